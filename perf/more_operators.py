"""What is measured of the INT8 product, the gated feed-forward block and
gradient clipping.

The operators (include/nvfp4.h has their contracts):

* int8: y = x W^T with x quantised to 8-bit integers, one scale for each
  token, and W quantised ahead with one scale for each output channel; the
  sums are whole numbers.
* gated: h = act(x Wg^T) * (x Wu^T) in one product over FP8 operands (one
  fp32 scale per 128 elements), W = [Wg; Wu] of 2F rows; training keeps
  [x Wg^T, x Wu^T] too.  With experts > 0 each expert's rows meet its own W,
  read through the router's index.
* backward: from the gradient of h and the kept products the gradients of
  x Wg^T and x Wu^T as FP8 operands of the products that follow (rows and
  transposed, from one read); with groups > 0 every expert's transposed
  columns start on a block border.
* clip: the norm over a list of gradients, and the gradients scaled to it.

``run`` computes them with elementary torch operations in fp32 (``own``
false) or through the framework (``own`` true).
"""
import math

import torch

own = False

BLOCK = 128
TINY = 2.0 ** -100          # a block's (a row's) largest magnitude is taken as at least this
F8 = torch.float8_e4m3fn
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token through a linear layer: the weight is streamed, launches count
        {"name": "int8_decode", "op": "int8", "M": 1, "N": 8192, "K": 8192, "x": "bf16", "out": "bf16"},
        # a ragged batch of requests, odd output width, K that ends inside a block
        {"name": "int8_ragged", "op": "int8", "M": 203, "N": 6151, "K": 2064, "x": "f32", "out": "f32"},
        # a prompt of 4096 tokens through the linear layer's workload
        {"name": "int8_prompt", "op": "int8", "M": 4096, "N": 8192, "K": 8192, "x": "bf16", "out": "bf16"},
        # one serving step of 16 requests through a dense block's first half
        {"name": "gated_decode", "op": "gated", "M": 16, "F": 8192, "K": 8192, "b_rows": 128, "act": "silu",
         "save": False, "out": "bf16"},
        # a training batch through it, the products kept for the backward
        {"name": "gated_train", "op": "gated", "M": 4096, "F": 8192, "K": 8192, "b_rows": 128, "act": "silu",
         "save": True, "out": "bf16"},
        # serving step of the mixture: 512 tokens, top-8 of 256 experts
        {"name": "gated_experts_serve", "op": "gated_experts", "tokens": 512, "topk": 8, "experts": 256,
         "F": 2048, "K": 6144, "gather": True, "skew": 0.0, "act": "silu", "save": False, "out": "bf16"},
        # a mixture's training batch, uneven routing
        {"name": "gated_experts_train", "op": "gated_experts", "tokens": 8192, "topk": 8, "experts": 64,
         "F": 2048, "K": 6144, "gather": True, "skew": 0.3, "act": "gelu", "save": True, "out": "bf16"},
        # backward of the dense block's training batch
        {"name": "backward_dense", "op": "backward", "rows": 4096, "F": 8192, "groups": 0, "act": "silu",
         "layout": "both", "x": "bf16"},
        # backward of the mixture's: 64 experts' rows
        {"name": "backward_experts", "op": "backward", "rows": 32768, "F": 2048, "groups": 64, "act": "gelu",
         "layout": "both", "x": "bf16"},
        # the small parameters of a model: norms' gains, biases, a router
        {"name": "clip_small", "op": "clip", "tensors": 96, "least": 64, "most": 65536, "share_bf16": 0.5,
         "border": 64, "seed_sizes": 1},
        # the linear layers of a few blocks, odd sizes among them
        {"name": "clip_layers", "op": "clip", "tensors": 24, "least": 1 << 20, "most": 1 << 25,
         "share_bf16": 0.5, "border": 64, "seed_sizes": 2},
        # experts' fp32 weight gradients: 16 of gate, up and down
        {"name": "clip_experts", "op": "clip", "tensors": 48, "least": 6144 * 2048, "most": 6144 * 2048,
         "share_bf16": 0.0, "border": 64, "seed_sizes": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("int8", "int8", "int8", "gated", "gated", "gated_experts", "backward", "backward",
                     "clip", "clip"))
    if op == "int8":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 100, 8192), "K": 16 * _log(rng, 4, 512),
                "x": rng.choice(("f32", "bf16")), "out": rng.choice(("f32", "bf16"))}
    if op == "gated":
        return {"op": op, "M": _log(rng, 1, 4096), "F": 8 * _log(rng, 8, 1024), "K": 16 * _log(rng, 8, 512),
                "b_rows": rng.choice((128, 128, 1)), "act": rng.choice(("silu", "gelu")),
                "save": rng.random() < 0.5, "out": rng.choice(("f32", "bf16", "bf16"))}
    if op == "gated_experts":
        return {"op": op, "tokens": _log(rng, 16, 2048), "topk": rng.randint(1, 4),
                "experts": _log(rng, 4, 128), "F": 8 * _log(rng, 16, 256), "K": 16 * _log(rng, 16, 256),
                "gather": rng.random() < 0.5, "skew": rng.choice((0.0, 0.5, 1.0)),
                "act": rng.choice(("silu", "gelu")), "save": rng.random() < 0.5,
                "out": rng.choice(("f32", "bf16", "bf16"))}
    if op == "backward":
        groups = rng.choice((0, 0, rng.randint(1, 64)))
        return {"op": op, "rows": _log(rng, 1, 8192) if not groups else _log(rng, 64, 16384),
                "F": 8 * _log(rng, 8, 512), "groups": groups, "act": rng.choice(("silu", "gelu")),
                "layout": rng.choice(("rows", "cols", "both")), "x": rng.choice(("f32", "bf16"))}
    least = _log(rng, 1, 1 << 16)
    return {"op": op, "tensors": _log(rng, 1, 256), "least": least, "most": least * _log(rng, 1, 256),
            "share_bf16": rng.choice((0.0, 0.5, 1.0)), "border": rng.choice((1, 8, 64)), "seed_sizes": rng.randint(0, 1 << 20)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _ceil(a, b):
    return -(-a // b)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _operand(g, rows, K, block_rows, lead=(), scale=1.0):
    """E4M3 values and fp32 scales of an operand [.., rows, K] as a program
    has them after quantising: magnitudes up to 448, scales around
    ``scale`` * 4 / 448."""
    n = rows * K * (lead[0] if lead else 1)
    q = torch.empty(n, dtype=F8, device=DEV)
    step = 1 << 28
    for i in range(0, n, step):
        m = min(step, n - i)
        q[i:i + m] = (_randn(g, m) * 112.0).clamp_(-448, 448).to(F8)
    s = torch.rand(*lead, _ceil(K, BLOCK), _ceil(rows, block_rows), generator=g, device=DEV)
    return q.view(*lead, rows, K), (s + 0.5) * (scale * 4.0 / 448.0)


def _routing(g, tokens, topk, experts, skew):
    """Expert-sorted rows of a top-k router: (m_offsets int32, row_index int32,
    rows of the busiest expert)."""
    logits = _randn(g, tokens, experts)
    logits -= skew * torch.log1p(torch.arange(experts, device=DEV, dtype=torch.float32))
    e = torch.topk(logits, topk, dim=-1).indices.reshape(-1)
    order = torch.sort(e, stable=True).indices
    counts = torch.bincount(e, minlength=experts)
    off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return off, (order // topk).to(torch.int32), int(counts.max())


def _padded(total_m, groups):
    """Columns of an expert-wise transposed operand: every expert's tokens
    start on a block border."""
    return BLOCK * ((total_m + (BLOCK - 1) * min(groups, total_m)) // BLOCK)


def _sizes(case):
    """The tensors of a list of gradients: (elements, dtype) each."""
    r = torch.Generator().manual_seed(case["seed_sizes"])
    u = torch.rand(case["tensors"], generator=r, dtype=torch.float64)
    lo, hi = math.log(case["least"]), math.log(case["most"])
    n = torch.exp(lo + u * (hi - lo)).round().long().clamp(min=1).tolist()
    half = (torch.rand(case["tensors"], generator=r) < case["share_bf16"]).tolist()
    return [(m, "bf16" if h else "f32") for m, h in zip(n, half)]


def _places(sizes, border):
    """Where each tensor starts in its type's flat buffer, and the buffers' lengths."""
    total, at = {}, []
    for n, dt in sizes:
        at.append(total.get(dt, 0))
        total[dt] = at[-1] + _ceil(n, border) * border
    return at, total


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        # a few channels that are much larger than the others
        x = _randn(g, M, K) * torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        st["input"] = x.to(DTYPES[case["x"]])
        q = (_randn(g, N, K) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        st["w"] = (q, (torch.rand(N, generator=g, device=DEV) + 0.5) / (32.0 * K ** 0.5))
    elif op == "gated":
        st["a"] = _operand(g, case["M"], case["K"], 1)
        st["w"] = _operand(g, 2 * case["F"], case["K"], case["b_rows"], scale=case["K"] ** -0.5)
    elif op == "gated_experts":
        E = case["experts"]
        off, idx, most = _routing(g, case["tokens"], min(case["topk"], E), E, case["skew"])
        total = case["tokens"] * min(case["topk"], E)
        st["m_offsets"], st["total"], st["most"] = off, total, most
        st["row_index"] = idx if case["gather"] else None
        st["a"] = _operand(g, case["tokens"] if case["gather"] else total, case["K"], 1)
        st["w"] = _operand(g, 2 * case["F"], case["K"], BLOCK, (E,), case["K"] ** -0.5)
    elif op == "backward":
        rows, F = case["rows"], case["F"]
        st["dh"] = (_randn(g, rows, F) * 1e-3).to(DTYPES[case["x"]])
        st["gate_up"] = (_randn(g, rows, 2 * F) * 1.5).to(DTYPES[case["x"]])
        if case["groups"]:
            cut = torch.sort(torch.randint(0, rows + 1, (case["groups"] - 1,), generator=g, device=DEV)).values
            off = torch.zeros(case["groups"] + 1, dtype=torch.int32, device=DEV)
            off[1:-1] = cut.to(torch.int32)
            off[-1] = rows
            st["m_offsets"] = off
    else:
        scale = torch.rand(case["tensors"], generator=torch.Generator().manual_seed(seed)) * 3.0 - 4.0
        sizes = _sizes(case)
        places, total = _places(sizes, case["border"])
        # flat buffers of each type, as a program has them that reduces or saves them as a whole
        flat = {dt: torch.zeros(n, dtype=DTYPES[dt], device=DEV) for dt, n in total.items()}
        st["flat_out"] = {dt: torch.zeros_like(t) for dt, t in flat.items()}
        st["grads"] = [flat[dt][at:at + n] for (n, dt), at in zip(sizes, places)]
        st["out"] = [st["flat_out"][dt][at:at + n] for (n, dt), at in zip(sizes, places)]
        for t, s in zip(st["grads"], scale.tolist()):
            t.copy_(_randn(g, t.numel()) * 10.0 ** s)
        # below the norm, as when a step's gradients are too large
        st["max_norm"] = 0.3 * math.sqrt(sum(float(t.double().square().sum()) for t in st["grads"]))
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _plain_int8(st):
    x = st["input"].float()
    amax = x.abs().amax(1, keepdim=True).clamp_min(TINY)
    top = torch.full_like(amax, 127.0)
    s, r = torch.div(amax, top), torch.div(top, amax)
    q = torch.round(x * r)
    wq, ws = st["w"]
    y = (q @ wq.float().t()) * s * ws
    return q.to(torch.int8), s[:, 0], y.to(DTYPES[st["out"]])


def _values(operand, block_rows, dtype=torch.float32):
    """The values of an operand [.., rows, K]."""
    q, s = operand
    rows, K = q.shape[-2:]
    s = s.to(dtype).repeat_interleave(block_rows, -1)[..., :rows].transpose(-1, -2)
    s = s.repeat_interleave(BLOCK, -1)[..., :K]
    return q.to(dtype) * s


def _gate(g, act):
    """sigma(z) and z' with act(g) = g sigma(z(g)): silu has z = g, gelu (its
    tanh form) z = 2 sqrt(2 / pi) (g + 0.044715 g^3)."""
    if act == "silu":
        return 1.0 / (1.0 + torch.exp(-g)), torch.ones_like(g)
    z = GELU_A * (g + GELU_B * g * g * g)
    return 1.0 / (1.0 + torch.exp(-z)), GELU_A * (1.0 + 3.0 * GELU_B * g * g)


def _gated_out(gu, st):
    F = st["F"]
    g, u = gu[:, :F], gu[:, F:]
    h = (g * _gate(g, st["act"])[0] * u).to(DTYPES[st["out"]])
    return {"h": h, "gate_up": gu.to(torch.bfloat16)} if st["save"] else {"h": h}


def _plain_gated(st):
    return _gated_out(_values(st["a"], 1) @ _values(st["w"], st["b_rows"]).t(), st)


def _plain_gated_experts(st):
    off, total, most = st["m_offsets"].long(), st["total"], st["most"]
    a = _values(st["a"], 1)
    if st["row_index"] is not None:
        a = a[st["row_index"].long()]
    E = off.numel() - 1
    r = torch.arange(total, device=a.device)
    e = torch.searchsorted(off, r, right=True) - 1
    slot = r - off[e]
    xt = a.new_zeros(E, a.shape[1], most)          # each expert's rows, padded to the busiest
    xt[e, :, slot] = a
    y = torch.bmm(_values(st["w"], BLOCK), xt)     # [E, 2F, most]
    return _gated_out(y[e, :, slot], st)


def _segments(off, total, P):
    """For each grouped row its column in the padded order, and whether it
    lies in a group."""
    off = off.long()
    counts = off[1:] - off[:-1]
    blocks = (counts + BLOCK - 1) // BLOCK
    pad = torch.cumsum(blocks * BLOCK, 0) - blocks * BLOCK
    r = torch.arange(total, device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    used = e < counts.numel()
    e = e.clamp(max=counts.numel() - 1)
    return (pad[e] + r - off[e]).clamp(max=P - 1), used


def _quant_rows(x):
    """x [R, C] (fp32) -> E4M3 [R, C] and scales [C / 128, R] of 1 x 128 blocks."""
    R, C = x.shape
    p = torch.nn.functional.pad(x, (0, -C % BLOCK)).view(R, _ceil(C, BLOCK), BLOCK)
    amax = p.abs().amax(2).clamp_min(TINY)
    top = torch.full_like(amax, 448.0)
    s, r = torch.div(amax, top), torch.div(top, amax)
    q = (p * r[:, :, None]).to(F8).view(R, -1)[:, :C].contiguous()
    return q, s.t().contiguous()


def _plain_backward(st):
    dh, gu, F = st["dh"].float(), st["gate_up"].float(), st["F"]
    g, u = gu[:, :F], gu[:, F:]
    sig, dz = _gate(g, st["act"])
    d = torch.cat([dh * u * (sig + g * sig * (1.0 - sig) * dz), dh * (g * sig)], 1)
    res = {}
    if st["layout"] in ("rows", "both"):
        res["rows"] = _quant_rows(d)
    if st["layout"] in ("cols", "both"):
        if st["groups"]:
            P = _padded(d.shape[0], st["groups"])
            cols, used = _segments(st["m_offsets"], d.shape[0], P)
            p = d.new_zeros(P, 2 * F)
            p[cols[used]] = d[used]
            res["cols"] = _quant_rows(p.t())
        else:
            res["cols"] = _quant_rows(torch.nn.functional.pad(d.t(), (0, -d.shape[0] % 16)))
    return res


def _plain_clip(st):
    # the sum over all elements is long: 64 bits
    sums = torch.stack([t.float().square().sum(dtype=torch.float64) for t in st["grads"]])
    norm = torch.sqrt(sums.sum())
    c = torch.where(norm > st["max_norm"], st["max_norm"] / norm, 1.0).float()
    done = [o.copy_(t.float() * c) for t, o in zip(st["grads"], st["out"])]
    assert len(done) == st["tensors"]
    return {"norm": norm.float().reshape(1), "grads": st["flat_out"]}


PLAIN = {"int8": _plain_int8, "gated": _plain_gated, "gated_experts": _plain_gated_experts,
         "backward": _plain_backward, "clip": _plain_clip}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(st):
    op = st["op"]
    if own:
        import nvfp4_block_scaled_gemm_amd as nv
        if op == "int8":
            a = nv.nvfp4_int8_quantize(st["input"])
            return a[0], a[1], nv.nvfp4_int8_gemm(a, st["w"], out_dtype=st["out"])
        if op == "gated":
            r = nv.nvfp4_fp8_gated_gemm(st["a"], st["w"], act=st["act"], out_dtype=st["out"],
                                        gate_up=st["save"])
            return {"h": r[0], "gate_up": r[1]} if st["save"] else {"h": r}
        if op == "gated_experts":
            r = nv.nvfp4_fp8_grouped_gated_gemm(st["m_offsets"], st["total"], st["a"], st["w"], act=st["act"],
                                                out_dtype=st["out"], gate_up=st["save"],
                                                row_index=st["row_index"])
            return {"h": r[0], "gate_up": r[1]} if st["save"] else {"h": r}
        if op == "backward":
            if st["groups"]:
                r = nv.nvfp4_fp8_grouped_gated_backward(st["dh"], st["gate_up"], st["m_offsets"],
                                                        act=st["act"], layout=st["layout"])
            else:
                r = nv.nvfp4_fp8_gated_backward(st["dh"], st["gate_up"], act=st["act"], layout=st["layout"])
            return {"rows": r[0], "cols": r[1]} if st["layout"] == "both" else {st["layout"]: r}
        norm = nv.nvfp4_clip_grads(st["grads"], st["max_norm"], out=st["out"])
        return {"norm": norm, "grads": st["flat_out"]}
    return PLAIN[op](st)


# --------------------------------------------------------------------------
# the least a pass has to move and compute
# --------------------------------------------------------------------------

def _size(name):
    return 4 if name == "f32" else 2


def _op_bytes(rows, K, block_rows):
    return rows * K + 4 * _ceil(K, BLOCK) * _ceil(rows, block_rows)


def work(case):
    op = case["op"]
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * (_size(case["x"]) + 1) + N * K + 4 * (M + N) + M * N * _size(case["out"]),
                "flops": 2 * M * N * K}
    if op in ("gated", "gated_experts"):
        F, K = case["F"], case["K"]
        if op == "gated":
            rows = case["M"]
            b = _op_bytes(rows, K, 1) + _op_bytes(2 * F, K, case["b_rows"])
        else:
            E = case["experts"]
            rows = case["tokens"] * min(case["topk"], E)
            b = _op_bytes(case["tokens"] if case["gather"] else rows, K, 1)
            b += min(E, rows) * _op_bytes(2 * F, K, BLOCK)
        out = _size(case["out"]) + (4 if case["save"] else 0)
        return {"bytes": b + rows * F * out, "flops": 4 * rows * F * K}
    if op == "backward":
        n = case["rows"] * case["F"]
        both = 2 if case["layout"] == "both" else 1
        return {"bytes": n * (3 * _size(case["x"]) + 2 * both) + 8 * both * _ceil(n, BLOCK), "flops": 20 * n}
    sizes = _sizes(case)
    return {"bytes": 2 * sum(n * _size(dt) for n, dt in sizes), "flops": 3 * sum(n for n, _ in sizes)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_quant(x):
    """x [R, C] float64 -> E4M3 values and scales of 1 x 128 blocks."""
    R, C = x.shape
    vals, scales = torch.empty_like(x), x.new_empty(_ceil(C, BLOCK), R)
    for i in range(_ceil(C, BLOCK)):
        b = x[:, i * BLOCK:(i + 1) * BLOCK]
        s = torch.clamp(torch.amax(torch.abs(b), 1), min=TINY) / 448.0
        v = b / s[:, None]
        # nearest of 4 significant bits (steps of 2^-9 below 2^-6), ties to even
        step = torch.exp2(torch.floor(torch.log2(torch.clamp(torch.abs(v), min=2.0 ** -6))) - 3)
        vals[:, i * BLOCK:(i + 1) * BLOCK] = torch.clamp(torch.round(v / step) * step, -448, 448)
        scales[i] = s
    return vals, scales


def _exact_act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def _exact_product(a, w, block_rows):
    """Sum over blocks of K of the scaled block products, 64 bits."""
    (aq, sa), (bq, sb) = a, w
    y = torch.zeros(aq.shape[0], bq.shape[0], dtype=torch.float64, device=DEV)
    cols = torch.arange(bq.shape[0], device=DEV) // block_rows
    for i in range(sa.shape[0]):
        k = slice(i * BLOCK, (i + 1) * BLOCK)
        y += (aq[:, k].double() @ bq[:, k].double().t()) * (sa[i].double()[:, None] * sb[i].double()[cols][None, :])
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "int8":
        # the definition rounds 127 / A and its product with x to fp32
        x = st["input"].double()
        A = torch.clamp(torch.amax(torch.abs(x), 1), min=TINY)
        q = torch.round((x * (127.0 / A).float().double()[:, None]).float().double())
        s = (A / 127.0).float().double()
        wq, ws = st["w"]
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
        for i in range(_ceil(case["K"], BLOCK)):
            k = slice(i * BLOCK, (i + 1) * BLOCK)
            y += q[:, k] @ wq[:, k].double().t()
        y *= s[:, None] * ws.double()[None, :]
        return q.to(torch.int8), A / 127.0, y
    if op in ("gated", "gated_experts"):
        F = case["F"]
        if op == "gated":
            gu = _exact_product(st["a"], st["w"], case["b_rows"])
        else:
            off = st["m_offsets"].tolist()
            gu = torch.zeros(st["total"], 2 * F, dtype=torch.float64, device=DEV)
            a = _values(st["a"], 1, torch.float64)
            for e in range(case["experts"]):
                if off[e] < off[e + 1]:
                    rows = slice(off[e], off[e + 1])
                    x = a[rows] if st["row_index"] is None else a[st["row_index"][rows].long()]
                    gu[rows] = x @ _values((st["w"][0][e], st["w"][1][e]), BLOCK, torch.float64).t()
        h = _exact_act(gu[:, :F], case["act"]) * gu[:, F:]
        return {"h": h, "gate_up": gu} if case["save"] else {"h": h}
    if op == "backward":
        # the gradient of sum(dh * act(g) * u) by automatic differentiation
        gu = st["gate_up"].double().requires_grad_(True)
        F = case["F"]
        h = _exact_act(gu[:, :F], case["act"]) * gu[:, F:]
        d, = torch.autograd.grad(h, gu, st["dh"].double())
        res = {}
        if case["layout"] in ("rows", "both"):
            res["rows"] = _exact_quant(d)
        if case["layout"] in ("cols", "both"):
            if case["groups"]:
                parts, off = [], st["m_offsets"].tolist()
                for lo, hi in zip(off[:-1], off[1:]):
                    parts.append(torch.nn.functional.pad(d[lo:hi].t(), (0, -(hi - lo) % BLOCK)))
                t = torch.cat(parts, 1)
                t = torch.nn.functional.pad(t, (0, _padded(case["rows"], case["groups"]) - t.shape[1]))
            else:
                t = torch.nn.functional.pad(d.t(), (0, -case["rows"] % 16))
            res["cols"] = _exact_quant(t)
        return res
    norm = math.sqrt(math.fsum(float(t.double().pow(2).sum()) for t in st["grads"]))
    c = min(1.0, st["max_norm"] / norm)
    flat = {dt: torch.zeros(t.shape, dtype=torch.float64, device=DEV) for dt, t in st["flat_out"].items()}
    for (n, dt), at, t in zip(_sizes(case), _places(_sizes(case), case["border"])[0], st["grads"]):
        flat[dt][at:at + n] = t.double() * c
    return {"norm": torch.tensor([norm], dtype=torch.float64), "grads": flat}
