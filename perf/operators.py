"""What is measured of the FP8 block-128 products and the expert router.

The operators (include/nvfp4.h has their contracts):

* quantize: x -> E4M3 bytes with one fp32 scale per 1 x 128 (or 128 x 128)
  block, along the rows, along the columns (transposed operand) or both from
  one read; for experts the transposed operand starts each expert's tokens on
  a block border.
* gemm: y = A . B^T of two such operands; forward, input gradient and weight
  gradient (accumulated into fp32) are this one product.
* grouped: the same for the experts of a mixture, tokens read through the
  router's index; wgrad: the experts' weight gradients.
* route: top-k of the router's logits, per-expert counts, the expert-sorted
  order and the balance loss; train: that and the gradient of the logits.

``run`` computes them with elementary torch operations in fp32 (``own``
false) or through the framework (``own`` true).
"""
import math

import torch

own = False

BLOCK = 128
TINY = 2.0 ** -100          # a block's largest magnitude is taken as at least this
F8 = torch.float8_e4m3fn
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one serving step's activations before a linear layer: launch latency
        {"name": "quant_decode", "op": "quantize", "batch": 1, "rows": 32, "cols": 8192, "groups": 0,
         "block_rows": 1, "layout": "rows", "x": "bf16"},
        # an output gradient of 64 experts (top-8 of 4096 tokens): both operands of its backward
        {"name": "quant_experts", "op": "quantize", "batch": 1, "rows": 32768, "cols": 4096, "groups": 64,
         "block_rows": 1, "layout": "both", "x": "bf16"},
        # a layer's master weight, for the forward and the input gradient
        {"name": "quant_weight", "op": "quantize", "batch": 1, "rows": 8192, "cols": 8192, "groups": 0,
         "block_rows": 128, "layout": "both", "x": "f32"},
        # one token through a linear layer: the weight is streamed
        {"name": "gemm_decode_m1", "op": "gemm", "M": 1, "N": 8192, "K": 8192, "b_rows": 128,
         "out": "bf16", "accumulate": False},
        # a ragged batch of requests, odd output width, K that ends inside a block
        {"name": "gemm_ragged_m203", "op": "gemm", "M": 203, "N": 6151, "K": 2064, "b_rows": 128,
         "out": "f32", "accumulate": False},
        # the linear layer's workload (forward; the input gradient has the same form)
        {"name": "gemm_linear", "op": "gemm", "M": 4096, "N": 8192, "K": 8192, "b_rows": 128,
         "out": "bf16", "accumulate": False},
        # its weight gradient, accumulated over microbatches in fp32
        {"name": "gemm_wgrad", "op": "gemm", "M": 8192, "N": 8192, "K": 4096, "b_rows": 1,
         "out": "f32", "accumulate": True},
        # serving step of the mixture: 512 tokens, top-8 of 256 experts
        {"name": "grouped_serve", "op": "grouped", "tokens": 512, "topk": 8, "experts": 256, "N": 4096,
         "K": 6144, "gather": True, "skew": 0.0, "out": "bf16"},
        # training batch, uneven routing
        {"name": "grouped_train", "op": "grouped", "tokens": 8192, "topk": 8, "experts": 64, "N": 4096,
         "K": 6144, "gather": False, "skew": 0.3, "out": "bf16"},
        # the experts' weight gradients of a training batch
        {"name": "grouped_wgrad", "op": "wgrad", "tokens": 4096, "topk": 8, "experts": 64, "N": 4096,
         "K": 2048, "skew": 0.3, "out": "f32"},
        # the serving step's router
        {"name": "route_serve", "op": "route", "tokens": 512, "experts": 256, "topk": 8, "x": "f32",
         "renorm": True, "masked": 0.0, "train": False},
        # a training batch's router, padded tokens among them, forward and backward
        {"name": "route_train", "op": "route", "tokens": 65536, "experts": 256, "topk": 8, "x": "bf16",
         "renorm": False, "masked": 0.05, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "quantize", "gemm", "gemm", "gemm", "grouped", "wgrad", "route", "route"))
    if op == "quantize":
        groups = rng.choice((0, 0, rng.randint(1, 64)))
        block_rows = 1 if groups else rng.choice((1, 1, 128))
        batch = _log(rng, 1, 8) if block_rows == 128 else 1
        return {"op": op, "batch": batch, "rows": _log(rng, 1, 8192) if not groups else _log(rng, 64, 16384),
                "cols": 16 * _log(rng, 8, 512), "groups": groups, "block_rows": block_rows,
                "layout": rng.choice(("rows", "cols", "both")) if not groups else rng.choice(("cols", "both")),
                "x": rng.choice(("f32", "bf16"))}
    if op == "gemm":
        out = rng.choice(("f32", "bf16"))
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 100, 8192), "K": 16 * _log(rng, 8, 512),
                "b_rows": rng.choice((128, 128, 1)), "out": out,
                "accumulate": out == "f32" and rng.random() < 0.5}
    if op == "grouped":
        experts = _log(rng, 4, 128)
        return {"op": op, "tokens": _log(rng, 16, 2048), "topk": rng.randint(1, 4), "experts": experts,
                "N": 8 * _log(rng, 32, 512), "K": 16 * _log(rng, 16, 256), "gather": rng.random() < 0.5,
                "skew": rng.choice((0.0, 0.5, 1.0)), "out": rng.choice(("f32", "bf16"))}
    if op == "wgrad":
        return {"op": op, "tokens": _log(rng, 64, 2048), "topk": rng.randint(1, 4), "experts": _log(rng, 4, 32),
                "N": 16 * _log(rng, 8, 256), "K": 16 * _log(rng, 8, 128), "skew": rng.choice((0.0, 0.5, 1.0)),
                "out": rng.choice(("f32", "bf16"))}
    experts = _log(rng, 8, 512)
    return {"op": op, "tokens": _log(rng, 1, 32768), "experts": experts, "topk": rng.randint(1, 8),
            "x": rng.choice(("f32", "bf16")), "renorm": rng.random() < 0.5,
            "masked": rng.choice((0.0, 0.2)), "train": rng.random() < 0.5}


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
    topk = min(topk, experts)
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


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = _randn(g, case["batch"], rows, cols)
        # a few channels that are much larger than the others
        x *= torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 30.0, 1.0)
        x = x.to(DTYPES[case["x"]])
        st["x"] = x if case["block_rows"] == BLOCK else x[0]
        if case["groups"]:
            cut = torch.sort(torch.randint(0, rows + 1, (case["groups"] - 1,), generator=g, device=DEV)).values
            off = torch.zeros(case["groups"] + 1, dtype=torch.int32, device=DEV)
            off[1:-1] = cut.to(torch.int32)
            off[-1] = rows
            st["m_offsets"] = off
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["a"] = _operand(g, M, K, 1)
        st["b"] = _operand(g, N, K, case["b_rows"], scale=K ** -0.5)
        if case["accumulate"]:
            st["y"] = _randn(g, M, N)
    elif op == "grouped":
        E = case["experts"]
        off, idx, most = _routing(g, case["tokens"], case["topk"], E, case["skew"])
        total = case["tokens"] * min(case["topk"], E)
        st["m_offsets"], st["total"], st["most"] = off, total, most
        st["row_index"] = idx if case["gather"] else None
        st["a"] = _operand(g, case["tokens"] if case["gather"] else total, case["K"], 1)
        st["b"] = _operand(g, case["N"], case["K"], BLOCK, (E,), case["K"] ** -0.5)
    elif op == "wgrad":
        E = case["experts"]
        off, _, most = _routing(g, case["tokens"], case["topk"], E, case["skew"])
        total = case["tokens"] * min(case["topk"], E)
        P = _padded(total, E)
        st["m_offsets"], st["total"], st["most"] = off, total, most
        # columns between the experts' tokens hold zeros, as the quantiser leaves them
        cols, used = _segments(off, total, P)
        keep = torch.zeros(P, dtype=torch.bool, device=DEV)
        keep[cols[used]] = True
        for name, rows in (("a", case["N"]), ("b", case["K"])):
            q, s = _operand(g, rows, P, 1)
            st[name] = (torch.where(keep, q.view(torch.uint8), 0).view(F8), s)
    else:
        T, E = case["tokens"], case["experts"]
        st["topk"] = min(case["topk"], E)
        x = _randn(g, T, E) * 1.5 - 0.3 * torch.log1p(torch.arange(E, device=DEV, dtype=torch.float32))
        st["x"] = x.to(DTYPES[case["x"]])
        st["mask"] = torch.rand(T, generator=g, device=DEV) >= case["masked"] if case["masked"] else None
        if case["train"]:
            st["d_weights"] = _randn(g, T, st["topk"])
            st["d_loss"] = torch.full((1,), 0.01 * E, device=DEV)
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _segments(off, total, P):
    """For each grouped row its column in the padded order, and whether it
    lies in a group."""
    off = off.long()
    counts = off[1:] - off[:-1]
    pad = torch.cumsum(_ceil_t(counts) * BLOCK, 0) - _ceil_t(counts) * BLOCK
    r = torch.arange(total, device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    used = e < counts.numel()
    e = e.clamp(max=counts.numel() - 1)
    return (pad[e] + r - off[e]).clamp(max=P - 1), used


def _ceil_t(counts):
    return (counts + BLOCK - 1) // BLOCK


def _quant_blocks(x, block_rows):
    """x [B, R, C] (fp32) -> E4M3 [B, R, C], scales [B, C / 128, R / block_rows]."""
    B, R, C = x.shape
    pr, pc = -R % block_rows, -C % BLOCK
    p = torch.nn.functional.pad(x, (0, pc, 0, pr))
    p = p.view(B, (R + pr) // block_rows, block_rows, (C + pc) // BLOCK, BLOCK)
    amax = p.abs().amax(dim=(2, 4)).clamp_min(TINY)
    top = torch.full_like(amax, 448.0)
    s, r = torch.div(amax, top), torch.div(top, amax)
    q = (p * r[:, :, None, :, None]).to(F8)
    q = q.view(B, R + pr, C + pc)[:, :R, :C].contiguous()
    return q, s.transpose(1, 2).contiguous()


def _plain_quantize(st):
    x = st["x"].float()
    x = x if x.dim() == 3 else x[None]
    res = []
    if st["layout"] in ("rows", "both"):
        res.append(_quant_blocks(x, st["block_rows"]))
    if st["layout"] in ("cols", "both"):
        if st["groups"]:
            P = _padded(x.shape[1], st["groups"])
            cols, used = _segments(st["m_offsets"], x.shape[1], P)
            p = x.new_zeros(P, x.shape[2])
            p[cols[used]] = x[0][used]
            xt = p.t()[None]
        else:
            xt = torch.nn.functional.pad(x.transpose(1, 2), (0, -x.shape[1] % 16))
        res.append(_quant_blocks(xt, st["block_rows"]))
    flat = st["x"].dim() == 2
    return [(q[0], s[0]) if flat else (q, s) for q, s in res]


def _values(operand, block_rows, dtype=torch.float32):
    """The values of an operand [.., rows, K]."""
    q, s = operand
    rows, K = q.shape[-2:]
    s = s.to(dtype).repeat_interleave(block_rows, -1)[..., :rows].transpose(-1, -2)
    s = s.repeat_interleave(BLOCK, -1)[..., :K]
    return q.to(dtype) * s


def _plain_gemm(st):
    y = _values(st["a"], 1) @ _values(st["b"], st["b_rows"]).t()
    return st["y"].add_(y) if st["accumulate"] else y.to(DTYPES[st["out"]])


def _plain_grouped(st):
    off, total, most = st["m_offsets"], st["total"], st["most"]
    a = _values(st["a"], 1)
    if st["row_index"] is not None:
        a = a[st["row_index"].long()]
    off = off.long()
    E = off.numel() - 1
    r = torch.arange(total, device=a.device)
    e = torch.searchsorted(off, r, right=True) - 1
    slot = r - off[e]
    xt = a.new_zeros(E, a.shape[1], most)          # each expert's rows, padded to the busiest
    xt[e, :, slot] = a
    y = torch.bmm(_values(st["b"], BLOCK), xt)     # [E, N, most]
    return y[e, :, slot].to(DTYPES[st["out"]])


def _plain_wgrad(st):
    off = st["m_offsets"].long()
    counts = off[1:] - off[:-1]
    pad = torch.cumsum(_ceil_t(counts) * BLOCK, 0) - _ceil_t(counts) * BLOCK
    j = torch.arange(st["most"], device=off.device)
    valid = j < counts[:, None]                                   # [E, most]
    cols = torch.where(valid, pad[:, None] + j, 0)
    a, b = _values(st["a"], 1), _values(st["b"], 1)
    ae = a[:, cols].permute(1, 0, 2).contiguous() * valid[:, None, :]     # [E, N, most]
    be = b[:, cols].permute(1, 2, 0).contiguous()                 # [E, most, K]
    return torch.bmm(ae, be).to(DTYPES[st["out"]])


def _plain_route(st, dtype=torch.float32):
    """Ties go to the lowest expert; an expert at -inf, or of a masked token,
    is not chosen."""
    x, k = st["x"].to(dtype), st["topk"]
    T, E = x.shape
    if st["mask"] is not None:
        x = x.masked_fill(~st["mask"][:, None], -math.inf)
    top, idx = torch.sort(x, dim=-1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    chosen = top > -math.inf
    active = chosen[:, :1]
    z = torch.where(active, x - top[:, :1], -math.inf)
    ez = torch.exp(z)
    p = ez / torch.where(active, ez.sum(-1, keepdim=True), 1.0)   # [T, E]
    w = torch.where(chosen, torch.gather(p, 1, idx), 0.0)
    if st["renorm"]:
        ec = torch.where(chosen, torch.exp(top - top[:, :1]), 0.0)
        w = ec / torch.where(active, ec.sum(-1, keepdim=True), 1.0)
    flat = torch.where(chosen, idx, E).reshape(-1)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    off = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    off[1:] = torch.cumsum(counts, 0).to(torch.int32)
    order = torch.sort(flat, stable=True).indices
    live = torch.arange(T * k, device=x.device) < off[E]
    row_index = torch.where(live, order // k, -1).to(torch.int32)
    pair_row = torch.empty(T * k, dtype=torch.int32, device=x.device)
    pair_row[order] = torch.where(live, torch.arange(T * k, device=x.device), -1).to(torch.int32)
    n = active.sum().to(torch.float64)
    share = counts.to(torch.float64) / (n * k).clamp_min(1.0)
    mean_p = p.sum(0, dtype=torch.float64) / n.clamp_min(1.0)
    loss = (E * (share * mean_p).sum()).to(dtype).reshape(1)
    out = {"expert_index": torch.where(chosen, idx, -1).to(torch.int32), "weights": w,
           "counts": counts.to(torch.int32), "m_offsets": off, "row_index": row_index,
           "pair_row": pair_row.view(T, k), "routed": n.to(torch.int32).reshape(1), "loss": loss}
    if st["train"]:
        dl, dw = st["d_loss"].to(dtype), torch.where(chosen, st["d_weights"].to(dtype), 0.0)
        dp = (dl * E * share.to(dtype) / n.clamp_min(1.0).to(dtype)).expand(T, E)
        dx = torch.zeros_like(x)
        if st["renorm"]:
            dx.scatter_add_(1, idx, w * (dw - (w * dw).sum(-1, keepdim=True)))
        else:
            dp = dp.scatter_add(1, idx, dw)
        dx = dx + p * (dp - (p * dp).sum(-1, keepdim=True))
        out["d_logits"] = torch.where(active, dx, 0.0)
    return out


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(st):
    if own:
        import nvfp4_block_scaled_gemm_amd as nv
        op = st["op"]
        if op == "quantize":
            if st["groups"]:
                return nv.nvfp4_fp8_grouped_quantize(st["x"], st["m_offsets"], layout=st["layout"])
            return nv.nvfp4_fp8_quantize(st["x"], block_rows=st["block_rows"], layout=st["layout"])
        if op == "gemm":
            if st["accumulate"]:
                return nv.nvfp4_fp8_gemm(st["a"], st["b"], out_dtype="f32", y=st["y"], accumulate=True)
            return nv.nvfp4_fp8_gemm(st["a"], st["b"], out_dtype=st["out"])
        if op == "grouped":
            return nv.nvfp4_fp8_grouped_gemm(st["m_offsets"], st["total"], st["a"], st["b"],
                                             out_dtype=st["out"], row_index=st["row_index"])
        if op == "wgrad":
            return nv.nvfp4_fp8_grouped_wgrad(st["m_offsets"], st["total"], st["a"], st["b"],
                                              out_dtype=st["out"])
        r = nv.nvfp4_moe_route(st["x"], st["topk"], mask=st["mask"], renormalize=st["renorm"])
        out = r._asdict()
        if st["train"]:
            out["d_logits"] = nv.nvfp4_moe_route_backward(st["x"], r, d_weights=st["d_weights"],
                                                          d_loss=st["d_loss"], mask=st["mask"],
                                                          renormalize=st["renorm"])
        return out
    op = st["op"]
    if op == "quantize":
        res = _plain_quantize(st)
        return res[0] if len(res) == 1 else tuple(res)
    if op == "gemm":
        return _plain_gemm(st)
    if op == "grouped":
        return _plain_grouped(st)
    if op == "wgrad":
        return _plain_wgrad(st)
    out = _plain_route(st)
    if st["train"]:
        out["d_logits"] = out["d_logits"].to(st["x"].dtype)
    return out


# --------------------------------------------------------------------------
# the least a pass has to move and compute
# --------------------------------------------------------------------------

def _size(name):
    return 4 if name == "f32" else 2


def _op_bytes(rows, K, block_rows):
    return rows * K + 4 * _ceil(K, BLOCK) * _ceil(rows, block_rows)


def work(case):
    op = case["op"]
    if op == "quantize":
        B, R, C = case["batch"], case["rows"], case["cols"]
        n = B * R * C
        b = n * _size(case["x"])
        one = n + 4 * B * _ceil(C, BLOCK) * _ceil(R, case["block_rows"])
        b += one * (2 if case["layout"] == "both" else 1)
        return {"bytes": b, "flops": 2 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        out = M * N * _size(case["out"]) * (2 if case["accumulate"] else 1)
        return {"bytes": _op_bytes(M, K, 1) + _op_bytes(N, K, case["b_rows"]) + out, "flops": 2 * M * N * K}
    if op in ("grouped", "wgrad"):
        E, N, K = case["experts"], case["N"], case["K"]
        total = case["tokens"] * min(case["topk"], E)
        live = min(E, total)
        if op == "wgrad":
            b = _op_bytes(N, total, 1) + _op_bytes(K, total, 1) + E * N * K * _size(case["out"])
        else:
            b = live * _op_bytes(N, K, BLOCK) + total * N * _size(case["out"])
            b += _op_bytes(case["tokens"] if case["gather"] else total, K, 1)
        return {"bytes": b, "flops": 2 * total * N * K}
    T, E, k = case["tokens"], case["experts"], min(case["topk"], case["experts"])
    b = T * E * _size(case["x"]) + T * k * 16 + 8 * E
    if case["train"]:
        b += T * E * _size(case["x"]) + T * k * 4
    return {"bytes": b, "flops": T * E * (12 if case["train"] else 5)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_blocks(x, block_rows):
    """x [R, C] float64 -> rounded values and scales, block by block along C."""
    R, C = x.shape
    nb = _ceil(C, BLOCK)
    wide = x.new_zeros(_ceil(R, block_rows) * block_rows, nb * BLOCK)
    wide[:R, :C] = x
    amax = wide.abs().unflatten(1, (nb, BLOCK)).unflatten(0, (-1, block_rows)).amax((1, 3)).clamp_min(TINY)
    s = amax / torch.full_like(amax, 448.0)
    full = s.repeat_interleave(block_rows, 0).repeat_interleave(BLOCK, 1)
    v = wide / full
    # nearest of 4 significant bits (steps of 2^-9 below 2^-6), ties to even
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)[:R, :C], s.t()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        xs = x if x.dim() == 3 else x[None]
        found = []
        if case["layout"] in ("rows", "both"):
            found.append([_exact_blocks(m, case["block_rows"]) for m in xs])
        if case["layout"] in ("cols", "both"):
            if case["groups"]:
                parts, off = [], st["m_offsets"].tolist()
                for lo, hi in zip(off[:-1], off[1:]):
                    part = xs[0, lo:hi].t()
                    parts.append(torch.nn.functional.pad(part, (0, -(hi - lo) % BLOCK)))
                t = torch.cat(parts, 1)
                t = torch.nn.functional.pad(t, (0, _padded(case["rows"], case["groups"]) - t.shape[1]))
                found.append([_exact_blocks(t, 1)])
            else:
                pad = -case["rows"] % 16
                found.append([_exact_blocks(torch.nn.functional.pad(m.t(), (0, pad)), case["block_rows"])
                              for m in xs])
        both = [tuple(torch.stack(t) if x.dim() == 3 else t[0] for t in zip(*f)) for f in found]
        return both[0] if len(both) == 1 else tuple(both)
    if op == "gemm":
        (aq, sa), (bq, sb) = st["a"], st["b"]
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
        cols = torch.arange(case["N"], device=DEV) // case["b_rows"]
        for i in range(_ceil(case["K"], BLOCK)):
            k = slice(i * BLOCK, (i + 1) * BLOCK)
            c = aq[:, k].double() @ bq[:, k].double().t()
            y += c * sa[i].double()[:, None] * sb[i].double()[cols][None, :]
        return y + st["y"].double() if case["accumulate"] else y
    if op == "grouped":
        off = st["m_offsets"].tolist()
        y = torch.zeros(st["total"], case["N"], dtype=torch.float64, device=DEV)
        a = _values(st["a"], 1, torch.float64)
        if case["gather"]:
            a = a[st["row_index"].long()]
        q, s = st["b"]
        for e in range(case["experts"]):
            if off[e] < off[e + 1]:
                y[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ _values((q[e], s[e]), BLOCK, torch.float64).t()
        return y
    if op == "wgrad":
        off, at = st["m_offsets"].tolist(), 0
        dw = torch.zeros(case["experts"], case["N"], case["K"], dtype=torch.float64, device=DEV)
        a, b = _values(st["a"], 1, torch.float64), _values(st["b"], 1, torch.float64)
        for e in range(case["experts"]):
            n = off[e + 1] - off[e]
            dw[e] = a[:, at:at + n] @ b[:, at:at + n].t()
            at += _ceil(n, BLOCK) * BLOCK
        return dw
    # the loss's gradient from its definition by automatic differentiation
    x = st["x"].double().requires_grad_(True)
    T, E = x.shape
    k = st["topk"]
    rows = torch.arange(T, device=DEV) if st["mask"] is None else st["mask"].nonzero()[:, 0]
    n = rows.numel()
    w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    loss = x.new_zeros(1)
    if n:
        p = torch.softmax(x[rows], -1)
        idx = torch.sort(st["x"][rows].float(), dim=-1, descending=True, stable=True).indices[:, :k]
        share = torch.bincount(idx.reshape(-1), minlength=E).double() / (n * k)
        loss = (E * (share * p.mean(0)).sum()).reshape(1)
        wr = torch.gather(p, 1, idx)
        if case["renorm"]:
            wr = wr / wr.sum(-1, keepdim=True)
        w = w.index_put((rows,), wr)
    out = {"weights": w.detach(), "loss": loss.detach()}
    if case["train"]:
        total = (loss * st["d_loss"].double()).sum() + (w * st["d_weights"].double()).sum()
        out["d_logits"] = torch.autograd.grad(total, x)[0] if n else torch.zeros_like(x)
    return out
