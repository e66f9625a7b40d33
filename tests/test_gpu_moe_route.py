"""The expert router on the GPU against the fp64 oracle: choices, counts and
order exactly, weights, loss and gradients within fp32 rounding."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
from oracle import moe_route_backward_ref, moe_route_ref
from tests.gpu_util import need_gpu, note, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"
# exp of a rounded argument below 88: 88 * 2^-24 in the argument and 2^-22 in
# the function, the same again in the sum's terms, and the sum and quotient
REL = 2 * 88 * 2.0 ** -24 + 2.0 ** -20


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def logits_of(T, E, seed, dtype):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * 2
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def check(x, k, mask=None, renorm=False, route=None):
    r = route or nv.nvfp4_moe_route(x.to(DEV), k, mask=None if mask is None else mask.to(DEV), renormalize=renorm)
    ref = moe_route_ref(x.float().numpy(), k, None if mask is None else mask.numpy(), renorm)
    for name in ("expert_index", "counts", "m_offsets", "row_index", "pair_row"):
        assert np.array_equal(np_(getattr(r, name)), ref[name]), name
    assert int(r.routed) == ref["routed"]
    w = np_(r.weights)
    assert np.all(np.abs(w - ref["weights"]) <= REL * ref["weights"] + 1e-37)
    # fp32 sums over at most 256 tokens of a workgroup, then wider
    assert abs(float(r.loss) - ref["loss"]) <= (REL + 512 * 2.0 ** -24) * ref["loss"]
    return r, ref


CASES = [(1, 8, 2), (1, 1, 1), (3, 64, 6), (16, 128, 8), (17, 7, 7), (64, 256, 8), (300, 60, 4), (257, 100, 3),
         (40, 257, 5), (33, 512, 16), (50, 1024, 9), (20, 1000, 8), (1000, 16, 2), (5000, 72, 2),
         (64, 200, 8), (65, 200, 8), (16, 1024, 16), (33, 8, 8), (100, 256, 8), (0, 40, 3)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("dtype,renorm,masked", [("fp32", False, False), ("fp32", True, True),
                                                 ("bf16", True, False), ("bf16", False, True)])
def test_route(T, E, k, dtype, renorm, masked):
    x = logits_of(T, E, T + E, dtype)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.7 if masked else None
    note(f"route {T}x{E} top {k} {dtype} renorm {renorm} masked {masked}")
    check(x, k, mask, renorm)


@pytest.mark.parametrize("T,E,k", [(64, 256, 2), (64, 255, 7), (64, 256, 7), (48, 256, 15), (48, 256, 16), (64, 128, 16),
                                   (64, 64, 16), (32, 512, 16), (33, 496, 4), (16, 1024, 1), (17, 1024, 1)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_both_sides_of_one_launch(T, E, k, dtype):
    x = logits_of(T, E, T * k + E, dtype)
    note(f"route {T}x{E} top {k} {dtype}")
    r, ref = check(x, k, torch.arange(T) % 5 != 3, True)
    back(x, k, r, ref, torch.arange(T) % 5 != 3, True)


@pytest.mark.parametrize("E", [8, 64, 256, 300, 1024])
def test_ties_go_to_the_lowest_expert(E):
    x = torch.zeros(70, E)
    x[10:40] = torch.randint(0, 3, (30, E), generator=torch.Generator().manual_seed(E)).float()
    x[40:] = -0.0
    note(f"route ties E {E}")
    check(x, 5)
    check(x.bfloat16(), 5, renorm=True)


@pytest.mark.parametrize("T,E,k", [(12, 8, 1), (64, 40, 5), (70, 256, 8), (40, 1024, 16), (300, 512, 3)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_zeros_of_either_sign_are_equal(T, E, k, dtype):
    """Rows of -1, -0 and +0 with fewer ones than choices, so that the border of
    the choice lies among zeros: the lowest experts of them, whatever their sign."""
    g = torch.Generator().manual_seed(T + E)
    x = torch.tensor([-1.0, -0.0, 0.0])[torch.randint(0, 3, (T, E), generator=g)]
    x[1::2, E // 2] = 1.0
    x[0, :3] = torch.tensor([-0.0, 0.0, -1.0])
    note(f"route zeros of either sign {T}x{E} top {k} {dtype}")
    check(x.bfloat16() if dtype == "bf16" else x, k)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_closed_experts_and_empty_rows(renorm, dtype):
    """-inf closes an expert; rows with fewer open experts than choices, with
    none, at the type's lowest value, and with very large spreads."""
    x = logits_of(90, 40, 5, dtype)
    x[0] = -float("inf")
    x[1, 1:] = -float("inf")
    x[2, ::2] = -float("inf")
    x[3] = torch.finfo(x.dtype).min
    x[4, 3:] = torch.finfo(x.dtype).min
    x[5] = torch.linspace(-80, 80, 40)
    x[:, 17] = -float("inf")
    mask = torch.ones(90, dtype=torch.bool)
    mask[80:] = False
    note(f"route closed experts {dtype} renorm {renorm}")
    r, ref = check(x, 6, mask, renorm)
    assert ref["counts"][17] == 0 and ref["routed"] == 79
    back(x, 6, r, ref, mask, renorm)


@pytest.mark.parametrize("T,E,k", [(9, 8, 8), (80, 40, 16), (70, 300, 4)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
def test_far_logits_keep_fp32_weights_and_gradients(T, E, k, dtype, renorm):
    """Every logit but one lies 20 to 80 below the top, in steps of 1/2, so the
    distances are exact.  Counted in 2^-24 relative: exp 3 (two of the
    instruction, one of its correction), the reciprocal and the product 2, one
    more for second-order terms; the sum is 1 and rounds away at most
    E exp(-20) = E * 0.035.  A gradient of an expert that was not chosen is
    -p <p, dw> with positive dw: the same error twice."""
    g = torch.Generator().manual_seed(E)
    x = -0.5 * torch.randint(40, 161, (T, E), generator=g).float()
    x[torch.arange(T), torch.randint(0, E, (T,), generator=g)] = 0.0
    x = x.bfloat16() if dtype == "bf16" else x
    note(f"route far logits {T}x{E} top {k} {dtype} renorm {renorm}")
    r = nv.nvfp4_moe_route(x.to(DEV), k, renormalize=renorm)
    ref = moe_route_ref(x.float().numpy(), k, None, renorm)
    assert np.array_equal(np_(r.expert_index), ref["expert_index"])
    rel = (6 + 0.035 * E) * 2.0 ** -24
    assert np.abs(np_(r.weights) / ref["weights"] - 1).max() <= rel
    if dtype == "bf16" or renorm or E == k:
        return
    dw = torch.rand(T, k, generator=g) + 0.5
    got = np_(nv.nvfp4_moe_route_backward(x.to(DEV), r, dw.to(DEV)))
    want = moe_route_backward_ref(ref, k, dw.numpy(), 0.0)
    rest = np.ones((T, E), bool)
    np.put_along_axis(rest, ref["expert_index"], False, 1)
    assert np.abs(got[rest] / want[rest] - 1).max() <= 2 * rel


@pytest.mark.parametrize("T", [8, 300])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_nan_logit_shows_in_its_token_alone(T, renorm, dtype):
    """NaN is outside the contract, but must not turn into a plausible weight;
    logits at the lowest value and at -inf beside it stay zeros."""
    x = logits_of(T, 20, 6, dtype)
    x[1, 3], x[2, 5:], x[3, 5:] = float("nan"), torch.finfo(x.dtype).min, -float("inf")
    x = x.to(DEV)
    note(f"route nan logit T {T} renorm {renorm} {dtype}")
    r = nv.nvfp4_moe_route(x, 3, renormalize=renorm)
    g = nv.nvfp4_moe_route_backward(x, r, torch.ones(T, 3, device=DEV), torch.ones(1, device=DEV), renormalize=renorm)
    rest = torch.arange(T, device=DEV) != 1
    assert bool(r.weights[1].isnan().all()) and bool(r.weights[rest].isfinite().all())
    assert bool(g[1].isnan().any()) and bool(g[rest].isfinite().all())
    assert not bool(g[2:4, 5:].any())


def test_all_masked_and_no_tokens():
    note("route with no token")
    for x, mask in ((logits_of(9, 12, 1, "fp32"), torch.zeros(9, dtype=torch.bool)),
                    (torch.empty(0, 12), None), (torch.full((5, 12), -float("inf")), None)):
        r = nv.nvfp4_moe_route(x.to(DEV), 3, mask=None if mask is None else mask.to(DEV))
        assert not np_(r.counts).any() and not np_(r.m_offsets).any() and float(r.loss) == 0 and int(r.routed) == 0
        assert (np_(r.row_index) == -1).all() and (np_(r.expert_index) == -1).all() and (np_(r.weights) == 0).all()
        g = nv.nvfp4_moe_route_backward(x.to(DEV), r, torch.ones(x.shape[0], 3, device=DEV),
                                        torch.ones(1, device=DEV), mask=None if mask is None else mask.to(DEV))
        assert g.shape == x.shape and not np_(g).any()


def back(x, k, r, ref, mask=None, renorm=False, use=("w", "l")):
    T, E = x.shape
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    dl = 0.37
    g = nv.nvfp4_moe_route_backward(
        x.to(DEV), r, dw.to(DEV) if "w" in use else None,
        torch.tensor([dl], device=DEV) if "l" in use else None,
        mask=None if mask is None else mask.to(DEV), renormalize=renorm)
    assert g.dtype == x.dtype
    want = moe_route_backward_ref(ref, k, dw.numpy() if "w" in use else np.zeros((T, k)),
                                  dl if "l" in use else 0.0, renorm)
    # every term is a product of values off by REL; the inner product sums
    # E + k of them in fp32
    p, c = ref["p"], dl * E * ref["counts"] / max(1, ref["routed"]) ** 2 / k
    size = p * (c + (p * c).sum(1, keepdims=True) + np.abs(dw.numpy()).sum(1, keepdims=True))
    chosen = ref["expert_index"]
    for t in range(T):
        for j in range(k):
            if chosen[t, j] >= 0:
                size[t, chosen[t, j]] += ref["weights"][t, j] * np.abs(dw[t].numpy()).sum()
    tol = (4 * REL + (E + k) * 2.0 ** -24) * size + 1e-37
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = np_(g)
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (bad[:4].tolist(), got[tuple(bad[0])], want[tuple(bad[0])], tol[tuple(bad[0])])


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (17, 7, 7), (64, 256, 8), (300, 60, 4), (40, 257, 5), (33, 512, 16),
                                   (20, 1000, 8)])
@pytest.mark.parametrize("dtype,renorm,masked", [("fp32", False, False), ("fp32", True, True),
                                                 ("bf16", False, True), ("bf16", True, False)])
@pytest.mark.parametrize("use", [("w", "l"), ("w",), ("l",), ()])
def test_backward(T, E, k, dtype, renorm, masked, use):
    x = logits_of(T, E, T + E, dtype)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.7 if masked else None
    note(f"route backward {T}x{E} top {k} {dtype} renorm {renorm} masked {masked} {use}")
    r, ref = check(x, k, mask, renorm)
    back(x, k, r, ref, mask, renorm, use)


def test_gradient_against_differences():
    """The kernels' own loss and weights, moved: fp32 rounding over a step of
    2^-6 leaves about 1e-4; the second-order error is of the same size."""
    x = logits_of(6, 20, 3, "fp32")
    k, h = 3, 2.0 ** -6
    dw = torch.randn(6, k, generator=torch.Generator().manual_seed(4))
    note("route gradient against differences")
    r = nv.nvfp4_moe_route(x.to(DEV), k)
    g = np_(nv.nvfp4_moe_route_backward(x.to(DEV), r, dw.to(DEV), torch.tensor([0.5], device=DEV)))

    def value(y):
        q = nv.nvfp4_moe_route(y.to(DEV), k)
        if not torch.equal(q.expert_index, r.expert_index):
            return None
        return 0.5 * float(q.loss.double()) + float((q.weights.double().cpu() * dw.double()).sum())

    seen = 0
    for t in range(6):
        for e in range(20):
            up, dn = x.clone(), x.clone()
            up[t, e] += h
            dn[t, e] -= h
            a, b = value(up), value(dn)
            if a is not None and b is not None:
                seen += 1
                assert abs((a - b) / (2 * h) - g[t, e]) < 5e-4
    assert seen > 60


@pytest.mark.parametrize("T,E,k", [(20000, 256, 8), (70000, 32, 2)])
def test_many_tokens(T, E, k):
    """Several 256-token runs a workgroup; checked with tensor operations."""
    x = logits_of(T, E, 7, "bf16").to(DEV)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(2)).to(DEV) < 0.9
    note(f"route {T}x{E}")
    r = nv.nvfp4_moe_route(x, k, mask=mask)
    idx = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :k]
    idx = torch.where(mask[:, None], idx, -1)
    assert torch.equal(r.expert_index.long(), idx)
    flat = torch.where(idx < 0, E, idx).reshape(-1)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    assert torch.equal(r.counts.long(), counts)
    assert torch.equal(r.m_offsets[1:].long(), torch.cumsum(counts, 0)) and int(r.m_offsets[0]) == 0
    order = torch.sort(flat, stable=True).indices
    total = int(counts.sum())
    assert torch.equal(r.row_index[:total].long(), (order // k)[:total]) and bool((r.row_index[total:] == -1).all())
    live = r.pair_row.reshape(-1) >= 0
    assert torch.equal(r.row_index[r.pair_row.reshape(-1)[live].long()].long(),
                       (torch.arange(T * k, device=DEV) // k)[live])
    p = torch.softmax(x[mask].double(), -1)
    n = int(mask.sum())
    loss = float(E * (counts.double() / (n * k) * p.mean(0)).sum())
    assert int(r.routed) == n and abs(float(r.loss) - loss) <= (REL + 512 * 2.0 ** -24) * loss
    again = nv.nvfp4_moe_route(x, k, mask=mask)
    assert all(torch.equal(a, b) for a, b in zip(r, again))


def test_strided_logits_workspace_and_out():
    wide = logits_of(50, 300, 11, "bf16")
    view = wide.to(DEV)[:, 3:3 + 64]
    ws = torch.empty(nv.nvfp4_moe_route_workspace_bytes(50, 64), dtype=torch.uint8, device=DEV)
    note("route strided logits")
    r = nv.nvfp4_moe_route(view, 4, workspace=ws)
    x = wide[:, 3:67].contiguous()
    _, ref = check(x, 4, route=r)
    out = torch.full((50, 100), 9.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.randn(50, 4, device=DEV)
    g = nv.nvfp4_moe_route_backward(view, r, dw, out=out[:, 5:69])
    assert torch.equal(g, nv.nvfp4_moe_route_backward(x.to(DEV), r, dw))
    assert bool((out[:, :5] == 9.0).all()) and bool((out[:, 69:] == 9.0).all())


@pytest.mark.parametrize("T", [0, 9, 700])
def test_outputs_are_tensors_of_their_own(T):
    """Scaling the weights in place leaves what a backward saved as it was,
    and keeping the loss keeps nothing else alive."""
    x = logits_of(T, 16, 3, "fp32").to(DEV)
    note(f"route outputs T {T}")
    r = nv.nvfp4_moe_route(x, 4)
    held = [t.untyped_storage().data_ptr() for t in r if t.numel()]
    assert len(set(held)) == len(held)
    before = {n: t._version for n, t in r._asdict().items()}
    r.weights.mul_(2.0)
    assert {n for n, t in r._asdict().items() if t._version != before[n]} == {"weights"}
    assert r.loss.untyped_storage().nbytes() == 4


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, k):
        r = nv.nvfp4_moe_route(x, k)
        ctx.save_for_backward(x, r.expert_index, r.counts, r.routed)
        ctx.mark_non_differentiable(r.expert_index)
        return r.weights, r.expert_index

    @staticmethod
    def backward(ctx, d_weights, _):
        x, index, counts, routed = ctx.saved_tensors
        r = nv.MoeRoute(index, None, counts, None, None, None, routed, None)
        return nv.nvfp4_moe_route_backward(x, r, d_weights.contiguous()), None


def test_weights_scaled_in_place_before_the_backward():
    x = logits_of(30, 16, 4, "fp32").to(DEV)
    dw = torch.randn(30, 4, generator=torch.Generator().manual_seed(1)).to(DEV)
    note("route weights scaled in place")
    z = x.clone().requires_grad_(True)
    w, _ = _Route.apply(z, 4)
    w.mul_(2.0)
    w.backward(dw)
    assert torch.equal(z.grad, nv.nvfp4_moe_route_backward(x, nv.nvfp4_moe_route(x, 4), 2 * dw))


def test_captured_and_replayed():
    """Two graphs with their own outputs and workspaces, replayed beside eager
    calls with changing logits."""
    xs = [logits_of(700, 48, 30 + i, "fp32").to(DEV) for i in range(3)]
    dw, dl = torch.randn(700, 2, device=DEV), torch.ones(1, device=DEV)
    ins = [xs[0].clone(), xs[0].clone()]
    graphs, outs = [], []
    note("route captured")
    nv.nvfp4_moe_route(xs[0], 2)
    torch.cuda.synchronize()
    for xin in ins:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = nv.nvfp4_moe_route(xin, 2)
            g = nv.nvfp4_moe_route_backward(xin, r, dw, dl)
        graphs.append(gr)
        outs.append((*r, g))
    for i in (1, 2, 0, 1):
        for j, gr in enumerate(graphs):
            ins[j].copy_(xs[(i + j) % 3])
            gr.replay()
        for j in range(2):
            x = xs[(i + j) % 3]
            r = nv.nvfp4_moe_route(x, 2)
            g = nv.nvfp4_moe_route_backward(x, r, dw, dl)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[j], (*r, g)))


def test_wrappers_refuse():
    x = torch.zeros(4, 8, device=DEV)
    r = nv.nvfp4_moe_route(x, 2)
    for call in (lambda: nv.nvfp4_moe_route(x, 0), lambda: nv.nvfp4_moe_route(x, 9),
                 lambda: nv.nvfp4_moe_route(x.half(), 2),
                 lambda: nv.nvfp4_moe_route(x, 2, mask=torch.ones(3, dtype=torch.bool, device=DEV)),
                 lambda: nv.nvfp4_moe_route(x, 2, mask=torch.ones(4, device=DEV)),
                 lambda: nv.nvfp4_moe_route_backward(x[:3], r),
                 lambda: nv.nvfp4_moe_route_backward(x, r, torch.ones(4, 3, device=DEV)),
                 lambda: nv.nvfp4_moe_route_backward(x, r, d_loss=torch.ones(2, device=DEV)),
                 lambda: nv.nvfp4_moe_route_backward(x, r, out=torch.empty(4, 8, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_moe_route(torch.zeros(4, 1100, device=DEV), 2)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_moe_route(x, 2, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
