"""A mixture layer's training step through the framework's calls together:
router, quantisers, experts' products forward and backward, weight gradients,
the router's backward -- against the same layer in fp64."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
from tests.gpu_util import need_gpu, note

pytestmark = pytest.mark.gpu
DEV = "cuda"


def values_of(op, block_rows=1):
    q, s = op
    rows, K = q.shape[-2:]
    f = s.double().repeat_interleave(block_rows, -1)[..., :rows].transpose(-1, -2)
    return q.double() * f.repeat_interleave(128, -1)[..., :K]


def step(x, logits, w, mask, dy, k):
    """One forward and backward of out[t] = sum_j weight_j * (x_t . W_e(j)^T)."""
    route = nv.nvfp4_moe_route(logits, k, mask=mask)
    total = route.row_index.numel()
    xq = nv.nvfp4_fp8_quantize(x)
    wq, wt = nv.nvfp4_fp8_quantize(w, block_rows=128, layout="both")
    h = torch.zeros(total, w.shape[1], device=x.device)
    nv.nvfp4_fp8_grouped_gemm(route.m_offsets, total, xq, wq, "f32", y=h, row_index=route.row_index)
    live = route.pair_row >= 0
    rows = route.pair_row.clamp_min(0).long()
    hk = h[rows] * live[..., None]
    out = (hk * route.weights[..., None]).sum(1)
    # backward: dh in grouped order, weights' gradients, then the products'
    d_weights = (hk * dy[:, None]).sum(-1)
    dh = torch.zeros(total, w.shape[1], device=x.device)
    dh[rows[live]] = (dy[:, None] * route.weights[..., None])[live]
    dhq, dht = nv.nvfp4_fp8_grouped_quantize(dh, route.m_offsets, layout="both")
    xt = nv.nvfp4_fp8_grouped_quantize(x, route.m_offsets, row_index=route.row_index)
    dw = nv.nvfp4_fp8_grouped_wgrad(route.m_offsets, total, dht, xt)
    dxg = torch.zeros(total, w.shape[2], device=x.device)
    nv.nvfp4_fp8_grouped_gemm(route.m_offsets, total, dhq, wt, "f32", y=dxg)
    dx = (dxg[rows] * live[..., None]).sum(1)
    dl = nv.nvfp4_moe_route_backward(logits, route, d_weights, torch.ones(1, device=x.device), mask=mask)
    return route, out, dx, dw, dl, (xq, wq, wt, dhq, dht, xt)


def test_training_step_of_a_mixture_layer():
    need_gpu()
    T, E, k, N, K = 150, 6, 2, 144, 272
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(T, K, generator=g).to(DEV), (torch.randn(E, N, K, generator=g) * K ** -0.5).to(DEV)
    logits, dy = torch.randn(T, E, generator=g).to(DEV), torch.randn(T, N, generator=g).to(DEV)
    mask = (torch.rand(T, generator=g) < 0.9).to(DEV)
    note("fp8 mixture layer step")
    route, out, dx, dw, dl, (xq, wq, wt, dhq, dht, xt) = step(x, logits, w, mask, dy, k)
    off, total = route.m_offsets.tolist(), route.row_index.numel()
    live = route.pair_row >= 0
    idx, rows = route.expert_index.long().clamp_min(0), route.pair_row.long().clamp_min(0)
    # the same layer in fp64 on the quantised values, expert by expert
    xv, wv, dv = values_of(xq), values_of(wq, 128), values_of(dhq)
    h = torch.einsum("tk,tjnk->tjn", xv.cpu(), wv[idx].cpu()).to(DEV) * live[..., None]
    want = (h * route.weights.double()[..., None]).sum(1)
    # off by fp32 accumulation alone: a hundredth of the 2^-4 of a rounding
    def near(a, b, rel):
        assert float((a.double() - b).norm()) <= rel * float(b.norm())
    near(out, want, 2e-6)
    dgr = dv[rows] * live[..., None]
    near(dx, torch.einsum("tjn,tjnk->tk", dgr.cpu(), wv[idx].cpu()).to(DEV), 2e-6)
    at = 0
    a, b = values_of(dht), values_of(xt)
    for e in range(E):
        n = off[e + 1] - off[e]
        near(dw[e], a[:, at:at + n] @ b[:, at:at + n].t(), 2e-6)
        # and the quantised gradient against the unquantised one: both
        # operands are off by up to 2^-4 relative, about a third of it in rms
        tok = route.row_index[off[e]:off[e + 1]].long()
        wt_e = (route.weights * (route.expert_index == e)).sum(1)[tok].double()
        near(dw[e], (dy[tok].double() * wt_e[:, None]).t() @ x[tok].double(), 2 ** -4)
        at += -(-n // 128) * 128
    # the router's gradient through the layer, by automatic differentiation
    z = logits.double().requires_grad_(True)
    p = torch.softmax(z[mask], -1)
    share = route.counts.double() / (mask.sum() * k)
    loss = E * (share * p.mean(0)).sum()
    wts = torch.gather(p, 1, idx[mask])
    total_loss = loss + (wts * (h[mask] * dy[mask].double()[:, None]).sum(-1)).sum()
    ref = torch.autograd.grad(total_loss, z)[0]
    near(dl, ref, 1e-5)
    assert abs(float(route.loss) - float(loss.detach())) <= 1e-6 * float(loss.detach())
    assert total == T * k and off[-1] == int(live.sum())


@pytest.mark.parametrize("T", [1, 4, 16, 64])
def test_a_decode_step_captured_and_replayed(T):
    """Router, quantiser and experts' product of few tokens in a graph, with
    eager steps between the replays; against eager and against fp64."""
    need_gpu()
    E, k, N, K = 32, 4, 272, 1040
    g = torch.Generator().manual_seed(T)
    wq = nv.nvfp4_fp8_quantize((torch.randn(E, N, K, generator=g) * K ** -0.5).to(DEV), block_rows=128)
    xs = [(torch.randn(T, K, generator=g).to(DEV), torch.randn(T, E, generator=g).to(DEV)) for _ in range(4)]

    def decode(x, logits):
        route = nv.nvfp4_moe_route(logits, k, renormalize=True)
        xq = nv.nvfp4_fp8_quantize(x)
        h = nv.nvfp4_fp8_grouped_gemm(route.m_offsets, T * k, xq, wq, "f32", row_index=route.row_index)
        return (h[route.pair_row.long()] * route.weights[..., None]).sum(1), route, xq

    note(f"fp8 mixture decode step T {T}")
    eager = [decode(*v) for v in xs]
    wv = values_of(wq, 128).cpu()
    for out, route, xq in eager:
        w = wv[route.expert_index.long().cpu()]                       # [T, k, N, K]
        h = (w * values_of(xq).cpu()[:, None, None, :]).sum(-1)
        want = (h * route.weights.double().cpu()[..., None]).sum(1)
        # fp32 accumulation alone, as above
        assert float((out.double().cpu() - want).norm()) <= 2e-6 * float(want.norm())
    xin, lin = xs[0][0].clone(), xs[0][1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed, _, _ = decode(xin, lin)
    for i in (1, 2, 3, 0, 2):
        xin.copy_(xs[i][0])
        lin.copy_(xs[i][1])
        graph.replay()
        again = decode(*xs[i])[0]
        torch.cuda.synchronize()
        assert torch.equal(replayed, eager[i][0]) and torch.equal(again, eager[i][0])


def test_the_router_feeds_the_4_bit_experts():
    """nvfp4_grouped_gemm reads the router's order as it stands."""
    need_gpu()
    T, E, k, N, K = 96, 8, 2, 64, 512
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(T, K, generator=g).to(DEV), torch.randn(E * N, K, generator=g).to(DEV)
    note("router and the 4-bit grouped product")
    route = nv.nvfp4_moe_route(torch.randn(T, E, generator=g).to(DEV), k)
    a, b = nv.nvfp4_quantize(x), nv.nvfp4_quantize(w)
    be = (b[0].view(E, N, -1), b[1].view(E, N, -1), b[2].repeat(E))
    y = nv.nvfp4_grouped_gemm(route.m_offsets, T * k, a, be, "f32", row_index=route.row_index)
    dense = nv.nvfp4_gemm(a, b, "f32").view(T, E, N)
    e = route.expert_index.long()
    want = torch.gather(dense, 1, e[..., None].expand(-1, -1, N))
    got = y[route.pair_row.long()]
    assert float((got - want).norm()) <= 1e-5 * float(want.norm())
