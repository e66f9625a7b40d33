"""Feed-forward layers through the framework's calls together: a dense gated
block's and a mixture's training step (fused product, its backward, weight
gradients, clipping), the trained weights served in INT8, and decode steps in a
graph -- against the same layers in fp64."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
from oracle import act_ref, int8_gemm_ref, int8_quantize_ref, moe_route_ref
from tests.gpu_util import need_gpu, note, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def values_of(op, block_rows=1):
    q, s = op
    rows, K = q.shape[-2:]
    f = s.double().cpu().repeat_interleave(block_rows, -1)[..., :rows].transpose(-1, -2)
    return q.cpu().double() * f.repeat_interleave(128, -1)[..., :K]


def act(g, kind):
    v, d = act_ref(g.numpy(), kind)
    return torch.from_numpy(v), torch.from_numpy(d)


def near(a, b, rel):
    assert float((a.double().cpu() - b).norm()) <= rel * float(b.norm())


# fp32 accumulation alone (a hundredth of the 2^-4 of an E4M3 rounding would be
# far more); one rounding to bf16; an operand quantised to E4M3: each element off
# by up to 2^-4, in rms about a third of that
SUMS, BF16, E4M3 = 2e-6, 2.0 ** -8, 2.0 ** -4


def quantised(op, value):
    """An FP8 operand's values against what was quantised; returns them."""
    v = values_of(op)[:, :value.shape[1]]
    near(v, value, E4M3)
    return v


@pytest.mark.parametrize("T,D,F,kind", [(96, 272, 144, "silu"), (200, 256, 256, "gelu"), (37, 400, 176, "silu")])
def test_training_steps_of_a_dense_block(T, D, F, kind):
    need_gpu()
    g = torch.Generator().manual_seed(T)
    w, wd = (torch.randn(2 * F, D, generator=g) * D ** -0.5).to(DEV), (torch.randn(D, F, generator=g) * F ** -0.5).to(DEV)
    dw, dwd = torch.zeros_like(w), torch.zeros_like(wd)
    wr, wt = nv.nvfp4_fp8_quantize(w, block_rows=128, layout="both")
    dr, dt = nv.nvfp4_fp8_quantize(wd, block_rows=128, layout="both")
    wv, dv = values_of(wr, 128), values_of(dr, 128)
    want_w, want_wd = torch.zeros(2 * F, D, dtype=torch.float64), torch.zeros(D, F, dtype=torch.float64)
    for micro in range(2):                                  # two microbatches into one gradient
        x, dy = torch.randn(T, D, generator=g).to(DEV), torch.randn(T, D, generator=g).to(DEV)
        note(f"feed-forward training step T {T} D {D} F {F} {kind} {micro}")
        xr, xt = nv.nvfp4_fp8_quantize(x, layout="both")
        h, gu = nv.nvfp4_fp8_gated_gemm(xr, wr, kind, gate_up=True)
        hr, ht = nv.nvfp4_fp8_quantize(h, layout="both")
        y = nv.nvfp4_fp8_gemm(hr, dr, "f32")
        dyr, dyt = nv.nvfp4_fp8_quantize(dy, layout="both")
        dh = nv.nvfp4_fp8_gemm(dyr, dt, "f32")
        gr, gc = nv.nvfp4_fp8_gated_backward(dh, gu, kind)
        dx = nv.nvfp4_fp8_gemm(gr, wt, "f32")
        nv.nvfp4_fp8_gemm(gc, xt, "f32", y=dw, accumulate=True)
        nv.nvfp4_fp8_gemm(dyt, ht, "f32", y=dwd, accumulate=True)
        # the same in fp64 on the quantised values
        p = values_of(xr) @ wv.t()
        v, slope = act(p[:, :F], kind)
        near(gu, p, BF16)
        near(h, v * p[:, F:], BF16)
        hv = quantised(hr, h.double().cpu())
        near(y, hv @ dv.t(), SUMS)
        near(dh, values_of(dyr) @ dv, SUMS)
        kept = gu.double().cpu()
        v, slope = act(kept[:, :F], kind)
        d = dh.double().cpu()
        grad = torch.cat([d * kept[:, F:] * slope, d * v], 1)
        gv = quantised(gr, grad)
        quantised(gc, grad.t())
        near(dx, gv @ wv, SUMS)
        want_w += values_of(gc) @ values_of(xt).t()
        want_wd += values_of(dyt) @ values_of(ht).t()
        # and the step against the unquantised one: every operand off as above,
        # three of them in a row
        p = x.double().cpu() @ w.double().cpu().t()
        v, slope = act(p[:, :F], kind)
        near(y, (v * p[:, F:]) @ wd.double().cpu().t(), 3 * E4M3)
        d = dy.double().cpu() @ wd.double().cpu()
        near(dx, torch.cat([d * p[:, F:] * slope, d * v], 1) @ w.double().cpu(), 3 * E4M3)
    near(dw, want_w, SUMS)
    near(dwd, want_wd, SUMS)
    norm = float(torch.sqrt(want_w.square().sum() + want_wd.square().sum()))
    n = nv.nvfp4_clip_grads([dw, dwd], 0.3 * norm)
    assert abs(float(n) / norm - 1) < SUMS
    near(dw, 0.3 * want_w, SUMS)
    near(dwd, 0.3 * want_wd, SUMS)
    # a step down the gradient, and the new weights served in 8-bit integers
    w -= 0.01 * dw
    wd -= 0.01 * dwd
    x = torch.randn(5, D, generator=g).to(DEV)
    wi, di = nv.nvfp4_int8_quantize(w), nv.nvfp4_int8_quantize(wd)
    p = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(x), wi, "f32")
    assert np.array_equal(np_(p), int8_gemm_ref(*int8_quantize_ref(np_(x)), *int8_quantize_ref(np_(w))))
    v, _ = act(p.double().cpu()[:, :F], kind)
    h = (v * p.double().cpu()[:, F:]).float().to(DEV)
    y = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(h), di, "f32")
    # a row's integers are off by half a step of its largest over 127, a few
    # hundredths of its rms at most, in both operands of both products
    q = x.double().cpu() @ w.double().cpu().t()
    v, _ = act(q[:, :F], kind)
    near(y, (v * q[:, F:]) @ wd.double().cpu().t(), 0.05)


def test_training_step_of_a_gated_mixture():
    need_gpu()
    T, E, k, F, D = 150, 6, 2, 176, 272
    g = torch.Generator().manual_seed(0)
    x, dy = torch.randn(T, D, generator=g).to(DEV), torch.randn(T, D, generator=g).to(DEV)
    w, wd = (torch.randn(E, 2 * F, D, generator=g) * D ** -0.5).to(DEV), (torch.randn(E, D, F, generator=g) * F ** -0.5).to(DEV)
    route = moe_route_ref(torch.randn(T, E, generator=g).numpy(), k)
    off, idx = torch.from_numpy(route["m_offsets"]).to(DEV), torch.from_numpy(route["row_index"]).to(DEV)
    rows, weights = torch.from_numpy(route["pair_row"]).long(), torch.from_numpy(route["weights"])
    total = T * k
    note("feed-forward mixture training step")
    xr = nv.nvfp4_fp8_quantize(x)
    xt = nv.nvfp4_fp8_grouped_quantize(x, off, row_index=idx)
    wr, wt = nv.nvfp4_fp8_quantize(w, block_rows=128, layout="both")
    dr, dt = nv.nvfp4_fp8_quantize(wd, block_rows=128, layout="both")
    h, gu = nv.nvfp4_fp8_grouped_gated_gemm(off, total, xr, wr, gate_up=True, row_index=idx)
    hr, ht = nv.nvfp4_fp8_grouped_quantize(h, off, layout="both")
    y = nv.nvfp4_fp8_grouped_gemm(off, total, hr, dr, "f32")
    # gradient of each grouped row: its token's, times the router's weight
    scale = torch.zeros(total, dtype=torch.float64)
    scale[rows.reshape(-1)] = weights.reshape(-1)
    dyg = (dy.double().cpu()[idx.cpu().long()] * scale[:, None]).float().to(DEV)
    dyr, dyt = nv.nvfp4_fp8_grouped_quantize(dyg, off, layout="both")
    dh = nv.nvfp4_fp8_grouped_gemm(off, total, dyr, dt, "f32")
    gr, gc = nv.nvfp4_fp8_grouped_gated_backward(dh, gu, off)
    dxg = nv.nvfp4_fp8_grouped_gemm(off, total, gr, wt, "f32")
    dw = nv.nvfp4_fp8_grouped_wgrad(off, total, gc, xt)
    dwd = nv.nvfp4_fp8_grouped_wgrad(off, total, dyt, ht)
    n = nv.nvfp4_clip_grads([dw, dwd], 1e-2)

    wv, dv, xv, hv, dyv, gv = (values_of(o, b) for o, b in ((wr, 128), (dr, 128), (xr, 1), (hr, 1), (dyr, 1), (gr, 1)))
    want_w, want_wd, at = torch.zeros(E, 2 * F, D, dtype=torch.float64), torch.zeros(E, D, F, dtype=torch.float64), 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        p = xv[idx[lo:hi].cpu().long()] @ wv[e].t()
        v, _ = act(p[:, :F], "silu")
        near(gu[lo:hi], p, BF16)
        near(h[lo:hi], v * p[:, F:], BF16)
        near(y[lo:hi], hv[lo:hi] @ dv[e].t(), SUMS)
        near(dh[lo:hi], dyv[lo:hi] @ dv[e], SUMS)
        kept, d = gu[lo:hi].double().cpu(), dh[lo:hi].double().cpu()
        v, slope = act(kept[:, :F], "silu")
        grad = torch.cat([d * kept[:, F:] * slope, d * v], 1)
        near(gv[lo:hi], grad, E4M3)
        near(dxg[lo:hi], gv[lo:hi] @ wv[e], SUMS)
        cols = slice(at, at + hi - lo)
        near(values_of(gc)[:, cols], grad.t(), E4M3)
        want_w[e] = values_of(gc)[:, cols] @ values_of(xt)[:, cols].t()
        want_wd[e] = values_of(dyt)[:, cols] @ values_of(ht)[:, cols].t()
        at += -(-(hi - lo) // 128) * 128
    norm = float(torch.sqrt(want_w.square().sum() + want_wd.square().sum()))
    assert abs(float(n) / norm - 1) < SUMS
    near(dw, want_w * (1e-2 / norm), SUMS)
    near(dwd, want_wd * (1e-2 / norm), SUMS)


@pytest.mark.parametrize("T", [1, 16, 64])
def test_a_decode_step_captured_and_replayed(T):
    """A mixture's gated experts and a dense block of few tokens in one graph, with
    eager steps between the replays; every replay equals the eager step."""
    need_gpu()
    E, k, F, D = 16, 4, 144, 1040
    g = torch.Generator().manual_seed(T)
    we = nv.nvfp4_fp8_quantize((torch.randn(E, 2 * F, D, generator=g) * D ** -0.5).to(DEV), block_rows=128)
    wd = nv.nvfp4_fp8_quantize((torch.randn(2 * F, D, generator=g) * D ** -0.5).to(DEV), block_rows=128)
    wi = nv.nvfp4_int8_quantize(torch.randn(D, F, generator=g).to(DEV))
    xs = [(torch.randn(T, D, generator=g).to(DEV), torch.randn(T, E, generator=g).to(DEV)) for _ in range(4)]

    def step(x, logits):
        route = nv.nvfp4_moe_route(logits, k, renormalize=True)
        xq = nv.nvfp4_fp8_quantize(x)
        h, gu = nv.nvfp4_fp8_grouped_gated_gemm(route.m_offsets, T * k, xq, we, gate_up=True,
                                                row_index=route.row_index)
        back = nv.nvfp4_fp8_grouped_gated_backward(h, gu, route.m_offsets, layout="both")
        dense = nv.nvfp4_fp8_gated_gemm(xq, wd, "gelu")
        y = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(dense), wi, "f32")
        return [h, gu, dense, y, back[0][0].view(torch.uint8), back[0][1], back[1][0].view(torch.uint8), back[1][1]]

    note(f"feed-forward decode step T {T}")
    eager = [step(*v) for v in xs]
    xin, lin = xs[0][0].clone(), xs[0][1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step(xin, lin)
    for i in (1, 2, 3, 0, 2):
        xin.copy_(xs[i][0])
        lin.copy_(xs[i][1])
        graph.replay()
        again = step(*xs[i])
        torch.cuda.synchronize()
        for a, b, c in zip(replayed, again, eager[i]):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_two_streams_at_once():
    """The same operators on two streams with nothing shared: each gives what it
    gives alone."""
    need_gpu()
    g = torch.Generator().manual_seed(3)
    jobs = []
    for i in range(2):
        x = nv.nvfp4_fp8_quantize(torch.randn(300, 512, generator=g).to(DEV))
        w = nv.nvfp4_fp8_quantize((torch.randn(400, 512, generator=g) * 0.05).to(DEV), block_rows=128)
        grads = [torch.randn(50000, generator=g).to(DEV), torch.randn(777, generator=g).to(DEV).to(torch.bfloat16)]
        jobs.append((x, w, grads, [torch.empty_like(t) for t in grads]))

    def run(job, stream=None):
        x, w, grads, out = job
        h, gu = nv.nvfp4_fp8_gated_gemm(x, w, gate_up=True, stream=stream)
        r = nv.nvfp4_fp8_gated_backward(h, gu, layout="rows", stream=stream)
        n = nv.nvfp4_clip_grads(grads, 3.0, out=out, stream=stream)
        return [h, gu, r[0].view(torch.uint8), r[1], n, *out]
    note("feed-forward operators on two streams")
    alone = [[t.clone() for t in run(j)] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        both = [run(j, s) for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
