"""Gradient norm and clipping on the GPU against fp64."""
import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
from oracle import clip_ref
from tests.gpu_util import need_gpu, note, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def grads_of(sizes, seed, kinds="mixed", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n, generator=g) * scale * 10.0 ** float(torch.randint(-3, 2, (1,), generator=g))
        out.append(t.to(torch.bfloat16) if kinds == "bf16" or (kinds == "mixed" and i % 2) else t)
    return out


def check(outs, grads, coefficient):
    """out = g * c: c is off by the norm's and its own rounding (2^-23 together,
    the 64-bit sums add nothing), the fp32 product rounds once, bf16 once more."""
    for o, g in zip(outs, grads):
        want = np_(g).astype(np.float64) * coefficient
        tol = (2.0 ** -23 + 2.0 ** -24) * np.abs(want) + 2.0 ** -149
        if o.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -134
        assert o.shape == g.shape
        assert (np.abs(np_(o).astype(np.float64) - want) <= tol).all()


SIZES = [[1], [7, 0, 3], [2048, 2049, 1, 4097], [100000], [64] * 130, [5] * 400, [1 << 20, 17, 300000, 8192]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("kinds", ["f32", "bf16", "mixed"])
def test_clip(sizes, kinds):
    grads = grads_of(sizes, len(sizes) + sizes[0], kinds)
    norm, _, _ = clip_ref([np_(g) for g in grads], 1.0)
    for part in (0.37, 1.5):
        note(f"clip {len(sizes)} tensors {kinds} part {part}")
        top = norm * part
        on = [g.clone().to(DEV) for g in grads]
        n2 = nv.nvfp4_grad_norm_sq(on)
        assert n2.dtype == torch.float64 and abs(float(n2) - norm ** 2) <= 1e-13 * norm ** 2
        outs = [torch.empty_like(g) for g in on]
        n = nv.nvfp4_clip_grads(on, top, out=outs)
        assert n.dtype == torch.float32 and abs(float(n) - norm) <= 2.0 ** -23 * norm
        check(outs, grads, min(1.0, part))
        for a, b in zip(on, grads):                         # read only
            assert torch.equal(a.cpu(), b)
        n_in = nv.nvfp4_clip_grads(on, top)
        assert torch.equal(n_in, n)
        for a, b in zip(on, outs):                          # in place: the same values
            assert torch.equal(a, b)


@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5, 8])
def test_clip_of_views_at_any_address(shift):
    """Views that start off 16-byte borders, both types, into outputs of either
    type at other borders; what lies beside them stays."""
    for dt in (torch.float32, torch.bfloat16):
        for odt in (torch.float32, torch.bfloat16):
            for other in (0, shift, 1):
                base = torch.randn(30000, generator=torch.Generator().manual_seed(shift)).to(dt).to(DEV)
                room = torch.full((30000,), 9.0, dtype=odt, device=DEV)
                spans = [(shift, 5000), (6000 + shift, 6001 + shift), (9000 + shift, 25013)]
                g = [base[a:b] for a, b in spans]
                o = [room[a + other:b + other] for a, b in spans]
                note(f"clip views shift {shift} {dt} -> {odt} other {other}")
                norm, _, _ = clip_ref([np_(t) for t in g], 1.0)
                nv.nvfp4_clip_grads(g, 0.1 * norm, out=o)
                check(o, [t.cpu() for t in g], 0.1)
                keep = torch.ones(30000, dtype=torch.bool)
                for a, b in spans:
                    keep[a + other:b + other] = False
                assert (room.cpu()[keep] == 9).all()


def test_norm_of_extreme_values():
    note("clip extreme values")
    big = torch.full((1000,), 3e38, device=DEV)
    tiny = torch.full((1000,), 1e-40, device=DEV)
    assert abs(float(nv.nvfp4_grad_norm_sq([big])) / (1000 * float(np.float32(3e38)) ** 2) - 1) < 1e-12
    want = float(np.float32(1e-40))
    assert abs(float(nv.nvfp4_grad_norm_sq([tiny])) / (1000 * want ** 2) - 1) < 1e-12
    n = nv.nvfp4_clip_grads([big], 1.0)
    assert torch.isinf(n).all() or float(n) > 3e38          # beyond fp32, though the sum is not
    assert abs(float(big.double().norm()) - 1) < 1e-6       # and it clips by the sum
    zeros = torch.zeros(100, device=DEV)
    assert float(nv.nvfp4_clip_grads([zeros], 1.0)) == 0 and (zeros == 0).all()
    some = torch.ones(100, device=DEV)
    assert float(nv.nvfp4_clip_grads([some], 0.0)) == 10 and (some == 0).all()
    some = torch.ones(100, device=DEV)
    assert float(nv.nvfp4_clip_grads([some], math.inf)) == 10 and (some == 1).all()
    assert float(nv.nvfp4_clip_grads([some], 10.0)) == 10 and (some == 1).all()   # at the border
    none = [torch.empty(0, device=DEV), torch.empty(0, dtype=torch.bfloat16, device=DEV)]
    assert float(nv.nvfp4_clip_grads(none, 1.0)) == 0 and float(nv.nvfp4_grad_norm_sq(none)) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    g = [torch.randn(5000, device=DEV), torch.randn(300, device=DEV).to(torch.bfloat16)]
    g[0][4321] = bad
    before = [t.clone() for t in g]
    note(f"clip {bad}")
    n = nv.nvfp4_clip_grads(g, 1e-3)
    assert not torch.isfinite(n).any()
    out = [torch.zeros_like(t) for t in g]
    nv.nvfp4_clip_grads(g, 1e-3, out=out)
    for a, b, o in zip(g, before, out):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(o.view(torch.int16), b.view(torch.int16))


def test_a_norm_from_elsewhere():
    """Shards' sums added before clipping, as several processes do it."""
    grads = grads_of([3000, 500, 12345], 3)
    norm, _, _ = clip_ref([np_(g) for g in grads], 1.0)
    on = [g.clone().to(DEV) for g in grads]
    note("clip with a given norm")
    total = nv.nvfp4_grad_norm_sq(on[:1]) + nv.nvfp4_grad_norm_sq(on[1:])
    for part in (on[:1], on[1:]):
        n = nv.nvfp4_clip_grads(part, 0.25 * norm, norm_sq=total)
        assert abs(float(n) - norm) <= 2.0 ** -23 * norm
    check(on, grads, 0.25)


def test_workspaces_and_refusals():
    on = [g.to(DEV) for g in grads_of([300, 40], 1)]
    ws = torch.empty(nv.nvfp4_grad_workspace_bytes(2), dtype=torch.uint8, device=DEV)
    note("clip workspaces and refusals")
    a = nv.nvfp4_grad_norm_sq(on, workspace=ws)
    assert torch.equal(a, nv.nvfp4_grad_norm_sq(on))
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_grad_norm_sq(on, workspace=ws[:64])
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_clip_grads([on[0], on[0]], 1.0)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_clip_grads([on[0]], 1.0, out=[on[0].view(torch.float32)[:300].view(torch.bfloat16)[:300]])
    for call in (lambda: nv.nvfp4_clip_grads([on[0].view(10, 30).t()], 1.0),
                 lambda: nv.nvfp4_clip_grads([on[0].half()], 1.0), lambda: nv.nvfp4_clip_grads([on[0], on[1].cpu()], 1.0),
                 lambda: nv.nvfp4_clip_grads(on, 1.0, out=[on[0]]), lambda: nv.nvfp4_clip_grads(on, float("nan")),
                 lambda: nv.nvfp4_clip_grads(on, 1.0, out=[on[0], on[1][:20]]),
                 lambda: nv.nvfp4_clip_grads(on, 1.0, norm_sq=torch.ones(1, device=DEV))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("count", [3, 300])
def test_clip_captured_and_replayed(count):
    lists = [[g.to(DEV) for g in grads_of([4000 + 7 * i for i in range(count)], s)] for s in range(3)]
    norms = [clip_ref([np_(g) for g in gs], 1.0)[0] for gs in lists]
    top = 0.5 * min(norms)
    note(f"clip graph {count}")
    out = [torch.empty_like(g) for g in lists[0]]
    eager = []
    for gs in lists:
        n = nv.nvfp4_clip_grads(gs, top, out=out)
        eager.append((n.clone(), [o.clone() for o in out]))
    held = [g.clone() for g in lists[0]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = nv.nvfp4_clip_grads(lists[1], top, out=out, stream=side)
    side.synchronize()
    assert torch.equal(n, eager[1][0]) and all(torch.equal(a, b) for a, b in zip(out, eager[1][1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = nv.nvfp4_clip_grads(held, top, out=out)
    for i in (1, 2, 0, 1):
        for h, g in zip(held, lists[i]):
            h.copy_(g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, eager[i][0]) and all(torch.equal(a, b) for a, b in zip(out, eager[i][1]))
        nv.nvfp4_grad_norm_sq(lists[i])


def test_clip_of_a_tensor_past_31_bits():
    n = (1 << 31) + 4099
    g = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    g[-1], g[1 << 31] = 3.0, 2.0
    note(f"clip {n} elements")
    norm = math.sqrt(n - 2 + 9 + 4)
    assert float(nv.nvfp4_grad_norm_sq([g])) == n - 2 + 9 + 4      # whole numbers: exact
    out = torch.empty_like(g)
    top = nv.nvfp4_clip_grads([g], 0.5 * norm, out=[out])
    assert abs(float(top) - norm) <= 2.0 ** -23 * norm
    assert float(out[-1]) == 1.5 and float(out[1 << 31]) == 1.0 and bool((out[: 1 << 31] == 0.5).all())
    assert bool((out[(1 << 31) + 1:-1] == 0.5).all())


@pytest.mark.parametrize("dt,odt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_empty_tensors_into_another_type(dt, odt):
    grads = [torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dt) for n in (5, 0, 300, 0)]
    on = [g.to(DEV) for g in grads]
    norm, _, _ = clip_ref([np_(g) for g in grads], 1.0)
    note(f"clip with empty tensors {dt} -> {odt}")
    out = [torch.empty(g.shape, dtype=odt, device=DEV) for g in on]
    n = nv.nvfp4_clip_grads(on, 0.4 * norm, out=out)
    assert abs(float(n) - norm) <= 2.0 ** -23 * norm
    check(out, grads, 0.4)
