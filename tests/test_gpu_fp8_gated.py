"""Gated feed-forward block on FP8 operands on the GPU against the fp64 oracle:
the fused product (dense and per expert) and its backward."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
import workloads as wl
from oracle import (E4M3_TABLE, act_ref, fp8_dequantize_ref, gated_backward_ref, gated_ref, gated_tolerance,
                    sums_tolerance)
from tests.gpu_util import need_gpu, note, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def operand(rng, rows, K, block_rows=1, lead=(), size=1.0):
    """E4M3 bytes of normal values and scales such that values are around
    ``size``, over a factor of eight."""
    v = torch.from_numpy(rng.standard_normal((*lead, rows, K)).astype(np.float32) * 100).clamp(-448, 448)
    q = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    s = (np.exp2(rng.uniform(-1.5, 1.5, (*lead, -(-K // 128), -(-rows // block_rows)))) * size / 100).astype(np.float32)
    return q, s


def gpu(op):
    return torch.from_numpy(op[0]).to(DEV).view(torch.float8_e4m3fn), torch.from_numpy(op[1]).to(DEV)


def check(h, kept, a, w, block_rows, act, out, rows=None):
    """h and the kept products against the oracle; rows: those that are checked."""
    if rows is not None:
        a = a[0][rows], a[1][:, rows]
        h, kept = h[torch.from_numpy(rows).to(DEV)], None if kept is None else kept[torch.from_numpy(rows).to(DEV)]
    F = w[0].shape[0] // 2
    ref, g, u, bg, bu = gated_ref(*a, *w, block_rows, act)
    av, wv = fp8_dequantize_ref(*a), fp8_dequantize_ref(*w, block_rows)
    tg, tu = (sums_tolerance(b, av, v, out) for b, v in ((bg, wv[:F]), (bu, wv[F:])))

    def near(got, want, tol, what):
        got = np_(got).astype(np.float64)
        assert got.shape == want.shape
        bad = np.argwhere(~(np.abs(got - want) <= tol))
        assert bad.size == 0, (what, bad[:4].tolist(), got[tuple(bad[0])], want[tuple(bad[0])], tol[tuple(bad[0])])
    near(h, ref, gated_tolerance(g, u, tg, tu, act, out), "h")
    if kept is not None:
        # rounded once to bf16
        want, tol = np.concatenate([g, u], 1), np.concatenate([tg, tu], 1)
        near(kept, want, tol + 2.0 ** -8 * (np.abs(want) + tol), "gate_up")


SHAPES = [(1, 1, 16), (1, 24, 128), (2, 17, 144), (3, 256, 6144), (4, 40, 6160), (5, 8, 2064), (16, 128, 256),
          (16, 8200, 144), (17, 100, 512), (31, 130, 400), (33, 1000, 640), (48, 64, 2048), (64, 96, 272), (65, 129, 1040),
          (100, 513, 384), (128, 128, 128), (130, 2100, 256), (200, 333, 1552), (257, 640, 112), (70, 4160, 1040),
          (600, 1000, 272), (1000, 264, 2064)]


@pytest.mark.parametrize("M,F,K", SHAPES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out,act", [("f32", "silu"), ("bf16", "gelu"), ("bf16", "silu"), ("f32", "gelu")])
def test_gated(M, F, K, block_rows, out, act):
    rng = np.random.default_rng(M * 7 + F * 3 + K)
    # products around 2.5, where the activations bend
    a, w = operand(rng, M, K), operand(rng, 2 * F, K, block_rows, size=2.5 * K ** -0.5)
    note(f"fp8 gated {M}x{F}x{K} block_rows {block_rows} {act} {out}")
    h, kept = nv.nvfp4_fp8_gated_gemm(gpu(a), gpu(w), act, out, gate_up=True)
    check(h, kept, a, w, block_rows, act, out)
    assert torch.equal(nv.nvfp4_fp8_gated_gemm(gpu(a), gpu(w), act, out), h)


@pytest.mark.parametrize("M,F,K", [(1024, 1100, 384), (1000, 4100, 144), (1000, 2240, 272), (2500, 4096, 144),
                                   (4100, 2048, 272)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gated_many_tiles(M, F, K, block_rows, out):
    rng = np.random.default_rng(M + F + K)
    a, w = operand(rng, M, K), operand(rng, 2 * F, K, block_rows, size=2.5 * K ** -0.5)
    note(f"fp8 gated {M}x{F}x{K} block_rows {block_rows} {out} (many tiles)")
    h, kept = nv.nvfp4_fp8_gated_gemm(gpu(a), gpu(w), "silu", out, gate_up=True)
    rows = np.unique(np.concatenate([[0, 127, 128, 255, 256, M - 1], rng.choice(M, 24, replace=False)]))
    check(h, kept, a, w, block_rows, "silu", out, rows=rows)


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("F", [40, 61])
def test_gated_strided_outputs(M, F):
    rng = np.random.default_rng(M)
    K = 272
    a, w = operand(rng, M, K), operand(rng, 2 * F, K, 128, size=0.2)
    for out, dt in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        for lead in (0, 1):
            h = torch.full((M, F + 9), 7.0, dtype=dt, device=DEV)
            kept = torch.full((M, 2 * F + 11), 7.0, dtype=torch.bfloat16, device=DEV)
            note(f"fp8 gated strided M {M} F {F} {out} lead {lead}")
            hv, kv = h[:, lead:lead + F], kept[:, lead:lead + 2 * F]
            nv.nvfp4_fp8_gated_gemm(gpu(a), gpu(w), "gelu", out, h=hv, gate_up=kv)
            check(hv, kv, a, w, 128, "gelu", out)
            assert (h[:, :lead] == 7).all() and (h[:, lead + F:] == 7).all()
            assert (kept[:, :lead] == 7).all() and (kept[:, lead + 2 * F:] == 7).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [2, 100])
def test_gated_of_far_values(act, M):
    """Gates far beyond where sigma is 0 or 1 in fp32, up to 3e38, and zeros: no NaN,
    act(g) is g or 0."""
    K, F = 128, 32
    q = np.zeros((M, K), np.uint8)
    q[:, 0] = 0x38                                          # x = (1, 0, ..)
    w = np.zeros((2 * F, K), np.uint8)
    w[:, 0] = 0x38
    gate = np.array([0, 1e-30, -1e-30, 20, -20, 86.9, -86.9, 88, -88, 104, -104, 9.8, -9.8, 10, -10, 1e4, -1e4, 1e20,
                     -1e20, 3e38, -3e38] + [1.0] * 11, np.float32)
    s = np.concatenate([gate, np.full(F, 0.5, np.float32)])[None]
    a = (q, np.ones((1, M), np.float32))
    note(f"fp8 gated far values {act} M {M}")
    for out in ("f32", "bf16"):
        h = np_(nv.nvfp4_fp8_gated_gemm(gpu(a), gpu((w, s)), act, out)).astype(np.float64)
        assert np.isfinite(h).all()
        g = gate.astype(np.float64)[None]
        tol = gated_tolerance(g, 0.5, 0.0, 0.0, act, out)
        assert (np.abs(h - act_ref(g, act)[0] * 0.5) <= tol).all()


def test_gated_nan_scales_and_empty():
    rng = np.random.default_rng(0)
    for M, F in ((4, 40), (200, 70)):
        a, w = operand(rng, M, 256), operand(rng, 2 * F, 256, 1, size=0.2)
        a[1][1, 2], w[1][0, 5], w[1][1, F + 9] = np.nan, np.nan, np.nan
        note(f"fp8 gated NaN scales M {M}")
        h = nv.nvfp4_fp8_gated_gemm(gpu(a), gpu(w))
        want = torch.zeros(M, F, dtype=torch.bool)
        want[2], want[:, 5], want[:, 9] = True, True, True
        assert torch.equal(h.isnan().cpu(), want)
    f8 = torch.float8_e4m3fn
    note("fp8 gated empty")
    none = torch.zeros(0, 64, device=DEV).to(f8), torch.zeros(1, 0, device=DEV)
    w2 = torch.zeros(8, 64, device=DEV).to(f8), torch.ones(1, 8, device=DEV)
    assert nv.nvfp4_fp8_gated_gemm(none, w2).shape == (0, 4)
    k0 = torch.zeros(5, 0, device=DEV).to(f8), torch.zeros(0, 5, device=DEV)
    w0 = torch.zeros(8, 0, device=DEV).to(f8), torch.zeros(0, 8, device=DEV)
    h, kept = nv.nvfp4_fp8_gated_gemm(k0, w0, gate_up=True)
    assert (h == 0).all() and (kept == 0).all() and h.shape == (5, 4)


def test_gated_refusals():
    rng = np.random.default_rng(0)
    a, w = gpu(operand(rng, 4, 256)), gpu(operand(rng, 32, 256, 128))
    odd = gpu(operand(rng, 31, 256, 1))
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for call in (lambda: nv.nvfp4_fp8_gated_gemm(a, odd), lambda: nv.nvfp4_fp8_gated_gemm(a, w, "relu"),
                 lambda: nv.nvfp4_fp8_gated_gemm(a, w, out_dtype="f16"),
                 lambda: nv.nvfp4_fp8_gated_gemm(a, gpu(operand(rng, 32, 272, 128))),
                 lambda: nv.nvfp4_fp8_gated_gemm(gpu(operand(rng, 256, 256, 128)), w),
                 lambda: nv.nvfp4_fp8_gated_gemm(a, w, h=torch.empty(4, 32, dtype=torch.bfloat16, device=DEV)),
                 lambda: nv.nvfp4_fp8_gated_gemm(a, w, gate_up=torch.empty(4, 32, device=DEV)),
                 lambda: nv.nvfp4_fp8_gated_gemm(a, w, gate_up=torch.empty(32, 4, dtype=torch.bfloat16, device=DEV).t()),
                 lambda: nv.nvfp4_fp8_grouped_gated_gemm(off, 4, a, w),
                 lambda: nv.nvfp4_fp8_grouped_gated_gemm(off, 4, a, gpu(operand(rng, 32, 256, 1, (1,)))),
                 lambda: nv.nvfp4_fp8_grouped_gated_gemm(off, 5, a, gpu(operand(rng, 32, 256, 128, (1,)))),
                 lambda: nv.nvfp4_fp8_gated_backward(torch.zeros(4, 12, device=DEV), torch.zeros(4, 24, device=DEV)),
                 lambda: nv.nvfp4_fp8_gated_backward(torch.zeros(4, 16, device=DEV), torch.zeros(4, 16, device=DEV)),
                 lambda: nv.nvfp4_fp8_gated_backward(torch.zeros(4, 16, device=DEV), torch.zeros(4, 32, device=DEV),
                                                     layout="x"),
                 lambda: nv.nvfp4_fp8_gated_backward(torch.zeros(4, 16, device=DEV), torch.zeros(4, 32, device=DEV),
                                                     layout="rows", out=a)):
        with pytest.raises(ValueError):
            call()


# ---- experts ----------------------------------------------------------------

@pytest.mark.parametrize("counts", [[5], [1, 0, 2, 1], [3, 0, 40, 17, 0, 9], [130, 0, 1, 300], [20] * 70, [64] * 9,
                                    [700, 900, 500]])
@pytest.mark.parametrize("F,K", [(96, 272), (77, 400)])
@pytest.mark.parametrize("out,gather", [("bf16", True), ("bf16", False), ("f32", True)])
def test_experts(counts, F, K, out, gather):
    rng = np.random.default_rng(sum(counts) + F)
    G, total = len(counts), sum(counts)
    off = wl.ragged_offsets(counts)
    tokens = max(1, total // 2) if gather else total
    a = operand(rng, tokens, K)
    w = operand(rng, 2 * F, K, 128, (G,), size=2.5 * K ** -0.5)
    idx = torch.from_numpy(rng.integers(0, tokens, total).astype(np.int32)) if gather else None
    if gather and total > 4:
        idx[3], idx[4] = -1, tokens                       # rows of zeros
    note(f"fp8 gated experts {counts[:6]} F {F} K {K} {out} gather {gather}")
    h, kept = nv.nvfp4_fp8_grouped_gated_gemm(off.to(DEV), total, gpu(a), gpu(w), "silu", out, gate_up=True,
                                              row_index=None if idx is None else idx.to(DEV))
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        src = np.arange(lo, hi) if idx is None else idx[lo:hi].numpy()
        ok = (src >= 0) & (src < tokens)
        src = np.clip(src, 0, tokens - 1)
        ae = np.where(ok[:, None], a[0][src], 0).astype(np.uint8), np.ascontiguousarray(a[1][:, src])
        check(h[lo:hi], kept[lo:hi], ae, (w[0][e], w[1][e]), 128, "silu", out)


@pytest.mark.parametrize("F", [2048, 264])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_experts_many_tiles(F, out):
    """Enough rows for the large shapes; one expert busy, some idle; sampled rows."""
    rng = np.random.default_rng(F)
    counts = [1500, 0, 600, 300, 0, 1100, 900, 2]
    K, G, total = 272, len(counts), sum(counts)
    off = wl.ragged_offsets(counts)
    a, w = operand(rng, total, K), operand(rng, 2 * F, K, 128, (G,), size=0.15)
    note(f"fp8 gated experts many tiles F {F} {out}")
    h, kept = nv.nvfp4_fp8_grouped_gated_gemm(off.to(DEV), total, gpu(a), gpu(w), "gelu", out, gate_up=True)
    for e in range(G):
        if counts[e]:
            r = np.unique(np.concatenate([[0, counts[e] - 1], rng.choice(counts[e], min(counts[e], 12), replace=False)]))
            r = r + int(off[e])
            check(h, kept, a, (w[0][e], w[1][e]), 128, "gelu", out, rows=r)


@pytest.mark.parametrize("total", [12, 900])
def test_experts_leave_rows_of_no_group(total):
    rng = np.random.default_rng(3)
    used = total * 2 // 3
    off = wl.ragged_offsets([used // 3, 0, used - used // 3])
    a, w = operand(rng, total, 256), operand(rng, 80, 256, 128, (3,), size=0.2)
    h = torch.full((total, 40), 7.0, dtype=torch.bfloat16, device=DEV)
    kept = torch.full((total, 80), 7.0, dtype=torch.bfloat16, device=DEV)
    note(f"fp8 gated experts, rows behind the last group, {total}")
    nv.nvfp4_fp8_grouped_gated_gemm(off.to(DEV), total, gpu(a), gpu(w), h=h, gate_up=kept)
    assert (h[used:] == 7).all() and (kept[used:] == 7).all() and not (h[:used] == 7).all(1).any()
    dh = torch.randn(total, 40, generator=torch.Generator().manual_seed(0)).to(DEV)
    q = torch.full((total, 80), 0x11, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s = torch.full((1, total), -3.0, device=DEV)
    nv.nvfp4_fp8_grouped_gated_backward(dh, kept, off.to(DEV), layout="rows", out=(q, s))
    assert (q.view(torch.uint8)[used:] == 0x11).all() and (s[:, used:] == -3).all() and (s[:, :used] > 0).all()


# ---- backward ---------------------------------------------------------------

def grad_inputs(rng, rows, F, dh_dtype, gu_dtype):
    dh = torch.from_numpy(rng.standard_normal((rows, F)).astype(np.float32) * np.exp2(rng.integers(-12, 3, (rows, 1))).astype(np.float32))
    gu = torch.from_numpy(rng.standard_normal((rows, 2 * F)).astype(np.float32) * 3)
    return dh.to(dh_dtype), gu.to(gu_dtype)


def check_operand(op, ref, err, what):
    """An FP8 operand [rows, K] of values ``ref`` that were off by at most ``err``
    before: the scale is the block's largest magnitude over 448, rounded; the
    bytes round to 4 significant bits (half a step: 2^-4 of the value, 2^-10 of
    the scale below 2^-6), after a product with the reciprocal scale (three
    roundings more)."""
    q, s = np_(op[0].view(torch.uint8)), np_(op[1]).astype(np.float64)
    rows, K = ref.shape
    assert q.shape == ref.shape and s.shape == (-(-K // 128), rows)
    starts = np.arange(0, K, 128)
    amax = np.maximum(np.maximum.reduceat(np.abs(ref), starts, axis=1), 2.0 ** -100).T
    emax = np.maximum.reduceat(err, starts, axis=1).T
    assert (np.abs(s - amax / 448) <= emax / 448 + 2.0 ** -23 * (amax + emax) / 448).all(), what
    full = np.repeat(s.T, 128, 1)[:, :K]
    got = E4M3_TABLE[q] * full
    tol = err + 2.0 ** -22 * np.abs(ref)
    tol = tol + np.maximum(2.0 ** -4 * (np.abs(ref) + tol), 2.0 ** -10 * full * (1 + 2.0 ** -20))
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (what, bad[:4].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])], tol[tuple(bad[0])])


def turned(v, width):
    """v [rows, cols] -> [cols, width], zeros behind the rows."""
    out = np.zeros((v.shape[1], width))
    out[:, :v.shape[0]] = v.T
    return out


@pytest.mark.parametrize("rows,F", [(1, 8), (1, 128), (7, 72), (15, 64), (16, 256), (17, 136), (64, 128), (129, 200),
                                    (200, 1024), (300, 384), (33, 1032)])
@pytest.mark.parametrize("types", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                   (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(rows, F, types, act):
    rng = np.random.default_rng(rows + F)
    dh, gu = grad_inputs(rng, rows, F, *types)
    note(f"fp8 gated backward {rows}x{F} {types} {act}")
    r, c = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), act)
    ref, err = gated_backward_ref(dh.float().numpy(), gu.float().numpy(), act)
    check_operand(r, ref, err, "rows")
    width = -(-rows // 16) * 16
    check_operand(c, turned(ref, width), turned(err, width), "cols")
    one = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), act, layout="rows")
    two = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), act, layout="cols")
    for x, y in ((r, one), (c, two)):
        assert torch.equal(x[0].view(torch.uint8), y[0].view(torch.uint8)) and torch.equal(x[1], y[1])


def test_backward_against_differences():
    """dg and du as differences of h itself, within the E4M3 rounding."""
    rng = np.random.default_rng(5)
    gu, dh = rng.standard_normal((6, 32)).astype(np.float32) * 2, rng.standard_normal((6, 16)).astype(np.float32)
    for act in ("silu", "gelu"):
        step = 1e-5
        g, u = gu[:, :16].astype(np.float64), gu[:, 16:].astype(np.float64)
        dg = dh * u * (act_ref(g + step, act)[0] - act_ref(g - step, act)[0]) / (2 * step)
        du = dh * act_ref(g, act)[0]
        note(f"fp8 gated backward, differences {act}")
        r = nv.nvfp4_fp8_gated_backward(torch.from_numpy(dh).to(DEV), torch.from_numpy(gu).to(DEV), act, layout="rows")
        ref = np.concatenate([dg, du], 1)
        check_operand(r, ref, 1e-6 * np.abs(ref) + 1e-9, act)


@pytest.mark.parametrize("F", [128, 72])
def test_backward_strides_out_and_empty(F):
    rng = np.random.default_rng(F)
    dh, gu = grad_inputs(rng, 37, F, torch.bfloat16, torch.bfloat16)
    wide_d = torch.zeros(37, F + 24, dtype=torch.bfloat16, device=DEV)
    wide_g = torch.zeros(37, 2 * F + 40, dtype=torch.bfloat16, device=DEV)
    wide_d[:, 8:8 + F], wide_g[:, 16:16 + 2 * F] = dh.to(DEV), gu.to(DEV)
    note(f"fp8 gated backward strided F {F}")
    want = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV))
    for layout in ("rows", "cols", "both"):
        out = nv.nvfp4_fp8_gated_backward(torch.zeros_like(dh).to(DEV), gu.to(DEV), layout=layout)
        got = nv.nvfp4_fp8_gated_backward(wide_d[:, 8:8 + F], wide_g[:, 16:16 + 2 * F], layout=layout, out=out)
        pairs = zip(want, got) if layout == "both" else ((want[layout == "cols"], got),)
        for x, y in pairs:
            assert torch.equal(x[0].view(torch.uint8), y[0].view(torch.uint8)) and torch.equal(x[1], y[1])
    e = nv.nvfp4_fp8_gated_backward(dh.to(DEV)[:0], gu.to(DEV)[:0])
    assert e[0][0].shape == (0, 2 * F) and e[1][0].shape == (2 * F, 0)
    with pytest.raises(nv.Nvfp4Error):                     # off a 16-byte border
        nv.nvfp4_fp8_gated_backward(wide_d[:, 1:1 + F], wide_g[:, 16:16 + 2 * F])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_of_special_values(act):
    """Far gates give neither NaN nor infinity; a NaN or an infinity marks its
    blocks, and those only."""
    rows, F = 8, 256
    gate = torch.tensor([0.0, -0.0, 20, -20, 86, -86, 88, -88, 104, -104, 9.8, -9.8, 10, -10, 1e10, -1e10, 1e30, -1e30,
                         3e38, -3e38]).repeat(13)[:F]
    gu = torch.cat([gate.expand(rows, F), torch.full((rows, F), 0.5)], 1).contiguous()
    dh = torch.ones(rows, F)
    note(f"fp8 gated backward special values {act}")
    r, c = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), act)
    ref, err = gated_backward_ref(dh.numpy(), np.clip(gu.numpy(), -200, 200), act)
    v, _ = act_ref(np.clip(gate.numpy(), -200, 200), act)
    ref[:, F:] = np.where(np.abs(gate.numpy()) > 200, np.maximum(gate.numpy().astype(np.float64), 0), v)
    err[:, F:] = np.abs(ref[:, F:]) * 2.0 ** -20 + 2.0 ** -110
    check_operand(r, ref, err, "rows")
    check_operand(c, turned(ref, 16), turned(err, 16), "cols")
    dh[2, 5], gu = float("inf"), torch.ones(rows, 2 * F)
    gu[4, 130] = float("nan")
    r, c = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), act)
    want = torch.zeros(4, rows, dtype=torch.bool)
    want[0, 2] = want[2, 2] = want[1, 4] = want[3, 4] = True
    assert torch.equal(r[1].isnan().cpu(), want)
    want_c = torch.zeros(1, 2 * F, dtype=torch.bool)
    want_c[0, [5, F + 5, 130, F + 130]] = True
    assert torch.equal(c[1].isnan().cpu(), want_c)
    assert (r[0].view(torch.uint8).view(rows, 4, 128)[want.t().to(DEV)] == 0).all()


@pytest.mark.parametrize("counts", [[5], [0, 128, 0, 1, 129], [300, 0, 0], [1] * 70, [0, 0]])
@pytest.mark.parametrize("F", [128, 72])
def test_grouped_backward(counts, F):
    rng = np.random.default_rng(sum(counts))
    off, total = wl.ragged_offsets(counts), sum(counts)
    dh, gu = grad_inputs(rng, total, F, torch.bfloat16, torch.bfloat16)
    note(f"fp8 grouped gated backward {counts[:6]} F {F}")
    r, c = nv.nvfp4_fp8_grouped_gated_backward(dh.to(DEV), gu.to(DEV), off.to(DEV), "gelu")
    P = nv.nvfp4_fp8_grouped_columns(total, len(counts))
    if total == 0:
        assert r[0].shape == (0, 2 * F) and c[0].shape == (2 * F, 0)
        return
    dense = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), "gelu", layout="rows")
    assert torch.equal(r[0].view(torch.uint8), dense[0].view(torch.uint8)) and torch.equal(r[1], dense[1])
    ref, err = gated_backward_ref(dh.float().numpy(), gu.float().numpy(), "gelu")
    wide, werr, at = np.zeros((2 * F, P)), np.zeros((2 * F, P)), 0
    for lo, hi in zip(off[:-1].tolist(), off[1:].tolist()):
        wide[:, at:at + hi - lo], werr[:, at:at + hi - lo] = ref[lo:hi].T, err[lo:hi].T
        at += -(-(hi - lo) // 128) * 128
    check_operand(c, wide, werr, "cols")
    two = nv.nvfp4_fp8_grouped_gated_backward(dh.to(DEV), gu.to(DEV), off.to(DEV), "gelu", layout="cols")
    assert torch.equal(c[0].view(torch.uint8), two[0].view(torch.uint8)) and torch.equal(c[1], two[1])


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [30, 10, -5, 1000], [-7, 100, 60, 60], [2 ** 31 - 1, 0, 5, -2 ** 31]])
@pytest.mark.parametrize("total", [90, 700])
def test_offsets_that_are_none_stay_inside(offsets, total):
    """Offsets that are not running sums: what is written is anyone's guess, but it
    lies inside the outputs' rows."""
    rng = np.random.default_rng(9)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    F, K = 40, 144
    a, w = gpu(operand(rng, total, K)), gpu(operand(rng, 2 * F, K, 128, (3,), size=0.2))
    idx = torch.randint(-5, total + 5, (total,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to(DEV)
    room_h = torch.full((total + 40, F), 7.0, dtype=torch.bfloat16, device=DEV)
    room_k = torch.full((total + 40, 2 * F), 7.0, dtype=torch.bfloat16, device=DEV)
    note(f"fp8 gated, offsets {offsets} of {total}")
    for index in (None, idx):
        nv.nvfp4_fp8_grouped_gated_gemm(off, total, a, w, h=room_h[20:-20], gate_up=room_k[20:-20], row_index=index)
    P = nv.nvfp4_fp8_grouped_columns(total, 3)
    room_q = torch.full((total + 64, 2 * F), 3, dtype=torch.uint8, device=DEV)
    room_t = torch.full((2 * F + 32, P), 3, dtype=torch.uint8, device=DEV)
    s, st = torch.empty(1, total, device=DEV), torch.empty(P // 128, 2 * F, device=DEV)
    f8 = torch.float8_e4m3fn
    nv.nvfp4_fp8_grouped_gated_backward(torch.ones(total, F, device=DEV), torch.ones(total, 2 * F, device=DEV), off,
                                        out=((room_q[32:-32].view(f8), s), (room_t[16:-16].view(f8), st)))
    for t, edge, v in ((room_h, 20, 7), (room_k, 20, 7), (room_q, 32, 3), (room_t, 16, 3)):
        assert (t[:edge] == v).all() and (t[-edge:] == v).all()


def test_gated_far_rows():
    """Outputs past 2^31 elements; sampled rows."""
    M, F, K = 70000, 16400, 16
    rng = np.random.default_rng(4)
    a, w = operand(rng, M, K), operand(rng, 2 * F, K, 128, size=0.6)
    note(f"fp8 gated {M}x{F}x{K}: {M * 2 * F} kept products")
    h, kept = nv.nvfp4_fp8_gated_gemm(gpu(a), gpu(w), gate_up=True)
    rows = np.array([0, 32767, 65472, 65473, 69999])
    check(h, kept, a, w, 128, "silu", "bf16", rows=rows)
    note("fp8 gated backward of them")
    r = nv.nvfp4_fp8_gated_backward(h, kept, layout="rows")
    at = torch.from_numpy(rows).to(DEV)
    few = nv.nvfp4_fp8_gated_backward(h[at], kept[at], layout="rows")
    assert torch.equal(r[0][at].view(torch.uint8), few[0].view(torch.uint8)) and torch.equal(r[1][:, at], few[1])


# ---- the activations' tails ----------------------------------------------------

TAILS = {"silu": [-70, -86.5, -87, -87.5, -88, -90, -95, -100, -102.5, -104, -106, -150, 87, 88, 104, 150, 0.0, 1e-30],
         "gelu": [-9, -9.8, -9.9, -9.95, -10, -10.1, -10.2, -10.3, -10.5, -10.6, -10.8, -15, 9.9, 10, 10.7, 15, 0.0, 1e-30]}


def tail_error(g, act):
    """Largest error of sigma(z(g)) in fp32: relative, 8 roundings and gelu's z off by
    4 more (each moves exp by |z| 2^-24); below the normal numbers two roundings to
    multiples of 2^-149."""
    z = np.abs(g) if act == "silu" else 2 * np.sqrt(2 / np.pi) * (np.abs(g) + 0.044715 * np.abs(g) ** 3)
    sigma = np.where(g >= 0, 1.0, np.exp(-z))
    return (8 + (4 * z if act == "gelu" else 0)) * 2.0 ** -24 * sigma + 2 * 2.0 ** -150


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [2, 100])
def test_gated_tails(act, M):
    """Gates whose sigma is small or below the normal numbers, times an up projection
    that brings their products back: act(g) is not cut to zero."""
    K, F = 128, 32
    gate = np.resize(np.array(TAILS[act], np.float32), F)
    q, w = np.zeros((M, K), np.uint8), np.zeros((2 * F, K), np.uint8)
    q[:, 0] = w[:, 0] = 0x38                                 # 1
    up = 2.0 ** 100
    s = np.concatenate([gate, np.full(F, up, np.float32)])[None]
    g = gate.astype(np.float64)
    v = act_ref(g, act)[0]
    # g sigma rounds (below the normal numbers by up to 2^-150), and so does its product
    tol = up * (np.abs(g) * tail_error(g, act) + 2.0 ** -150) + 2 * 2.0 ** -24 * np.abs(v * up)
    note(f"fp8 gated tails {act} M {M}")
    for out in ("f32", "bf16"):
        h = np_(nv.nvfp4_fp8_gated_gemm(gpu((q, np.ones((1, M), np.float32))), gpu((w, s)), act, out)).astype(np.float64)
        t = tol if out == "f32" else tol + 2.0 ** -8 * (np.abs(v * up) + tol)
        bad = np.argwhere(~(np.abs(h - v * up) <= t))
        assert bad.size == 0, [(gate[j], h[i, j], (v * up)[j], t[j]) for i, j in bad[:4]]


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_tails(act):
    """The same of the gradients, one to a block (the transposed layout of one row), so
    that a scale shows its value."""
    gate = np.resize(np.array(TAILS[act], np.float32), 64)
    g, up = gate.astype(np.float64), 2.0 ** 60
    v, d = act_ref(g, act)
    sig = np.where(g == 0, 0.5, v / np.where(g == 0, 1.0, g))
    # |g z'| of act' = sigma + g sigma z' (1 - sigma)
    far = np.abs(g) if act == "silu" else 2 * np.sqrt(2 / np.pi) * (np.abs(g) + 3 * 0.044715 * np.abs(g) ** 3)
    dh, u = np.full(64, 2.0 ** 60, np.float32), np.full(64, up, np.float32)
    e = tail_error(g, act)
    dg, du = 2.0 ** 120 * d, 2.0 ** 60 * v
    parts = np.abs(sig) + np.abs(d - sig)
    # sigma's error in both parts (their 1 - sigma has it too where it is small), 8 roundings
    # more; a part below the normal numbers rounds by up to 2^-150
    err_dg = 2.0 ** 120 * ((1 + far) * 2 * e + 8 * 2.0 ** -24 * parts + (2 + far) * 2.0 ** -150)
    err_du = 2.0 ** 60 * (np.abs(g) * e + 2.0 ** -150) + 2 * 2.0 ** -24 * np.abs(du)
    note(f"fp8 gated backward tails {act}")
    c = nv.nvfp4_fp8_gated_backward(torch.from_numpy(dh)[None].to(DEV),
                                    torch.from_numpy(np.concatenate([gate, u]))[None].to(DEV), act, layout="cols")
    ref, err = np.concatenate([dg, du])[None], np.concatenate([err_dg, err_du])[None]
    check_operand(c, turned(ref, 16), turned(err, 16), "cols")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_rounds_as_fp32(act):
    """The slope's rounding errors over normal gates, in rms: a rounding to fp32 is off by
    2^-24 / sqrt(3) / m of the value, m its significand, 2^-24 * 0.577 * 0.7355 = 2.53e-8 in rms
    for m spread over its logarithm.  act' = sigma + act turn rounds once itself and takes
    over sigma's rounding; act, turn and the exponential (three roundings, the hardware's
    exp2 off by one unit) reach it with weights around 1/4: sqrt(2 + 5/16) = 1.52
    roundings.  The scale that shows it adds one: sqrt(2 + 5/16 + 1) = 1.82.  Not more
    than 2.1 of them; a rounding more in sigma (1 + t, or its reciprocal) gives 2.1 to 2.3."""
    g = torch.randn(1, 8192, generator=torch.Generator().manual_seed(7)) * 1.5
    gu, dh = torch.cat([g, torch.ones_like(g)], 1), torch.ones_like(g)
    note(f"fp8 gated backward rounding {act}")
    c = nv.nvfp4_fp8_gated_backward(dh.to(DEV), gu.to(DEV), act, layout="cols")
    got = np_(c[1]).astype(np.float64)[0, :8192] * 448
    want = np.abs(act_ref(g.numpy()[0], act)[1])
    assert np.linalg.norm(got - want) <= 2.1 * 2.53e-8 * np.linalg.norm(want)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_that_are_not_finite(act):
    """act(inf) = inf, act(-inf) and act(NaN) are NaN, as is act' of all three; the blocks
    that hold them are marked, finite gates beside them are not."""
    inf = float("inf")
    gate = torch.tensor([inf, -inf, float("nan"), 3e38, -3e38, 1.0, 0.0, -1.0])
    note(f"fp8 gated, gates that are not finite, {act}")
    for M in (2, 100):
        q = torch.zeros(M, 128)
        w = torch.zeros(16, 128)
        q[:, 0] = w[:, 0] = 1
        f8 = torch.float8_e4m3fn
        h = nv.nvfp4_fp8_gated_gemm((q.to(f8).to(DEV), torch.ones(1, M, device=DEV)),
                                    (w.to(f8).to(DEV), torch.cat([gate, torch.ones(8)])[None].to(DEV)), act, "f32").cpu()
        assert (h[:, 0] == inf).all() and h[:, 1:3].isnan().all() and h[:, 3:].isfinite().all()
    gu = torch.cat([gate, torch.ones(8)])[None]
    _, s = nv.nvfp4_fp8_gated_backward(torch.ones(1, 8, device=DEV), gu.to(DEV), act, layout="cols")
    assert s.cpu().isnan().tolist() == [[True] * 3 + [False] * 5 + [True] * 3 + [False] * 5]
