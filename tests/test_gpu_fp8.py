"""FP8 block-128 operators on the GPU against the fp64 oracle: the quantisers
byte for byte, the products within the error of fp32 accumulation
(oracle.fp8_tolerance derives it)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
import workloads as wl
from oracle import (E4M3_TABLE, fp8_dequantize_ref, fp8_gemm_ref, fp8_grouped_quantize_t_ref, fp8_quantize_ref, fp8_quantize_t_ref,
                    fp8_tolerance)
from tests.gpu_util import need_gpu, note, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def bytes_of(q):
    return np_(q.view(torch.uint8))


def same(op, ref):
    q, s = bytes_of(op[0]), np_(op[1])
    rq, rs = ref
    assert q.shape == rq.shape and s.shape == rs.shape
    assert np.array_equal(s, rs, equal_nan=True), np.argwhere(s != rs)[:4]
    assert np.array_equal(q, rq), np.argwhere(q != rq)[:4]


def values(rows, cols, seed, dtype="bf16", spread=8.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x = x * torch.exp2(torch.randint(-int(spread), int(spread) + 1, (rows, 1), generator=g).float())
    return x.to(torch.bfloat16) if dtype == "bf16" else x


# ---- quantisers -------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (7, 144), (64, 256), (129, 400), (200, 2064)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_both_layouts(dtype, rows, cols, block_rows):
    x = values(rows, cols, rows + cols, dtype)
    note(f"fp8 quantize {dtype} {rows}x{cols} block_rows {block_rows}")
    r, t = nv.nvfp4_fp8_quantize(x.to(DEV), block_rows=block_rows, layout="both")
    only_r = nv.nvfp4_fp8_quantize(x.to(DEV), block_rows=block_rows)
    only_t = nv.nvfp4_fp8_quantize(x.to(DEV), block_rows=block_rows, layout="cols")
    ref, ref_t = fp8_quantize_ref(x.float().numpy(), block_rows), fp8_quantize_t_ref(x.float().numpy(), block_rows)
    same(r, ref)
    same(only_r, ref)
    same(t, ref_t)
    same(only_t, ref_t)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_blocks(block_rows):
    x = torch.zeros(260, 384)
    x[1, 3], x[2, 200], x[130, 130] = float("nan"), float("inf"), -float("inf")
    x[3], x[4, :128], x[5, 0] = 1e-40, 3e38, -0.0
    x[140:, 256:] = torch.randn(120, 128, generator=torch.Generator().manual_seed(1)) * 1e-30
    note(f"fp8 quantize special blocks {block_rows}")
    r, t = nv.nvfp4_fp8_quantize(x.to(DEV), block_rows=block_rows, layout="both")
    same(r, fp8_quantize_ref(x.numpy(), block_rows))
    same(t, fp8_quantize_t_ref(x.numpy(), block_rows))


def test_quantize_batches_strides_and_out():
    w = torch.stack([values(200, 272, 5 + i, "fp32") for i in range(3)])
    note("fp8 quantize batch")
    r, t = nv.nvfp4_fp8_quantize(w.to(DEV), block_rows=128, layout="both")
    r1 = nv.nvfp4_fp8_quantize(w.to(DEV), block_rows=1)
    for i in range(3):
        same((r[0][i], r[1][i]), fp8_quantize_ref(w[i].numpy(), 128))
        same((t[0][i], t[1][i]), fp8_quantize_t_ref(w[i].numpy(), 128))
        same((r1[0][i], r1[1][i]), fp8_quantize_ref(w[i].numpy(), 1))
    wide = values(50, 512, 9)
    out = nv.nvfp4_fp8_quantize(wide.to(DEV)[:, 64:64 + 160].contiguous())
    note("fp8 quantize strided rows into given buffers")
    got = nv.nvfp4_fp8_quantize(wide.to(DEV)[:, 64:64 + 160], out=out)
    assert got[0].data_ptr() == out[0].data_ptr()
    same(got, fp8_quantize_ref(wide[:, 64:224].float().numpy()))
    assert nv.nvfp4_fp8_quantize(torch.empty(0, 64, device=DEV))[0].shape == (0, 64)


@pytest.mark.parametrize("counts", [[5], [0, 128, 0, 1, 129], [300, 0, 0], [1] * 70, [0, 0]])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_quantize(counts, gather):
    off = wl.ragged_offsets(counts)
    total = int(off[-1])
    src = values(max(total, 1), 144, total + gather)[:max(total, 1) if gather else total]
    idx = torch.randint(-1, src.shape[0] + 1, (total,), generator=torch.Generator().manual_seed(2)).int()
    x = src.float()
    if gather:
        x = torch.where(((idx >= 0) & (idx < src.shape[0]))[:, None], x[idx.long().clamp(0, src.shape[0] - 1)], 0.0)
    note(f"fp8 grouped quantize {counts[:6]} gather {gather}")
    r, t = nv.nvfp4_fp8_grouped_quantize(src.to(DEV), off.to(DEV), layout="both",
                                         row_index=idx.to(DEV) if gather else None)
    if total == 0:
        assert r[0].shape == (0, 144) and t[0].shape == (144, 0)
        return
    same(r, fp8_quantize_ref(x.numpy()))
    same(t, fp8_grouped_quantize_t_ref(x.numpy(), off.tolist()))


def test_grouped_quantize_leaves_rows_of_no_group():
    x = values(40, 128, 3)
    off = torch.tensor([0, 10, 25], dtype=torch.int32)
    q = torch.full((40, 128), 0x11, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s = torch.full((1, 40), -3.0, device=DEV)
    note("fp8 grouped quantize, rows behind the last group")
    nv.nvfp4_fp8_grouped_quantize(x.to(DEV), off.to(DEV), layout="rows", out=(q, s))
    assert (bytes_of(q)[25:] == 0x11).all() and (np_(s)[:, 25:] == -3.0).all()
    rq, rs = fp8_quantize_ref(x[:25].float().numpy())
    assert np.array_equal(bytes_of(q)[:25], rq) and np.array_equal(np_(s)[:, :25], rs)


# ---- products ---------------------------------------------------------------

def rand_operand(rng, rows, K, block_rows=1, lead=()):
    """Random finite E4M3 bytes and scales over three decades."""
    q = rng.integers(0, 256, (*lead, rows, K)).astype(np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x3C
    s = np.exp2(rng.uniform(-8, 2, (*lead, -(-K // 128), -(-rows // block_rows)))).astype(np.float32)
    return q, s


def to_gpu(op):
    return (torch.from_numpy(op[0]).to(DEV).view(torch.float8_e4m3fn), torch.from_numpy(op[1]).to(DEV))


def close(y, a, b, block_rows, out, rows=None, add=None):
    """y against the oracle; rows: the rows of y and a that are checked."""
    aq, sa = (a[0], a[1]) if rows is None else (a[0][rows], a[1][:, rows])
    ref, base = fp8_gemm_ref(aq, sa, b[0], b[1], block_rows)
    tol = fp8_tolerance(ref, base, fp8_dequantize_ref(aq, sa), fp8_dequantize_ref(b[0], b[1], block_rows), out)
    if add is not None:          # one more fp32 addition
        ref = ref + add
        tol = tol + 2.0 ** -24 * (np.abs(ref) + tol)
    got = np_(y).astype(np.float64)
    got = got if rows is None else got[rows]
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (bad[:4].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])], tol[tuple(bad[0])])


SHAPES = [(1, 1, 16), (1, 300, 128), (2, 17, 144), (3, 256, 1024), (5, 8, 2064), (16, 128, 256), (17, 200, 512),
          (31, 130, 400), (33, 1000, 640), (48, 64, 8192), (64, 96, 272), (65, 129, 1040), (100, 513, 384),
          (128, 128, 128), (130, 4100, 256), (200, 333, 1552), (257, 640, 112), (70, 8300, 2064), (600, 1000, 1040),
          (1000, 520, 8192)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm(M, N, K, block_rows, out):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    note(f"fp8 gemm {M}x{N}x{K} block_rows {block_rows} {out}")
    y = nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), out)
    close(y, a, b, block_rows if N > 1 else 1, out)


@pytest.mark.parametrize("M,N,K", [(1024, 1100, 384), (4096, 1024, 256), (2500, 4200, 144), (4096, 4096, 128),
                                   (8192, 8200, 272)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_gemm_many_tiles(M, N, K, block_rows):
    """Enough tiles for the large tile shapes, ragged edges; sampled rows."""
    rng = np.random.default_rng(M + N + K)
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    note(f"fp8 gemm {M}x{N}x{K} block_rows {block_rows} (many tiles)")
    y = nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "f32")
    rows = np.unique(np.concatenate([[0, 127, 128, 255, 256, M - 1], rng.choice(M, 40, replace=False)]))
    close(y, a, b, block_rows, "f32", rows=rows)


@pytest.mark.parametrize("M,N,K", [(20, 16400, 272), (90, 16400, 144), (512, 4104, 272), (1000, 8200, 144),
                                   (1000, 4500, 272), (2500, 8200, 144)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_gemm_many_tiles_bf16(M, N, K, block_rows):
    """The 8-bit products' tile shapes, ragged edges; sampled rows."""
    rng = np.random.default_rng(M + N + K)
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    note(f"fp8 gemm {M}x{N}x{K} block_rows {block_rows} bf16 (many tiles)")
    y = nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "bf16")
    rows = np.unique(np.concatenate([[0, M // 2, M - 1], rng.choice(M, min(M, 24), replace=False)]))
    close(y, a, b, block_rows, "bf16", rows=rows)


@pytest.mark.parametrize("M,N,K,block_rows", [(1, 512, 512, 128), (40, 300, 272, 1), (300, 257, 384, 1),
                                              (300, 257, 384, 128), (600, 1500, 400, 1), (70, 8300, 272, 128)])
def test_gemm_accumulates(M, N, K, block_rows):
    rng = np.random.default_rng(M + N)
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    y0 = rng.standard_normal((M, N)).astype(np.float32) * 1e3
    y = torch.from_numpy(y0).to(DEV)
    note(f"fp8 gemm accumulate {M}x{N}x{K}")
    assert nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "f32", y=y, accumulate=True) is y
    close(y, a, b, block_rows, "f32", add=y0.astype(np.float64))


@pytest.mark.parametrize("M", [1, 3, 4, 5])
@pytest.mark.parametrize("N,K", [(300, 6144), (4099, 6160), (133, 8208), (72, 6128), (200, 4112)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out,add", [("f32", False), ("f32", True), ("bf16", False)])
def test_gemm_few_rows_of_long_k(M, N, K, block_rows, out, add):
    """Both sides of the borders (4 rows, K = 6144) of the widest split of K;
    numbers of blocks that the waves do not share evenly, a last block cut."""
    rng = np.random.default_rng(M + N + K)
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    y0 = rng.standard_normal((M, N)).astype(np.float32) * 1e3 if add else None
    note(f"fp8 gemm {M}x{N}x{K} block_rows {block_rows} {out} add {add}")
    y = nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), out, y=torch.from_numpy(y0).to(DEV) if add else None, accumulate=add)
    close(y, a, b, block_rows, out, add=y0.astype(np.float64) if add else None)


@pytest.mark.parametrize("M,N,K,block_rows", [(40, 1500, 272, 128), (500, 500, 272, 1), (600, 1500, 400, 128),
                                              (1024, 4100, 144, 128), (1024, 4100, 144, 1), (2000, 4100, 144, 128),
                                              (2000, 4100, 144, 1), (2, 4099, 4112, 128), (2, 4099, 8208, 1)])
def test_gemm_accumulates_in_every_shape(M, N, K, block_rows):
    rng = np.random.default_rng(M + N)
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    y0 = rng.standard_normal((M, N)).astype(np.float32) * 1e3
    y = torch.from_numpy(y0).to(DEV)
    note(f"fp8 gemm accumulate {M}x{N}x{K} block_rows {block_rows}")
    nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "f32", y=y, accumulate=True)
    close(y, a, b, block_rows, "f32", add=y0.astype(np.float64))


@pytest.mark.parametrize("M,N", [(1, 130), (20, 130), (200, 130), (2100, 130)])
@pytest.mark.parametrize("out,ld,shift", [("bf16", 136, 0), ("bf16", 133, 1), ("f32", 132, 0), ("f32", 131, 3)])
def test_gemm_writes_only_its_view(M, N, out, ld, shift):
    """Row strides and bases that allow 16-byte stores and ones that do not;
    the bytes around y stay."""
    rng = np.random.default_rng(ld)
    K = 256
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, 128)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    buf = torch.full((M * ld + 64,), 7.0, dtype=dt, device=DEV)
    y = buf[shift:shift + M * ld].view(M, ld)[:, :N]
    note(f"fp8 gemm strided y M {M} {out} ld {ld} shift {shift}")
    nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), out, y=y)
    close(y, a, b, 128, out)
    rest = buf.clone()
    rest[shift:shift + M * ld].view(M, ld)[:, :N] = 7.0
    assert bool((rest == 7.0).all())


@pytest.mark.parametrize("M", [3, 40, 300, 1100])
def test_gemm_exact_codes_and_nan_scales(M):
    """Every finite code against a unit row: exact; a NaN scale marks its row
    (or column block) and no other."""
    K, N = 256, 256
    rng = np.random.default_rng(M)
    bq = np.tile(np.arange(256, dtype=np.uint8), (N, 1))
    bq[:, [0x7F, 0xFF]] = 0
    b = (bq, np.ones((2, 2), np.float32))
    aq = np.zeros((M, K), np.uint8)
    hot = rng.permutation(K)[:M] if M <= K else rng.integers(0, K, M)
    aq[np.arange(M), hot] = 0x38                     # 1.0
    a = (aq, np.ones((2, M), np.float32))
    note(f"fp8 gemm one-hot rows M {M}")
    y = np_(nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "f32"))
    vals = torch.from_numpy(bq).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(y, vals[:, hot].T)
    a[1][1, 1] = np.nan
    b[1][0, 1] = np.nan
    y = np_(nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "f32"))
    assert np.isnan(y[1]).all() and np.isnan(y[:, 128:]).all()
    assert np.isfinite(np.delete(y, 1, 0)[:, :128]).all()


def outliers(rng, rows, K, second):
    """Values of 0.5 to 1.5 and in each block of 128 two of 448, the second as
    the code given."""
    q = rng.choice(np.array([0x30, 0x34, 0x38, 0x3C, 0xB0, 0xB8], np.uint8), (rows, K))
    q[:, 3::128], q[:, 9::128] = 0x7E, second
    return q, np.exp2(rng.uniform(-2, 2, (-(-K // 128), rows))).astype(np.float32)


def few_rows_close(y, a, b, block_rows, out):
    """Few rows keep fp32 sums for bf16 outputs too: one rounding more."""
    ref, base = fp8_gemm_ref(*a, *b, block_rows)
    tol = fp8_tolerance(ref, base, fp8_dequantize_ref(*a), fp8_dequantize_ref(*b, block_rows), "f32")
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = np.argwhere(~(np.abs(np_(y).astype(np.float64) - ref) <= tol))
    assert bad.size == 0, (bad[:4].tolist(), np_(y)[tuple(bad[0])], ref[tuple(bad[0])], tol[tuple(bad[0])])


@pytest.mark.parametrize("M,N,K", [(1, 300, 4112), (2, 300, 6160), (3, 128, 256), (5, 8200, 400), (16, 520, 2064), (20, 130, 400),
                                   (30, 4000, 272)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_few_rows_with_outliers_that_cancel(M, N, K, block_rows, out):
    """The two largest products of every block cancel; what is left is a few
    thousandths of them."""
    rng = np.random.default_rng(M + N)
    a, b = outliers(rng, M, K, 0x7E), outliers(rng, N, K, 0xFE)
    b = b if block_rows == 1 else (b[0], np.ascontiguousarray(b[1][:, ::128]))
    note(f"fp8 gemm cancelling outliers {M}x{N}x{K} block_rows {block_rows} {out}")
    few_rows_close(nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), out), a, b, block_rows, out)


@pytest.mark.parametrize("counts,N,K", [([2, 0, 1, 3], 300, 4112), ([1, 0, 3, 9, 2, 17, 0, 33], 1032, 1040),
                                        ([1, 0, 2, 1, 3], 2056, 1040)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_few_grouped_rows_with_outliers_that_cancel(counts, N, K, out):
    rng = np.random.default_rng(N)
    off = wl.ragged_offsets(counts)
    a, bs = outliers(rng, int(off[-1]), K, 0x7E), [outliers(rng, N, K, 0xFE) for _ in counts]
    b = (np.stack([q for q, _ in bs]), np.stack([s[:, ::128] for _, s in bs]))
    note(f"fp8 grouped cancelling outliers {counts} N {N} K {K} {out}")
    y = nv.nvfp4_fp8_grouped_gemm(off.to(DEV), int(off[-1]), to_gpu(a), to_gpu(b), out)
    for e, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        if lo < hi:
            few_rows_close(y[lo:hi], (a[0][lo:hi], a[1][:, lo:hi]), (b[0][e], b[1][e]), 128, out)


@pytest.mark.parametrize("M,N,K", [(2, 300, 4112), (40, 300, 272), (40, 1500, 272), (300, 1500, 400), (600, 1000, 1040),
                                   (2048, 8200, 144)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("small,large,second", [(None, 0x7E, 0xFE), (0x4F, 0x78, 0xF8), (0x4F, 0x78, 0x4F)])
def test_gemm_with_outliers(M, N, K, block_rows, out, small, large, second):
    """Every kernel, with blocks of a few large products that cancel or stand
    alone and many that lie just above the 8-bit instruction's last bit (7.5 of
    256^2: half of it is cut): fp32 outputs within fp32 sums, bf16 ones within
    2^-9 of the sum of magnitudes and their own rounding."""
    rng = np.random.default_rng(M + K)
    a, b = outliers(rng, M, K, 0x7E), outliers(rng, N, K, 0xFE)
    if small is not None:
        a[0][:], b[0][:] = 0x38, small
        a[0][:, 3::128] = b[0][:, 3::128] = large
        a[0][:, 9::128], b[0][:, 9::128] = (large, second) if second > 127 else (0x38, small)
    b = b if block_rows == 1 else (b[0], np.ascontiguousarray(b[1][:, ::128]))
    note(f"fp8 gemm outliers {M}x{N}x{K} block_rows {block_rows} {out} {large:#x} {second:#x}")
    y = nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), out)
    rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 24)]))
    a = (a[0][rows], a[1][:, rows])
    ref, base = fp8_gemm_ref(*a, *b, block_rows)
    tol = fp8_tolerance(ref, base, fp8_dequantize_ref(*a), fp8_dequantize_ref(*b, block_rows), "f32")
    if out == "bf16":
        tol = tol + 2.0 ** -9 * base
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = np_(y[torch.from_numpy(rows).to(DEV)]).astype(np.float64)
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (bad[:4].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])], tol[tuple(bad[0])])


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N", [(2, 300), (40, 300), (300, 1500), (1024, 4100)])
def test_gemm_scales_whose_product_is_tiny(M, N, block_rows):
    """Scales' products on both sides of 2^-126.  Below it they are rounded to a
    multiple of 2^-149, off by at most 2^-150 times the block's sum; results
    below 2^-126 likewise by 2^-150 each of five additions."""
    rng = np.random.default_rng(M)
    K = 400
    a, b = rand_operand(rng, M, K), rand_operand(rng, N, K, block_rows)
    a = (a[0], (np.exp2(rng.integers(-75, -60, a[1].shape)) * 1.37).astype(np.float32))
    b = (b[0], (np.exp2(rng.integers(-75, -60, b[1].shape)) * 1.61).astype(np.float32))
    note(f"fp8 gemm tiny scales {M}x{N} block_rows {block_rows}")
    y = np_(nv.nvfp4_fp8_gemm(to_gpu(a), to_gpu(b), "f32")).astype(np.float64)
    ref, base = fp8_gemm_ref(*a, *b, block_rows)
    va, vb = np.abs(E4M3_TABLE[a[0]]), np.abs(E4M3_TABLE[b[0]])
    tol = (128 + 3 + 4) * 2.0 ** -24 * base + 2.0 ** -150 * (va @ vb.T) + 5 * 2.0 ** -150
    bad = np.argwhere(~(np.abs(y - ref) <= tol))
    assert bad.size == 0, (bad[:4].tolist(), y[tuple(bad[0])], ref[tuple(bad[0])], tol[tuple(bad[0])])


def test_gemm_empty():
    f8 = torch.float8_e4m3fn
    a = (torch.empty(4, 0, dtype=f8, device=DEV), torch.empty(0, 4, device=DEV))
    b = (torch.empty(40, 0, dtype=f8, device=DEV), torch.empty(0, 1, device=DEV))
    note("fp8 gemm K = 0")
    y = torch.full((4, 40), 3.0, device=DEV)
    assert bool((nv.nvfp4_fp8_gemm(a, b, "f32", y=y, accumulate=True) == 3.0).all())
    assert bool((nv.nvfp4_fp8_gemm(a, b, "f32", y=y) == 0).all())
    z = (torch.empty(0, 128, dtype=f8, device=DEV), torch.empty(1, 0, device=DEV))
    w = (torch.empty(8, 128, dtype=f8, device=DEV), torch.empty(1, 1, device=DEV))
    assert nv.nvfp4_fp8_gemm(z, w).shape == (0, 8)


def test_gemm_past_4_gib():
    """An activation operand past 2^32 bytes, and the same rows read through an
    index below 2^31; rows on both sides of the 2^31 and 2^32 byte offsets."""
    M, N, K = 300000, 72, 16384
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    for i in range(0, M, 50000):
        q[i:i + 50000] = torch.randint(0, 120, (50000, K), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.rand(K // 128, M, device=DEV, generator=g)
    b = rand_operand(np.random.default_rng(5), N, K, 128)
    note("fp8 gemm past 4 GiB")
    y = nv.nvfp4_fp8_gemm((q.view(torch.float8_e4m3fn), s), to_gpu(b), "bf16")
    rows = [0, 131071, 131072, 131073, 262143, 262144, 262145, M - 1]
    close(y[rows], (np_(q[rows]), np_(s[:, rows])), b, 128, "bf16")


GROUPS = [[5], [0, 3, 0, 40, 1], [16] * 9, [130, 0, 257, 64, 1], [1, 2] * 40, [0, 0, 700], [33, 64, 65, 0],
          [0] * 70 + [5] + [0] * 80 + [20], [1] * 130]


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: f"G{len(c)}t{sum(c)}")
@pytest.mark.parametrize("N,K", [(72, 144), (300, 512), (8, 16)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped(counts, N, K, gather, out):
    rng = np.random.default_rng(sum(counts) + N)
    off = wl.ragged_offsets(counts)
    total, G = int(off[-1]), len(counts)
    a_rows = 37 if gather else total
    a, b = rand_operand(rng, a_rows, K), rand_operand(rng, N, K, 128, (G,))
    idx = rng.integers(-1, a_rows + 1, total).astype(np.int32)       # -1 and a_rows: a row of zeros
    note(f"fp8 grouped {len(counts)} groups {total} rows N {N} K {K} gather {gather} {out}")
    y = np_(nv.nvfp4_fp8_grouped_gemm(off.to(DEV), total, to_gpu(a), to_gpu(b), out,
                                      row_index=torch.from_numpy(idx).to(DEV) if gather else None))
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        if gather:
            ok = (idx[lo:hi] >= 0) & (idx[lo:hi] < a_rows)
            q = np.where(ok[:, None], a[0][idx[lo:hi].clip(0, a_rows - 1)], 0)
            s = np.where(ok[None, :], a[1][:, idx[lo:hi].clip(0, a_rows - 1)], 0).astype(np.float32)
        else:
            q, s = a[0][lo:hi], a[1][:, lo:hi]
        close(torch.from_numpy(y[lo:hi]), (q, s), (b[0][e], b[1][e]), 128, out)


@pytest.mark.parametrize("counts,N,K", [
    ([20, 0, 64, 65, 1] * 9, 2056, 144), ([20, 0, 64, 65, 1] * 18, 1032, 1040), ([0, 400, 3, 130, 128, 250, 289, 100], 4104, 144),
    ([0, 1000, 300, 257, 1, 511, 700, 256, 900, 640, 5, 833, 720, 610, 512, 900], 4104, 144),
    ([1, 0, 3, 9, 2, 17, 0, 33], 1032, 1040), ([1, 0, 2, 1, 3], 2056, 1040), ([40, 3, 0, 33, 70], 520, 2064)],
    ids=lambda c: f"G{len(c)}t{sum(c)}" if isinstance(c, list) else str(c))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_many_tiles(counts, N, K, gather, out):
    """Rows and columns for every tile shape; each expert's edge rows and some
    more."""
    rng = np.random.default_rng(sum(counts))
    off = wl.ragged_offsets(counts)
    total, G = int(off[-1]), len(counts)
    a_rows = 1111 if gather else total
    a, b = rand_operand(rng, a_rows, K), rand_operand(rng, N, K, 128, (G,))
    idx = rng.integers(0, a_rows, total).astype(np.int32)
    note(f"fp8 grouped {G} groups {total} rows N {N} K {K} gather {gather} {out} (many tiles)")
    y = nv.nvfp4_fp8_grouped_gemm(off.to(DEV), total, to_gpu(a), to_gpu(b), out,
                                  row_index=torch.from_numpy(idx).to(DEV) if gather else None)
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        rows = np.unique(np.concatenate([[lo, hi - 1], rng.integers(lo, hi, 10)]))
        src = idx[rows] if gather else rows
        close(y[rows], (a[0][src], a[1][:, src]), (b[0][e], b[1][e]), 128, out)


@pytest.mark.parametrize("counts,N,K", [([1, 2, 0, 1] * 16, 4104, 2064), ([1, 2, 0, 1] * 4, 4104, 2064), ([3, 1] * 12, 2100, 144),
                                        ([30, 26, 0, 41] * 2, 2056, 144),
                                        ([30, 26, 0, 41] * 8, 2056, 400), ([2] * 40, 4104, 1040)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_by_number_of_workgroups(counts, N, K, gather, out):
    """Both sides of four workgroups a CU, and of two for each element of K."""
    test_grouped_many_tiles(counts, N, K, gather, out)


def test_grouped_leaves_rows_of_no_group():
    rng = np.random.default_rng(4)
    a, b = rand_operand(rng, 50, 128), rand_operand(rng, 40, 128, 128, (2,))
    off = torch.tensor([0, 7, 30], dtype=torch.int32)
    y = torch.full((50, 40), 5.0, device=DEV)
    note("fp8 grouped, rows behind the last group")
    nv.nvfp4_fp8_grouped_gemm(off.to(DEV), 50, to_gpu(a), to_gpu(b), "f32", y=y)
    assert bool((y[30:] == 5.0).all())
    for e, (lo, hi) in enumerate(((0, 7), (7, 30))):
        close(y[lo:hi], (a[0][lo:hi], a[1][:, lo:hi]), (b[0][e], b[1][e]), 128, "f32")


def test_grouped_stays_inside_on_bad_offsets():
    """Offsets that run backwards or past the rows: nothing outside y is
    touched and the call ends."""
    rng = np.random.default_rng(5)
    a, b = rand_operand(rng, 40, 128), rand_operand(rng, 24, 128, 128, (4,))
    off = torch.tensor([0, 30, 10, 9000, -5], dtype=torch.int32)
    buf = torch.full((60, 24), 2.0, device=DEV)
    note("fp8 grouped, inconsistent offsets")
    nv.nvfp4_fp8_grouped_gemm(off.to(DEV), 40, to_gpu(a), to_gpu(b), "f32", y=buf[10:50])
    torch.cuda.synchronize()
    assert bool((buf[:10] == 2.0).all()) and bool((buf[50:] == 2.0).all())


def test_grouped_many_groups_and_past_4_gib():
    """More groups than a wave has lanes, and expert weights past 2^32 bytes."""
    G, N, K = 150, 4096, 7168
    g = torch.Generator(device=DEV).manual_seed(6)
    q = torch.randint(0, 120, (G, N, K), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.rand(G, K // 128, N // 128, device=DEV, generator=g)
    counts = [0] * G
    counts[0], counts[70], counts[149] = 3, 20, 40
    off = wl.ragged_offsets(counts)
    a = rand_operand(np.random.default_rng(6), 63, K)
    note("fp8 grouped, weights past 4 GiB")
    y = nv.nvfp4_fp8_grouped_gemm(off.to(DEV), 63, to_gpu(a), (q.view(torch.float8_e4m3fn), s), "f32")
    for e, lo, hi in ((0, 0, 3), (70, 3, 23), (149, 23, 63)):
        close(y[lo:hi], (a[0][lo:hi], a[1][:, lo:hi]), (np_(q[e]), np_(s[e])), 128, "f32")


@pytest.mark.parametrize("counts", [[5], [0, 130, 0, 1, 256], [128, 128], [0, 0, 0], [300, 7] * 5],
                         ids=lambda c: f"G{len(c)}t{sum(c)}")
@pytest.mark.parametrize("N,K", [(48, 80), (144, 272), (16, 128)])
@pytest.mark.parametrize("out,add", [("f32", False), ("bf16", False), ("f32", True)])
def test_wgrad(counts, N, K, out, add):
    off = wl.ragged_offsets(counts)
    total, G = int(off[-1]), len(counts)
    dy, x = values(total, N, 1, "fp32"), values(total, K, 2, "bf16")
    note(f"fp8 wgrad {counts[:6]} N {N} K {K} {out} add {add}")
    a = nv.nvfp4_fp8_grouped_quantize(dy.to(DEV), off.to(DEV))
    b = nv.nvfp4_fp8_grouped_quantize(x.to(DEV), off.to(DEV))
    dw0 = torch.randn(G, N, K, generator=torch.Generator().manual_seed(3)) * 100 if add else None
    dw = np_(nv.nvfp4_fp8_grouped_wgrad(off.to(DEV), total, a, b, out,
                                        dw=dw0.to(DEV) if add else None, accumulate=add))
    aq, sa, bq, sb = bytes_of(a[0]), np_(a[1]), bytes_of(b[0]), np_(b[1])
    at = 0
    for e, c in enumerate(counts):
        n = -(-c // 128) * 128
        part = lambda q, s: (q[:, at:at + n], s[at // 128:(at + n) // 128])  # noqa: E731
        if c == 0:
            assert np.array_equal(dw[e], dw0[e].numpy() if add else np.zeros((N, K)))
        else:
            close(torch.from_numpy(dw[e]), part(aq, sa), part(bq, sb), 1, out,
                  add=dw0[e].double().numpy() if add else None)
        at += n


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_wgrad_many_tiles(out):
    counts, N, K = [300, 0, 129, 5], 2032, 2000
    off = wl.ragged_offsets(counts)
    total = int(off[-1])
    note(f"fp8 wgrad {counts} N {N} K {K} {out} (many tiles)")
    a = nv.nvfp4_fp8_grouped_quantize(values(total, N, 4, "fp32").to(DEV), off.to(DEV))
    b = nv.nvfp4_fp8_grouped_quantize(values(total, K, 5, "bf16").to(DEV), off.to(DEV))
    dw = nv.nvfp4_fp8_grouped_wgrad(off.to(DEV), total, a, b, out)
    aq, sa, bq, sb = bytes_of(a[0]), np_(a[1]), bytes_of(b[0]), np_(b[1])
    at = 0
    for e, c in enumerate(counts):
        n = -(-c // 128) * 128
        part = lambda q, s: (q[:, at:at + n], s[at // 128:(at + n) // 128])  # noqa: E731
        if c == 0:
            assert bool((dw[e] == 0).all())
        else:
            rows = np.arange(e, N, 37)
            close(dw[e], part(aq, sa), part(bq, sb), 1, out, rows=rows)
        at += n


# ---- streams, graphs --------------------------------------------------------

def test_side_stream_and_graph_replays():
    """Quantise -> product -> accumulate on a side stream, and captured and
    replayed with new inputs beside the program's own eager work."""
    M, N, K = 70, 260, 512
    xs = [values(M, K, 20 + i).to(DEV) for i in range(4)]
    w = nv.nvfp4_fp8_quantize(values(N, K, 30, spread=1).to(DEV), block_rows=128)
    eager = [nv.nvfp4_fp8_gemm(nv.nvfp4_fp8_quantize(x), w, "f32") for x in xs]
    side = torch.cuda.Stream()
    note("fp8 on a side stream")
    side.wait_stream(torch.cuda.current_stream())
    a = nv.nvfp4_fp8_quantize(xs[0], stream=side)
    y = nv.nvfp4_fp8_gemm(a, w, "f32", stream=side)
    side.synchronize()
    assert torch.equal(y, eager[0])
    xin = xs[0].clone()
    note("fp8 captured")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = nv.nvfp4_fp8_quantize(xin)
        yg = nv.nvfp4_fp8_gemm(q, w, "f32")
    for i in (1, 2, 3, 0, 2):
        xin.copy_(xs[i])
        graph.replay()
        again = nv.nvfp4_fp8_gemm(nv.nvfp4_fp8_quantize(xs[i]), w, "f32")
        torch.cuda.synchronize()
        assert torch.equal(yg, eager[i]) and torch.equal(again, eager[i])


def test_results_do_not_change_between_calls():
    off = wl.ragged_offsets([40, 0, 200, 3])
    rng = np.random.default_rng(8)
    a, b = to_gpu(rand_operand(rng, 243, 272)), to_gpu(rand_operand(rng, 144, 272, 128, (4,)))
    note("fp8 grouped twice")
    one = nv.nvfp4_fp8_grouped_gemm(off.to(DEV), 243, a, b, "f32")
    two = nv.nvfp4_fp8_grouped_gemm(off.to(DEV), 243, a, b, "f32")
    assert torch.equal(one, two)


def test_wrappers_refuse_operands_that_do_not_fit():
    a = nv.nvfp4_fp8_quantize(values(4, 256, 1).to(DEV))
    w = nv.nvfp4_fp8_quantize(values(300, 256, 2).to(DEV), block_rows=128)
    other = nv.nvfp4_fp8_quantize(values(4, 128, 1).to(DEV))
    y = torch.empty(4, 300, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: nv.nvfp4_fp8_gemm(other, w), lambda: nv.nvfp4_fp8_gemm(w, a),
                 lambda: nv.nvfp4_fp8_gemm(a, w, "f16"), lambda: nv.nvfp4_fp8_gemm(a, w, "f32", y=y),
                 lambda: nv.nvfp4_fp8_gemm(a, w, "bf16", y=y, accumulate=True),
                 lambda: nv.nvfp4_fp8_gemm(a, w, y=y[:, :299]),
                 lambda: nv.nvfp4_fp8_gemm(a, w, "f32", accumulate=True),
                 lambda: nv.nvfp4_fp8_quantize(torch.empty(4, 24, device=DEV)),
                 lambda: nv.nvfp4_fp8_quantize(torch.empty(4, 32, device=DEV), layout="up")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_fp8_quantize(torch.empty(4, 34, device=DEV)[:, 2:])   # rows 8 bytes off a 16-byte border
