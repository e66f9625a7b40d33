"""INT8 operands and products on the GPU against the oracle, bit for bit: the
quantiser's integers and scales, and products whose sums are exact."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv
from oracle import int8_gemm_ref, int8_quantize_ref
from tests.gpu_util import need_gpu, note, np_

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def values(rows, cols, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def same(op, ref):
    q, s = np_(op[0]), np_(op[1])
    assert np.array_equal(s, ref[1], equal_nan=True), np.argwhere(s != ref[1])[:4]
    assert np.array_equal(q, ref[0]), np.argwhere(q != ref[0])[:4]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 512), (3, 528), (7, 1024), (9, 1040), (64, 2048), (6, 2064),
                                       (2, 4096), (3, 4112), (5, 8192), (2, 8208), (1, 32768), (2, 32784),
                                       (3, 100000), (1030, 64)])
def test_quantize(dtype, rows, cols):
    x = values(rows, cols, rows + cols, dtype)
    note(f"int8 quantize {dtype} {rows}x{cols}")
    same(nv.nvfp4_int8_quantize(x.to(DEV)), int8_quantize_ref(x.float().numpy()))


@pytest.mark.parametrize("cols", [64, 4096, 40000])
def test_quantize_special_rows(cols):
    x = torch.zeros(9, cols)
    x[1, cols - 1], x[2, 5], x[3, 0] = float("nan"), float("inf"), -float("inf")
    x[4, 7], x[5], x[6, ::2], x[7, 3] = 1e-40, 3e38, -0.0, -2.0 ** -120
    # ties: 127 of the largest, so that x * r is a whole number and a half
    x[8, :8] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5])
    note(f"int8 quantize special rows {cols}")
    ref = int8_quantize_ref(x.numpy())
    assert ref[0][8, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, 126]
    same(nv.nvfp4_int8_quantize(x.to(DEV)), ref)


def test_quantize_strides_out_and_empty():
    wide = values(50, 512, 9, "bf16")
    part = wide[:, 64:64 + 160]
    out = (torch.full((50, 160), 99, dtype=torch.int8, device=DEV), torch.zeros(50, device=DEV))
    note("int8 quantize strided rows into given buffers")
    got = nv.nvfp4_int8_quantize(wide.to(DEV)[:, 64:64 + 160], out=out)
    assert got[0] is out[0]
    same(got, int8_quantize_ref(part.float().numpy()))
    assert nv.nvfp4_int8_quantize(torch.empty(0, 64, device=DEV))[0].shape == (0, 64)
    with pytest.raises(ValueError):
        nv.nvfp4_int8_quantize(wide.to(DEV)[:, 64:64 + 160], out=(out[0][:40], out[1][:40]))
    with pytest.raises(ValueError):
        nv.nvfp4_int8_quantize(wide.to(DEV).t())
    with pytest.raises(nv.Nvfp4Error):                         # rows off a 16-byte border
        nv.nvfp4_int8_quantize(wide.to(DEV)[:, 1:33])


def operand(rng, rows, K):
    return (rng.integers(-128, 128, (rows, K)).astype(np.int8),
            np.exp2(rng.uniform(-10, 2, rows)).astype(np.float32))


def gpu(op):
    return torch.from_numpy(op[0]).to(DEV), torch.from_numpy(op[1]).to(DEV)


def check(a, b, out, rows=None, **kw):
    y = nv.nvfp4_int8_gemm(gpu(a), gpu(b), out, **kw)
    got = np_(y if rows is None else y[torch.from_numpy(rows).to(DEV)])
    ref = int8_gemm_ref(a[0] if rows is None else a[0][rows], a[1] if rows is None else a[1][rows], *b)
    if out == "bf16":
        ref = torch.from_numpy(ref).to(torch.bfloat16).float().numpy()
    assert np.array_equal(got, ref, equal_nan=True), np.argwhere(got != ref)[:4]
    return y


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 300, 128), (2, 17, 144), (3, 256, 6144), (4, 133, 8208), (5, 72, 6160),
                                   (8, 4100, 272), (9, 5000, 272), (16, 8200, 144), (17, 200, 512), (33, 1000, 640),
                                   (48, 64, 8192), (64, 96, 272), (65, 129, 1040), (128, 128, 128), (130, 4100, 256),
                                   (200, 333, 1552), (257, 640, 112), (70, 8300, 2064), (600, 1000, 1040),
                                   (1000, 520, 8192), (90, 16400, 144), (512, 4104, 272), (16, 7, 131056)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm(M, N, K, out):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    note(f"int8 gemm {M}x{N}x{K} {out}")
    check(operand(rng, M, K), operand(rng, N, K), out)


@pytest.mark.parametrize("M,N,K", [(1024, 1100, 384), (1000, 8200, 144), (2500, 4200, 144), (4096, 4096, 128),
                                   (2500, 8200, 272), (4100, 8200, 400)])
def test_gemm_many_tiles(M, N, K):
    """Enough tiles for the large tile shapes, ragged edges; sampled rows."""
    rng = np.random.default_rng(M + N + K)
    rows = np.unique(np.concatenate([[0, 127, 128, 255, 256, M - 1], rng.choice(M, 40, replace=False)]))
    note(f"int8 gemm {M}x{N}x{K} (many tiles)")
    check(operand(rng, M, K), operand(rng, N, K), "bf16", rows=rows)


@pytest.mark.parametrize("M,N", [(3, 40), (40, 1500), (300, 300), (1024, 4100)])
def test_gemm_largest_sums(M, N):
    """All -128 at the longest K: sums of 2147221504, the largest there are."""
    K = 131056 if M < 1024 else 2048
    a = (np.full((M, K), -128, np.int8), np.ones(M, np.float32))
    b = (np.full((N, K), -128, np.int8), np.ones(N, np.float32))
    b[0][N // 2] = 127
    note(f"int8 gemm largest sums {M}x{N}x{K}")
    y = nv.nvfp4_int8_gemm(gpu(a), gpu(b), "f32")
    want = torch.full((N,), 16384.0 * K)
    want[N // 2] = -128.0 * 127 * K
    assert torch.equal(y.cpu(), want.float().expand(M, N))


@pytest.mark.parametrize("M", [2, 40, 300])
def test_gemm_strided_outputs_and_nan_scales(M):
    rng = np.random.default_rng(M)
    N, K = 333, 272
    a, b = operand(rng, M, K), operand(rng, N, K)
    a[1][1], b[1][7] = np.nan, np.nan
    for dt, name in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        for lead in (0, 1):
            wide = torch.full((M, N + 13), 5.0, dtype=dt, device=DEV)
            note(f"int8 gemm strided {name} M {M} lead {lead}")
            y = check(a, b, name, y=wide[:, lead:lead + N])
            assert y.data_ptr() == wide[:, lead:].data_ptr()
            assert (wide[:, lead + N:] == 5).all() and (wide[:, :lead] == 5).all()


def test_gemm_empty_and_refusals():
    rng = np.random.default_rng(0)
    a, b = operand(rng, 4, 64), operand(rng, 6, 64)
    e = (torch.zeros(0, 64, dtype=torch.int8, device=DEV), torch.zeros(0, device=DEV))
    z = (torch.zeros(4, 0, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV))
    note("int8 gemm empty")
    assert nv.nvfp4_int8_gemm(e, gpu(b)).shape == (0, 6) and nv.nvfp4_int8_gemm(gpu(a), e).shape == (4, 0)
    assert (nv.nvfp4_int8_gemm(z, z, "f32") == 0).all()
    q = nv.nvfp4_int8_quantize(torch.zeros(4, 0, device=DEV))
    same(q, int8_quantize_ref(np.zeros((4, 0), np.float32)))
    assert (nv.nvfp4_int8_gemm(q, q, "f32") == 0).all()
    with pytest.raises(ValueError):
        nv.nvfp4_int8_gemm(gpu(a), gpu(operand(rng, 6, 80)))
    with pytest.raises(ValueError):
        nv.nvfp4_int8_gemm(gpu(a), gpu(b), "f16")
    with pytest.raises(ValueError):
        nv.nvfp4_int8_gemm(gpu(a), gpu(b), y=torch.empty(4, 5, dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("M", [1, 20, 200])
def test_a_linear_layer_captured_and_replayed(M):
    """Quantise and multiply on a side stream and in a graph, eager work between
    the replays."""
    K, N = 1040, 720
    g = torch.Generator().manual_seed(M)
    w = nv.nvfp4_int8_quantize(torch.randn(N, K, generator=g).to(DEV))
    xs = [torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV) for _ in range(4)]

    def layer(x, stream=None):
        return nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(x, stream=stream), w, "f32", stream=stream)
    note(f"int8 layer graph M {M}")
    eager = [layer(x) for x in xs]
    ref = int8_gemm_ref(*int8_quantize_ref(np_(xs[1])), np_(w[0]), np_(w[1]))
    assert np.array_equal(np_(eager[1]), ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    on_side = layer(xs[2], stream=side)
    side.synchronize()
    assert torch.equal(on_side, eager[2])
    xin = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(xin)
    for i in (1, 2, 3, 0, 2):
        xin.copy_(xs[i])
        graph.replay()
        again = layer(xs[i])
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i]) and torch.equal(again, eager[i])


def test_far_rows():
    """Operands and outputs past 2^31 elements; sampled rows."""
    M, K, N = 70000, 32768, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    rng = np.random.default_rng(0)
    b = operand(rng, N, K)
    rows = torch.tensor([0, 32767, 65535, 65536, 69999], device=DEV)
    note(f"int8 far rows {M}x{K}")
    q = nv.nvfp4_int8_quantize(x)
    ref = int8_quantize_ref(np_(x[rows]))
    same((q[0][rows], q[1][rows]), ref)
    y = nv.nvfp4_int8_gemm(q, gpu(b), "f32")
    assert np.array_equal(np_(y[rows]), int8_gemm_ref(*ref, *b))
    del x, y
    a = (q[0][:1024, :16].contiguous(), q[1][:1024])
    w = (q[0].view(-1, 16)[:2200000].contiguous(), torch.ones(2200000, device=DEV))
    note("int8 outputs past 2^31 elements")
    y = nv.nvfp4_int8_gemm(a, w, "bf16")
    part = nv.nvfp4_int8_gemm((a[0][1000:], a[1][1000:]), (w[0][-100:].contiguous(), w[1][-100:]), "bf16")
    assert torch.equal(y[1000:, -100:], part)
