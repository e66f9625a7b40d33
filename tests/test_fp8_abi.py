"""Argument checks of the FP8 and router entry points (no GPU: every call here
is refused, or has nothing to do, before anything is enqueued)."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv

P = ctypes.c_void_p(0x10000)
P8 = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)
INV, UNS, OK = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED, nv.NVFP4_OK


def _call(name, defaults, kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(nv.load(), name)(*args.values(), None)


QUANT = dict(x=P, x_dtype=nv.NVFP4_BF16, batch=1, rows=4, cols=32, ld_x=32, block_rows=1, q=P, s=P,
             qt=None, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(cols=24, ld_x=24), INV), (dict(rows=-1), INV), (dict(batch=-1), INV), (dict(x_dtype=2), INV),
    (dict(block_rows=64), INV), (dict(block_rows=0), INV), (dict(ld_x=16), INV), (dict(x=None), INV),
    (dict(q=None), INV), (dict(s=None), INV), (dict(q=None, s=None), INV), (dict(qt=P), INV),
    (dict(st=P), INV), (dict(x=P8), UNS), (dict(ld_x=36), UNS), (dict(q=P8), UNS), (dict(s=ODD), UNS),
    (dict(qt=P8, st=P), UNS), (dict(rows=1 << 31), UNS), (dict(rows=0), OK), (dict(batch=0), OK),
    (dict(cols=0, ld_x=0), OK),
])
def test_quantize_checks(kw, status):
    assert _call("nvfp4_fp8_quantize", QUANT, kw) == status


GQUANT = dict(x=P, x_dtype=nv.NVFP4_F32, G=3, m_offsets=P, row_index=None, total_m=8, x_rows=8, cols=32,
              ld_x=32, q=None, s=None, qt=P, st=P)


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), INV), (dict(G=0), INV), (dict(m_offsets=None), INV), (dict(row_index=P, x_rows=-1), INV),
    (dict(cols=40), INV), (dict(qt=None), INV), (dict(qt=None, st=None), INV), (dict(x=P8), UNS),
    (dict(row_index=P, x_rows=1 << 31), UNS), (dict(total_m=0), OK), (dict(G=0, total_m=0), OK),
])
def test_grouped_quantize_checks(kw, status):
    assert _call("nvfp4_fp8_grouped_quantize", GQUANT, kw) == status


@pytest.mark.parametrize("total,G,want", [(0, 4, 0), (5, 0, 0), (1, 4, 128), (128, 1, 128), (129, 1, 256),
                                          (3, 100, 384), (4096, 64, 12160)])
def test_grouped_columns(total, G, want):
    assert nv.nvfp4_fp8_grouped_columns(total, G) == want


def test_grouped_columns_hold_every_split():
    for total in (1, 2, 127, 128, 300):
        for G in (1, 2, 5):
            worst = max(sum(-(-c // 128) * 128 for c in split)
                        for split in _splits(total, min(G, 3), step=max(1, total // 7)))
            assert worst <= nv.nvfp4_fp8_grouped_columns(total, G)


def _splits(total, G, step):
    if G == 1:
        return [(total,)]
    return [(c, *rest) for c in list(range(0, total + 1, step)) + [total]
            for rest in _splits(total - c, G - 1, step)]


GEMM = dict(M=8, N=8, K=128, a_q=P, a_s=P, b_q=P, b_s=P, b_block_rows=128, y=P, y_dtype=nv.NVFP4_F32,
            ld_y=8, flags=0)


@pytest.mark.parametrize("kw,status", [
    (dict(K=24), INV), (dict(M=-1), INV), (dict(N=-1), INV), (dict(b_block_rows=2), INV), (dict(ld_y=7), INV),
    (dict(y_dtype=3), INV), (dict(flags=2), INV), (dict(flags=1, y_dtype=nv.NVFP4_BF16), INV),
    (dict(y=None), INV), (dict(a_q=None), INV), (dict(a_s=None), INV), (dict(b_q=None), INV),
    (dict(b_s=None), INV), (dict(a_q=P8), UNS), (dict(b_q=P8), UNS), (dict(a_s=ODD), UNS),
    (dict(y=ODD), UNS), (dict(K=(1 << 22) + 16), UNS), (dict(M=1 << 31), UNS), (dict(M=0), OK),
    (dict(N=0, ld_y=0), OK),
])
def test_gemm_checks(kw, status):
    assert _call("nvfp4_fp8_gemm", GEMM, kw) == status


GROUPED = dict(G=4, m_offsets=P, row_index=None, total_m=8, a_rows=0, N=8, K=128, a_q=P, a_s=P, b_q=P, b_s=P,
               y=P, y_dtype=nv.NVFP4_BF16, ld_y=8)


@pytest.mark.parametrize("kw,status", [
    (dict(K=40), INV), (dict(G=-1), INV), (dict(G=0), INV), (dict(total_m=-1), INV), (dict(a_rows=-1), INV),
    (dict(a_rows=7), INV), (dict(m_offsets=None), INV), (dict(ld_y=4), INV), (dict(b_q=None), INV),
    (dict(y_dtype=9), INV), (dict(a_q=P8), UNS), (dict(row_index=P, a_rows=1 << 24), UNS),
    (dict(N=1 << 31), UNS), (dict(total_m=0), OK), (dict(G=0, total_m=0), OK), (dict(N=0, ld_y=0), OK),
])
def test_grouped_checks(kw, status):
    assert _call("nvfp4_fp8_grouped_gemm", GROUPED, kw) == status


def test_the_walk_over_groups_ends():
    """The kernels take 64 groups at a time and count them in 32 bits: past 2^31 - 65 the
    count would turn negative before it reaches the end."""
    for G in ((1 << 31) - 64, (1 << 31) - 1):
        assert _call("nvfp4_fp8_grouped_gemm", GROUPED, dict(G=G)) == UNS
        assert _call("nvfp4_fp8_grouped_gemm", GROUPED, dict(G=G, N=1 << 20, ld_y=1 << 20)) == UNS
        assert _call("nvfp4_fp8_grouped_quantize", GQUANT, dict(G=G)) == UNS
    assert _call("nvfp4_fp8_grouped_gemm", GROUPED, dict(G=(1 << 31) - 65, total_m=0)) == OK


WGRAD = dict(G=4, m_offsets=P, total_m=8, N=8, K=8, a_q=P, a_s=P, b_q=P, b_s=P, dw=P, dw_dtype=nv.NVFP4_F32,
             flags=0)


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), INV), (dict(G=0), INV), (dict(N=-1), INV), (dict(K=-1), INV), (dict(m_offsets=None), INV),
    (dict(dw=None), INV), (dict(b_s=None), INV), (dict(flags=1, dw_dtype=nv.NVFP4_BF16), INV),
    (dict(flags=4), INV), (dict(a_q=P8), UNS), (dict(total_m=1 << 23), UNS), (dict(N=0), OK), (dict(K=0), OK),
    (dict(G=0, total_m=0), OK),
])
def test_wgrad_checks(kw, status):
    assert _call("nvfp4_fp8_grouped_wgrad", WGRAD, kw) == status


@pytest.mark.parametrize("name,defaults,kw", [
    ("nvfp4_fp8_quantize", QUANT, dict(batch=1 << 24, rows=1, cols=16, ld_x=16, block_rows=128)),
    ("nvfp4_fp8_quantize", QUANT, dict(rows=1 << 30, cols=1 << 20, ld_x=1 << 20)),
    ("nvfp4_fp8_quantize", QUANT, dict(batch=1 << 30, rows=1 << 30, cols=1 << 30, ld_x=1 << 30)),
    ("nvfp4_fp8_grouped_quantize", GQUANT, dict(total_m=1 << 30, x_rows=1 << 30, cols=1 << 14, ld_x=1 << 14)),
    ("nvfp4_fp8_gemm", GEMM, dict(M=1, N=1 << 28, K=16, ld_y=1 << 28)),
    ("nvfp4_fp8_gemm", GEMM, dict(M=2, N=1 << 27, K=4096, ld_y=1 << 27)),
    ("nvfp4_fp8_gemm", GEMM, dict(M=1 << 30, N=16, K=16, ld_y=16, y_dtype=nv.NVFP4_BF16)),
    ("nvfp4_fp8_grouped_gemm", GROUPED, dict(G=4, total_m=32, N=48 << 20, K=1 << 22, ld_y=48 << 20)),
    ("nvfp4_fp8_grouped_wgrad", WGRAD, dict(G=1 << 25, N=16, K=16)),
    ("nvfp4_fp8_grouped_wgrad", WGRAD, dict(G=1 << 30, N=1 << 30, K=1 << 30, dw_dtype=nv.NVFP4_BF16)),
])
def test_launches_past_a_grid_are_refused(name, defaults, kw):
    assert _call(name, defaults, kw) == UNS


ROUTE = dict(T=8, E=16, topk=2, logits=P, dtype=nv.NVFP4_F32, ld=16, mask=None, flags=0, expert_index=P,
             weights=P, counts=P, m_offsets=P, row_index=P, pair_row=P, routed=P, loss=P, workspace=P,
             workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(E=0), INV), (dict(topk=0), INV), (dict(topk=17), INV), (dict(dtype=7), INV),
    (dict(flags=2), INV), (dict(ld=15), INV), (dict(logits=None), INV), (dict(counts=None), INV),
    (dict(loss=None), INV), (dict(workspace=None), INV), (dict(workspace_bytes=16), INV),
    (dict(pair_row=None), INV), (dict(E=1025, ld=1025), UNS), (dict(E=64, ld=64, topk=17), UNS),
    (dict(T=1 << 30, topk=2), UNS), (dict(logits=ODD), UNS), (dict(weights=ODD), UNS),
])
def test_route_checks(kw, status):
    assert _call("nvfp4_moe_route", ROUTE, kw) == status


BACK = dict(T=8, E=16, topk=2, logits=P, dtype=nv.NVFP4_F32, ld=16, mask=None, flags=0, expert_index=P,
            counts=P, routed=P, d_weights=P, d_loss=P, d_logits=P, ld_d=16)


@pytest.mark.parametrize("kw,status", [
    (dict(topk=17), INV), (dict(ld=1), INV), (dict(ld_d=15), INV), (dict(expert_index=None), INV),
    (dict(counts=None), INV), (dict(routed=None), INV), (dict(d_logits=None), INV), (dict(flags=8), INV),
    (dict(d_weights=ODD), UNS), (dict(d_logits=ODD), UNS), (dict(E=2000, ld=2000, ld_d=2000), UNS),
    (dict(T=0), OK),
])
def test_route_backward_checks(kw, status):
    assert _call("nvfp4_moe_route_backward", BACK, kw) == status


def test_route_workspace():
    assert nv.nvfp4_moe_route_workspace_bytes(-1, 8) == 0
    assert nv.nvfp4_moe_route_workspace_bytes(0, 8) > 0
    assert nv.nvfp4_moe_route_workspace_bytes(1 << 20, 256) >= nv.nvfp4_moe_route_workspace_bytes(16, 256)


def test_wrappers_refuse_before_the_library():
    x = torch.zeros(4, 32)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: nv.nvfp4_fp8_quantize(x), lambda: nv.nvfp4_fp8_grouped_quantize(x, off),
                 lambda: nv.nvfp4_moe_route(x, 2), lambda: nv.nvfp4_fp8_quantize(x.half()),
                 lambda: nv.Fp8Packed((x.to(torch.float8_e4m3fn), torch.zeros(1, 4))),
                 lambda: nv.Fp8Packed((x, torch.zeros(1, 4))),
                 lambda: nv.Fp8Packed((x.to(torch.float8_e4m3fn), torch.zeros(2, 4)))):
        with pytest.raises(ValueError):
            call()
