"""Argument checks of the gated blocks, the INT8 operands and gradient clipping
(no GPU: every call here is refused, or has nothing to do, before anything is
enqueued)."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_gemm_amd as nv

P = ctypes.c_void_p(0x10000)
P8 = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)
BYTE = ctypes.c_void_p(0x10001)
INV, UNS, OK = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED, nv.NVFP4_OK
BF, F32 = nv.NVFP4_BF16, nv.NVFP4_F32


def _call(name, defaults, kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(nv.load(), name)(*args.values(), None)


GATED = dict(M=8, F=24, K=128, a_q=P, a_s=P, w_q=P, w_s=P, w_block_rows=128, act=0, h=P, h_dtype=BF, ld_h=24,
             gate_up=P, ld_gate_up=48)


@pytest.mark.parametrize("kw,status", [
    (dict(K=24), INV), (dict(M=-1), INV), (dict(F=-1), INV), (dict(w_block_rows=2), INV), (dict(act=2), INV),
    (dict(act=-1), INV), (dict(h_dtype=2), INV), (dict(h=None), INV), (dict(ld_h=23), INV),
    (dict(ld_gate_up=47), INV), (dict(a_q=None), INV), (dict(a_s=None), INV), (dict(w_q=None), INV),
    (dict(w_s=None), INV), (dict(a_q=P8), UNS), (dict(w_q=P8), UNS), (dict(w_s=ODD), UNS), (dict(h=BYTE), UNS),
    (dict(h=ODD, h_dtype=F32), UNS), (dict(gate_up=BYTE), UNS), (dict(K=(1 << 22) + 16), UNS),
    (dict(F=(1 << 27) + 1, ld_h=1 << 28, ld_gate_up=1 << 29), UNS), (dict(M=1 << 31), UNS),
    (dict(M=1 << 30, F=1 << 27, ld_h=1 << 27, ld_gate_up=1 << 28), UNS),
    (dict(M=0), OK), (dict(F=0), OK),
])
def test_gated_checks(kw, status):
    assert _call("nvfp4_fp8_gated_gemm", GATED, kw) == status


GGATED = dict(G=3, m_offsets=P, row_index=None, total_m=8, a_rows=8, F=24, K=128, a_q=P, a_s=P, w_q=P, w_s=P, act=1,
              h=P, h_dtype=BF, ld_h=24, gate_up=None, ld_gate_up=0)


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), INV), (dict(G=0), INV), (dict(m_offsets=None), INV), (dict(a_rows=7), INV), (dict(a_rows=-1), INV),
    (dict(K=8), INV), (dict(act=3), INV), (dict(ld_h=8), INV), (dict(gate_up=P, ld_gate_up=24), INV),
    (dict(row_index=P, a_rows=1 << 25), UNS), (dict(w_q=ODD), UNS), (dict(F=(1 << 27) + 16, ld_h=1 << 28), UNS),
    (dict(total_m=0, a_rows=0), OK), (dict(F=0), OK), (dict(G=0, total_m=0, a_rows=0), OK),
])
def test_grouped_gated_checks(kw, status):
    assert _call("nvfp4_fp8_grouped_gated_gemm", GGATED, kw) == status


BACK = dict(dh=P, dh_dtype=BF, ld_dh=24, gate_up=P, gate_up_dtype=BF, ld_gate_up=48, act=0, rows=8, F=24, q=P, s=P,
            qt=P, st=P)


@pytest.mark.parametrize("kw,status", [
    (dict(F=12), INV), (dict(F=-8), INV), (dict(rows=-1), INV), (dict(dh_dtype=2), INV), (dict(gate_up_dtype=-1), INV),
    (dict(act=2), INV), (dict(ld_dh=16), INV), (dict(ld_gate_up=40), INV), (dict(dh=None), INV),
    (dict(gate_up=None), INV), (dict(q=None), INV), (dict(st=None), INV), (dict(q=None, s=None, qt=None, st=None), INV),
    (dict(dh=P8), UNS), (dict(gate_up=P8), UNS), (dict(ld_dh=28), UNS), (dict(ld_gate_up=52), UNS), (dict(q=P8), UNS),
    (dict(qt=P8), UNS), (dict(s=ODD), UNS), (dict(rows=1 << 31), UNS),
    (dict(F=1 << 28, ld_dh=1 << 28, ld_gate_up=1 << 29), UNS),
    (dict(rows=1 << 30, F=1 << 27, ld_dh=1 << 27, ld_gate_up=1 << 28), UNS),
    (dict(rows=0), OK), (dict(F=0), OK),
])
def test_backward_checks(kw, status):
    assert _call("nvfp4_fp8_gated_backward", BACK, kw) == status
    grouped = dict(G=2, m_offsets=P, **BACK)
    assert _call("nvfp4_fp8_grouped_gated_backward", {("total_m" if k == "rows" else k): v for k, v in grouped.items()},
                 {("total_m" if k == "rows" else k): v for k, v in kw.items()}) == status


def test_grouped_backward_needs_groups():
    grouped = dict(G=2, m_offsets=P, **BACK)
    for kw, status in ((dict(G=0), INV), (dict(G=-1), INV), (dict(m_offsets=None), INV), (dict(G=0, rows=0), OK)):
        assert _call("nvfp4_fp8_grouped_gated_backward", grouped, kw) == status


def test_gated_calls_of_too_many_groups():
    """Experts are counted in 32 bits, an expert's rows of its weight twice over."""
    many = (1 << 30) + 1
    assert _call("nvfp4_fp8_grouped_gated_gemm", GGATED, dict(G=many)) == UNS
    assert _call("nvfp4_fp8_grouped_gated_gemm", GGATED, dict(G=many, row_index=P)) == UNS
    assert _call("nvfp4_fp8_grouped_gated_backward", dict(G=2, m_offsets=P, **BACK), dict(G=many)) == UNS
    for kw in (dict(G=many, total_m=0, a_rows=0), dict(G=many, F=0)):
        assert _call("nvfp4_fp8_grouped_gated_gemm", GGATED, kw) == UNS


QUANT = dict(x=P, x_dtype=BF, rows=4, cols=32, ld_x=32, q=P, s=P)


@pytest.mark.parametrize("kw,status", [
    (dict(cols=24, ld_x=24), INV), (dict(rows=-1), INV), (dict(x_dtype=2), INV), (dict(ld_x=16), INV),
    (dict(x=None), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(q=None, s=None), INV), (dict(x=P8), UNS),
    (dict(ld_x=36), UNS), (dict(q=P8), UNS), (dict(s=ODD), UNS), (dict(rows=1 << 31), UNS),
    (dict(rows=1 << 30, cols=65536, ld_x=65536), UNS), (dict(rows=0), OK),
    (dict(rows=0, x=None, q=None, s=None), OK), (dict(cols=0, ld_x=0, s=None), INV),
])
def test_int8_quantize_checks(kw, status):
    assert _call("nvfp4_int8_quantize", QUANT, kw) == status


INT8 = dict(M=8, N=8, K=128, a_q=P, a_s=P, b_q=P, b_s=P, y=P, y_dtype=F32, ld_y=8)


@pytest.mark.parametrize("kw,status", [
    (dict(K=24), INV), (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-16), INV), (dict(y_dtype=2), INV),
    (dict(ld_y=7), INV), (dict(y=None), INV), (dict(a_q=None), INV), (dict(a_s=None), INV), (dict(b_q=None), INV),
    (dict(b_s=None), INV), (dict(K=0, a_s=None), INV), (dict(a_q=P8), UNS), (dict(b_q=P8), UNS), (dict(a_s=ODD), UNS),
    (dict(b_s=ODD), UNS), (dict(y=ODD), UNS), (dict(K=1 << 17), UNS), (dict(M=1 << 31), UNS), (dict(N=1 << 31), UNS),
    (dict(M=1 << 30, N=1 << 30, ld_y=1 << 30), UNS), (dict(M=0), OK), (dict(N=0), OK),
])
def test_int8_gemm_checks(kw, status):
    assert _call("nvfp4_int8_gemm", INT8, kw) == status


def _grads(*rows):
    return (nv.Grad * max(len(rows), 1))(*[nv.Grad(*r) for r in rows])


ONE = (0x10000, 0, 16, F32, F32)


@pytest.mark.parametrize("grads,kw,status", [
    ([ONE], dict(count=-1), INV), ([ONE], dict(grads=None), INV), ([ONE], dict(norm_sq=None), INV),
    ([ONE], dict(workspace=None), INV), ([ONE], dict(workspace_bytes=8), INV), ([ONE], dict(workspace=ODD), UNS),
    ([ONE], dict(norm_sq=ctypes.c_void_p(0x10004)), UNS), ([(0, 0, 16, F32, F32)], {}, INV),
    ([(0x10000, 0, -1, F32, F32)], {}, INV), ([(0x10000, 0, 16, 2, F32)], {}, INV),
    ([(0x10002, 0, 16, F32, F32)], {}, UNS), ([(0x10001, 0, 16, BF, F32)], {}, UNS),
    ([(0x10000, 0, (1 << 42) + 1, F32, F32)], {}, UNS),
    ([(0x10000, 0, 1 << 41, BF, BF), (0x10000, 0, (1 << 41) + 1, BF, BF)], {}, UNS),
    ([ONE], dict(count=(1 << 20) + 1), UNS),
])
def test_norm_checks(grads, kw, status):
    arr = _grads(*grads)
    args = dict(count=len(grads), grads=ctypes.addressof(arr), norm_sq=P, workspace=P, workspace_bytes=1 << 20)
    assert _call("nvfp4_grad_norm_sq", args, kw) == status


A, B = 0x10000, 0x20000


@pytest.mark.parametrize("grads,kw,status", [
    ([ONE], dict(max_norm=-1.0), INV), ([ONE], dict(max_norm=float("nan")), INV), ([ONE], dict(count=-1), INV),
    ([ONE], dict(workspace=None), INV), ([ONE], dict(norm=ODD), UNS), ([ONE], dict(norm_sq=ODD), UNS),
    ([(A, 0, 16, F32, BF)], {}, INV),                            # in place keeps its type
    ([(A, A, 16, F32, BF)], {}, INV), ([(A, B, 16, F32, 2)], {}, INV), ([(A, B + 2, 16, F32, F32)], {}, UNS),
    ([(A, 0, 16, F32, F32), (A, 0, 16, F32, F32)], {}, INV),     # the same gradient twice
    ([(A, 0, 16, F32, F32), (A + 60, 0, 16, F32, F32)], {}, INV),
    ([(A + 60, 0, 16, F32, F32), (A, 0, 16, F32, F32)], {}, INV),
    ([(A, A + 32, 16, F32, F32)], {}, INV),                      # moved over itself
    ([(A, B, 16, F32, F32), (B + 4, 0x30000, 4, F32, F32)], {}, INV),
    ([(A, B, 16, F32, BF), (A + 64, B + 16, 4, F32, F32)], {}, INV),
    ([(A, 0, 1 << 12, F32, F32), (A + 256, B, 4, F32, F32)], {}, INV),
])
def test_clip_checks(grads, kw, status):
    arr = _grads(*grads)
    args = dict(count=len(grads), grads=ctypes.addressof(arr), max_norm=1.0, norm_sq=None, norm=P, workspace=P,
                workspace_bytes=1 << 20)
    assert _call("nvfp4_clip_grads", args, kw) == status


@pytest.mark.parametrize("empty", [(0, 0, 0, F32, BF), (0, 0, 0, BF, F32), (A, 0, 0, F32, BF), (A, A, 0, BF, F32)])
def test_clip_checks_of_empty_tensors(empty):
    """A tensor without elements has no place and so is not in place: the call passes
    the list's checks and is refused for what is looked at after them."""
    arr = _grads((A, B, 16, F32, BF), empty)
    args = dict(count=2, grads=ctypes.addressof(arr), max_norm=1.0, norm_sq=None, norm=ODD, workspace=P,
                workspace_bytes=1 << 20)
    assert _call("nvfp4_clip_grads", args, {}) == UNS
    arr[1].out_dtype = 2
    assert _call("nvfp4_clip_grads", args, {}) == INV


FAR = ctypes.c_void_p(0x800000)


def _at(address):
    return ctypes.c_void_p(address)


@pytest.mark.parametrize("grads,kw", [
    ([(A, 0, 16, F32, F32)], dict(norm=_at(A + 60))), ([(A, B, 16, F32, F32)], dict(norm=_at(A))),
    ([(A, B, 16, F32, BF)], dict(norm=_at(B + 28))),
    ([(A, 0, 16, F32, F32)], dict(workspace=_at(A + 56))), ([(A, B, 16, F32, F32)], dict(workspace=_at(B - (1 << 16)))),
    ([(A, 0, 16, F32, F32)], dict(norm_sq=_at(A + 8))), ([(A, B, 16, F32, F32)], dict(norm_sq=_at(B))),
    ([(A, B, 16, F32, F32)], dict(norm=_at(0x900004), norm_sq=_at(0x900000))),
    ([(A, B, 16, F32, F32)], dict(norm=_at(0x900000), norm_sq=_at(0x900000))),
    ([(A, B, 16, F32, F32)], dict(norm=_at(0x800010))),
])
def test_clip_checks_of_its_own_memory(grads, kw):
    """Workgroups read the squared norm, the workspace and the gradients while others
    write: none of what is written may lie in what is read, or in another result."""
    arr = _grads(*grads)
    args = dict(count=len(grads), grads=ctypes.addressof(arr), max_norm=1.0, norm_sq=None, norm=_at(0x700000),
                workspace=FAR, workspace_bytes=1 << 20)
    assert _call("nvfp4_clip_grads", args, kw) == INV


def test_norm_checks_of_its_workspace():
    for at in (A, A + 56, A - 8):
        arr = _grads((A, 0, 16, F32, F32))
        args = dict(count=1, grads=ctypes.addressof(arr), norm_sq=FAR, workspace=_at(at), workspace_bytes=1 << 20)
        assert _call("nvfp4_grad_norm_sq", args, {}) == INV


def test_clip_checks_long_lists():
    rows = [(A + 64 * i, 0, 16, F32, F32) for i in range(300)]
    arr = _grads(*rows, (A + 64 * 150 + 4, 0, 1, F32, F32))
    args = dict(count=301, grads=ctypes.addressof(arr), max_norm=1.0, norm_sq=None, norm=P, workspace=P,
                workspace_bytes=1 << 20)
    assert _call("nvfp4_clip_grads", args, {}) == INV


def test_grad_workspace_bytes():
    assert nv.nvfp4_grad_workspace_bytes(-1) == 0
    sizes = [nv.nvfp4_grad_workspace_bytes(n) for n in (0, 1, 100, 113, 1000)]
    assert all(s % 8 == 0 and s > 0 for s in sizes) and sizes == sorted(sizes)


def test_tensor_wrappers_refuse():
    f = torch.float8_e4m3fn
    a = (torch.zeros(4, 64).to(f), torch.ones(1, 4))
    w = (torch.zeros(32, 64).to(f), torch.ones(1, 32))
    q8 = (torch.zeros(4, 64, dtype=torch.int8), torch.ones(4))
    off = torch.zeros(2, dtype=torch.int32)
    for call in (
            lambda: nv.nvfp4_fp8_gated_gemm(a, w), lambda: nv.nvfp4_fp8_grouped_gated_gemm(off, 4, a, w),
            lambda: nv.nvfp4_fp8_gated_backward(torch.zeros(4, 16), torch.zeros(4, 32)),
            lambda: nv.nvfp4_fp8_grouped_gated_backward(torch.zeros(4, 16), torch.zeros(4, 32), off),
            lambda: nv.nvfp4_int8_quantize(torch.zeros(4, 32)), lambda: nv.nvfp4_int8_gemm(q8, q8),
            lambda: nv.Int8Packed((torch.zeros(4, 64), torch.ones(4))),
            lambda: nv.Int8Packed((torch.zeros(4, 24, dtype=torch.int8), torch.ones(4))),
            lambda: nv.Int8Packed((torch.zeros(4, 64, dtype=torch.int8), torch.ones(3))),
            lambda: nv.Int8Packed((torch.zeros(64, 4, dtype=torch.int8).t(), torch.ones(4))),
            lambda: nv.nvfp4_grad_norm_sq([]), lambda: nv.nvfp4_grad_norm_sq([torch.zeros(4)]),
            lambda: nv.nvfp4_clip_grads([], 1.0), lambda: nv.nvfp4_clip_grads([torch.zeros(4)], 1.0),
            lambda: nv.nvfp4_clip_grads([torch.zeros(4)], -1.0),
            lambda: nv.nvfp4_clip_grads([torch.zeros(4)], 1.0, out=[])):
        with pytest.raises(ValueError):
            call()
