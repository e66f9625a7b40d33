"""CPU oracle of the gated feed-forward block, the INT8 operands and products,
and gradient clipping (numpy, fp64), written from the definitions in
include/nvfp4.h."""
from __future__ import annotations

import math

import numpy as np

from .fp8_ref import FP8_BLOCK, fp8_dequantize_ref

INT8_TINY = np.float32(2.0 ** -100)
# the largest slope of either activation: silu 1.0998.., gelu (tanh form) 1.1289..
ACT_SLOPE = 1.13


def _sigma(z):
    """1 / (1 + exp(-z)) without cancelling on either side."""
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act_ref(g, act: str):
    """(act(g), act'(g)) in fp64, to full relative precision in the tails."""
    g = np.asarray(g, np.float64)
    if act == "silu":
        z, dz = g, 1.0
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g)
    s = _sigma(z)
    return g * s, s * (1.0 + g * dz * _sigma(-z))


def act_error(g, act: str):
    """Largest relative error of act(g) and of sigma(z(g)) in fp32, given g
    exactly: exp within 2 ulp, 1 + e, the reciprocal (1 ulp) and the product
    with g, together below 8 * 2^-24; gelu's z is off by 4 roundings, each of
    which moves exp by |z| 2^-24."""
    g = np.clip(np.asarray(g, np.float64), -10, 10)
    z = 2 * math.sqrt(2.0 / math.pi) * (np.abs(g) + 0.044715 * np.abs(g) ** 3) if act == "gelu" else 0.0
    return (8.0 + 4.0 * z) * 2.0 ** -24


def gated_ref(a_q, a_s, w_q, w_s, w_block_rows: int, act: str):
    """(h [M, F], g, u, sum|x Wg|, sum|x Wu|) of FP8 operands in fp64."""
    a, w = fp8_dequantize_ref(a_q, a_s), fp8_dequantize_ref(w_q, w_s, w_block_rows)
    F = w.shape[0] // 2
    y, base = a @ w.T, np.abs(a) @ np.abs(w).T
    return act_ref(y[:, :F], act)[0] * y[:, F:], y[:, :F], y[:, F:], base[:, :F], base[:, F:]


def sums_tolerance(base, a, b, out_dtype: str):
    """Largest error of a product's sums before its result is rounded: the fp32
    part of oracle.fp8_tolerance and, for bf16 outputs, its term of the 8-bit
    instructions."""
    K = a.shape[1]
    tol = (128 + 3 + -(-K // FP8_BLOCK)) * 2.0 ** -24 * base
    if out_dtype == "bf16":
        starts = np.arange(0, K, FP8_BLOCK)
        ma, mb = (np.maximum.reduceat(np.abs(v), starts, axis=1) for v in (a, b))
        tol = tol + 2.0 ** -10 * (ma @ mb.T)
    return tol


def gated_tolerance(g, u, tol_g, tol_u, act: str, out_dtype: str):
    """Largest error of h = act(g) u given those of g and u: the activation moves
    by at most its largest slope times g's error and has an error of its own
    (act_error; below 2^-115 where sigma is cut to zero), two products round,
    and bf16 rounds once more by at most 2^-8 of the value."""
    v = np.abs(act_ref(g, act)[0])
    tol_v = ACT_SLOPE * tol_g
    tol_v = tol_v + act_error(np.abs(g) + tol_g, act) * (v + tol_v) + 2.0 ** -115
    tol = tol_v * (np.abs(u) + tol_u) + v * tol_u
    tol = tol + 2 * 2.0 ** -24 * (v * np.abs(u) + tol)
    if out_dtype == "bf16":
        tol = tol + 2.0 ** -8 * (v * np.abs(u) + tol)
    return tol


def gated_backward_ref(dh, gate_up, act: str):
    """([dg, du], its largest error in fp32) in fp64.  act' = sigma (1 + z' g (1 -
    sigma)): the second factor is a sum whose parts are each off by sigma's
    relative error and a few roundings."""
    dh, gu = np.asarray(dh, np.float64), np.asarray(gate_up, np.float64)
    F = dh.shape[1]
    g, u = gu[:, :F], gu[:, F:]
    v, d = act_ref(g, act)
    rel = 2 * act_error(g, act) + 6 * 2.0 ** -24
    sig = np.where(g == 0, 0.5, v / np.where(g == 0, 1.0, g))
    part = np.abs(sig) + np.abs(d - sig)          # both parts of act'
    err = np.concatenate([np.abs(dh * u) * part * rel, np.abs(dh * v) * rel], 1)
    # where sigma is cut to zero
    err = err + 2.0 ** -115 * np.concatenate([np.abs(dh * u), np.abs(dh)], 1)
    return np.concatenate([dh * u * d, dh * v], 1), err


def int8_quantize_ref(x):
    """x [rows, cols] (fp32-exact values) -> (q int8, s fp32 [rows])."""
    x = np.asarray(x, np.float32)
    finite = np.isfinite(x).all(axis=1)
    a = np.abs(np.where(finite[:, None], x, 0)).max(axis=1, initial=0).astype(np.float32)
    a = np.maximum(a, INT8_TINY)
    s, r = (a / np.float32(127)).astype(np.float32), (np.float32(127) / a).astype(np.float32)
    v = (np.where(finite[:, None], x, 0) * r[:, None]).astype(np.float32)
    q = np.rint(v).astype(np.int8)
    return q, np.where(finite, s, np.float32(np.nan)).astype(np.float32)


def int8_gemm_ref(a_q, a_s, b_q, b_s):
    """y fp32, bit for bit: the exact sum rounded to fp32, then the two scales."""
    total = np.asarray(a_q, np.float64) @ np.asarray(b_q, np.float64).T  # exact: below 2^53
    y = total.astype(np.float32)
    with np.errstate(invalid="ignore"):
        return (y * np.asarray(a_s, np.float32)[:, None]).astype(np.float32) * np.asarray(b_s, np.float32)[None, :]


def clip_ref(grads, max_norm: float, norm_sq: float | None = None):
    """(norm, coefficient, clipped values in fp64) of a list of arrays."""
    if norm_sq is None:
        norm_sq = math.fsum(float(v) for g in grads for v in np.square(np.asarray(g, np.float64)).ravel())
    norm = math.sqrt(norm_sq)
    c = max_norm / norm if math.isfinite(norm) and norm > max_norm else 1.0
    return norm, c, [np.asarray(g, np.float64) * c for g in grads]
