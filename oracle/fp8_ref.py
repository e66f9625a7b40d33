"""CPU oracle of the FP8 block-128 operands and products and of the expert
router (numpy, fp64), written from the definitions in include/nvfp4.h."""
from __future__ import annotations

import numpy as np

FP8_BLOCK = 128
FP8_TINY = np.float32(2.0 ** -100)
FP8_MAX = np.float32(448.0)


def _e4m3_table() -> np.ndarray:
    """Values of the 256 E4M3FN codes (1 sign, 4 exponent bits of bias 7, 3
    mantissa bits; exponent 0 subnormal; 0x7F and 0xFF NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0))
    v = np.where(c & 0x80, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


E4M3_TABLE = _e4m3_table()


def e4m3_encode(v) -> np.ndarray:
    """Codes of finite |v| <= 448 (1 + small): nearest value, ties to the even
    code, sign kept."""
    a = np.abs(np.asarray(v, np.float64))
    mags = E4M3_TABLE[:127]
    lo = np.clip(np.searchsorted(mags, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    mid = (mags[lo] + mags[hi]) / 2
    up = (a > mid) | ((a == mid) & (lo % 2 == 1))
    code = np.where(up, hi, lo)
    return (code | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def fp8_quantize_ref(x, block_rows: int = 1):
    """x [rows, cols] (fp32-exact values) -> (q uint8 [rows, cols],
    s fp32 [ceil(cols/128), ceil(rows/block_rows)]), rows layout."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // FP8_BLOCK)
    p = np.zeros((nr * block_rows, nc * FP8_BLOCK), np.float32)
    p[:rows, :cols] = x
    p = p.reshape(nr, block_rows, nc, FP8_BLOCK)
    finite = np.isfinite(p).all(axis=(1, 3))
    a = np.abs(np.where(np.isfinite(p), p, 0)).max(axis=(1, 3))
    a = np.maximum(a, FP8_TINY).astype(np.float32)
    s = (a / FP8_MAX).astype(np.float32)
    r = (FP8_MAX / a).astype(np.float32)
    keep = finite[:, None, :, None]
    v = (np.where(keep, p, 0) * r[:, None, :, None]).astype(np.float32)
    q = np.where(keep, e4m3_encode(v), 0).astype(np.uint8)
    s = np.where(finite, s, np.float32(np.nan)).astype(np.float32)
    q = q.reshape(nr * block_rows, nc * FP8_BLOCK)[:rows, :cols]
    return q, np.ascontiguousarray(s.T)


def fp8_quantize_t_ref(x, block_rows: int = 1):
    """The transposed layout: q [cols, rows rounded up to 16], blocks along
    the columns of x."""
    x = np.asarray(x, np.float32)
    pad = np.zeros((-(-x.shape[0] // 16) * 16, x.shape[1]), np.float32)
    pad[:x.shape[0]] = x
    return fp8_quantize_ref(pad.T, block_rows)


def fp8_grouped_columns_ref(total_m: int, G: int) -> int:
    return (total_m + 127 * min(G, total_m)) // 128 * 128


def fp8_grouped_quantize_t_ref(x, offsets):
    """Transposed layout of rows sorted by group, each group's tokens starting
    at a multiple of 128 columns."""
    x = np.asarray(x, np.float32)
    G = len(offsets) - 1
    wide = np.zeros((fp8_grouped_columns_ref(x.shape[0], G), x.shape[1]), np.float32)
    at = 0
    for e in range(G):
        part = x[offsets[e]:offsets[e + 1]]
        wide[at:at + len(part)] = part
        at += -(-len(part) // 128) * 128
    return fp8_quantize_ref(wide.T)


def fp8_dequantize_ref(q, s, block_rows: int = 1) -> np.ndarray:
    """Values of an operand [rows, K] in fp64 (exact)."""
    rows, K = q.shape
    f = np.repeat(np.repeat(np.asarray(s, np.float64).T, block_rows, 0)[:rows], FP8_BLOCK, 1)[:, :K]
    return E4M3_TABLE[np.asarray(q)] * f


def fp8_gemm_ref(a_q, a_s, b_q, b_s, b_block_rows: int = 1):
    """(y, sum_k |A B|) of y[m, n] = sum_k A(m, k) B(n, k) in fp64."""
    a = fp8_dequantize_ref(a_q, a_s)
    b = fp8_dequantize_ref(b_q, b_s, b_block_rows)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def fp8_tolerance(y_ref, base, a, b, out_dtype: str):
    """Largest error of the product of operands with values a [M, K] and
    b [N, K].  fp32 outputs: 128 fp32 additions in a block, the product of two
    scales and of them with the block's sum, and one addition per block, each
    off by at most 2^-24 of a partial sum that sum |A B| bounds.  bf16 outputs
    round once more, by at most 2^-8 of the value, and their blocks are summed
    by the 8-bit matrix instruction, which cuts each product 2^-16 below the
    largest running sum.  For operands without outliers that costs up to
    2^-11.2 of the largest of 128 products (an in-bounds check of the
    instruction alone), counted here as 2^-10 of max |A| max |B|.  It is no
    bound for all operands: that is 2^-9 sum |A B|, and blocks of one outlier
    and 127 small products come near it."""
    K = a.shape[1]
    tol = (128 + 3 + -(-K // FP8_BLOCK)) * 2.0 ** -24 * base
    if out_dtype == "bf16":
        starts = np.arange(0, K, FP8_BLOCK)
        ma, mb = (np.maximum.reduceat(np.abs(v), starts, axis=1) for v in (a, b))
        tol = tol + 2.0 ** -10 * (ma @ mb.T)
        tol = tol + 2.0 ** -8 * (np.abs(y_ref) + tol)
    return tol


def moe_route_ref(logits, topk: int, mask=None, renormalize: bool = False):
    """Router in fp64, token by token.  Returns a dict of the outputs of
    nvfp4_moe_route and ``p`` (probabilities)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    idx = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    p = np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:topk]
        if not order:
            continue
        ez = np.exp(x[t] - x[t, order[0]])
        p[t] = ez / ez.sum()
        idx[t, :len(order)] = order
        w[t, :len(order)] = ez[order] / ez[order].sum() if renormalize else p[t, order]
    counts = np.bincount(idx[idx >= 0], minlength=E).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    row_index = np.full(T * topk, -1, np.int32)
    pair_row = np.full((T, topk), -1, np.int32)
    nxt = off[:-1].copy()
    for t in range(T):
        for j in range(topk):
            e = idx[t, j]
            if e >= 0:
                row_index[nxt[e]], pair_row[t, j] = t, nxt[e]
                nxt[e] += 1
    n = int((idx[:, 0] >= 0).sum())
    loss = E * float((counts / (n * topk) * p.sum(0) / n).sum()) if n else 0.0
    return dict(expert_index=idx, weights=w, counts=counts, m_offsets=off, row_index=row_index,
                pair_row=pair_row, routed=n, loss=loss, p=p)


def moe_route_backward_ref(r, topk: int, d_weights, d_loss: float, renormalize: bool = False):
    """Gradient of the logits, token by token, from moe_route_ref's answer."""
    p, idx = r["p"], r["expert_index"]
    T, E = p.shape
    n = r["routed"]
    c = d_loss * E * r["counts"] / (n * topk) / n if n else np.zeros(E)
    dx = np.zeros((T, E))
    for t in range(T):
        sel = idx[t][idx[t] >= 0]
        if not len(sel):
            continue
        dp, dw = c.copy(), np.asarray(d_weights[t], np.float64)[:len(sel)]
        if renormalize:
            w = r["weights"][t][:len(sel)]
            dx[t, sel] += w * (dw - (w * dw).sum())
        else:
            dp[sel] += dw
        dx[t] += p[t] * (dp - (p[t] * dp).sum())
    return dx
