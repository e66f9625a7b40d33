"""The FP8 and router oracle against independent definitions (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import (E4M3_TABLE, e4m3_encode, fp8_dequantize_ref, fp8_gemm_ref,
                    fp8_grouped_columns_ref, fp8_grouped_quantize_t_ref, fp8_quantize_ref,
                    fp8_quantize_t_ref, moe_route_backward_ref, moe_route_ref)


def test_e4m3_table_and_encoder_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, E4M3_TABLE, equal_nan=True)
    # every value, every midpoint and its fp32 neighbours
    mags = E4M3_TABLE[:127]
    mid = ((mags[1:] + mags[:-1]) / 2).astype(np.float32)
    v = np.concatenate([mags.astype(np.float32), mid, np.nextafter(mid, np.float32(0)),
                        np.nextafter(mid, np.float32(1e9))])
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(e4m3_encode(v), want)


@pytest.mark.parametrize("rows,cols,block_rows", [(3, 16, 1), (5, 400, 1), (130, 272, 128), (1, 128, 128)])
def test_quantize_is_within_half_a_step(rows, cols, block_rows):
    rng = np.random.default_rng(rows + cols)
    x = (rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-20, 20, (rows, 1)))).astype(np.float32)
    q, s = fp8_quantize_ref(x, block_rows)
    assert q.shape == (rows, cols) and s.shape == (-(-cols // 128), -(-rows // block_rows))
    v = fp8_dequantize_ref(q, s, block_rows)
    step = np.repeat(np.repeat(s.T.astype(np.float64), block_rows, 0)[:rows], 128, 1)[:, :cols]
    # half a step is 2^-4 of the value, or half of the smallest 2^-9; the
    # scale, its reciprocal and the product round by 2^-24 each
    assert np.all(np.abs(v - x) <= (2.0 ** -4 + 2.0 ** -21) * np.abs(x) + 2.0 ** -10 * (1 + 2.0 ** -21) * step)


def test_quantize_special_blocks():
    x = np.zeros((6, 256), np.float32)
    x[1, 3] = np.nan
    x[2, 200] = np.inf
    x[3, :] = np.float32(1e-40)
    x[4, :] = np.float32(3e38)
    x[5, 0] = -0.0
    q, s = fp8_quantize_ref(x)
    assert np.isnan(s[0, 1]) and np.isnan(s[1, 2]) and np.isfinite(s[1, 1]) and np.isfinite(s[0, 2])
    assert not q[1, :128].any() and not q[2, 128:].any() and not q[0].any()
    assert q[5, 0] == 0x80 and np.all(q[4] == 126)
    assert np.all(s[:, 0] == np.float32(2.0 ** -100) / np.float32(448))


def test_layouts_hold_the_same_tensor():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((37, 48)).astype(np.float32)
    qt, st = fp8_quantize_t_ref(x)
    assert qt.shape == (48, 48) and st.shape == (1, 48) and not qt[:, 37:].any()
    q, _ = fp8_quantize_ref(x, 128)
    qt128, _ = fp8_quantize_t_ref(x, 128)
    assert np.array_equal(q, qt128[:, :37].T)
    off = [0, 5, 5, 37]
    g, gs = fp8_grouped_quantize_t_ref(x, off)
    assert g.shape == (48, fp8_grouped_columns_ref(37, 3)) and gs.shape == (g.shape[1] // 128, 48)
    first, fs = fp8_quantize_t_ref(x[:5])
    assert np.array_equal(g[:, :5], first[:, :5]) and np.array_equal(gs[0], fs[0])
    last, ls = fp8_quantize_t_ref(x[5:])
    assert np.array_equal(g[:, 128:160], last[:, :32]) and np.array_equal(gs[1], ls[0])


def test_gemm_ref_is_the_triple_sum():
    rng = np.random.default_rng(2)
    aq, bq = (rng.integers(0, 127, (r, 144)).astype(np.uint8) for r in (3, 130))
    sa, sb = rng.random((2, 3)).astype(np.float32), rng.random((2, 2)).astype(np.float32)
    y, base = fp8_gemm_ref(aq, sa, bq, sb, 128)
    for m, n in ((0, 0), (2, 129), (1, 127)):
        want = sum(E4M3_TABLE[aq[m, k]] * float(sa[k // 128, m]) * E4M3_TABLE[bq[n, k]]
                   * float(sb[k // 128, n // 128]) for k in range(144))
        assert abs(y[m, n] - want) <= 1e-12 * base[m, n]


@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    T, E, k = 5, 7, 3
    x = rng.standard_normal((T, E))
    x[2, 1:] = -np.inf                      # fewer experts than choices
    x[3] = -np.inf                          # none at all
    mask = np.array([1, 1, 1, 1, 0])
    dw, dl = rng.standard_normal((T, k)), 0.7
    r = moe_route_ref(x, k, mask, renorm)
    assert r["routed"] == 3 and r["counts"].sum() == 7
    g = moe_route_backward_ref(r, k, dw, dl, renorm)

    def value(y):
        q = moe_route_ref(y, k, mask, renorm)
        assert np.array_equal(q["expert_index"], r["expert_index"])
        return dl * q["loss"] + float((q["weights"] * np.where(q["expert_index"] >= 0, dw, 0)).sum())

    h = 1e-6
    for t in range(T):
        for e in range(E):
            if x[t, e] == -np.inf:
                assert g[t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central differences: O(h^2) truncation and 1e-16 / h rounding
            assert abs((value(up) - value(dn)) / (2 * h) - g[t, e]) < 1e-8


def test_even_load_has_loss_one():
    x = np.eye(4) * 30.0
    r = moe_route_ref(x, 1)
    assert abs(r["loss"] - 1.0) < 1e-9 and r["counts"].tolist() == [1, 1, 1, 1]
    assert r["row_index"].tolist() == [0, 1, 2, 3]
