"""The 4-bit KV row written out as its definition -- TEST INFRASTRUCTURE ONLY.

include/skv.h gives the format ("KV rows in 4 bits"): 36 groups of 16 values,
e2m1 codes, an e4m3 scale a group, one exponent a row.  Everything here is
float64 and looks values up in the formats' value tables; nothing is shared
with the library or its kernels.

Parity status: pinned in tests/test_oracle_q4.py by rows whose packed bytes are
derived by hand, by the tables' closed forms, and by a scalar search over all
codes and scales.
"""
from __future__ import annotations

import numpy as np

DIM, GROUPS, GROUP = 576, 36, 16
ROW_BYTES, SCALES_AT, EXP_AT = 336, 288, 324

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3 codes 0..126 (127 is a NaN): 3 fraction bits, bias 7, subnormals below 2^-6
E4M3 = np.array([m * 2.0 ** -9 if p == 0 else (8 + m) * 2.0 ** (p - 10) for p in range(16) for m in range(8)][:127])


def nearest(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table value nearest to each x >= 0 (ties to the even index; above the table: its last)."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def pack(x: np.ndarray) -> np.ndarray:
    """Rows [n][576] (bf16 values as float64) -> packed rows [n][336] uint8."""
    x = np.asarray(x, np.float64)
    n = x.shape[0]
    g = x.reshape(n, GROUPS, GROUP)
    fine = np.isfinite(g).all(-1)
    a = np.where(fine, np.abs(np.where(np.isfinite(g), g, 0.0)).max(-1), 0.0)
    top = a.max(-1)
    # the least e with 2688 * 2^e >= top: frexp gives top / 2688 = m * 2^e, m in [0.5, 1)
    m, e = np.frexp(top / 2688.0)
    e = np.where(m == 0.5, e - 1, e)
    e = np.where(top > 0, np.clip(e, -100, 116), -100)
    unit = np.ldexp(1.0, e)[:, None]
    si = nearest(a / unit / 6.0, E4M3)
    scale = E4M3[si] * unit
    live = fine & (si > 0)
    safe = np.where(live, scale, 1.0)[..., None]
    code = nearest(np.where(live[..., None], np.abs(g), 0.0) / safe, E2M1)
    code = np.where(live[..., None], code + 8 * np.signbit(g), 0).astype(np.uint8).reshape(n, DIM // 2, 2)
    out = np.zeros((n, ROW_BYTES), np.uint8)
    out[:, :SCALES_AT] = code[..., 0] | (code[..., 1] << 4)
    out[:, SCALES_AT:EXP_AT] = np.where(fine, si, 127)
    out[:, EXP_AT] = e + 127
    return out


def values(packed: np.ndarray) -> np.ndarray:
    """Packed rows [..., 336] -> the values they stand for [..., 576], float64."""
    p = np.asarray(packed, np.uint8)
    codes = np.concatenate([E2M1, -E2M1])
    scales = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])  # pack writes no negative one
    b = p[..., :SCALES_AT]
    v = codes[np.stack([b & 15, b >> 4], -1)].reshape(*p.shape[:-1], GROUPS, GROUP)
    v = v * scales[p[..., SCALES_AT:EXP_AT]][..., None]
    return (v * np.ldexp(1.0, p[..., EXP_AT].astype(int) - 127)[..., None, None]).reshape(*p.shape[:-1], DIM)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """float64 values that bf16 holds exactly (or NaN) -> their bits."""
    f = np.asarray(x, np.float64).astype(np.float32)
    bits = f.view(np.uint32)
    assert np.all(np.isnan(f) | ((bits & 0xFFFF) == 0)), "a value bf16 does not hold"
    return (bits >> 16).astype(np.uint16)


def test_rows(n: int, seed: int) -> np.ndarray:
    """bf16 rows [n][576] as bits: latents of many sizes, and, from row 1 on, the rows where rounding can go wrong."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, DIM)) * np.exp2(rng.uniform(-3, 3, (n, 1))) * np.exp2(rng.uniform(-2, 2, DIM))
    x[:, 512:] *= 3
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # truncated: any bf16 will do
    # a row on which every value is a tie between two codes of scale 1 (or an end of them), sizes 0.25 .. 5 and 6
    ties = np.tile(np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25]), GROUPS)
    big = np.float32(3.3895313892515355e38)
    special = [
        np.zeros(DIM), -np.zeros(DIM), ties * 448, ties * 2.0 ** -30,
        np.where(np.arange(DIM) == 77, np.nan, x[0]), np.where(np.arange(DIM) == 575, -np.inf, x[0]),
        np.full(DIM, np.nan), np.full(DIM, big), np.where(np.arange(DIM) < 16, big, x[0]),
        np.full(DIM, 2.0 ** -133), x[0] * 2.0 ** -126, x[0] * 2.0 ** -112, x[0] * 2.0 ** 118,
        np.where(np.arange(DIM) < 560, x[0] * 2.0 ** -15, 2688.0),  # groups whose scale is an e4m3 subnormal or 0
        np.full(DIM, 2688.0), np.full(DIM, 2704.0), np.where(np.arange(DIM) == 3, 1.0, 0.0),
    ]
    for i, s in enumerate(special):
        if i + 1 < n:
            bits[i + 1] = (np.asarray(s, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    # scale ties: a group's largest value 6 * (midpoint of two e4m3 values), the row's exponent held at 0 by 2688
    if n > 40:
        mid = (E4M3[1:] + E4M3[:-1]) / 2 * 6
        for r in range(4):
            row = np.zeros((GROUPS, GROUP))
            row[0, 0] = 2688.0
            row[1:, 0] = mid[r * 30:r * 30 + 35]
            row[1:, 1] = -row[1:, 0] / 2
            bits[20 + r] = (row.reshape(-1).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return bits


test_rows.__test__ = False  # not a pytest function
