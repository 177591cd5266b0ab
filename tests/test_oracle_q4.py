"""The 4-bit row's oracle against rows packed by hand, the formats' closed
forms and a scalar search (CPU only)."""
import numpy as np
import pytest

from oracle import attention as att
from oracle import q4


def test_tables_are_the_formats():
    assert len(q4.E4M3) == 127 and q4.E4M3[-1] == 448 and q4.E4M3[1] == 2.0 ** -9 and q4.E4M3[8] == 2.0 ** -6
    assert np.all(np.diff(q4.E4M3) > 0) and np.all(np.diff(q4.E2M1) > 0)
    assert q4.E2M1[-1] * q4.E4M3[-1] == 2688


def test_a_row_packed_by_hand():
    # one group holds 0..7 and their negatives; its largest value 7 gives e: 2688 * 2^-9 = 5.25 < 7 <= 10.5, so e = -8;
    # scale 7 * 256 / 6 = 298.67 -> e4m3 288 (code 0x79: 2^8 * 1.125); unit 288 / 256 = 1.125
    x = np.zeros((1, 576))
    x[0, 16:24] = np.arange(8)
    x[0, 24:32] = -np.arange(8.0)
    p = q4.pack(x)
    assert p[0, 324] == 127 - 8 and p[0, 289] == 0x79 and not p[0, 325:].any()
    # x / 1.125: 0 .889 1.778 2.667 3.556 4.444 5.333 6.222 -> codes 0, 1 (2), 2 (4), 3 (5), 4 (6), 4 (6), 6 (7), 6 (7)
    assert list(p[0, 8:16]) == [0x20, 0x54, 0x66, 0x77, 0x28 | 0x80, 0xDC, 0xEE, 0xFF]
    assert not p[0, :8].any() and not p[0, 16:288].any()
    v = q4.values(p)[0]
    assert list(v[16:24]) == [0, 1.125, 2.25, 3.375, 4.5, 4.5, 6.75, 6.75]
    assert np.array_equal(v[24:32], -v[16:24])


def test_zero_bytes_are_a_zero_row_and_bad_groups_read_nan():
    assert not q4.values(np.zeros(336, np.uint8)).any()
    x = np.ones((1, 576))
    x[0, 5] = np.nan
    x[0, 575] = np.inf
    v = q4.values(q4.pack(x))[0]
    # ones: e = -11, scale 2048 / 6 = 341.3 -> 352, code 2048 / 352 = 5.8 -> 6, value 6 * 352 / 2048
    assert np.isnan(v[:16]).all() and np.isnan(v[560:]).all() and np.all(v[16:560] == 1.03125)


def test_every_value_is_a_bf16_and_within_the_formats_error():
    bits = q4.test_rows(64, 3)
    x = att.bf16_rows_to_f64(bits.view(np.uint8))
    v = q4.values(q4.pack(x))
    assert np.array_equal(np.isnan(v), np.repeat(~np.isfinite(x.reshape(-1, 36, 16)).all(-1), 16, axis=1).reshape(-1, 576))
    q4.bf16_bits(v)
    ok = ~np.isnan(v).any(1) & (np.abs(x).max(1) > 2.0 ** -89) & (np.abs(x).max(1) < 2.0 ** 127)
    # a code's rounding is at most 1 (between 4 and 6) of a largest value 6; the scale's at most 2^-4; saturation 6.4 to 6
    a = np.abs(x).reshape(-1, 36, 16).max(-1).repeat(16, -1).reshape(-1, 576)
    floor = np.abs(x).max(1, keepdims=True) * 2.0 ** -17  # groups below the smallest scale
    assert np.all(np.abs(v - x)[ok] <= (a / 6 * 1.07 + floor)[ok])


@pytest.mark.parametrize("seed", [1, 2])
def test_codes_are_the_nearest_by_search(seed):
    """Scalar search over every code of the chosen scale, and over every scale."""
    bits = q4.test_rows(8, seed)[:2]
    x = att.bf16_rows_to_f64(bits.view(np.uint8))
    p = q4.pack(x)
    v = q4.values(p)
    for r in range(2):
        e = int(p[r, 324]) - 127
        if np.abs(x[r]).max() > 0:
            assert 2688 * 2.0 ** e >= np.abs(x[r]).max() > 2688 * 2.0 ** (e - 1)
        for g in range(36):
            s = q4.E4M3[p[r, 288 + g]]
            want = np.abs(x[r, 16 * g:16 * g + 16]).max() * 2.0 ** -e / 6
            assert abs(s - want) == min(abs(t - want) for t in q4.E4M3)
            for i in range(16 * g, 16 * g + 16):
                got = abs(abs(v[r, i]) - abs(x[r, i]))
                assert got == min(abs(c * s * 2.0 ** e - abs(x[r, i])) for c in q4.E2M1)
