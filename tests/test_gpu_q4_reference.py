"""skv_attend_q4 where its running reference is stale or rises: scores that rise
from block to block by chosen steps, peaked and flat heads.

The bound on out is tight.  The kernel computes sum_j P_j v_j / sum_j P_j with the
same P_j in both sums: p_j rounded to bf16, P_j = p_j (1 + d_j) with |d_j| <= u = 2^-8
(half a step relative to the value).  Before the output's own rounding it is therefore off by
    | sum_j w_j d_j (v_j - out) | / | sum_j w_j (1 + d_j) |  <=  u / (1 - u) * sum_j w_j |v_j - out|
where w_j are the exact softmax weights: nothing at all for a head that one key dominates,
whatever that key's P rounds to.  To this come the errors of the scores, the exponentials
and the fp32 sums: relative errors of p_j of at most e_j move out by at most 2 max e_j * sum_j w_j
|v_j - out|; e = ds + MISC as in tests/attention_check.py, without the rounding of exchanged scores
(they cross as fp32).  fp32 accumulation over up to 4096 keys and the joining of splits: MISC
of the largest value.  The output lies between the bf16 roundings of the ends of that interval."""
import numpy as np
import pytest
import torch

import attention_check as ac
import test_gpu_q4 as g4
from oracle import attention as att
from oracle import q4

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
CODE = {0.0: 0, 0.5: 1, 1.0: 2, 1.5: 3, 2.0: 4, 3.0: 5, 4.0: 6, 6.0: 7}


def _bf16_round(x):
    """float64 -> the nearest bf16 (ties to even), as float64; the exponent range is not touched."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def check(q, keys, scale, out, lse, what):
    """One unit: q [H][576], keys [k][576] float64; out [H][512] as float64, lse [H]."""
    x = q @ keys.T * scale
    want, want_lse = att.attend(q, keys, np.ones(len(keys), bool), scale)
    w = np.exp(x - want_lse[:, None])
    v = keys[:, :512]
    a = np.abs(q) @ np.abs(keys).T
    e = (scale * ac.ACC * a + 2.0 ** -23 * np.abs(x)).max(axis=1) + ac.MISC
    vmax = np.abs(v).max()
    for h in range(len(q)):
        spread = w[h] @ np.abs(v - want[h])
        tol = (U / (1 - U) + 2 * e[h]) * spread + ac.MISC * vmax
        lo, hi = _bf16_round(want[h] - tol), _bf16_round(want[h] + tol)
        bad = (out[h] < lo) | (out[h] > hi)
        assert not bad.any(), (what, h, np.abs(out[h] - want[h]).max(), tol.max())
    lse_tol = e + (len(keys) / 32 + 64) * 2.0 ** -24 + ac.MISC
    assert np.all(np.abs(lse - want_lse) <= lse_tol), (what, np.abs(lse - want_lse).max())


def _rows(rng, x, exponent=0, gain=0x38):
    """Packed rows [n][336] of random value codes whose value 512 is x [n] (a code, under the scale `gain`); the other
    rope values are zero."""
    n = len(x)
    p = np.zeros((n, q4.ROW_BYTES), np.uint8)
    p[:, :256] = rng.integers(0, 256, (n, 256))
    p[:, 288:320] = rng.integers(0x30, 0x40, (n, 32))  # scales 0.5 .. 1.875
    p[:, 256] = [CODE[float(v)] for v in x]
    p[:, 320] = gain
    p[:, 324] = 127 + exponent
    return p


class Units:
    """A context of packed rows whose units hold the given rows in order."""

    def __init__(self, packed):
        self.packed = packed  # [B][L][k][336]
        B, L, k = packed.shape[:3]
        self.ctx = g4._ctx(B, L, k, k, k, B)
        self.req = torch.tensor([self.ctx.publish(k, rows=np.ascontiguousarray(packed[b])) for b in range(B)],
                                dtype=torch.int32, device="cuda")
        topk = torch.arange(k, dtype=torch.int32, device="cuda").expand(B, L, k).contiguous()
        self.slots = torch.empty_like(topk)
        n = torch.empty((2, B, L), dtype=torch.int32, device="cuda")
        self.ctx.assemble(self.req, topk, self.slots, n[0], n[1])

    def attend(self, q, scale, sms):
        """q [units][128][576] of bf16 values -> out as float64, lse."""
        out, lse = g4._outputs(q.shape[0])
        self.ctx.set_attend_sms(sms)
        self.ctx.attend_q4(self.req, torch.from_numpy(q).to(torch.bfloat16).cuda(), self.slots, out, lse, sm_scale=scale)
        assert self.ctx.get_device_error() == 0
        return out.double().cpu().numpy(), lse.cpu().numpy()


def _queries(rng, units, rises, unit=1.0):
    """q whose only score dim is value 512: heads with q_512 = rises (cycled, permuted per unit)."""
    q = np.zeros((units, 128, 576))
    for n in range(units):
        q[n, :, 512] = _bf16_round(rng.permutation(np.resize(rises, 128)) * unit)
    return q


# A score is q_512 * x / 8 in log2, x one of 0 .. 6: a head with q_512 = 4 r / 3 rises by r where x goes from 0 to 6.
RISES = np.array([0, 1, 7.9, 8.1, 15, 20, 22, 22.5, 23, 23.3, 23.7, 24.2, 25, 26, 31, 40, 60, -3, -40])
SCALE = np.log(2.0) / 8


@pytest.mark.parametrize("at", [5, 37])  # the peak's place in its block: either CTA's half
@pytest.mark.parametrize("sms", [2, 0])
@pytest.mark.parametrize("steps", [(0, 6), (0, 6, 0, 0, 0), (0, 2, 3, 6, 4), (0, 0, 0, 0, 6), (6, 0, 0), (1.5, 2, 2, 3, 6, 6, 0.5)])
def test_blocks_whose_maxima_rise(steps, sms, at):
    """Every block's keys have x = 0 but one, which has the step's; two units a pair of SMs (sms = 2), or each unit's blocks
    over all pairs."""
    rng = np.random.default_rng(len(steps) + at)
    k = 64 * len(steps) - 9  # the last block is ragged
    x = np.zeros((2, 1, k))
    for i, s in enumerate(steps):
        x[0, 0, 64 * i + at] = s
        x[1, 0, 64 * i + at] = steps[(i + 1) % len(steps)]
    packed = np.stack([_rows(rng, x[b, 0])[None] for b in range(2)])
    u = Units(packed)
    q = _queries(rng, 2, RISES * 4 / 3)
    out, lse = u.attend(q, SCALE, sms)
    for n in range(2):
        check(q[n], q4.values(packed[n, 0]), SCALE, out[n], lse[n], n)
    u.ctx.close()


@pytest.mark.parametrize("sms", [2, 0])
def test_a_dominating_key_gives_its_values_whatever_its_weight_rounds_to(sms):
    """Heads whose one large p is any number between 2^17 and 2^24 of the reference's: out is that key's row to
    within the others' weight, not to within p's rounding."""
    rng = np.random.default_rng(41)
    k = 256
    x = np.zeros(k)
    x[200] = 6
    packed = _rows(rng, x)[None, None]
    u = Units(packed)
    q = _queries(rng, 1, np.linspace(17, 24, 128) * 4 / 3)
    out, lse = u.attend(q, SCALE, sms)
    keys = q4.values(packed[0, 0])
    check(q[0], keys, SCALE, out[0], lse[0], "")
    # and so, beyond the bound: where the others weigh less than a quarter of a step, the very values
    heavy = q[0, :, 512] > 22 * 4 / 3
    row = keys[200, :512]
    large = np.abs(row) >= np.abs(keys[:, :512]).max() / 8
    assert heavy.sum() > 20 and large.sum() > 100
    assert np.array_equal(out[0][heavy][:, large], np.broadcast_to(row[large], (heavy.sum(), large.sum())))
    u.ctx.close()


@pytest.mark.parametrize("sms", [2, 0])
@pytest.mark.parametrize("scale", [1 / 24, 0.2])
def test_rows_as_a_cache_holds_them_within_the_tight_bound(scale, sms):
    rng = np.random.default_rng(43)
    k = 700
    x = (rng.standard_normal((2, k, 576)) * np.exp2(rng.uniform(-1, 1, 576)) * np.exp2(rng.uniform(-2, 2, (2, k, 1)))).astype(np.float32)
    packed = q4.pack(x.reshape(-1, 576)).reshape(2, 1, k, q4.ROW_BYTES)
    u = Units(packed)
    q = _bf16_round(rng.standard_normal((2, 128, 576)))
    out, lse = u.attend(q, scale, sms)
    for n in range(2):
        check(q[n], q4.values(packed[n, 0]), scale, out[n], lse[n], n)
    u.ctx.close()


@pytest.mark.parametrize("sms", [2, 0])
@pytest.mark.parametrize("rise", [20, 23.9, 24.1, 40])
def test_large_values_under_a_stale_reference_stay_finite(rise, sms):
    """Values up to 2^103.5, eight of whose keys rise by `rise` above the reference of the block before: under that
    reference their sum of P v would pass the range of fp32 at 2^23.9, under one that keeps P at 2^8 it does not."""
    rng = np.random.default_rng(47)
    k = 192
    x = np.zeros(k)
    x[100:108] = 6
    packed = _rows(rng, x, exponent=100)[None, None]
    packed[0, 0, 100:108, :256] = 0x77  # the largest code, all of one sign
    u = Units(packed)
    q = _queries(rng, 1, np.array([rise]) * 4 / 3, unit=2.0 ** -100)
    out, lse = u.attend(q, SCALE, sms)
    assert np.isfinite(out).all()
    check(q[0], q4.values(packed[0, 0]), SCALE, out[0], lse[0], "")
    u.ctx.close()
