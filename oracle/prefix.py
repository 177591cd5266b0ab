"""Attention over a prefix that a batch shares, the join of attention results, the
weights of the prefix's tokens and the eviction of the lightest, written out as
their definitions in 64 bits -- TEST INFRASTRUCTURE ONLY (include/skv.h,
skv_attend_prefix, skv_join, skv_weigh_prefix, skv_evict_prefix).

Tensors (torch, of any device), one layer at a time:

    s_ij = scale q_i . k_j
    lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) k_j[:512]
    weight_j = before_j + gain sum_i exp(s_ij - lse_i)

Each comes with a bound on what the kernels may be off by, from the roundings
they make (u below, the half step of bf16):

- A score is a sum of 576 exact products in fp32, 36 steps of 16 on the tensor
  cores: off by at most ds_ij = STEPS scale |q_i| . |k_j|.
- P is rounded to bf16, and the output divided by the sum of the rounded P, so
  an error of P moves out_i by at most its share of |v_j - out_i|, which is at
  most |v_j| + |out_i|: (u + 2 ds) (sum_j w_ij |v_j| + |out_i|); then out itself
  is rounded (u |out_i|).
- An exponential, a logarithm, a division and the sums of n numbers: MISC + n 2^-24.
- The exponent's argument in a weight holds the scale and the lse times log2 e,
  each rounded: off by at most 2^-23 (|s_ij| + |lse_i| + 1) relative to the term.

Parity status: pinned in tests/test_oracle_prefix.py by hand-made cases and by
identities (a split prefix joined, shares that sum to the batch's heads).
"""
from __future__ import annotations

import math

import torch

U_BF16 = 2.0 ** -8
STEPS = 37 * 2.0 ** -22
MISC = 1e-5


def scores(q, rows, scale):
    """q [i][576], rows [j][576] -> [i][j]."""
    return q.double() @ rows.double().T * scale


def attend(q, rows, scale):
    """-> out [i][512], lse [i], and the bounds on both."""
    if rows.shape[0] == 0:
        zero = q.new_zeros((q.shape[0], 512), dtype=torch.float64)
        none = q.new_full((q.shape[0],), -math.inf, dtype=torch.float64)
        return zero, none, zero, torch.zeros_like(none)
    s = scores(q, rows, scale)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[:, None])
    v = rows[:, :512].double()
    out = w @ v
    ds = (STEPS * scale * (q.double().abs() @ rows.double().abs().T)).amax(-1)
    n = rows.shape[0] * 2.0 ** -24
    spread = w @ v.abs() + out.abs()
    return out, lse, (U_BF16 + 2 * ds + MISC + n)[:, None] * spread + U_BF16 * out.abs() + 1e-30, ds + MISC + n


def join(outs, lses):
    """Parts outs[p] [i][512], lses[p] [i] -> out, lse."""
    lse = torch.stack([e.double() for e in lses])
    both = torch.logsumexp(lse, 0)
    out = torch.zeros_like(outs[0], dtype=torch.float64)
    for o, e in zip(outs, lse):
        out += torch.where((e == -math.inf)[..., None], 0.0, torch.exp(e - both)[..., None] * o.double())
    return out, both


def weigh(q, rows, lse, scale, before=None, gain=1.0):
    """-> the weights [j], and the bound on them."""
    n = rows.shape[0]
    w = torch.zeros(n, dtype=torch.float64, device=q.device) if before is None else before.double()
    live = lse != -math.inf
    q, lse = q[live], lse[live].double()
    s = scores(q, rows, scale)
    p = torch.exp(s - lse[:, None])
    ds = STEPS * scale * (q.double().abs() @ rows.double().abs().T)
    off = (p * (ds + 2.0 ** -23 * (s.abs() + lse.abs()[:, None] + 1) + 2.0 ** -21)).sum(0) + q.shape[0] * 2.0 ** -24 * p.sum(0)
    return w + gain * p.sum(0), abs(gain) * off + 2.0 ** -23 * (w.abs() + abs(gain) * p.sum(0)) + 1e-37


def evict(weights, keep, first, last):
    """The tokens that stay, ascending, of weights [j]."""
    n = len(weights)
    w = [float(x) for x in weights]
    rank = sorted(range(n), key=lambda j: (not (j < first or j >= n - last), math.isnan(w[j]), 0.0 if math.isnan(w[j]) else -w[j], j))
    return sorted(rank[:keep])
