"""How far a bf16 result of linear attention may be off where the factors of its last products are split into two bf16 parts.

A rounding to bf16 is off by at most half a step, 2^-8 of the value.  The result has one of its own: 2^-8 |ref|.  A factor
(a weighted score, an entry of the state, a decayed key) in two parts is off by at most 2^-8 of what the first part left,
2^-16 of the factor.  These errors are independent of one another, so a sum of n terms is off by at most 2^-16 / sqrt(3) of
the terms' root sum square, which is what the result's own rms is; a result has at most two such sums (scores; states that
were themselves summed from split keys): sqrt(2) 2^-16 / sqrt(3) = 1.25e-5 of the rms, one sigma.  SPLIT is 6 sigma, times 2
for elements whose terms are larger than the head's average (the rms is the whole head's; |ref| counts where it is larger).
One part alone would leave sigma = 2^-8 / sqrt(3) = 2.3e-3 of the rms, 15 times SPLIT, in the elements that are small
themselves."""

import math

import torch

ROUND = 2.0 ** -8
SPLIT = 2 * 6 * math.sqrt(2.0) * 2.0 ** -16 / math.sqrt(3.0)


def beyond_rounding(got, ref):
    """Max over elements of what is left of |got - ref| without half a bf16 step of ref, relative to the larger of |ref| and
    the rms of the head's elements that are not zero; [b, L, heads, d]."""
    got, ref = got.double(), ref.double()
    if ref.numel() == 0:
        return 0.0
    n = (ref != 0).sum(dim=(0, 1, 3), keepdim=True).clamp(min=1)
    rms = (ref.square().sum(dim=(0, 1, 3), keepdim=True) / n).sqrt()
    size = torch.maximum(ref.abs(), torch.where(rms > 0, rms, torch.ones_like(rms)))
    return float((((got - ref).abs() - ROUND * ref.abs()) / size).max())
