"""The bound of mixer_bounds tells factors in two bf16 parts from factors in one: the operator in fp64 with its weighted scores
and its state rounded the one way and the other."""

import pytest
import torch

import mixer_bounds as B
import mixer_ref as R


def in_parts(x, parts):
    out, left = torch.zeros_like(x), x
    for _ in range(parts):
        p = left.float().to(torch.bfloat16).double()
        out, left = out + p, left - p
    return out


def chunk(q, k, v, g, scale, h0, score_parts, state_parts):
    """y of a chunk [b, n, heads, d] with a state before it, its factors in so many bf16 parts."""
    q, k, v = (x.double() for x in (q, k, v))
    n = torch.arange(q.shape[1], dtype=torch.float64)
    gap = n[:, None] - n[None, :]
    w = torch.where(gap >= 0, torch.exp(g.double()[:, None, None] * gap.clamp(min=0)), torch.zeros((), dtype=torch.float64))
    p = in_parts(scale * torch.einsum("bihd,bjhd->bhij", q, k) * w, score_parts)
    far = torch.einsum("bihk,bhkv->bihv", q, in_parts(h0.double(), state_parts)) * torch.exp(g.double() * (n[:, None] + 1))[None, :, :, None]
    return (torch.einsum("bhij,bjhv->bihv", p, v) + scale * far).float().to(torch.bfloat16)


@pytest.mark.parametrize("n,d", [(16, 64), (64, 64), (64, 128)])
def test_the_bound_tells_two_parts_from_one(n, d):
    gen = torch.Generator().manual_seed(n + d)
    b, H = 2, 3
    q, k, v = (torch.randn(b, n, H, d, generator=gen).to(torch.bfloat16) for _ in range(3))
    h0, g = torch.randn(b, H, d, d, generator=gen), R.log_decays(H)
    ref, _ = R.linattn(q, k, v, g, d ** -0.5, h0=h0)
    off = lambda scores, states: B.beyond_rounding(chunk(q, k, v, g, d ** -0.5, h0, scores, states), ref)
    assert off(2, 2) < B.SPLIT
    assert off(1, 2) > 2 * B.SPLIT and off(2, 1) > 2 * B.SPLIT
