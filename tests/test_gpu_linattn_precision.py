"""bf16 linear attention to the precision that its split factors promise (the bound is derived in mixer_bounds.py), and the
gradients of short blocks without a state, which run on kernels of their own: head sizes, shared heads, padding."""

import math

import pytest
import torch

import mixer_bounds as B
import mixer_ref as R
from test_gpu_linattn import DEV, TOL_F32, make, r2l, state  # noqa: F401  (r2l is a fixture)

pytestmark = pytest.mark.gpu


def outputs(r2l, q, k, v, g, ref_kw, **kw):
    scale = q.shape[3] ** -0.5
    ref, href = R.linattn(q, k, v, g, scale, **ref_kw)
    for want in ((False, True) if not (kw.get("reverse") and kw.get("block_len")) else (False,)):
        y, h = r2l.r2l_linattn(q, k, v, g, want_h_last=want, **kw)
        assert B.beyond_rounding(y, ref) < B.SPLIT
        assert not want or R.rel_err_state(h, href) < TOL_F32
    return ref


def gradients(r2l, q, k, v, g, dy, ref_kw, **kw):
    want = R.linattn_grads(q, k, v, g, q.shape[3] ** -0.5, dy, **ref_kw)
    got = r2l.r2l_linattn_bwd(q, k, v, g, dy, **kw)
    for n, w in zip(("dq", "dk", "dv"), want):
        assert got[n].shape == w.shape and B.beyond_rounding(got[n], w) < B.SPLIT, n


def both(r2l, L, d, H, qh=None, kh=None, vh=None, reverse=False, block=None, lens=None, h0=False, b=2, seed=0, fused=False):
    q, k, v, g = make(seed, b, L, H, qh or H, kh or H, vh or H, *d, "bf16", fused)
    s = state(seed + 1, b, H, *d) if h0 else None
    n = torch.tensor(lens, dtype=torch.int32, device=DEV) if lens else None
    ref_kw = dict(reverse=reverse, block=block, lens=lens, h0=s)
    kw = dict(reverse=reverse, block_len=block, seq_lens=n, h0=s)
    ref = outputs(r2l, q, k, v, g, ref_kw, **kw)
    dy = torch.randn(ref.shape, generator=torch.Generator().manual_seed(seed + 2)).to(q.dtype).to(DEV)
    gradients(r2l, q, k, v, g, dy, ref_kw, **kw)
    assert r2l.r2l_mixer_device_status() == r2l.R2L_OK


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("L,d", [(16, (64, 64)), (48, (64, 64)), (30, (128, 128)), (64, (128, 128)), (65, (64, 64)), (130, (128, 128)),
                                 (300, (64, 128)), (300, (128, 64)), (1500, (64, 64))])
def test_split_factors_keep_their_precision(r2l, L, d, h0, reverse):
    both(r2l, L, d, 3, h0=h0, reverse=reverse, seed=L)


@pytest.mark.parametrize("L", [1, 2, 5, 15, 16, 17, 31, 33, 48, 64])
@pytest.mark.parametrize("reverse", [False, True])
def test_short_blocks_of_every_length(r2l, L, reverse):
    both(r2l, L, (64, 64), 3, reverse=reverse, seed=L)
    both(r2l, L, (128, 128), 2, reverse=reverse, seed=L + 1)


@pytest.mark.parametrize("d", [(32, 128), (128, 32), (40, 72), (72, 40), (64, 128), (128, 64), (96, 104)])
@pytest.mark.parametrize("L", [5, 32, 50])
def test_short_blocks_of_head_sizes(r2l, d, L):
    for reverse in (False, True):
        both(r2l, L, d, 2, reverse=reverse, seed=sum(d) + L)


@pytest.mark.parametrize("qh,kh,vh", [(1, 1, 4), (4, 2, 2), (2, 4, 1), (1, 2, 4), (4, 1, 1)])
@pytest.mark.parametrize("L,d", [(7, (64, 64)), (48, (64, 32)), (20, (128, 128)), (64, (40, 128)), (100, (64, 64))])
def test_shared_heads(r2l, qh, kh, vh, L, d):
    for reverse in (False, True):
        both(r2l, L, d, 4, qh, kh, vh, reverse=reverse, fused=True, seed=qh + L)


@pytest.mark.parametrize("L,block,d", [(60, 20, (64, 64)), (64, 16, (128, 128)), (96, 48, (128, 64)), (128, 64, (72, 128)), (14, 1, (64, 64))])
@pytest.mark.parametrize("kh", [1, 4])
def test_blocks_right_to_left(r2l, L, block, d, kh):
    both(r2l, L, d, 4, kh, kh, 4, reverse=True, block=block, b=3, seed=block)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("kh", [1, 4])
@pytest.mark.parametrize("L,d", [(16, (64, 64)), (33, (128, 128)), (64, (64, 128))])
def test_padded_short_batch(r2l, L, d, kh, reverse):
    both(r2l, L, d, 4, kh, kh, kh, reverse=reverse, lens=[0, 1, 15, 16, L // 2, L - 1, L], b=7, seed=L)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("L,d,kh", [(12, 64, 1), (30, 128, 1), (30, 128, 4), (64, 128, 2), (100, 64, 1)])
def test_gradients_past_a_rows_end_and_beside_a_bad_token(r2l, L, d, kh, bad):
    """fp32 parts of shared heads too: what padding holds changes no bit, and a bad token stays with those that see it.

    Short blocks keep the bits of the others.  Chunks (L > 64) sum an output that met a masked bad value again, the same at
    most 64 products in another order, in fp32: each order is off by at most 64 2^-24 of the sum of the terms' sizes, which is
    at most sqrt(64) of their root sum square; 2 * 64 * 2^-24 * 8 = 6.1e-5 of the rms between the two, and half a step of
    rounding on either side."""
    b, H = 3, 4
    q, k, v, g = make(43, b, L, H, kh, kh, kh, d, d, "bf16")
    dy = torch.randn(b, L, H, d, generator=torch.Generator().manual_seed(44)).to(q.dtype).to(DEV)
    lens = torch.tensor([L - 5, L, L - 3], dtype=torch.int32, device=DEV)
    for reverse in (False, True):
        kw = dict(seq_lens=lens, reverse=reverse)
        want = r2l.r2l_linattn_bwd(q, k, v, g, dy, **kw)
        x = [t.clone() for t in (q, k, v, dy)]
        for t in x:
            t[0, L - 5:] = bad
            t[2, L - 3:] = bad
        got = r2l.r2l_linattn_bwd(*x[:3], g, x[3], **kw)
        assert all(torch.equal(got[n], want[n]) for n in ("dq", "dk", "dv"))
        # dq of the tokens before t (in scan order) sees neither k nor v of t; dk and dv of those behind it no q nor dy
        t = 6
        before, behind = (slice(t + 1, None), slice(0, t)) if reverse else (slice(0, t), slice(t + 1, None))
        for which, names, keep in ((1, ("dq",), before), (2, ("dq",), before), (0, ("dk", "dv"), behind), (3, ("dk", "dv"), behind)):
            x = [a.clone() for a in (q, k, v, dy)]
            x[which][1, t, 0] = bad
            got = r2l.r2l_linattn_bwd(*x[:3], g, x[3], **kw)
            for n in names:
                a, w = got[n][1, keep].double(), want[n][1, keep].double()
                if L <= 64:
                    assert torch.equal(a, w), (which, n)
                else:
                    rms = want[n][1].double().square().mean().sqrt()
                    assert bool(((a - w).abs() <= 2 * B.ROUND * w.abs() + 2 * 64 * 2.0 ** -24 * 8 * rms).all()), (which, n)
                assert not torch.isfinite(got[n][1, t, 0].float()).all()
            for n in ("dq", "dk", "dv"):
                assert torch.equal(got[n][0], want[n][0]) and torch.equal(got[n][2], want[n][2])
