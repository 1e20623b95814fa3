"""GPU parity of linear attention (r2l_linattn, r2l_linattn_step, r2l_linattn_bwd) against the fp64 recurrence.

Tolerances, relative to max(|ref|, rms of the element's head), fixed before the first run:
  fp32 (outputs, gradients, states of any input type): 1e-5 = 168 half-steps of fp32.  An output is a sum of up
      to 128 L products with about 4 roundings of 2^-24 each on the way; they add like a random walk, as the
      products themselves do, so that relative to the rms about 4 sqrt(2) 2^-24 remain (3e-7), 6 times that for the
      largest of a million elements, and a factor of 5 for sums that are not that random.
  bf16 outputs and gradients: 2^-8 (the rounding of the output) + 6 * 2^-8 / sqrt(3) (a score and a state entry are
      rounded to bf16 at most once before the last product: uniform errors of at most 2^-8 each, on disjoint parts of
      the sum, 6 sigma) = 1.8e-2.
"""

import math

import pytest
import torch

import mixer_ref as R

pytestmark = pytest.mark.gpu

TOL_F32 = 1e-5
TOL_BF16 = 2.0 ** -8 + 6 * 2.0 ** -8 / math.sqrt(3.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


@pytest.fixture(scope="module")
def r2l():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import reverse_mamba_selective_b200 as pkg

    pkg.load_mixer()
    return pkg


def tol(t):
    return TOL_F32 if t == torch.float32 else TOL_BF16


def make(seed, b, L, H, qh, kh, vh, dk, dv, dtype, fused=False):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    n = lambda *s: torch.randn(*s, generator=gen).to(t).to(DEV)
    if fused:  # q, k and v as slices of one projection's output
        w = qh * dk + kh * dk + vh * dv
        x = n(b, L, w + 16)
        q = x[..., : qh * dk].view(b, L, qh, dk)
        k = x[..., qh * dk : (qh + kh) * dk].view(b, L, kh, dk)
        v = x[..., (qh + kh) * dk : w].view(b, L, vh, dv)
    else:
        q, k, v = n(b, L, qh, dk), n(b, L, kh, dk), n(b, L, vh, dv)
    return q, k, v, R.log_decays(H).to(DEV)


def state(seed, b, H, dk, dv):
    return torch.randn(b, H, dk, dv, generator=torch.Generator().manual_seed(seed)).to(DEV)


def check(r2l, case, seed=0, g=None):
    c = dict(b=1, L=1, H=2, qh=None, kh=None, vh=None, dk=64, dv=64, dtype="bf16", reverse=False, block=None, lens=None,
             h0=False, fused=False)
    c.update(case)
    H = c["H"]
    q, k, v, gg = make(seed, c["b"], c["L"], H, c["qh"] or H, c["kh"] or H, c["vh"] or H, c["dk"], c["dv"], c["dtype"], c["fused"])
    g = gg if g is None else g
    whole = not (c["reverse"] and c["block"] and c["block"] != c["L"])
    h0 = state(seed + 1, c["b"], H, c["dk"], c["dv"]) if c["h0"] else None
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=DEV) if c["lens"] else None
    scale = c["dk"] ** -0.5
    kw = dict(reverse=c["reverse"], block_len=c["block"], seq_lens=lens, h0=h0)
    y, h = r2l.r2l_linattn(q, k, v, g, want_h_last=whole, **kw)
    ref, href = R.linattn(q, k, v, g, scale, c["reverse"], c["block"], c["lens"], h0)
    assert y.shape == ref.shape and y.dtype == q.dtype
    assert R.rel_err_per_head(y, ref) < tol(q.dtype)
    if whole:
        assert R.rel_err_state(h, href) < TOL_F32
    # without the final state the outputs are the same operator's
    y2, none = r2l.r2l_linattn(q, k, v, g, **kw)
    assert none is None and R.rel_err_per_head(y2, ref) < tol(q.dtype)
    # gradients
    dy = torch.randn(ref.shape, generator=torch.Generator().manual_seed(seed + 2)).to(q.dtype).to(DEV)
    dh = 0.1 * state(seed + 3, c["b"], H, c["dk"], c["dv"]) if whole else None
    got = r2l.r2l_linattn_bwd(q, k, v, g, dy, dh_last=dh, **kw)
    want = R.linattn_grads(q, k, v, g, scale, dy, c["reverse"], c["block"], c["lens"], h0, dh)
    for name, w in zip(("dq", "dk", "dv"), want):
        assert got[name].dtype == q.dtype and got[name].shape == w.shape
        assert R.rel_err_per_head(got[name], w) < tol(q.dtype), name
    if c["h0"]:
        assert R.rel_err_state(got["dh0"], want[3]) < TOL_F32
    else:
        assert got["dh0"] is None
    assert r2l.r2l_mixer_device_status() == r2l.R2L_OK


LENGTHS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 257]


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("reverse", [False, True])
def test_lengths(r2l, L, reverse):
    check(r2l, dict(b=2, L=L, H=3, dk=64, dv=64, reverse=reverse, h0=L % 2 == 1), seed=L)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (8, 8), (96, 40), (16, 120), (72, 104), (120, 8)])
@pytest.mark.parametrize("L", [5, 70, 150])
def test_head_sizes(r2l, dk, dv, L):
    check(r2l, dict(b=1, L=L, H=2, dk=dk, dv=dv, h0=True), seed=dk + dv)
    check(r2l, dict(b=1, L=L, H=2, dk=dk, dv=dv, reverse=True), seed=dk + dv + 1)


@pytest.mark.parametrize("qh,kh,vh", [(1, 1, 4), (4, 2, 2), (2, 4, 1), (1, 2, 4), (4, 1, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_heads(r2l, qh, kh, vh, dtype):
    check(r2l, dict(b=2, L=90, H=4, qh=qh, kh=kh, vh=vh, dk=40, dv=64, dtype=dtype, h0=True), seed=qh * 100 + kh * 10 + vh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,block", [(64, 16), (64, 32), (128, 64), (60, 20), (48, 1), (195, 65), (300, 100), (260, 130)])
def test_reverse_blocks(r2l, L, block, dtype):
    check(r2l, dict(b=3, L=L, H=2, dk=64, dv=48, dtype=dtype, reverse=True, block=block), seed=block)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_padded_batch(r2l, dtype, reverse):
    check(r2l, dict(b=7, L=150, H=2, dk=64, dv=64, dtype=dtype, reverse=reverse, lens=[0, 1, 63, 64, 65, 149, 150], h0=True),
          seed=5)


@pytest.mark.parametrize("L", [1, 3, 8, 9, 70, 200])
@pytest.mark.parametrize("dk,dv", [(64, 64), (4, 4), (100, 36), (128, 128), (20, 124)])
def test_fp32(r2l, L, dk, dv):
    check(r2l, dict(b=2, L=L, H=2, dk=dk, dv=dv, dtype="f32", h0=True), seed=L + dk)
    check(r2l, dict(b=2, L=L, H=2, dk=dk, dv=dv, dtype="f32", reverse=True), seed=L + dk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
def test_fused_projection_slices(r2l, dtype, reverse):
    check(r2l, dict(b=2, L=130, H=4, qh=2, kh=2, dk=64, dv=32, dtype=dtype, fused=True, reverse=reverse), seed=11)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [5, 140])
def test_extreme_decays(r2l, dtype, L):
    # gamma = 0, gamma = 1, a decay that reaches the denormals within a chunk, and a very slow one
    g = torch.tensor([-math.inf, 0.0, -30.0, -1e-5, -3.4e38], dtype=torch.float32, device=DEV)
    check(r2l, dict(b=1, L=L, H=5, dk=32, dv=32, dtype=dtype, h0=True), seed=3, g=g)
    check(r2l, dict(b=1, L=L, H=5, dk=32, dv=32, dtype=dtype, reverse=True), seed=4, g=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequence_of_few_heads(r2l, dtype):
    # one sequence, two heads: divided over the SMs; a slow head keeps what thousands of tokens left behind
    g = torch.tensor([-1e-4, -0.02], dtype=torch.float32, device=DEV)
    check(r2l, dict(b=1, L=3001, H=2, dk=64, dv=64, dtype=dtype, h0=True), seed=8, g=g)
    check(r2l, dict(b=1, L=3001, H=2, dk=64, dv=64, dtype=dtype, reverse=True, lens=[2900]), seed=9, g=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,H,qh,dk,dv", [(1, 2, 2, 128, 128), (5, 4, 1, 64, 40), (33, 3, 3, 96, 64)])
def test_step_continues_the_sequence(r2l, dtype, b, H, qh, dk, dv):
    q, k, v, g = make(21, b, 5, H, qh, qh, H, dk, dv, dtype)
    h0 = state(22, b, H, dk, dv)
    ref, href = R.linattn(q, k, v, g, dk ** -0.5, h0=h0)
    h = h0.clone()
    ys = []
    for t in range(5):
        if t == 2:  # out of place
            h2 = torch.empty_like(h)
            before = h.clone()
            ys.append(r2l.r2l_linattn_step(q[:, t], k[:, t], v[:, t], g, h, h_out=h2))
            assert torch.equal(h, before)
            h = h2
        else:
            ys.append(r2l.r2l_linattn_step(q[:, t], k[:, t], v[:, t], g, h))
    assert R.rel_err_per_head(torch.stack(ys, 1), ref) < tol(q.dtype)
    assert R.rel_err_state(h, href) < TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_block_then_steps(r2l, dtype):
    # as a server uses them: prompt -> state, a block resumed from it in place, then single tokens
    b, H, dk, dv = 2, 3, 64, 64
    q, k, v, g = make(31, b, 90, H, H, H, H, dk, dv, dtype)
    ref, href = R.linattn(q, k, v, g, dk ** -0.5)
    y1, h = r2l.r2l_linattn(q[:, :70].contiguous(), k[:, :70].contiguous(), v[:, :70].contiguous(), g, want_h_last=True)
    y2, h2 = r2l.r2l_linattn(q[:, 70:86].contiguous(), k[:, 70:86].contiguous(), v[:, 70:86].contiguous(), g, h0=h, h_last=h)
    assert h2 is h
    ys = [y1, y2] + [r2l.r2l_linattn_step(q[:, t], k[:, t], v[:, t], g, h)[:, None] for t in range(86, 90)]
    assert R.rel_err_per_head(torch.cat(ys, 1), ref) < tol(q.dtype)
    assert R.rel_err_state(h, href) < TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_values_stay_where_they_belong(r2l, dtype, bad):
    """Padding behind a row, later tokens, other rows, blocks and heads do not reach an output."""
    b, L, H, d = 3, 150, 2, 64
    q, k, v, g = make(41, b, L, H, H, H, H, d, d, dtype)
    lens = [70, 150, 100]
    want, hwant = r2l.r2l_linattn(q, k, v, g, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), want_h_last=True)
    dy = torch.randn(want.shape, generator=torch.Generator().manual_seed(1)).to(q.dtype).to(DEV)
    gw = r2l.r2l_linattn_bwd(q, k, v, g, dy, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    q2, k2, v2, dy2 = q.clone(), k.clone(), v.clone(), dy.clone()
    for x in (q2, k2, v2, dy2):  # behind the rows
        x[0, 70:] = bad
        x[2, 100:] = bad
    got, hgot = r2l.r2l_linattn(q2, k2, v2, g, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), want_h_last=True)
    assert torch.equal(got, want) and torch.equal(hgot, hwant)
    gg = r2l.r2l_linattn_bwd(q2, k2, v2, g, dy2, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    for n in ("dq", "dk", "dv"):
        assert torch.equal(gg[n], gw[n])
    # a later token of the same sequence (in the same group of 64), another head, another row
    full, _ = r2l.r2l_linattn(q, k, v, g)
    for which in (1, 2):
        q3, k3, v3 = q.clone(), k.clone(), v.clone()
        (q3, k3, v3)[which][1, 90, 0] = bad
        out, _ = r2l.r2l_linattn(q3, k3, v3, g)
        assert torch.equal(out[1, :90], full[1, :90]) and torch.equal(out[1, :, 1], full[1, :, 1])
        assert torch.equal(out[0], full[0]) and torch.equal(out[2], full[2])
        assert not torch.isfinite(out[1, 90, 0].float()).all()
    # blocks, right to left
    blk, _ = r2l.r2l_linattn(q, k, v, g, reverse=True, block_len=30)
    k3, v3 = k.clone(), v.clone()
    k3[1, 31, 0] = bad
    v3[1, 31, 0] = bad
    out, _ = r2l.r2l_linattn(q, k3, v3, g, reverse=True, block_len=30)
    keep = torch.ones(L, dtype=torch.bool)
    keep[30:32] = False
    assert torch.equal(out[:, keep], blk[:, keep]) and torch.equal(out[0], blk[0]) and torch.equal(out[2], blk[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(r2l, dtype):
    """d/de of the sum of y . dy + h_last . dh along random directions, by central differences of the fp64 operator."""
    b, L, H, d = 1, 70, 2, 16
    q, k, v, g = make(51, b, L, H, H, H, H, d, d, dtype)
    h0 = state(52, b, H, d, d)
    dy = torch.randn(b, L, H, d, generator=torch.Generator().manual_seed(53)).to(q.dtype).to(DEV)
    dh = state(54, b, H, d, d)
    got = r2l.r2l_linattn_bwd(q, k, v, g, dy, h0=h0, dh_last=dh)
    gen = torch.Generator().manual_seed(55)

    def value(qq, kk, vv, hh):
        y, h = R.linattn(qq, kk, vv, g, d ** -0.5, h0=hh)
        return float((y * dy.double()).sum() + (h * dh.double()).sum())

    base = [x.double() for x in (q, k, v, h0)]
    for i, name in enumerate(("dq", "dk", "dv", "dh0")):
        u = torch.randn(base[i].shape, generator=gen).double().to(DEV)
        e = 1e-5
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + e * u, base[i] - e * u
        slope = (value(*hi) - value(*lo)) / (2 * e)
        inner = float((got[name].double() * u).sum())
        size = float(got[name].double().norm() * u.norm()) / math.sqrt(u.numel())
        # rounding: at most 2^-8 an element (two in bf16 before it), random over the sum: 6 sigma of its 2-norm
        assert abs(slope - inner) < (6 * 3 * 2.0 ** -8 if dtype == "bf16" and name != "dh0" else 1e-4) * size, name


def test_other_stream_and_graph(r2l):
    """Calls on a side stream, and a captured sequence of calls replayed on new inputs, give the plain calls' bits."""
    b, L, H, d = 2, 200, 2, 64
    q, k, v, g = make(61, b, L, H, 1, 1, H, d, d, "bf16")
    dy = torch.randn(b, L, H, d, generator=torch.Generator().manual_seed(62)).to(q.dtype).to(DEV)
    want = r2l.r2l_linattn(q, k, v, g, want_h_last=True)
    wg = r2l.r2l_linattn_bwd(q, k, v, g, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r2l.r2l_linattn(q, k, v, g, want_h_last=True, stream=s)
    gg = r2l.r2l_linattn_bwd(q, k, v, g, dy, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, w in zip(got, want):
        assert torch.equal(a, w)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(gg[n], wg[n])
    graph = torch.cuda.CUDAGraph()
    qs, ks, vs = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    with torch.cuda.graph(graph):
        cy, ch = r2l.r2l_linattn(qs, ks, vs, g, want_h_last=True)
        cg = r2l.r2l_linattn_bwd(qs, ks, vs, g, dy)
        one = r2l.r2l_linattn_step(qs[:, 0], ks[:, 0], vs[:, 0], g, ch)
    for _ in range(2):
        qs.copy_(q), ks.copy_(k), vs.copy_(v)
        graph.replay()
        assert torch.equal(cy, want[0])
        for n in ("dq", "dk", "dv"):
            assert torch.equal(cg[n], wg[n])
    h = want[1].clone()
    assert torch.equal(one, r2l.r2l_linattn_step(q[:, 0], k[:, 0], v[:, 0], g, h)) and torch.equal(ch, h)
    del graph


def test_same_results_every_time(r2l):
    q, k, v, g = make(71, 2, 1000, 2, 1, 1, 2, 128, 128, "bf16")
    dy = torch.randn(2, 1000, 2, 128, generator=torch.Generator().manual_seed(72)).to(q.dtype).to(DEV)
    first = r2l.r2l_linattn(q, k, v, g, want_h_last=True), r2l.r2l_linattn_bwd(q, k, v, g, dy)
    for _ in range(3):
        again = r2l.r2l_linattn(q, k, v, g, want_h_last=True), r2l.r2l_linattn_bwd(q, k, v, g, dy)
        assert all(torch.equal(a, b) for a, b in zip(first[0], again[0]))
        assert all(torch.equal(first[1][n], again[1][n]) for n in ("dq", "dk", "dv"))


def test_empty(r2l):
    g = R.log_decays(2).to(DEV)
    z = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)
    y, h = r2l.r2l_linattn(z(0, 5, 2, 8), z(0, 5, 2, 8), z(0, 5, 2, 8), g, want_h_last=True)
    assert y.shape == (0, 5, 2, 8) and h.shape == (0, 2, 8, 8)
    h0 = state(1, 3, 2, 8, 16)
    y, h = r2l.r2l_linattn(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 16), g, h0=h0, want_h_last=True)
    assert y.shape == (3, 0, 2, 16) and torch.equal(h, h0)
    y, h = r2l.r2l_linattn(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 16), g, want_h_last=True)
    assert torch.equal(h, torch.zeros_like(h0))
    got = r2l.r2l_linattn_bwd(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 16), g, z(3, 0, 2, 16), h0=h0, dh_last=h0)
    assert torch.equal(got["dh0"], h0)


def test_whole_mixer_step(r2l):
    """The two operators as a layer uses them: fused projection -> norm and rotation in place -> attention -> gradients."""
    b, L, H, kh, d = 2, 100, 4, 2, 64
    gen = torch.Generator().manual_seed(81)
    qkv = torch.randn(b, L, (H + 2 * kh) * d, generator=gen).to(torch.bfloat16).to(DEV)
    q = qkv[..., : H * d].view(b * L, H, d)
    k = qkv[..., H * d : (H + kh) * d].view(b * L, kh, d)
    v = qkv[..., (H + kh) * d :].view(b, L, kh, d)
    w = (1 + 0.1 * torch.randn(2, d, generator=gen)).to(DEV)
    pos = torch.arange(L, device=DEV).repeat(b)
    inv = torch.exp(-math.log(1e4) * torch.arange(d // 2, device=DEV) * 2 / d).float()
    g = R.log_decays(H).to(DEV)
    q0, k0 = q.clone(), k.clone()
    nq, nk = r2l.r2l_qk_norm_rope(q, k, w[0].contiguous(), w[1].contiguous(), pos, inv)
    y, _ = r2l.r2l_linattn(nq.view(b, L, H, d), nk.view(b, L, kh, d), v, g)
    dy = torch.randn(b, L, H, d, generator=gen).to(torch.bfloat16).to(DEV)
    ga = r2l.r2l_linattn_bwd(nq.view(b, L, H, d), nk.view(b, L, kh, d), v, g, dy)
    gn = r2l.r2l_qk_norm_rope_bwd(q, k, w[0].contiguous(), w[1].contiguous(), pos, inv, ga["dq"].view(b * L, H, d),
                                  ga["dk"].view(b * L, kh, d))
    assert torch.equal(q, q0) and torch.equal(k, k0)
    # the chain with each stored tensor rounded where the layer stores it
    rq, rk = R.norm_rope(q, w[0], pos, inv, 1e-6, False), R.norm_rope(k, w[1], pos, inv, 1e-6, False)
    assert R.rel_err_per_head(nq[None], rq[None]) < 2.0 ** -8 + 1e-5
    ref, _ = R.linattn(nq.view(b, L, H, d), nk.view(b, L, kh, d), v, g, d ** -0.5)
    assert R.rel_err_per_head(y, ref) < TOL_BF16
    want = R.linattn_grads(nq.view(b, L, H, d), nk.view(b, L, kh, d), v, g, d ** -0.5, dy)
    assert R.rel_err_per_head(ga["dv"], want[2]) < TOL_BF16
    dq, dqw = R.norm_rope_grads(q, w[0], pos, inv, 1e-6, False, ga["dq"].view(b * L, H, d))
    assert R.rel_err_per_head(gn["dq"][None], dq[None]) < 2.0 ** -8 + 1e-5
    assert float((gn["dq_weight"].double() - dqw).norm() / dqw.norm()) < 1e-5
