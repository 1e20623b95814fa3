"""Linear attention on short blocks (with and without states, padded, many at once), and calls whose memory is the hard
part: states updated in place, far offsets, two streams at once.  Reference and tolerances are those of
test_gpu_linattn.py (derived there)."""

import math

import pytest
import torch

import mixer_ref as R
from test_gpu_linattn import DEV, TOL_F32, check, make, r2l, state, tol  # noqa: F401  (r2l is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("L", [16, 17, 33, 64])
def test_padded_short_batch(r2l, L, h0, reverse):
    lens = [0, 1, 15, 16, L // 2, L - 1, L]
    check(r2l, dict(b=7, L=L, H=3, dk=64, dv=64, reverse=reverse, lens=[min(n, L) for n in lens], h0=h0), seed=L)


@pytest.mark.parametrize("dk,dv", [(8, 8), (8, 128), (128, 8), (40, 72), (72, 40), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("L", [5, 32])
def test_head_sizes_of_short_blocks(r2l, dk, dv, L):
    for reverse in (False, True):
        for h0 in (False, True):
            check(r2l, dict(b=2, L=L, H=2, dk=dk, dv=dv, reverse=reverse, h0=h0), seed=dk + dv + L)


@pytest.mark.parametrize("qh,kh,vh", [(4, 1, 1), (1, 4, 2), (2, 2, 4)])
@pytest.mark.parametrize("L", [3, 48])
def test_shared_heads_of_short_blocks(r2l, qh, kh, vh, L):
    for h0 in (False, True):
        check(r2l, dict(b=3, L=L, H=4, qh=qh, kh=kh, vh=vh, dk=64, dv=32, h0=h0, fused=True), seed=qh + L)


@pytest.mark.parametrize("L,d", [(1, 64), (16, 64), (20, 64), (20, 128), (64, 64)])
def test_more_blocks_than_the_gpu_holds_at_once(r2l, L, d):
    # several items for every CTA: 1500 (sequence, head) pairs
    b, H = 75, 20
    q, k, v, g = make(L + d, b, L, H, H, 4, H, d, d, "bf16")
    h0 = state(1, b, H, d, d)
    ref, href = R.linattn(q, k, v, g, d ** -0.5, h0=h0)
    y, h = r2l.r2l_linattn(q, k, v, g, h0=h0, want_h_last=True)
    assert R.rel_err_per_head(y, ref) < tol(q.dtype) and R.rel_err_state(h, href) < TOL_F32
    y, none = r2l.r2l_linattn(q, k, v, g, h0=h0)
    assert none is None and R.rel_err_per_head(y, ref) < tol(q.dtype)
    ref, href = R.linattn(q, k, v, g, d ** -0.5, reverse=True)
    y, h = r2l.r2l_linattn(q, k, v, g, reverse=True, want_h_last=True)
    assert R.rel_err_per_head(y, ref) < tol(q.dtype) and R.rel_err_state(h, href) < TOL_F32
    y, _ = r2l.r2l_linattn(q, k, v, g, reverse=True, block_len=L)
    assert R.rel_err_per_head(y, ref) < tol(q.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,H", [(7, 3), (16, 3), (50, 3), (65, 3), (900, 1)])
def test_states_in_place(r2l, dtype, L, H):
    # 900 tokens of two sequences are divided over the SMs: the parts read the first state while the last is written
    lens = torch.tensor([L, L - 3], dtype=torch.int32, device=DEV)
    q, k, v, g = make(L, 2, L, H, H, H, H, 64, 64, dtype)
    h0 = state(2, 2, H, 64, 64)
    for reverse in (False, True):
        y, h = r2l.r2l_linattn(q, k, v, g, h0=h0, want_h_last=True, seq_lens=lens, reverse=reverse)
        s = h0.clone()
        y2, s2 = r2l.r2l_linattn(q, k, v, g, h0=s, h_last=s, seq_lens=lens, reverse=reverse)
        assert s2 is s and torch.equal(s, h) and torch.equal(y, y2)


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("L", [12, 30])
def test_non_finite_values_stay_in_their_block(r2l, L, bad, with_state):
    b, H, d = 3, 2, 64
    q, k, v, g = make(41, b, L, H, H, H, H, d, d, "bf16")
    h0 = state(3, b, H, d, d) if with_state else None
    n = torch.tensor([L - 5, L, L - 3], dtype=torch.int32, device=DEV)
    for reverse in (False, True):
        kw = dict(h0=h0, seq_lens=n, reverse=reverse)
        want, hw = r2l.r2l_linattn(q, k, v, g, want_h_last=with_state, **kw)
        dy = torch.randn(want.shape, generator=torch.Generator().manual_seed(1)).to(q.dtype).to(DEV)
        gw = r2l.r2l_linattn_bwd(q, k, v, g, dy, **kw)
        assert not want[0, L - 5:].any() and not want[2, L - 3:].any()
        x = [t.clone() for t in (q, k, v, dy)]
        for t in x:
            t[0, L - 5:] = bad
            t[2, L - 3:] = bad
        got, hg = r2l.r2l_linattn(*x[:3], g, want_h_last=with_state, **kw)
        assert torch.equal(got, want) and (hw is None or torch.equal(hg, hw))
        gg = r2l.r2l_linattn_bwd(*x[:3], g, x[3], **kw)
        assert all(torch.equal(gg[m], gw[m]) for m in ("dq", "dk", "dv"))
        # a token that others must not see: a later one in scan order, in k or v of one head
        t = 8
        ahead = slice(t + 1, None) if reverse else slice(0, t)
        for which in (1, 2):
            x = [a.clone() for a in (q, k, v)]
            x[which][1, t, 0] = bad
            got, hg = r2l.r2l_linattn(*x, g, want_h_last=with_state, **kw)
            assert torch.equal(got[1, ahead], want[1, ahead]) and torch.equal(got[1, :, 1], want[1, :, 1])
            assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
            assert not torch.isfinite(got[1, t, 0].float()).all()
            if with_state:
                assert torch.equal(hg[0], hw[0]) and torch.equal(hg[2], hw[2]) and torch.equal(hg[1, 1], hw[1, 1])


@pytest.mark.parametrize("dtype,L", [("bf16", 20), ("bf16", 130), ("f32", 20)])
def test_offsets_past_32_bits(r2l, dtype, L):
    """Tokens far apart: element offsets of 2^32 and byte offsets beyond."""
    H, d, t = 2, 64, torch.bfloat16 if dtype == "bf16" else torch.float32
    far = 2 ** 32 // L + 4096
    far -= far % 8
    buf = torch.empty((L - 1) * far + 3 * H * d, dtype=t, device=DEV)
    x = buf.as_strided((1, L, 3 * H, d), (L * far, far, d, 1))
    x.copy_(torch.randn(1, L, 3 * H, d, generator=torch.Generator().manual_seed(1)).to(t).to(DEV))
    q, k, v = x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:]
    g, h0 = R.log_decays(H).to(DEV), state(2, 1, H, d, d)
    near = [a.contiguous() for a in (q, k, v)]
    for kw in (dict(), dict(h0=h0, want_h_last=True)):
        a, b = r2l.r2l_linattn(q, k, v, g, **kw), r2l.r2l_linattn(*near, g, **kw)
        assert torch.equal(a[0], b[0]) and (a[1] is None or torch.equal(a[1], b[1]))
    dy = torch.randn(1, L, H, d, generator=torch.Generator().manual_seed(3)).to(t).to(DEV)
    a, b = r2l.r2l_linattn_bwd(q, k, v, g, dy), r2l.r2l_linattn_bwd(*near, g, dy)
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv"))
    pos, inv = torch.arange(L, device=DEV), torch.rand(d // 2, generator=torch.Generator().manual_seed(4)).to(DEV)
    a = r2l.r2l_qk_norm_rope(q[0], k[0], None, None, pos, inv)
    b = r2l.r2l_qk_norm_rope(near[0][0], near[1][0], None, None, pos, inv)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_calls_at_once(r2l):
    """Calls on two streams that overlap, each with workspaces of its own, give the bits of the calls one by one."""
    cases = [make(5, 1, 3000, 2, 2, 2, 2, 64, 64, "bf16"), make(6, 2, 1500, 4, 1, 1, 4, 64, 64, "bf16")]
    dys = [torch.randn(*c[2].shape[:2], c[3].shape[0], 64, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)
           for c in cases]

    def run(c, dy):
        y, h = r2l.r2l_linattn(*c, want_h_last=True)
        got = r2l.r2l_linattn_bwd(*c, dy)
        return [y, h, got["dq"], got["dk"], got["dv"]]

    want = [run(c, dy) for c, dy in zip(cases, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cases[i], dys[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_two_graphs_share_a_workspace(r2l):
    """Captured calls that use one workspace (segments' states, shared heads' gradients), replayed in turn."""
    cases = [make(5, 1, 3000, 2, 1, 1, 2, 64, 64, "bf16"), make(6, 2, 1500, 2, 2, 1, 2, 64, 64, "bf16")]
    dys = [torch.randn(*c[2].shape[:2], c[3].shape[0], 64, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)
           for c in cases]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)

    def run(c, dy, **kw):
        y, h = r2l.r2l_linattn(*c, want_h_last=True, **kw)
        g = r2l.r2l_linattn_bwd(*c, dy, **kw)
        return [y, h, g["dq"], g["dk"], g["dv"]]

    want = [run(c, dy) for c, dy in zip(cases, dys)]
    graphs, got = [], []
    for c, dy in zip(cases, dys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(run(c, dy, workspace=ws))
    for i in (0, 1, 0, 1):
        graphs[i].replay()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(r2l.MixerError):
        r2l.r2l_linattn(*cases[0], workspace=small)
    del graphs


def test_binding_refusals(r2l):
    q, k, v, g = make(1, 2, 20, 4, 4, 2, 4, 64, 64, "bf16")
    ok = lambda **kw: r2l.r2l_linattn(q, k, v, g, **kw)
    for bad, err in ((lambda: r2l.r2l_linattn(q, k, v, None), TypeError), (lambda: r2l.r2l_linattn(q, k.float(), v, g), TypeError),
                     (lambda: r2l.r2l_linattn(q.half(), k.half(), v.half(), g), TypeError),
                     (lambda: r2l.r2l_linattn(q, k[..., :32], v, g), ValueError),
                     (lambda: r2l.r2l_linattn(q, k, v.transpose(1, 2), g), ValueError),
                     (lambda: r2l.r2l_linattn(q[:1].expand(2, -1, -1, -1), k, v, g), ValueError),
                     (lambda: r2l.r2l_linattn(q, k, v, g[:3].contiguous()), r2l.MixerError),
                     (lambda: r2l.r2l_linattn(q.cpu(), k, v, g), TypeError),
                     (lambda: ok(h0=torch.zeros(2, 4, 64, 32, device=DEV)), ValueError),
                     (lambda: ok(h0=torch.zeros(2, 4, 64, 64, device=DEV, dtype=torch.bfloat16)), TypeError),
                     (lambda: ok(reverse=True, block_len=6), r2l.MixerError),
                     (lambda: ok(reverse=True, block_len=10, want_h_last=True), r2l.MixerError),
                     (lambda: ok(seq_lens=torch.zeros(2, dtype=torch.int64, device=DEV)), TypeError),
                     (lambda: r2l.r2l_linattn_step(q[:, 0], k[:, 0], v[:, 0], g, None), ValueError),
                     (lambda: r2l.r2l_linattn_bwd(q, k, v, g, None), ValueError),
                     (lambda: r2l.r2l_qk_norm_rope(q[0], k[0], None, None, [1] * 20, torch.ones(32, device=DEV)), TypeError)):
        with pytest.raises(err):
            bad()
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("L,H,kh,dk,dv", [(1300, 2, 1, 64, 48), (2111, 1, 1, 128, 32)])
def test_divided_sequences_of_a_padded_batch(r2l, L, H, kh, dk, dv, dtype, reverse):
    # divided over the SMs; rows that end before, at and inside a segment's first token
    check(r2l, dict(b=4, L=L, H=H, qh=kh, kh=kh, dk=dk, dv=dv, dtype=dtype, reverse=reverse, lens=[0, 193, L // 2, L], h0=True), seed=L)
