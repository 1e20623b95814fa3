"""GPU parity of the per-head norm with the rotary embedding (r2l_qk_norm_rope and its gradients) against fp64.

Tolerances, relative to max(|ref|, rms of the head's outputs), fixed before the first run: fp32 1e-5 (sums of at
most 256 squares, one reciprocal root, a rotation: a few 2^-24 each); bf16 2^-8 for the rounding of the result on
top of that.  Weight gradients (fp32 sums over all tokens and heads): 1e-5 of their norm.
"""

import math

import pytest
import torch

import mixer_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}
DEV = "cuda"


@pytest.fixture(scope="module")
def r2l():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import reverse_mamba_selective_b200 as pkg

    pkg.load_mixer()
    return pkg


def make(seed, n, hq, hk, d, rot, dtype, fused=False, pos_dtype=torch.int64, pos0=0):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    x = torch.randn(n, (hq + 2 * hk) * d, generator=gen).to(t).to(DEV)
    q, k = x[:, : hq * d].view(n, hq, d), x[:, hq * d : (hq + hk) * d].view(n, hk, d)
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = (1 + 0.2 * torch.randn(2, d, generator=gen)).to(DEV)
    pos = (pos0 + torch.randint(0, 1000, (n,), generator=gen)).to(pos_dtype).to(DEV)
    inv = torch.exp(-math.log(1e6) * torch.arange(rot // 2) * 2.0 / max(rot, 1)).float().to(DEV) if rot else None
    dq = torch.randn(n, hq, d, generator=gen).to(t).to(DEV)
    dk = torch.randn(n, hk, d, generator=gen).to(t).to(DEV)
    return q, k, w[0].contiguous(), w[1].contiguous(), pos, inv, dq, dk


def check(r2l, n, hq, hk, d, rot, dtype, inter=False, fused=False, weights=True, seed=0, eps=1e-6, **kw):
    q, k, qw, kw_, pos, inv, dq, dk = make(seed, n, hq, hk, d, rot, dtype, fused, **kw)
    if not weights:
        qw = kw_ = None
    got = r2l.r2l_qk_norm_rope(q, k, qw, kw_, pos if rot else None, inv, eps=eps, interleaved=inter)
    g = r2l.r2l_qk_norm_rope_bwd(q, k, qw, kw_, pos if rot else None, inv, dq, dk, eps=eps, interleaved=inter)
    for x, w, out, dy, name in ((q, qw, got[0], dq, "q"), (k, kw_, got[1], dk, "k")):
        ref = R.norm_rope(x, w, pos, inv, eps, inter)
        assert out.dtype == x.dtype and R.rel_err_per_head(out[None], ref[None]) < TOL[dtype], name
        dx, dw = R.norm_rope_grads(x, w, pos, inv, eps, inter, dy)
        assert R.rel_err_per_head(g["d" + name][None], dx[None]) < TOL[dtype], name
        size = float(dw.norm())
        assert float((g["d" + name + "_weight"].double() - dw).norm()) <= 1e-5 * size, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (256, 256), (80, 80), (96, 48), (128, 64), (32, 8), (10, 6), (2, 2),
                                   (64, 0), (250, 250), (200, 100)])
def test_head_sizes(r2l, dtype, inter, d, rot):
    check(r2l, 37, 3, 2, d, rot, dtype, inter, seed=d + rot)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 64, 593, 2001])
def test_token_counts(r2l, dtype, n):
    check(r2l, n, 4, 1, 64, 64, dtype, seed=n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (16, 8), (7, 3), (40, 1)])
def test_head_counts_in_a_fused_projection(r2l, dtype, hq, hk):
    check(r2l, 45, hq, hk, 128, 128, dtype, fused=True, seed=hq)
    check(r2l, 45, hq, hk, 36, 36, dtype, fused=True, seed=hq)  # single-channel path


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_positions_and_int32(r2l, dtype):
    # fp32 angles would be off by up to a radian at ten million; negative positions rotate backwards
    check(r2l, 50, 2, 2, 128, 128, dtype, pos0=10_000_000)
    check(r2l, 50, 2, 2, 128, 128, dtype, pos0=-3_000_000)
    check(r2l, 50, 2, 2, 128, 128, dtype, pos0=2_000_000_000, pos_dtype=torch.int32)


def test_unit_weights_and_large_eps(r2l):
    check(r2l, 20, 2, 1, 64, 64, "bf16", weights=False)
    check(r2l, 20, 2, 1, 64, 64, "f32", weights=False, eps=0.5)


def test_zero_rows_and_one_operand_without_heads(r2l):
    q, k, qw, kw, pos, inv, dq, dk = make(3, 6, 2, 1, 64, 64, "bf16")
    q[2] = 0
    out, _ = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv)
    assert torch.equal(out[2], torch.zeros_like(out[2]))
    none = k[:, :0].contiguous()
    full = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv)[0]
    only, empty = r2l.r2l_qk_norm_rope(q, none, qw, kw, pos, inv)
    assert torch.equal(only, full) and empty.shape == (6, 0, 64)
    g = r2l.r2l_qk_norm_rope_bwd(q, none, qw, kw, pos, inv, dq, dk[:, :0].contiguous())
    assert torch.equal(g["dk_weight"], torch.zeros_like(kw))
    z = q[:0]
    a, b = r2l.r2l_qk_norm_rope(z, k[:0], qw, kw, pos[:0], inv)
    assert a.shape == (0, 2, 64) and b.shape == (0, 1, 64)
    g = r2l.r2l_qk_norm_rope_bwd(z, k[:0], qw, kw, pos[:0], inv, z, k[:0])
    assert torch.equal(g["dq_weight"], torch.zeros_like(qw)) and torch.equal(g["dk_weight"], torch.zeros_like(kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 36])
def test_in_place_and_strided_outputs(r2l, dtype, d):
    q, k, qw, kw, pos, inv, _, _ = make(4, 33, 4, 2, d, d, dtype, fused=True)
    want = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv)
    out = torch.full((33, 4 * d + 2 * d + 8), 7.0, dtype=q.dtype, device=DEV)
    qo, ko = out[:, : 4 * d].view(33, 4, d), out[:, 4 * d : 6 * d].view(33, 2, d)
    r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert bool((out[:, 6 * d :] == 7.0).all())
    a, b = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv, q_out=q, k_out=k)
    assert a is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_heads(r2l, dtype):
    # a slice that starts off a 16-byte boundary takes the single-channel path, with the same values
    q, k, qw, kw, pos, inv, _, _ = make(5, 19, 2, 1, 64, 64, dtype)
    x = torch.zeros(19, 2 * 64 + 3, dtype=q.dtype, device=DEV)
    x[:, 1 : 1 + 128] = q.reshape(19, 128)
    u = x[:, 1 : 1 + 128].view(19, 2, 64)
    a, b = r2l.r2l_qk_norm_rope(u, k, qw, kw, pos, inv)
    ref = R.norm_rope(u, qw, pos, inv, 1e-6, False)
    assert R.rel_err_per_head(a[None], ref[None]) < TOL[dtype]


def test_gradients_against_differences(r2l):
    n, d = 9, 32
    q, k, qw, kw, pos, inv, dq, dk = make(6, n, 2, 1, d, d, "f32")
    g = r2l.r2l_qk_norm_rope_bwd(q, k, qw, kw, pos, inv, dq, dk)
    gen = torch.Generator().manual_seed(7)
    f = lambda x, w: float((R.norm_rope(x, w, pos, inv, 1e-6, False) * dq.double()).sum())
    u, uw = (torch.randn(s, generator=gen).double().to(DEV) for s in (q.shape, qw.shape))
    e = 1e-6
    slope = (f(q.double() + e * u, qw.double()) - f(q.double() - e * u, qw.double())) / (2 * e)
    assert abs(slope - float((g["dq"].double() * u).sum())) < 1e-4 * float(g["dq"].double().norm())
    slope = (f(q.double(), qw.double() + e * uw) - f(q.double(), qw.double() - e * uw)) / (2 * e)
    assert abs(slope - float((g["dq_weight"].double() * uw).sum())) < 1e-4 * float(g["dq_weight"].double().norm())


def test_non_finite_rows_stay_alone(r2l):
    q, k, qw, kw, pos, inv, dq, dk = make(8, 12, 2, 2, 64, 64, "bf16")
    want = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv)
    gw = r2l.r2l_qk_norm_rope_bwd(q, k, qw, kw, pos, inv, dq, dk)
    q[3, 1] = math.nan
    got = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv)
    keep = torch.ones(12, 2, dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])
    g = r2l.r2l_qk_norm_rope_bwd(q, k, qw, kw, pos, inv, dq, dk)
    assert torch.equal(g["dq"][keep], gw["dq"][keep]) and torch.equal(g["dk_weight"], gw["dk_weight"])


def test_stream_and_graph(r2l):
    q, k, qw, kw, pos, inv, dq, dk = make(9, 700, 4, 2, 128, 128, "bf16")
    want = r2l.r2l_qk_norm_rope(q, k, qw, kw, pos, inv)
    wg = r2l.r2l_qk_norm_rope_bwd(q, k, qw, kw, pos, inv, dq, dk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r2l.r2l_qk_norm_rope_bwd(q, k, qw, kw, pos, inv, dq, dk, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(got[n], wg[n]) for n in wg)
    graph = torch.cuda.CUDAGraph()
    qs = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        a, b = r2l.r2l_qk_norm_rope(qs, k, qw, kw, pos, inv)
        cg = r2l.r2l_qk_norm_rope_bwd(qs, k, qw, kw, pos, inv, dq, dk)
    for _ in range(2):
        qs.copy_(q)
        graph.replay()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert all(torch.equal(cg[n], wg[n]) for n in wg)
    del graph


@pytest.mark.parametrize("n,d", [(40001, 16), (20011, 64), (10007, 20)])
def test_several_tokens_a_group(r2l, n, d):
    # more tokens than the gradient kernel has groups of lanes: each walks over several, the loads running on between them
    check(r2l, n, 3, 1, d, d, "bf16", seed=n)


def test_two_graphs_share_a_workspace(r2l):
    """Two captured gradient calls with one workspace, replayed in turn, give the plain calls' bits."""
    cases = [make(s, n, 4, 2, 64, 64, "bf16") for s, n in ((1, 700), (2, 300))]
    want = [r2l.r2l_qk_norm_rope_bwd(*c) for c in cases]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    graphs, got = [], []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(r2l.r2l_qk_norm_rope_bwd(*c, workspace=ws))
    for i in (0, 1, 0, 1):
        graphs[i].replay()
        assert all(torch.equal(got[i][m], want[i][m]) for m in want[i])
    del graphs
