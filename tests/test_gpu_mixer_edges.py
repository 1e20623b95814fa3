"""The mixer's operators at the edges of what their documentation allows: sums over nothing, infinite states, streams that
the outputs are made for, the longest rows.  Reference and tolerances are those of test_gpu_linattn.py."""

import pytest
import torch

import mixer_ref as R
from test_gpu_linattn import DEV, TOL_F32, TYPES, make, r2l, state, tol  # noqa: F401  (r2l is a fixture)

pytestmark = pytest.mark.gpu


def dirty(*sizes):
    """Leaves blocks full of ones with the allocator, so that memory that is not written shows."""
    blocks = [torch.ones(max(n, 1), device=DEV) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,H", [(0, 64, 2), (64, 0, 2), (0, 0, 2), (64, 64, 0)])
def test_sums_over_nothing_are_zero(r2l, dtype, dk, dv, H):
    b, L, t = 2, 70, TYPES[dtype]
    q, k = (torch.ones(b, L, 2, dk, dtype=t, device=DEV) for _ in range(2))
    v = torch.ones(b, L, 2, dv, dtype=t, device=DEV)
    g = R.log_decays(H).to(DEV)
    h0 = torch.ones(b, H, dk, dv, device=DEV)
    zeros = lambda x: x is not None and torch.equal(x, torch.zeros_like(x))
    dirty(b * L * 64, b * L * 128)
    y, h = r2l.r2l_linattn(q, k, v, g, h0=h0, want_h_last=True)
    assert y.shape == (b, L, H, dv) and zeros(y) and h.shape == (b, H, dk, dv)
    y = torch.ones(b, L, H, dv, dtype=t, device=DEV)
    assert zeros(r2l.r2l_linattn(q, k, v, g, reverse=True, block_len=10, y=y)[0])
    y = torch.ones(b, H, dv, dtype=t, device=DEV)
    assert zeros(r2l.r2l_linattn_step(q[:, 0], k[:, 0], v[:, 0], g, h0, y=y))
    dirty(b * L * 64, b * L * 128)
    got = r2l.r2l_linattn_bwd(q, k, v, g, torch.ones(b, L, H, dv, dtype=t, device=DEV), h0=h0)
    assert zeros(got["dq"]) and zeros(got["dk"]) and zeros(got["dv"]) and got["dh0"].shape == h0.shape


def test_rows_of_more_pieces_than_32_bits_count(r2l):
    """A short sequence in a row of 2^27 tokens and more: 2^31 16-byte pieces of zeros stand behind it."""
    L, n, d = 2 ** 27 + 2 ** 20, 100, 128
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    gen = torch.Generator().manual_seed(1)
    first = [torch.randn(1, n, 1, w, generator=gen).to(torch.bfloat16).to(DEV) for w in (8, 8, d)]
    g = torch.tensor([-0.1], device=DEV)
    want = r2l.r2l_linattn(*first, g)[0]
    q, k, v = (torch.empty(1, L, 1, w, dtype=torch.bfloat16, device=DEV) for w in (8, 8, d))  # what padding holds does not count
    for x, f in zip((q, k, v), first):
        x[:, :n] = f
    y = torch.ones(1, L, 1, d, dtype=torch.bfloat16, device=DEV)
    r2l.r2l_linattn(q, k, v, g, seq_lens=torch.tensor([n], dtype=torch.int32, device=DEV), y=y)
    # two results, each rounded by half a step at most
    assert R.rel_err_per_head(y[:, :n], want) <= 2 * 2.0 ** -8
    bits = y[:, n:].view(torch.int32)
    assert int(bits.amax()) == int(bits.amin()) == 0
    del q, k, v, y, bits
    torch.cuda.empty_cache()


def same_with_infinities(got, ref, err, bound):
    """The reference's infinities, signs and all, where it has them, and its values within the bound elsewhere."""
    got, ref = got.double(), ref.double()
    assert not ref.isnan().any()
    at = ref.isinf()
    assert torch.equal(got[at], ref[at]) and torch.isfinite(got[~at]).all()
    zero = torch.zeros_like(ref)
    assert err(torch.where(at, zero, got), torch.where(at, zero, ref)) < bound


def infinite_state(seed, b, H, d):
    s = state(seed, b, H, d, d)
    s[:, :, 3, 5] = float("inf")
    s[:, :, 7, 9] = -float("inf")
    return s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("L,d", [(1, 64), (16, 64), (40, 64), (40, 128), (70, 128), (200, 64), (2500, 64)])
def test_an_infinite_state_stays_infinite(r2l, L, d, dtype, reverse):
    # a decay of 1 (a second part of zero), and some whose fp32 rounding lies below and above them
    g = torch.tensor([0.0, -1e-4, -0.02, -0.1], device=DEV)
    H = len(g)
    q, k, v, _ = make(L + d, 1, L, H, H, H, H, d, d, dtype)
    h0, dh = infinite_state(1, 1, H, d), infinite_state(2, 1, H, d)
    y, h = r2l.r2l_linattn(q, k, v, g, h0=h0, want_h_last=True, reverse=reverse)
    ref, href = R.linattn(q, k, v, g, d ** -0.5, reverse, h0=h0)
    same_with_infinities(h, href, R.rel_err_state, TOL_F32)
    same_with_infinities(y, ref, R.rel_err_per_head, tol(q.dtype))
    dy = torch.randn(ref.shape, generator=torch.Generator().manual_seed(3)).to(q.dtype).to(DEV)
    got = r2l.r2l_linattn_bwd(q, k, v, g, dy, h0=h0, dh_last=dh, reverse=reverse)
    want = R.linattn_grads(q, k, v, g, d ** -0.5, dy, reverse, h0=h0, dh_last=dh)
    same_with_infinities(got["dh0"], want[3], R.rel_err_state, TOL_F32)
    for n, w in zip(("dq", "dk", "dv"), want):
        same_with_infinities(got[n], w, R.rel_err_per_head, tol(q.dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinite_state_stays_infinite_in_steps(r2l, dtype):
    g = torch.tensor([0.0, -1e-4, -0.02, -0.1, -3.0], device=DEV)
    H, d = len(g), 64
    q, k, v, _ = make(4, 2, 5, H, H, H, H, d, d, dtype)
    h = infinite_state(5, 2, H, d)
    ref, href = R.linattn(q, k, v, g, d ** -0.5, h0=h)
    y = torch.stack([r2l.r2l_linattn_step(q[:, t], k[:, t], v[:, t], g, h) for t in range(5)], 1)
    same_with_infinities(h, href, R.rel_err_state, TOL_F32)
    same_with_infinities(y, ref, R.rel_err_per_head, tol(q.dtype))


def side_calls(r2l, seed, stream):
    """Every entry point that makes its outputs, as a call on the given stream that returns them."""
    b, L, H, d = 2, 700, 2, 64
    q, k, v, g = make(seed, b, L, H, 1, 1, H, d, d, "bf16")
    dy = torch.randn(b, L, H, d, generator=torch.Generator().manual_seed(seed)).to(q.dtype).to(DEV)
    h = state(seed, b, H, d, d)
    pos, inv = torch.arange(L, device=DEV), torch.rand(d // 2, generator=torch.Generator().manual_seed(seed)).to(DEV)
    h2, one = torch.empty_like(h), dy[0, :, :1].contiguous()
    return [lambda: list(r2l.r2l_linattn(q, k, v, g, want_h_last=True, stream=stream)),
            lambda: [t for t in r2l.r2l_linattn_bwd(q, k, v, g, dy, h0=h, stream=stream).values()],
            lambda: [r2l.r2l_linattn_step(q[:, 0], k[:, 0], v[:, 0], g, h, h_out=h2, stream=stream)],
            lambda: list(r2l.r2l_qk_norm_rope(q[0], k[0], None, None, pos, inv, stream=stream)),
            lambda: [t for t in r2l.r2l_qk_norm_rope_bwd(q[0], k[0], None, None, pos, inv, one, one, stream=stream).values()]]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("raw", [False, True])
def test_outputs_for_another_stream_take_none_of_this_ones_memory(r2l, which, raw):
    """A block that this stream has freed, with work on it still to come, is not what a call on another stream writes."""
    s = torch.cuda.Stream()
    call = side_calls(r2l, 1, s.cuda_stream if raw else s)[which]
    want = [t.clone() for t in side_calls(r2l, 1, None)[which]()]
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want] + [1 << 19, 1 << 20]
    held = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes]
    kept = [torch.zeros_like(t) for t in held]
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(200_000_000)
    for a, t in zip(kept, held):
        a.copy_(t)
    del held, t  # freed here, read by this stream after its sleep
    got = call()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    assert all(bool((a == 7).all()) for a in kept)


@pytest.mark.parametrize("which", range(5))
def test_outputs_of_another_stream_last_as_long_as_this_one_reads_them(r2l, which):
    s = torch.cuda.Stream()
    first, second = side_calls(r2l, 1, s)[which], side_calls(r2l, 2, s)[which]
    want = [t.clone() for t in side_calls(r2l, 1, None)[which]()]
    s.wait_stream(torch.cuda.current_stream())
    got = first()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]
    del got  # read by this stream after its sleep
    for _ in range(3):
        second()
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(copies, want))


def test_another_stream_within_a_capture(r2l):
    s = torch.cuda.Stream()
    calls, want = side_calls(r2l, 3, s), [[t.clone() for t in c()] for c in side_calls(r2l, 3, None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = [c() for c in calls]
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for x, y in zip(got, want) for a, w in zip(x, y))
    del graph


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 20, 90, 700])
def test_a_scale_outputs_and_workspaces_of_the_caller(r2l, dtype, L):
    b, H, d, scale = 2, 2, 64, -0.7
    q, k, v, g = make(L, b, L, H, H, 1, H, d, d, dtype)
    h0, dh = state(1, b, H, d, d), state(2, b, H, d, d)
    ref, href = R.linattn(q, k, v, g, scale, h0=h0)
    y, h = torch.empty(b, L, H, d, dtype=q.dtype, device=DEV), torch.empty_like(h0)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    keep = h0.clone()
    a, c = r2l.r2l_linattn(q, k, v, g, scale=scale, h0=h0, h_last=h, y=y, workspace=ws)
    assert a is y and c is h and torch.equal(h0, keep)
    assert R.rel_err_per_head(y, ref) < tol(q.dtype) and R.rel_err_state(h, href) < TOL_F32
    dy = torch.randn(ref.shape, generator=torch.Generator().manual_seed(3)).to(q.dtype).to(DEV)
    got = r2l.r2l_linattn_bwd(q, k, v, g, dy, scale=scale, dh_last=dh, want_dh0=True, workspace=ws)  # from a state of zeros
    want = R.linattn_grads(q, k, v, g, scale, dy, dh_last=dh)
    for n, w in zip(("dq", "dk", "dv"), want):
        assert R.rel_err_per_head(got[n], w) < tol(q.dtype), n
    assert R.rel_err_state(got["dh0"], want[3]) < TOL_F32
    assert r2l.r2l_linattn_bwd(q, k, v, g, dy, scale=scale, h0=h0, want_dh0=False)["dh0"] is None
    one = r2l.r2l_linattn_step(q[:, 0], k[:, 0], v[:, 0], g, h0.clone(), scale=scale)
    assert R.rel_err_per_head(one[:, None], R.linattn(q[:, :1], k[:, :1], v[:, :1], g, scale, h0=h0)[0]) < tol(q.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("L", [20, 90, 1500])
def test_lengths_outside_the_row_are_clamped(r2l, L, reverse, dtype):
    b, H, d = 4, 2, 64
    q, k, v, g = make(L, b, L, H, H, H, H, d, d, dtype)
    h0 = state(1, b, H, d, d)
    lens = lambda *n: torch.tensor(n, dtype=torch.int32, device=DEV)
    dy = torch.randn(b, L, H, d, generator=torch.Generator().manual_seed(3)).to(q.dtype).to(DEV)

    def run(n):
        g2 = r2l.r2l_linattn_bwd(q, k, v, g, dy, h0=h0, seq_lens=n, reverse=reverse)
        return [*r2l.r2l_linattn(q, k, v, g, h0=h0, want_h_last=True, seq_lens=n, reverse=reverse), *g2.values()]

    far, near = run(lens(-2 ** 31, -1, 2 ** 31 - 1, L + 1)), run(lens(0, 0, L, L))
    assert all(torch.equal(a, c) for a, c in zip(far, near))


def test_lengths_are_read_at_every_replay(r2l):
    b, L, H, d = 3, 130, 2, 64
    q, k, v, g = make(5, b, L, H, H, H, H, d, d, "bf16")
    n = torch.tensor([L, L, L], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = r2l.r2l_linattn(q, k, v, g, seq_lens=n, want_h_last=True)
    for lens in ([1, 70, 130], [0, 129, 64], [130, 5, 65]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want = r2l.r2l_linattn(q, k, v, g, seq_lens=n, want_h_last=True)
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    del graph


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq,hk,d", [(1, 300, 0, 64), (2, 0, 257, 64), (3, 1, 200, 20), (70000, 1, 1, 8), (1, 1, 1, 256)])
def test_many_heads_or_tokens_of_the_norm(r2l, n, hq, hk, d, dtype):
    gen = torch.Generator().manual_seed(n)
    t = TYPES[dtype]
    x = [torch.randn(n, h, d, generator=gen).to(t).to(DEV) for h in (hq, hk, hq, hk)]
    pos, inv = torch.arange(n, device=DEV), torch.rand(d // 2, generator=gen).to(DEV)
    w = torch.rand(d, generator=gen).to(DEV)
    out = r2l.r2l_qk_norm_rope(x[0], x[1], w, None, pos, inv)
    got = r2l.r2l_qk_norm_rope_bwd(x[0], x[1], w, None, pos, inv, x[2], x[3])
    bound = 1e-5 if dtype == "f32" else 2.0 ** -8 + 1e-5
    for i, (name, wt) in enumerate((("q", w), ("k", None))):
        if x[i].shape[1] == 0:
            assert not got[f"d{name}_weight"].any()
            continue
        ref = R.norm_rope(x[i], wt, pos, inv, 1e-6, False)
        dx, dw = R.norm_rope_grads(x[i], wt, pos, inv, 1e-6, False, x[2 + i])
        assert R.rel_err_per_head(out[i][None], ref[None]) < bound
        assert R.rel_err_per_head(got[f"d{name}"][None], dx[None]) < bound
        assert float((got[f"d{name}_weight"].double() - dw).norm()) <= 1e-5 * float(dw.norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_heads_off_their_16_byte_boundaries(r2l, dtype):
    # every operand dense, one element into its storage
    n, h, d = 33, 3, 64
    gen = torch.Generator().manual_seed(9)
    off = lambda *s: torch.randn(1 + torch.Size(s).numel(), generator=gen).to(TYPES[dtype]).to(DEV)[1:].view(*s)
    q, k, dq, dk = (off(n, h, d) for _ in range(4))
    w = torch.rand(d + 1, generator=gen).to(DEV)[1:]
    pos, inv = torch.arange(n + 1, device=DEV)[1:], torch.rand(d // 2 + 1, generator=gen).to(DEV)[1:]
    args = lambda f: [f(q), f(k), f(w), f(w), f(pos), f(inv)]
    same, copy = (lambda t: t), (lambda t: t.clone())
    for a, c in zip(r2l.r2l_qk_norm_rope(*args(same)), (R.norm_rope(t, w, pos, inv, 1e-6, False) for t in (q, k))):
        assert R.rel_err_per_head(a[None], c[None]) < (1e-5 if dtype == "f32" else 2.0 ** -8 + 1e-5)
    a = r2l.r2l_qk_norm_rope_bwd(*args(same), dq, dk)
    c = r2l.r2l_qk_norm_rope_bwd(*args(copy), dq.clone(), dk.clone())
    for m in a:
        # two results of one sum, in another order, each rounded once: 1e-5 and a half step either way
        assert R.rel_err_per_head(a[m].reshape(1, 1, 1, -1), c[m].reshape(1, 1, 1, -1)) < (2e-5 if a[m].dtype == torch.float32 else 2 * 2.0 ** -8 + 2e-5), m


def test_calls_of_several_threads(r2l):
    """Threads with streams of their own, every kernel's first launches among them, get the bits of calls one by one."""
    import threading

    want = [[[t.clone() for t in c()] for c in side_calls(r2l, seed, None)] for seed in range(4)]
    torch.cuda.synchronize()
    bad = []

    def work(seed):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = [c() for c in side_calls(r2l, seed, None)]
                s.synchronize()
                bad.extend(seed for x, y in zip(got, want[seed]) for a, w in zip(x, y) if not torch.equal(a, w))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
