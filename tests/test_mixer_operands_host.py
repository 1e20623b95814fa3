"""What the mixer binding makes of its operands' strides, without a GPU: tensors of the CPU that say they are on cuda:0, and
calls that are refused before anything is launched."""

import ctypes

import pytest
import torch


class OnCuda(torch.Tensor):
    """A CPU tensor that the binding takes for one on cuda:0."""

    is_cuda = True

    def get_device(self):
        return 0


def cuda(t):
    return t.as_subclass(OnCuda)


@pytest.fixture(scope="module")
def r2l():
    from reverse_mamba_selective_b200 import _build

    _build.build()
    import reverse_mamba_selective_b200 as pkg

    pkg.load_mixer()
    return pkg


def tokens(*lead, heads=4, d=64):
    return torch.zeros(*lead, heads, d, dtype=torch.bfloat16)


# what lies in memory, and the tokens it is broadcast to
BROADCAST = [((1, 1), (1, 50)), ((3, 1), (3, 50)), ((1, 1), (3, 50)), ((1, 50), (3, 50)), ((1, 1), (8, 1)), ((1,), (128,))]


@pytest.mark.parametrize("held,lead", BROADCAST)
def test_tokens_that_share_their_memory_are_refused(held, lead):
    from reverse_mamba_selective_b200 import mixer

    t = cuda(tokens(*held)).expand(*lead, 4, 64)
    with pytest.raises(ValueError):
        mixer._heads("x", t, torch.bfloat16, lead, 0)


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("held,lead", BROADCAST)
def test_no_entry_point_takes_a_broadcast_operand(r2l, held, lead, which):
    x = [cuda(tokens(*lead)) for _ in range(3)]
    x[which] = cuda(tokens(*held)).expand(*lead, 4, 64)
    g = cuda(torch.zeros(4))
    with pytest.raises(ValueError):
        if len(lead) == 2:
            r2l.r2l_linattn(*x, g)
        else:
            r2l.r2l_linattn_step(*x, g, cuda(torch.zeros(lead[0], 4, 64, 64)))
    if len(lead) == 2:
        with pytest.raises(ValueError):
            r2l.r2l_linattn_bwd(*x, g, cuda(tokens(*lead)))


@pytest.mark.parametrize("which", ["q", "k", "q_out", "k_out"])
def test_norm_and_rotation_take_no_broadcast_operand_or_output(r2l, which):
    x = {n: cuda(tokens(20)) for n in ("q", "k", "q_out", "k_out")}
    x[which] = cuda(tokens(1)).expand(20, 4, 64)
    with pytest.raises(ValueError):
        r2l.r2l_qk_norm_rope(x["q"], x["k"], None, None, None, None, q_out=x["q_out"], k_out=x["k_out"])
    if which in ("q", "k"):
        with pytest.raises(ValueError):
            r2l.r2l_qk_norm_rope_bwd(x["q"], x["k"], None, None, None, None, cuda(tokens(20)), cuda(tokens(20)))


@pytest.mark.parametrize("make,lead,stride", [
    (lambda: tokens(3, 50), (3, 50), 0),
    (lambda: tokens(3, 50, heads=9)[:, :, 2:6], (3, 50), 9 * 64),
    (lambda: tokens(3, 50, heads=9)[:1, :, 2:6], (1, 50), 9 * 64),
    (lambda: tokens(3, 50, heads=9)[:, :1, 2:6], (3, 1), 50 * 9 * 64),
    (lambda: tokens(3, 50, heads=9)[:, 7, 2:6], (3,), 50 * 9 * 64),
    (lambda: tokens(3, 50, heads=9)[1:2, 7, 2:6], (1,), 0),
    (lambda: tokens(1, 1).expand(1, 1, 4, 64), (1, 1), 0),
    (lambda: tokens(3, 50)[:, ::2], (3, 25), 2 * 4 * 64),
    (lambda: tokens(0, 50), (0, 50), 0),
])
def test_tokens_with_memory_of_their_own_are_taken(make, lead, stride):
    from reverse_mamba_selective_b200 import mixer

    assert mixer._heads("x", cuda(make()), torch.bfloat16, lead, 0) == stride


@pytest.mark.parametrize("make,lead", [
    (lambda: tokens(3, 50)[:, :49], (3, 49)),                         # rows further apart than their tokens say
    (lambda: tokens(50, 3).transpose(0, 1), (3, 50)),                 # tokens of a row further apart than the rows
    (lambda: tokens(3, 50).transpose(2, 3), (3, 50)),                 # channels not dense
    (lambda: torch.zeros(4000, dtype=torch.bfloat16).as_strided((5, 4, 64), (128, 64, 1)), (5,)),  # tokens that overlap in part
])
def test_tokens_not_evenly_spaced_are_refused(make, lead):
    from reverse_mamba_selective_b200 import mixer

    with pytest.raises(ValueError):
        mixer._heads("x", cuda(make()), torch.bfloat16, lead, 0)


def args(r2l, **over):
    a = dict(batch=2, seqlen=6, block_len=6, n_heads=4, q_heads=4, k_heads=2, v_heads=4, d_k=64, d_v=32, reverse=0,
             dtype=r2l.R2L_BF16, scale=0.125, q=4096, k=8192, v=12288, q_stride=0, k_stride=0, v_stride=0, log_decay=256,
             seq_lens=None)
    a.update(over)
    return r2l.LinattnArgs(**a)


@pytest.mark.parametrize("over", [dict(d_k=0), dict(d_v=0), dict(n_heads=0)])
def test_outputs_of_empty_sums_are_checked(r2l, over):
    lib = r2l.load_mixer()
    a = args(r2l, **over)
    one = args(r2l, **over, seqlen=1, block_len=1)
    assert lib.r2l_linattn(ctypes.byref(a), None, None, 16392, None, 0, None) == r2l.R2L_ERR_INVALID_ARG
    assert lib.r2l_linattn_step(ctypes.byref(one), 4096, 4096, 16392, None) == r2l.R2L_ERR_INVALID_ARG
    for o in ((8, None, None), (None, 8, None), (None, None, 8)):
        assert lib.r2l_linattn_bwd(ctypes.byref(a), 16384, None, None, *o, None, None, 0, None) == r2l.R2L_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour on a machine without a GPU")
def test_outputs_of_empty_sums_are_written(r2l):
    """Zeros have to be written where an output is not empty: without a GPU that fails, and does not pass in silence."""
    lib = r2l.load_mixer()
    run = lambda y, **over: lib.r2l_linattn(ctypes.byref(args(r2l, **over)), None, None, y, None, 0, None)
    assert run(16384, d_k=0) == r2l.R2L_ERR_CUDA
    assert run(16384, d_v=0) == run(16384, n_heads=0) == run(16384, d_k=0, seqlen=0) == run(None, d_k=0) == r2l.R2L_OK
    one = dict(seqlen=1, block_len=1)
    step = lambda **over: lib.r2l_linattn_step(ctypes.byref(args(r2l, **one, **over)), 4096, 4096, 16384, None)
    assert step(d_k=0) == r2l.R2L_ERR_CUDA and step(d_v=0) == r2l.R2L_OK
    grad = lambda dq, dk, dv, **over: lib.r2l_linattn_bwd(ctypes.byref(args(r2l, **over)), 16384, None, None, dq, dk, dv, None, None, 0, None)
    assert grad(None, None, 16384, d_k=0) == grad(16384, None, None, d_v=0) == grad(None, 16384, None, d_v=0) == r2l.R2L_ERR_CUDA
    assert grad(16384, 32768, None, d_k=0) == grad(None, None, 16384, d_v=0) == r2l.R2L_OK


@pytest.mark.parametrize("dtype", [0, 1])
def test_rows_at_the_end_of_the_token_counters(r2l, dtype):
    """The kernels count tokens in 32 bits, some chunks ahead: runs that would pass the end are refused."""
    lib = r2l.load_mixer()
    size = lambda n, b=1: lib.r2l_linattn_workspace_size(ctypes.byref(args(r2l, batch=b, seqlen=n, block_len=n, dtype=dtype)))
    run = lambda n, b=1: lib.r2l_linattn(ctypes.byref(args(r2l, batch=b, seqlen=n, block_len=n, dtype=dtype)), None, None, 16384,
                                         1 << 20, 1 << 40, None)
    for n, b in ((2 ** 31 - 1, 1), (2 ** 31 - 8, 1), (2 ** 31 - 256, 1), (2 ** 30, 2)):
        assert run(n, b) == r2l.R2L_ERR_UNSUPPORTED and size(n, b) == 0
    assert size(2 ** 31 - 257) > 0


@pytest.mark.parametrize("tokens", [2 ** 31, 2 ** 32 + 4])
def test_sizes_past_32_bits_are_refused_and_not_cut_off(r2l, tokens):
    far = lambda *shape, dtype=torch.bfloat16: cuda(torch.empty(*shape, dtype=dtype, device="meta"))
    with pytest.raises(ValueError, match="2\\^31"):
        r2l.r2l_qk_norm_rope(far(tokens, 1, 2), far(tokens, 0, 2), None, None, None, None)
    x, g = far(1, tokens, 1, 8), far(1, dtype=torch.float32)
    with pytest.raises(ValueError, match="2\\^31"):
        r2l.r2l_linattn(x, x, x, g)
    x = far(tokens, 1, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        r2l.r2l_linattn_step(x, x, x, g, far(tokens, 1, 8, 8, dtype=torch.float32))
    x = far(1, 64, 1, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        r2l.r2l_linattn(x, x, x, g, reverse=True, block_len=(1 << 32) + 64)
