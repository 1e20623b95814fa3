"""Host-side checks of libr2l_mixer.so that need no GPU: exports, struct layout, refusals, empty problems."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "r2l_mixer.h")
CUDA_INC = "/usr/local/cuda/include"


@pytest.fixture(scope="module")
def r2l():
    from reverse_mamba_selective_b200 import _build

    _build.build()
    import reverse_mamba_selective_b200 as pkg

    pkg.load_mixer()
    return pkg


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*R2L_API\s+(?:r2l_status|const char \*|int|size_t)\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


def test_library_exports_exactly_the_header(r2l):
    from reverse_mamba_selective_b200 import mixer

    out = subprocess.run(["nm", "-D", "--defined-only", mixer.MIXER_LIB_PATH], capture_output=True, text=True).stdout
    assert {ln.split()[-1] for ln in out.splitlines() if " T " in ln} == set(declared_functions())
    assert r2l.r2l_mixer_abi_version() == 100


@pytest.mark.parametrize("cname,pyname", [("r2l_linattn_args", "LinattnArgs"), ("r2l_qk_norm_rope_args", "QkNormRopeArgs")])
def test_struct_layout_matches_c(r2l, tmp_path, cname, pyname):
    cls = getattr(r2l, pyname)
    fields = [f for f, _ in cls._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"r2l_mixer.h\"\nint main(void){\n"
                    f"printf(\"%zu\\n\", sizeof({cname}));\n"
                    + "".join(f"printf(\"%zu\\n\", offsetof({cname}, {f}));\n" for f in fields) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), "-I", CUDA_INC, "-o", str(exe), str(prog)])
    vals = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert vals[0] == ctypes.sizeof(cls)
    assert vals[1:] == [getattr(cls, f).offset for f in fields]


def la(r2l, **over):
    a = dict(batch=2, seqlen=128, block_len=128, n_heads=4, q_heads=4, k_heads=2, v_heads=4, d_k=64, d_v=32, reverse=0,
             dtype=r2l.R2L_BF16, scale=0.125, q=4096, k=8192, v=12288, q_stride=0, k_stride=0, v_stride=0, log_decay=256,
             seq_lens=None)
    a.update(over)
    return r2l.LinattnArgs(**a)


def code(r2l, st):
    return r2l.status_string(st).split(":")[0]


BAD = "R2L_ERR_INVALID_ARG"
LA_REFUSED = [
    (dict(batch=-1), BAD), (dict(seqlen=-1), BAD), (dict(n_heads=-4), BAD), (dict(d_k=-8), BAD),
    (dict(dtype=5), BAD),
    (dict(d_k=136), "R2L_ERR_UNSUPPORTED"), (dict(d_v=256), "R2L_ERR_UNSUPPORTED"),
    (dict(d_k=60), BAD), (dict(d_v=36), BAD),
    (dict(q_heads=3), BAD), (dict(k_heads=0), BAD), (dict(v_heads=8), BAD),
    (dict(q_stride=128), BAD), (dict(k_stride=132), BAD), (dict(v_stride=-128), BAD), (dict(v_stride=1 << 40), BAD),
    (dict(q=None), BAD), (dict(k=8200), BAD), (dict(v=12290), BAD), (dict(log_decay=None), BAD), (dict(log_decay=258), BAD),
    (dict(seq_lens=4098), BAD),
    (dict(reverse=1, block_len=0), BAD), (dict(reverse=1, block_len=100), BAD), (dict(reverse=1, block_len=64, seq_lens=4096), BAD),
    (dict(batch=1 << 20, seqlen=1 << 12, block_len=1 << 12), "R2L_ERR_UNSUPPORTED"),
]


@pytest.mark.parametrize("over,want", LA_REFUSED)
def test_linattn_refusals(r2l, over, want):
    lib = r2l.load_mixer()
    a = la(r2l, **over)
    assert code(r2l, lib.r2l_linattn(ctypes.byref(a), None, None, 16384, 1 << 20, 1 << 40, None)) == want
    assert code(r2l, lib.r2l_linattn_bwd(ctypes.byref(a), 16384, None, None, 32768, 65536, 131072, None, 1 << 20, 1 << 40, None)) == want
    assert lib.r2l_linattn_workspace_size(ctypes.byref(a)) == 0
    assert lib.r2l_linattn_bwd_workspace_size(ctypes.byref(a)) == 0


def test_linattn_output_and_state_refusals(r2l):
    lib = r2l.load_mixer()
    run = lambda a, h0=None, h1=None, y=16384, ws=1 << 20, n=1 << 40: code(
        r2l, lib.r2l_linattn(ctypes.byref(a), h0, h1, y, ws, n, None))
    assert code(r2l, lib.r2l_linattn(None, None, None, 16384, None, 0, None)) == BAD
    assert run(la(r2l), y=None) == BAD and run(la(r2l), y=16392) == BAD
    assert run(la(r2l), h0=4) == BAD and run(la(r2l), h1=8) == BAD
    blocks = dict(reverse=1, block_len=32)
    assert run(la(r2l, **blocks), h0=4096) == BAD and run(la(r2l, **blocks), h1=4096) == BAD
    grad = lambda a, dy=16384, h0=None, dh=None, o=(32768, 65536, 131072), dh0=None, ws=1 << 20, n=1 << 40: code(
        r2l, lib.r2l_linattn_bwd(ctypes.byref(a), dy, h0, dh, *o, dh0, ws, n, None))
    assert grad(la(r2l), dy=None) == BAD and grad(la(r2l), o=(32768, None, 131072)) == BAD
    assert grad(la(r2l), o=(32768, 65536, 131080)) == BAD
    assert grad(la(r2l, **blocks), dh=4096) == BAD and grad(la(r2l, **blocks), dh0=4096) == BAD
    need = lib.r2l_linattn_bwd_workspace_size(ctypes.byref(la(r2l)))
    assert need >= 2 * 128 * 4 * 64 * 4  # the shared key heads' parts
    assert grad(la(r2l), n=need - 1) == BAD and grad(la(r2l), ws=None) == BAD and grad(la(r2l), ws=(1 << 20) + 16) == BAD
    step = lambda a, h=4096, o=4096, y=16384: code(r2l, lib.r2l_linattn_step(ctypes.byref(a), h, o, y, None))
    assert step(la(r2l)) == BAD  # one token only
    one = dict(seqlen=1, block_len=1)
    assert step(la(r2l, **one, reverse=1)) == BAD and step(la(r2l, **one, seq_lens=4096)) == BAD
    assert step(la(r2l, **one), h=None) == BAD and step(la(r2l, **one), o=None) == BAD and step(la(r2l, **one), y=None) == BAD
    assert step(la(r2l, **one), h=4100) == BAD


def test_gradient_of_the_state_is_not_written_over_a_state(r2l):
    lib = r2l.load_mixer()
    grad = lambda h0, dh, dh0: code(r2l, lib.r2l_linattn_bwd(
        ctypes.byref(la(r2l)), 16384, h0, dh, 32768, 65536, 131072, dh0, 1 << 20, 1 << 40, None))
    assert grad(4096, 8192, 4096) == BAD and grad(4096, 8192, 8192) == BAD and grad(None, 8192, 8192) == BAD


def test_empty_problems_are_noops(r2l):
    lib = r2l.load_mixer()
    for over in (dict(batch=0), dict(n_heads=0), dict(d_k=0), dict(d_v=0), dict(seqlen=0)):
        a = la(r2l, **over, q=None, k=None, v=None)
        assert lib.r2l_linattn(ctypes.byref(a), None, None, None, None, 0, None) == r2l.R2L_OK
        assert lib.r2l_linattn_bwd(ctypes.byref(a), None, None, None, None, None, None, None, None, 0, None) == r2l.R2L_OK
    for over in (dict(tokens=0), dict(head_dim=0, rot_dim=0), dict(q_heads=0, k_heads=0)):
        a = rope(r2l, **over, q=None, k=None)
        assert lib.r2l_qk_norm_rope(ctypes.byref(a), None, 0, None, 0, None) == r2l.R2L_OK
        assert lib.r2l_qk_norm_rope_bwd(ctypes.byref(a), None, None, None, None, None, None, None, 0, None) == r2l.R2L_OK


def rope(r2l, **over):
    a = dict(tokens=10, q_heads=4, k_heads=2, head_dim=64, rot_dim=64, interleaved=0, position_64=1, dtype=r2l.R2L_BF16,
             eps=1e-6, q=4096, k=8192, q_stride=0, k_stride=0, q_weight=256, k_weight=512, positions=1024, inv_freq=2048)
    a.update(over)
    return r2l.QkNormRopeArgs(**a)


@pytest.mark.parametrize("over,want", [
    (dict(tokens=-1), BAD), (dict(q_heads=-1), BAD), (dict(head_dim=-2), BAD), (dict(dtype=9), BAD),
    (dict(head_dim=258), "R2L_ERR_UNSUPPORTED"), (dict(head_dim=63), BAD), (dict(rot_dim=33), BAD), (dict(rot_dim=66), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(q_stride=255), BAD), (dict(k_stride=127), BAD),
    (dict(q=None), BAD), (dict(k=8193), BAD), (dict(q_weight=258), BAD), (dict(positions=None), BAD),
    (dict(positions=1028), BAD), (dict(inv_freq=None), BAD), (dict(inv_freq=2050), BAD),
])
def test_rope_refusals(r2l, over, want):
    lib = r2l.load_mixer()
    a = rope(r2l, **over)
    assert code(r2l, lib.r2l_qk_norm_rope(ctypes.byref(a), 16384, 0, 32768, 0, None)) == want
    assert code(r2l, lib.r2l_qk_norm_rope_bwd(ctypes.byref(a), 4096, 8192, 16384, 32768, 256, 512, 1 << 20, 1 << 30, None)) == want


def test_rope_output_refusals(r2l):
    lib = r2l.load_mixer()
    a = rope(r2l)
    run = lambda q, qs, k, ks: code(r2l, lib.r2l_qk_norm_rope(ctypes.byref(a), q, qs, k, ks, None))
    assert run(None, 0, 32768, 0) == BAD and run(16384, 0, None, 0) == BAD
    assert run(16385, 0, 32768, 0) == BAD and run(16384, 255, 32768, 0) == BAD and run(16384, 0, 32768, 64) == BAD
    need = lib.r2l_qk_norm_rope_bwd_workspace_size(ctypes.byref(a))
    assert need > 0
    grad = lambda dq=4096, out=16384, w=256, ws=1 << 20, n=need: code(
        r2l, lib.r2l_qk_norm_rope_bwd(ctypes.byref(a), dq, 8192, out, 32768, w, None, ws, n, None))
    assert grad(dq=None) == BAD and grad(out=None) == BAD and grad(w=258) == BAD
    assert grad(n=need - 1) == BAD and grad(ws=(1 << 20) + 128) == BAD and grad(ws=None) == BAD


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour on a machine without a GPU")
def test_no_cpu_fallback_without_gpu(r2l):
    lib = r2l.load_mixer()
    n = lib.r2l_linattn_workspace_size(ctypes.byref(la(r2l)))
    assert lib.r2l_linattn(ctypes.byref(la(r2l)), None, None, 16384, 1 << 20, n, None) == r2l.R2L_ERR_CUDA
    assert lib.r2l_mixer_last_error().decode() != ""
    assert lib.r2l_qk_norm_rope(ctypes.byref(rope(r2l)), 16384, 0, 32768, 0, None) == r2l.R2L_ERR_CUDA
    t = torch.zeros(1, 4, 2, 8)
    with pytest.raises(TypeError):
        r2l.r2l_linattn(t, t, t, torch.zeros(2))


def test_binding_fails_loudly_without_library(monkeypatch, tmp_path):
    import reverse_mamba_selective_b200.mixer as m

    monkeypatch.setattr(m, "_lib", None)
    monkeypatch.setattr(m, "MIXER_LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(ImportError):
        m.load_mixer()
