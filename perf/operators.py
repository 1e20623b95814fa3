"""Cases of the linear-attention operators: what is computed, on which sizes, and its plain form.

Two operators that go together in one mixer layer:

* linear attention with a fixed decay for each head -- a prompt or a block of tokens at once, one
  token of every sequence (the serving step), and the gradients;
* the per-head RMS norm of queries and keys with the rotary position embedding, and its gradients.

With ``own`` false, ``run`` computes them with elementary torch operations in fp32 (angles in fp64);
with ``own`` true it calls the package.  ``exact`` writes the definitions out in fp64, token by token.
"""

import math

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases

def _attn(op, name, **kw):
    c = dict(op=op, dtype="bf16", b=1, L=1, heads=16, qk_heads=16, dk=128, dv=128, reverse=False, block=0,
             lens=False, h0=False, h_last=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _rope(op, name, **kw):
    c = dict(op=op, dtype="bf16", tokens=1, q_heads=16, k_heads=8, dim=128, rot=128, interleaved=False, fused=True)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # prompt prefill of a batch of 8 requests, 4096 tokens each, 16 heads of 128; the states go on to the steps
        _attn("attn", "prefill_b8_L4096", b=8, L=4096, h_last=True),
        # one long prompt alone on the GPU: 16 heads are fewer than the SMs, so the sequence has to be divided
        _attn("attn", "long_b1_L32768", L=32768, h_last=True),
        # a right-padded batch of prompts of unequal length, queries and keys shared by groups of heads, odd sizes
        _attn("attn", "ragged_b6_L1021", b=6, L=1021, heads=12, qk_heads=4, dk=96, dv=64, lens=True, h_last=True),
        # parallel decoding: right to left over the active block of 32 tokens of 64 requests
        _attn("attn", "block_b64_L32", b=64, L=32, reverse=True, block=32),
        # the active block of 16 tokens of 32 requests, resumed from the cached state of the prefix
        _attn("attn", "resume_b32_L16", b=32, L=16, heads=32, qk_heads=32, h0=True, h_last=True),
        # serving, one token: a single request (latency)
        _attn("step", "step_b1", h0=True),
        # serving, one token of each of 128 requests
        _attn("step", "step_b128", b=128, h0=True),
        # training step of the prefill shape
        _attn("grad", "grad_b8_L4096", b=8, L=4096),
        # fp32 gradients through a carried state, odd length, 64 x 48 heads
        _attn("grad", "grad_f32_b2_L200", dtype="f32", b=2, L=200, heads=8, qk_heads=8, dk=64, dv=48, h0=True, h_last=True),
        # one token of each of 64 requests, out of the fused projection
        _rope("rope", "rope_64", tokens=64),
        # the tokens of the prefill above
        _rope("rope", "rope_32768", tokens=32768),
        # their gradients in training
        _rope("rope_grad", "rope_grad_16384", tokens=16384),
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "step", "grad", "rope", "rope_grad"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op in ("rope", "rope_grad"):
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        k = rng.choice([1, 2, 4, 8])
        q = k * rng.choice([1, 2, 4])
        cap = 8192 * 128 * 24 // (dim * (q + k))
        return _rope(op, None, dtype=dtype, tokens=_size(rng, 1, cap), q_heads=q, k_heads=k, dim=dim,
                     rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, fused=rng.random() < 0.6)
    group = rng.choice([1, 1, 2, 4])
    heads = group * rng.choice([1, 2, 4, 8, 8])
    dk, dv = rng.choice([32, 64, 80, 96, 128, 128]), rng.choice([32, 48, 64, 64, 128, 128])
    if op == "step":
        return _attn(op, None, dtype=dtype, b=_size(rng, 1, 128), heads=heads, qk_heads=heads // group, dk=dk, dv=dv, h0=True)
    cap = (1 << 16) if dtype == "f32" else (1 << 18)  # (token, head) pairs
    L = _size(rng, 1, 4000)
    block, reverse = 0, rng.random() < 0.4
    if reverse and rng.random() < 0.5:
        block = _size(rng, 1, 300)
        L = block * _size(rng, 1, max(1, 4000 // block))
    b = _size(rng, 1, max(1, min(64, cap // (L * heads))))
    plain = block == 0
    return _attn(op, None, dtype=dtype, b=b, L=L, heads=heads, qk_heads=heads // group, dk=dk, dv=dv, reverse=reverse,
                 block=block, lens=plain and not reverse and op == "attn" and rng.random() < 0.4,
                 h0=plain and rng.random() < 0.5, h_last=plain and rng.random() < 0.6)


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("rope", "rope_grad"):
        n = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["dim"]
        passes = 2 if c["op"] == "rope" else 3
        return {"bytes": passes * n * es + c["tokens"] * 8 + 2 * c["dim"] * 4 + c["rot"] * 2,
                "flops": n * (8 if c["op"] == "rope" else 16)}
    rows = c["b"] * c["L"]
    qk, v = rows * c["qk_heads"] * c["dk"], rows * c["heads"] * c["dv"]
    state = c["b"] * c["heads"] * c["dk"] * c["dv"] * 4
    pairs = rows * c["heads"] * c["dk"] * c["dv"]
    if c["op"] == "step":
        return {"bytes": (2 * qk + 2 * v) * es + 2 * state, "flops": 4 * pairs}
    io = (2 * qk + 2 * v) * es + state * (int(c["h0"]) + int(c["h_last"]))
    if c["op"] == "attn":
        return {"bytes": io, "flops": 4 * pairs}
    # q, k, v and dy read; dq, dk and dv written; h0 and dh_last read, dh0 written
    return {"bytes": (4 * qk + 3 * v) * es + state * (2 * int(c["h0"]) + int(c["h_last"])), "flops": 12 * pairs}


# ------------------------------------------------------------------------------------------ inputs

def _log_decay(heads):
    # gamma_h = 1 - 2^(-1 - 7 h / heads): memories from two tokens to a few hundred
    h = torch.arange(heads, dtype=torch.float64)
    return torch.log1p(-torch.exp2(-1.0 - 7.0 * h / heads)).to(torch.float32).to(DEV)


def prepare(case, seed):
    c = dict(case)
    t = _TYPES[c["dtype"]]
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32) * std).to(dtype)

    s = {"case": c}
    if c["op"] in ("rope", "rope_grad"):
        n, hq, hk, d = c["tokens"], c["q_heads"], c["k_heads"], c["dim"]
        if c["fused"]:  # queries and keys as they lie in the output of one projection (with the values behind them)
            qkv = normal(n, (hq + 2 * hk) * d)
            s["q"], s["k"] = qkv[:, : hq * d].view(n, hq, d), qkv[:, hq * d : (hq + hk) * d].view(n, hk, d)
        else:
            s["q"], s["k"] = normal(n, hq, d), normal(n, hk, d)
        s["qw"], s["kw"] = 1.0 + normal(d, std=0.1, dtype=torch.float32), 1.0 + normal(d, std=0.1, dtype=torch.float32)
        # positions of a long context: a run of tokens that starts anywhere below 2^17
        start = torch.randint(0, 1 << 17, (1,), generator=gen, device=DEV)
        s["pos"] = start + torch.arange(n, device=DEV)
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
        s["inv_freq"] = torch.exp(-math.log(1e6) * 2.0 * i / c["rot"]).to(torch.float32)
        if c["op"] == "rope_grad":
            s["dq"], s["dk"] = normal(n, hq, d), normal(n, hk, d)
        return s
    b, L, h, hk, dk, dv = c["b"], c["L"], c["heads"], c["qk_heads"], c["dk"], c["dv"]
    lead = (b,) if c["op"] == "step" else (b, L)
    s["q"], s["k"], s["v"] = normal(*lead, hk, dk), normal(*lead, hk, dk), normal(*lead, h, dv)
    s["g"] = _log_decay(h)
    s["h0"] = normal(b, h, dk, dv, dtype=torch.float32) if c["h0"] else None
    s["lens"] = torch.randint(1, L + 1, (b,), generator=gen, device=DEV).to(torch.int32) if c["lens"] else None
    if c["op"] == "grad":
        s["dy"] = normal(b, L, h, dv)
        s["dh"] = normal(b, h, dk, dv, std=0.1, dtype=torch.float32) if c["h_last"] else None
    return s


# -------------------------------------------------------------------------------------- plain forms

def _plain_attn(c, q, k, v, g, h0, lens, want_h):
    """Chunks of C tokens, fp32: within a chunk by the matrix of pairs, across chunks by their states."""
    b, L, h = v.shape[:3]
    scale = 1.0 / math.sqrt(c["dk"])
    rep = h // q.shape[2]
    q, k, v = (x.float().transpose(1, 2) for x in (q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2), v))
    if c["block"]:  # every block is a sequence of its own
        nb = L // c["block"]
        q, k, v = (x.reshape(b, h, nb, c["block"], -1).transpose(1, 2).reshape(b * nb, h, c["block"], -1) for x in (q, k, v))
    rows, n = q.shape[0], q.shape[2]
    if c["reverse"]:
        q, k, v = q.flip(2), k.flip(2), v.flip(2)
    t = torch.arange(n, device=DEV)
    g = g.double()
    if lens is not None:
        live = (t < lens[:, None])[:, None, :, None]
        k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    h_last = None
    if want_h:
        left = (lens[:, None] if lens is not None else torch.full((rows, 1), n, device=DEV)) - 1 - t  # tokens after t
        w = torch.where(left >= 0, torch.exp(g[:, None, None] * left.clamp(min=0)), 0.0).float()  # [h, rows, n]
        h_last = torch.matmul((k * w.transpose(0, 1)[..., None]).transpose(2, 3), v)
        if h0 is not None:
            h_last = h_last + h0 * torch.exp(g[None, :] * (left[:, :1] + 1)).float()[..., None, None]
    C = 64
    nc = -(-n // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, nc * C - n)).reshape(rows, h, nc, C, -1) for x in (q, k, v))
    i = torch.arange(C, device=DEV)
    gap = i[:, None] - i[None, :]
    within = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), 0.0).float()  # [h, C, C]
    y = torch.matmul(torch.matmul(q, k.transpose(3, 4)) * within[None, :, None], v)
    tail = torch.exp(g[:, None] * (C - 1 - i)).float()  # to the end of the chunk
    states = torch.matmul((k * tail[None, :, None, :, None]).transpose(3, 4), v)  # [rows, h, nc, dk, dv]
    m = torch.arange(nc, device=DEV)
    skip = m[:, None] - 1 - m[None, :]
    across = torch.where(skip >= 0, torch.exp(g[:, None, None] * C * skip.clamp(min=0)), 0.0).float()  # [h, nc, nc]
    before = torch.matmul(across[None], states.flatten(3)).view_as(states)
    if h0 is not None:
        before = before + torch.exp(g[:, None] * C * m).float()[None, :, :, None, None] * h0[:, :, None]
    head = torch.exp(g[:, None] * (i + 1)).float()
    y = y + torch.matmul(q * head[None, :, None, :, None], before)
    y = (y * scale).reshape(rows, h, nc * C, -1)[:, :, :n]
    if lens is not None:
        y = torch.where(live, y, 0.0)
    if c["reverse"]:
        y = y.flip(2)
    if c["block"]:
        y = y.reshape(b, nb, h, n, -1).transpose(1, 2).reshape(b, h, L, -1)
    return y.transpose(1, 2), h_last


def _plain_step(c, s):
    rep = c["heads"] // c["qk_heads"]
    q, k, v = s["q"].float().repeat_interleave(rep, 1), s["k"].float().repeat_interleave(rep, 1), s["v"].float()
    h = s["h0"] * torch.exp(s["g"])[:, None, None] + k[..., None] * v[..., None, :]
    y = (q[..., None] * h).sum(2) / math.sqrt(c["dk"])
    return y.to(s["v"].dtype), h


def _plain_grad(c, s):
    ins = {n: s[n].detach().float().requires_grad_() for n in ("q", "k", "v")}
    h0 = s["h0"].detach().requires_grad_() if s["h0"] is not None else None
    y, h_last = _plain_attn(c, ins["q"], ins["k"], ins["v"], s["g"], h0, None, c["h_last"])
    outs, grads = [y], [s["dy"].float()]
    if c["h_last"]:
        outs.append(h_last)
        grads.append(s["dh"])
    leaves = list(ins.values()) + ([h0] if h0 is not None else [])
    got = torch.autograd.grad(outs, leaves, grads)
    t = s["q"].dtype
    return [x.to(t) for x in got[:3]] + [x for x in got[3:]]


def _angles(c, s):
    a = s["pos"].double()[:, None] * s["inv_freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _halves(c, x):
    r = c["rot"]
    if c["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2]
    return x[..., : r // 2], x[..., r // 2 : r]


def _joined(c, a, b, rest):
    x = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([x, rest], -1)


def _plain_rope(c, x, w, cos, sin):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    a, b = _halves(c, y)
    return _joined(c, a * cos - b * sin, b * cos + a * sin, y[..., c["rot"] :])


def _plain_rope_grad(c, x, w, cos, sin, dy):
    a, b = _halves(c, dy)
    u = _joined(c, a * cos + b * sin, b * cos - a * sin, dy[..., c["rot"] :])  # the rotation taken back
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    z = x * inv
    dx = inv * (u * w - z * (u * w * z).mean(-1, keepdim=True))
    return dx, (u * z).double().sum((0, 1)).float()


# ---------------------------------------------------------------------------------------------- run

def _run_plain(c, s):
    op = c["op"]
    if op == "attn":
        y, h = _plain_attn(c, s["q"], s["k"], s["v"], s["g"], s["h0"], s["lens"], c["h_last"])
        y = y.to(s["q"].dtype)
        return [y, h] if c["h_last"] else [y]
    if op == "step":
        return list(_plain_step(c, s))
    if op == "grad":
        return _plain_grad(c, s)
    t = s["q"].dtype
    cos, sin = _angles(c, s)
    if op == "rope":
        return [_plain_rope(c, s["q"].float(), s["qw"], cos, sin).to(t), _plain_rope(c, s["k"].float(), s["kw"], cos, sin).to(t)]
    dq, dqw = _plain_rope_grad(c, s["q"].float(), s["qw"], cos, sin, s["dq"].float())
    dk, dkw = _plain_rope_grad(c, s["k"].float(), s["kw"], cos, sin, s["dk"].float())
    return [dq.to(t), dk.to(t), dqw, dkw]


def _run_own(c, s):
    import reverse_mamba_selective_b200 as r2l

    op = c["op"]
    if op == "attn":
        y, h = r2l.r2l_linattn(s["q"], s["k"], s["v"], s["g"], reverse=c["reverse"], block_len=c["block"] or None,
                               seq_lens=s["lens"], h0=s["h0"], want_h_last=c["h_last"])
        return [y, h] if c["h_last"] else [y]
    if op == "step":
        h = torch.empty_like(s["h0"])  # not in place, so that every pass starts from the same state
        return [r2l.r2l_linattn_step(s["q"], s["k"], s["v"], s["g"], s["h0"], h_out=h), h]
    if op == "grad":
        g = r2l.r2l_linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["dy"], reverse=c["reverse"], block_len=c["block"] or None,
                                h0=s["h0"], dh_last=s["dh"])
        return [g["dq"], g["dk"], g["dv"]] + ([g["dh0"]] if c["h0"] else [])
    if op == "rope":
        return list(r2l.r2l_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["inv_freq"], eps=1e-6,
                                         interleaved=c["interleaved"]))
    g = r2l.r2l_qk_norm_rope_bwd(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["inv_freq"], s["dq"], s["dk"], eps=1e-6,
                                 interleaved=c["interleaved"])
    return [g["dq"], g["dk"], g["dq_weight"], g["dk_weight"]]


def run(state):
    c = state["case"]
    return _run_own(c, state) if own else _run_plain(c, state)


# -------------------------------------------------------------------------------------------- exact

def _exact_attn(c, s):
    """S_t = e^g S + k_t v_t^T, y_t = q_t . S_t / sqrt(dk), one token after another in the order of the scan."""
    b, L, h, dv = s["v"].shape
    rep, dk = h // c["qk_heads"], c["dk"]
    q, k, v = s["q"].double().repeat_interleave(rep, 2), s["k"].double().repeat_interleave(rep, 2), s["v"].double()
    decay = torch.exp(s["g"].double())[None, :, None, None]
    zero = torch.zeros(b, h, dk, dv, dtype=torch.float64, device=DEV)
    S = s["h0"].double() if s["h0"] is not None else zero.clone()
    y = torch.zeros(b, L, h, dv, dtype=torch.float64, device=DEV)
    block = c["block"] or L
    for n in range(L):
        t = L - 1 - n if c["reverse"] else n
        if n and n % block == 0:
            S = zero.clone()
        new = S * decay + k[:, t, :, :, None] * v[:, t, :, None, :]
        out = torch.matmul(q[:, t, :, None, :], new)[:, :, 0] / math.sqrt(dk)
        if s["lens"] is not None:
            live = (t < s["lens"])[:, None, None, None]
            new, out = torch.where(live, new, S), torch.where(live[..., 0], out, 0.0)
        S, y[:, t] = new, out
    return [y, S] if c["h_last"] else [y]


def _exact_grad(c, s):
    """The recurrence's adjoint, token by token: dq from the states, dk and dv from the states' gradients."""
    b, L, h, dv = s["v"].shape
    rep, dk = h // c["qk_heads"], c["dk"]
    scale = 1.0 / math.sqrt(dk)
    q, k, v = s["q"].double().repeat_interleave(rep, 2), s["k"].double().repeat_interleave(rep, 2), s["v"].double()
    dy = s["dy"].double()
    decay = torch.exp(s["g"].double())[None, :, None, None]
    S = s["h0"].double() if s["h0"] is not None else torch.zeros(b, h, dk, dv, dtype=torch.float64, device=DEV)
    A = s["dh"].double() if s["dh"] is not None else torch.zeros(b, h, dk, dv, dtype=torch.float64, device=DEV)
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    block = c["block"] or L
    order = list(range(L))[::-1] if c["reverse"] else list(range(L))
    for n, t in enumerate(order):
        S = k[:, t, :, :, None] * v[:, t, :, None, :] + (S * decay if n == 0 or n % block else 0.0)
        dq[:, t] = torch.matmul(S, dy[:, t, :, :, None])[..., 0] * scale
    for n in range(L - 1, -1, -1):
        t = order[n]
        A = A + scale * q[:, t, :, :, None] * dy[:, t, :, None, :]
        dkk[:, t] = torch.matmul(A, v[:, t, :, :, None])[..., 0]
        dvv[:, t] = torch.matmul(k[:, t, :, None, :], A)[:, :, 0]
        A = A * decay if n == 0 or n % block else torch.zeros_like(A)
    kh = c["qk_heads"]
    got = [dq.view(b, L, kh, rep, dk).sum(3), dkk.view(b, L, kh, rep, dk).sum(3), dvv]
    return got + ([A] if s["h0"] is not None else [])


def _exact_rope(c, s):
    r, d = c["rot"], c["dim"]
    i = torch.arange(r // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
    a = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    outs, weights = [], []
    for name, wname in (("q", "qw"), ("k", "kw")):
        x, w = s[name].double(), s[wname].double()
        inv = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6)
        if c["op"] == "rope":
            y = x * inv * w
            z = y.clone()
            z[..., first] = y[..., first] * cos - y[..., second] * sin
            z[..., second] = y[..., second] * cos + y[..., first] * sin
            outs.append(z)
            continue
        dy = s["d" + name].double()
        u = dy.clone()
        u[..., first] = dy[..., first] * cos + dy[..., second] * sin
        u[..., second] = dy[..., second] * cos - dy[..., first] * sin
        weights.append((u * x * inv).sum((0, 1)))
        u = u * w
        outs.append(inv * u - x * inv ** 3 * (u * x).sum(-1, keepdim=True) / d)
    return outs + weights


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "attn":
        return _exact_attn(c, s)
    if c["op"] == "step":
        one = {**s, **{n: s[n][:, None] for n in ("q", "k", "v")}}
        y, h = _exact_attn({**c, "h_last": True}, one)
        return [y[:, 0], h]
    if c["op"] == "grad":
        return _exact_grad(c, s)
    return _exact_rope(c, s)
