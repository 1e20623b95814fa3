"""The mixer operators written out in fp64, one token after another (no chunks, no shared code with the library)."""

import math

import torch


def order(L, reverse, n=None):
    n = L if n is None else n
    return list(range(n))[::-1] if reverse else list(range(n))


def linattn(q, k, v, g, scale, reverse=False, block=None, lens=None, h0=None):
    """(y, h_last) of S_t = e^g S + k_t v_t^T, y_t = scale q_t . S_t; q, k, v [b, L, heads, d] of any type."""
    b, L, H = v.shape[0], v.shape[1], g.shape[0]
    q, k, v = (x.double().repeat_interleave(H // x.shape[2], 2) for x in (q, k, v))
    dk, dv = q.shape[3], v.shape[3]
    decay = torch.exp(g.double())[:, None, None]
    y = torch.zeros(b, L, H, dv, dtype=torch.float64, device=q.device)
    last = torch.zeros(b, H, dk, dv, dtype=torch.float64, device=q.device)
    for r in range(b):
        S = h0[r].double() if h0 is not None else torch.zeros_like(last[r])
        n = L if lens is None else int(lens[r])
        for i, t in enumerate(order(L, reverse, n)):
            if reverse and block and i and i % block == 0:
                S = torch.zeros_like(S)
            S = S * decay + k[r, t, :, :, None] * v[r, t, :, None, :]
            y[r, t] = scale * torch.einsum("hk,hkv->hv", q[r, t], S)
        last[r] = S
    return y, last


def linattn_grads(q, k, v, g, scale, dy, reverse=False, block=None, lens=None, h0=None, dh_last=None):
    """(dq, dk, dv, dh0) by the recurrence's adjoint, token by token, in fp64."""
    b, L, H = v.shape[0], v.shape[1], g.shape[0]
    groups = [x.shape[2] for x in (q, k, v)]
    q, k, v = (x.double().repeat_interleave(H // x.shape[2], 2) for x in (q, k, v))
    dy = dy.double()
    decay = torch.exp(g.double())[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dh0 = torch.zeros(b, H, q.shape[3], v.shape[3], dtype=torch.float64, device=q.device)
    for r in range(b):
        n = L if lens is None else int(lens[r])
        toks = order(L, reverse, n)
        S = h0[r].double() if h0 is not None else torch.zeros_like(dh0[r])
        for i, t in enumerate(toks):
            if reverse and block and i and i % block == 0:
                S = torch.zeros_like(S)
            S = S * decay + k[r, t, :, :, None] * v[r, t, :, None, :]
            dq[r, t] = scale * torch.einsum("hkv,hv->hk", S, dy[r, t])
        A = dh_last[r].double() if dh_last is not None else torch.zeros_like(dh0[r])
        for i in range(n - 1, -1, -1):
            t = toks[i]
            A = A + scale * q[r, t, :, :, None] * dy[r, t, :, None, :]
            dk[r, t] = torch.einsum("hkv,hv->hk", A, v[r, t])
            dv[r, t] = torch.einsum("hkv,hk->hv", A, k[r, t])
            A = torch.zeros_like(A) if reverse and block and i and i % block == 0 else A * decay
        dh0[r] = A
    out = [x.view(b, L, n, H // n, x.shape[3]).sum(3) for x, n in zip((dq, dk, dv), groups)]
    return out[0], out[1], out[2], dh0


def rotate(x, cos, sin, interleaved):
    """The rotary embedding of the first 2 * cos.shape[-1] channels of x [tokens, heads, d]."""
    r = 2 * cos.shape[-1]
    i = torch.arange(r // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    x = x.double()
    z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        z = z * w.double()
    if inv_freq is None:
        return z
    t = (pos.double()[:, None] * inv_freq.double())[:, None]
    return rotate(z, torch.cos(t), torch.sin(t), interleaved)


def norm_rope_grads(x, w, pos, inv_freq, eps, interleaved, dy):
    """(dx, dw) in fp64."""
    x, u = x.double(), dy.double()
    d = x.shape[-1]
    if inv_freq is not None:
        t = (pos.double()[:, None] * inv_freq.double())[:, None]
        u = rotate(u, torch.cos(t), -torch.sin(t), interleaved)
    r = torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dw = (u * x / r).sum((0, 1))
    if w is not None:
        u = u * w.double()
    return u / r - x * (u * x).sum(-1, keepdim=True) / (d * r ** 3), dw


def rel_err_per_head(got, ref):
    """Max over elements of |got - ref| / max(|ref|, rms of ref over the element's head) for [b, L, heads, d]: the
    heads' decays differ, and with them their outputs' size."""
    got, ref = got.double(), ref.double()
    if ref.numel() == 0:
        return 0.0
    rms = ref.square().mean(dim=(0, 1, 3), keepdim=True).sqrt()
    rms = torch.where(rms > 0, rms, torch.ones_like(rms))
    return float(((got - ref).abs() / torch.maximum(ref.abs(), rms)).max())


def rel_err_state(got, ref):
    """The same for states [b, heads, dk, dv]."""
    got, ref = got.double(), ref.double()
    if ref.numel() == 0:
        return 0.0
    rms = ref.square().mean(dim=(2, 3), keepdim=True).sqrt()
    rms = torch.where(rms > 0, rms, torch.ones_like(rms))
    return float(((got - ref).abs() / torch.maximum(ref.abs(), rms)).max())


def log_decays(heads, lo=1.0, span=7.0):
    return torch.tensor([math.log1p(-(2.0 ** (-lo - span * h / max(heads, 1)))) for h in range(heads)], dtype=torch.float32)
