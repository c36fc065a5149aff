"""The gated delta rule and the query/key norms in 64 bits, token by token, on the CPU.

Written from the definitions, with torch only: no code is shared with the library's
kernels or with its chunked formulas.
"""

import torch

F64 = torch.float64


def heads(x, H):
    """[B,Hk,...] -> [B,H,...]: value head h reads key head h // (H / Hk)."""
    return x[:, torch.arange(H) // (H // x.shape[1])]


def forward(q, k, v, beta, log_alpha, scale, S0=None):
    """y [B,H,T,dv] and the last state [B,H,dv,dk]; differentiable."""
    B, H, T, dv = v.shape
    q, k = heads(q, H), heads(k, H)
    S = torch.zeros(B, H, dv, q.shape[-1], dtype=F64) if S0 is None else S0
    y = []
    for t in range(T):
        Sd = torch.exp(log_alpha[:, :, t])[..., None, None] * S
        e = v[:, :, t] - torch.einsum("bhvk,bhk->bhv", Sd, k[:, :, t])
        S = Sd + torch.einsum("bh,bhv,bhk->bhvk", beta[:, :, t], e, k[:, :, t])
        y.append(scale * torch.einsum("bhvk,bhk->bhv", S, q[:, :, t]))
    return torch.stack(y, 2), S


def gradients(q, k, v, beta, log_alpha, scale, S0, dy, dST=None):
    """Gradients of <dy, y> + <dST, S_T> by the reverse recurrence of the definition."""
    B, H, T, dv = v.shape
    Hk = q.shape[1]
    qh, kh = heads(q, H), heads(k, H)
    S = torch.zeros(B, H, dv, q.shape[-1], dtype=F64) if S0 is None else S0
    seen = []
    for t in range(T):
        Sd = torch.exp(log_alpha[:, :, t])[..., None, None] * S
        e = v[:, :, t] - (Sd @ kh[:, :, t, :, None])[..., 0]
        S = Sd + (beta[:, :, t, None] * e)[..., None] * kh[:, :, t, None, :]
        seen.append((Sd, e, S))
    lam = torch.zeros_like(S) if dST is None else dST.clone()
    dq, dk = torch.zeros_like(qh), torch.zeros_like(kh)
    dv_, db, dl = torch.zeros_like(v), torch.zeros_like(beta), torch.zeros_like(beta)
    for t in reversed(range(T)):
        Sd, e, S = seen[t]
        g = scale * dy[:, :, t]
        dq[:, :, t] = (S.mT @ g[..., None])[..., 0]
        lam = lam + g[..., None] * qh[:, :, t, None, :]
        du = (lam @ kh[:, :, t, :, None])[..., 0]
        db[:, :, t] = (du * e).sum(-1)
        de = beta[:, :, t, None] * du
        dv_[:, :, t] = de
        dk[:, :, t] = (lam.mT @ (beta[:, :, t, None] * e)[..., None] - Sd.mT @ de[..., None])[..., 0]
        lam = lam - de[..., None] * kh[:, :, t, None, :]
        dl[:, :, t] = (lam * Sd).sum((-1, -2))
        lam = torch.exp(log_alpha[:, :, t])[..., None, None] * lam
    share = lambda x: x.reshape(B, Hk, H // Hk, T, -1).sum(2)  # noqa: E731
    return dict(dq=share(dq), dk=share(dk), dv=dv_, dbeta=db, dlog_alpha=dl, dS0=lam)


def draw(B, H, Hk, T, dk, dv, dtype="f32", S0=False, mask="none", seed=0, unit=True):
    """Inputs in the I/O dtype (gates and S0 float32), on the CPU.

    mask: "none"; "docs" (resets at the first token, in a row, at and around chunk borders,
    and padding tokens); "empty" (one batch row's update masked out throughout); "reset" (a
    reset at every token)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k = r(B, Hk, T, dk), r(B, Hk, T, dk)
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    d = dict(q=q.to(td), k=k.to(td), v=r(B, H, T, dv).to(td), dy=r(B, H, T, dv).to(td))
    d["beta"] = torch.sigmoid(r(B, H, T))
    d["log_alpha"] = torch.log1p(-10.0 ** (3 * torch.rand((B, H, T), generator=g) - 4))
    d["S0"] = r(B, H, dv, dk) / dk ** 0.5 if S0 else None
    if mask == "docs":
        for t in (0, 1, 5, 31, 32, 63, 64, 65, 100, 127, 128, 200):
            if t < T:
                d["log_alpha"][:, (t % H):, t] = float("-inf")
        d["log_alpha"][:, :, T // 2] = -500.0
        d["beta"][:, :, 7 % T] = 0.0
        d["beta"][:, :, T - T // 4:] = 0.0
    elif mask == "empty":
        d["beta"][0] = 0.0
    elif mask == "reset":
        d["log_alpha"][:] = float("-inf")
    return d


def f64(d):
    return {n: None if x is None else x.to(F64) for n, x in d.items()}


def rel2(got, ref):
    """2-norm of the difference over the reference's (over 1 where that is zero)."""
    got, ref = got.detach().cpu().to(F64), ref.to(F64)
    n = ref.norm()
    return float((got - ref).norm() / (n if n > 0 else 1.0))


def norm_rope(x, w, pos, inv_freq, norm, eps):
    """[B,T,H,d] -> [B,H,T,d] in 64 bits; differentiable."""
    ss = x.square().sum(-1, keepdim=True)
    u = x / torch.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)
    if w is not None:
        u = u * w
    if inv_freq is not None and inv_freq.numel():
        h = inv_freq.numel()
        a = pos.to(F64)[..., None, None] * inv_freq.to(F64)
        c, s = torch.cos(a), torch.sin(a)
        u = torch.cat([u[..., :h] * c - u[..., h:2 * h] * s,
                       u[..., h:2 * h] * c + u[..., :h] * s, u[..., 2 * h:]], -1)
    return u.transpose(1, 2)
