"""Measured cases of the gated delta rule and of the query/key norms in front of it.

Four operators of one layer. Its queries and keys are normalised per head and rotated by
their positions (``gradlev_qk_norm_rope_fwd`` / ``_bwd``); a state S_t [d_v, d_k] per value
head then learns to return v_t for k_t, with a retention alpha_t and a step beta_t:

    S'  = alpha_t S_{t-1}
    S_t = S' + beta_t (v_t - S' k_t) k_t^T
    y_t = scale S_t q_t

in chunks over whole sequences (``gradlev_delta_fwd``, ``gradlev_delta_bwd``) or token by
token on states that stay in a pool (``gradlev_delta_step``).

``own`` False: elementary torch operations in 32 bits. ``own`` True: the library's calls.
``exact``: the recurrences as they stand above, token by token in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens per chunk of the plain form
NEG_INF = float("-inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request, one token: the smallest call of serving
        dict(name="step_one", op="step", dt="bf16", B=1, H=16, Hk=16, T=1, dk=128, dv=128, pool=4),
        # a batch of requests, one token each, states picked out of a larger pool; one row in
        # eight is padding of the batch
        dict(name="step_batch", op="step", dt="bf16", B=64, H=16, Hk=8, T=1, dk=128, dv=128,
             pool=96),
        # a few tokens at once (drafted tokens being checked) on the float32 layer
        dict(name="step_f32_T5", op="step", dt="f32", B=4, H=8, Hk=8, T=5, dk=64, dv=64, pool=4),
        # a prompt of ragged length read by one request
        dict(name="prefill_T1000", op="fwd", dt="bf16", B=1, H=16, Hk=8, T=1000, dk=128, dv=128,
             S0=False, docs=False),
        # the next part of a long document, from the state of the parts before
        dict(name="prefill_T32768", op="fwd", dt="bf16", B=1, H=16, Hk=16, T=32768, dk=128, dv=256,
             S0=True, docs=False),
        # training on packed documents, small and ragged: resets and padding inside the sequence
        dict(name="train_T257", op="train", dt="bf16", B=2, H=4, Hk=2, T=257, dk=128, dv=128,
             S0=False, docs=True),
        # training at the bench's layer size
        dict(name="train_T4096", op="train", dt="bf16", B=8, H=16, Hk=16, T=4096, dk=128, dv=128,
             S0=False, docs=False),
        # training on one long sequence, value heads twice as wide
        dict(name="train_T32768", op="train", dt="bf16", B=1, H=16, Hk=16, T=32768, dk=128, dv=256,
             S0=False, docs=False),
        # the float32 layer
        dict(name="train_f32", op="train", dt="f32", B=4, H=8, Hk=8, T=2048, dk=64, dv=64,
             S0=False, docs=False),
        # queries and keys of a batch of single tokens, at far positions
        dict(name="norm_T1", op="norm", dt="bf16", B=64, T=1, H=16, Hk=8, d=128, rot=128,
             kind="rms", start=1000000, bwd=False),
        # forward over a training batch
        dict(name="norm_T4096", op="norm", dt="bf16", B=8, T=4096, H=16, Hk=16, d=128, rot=64,
             kind="l2", start=0, bwd=False),
        # forward and gradients over a training batch, with learned weights
        dict(name="norm_train", op="norm", dt="bf16", B=8, T=4096, H=16, Hk=16, d=128, rot=128,
             kind="rms", start=0, bwd=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "train", "norm", "fwd", "train"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    Hk = _log_int(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 2])
    if op == "norm":
        d = 8 * rng.randint(4, 16)
        rows = _log_int(rng, 1, 8 * 4096 * 32 // (H + Hk) * (128 if dt == "bf16" else 64) // 128)
        B = min(rows, _log_int(rng, 1, 64))
        return dict(op="norm", dt=dt, B=B, T=max(1, rows // B), H=H, Hk=Hk, d=d,
                    rot=16 * rng.randint(0, d // 16), kind=rng.choice(["l2", "rms"]),
                    start=_log_int(rng, 1, 4000000), bwd=rng.random() < 0.5)
    if dt == "bf16" and rng.random() < 0.75:  # the widths of the bench's layers
        dk, dv = 128, rng.choice([128, 128, 256])
    else:
        dk, dv = 8 * rng.randint(2, 16), 8 * rng.randint(2, 16)
    if op == "step":
        B = _log_int(rng, 1, 128)
        return dict(op="step", dt=dt, B=B, H=H, Hk=Hk, T=rng.choice([1, 1, 1, 2, 3, 8]), dk=dk,
                    dv=dv, pool=B + rng.randint(0, 40))
    B = _log_int(rng, 1, 8)
    # at most the listed cases' work, and at most 16384 chunks of the plain form in a row
    most = (8 * 16 * 4096) // (B * H) if dt == "bf16" else (4 * 8 * 2048 * 64 * 64) // (
        B * H * dk * dv)
    T = _log_int(rng, 1, max(1, min(32768, most * 128 // max(dv, 128))))
    return dict(op=op, dt=dt, B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv, S0=rng.random() < 0.5,
                docs=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    dt = DT[case["dt"]]
    s = dict(case=case)
    B, T, H, Hk = case["B"], case["T"], case["H"], case["Hk"]
    if case["op"] == "norm":
        d = case["d"]
        # one packed projection [B, T, H + Hk, d]: queries and keys are views of it
        qk = (normal(B, T, H + Hk, d) * (0.5 + uniform(1, 1, H + Hk, 1))).to(dt)
        s.update(q=qk[:, :, :H], k=qk[:, :, H:])
        s.update(wq=1 + 0.2 * normal(d), wk=1 + 0.2 * normal(d))
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) /
                                     max(half, 1))).float()
        first = (case["start"] * uniform(B, 1)).to(torch.int32)
        s["pos"] = first + torch.arange(T, device=DEV, dtype=torch.int32)
        if case["bwd"]:
            s.update(dyq=normal(B, H, T, d).to(dt), dyk=normal(B, Hk, T, d).to(dt))
    else:
        dk, dv = case["dk"], case["dv"]

        def unit(*shape):
            x = normal(*shape)
            return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

        s.update(q=unit(B, Hk, T, dk), k=unit(B, Hk, T, dk), v=normal(B, H, T, dv).to(dt))
        s["beta"] = torch.sigmoid(normal(B, H, T))
        # retention 1 - 10^U(-4, -1)
        s["log_alpha"] = torch.log1p(-10.0 ** (3 * uniform(B, H, T) - 4))
        s["scale"] = dk ** -0.5
        if case["op"] == "step":
            P = case["pool"]
            s["S"] = normal(P, H, dv, dk) / dk ** 0.5
            slots = torch.randperm(P, generator=g, device=DEV)[:B].to(torch.int32)
            s["slots"] = torch.where(torch.arange(B, device=DEV) % 8 == 7, -1, slots).to(
                torch.int32)
        else:
            if case["docs"]:
                # documents of about 100 tokens, each starting from an empty state, and a few
                # padding tokens (no update)
                start = uniform(B, 1, T) < 0.01
                pad = uniform(B, 1, T) < 0.03
                s["log_alpha"] = torch.where(start, NEG_INF, s["log_alpha"]).contiguous()
                s["beta"] = torch.where(pad, 0.0, s["beta"]).contiguous()
            s["S0"] = normal(B, H, dv, dk) / dk ** 0.5 if case["S0"] else None
            if case["op"] == "train":
                s["dy"] = normal(B, H, T, dv).to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    with torch.no_grad():
        return _run_plain(s, case)


def _run_own(s, case):
    import token_weight_scans_b200 as tw
    if case["op"] == "step":
        y = tw.gradlev_delta_step(s["q"], s["k"], s["v"], s["beta"], s["log_alpha"], s["S"],
                                  slots=s["slots"], scale=s["scale"])
        return dict(y=y, S=s["S"])
    if case["op"] == "fwd":
        y, ST = tw.gradlev_delta_fwd(s["q"], s["k"], s["v"], s["beta"], s["log_alpha"], s["S0"],
                                     scale=s["scale"])
        return dict(y=y, ST=ST)
    if case["op"] == "train":
        args = (s["q"], s["k"], s["v"], s["beta"], s["log_alpha"])
        ckpt = torch.empty(tw.gradlev_delta_ckpt_bytes(
            case["B"], case["H"], case["Hk"], case["T"], case["dk"], case["dv"],
            tw.BF16 if case["dt"] == "bf16" else tw.F32), dtype=torch.uint8, device=DEV)
        y, _ = tw.gradlev_delta_fwd(*args, s["S0"], scale=s["scale"], want_ST=False, ckpt=ckpt)
        out = tw.gradlev_delta_bwd(*args, s["dy"], s["S0"], scale=s["scale"], ckpt=ckpt,
                                   want_dS0=s["S0"] is not None)
        return dict(y=y, **{n: t for n, t in out.items() if t is not None})
    args = (s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"])
    yq, yk = tw.gradlev_qk_norm_rope_fwd(*args, norm=case["kind"])
    if not case["bwd"]:
        return dict(yq=yq, yk=yk)
    out = tw.gradlev_qk_norm_rope_bwd(s["dyq"], s["dyk"], *args, norm=case["kind"])
    return dict(yq=yq, yk=yk, **out)


# ------------------------------------------------------------------ plain forms
def _chunks(x, T):
    """[B, H, T, ...] -> [B, H, N, CHUNK, ...] in float32, the last chunk filled with zeros."""
    N = -(-T // CHUNK)
    if N * CHUNK != T:
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (N * CHUNK - T,) + x.shape[3:])], 2)
    return x.view(x.shape[:2] + (N, CHUNK) + x.shape[3:])


def _delta_plain(q, k, v, beta, log_alpha, S, scale):
    """The chunked form, all [B, H, T, .] float32. Returns y and the last state."""
    T = v.shape[2]
    q, k, v, b, la = (_chunks(x, T) for x in (q, k, v, beta, log_alpha))
    reset = torch.isinf(la)
    L = torch.where(reset, 0.0, la).cumsum(-1)
    seg = reset.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    seen = low & (seg[..., :, None] == seg[..., None, :])
    M = torch.where(seen, L[..., :, None] - L[..., None, :], 0.0).exp() * seen
    G = L.exp() * (seg == 0)
    A = ((k @ k.transpose(-1, -2)) * M * b[..., :, None]).tril(-1)
    # (I + A)^{-1} by doubling: the inverses of the diagonal blocks of size s join to those of 2 s
    at = torch.arange(CHUNK, device=v.device)
    X = torch.eye(CHUNK, device=v.device).expand_as(A)
    for level in range(6):
        i, j = at[:, None] >> level, at[None, :] >> level
        X = X - X @ (A * ((i == j + 1) & (i % 2 == 1))) @ X
    U = X @ (b[..., None] * v)
    W = X @ ((b * G)[..., None] * k)
    P = (q @ k.transpose(-1, -2)) * M
    Gq = G[..., None] * q
    Ke = M[..., -1, :, None] * k
    y = []
    for n in range(v.shape[2]):
        u = U[:, :, n] - W[:, :, n] @ S.transpose(-1, -2)
        y.append(scale * (Gq[:, :, n] @ S.transpose(-1, -2) + P[:, :, n] @ u))
        S = G[:, :, n, -1, None, None] * S + u.transpose(-1, -2) @ Ke[:, :, n]
    return torch.cat(y, 2)[:, :, :T], S


def _norm_plain(x, w, pos, inv_freq, kind, eps):
    """[B, T, H, d] float32 -> [B, H, T, d]."""
    ss = x.square().sum(-1, keepdim=True)
    x = x / ((ss / x.shape[-1] if kind == "rms" else ss) + eps).sqrt() * w
    half = inv_freq.numel()
    a = pos.double()[..., None, None] * inv_freq.double()
    c, s = torch.cos(a).float(), torch.sin(a).float()
    x1, x2, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s, rest], -1).transpose(1, 2)


EPS = 1e-6


def _run_plain(s, case):
    if case["op"] == "norm":
        dt = s["q"].dtype
        names = ("q", "k", "wq", "wk")
        f = [s[n].float() for n in names]
        if not case["bwd"]:
            return dict(yq=_norm_plain(f[0], f[2], s["pos"], s["inv_freq"], case["kind"],
                                       EPS).to(dt),
                        yk=_norm_plain(f[1], f[3], s["pos"], s["inv_freq"], case["kind"],
                                       EPS).to(dt))
        with torch.enable_grad():
            f = [x.requires_grad_() for x in f]
            # the weights' gradients are long sums: float64 copies of the weights collect them
            w64 = [w.detach().double().requires_grad_() for w in f[2:]]
            out = {}
            for n, x, w, dy in (("q", f[0], w64[0], s["dyq"]), ("k", f[1], w64[1], s["dyk"])):
                y = _norm_plain(x, _Spread.apply(w, x), s["pos"], s["inv_freq"], case["kind"], EPS)
                dx, dw = torch.autograd.grad(y, (x, w), dy.float())
                out.update({"y" + n: y.detach().to(dt), "d" + n: dx.to(dt),
                            "dw" + n: dw.float()})
        return out
    H, Hk = case["H"], case["Hk"]
    dt = s["v"].dtype

    def heads(x):
        return x.float().repeat_interleave(H // Hk, 1)

    if case["op"] == "step":
        q, k, v = heads(s["q"]), heads(s["k"]), s["v"].float()
        live = s["slots"] >= 0
        slots = s["slots"].long()
        S = s["S"][slots.clamp(min=0)]
        y = torch.zeros_like(v)
        for t in range(case["T"]):
            S = S * s["log_alpha"][:, :, t].exp()[..., None, None]
            e = v[:, :, t] - (S * k[:, :, t, None, :]).sum(-1)
            S = S + (s["beta"][:, :, t, None] * e)[..., None] * k[:, :, t, None, :]
            y[:, :, t] = s["scale"] * (S * q[:, :, t, None, :]).sum(-1)
        # rows without a state write nothing and answer with zeros
        rows = torch.arange(case["pool"], device=v.device)[:, None] == slots[None, :]
        hit = rows.any(1)
        s["S"].copy_(torch.where(hit[:, None, None, None], S[rows.to(torch.int8).argmax(1)],
                                 s["S"]))
        return dict(y=torch.where(live[:, None, None, None], y, 0.0).to(dt), S=s["S"])
    names = ("q", "k", "v", "beta", "log_alpha")
    f = {n: s[n].float() for n in names}
    S0 = s["S0"] if s["S0"] is not None else torch.zeros(
        case["B"], H, case["dv"], case["dk"], device=DEV)
    if case["op"] == "fwd":
        y, ST = _delta_plain(heads(f["q"]), heads(f["k"]), f["v"], f["beta"], f["log_alpha"], S0,
                             s["scale"])
        return dict(y=y.to(dt), ST=ST)
    with torch.enable_grad():
        for n in names:
            f[n] = f[n].clone().requires_grad_()
        S0 = S0.clone().requires_grad_()
        y, _ = _delta_plain(heads(f["q"]), heads(f["k"]), f["v"], f["beta"], f["log_alpha"], S0,
                            s["scale"])
        wrt = [f[n] for n in names] + ([S0] if s["S0"] is not None else [])
        grads = torch.autograd.grad(y, wrt, s["dy"].float())
    out = {"d" + n: x.to(dt) for n, x in zip(names + ("S0",), grads)}
    return dict(y=y.detach().to(dt), **out)


class _Spread(torch.autograd.Function):
    """A float64 weight read in 32 bits, its gradient summed in 64."""

    @staticmethod
    def forward(ctx, w, like):
        return w.float().expand_as(like).contiguous()

    @staticmethod
    def backward(ctx, g):
        return g.flatten(0, -2).sum(0, dtype=torch.float64), None


# ------------------------------------------------------------------ work
def work(case):
    es = 2 if case["dt"] == "bf16" else 4
    B, T, H, Hk = case["B"], case["T"], case["H"], case["Hk"]
    if case["op"] == "norm":
        n = B * T * (H + Hk) * case["d"]
        by = 2 * n * es + (2 * n * es if case["bwd"] else 0) + B * T * 4 + 16 * case["d"]
        return dict(bytes=by, flops=n * (20 if case["bwd"] else 7))
    dk, dv = case["dk"], case["dv"]
    qk, vv, gates, st = B * Hk * T * dk * es, B * H * T * dv * es, B * H * T * 4, B * H * dk * dv
    if case["op"] == "step":
        live = B - B // 8
        return dict(bytes=2 * qk + 2 * vv + 2 * gates + 8 * st * live // B,
                    flops=7 * st * T * live // B)
    S0 = 4 * st if case["S0"] else 0
    fwd = 6 * st * T
    if case["op"] == "fwd":
        return dict(bytes=2 * qk + 2 * vv + 2 * gates + S0 + 4 * st, flops=fwd)
    return dict(bytes=4 * qk + 4 * vv + 2 * gates + 2 * B * H * T * es + S0 +
                (es * st if case["S0"] else 0), flops=fwd + 14 * st * T)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    B, H, Hk, T, dk, dv = (case[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
    r = H // Hk
    group = torch.arange(H, device=DEV) // r
    # token-major copies: q[t] is [B, H, dk]
    q, k, v, b, a = (x.double().transpose(1, 2).transpose(0, 1).contiguous()
                     for x in (s["q"][:, group], s["k"][:, group], s["v"], s["beta"],
                               s["log_alpha"].double().exp()))

    def token(S, t):
        Sd = a[t][..., None, None] * S
        e = v[t] - torch.matmul(Sd, k[t][..., None])[..., 0]
        return Sd, e, Sd + (b[t][..., None] * e)[..., None] * k[t][..., None, :]

    y = torch.empty(T, B, H, dv, dtype=torch.float64, device=DEV)

    def out(S, t):
        torch.matmul(S, q[t][..., None] * s["scale"], out=y[t].unsqueeze(-1))

    def back(x):  # token-major -> [B, H, T, ...]
        return x.transpose(0, 1).transpose(1, 2)

    if case["op"] == "step":
        S = s["S"].double()[s["slots"].long().clamp(min=0)]
        for t in range(T):
            S = token(S, t)[2]
            out(S, t)
        live = s["slots"] >= 0
        y[:, ~live] = 0
        pool = s["S"].double()
        pool[s["slots"].long()[live]] = S[live]
        return dict(y=back(y), S=pool)
    S = s["S0"].double() if s["S0"] is not None else torch.zeros(B, H, dv, dk, dtype=torch.float64,
                                                                 device=DEV)
    part, starts = 64, []
    for t in range(T):
        if t % part == 0 and case["op"] == "train":
            starts.append(S)
        S = token(S, t)[2]
        out(S, t)
    if case["op"] == "fwd":
        return dict(y=back(y), ST=S)
    dq, dk_, dv_, db, dl = (torch.empty_like(x) for x in (q, k, v, b, a))
    dy = s["dy"].double().transpose(1, 2).transpose(0, 1).contiguous()
    lam = torch.zeros_like(S)
    for n in reversed(range(len(starts))):
        S, seen = starts[n], []
        for t in range(n * part, min(T, (n + 1) * part)):
            Sd, e, S = token(S, t)
            seen.append((Sd, e, S))
        for t in reversed(range(n * part, min(T, (n + 1) * part))):
            Sd, e, S = seen[t - n * part]
            g = s["scale"] * dy[t]
            dq[t] = torch.matmul(S.transpose(-1, -2), g[..., None])[..., 0]
            lam = lam + g[..., None] * q[t][..., None, :]
            du = torch.matmul(lam, k[t][..., None])[..., 0]
            db[t] = (du * e).sum(-1)
            de = b[t][..., None] * du
            dv_[t] = de
            dk_[t] = (torch.matmul(lam.transpose(-1, -2), (b[t][..., None] * e)[..., None]) -
                      torch.matmul(Sd.transpose(-1, -2), de[..., None]))[..., 0]
            lam = lam - de[..., None] * k[t][..., None, :]
            dl[t] = (lam * Sd).sum((-1, -2))
            lam = a[t][..., None, None] * lam

    def shared(x):  # the value heads of a key head add up
        return x.view(B, Hk, r, T, dk).sum(2)

    res = dict(y=back(y), dq=shared(back(dq)), dk=shared(back(dk_)), dv=back(dv_), dbeta=back(db),
               dlog_alpha=back(dl))
    if s["S0"] is not None:
        res["dS0"] = lam
    return res


def _exact_norm(s, case):
    d, half = case["d"], case["rot"] // 2
    ang = s["pos"].double()[:, None, :, None] * s["inv_freq"].double()
    res = {}
    for n, dy in (("q", s.get("dyq")), ("k", s.get("dyk"))):
        x = s[n].double().transpose(1, 2)  # [B, H, T, d]
        w = s["w" + n].double()
        div = d if case["kind"] == "rms" else 1
        r = (x.pow(2).sum(-1, keepdim=True) / div + EPS).rsqrt()
        z = x * r
        turn = torch.polar(torch.ones_like(ang), ang)
        y = z * w
        pair = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
        res["y" + n] = torch.cat([pair.real, pair.imag, y[..., 2 * half:]], -1)
        if dy is None:
            continue
        g = dy.double()
        pair = torch.complex(g[..., :half], g[..., half:2 * half]) * turn.conj()
        g = torch.cat([pair.real, pair.imag, g[..., 2 * half:]], -1)
        res["dw" + n] = (g * z).sum((0, 1, 2))
        g = g * w
        res["d" + n] = ((g - z * (g * z).sum(-1, keepdim=True) / div) * r).transpose(1, 2)
    return res
