"""GPU tests of the gated delta rule (gradlev_delta_fwd, _bwd, _step) against the 64-bit
token-by-token reference.

Tolerances (2-norm of the difference over the reference's), fixed before the first run:
- float32 and every CUDA-core product: a value is at the end of at most four products in a
  row (K S^T, Z R, P D, the state update), each a sum of at most 256 terms with a rounding
  of 2^-24 apiece: 4 * 256 * 2^-24 = 6.1e-5. The rule contracts, so errors of earlier
  tokens do not add up beyond that.
- bf16 I/O: half a step, 2^-8, per rounding to bf16 on the way to an output. The outputs'
  own rounding is one; the tensor-core kernels round their operands too. Independent
  roundings add up as squares: sqrt(n) 2^-8 with the n below.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

F32_TOL = 4 * 256 * 2.0 ** -24
HALF = 2.0 ** -8
# roundings to bf16 on the way: y: W, S, D, P, itself. dv: P T, W', dS, dY G Q, E, itself.
# dq and dk: those of D and E, the states, X, Y, themselves. Gates: D and E twice over.
ROUNDINGS = dict(y=5, dv=6, dq=8, dk=10, dbeta=10, dlog_alpha=12, dS0=8)
NAMES = ("q", "k", "v", "beta", "log_alpha")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    yield


def tol(name, dtype):
    if name in ("ST", "S") or dtype == "f32":
        return F32_TOL
    return F32_TOL + ROUNDINGS[name] ** 0.5 * HALF


def dev(d):
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def code(dtype):
    return tw.BF16 if dtype == "bf16" else tw.F32


def check(got, want, dtype, names=None):
    for n in names or want:
        assert torch.isfinite(got[n].float()).all(), n
        err = ref.rel2(got[n], want[n])
        assert err <= tol(n, dtype), (n, err, tol(n, dtype))


CASES = [
    # (B, H, Hk, T, dk, dv, dtype, S0, mask)
    (1, 1, 1, 1, 8, 8, "f32", False, "none"),
    (1, 1, 1, 1, 8, 8, "f32", True, "none"),
    (2, 4, 2, 33, 16, 24, "f32", True, "docs"),
    (1, 2, 1, 100, 64, 64, "f32", False, "none"),
    (1, 2, 2, 257, 128, 128, "f32", True, "docs"),
    (1, 1, 1, 70, 256, 64, "f32", True, "none"),
    (1, 1, 1, 40, 64, 256, "f32", False, "none"),
    (1, 1, 1, 45, 256, 256, "f32", True, "none"),
    (1, 6, 2, 64, 40, 72, "f32", False, "docs"),
    (2, 2, 2, 31, 16, 16, "f32", True, "empty"),
    (1, 2, 2, 65, 16, 16, "f32", True, "reset"),
    (2, 4, 2, 33, 16, 24, "bf16", True, "docs"),
    (1, 2, 1, 100, 64, 64, "bf16", False, "none"),
    (1, 1, 1, 1, 128, 128, "bf16", False, "none"),
    (1, 1, 1, 1, 128, 256, "bf16", True, "none"),
    (1, 2, 2, 63, 128, 128, "bf16", True, "none"),
    (1, 2, 2, 64, 128, 128, "bf16", False, "none"),
    (1, 2, 1, 65, 128, 256, "bf16", True, "none"),
    (2, 4, 2, 257, 128, 128, "bf16", True, "docs"),
    (1, 3, 1, 200, 128, 256, "bf16", True, "docs"),
    (2, 2, 2, 130, 128, 128, "bf16", True, "empty"),
    (1, 2, 2, 130, 128, 128, "bf16", True, "reset"),
    (1, 2, 2, 1100, 128, 128, "bf16", True, "none"),
    # heads narrower than the tensor-core tiles
    (2, 2, 1, 150, 64, 64, "bf16", True, "docs"),
    (1, 3, 3, 257, 8, 8, "bf16", True, "none"),
    (2, 2, 2, 130, 72, 200, "bf16", True, "none"),
    (1, 2, 1, 1000, 120, 136, "bf16", True, "docs"),
    (1, 2, 1, 257, 128, 40, "bf16", False, "none"),
    (2, 2, 1, 100, 136, 64, "bf16", True, "none"),
    # the same with gates enough for the tensor-core gradients (few gates, or narrow heads with
    # fewer than 8192, take the float32 kernels)
    (20, 64, 32, 1, 128, 128, "bf16", True, "none"),
    (9, 2, 2, 63, 128, 128, "bf16", True, "none"),
    (9, 2, 2, 64, 128, 128, "bf16", False, "none"),
    (9, 2, 1, 65, 128, 256, "bf16", True, "none"),
    (3, 3, 1, 200, 128, 256, "bf16", True, "docs"),
    (5, 2, 2, 130, 128, 128, "bf16", True, "empty"),
    (5, 2, 2, 130, 128, 128, "bf16", True, "reset"),
    (4, 2, 1, 150, 64, 64, "bf16", True, "docs"),
    (5, 2, 2, 130, 72, 200, "bf16", True, "none"),
    (3, 2, 1, 257, 128, 40, "bf16", False, "none"),
    (8, 4, 2, 257, 40, 72, "bf16", True, "docs"),
    (4, 8, 8, 257, 24, 136, "bf16", True, "none"),
    # few long scans, walked in segments
    (1, 2, 1, 1283, 128, 256, "bf16", True, "none"),
    (1, 2, 1, 1283, 128, 256, "bf16", False, "docs"),
    (1, 1, 1, 2049, 128, 128, "bf16", True, "docs"),
    (2, 3, 3, 770, 128, 128, "bf16", False, "empty"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(case):
    B, H, Hk, T, dk, dv, dtype, S0, mask = case
    d = ref.draw(B, H, Hk, T, dk, dv, dtype, S0, mask, seed=T + dk)
    g = dev(d)
    x = ref.f64(d)
    scale = dk ** -0.5
    dST = torch.randn(B, H, dv, dk, generator=torch.Generator().manual_seed(9)).to(d["v"].dtype)
    y64, S64 = ref.forward(*[x[n] for n in NAMES], scale, x["S0"])
    want = ref.gradients(*[x[n] for n in NAMES], scale, x["S0"], x["dy"], dST.to(ref.F64))
    args = [g[n] for n in NAMES]
    ck = torch.empty(tw.gradlev_delta_ckpt_bytes(B, H, Hk, T, dk, dv, code(dtype)),
                     dtype=torch.uint8, device="cuda")
    y, ST = tw.gradlev_delta_fwd(*args, g["S0"])
    check(dict(y=y, ST=ST), dict(y=y64, ST=S64), dtype)
    y, none = tw.gradlev_delta_fwd(*args, g["S0"], want_ST=False, ckpt=ck)
    assert none is None
    check(dict(y=y), dict(y=y64), dtype)
    out = tw.gradlev_delta_bwd(*args, g["dy"], g["S0"], dST.cuda(), ckpt=ck)
    if mask == "reset":  # every token starts anew: nothing flows through the gates
        assert not out["dlog_alpha"].any() and not out["dS0"].any()
        check(out, want, dtype, ["dq", "dk", "dv", "dbeta"])
    else:
        check(out, want, dtype)
    # without checkpoints the states are recomputed: the same bits
    again = tw.gradlev_delta_bwd(*args, g["dy"], g["S0"], dST.cuda())
    for n in out:
        assert torch.equal(out[n], again[n]), n
    # checkpoints of a forward that also gave the last state
    y, ST = tw.gradlev_delta_fwd(*args, g["S0"], ckpt=ck)
    check(dict(y=y, ST=ST), dict(y=y64, ST=S64), dtype)
    out = tw.gradlev_delta_bwd(*args, g["dy"], g["S0"], dST.cuda(), ckpt=ck)
    check(out, want, dtype, [n for n in want if mask != "reset" or n in ("dq", "dk", "dv", "dbeta")])


@pytest.mark.parametrize("B,H,dtype,d", [(1, 2, "f32", 32), (1, 2, "bf16", 128), (40, 8, "bf16", 128)])
def test_first_token_of_an_empty_state_has_no_gate_gradient(B, H, dtype, d):
    """One token and no start state: log_alpha multiplies zero, so its gradient is zero itself."""
    g = dev(ref.draw(B, H, H, 1, d, d, dtype, False, seed=3))
    out = tw.gradlev_delta_bwd(*[g[n] for n in NAMES], g["dy"])
    assert not out["dlog_alpha"].any()


@pytest.mark.parametrize("dtype,dv", [("f32", 32), ("bf16", 128), ("bf16", 256)])
def test_split_sequence_carries_the_state(dtype, dv):
    B, H, Hk, T, dk, cut = 8 if dtype == "bf16" else 1, 2, 1, 150, 128 if dtype == "bf16" else 32, 77
    d = ref.draw(B, H, Hk, T, dk, dv, dtype, True, seed=4)
    g = dev(d)
    x = ref.f64(d)
    want = ref.gradients(*[x[n] for n in NAMES], dk ** -0.5, x["S0"], x["dy"])
    y64, S64 = ref.forward(*[x[n] for n in NAMES], dk ** -0.5, x["S0"])
    part = lambda t, s: t[:, :, s].contiguous()  # noqa: E731
    a, b = slice(0, cut), slice(cut, T)
    A, Bp = ([part(g[n], s) for n in NAMES] for s in (a, b))
    ya, Sa = tw.gradlev_delta_fwd(*A, g["S0"])
    yb, Sb = tw.gradlev_delta_fwd(*Bp, Sa)
    check(dict(y=torch.cat([ya, yb], 2), ST=Sb), dict(y=y64, ST=S64), dtype)
    gb = tw.gradlev_delta_bwd(*Bp, part(g["dy"], b), Sa)
    ga = tw.gradlev_delta_bwd(*A, part(g["dy"], a), g["S0"], gb["dS0"])
    joined = {n: torch.cat([ga[n], gb[n]], 2) for n in ga if n != "dS0"}
    check(dict(joined, dS0=ga["dS0"]), want, dtype)


@pytest.mark.parametrize("B,H,Hk,T,dk,dv,dtype", [
    (1, 2, 2, 1, 128, 128, "bf16"), (3, 4, 2, 1, 128, 256, "bf16"), (2, 2, 1, 9, 64, 64, "f32"),
    (2, 2, 1, 3, 32, 40, "f32"), (2, 2, 2, 2, 256, 33, "bf16"), (1, 1, 1, 4, 4, 1, "f32"),
    (9, 2, 2, 2, 100, 128, "bf16"),
    (40, 32, 16, 2, 128, 100, "bf16"), (75, 32, 32, 1, 24, 130, "f32"),  # 8 rows per lane group
])
def test_step(B, H, Hk, T, dk, dv, dtype):
    d = ref.draw(B, H, Hk, T, dk, dv, dtype, True, "docs" if T == 9 else "none", seed=dk + T)
    g, x = dev(d), ref.f64(d)
    y64, S64 = ref.forward(*[x[n] for n in NAMES], 0.3, x["S0"])
    S = g["S0"].clone()
    y = tw.gradlev_delta_step(*[g[n] for n in NAMES], S, scale=0.3)
    check(dict(y=y, S=S), dict(y=y64, S=S64), dtype)
    # one call per token: the same bits
    S2, ys = g["S0"].clone(), []
    for t in range(T):
        ys.append(tw.gradlev_delta_step(*[g[n][:, :, t:t + 1].contiguous() for n in NAMES], S2,
                                        scale=0.3))
    assert torch.equal(torch.cat(ys, 2), y) and torch.equal(S, S2)


def test_step_slots():
    """Padding rows, slots outside the pool and repeated slots answer with zeros and write no
    state; pool rows that no row names keep their bits."""
    B, H, dk, dv, pool = 7, 2, 64, 48, 6
    d = ref.draw(B, H, 1, 2, dk, dv, "f32", seed=2)
    g, x = dev(d), ref.f64(d)
    slots = torch.tensor([3, -1, 0, 3, 6, 5, 2 ** 31 - 1], dtype=torch.int32)
    first = torch.randn(pool, H, dv, dk, generator=torch.Generator().manual_seed(3))
    S = first.cuda()
    y = tw.gradlev_delta_step(*[g[n] for n in NAMES], S, slots=slots.cuda(), scale=1.0)
    live = [0, 2, 5]
    y64, S64 = ref.forward(*[x[n][live] for n in NAMES], 1.0, first[slots[live].long()].double())
    check(dict(y=y[live], S=S[slots[live].long().cuda()]), dict(y=y64, S=S64), "f32")
    assert not y[[1, 3, 4, 6]].any()
    assert torch.equal(S[[1, 2, 4]].cpu(), first[[1, 2, 4]])


@pytest.mark.parametrize("B,H,T,dk,dv,dtype", [
    (1, 2, 40, 32, 32, "f32"), (2, 2, 100, 136, 64, "bf16"), (2, 4, 100, 128, 128, "bf16"),
    (4, 4, 100, 128, 128, "bf16"),
    (1, 2, 1283, 128, 256, "bf16"), (2, 2, 3, 64, 64, "bf16")])
def test_a_reset_first_token_forgets_any_state(B, H, T, dk, dv, dtype):
    """What S0 or the pool holds, NaN and infinities among it, does not matter to a scan whose
    first token is a reset; the other scans of the call keep theirs."""
    d = ref.draw(B, H, H, T, dk, dv, dtype, True, seed=8)
    d["log_alpha"][:, 0, 0] = float("-inf")
    d["S0"][:, 0] = 0.0
    g = dev(d)
    args, zero = [g[n] for n in NAMES], g["S0"]
    junk = zero.clone()
    junk[:, 0] = float("nan")
    junk[:, 0, ::2] = float("inf")
    for want_ST in (False, True):
        got, want = (tw.gradlev_delta_fwd(*args, s, want_ST=want_ST) for s in (junk, zero))
        assert torch.equal(got[0], want[0]) and torch.isfinite(got[0].float()).all()
        assert not want_ST or torch.equal(got[1], want[1])
    got, want = (tw.gradlev_delta_bwd(*args, g["dy"], s) for s in (junk, zero))
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.isfinite(got[n].float()).all(), n
    a, b = junk.clone(), zero.clone()
    ya, yb = (tw.gradlev_delta_step(*args, s) for s in (a, b))
    assert torch.equal(ya, yb) and torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 24, 40), ("bf16", 128, 128), ("bf16", 128, 256),
                                         ("bf16", 40, 72), ("bf16", 72, 136)])
def test_outputs_stay_inside_their_buffers(dtype, dk, dv):
    B, H, Hk, T = 8, 2, 2, 70
    d = dev(ref.draw(B, H, Hk, T, dk, dv, dtype, True, seed=6))
    args = [d[n] for n in NAMES]
    size = (B, H, Hk, T, dk, dv, code(dtype))
    held = []

    def buf(shape, dt):  # a tensor with 1 KB of pattern on both sides
        n = int(np.prod(shape)) * torch.empty(0, dtype=dt).element_size()
        raw = torch.full((n + 2048,), 0x5A, dtype=torch.uint8, device="cuda")
        held.append((raw, n))
        return raw[1024:1024 + n].view(dt).view(shape)

    dt, f32, u8 = d["v"].dtype, torch.float32, torch.uint8
    y, ST = buf((B, H, T, dv), dt), buf((B, H, dv, dk), f32)
    ck = buf((tw.gradlev_delta_ckpt_bytes(*size),), u8)
    wf, wb = (buf((tw.gradlev_delta_workspace_bytes(*size, b),), u8) for b in (0, 1))
    out = dict(dq=buf((B, Hk, T, dk), dt), dk=buf((B, Hk, T, dk), dt), dv=buf((B, H, T, dv), dt),
               dbeta=buf((B, H, T), dt), dlog_alpha=buf((B, H, T), dt),
               dS0=buf((B, H, dv, dk), dt))
    tw.gradlev_delta_fwd(*args, d["S0"], y=y, ST=ST, ckpt=ck, workspace=wf)
    tw.gradlev_delta_bwd(*args, d["dy"], d["S0"], ckpt=ck, workspace=wb, out=out)
    tw.gradlev_delta_bwd(*args, d["dy"], d["S0"], workspace=wb, out=out)
    torch.cuda.synchronize()
    for raw, n in held:
        assert (raw[:1024] == 0x5A).all() and (raw[1024 + n:] == 0x5A).all()
    assert tw.gradlev_device_status(wf) == 0 and tw.gradlev_device_status(wb) == 0


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 32, 32), ("bf16", 128, 128)])
def test_graph_replay_and_streams(dtype, dk, dv):
    """A captured pass replayed on new inputs, and a pass on another stream, give the bits of
    an eager pass; two graphs with their own workspaces do not disturb each other."""
    B, H, Hk, T = 2, 4, 2, 200
    size = (B, H, Hk, T, dk, dv, code(dtype))
    sets = [dev(ref.draw(B, H, Hk, T, dk, dv, dtype, True, seed=s)) for s in (1, 2, 3)]

    def bufs():
        return dict(ck=torch.empty(tw.gradlev_delta_ckpt_bytes(*size), dtype=torch.uint8, device="cuda"),
                    wf=torch.empty(tw.gradlev_delta_workspace_bytes(*size, 0), dtype=torch.uint8, device="cuda"),
                    wb=torch.empty(tw.gradlev_delta_workspace_bytes(*size, 1), dtype=torch.uint8, device="cuda"))

    def one(d, b):
        args = [d[n] for n in NAMES]
        y, ST = tw.gradlev_delta_fwd(*args, d["S0"], ckpt=b["ck"], workspace=b["wf"])
        out = tw.gradlev_delta_bwd(*args, d["dy"], d["S0"], ckpt=b["ck"], workspace=b["wb"])
        return dict(out, y=y, ST=ST)

    eager = [one(d, bufs()) for d in sets]
    graphs = []
    for d in sets[:2]:
        held = {n: x.clone() for n, x in d.items()}
        b = bufs()
        one(held, b)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = one(held, b)
        graphs.append((gr, held, res, b))
    for gr, *_ in graphs:
        gr.replay()
    for i, (gr, held, res, _) in enumerate(graphs):
        for n in res:
            assert torch.equal(res[n], eager[i][n]), n
    gr, held, res, _ = graphs[0]
    for n in held:
        held[n].copy_(sets[2][n])
    gr.replay()
    torch.cuda.synchronize()
    for n in res:
        assert torch.equal(res[n], eager[2][n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        res = one(sets[1], bufs())
    side.synchronize()
    for n in res:
        assert torch.equal(res[n], eager[1][n]), n


def test_the_layer_end_to_end():
    """The operators as a layer uses them: norms and rotation from a packed projection, the
    chunked rule over a prompt, then token by token; and the gradients of the training form."""
    B, T, H, Hk, d, dv, prompt = 2, 90, 4, 2, 128, 128, 83
    gen = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    td = torch.bfloat16
    packed = r(B, T, 2 * Hk, d).to(td)
    v, dy = r(B, H, T, dv).to(td), r(B, H, T, dv).to(td)
    beta = torch.sigmoid(r(B, H, T))
    la = torch.log1p(-10.0 ** (3 * torch.rand((B, H, T), generator=gen) - 4))
    wq, wk = 1 + 0.1 * r(d), torch.ones(d)
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float()
    pos = (torch.tensor([[5], [70000]]) + torch.arange(T)).to(torch.int32)
    # 64-bit chain
    leaves = [x.to(ref.F64).requires_grad_() for x in (packed, wq, wk, v)]
    p64, wq64, wk64, v64 = leaves
    q64 = ref.norm_rope(p64[:, :, :Hk], wq64, pos, inv, "l2", 1e-6)
    k64 = ref.norm_rope(p64[:, :, Hk:], wk64, pos, inv, "l2", 1e-6)
    y64, S64 = ref.forward(q64, k64, v64, beta.double(), la.double(), d ** -0.5)
    (y64 * dy.double()).sum().backward()
    # the library
    pk, vg, bg, lg, dyg, posg = (x.cuda() for x in (packed, v, beta, la, dy, pos))
    args = (pk[:, :, :Hk], pk[:, :, Hk:], wq.cuda(), wk.cuda(), posg, inv.cuda())
    q, k = tw.gradlev_qk_norm_rope_fwd(*args)
    ck = torch.empty(tw.gradlev_delta_ckpt_bytes(B, H, Hk, T, d, dv, tw.BF16), dtype=torch.uint8,
                     device="cuda")
    y, ST = tw.gradlev_delta_fwd(q, k, vg, bg, lg, ckpt=ck)
    g = tw.gradlev_delta_bwd(q, k, vg, bg, lg, dyg, ckpt=ck)
    dpk = torch.empty_like(pk)
    gn = tw.gradlev_qk_norm_rope_bwd(g["dq"], g["dk"], *args, out=dict(
        dq=dpk[:, :, :Hk], dk=dpk[:, :, Hk:], dwq=torch.empty(d, device="cuda"),
        dwk=torch.empty(d, device="cuda")))
    # q and k round once more, in front of everything
    extra = 2 ** 0.5
    assert ref.rel2(y, y64.detach()) <= extra * tol("y", "bf16")
    assert ref.rel2(g["dv"], v64.grad) <= extra * tol("dv", "bf16")
    assert ref.rel2(dpk, p64.grad) <= extra * tol("dk", "bf16")
    assert ref.rel2(gn["dwq"], wq64.grad) <= extra * tol("dq", "bf16")
    assert ref.rel2(gn["dwk"], wk64.grad) <= extra * tol("dk", "bf16")
    # serving: the prompt in chunks, the rest token by token
    cut = lambda t, a, b: t[:, :, a:b].contiguous()  # noqa: E731
    yp, S = tw.gradlev_delta_fwd(*[cut(t, 0, prompt) for t in (q, k, vg, bg, lg)])
    ys = [yp]
    for t in range(prompt, T):
        ys.append(tw.gradlev_delta_step(*[cut(x, t, t + 1) for x in (q, k, vg, bg, lg)], S))
    assert ref.rel2(torch.cat(ys, 2), y64.detach()) <= extra * tol("y", "bf16")
    assert ref.rel2(S, ST.cpu()) <= 2 * F32_TOL


@pytest.mark.parametrize("site,want_ST", [(5, False), (5, True), (6, False)])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_device_usable(site, want_ST):
    B, H, T, d = 1, 2, 600, 128
    g = dev(ref.draw(B, H, H, T, d, d, "bf16", True, seed=5))
    args = [g[n] for n in NAMES]
    size = (B, H, H, T, d, d, tw.BF16)
    ws = [torch.empty(tw.gradlev_delta_workspace_bytes(*size, b), dtype=torch.uint8, device="cuda")
          for b in (0, 1)]
    ck = torch.empty(tw.gradlev_delta_ckpt_bytes(*size), dtype=torch.uint8, device="cuda")

    def run():
        y, ST = tw.gradlev_delta_fwd(*args, g["S0"], want_ST=want_ST, ckpt=ck, workspace=ws[0])
        out = tw.gradlev_delta_bwd(*args, g["dy"], ckpt=ck, workspace=ws[1])
        return dict(out, y=y, ST=ST), [tw.gradlev_device_status(w) for w in ws]

    good, status = run()
    assert status == [0, 0]
    tw.lib().gradlev_debug_inject_timeout(site, 20)
    _, status = run()
    assert status[site - 5] == 5  # GRADLEV_ERR_TIMEOUT
    again, status = run()
    assert status == [0, 0]
    for n in good:
        assert good[n] is None or torch.equal(good[n], again[n]), n


def test_calls_on_a_stream_of_their_own():
    """stream=: the work goes to that stream, with buffers the call allocates itself."""
    d = dev(ref.draw(2, 4, 2, 200, 128, 128, "bf16", True, seed=6))
    args = [d[n] for n in NAMES]
    y0, S0 = tw.gradlev_delta_fwd(*args, d["S0"])
    g0 = tw.gradlev_delta_bwd(*args, d["dy"], d["S0"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y, S = tw.gradlev_delta_fwd(*args, d["S0"], stream=side)
        g = tw.gradlev_delta_bwd(*args, d["dy"], d["S0"], stream=side)
        torch.empty(1 << 22, device="cuda").fill_(1.0)  # would reuse what the calls let go
    side.synchronize()
    assert torch.equal(y, y0) and torch.equal(S, S0)
    for n in g0:
        assert torch.equal(g[n], g0[n]), n


def test_binding_refusals():
    d = dev(ref.draw(1, 2, 1, 8, 16, 16, S0=True))
    args = [d[n] for n in NAMES]

    def bad(i, t):
        return args[:i] + [t] + args[i + 1:]

    for a in (bad(0, args[0].transpose(2, 3)), bad(1, args[1][:, :, :4]), bad(2, args[2].bfloat16()),
              bad(3, args[3].double()), bad(4, args[4][0]), bad(0, args[0].half()),
              bad(1, args[1].cpu())):
        with pytest.raises(tw.GradlevError):
            tw.gradlev_delta_fwd(*a)
        with pytest.raises(tw.GradlevError):
            tw.gradlev_delta_bwd(*a, d["dy"])
        with pytest.raises(tw.GradlevError):
            tw.gradlev_delta_step(*a, d["S0"])
    tiny = torch.empty(8, dtype=torch.uint8, device="cuda")
    with pytest.raises(tw.GradlevError, match="too small"):
        tw.gradlev_delta_fwd(*args, workspace=tiny)
    with pytest.raises(tw.GradlevError, match="too small"):
        tw.gradlev_delta_fwd(*args, ckpt=tiny)
    with pytest.raises(tw.GradlevError, match="too small"):
        tw.gradlev_delta_bwd(*args, d["dy"], ckpt=tiny)
    with pytest.raises(tw.GradlevError):
        tw.gradlev_delta_step(*args, d["S0"], slots=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(tw.GradlevError):
        tw.gradlev_delta_bwd(*args, d["dy"], dST=d["S0"].bfloat16())


def _room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip(f"needs {gb} GB")


@pytest.mark.parametrize("dtype,T,gb", [("bf16", 1 << 20, 110), ("f32", 1 << 19, 125)])
def test_offsets_past_32_bits(dtype, T, gb):
    """Tensors of more than 2^31 elements and states of more than 2^32: the first 1024 tokens
    and the last (behind a reset) have the bits of a call on them alone."""
    _room(gb)
    H, d, tail = 18, 128, 1024
    size = (1, H, H, T, d, d, code(dtype))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v, dy = (torch.randn(1, H, T, d, generator=gen, dtype=dt, device="cuda") for _ in range(4))
    k *= d ** -0.5 / 1.5  # |k|^2 below 1
    beta = torch.rand(1, H, T, generator=gen, device="cuda")
    la = -0.1 * torch.rand(1, H, T, generator=gen, device="cuda")
    la[:, :, T - tail] = float("-inf")
    full = (q, k, v, beta, la, dy)
    first, last = ([x[:, :, s].contiguous() for x in full] for s in (slice(tail), slice(T - tail, T)))

    def run(a):
        n = a[0].shape[2]
        ck = torch.empty(tw.gradlev_delta_ckpt_bytes(1, H, H, n, d, d, size[-1]), dtype=torch.uint8,
                         device="cuda")
        y, ST = tw.gradlev_delta_fwd(*a[:5], ckpt=ck)
        return dict(tw.gradlev_delta_bwd(*a, ckpt=ck), y=y, ST=ST)

    got, front, back = run(full), run(first), run(last)
    assert torch.equal(got["y"][:, :, :tail], front["y"])
    assert torch.equal(got["ST"], back["ST"])
    for n in ("y", "dq", "dk", "dv", "dbeta", "dlog_alpha"):
        assert torch.equal(got[n][:, :, T - tail:], back[n]), n


def test_step_in_a_pool_past_32_bits():
    _room(25)
    pool, H, d = 8300, 32, 128  # 4.35e9 elements
    g = dev(ref.draw(2, H, H, 1, d, d, "f32", True, seed=12))
    args, S = [g[n] for n in NAMES], torch.zeros(pool, H, d, d, device="cuda")
    at = torch.tensor([pool - 1, 0], device="cuda")
    S[at] = g["S0"]
    y = tw.gradlev_delta_step(*args, S, slots=at.int())
    want = tw.gradlev_delta_step(*args, g["S0"])
    assert torch.equal(y, want) and torch.equal(S[at], g["S0"]) and not S[1:pool - 1].any()


def test_calls_at_once_on_two_streams():
    """Passes that overlap on the GPU, a workspace each (their own allocations): the bits of passes
    one after the other."""
    sets = [dev(ref.draw(2, 4, h, 700, 128, d, "bf16", True, seed=20 + h)) for h, d in ((4, 128), (2, 256))]

    def one(d, stream=None):
        args = [d[n] for n in NAMES]
        y, ST = tw.gradlev_delta_fwd(*args, d["S0"], stream=stream)
        return dict(tw.gradlev_delta_bwd(*args, d["dy"], d["S0"], stream=stream), y=y, ST=ST)

    alone = [one(d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [one(d, st) for d, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for g, a in zip(got, alone):
        for n in a:
            assert torch.equal(g[n], a[n]), n
