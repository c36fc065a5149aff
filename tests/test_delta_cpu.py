"""Gated delta rule and query/key norms without a GPU: the 64-bit reference against
autograd and differences, and every refusal of the entry points and the binding."""

import ctypes

import pytest
import torch

import token_weight_scans_b200 as tw
from tests import delta_ref as ref
from token_weight_scans_b200 import build as tw_build

P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: the checks come first
NULL = P(0)
NAMES = ("q", "k", "v", "beta", "log_alpha", "S0")


@pytest.fixture(scope="module")
def L():
    tw_build.build()
    return tw.lib()


def test_reference_gradients_match_autograd_and_differences():
    d = ref.f64(ref.draw(2, 4, 2, 9, 8, 6, S0=True, seed=3))
    dST = torch.randn(2, 4, 6, 8, dtype=ref.F64, generator=torch.Generator().manual_seed(1))
    leaves = {n: d[n].clone().requires_grad_() for n in NAMES}

    def loss(**over):
        x = {**{n: d[n] for n in NAMES}, **over}
        y, S = ref.forward(x["q"], x["k"], x["v"], x["beta"], x["log_alpha"], 0.3, x["S0"])
        return (y * d["dy"]).sum() + (S * dST).sum()

    loss(**leaves).backward()
    got = ref.gradients(*[d[n] for n in NAMES[:5]], 0.3, d["S0"], d["dy"], dST)
    for n in NAMES:
        assert ref.rel2(got["d" + n], leaves[n].grad) < 1e-13, n
        # central differences: error of order h^2 and eps / h
        way = torch.randn(d[n].shape, dtype=ref.F64, generator=torch.Generator().manual_seed(5))
        h = 1e-5
        diff = (loss(**{n: d[n] + h * way}) - loss(**{n: d[n] - h * way})) / (2 * h)
        assert abs(float(diff - (got["d" + n] * way).sum())) < 1e-7 * (1 + abs(float(diff))), n


def test_reset_and_padding_in_the_reference():
    """log_alpha = -inf cuts the sequence; beta = 0 leaves the state to its decay."""
    d = ref.f64(ref.draw(1, 1, 1, 8, 8, 8, seed=1))
    d["log_alpha"][..., 5] = float("-inf")
    y, S = ref.forward(*[d[n] for n in NAMES[:5]], 1.0)
    y2, S2 = ref.forward(*[d[n][:, :, 5:] for n in NAMES[:5]], 1.0)
    assert torch.equal(y[:, :, 5:], y2) and torch.equal(S, S2)
    g = ref.gradients(*[d[n] for n in NAMES[:5]], 1.0, None, d["dy"])
    assert float(g["dlog_alpha"][..., 5]) == 0.0


def fwd(L, B=1, H=2, Hk=1, T=8, dk=16, dv=16, dt=0, ws_bytes=1 << 30, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, beta=FAKE, la=FAKE, S0=NULL, y=FAKE, ST=NULL, ckpt=NULL,
             ws=FAKE)
    a.update(over)
    return L.gradlev_delta_fwd(B, H, Hk, T, dk, dv, dt, a["q"], a["k"], a["v"], a["beta"], a["la"],
                               1.0, a["S0"], a["y"], a["ST"], a["ckpt"], a["ws"], ws_bytes, NULL)


def bwd(L, B=1, H=2, Hk=1, T=8, dk=16, dv=16, dt=0, ws_bytes=1 << 30, **over):
    a = {n: FAKE for n in ("q", "k", "v", "beta", "la", "dy", "dq", "gk", "gv", "db", "dl", "ws")}
    a.update({n: NULL for n in ("S0", "dST", "dS0", "ckpt")})
    a.update(over)
    return L.gradlev_delta_bwd(B, H, Hk, T, dk, dv, dt, a["q"], a["k"], a["v"], a["beta"], a["la"],
                               1.0, a["S0"], a["dy"], a["dST"], a["dq"], a["gk"], a["gv"], a["db"],
                               a["dl"], a["dS0"], a["ckpt"], a["ws"], ws_bytes, NULL)


def step(L, B=1, H=2, Hk=1, T=1, dk=16, dv=16, dt=0, pool=4, **over):
    a = {n: FAKE for n in ("q", "k", "v", "beta", "la", "S", "y")}
    a["slots"] = FAKE
    a.update(over)
    return L.gradlev_delta_step(B, H, Hk, T, dk, dv, dt, a["q"], a["k"], a["v"], a["beta"],
                                a["la"], 1.0, a["slots"], pool, a["S"], a["y"], NULL)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_sizes_are_refused(L, call):
    for n in ("B", "H", "Hk", "T", "dk", "dv"):
        for v in (0, -1):
            assert call(L, **{n: v}) == 1, n
    assert call(L, dt=7) == 1
    assert call(L, H=3, Hk=2) == 2
    assert call(L, dk=260 if call is step else 264) == 2
    assert call(L, dk=6) == 2
    assert call(L, B=1 << 15, H=1 << 10, T=1 << 10) == 2
    if call is not step:
        assert call(L, dk=12) == 2 and call(L, dv=12) == 2 and call(L, dv=264) == 2


def test_sizes_agree_with_the_queries(L):
    for shape, ok in (((1, 2, 1, 8, 16, 16, 0), 0), ((1, 2, 1, 8, 256, 256, 0), 0),
                      ((1, 3, 2, 8, 16, 16, 0), 2), ((1, 2, 1, 8, 12, 16, 1), 2),
                      ((1, 2, 1, 0, 16, 16, 1), 1)):
        assert L.gradlev_delta_supported(*shape) == ok
        assert (L.gradlev_delta_ckpt_bytes(*shape) > 0) == (ok == 0)
        for b in (0, 1):
            assert (L.gradlev_delta_workspace_bytes(*shape, b) >= 256) == (ok == 0)


@pytest.mark.parametrize("call,names", [
    (fwd, ("q", "k", "v", "beta", "la", "y", "ws")),
    (bwd, ("q", "k", "v", "beta", "la", "dy", "dq", "gk", "gv", "db", "dl", "ws")),
    (step, ("q", "k", "v", "beta", "la", "S", "y"))])
def test_null_and_misaligned_pointers_are_refused(L, call, names):
    for n in names:
        assert call(L, **{n: NULL}) == 1, n
        assert call(L, **{n: P(4096 + 2)}) == 1, n
    if call is fwd:
        for n in ("S0", "ST"):
            assert call(L, **{n: P(4096 + 4)}) == 1
    if call is bwd:
        for n in ("S0", "dST", "dS0"):
            assert call(L, **{n: P(4096 + 4)}) == 1
    if call is not step:
        assert call(L, ckpt=P(4096 + 16)) == 1 and call(L, ws=P(4096 + 16)) == 1


def test_small_workspaces_are_refused(L):
    need = [L.gradlev_delta_workspace_bytes(1, 2, 1, 8, 16, 16, 0, b) for b in (0, 1)]
    assert fwd(L, ws_bytes=need[0] - 1) == 3
    assert bwd(L, ws_bytes=need[1] - 1) == 3


def test_step_without_slots_needs_a_state_per_row(L):
    assert step(L, B=5, pool=4, slots=NULL) == 1
    assert step(L, pool=0) == 1


def norm(L, B=1, T=2, Hq=2, Hk=1, d=32, rot=16, dt=0, kind=0, eps=1e-6, qs=(128, 64, 32),
         bwd=False, ws_bytes=1 << 20, **over):
    a = {n: FAKE for n in ("q", "k", "wq", "wk", "pos", "freq", "yq", "yk", "dwq", "dwk", "ws")}
    a.update(over)
    s = (ctypes.c_longlong * 3)(*qs)
    ks = (ctypes.c_longlong * 3)(64, 32, 32)
    if not bwd:
        return L.gradlev_qk_norm_rope_fwd(B, T, Hq, Hk, d, rot, dt, kind, eps, a["q"], s, a["k"],
                                          ks, a["wq"], a["wk"], a["pos"], a["freq"], a["yq"],
                                          a["yk"], NULL)
    return L.gradlev_qk_norm_rope_bwd(B, T, Hq, Hk, d, rot, dt, kind, eps, a["yq"], a["yk"], a["q"],
                                      s, a["k"], ks, a["wq"], a["wk"], a["pos"], a["freq"],
                                      a["q"], s, a["k"], ks, a["dwq"], a["dwk"], a["ws"], ws_bytes, NULL)


@pytest.mark.parametrize("b", [False, True])
def test_norm_refusals(L, b):
    for n in ("B", "T", "Hq", "Hk", "d"):
        assert norm(L, bwd=b, **{n: 0}) == 1, n
    assert norm(L, bwd=b, rot=-16) == 1
    assert norm(L, bwd=b, dt=5) == 1 and norm(L, bwd=b, kind=2) == 1
    assert norm(L, bwd=b, eps=-1.0) == 1 and norm(L, bwd=b, eps=float("nan")) == 1
    assert norm(L, bwd=b, d=36) == 2 and norm(L, bwd=b, d=264) == 2
    assert norm(L, bwd=b, rot=8) == 2 and norm(L, bwd=b, rot=48) == 2
    assert norm(L, bwd=b, B=1 << 20, T=1 << 20) == 2
    for n in ("q", "k", "yq", "yk", "freq"):
        assert norm(L, bwd=b, **{n: NULL}) == 1, n
        assert norm(L, bwd=b, **{n: P(4096 + 2)}) == 1, n
    assert norm(L, bwd=b, qs=(128, 66, 32)) == 1  # rows that a 16-byte load cannot start at
    assert norm(L, bwd=b, qs=(128, -64, 32)) == 1
    if b:
        assert norm(L, bwd=True, dwq=NULL) == 1 and norm(L, bwd=True, wk=NULL) == 1
        assert norm(L, bwd=True, ws_bytes=16) == 3 and norm(L, bwd=True, ws=NULL) == 1


def test_the_binding_refuses_before_any_call():
    d = ref.draw(1, 2, 1, 4, 16, 16)
    args = [d[n] for n in NAMES[:5]]
    with pytest.raises(tw.GradlevError, match="CUDA device"):
        tw.gradlev_delta_fwd(*args)
    with pytest.raises(tw.GradlevError, match="CUDA device"):
        tw.gradlev_delta_bwd(*args, d["dy"])
    with pytest.raises(tw.GradlevError, match="CUDA device"):
        tw.gradlev_delta_step(*args, torch.zeros(1, 2, 16, 16))
    x = torch.zeros(1, 4, 2, 32)
    with pytest.raises(tw.GradlevError, match="CUDA device"):
        tw.gradlev_qk_norm_rope_fwd(x, x)
    with pytest.raises(tw.GradlevError, match="not one of"):
        tw.gradlev_qk_norm_rope_fwd(x, x, norm="max")


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_products_of_sizes_past_64_bits_are_refused(L, call):
    big = 1 << 30
    assert call(L, B=big, H=big, Hk=1, T=1 << 10) == 2  # 2^70: 0 modulo 2^64
    assert call(L, B=big, H=big, Hk=1, T=1) == 2
    assert call(L, B=1, H=1, T=1, dv=2 ** 31 - 8) == 2
    if call is not step:
        for shape in ((big, big, 1, 1 << 10, 16, 16, 0), (big, big, 1, 1, 16, 16, 1)):
            assert L.gradlev_delta_supported(*shape) == 2
            assert L.gradlev_delta_workspace_bytes(*shape, 1) == 0
    for b in (False, True):
        assert norm(L, bwd=b, B=big, T=big, Hq=1 << 9, Hk=1 << 9) == 2


def test_outputs_over_their_inputs_or_themselves_are_refused(L):
    assert fwd(L, S0=P(8192), ST=P(8192)) == 1
    for qs in ((0, 64, 32), (128, 0, 32), (128, 64, 0)):  # gradients of many rows in one place
        assert norm(L, bwd=True, B=2, qs=qs) == 1
