"""GPU tests of the norms and rotation of queries and keys against the 64-bit formula.

Tolerances (2-norm of the difference over the reference's): float32 sums of at most 256
terms with 2^-24 apiece, twice (the norm and, backwards, its gradient's dot product), and
2^-22 for sine and cosine of a reduced angle: 2 * 256 * 2^-24 + 2^-22. bf16 outputs add one
rounding, 2^-8. The weights' gradients are float32 sums over the rows of terms that are
formed as above."""

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
F32_TOL = 2 * 256 * 2.0 ** -24 + 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    yield


CASES = [
    # (B, T, Hq, Hk, d, rot, dtype, norm, weights, start)
    (1, 1, 1, 1, 8, 0, "f32", "l2", "none", 0),
    (2, 3, 4, 2, 16, 16, "f32", "rms", "both", 0),
    (2, 5, 3, 1, 40, 32, "bf16", "l2", "q", 1000),
    (1, 7, 16, 16, 128, 128, "bf16", "rms", "both", 2000000000),
    (3, 33, 5, 2, 64, 16, "f32", "rms", "k", 4000000),
    (2, 9, 2, 2, 256, 256, "bf16", "l2", "both", 50),
    (1, 11, 7, 3, 248, 48, "f32", "l2", "both", None),
    (64, 1, 16, 8, 128, 64, "bf16", "rms", "both", 123456),
    (2, 300, 2, 2, 128, 128, "f32", "rms", "both", None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(case):
    B, T, Hq, Hk, d, rot, dtype, norm, weights, start = case
    gen = torch.Generator().manual_seed(d + T)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    pad = 8  # columns between the rows that nothing may touch
    packed = r(B, T, Hq + Hk, d + pad).to(td)
    dyq, dyk = r(B, Hq, T, d).to(td), r(B, Hk, T, d).to(td)
    wq = 1 + 0.3 * r(d) if weights in ("q", "both") else None
    wk = 1 + 0.3 * r(d) if weights in ("k", "both") else None
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))
    inv = inv.float() if rot else None
    pos = None if start is None else (start + torch.arange(B * T).view(B, T)).to(torch.int32)
    p64 = packed.to(ref.F64).requires_grad_()
    w64 = [None if w is None else w.to(ref.F64).requires_grad_() for w in (wq, wk)]
    at = pos if pos is not None else torch.arange(T).expand(B, T)
    q64 = ref.norm_rope(p64[:, :, :Hq, :d], w64[0], at, inv, norm, 1e-5)
    k64 = ref.norm_rope(p64[:, :, Hq:, :d], w64[1], at, inv, norm, 1e-5)
    ((q64 * dyq.to(ref.F64)).sum() + (k64 * dyk.to(ref.F64)).sum()).backward()
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    pk = packed.cuda()
    args = (pk[:, :, :Hq, :d], pk[:, :, Hq:, :d], cu(wq), cu(wk), cu(pos), cu(inv))
    tol = F32_TOL + (2.0 ** -8 if dtype == "bf16" else 0.0)
    yq, yk = tw.gradlev_qk_norm_rope_fwd(*args, norm=norm, eps=1e-5)
    assert ref.rel2(yq, q64.detach()) <= tol and ref.rel2(yk, k64.detach()) <= tol
    dpk = torch.full_like(pk, 7.0)
    out = dict(dq=dpk[:, :, :Hq, :d], dk=dpk[:, :, Hq:, :d])
    for n, w in (("dwq", wq), ("dwk", wk)):
        if w is not None:
            out[n] = torch.empty(d, device="cuda")
    got = tw.gradlev_qk_norm_rope_bwd(cu(dyq), cu(dyk), *args, norm=norm, eps=1e-5, out=out)
    assert (dpk[..., d:] == 7.0).all()
    if not (norm == "l2" and d == 8 and rot == 0 and T == 1):
        assert ref.rel2(dpk[..., :d], p64.grad[..., :d]) <= tol
    for n, w in (("dwq", w64[0]), ("dwk", w64[1])):
        if w is not None:
            assert ref.rel2(got[n], w.grad) <= F32_TOL, n
    # contiguous gradients, and the same bits again
    got2 = tw.gradlev_qk_norm_rope_bwd(cu(dyq), cu(dyk), *args, norm=norm, eps=1e-5)
    for n in got:
        assert torch.equal(got[n], got2[n]), n
    # in place of the inputs
    tw.gradlev_qk_norm_rope_bwd(cu(dyq), cu(dyk), *args, norm=norm, eps=1e-5, out=dict(
        {n: torch.empty(d, device="cuda") for n in out if n[1] == "w"}, dq=args[0], dk=args[1]))
    assert torch.equal(args[0], got["dq"]) and torch.equal(args[1], got["dk"])


def test_permuted_and_broadcast_strides():
    """Any order of the axes, and one row read for every head."""
    gen = torch.Generator().manual_seed(1)
    B, T, H, d = 2, 6, 3, 32
    x = torch.randn(H, B, T, d, generator=gen).cuda()
    q = x.permute(1, 2, 0, 3)
    k = x[:1].permute(1, 2, 0, 3).expand(B, T, H, d)
    yq, yk = tw.gradlev_qk_norm_rope_fwd(q, k)
    zq, zk = tw.gradlev_qk_norm_rope_fwd(q.contiguous(), k.contiguous())
    assert torch.equal(yq, zq) and torch.equal(yk, zk)


def test_refusals():
    x = torch.zeros(1, 4, 2, 32, device="cuda")
    for q, k in ((x[..., ::2], x), (x, x.bfloat16()), (x, x[:, :3]), (x[0], x),
                 (x[..., 1:25], x[..., 1:25]), (x.half(), x.half())):
        with pytest.raises(tw.GradlevError):
            tw.gradlev_qk_norm_rope_fwd(q, k)
    with pytest.raises(tw.GradlevError):
        tw.gradlev_qk_norm_rope_fwd(x, x, pos=torch.zeros(1, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(tw.GradlevError):
        tw.gradlev_qk_norm_rope_fwd(x, x, wq=torch.ones(16, device="cuda"))
    with pytest.raises(tw.GradlevError):
        tw.gradlev_qk_norm_rope_fwd(x, x, inv_freq=torch.ones(4, device="cuda"))
    with pytest.raises(tw.GradlevError):
        tw.gradlev_qk_norm_rope_bwd(x, x, x, x)
