"""GPU tests of the gated delta rule where keys are alike.

Keys of one head usually share a direction. Their errors e_t then nearly cancel in the sums over a
chunk (each token takes back what the one before it wrote), so that a rounding of the terms costs
more than a rounding of the sum. The bounds are those of the other delta tests, sqrt(n) 2^-8 for
the n roundings to bf16 on the way to an output and 4 * 256 * 2^-24 for float32: a rounding counts
once, whatever the keys are.
"""

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402
from tests.test_gpu_delta import NAMES, check, code, dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    yield


def alike(B, H, Hk, T, dk, dv, dtype, cosine, beta, seed):
    """Queries and keys of unit length whose mean cosine is `cosine` within a head; beta: one
    value, or None (sigmoid of a normal)."""
    d = ref.draw(B, H, Hk, T, dk, dv, dtype, True, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    common = torch.randn((B, Hk, 1, dk), generator=g)
    common /= common.norm(dim=-1, keepdim=True)
    for n in ("q", "k"):
        x = torch.randn((B, Hk, T, dk), generator=g) / dk ** 0.5
        x = cosine ** 0.5 * common + (1 - cosine) ** 0.5 * x
        d[n] = (x / x.norm(dim=-1, keepdim=True)).to(d[n].dtype)
    if beta is not None:
        d["beta"] = torch.full((B, H, T), beta)
    return d


SHAPES = [
    # (B, H, Hk, T, dk, dv, dtype): the tensor cores, narrower heads, segments, a small call, float32
    (3, 4, 2, 200, 128, 128, "bf16"), (6, 3, 3, 260, 64, 72, "bf16"),
    (9, 4, 2, 257, 40, 72, "bf16"), (1, 2, 1, 1283, 128, 256, "bf16"),
    (1, 2, 2, 200, 128, 128, "bf16"), (1, 2, 1, 200, 64, 64, "f32"),
]


@pytest.mark.parametrize("cosine,beta", [(0.5, None), (0.9, None), (0.9, 1.0), (0.9, 1.9)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_alike_keys(shape, cosine, beta):
    B, H, Hk, T, dk, dv, dtype = shape
    d = alike(*shape, cosine, beta, seed=T + dk)
    g, x = dev(d), ref.f64(d)
    scale = dk ** -0.5
    y64, S64 = ref.forward(*[x[n] for n in NAMES], scale, x["S0"])
    want = ref.gradients(*[x[n] for n in NAMES], scale, x["S0"], x["dy"])
    args = [g[n] for n in NAMES]
    y, ST = tw.gradlev_delta_fwd(*args, g["S0"])
    check(dict(y=y, ST=ST), dict(y=y64, ST=S64), dtype)
    ck = torch.empty(tw.gradlev_delta_ckpt_bytes(B, H, Hk, T, dk, dv, code(dtype)),
                     dtype=torch.uint8, device="cuda")
    y, _ = tw.gradlev_delta_fwd(*args, g["S0"], want_ST=False, ckpt=ck)
    out = tw.gradlev_delta_bwd(*args, g["dy"], g["S0"], ckpt=ck)
    check(dict(out, y=y), dict(want, y=y64), dtype)
