"""GPU tests of the gated delta rule over the whole range of its gates: decays between the mild
ones of training and a reset, sums of them on either side of where a chunk's decays leave one
float32 factor (80), and tokens without a step at the ends of a chunk.

References are the 64-bit recurrences, tolerances those of the other delta tests: in bf16
sqrt(n) 2^-8 for the n roundings on the way to an output, in float32 4 * 256 * 2^-24. They hold
for the tokens without a step alone as well, whose gradients no larger neighbour can hide.
"""

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402
from tests.test_gpu_delta import NAMES, check, code, dev, tol  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    yield


def gates(kind, B, H, T, seed):
    """log_alpha [B,H,T]. "wide": every token anywhere between -0.5 and -86, on a scale of
    factors. "half": mild but for one half of each chunk of 64, which takes a total of 55 to 95.
    "early": tokens 12 to 31 of each chunk share 56 to 79 nats, the rest have 0.01 each. (And "docs", the mask
    of the other tests: resets and padding.)"""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand((B, H, T), generator=g)
    if kind == "wide":
        return -0.5 * 172.0 ** u
    n = -(-T // 64)
    la = -0.02 * u if kind == "half" else torch.full((B, H, T), -0.01)
    for b in range(B):
        for h in range(H):
            for c in range(n):
                r = torch.rand(2, generator=g).tolist()
                if kind == "half":
                    lo, hi = (0, 32) if r[0] < 0.5 else (32, 64)
                    total = 55 + 40 * r[1]
                else:
                    lo, hi, total = 12, 32, 56 + 23 * r[1]
                part = torch.rand(hi - lo, generator=g) + 0.1
                at = torch.arange(64 * c + lo, 64 * c + hi)
                at = at[at < T]
                la[b, h, at] = -(total * part / part.sum())[:len(at)]
    return la


CASES = [
    # (B, H, Hk, T, dk, dv, dtype): the tensor cores, in segments too; a small call; float32
    (9, 4, 2, 150, 128, 128, "bf16"), (16, 4, 4, 130, 64, 40, "bf16"),
    (14, 4, 2, 150, 64, 64, "bf16"), (9, 8, 4, 130, 24, 136, "bf16"),
    (1, 2, 1, 1283, 128, 256, "bf16"), (1, 2, 2, 150, 128, 128, "bf16"),
    (2, 2, 1, 100, 136, 64, "bf16"), (2, 3, 3, 150, 64, 48, "f32"),
]


@pytest.mark.parametrize("kind", ["wide", "half", "early", "docs"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_strong_decays(case, kind):
    B, H, Hk, T, dk, dv, dtype = case
    d = ref.draw(B, H, Hk, T, dk, dv, dtype, True, "docs" if kind == "docs" else "none", seed=T + dk)
    if kind != "docs":
        d["log_alpha"] = gates(kind, B, H, T, seed=dk + dv)
    still = (torch.arange(T) % 64 < 4) | (torch.arange(T) % 64 >= 60)
    d["beta"][:, :, still] = 0.0
    d["beta"][:, :, 40 % T::64] = 1e-7
    g, x = dev(d), ref.f64(d)
    scale = dk ** -0.5
    y64, S64 = ref.forward(*[x[n] for n in NAMES], scale, x["S0"])
    S64[S64.abs() < 2.0 ** -126] = 0.0  # a last state that decayed below what float32 holds
    want = ref.gradients(*[x[n] for n in NAMES], scale, x["S0"], x["dy"])
    args = [g[n] for n in NAMES]
    y, ST = tw.gradlev_delta_fwd(*args, g["S0"])
    check(dict(y=y, ST=ST), dict(y=y64, ST=S64), dtype)
    ck = torch.empty(tw.gradlev_delta_ckpt_bytes(B, H, Hk, T, dk, dv, code(dtype)),
                     dtype=torch.uint8, device="cuda")
    y, _ = tw.gradlev_delta_fwd(*args, g["S0"], want_ST=False, ckpt=ck)
    out = tw.gradlev_delta_bwd(*args, g["dy"], g["S0"], ckpt=ck)
    check(dict(out, y=y), dict(want, y=y64), dtype)
    for n in ("dbeta", "dlog_alpha"):
        err = ref.rel2(out[n][:, :, still.cuda()], want[n][:, :, still])
        assert err <= tol(n, dtype), (n, err)
