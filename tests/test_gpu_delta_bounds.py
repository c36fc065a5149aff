"""GPU tests of how near the gated delta rule comes to the 64-bit recurrence, close enough to
notice a rounding too many.

A rounding to bf16 is uniform within half a step, 2^-8 of a value's leading power of two: 2^-8 /
sqrt(3) of that power in the mean square. Over values as normal numbers are spread, the mean square
of the leading power is 0.54 of the value's. Independent roundings add up as squares:
sqrt(0.54 n / 3) 2^-8 for the n that an output sees on the tensor cores, itself among them (what
goes by two bf16 counts for none):
  y: Wq, y;                 dq: the state, dq;          dk: the state, its gradient, dk;
  dv, dbeta, dS0: Kw, F, themselves;
  dlog_alpha: the state, its gradient, Kw, F, dlog_alpha.
float32: products of operands that are split into two parts are 2^-21 off, and their sums of at
most 256 terms add sqrt(256) 2^-24; four in a row, independent of each other. The float32 state of
a bf16 forward goes by three bf16, as many bits as float32 has; what is left are the tensor core's
24 additions to it per chunk, each cut to 2^-23.

In float32 dlog_alpha gets the factor of `cancellation`. It is a sum over the pairs of tokens
i >= t > j of a chunk of 32,
  X_ij q_i.k_j - Y_ij k_i.k_j,  X_ij = scale M_ij beta_j dy_i.D_j,  Y_ij = M_ij beta_i beta_j E_i.D_j,
and what flows through the chunk's ends. Each pair carries the error above relative to itself, so
that the sum's is that times the root of the sum of the pairs' squares, which is more than the sum
where keys are alike: there what the pairs of one token add, those of the next take away.
"""

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402
from tests.test_gpu_delta import NAMES, code, dev  # noqa: E402
from tests.test_gpu_delta_alike import alike  # noqa: E402

pytestmark = pytest.mark.gpu

ROUNDING = 2.0 ** -8 * (0.54 / 3) ** 0.5
SEEN = dict(y=2, dv=3, dS0=3, dq=2, dk=3, dbeta=3, dlog_alpha=5)
F32 = 4 ** 0.5 * (2.0 ** -21 + 256 ** 0.5 * 2.0 ** -24)
STATE = 24 * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    yield


def cancellation(x, want, scale):
    """2-norm over the tokens of the root of the sum of the squares of a token's pairs, over that of
    dlog_alpha (at least 1)."""
    B, H, T, _ = x["v"].shape
    q, k = ref.heads(x["q"], H), ref.heads(x["k"], H)
    S, D = x["S0"], []
    for t in range(T):
        Sd = torch.exp(x["log_alpha"][:, :, t])[..., None, None] * S
        D.append(x["v"][:, :, t] - (Sd @ k[:, :, t, :, None])[..., 0])
        S = Sd + (x["beta"][:, :, t, None] * D[-1])[..., None] * k[:, :, t, None, :]
    D, E = torch.stack(D, 2), want["dv"] / x["beta"][..., None]
    total = 0.0
    for a in range(0, T, 32):
        c = slice(a, min(a + 32, T))
        L, b = x["log_alpha"][:, :, c].cumsum(-1), x["beta"][:, :, c]
        M = (L[..., :, None] - L[..., None, :]).exp().tril(-1)
        X = scale * M * b[..., None, :] * (x["dy"][:, :, c] @ D[:, :, c].mT)
        Y = M * b[..., :, None] * b[..., None, :] * (E[:, :, c] @ D[:, :, c].mT)
        pairs = (X * (q[:, :, c] @ k[:, :, c].mT)) ** 2 + (Y * (k[:, :, c] @ k[:, :, c].mT)) ** 2
        n = pairs.shape[-1]
        for t in range(1, n):
            total += float(pairs[..., t:, :t].sum())
    return max(1.0, total ** 0.5 / float(want["dlog_alpha"].norm()))


def errors(shape, cosine, beta, seed):
    B, H, Hk, T, dk, dv, dtype = shape
    d = alike(*shape, cosine, beta, seed=seed)
    g, x = dev(d), ref.f64(d)
    scale = dk ** -0.5
    y64, S64 = ref.forward(*[x[n] for n in NAMES], scale, x["S0"])
    want = ref.gradients(*[x[n] for n in NAMES], scale, x["S0"], x["dy"])
    args = [g[n] for n in NAMES]
    y0, ST = tw.gradlev_delta_fwd(*args, g["S0"])
    ck = torch.empty(tw.gradlev_delta_ckpt_bytes(B, H, Hk, T, dk, dv, code(dtype)),
                     dtype=torch.uint8, device="cuda")
    y, _ = tw.gradlev_delta_fwd(*args, g["S0"], want_ST=False, ckpt=ck)
    out = tw.gradlev_delta_bwd(*args, g["dy"], g["S0"], ckpt=ck)
    e = {n: ref.rel2(out[n], want[n]) for n in want}
    e.update(y=max(ref.rel2(y, y64), ref.rel2(y0, y64)), ST=ref.rel2(ST, S64))
    return e, cancellation(x, want, scale) if dtype == "f32" else None


# the smallest calls that take the tensor cores, and some more; then the float32 kernels
@pytest.mark.parametrize("shape", [
    (1, 5, 5, 205, 128, 128, "bf16"), (1, 5, 1, 820, 64, 64, "bf16"), (9, 4, 4, 500, 24, 40, "bf16"),
    (1, 3, 3, 2731, 24, 40, "bf16"), (1, 3, 3, 2731, 56, 64, "bf16"), (2, 4, 4, 300, 128, 256, "bf16"),
    (1, 5, 5, 204, 128, 128, "bf16"), (1, 3, 3, 300, 64, 64, "f32"), (1, 2, 2, 300, 128, 128, "f32"),
], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("cosine,beta", [(0.0, None), (0.5, None), (0.9, 1.0)])
def test_errors_are_those_of_the_roundings(shape, cosine, beta):
    for seed in range(3):
        e, factor = errors(shape, cosine, beta, seed)
        for n, err in e.items():
            if shape[-1] == "f32":
                tol = F32 * (factor if n == "dlog_alpha" else 1.0)
            elif n == "ST":
                tol = STATE
            else:
                tol = SEEN[n] ** 0.5 * ROUNDING
            assert err <= tol, (n, seed, err, tol)
