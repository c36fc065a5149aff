"""GPU tests of the norms' gradients row by row.

dx = r (g w - z <z, g w> / n) loses what lies along z, so a row's error is measured against
r |g w|, the size of what is subtracted: sums of at most 256 float32 terms, twice, 2^-22 for the
angles, and half a step of the output's type."""

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("B,T,H,d,rot", [(1, 1, 1, 8, 0), (1, 1, 1, 16, 16), (1, 3, 2, 24, 16),
                                         (2, 5, 3, 128, 64), (1, 2, 1, 256, 256)])
def test_gradients_of_every_row(B, T, H, d, rot, norm, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn((B, T, H, d), generator=gen).to(td)
        dy = torch.randn((B, H, T, d), generator=gen).to(td)
        inv = 100.0 ** (-torch.arange(rot // 2) / max(rot // 2, 1)) if rot else None
        x64 = x.double().requires_grad_()
        pos = torch.arange(T).expand(B, T)
        (ref.norm_rope(x64, None, pos, inv, norm, 1e-6) * dy.double()).sum().backward()
        out = tw.gradlev_qk_norm_rope_bwd(
            dy.cuda(), dy.cuda(), x.cuda(), x.cuda(),
            inv_freq=None if inv is None else inv.cuda(), norm=norm)
        n = d if norm == "rms" else 1
        r = (x.double().square().sum(-1) / n + 1e-6) ** -0.5
        size = r * dy.double().norm(dim=-1).transpose(1, 2)
        tol = 2 * 256 * 2.0 ** -24 + 2.0 ** -22 + (2.0 ** -8 if dtype == "bf16" else 0.0)
        for name in ("dq", "dk"):
            err = (out[name].cpu().double() - x64.grad).norm(dim=-1) / size
            assert float(err.max()) <= tol, (name, seed, float(err.max()))
