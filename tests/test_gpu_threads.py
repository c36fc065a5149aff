"""GPU test of the scans and the two-layer reconstruction called by several host threads at once,
with widths that need different amounts of shared memory in the same kernels."""

import threading

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402

pytestmark = pytest.mark.gpu


def scan(d, dt, gen):
    B, H, T = 1, 2, 20
    r = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    x, g = r(B, H, T, d).to(dt), r(B, H, T, d).to(dt)
    eta, alpha, W0 = 0.01 * torch.ones(B, H, T, device="cuda"), torch.sigmoid(r(B, H, T) + 4), r(H, d, d)
    size = (B, H, T, d, d, tw.BF16 if dt == torch.bfloat16 else tw.F32)
    y = torch.empty_like(g)
    ws = torch.empty(tw.gradlev_scan_workspace_bytes(*size, 0), dtype=torch.uint8, device="cuda")
    held = (x, g, eta, alpha, W0, y, ws)
    at = [t.data_ptr() for t in held]
    return held, y, lambda s: tw.lib().gradlev_scan_fwd(*size, *at[:6], None, at[6], ws.numel(), s)


def mlp2(d, dt, gen):
    B, H, T = 1, 2, 20
    r = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    rows = [(0.1 * r(B, H, T, d)).to(dt) for _ in range(4)]  # x, g1hat, g2hat, v
    eta, alpha, W = 0.01 * torch.ones(B, H, T, device="cuda"), torch.sigmoid(r(B, H, T) + 4), 0.1 * r(H, d, d)
    size = (B, H, T, d, d, d, tw.BF16 if dt == torch.bfloat16 else tw.F32)
    out = [torch.empty_like(rows[0]) for _ in range(5)]
    dW = torch.empty(B, H, d, d, device="cuda")
    ws = torch.empty(tw.gradlev_mlp2_workspace_bytes(*size), dtype=torch.uint8, device="cuda")
    held = (*rows, eta, alpha, W, W, *out, dW, ws)
    at = [t.data_ptr() for t in held]
    return held, dW, lambda s: tw.lib().gradlev_mlp2_recon(*size, *at[:8], 0, *at[8:], ws.numel(), s)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("make", [scan, mlp2])
def test_threads_with_different_widths(make, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    gen = torch.Generator().manual_seed(1)
    calls = [make(d, getattr(torch, dtype), gen) for d in (64, 8, 32, 16)]
    main = torch.cuda.current_stream()
    want = []
    for _, y, call in calls:
        assert call(main.cuda_stream) == 0
        want.append(y.clone())
        y.zero_()
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(len(calls)), []

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        status = {calls[i][2](stream.cuda_stream) for _ in range(2000)}
        stream.synchronize()
        if status != {0} or not torch.equal(calls[i][1], want[i]):
            wrong.append((i, status))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
