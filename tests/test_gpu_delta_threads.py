"""GPU test of the gated delta rule called by several host threads at once: each with its own
sizes, buffers and stream, and the results of calls one after the other."""

import threading

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import delta_ref as ref  # noqa: E402
from tests.test_gpu_delta import NAMES, code, dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_threads_with_different_widths(dtype):
    """The widest heads need ten times the shared memory of the narrowest, in the same kernels."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    sets = [dev(ref.draw(1, 2, 1, 40, d, d, dtype, True, seed=d)) for d in (256, 16, 160, 8)]

    alone = [dict(zip(("y", "ST"), tw.gradlev_delta_fwd(*[d[n] for n in NAMES], d["S0"])))
             for d in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        d = sets[i]
        B, H, T, dv = d["v"].shape
        size = (B, H, d["q"].shape[1], T, d["q"].shape[3], dv, code(dtype))
        y, ST = torch.empty_like(d["v"]), torch.empty_like(d["S0"])
        ws = torch.empty(tw.gradlev_delta_workspace_bytes(*size, 0), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        at = [d[n].data_ptr() for n in NAMES]
        call = (*size, *at, size[4] ** -0.5, d["S0"].data_ptr(), y.data_ptr(), ST.data_ptr(), None,
                ws.data_ptr(), ws.numel(), stream.cuda_stream)
        start.wait()
        status = {tw.lib().gradlev_delta_fwd(*call) for _ in range(2000)}
        stream.synchronize()
        if status != {0} or not torch.equal(y, alone[i]["y"]) or not torch.equal(ST, alone[i]["ST"]):
            wrong.append((i, status))

    start = threading.Barrier(len(sets))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
