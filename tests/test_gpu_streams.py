"""GPU tests of calls with stream=: memory that the current stream has let go of, but not yet
written for the last time, must not become a buffer of a call on another stream."""

import pytest

torch = pytest.importorskip("torch")

import token_weight_scans_b200 as tw  # noqa: E402
from tests import calls  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", calls.NAMES)
def test_pending_writes_of_the_current_stream_do_not_reach_a_call(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_weight_scans_b200 import build
    build.build()
    tw.lib()
    call = calls.all_calls("cuda")[name]
    alone = call()
    sizes = [t.numel() * t.element_size() for t in alone.values()] + [1 << k for k in range(9, 25)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):  # the first time the given stream has no memory yet
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda._sleep(50_000_000)
        for b in blocks:
            b.fill_(0xFF)
        del b, blocks
        got = call(stream=side)
        torch.cuda.synchronize()
        for n in alone:
            assert torch.equal(got[n], alone[n]), n
