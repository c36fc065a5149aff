"""Calls with stream=, without a GPU: what a call allocates must come from the given stream's
memory, and both streams must hold what they use."""

import contextlib
import types

import pytest
import torch

import token_weight_scans_b200 as tw
from tests import calls
from token_weight_scans_b200 import build as tw_build

CPU = torch.device("cpu")


@pytest.mark.parametrize("name", calls.NAMES)
def test_buffers_are_allocated_on_the_given_stream(name, monkeypatch):
    tw_build.build()
    real, now, seen, held = tw.lib(), [], [], []
    mine, side = (types.SimpleNamespace(device=CPU, cuda_stream=n) for n in (1, 2))

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    class Lib:  # sizes from the library, no launch
        def __getattr__(self, entry):
            if entry != name:
                return getattr(real, entry)
            return lambda *a: seen.append((a[-1], list(now))) or 0

    def made_on(make):
        def f(*a, **k):
            t = make(*a, **k)
            t.made = now[-1] if now else mine
            return t
        return f

    monkeypatch.setattr(tw, "lib", lambda: Lib())
    monkeypatch.setattr(tw, "_cuda_device", lambda x: CPU)
    monkeypatch.setattr(tw, "_on", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1] if now else mine)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: now[-1].cuda_stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.append((t, s)))
    call = calls.all_calls("cpu")[name]
    for make in ("empty", "empty_like"):
        monkeypatch.setattr(torch, make, made_on(getattr(torch, make)))
    monkeypatch.setattr(torch.Tensor, "new_empty", made_on(torch.Tensor.new_empty))
    out = call(stream=side)
    (raw, during), = seen
    assert (raw.value if hasattr(raw, "value") else raw) == 2
    assert during == [side]
    for n, t in out.items():
        assert t.made is side, n
        assert any(h is t and s is mine for h, s in held), n  # the caller reads it on its own
