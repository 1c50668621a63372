"""The device and the stream that the binding calls a grouped-head entry point with, on the host: the library and torch's
device calls are fakes, so that two devices can be played."""
import contextlib
import types

import pytest
import torch

import compressed_sparse_attention_13_b200 as K


class Machine:
    """A current device, the streams of each, and what the entry point saw."""

    def __init__(self, monkeypatch, status=0):
        self.current, self.seen, self.status = 0, [], status

        @contextlib.contextmanager
        def device(d):
            before, self.current = self.current, d
            try:
                yield
            finally:
                self.current = before

        def call(*args):
            self.seen.append((self.current, args[2:]))
            return self.status

        monkeypatch.setattr(K, "_lib", types.SimpleNamespace(prompt_attn=call, csa_strerror=lambda st: b"no"))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=100 + self.current))
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)


P = K.gqa_params(8, 2, 128, 0.1)
GIVEN = types.SimpleNamespace(cuda_stream=7)


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("stream,want", [(None, None), (GIVEN, 7)])
def test_a_call_runs_on_the_device_of_its_tensors(monkeypatch, dev, stream, want):
    m = Machine(monkeypatch)
    K._launch("prompt_attn", P, 3, ("a", "b"), stream, dev)
    assert m.seen == [(dev, ("a", "b", want or 100 + dev))]
    assert m.current == 0


def test_a_refusal_leaves_the_callers_device(monkeypatch):
    m = Machine(monkeypatch, status=-1)
    with pytest.raises(K.CsaError, match="prompt_attn"):
        K._launch("prompt_attn", P, 3, (), None, 1)
    assert m.current == 0 and m.seen == [(1, (101,))]
