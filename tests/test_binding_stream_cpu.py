"""The stream context of the recurrence's and norms' calls (no GPU needed): whatever a
call refuses, the caller's stream is current again and the refusal is what they see."""
import pytest
import torch

import gated_delta_rule_attn_b200 as la

DEV = torch.device("cuda", 0)


class Stream:
    device, cuda_stream = DEV, 77


class Ctx:
    def __init__(self, log):
        self.log = log

    def __enter__(self):
        self.log.append("enter")

    def __exit__(self, *exc):
        self.log.append("exit")


class OnDevice(torch.Tensor):
    """A tensor that says it is on the GPU and keeps what it was recorded on."""
    device = DEV
    seen = None
    broken = False

    def record_stream(self, s):
        if self.broken:
            raise RuntimeError("cannot be recorded")
        self.seen = s


def on_device():
    return torch.zeros(3).as_subclass(OnDevice)


@pytest.fixture
def log(monkeypatch):
    log = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: Ctx(log))
    return log


def test_a_refused_tensor_elsewhere_leaves_the_stream(log):
    good = on_device()
    with pytest.raises(ValueError, match="the refusal"):
        with la._On(DEV, Stream(), good, torch.zeros(3), None):
            raise ValueError("the refusal")
    assert log == ["enter", "exit"]


def test_anything_given_for_a_tensor_leaves_the_stream(log):
    with pytest.raises(ValueError, match="the refusal"):
        with la._On(DEV, Stream(), [1.0], "x", 3):
            raise ValueError("the refusal")
    assert log == ["enter", "exit"]


def test_a_tensor_that_cannot_be_recorded_leaves_the_stream(log):
    t = on_device()
    t.broken = True
    with pytest.raises(RuntimeError):
        with la._On(DEV, Stream(), t):
            pass
    assert log == ["enter", "exit"]


def test_a_call_records_its_tensors(log):
    ts, s = [on_device(), None, on_device()], Stream()
    with la._On(DEV, s, *ts) as handle:
        assert handle == 77 and log == ["enter"]
    assert log == ["enter", "exit"] and ts[0].seen is s and ts[2].seen is s
