"""What the training operators' Python layer does around the library calls, on
stand-ins for CUDA tensors (no GPU needed)."""
import contextlib

import pytest
import torch

from newton_schulz_quintic_gb300 import training

DEV = torch.device("cuda", 0)


class Stub:
    """A CUDA tensor as far as the argument checks look at one."""

    is_cuda, device = True, DEV

    def __init__(self, shape, dtype, log=None, contiguous=True):
        self.shape = (shape,) if isinstance(shape, int) else tuple(shape)
        self.dtype, self.log, self.contiguous = dtype, log, contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def stride(self, axis=None):
        s = [1] * len(self.shape)
        for k in range(len(s) - 2, -1, -1):
            s[k] = s[k + 1] * self.shape[k + 1]
        return tuple(s) if axis is None else s[axis]

    def data_ptr(self):
        return 0x1000

    def reshape(self, *_):
        if not self.contiguous:
            self.log.append("copy")
        return Stub((self.numel(),), self.dtype)


@pytest.fixture
def log(monkeypatch):
    """The order of events of a call: its stream's block, copies, the library call."""
    events = []

    @contextlib.contextmanager
    def on(device, stream):
        events.append(("enter", device, stream))
        yield
        events.append("exit")

    monkeypatch.setattr(training, "_on", on)
    monkeypatch.setattr(training, "_call", lambda name, *a: events.append(name))
    monkeypatch.setattr(training, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(training, "_empty", lambda shape, dtype, device: Stub(shape, dtype))
    return events


@pytest.mark.parametrize("stream", [None, object()])
def test_ids_are_copied_on_the_stream_of_the_call(log, stream):
    ids = Stub((4, 6), torch.int64, log, contiguous=False)
    training.embed_lookup(Stub((50, 8), torch.float32), ids, stream=stream)
    assert log == [("enter", DEV, stream), "copy", "ns_embed_lookup", "exit"]
    log.clear()
    training.embed_grad(Stub((24, 8), torch.float32), ids, vocab=50, stream=stream)
    assert log == [("enter", DEV, stream), "copy", "ns_embed_grad", "exit"]


@pytest.mark.parametrize("device", [DEV, "cuda:0", "cuda", torch.device("cuda"), 0])
def test_an_empty_checkpoint_knows_its_device(log, monkeypatch, device):
    # whatever names the device, calls compare it with tensors' and take its index
    monkeypatch.setattr(training, "_current_device", lambda: 0)
    ck = training.Checkpoint8.empty(4, 40, device)
    assert ck.device == DEV and ck.device.index == 0
    training.checkpoint_load(ck)
    training.checkpoint_wgrad(Stub((4, 8), torch.float32), ck)
    assert [e for e in log if isinstance(e, str) and e != "exit"] == ["ns_ckpt_load", "ns_ckpt_wgrad"]


def test_an_empty_checkpoint_is_on_a_gpu(log):
    with pytest.raises(ValueError):
        training.Checkpoint8.empty(4, 40, "cpu")
