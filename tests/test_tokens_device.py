"""The token operators run on their tensors' device, also where another one is
current (checked without a GPU: the library and the device calls are stand-ins)."""

import contextlib

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import _lib as L


class Stand:
    """What the wrappers look at in a tensor."""

    def __init__(self, *shape, dtype=torch.float32, device=1):
        self.shape, self.dtype, self._device = torch.Size(shape), dtype, device

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = torch.empty(self.shape, device="meta").stride()
        return s if i is None else s[i]

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 4


@pytest.fixture
def machine(monkeypatch):
    """Two devices, device 0 current; the log of (call, device, stream)."""
    now, log = [0], []

    class Library:
        def __getattr__(self, name):
            return lambda *args: log.append((name, now[0], args[-1])) or L.GS_OK

    @contextlib.contextmanager
    def on(device):
        before, now[0] = now[0], device
        try:
            yield
        finally:
            now[0] = before

    class Stream:
        cuda_stream, device_index = 77, 1

    library = Library()
    monkeypatch.setattr(L, "lib", lambda: library)
    monkeypatch.setattr(L, "_RAW_STREAM", None)  # looked up again, as what follows
    monkeypatch.setattr(L, "_DEVICE", None, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", on)
    return log, Stream()


def calls(device, stream):
    def t(*shape, dtype=torch.float32):
        return Stand(*shape, dtype=dtype, device=device)

    q, pos, lists, lse = t(1, 9, 2, 64), t(1, 9, 3), t(1, 2, 1, 4), t(1, 2, 9)
    sums = t(1, 2, 1, 64), t(1, 2, 1)
    x, ws = t(9, 64), t(1000)
    L.gs_rope_axes(q, q, q, q, pos, t(32), (8, 12, 12), stream=stream)
    L.gs_norm_gate_fwd(x, x, None, None, None, x, x, t(2, 9), 9, stream=stream)
    L.gs_norm_gate_bwd(x, x, x, x, None, None, None, t(2, 9), x, x, None, None, None, 9, ws, stream=stream)
    L.gs_block_summary(q, *sums, stream=stream)
    L.gs_block_select(q, *sums, 64, 2, lists, stream=stream)
    L.gs_block_attn_fwd(q, q, q, lists, q, lse, stream=stream)
    L.gs_block_attn_bwd(q, q, q, q, q, lse, lists, q, q, q, ws, stream=stream)


@pytest.mark.parametrize("device", [0, 1])
def test_launches_are_on_the_tensors_device(machine, device):
    log, _ = machine
    calls(device, None)
    assert len(log) == 7
    assert all(at == device and stream == 1000 + device for _, at, stream in log), log
    assert torch.cuda.current_device() == 0


def test_a_given_stream_is_used_there(machine):
    log, stream = machine
    calls(1, stream)
    assert len(log) == 7 and all(at == 1 and s == 77 for _, at, s in log), log
