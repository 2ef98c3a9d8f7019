"""Which device and stream the adapter and expert calls of the binding run on
(CPU only: the library and the device state are stand-ins)."""
import contextlib

import pytest
import torch

import bf16_activation_quantized_amd as w4


class Device:
    """A process with several devices: the current one, and the library's calls
    with the device each was made on."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []
        dev = self

        @contextlib.contextmanager
        def device(d):
            before, dev.current = dev.current, d
            try:
                yield
            finally:
                dev.current = before

        class Stream:
            def __init__(self, index):
                self.device, self.cuda_stream = torch.device("cuda", index), 0x100 + index

        class Lib:
            def __getattr__(self, name):
                def f(*args):
                    dev.calls.append((name, dev.current, args))
                    return 256 if name.endswith("_bytes") else 0
                return f

        self.Stream = Stream
        monkeypatch.setattr(torch.cuda, "current_device", lambda: dev.current)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        monkeypatch.setattr(w4, "_current_raw_stream", lambda d: 0x200 + d)
        monkeypatch.setattr(w4, "_lib_handle", Lib())


class Tensor:
    """Stands for a device tensor of a shape."""

    def __init__(self, *shape, dev=1):
        self.shape, self.dev = shape, dev

    def get_device(self):
        return self.dev


@pytest.fixture()
def on_device_1(monkeypatch):
    """Tensors on device 1 while device 0 is current."""
    monkeypatch.setattr(w4, "_rank", lambda t, name, dtype, dims: t.shape)
    monkeypatch.setattr(w4, "_in", lambda t, name, dtype, shape, dev: 0x10000)
    monkeypatch.setattr(w4, "_out", lambda t, name, dtype, shape, like, dev, stream: (t, 0x10000))
    return Device(monkeypatch)


def lora(**kw):
    t = Tensor
    return w4.w4a16_gemm_lora(t(4, 256), t(64, 128), t(64, 2), t(3, 16, 256), t(3, 64, 16), t(4), **kw)


def test_sizes_are_asked_on_the_tensors_device(on_device_1):
    """The projection's plan, and with it the workspace, depends on the device's
    compute units: the size comes from the device that the call runs on."""
    lora()
    assert [(n, d) for n, d, _ in on_device_1.calls] == [("w4a16_gemm_lora_workspace_bytes", 1),
                                                         ("w4a16_gemm_lora", 1)]
    assert on_device_1.current == 0


def test_a_stream_of_another_device_is_refused(on_device_1):
    t = Tensor
    calls = [lora, lambda **kw: w4.w4a16_expert_sort(t(8, 2), 4, **kw),
             lambda **kw: w4.w4a16_expert_gather(t(8, 64), t(8, 2), **kw),
             lambda **kw: w4.w4a16_expert_gather_grad(t(16, 64), t(8, 2), **kw),
             lambda **kw: w4.w4a16_expert_combine(t(16, 64), t(8, 2), **kw)]
    own = on_device_1.Stream(1)
    for f in calls:
        on_device_1.calls.clear()
        with pytest.raises(ValueError, match="device"):
            f(stream=on_device_1.Stream(0))
        assert not [n for n, _, _ in on_device_1.calls if not n.endswith("_bytes")]
        f(stream=own)
        assert on_device_1.calls[-1][1] == 1 and on_device_1.calls[-1][2][-1] == own.cuda_stream
        f()                                             # the tensors' device's current stream
        assert on_device_1.calls[-1][1] == 1 and on_device_1.calls[-1][2][-1] == 0x201
        f(stream=0x7000)                                # an address is taken as it is
        assert on_device_1.calls[-1][2][-1] == 0x7000
