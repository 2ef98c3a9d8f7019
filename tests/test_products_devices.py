"""Which device and stream the 8-bit products and the input gradients run on
(CPU only: the library and the device state are stand-ins)."""
import pytest
import torch

import bf16_activation_quantized_amd as w4
from test_binding_devices import Device, Tensor, on_device_1   # noqa: F401  (fixture)

t = Tensor
CALLS = {
    "w4a16_fp8_quantize": lambda **kw: w4.w4a16_fp8_quantize(t(4, 256), q=t(4, 256), scales=t(4, 2), **kw),
    "w4a16_fp8_gemm": lambda **kw: w4.w4a16_fp8_gemm(t(4, 256), t(4, 2), t(128, 256), t(1, 2), **kw),
    "w4a16_fp8_gemm_grouped": lambda **kw: w4.w4a16_fp8_gemm_grouped(t(4, 256), t(4, 2), t(3, 128, 256), t(3, 1, 2),
                                                                     t(3), **kw),
    "w4a16_fp8_gemm_grad": lambda **kw: w4.w4a16_fp8_gemm_grad(t(4, 128), t(4, 1), t(128, 256), t(1, 2), **kw),
    "w4a16_gemm_grad": lambda **kw: w4.w4a16_gemm_grad(t(4, 64), t(64, 128), t(64, 2), **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_device_and_stream(on_device_1, name):   # noqa: F811
    f = CALLS[name]
    w4._bytes_of.cache_clear()
    f()
    assert on_device_1.calls[-1][0] == name and all(d == 1 for _, d, _ in on_device_1.calls)   # sizes too
    assert on_device_1.calls[-1][2][-1] == 0x201 and on_device_1.current == 0
    on_device_1.calls.clear()
    with pytest.raises(ValueError, match="device"):
        f(stream=on_device_1.Stream(0))
    assert not [n for n, _, _ in on_device_1.calls if not n.endswith("_bytes")]
    own = on_device_1.Stream(1)
    f(stream=own)
    assert on_device_1.calls[-1][1] == 1 and on_device_1.calls[-1][2][-1] == own.cuda_stream
    f(stream=0x7000)
    assert on_device_1.calls[-1][2][-1] == 0x7000
    w4._bytes_of.cache_clear()      # (the stand-in's sizes)


def test_wrong_arguments_raise():
    x, q = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 256).to(torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        w4.w4a16_fp8_quantize(x)
    with pytest.raises(TypeError):
        w4.w4a16_fp8_gemm(x, s, q, s)
    with pytest.raises(ValueError):
        w4.w4a16_fp8_gemm(q[0], s, q, s)
    with pytest.raises(TypeError):
        w4.w4a16_fp8_gemm_grouped(q, s, q, s, None)
    with pytest.raises(ValueError):
        w4.w4a16_gemm_grad(x, torch.zeros(3, 256, 128, dtype=torch.uint8), x)
