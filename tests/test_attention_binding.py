"""The binding of the attention operators where torch lacks the private functions that save it host time."""
import subprocess

import torch

from mixture_experts_gemv_b200 import _lib


def test_the_binding_does_without_torchs_private_functions(monkeypatch):
    kept = {name: getattr(_lib, name) for name in ("_torch", "_dtype_codes", "_raw_stream", "_device")}
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    for name, value in kept.items():
        monkeypatch.setattr(_lib, name, value)   # put back afterwards
    _lib._setup()
    assert _lib._device is torch.cuda.current_device
    asked = []
    monkeypatch.setattr(_lib, "_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: asked.append(index) or torch.cuda.ExternalStream)
    monkeypatch.setattr(torch.cuda.ExternalStream, "cuda_stream", 77, raising=False)
    got = []
    _lib._call(lambda *a: got.append(a) or _lib.MOE_OK, 3, None, 1, 2)
    assert got == [(1, 2, 77)] and asked == [3]


def test_the_library_shares_no_variable_with_another_copy_of_itself():
    """A variable that the linker makes one of a kind in the process would be shared by a second copy of the library,
    whose kernels are its own."""
    from mixture_experts_gemv_b200 import build
    names = subprocess.run(["nm", "-D", build.build()], check=True, capture_output=True, text=True).stdout
    unique = [line for line in names.splitlines() if line.split()[-2:-1] == ["u"]]
    assert "moe_attention_decode" in names and not unique, unique[:5]
