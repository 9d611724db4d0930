"""The C++ calls of csrc/torch_calls.cpp (checks, buffers and launch of the
adapters and of clipping), bound to the library that binding.py has loaded.
The extension module is loaded by the first call that needs it; without it
that call fails."""
from __future__ import annotations

import ctypes

import torch  # noqa: F401  (its libraries are what _torch_calls links to)

from . import binding as _b

_module = None


def calls():
    global _module
    if _module is None:
        from . import _torch_calls
        _torch_calls.bind(_b._check, *(
            ctypes.cast(getattr(_b._lib, name), ctypes.c_void_p).value for name in (
                "snack_lora_workspace", "snack_lora_fwd", "snack_lora_bwd",
                "snack_grad_workspace", "snack_grad_norm", "snack_grad_clip")))
        _module = _torch_calls
    return _module
