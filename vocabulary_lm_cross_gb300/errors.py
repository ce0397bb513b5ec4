"""Errors that kernels detected on the device after their call had returned."""
from __future__ import annotations

import torch

from . import capi


def take_device_errors(device=None) -> int:
    """The DEVERR_* bits (capi.py) that linear and gated layers called without dev_err
    have left on `device` since the last call; they are cleared.  Waits for the current
    stream; layers on other streams count once they have run."""
    dev = torch.device("cuda" if device is None else device)
    with torch.cuda.device(dev):
        out = torch.zeros(1, dtype=torch.int32, device="cuda")
        capi.check(capi.lib().vlmce_take_device_errors(
            out.data_ptr(), torch.cuda.current_stream().cuda_stream), "vlmce_take_device_errors")
        return int(out)


def check_device_errors(device=None) -> None:
    """Raise if take_device_errors() finds any."""
    bits = take_device_errors(device)
    if bits & capi.DEVERR_TIMEOUT:
        raise RuntimeError("a kernel's wait gave up: results since the last check are invalid")
    if bits:
        raise RuntimeError(f"device error bits {bits:#x}")
