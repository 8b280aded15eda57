"""Where a call of the layer objects launches and allocates."""
from __future__ import annotations

import contextlib

import torch

_NOTHING = contextlib.nullcontext()


def resolve_device(device) -> torch.device:
    """`device` with its index filled in (the current device for a bare "cuda")."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def on(device: torch.device, stream=None):
    """Context in which `device` is current and `stream` (None: the device's current
    stream; a torch stream or a cudaStream_t) is its current stream, so that what is
    launched and what torch allocates inside belong to the same stream."""
    if stream is None:
        return _NOTHING if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)
