"""What the modules over the native bindings share."""
from __future__ import annotations

import importlib
import os

import torch

from . import EcwError, lib

_HERE = os.path.dirname(os.path.abspath(__file__))
_bound = {}


def native(name):
    """The native binding `name`, with the library loaded (raises if they have not been built)."""
    m = _bound.get(name)
    if m is None:
        L = lib()
        path = os.path.join(_HERE, f"{name}.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} missing: run __graft_entry__.build() (or "
                              "python entropy_coded_weight_amd/build.py) first")
        m = importlib.import_module(f".{name}", __package__)
        m.init(L._name, EcwError)
        _bound[name] = m
    return m


def on(stream, tensors, call):
    """call() with `stream` current; the tensors live on until its work is done."""
    tensors = [t for t in tensors if isinstance(t, torch.Tensor) and t.is_cuda]
    for t in tensors:  # work goes to the tensors' device, whose current stream would be another one
        if t.device != stream.device:
            raise ValueError(f"the stream is on {stream.device}, an operand on {t.device}")
    with torch.cuda.stream(stream):
        for t in tensors:
            t.record_stream(stream)
        return call()
