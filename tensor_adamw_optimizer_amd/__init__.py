"""Fused multi-tensor AdamW for AMD MI355X (gfx950).

The update runs in ``libapexw.so`` (HIP kernels behind the C ABI of
``include/apexw.h``); ``_lib`` is its ctypes binding and ``AdamW`` a torch
wrapper that supplies device memory and the stream.  ``ops`` has the operators
of a model around the step: the gated feed-forward block, the linear cross
entropy and the norm of queries and keys with rotation.  Importing the package
does not load the library; the first call that needs it does, and raises if
it has not been built.
"""
import importlib

from . import _lib
from ._lib import ApexwError

__all__ = ["AdamW", "ApexwError", "_lib", "ops"]


def __getattr__(name):
    if name == "AdamW":
        from .optim import AdamW
        return AdamW
    if name == "ops":
        return importlib.import_module(".ops", __name__)
    raise AttributeError(name)
