"""B200-native DiT-MoE sparse expert layer (forward, backward, the balance loss's
statistics and gradients, the optimizer's step): C-ABI library + thin binding.

``inputs`` (seeded synthetic workloads) and ``metrics`` (work accounting) load
without a GPU.  The compute entry points live in ``binding`` (ctypes over
``libmoe.so``), ``layer`` (buffer management around the four calls) and ``optim``
(gradient norm and AdamW); they load the CUDA library on import and fail loudly when it is missing.
"""
import importlib

__all__ = ["inputs", "metrics", "binding", "layer", "optim"]


def __getattr__(name):
    if name in __all__:
        return importlib.import_module(f"{__name__}.{name}")
    raise AttributeError(name)
