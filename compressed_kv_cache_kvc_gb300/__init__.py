"""Compressed-KV decode step for GB300 (sm_103a).

The compute lives in the CUDA library ``libkvc.so`` (C ABI: ``include/kvc.h``);
``KVCache``, ``BlockScaledCache``, ``Rotary`` and ``prompt_attention`` are thin bindings that
pass device pointers and the torch CUDA stream to it.
"""
from . import workloads  # noqa: F401

__all__ = ["BlockScaledCache", "KVCache", "Rotary", "document_runs", "prompt_attention", "workloads"]


def __getattr__(name):
    if name == "KVCache":
        from .cache import KVCache
        return KVCache
    if name == "BlockScaledCache":
        from .block_cache import BlockScaledCache
        return BlockScaledCache
    if name == "Rotary":
        from .rotary import Rotary
        return Rotary
    if name in ("prompt_attention", "document_runs"):
        from . import prompt
        return getattr(prompt, name)
    raise AttributeError(name)
