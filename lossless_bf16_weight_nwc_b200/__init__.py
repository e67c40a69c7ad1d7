"""Lossless BF16 weight compression with a fused decode-GEMV for B200 (sm_100a).

The product is the C-ABI library libnwc.so (include/nwc.h); `_lib` binds it
with ctypes (loaded on first use, and it raises if the library is missing).
`synth` generates the seeded synthetic inputs; `autotune` picks a matrix's
tile width and code limit by timing the library's GEMV on the device;
`sharded` splits a matrix by output rows over a process group; `paged` holds
what a decode layer does between its projections (norms with the position
rotation, a paged key/value cache, attention over shared prefixes).
"""
import importlib

_PAGED = ("AttentionBlock", "PagedBatch", "PagedKV", "qk_norm_rope", "rope_frequencies")
__all__ = ["CompressedMatrix", "lib", *_PAGED]


def __getattr__(name):
    if name == "lib":
        return importlib.import_module(__name__ + "._lib")
    if name == "CompressedMatrix":
        return importlib.import_module(__name__ + "._lib").CompressedMatrix
    if name in _PAGED:
        return getattr(importlib.import_module(__name__ + ".paged"), name)
    raise AttributeError(name)
