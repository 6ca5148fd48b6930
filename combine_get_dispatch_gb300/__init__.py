"""GB300-native DeepEP-style MoE dispatch / combine, with the router and the
experts' products around them, the whole layer for a few tokens and the update of
the experts' weights.

The product is libep.so (C ABI in include/ep.h, CUDA kernels for sm_103a in
csrc/); `ep` is its thin ctypes binding and `synth` the seeded workload
generator used by tests and the benchmark.
"""
from . import ep, synth  # noqa: F401

__all__ = ["ep", "synth"]
