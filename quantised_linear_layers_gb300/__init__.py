"""Fine-grained-scaled FP8 and microscaled 4-bit linear layers for GB300 (sm_103a).

The compute path is the CUDA library ``libqlinear.so`` (built from ``csrc/``)
behind a C ABI; ``ops`` is a thin binding over it (ctypes, and ``_fp4.so`` for the
4-bit calls). ``linear`` has the FP8 layer, ``fp4`` the 4-bit layers. Importing the
package does not load the library; the first op call does, and raises if it is
missing.
"""
__all__ = ["ops", "linear", "fp4", "synthetic"]
