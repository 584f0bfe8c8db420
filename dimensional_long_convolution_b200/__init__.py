"""B200-native gated nD FFT long convolution (HyenaND hot path).

The product is the C-ABI shared library libhyena_nd.so (include/hyena_nd.h),
built from csrc/ for sm_100a.  ``hyena_nd`` is its thin Python binding, ``hyena_nd_block`` that of the operators
around the convolution (include/hyena_nd_block.h).
"""
from . import workloads  # noqa: F401

__all__ = ["workloads", "hyena_nd", "hyena_nd_block"]
