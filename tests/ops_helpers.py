"""Helpers of the tests of the operators around the layer.  Test code only."""
import numpy as np

from gen.layers import bf16_bits_to_f32, f32_to_bf16_bits


def _bf16(a):
    return bf16_bits_to_f32(f32_to_bf16_bits(a)).astype(np.float64)


def rounded_from(got, ref, tol, bf16):
    """Where `got` is the value, in its type, of some number within tol of ref.  Rounding to
    nearest keeps order, so for bf16 that is: between the roundings of ref - tol and ref + tol
    (taken outwards to fp32 first)."""
    lo, hi = ref - tol, ref + tol
    if bf16:
        lo = _bf16(np.nextafter(lo.astype(np.float32), np.float32(-np.inf)))
        hi = _bf16(np.nextafter(hi.astype(np.float32), np.float32(np.inf)))
    return (lo <= got) & (got <= hi)
