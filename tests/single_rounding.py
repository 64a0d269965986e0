"""a b + c of fp32 tensors in one rounding, without an fp32 FMA."""
import torch


def fma(a, b, c):
    """a b is exact in 64 bits; the sum is rounded to odd there (its last bit set
    where it is inexact), after which the rounding to 24 bits is that of the
    exact value."""
    p, c = a.double() * b.double(), c.double()
    s = p + c
    t = s - p
    e = (p - (s - t)) + (c - t)  # s + e is exact
    bits = s.view(torch.int64)
    up = (e > 0) == (s > 0)  # away from zero is one more in the bits
    odd = torch.where((e != 0) & (bits & 1 == 0), torch.where(up, bits + 1, bits - 1), bits)
    return odd.view(torch.float64).float()
