"""Plain 64-bit forms and error bounds for the tests of the bf16 / fp16 operators (CPU)."""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


def floor_step(dtype):
    """Half the distance between the smallest subnormals: what a rounding near zero is off by."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def randn(shape, dtype, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * std).to(dtype)


def ints(shape, dtype, seed, lo=-2, hi=2):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=gen).to(dtype)


def spans(splits, M):
    """Row ranges of the groups, clamped as the library clamps them, and the rows they cover."""
    out, at = [], 0
    for m in splits:
        e = min(at + max(int(m), 0), M)
        out.append((at, e))
        at = e
    return out, at


def product(a, b):
    """(a @ b, sum of |a| |b|) in 64 bits."""
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


def assert_close(got, want, mag, terms, what, dtype=None):
    """got (device, any dtype) against the 64-bit want.  One rounding of the result to got's type,
    plus the fp32 accumulation: each of the `terms` products is exact in fp32 up to 2^-24 and enters
    at most `terms` additions that may each be off by a whole unit 2^-23 of a partial sum, itself at
    most mag = sum |a| |b|."""
    got64 = got.detach().cpu().double()
    dt = dtype or got.dtype
    tol = half_step(dt) * want.abs() * (1 + 2.0 ** -8) + (terms + 8) * 2.0 ** -23 * mag + floor_step(dt)
    bad = ~((got64 - want).abs() <= tol)
    if bad.any():
        i = tuple(int(v[0]) for v in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {got64[i]}, "
                             f"want {want[i]}, tolerance {tol[i]}")


def np_ids(n, groups, seed, drop=0.0):
    r = np.random.RandomState(seed)
    ids = r.randint(0, groups, size=n).astype(np.int32)
    ids[r.rand(n) < drop] = -1
    return ids
