"""Error bounds of the row operators' tests, from the arithmetic of the kernels: float32
sums and products (unit roundoff 2^-24), then one rounding to the output's type."""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype, ref):
    """Largest error of one rounding to dtype: half an epsilon of the value, or half the
    smallest subnormal."""
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(ref) * (fi.eps / 2), float(fi.smallest_normal) * fi.eps / 2)


def row_sum_ops(d):
    """Float32 operations that one term of a sum over a row can pass through: a lane adds
    at most d / 16 + 8 elements (at least 16 lanes share a row of over 128 elements) and
    the lanes meet in a tree of up to 10 levels plus a few scalings."""
    return d / 16 + 32


def assert_near(name, got, ref, bound):
    """|got - ref| <= bound for every element; got is a tensor, ref and bound float64."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    over = np.abs(got - ref) - bound
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[worst] <= 0, (
        f"{name}: {got[worst]} for {ref[worst]}, off by {abs(got[worst] - ref[worst])}, bound "
        f"{np.broadcast_to(bound, ref.shape)[worst]} at {worst}")


def wide(t, offset=1, pad=3):
    """The same values as a slice of a wider tensor: rows with another stride and, for an
    odd offset, off any alignment but their type's."""
    T, d = t.shape
    big = torch.full((T, d + offset + pad), float("nan"), dtype=t.dtype, device=t.device)
    v = big[:, offset:offset + d]
    v.copy_(t)
    return v
