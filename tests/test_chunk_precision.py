"""The bound of the attention of chunks with 16-bit inputs sees the parts in which weights enter.

A weight p enters its product rounded to the type: with m stored bits an error of at most
2^-(m+1) p, half a step (2^-8 bf16, 2^-11 fp16).  Its second part, the rounded remainder, leaves
2^-17 (bf16) or 2^-23 (fp16) of p, as test_paged_precision.py works out.  A 16-bit output takes
one part, an fp32 output two.
"""
import numpy as np
import pytest

from oracle import paged as ref
from test_gpu_chunk import TWO_PARTS
from test_gpu_paged import U, _t


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_bounds_see_parts(dtype):
    """One part breaks the bound of an fp32 output, and keeps that of a 16-bit one; half of the
    type's bits break that too."""
    import torch
    rng = np.random.default_rng(12)
    n, D, rows = 64, 64, 40
    cast = lambda x: torch.from_numpy(np.asarray(x)).to(_t(dtype)).double().numpy()
    q, k, v = cast(rng.standard_normal((rows, 1, D))), cast(rng.standard_normal((n // 16, 1, 16, D))), cast(rng.standard_normal((n // 16, 1, 16, D)))
    want, _, s = ref.attend(q, k, v, np.arange(n // 16)[None].repeat(rows, 0), np.full(rows, n))
    x = q[:, 0] @ k[:, 0].reshape(n, D).T * D ** -0.5
    p = np.exp2((x - x.max(1, keepdims=True)) / np.log(2) + (10 if dtype == "f16" else 0))
    one = cast(p)
    step = 2.0 ** np.floor(np.log2(p)) * U[dtype] ** 0.5
    coarse = np.round(p / step) * step
    out = lambda w: (w @ v[:, 0].reshape(n, D) / p.sum(1, keepdims=True))[:, None]
    small = (2.0 ** -35 * s["n"] * np.abs(v).max() if dtype == "f16" else 0 * s["n"])[..., None]
    worst = lambda o, weight, rounding: float((np.abs(o - want) / (s["absv"] * weight + small + rounding * np.abs(want) + 1e-30)).max())
    assert worst(out(one), TWO_PARTS[dtype], U["f32"]) > 1.5
    assert worst(out(one + cast(p - one)), TWO_PARTS[dtype], U["f32"]) <= 1.0
    assert worst(cast(out(one)), U[dtype], U[dtype]) <= 1.0
    assert worst(cast(out(coarse)), U[dtype], U[dtype]) > 1.5
