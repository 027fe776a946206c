"""The attention of chunks where parts of a tile see nothing but scores of minus infinity, and at a scale
of 0."""
import pytest

from test_gpu_chunk import _run, _step, _want, check
from test_gpu_paged import Case, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, D", [("bf16", 64), ("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_under_scores_of_minus_infinity(dtype, D, value):
    """Keys of minus infinity have no weight, and 0 times a value that is not finite is no number: in that
    element of every row that sees it, wherever the context is cut; the other elements stay."""
    import torch
    cu, lens, rows = _step([(2, 20000)])
    c = Case(22, lens, 2, 1, D, 64, dtype)
    q = c.q(rows).abs() + 0.5
    c.k[_i32(c.table[0, :100]).long()] = -float("inf")          # of 6400 tokens: whole parts see nothing else
    clean, want_lse = _run(c, q, cu, lens)
    assert torch.isfinite(clean).all()
    c.v[int(c.table[0, 40]), 0, 5, 3] = value
    o, lse = _run(c, q, cu, lens)
    assert torch.isnan(o[..., 3]).all()
    assert torch.equal(lse, want_lse)
    rest = [e for e in range(D) if e != 3]
    assert torch.equal(o[..., rest], clean[..., rest])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite_at_a_scale_of_zero(dtype, value):
    """0 times what such a query gives is no number; other rows and heads have the plain mean."""
    import torch
    cu, lens, rows = _step([(40, 100), (1, 50)])
    c = Case(23, lens, 4, 2, 64, 32, dtype)
    q = c.q(rows)
    clean, clean_lse = _run(c, q, cu, lens, scale=0.0)
    check(clean, clean_lse, _want(c, q, cu, lens, scale=0.0), "f32", dtype, 64)
    q[7, 1, 9] = value
    o, lse = _run(c, q, cu, lens, scale=0.0)
    assert torch.isnan(o[7, 1]).all() and bool(torch.isnan(lse[7, 1]))
    o[7, 1], lse[7, 1] = clean[7, 1], clean_lse[7, 1]
    assert torch.equal(o, clean) and torch.equal(lse, clean_lse)
