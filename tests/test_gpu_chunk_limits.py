"""The attention of chunks where its plan takes many steps, where parts of a tile see nothing but
scores of minus infinity, at a scale of 0, where wide fp32 heads hold values that are not finite, and
where requests share pages."""
import numpy as np
import pytest

from oracle import paged as pref
from oracle import serve as ref
import test_gpu_chunk as chunk
from test_gpu_chunk import _run, _step, _want, check
from test_gpu_paged import Case, _f64, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_tiles_than_steps_of_the_plan_take(dtype):
    """2500 tiles (128 heads a group: a row each) of three requests in one step of requests, two borders of
    1024 tiles among them, rows of no request on both sides.  Rows at the borders against the oracle; all
    of them against single rows, each side within 2^-10 (an error of a score of D 2^-24 times at most
    2^4, weights of 2^-17, both twice in a mean of |v| < 2^3)."""
    from gated_deltanet_prefill_chunkwise_amd import ops
    step, most = [(1100, 0), (0, 9), (900, 7), (500, 100)], 20
    cu, lens, rows = _step(step, front=3, behind=4)
    c = Case(21, lens, 128, 1, 64, 16, dtype)
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens, max_len=most)
    req, sees = ref.chunk_rows(cu, lens, rows, most)
    at = np.unique(np.concatenate([np.arange(x - 3, x + 4) for x in (3, 3 + 1024, 3 + 1100, 3 + 2000, 3 + 2048, 3 + 2500)]))
    at = at[(at >= 0) & (at < rows)]
    want = pref.attend(_f64(q)[at], _f64(c.k), _f64(c.v), c.table, sees[at], req=req[at], max_len=most)
    v = _f64(c.v)
    want[2]["vmax"] = np.full(want[1].shape, np.abs(v[np.isfinite(v)]).max())
    check(o[at], lse[at], want, "f32", dtype, 64)
    p, pl = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(sees), row_req=_i32(req), max_len=most, want_lse=True)
    assert float((o - p).abs().max()) <= 2.0 ** -9
    none = (sees <= 0).nonzero()[0]
    assert len(none) == 7 and not o[none].any() and bool((lse[none] == -float("inf")).all())
    some = sees > 0
    assert float((lse - pl)[some].abs().max()) <= 2.0 ** -9


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


@pytest.mark.parametrize("D", [128, 256])
def test_later_tokens_do_not_reach_earlier_rows_of_wide_heads(D):
    chunk.test_later_tokens_do_not_reach_earlier_rows("f32", D)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_requests_that_share_pages(dtype):
    """A common beginning: the same pages in the tables of several requests, and twice in one."""
    cu, lens, rows = _step([(40, 200), (3, 237), (1, 100), (70, 170)])
    c = Case(24, lens, 8, 2, 64, 16, dtype)
    c.table[1, :10] = c.table[0, :10]
    c.table[2, :6] = c.table[0, 3]
    c.table[3, 1:5] = c.table[0, 1:5]
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens)
    check(o, lse, _want(c, q, cu, lens), "f32", dtype, 64)
