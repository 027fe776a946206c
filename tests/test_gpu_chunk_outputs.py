"""16-bit outputs of the attention of chunks: the weights of 16-bit inputs enter in two parts whatever
the output's type, so that beside fp32's roundings and its own o errs by 2^-17 (bf16) or 2^-23 (fp16, and
2^-35 of the largest weight for each key) of the weighted mean of |v|, as sgdn_paged_attend's does; and
the calls that the other tests make with an fp32 output, with one of 16 bits."""
import numpy as np
import pytest

import test_gpu_chunk as chunk
from test_gpu_chunk import TWO_PARTS, _run, _step, _want
from test_gpu_paged import U, Case, _f64, _t

pytestmark = pytest.mark.gpu


def check(o, lse, want, out, dtype, D):
    """test_gpu_chunk.check, with a second part for every output."""
    chunk.check(o, lse, want, out, dtype, D)
    ro, rl, s = want
    score = D * U["f32"] * s["qk"] + 2 * U["f32"] * s["xmax"] + 2.0 ** -21
    small = 2.0 ** -35 * s["n"] * s["vmax"] if dtype == "f16" else 0.0 * s["n"]
    tiny = 2.0 ** -25 if out == "f16" else 1e-30
    tol = s["absv"] * (TWO_PARTS[dtype] + 2 * score + 2 * s["n"] * U["f32"])[..., None] + U[out] * np.abs(ro) + tiny + small[..., None]
    worst = float((np.abs(_f64(o) - ro) / tol).max())
    print(f"err / bound of two parts: {worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("bf16", "f16"), ("f16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("Hq, Hkv, D, P", [(8, 2, 128, 64), (5, 5, 64, 128), (16, 1, 256, 64), (33, 1, 128, 16)])
def test_weights_of_two_parts(Hq, Hkv, D, P, dtype, out):
    cu, lens, rows = _step(chunk.STEP, front=2, behind=9)
    c = Case(Hq * D + P + 1, lens, Hq, Hkv, D, P, dtype)
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens, out_dtype=_t(out))
    check(o, lse, _want(c, q, cu, lens), out, dtype, D)


@pytest.fixture(params=["bf16", "f16"])
def out(request, monkeypatch):
    """The other file's calls with an output of the inputs' 16-bit type."""
    t, run = request.param, chunk._run
    monkeypatch.setattr(chunk, "_run", lambda *a, **kw: run(*a, **dict(dict(out_dtype=_t(t)), **kw)))
    monkeypatch.setattr(chunk, "check", lambda o, lse, want, _, dtype, D, own=chunk.check: _both(own, o, lse, want, t, dtype, D))
    return t


def _both(own, o, lse, want, t, dtype, D):
    with pytest.MonkeyPatch.context() as m:
        m.setattr(chunk, "check", own)
        check(o, lse, want, t, dtype, D)


@pytest.mark.parametrize("Hq, Hkv, D, P", [(8, 2, 128, 64), (3, 3, 64, 16), (16, 2, 256, 32)])
@pytest.mark.parametrize("new, cached", [(1, 0), (1, 5000), (127, 1), (129, 129), (300, 2000), (40, 9001)])
def test_one_request(new, cached, Hq, Hkv, D, P, out):
    chunk.test_one_request(new, cached, Hq, Hkv, D, P, out)


def test_lengths_that_leave_rows_empty(out):
    chunk.test_lengths_that_leave_rows_empty(out)


def test_pages_that_are_none(out):
    chunk.test_pages_that_are_none(out)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_later_tokens_do_not_reach_earlier_rows(D, out):
    chunk.test_later_tokens_do_not_reach_earlier_rows(out, D)


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0, 1e-30])
def test_scales(scale, out):
    chunk.test_scales(scale, out)


def test_large_scores(out):
    chunk.test_large_scores(out)


def test_lowest_and_infinite_scores(out):
    chunk.test_lowest_and_infinite_scores(out)


@pytest.mark.parametrize("Hq, Hkv, D, P, new, cached", [(8, 1, 128, 64, 3, 60000), (4, 1, 64, 16, 1, 30000), (2, 1, 256, 32, 2, 20011)])
def test_few_rows_over_long_contexts(Hq, Hkv, D, P, new, cached, out):
    chunk.test_few_rows_over_long_contexts(Hq, Hkv, D, P, out, new, cached)
