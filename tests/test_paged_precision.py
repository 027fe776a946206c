"""Attention with 16-bit inputs errs by two-part softmax weights and the output's own rounding,
whichever kernel takes a row: single rows, and rows that share their lists with their neighbours.

The bound is that of test_gpu_paged.py with the weights' term written out.  A weight p enters its
product as p1 + p2, p1 = p rounded to the type, p2 = p - p1 rounded to the type.  With a step of
2^-m at 1 (m = 7 bf16, 10 fp16), |p - p1| <= 2^-(m+1) for p in [1, 2), and what is left of that
lies in a binade whose step is at most 2^-(m+2) 2^-m: an error of at most 2^-(2m+3) p, 2^-17 for
bf16 and 2^-23 for fp16.  fp16 has no step below 2^-24: there the error is at most 2^-25, and the
row's largest weight is at least 2^10 at that scale, so 2^-35 of it for each of n keys.
"""
import numpy as np
import pytest

from oracle import paged as ref
from test_gpu_paged import LENS, U, Case, _f64, _i32, _lists, _prompt, _t

TWO_PARTS = {"bf16": (2.0 ** -17, 0.0), "f16": (2.0 ** -23, 2.0 ** -35)}


def worst(o, want, out, dtype, D, vmax):
    """Largest error over its bound."""
    ro, _, s = want
    u = U["f32"]
    score = D * u * s["qk"] + 2 * u * s["xmax"] + 2.0 ** -21
    rel, floor = TWO_PARTS[dtype]
    tol = s["absv"] * (rel + 2 * score + 2 * s["n"] * u)[..., None] + (floor * vmax * s["n"])[..., None] + U[out] * np.abs(ro) + 1e-30
    return float((np.abs(o - ro) / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_bound_sees_a_lost_part(dtype):
    """Weights of one part break the bound, of two parts keep it, with a 16-bit output."""
    import torch
    rng = np.random.default_rng(11)
    n, D, rows = 64, 64, 40
    cast = lambda x: torch.from_numpy(np.asarray(x)).to(_t(dtype)).double().numpy()
    q, k, v = cast(rng.standard_normal((rows, 1, D))), cast(rng.standard_normal((n // 16, 1, 16, D))), cast(rng.standard_normal((n // 16, 1, 16, D)))
    want = ref.attend(q, k, v, np.arange(n // 16)[None].repeat(rows, 0), np.full(rows, n))
    x = q[:, 0] @ k[:, 0].reshape(n, D).T * D ** -0.5
    p = np.exp2((x - x.max(1, keepdims=True)) / np.log(2) + (10 if dtype == "f16" else 0))
    one = cast(p)
    got = [cast(w @ v[:, 0].reshape(n, D) / p.sum(1, keepdims=True))[:, None] for w in (one, one + cast(p - one))]
    far, near = (worst(o, want, dtype, dtype, D, np.abs(v).max()) for o in got)
    assert far > 1.5 and near <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("Hq, Hkv, D, P, K", [(8, 1, 64, 16, 5), (8, 1, 128, 32, 3), (16, 2, 256, 16, 4), (5, 1, 128, 16, 5)])
def test_rows_that_share_lists(Hq, Hkv, D, P, K, dtype, out):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    gp = 1 << (Hq // Hkv - 1).bit_length()
    R = 256 * (128 // gp) // Hkv + 50
    c, req, length, lists, q = _prompt(Hq + D + P, Hq, Hkv, D, P, dtype, K, np.array([R + 70]), [R], alike=16)
    t = [_i32(x) for x in (c.table, length, lists, req)]
    ws = torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda")
    o, _ = ops.paged_attend_sparse(q, c.k, c.v, t[0], t[1], t[2], row_req=t[3], out_dtype=_t(out), workspace=ws)
    torch.cuda.synchronize()
    assert (ws.view(torch.int32) == 1).sum() >= 40, "rows that share their lists, and not single rows alone"
    rows = np.unique(c.rng.integers(100, R, 120))
    want = ref.attend(_f64(q[rows]), _f64(c.k), _f64(c.v), c.table, length[rows], req[rows], blocks=lists[rows])
    v = _f64(c.v)
    err = worst(_f64(o[torch.from_numpy(rows).cuda()]), want, out, dtype, D, np.abs(v[np.isfinite(v)]).max())
    print(f"err / bound {err:.3f}")
    assert err <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("Hq, Hkv, D, P", [(4, 1, 64, 16), (8, 2, 128, 64), (16, 1, 256, 64), (20, 1, 64, 32)])
@pytest.mark.parametrize("sparse", [False, True])
def test_single_rows(Hq, Hkv, D, P, dtype, out, sparse):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(Hq + D + P + 2, LENS, Hq, Hkv, D, P, dtype)
    q = c.q(len(LENS))
    lists = _lists(c.rng, len(LENS), Hkv, 3, -(-c.lens // P)) if sparse else None
    args = (q, c.k, c.v, _i32(c.table), _i32(c.lens))
    o, _ = ops.paged_attend_sparse(*args, _i32(lists), out_dtype=_t(out)) if sparse else ops.paged_attend(*args, out_dtype=_t(out))
    torch.cuda.synchronize()
    want = ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens, blocks=lists)
    v = _f64(c.v)
    err = worst(_f64(o), want, out, dtype, D, np.abs(v[np.isfinite(v)]).max())
    print(f"err / bound {err:.3f}")
    assert err <= 1.0
