"""The choice of blocks at magnitudes near the ends of the types: the lists equal those of the exact
scores, whatever the size of the queries, and for summaries of every size that paged_write makes
(2^-126 to 2^121), as far as heads of a group that differ by 2^d read summaries of 2^(d - 133) or more."""
import numpy as np
import pytest

from oracle import paged as ref
from test_gpu_paged import _f64, _i32, _t

pytestmark = pytest.mark.gpu


def _call(Hq, Hkv, D, dtype, rows, q_exp, page_exp, seed):
    """Queries and summaries whose powers of two span the given ranges (q_exp by head)."""
    import torch
    rng = np.random.default_rng(seed)
    n = 60
    codes = rng.integers(-127, 128, (n, Hkv, D)).astype(np.int8)
    scale = np.ldexp(1.0, rng.integers(page_exp[0], page_exp[1] + 1, (n, Hkv))).astype(np.float32)
    x = rng.standard_normal((rows, Hq, D)).clip(-3, 3)
    q = torch.from_numpy(np.ldexp(x, rng.integers(q_exp[0], q_exp[1] + 1, (rows, Hq, 1)))).cuda().to(_t(dtype))
    assert torch.isfinite(q).all()
    table = rng.permutation(n)[None].astype(np.int32)
    length = rng.integers(500, n * 16 + 1, rows).astype(np.int32)
    return codes, scale, q, table, length


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq, Hkv, D", [(2, 2, 64), (4, 2, 128), (16, 2, 64), (16, 1, 256), (20, 1, 128)])
@pytest.mark.parametrize("q_exp, page_exp", [
    ((120, 125), (-9, -6)),         # products of codes and large queries alone pass fp32
    ((119, 125), (-126, -100)),
    ((-140, -120), (-40, -30)),     # ... and of small ones fall below it
    ((-120, -120), (-126, -118)),
    ((-3, 3), (100, 121)),          # the largest summaries, the smallest
    ((0, 6), (-126, -119)),
    ((60, 66), (90, 121)),
    ((-60, 60), (-10, 10)),         # heads of one row far apart
])
def test_select_far_magnitudes(q_exp, page_exp, Hq, Hkv, D, dtype):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    for rows in (3, (1 << 16) // (Hkv * D) + 70):        # single rows, rows that share pages
        codes, scale, q, table, length = _call(Hq, Hkv, D, dtype, rows, q_exp, page_exp, Hq + D)
        req = np.zeros(rows, np.int32)
        got = ops.paged_select(q, torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(), _i32(table), _i32(length),
                               16, 7, row_req=_i32(req))
        torch.cuda.synchronize()
        pick = np.unique(np.r_[np.arange(min(rows, 40)), rows - 1])
        want = ref.select(_f64(q[pick]), codes, scale, table, length[pick], 16, 7, req=req[pick])
        assert np.array_equal(got.cpu().numpy()[pick], want), rows
