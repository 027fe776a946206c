"""GPU parity of the attention of chunks against the fp64 oracle: the bounds are those of the
attention of single rows (test_gpu_paged.check).  Weights of 16-bit inputs err by 2^-17 (bf16) or
2^-23 (fp16) of themselves for an fp32 output, where they enter in two parts, and by half a step
of the type (2^-8, 2^-11) for a 16-bit one, as the header says; by nothing with fp32 inputs."""
import numpy as np
import pytest

from oracle import serve as ref
from test_gpu_paged import U, Case, _f64, _i32, _t

pytestmark = pytest.mark.gpu

TWO_PARTS = {"f32": 0.0, "bf16": 2.0 ** -17, "f16": 2.0 ** -23}


def check(o, lse, want, out, dtype, D):
    ro, rl, s = want
    o, lse = _f64(o), _f64(lse)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.isfinite(o).all()
    u = U["f32"]
    score = D * u * s["qk"] + 2 * u * s["xmax"] + 2.0 ** -21
    sums = s["n"] * u
    # fp16: nothing lies under 2^-24, so a remainder errs by 2^-25 at weights of up to 2^10 or more (2^-35 of the largest), for each key
    small = 2.0 ** -35 * s["n"] if dtype == "f16" else 0.0
    vmax = s.get("vmax", np.zeros(rl.shape))
    tiny = 2.0 ** -25 if out == "f16" else 1e-30          # half the smallest step of an fp16 o
    weight = TWO_PARTS[dtype] if out == "f32" or dtype == "f32" else U[dtype]
    tol = s["absv"] * (weight + 2 * score + 2 * sums)[..., None] + U[out] * np.abs(ro) + tiny + (small * vmax)[..., None] * np.ones(D)
    err = np.abs(o - ro)
    worst = float((err / tol).max())
    ltol = (score + sums + 4 * u * np.abs(np.where(empty, 0, rl)) + 2.0 ** -22)[~empty]
    lworst = float((np.abs(lse[~empty] - rl[~empty]) / ltol).max()) if ltol.size else 0.0
    print(f"err / bound: o {worst:.3f}  lse {lworst:.3f}")
    assert worst <= 1.0 and lworst <= 1.0
    assert not o[empty].any()


def _want(c, q, cu, lens, **kw):
    want = ref.attend_chunk(_f64(q), _f64(c.k), _f64(c.v), c.table, cu, lens, **kw)
    v = _f64(c.v)
    want[2]["vmax"] = np.full(want[1].shape, np.abs(v[np.isfinite(v)]).max() if np.isfinite(v).any() else 0.0)
    return want


def _run(c, q, cu, lens, **kw):
    from gated_deltanet_prefill_chunkwise_amd import ops
    return ops.paged_attend_chunk(q, c.k, c.v, _i32(c.table), _i32(cu), _i32(lens), want_lse=True, **kw)


# (new, cached) of requests: single tokens, borders of stages and tiles, prompts, no rows, nothing cached
STEP = [(1, 0), (1, 15), (1, 16), (5, 0), (0, 40), (16, 17), (33, 31), (64, 64), (1, 200), (0, 0), (65, 0), (7, 127), (90, 43)]
SHAPES = [  # Hq, Hkv, D, P
    (4, 1, 64, 16), (8, 2, 128, 64), (6, 2, 128, 32), (5, 5, 64, 128), (16, 1, 256, 64), (15, 3, 64, 16), (8, 1, 256, 16),
    (20, 1, 64, 32), (33, 1, 128, 64), (4, 4, 128, 16), (7, 7, 256, 32), (150, 1, 64, 64), (260, 2, 128, 32),
]


def _step(step, front=0, behind=0):
    new, cached = np.array(step).T
    cu = front + np.concatenate([[0], np.cumsum(new)])
    return cu, new + cached, int(cu[-1]) + behind


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("Hq, Hkv, D, P", SHAPES)
def test_chunk(Hq, Hkv, D, P, dtype, out):
    cu, lens, rows = _step(STEP if Hq < 100 else STEP[:8], front=2, behind=9)
    c = Case(Hq * D + P, lens, Hq, Hkv, D, P, dtype)
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens, out_dtype=_t(out))
    check(o, lse, _want(c, q, cu, lens), out, dtype, D)


@pytest.mark.parametrize("new, cached", [(1, 0), (1, 1), (1, 5000), (2, 63), (127, 1), (128, 0), (129, 129), (300, 2000), (1000, 0), (40, 9001)])
@pytest.mark.parametrize("Hq, Hkv, D, P, dtype", [(8, 2, 128, 64, "bf16"), (16, 2, 256, 32, "f16"), (3, 3, 64, 16, "bf16"), (5, 1, 64, 128, "f32")])
def test_one_request(new, cached, Hq, Hkv, D, P, dtype):
    if new * (new + cached) * Hq > 6_000_000:
        new = max(1, 6_000_000 // (Hq * (new + cached)))
    cu, lens, rows = _step([(new, cached)])
    c = Case(new + cached, lens, Hq, Hkv, D, P, dtype)
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens)
    check(o, lse, _want(c, q, cu, lens), "f32", dtype, D)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_requests(dtype):
    """More requests than one step of the plan takes, most without rows."""
    rng = np.random.default_rng(2)
    B = 2500
    new = np.where(rng.random(B) < 0.1, rng.integers(1, 4, B), 0)
    new[1023], new[1024], new[B - 1] = 40, 3, 2
    cached = np.where(new > 0, rng.integers(0, 40, B), 0)
    cu, lens, rows = _step(list(zip(new, cached)), front=1, behind=3)
    c = Case(7, lens, 4, 2, 64, 16, dtype)
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens)
    check(o, lse, _want(c, q, cu, lens), "f32", dtype, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_lengths_that_leave_rows_empty(dtype):
    """Fewer tokens than rows, none, negative ones, rows cut at max_len, rows beyond the call's."""
    cu = np.array([0, 5, 5, 25, 30, 47, 90])
    lens = np.array([3, 0, 7, -4, 17, 60])
    c = Case(3, np.maximum(lens, 0), 8, 2, 64, 16, dtype)
    q = c.q(70)                                       # the last request's rows end inside
    o, lse = _run(c, q, cu, lens)
    want = _want(c, q, cu, lens)
    assert np.isneginf(want[1]).sum() == (2 + 13 + 5) * 8
    check(o, lse, want, "f32", dtype, 64)
    o, lse = _run(c, q, cu, lens, max_len=9)
    check(o, lse, _want(c, q, cu, lens, max_len=9), "f32", dtype, 64)
    o, lse = _run(c, q, np.zeros(7, int), lens)       # no rows of any request
    assert not o.any() and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_pages_that_are_none(dtype):
    """A context with holes: pages outside the cache take no part, whole stages of them too."""
    cu, lens, rows = _step([(40, 400), (3, 90), (1, 300), (200, 0), (5, 30)])
    c = Case(4, lens, 6, 2, 64, 16, dtype)
    n_pages = c.k.shape[0]
    c.table[0, 1], c.table[0, 4:12], c.table[0, 26] = -1, n_pages, 2 ** 31 - 1
    c.table[1, 5], c.table[2, :18] = -3, -1
    c.table[4, :] = n_pages + 5                       # nothing left at all
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens)
    check(o, lse, _want(c, q, cu, lens), "f32", dtype, 64)


@pytest.mark.parametrize("dtype, D", [("bf16", 128), ("f16", 64), ("bf16", 256), ("f32", 64)])
def test_later_tokens_do_not_reach_earlier_rows(dtype, D):
    """Keys and values of a request's own new tokens that are not finite change only the rows that see them."""
    import torch
    P, new, cached = 32, 150, 75
    cu, lens, rows = _step([(new, cached), (30, 3)])
    c = Case(5, lens, 4, 2, D, P, dtype)
    q = c.q(rows)
    clean, lse = _run(c, q, cu, lens)
    for at, value in ((cached + 61, float("nan")), (cached + 140, float("inf")), (cached + 17, -float("inf"))):
        page, off = int(c.table[0, at // P]), at % P
        for t, name in ((c.v, "v"), (c.k, "k")):
            keep = t[page, :, off].clone()
            t[page, 0, off, 3] = value
            o, l = _run(c, q, cu, lens)
            first = at - cached                       # the first row that sees it
            heads = slice(0, 2)                       # of key/value head 0
            assert torch.equal(torch.isfinite(o[:first]), torch.ones_like(o[:first], dtype=torch.bool)), (name, value)
            check(o[:first].contiguous(), l[:first].contiguous(), _cut(c, q, cu, lens, first), "f32", dtype, D)
            if name == "v":
                assert not torch.isfinite(o[first:new, heads, 3]).any()
                rest = torch.cat([o[first:new, heads, :3], o[first:new, heads, 4:]], -1)
                assert torch.isfinite(rest).all() and torch.isfinite(l).all()
            elif value != value:
                assert torch.isnan(o[first:new, heads]).all()
            assert torch.isfinite(o[:new, 2:]).all() and torch.equal(o[new:], clean[new:]) and torch.equal(l[new:], lse[new:])
            t[page, :, off] = keep


def _cut(c, q, cu, lens, first):
    """The oracle's rows in front of `first` (the first request's)."""
    want = ref.attend_chunk(_f64(q)[:first], np.nan_to_num(_f64(c.k), posinf=0, neginf=0), np.nan_to_num(_f64(c.v), posinf=0, neginf=0),
                            c.table[:1], [0, first], [int(lens[0]) - (int(cu[1]) - first)])
    want[2]["vmax"] = np.full(want[1].shape, 10.0)
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0, 1e-30])
def test_scales(scale, dtype):
    cu, lens, rows = _step([(70, 100), (1, 50)])
    c = Case(6, lens, 4, 2, 64, 32, dtype)
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens, scale=scale)
    check(o, lse, _want(c, q, cu, lens, scale=scale), "f32", dtype, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_large_scores(dtype):
    """Scores of some hundreds that rise and fall along the context, so that the reference moves often."""
    cu, lens, rows = _step([(80, 300)])
    c = Case(9, lens, 4, 1, 64, 16, dtype, spread=1.0)
    ramp = np.abs(((np.arange(380) * 7) % 97) - 48) / 8.0
    for t, x in enumerate(ramp):
        c.k[int(c.table[0, t // 16]), :, t % 16] *= float(x)
    q = c.q(rows) * 3
    o, lse = _run(c, q, cu, lens, scale=1.0)
    check(o, lse, _want(c, q, cu, lens, scale=1.0), "f32", dtype, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_lowest_and_infinite_scores(dtype):
    """Keys of the type's lowest value and of minus infinity, seen by every row: weights of 0, not NaN, while others are seen too."""
    import torch
    cu, lens, rows = _step([(40, 64)])
    c = Case(10, lens, 2, 1, 64, 16, dtype)
    q = c.q(rows).abs() + 0.5
    low = float(torch.finfo(_t(dtype)).min)
    for page, value in ((0, low), (1, -float("inf"))):
        c.k[int(c.table[0, page])] = value
    o, lse = _run(c, q, cu, lens, scale=0.1)
    want = ref.attend_chunk(_f64(q), np.where(np.isneginf(_f64(c.k)), -1e300, _f64(c.k)), _f64(c.v), c.table, cu, lens, scale=0.1)
    seen = _f64(c.k)[c.table[0, 2:]]                 # the bound's sizes without the keys that have no weight
    big = float(np.nanmax(np.abs(np.where(np.isfinite(seen), seen, 0)))) * float(q.max()) * 64 * 0.1
    want[2]["qk"] = np.full(want[1].shape, big)
    want[2]["xmax"] = want[2]["qk"]
    want[2]["vmax"] = np.full(want[1].shape, 10.0)
    check(o, lse, want, "f32", dtype, 64)


def test_strided_queries_given_outputs_and_workspace():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    cu, lens, rows = _step([(40, 20), (3, 100)], behind=4)
    c = Case(11, lens, 8, 2, 128, 64, "bf16")
    wide = c.g(c.rng.standard_normal((rows, 12, 128)))
    q = wide[:, 2:10]
    o, lse = torch.full((rows, 8, 128), 7.0, device="cuda", dtype=torch.float16), torch.full((rows, 8), 7.0, device="cuda")
    shape = ops._paged(rows, 8, c.k.shape, torch.bfloat16, torch.float16, *c.table.shape, None)
    ws = torch.full((ops.paged_chunk_workspace_bytes(shape),), 255, dtype=torch.uint8, device="cuda")
    r = _run(c, q, cu, lens, o=o, lse=lse, workspace=ws)
    assert r[0] is o and r[1] is lse
    check(o, lse, _want(c, q, cu, lens), "f16", "bf16", 128)
    plain, _ = ops.paged_attend_chunk(q.contiguous(), c.k, c.v, _i32(c.table), _i32(cu), _i32(lens), out_dtype=torch.float16)
    assert torch.equal(plain, o)
    with pytest.raises(ops.SgdnError) as e:
        _run(c, q, cu, lens, o=o, workspace=ws[:-1])
    assert e.value.status == -3


def test_agrees_with_single_rows():
    """The same rows by sgdn_paged_attend: both within their bounds of the oracle, and of each other."""
    from gated_deltanet_prefill_chunkwise_amd import ops
    cu, lens, rows = _step([(1, 700), (60, 500), (1, 3), (200, 0)])
    c = Case(12, lens, 16, 4, 128, 64, "bf16")
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens)
    req, sees = ref.chunk_rows(cu, lens, rows)
    p, pl = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(sees), row_req=_i32(req), want_lse=True)
    want = _want(c, q, cu, lens)
    check(o, lse, want, "f32", "bf16", 128)
    check(p, pl, want, "f32", "bf16", 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_pages(dtype):
    """Pages whose elements lie beyond 2^31 and 2^32 elements of the cache."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    P, Hkv, D, new, cached = 128, 8, 128, 30, 500
    per = Hkv * P * D
    n_pages = (1 << 32) // per + 40
    k = torch.zeros((n_pages, Hkv, P, D), device="cuda", dtype=_t(dtype))
    v = torch.zeros_like(k)
    n = -(-(new + cached) // P)
    far = np.array([n_pages - 1, (1 << 31) // per, (1 << 32) // per, 3, n_pages - 7])[:n]
    for p in far:
        k[p].normal_()
        v[p].normal_()
    q = torch.randn((new, 16, D), device="cuda").to(_t(dtype))
    o, lse = ops.paged_attend_chunk(q, k, v, _i32(far[None]), _i32([0, new]), _i32([new + cached]), want_lse=True)
    near = torch.from_numpy(far).cuda()
    table = np.arange(n, dtype=np.int32)[None]
    want = ref.attend_chunk(_f64(q), _f64(k[near]), _f64(v[near]), table, [0, new], [new + cached])
    check(o, lse, want, "f32", dtype, D)


def test_binding_refusals():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    cu, lens, rows = _step([(10, 20)])
    c = Case(13, lens, 4, 2, 64, 16, "bf16")
    q, table, cu, lens = c.q(rows), _i32(c.table), _i32(cu), _i32(lens)
    call = lambda **kw: ops.paged_attend_chunk(**dict(dict(q=q, k_cache=c.k, v_cache=c.v, table=table, cu=cu, lens=lens), **kw))  # noqa: E731
    for kw in (dict(q=q.half()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(cu=cu[:-1]), dict(cu=cu.long()), dict(lens=lens.cpu()),
               dict(lens=torch.cat([lens, lens])), dict(table=table[0]), dict(v_cache=c.v.half()), dict(k_cache=c.k[0]),
               dict(o=torch.zeros(1, device="cuda")), dict(lse=torch.zeros((rows, 4), device="cuda", dtype=torch.float16)),
               dict(max_len=0), dict(max_len=1 << 32), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
               dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw, status in ((dict(max_len=1 << 20), -2), (dict(scale=float("inf")), -1), (dict(q=c.g(np.zeros((rows, 3, 64)))), -2)):
        with pytest.raises(ops.SgdnError) as e:
            call(**kw)
        assert e.value.status == status
    none, _ = call(q=q[:0])
    assert none.shape == (0, 4, 64)


@pytest.mark.parametrize("Hq, Hkv, D, P, dtype, new, cached", [
    (8, 1, 128, 64, "bf16", 3, 60000), (4, 1, 64, 16, "f16", 1, 30000), (2, 1, 256, 32, "bf16", 2, 20011), (3, 1, 64, 16, "f32", 5, 12000),
    (2, 1, 256, 64, "f32", 1, 9000), (4, 2, 128, 64, "f32", 2, 9000),
])
def test_few_rows_over_long_contexts(Hq, Hkv, D, P, dtype, new, cached):
    """Tiles of many parts, which several sets of waves join; a context with a hole as long as some of them."""
    cu, lens, rows = _step([(new, cached)], behind=1)
    c = Case(cached, lens, Hq, Hkv, D, P, dtype)
    c.table[0, 2000 // P:8000 // P] = -1
    q = c.q(rows)
    o, lse = _run(c, q, cu, lens)
    check(o, lse, _want(c, q, cu, lens), "f32", dtype, D)
