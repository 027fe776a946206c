"""GPU parity of the paged attention operators against the fp64 oracle.

Integers (bookkeeping, summaries, picked blocks) must be equal.  Attention is
held to a bound made of its roundings.  With u(t) half a step of type t
(2^-24 fp32, 2^-11 fp16, 2^-8 bf16), n keys, X = max |x| and Q = max scale
sum |q k| over the row's keys, all from the oracle:
  scores      D u(f32) Q from the sum of D products, 2 u(f32) X from scaling;
              an error e of a score is an error e of the weight's logarithm,
              and 2^-21 is allowed to the exponential itself
  weights     u(type) each where they are rounded to 16 bits; none for fp32
              inputs, u^2 for an fp32 o (two parts)
  sums        n u(f32) for each of the two sums
  output      u(o type) |o|
The first three act on sum p |v|, and twice: in the numerator and the sum.
"""
import numpy as np
import pytest

from oracle import paged as ref

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _t(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _f64(t):
    return t.double().cpu().numpy()


def _i32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Case:
    """Requests with a cache whose every unused place holds NaN."""

    def __init__(self, seed, lens, Hq, Hkv, D, P, dtype, width=None, extra=3, spread=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.P, self.Hq, self.Hkv, self.D, self.dtype = P, Hq, Hkv, D, dtype
        self.lens = np.asarray(lens)
        blocks = -(-self.lens // P)
        W = max(int(blocks.max()), 1) if width is None else width
        n_pages = int(blocks.sum()) + extra
        ids = rng.permutation(n_pages)
        # beyond a request's pages: numbers of pages that do not exist
        table = rng.choice(np.array([-1, -7, n_pages, 2 ** 31 - 1]), (len(lens), W)).astype(np.int32)
        k, v = rng.standard_normal((2, n_pages, Hkv, P, D)) * spread
        used = np.zeros((n_pages, P), bool)
        at = 0
        for b, n in enumerate(self.lens):
            for j in range(blocks[b]):
                table[b, j] = ids[at]
                used[ids[at], :min(P, n - j * P)] = True
                at += 1
        hole = ~used[:, None, :, None]
        k, v = np.where(hole, np.nan, k), np.where(hole, np.inf, v)
        g = lambda x: torch.from_numpy(x).cuda().to(_t(dtype))
        self.table, self.k, self.v = table, g(k), g(v)
        self.rng, self.g = rng, g

    def q(self, rows):
        return self.g(self.rng.standard_normal((rows, self.Hq, self.D)))


def check(o, lse, want, out, dtype, D):
    ro, rl, s = want
    o, lse = _f64(o), _f64(lse)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.isfinite(o).all()
    u = U["f32"]
    score = D * u * s["qk"] + 2 * u * s["xmax"] + 2.0 ** -21
    weight = 0.0 if dtype == "f32" else U[dtype] ** 2 if out == "f32" else U[dtype]
    sums = s["n"] * u
    tol = s["absv"] * (weight + 2 * score + 2 * sums)[..., None] + U[out] * np.abs(ro) + 1e-30
    err = np.abs(o - ro)
    worst = float((err / tol).max())
    ltol = (score + sums + 4 * u * np.abs(np.where(empty, 0, rl)) + 2.0 ** -22)[~empty]
    lworst = float((np.abs(lse[~empty] - rl[~empty]) / ltol).max()) if ltol.size else 0.0
    print(f"err / bound: o {worst:.3f}  lse {lworst:.3f}")
    assert worst <= 1.0 and lworst <= 1.0
    assert not o[empty].any()


# attend ---------------------------------------------------------------------

LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 531]
SHAPES = [  # Hq, Hkv, D, P
    (4, 1, 64, 16), (8, 2, 128, 64), (6, 2, 128, 32), (5, 5, 64, 128), (16, 1, 256, 64),
    (15, 3, 64, 16), (8, 1, 256, 16), (20, 1, 64, 32), (33, 1, 128, 64), (32, 2, 128, 128),
]


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
                                        ("f32", "f32"), ("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("Hq, Hkv, D, P", SHAPES)
def test_attend(Hq, Hkv, D, P, dtype, out):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(Hq + D + P, LENS, Hq, Hkv, D, P, dtype)
    q = c.q(len(LENS))
    o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(c.lens), out_dtype=_t(out), want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens), out, dtype, D)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n, B", [(1, 1), (700, 1), (5003, 1), (4999, 3), (1023, 40)])
def test_attend_splits(n, B, dtype):
    """Few rows: the length is split and joined; the parts of short rows are empty."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    lens = np.maximum(0, n - 977 * np.arange(B) % (n + 1))
    c = Case(n + B, lens, 4, 2, 128, 64, dtype, width=5003 // 64 + 1)
    q = c.q(B)
    o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(lens), want_lse=True)
    o2, _ = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(lens), max_len=max(n, 1))
    torch.cuda.synchronize()
    want = ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, lens)
    check(o, lse, want, "f32", dtype, 128)
    check(o2, lse, want, "f32", dtype, 128)


def test_attend_rows_of_requests():
    """Several rows of a request (causal), rows of no request, and lengths cut by max_len."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(41, [300, 77], 4, 2, 64, 32, "bf16")
    req = np.array([0, 0, 1, 1, 0, -1, 2, 7, 1, 0], np.int32)
    length = np.array([1, 299, 77, 40, 300, 50, 50, 3, 0, -5], np.int32)
    q = c.q(len(req))
    o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(length), row_req=_i32(req), want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, length, req), "f32", "bf16", 64)
    o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(length), row_req=_i32(req), want_lse=True, max_len=60)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, length, req, max_len=60), "f32", "bf16", 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attend_large_scores(dtype):
    """Scores up to about 300 either way, rising and falling along the keys, so that
    the reference moves late and far."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    n, D, P = 900, 64, 64
    c = Case(51, [n, n, n], 2, 1, D, P, dtype)
    ramp = np.zeros((3, 15 * P))
    ramp[0, :n] = np.linspace(-1, 1, n)
    ramp[1, :n] = np.linspace(1, -1, n)
    ramp[2, :n] = np.sin(np.arange(n) / 7.0)
    k = _f64(c.k)
    for b in range(3):
        for j in range(15):
            page, m = c.table[b, j], min(P, n - j * P)
            k[page, 0, :m] = 0.05 * k[page, 0, :m] + 6.0 * ramp[b, j * P:j * P + m, None]
    c.k = c.g(k)
    q = c.g(np.ones((3, 2, D)) * np.array([1.0, -1.0])[None, :, None] * 6.0)
    o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(c.lens), want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens), "f32", dtype, D)


def test_attend_lowest_and_infinite_values():
    """Values that a mask would use are ordinary numbers in the cache: the type's lowest key
    entry gives weight 0 beside others and the plain mean where all have it; an infinite
    score gives NaN, as the formula does, and only in its own row."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    for dtype in ("bf16", "f32"):
        c = Case(52, [40, 40, 40], 1, 1, 64, 16, dtype, spread=0.5)
        low = float(torch.finfo(_t(dtype)).min)
        c.k[c.table[0, 0], 0, 5] = low        # one key
        for j in range(3):
            c.k[c.table[1, j], 0, :min(16, 40 - 16 * j)] = low   # every key: equal scores
        c.k[c.table[2, 1], 0, 3, 0] = float("inf")
        q = torch.full((3, 1, 64), 2.0 ** -7, device="cuda").to(_t(dtype))
        o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(c.lens), scale=1.0, want_lse=True)
        torch.cuda.synchronize()
        k = _f64(c.k)
        keep = c.k[c.table[0, 0], 0, 5].clone()
        vals = np.concatenate([_f64(c.v[c.table[0, j], 0, :min(16, 40 - 16 * j)]) for j in range(3)])
        keys = np.concatenate([k[c.table[0, j], 0, :min(16, 40 - 16 * j)] for j in range(3)])
        x = keys @ np.full(64, 2.0 ** -7)
        w = np.exp(x - x.max())
        assert w[5] == 0.0 and torch.equal(keep, c.k[c.table[0, 0], 0, 5])
        assert np.allclose(_f64(o[0, 0]), w @ vals / w.sum(), rtol=0, atol=1e-4)
        mean = np.concatenate([_f64(c.v[c.table[1, j], 0, :min(16, 40 - 16 * j)]) for j in range(3)]).mean(0)
        assert np.allclose(_f64(o[1, 0]), mean, rtol=0, atol=1e-4)
        assert torch.isnan(o[2]).all()


def test_attend_strided_q_and_given_outputs():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(61, [1000, 33, 64], 4, 2, 128, 64, "bf16")
    fused = c.g(c.rng.standard_normal((3, 4 + 2 + 2, 128)))
    q = fused[:, :4]
    assert not q.is_contiguous()
    t, n = _i32(c.table), _i32(c.lens)
    o, lse = torch.full((3, 4, 128), 7.0, device="cuda"), torch.full((3, 4), 7.0, device="cuda")
    shape = ops._paged(3, 4, c.k.shape, c.k.dtype, o.dtype, 3, c.table.shape[1], None)
    ws = torch.empty(ops.paged_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    r, rl = ops.paged_attend(q, c.k, c.v, t, n, o=o, lse=lse, workspace=ws)
    assert r is o and rl is lse
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens), "f32", "bf16", 128)
    with pytest.raises(ops.SgdnError):
        ops.paged_attend(q, c.k, c.v, t, n, workspace=ws[:ws.numel() - 1])


def test_attend_page_numbers_that_are_none():
    """A damaged table: the keys of a page that does not exist take no part."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(62, [200, 150, 64], 4, 2, 64, 32, "bf16")
    c.table[0, 2], c.table[1, 0], c.table[1, 4] = -3, c.k.shape[0], 2 ** 31 - 1
    c.table[2] = -1
    q = c.q(3)
    o, lse = ops.paged_attend(q, c.k, c.v, _i32(c.table), _i32(c.lens), want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens), "f32", "bf16", 64)


def test_attend_far_pages():
    """A cache of more than 2^31 elements: offsets pass 32 bits."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    P, Hkv, D = 64, 4, 128
    n_pages = (2 ** 31 + 2 ** 26) // (P * Hkv * D)
    k = torch.empty((n_pages, Hkv, P, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = np.array([[n_pages - 1, 0, n_pages - 3], [2, n_pages - 2, 1]], np.int32)
    g = torch.Generator(device="cuda").manual_seed(3)
    slots = np.array([[table[b, t // P] * P + t % P for t in range(150)] for b in range(2)], np.int32)
    new_k, new_v = torch.randn((2, 300, Hkv, D), generator=g, device="cuda").bfloat16()
    codes = torch.zeros((n_pages, Hkv, D), dtype=torch.int8, device="cuda")
    scale = torch.zeros((n_pages, Hkv), device="cuda")
    ops.paged_write(new_k, new_v, _i32(slots.reshape(-1)), k, v, codes, scale)
    q = torch.randn((2, 8, D), generator=g, device="cuda").bfloat16()
    length = np.array([150, 149], np.int32)
    o, lse = ops.paged_attend(q, k, v, _i32(table), _i32(length), want_lse=True)
    lists = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda").expand(2, Hkv, 3).contiguous()
    o2, _ = ops.paged_attend_sparse(q, k, v, _i32(table), _i32(length), lists)
    torch.cuda.synchronize()
    near = np.arange(6, dtype=np.int32).reshape(2, 3)
    kk, vv = (t[torch.from_numpy(table.reshape(-1)).long().cuda()] for t in (k, v))
    want = ref.attend(_f64(q), np.nan_to_num(_f64(kk)), np.nan_to_num(_f64(vv)), near, length)
    check(o, lse, want, "f32", "bf16", D)
    check(o2, lse, want, "f32", "bf16", D)
    full = table[:, :2].reshape(-1)
    for p in full:
        for h in range(Hkv):
            cc, ss = ref.quantise(_f64(k[int(p), h]).mean(0))
            assert np.array_equal(codes[int(p), h].cpu().numpy(), cc) and float(scale[int(p), h]) == ss


# attend_sparse --------------------------------------------------------------


def _lists(rng, rows, Hkv, K, nb):
    out = np.full((rows, Hkv, K), -1, np.int32)
    for r in range(rows):
        for h in range(Hkv):
            m = min(K, int(nb[r]))
            out[r, h, :m] = np.sort(rng.permutation(int(nb[r]))[:m])
    return out


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("Hq, Hkv, D, P", SHAPES)
def test_attend_sparse(Hq, Hkv, D, P, dtype, out):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(Hq + D + P + 1, LENS, Hq, Hkv, D, P, dtype)
    q = c.q(len(LENS))
    lists = _lists(c.rng, len(LENS), Hkv, 5, -(-c.lens // P))
    o, lse = ops.paged_attend_sparse(q, c.k, c.v, _i32(c.table), _i32(c.lens), _i32(lists),
                                     out_dtype=_t(out), want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens, blocks=lists), out, dtype, D)


def test_attend_sparse_odd_lists():
    """Any order, holes, blocks beyond the row, one listed twice, none at all, one entry."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(71, [500, 500, 130], 4, 2, 128, 32, "bf16")
    lists = np.full((3, 2, 9), -1, np.int32)
    lists[0, 0] = [15, -1, 3, 0, -1, 16, 2 ** 31 - 1, 7, -2 ** 31]
    lists[0, 1] = [4, 4, 4, -1, -1, 1, 4, -1, 1]
    lists[1, 1, 8] = 15
    lists[2, 0] = [4, 5, 6, 7, 3, 8, 9, 10, 4]
    q = c.q(3)
    for L in (lists, lists[:, :, 8:].copy()):
        o, lse = ops.paged_attend_sparse(q, c.k, c.v, _i32(c.table), _i32(c.lens), _i32(L), want_lse=True)
        torch.cuda.synchronize()
        check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, c.lens, blocks=L), "f32", "bf16", 128)


@pytest.mark.parametrize("rows, Hq, Hkv, K", [(700, 4, 1, 6), (150, 16, 2, 3), (37, 20, 1, 4)])
def test_attend_sparse_many_rows(rows, Hq, Hkv, K):
    """Every token of two requests (more units than are split), and padding rows behind them."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    lens = np.array([rows - rows // 3 + 90, rows // 3 + 40])
    c = Case(rows, lens, Hq, Hkv, 64, 16, "bf16")
    n = [rows - rows // 3, rows // 3]
    req = np.r_[np.zeros(n[0]), np.ones(n[1]), -np.ones(5)].astype(np.int32)
    length = np.r_[lens[0] - n[0] + 1 + np.arange(n[0]), lens[1] - n[1] + 1 + np.arange(n[1]), np.zeros(5)].astype(np.int32)
    lists = _lists(c.rng, rows + 5, Hkv, K, -(-length // 16))
    q = c.q(rows + 5)
    o, lse = ops.paged_attend_sparse(q, c.k, c.v, _i32(c.table), _i32(length), _i32(lists), row_req=_i32(req),
                                     out_dtype=_t("bf16"), want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, length, req, blocks=lists), "bf16", "bf16", 64)


# select ---------------------------------------------------------------------


def _summaries(rng, n_pages, Hkv, D, coarse=False):
    import torch
    if coarse:                                   # few values: many equal scores
        codes = rng.integers(-1, 2, (n_pages, Hkv, D)).astype(np.int8)
        scale = 2.0 ** rng.integers(-1, 1, (n_pages, Hkv))
    else:
        codes = rng.integers(-127, 128, (n_pages, Hkv, D)).astype(np.int8)
        scale = 2.0 ** rng.integers(-9, -5, (n_pages, Hkv))
    scale = scale.astype(np.float32)
    return codes, scale, torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq, Hkv, D, G_note", [(4, 4, 64, 1), (6, 3, 128, 2), (9, 3, 64, 3), (8, 2, 256, 4), (6, 1, 128, 6),
                                                (16, 2, 128, 8), (16, 1, 64, 16), (20, 1, 128, 20), (40, 1, 64, 40)])
@pytest.mark.parametrize("coarse", [False, True])
def test_select(Hq, Hkv, D, G_note, dtype, coarse):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(Hq + D)
    P, B, W = 16, 5, 90
    codes, scale, dc, ds = _summaries(rng, B * W, Hkv, D, coarse)
    table = rng.permutation(B * W).reshape(B, W).astype(np.int32)
    table[1, 7], table[2, 3] = -1, B * W
    q = torch.from_numpy(rng.integers(-2, 3, (B, Hq, D)) if coarse else rng.standard_normal((B, Hq, D))).cuda().to(_t(dtype))
    length = np.array([0, 1400, 1, 333, 16 * 90], np.int32)
    for K, sink, local in ((4, 1, 1), (17, 0, 3), (90, 2, 2), (100, 1, 1)):
        got = ops.paged_select(q, dc, ds, _i32(table), _i32(length), P, K, n_sink=sink, n_local=local)
        torch.cuda.synchronize()
        want = ref.select(_f64(q), codes, scale, table, length, P, K, n_sink=sink, n_local=local)
        assert np.array_equal(got.cpu().numpy(), want), (K, sink, local)


@pytest.mark.parametrize("W", [64, 65, 256, 257, 1024, 1025, 2048, 2049, 4096, 4097, 16384])
def test_select_widths(W):
    """Every size class of the choice, at its borders."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(W)
    B, Hkv, D, P = 2, 1, 64, 16
    codes, scale, dc, ds = _summaries(rng, W + 3, Hkv, D, coarse=W % 2 == 1)
    table = np.stack([rng.permutation(W + 3)[:W] for _ in range(B)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((B, 2, D))).cuda().bfloat16()
    length = np.array([W * P, W * P - 5], np.int32)
    for K in (2, 33):
        got = ops.paged_select(q, dc, ds, _i32(table), _i32(length), P, K)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), ref.select(_f64(q), codes, scale, table, length, P, K))


@pytest.mark.parametrize("Hq, Hkv", [(2, 2), (4, 2), (8, 2), (16, 2), (16, 1), (6, 2), (24, 1)])
def test_select_rows_of_requests(Hq, Hkv):
    """Packed rows of several requests (tiles of rows that span them), rows of none, and a
    request that comes twice in a tile."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(Hq)
    P, W, B, D = 16, 40, 4, 64
    codes, scale, dc, ds = _summaries(rng, B * W, Hkv, D)
    table = rng.permutation(B * W).reshape(B, W).astype(np.int32)
    req = np.r_[[0] * 7, [1], [2] * 30, [-1], [1] * 5, [3, 0, 3, 9, 3], [-1] * 3].astype(np.int32)
    length = rng.integers(1, W * P + 1, len(req)).astype(np.int32)
    length[-3:], length[4] = 0, -1
    q = torch.from_numpy(rng.standard_normal((len(req), Hq, D))).cuda().bfloat16()
    for max_len in (None, 300):
        got = ops.paged_select(q, dc, ds, _i32(table), _i32(length), P, 6, row_req=_i32(req), max_len=max_len)
        torch.cuda.synchronize()
        want = ref.select(_f64(q), codes, scale, table, length, P, 6, req=req, max_len=max_len)
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq, Hkv, D", [(2, 2, 64), (4, 2, 256), (8, 2, 128), (6, 2, 64), (16, 2, 128), (16, 1, 256), (24, 1, 128)])
def test_select_many_rows_of_requests(Hq, Hkv, D, dtype):
    """So many rows that those of a request share its pages, across the borders of requests."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(Hq + D)
    P, W, B = 16, 21, 6
    codes, scale, dc, ds = _summaries(rng, B * W, Hkv, D)
    table = rng.permutation(B * W).reshape(B, W).astype(np.int32)
    table[2, 5], table[3, 2] = -1, B * W
    n = (1 << 17) // (Hkv * D) + 60
    req = np.r_[[5] * 7, [1] * (n // 3), [3, 0, 3, 9, 3], [-1], [2] * (n - n // 3), [4] * 2, [-1] * 3].astype(np.int32)
    length = rng.integers(1, W * P + 1, len(req)).astype(np.int32)
    length[-3:], length[40:42] = 0, (-1, 0)
    q = torch.from_numpy(rng.standard_normal((len(req), Hq, D))).cuda().to(_t(dtype))
    for K, max_len in ((6, None), (16, 300)):
        got = ops.paged_select(q, dc, ds, _i32(table), _i32(length), P, K, row_req=_i32(req), max_len=max_len)
        torch.cuda.synchronize()
        want = ref.select(_f64(q), codes, scale, table, length, P, K, req=req, max_len=max_len)
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("Hq, Hkv, D", [(2, 2, 128), (8, 2, 64), (16, 2, 256), (16, 1, 128)])
def test_select_prompt_and_single_rows(Hq, Hkv, D):
    """A prompt between new tokens of other requests, more of them than a workgroup takes one by one."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(D)
    P, W, B = 16, 37, 60
    codes, scale, dc, ds = _summaries(rng, B * W, Hkv, D)
    table = rng.permutation(B * W).reshape(B, W).astype(np.int32)
    n = (1 << 17) // (Hkv * D) + 2 * B * B
    req = np.r_[np.arange(1, 30), np.zeros(n), np.arange(30, B), -1].astype(np.int32)
    length = rng.integers(1, W * P + 1, len(req)).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((len(req), Hq, D))).cuda().bfloat16()
    got = ops.paged_select(q, dc, ds, _i32(table), _i32(length), P, 8, row_req=_i32(req))
    torch.cuda.synchronize()
    rows = np.r_[np.arange(0, 64), rng.integers(64, n, 200), np.arange(len(req) - 64, len(req))]
    want = ref.select(_f64(q[rows]), codes, scale, table, length[rows], P, 8, req=req[rows])
    assert np.array_equal(got.cpu().numpy()[rows], want)


def test_select_values_that_are_not_finite():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(8)
    codes, scale, dc, ds = _summaries(rng, 30, 1, 64)
    scale[3], scale[9] = np.nan, np.nan
    ds = torch.from_numpy(scale).cuda()
    q = rng.standard_normal((2, 2, 64))
    q[0, 0, :5] = [np.nan, np.inf, -np.inf, 3.0, 1e-30]
    q[1] = np.nan
    q = torch.from_numpy(q).cuda().float()
    table = np.tile(np.arange(30, dtype=np.int32), (2, 1))
    length = np.array([480, 470], np.int32)
    for K in (5, 29):
        got = ops.paged_select(q, dc, ds, _i32(table), _i32(length), 16, K)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), ref.select(_f64(q), codes, scale, table, length, 16, K))


# write ----------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hkv, D, P", [(1, 64, 16), (2, 128, 64), (3, 256, 32), (8, 128, 128), (5, 64, 64)])
def test_write(Hkv, D, P, dtype):
    """Pages begun in earlier calls, completed, several in one call, rows without a slot; all
    else stays."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(P + D + Hkv)
    n_pages = 12
    g = lambda x: torch.from_numpy(x).cuda().to(_t(dtype))
    k_cache, v_cache = (g(rng.standard_normal((n_pages, Hkv, P, D))) for _ in range(2))
    codes = torch.full((n_pages, Hkv, D), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((n_pages, Hkv), 7.0, device="cuda")
    want = [x.float().cpu().numpy() for x in (k_cache, v_cache)] + [codes.cpu().numpy(), scale.cpu().numpy()]
    page = rng.permutation(n_pages)
    run = lambda b, lo, hi: [int(page[b + t // P]) * P + t % P for t in range(lo, hi)]
    calls = [
        run(0, 0, P // 2) + run(4, 0, 2 * P + 3) + [-1, n_pages * P, 2 ** 31 - 1],
        run(0, P // 2, P),                       # completes a page begun before
        run(0, P, P + 1),                        # one row that completes nothing
        run(4, 2 * P + 3, 3 * P - 1) + run(0, P + 1, 2 * P),
        run(4, 3 * P - 1, 3 * P),                # one row that completes a page
        [-5] * 3 + run(8, 0, 4 * P),
    ]
    for slots in calls:
        n = len(slots)
        k, v = (g(rng.standard_normal((n, Hkv, D)) * 2.0 ** rng.integers(-3, 3, (n, 1, 1))) for _ in range(2))
        ops.paged_write(k, v, _i32(slots), k_cache, v_cache, codes, scale)
        torch.cuda.synchronize()
        ref.write(k.float().cpu().numpy(), v.float().cpu().numpy(), slots, *want)
        for got, w in zip((k_cache, v_cache, codes, scale), want):
            assert np.array_equal(got.float().cpu().numpy(), w.astype(np.float32))


def test_write_summary_borders():
    """Means that are 0, tiny, huge, exactly half way, and not finite."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    P, D = 16, 64
    k = np.zeros((6 * P, 1, D), np.float32)
    k[P:2 * P, 0, 0] = 2.0 ** -126
    k[2 * P:3 * P, 0, :3] = [3.0e38, -3.0e38, 1.0e38]
    k[3 * P:4 * P, 0, :6] = [64.0, 0.5, 1.5, 2.5, -0.5, 127.5]
    k[4 * P:5 * P, 0, :4] = [np.inf, 1.0, -3.0, np.nan]
    k[5 * P, 0, 0], k[5 * P + 1, 0, 0], k[5 * P + 2, 0, 1] = 1e30, -1e30, 1.0   # cancels in 64 bits
    k_cache, v_cache = torch.zeros((2, 6, 1, P, D), device="cuda")
    codes, scale = torch.zeros((6, 1, D), dtype=torch.int8, device="cuda"), torch.zeros((6, 1), device="cuda")
    kk = torch.from_numpy(k).cuda()
    ops.paged_write(kk, kk, _i32(np.arange(6 * P)), k_cache, v_cache, codes, scale)
    torch.cuda.synchronize()
    for p in range(6):
        with np.errstate(invalid="ignore"):
            c, s = ref.quantise(k[p * P:(p + 1) * P, 0].astype(np.float64).sum(0) / P)
        assert float(scale[p, 0]) == s and np.array_equal(codes[p, 0].cpu().numpy(), c), p


def test_write_views_without_summaries():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(9)
    fused = torch.from_numpy(rng.standard_normal((40, 8 + 2 + 2, 128))).cuda().bfloat16()
    k, v = fused[:, 8:10], fused[:, 10:]
    k_cache, v_cache = torch.zeros((2, 2, 2, 32, 128), dtype=torch.bfloat16, device="cuda")
    ops.paged_write(k, v, _i32(np.arange(40) + 5), k_cache, v_cache)
    torch.cuda.synchronize()
    for cache, x in ((k_cache, k), (v_cache, v)):
        flat = cache.transpose(1, 2).reshape(64, 2, 128)
        assert torch.equal(flat[5:45], x) and not flat[:5].any() and not flat[45:].any()
    with pytest.raises(ValueError, match="contiguous"):
        ops.paged_write(fused[:, 8:12:2], v, _i32(np.arange(40)), k_cache, v_cache)


# plan and release -----------------------------------------------------------


def _plan_state(rng, B, W, P, n_pages, cached):
    lens = np.minimum(cached, W * P).astype(np.int32)
    blocks = -(-lens // P)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = ids[at:at + blocks[b]]
        at += blocks[b]
    taken = int(rng.integers(0, 5 * n_pages))
    ring = np.full(n_pages, -9, np.int32)
    ring[(taken + np.arange(n_pages - at)) % n_pages] = ids[at:]
    return lens, table, ring, np.array([taken, taken + n_pages - at], np.int64)


def _compare_plan(got, want, table):
    for n in ("lens", "cu", "page_cu", "slot", "row_req", "row_len", "status", "free_pos"):
        assert np.array_equal(got[n].cpu().numpy(), want[n]), n
    assert np.array_equal(table.cpu().numpy(), want["table"])


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B, W, P, most, rows, pages", [
    (1, 4, 16, 1, 1, 40), (7, 6, 16, 40, 300, 60), (128, 8, 64, 1, 130, 1100), (300, 3, 32, 9, 2000, 1000),
    (1024, 4, 16, 3, 4096, 5000), (1025, 4, 16, 3, 4096, 5000), (2500, 2, 16, 8, 9000, 5100),
    (20, 40, 128, 3000, 30000, 900), (40, 6, 16, 60, 500, 90), (64, 4, 16, 30, 0, 300)])
def test_plan(B, W, P, most, rows, pages, inplace):
    """Room for all, too few pages, too few rows, tables too narrow, negative numbers."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(B + rows)
    cached = rng.integers(0, max(1, min(W * P, (pages - 4) * P // B)), B)
    lens, table, ring, pos = _plan_state(rng, B, W, P, pages, cached)
    add = rng.integers(0, most + 1, B).astype(np.int32)
    if B > 5:
        add[3], lens[4] = -1, -8
    want = ref.plan(lens, add, table, ring, pos, P, rows)
    d = [torch.from_numpy(x).cuda() for x in (lens, add, table, ring, pos)]
    kw = dict(lens_out=d[0], free_pos_out=d[4]) if inplace else {}
    got = ops.paged_plan(*d, P, rows, **kw)
    torch.cuda.synchronize()
    _compare_plan(got, want, d[2])
    if not inplace:                              # nothing else was touched; again gives the same
        assert np.array_equal(d[0].cpu().numpy(), lens) and np.array_equal(d[4].cpu().numpy(), pos)
        again = ops.paged_plan(*d, P, rows, out=got)
        torch.cuda.synchronize()
        _compare_plan(again, want, d[2])


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B, W, P, pages", [(1, 3, 16, 9), (40, 300, 16, 5000), (1500, 3, 64, 5000), (2, 5000, 16, 9000)])
def test_release(B, W, P, pages, inplace):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(B + W)
    lens, table, ring, pos = _plan_state(rng, B, W, P, pages, rng.integers(0, pages * P // B - 15, B))
    done = (rng.random(B) < 0.5).astype(np.uint8)
    done[0] = 3
    if B > 9:
        lens[7], done[7] = -4, 1
    want = ref.release(lens, done, table, ring, pos, P)
    d = [torch.from_numpy(x).cuda() for x in (lens, done, table, ring, pos)]
    kw = dict(lens_out=d[0], free_pos_out=d[4]) if inplace else {}
    n, p = ops.paged_release(*d, P, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(n.cpu().numpy(), want[0]) and np.array_equal(d[3].cpu().numpy(), want[1])
    assert np.array_equal(p.cpu().numpy(), want[2]) and np.array_equal(d[2].cpu().numpy(), table)


def test_binding_refusals():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(81, [20, 30], 4, 2, 64, 16, "bf16")
    t, n, q = _i32(c.table), _i32(c.lens), c.q(2)
    lists = torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda")
    call = lambda **kw: ops.paged_attend(**{**dict(q=q, k_cache=c.k, v_cache=c.v, table=t, row_len=n), **kw})
    for kw in (dict(q=q.float()), dict(q=q[:, :, ::2]), dict(q=q[:, :3]), dict(v_cache=c.v.float()), dict(v_cache=c.v[:-1]),
               dict(k_cache=c.k.transpose(2, 3)), dict(table=t.long()), dict(row_len=n[:1]), dict(row_len=n.cpu()),
               dict(row_req=n[:1]), dict(o=torch.empty((2, 4, 32), device="cuda")), dict(table=t[:1]),
               dict(lse=torch.empty((2, 3), device="cuda")), dict(max_len=10 ** 6), dict(scale=float("nan")),
               dict(out_dtype=torch.float64)):
        with pytest.raises((ValueError, ops.SgdnError)):
            call(**kw)
    for bad in (lists.long(), lists[:1], lists[:, :1], lists[:, :, :0], None):
        with pytest.raises((ValueError, ops.SgdnError)):
            ops.paged_attend_sparse(q, c.k, c.v, t, n, bad)
    codes, scale = torch.zeros((len(c.k), 2, 64), dtype=torch.int8, device="cuda"), torch.ones((len(c.k), 2), device="cuda")
    sel = lambda **kw: ops.paged_select(**{**dict(q=q, codes=codes, code_scale=scale, table=t, row_len=n, page=16, n_blocks=3), **kw})
    for kw in (dict(page=48), dict(n_blocks=1), dict(n_local=0), dict(codes=codes.int()), dict(code_scale=scale[:, :1]),
               dict(q=q[:, :3]), dict(blocks=lists[:, :, :2])):
        with pytest.raises((ValueError, ops.SgdnError)):
            sel(**kw)
    assert sel().shape == (2, 2, 3)
    with pytest.raises(ops.SgdnError):
        ops.paged_write(q[:, :2], q[:, 2:], n, c.k, c.v, codes)       # codes without their scale
    ops.paged_attend(q[:0], c.k, c.v, t, n[:0])                       # nothing to do
    torch.cuda.synchronize()


def test_max_len_as_given():
    """An upper bound that is a tensor counts with its value at the call; 0 is none."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = Case(83, [20, 60], 4, 2, 64, 16, "f32")
    t, n, q = _i32(c.table), _i32(c.lens), c.q(2)
    codes, _, dc, ds = _summaries(c.rng, len(c.k), 2, 64)
    most = torch.tensor(60)
    for m in (60, 33, 1):
        most.fill_(m)
        o, lse = ops.paged_attend(q, c.k, c.v, t, n, max_len=most, want_lse=True)
        got = ops.paged_select(q, dc, ds, t, n, torch.tensor(16), 2, max_len=most)
        torch.cuda.synchronize()
        want = ref.attend(_f64(q), _f64(c.k), _f64(c.v), c.table, np.minimum(c.lens, m), np.arange(2))
        check(o, lse, want, "f32", "f32", 64)
        assert np.array_equal(got.cpu().numpy(), ref.select(_f64(q), codes, _f64(ds).astype(np.float32), c.table, c.lens, 16, 2, max_len=m))
    for m in (0, -5, 61.0):
        with pytest.raises((ValueError, TypeError)):
            ops.paged_attend(q, c.k, c.v, t, n, max_len=m)


# attend_sparse of prompts ----------------------------------------------------


def _prompt(seed, Hq, Hkv, D, P, dtype, K, lens, new, nan=None, pad=3, alike=8):
    """Every new token of the given requests as a row; lists that `alike` rows in a row mostly share."""
    c = Case(seed, lens, Hq, Hkv, D, P, dtype)
    req = np.r_[np.repeat(np.arange(len(lens)), new), -np.ones(pad)].astype(np.int32)
    length = np.r_[np.concatenate([n - m + 1 + np.arange(m) for n, m in zip(lens, new)]), np.zeros(pad)].astype(np.int32)
    R = len(req)
    nb = -(-length // P)
    lists = np.full((R, Hkv, K), -1, np.int32)
    for r in range(R):
        rng = np.random.default_rng([seed, r // alike])
        for h in range(Hkv):
            order = rng.permutation(max(int(nb.max()), 1))
            pick = [j for j in order if j < nb[r]][:K - 1]
            if nb[r] > 0 and c.rng.random() < 0.3 and pick:
                pick[c.rng.integers(len(pick))] = int(nb[r]) - 1
            if nb[r] > 0:
                pick.append(int(nb[r]) - 1)
            lists[r, h, :len(pick)] = sorted(pick) if K % 2 else pick   # a block may come twice
    return c, req, length, lists, c.q(R)


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("Hq, Hkv, D, P, K", [
    (8, 1, 64, 16, 5), (8, 1, 128, 64, 3), (8, 1, 256, 32, 4), (16, 1, 64, 32, 6), (12, 1, 128, 16, 7),
    (5, 1, 64, 64, 3), (2, 2, 64, 16, 9), (3, 1, 128, 128, 2), (2, 1, 64, 16, 4), (1, 1, 64, 32, 5)])
def test_attend_sparse_prompts(Hq, Hkv, D, P, K, dtype, out):
    """Tiles of rows that share lists: within a request, across a border, with padding rows behind."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    G = Hq // Hkv
    gp = 1 << (G - 1).bit_length()
    R = 256 * (128 // gp) // Hkv + 50              # as many tiles as it takes
    new = [R - R // 3, R // 3 - 1, 1]
    lens = np.array(new) + [70, 3, 200]
    c, req, length, lists, q = _prompt(Hq + D + P, Hq, Hkv, D, P, dtype, K, lens, new, alike=16)
    t = [_i32(x) for x in (c.table, length, lists, req)]
    ws = torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda")
    o, lse = ops.paged_attend_sparse(q, c.k, c.v, t[0], t[1], t[2], row_req=t[3], out_dtype=_t(out), want_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert (ws.view(torch.int32) == 1).sum() >= 40, "tiles, and not single rows alone"
    rows = np.unique(np.r_[np.arange(0, 40), c.rng.integers(0, len(req), 60), new[0] - 20 + np.arange(40), len(req) - 30 + np.arange(30)])
    want = ref.attend(_f64(q[rows]), _f64(c.k), _f64(c.v), c.table, length[rows], req[rows], blocks=lists[rows])
    i = torch.from_numpy(rows).cuda()
    check(o[i], lse[i], want, out, dtype, D)


def test_far_pages_of_prompts():
    """Tiles and the choice of blocks where offsets into the cache and the summaries pass 32 bits."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    P, Hkv, D, R = 64, 4, 128, 900
    n_pages = (2 ** 31 + 2 ** 26) // (P * Hkv * D)
    k = torch.empty((n_pages, Hkv, P, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(4)
    table = np.array([[n_pages - 1, 0, n_pages - 3, 2, n_pages - 2, 1] + list(range(n_pages - 20, n_pages - 8))], np.int32)
    for p in table[0]:
        k[int(p)], v[int(p)] = torch.randn((2, Hkv, P, D), generator=g, device="cuda").bfloat16()
    q = torch.randn((R, 8, D), generator=g, device="cuda").bfloat16()
    length = 200 + np.arange(R, dtype=np.int32)
    lists = np.broadcast_to(np.array([0, 2, 3], np.int32), (R, Hkv, 3)).copy()
    ws = torch.zeros(1 << 12, dtype=torch.uint8, device="cuda")
    o, lse = ops.paged_attend_sparse(q, k, v, _i32(table), _i32(length), _i32(lists), row_req=_i32(np.zeros(R)), want_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert (ws.view(torch.int32) == 1).sum() >= 40
    rows = np.r_[np.arange(0, R, 37), R - 1]
    i = torch.from_numpy(rows).cuda()
    at = torch.from_numpy(table[0]).long().cuda()
    near = np.arange(table.shape[1], dtype=np.int32)[None]
    want = ref.attend(_f64(q[i]), _f64(k[at]), _f64(v[at]), near, length[rows], np.zeros(len(rows), int), blocks=lists[rows])
    check(o[i], lse[i], want, "f32", "bf16", D)
    del k, v
    n_pages = (2 ** 31 + 2 ** 27) // (Hkv * D)             # summaries are a P-th of the keys
    codes = torch.zeros((n_pages, Hkv, D), dtype=torch.int8, device="cuda")
    scale = torch.ones((n_pages, Hkv), device="cuda")
    table = np.array([[n_pages - 1, 0, n_pages - 3, 2, n_pages - 2, 1] + list(range(n_pages - 20, n_pages - 8))], np.int32)
    at = torch.from_numpy(table[0]).long().cuda()
    codes[at] = torch.randint(-127, 128, (table.shape[1], Hkv, D), generator=g, device="cuda").to(torch.int8)
    for n in (R, 3):                                       # rows that share pages, single rows
        got = ops.paged_select(q[:n], codes, scale, _i32(table), _i32(length[:n]), P, 4, row_req=_i32(np.zeros(n)))
        torch.cuda.synchronize()
        pick = rows[rows < n]
        want = ref.select(_f64(q)[pick], codes[at].cpu().numpy(), scale[at].cpu().numpy(), near, length[pick], P, 4, req=np.zeros(len(pick), int))
        assert np.array_equal(got.cpu().numpy()[pick], want)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3, 3.0])
def test_attend_scale(scale):
    """Scales of either sign and 0, for single rows and for tiles of rows."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    R = 256 * 16 + 9
    c, req, length, lists, q = _prompt(9, 8, 1, 64, 32, "bf16", 3, np.array([R + 60]), [R], pad=0, alike=16)
    t = [_i32(x) for x in (c.table, length, lists, req)]
    rows = np.arange(0, R, 57)
    i = torch.from_numpy(rows).cuda()
    for n in (R, 40):
        o, lse = ops.paged_attend_sparse(q[-n:], c.k, c.v, t[0], t[1][-n:], t[2][-n:], row_req=t[3][-n:], scale=scale, want_lse=True)
        torch.cuda.synchronize()
        pick = rows[rows >= R - n]
        j = torch.from_numpy(pick - (R - n)).cuda()
        want = ref.attend(_f64(q[torch.from_numpy(pick).cuda()]), _f64(c.k), _f64(c.v), c.table, length[pick], req[pick], scale, lists[pick])
        check(o[j], lse[j], want, "f32", "bf16", 64)


@pytest.mark.parametrize("alike", [1, 16])
def test_attend_sparse_prompts_see_only_their_own(alike):
    """A row's result does not change with what other rows of its tile list or see: values
    that are not finite in their blocks, in later tokens, or an infinite score of one."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    R = 256 * 16 + 9
    c, req, length, lists, q = _prompt(5, 8, 1, 64, 16, "bf16", 4, np.array([R + 60]), [R], pad=0, alike=alike)
    t = [_i32(x) for x in (c.table, length, lists, req)]
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    call = lambda: ops.paged_attend_sparse(q, c.k, c.v, t[0], t[1], t[2], row_req=t[3], want_lse=True, workspace=ws)
    o, lse = call()
    assert ((ws.view(torch.int32) == 1).sum() >= 100) == (alike > 1)     # tiles, or single rows alone
    bad = c.table[0, [3, 40, 100]]
    c.v[bad[0], 0, 5, 7], c.v[bad[1], 0, 2] = float("nan"), float("inf")
    c.k[bad[2], 0, 9, 3] = float("inf")
    o2, lse2 = call()
    torch.cuda.synchronize()
    hit, spoilt = np.zeros(R, bool), np.zeros(R, bool)
    above = (_f64(q)[:, :, 3] > 0).any(-1)       # else the infinite key's scores are -inf, which weigh 0
    for j, place in ((3, 5), (40, 2), (100, 9)):
        one = (lists[:, 0] == j).any(-1) & (length > 16 * j + place)
        hit |= one
        spoilt |= one & (above if j == 100 else True)
    assert 0 < hit.sum() < R
    clean = torch.from_numpy(~hit).cuda()
    # the kernel for single rows sums in another order than the tiles: equal within both bounds
    rows = np.flatnonzero(~hit)[::41]
    want = ref.attend(_f64(q[rows]), np.nan_to_num(_f64(c.k)), np.nan_to_num(_f64(c.v)), c.table, length[rows], req[rows], blocks=lists[rows])
    i = torch.from_numpy(rows).cuda()
    check(o2[i], lse2[i], want, "f32", "bf16", 64)
    check(o[i], lse[i], want, "f32", "bf16", 64)
    assert torch.isfinite(o2[clean]).all() and torch.isfinite(o).all()
    assert not torch.isfinite(o2[torch.from_numpy(spoilt).cuda()].reshape(int(spoilt.sum()), -1)).all(-1).any()
