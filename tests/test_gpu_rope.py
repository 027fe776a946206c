"""GPU parity of rotary positions and head norms against the fp64 oracle.

Tolerance, with u = 2^-24, half a step of fp32: an element is a c - b s of its pair.
  angle     r = t - n pi/2 in fp64, to fp32: u/2 (r < 1);  c and s of it: 2 u for their
            polynomials' roundings, 2^-28 for what the series drop
  products  magnitude to fp32 and times it: 2 u;  product and sum: 2 u
together under 7 u of (|a| + |b|) magnitude, so 2^-21 of that.  A norm adds the sum's
conversion, square root, quotient, two products and the weight's sum: 6 u of |a| and |b|,
together under 2^-20.  Then u(type) of the value for the output's rounding, and half the
smallest step (2^-25) in fp16 and half of 2^-133 in bf16 where values lie below the normals.
"""
import numpy as np
import pytest

from oracle import serve as ref

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def _t(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _f64(t):
    return t.double().cpu().numpy()


def check(y, want, size, dtype, norm):
    tol = (2.0 ** -20 if norm else 2.0 ** -21) * size + U[dtype] * np.abs(want) + TINY[dtype]
    err = np.abs(_f64(y) - want)
    assert np.isfinite(_f64(y)).all()
    worst = float((err / tol).max()) if err.size else 0.0
    print(f"err / bound {worst:.3f}")
    assert worst <= 1.0


def _case(seed, R, Hq, Hk, D, rot, dtype, gated=False, far=10 ** 6):
    """One projection's output with q, k, v (with a gate beside each query head if `gated`), and the places."""
    import torch
    rng = np.random.default_rng(seed)
    wide = 2 if gated else 1
    fused = torch.from_numpy(rng.standard_normal((R, wide * Hq + 2 * Hk, D))).cuda().to(_t(dtype))
    q = fused[:, :wide * Hq].unflatten(1, (Hq, wide))[:, :, 0]
    k = fused[:, wide * Hq:wide * Hq + Hk]
    pos = rng.integers(0, far, R).astype(np.int32)
    return fused, q, k, pos, rng


SHAPES = [  # R, Hq, Hk, D, rot
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (37, 16, 2, 256, 64), (5, 7, 1, 80, 40), (130, 15, 3, 64, 20), (3, 2, 2, 8, 2),
    (9, 3, 5, 72, 72), (11, 4, 4, 96, 0), (64, 5, 1, 256, 256), (2, 40, 8, 128, 130 - 4), (4100, 2, 1, 32, 16), (6, 1, 0, 16, 10),
]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R, Hq, Hk, D, rot", SHAPES)
def test_rope(R, Hq, Hk, D, rot, dtype, layout):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    _, q, k, pos, rng = _case(R + D, R, Hq, Hk, D, rot, dtype, gated=R % 2 == 1)
    f, m = (ops.rope_freqs(rot, scaling="by_pair", factor=8, original=4096) if rot else (torch.zeros(0, dtype=torch.float64), 1.5))
    yq, yk = ops.rope(q, k if Hk else None, torch.from_numpy(pos).cuda(), f.cuda(), layout=layout, magnitude=m)
    check(yq, *ref.rope(_f64(q), pos, f.numpy(), layout, m), dtype, False)
    if Hk:
        check(yk, *ref.rope(_f64(k), pos, f.numpy(), layout, m), dtype, False)
    else:
        assert yk is None
    if rot == 0:
        assert torch.equal(yq, q)
    if rot < D:
        assert torch.equal(yq[..., rot:], q[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype, w_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("R, Hq, Hk, D, rot", SHAPES)
def test_norm_rope(R, Hq, Hk, D, rot, dtype, w_dtype, layout):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    _, q, k, pos, rng = _case(R + D + 1, R, Hq, Hk, D, rot, dtype, gated=R % 2 == 1)
    wq, wk = (torch.from_numpy(rng.standard_normal(D) * 0.2).cuda().to(_t(w_dtype)) for _ in range(2))
    f = ops.rope_freqs(rot, 5e5)[0] if rot else torch.zeros(0, dtype=torch.float64)
    eps = 1e-5
    yq, yk = ops.norm_rope(q, k if Hk else None, wq, wk if Hk else None, torch.from_numpy(pos).cuda(), f.cuda(), layout=layout,
                           weight_offset=1.0, eps=eps)
    e = float(np.float32(eps))
    check(yq, *ref.rope(ref.norm(_f64(q), _f64(wq), 1.0, e), pos, f.numpy(), layout, 1.0), dtype, True)
    if Hk:
        check(yk, *ref.rope(ref.norm(_f64(k), _f64(wk), 1.0, e), pos, f.numpy(), layout, 1.0), dtype, True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_places(layout):
    """Up to the last place that 32 bits hold, and past it by the offset."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    _, q, k, _, _ = _case(5, 6, 4, 2, 128, 128, "f32")
    pos = np.array([2 ** 31 - 1, 2 ** 31 - 2, 10 ** 9 + 7, 0, 1, 2 ** 24 + 1], np.int32)
    f, _ = ops.rope_freqs(128)
    for offset in (0, 2 ** 31 - 1):
        yq, yk = ops.rope(q, k, torch.from_numpy(pos).cuda(), f.cuda(), layout=layout, pos_offset=offset)
        place = pos.astype(np.int64) + offset
        check(yq, *ref.rope(_f64(q), place, f.numpy(), layout, 1.0), "f32", False)
        check(yk, *ref.rope(_f64(k), place, f.numpy(), layout, 1.0), "f32", False)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("layout, rot", [("half", 64), ("half", 20), ("interleaved", 64)])
def test_in_place_rows_left_out_and_nothing_else_written(norm, layout, rot):
    """q and k turned where they lie; rows in front of place 0 and all that is not q or k stay, NaN included."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    fused, q, k, _, rng = _case(8, 200, 6, 2, 64, rot, "bf16", gated=True)
    length = rng.integers(-1, 40, 200).astype(np.int32)
    left = torch.from_numpy(length <= 0).cuda()
    fused[left] = float("nan")
    before, q0, k0 = fused.clone(), q.clone(), k.clone()
    f, _ = ops.rope_freqs(rot)
    pos, fd = torch.from_numpy(length).cuda(), f.cuda()
    call = (lambda *a, **kw: ops.norm_rope(a[0], a[1], None, None, *a[2:], weight_offset=1.0, **kw)) if norm else ops.rope
    yq, yk = call(q, k, pos, fd, layout=layout, pos_offset=-1, q_out=q, k_out=k)
    assert yq is q and yk is k
    live = length > 0
    n = (lambda x: ref.norm(x, None, 1.0, float(np.float32(1e-6)))) if norm else (lambda x: x)
    check(q[~left], *ref.rope(n(_f64(q0)[live]), length[live] - 1, f.numpy(), layout, 1.0), "bf16", norm)
    check(k[~left], *ref.rope(n(_f64(k0)[live]), length[live] - 1, f.numpy(), layout, 1.0), "bf16", norm)
    assert torch.isnan(fused[left]).all()
    rest = fused.clone()
    rest[:, :12].unflatten(1, (6, 2))[:, :, 0] = before[:, :12].unflatten(1, (6, 2))[:, :, 0]
    rest[:, 12:14] = before[:, 12:14]
    assert bool(((rest == before) | left[:, None, None]).all())
    # heads in front of rows, and into given outputs: the same bits
    hq, hk = q0.permute(1, 0, 2).contiguous().permute(1, 0, 2), k0.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    oq, ok = torch.full_like(hq, 3.0), torch.full((200, 2, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    call(hq, hk, pos, fd, layout=layout, pos_offset=-1, q_out=oq, k_out=ok)
    assert torch.equal(oq[~left], q[~left]) and torch.equal(ok[~left], k[~left])
    assert bool((oq[left] == 3.0).all()) and bool((ok[left] == 3.0).all())


@pytest.mark.parametrize("dtype, small, large", [("bf16", -125, 126), ("f32", -125, 126), ("f16", -14, 14)])
def test_norm_of_any_magnitude(dtype, small, large):
    """Heads whose squares leave fp32 are normed like their multiples by a power of two."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.uniform(1.0, 1.9, (4, 3, 64)) * rng.choice([-1, 1], (4, 3, 64))).cuda().to(_t(dtype))
    pos, f = torch.arange(4, dtype=torch.int32, device="cuda"), ops.rope_freqs(32)[0].cuda()
    want, _ = ops.norm_rope(x, None, None, None, pos, f, eps=0.0, weight_offset=1.0)
    for e in (small, -30 if small < -30 else small, large):
        y = (x.double() * 2.0 ** e).to(_t(dtype))
        got, _ = ops.norm_rope(y, None, None, None, pos, f, eps=0.0, weight_offset=1.0)
        assert torch.equal(got, want), e


def test_l2_norm_for_the_linear_layers():
    """rot = 0, no weights: x / sqrt(sum x^2 + eps)."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    rng = np.random.default_rng(4)
    q, k = (torch.from_numpy(rng.standard_normal((50, 16, 128)) * 3).cuda().bfloat16() for _ in range(2))
    none = torch.zeros(0, dtype=torch.float64, device="cuda")
    pos = torch.zeros(50, dtype=torch.int32, device="cuda")
    yq, yk = ops.norm_rope(q, k, None, None, pos, none, eps=1e-6 / 128, weight_offset=128 ** -0.5)
    for x, y in ((q, yq), (k, yk)):
        want = _f64(x) / np.sqrt((_f64(x) ** 2).sum(-1, keepdims=True) + 1e-6)
        check(y, want, np.abs(want), "bf16", True)


def test_values_that_are_not_finite():
    """They stay in their own pair (rope) or head (norm)."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    _, q, k, pos, _ = _case(6, 8, 4, 2, 128, 64, "bf16")
    q, k = q.clone(), k.clone()
    p, f = torch.from_numpy(pos).cuda(), ops.rope_freqs(64)[0].cuda()
    clean = ops.rope(q, k, p, f), ops.norm_rope(q, k, None, None, p, f, weight_offset=1.0)
    q[3, 1, 7], k[2, 0, 100] = float("nan"), float("inf")
    yq, yk = ops.rope(q, k, p, f)
    bad = torch.zeros_like(yq, dtype=torch.bool)
    bad[3, 1, 7] = bad[3, 1, 39] = True
    assert torch.isnan(yq[bad]).all() and torch.equal(yq[~bad], clean[0][0][~bad])
    bad = torch.zeros_like(yk, dtype=torch.bool)
    bad[2, 0, 100] = True
    assert torch.isinf(yk[bad]).all() and torch.equal(yk[~bad], clean[0][1][~bad])
    yq, yk = ops.norm_rope(q, k, None, None, p, f, weight_offset=1.0)
    assert torch.isnan(yq[3, 1]).all()
    assert torch.isnan(yk[2, 0, 100]) and not yk[2, 0, :100].any() and not yk[2, 0, 101:].any()
    yq[3, 1], yk[2, 0] = clean[1][0][3, 1], clean[1][1][2, 0]
    assert torch.equal(yq, clean[1][0]) and torch.equal(yk, clean[1][1])


def test_more_rows_than_a_grid_of_one_wave_each():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    R = 300001
    x = torch.randn((R, 1, 8), device="cuda")
    pos = torch.arange(R, dtype=torch.int32, device="cuda")
    f = ops.rope_freqs(8)[0]
    y, _ = ops.rope(x, None, pos, f.cuda())
    at = np.r_[0:5, R // 2:R // 2 + 5, R - 5:R]
    check(y[at], *ref.rope(_f64(x[at]), at, f.numpy(), "half", 1.0), "f32", False)


def test_refusals():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    x, pos, f = torch.zeros((4, 2, 64), device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), ops.rope_freqs(64)[0].cuda()
    w = torch.zeros(64, device="cuda")
    for call in (
            lambda: ops.rope(x, x.half(), pos, f), lambda: ops.rope(x, x[:3], pos, f), lambda: ops.rope(x, x[..., :32], pos, f),
            lambda: ops.rope(x, None, pos[:3], f), lambda: ops.rope(x, None, pos.long(), f), lambda: ops.rope(x, None, pos, f.float()),
            lambda: ops.rope(x, None, pos, f[None]), lambda: ops.rope(x, None, pos.cpu(), f), lambda: ops.rope(x, None, pos, f.cpu()),
            lambda: ops.rope(x.transpose(1, 2), None, pos, f), lambda: ops.rope(x[0], None, pos, f), lambda: ops.rope(x.double(), None, pos, f),
            lambda: ops.rope(x, None, pos, f, layout="other"), lambda: ops.rope(x, None, pos, f, pos_offset=1 << 31),
            lambda: ops.rope(x, None, pos, f, q_out=x[:3]), lambda: ops.rope(x, None, pos, f, q_out=x.half()),
            lambda: ops.norm_rope(x, x, w, w.half(), pos, f), lambda: ops.norm_rope(x, x, w[:32], w, pos, f),
            lambda: ops.norm_rope(x, x, w, w.cpu(), pos, f)):
        with pytest.raises(ValueError):
            call()
    for call, status in (
            (lambda: ops.rope(x, None, pos, ops.rope_freqs(66)[0].cuda()), -1),                 # rot > d
            (lambda: ops.rope(x.expand(4, 2, 64)[:, :1].expand(4, 3, 64), None, pos, f), -1),    # one head three times
            (lambda: ops.rope(torch.zeros((4, 2, 66), device="cuda")[..., :64], None, pos, f), -1),
            (lambda: ops.rope(torch.zeros((4, 2, 66), device="cuda"), None, pos, f), -2),
            (lambda: ops.norm_rope(x, None, w, None, pos, f, eps=-1.0), -1)):
        with pytest.raises(ops.SgdnError) as e:
            call()
        assert e.value.status == status
