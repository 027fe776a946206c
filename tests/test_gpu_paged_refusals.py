"""Steps that do not fit: requests refused for pages (1) and for rows (4), one after the other, in
the page bookkeeping of every launch form and in serving steps that go on with what was admitted."""
import numpy as np
import pytest

import test_gpu_paged_flow as flow
from oracle import paged as ref
from test_gpu_paged import _compare_plan, _f64, _i32, _plan_state, check

P = 16


def _state(B, first, rows, spare, seed):
    """B requests of a few tokens, every third of which starts a page with its new ones.  The ring
    holds `spare` pages, `first` requests want many rows; the others one or none."""
    rng = np.random.default_rng(seed)
    cached = rng.integers(1, 3 * P - 8, B)
    cached[::3] = P * rng.integers(0, 3, len(cached[::3]))
    blocks = -(-cached // P)
    lens, table, ring, pos = _plan_state(rng, B, 5, P, int(blocks.sum()) + spare, cached)
    add = rng.integers(0, 2, B).astype(np.int32)
    add[:first] = rng.integers(0, 8, first)
    add[rng.integers(0, B, B // 20)] = -1
    lens[rng.integers(0, B, B // 30)] = -3
    add[rng.integers(0, B, B // 30)] = 5 * P
    return lens, add, table, ring, pos


CASES = [  # B, first, rows, spare; the sums run over chunks of up to 1024 requests
    (900, 300, 1000, 150),           # one launch
    (900, 300, 1100, 150),           # rows in a second launch
    (3000, 600, 5000, 250),                # pages end in the first chunk, rows never
    (3000, 600, 2500, 250),                # ... rows in the second or third
    (2600, 1000, 1500, 120),               # both in the first
    (2600, 1000, 1500, 0),                 # no page at all
    (1500, 700, 1200, 5000),               # rows alone
]


def _plan(case, seed):
    B, first, rows, spare = case
    state = _state(B, first, rows, spare, seed)
    return state, rows, ref.plan(*state, P, rows)


def test_reasons_occur():
    """What the cases are for: by chunk of 1024 requests, the reasons and whether some get rows."""
    seen = []
    for case in CASES:
        state, rows, want = _plan(case, 1)
        status, got = want["status"], np.diff(want["cu"])
        seen.append([(set(status[i:i + 1024]), int(got[i:i + 1024].sum())) for i in range(0, len(status), 1024)])
    for chunks in seen[:2]:
        assert chunks[0][0] >= {0, 1, 2, 4, 8}
    assert 1 in seen[2][0][0] and all(4 not in s for s, _ in seen[2]) and seen[2][1][1] > 0 and seen[2][2][1] > 0
    assert 1 in seen[3][0][0] and 4 not in seen[3][0][0] and 4 in seen[3][2][0] and seen[3][1][1] > 0
    assert {1, 4} <= seen[4][0][0] and 0 in seen[4][1][0]
    assert 1 in seen[5][0][0] and seen[5][0][1] > 0
    assert 4 in seen[6][0][0] and not any(1 in s for s, _ in seen[6])


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_plan_refuses(case, inplace):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    for seed in (1, 2):
        state, rows, want = _plan(case, seed)
        d = [torch.from_numpy(x).cuda() for x in state]
        got = ops.paged_plan(*d, P, rows, **(dict(lens_out=d[0], free_pos_out=d[4]) if inplace else {}))
        torch.cuda.synchronize()
        _compare_plan(got, want, d[2])


PAGES, ROWS, STEPS = 26, 96, 16


def _adds(rng, step):
    """New tokens and ended requests of a step; prompts that often find too few pages or rows."""
    add, done = rng.integers(0, 2, flow.B), np.zeros(flow.B, np.uint8)
    for b in rng.permutation(flow.B)[:step % 3]:
        add[b] = rng.integers(30, 120)
    if step % 5 == 4:
        for b in rng.permutation(flow.B)[:2]:
            done[b], add[b] = 1, 0
    return add, done


def test_serving_steps_refuse():
    """The steps below contain both reasons, and requests that are admitted in the same step."""
    rng = np.random.default_rng(8)
    lens, table = np.zeros(flow.B, np.int32), np.full((flow.B, flow.W), -1, np.int32)
    ring, pos, seen, beside = np.arange(PAGES, dtype=np.int32), np.array([0, PAGES]), set(), set()
    for step in range(STEPS):
        add, done = _adds(rng, step)
        lens, ring, pos = ref.release(lens, done, table, ring, pos, flow.P)
        r = ref.plan(lens, add, table, ring, pos, flow.P, ROWS)
        lens, table, pos = r["lens"], r["table"], r["free_pos"]
        seen |= set(r["status"].tolist())
        if r["cu"][-1] > 0:
            beside |= set(r["status"].tolist())
    assert {0, 1, 4} <= seen and {1, 4} <= beside and lens.max() > 60


@pytest.mark.gpu
def test_serving_goes_on(monkeypatch):
    import torch
    monkeypatch.setattr(flow, "PAGES", PAGES)
    s, rng, seen = flow.Server(3), np.random.default_rng(8), set()
    for step in range(STEPS):
        add, done = _adds(rng, step)
        q, k, v = s.tokens(ROWS)
        plan, blocks, part, full = s.step(_i32(add), torch.from_numpy(done).cuda(), ROWS, q, k, v)
        torch.cuda.synchronize()
        want, h = s.mirror(add, done, ROWS, k, v), s.h
        seen |= set(want["status"].tolist())
        for n in ("cu", "page_cu", "slot", "row_req", "row_len", "status"):
            assert np.array_equal(plan[n].cpu().numpy(), want[n]), (step, n)
        for n, t in (("lens", s.lens), ("table", s.table), ("ring", s.ring), ("pos", s.pos)):
            assert np.array_equal(t.cpu().numpy(), h[n]), (step, n)
        assert np.array_equal(blocks.cpu().numpy(), ref.select(
            _f64(q), h["codes"], h["scale"], h["table"], want["row_len"], flow.P, flow.KEEP, req=want["row_req"])), step
        args = (_f64(q), h["k"], h["v"], h["table"], want["row_len"], want["row_req"])
        check(*full, ref.attend(*args), "f32", s.dtype, flow.D)
        check(*part, ref.attend(*args, blocks=blocks.cpu().numpy()), "f32", s.dtype, flow.D)
    assert {0, 1, 4} <= seen
