"""Pins of the paged attention oracle: hand-worked bookkeeping, summaries at the
borders of their rounding, attention against closed forms, block choice by
crafted scores."""
import math

import numpy as np
import pytest

from oracle import paged


def test_plan_by_hand():
    # pages of 4 tokens; request 0 has 3 tokens and gets 3 (one page more),
    # request 1 is new and gets 4 (one page), request 2 gets none
    table = np.full((3, 4), -1, np.int32)
    table[0, 0], table[2, 0] = 9, 7
    ring = np.array([5, 6, 8, 0], np.int32)
    r = paged.plan([3, 0, 2], [3, 4, 0], table, ring, [5, 8], 4, 9)   # entries 5, 6, 7 -> 6, 8, 0
    assert r["table"][0, :2].tolist() == [9, 6] and r["table"][1, 0] == 8
    assert r["slot"].tolist() == [39, 24, 25, 32, 33, 34, 35, -1, -1]
    assert r["row_req"].tolist() == [0, 0, 0, 1, 1, 1, 1, -1, -1]
    assert r["row_len"].tolist() == [4, 5, 6, 1, 2, 3, 4, 0, 0]
    assert r["cu"].tolist() == [0, 3, 7, 7] and r["page_cu"].tolist() == [0, 1, 2, 2]
    assert r["lens"].tolist() == [6, 4, 2] and r["free_pos"].tolist() == [7, 8]
    assert r["status"].tolist() == [0, 0, 0]


def test_plan_refuses_in_order():
    table = np.full((5, 3), -1, np.int32)
    ring = np.arange(8, dtype=np.int32)
    # two pages free: 0 takes one, 1 needs two (refused), 2 would need one (the sum is past
    # the ring: refused), 3 needs none and is admitted, 4 needs four pages of three
    r = paged.plan([0, 0, 0, 1, 0], [4, 8, 1, 2, 13], table, ring, [0, 2], 4, 100)
    assert r["status"].tolist() == [0, 1, 1, 0, 2]
    assert r["lens"].tolist() == [4, 0, 0, 3, 0] and r["free_pos"].tolist() == [1, 2]
    r = paged.plan([0, 0, 0], [3, 3, -1], table[:3], ring, [0, 8], 4, 5)
    assert r["status"].tolist() == [0, 4, 8]


def test_release_then_plan_keeps_every_page():
    rng = np.random.default_rng(3)
    P, W, B, n_pages = 16, 6, 5, 40
    ring, pos = rng.permutation(n_pages).astype(np.int32), np.array([0, n_pages], np.int64)
    lens, table = np.zeros(B, np.int32), np.full((B, W), -1, np.int32)
    for _ in range(40):
        done = rng.random(B) < 0.2
        lens, ring, pos = paged.release(lens, done, table, ring, pos, P)
        add = rng.integers(0, 30, B)
        r = paged.plan(lens, add, table, ring, pos, P, 200)
        lens, table, pos = r["lens"], r["table"], r["free_pos"]
        held = [table[b, j] for b in range(B) for j in range(paged.pages_of(lens[b], P))]
        free = [ring[i % n_pages] for i in range(pos[0], pos[1])]
        assert sorted(map(int, held + free)) == list(range(n_pages))


@pytest.mark.parametrize("x, codes, scale", [
    ([64.0, -1.0, 0.5, 1.5], [64, -1, 0, 2], 1.0),           # ties to even
    ([127.4, 1.0], [127, 1], 1.0),
    ([127.5, -127.9], [127, -127], 1.0),                      # held at 127
    ([128.0, 1.0], [64, 0], 2.0),
    ([0.0, 0.0], [0, 0], 1.0),
    ([math.inf, 3.0, math.nan], [0, 96, 0], 2.0 ** -5),
    ([2.0 ** -149], [0], 2.0 ** -126),                        # fp32's smallest: the scale stays normal
])
def test_quantise(x, codes, scale):
    c, s = paged.quantise(np.array(x))
    assert c.tolist() == codes and s == scale


def test_attend_closed_forms():
    P, D = 16, 64
    k = np.zeros((3, 1, P, D))
    v = np.random.default_rng(5).standard_normal((3, 1, P, D))
    table = np.array([[2, 0]], np.int32)
    q = np.ones((1, 2, D))
    o, lse, _ = paged.attend(q, k, v, table, [20])
    mean = np.concatenate([v[2, 0], v[0, 0, :4]]).mean(0)     # equal scores: the mean
    assert np.allclose(o[0, 0], mean) and np.allclose(lse, math.log(20))
    k[0, 0, 3] = 100.0                                        # one key takes everything
    o, _, _ = paged.attend(q, k, v, table, [20])
    assert np.allclose(o[0, 1], v[0, 0, 3])
    o, lse, _ = paged.attend(q, k, v, table, [0])
    assert not o.any() and np.isneginf(lse).all()


def test_attend_over_all_blocks_is_attend():
    rng = np.random.default_rng(6)
    P, D = 16, 64
    k, v = rng.standard_normal((2, 9, 2, P, D))
    table = rng.permutation(8).reshape(2, 4).astype(np.int32)
    q, length = rng.standard_normal((2, 4, D)), [50, 17]
    full = paged.attend(q, k, v, table, length)
    lists = np.tile(np.array([3, 1, -1, 0, 2], np.int32), (2, 2, 1))
    part = paged.attend(q, k, v, table, length, blocks=lists)
    assert np.allclose(full[0], part[0]) and np.allclose(full[1], part[1])


def test_select_crafted():
    D, page = 64, 16
    codes = np.zeros((8, 1, D), np.int8)
    codes[:, 0, 0] = [1, 5, 3, 5, 9, 2, 0, 0]
    scale = np.ones((8, 1), np.float32)
    table = np.arange(8, dtype=np.int32)[None]
    q = np.zeros((1, 1, D))
    q[0, 0, 0] = 1.0
    pick = lambda n, **kw: paged.select(q, codes, scale, table, [7 * page - 3], page, n, **kw)[0, 0].tolist()
    assert pick(4) == [0, 1, 4, 6]                # 0 and 6 forced, 4 best, 1 before 3 (equal)
    assert pick(5) == [0, 1, 3, 4, 6]
    assert pick(3, n_sink=0, n_local=2) == [4, 5, 6]
    assert pick(9) == [0, 1, 2, 3, 4, 5, 6, -1, -1]
    scale[4] = 0.25                               # 9 / 4 is under 3
    assert pick(4) == [0, 1, 3, 6]
    table[0, 3] = 99                              # no such page: ranks last
    assert pick(4) == [0, 1, 2, 6]
