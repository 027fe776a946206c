"""The paged attention operators: their plain forms, their 64-bit definitions and the cases
they are measured on.

A softmax attention layer that is served beside the gated linear layers keeps its keys and
values in pages of a cache.  Five operators make up its path:

  plan      block tables and slot maps from request lengths (and finished requests' pages back)
  write     new keys and values into their slots, and an 8-bit summary of each page completed
  attend    one new token per row over its whole cached sequence
  select    the blocks (pages) that a cheap score over the summaries picks for each row
  sparse    attention of each row over its picked blocks

Notation: P tokens per page, W pages per table row, R rows (new tokens), Hq query heads in groups
of G over Hkv key/value heads, D elements per head.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # One token for each of 128 running requests: bookkeeping ahead of every decode step.
        dict(name="plan_step", op="plan", batch=128, width=2048, page=64, cached=131072, new=1, done=0, prompts=0),
        # A serving step that swaps an eighth of 64 requests for long prompts.
        dict(name="plan_turnover", op="plan", batch=64, width=512, page=64, cached=32000, new=1, done=8, prompts=8),
        # One new token for each of 128 requests.
        dict(name="write_step", op="write", batch=128, new=1, cached=2000, hkv=8, d=128, page=64, type="bf16"),
        # A batch of prompts, ragged, 32K tokens in all.
        dict(name="write_prompts", op="write", batch=8, new=8192, cached=100, hkv=8, d=128, page=64, type="bf16"),
        # A lone request at a short context: latency alone.
        dict(name="attend_one", op="attend", batch=1, cached=4096, hq=32, hkv=8, d=128, page=64, type="bf16"),
        # The decode step of a full batch, ragged.
        dict(name="attend_batch", op="attend", batch=128, cached=8192, hq=32, hkv=8, d=128, page=64, type="bf16"),
        # Two requests at the longest context, few and wide heads.
        dict(name="attend_long", op="attend", batch=2, cached=131072, hq=16, hkv=2, d=256, page=64, type="f16"),
        # Everything odd: 32-bit, small pages, five heads a group, uneven lengths.
        dict(name="attend_odd", op="attend", batch=7, cached=5001, hq=15, hkv=3, d=64, page=16, type="f32"),
        # Choice of 64 blocks for each decoded token at long contexts.
        dict(name="select_step", op="select", batch=32, new=1, cached=131072, hq=32, hkv=8, d=128, page=64, blocks=64, type="bf16"),
        # Choice of 16 blocks for every token of four prompts.
        dict(name="select_prompts", op="select", batch=4, new=2048, cached=16384, hq=16, hkv=2, d=256, page=64, blocks=16, type="bf16"),
        # Decode over 64 of up to 512 blocks.
        dict(name="sparse_step", op="sparse", batch=32, new=1, cached=32768, hq=32, hkv=8, d=128, page=64, blocks=64, type="bf16"),
        # Every token of four prompts over its 16 blocks.
        dict(name="sparse_prompts", op="sparse", batch=4, new=1024, cached=16384, hq=16, hkv=2, d=256, page=64, blocks=16, type="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "select", "sparse"])
    cost = lambda c: max(work(c)["bytes"], work(c)["flops"] / 50)  # noqa: E731
    most = max(cost(c) for c in listed() if c["op"] == op)
    while True:
        case = _draw(rng, op)
        if cost(case) <= most:
            return case


def _draw(rng, op):
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "plan":
        batch = _log(rng, 1, 512)
        cached = _log(rng, 1, 131072)
        done = rng.randint(0, batch // 8)
        return dict(op=op, batch=batch, width=cached // page + 300, page=page, cached=cached,
                    new=rng.choice([1, 1, _log(rng, 1, 64)]), done=done, prompts=rng.randint(0, batch // 8))
    heads = dict(hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128, 128, 256]), page=page,
                 type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    row = heads["hkv"] * heads["d"] * BYTES[heads["type"]] * 2
    if op == "write":
        new = rng.choice([1, _log(rng, 1, 8192)])
        batch = _log(rng, 1, max(1, min(256, (1 << 28) // (new * row))))
        return dict(op=op, batch=batch, new=new, cached=_log(rng, 1, 2000), **heads)
    heads["hq"] = heads["hkv"] * rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "attend":
        cached = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(256, (1 << 31) // (cached * row))))
        return dict(op=op, batch=batch, cached=cached, **heads)
    blocks = _log(rng, 4, 64)
    if rng.random() < 0.5:
        batch, new, cached = _log(rng, 1, 32), 1, _log(rng, 1, 32768)
    else:
        new = _log(rng, 2, 1024)
        batch, cached = _log(rng, 1, max(1, 2048 // new)), new + _log(rng, 1, 15360)
        blocks = min(blocks, 1024 // page)
    if op == "select":      # more blocks than are picked: otherwise nothing is chosen
        cached = new + _log(rng, 4 * blocks * page, 8 * blocks * page if new > 1 else 131072)
    return dict(op=op, batch=batch, new=new, cached=cached, blocks=max(blocks, 2), **heads)


# What a case is made of ------------------------------------------------------------------------


def _lengths(case):
    """Cached lengths (before the step) and new tokens of each request: ragged, the first the longest.
    They belong to the case, so that its outputs have one shape."""
    rng = np.random.default_rng([case["batch"], case["cached"], case["page"], 17])
    b, n = case["batch"], case.get("new", 1)
    cached = np.maximum(1, (case["cached"] * rng.uniform(0.25, 1.0, b)).astype(np.int64))
    cached[0] = case["cached"]
    new = np.maximum(1, (n * rng.uniform(0.3, 1.0, b)).astype(np.int64)) if n > 1 else np.ones(b, np.int64)
    new[0] = n
    return cached, new


def _mean_lengths(case):
    b, n = case["batch"], case.get("new", 1)
    cached = case["cached"] * (1 + 0.625 * (b - 1))
    new = n * (1 + 0.65 * (b - 1)) if n > 1 else b
    return cached, new


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _table(lengths, page, seed, spare=8):
    """A block table whose rows are pages in random order, and the number of pages of the cache."""
    blocks = -(-lengths // page)
    total = int(blocks.sum())
    pages = total + spare
    order = np.random.default_rng([seed, 23]).permutation(pages)[:total]
    width = int(blocks.max())
    table = np.full((len(lengths), width), -1, np.int32)
    table[np.arange(width)[None, :] < blocks[:, None]] = order
    return table, pages


def _rows(cached, new):
    """Request and visible length of each row: the new tokens of every request, one after the other."""
    req = np.repeat(np.arange(len(new)), new)
    first = np.repeat(np.cumsum(new) - new, new)
    return req, np.repeat(cached, new) + np.arange(len(req)) - first + 1


def _prepare_plan(case, seed):
    rng = np.random.default_rng([case["batch"], case["cached"], 5])
    b, p, w = case["batch"], case["page"], case["width"]
    cached, _ = _lengths(case)
    cached = np.minimum(cached, w * p - 64)
    new = np.full(b, case["new"], np.int64)
    done = np.zeros(b, np.uint8)
    order = rng.permutation(b)
    gone, fresh = order[:case["done"]], order[case["done"]:case["done"] + case["prompts"]]
    done[gone] = 1
    new[gone] = 0
    cached[fresh] = 0
    new[fresh] = rng.integers(1, min(32768, w * p - 1) + 1, len(fresh))
    blocks = -(-cached // p)
    need = int((-(-(cached + new) // p) - blocks).sum())
    held = int(blocks.sum())
    pages = held + need + 16
    rng = np.random.default_rng([seed, 7])
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((b, w), -1, np.int32)
    table[np.arange(w)[None, :] < blocks[:, None]] = ids[:held]
    # the ring of free pages: as long as the cache, entries taken .. returned - 1 are free
    taken = int(rng.integers(0, 3 * pages))
    ring = np.zeros(pages, np.int32)
    ring[(taken + np.arange(pages - held)) % pages] = ids[held:]
    return dict(op="plan", page=p, rows=int(new.sum()), any_done=case["done"] > 0, lens=_int32(cached), add=_int32(new),
                done=torch.from_numpy(done).cuda(), table=_int32(table), ring=_int32(ring),
                pos=torch.tensor([taken, taken + pages - held], dtype=torch.int64, device="cuda"))


def _cache(pages, case, g):
    shape = (pages, case["hkv"], case["page"], case["d"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16 if case["type"] == "bf16" else torch.float32).to(
        TYPES[case["type"]]) for _ in range(2)]


def prepare(case, seed):
    if case["op"] == "plan":
        return _prepare_plan(case, seed)
    g = _generator(seed)
    dt, p, hkv, d = TYPES[case["type"]], case["page"], case["hkv"], case["d"]
    cached, new = _lengths(case)
    if case["op"] == "attend":
        table, pages = _table(cached, p, seed)
        k, v = _cache(pages, case, g)
        q = torch.randn((len(cached), case["hq"], d), generator=g, device="cuda").to(dt)
        return dict(op="attend", q=q, k=k, v=v, table=_int32(table), lens=_int32(cached), most=int(cached.max()))
    if case["op"] != "write" and case["new"] > 1:
        cached = np.maximum(cached - new, 0)     # the prompt's own tokens are the last of the context
    table, pages = _table(cached + new, p, seed)
    req, length = _rows(cached, new)
    if case["op"] == "write":
        k, v = _cache(pages, case, g)
        slot = table[req, (length - 1) // p].astype(np.int64) * p + (length - 1) % p
        fused = torch.randn((len(req), 2, hkv, d), generator=g, device="cuda").to(dt)   # one projection's output
        codes = torch.zeros((pages, hkv, d), dtype=torch.int8, device="cuda")
        scale = torch.ones((pages, hkv), dtype=torch.float32, device="cuda")
        return dict(op="write", k=fused[:, 0], v=fused[:, 1], slot=_int32(slot), k_cache=k, v_cache=v, codes=codes, scale=scale,
                    most=min(len(req), len(req) // p + len(new)))
    s = dict(op=case["op"], table=_int32(table), req=_int32(req), len=_int32(length), page=p, blocks=case["blocks"],
             cu=_int32(np.concatenate([[0], np.cumsum(new)])), longest=int(new.max()), most=int(length.max()))
    width, rows = table.shape[1], len(req)
    s["q"] = torch.randn((rows, case["hq"], d), generator=g, device="cuda").to(dt)
    if case["op"] == "select":
        mean = torch.randn((pages, hkv, d), generator=g, device="cuda") * 0.25
        s["codes"], s["scale"] = _quantise(mean.double())
        return s
    # lists as a selection leaves them: neighbouring rows look for much the same blocks
    s["k"], s["v"] = _cache(pages, case, g)
    topic = torch.randn((rows // 32 + len(new) + 1, hkv, width), generator=g, device="cuda")
    drift = torch.from_numpy(np.cumsum(np.r_[False, (req[1:] != req[:-1]) | (np.arange(1, rows) % 32 == 0)])).cuda()
    score = topic[drift] + 0.3 * torch.randn((rows, hkv, width), generator=g, device="cuda")
    s["lists"] = _choose(score, s["len"], p, case["blocks"], 1, 2)
    return s


# The plain forms -------------------------------------------------------------------------------


def _plan_plain(s):
    p, rows, ring, table, b = s["page"], s["rows"], s["ring"], s["table"], s["lens"].numel()
    lens, pos, w = s["lens"].long(), s["pos"].clone(), s["table"].shape[1]
    f = ring.numel()
    dev = ring.device
    blocks = torch.div(lens + (p - 1), p, rounding_mode="floor")
    if s["any_done"]:
        give = torch.where(s["done"] != 0, blocks, 0)
        at = give.cumsum(0) - give
        col = torch.arange(w, device=dev)
        where = torch.where(col[None, :] < give[:, None], (pos[1] + at[:, None] + col[None, :]) % f, f)
        ring_now = torch.cat([ring, ring.new_zeros(1)]).scatter_(0, where.reshape(-1), table.reshape(-1))[:f]
        ring.copy_(ring_now)
        pos[1] += give.sum()
        lens = torch.where(s["done"] != 0, 0, lens)
        blocks = torch.where(s["done"] != 0, 0, blocks)
    add = s["add"].long()
    total = lens + add
    after = torch.div(total + (p - 1), p, rounding_mode="floor")
    status = torch.where((add < 0) | (lens < 0), 8, torch.where(after > w, 2, 0))
    need, want = torch.where(status == 0, after - blocks, 0), torch.where(status == 0, add, 0)
    status = torch.where((status == 0) & (need > 0) & (need.cumsum(0) > pos[1] - pos[0]), 1, status)
    status = torch.where((status == 0) & (want > 0) & (want.cumsum(0) > rows), 4, status)
    need, want = torch.where(status == 0, need, 0), torch.where(status == 0, want, 0)
    zero = need.new_zeros(1)
    page_cu, cu = torch.cat([zero, need.cumsum(0)]), torch.cat([zero, want.cumsum(0)])
    r = torch.arange(rows, device=dev)
    req = torch.searchsorted(cu, r, right=True) - 1
    live = r < cu[-1]
    q = req.clamp(0, b - 1)
    at = lens[q] + r - cu[q]
    block = torch.div(at, p, rounding_mode="floor")
    fresh = live & (block >= blocks[q])
    held = table[q, block.clamp(0, w - 1)].long()
    page = torch.where(fresh, ring[(pos[0] + page_cu[q] + block - blocks[q]) % f].long(), held)
    table[q, block.clamp(0, w - 1)] = torch.where(live, page, held).int()
    ints = lambda x: x.to(torch.int32)  # noqa: E731
    taken = torch.stack([pos[0] + page_cu[-1], pos[1]])
    return dict(lens=ints(lens + want), cu=ints(cu), page_cu=ints(page_cu), slot=ints(torch.where(live, page * p + at % p, -1)),
                row_req=ints(torch.where(live, req, -1)), row_len=ints(torch.where(live, at + 1, 0)), free_pos=taken,
                status=ints(status), table=table, ring=ring)


def _quantise(mean):
    """Codes and a power of two for each vector: the smallest 2^e with max|mean| <= 2^(e + 7), at least 2^-126."""
    top = mean.abs().amax(-1)
    _, e = torch.frexp(top)
    scale = ((e - 7).clamp(min=-126, max=127) + 127).int().bitwise_left_shift(23).view(torch.float32)   # the power by its bits
    scale = torch.where(top > 0, scale, 1.0)
    codes = torch.round(mean / scale[..., None]).clamp(-127, 127)
    return codes.to(torch.int8), scale


def _write_plain(s):
    kc, vc, p = s["k_cache"], s["v_cache"], s["k_cache"].shape[2]
    slot = s["slot"].long()
    page, off = torch.div(slot, p, rounding_mode="floor"), slot % p
    kc[page, :, off] = s["k"]
    vc[page, :, off] = s["v"]
    # pages whose last slot is written now: at most `most` of them
    full = off == p - 1
    pick = torch.argsort((~full).to(torch.uint8), stable=True)[:s["most"]]
    valid = full[pick]
    at = torch.where(valid, page[pick], page[pick[0]])
    codes, scale = _quantise(kc[at].double().sum(2) / p)
    s["codes"][at] = torch.where(valid[0], codes, s["codes"][at])
    s["scale"][at] = torch.where(valid[0], scale, s["scale"][at])
    return dict(k_cache=kc, v_cache=vc, summary=s["codes"] * s["scale"][..., None])


def _softmax(q, k, v, live):
    """q [.., G, D], k and v [.., T, D], live [.., 1, T]: the output and the log of the sum."""
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()) * (1.0 / math.sqrt(q.shape[-1]))
    x = torch.where(live, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.where(live, torch.exp(x - top), 0.0)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, torch.where(live.transpose(-1, -2), v, 0.0)) / total
    some = live.any(-1, keepdim=True)
    return torch.where(some, o, 0.0), torch.where(some, top + torch.log(total), -math.inf).squeeze(-1)


def _attend_plain(s):
    q, kc, vc = s["q"], s["k"], s["v"]
    pages, hkv, p, d = kc.shape
    b, hq, _ = q.shape
    n = -(-s["most"] // p)
    table = s["table"][:, :n].long().clamp(min=0)
    k = kc[table].float().transpose(1, 2).reshape(b, hkv, n * p, d)
    v = vc[table].float().transpose(1, 2).reshape(b, hkv, n * p, d)
    live = torch.arange(n * p, device=q.device) < s["lens"][:, None]
    o, lse = _softmax(q.float().reshape(b, hkv, hq // hkv, d), k, v, live[:, None, None, :])
    return dict(o=o.reshape(q.shape).to(q.dtype), lse=lse.reshape(b, hq))


def _choose(score, length, p, blocks, n_sink, n_local):
    """The `blocks` best of each row's blocks, the first and last ones always, in rising order; -1 after them."""
    n = torch.div(length.long() + (p - 1), p, rounding_mode="floor")[:, None, None]
    j = torch.arange(score.shape[-1], device=score.device)
    score = torch.where((j < n_sink) | (j >= n - n_local), math.inf, score)
    score = torch.where(j < n, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.arange(score.shape[-1], device=score.device)
    best = torch.where(rank < torch.clamp(n, max=blocks), best, score.shape[-1]).sort(-1).values[..., :blocks]
    best = torch.where(best < score.shape[-1], best, -1).to(torch.int32)
    return torch.nn.functional.pad(best, (0, blocks - best.shape[-1]), value=-1).contiguous()


def _select_plain(s):
    q, table = s["q"], s["table"].long().clamp(min=0)
    rows, hq, d = q.shape
    pages, hkv, _ = s["codes"].shape
    b, w = table.shape
    g = hq // hkv
    codes, scale = _quantise(q.double())
    req = s["req"].long()
    at = torch.arange(rows, device=q.device) - s["cu"].long()[req]     # place among the request's rows
    padded = torch.zeros((b, s["longest"], hkv, g, d), device=q.device)
    padded[req, at] = codes.float().reshape(rows, hkv, g, d)
    padded = padded.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    keys = s["codes"][table].float().permute(0, 2, 3, 1).contiguous()          # [b, hkv, d, w]
    dot = torch.matmul(padded, keys).reshape(b, hkv, s["longest"], g, w)        # whole numbers under 2^24: exact
    dot = dot.permute(0, 2, 1, 3, 4)[req, at]                                   # [rows, hkv, g, w]
    mean = s["scale"][table].permute(0, 2, 1)[req]                              # [rows, hkv, w]
    score = ((dot * scale.reshape(rows, hkv, g, 1)) * mean[:, :, None, :]).amax(2)
    return dict(blocks=_choose(score, s["len"], s["page"], s["blocks"], 1, 1))


def _sparse_plain(s):
    q, kc, vc, lists = s["q"], s["k"], s["v"], s["lists"].long()
    pages, hkv, p, d = kc.shape
    rows, hq, _ = q.shape
    n = lists.shape[-1]
    page = s["table"].long()[s["req"].long()[:, None, None], lists.clamp(min=0)].clamp(min=0)
    head = torch.arange(hkv, device=q.device)[None, :, None]
    at = lists[..., None] * p + torch.arange(p, device=q.device)
    live = (lists[..., None] >= 0) & (at < s["len"].long()[:, None, None, None])
    o, lse = _softmax(q.float().reshape(rows, hkv, hq // hkv, d), kc[page, head].float().reshape(rows, hkv, n * p, d),
                      vc[page, head].float().reshape(rows, hkv, n * p, d), live.reshape(rows, hkv, 1, n * p))
    return dict(o=o.reshape(q.shape).to(q.dtype), lse=lse.reshape(rows, hq))


# One pass --------------------------------------------------------------------------------------


def _run_own(s):
    from gated_deltanet_prefill_chunkwise_amd import ops
    if s["op"] == "plan":
        lens, pos = s["lens"], s["pos"]
        if s["any_done"]:
            lens, pos = ops.paged_release(lens, s["done"], s["table"], s["ring"], pos, s["page"])
        r = ops.paged_plan(lens, s["add"], s["table"], s["ring"], pos, s["page"], s["rows"])
        return dict(r, table=s["table"], ring=s["ring"])
    if s["op"] == "write":
        ops.paged_write(s["k"], s["v"], s["slot"], s["k_cache"], s["v_cache"], s["codes"], s["scale"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], summary=s["codes"] * s["scale"][..., None])
    if s["op"] == "attend":
        o, lse = ops.paged_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], max_len=s["most"], out_dtype=s["q"].dtype, want_lse=True)
        return dict(o=o, lse=lse)
    if s["op"] == "select":
        return dict(blocks=ops.paged_select(s["q"], s["codes"], s["scale"], s["table"], s["len"], s["page"], s["blocks"], row_req=s["req"],
                                            n_sink=1, n_local=1, max_len=s["most"]))
    o, lse = ops.paged_attend_sparse(s["q"], s["k"], s["v"], s["table"], s["len"], s["lists"], row_req=s["req"], out_dtype=s["q"].dtype,
                                     want_lse=True)
    return dict(o=o, lse=lse)


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan_plain, "write": _write_plain, "attend": _attend_plain, "select": _select_plain, "sparse": _sparse_plain}[state["op"]](state)


# What a pass cannot do without -----------------------------------------------------------------


def work(case):
    cached, new = _mean_lengths(case)
    p, b = case["page"], case["batch"]
    if case["op"] == "plan":
        rows = (b - case["done"] - case["prompts"]) * case["new"] + case["prompts"] * min(32768, case["width"] * p) / 2
        moved = rows / p + case["done"] * 0.6 * case["cached"] / p
        return {"bytes": 4.0 * (2 * b + 2 * moved + 3 * rows + 4 * b), "flops": 0.0}
    e, hkv, d = BYTES[case["type"]], case["hkv"], case["d"]
    if case["op"] == "write":
        done = new / p
        return {"bytes": 4.0 * new * hkv * d * e + 4 * new + done * hkv * (d + 4), "flops": done * p * hkv * d}
    hq = case["hq"]
    if case["op"] == "attend":
        return {"bytes": 2.0 * cached * hkv * d * e + 2 * b * hq * d * e + 4 * cached / p, "flops": 4.0 * cached * hq * d}
    ctx = case["cached"] * (1 + 0.625 * (b - 1)) / b          # of one request
    seen = ctx - (new / b) / 2                                # of one row, on average
    if case["op"] == "select":
        return {"bytes": b * ctx / p * (hkv * (d + 4) + 4) + new * (hq * d * e + hkv * case["blocks"] * 4), "flops": 2.0 * new * hq * d * seen / p}
    keys = min(case["blocks"] * p, seen)
    pages = b * min(ctx, keys * new / b)
    return {"bytes": 2.0 * pages * hkv * d * e + 2 * new * hq * d * e + new * hkv * case["blocks"] * 4, "flops": 4.0 * new * hq * keys * d}


# The definitions, in 64 bits --------------------------------------------------------------------


def _host(t):
    return t.cpu().numpy()


def _exact_plan(s):
    lens, add, done = (_host(s[n]).astype(np.int64) for n in ("lens", "add", "done"))
    table, ring, p, rows = _host(s["table"]).copy(), _host(s["ring"]).copy(), s["page"], s["rows"]
    taken, back = (int(x) for x in _host(s["pos"]))
    f, w = len(ring), table.shape[1]
    for b in range(len(lens)):
        if done[b] and s["any_done"]:
            for j in range(-(-lens[b] // p)):
                ring[back % f] = table[b, j]
                back += 1
            lens[b] = 0
    first, slot, req, length, cu, page_cu, status = taken, [], [], [], [0], [0], []
    wanted = pages = 0
    for b in range(len(lens)):
        have, after = -(-lens[b] // p), -(-(lens[b] + add[b]) // p)
        why = 8 if add[b] < 0 or lens[b] < 0 else 2 if after > w else 0
        if why == 0:
            pages += after - have
            wanted += add[b]
            why = 1 if after > have and pages > back - first else 4 if add[b] > 0 and wanted > rows else 0
        if why == 0:
            for j in range(have, after):
                table[b, j] = ring[taken % f]
                taken += 1
            for t in range(lens[b], lens[b] + add[b]):
                slot.append(int(table[b, t // p]) * p + t % p)
                req.append(b)
                length.append(t + 1)
            lens[b] += add[b]
        cu.append(len(slot))
        page_cu.append(taken - first)
        status.append(why)
    pad = rows - len(slot)
    as_int = lambda x: torch.tensor(np.asarray(x, np.int64), dtype=torch.int32)  # noqa: E731
    return dict(lens=as_int(lens), cu=as_int(cu), page_cu=as_int(page_cu), slot=as_int(slot + [-1] * pad), row_req=as_int(req + [-1] * pad),
                row_len=as_int(length + [0] * pad), free_pos=torch.tensor([taken, back]), status=as_int(status), table=as_int(table), ring=as_int(ring))


def _exact_summary(keys):
    """keys [n, Hkv, P, D] as float64 arrays: the values that a page's codes stand for."""
    m = keys.mean(2)
    top = np.abs(m).max(-1)
    unit = np.where(top > 0, np.exp2(np.maximum(np.floor(np.log2(np.where(top > 0, top, 1.0))) - 6, -126)), 1.0)[..., None]
    return np.clip(np.rint(m / unit), -127, 127), unit


def _exact_write(s):
    p = s["k_cache"].shape[2]
    slot = _host(s["slot"])
    k = s["k"].double().cpu().numpy()
    value = (s["codes"].double() * s["scale"].double()[..., None]).cpu().numpy()
    full = np.nonzero(slot % p == p - 1)[0]
    for i in full:
        page = slot[i] // p
        keys = s["k_cache"][page].double().cpu().numpy()
        for r in range(max(0, i - p + 1), i + 1):
            if slot[r] // p == page:
                keys[:, slot[r] % p] = k[r]
        c, unit = _exact_summary(keys[None])
        value[page] = (c * unit)[0]
    return dict(k_cache=None, v_cache=None, summary=torch.from_numpy(value))


def _exact_row(q, k, v):
    """q [Hkv, G, D], k and v [Hkv, T, D] in float64, one row."""
    x = torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(q.shape[-1])
    return torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v), torch.logsumexp(x, -1)


def _exact_attend(s):
    hkv, p, d = s["k"].shape[1:]
    q = s["q"].double()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b, n in enumerate(_host(s["lens"])):
        ids = s["table"][b, :-(-int(n) // p)].long()
        k, v = (c[ids].double().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] for c in (s["k"], s["v"]))
        a, z = _exact_row(q[b].reshape(hkv, -1, d), k, v)
        o[b], lse[b] = a.reshape(-1, d), z.reshape(-1)
    return dict(o=o, lse=lse)


def _exact_select(s):
    q = s["q"].double().cpu().numpy()
    rows, hq, d = q.shape
    hkv = s["codes"].shape[1]
    top = np.abs(q).max(-1, keepdims=True)
    unit = np.where(top > 0, np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0))) - 6), 1.0)
    q = (np.clip(np.rint(q / unit), -127, 127) * unit).reshape(rows, hkv, -1, d)
    value = s["codes"].double().cpu().numpy() * s["scale"].double().cpu().numpy()[..., None]
    table, req, length = _host(s["table"]), _host(s["req"]), _host(s["len"])
    out = np.full((rows, hkv, s["blocks"]), -1, np.int32)
    for b in np.unique(req):
        mine = np.nonzero(req == b)[0]
        keys = value[np.maximum(table[b], 0)]
        for h in range(hkv):
            score = (q[mine, h].reshape(-1, d) @ keys[:, h].T).reshape(len(mine), -1, keys.shape[0]).max(1)
            for r, x in zip(mine, score):
                n = -(-int(length[r]) // s["page"])
                x = x[:n].copy()
                x[0] = x[n - 1] = np.inf
                best = np.sort(np.argsort(-x, kind="stable")[:s["blocks"]])
                out[r, h, :len(best)] = best
    return dict(blocks=torch.from_numpy(out))


def _exact_sparse(s):
    hkv, p, d = s["k"].shape[1:]
    rows = s["q"].shape[0]
    q = s["q"].double().reshape(rows, hkv, -1, d)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    table, length = s["table"].long(), s["len"].long()
    for h in range(hkv):
        for r0 in range(0, rows, 256):
            r = slice(r0, min(rows, r0 + 256))
            j = s["lists"][r, h].long()                                      # [n, K]
            ids = torch.gather(table[s["req"][r].long()], 1, j.clamp(min=0)).clamp(min=0)
            seen = ((j[..., None] * p + torch.arange(p, device=j.device) < length[r, None, None]) & (j[..., None] >= 0)).flatten(1)
            k, v = (c[ids, h].double().flatten(1, 2) for c in (s["k"], s["v"]))
            x = (torch.bmm(q[r, h], k.transpose(1, 2).contiguous()) / math.sqrt(d)).masked_fill(~seen[:, None], -math.inf)
            lse[r, h] = torch.logsumexp(x, -1)
            o[r, h] = torch.bmm(torch.exp(x - lse[r, h][..., None]), v)
    return dict(o=o.reshape(rows, -1, d), lse=lse.reshape(rows, -1))


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "write": _exact_write, "attend": _exact_attend, "select": _exact_select, "sparse": _exact_sparse}[s["op"]](s)
