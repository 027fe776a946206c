"""Operators around the paged cache: their plain forms, their 64-bit definitions and the cases they
are measured on.

What a softmax attention layer that is served beside the gated linear layers does with the output of
its joint projection before and after the cache write:

  rope    rotary positions of queries and keys
  norm    a norm of every query and key head, and the rotation, in one pass
  chunk   attention of chunks of new tokens (prompts, pieces of them, single tokens) over the cache

Notation: R rows (new tokens), Hq query heads in groups of G over Hkv key/value heads, D elements
per head, P tokens per page.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # The one token of a lone request: latency alone.
        dict(name="rope_one", op="rope", batch=1, new=1, cached=4096, hq=32, hkv=8, d=128, rot=128, layout="half", stretch=1, type="bf16"),
        # A batch of prompts, ragged, at far positions of a context stretched eightfold.
        dict(name="rope_prompts", op="rope", batch=8, new=8192, cached=1000000, hq=32, hkv=8, d=128, rot=128, layout="interleaved", stretch=8, type="bf16"),
        # Everything odd: 32-bit, part of the head, halves that end inside an access.
        dict(name="rope_odd", op="rope", batch=5, new=401, cached=5001, hq=15, hkv=3, d=64, rot=20, layout="half", stretch=2, type="f32"),
        # One token for each of 128 running requests, few and wide heads, a quarter rotated.
        dict(name="norm_step", op="norm", batch=128, new=1, cached=32000, hq=16, hkv=2, d=256, rot=64, layout="half", stretch=1, type="bf16"),
        # The same batch of prompts with normed heads.
        dict(name="norm_prompts", op="norm", batch=8, new=8192, cached=4096, hq=32, hkv=8, d=128, rot=128, layout="half", stretch=1, type="bf16"),
        # Odd sizes: heads of 80, one key head, 16-bit floats.
        dict(name="norm_odd", op="norm", batch=3, new=777, cached=100, hq=7, hkv=1, d=80, rot=40, layout="interleaved", stretch=4, type="f16"),
        # A few drafted tokens of a lone request.
        dict(name="chunk_short", op="chunk", batch=1, new=16, singles=0, pad=0, cached=4096, hq=32, hkv=8, d=128, page=64, type="bf16"),
        # One prompt from its first token.
        dict(name="chunk_prompt", op="chunk", batch=1, new=8192, singles=0, pad=0, cached=0, hq=32, hkv=8, d=128, page=64, type="bf16"),
        # The last piece of a prompt at the longest context, few and wide heads.
        dict(name="chunk_long", op="chunk", batch=1, new=512, singles=0, pad=0, cached=131072, hq=16, hkv=2, d=256, page=64, type="f16"),
        # A serving step: 60 running requests, pieces of four prompts, and the rows behind them of a step of fixed size.
        dict(name="chunk_mixed", op="chunk", batch=4, new=1024, singles=60, pad=100, cached=16384, hq=32, hkv=8, d=128, page=64, type="bf16"),
        # A batch of ragged prompts, a key head for each query head.
        dict(name="chunk_prompts", op="chunk", batch=8, new=2048, singles=0, pad=0, cached=1000, hq=16, hkv=16, d=64, page=32, type="bf16"),
        # Everything odd: 32-bit, small pages, five heads a group, uneven lengths.
        dict(name="chunk_odd", op="chunk", batch=3, new=301, singles=2, pad=5, cached=1501, hq=15, hkv=3, d=64, page=16, type="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / (50 if case["type"] != "f32" else 8))


def draw(rng):
    op = rng.choice(["rope", "norm", "chunk"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        case = _draw_chunk(rng) if op == "chunk" else _draw_heads(rng, op)
        # scores that the plain form writes down: no more than the largest listed case's
        if _cost(case) <= most and (op != "chunk" or case["batch"] * case["hq"] * case["new"] * (case["new"] + case["cached"]) <= 1 << 31):
            return case


def _draw_heads(rng, op):
    d = rng.choice([32, 64, 80, 96, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    rot = rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)])
    new = rng.choice([1, _log(rng, 1, 8192)])
    batch = _log(rng, 1, max(1, min(512, (1 << 29) // (new * (hq + hkv) * d * BYTES[kind]))))
    return dict(op=op, batch=batch, new=new, cached=_log(rng, 1, 1000000), hq=hq, hkv=hkv, d=d, rot=rot,
                layout=rng.choice(["half", "interleaved"]), stretch=rng.choice([1, 2, 4, 8, 32]), type=kind)


def _draw_chunk(rng):
    page = rng.choice([16, 32, 64, 64, 128])
    hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128, 256])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    new = _log(rng, 2, 8192)
    cached = rng.choice([0, _log(rng, 1, 131072)])
    row = hkv * d * BYTES[kind] * 2
    batch = _log(rng, 1, max(1, min(16, (1 << 30) // ((new + cached) * row))))
    singles = rng.choice([0, _log(rng, 1, max(1, min(128, (1 << 31) // ((1 + cached) * row))))])
    return dict(op="chunk", batch=batch, new=new, singles=singles, pad=rng.choice([0, _log(rng, 1, 200)]), cached=cached, hq=hq, hkv=hkv, d=d,
                page=page, type=kind)


# What a case is made of ------------------------------------------------------------------------


def _lengths(case):
    """Cached lengths (before the step) and new tokens of each request: ragged, the first of the chunks the
    longest, and the requests with a single token between them.  They belong to the case, so that its outputs have one shape."""
    rng = np.random.default_rng([case["batch"], case["cached"], case["new"], 19])
    b, n, one = case["batch"], case["new"], case.get("singles", 0)
    cached = (case["cached"] * rng.uniform(0.25, 1.0, b + one)).astype(np.int64)
    new = np.maximum(1, (n * rng.uniform(0.3, 1.0, b + one)).astype(np.int64))
    cached[0], new[0] = case["cached"], n
    new[b:] = 1
    order = np.concatenate([[0], 1 + rng.permutation(b + one - 1)]) if one else np.arange(b)
    return cached[order], new[order], order < b


def _int32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _table(lengths, page, seed, spare=8):
    """A block table whose rows are pages in random order, and the number of pages of the cache."""
    blocks = -(-lengths // page)
    total = int(blocks.sum())
    order = np.random.default_rng([seed, 23]).permutation(total + spare)[:total]
    width = max(1, int(blocks.max()))
    table = np.full((len(lengths), width), -1, np.int32)
    table[np.arange(width)[None, :] < blocks[:, None]] = order
    return table, total + spare


def _normal(shape, g, kind):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
    return x.to(TYPES[kind])


def _frequencies(rot, stretch):
    """Radians per token of each pair.  Where the context is stretched, pairs that turn less than once in
    8192 tokens are slowed by the factor, those that turn more than 4 times are not, those between in part."""
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    if stretch == 1:
        return f
    turns = f * 8192 / (2 * math.pi)
    keep = np.clip((turns - 1.0) / 3.0, 0.0, 1.0)
    return f * (keep + (1.0 - keep) / stretch)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cached, new, chunks = _lengths(case)
    hq, hkv, d, kind = case["hq"], case["hkv"], case["d"], case["type"]
    first = np.cumsum(new) - new
    total = int(new.sum())
    if case["op"] != "chunk":
        pos = np.repeat(cached - first, new) + np.arange(total)
        fused = _normal((total, hq + 2 * hkv, d), g, kind)          # one projection's output: q, k, v
        s = dict(op=case["op"], q=fused[:, :hq], k=fused[:, hq:hq + hkv], pos=_int32(pos), layout=case["layout"],
                 freqs=torch.from_numpy(_frequencies(case["rot"], case["stretch"])).cuda(),
                 magnitude=1.0 + 0.1 * math.log(case["stretch"]))
        if case["op"] == "norm":
            s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[kind]), (
                1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[kind])
            s["eps"] = 1e-6
        return s
    p, lens = case["page"], cached + new
    table, pages = _table(lens, p, seed)
    k, v = _normal((pages, hkv, p, d), g, kind), _normal((pages, hkv, p, d), g, kind)
    q = _normal((total + case["pad"], hq, d), g, kind)
    s = dict(op="chunk", q=q, k=k, v=v, table=_int32(table), cu=_int32(np.concatenate([[0], np.cumsum(new)])), lens=_int32(lens),
             most=int(lens.max()), groups=[])
    for mine in (chunks, ~chunks):                                  # padded together in the plain form
        if mine.any():
            s["groups"].append((torch.from_numpy(np.nonzero(mine)[0]).cuda(), int(new[mine].max()), int(lens[mine].max())))
    return s


# The plain forms -------------------------------------------------------------------------------


def _turn_plain(x, cos, sin, layout):
    """x [R, H, D] in 32 bits, cos and sin [R, 1, rot / 2]."""
    half = cos.shape[-1]
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _norm_plain(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _heads_plain(s):
    angle = s["pos"].double()[:, None, None] * s["freqs"]           # in 64 bits: far positions
    cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
    q, k = s["q"].float(), s["k"].float()
    if s["op"] == "norm":
        q, k = _norm_plain(q, s["wq"], s["eps"]), _norm_plain(k, s["wk"], s["eps"])
    return dict(q=_turn_plain(q, cos, sin, s["layout"]).to(s["q"].dtype), k=_turn_plain(k, cos, sin, s["layout"]).to(s["k"].dtype))


def _group_plain(s, mine, longest, most, o, lse):
    """The requests `mine`, padded to `longest` new tokens and `most` tokens in all; o and lse end with a row that takes what is padding."""
    q, kc, vc = s["q"], s["k"], s["v"]
    pages, hkv, p, d = kc.shape
    b, g = mine.numel(), q.shape[1] // hkv
    n = -(-most // p)
    table = s["table"][mine][:, :n].long().clamp(min=0)
    k = kc[table].float().transpose(1, 2).reshape(b, hkv, n * p, d)
    v = vc[table].float().transpose(1, 2).reshape(b, hkv, n * p, d)
    first, count = s["cu"][mine].long(), (s["cu"][mine + 1] - s["cu"][mine]).long()
    i = torch.arange(longest, device=q.device)
    real = i < count[:, None]
    row = torch.where(real, first[:, None] + i, q.shape[0])
    sees = torch.where(real, s["lens"][mine].long()[:, None] - count[:, None] + i + 1, 0)
    x = q[row.clamp(max=q.shape[0] - 1)].float().reshape(b, longest, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, longest * g, d)
    x = torch.matmul(x, k.transpose(-1, -2).contiguous()).mul_(1.0 / math.sqrt(d)).reshape(b, hkv, longest, g, n * p)
    x.masked_fill_(torch.arange(n * p, device=q.device) >= sees[:, None, :, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    some = (sees > 0)[:, None, :, None, None]
    y = torch.matmul(x.reshape(b, hkv, longest * g, n * p), v).reshape(b, hkv, longest, g, d)
    y = torch.where(some, y / total, 0.0)
    z = torch.where(some, top + torch.log(total), -math.inf)
    o[row] = y.permute(0, 2, 1, 3, 4).reshape(b, longest, hkv * g, d)
    lse[row] = z.permute(0, 2, 1, 3, 4).reshape(b, longest, hkv * g)


def _chunk_plain(s):
    q = s["q"]
    o = torch.zeros((q.shape[0] + 1,) + q.shape[1:], device=q.device)
    lse = torch.full((q.shape[0] + 1, q.shape[1]), -math.inf, device=q.device)
    _group_plain(s, *s["groups"][0], o, lse)
    if len(s["groups"]) > 1:
        _group_plain(s, *s["groups"][1], o, lse)
    return dict(o=o[:-1].to(q.dtype), lse=lse[:-1])


# One pass --------------------------------------------------------------------------------------


def _run_own(s):
    from gated_deltanet_prefill_chunkwise_amd import ops
    if s["op"] == "rope":
        q, k = ops.rope(s["q"], s["k"], s["pos"], s["freqs"], layout=s["layout"], magnitude=s["magnitude"])
        return dict(q=q, k=k)
    if s["op"] == "norm":
        q, k = ops.norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"], layout=s["layout"], magnitude=s["magnitude"], eps=s["eps"])
        return dict(q=q, k=k)
    o, lse = ops.paged_attend_chunk(s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], max_len=s["most"], out_dtype=s["q"].dtype, want_lse=True)
    return dict(o=o, lse=lse)


def run(state):
    if own:
        return _run_own(state)
    return _chunk_plain(state) if state["op"] == "chunk" else _heads_plain(state)


# What a pass cannot do without -----------------------------------------------------------------


def work(case):
    cached, new, _ = _lengths(case)
    rows, e, hq, hkv, d = float(new.sum()), BYTES[case["type"]], case["hq"], case["hkv"], case["d"]
    if case["op"] != "chunk":
        heads = rows * (hq + hkv)
        return {"bytes": 2 * heads * d * e + 4 * rows + 4 * case["rot"], "flops": heads * (3 * case["rot"] + (4 * d if case["op"] == "norm" else 0))}
    seen = float((new * cached + new * (new + 1) // 2).sum())       # (row, key) pairs
    tokens = float((cached + new).sum())
    rows += case["pad"]
    return {"bytes": 2 * tokens * hkv * d * e + rows * hq * (2 * d * e + 4) + 4 * tokens / case["page"], "flops": 4.0 * seen * hq * d}


# The definitions, in 64 bits --------------------------------------------------------------------


def _exact_heads(s):
    """Each pair is a complex number, turned by its angle."""
    half = s["freqs"].numel()
    unit = torch.polar(torch.full((), float(s["magnitude"]), dtype=torch.float64, device="cuda"), torch.outer(s["pos"].double(), s["freqs"]))
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if s["op"] == "norm":
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * s["w" + name].double()
        y = x.clone()
        place = torch.arange(half, device="cuda")
        re, im = (place, place + half) if s["layout"] == "half" else (2 * place, 2 * place + 1)
        z = torch.complex(x[..., re], x[..., im]) * unit[:, None, :]
        y[..., re], y[..., im] = z.real, z.imag
        out[name] = y
    return out


def _exact_chunk(s):
    hkv, p, d = s["k"].shape[1:]
    q = s["q"].double()
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    g = q.shape[1] // hkv
    for b, n in enumerate(lens):
        ids = s["table"][b, :-(-n // p)].long()
        for h in range(hkv):
            k, v = (c[ids, h].double().reshape(-1, d)[:n] for c in (s["k"], s["v"]))
            for r0 in range(cu[b], cu[b + 1], 1024):
                r1 = min(cu[b + 1], r0 + 1024)
                sees = torch.arange(n - cu[b + 1] + r0, n - cu[b + 1] + r1, device=q.device)   # last key of each row
                top = n - cu[b + 1] + r1                                                       # keys that any of them sees
                x = (q[r0:r1, h * g:(h + 1) * g].reshape(-1, d) @ k[:top].T.contiguous() / math.sqrt(d)).reshape(r1 - r0, g, top)
                x = x.masked_fill(torch.arange(top, device=q.device) > sees[:, None, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[r0:r1, h * g:(h + 1) * g] = z
                o[r0:r1, h * g:(h + 1) * g] = (torch.exp(x - z[..., None]).reshape(-1, top) @ v[:top]).reshape(r1 - r0, g, d)
    return dict(o=o, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_chunk(s) if case["op"] == "chunk" else _exact_heads(s)
