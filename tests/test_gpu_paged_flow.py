"""The paged attention operators together, as a server uses them: steps of bookkeeping, cache
write, block choice and attention against the fp64 oracle on mirrored arrays; the same captured
into a HIP graph and replayed; other streams; shared workspaces."""
import numpy as np
import pytest

from oracle import paged as ref
from test_gpu_paged import _f64, _i32, _t, check

pytestmark = pytest.mark.gpu

B, W, P, HKV, HQ, D, PAGES = 6, 24, 16, 2, 8, 64, 90
KEEP = 5


class Server:
    """Device state of one attention layer, and the same on the host."""

    def __init__(self, seed, dtype="bf16"):
        import torch
        rng = np.random.default_rng(seed)
        self.rng, self.dtype = rng, dtype
        dt = _t(dtype)
        shape = (PAGES, HKV, P, D)
        # a fresh cache holds anything
        self.k, self.v = torch.full(shape, float("nan"), device="cuda", dtype=dt), torch.full(shape, float("inf"), device="cuda", dtype=dt)
        self.codes = torch.full((PAGES, HKV, D), 77, dtype=torch.int8, device="cuda")
        self.scale = torch.full((PAGES, HKV), float("nan"), device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.ring = _i32(rng.permutation(PAGES))
        self.pos = torch.tensor([0, PAGES], dtype=torch.int64, device="cuda")
        self.h = dict(k=np.zeros(shape), v=np.zeros(shape), codes=np.zeros((PAGES, HKV, D), np.int8), scale=np.full((PAGES, HKV), np.nan),
                      lens=np.zeros(B, np.int32), table=self.table.cpu().numpy(), ring=self.ring.cpu().numpy(), pos=np.array([0, PAGES]))

    def tokens(self, rows):
        import torch
        fused = torch.from_numpy(self.rng.standard_normal((rows, HQ + 2 * HKV, D))).cuda().to(_t(self.dtype))
        return fused[:, :HQ], fused[:, HQ:HQ + HKV], fused[:, HQ + HKV:]

    def step(self, add, done, rows, q, k, v, out=None):
        """One step on the device, everything in place; returns the plan, blocks and outputs."""
        from gated_deltanet_prefill_chunkwise_amd import ops
        if done is not None:
            ops.paged_release(self.lens, done, self.table, self.ring, self.pos, P, lens_out=self.lens, free_pos_out=self.pos)
        plan = ops.paged_plan(self.lens, add, self.table, self.ring, self.pos, P, rows, lens_out=self.lens, free_pos_out=self.pos)
        ops.paged_write(k, v, plan["slot"], self.k, self.v, self.codes, self.scale)
        blocks = ops.paged_select(q, self.codes, self.scale, self.table, plan["row_len"], P, KEEP, row_req=plan["row_req"])
        part = ops.paged_attend_sparse(q, self.k, self.v, self.table, plan["row_len"], blocks, row_req=plan["row_req"], want_lse=True)
        full = ops.paged_attend(q, self.k, self.v, self.table, plan["row_len"], row_req=plan["row_req"], want_lse=True)
        return plan, blocks, part, full

    def mirror(self, add, done, rows, k, v):
        h = self.h
        if done is not None:
            h["lens"], h["ring"], h["pos"] = ref.release(h["lens"], done, h["table"], h["ring"], h["pos"], P)
        plan = ref.plan(h["lens"], add, h["table"], h["ring"], h["pos"], P, rows)
        h["lens"], h["table"], h["pos"] = plan["lens"], plan["table"], plan["free_pos"]
        ref.write(_f64(k), _f64(v), plan["slot"], h["k"], h["v"], h["codes"], h["scale"])
        return plan


def test_serving_steps():
    """Prompts, single tokens, finished requests, a step that does not fit, rows behind the last."""
    import torch
    s = Server(1)
    rows = 260
    for step in range(14):
        add = s.rng.integers(0, 2, B)
        done = np.zeros(B, np.uint8)
        if step % 3 == 0:
            add[s.rng.integers(B)] = s.rng.integers(30, 180)
        if step % 4 == 3:
            b = int(s.rng.integers(B))
            done[b], add[b] = 1, 0
        q, k, v = s.tokens(rows)
        before = s.k.clone(), s.v.clone()
        plan, blocks, part, full = s.step(_i32(add), torch.from_numpy(done).cuda(), rows, q, k, v)
        torch.cuda.synchronize()
        want = s.mirror(add, done, rows, k, v)
        h = s.h
        for n in ("cu", "page_cu", "slot", "row_req", "row_len", "status"):
            assert np.array_equal(plan[n].cpu().numpy(), want[n]), (step, n)
        for n, t in (("lens", s.lens), ("table", s.table), ("ring", s.ring), ("pos", s.pos)):
            assert np.array_equal(t.cpu().numpy(), h[n]), (step, n)
        written = np.zeros(PAGES * P, bool)
        written[want["slot"][want["slot"] >= 0]] = True
        keep = torch.from_numpy(~written.reshape(PAGES, P)).cuda()[:, None, :, None]
        for now, old in zip((s.k, s.v), before):      # nothing but the new slots was written
            same = (now == old) | (torch.isnan(now) & torch.isnan(old))
            assert bool((same | ~keep).all())
        assert np.array_equal(blocks.cpu().numpy(), ref.select(
            _f64(q), h["codes"], h["scale"], h["table"], want["row_len"], P, KEEP, req=want["row_req"])), step
        args = (_f64(q), h["k"], h["v"], h["table"], want["row_len"], want["row_req"])
        check(*full, ref.attend(*args), "f32", s.dtype, D)
        check(*part, ref.attend(*args, blocks=blocks.cpu().numpy()), "f32", s.dtype, D)
    assert (want["status"] == 0).all() and s.h["lens"].max() > 100


def _state(s):
    return [t.clone() for t in (s.k, s.v, s.codes, s.scale, s.lens, s.table, s.ring, s.pos)]


def _load(s, saved):
    for t, x in zip((s.k, s.v, s.codes, s.scale, s.lens, s.table, s.ring, s.pos), saved):
        t.copy_(x)


def _equal(a, b):
    return bool(((a == b) | ((a != a) & (b != b))).all())


def test_captured_step_replays():
    """A decode step of fixed size, captured once (everything in place, so that each replay is the
    next token); replays with eager work and synchronisation between, each against the eager run."""
    import torch
    s = Server(2)
    q, k, v = s.tokens(200)
    s.step(_i32([40, 3, 90, 0, 15, 31]), None, 200, q, k, v)
    rows = 8                                          # two rows are padding
    add = _i32([1, 1, 1, 1, 1, 1])
    q, k, v = (t.contiguous() for t in s.tokens(rows))
    qs, ks = ([t.clone()] + [torch.randn_like(t) for _ in range(4)] for t in (q, k))
    saved = _state(s)
    wants = []
    for i in range(5):
        q.copy_(qs[i])
        k.copy_(ks[i])
        plan, blocks, part, full = s.step(add, None, rows, q, k, v)
        wants.append([t.clone() for t in (*plan.values(), blocks, *part, *full)] + _state(s))
    torch.cuda.synchronize()
    _load(s, saved)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                     # warm-up outside the capture
        s.step(add, None, rows, q, k, v)
    torch.cuda.current_stream().wait_stream(side)
    _load(s, saved)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan, blocks, part, full = s.step(add, None, rows, q, k, v)
    _load(s, saved)
    for i in range(5):
        q.copy_(qs[i])
        k.copy_(ks[i])
        g.replay()
        torch.cuda.synchronize()
        got = [*plan.values(), blocks, *part, *full] + _state(s)
        for a, b in zip(got, wants[i]):
            assert _equal(a, b), i
        torch.ones(1 << 20, device="cuda").sum().item()


def _prompt_call(seed, rows=4200):
    import torch
    rng = np.random.default_rng(seed)
    n = rows + 50
    nb = -(-n // P)
    g = lambda *shape: torch.from_numpy(rng.standard_normal(shape)).cuda().bfloat16()
    k, v, q = g(nb, 1, P, D), g(nb, 1, P, D), g(rows, 8, D)
    table, length = rng.permutation(nb)[None], 51 + np.arange(rows)
    pick = np.sort(rng.integers(0, 3, (rows, 1, 4)) + np.arange(4) * 3 % 4, axis=-1)
    lists = np.where(pick < -(-length // P)[:, None, None], pick, -1)
    return dict(q=q, k_cache=k, v_cache=v, table=_i32(table), row_len=_i32(length), blocks=_i32(lists), row_req=_i32(np.zeros(rows)))


def test_captured_turnover():
    """Release and a plan of more rows than one launch takes, in place, replayed on other states."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    n, w, page, rows, pages = 50, 12, 32, 3000, 700
    rng = np.random.default_rng(31)

    def state():
        lens = rng.integers(0, 300, n).astype(np.int32)
        table, ring, ids = np.full((n, w), -1, np.int32), np.zeros(pages, np.int32), rng.permutation(pages)
        held = -(-lens // page)
        for b in range(n):
            table[b, :held[b]], ids = ids[:held[b]], ids[held[b]:]
        taken = int(rng.integers(0, 10 * pages))
        ring[(taken + np.arange(len(ids))) % pages] = ids
        done = (rng.random(n) < 0.3).astype(np.uint8)
        add = np.where(done, 0, rng.integers(0, 90, n)).astype(np.int32)
        return dict(lens=lens, done=done, add=add, table=table, ring=ring, pos=np.array([taken, taken + len(ids)], np.int64))

    d = {k: torch.from_numpy(x).cuda() for k, x in state().items()}

    def call():
        ops.paged_release(d["lens"], d["done"], d["table"], d["ring"], d["pos"], page, lens_out=d["lens"], free_pos_out=d["pos"])
        return ops.paged_plan(d["lens"], d["add"], d["table"], d["ring"], d["pos"], page, rows, lens_out=d["lens"], free_pos_out=d["pos"])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(5):
        s = state()
        for k, x in s.items():
            d[k].copy_(torch.from_numpy(x))
        graph.replay()
        torch.cuda.synchronize()
        lens, ring, pos = ref.release(s["lens"], s["done"], s["table"], s["ring"], s["pos"], page)
        want = ref.plan(lens, s["add"], s["table"], ring, pos, page, rows)
        for k in ("lens", "cu", "page_cu", "slot", "row_req", "row_len", "status", "free_pos"):
            assert np.array_equal(got[k].cpu().numpy(), want[k]), k
        assert np.array_equal(d["table"].cpu().numpy(), want["table"]) and np.array_equal(d["ring"].cpu().numpy(), ring)
        torch.ones(1 << 20, device="cuda").sum().item()


def test_captured_prompts_and_shared_workspace():
    """Tiles, single rows and splits in two graphs that use one workspace in turn."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    a = _prompt_call(3)
    b = {n: t for n, t in _prompt_call(4, 900).items()}
    c = {n: (t[:2].contiguous() if n in ("q", "row_len", "row_req") else t) for n, t in b.items() if n != "blocks"}
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    calls = (lambda: ops.paged_attend_sparse(**a, workspace=ws), lambda: ops.paged_attend(**c, workspace=ws),
             lambda: ops.paged_attend_sparse(**b, workspace=ws))
    want = [f()[0].clone() for f in calls]
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f()[0])
        graphs.append(g)
    for i in range(4):
        for j in (0, 1, 2, 1, 0):
            outs[j].fill_(7.0)
            ws.fill_(i * 50 + j)                      # what it held does not matter
            graphs[j].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[j], want[j]), (i, j)


def test_other_stream_and_two_at_once():
    """Calls on a stream that is not the current one, and on two streams at once; the tensors
    are dropped while the work is in flight."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    calls = [_prompt_call(i, 400 + 300 * i) for i in range(3)]
    want = [ops.paged_attend_sparse(**c)[0].clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for turn in range(6):
        for c, s in zip(calls, streams):
            copies = {n: t.clone() for n, t in c.items()}
            s.wait_stream(torch.cuda.current_stream())
            outs.append(ops.paged_attend_sparse(**copies, stream=s)[0])
            del copies                                # their memory goes back while the call runs
            torch.full((1 << 22,), float("nan"), device="cuda")
    for s in streams:
        s.synchronize()
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 3]), i


def test_other_stream_bookkeeping():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    s = Server(5)
    add = _i32([20, 0, 33, 1, 5, 60])
    want = ref.plan(s.h["lens"], [20, 0, 33, 1, 5, 60], s.h["table"], s.h["ring"], s.h["pos"], P, 130)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ops.paged_plan(s.lens, add, s.table, s.ring, s.pos, P, 130, stream=side)
    lens, pos = ops.paged_release(got["lens"], _i32([1] * B).byte(), s.table, s.ring, got["free_pos"], P, stream=side)
    side.synchronize()
    for n in ("slot", "row_req", "row_len", "cu", "status", "free_pos"):
        assert np.array_equal(got[n].cpu().numpy(), want[n]), n
    assert not lens.any() and int(pos[1] - pos[0]) == PAGES
    with pytest.raises(ValueError):
        ops.paged_plan(s.lens, add.cpu(), s.table, s.ring, s.pos, P, 130)


def test_repeats_are_identical():
    """No result depends on the order in which waves or workgroups finish."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    a = _prompt_call(7)
    one = {n: (t[-3:].contiguous() if n in ("q", "row_len", "row_req") else t) for n, t in a.items() if n != "blocks"}
    first = ops.paged_attend_sparse(**a, want_lse=True), ops.paged_attend(**one, want_lse=True)
    for _ in range(5):
        again = ops.paged_attend_sparse(**a, want_lse=True), ops.paged_attend(**one, want_lse=True)
        for x, y in zip(first, again):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
