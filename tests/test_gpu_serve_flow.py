"""A served layer's step with the rotation and the attention of chunks: plan, norm and rotation in
place, cache write, attention, against the fp64 oracle on mirrored arrays; the same captured into a
HIP graph and replayed; graphs that share a workspace; other streams; equal bits in equal calls."""
import numpy as np
import pytest

from oracle import paged as pref
from oracle import serve as ref
from test_gpu_chunk import check as check_chunk
from test_gpu_paged import Case, _f64, _i32, _t
from test_gpu_paged_flow import _equal
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu

B, W, P, HKV, HQ, D, ROT, PAGES = 5, 20, 16, 2, 8, 64, 32, 90


class Layer:
    """Device state of one attention layer, and the same on the host."""

    def __init__(self, seed, dtype="bf16", layout="half", out="f32"):
        import torch
        from gated_deltanet_prefill_chunkwise_amd import ops
        self.rng, self.dtype, self.layout, self.out = np.random.default_rng(seed), dtype, layout, out
        shape = (PAGES, HKV, P, D)
        self.k, self.v = (torch.full(shape, x, device="cuda", dtype=_t(dtype)) for x in (float("nan"), float("inf")))
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.ring = _i32(self.rng.permutation(PAGES))
        self.pos = torch.tensor([0, PAGES], dtype=torch.int64, device="cuda")
        self.wq, self.wk = (torch.from_numpy(self.rng.standard_normal(D) * 0.2).cuda().to(_t(dtype)) for _ in range(2))
        f, self.m = ops.rope_freqs(ROT, scaling="by_pair", factor=4.0, original=64)
        self.f = f.cuda()
        self.h = dict(k=np.zeros(shape), v=np.zeros(shape), lens=np.zeros(B, np.int32), table=self.table.cpu().numpy(),
                      ring=self.ring.cpu().numpy(), pos=np.array([0, PAGES]))

    def tokens(self, rows):
        """A projection's output: each query head with a gate behind it, keys, values."""
        import torch
        return torch.from_numpy(self.rng.standard_normal((rows, 2 * HQ + 2 * HKV, D))).cuda().to(_t(self.dtype))

    def split(self, x):
        return x[:, :2 * HQ:2], x[:, 2 * HQ:2 * HQ + HKV], x[:, 2 * HQ + HKV:]

    def step(self, x, add):
        """Everything in place but the queries, which attention takes whole; (plan, q, k, o, lse)."""
        from gated_deltanet_prefill_chunkwise_amd import ops
        rows = x.shape[0]
        plan = ops.paged_plan(self.lens, add, self.table, self.ring, self.pos, P, rows, lens_out=self.lens, free_pos_out=self.pos)
        q, k, v = self.split(x)
        whole = x.new_zeros((rows, HQ, D))
        ops.norm_rope(q, k, self.wq, self.wk, plan["row_len"], self.f, layout=self.layout, magnitude=self.m, weight_offset=1.0,
                      pos_offset=-1, q_out=whole, k_out=k)
        ops.paged_write(k, v, plan["slot"], self.k, self.v)
        o, lse = ops.paged_attend_chunk(whole, self.k, self.v, self.table, plan["cu"], self.lens, out_dtype=_t(self.out), want_lse=True)
        return plan, whole, k, o, lse

    def state(self):
        return [self.k, self.v, self.lens, self.table, self.ring, self.pos]


@pytest.mark.parametrize("dtype, out, layout", [("bf16", "bf16", "half"), ("f16", "f32", "interleaved"), ("f32", "f32", "half")])
def test_serving_steps(dtype, out, layout):
    """Prompts, pieces of prompts, single tokens, requests without rows, rows behind the last."""
    s, rows = Layer(1, dtype, layout, out), 230
    for step in range(8):
        add = s.rng.integers(0, 2, B)
        if step % 2 == 0:
            add[s.rng.integers(B)] = s.rng.integers(20, 90)
        if step == 5:
            add[:] = 0                                # nothing to do
        x = s.tokens(rows)
        before = x.clone()
        plan, q, k, o, lse = s.step(x, _i32(add))
        h = s.h
        want = pref.plan(h["lens"], add, h["table"], h["ring"], h["pos"], P, rows)
        assert (want["status"] == 0).all()
        h["lens"], h["table"], h["pos"] = want["lens"], want["table"], want["free_pos"]
        live, place = want["row_len"] > 0, want["row_len"][want["row_len"] > 0] - 1
        q0, k0, v0 = s.split(before)
        for got, was, w in ((q, q0, s.wq), (k, k0, s.wk)):
            normed = ref.norm(_f64(was)[live], _f64(w), 1.0, float(np.float32(1e-6)))
            y, size = ref.rope(normed, place, _f64(s.f), layout, s.m)
            if live.any():
                check_rope(got[np.flatnonzero(live)], y, size, dtype, True)
            assert bool((got[np.flatnonzero(~live)] == (was if got is k else 0 * was)[np.flatnonzero(~live)]).all())
        pref.write(_f64(k), _f64(v0), want["slot"], h["k"], h["v"])
        a = ref.attend_chunk(_f64(q), h["k"], h["v"], h["table"], want["cu"], h["lens"])
        a[2]["vmax"] = np.full(a[1].shape, np.abs(h["v"]).max())
        check_chunk(o, lse, a, out, dtype, D)
        assert bool((s.split(x)[0] == q0).all() and (s.split(x)[2] == v0).all())


def test_captured_step_replays():
    """A step of pieces and single tokens captured once: each replay is the next step, with eager
    work and synchronisation between, against the eager run."""
    import torch
    s = Layer(2)
    s.step(s.tokens(200), _i32([40, 3, 60, 0, 15]))
    x, add = s.tokens(40), _i32([1, 9, 1, 20, 2])     # seven rows are padding
    xs = [s.tokens(40) for _ in range(4)]
    saved = [t.clone() for t in s.state()]

    def load():
        for t, w in zip(s.state(), saved):
            t.copy_(w)

    wants = []
    for y in xs:
        x.copy_(y)
        plan, *rest = s.step(x, add)
        wants.append([t.clone() for t in (*plan.values(), *rest, *s.state())])
    torch.cuda.synchronize()
    load()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan, *rest = s.step(x, add)
    load()
    for i, y in enumerate(xs):
        x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((*plan.values(), *rest, *s.state()), wants[i]):
            assert _equal(a, b), i
        torch.ones(1 << 20, device="cuda").sum().item()


def _call(seed, step, Hq=8, Hkv=2, dtype="bf16", behind=3):
    new, cached = np.array(step).T
    cu, lens = np.concatenate([[0], np.cumsum(new)]), new + cached
    c = Case(seed, lens, Hq, Hkv, 64, 16, dtype)
    return dict(q=c.q(int(cu[-1]) + behind), k_cache=c.k, v_cache=c.v, table=_i32(c.table), cu=_i32(cu), lens=_i32(lens))


CALLS = [dict(step=[(70, 3000), (1, 500), (0, 9), (300, 0)]), dict(step=[(1, 900)] * 40), dict(step=[(33, 700), (2, 2)], dtype="f32"),
         dict(step=[(5, 4000)], Hq=32, Hkv=8, behind=0)]


def test_graphs_that_share_a_workspace():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    calls = [_call(i, **kw) for i, kw in enumerate(CALLS)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = [ops.paged_attend_chunk(**c)[0].clone() for c in calls]
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.paged_attend_chunk(**c, workspace=ws)[0])
        graphs.append(g)
    for i in range(3):
        for j in (0, 1, 2, 3, 1, 0):
            outs[j].fill_(7.0)
            ws.fill_(i * 80 + j)                      # what it held does not matter
            graphs[j].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[j], want[j]), (i, j)
        torch.ones(1 << 20, device="cuda").sum().item()


def test_other_stream_and_several_at_once():
    """Calls on streams that are not the current one, at the same time; the tensors are dropped
    while the work is in flight."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    f = ops.rope_freqs(64)[0].cuda()

    def run(c, **kw):
        place = c["table"].new_tensor(range(c["q"].shape[0]))
        q, _ = ops.rope(c["q"], None, place, f, **kw)
        return ops.paged_attend_chunk(**dict(c, q=q), **kw)[0]

    calls = [_call(10 + i, **kw) for i, kw in enumerate(CALLS)]
    want = [run(c).clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = []
    for turn in range(5):
        for c, s in zip(calls, streams):
            copies = {n: t.clone() for n, t in c.items()}
            place = torch.arange(c["q"].shape[0], dtype=torch.int32, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            q, _ = ops.rope(copies["q"], None, place, f, stream=s)
            copies["q"] = q
            outs.append(ops.paged_attend_chunk(**copies, stream=s)[0])
            del copies, q, place                      # their memory goes back while the calls run
            torch.full((1 << 22,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % len(calls)]), i


@pytest.mark.parametrize("kw", CALLS)
def test_equal_calls_give_equal_bits(kw):
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = _call(3, **kw)
    first = [t.clone() for t in ops.paged_attend_chunk(**c, want_lse=True)]
    for _ in range(4):
        for a, b in zip(first, ops.paged_attend_chunk(**c, want_lse=True)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cu", [[0, 50, 20, 60, 80], [90, 60, 30, 10, 0], [-5, 10, 10, 70, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 40, 41]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_starts_that_fall_stay_inside(cu, dtype):
    """Row starts that fall or lie outside give no meaning to rows, but nothing outside o and lse is written."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    c = _call(4, [(20, 100), (20, 7), (20, 300), (20, 0)], dtype=dtype, behind=0)
    rows = c["q"].shape[0]
    pad = 64
    o = torch.full((rows + 2 * pad, 8, 64), 7.0, device="cuda")
    lse = torch.full((rows + 2 * pad, 8), 7.0, device="cuda")
    need = ops.paged_chunk_workspace_bytes(ops._paged(rows, 8, c["k_cache"].shape, c["q"].dtype, torch.float32, *c["table"].shape, None))
    ws = torch.full((need + 512,), 99, dtype=torch.uint8, device="cuda")
    ops.paged_attend_chunk(**dict(c, cu=_i32(cu)), o=o[pad:-pad], lse=lse[pad:-pad], workspace=ws[256:-256])
    for t in (o[:pad], o[-pad:], lse[:pad], lse[-pad:]):
        assert bool((t == 7.0).all())
    assert bool((ws[:256] == 99).all() and (ws[-256:] == 99).all())
