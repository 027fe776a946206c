"""The C ABI of the paged attention operators: declared, exported, and bad
arguments refused before anything is enqueued.  CPU only (no compute)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgdn_attn.h")
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1008)    # not 16-byte aligned
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_prefill_chunkwise_amd import build, ops
    if not os.path.exists(ops.LIB_PATH):
        build.build()
    return ops.lib()


def test_header_and_exports(L):
    from gated_deltanet_prefill_chunkwise_amd import ops
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sgdn_\w+)\s*\(", text))
    assert names == {"sgdn_paged_" + n for n in ("release", "plan", "write", "workspace_bytes",
                                                 "attend", "attend_sparse", "select")}
    out = subprocess.run(["nm", "-D", "--defined-only", ops.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert names <= exported and names <= set(ops.EXPORTS)


def test_struct_layout(tmp_path):
    from gated_deltanet_prefill_chunkwise_amd import ops
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "sgdn_attn.h"',
             'int main(void) {', 'printf("%zu", sizeof(sgdn_paged));']
    lines += [f'printf(" %zu", offsetof(sgdn_paged, {f}));' for f, _ in ops.Paged._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(ops.Paged)] + [getattr(ops.Paged, f).offset
                                                for f, _ in ops.Paged._fields_]


def _shape(**kw):
    from gated_deltanet_prefill_chunkwise_amd import ops
    base = dict(rows=4, batch=4, n_q=8, n_kv=2, d=128, page=64, n_pages=100, width=20, max_len=0,
                dtype=1, o_dtype=0)
    base.update(kw)
    return ops.Paged(*[base[n] for n, _ in ops.Paged._fields_])


BAD_SHAPES = [
    (dict(rows=-1), EINVAL), (dict(n_q=0), EINVAL), (dict(n_kv=0), EINVAL), (dict(d=0), EINVAL),
    (dict(page=0), EINVAL), (dict(n_pages=0), EINVAL), (dict(dtype=3), EINVAL),
    (dict(dtype=-1), EINVAL), (dict(d=96), EUNSUPPORTED), (dict(page=48), EUNSUPPORTED),
    (dict(page=256), EUNSUPPORTED), (dict(n_q=9), EUNSUPPORTED),
    (dict(n_pages=1 << 26), EUNSUPPORTED),            # slots pass 31 bits
    (dict(rows=1 << 26), EUNSUPPORTED),
]
BAD_READS = BAD_SHAPES + [
    (dict(batch=0), EINVAL), (dict(width=0), EINVAL), (dict(max_len=-1), EINVAL),
    (dict(max_len=20 * 64 + 1), EINVAL), (dict(width=1 << 26), EUNSUPPORTED),
]


def _attend(L, shape=None, sparse=False, n_blocks=4, ws_bytes=1 << 40, scale=1.0, ldq=8 * 128, **ptr):
    p = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, req=FAKE, length=FAKE, blocks=FAKE, o=FAKE,
             lse=None, ws=FAKE)
    p.update(ptr)
    sp = ctypes.byref(_shape() if shape is None else shape)
    lists = (p["blocks"], n_blocks) if sparse else ()
    fn = L.sgdn_paged_attend_sparse if sparse else L.sgdn_paged_attend
    return fn(sp, p["q"], ldq, p["kc"], p["vc"], p["table"], p["req"], p["length"], *lists, scale,
              p["o"], p["lse"], p["ws"], ws_bytes, None)


def _select(L, shape=None, n_blocks=4, n_sink=1, n_local=1, ws_bytes=1 << 40, ldq=8 * 128, **ptr):
    p = dict(q=FAKE, codes=FAKE, scale=FAKE, table=FAKE, req=FAKE, length=FAKE, blocks=FAKE, ws=FAKE)
    p.update(ptr)
    sp = ctypes.byref(_shape() if shape is None else shape)
    return L.sgdn_paged_select(sp, p["q"], ldq, p["codes"], p["scale"], p["table"], p["req"],
                               p["length"], n_blocks, n_sink, n_local, p["blocks"], p["ws"],
                               ws_bytes, None)


def _write(L, shape=None, ldk=256, ldv=256, **ptr):
    p = dict(k=FAKE, v=FAKE, slot=FAKE, kc=FAKE, vc=FAKE, codes=FAKE, scale=FAKE)
    p.update(ptr)
    sp = ctypes.byref(_shape() if shape is None else shape)
    return L.sgdn_paged_write(sp, p["k"], p["v"], ldk, ldv, p["slot"], p["kc"], p["vc"],
                              p["codes"], p["scale"], None)


@pytest.mark.parametrize("kw, status", BAD_READS)
def test_bad_shapes_of_reading_calls(L, kw, status):
    from gated_deltanet_prefill_chunkwise_amd import ops
    s = _shape(**kw)
    assert _attend(L, s) == status and _attend(L, s, sparse=True) == status
    assert _select(L, s) == status
    assert ops.paged_workspace_bytes(s) == 0 and ops.paged_workspace_bytes(s, 4, True) == 0


@pytest.mark.parametrize("kw, status", BAD_SHAPES)
def test_bad_shapes_of_write(L, kw, status):
    assert _write(L, _shape(**kw)) == status


def test_attend_arguments(L):
    for sparse in (False, True):
        for name in ("q", "kc", "vc", "table", "length", "o", "ws"):
            assert _attend(L, sparse=sparse, **{name: None}) == EINVAL, name
        for name in ("q", "kc", "vc", "o", "ws"):
            assert _attend(L, sparse=sparse, **{name: ODD}) == EINVAL, name
        for scale in (float("nan"), float("inf"), 3e38):               # 3e38 log2(e) passes fp32
            assert _attend(L, sparse=sparse, scale=scale) == EINVAL
        for ldq in (8 * 128 - 8, 8 * 128 + 4, -1024):
            assert _attend(L, sparse=sparse, ldq=ldq) == EINVAL
        assert _attend(L, _shape(o_dtype=5), sparse=sparse) == EINVAL
        assert _attend(L, _shape(rows=5), sparse=sparse, req=None) == EINVAL   # row r is request r
        assert _attend(L, sparse=sparse, ws_bytes=256) == EWORKSPACE
        assert _attend(L, _shape(rows=0), sparse=sparse, q=None, o=None) == 0  # nothing to do
    assert _attend(L, sparse=True, n_blocks=0) == EINVAL
    assert _attend(L, sparse=True, n_blocks=4097) == EUNSUPPORTED
    assert _attend(L, sparse=True, blocks=None) == EINVAL
    assert L.sgdn_paged_attend(None, FAKE, 1024, FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, FAKE, None,
                               FAKE, 1 << 40, None) == EINVAL


def test_more_rows_than_a_launch_holds(L):
    """A launch holds fewer than 2^32 threads."""
    from gated_deltanet_prefill_chunkwise_amd import ops
    for kw in (dict(rows=(1 << 22) - 1, n_q=4, n_kv=4), dict(rows=1 << 21, n_q=80, n_kv=4)):   # 2^24 units of 256
        s = _shape(batch=kw["rows"], **kw)
        for sparse in (False, True):
            assert _attend(L, s, sparse=sparse, ldq=kw["n_q"] * 128) == EUNSUPPORTED
        assert ops.paged_workspace_bytes(s) == 0 and ops.paged_workspace_bytes(s, 4) == 0
    s = _shape(rows=(1 << 22) - 3, batch=4, n_q=4, n_kv=4)
    assert _attend(L, s, q=None, ldq=512) == EINVAL                     # enough room: the next check
    for n, ok in ((1 << 20, False), ((1 << 20) - 4, True)):
        s = _shape(rows=n, batch=4, n_q=4, n_kv=4)
        assert _select(L, s, q=None, ldq=512) == (EINVAL if ok else EUNSUPPORTED)
        assert (ops.paged_workspace_bytes(s, 4, True) > 0) == ok
    assert _write(L, _shape(rows=1 << 28, n_q=1, n_kv=1)) == EUNSUPPORTED


def test_attend_workspace(L):
    from gated_deltanet_prefill_chunkwise_amd import ops
    few = _shape(rows=1, batch=1, width=1000)
    need = ops.paged_workspace_bytes(few)
    assert need > 256 and need % 256 == 0           # split over the length
    assert _attend(L, few, ws_bytes=need - 1) == EWORKSPACE
    assert ops.paged_workspace_bytes(_shape(rows=4096)) == 256     # rows enough: no splits
    assert ops.paged_workspace_bytes(_shape(rows=0)) == 256


def test_select_arguments(L):
    from gated_deltanet_prefill_chunkwise_amd import ops
    for name in ("q", "codes", "scale", "table", "length", "blocks", "ws"):
        assert _select(L, **{name: None}) == EINVAL, name
    for name in ("q", "codes", "ws"):
        assert _select(L, **{name: ODD}) == EINVAL, name
    assert _select(L, n_blocks=0) == EINVAL
    assert _select(L, n_local=0) == EINVAL          # the last block may have no summary
    assert _select(L, n_sink=-1) == EINVAL
    assert _select(L, n_blocks=4, n_sink=2, n_local=3) == EINVAL
    assert _select(L, n_blocks=4097) == EUNSUPPORTED
    assert _select(L, _shape(width=16385)) == EUNSUPPORTED
    assert _select(L, _shape(rows=5), req=None) == EINVAL
    need = ops.paged_workspace_bytes(_shape(), 4, True)
    assert need >= 4 * 2 * 20 * 4
    assert _select(L, ws_bytes=need - 1) == EWORKSPACE
    assert _select(L, _shape(rows=0), q=None) == 0
    assert ops.paged_workspace_bytes(_shape(width=16385), 4, True) == 0


def test_write_arguments(L):
    for name in ("k", "v", "slot", "kc", "vc", "codes", "scale"):    # codes and scale go together
        assert _write(L, **{name: None}) == EINVAL, name
    for name in ("k", "v", "kc", "vc", "codes"):
        assert _write(L, **{name: ODD}) == EINVAL, name
    for ld in (255, 260, -256):
        assert _write(L, ldk=ld) == EINVAL and _write(L, ldv=ld) == EINVAL
    assert _write(L, _shape(rows=0), k=None) == 0


def test_plan_and_release_arguments(L):
    def plan(batch=2, page=64, width=8, rows=4, n_free=9, **ptr):
        names = ("lens", "add", "table", "ring", "pos", "lens_out", "pos_out", "cu", "page_cu",
                 "slot", "req", "length", "status")
        return L.sgdn_paged_plan(batch, page, width, rows, n_free, *[ptr.get(n, FAKE) for n in names], None)

    def release(batch=2, page=64, width=8, n_free=9, **ptr):
        names = ("lens", "done", "table", "ring", "pos", "lens_out", "pos_out")
        return L.sgdn_paged_release(batch, page, width, n_free, *[ptr.get(n, FAKE) for n in names], None)
    for call in (plan, release):
        for kw in (dict(batch=0), dict(page=0), dict(width=0), dict(n_free=0)):
            assert call(**kw) == EINVAL, kw
        assert call(page=24) == EUNSUPPORTED and call(width=1 << 26) == EUNSUPPORTED
        for name in ("lens", "table", "ring", "pos", "lens_out", "pos_out"):
            assert call(**{name: None}) == EINVAL, name
    assert plan(rows=-1) == EINVAL
    for name in ("add", "cu", "page_cu", "slot", "req", "length", "status"):
        assert plan(**{name: None}) == EINVAL, name
    assert release(done=None) == EINVAL


def test_binding_refuses_host_tensors():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    t = torch.zeros((1, 4), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    pos = torch.zeros(2, dtype=torch.int64)
    cache = torch.zeros((2, 1, 16, 64))
    with pytest.raises(ValueError, match="device tensor"):
        ops.paged_plan(one, one, t, one, pos, 16, 1)
    with pytest.raises(ValueError, match="device tensor"):
        ops.paged_release(one, one.byte(), t, one, pos, 16)
    with pytest.raises(ValueError, match="device tensor"):
        ops.paged_write(cache[:, :, 0], cache[:, :, 0], one, cache, cache)
    with pytest.raises(ValueError, match="device tensor"):
        ops.paged_attend(cache[:1, :, 0], cache, cache, t, one)
    with pytest.raises(ValueError, match="device tensor"):
        ops.paged_select(cache[:1, :, 0], torch.zeros((2, 1, 64), dtype=torch.int8),
                         torch.zeros((2, 1)), t, one, 16, 2)
