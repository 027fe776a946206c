"""The C ABI of the operators around the paged cache: declared, exported, frequencies against the
oracle, and bad arguments refused before anything is enqueued.  CPU only (no compute)."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import serve as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgdn_serve.h")
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
    assert names == {"sgdn_" + n for n in ("rope_freqs", "rope", "norm_rope", "paged_attend_chunk",
                                           "paged_chunk_workspace_bytes")}
    out = subprocess.run(["nm", "-D", "--defined-only", ops.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert names <= exported and names <= set(ops.EXPORTS)


def test_struct_layout(tmp_path):
    from gated_deltanet_prefill_chunkwise_amd import ops
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "sgdn_serve.h"',
             'int main(void) {', 'printf("%zu %zu", sizeof(sgdn_rope_shape), sizeof(sgdn_strides));']
    lines += [f'printf(" %zu", offsetof(sgdn_rope_shape, {f}));' for f, _ in ops.RopeShape._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(ops.RopeShape), ctypes.sizeof(ops.Strides)] + [
        getattr(ops.RopeShape, f).offset for f, _ in ops.RopeShape._fields_]


# frequencies ----------------------------------------------------------------


@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=8), dict(scaling="base", factor=4),
    dict(scaling="by_pair", factor=8, original=4096), dict(scaling="by_pair", factor=1, original=4096),
    dict(scaling="by_pair", factor=40, original=100, low=1, high=1.0001),      # one pair's border: a = b
    dict(scaling="by_turns", factor=8, original=8192, low=1, high=4),
])
@pytest.mark.parametrize("rot, base", [(64, 10000.0), (128, 500000.0), (20, 10000.0), (4, 10.0), (256, 1e6)])
def test_freqs(rot, base, kw):
    """Both sides form them with a few operations in fp64: 2^-45 of the value covers 2^7 roundings,
    the power's own among them (its exponent is at most 2 ln(base) < 2^5 times a relative 2^-52)."""
    from gated_deltanet_prefill_chunkwise_amd import ops
    f, m = ops.rope_freqs(rot, base, **kw)
    want, wm = ref.freqs(rot, base, **kw)
    assert f.dtype.is_floating_point and f.shape == (rot // 2,)
    assert np.all(np.abs(f.numpy() - want) <= 2.0 ** -45 * want) and abs(m - wm) < 1e-14


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=-2), dict(rot=7), dict(rot=258), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
    dict(scaling="base", rot=2, factor=2), dict(scaling="by_pair", factor=2), dict(scaling="by_turns", factor=2, original=-1),
    dict(scaling="by_turns", factor=2, original=4096, low=0.0), dict(scaling="by_turns", factor=2, original=4096, low=4, high=4),
    dict(scaling="by_pair", factor=float("inf"), original=4096),
])
def test_freqs_refused(kw):
    from gated_deltanet_prefill_chunkwise_amd import ops
    with pytest.raises(ops.SgdnError) as e:
        ops.rope_freqs(**dict(dict(rot=64), **kw))
    assert e.value.status == EINVAL


def test_freqs_arguments(L):
    from gated_deltanet_prefill_chunkwise_amd import ops
    with pytest.raises(ValueError):
        ops.rope_freqs(64, scaling="other")
    with pytest.raises(ValueError):
        ops.rope_freqs((1 << 32) + 64)
    out = (ctypes.c_double * 128)()
    m = ctypes.c_double()
    for args in ((64, 5), (64, -1)):
        assert L.sgdn_rope_freqs(*args, 1e4, 2.0, 4096.0, 1.0, 4.0, out, ctypes.addressof(m)) == EINVAL
    assert L.sgdn_rope_freqs(64, 0, 1e4, 1.0, 0.0, 1.0, 4.0, None, ctypes.addressof(m)) == EINVAL
    assert L.sgdn_rope_freqs(64, 0, 1e4, 1.0, 0.0, 1.0, 4.0, out, None) == EINVAL


# rotation and norms ---------------------------------------------------------


def _rope(L, norm=False, eps=1e-6, offset=0.0, magnitude=1.0, freqs=FAKE, pos=FAKE, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE,
          q_out=FAKE, k_out=FAKE, **kw):
    from gated_deltanet_prefill_chunkwise_amd import ops
    base = dict(rows=4, n_q=8, n_k=2, d=128, rot=64, layout=0, dtype=1, w_dtype=1, q_row=1024, q_head=128, k_row=256,
                k_head=128, qo_row=1024, qo_head=128, ko_row=256, ko_head=128)
    base.update(kw)
    v = list(base.values())
    s = ops.RopeShape(*v[:8], *(ops.Strides(*v[i:i + 2]) for i in range(8, 16, 2)))
    weights = (wq, wk, offset, eps) if norm else ()
    fn = L.sgdn_norm_rope if norm else L.sgdn_rope
    return fn(ctypes.byref(s), q, k, *weights, pos, 0, freqs, magnitude, q_out, k_out, None)


ROPE_REFUSED = [
    (dict(rows=-1), EINVAL), (dict(n_q=-1), EINVAL), (dict(n_k=-1), EINVAL), (dict(d=0), EINVAL), (dict(rot=-2), EINVAL),
    (dict(rot=130), EINVAL), (dict(dtype=3), EINVAL), (dict(dtype=-1), EINVAL), (dict(layout=2), EINVAL),
    (dict(layout=-1), EINVAL), (dict(rot=63), EUNSUPPORTED), (dict(d=132), EUNSUPPORTED), (dict(d=264), EUNSUPPORTED),
    (dict(d=130, dtype=0), EUNSUPPORTED), (dict(n_q=65535, n_k=1), EUNSUPPORTED), (dict(rows=(1 << 26) - 3), EUNSUPPORTED),
    (dict(magnitude=float("inf")), EINVAL), (dict(magnitude=1e39), EINVAL), (dict(magnitude=float("nan")), EINVAL),
    (dict(pos=None), EINVAL), (dict(freqs=None), EINVAL), (dict(freqs=ctypes.c_void_p(0x1004)), EINVAL),
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(q_out=None), EINVAL), (dict(k_out=None), EINVAL),
    (dict(q=ODD), EINVAL), (dict(k=ODD), EINVAL), (dict(q_out=ODD), EINVAL), (dict(k_out=ODD), EINVAL),
    (dict(q_row=1028), EINVAL), (dict(q_head=132), EINVAL), (dict(q_row=127), EINVAL), (dict(q_head=120), EINVAL),
    (dict(q_row=1016), EINVAL),                       # rows that overlap
    (dict(ko_row=0), EINVAL), (dict(ko_head=0), EINVAL), (dict(qo_row=-1024), EINVAL), (dict(q_row=(1 << 36) + 8), EINVAL),
    (dict(q_head=128, q_row=128), EINVAL),            # heads of a row on the next row's
    (dict(qo_row=2048), EINVAL), (dict(ko_row=512, ko_head=256), EINVAL),   # in place, with other strides
]


@pytest.mark.parametrize("kw, status", ROPE_REFUSED)
@pytest.mark.parametrize("norm", [False, True])
def test_rope_refused(L, norm, kw, status):
    assert _rope(L, norm, **kw) == status


def test_norm_refused(L):
    for kw in (dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(offset=float("nan")),
               dict(offset=float("inf")), dict(w_dtype=3), dict(wq=ODD), dict(wk=ODD)):
        assert _rope(L, True, **kw) == EINVAL, kw


def test_rope_of_nothing(L):
    for norm in (False, True):
        none = dict(q=None, k=None, q_out=None, k_out=None, pos=None, freqs=None)
        assert _rope(L, norm, rows=0, **none) == 0
        assert _rope(L, norm, n_q=0, n_k=0, **none) == 0
        assert _rope(L, norm, rows=0, d=0, **none) == EINVAL


# attention of chunks --------------------------------------------------------


def _shape(**kw):
    from gated_deltanet_prefill_chunkwise_amd import ops
    base = dict(rows=40, batch=4, n_q=8, n_kv=2, d=128, page=64, n_pages=100, width=20, max_len=0,
                dtype=1, o_dtype=0)
    base.update(kw)
    return ops.Paged(*[base[n] for n, _ in ops.Paged._fields_])


def _chunk(L, ws_bytes=1 << 40, scale=1.0, ldq=8 * 128, ptr=None, **kw):
    p = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, cu=FAKE, lens=FAKE, o=FAKE, lse=None, ws=FAKE)
    p.update(ptr or {})
    return L.sgdn_paged_attend_chunk(ctypes.byref(_shape(**kw)), p["q"], ldq, p["kc"], p["vc"], p["table"], p["cu"],
                                     p["lens"], scale, p["o"], p["lse"], p["ws"], ws_bytes, None)


CHUNK_REFUSED = [
    (dict(rows=-1), EINVAL), (dict(n_q=0), EINVAL), (dict(n_kv=0), EINVAL), (dict(d=0), EINVAL), (dict(page=0), EINVAL),
    (dict(n_pages=0), EINVAL), (dict(dtype=3), EINVAL), (dict(o_dtype=3), EINVAL), (dict(d=96), EUNSUPPORTED),
    (dict(page=48), EUNSUPPORTED), (dict(n_q=9), EUNSUPPORTED), (dict(n_pages=1 << 26), EUNSUPPORTED),
    (dict(rows=1 << 26), EUNSUPPORTED), (dict(n_kv=65536, n_q=65536), EUNSUPPORTED), (dict(batch=0), EINVAL), (dict(width=0), EINVAL), (dict(max_len=-1), EINVAL),
    (dict(max_len=20 * 64 + 1), EINVAL), (dict(width=1 << 26), EUNSUPPORTED),
    (dict(width=(1 << 25) - 1), EUNSUPPORTED), (dict(width=(1 << 25) - 1, max_len=(1 << 31) - 127), EUNSUPPORTED),
    (dict(scale=float("nan")), EINVAL), (dict(scale=3e38), EINVAL), (dict(ldq=1020), EINVAL), (dict(ldq=1028), EINVAL),
]


@pytest.mark.parametrize("kw, status", CHUNK_REFUSED)
def test_chunk_refused(L, kw, status):
    assert _chunk(L, **kw) == status
    if "scale" not in kw and "ldq" not in kw and "o_dtype" not in kw:
        assert L.sgdn_paged_chunk_workspace_bytes(ctypes.byref(_shape(**kw))) == 0


def test_chunk_pointers(L):
    for n in ("q", "kc", "vc", "table", "cu", "lens", "o", "ws"):
        assert _chunk(L, ptr={n: None}) == EINVAL, n
    for n in ("q", "kc", "vc", "o", "ws"):
        assert _chunk(L, ptr={n: ODD}) == EINVAL, n
    assert L.sgdn_paged_attend_chunk(None, *[None] * 1, 0, *[None] * 5, 1.0, None, None, None, 0, None) == EINVAL
    assert L.sgdn_paged_chunk_workspace_bytes(None) == 0


def test_chunk_workspace(L):
    need = L.sgdn_paged_chunk_workspace_bytes(ctypes.byref(_shape()))
    assert need > 0
    # the longest contexts, the most rows and heads: sizes beyond 32 bits are held
    assert L.sgdn_paged_chunk_workspace_bytes(ctypes.byref(_shape(width=(1 << 25) - 1, max_len=(1 << 31) - 128))) > 0
    assert L.sgdn_paged_chunk_workspace_bytes(ctypes.byref(_shape(rows=1 << 24, batch=1 << 30))) > 32 << 24
    assert _chunk(L, ws_bytes=need - 1) == EWORKSPACE
    assert _chunk(L, rows=0, ptr={n: None for n in ("q", "kc", "vc", "table", "cu", "lens", "o", "ws")}) == 0


def test_binding_refuses_host_tensors():
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    f, _ = ops.rope_freqs(64)
    x, pos = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ops.rope(x, None, pos, f), lambda: ops.norm_rope(x, x, None, None, pos, f),
                 lambda: ops.rope(None, None, pos, f), lambda: ops.rope(x, None, pos, f, k_out=x)):
        with pytest.raises(ValueError):
            call()
    cache, table = torch.zeros(3, 1, 16, 64), torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.paged_attend_chunk(x, cache, cache, table, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
