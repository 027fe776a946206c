"""Thin Python binding of libsgdn.so (C ABI in include/sgdn.h, for the paged
attention operators ``paged_*`` include/sgdn_attn.h, and for what stands around
them, ``rope*``, ``norm_rope`` and ``paged_attend_chunk``, include/sgdn_serve.h).

Argument marshalling only: every step of the prefill runs in the library's HIP
kernels.  Tensors are torch device tensors (torch provides memory and the
stream).  The library is loaded on first use; a missing library raises.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsgdn.so")

SGDN_F32, SGDN_BF16, SGDN_F16 = 0, 1, 2
SOLVES = {"exact": 0, "blockadj": 1}
EXPORTS = ("sgdn_workspace_bytes", "sgdn_event_capacity", "sgdn_prefill_dense", "sgdn_select",
           "sgdn_prefill_sparse", "sgdn_decode_step", "sgdn_status_string", "sgdn_fp64_selftest",
           "sgdn_select_noalloc",
           "sgdn_paged_release", "sgdn_paged_plan", "sgdn_paged_write",
           "sgdn_paged_workspace_bytes", "sgdn_paged_attend", "sgdn_paged_attend_sparse",
           "sgdn_paged_select",
           "sgdn_rope_freqs", "sgdn_rope", "sgdn_norm_rope", "sgdn_paged_chunk_workspace_bytes",
           "sgdn_paged_attend_chunk")
NOALLOC_SCRATCH_BYTES = 4 << 20   # SGDN_NOALLOC_SCRATCH_BYTES


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "seqlen", "n_qk", "n_v", "d_k", "d_v", "dtype", "solve", "o_dtype")] + \
               [("cu_seqlens", ctypes.c_void_p)]


class SparseParams(ctypes.Structure):
    _fields_ = [("keep_budget", ctypes.c_float), ("tier_rate", ctypes.c_float * 3),
                ("tail", ctypes.c_int32),
                ("r_window", ctypes.c_int32), ("norm_weight", ctypes.c_void_p),
                ("fixed_tiers", ctypes.c_int32), ("unit_visibility", ctypes.c_int32),
                ("rank_key", ctypes.c_void_p), ("ablate", ctypes.c_int32),
                ("aux_stream", ctypes.c_void_p), ("aux_events", ctypes.c_void_p * 2)]


ABLATE = {"deferred_w": 1, "compact_states": 2, "csr": 4, "mapped_o": 8,
          "tier_schedule": 16}   # SGDN_ABLATE_* bits


class Stats(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("E_max", ctypes.c_int32),
                ("n_tier", ctypes.c_int32 * 3), ("k", ctypes.c_int32 * 3),
                ("n_snapshots", ctypes.c_int32), ("nonfinite_input", ctypes.c_int32),
                ("nonfinite_output", ctypes.c_int32)]


class Paged(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("rows", "batch", "n_q", "n_kv", "d", "page", "n_pages", "width", "max_len",
                 "dtype", "o_dtype")]


# bits of Stats.nonfinite_input / nonfinite_output (SGDN_NF_*)
NF_INPUT = {"q": 1, "k": 2, "v": 4, "a": 8, "beta": 16, "z": 32, "s0": 64}
NF_OUTPUT = {"o": 1, "s_final": 2}
STAT_FIELDS = ("E", "E_max", "n_low", "n_medium", "n_high", "k_low", "k_medium", "k_high",
               "n_snapshots", "nonfinite_input", "nonfinite_output")


class Strides(ctypes.Structure):
    _fields_ = [("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class RopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("rows", "n_q", "n_k", "d", "rot", "layout", "dtype", "w_dtype")] + \
               [(n, Strides) for n in ("q", "k", "q_out", "k_out")]


class Debug(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("g", "gamma", "prefix", "score", "eta", "U", "mask", "tier")] + \
               [("events", ctypes.POINTER(ctypes.c_void_p)), ("n_events", ctypes.c_int32)]


EV_NAMES = ("start", "intra", "prefix", "gate", "select", "deferred_w", "hscan", "o")


STATS_INTS = ctypes.sizeof(Stats) // 4

_lib = None


class SgdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def lib():
    """Load libsgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m gated_deltanet_prefill_chunkwise_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        P = ctypes.POINTER(Problem)
        SP = ctypes.POINTER(SparseParams)
        L.sgdn_workspace_bytes.argtypes = [P, i32, SP]
        L.sgdn_workspace_bytes.restype = sz
        L.sgdn_event_capacity.argtypes = [P, SP, ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_int32)]
        L.sgdn_event_capacity.restype = i32
        L.sgdn_fp64_selftest.argtypes = [vp, vp, vp, vp, ctypes.c_int64, vp]
        L.sgdn_fp64_selftest.restype = i32
        L.sgdn_prefill_dense.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
        L.sgdn_prefill_dense.restype = i32
        L.sgdn_select.argtypes = [P, vp, vp, vp, SP, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.sgdn_select.restype = i32
        L.sgdn_select_noalloc.argtypes = [P, vp, vp, vp, SP, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sgdn_select_noalloc.restype = i32
        L.sgdn_prefill_sparse.argtypes = [P, vp, vp, vp, vp, vp, vp, SP, vp, vp, vp, vp, vp, vp,
                                          sz, vp, vp]
        L.sgdn_prefill_sparse.restype = i32
        L.sgdn_decode_step.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sgdn_decode_step.restype = i32
        PG, f32, i64 = ctypes.POINTER(Paged), ctypes.c_float, ctypes.c_int64
        L.sgdn_paged_release.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.sgdn_paged_plan.argtypes = [i32, i32, i32, i32, i32] + [vp] * 14
        L.sgdn_paged_write.argtypes = [PG, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp]
        L.sgdn_paged_workspace_bytes.argtypes = [PG, i32, i32]
        L.sgdn_paged_workspace_bytes.restype = sz
        L.sgdn_paged_attend.argtypes = [PG, vp, i64, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz, vp]
        L.sgdn_paged_attend_sparse.argtypes = [PG, vp, i64, vp, vp, vp, vp, vp, vp, i32, f32, vp,
                                               vp, vp, sz, vp]
        L.sgdn_paged_select.argtypes = [PG, vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, sz,
                                        vp]
        for name in ("release", "plan", "write", "attend", "attend_sparse", "select"):
            getattr(L, "sgdn_paged_" + name).restype = i32
        RS, f64 = ctypes.POINTER(RopeShape), ctypes.c_double
        L.sgdn_rope_freqs.argtypes = [i32, i32, f64, f64, f64, f64, f64, vp, vp]
        L.sgdn_rope.argtypes = [RS, vp, vp, vp, i32, vp, f64, vp, vp, vp]
        L.sgdn_norm_rope.argtypes = [RS, vp, vp, vp, vp, f32, f32, vp, i32, vp, f64, vp, vp, vp]
        L.sgdn_paged_chunk_workspace_bytes.argtypes = [PG]
        L.sgdn_paged_chunk_workspace_bytes.restype = sz
        L.sgdn_paged_attend_chunk.argtypes = [PG, vp, i64, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz,
                                              vp]
        for name in ("rope_freqs", "rope", "norm_rope", "paged_attend_chunk"):
            getattr(L, "sgdn_" + name).restype = i32
        L.sgdn_status_string.argtypes = [i32]
        L.sgdn_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().sgdn_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _code(dtype):
    """sgdn_dtype of an input tensor dtype (fp32 or bf16)."""
    import torch
    codes = {torch.float32: SGDN_F32, torch.bfloat16: SGDN_BF16}
    if dtype not in codes:
        raise ValueError(f"inputs must be float32 or bfloat16, got {dtype}")
    return codes[dtype]


def _ocode(dtype):
    """sgdn_dtype of the output o (fp32, bf16 or fp16)."""
    import torch
    codes = {torch.float32: SGDN_F32, torch.bfloat16: SGDN_BF16, torch.float16: SGDN_F16}
    if dtype not in codes:
        raise ValueError(f"o must be float32, bfloat16 or float16, got {dtype}")
    return codes[dtype]


def batch_shape(q, cu_seqlens=None, max_seqlen=None):
    """(B, T) of a call.  Packed sequences (``cu_seqlens`` int32 [B + 1] on the
    device, q [1, N_tok, Nq, d]): B = len(cu_seqlens) - 1 and T = the longest
    sequence (read back from the device unless ``max_seqlen`` is given)."""
    if cu_seqlens is None:
        return q.shape[0], q.shape[1]
    import torch
    _check(cu_seqlens, "cu_seqlens", torch.int32)
    if q.shape[0] != 1:
        raise ValueError("packed sequences take q, k, v, a, beta, z of batch 1 [1, N_tok, ...]")
    B = cu_seqlens.numel() - 1
    if B < 1:
        raise ValueError("cu_seqlens needs at least two offsets")
    if max_seqlen is None:
        max_seqlen = int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    return B, max(int(max_seqlen), 1)


def problem(q, v, solve="exact", out_dtype=None, cu_seqlens=None, max_seqlen=None) -> Problem:
    B, T = batch_shape(q, cu_seqlens, max_seqlen)
    Nq, d = q.shape[2], q.shape[3]
    Nv, dv = v.shape[2], v.shape[3]
    od = _ocode(out_dtype) if out_dtype is not None else SGDN_F32
    return Problem(B, T, Nq, Nv, d, dv, _code(q.dtype), SOLVES[solve], od,
                   None if cu_seqlens is None else cu_seqlens.data_ptr())


def sparse_params(keep_budget=0.29, norm_weight=None, tail=16, r_window=16, fixed_tiers=False,
                  unit_visibility=False, rank_key=None, ablate=(), aux=None,
                  tier_rate=None) -> SparseParams:
    """Selector parameters; ``rank_key`` (device fp32 [B, Nv/2, C]) and the
    flags are the selector ablations, ``ablate`` names kernel-pipeline
    ablations (keys of ABLATE), ``tier_rate`` a (rho_L, rho_M, rho_H)
    override of the budget's tier rates, all described in include/sgdn.h.
    ``aux`` is an (aux stream, fork event, join event) triple of torch
    objects, or None for the one-stream schedule."""
    bits = 0
    for name in ablate:
        bits |= ABLATE[name]
    rates = (ctypes.c_float * 3)(*((0.0, 0.0, 0.0) if tier_rate is None else tier_rate))
    p = SparseParams(float(keep_budget), rates, tail, r_window,
                     None if norm_weight is None else norm_weight.data_ptr(),
                     int(bool(fixed_tiers)), int(bool(unit_visibility)),
                     None if rank_key is None else rank_key.data_ptr(), bits)
    if aux is not None:
        stream, ev0, ev1 = aux
        p.aux_stream = stream.cuda_stream
        p.aux_events[0] = ev0.cuda_event
        p.aux_events[1] = ev1.cuda_event
    return p


_aux = {}


def aux_stream(device=None):
    """The binding's second stream and fork / join events for ``device``
    (created once per device and kept; the library itself holds none).  The
    stream has the default priority; the events are recorded once so that
    their handles exist."""
    import torch
    idx = None if device is None else torch.device(device).index
    dev = torch.device("cuda", torch.cuda.current_device() if idx is None else idx)
    if dev not in _aux:
        with torch.cuda.device(dev):
            st = torch.cuda.Stream(device=dev)
            evs = (torch.cuda.Event(enable_timing=False), torch.cuda.Event(enable_timing=False))
            for e in evs:
                e.record(st)
            st.synchronize()
        _aux[dev] = (st, *evs)
    return _aux[dev]


def event_capacity(prob: Problem, params: SparseParams):
    """((k_L, k_M, k_H), E_max per sequence) as the library sizes them."""
    k = (ctypes.c_int32 * 3)()
    e = ctypes.c_int32()
    st = lib().sgdn_event_capacity(ctypes.byref(prob), ctypes.byref(params), k, ctypes.byref(e))
    if st != 0:
        raise SgdnError(st, "sgdn_event_capacity")
    return tuple(k), int(e.value)


def fp64_selftest(x, y, stream=None):
    """Run the selector's compiled binary64 division and square root on device
    fp64 tensors; returns (x / y, sqrt(x)) as device tensors."""
    import torch
    _check(x, "x", torch.float64)
    _check(y, "y", torch.float64)
    if x.shape != y.shape:
        raise ValueError("x and y must have the same shape")
    q = torch.empty_like(x)
    r = torch.empty_like(x)
    st = lib().sgdn_fp64_selftest(_ptr(x), _ptr(y), _ptr(q), _ptr(r), x.numel(), _stream(stream))
    if st != 0:
        raise SgdnError(st, "sgdn_fp64_selftest")
    return q, r


def workspace_bytes(prob: Problem, sparse: bool, params: SparseParams | None = None) -> int:
    return int(lib().sgdn_workspace_bytes(ctypes.byref(prob), int(sparse),
                                          None if params is None else ctypes.byref(params)))


def _check(t, name, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _stats_check(stats, B):
    import torch
    _check(stats, "stats", torch.int32)
    if stats is not None and tuple(stats.shape) != (B, STATS_INTS):
        raise ValueError(f"stats must be int32 [{B}, {STATS_INTS}]")


def _workspace(nbytes, device, workspace):
    import torch
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def debug_struct(events=None, **bufs) -> Debug:
    """Debug outputs (torch tensors by field name) and optional hipEvent_t handles."""
    d = Debug(*[None if bufs.get(n) is None else bufs[n].data_ptr() for n, _ in Debug._fields_[:8]])
    if events is not None:
        arr = (ctypes.c_void_p * len(events))(*events)
        d.events = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
        d.n_events = len(events)
        d._keep = arr
    return d


def prefill_dense(q, k, v, a, beta, s0=None, solve="exact", want_state=True, o=None,
                  s_final=None, workspace=None, debug=None, stream=None, out_dtype=None,
                  cu_seqlens=None, max_seqlen=None, stats=None):
    """Dense GDN-core prefill; returns (o, s_final).

    o is fp32 unless ``out_dtype`` (or a given ``o``) says otherwise.  With
    ``cu_seqlens`` the inputs hold packed sequences (see ``batch_shape``).
    ``stats`` (int32 [B, STATS_INTS] on the device) receives the per-sequence
    statistics, including the non-finite flags.
    """
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, n, q.dtype)
    _check(a, "a", torch.float32)
    _check(s0, "s0", torch.float32)
    if o is not None:
        out_dtype = o.dtype
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    _check(o, "o", out_dtype)
    prob = problem(q, v, solve, out_dtype, cu_seqlens, max_seqlen)
    B, Nv, dv = prob.batch, v.shape[2], v.shape[3]
    if o is None:
        o = torch.empty(v.shape, dtype=out_dtype, device=v.device)
    if want_state and s_final is None:
        s_final = torch.empty((B, Nv, q.shape[3], dv), dtype=torch.float32, device=q.device)
    _stats_check(stats, B)
    nbytes = workspace_bytes(prob, False)
    if nbytes == 0:
        raise SgdnError(-2, "sgdn_workspace_bytes")
    ws = _workspace(nbytes, q.device, workspace)
    dbg = None if debug is None else ctypes.byref(debug)
    st = lib().sgdn_prefill_dense(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                  _ptr(beta), _ptr(s0), _ptr(o), _ptr(s_final), _ptr(stats),
                                  _ptr(ws), ws.numel(), _stream(stream), dbg)
    if st != 0:
        raise SgdnError(st, "sgdn_prefill_dense")
    return o, s_final


def decode_step(q, k, v, a, beta, state, s_out=None, o=None, out_dtype=None, stream=None):
    """One-token decode step from ``state`` [B, Nv, d, dv] fp32; returns (o, s_out).

    q, k [B, Nq, d], v [B, Nv, dv], a [B, Nv] fp32, beta [B, Nv].  ``s_out``
    may be ``state`` itself (updated in place); by default a new tensor.
    """
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, n, q.dtype)
    _check(a, "a", torch.float32)
    _check(state, "state", torch.float32)
    if o is not None:
        out_dtype = o.dtype
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    _check(o, "o", out_dtype)
    B, Nq, d = q.shape
    Nv, dv = v.shape[1], v.shape[2]
    if o is None:
        o = torch.empty(v.shape, dtype=out_dtype, device=v.device)
    if s_out is None:
        s_out = torch.empty_like(state)
    _check(s_out, "s_out", torch.float32)
    for t, shape, n in ((k, (B, Nq, d), "k"), (a, (B, Nv), "a"), (beta, (B, Nv), "beta"),
                        (state, (B, Nv, d, dv), "state"), (s_out, (B, Nv, d, dv), "s_out"),
                        (o, (B, Nv, dv), "o")):
        if tuple(t.shape) != shape:
            raise ValueError(f"{n} must have shape {shape}, got {tuple(t.shape)}")
    prob = Problem(B, 1, Nq, Nv, d, dv, _code(q.dtype), 0, _ocode(out_dtype))
    st = lib().sgdn_decode_step(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                _ptr(beta), _ptr(state), _ptr(s_out), _ptr(o), _stream(stream))
    if st != 0:
        raise SgdnError(st, "sgdn_decode_step")
    return o, s_out


def select(score, gamma, eta, keep_budget=0.29, workspace=None, stream=None, cu_seqlens=None,
           fixed_tiers=False, unit_visibility=False, rank_key=None, noalloc=False, out=None,
           tier_rate=None):
    """Selector + CSR layout on fp32 statistics; returns a dict of device tensors.

    With ``cu_seqlens`` (int32 [B + 1] token offsets) sequence b has only its
    ceil(len_b / 64) valid chunks; the arrays keep the stride C.  ``noalloc``
    calls sgdn_select_noalloc (the library's static scratch, no workspace);
    ``out`` reuses a dict of output tensors from an earlier call.
    """
    import torch
    B, Nv, C = score.shape
    for t, n in ((score, "score"), (gamma, "gamma"), (eta, "eta")):
        _check(t, n, torch.float32)
    _check(cu_seqlens, "cu_seqlens", torch.int32)
    _check(rank_key, "rank_key", torch.float32)
    if rank_key is not None and tuple(rank_key.shape) != (B, Nv // 2, C):
        raise ValueError("rank_key must be [B, Nv/2, C]")
    if cu_seqlens is not None and cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must hold B + 1 offsets")
    T = C * 64
    prob = Problem(B, T, Nv // 2, Nv, 128, 128, SGDN_BF16, 1, SGDN_F32,
                   None if cu_seqlens is None else cu_seqlens.data_ptr())
    params = sparse_params(keep_budget, fixed_tiers=fixed_tiers, unit_visibility=unit_visibility,
                           rank_key=rank_key, tier_rate=tier_rate)
    NP, G = Nv // 2, (C + 1) // 2
    dev = score.device
    _, e_max = event_capacity(prob, params)
    shapes = dict(mask=((B, NP, C), torch.uint8), tier=((B, NP), torch.uint8),
                  row_pair=((B, NP), torch.int32), row_ptr=((B, NP + 1), torch.int32),
                  col=((B, e_max), torch.int32), pred=((B, NP, G), torch.int32),
                  group_slot=((B, NP, G), torch.int32), stats=((B, STATS_INTS), torch.int32))
    if out is not None:
        for name, (shape, dt) in shapes.items():
            _check(out[name], name, dt)
            if tuple(out[name].shape) != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(out[name].shape)}")
    else:
        out = {name: torch.empty(shape, dtype=dt, device=dev) for name, (shape, dt) in shapes.items()}
        out["col"].fill_(-1)
    return _select_call(prob, params, score, gamma, eta, out, workspace, noalloc, stream)


def _select_call(prob, params, score, gamma, eta, out, workspace, noalloc, stream):
    args = (_ptr(out["mask"]), _ptr(out["tier"]), _ptr(out["row_pair"]), _ptr(out["row_ptr"]),
            _ptr(out["col"]), _ptr(out["pred"]), _ptr(out["group_slot"]), _ptr(out["stats"]))
    if noalloc:
        st = lib().sgdn_select_noalloc(ctypes.byref(prob), _ptr(score), _ptr(gamma), _ptr(eta),
                                       ctypes.byref(params), *args, _stream(stream))
        if st != 0:
            raise SgdnError(st, "sgdn_select_noalloc")
        return out
    nbytes = workspace_bytes(prob, True, params)
    if nbytes == 0:
        raise SgdnError(-2, "sgdn_workspace_bytes")
    ws = _workspace(nbytes, score.device, workspace)
    st = lib().sgdn_select(ctypes.byref(prob), _ptr(score), _ptr(gamma), _ptr(eta),
                           ctypes.byref(params), *args, _ptr(ws), ws.numel(), _stream(stream))
    if st != 0:
        raise SgdnError(st, "sgdn_select")
    return out


def prefill_sparse(q, k, v, a, beta, z=None, keep_budget=0.29, solve="blockadj",
                   mask_override=None, s0=None, norm_weight=None, want_state=True, o=None,
                   s_final=None, stats=None, workspace=None, debug=None, stream=None,
                   out_dtype=None, cu_seqlens=None, max_seqlen=None, tail=16, fixed_tiers=False,
                   unit_visibility=False, rank_key=None, ablate=(), aux=True, tier_rate=None):
    """SparseGDN prefill; returns (o, s_final, stats[B, STATS_INTS] int32).

    o is fp32 unless ``out_dtype`` (or a given ``o``) says otherwise.  With
    ``cu_seqlens`` the inputs hold packed sequences (see ``batch_shape``).
    ``aux``: True uses the binding's second stream (``aux_stream``) for the
    H scan and O of the shorter chains (where the library forks: sequences
    longer than 64 chunks, see include/sgdn.h), False runs every kernel on
    ``stream``, or a (stream, event, event) triple of the caller's.
    """
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (z, "z")):
        _check(t, n, q.dtype)
    _check(a, "a", torch.float32)
    _check(s0, "s0", torch.float32)
    _check(mask_override, "mask_override", torch.uint8)
    _check(norm_weight, "norm_weight", torch.float32)
    if o is not None:
        out_dtype = o.dtype
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    _check(o, "o", out_dtype)
    prob = problem(q, v, solve, out_dtype, cu_seqlens, max_seqlen)
    _check(rank_key, "rank_key", torch.float32)
    if rank_key is not None and tuple(rank_key.shape) != (prob.batch, v.shape[2] // 2,
                                                         -(-prob.seqlen // 64)):
        raise ValueError("rank_key must be [B, Nv/2, C]")
    if aux is True:
        aux = aux_stream(q.device)
    elif aux is False:
        aux = None
    params = sparse_params(keep_budget, norm_weight, tail=tail, fixed_tiers=fixed_tiers,
                           unit_visibility=unit_visibility, rank_key=rank_key, ablate=ablate,
                           aux=aux, tier_rate=tier_rate)
    B, Nv, dv = prob.batch, v.shape[2], v.shape[3]
    if o is None:
        o = torch.empty(v.shape, dtype=out_dtype, device=v.device)
    if want_state and s_final is None:
        s_final = torch.empty((B, Nv, q.shape[3], dv), dtype=torch.float32, device=q.device)
    if stats is None:
        stats = torch.zeros((B, STATS_INTS), dtype=torch.int32, device=q.device)
    _stats_check(stats, B)
    nbytes = workspace_bytes(prob, True, params)
    if nbytes == 0:
        raise SgdnError(-2, "sgdn_workspace_bytes")
    ws = _workspace(nbytes, q.device, workspace)
    dbg = None if debug is None else ctypes.byref(debug)
    st = lib().sgdn_prefill_sparse(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                   _ptr(beta), _ptr(z), ctypes.byref(params), _ptr(mask_override),
                                   _ptr(s0), _ptr(o), _ptr(s_final), _ptr(stats), _ptr(ws),
                                   ws.numel(), _stream(stream), dbg)
    if st != 0:
        raise SgdnError(st, "sgdn_prefill_sparse")
    return o, s_final, stats



# Paged attention (include/sgdn_attn.h) ---------------------------------------
#
# The tensors of a call must share one device, which need not be the current
# one; ``stream`` is a stream of that device (default: its current stream).  On
# another stream than the current one a call allocates from that stream's
# memory and holds the tensors that it is given for it (``record_stream``).

PLAN_REFUSED = {"pages": 1, "width": 2, "rows": 4, "negative": 8}   # codes of paged_plan's status


class _On:
    """The call's device as the current one, and its stream."""

    __slots__ = ("device", "away", "other", "stream", "raw")

    def __init__(self, device, stream):
        import torch
        index = device.index
        self.device = device
        self.away = index != torch._C._cuda_getDevice()
        self.raw = torch._C._cuda_getCurrentRawStream(index)
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self.other = stream is not None and stream.cuda_stream != self.raw
        if self.other:
            self.stream = stream
            self.raw = stream.cuda_stream

    def empty(self, shape, dtype):
        """Memory that belongs to the call's stream, held for the current one too."""
        import torch
        if not self.other:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def call(self, name, *args, hold=()):
        fn = getattr(lib(), name)
        if self.away:
            import torch
            with torch.cuda.device(self.device):
                st = fn(*args, self.raw)
        else:
            st = fn(*args, self.raw)
        if st != 0:
            raise SgdnError(st, name)
        if self.other:
            for t in hold:
                if t is not None:
                    t.record_stream(self.stream)


def _paged_check(device, *tensors):
    """Each (name, tensor or None, element type or None, shape or None): a contiguous
    tensor of the call's device.  One pass, as it is much of a small call's time."""
    for name, t, dtype, shape in tensors:
        if t is None:
            continue
        if (t.device != device or (dtype is not None and t.dtype is not dtype)
                or not t.is_contiguous() or not t.is_cuda):
            _check(t, name, dtype)
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _row_view(t, name, device, dtype, shape):
    """[R, heads, d] whose rows are contiguous; returns its row stride.  ``shape``: None
    where any size will do."""
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    rows, heads, d = t.shape
    if t.shape != shape and any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if rows == 0:
        return heads * d
    ld, sh, se = t.stride()
    if (rows > 1 and ld < heads * d) or (heads > 1 and sh != d) or (d > 1 and se != 1):
        raise ValueError(f"each row of {name} must be contiguous, got strides {t.stride()}")
    return ld if rows > 1 else heads * d


def _int32(**sizes):
    """The library's sizes are 32 bits wide; ctypes would take them modulo 2^32."""
    for name, x in sizes.items():
        if not -(1 << 31) <= x < 1 << 31:
            raise ValueError(f"{name} must fit 32 bits, got {x}")


@functools.lru_cache(maxsize=256)
def _paged(rows, q_heads, cache_shape, dtype, out_dtype=None, batch=1, width=1, max_len=None):
    """The shape of a call, by its sizes (made once for each: small calls are bound by this side)."""
    n_pages, n_kv, page, d = cache_shape
    if max_len is not None and max_len < 1:
        raise ValueError(f"max_len must be positive (or None), got {max_len}")
    _int32(rows=rows, batch=batch, query_heads=q_heads, heads=n_kv, d=d, page=page,
           n_pages=n_pages, width=width, max_len=max_len or 0)
    code = _ocode(dtype)
    return Paged(rows, batch, q_heads, n_kv, d, page, n_pages, width,
                 0 if max_len is None else max_len, code,
                 code if out_dtype is None else _ocode(out_dtype))


def paged_workspace_bytes(shape: Paged, n_blocks=0, select=False) -> int:
    """Workspace of paged_attend (``n_blocks`` 0), paged_attend_sparse or paged_select."""
    _int32(n_blocks=n_blocks)
    return int(lib().sgdn_paged_workspace_bytes(ctypes.byref(shape), int(n_blocks), int(select)))


@functools.lru_cache(maxsize=256)
def _paged_bytes(n_blocks, select, *sizes):
    return paged_workspace_bytes(_paged(*sizes), n_blocks, select)


def _paged_ws(n_blocks, select, on, workspace, *sizes):
    """(pointer, bytes, tensor) of the call's workspace; ``sizes`` as for _paged."""
    nbytes = _paged_bytes(n_blocks, select, *sizes)
    if nbytes == 0:
        raise SgdnError(-2, "sgdn_paged_workspace_bytes")
    import torch
    if workspace is None:
        if nbytes <= 256:                  # none is used
            return None, 0, None
        workspace = on.empty(nbytes, torch.uint8)
    else:
        _paged_check(on.device, ("workspace", workspace, None, None))
        nbytes = workspace.numel() * workspace.element_size()
    return workspace.data_ptr(), nbytes, workspace


def _optional(t):
    return None if t is None else t.data_ptr()


def _table_shape(table):
    if table.dim() != 2:
        raise ValueError("table must be [B, W]")
    return table.shape


def paged_release(lens, done, table, free_list, free_pos, page, lens_out=None, free_pos_out=None,
                  stream=None):
    """Pages of ended requests back to the ring; returns (lens, free_pos).

    ``done`` uint8 [B]; ``free_list`` int32 [n_free] is updated in place;
    ``lens_out`` / ``free_pos_out`` may be ``lens`` / ``free_pos`` themselves
    (updated in place), by default new tensors.
    """
    import torch
    dev, i32, i64 = lens.device, torch.int32, torch.int64
    B, W = _table_shape(table)
    page = operator.index(page)
    _int32(batch=B, width=W, page=page, free_list=free_list.numel())
    _paged_check(dev, ("lens", lens, i32, (B,)), ("done", done, torch.uint8, (B,)),
                 ("table", table, i32, None), ("free_list", free_list, i32, None),
                 ("free_pos", free_pos, i64, (2,)), ("lens_out", lens_out, i32, (B,)),
                 ("free_pos_out", free_pos_out, i64, (2,)))
    on = _On(dev, stream)
    if lens_out is None:
        lens_out = on.empty((B,), i32)
    if free_pos_out is None:
        free_pos_out = on.empty((2,), i64)
    on.call("sgdn_paged_release", B, page, W, free_list.numel(), lens.data_ptr(), done.data_ptr(),
            table.data_ptr(), free_list.data_ptr(), free_pos.data_ptr(), lens_out.data_ptr(),
            free_pos_out.data_ptr(),
            hold=(lens, done, table, free_list, free_pos, lens_out, free_pos_out))
    return lens_out, free_pos_out


def paged_plan(lens, add, table, free_list, free_pos, page, rows, lens_out=None,
               free_pos_out=None, out=None, stream=None):
    """Pages, slots and row descriptors of a step's new tokens; returns a dict.

    ``table`` int32 [B, W] gets the new pages in place.  The dict holds lens,
    free_pos, cu and page_cu [B + 1], slot, row_req and row_len [rows] and
    status [B] (0, or why a request was refused: ``PLAN_REFUSED``).
    ``lens_out`` / ``free_pos_out`` may be ``lens`` / ``free_pos`` themselves;
    ``out`` reuses the dict of an earlier call of the same sizes.
    """
    import torch
    dev, i32, i64 = lens.device, torch.int32, torch.int64
    B, W = _table_shape(table)
    rows, page = int(rows), operator.index(page)
    if rows < 0:
        raise ValueError(f"rows must not be negative, got {rows}")
    _int32(batch=B, width=W, page=page, rows=rows, free_list=free_list.numel())
    _paged_check(dev, ("lens", lens, i32, (B,)), ("add", add, i32, (B,)),
                 ("table", table, i32, None), ("free_list", free_list, i32, None),
                 ("free_pos", free_pos, i64, (2,)), ("lens_out", lens_out, i32, (B,)),
                 ("free_pos_out", free_pos_out, i64, (2,)))
    on = _On(dev, stream)
    if out is None:
        cu, page_cu, slot, row_req, row_len, status, new = torch.split_with_sizes(
            on.empty((4 * B + 2 + 3 * rows,), i32), (B + 1, B + 1, rows, rows, rows, B, B))
        out = dict(cu=cu, page_cu=page_cu, slot=slot, row_req=row_req, row_len=row_len,
                   status=status, lens=new if lens_out is None else lens_out,
                   free_pos=on.empty((2,), i64) if free_pos_out is None else free_pos_out)
    else:
        out = dict(out)
        if lens_out is not None:
            out["lens"] = lens_out
        if free_pos_out is not None:
            out["free_pos"] = free_pos_out
        _paged_check(dev, *((n, out[n], i32, (size,)) for n, size in
                            (("cu", B + 1), ("page_cu", B + 1), ("slot", rows), ("row_req", rows),
                             ("row_len", rows), ("status", B), ("lens", B))),
                     ("free_pos", out["free_pos"], i64, (2,)))
    o = out
    on.call("sgdn_paged_plan", B, page, W, rows, free_list.numel(), lens.data_ptr(),
            add.data_ptr(), table.data_ptr(), free_list.data_ptr(), free_pos.data_ptr(),
            o["lens"].data_ptr(), o["free_pos"].data_ptr(), o["cu"].data_ptr(),
            o["page_cu"].data_ptr(), o["slot"].data_ptr(), o["row_req"].data_ptr(),
            o["row_len"].data_ptr(), o["status"].data_ptr(),
            hold=(lens, add, table, free_list, free_pos, *o.values()))
    return out


def paged_write(k, v, slot, k_cache, v_cache, codes=None, code_scale=None, stream=None):
    """New keys and values [R, Hkv, d] into their slots, in place.

    k and v may be views with a row stride (a joint projection's output).
    With ``codes`` int8 [n_pages, Hkv, d] and ``code_scale`` fp32
    [n_pages, Hkv] the pages that the rows complete are summarised there, for
    ``paged_select``.
    """
    import torch
    dev, dt = k_cache.device, k_cache.dtype
    if k_cache.dim() != 4:
        raise ValueError("the caches must be [n_pages, Hkv, page, d]")
    n_pages, n_kv, page, d = k_cache.shape
    rows = k.shape[0]
    _paged_check(dev, ("slot", slot, torch.int32, (rows,)), ("k_cache", k_cache, None, None),
                 ("v_cache", v_cache, dt, k_cache.shape),
                 ("codes", codes, torch.int8, (n_pages, n_kv, d)),
                 ("code_scale", code_scale, torch.float32, (n_pages, n_kv)))
    ldk = _row_view(k, "k", dev, dt, (rows, n_kv, d))
    ldv = _row_view(v, "v", dev, dt, (rows, n_kv, d))
    shape = _paged(rows, n_kv, k_cache.shape, dt)
    _On(dev, stream).call(
        "sgdn_paged_write", ctypes.byref(shape), k.data_ptr(), v.data_ptr(), ldk, ldv,
        slot.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _optional(codes),
        _optional(code_scale), hold=(k, v, slot, k_cache, v_cache, codes, code_scale))


def _attend(name, q, k_cache, v_cache, table, row_len, row_req, blocks, scale, max_len, o,
            out_dtype, want_lse, lse, workspace, stream):
    import torch
    dev, dt, i32 = k_cache.device, k_cache.dtype, torch.int32
    if k_cache.dim() != 4:
        raise ValueError("the caches must be [n_pages, Hkv, page, d]")
    n_kv, d = k_cache.shape[1], k_cache.shape[3]
    ldq = _row_view(q, "q", dev, dt, (None, None, d))
    rows, n_q, _ = q.shape
    B, W = _table_shape(table)
    max_len = None if max_len is None else operator.index(max_len)   # a key below: no tensor
    n_blocks, lists = 0, ()
    if blocks is not None:
        if blocks.dim() != 3 or blocks.shape[2] < 1:
            raise ValueError("blocks must be [R, Hkv, n_blocks]")
        n_blocks = blocks.shape[2]
        lists = (blocks.data_ptr(), n_blocks)
    if row_req is None and rows > B:
        raise ValueError("without row_req, row r is request r: more rows than requests")
    if o is not None:
        out_dtype = o.dtype
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    _paged_check(dev, ("k_cache", k_cache, None, None), ("v_cache", v_cache, dt, k_cache.shape),
                 ("table", table, i32, None), ("row_len", row_len, i32, (rows,)),
                 ("row_req", row_req, i32, (rows,)),
                 ("blocks", blocks, i32, (rows, n_kv, n_blocks)),
                 ("o", o, None, (rows, n_q, d)), ("lse", lse, torch.float32, (rows, n_q)))
    sizes = (rows, n_q, k_cache.shape, dt, out_dtype, B, W, max_len)
    shape = _paged(*sizes)
    on = _On(dev, stream)
    ws, nbytes, held = _paged_ws(n_blocks, False, on, workspace, *sizes)
    if o is None:
        o = on.empty((rows, n_q, d), out_dtype)
    if want_lse and lse is None:
        lse = on.empty((rows, n_q), torch.float32)
    on.call(name, ctypes.byref(shape), q.data_ptr(), ldq, k_cache.data_ptr(), v_cache.data_ptr(),
            table.data_ptr(), _optional(row_req), row_len.data_ptr(), *lists,
            d ** -0.5 if scale is None else float(scale), o.data_ptr(), _optional(lse), ws, nbytes,
            hold=(q, k_cache, v_cache, table, row_req, row_len, blocks, o, lse, held))
    return o, lse


def paged_attend(q, k_cache, v_cache, table, row_len, row_req=None, scale=None, max_len=None,
                 o=None, out_dtype=None, want_lse=False, lse=None, workspace=None, stream=None):
    """Attention of rows [R, Hq, d] over their whole cached sequence; returns (o, lse).

    Row r belongs to request ``row_req[r]`` (by default r) and sees its first
    ``row_len[r]`` tokens; rows that see nothing give 0 (lse -inf).  ``scale``
    is d**-0.5 by default, o fp32 unless ``out_dtype`` (or a given ``o``) says
    otherwise, lse None unless asked for.  ``max_len``: an upper bound of
    ``row_len`` that is known on the host (by default what the table holds;
    longer rows are cut to it): the work is split by it.
    """
    return _attend("sgdn_paged_attend", q, k_cache, v_cache, table, row_len, row_req, None, scale,
                   max_len, o, out_dtype, want_lse, lse, workspace, stream)


def paged_attend_sparse(q, k_cache, v_cache, table, row_len, blocks, row_req=None, scale=None,
                        max_len=None, o=None, out_dtype=None, want_lse=False, lse=None,
                        workspace=None, stream=None):
    """``paged_attend`` over the blocks listed in ``blocks`` int32
    [R, Hkv, n_blocks] only (-1: none), as ``paged_select`` returns them."""
    if blocks is None:
        raise ValueError("blocks must be given")
    return _attend("sgdn_paged_attend_sparse", q, k_cache, v_cache, table, row_len, row_req,
                   blocks, scale, max_len, o, out_dtype, want_lse, lse, workspace, stream)


def paged_select(q, codes, code_scale, table, row_len, page, n_blocks, row_req=None, n_sink=1,
                 n_local=1, max_len=None, blocks=None, workspace=None, stream=None):
    """The ``n_blocks`` blocks that each row and key/value head reads; returns
    int32 [R, Hkv, n_blocks], rising, -1 behind the last.

    ``codes`` and ``code_scale`` are the page summaries of ``paged_write``.  A
    row's first ``n_sink`` and last ``n_local`` blocks are always among them.
    """
    import torch
    dev, i32 = codes.device, torch.int32
    if codes.dim() != 3:
        raise ValueError("codes must be [n_pages, Hkv, d]")
    n_pages, n_kv, d = codes.shape
    page, n_blocks = operator.index(page), operator.index(n_blocks)
    n_sink, n_local = operator.index(n_sink), operator.index(n_local)
    _int32(n_blocks=n_blocks, n_sink=n_sink, n_local=n_local)
    ldq = _row_view(q, "q", dev, q.dtype, (None, None, d))
    rows = q.shape[0]
    B, W = _table_shape(table)
    max_len = None if max_len is None else operator.index(max_len)
    if row_req is None and rows > B:
        raise ValueError("without row_req, row r is request r: more rows than requests")
    _paged_check(dev, ("codes", codes, torch.int8, None),
                 ("code_scale", code_scale, torch.float32, (n_pages, n_kv)),
                 ("table", table, i32, None), ("row_len", row_len, i32, (rows,)),
                 ("row_req", row_req, i32, (rows,)),
                 ("blocks", blocks, i32, (rows, n_kv, n_blocks)))
    sizes = (rows, q.shape[1], (n_pages, n_kv, page, d), q.dtype, None, B, W, max_len)
    shape = _paged(*sizes)
    on = _On(dev, stream)
    ws, nbytes, held = _paged_ws(n_blocks, True, on, workspace, *sizes)
    if blocks is None:
        blocks = on.empty((rows, n_kv, n_blocks), i32)
    on.call("sgdn_paged_select", ctypes.byref(shape), q.data_ptr(), ldq, codes.data_ptr(),
            code_scale.data_ptr(), table.data_ptr(), _optional(row_req), row_len.data_ptr(),
            n_blocks, n_sink, n_local, blocks.data_ptr(), ws, nbytes,
            hold=(q, codes, code_scale, table, row_req, row_len, blocks, held))
    return blocks


# --- What stands around the paged cache (include/sgdn_serve.h) ---------------
# Streams and devices as above.

ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "by_pair": 3, "by_turns": 4}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _choice(name, value, choices):
    if value not in choices:
        raise ValueError(f"{name} must be one of {', '.join(choices)}, got {value!r}")
    return choices[value]


def rope_freqs(rot, base=10000.0, scaling="plain", factor=1.0, original=0, low=1.0, high=32.0,
               device=None):
    """Frequencies of the ``rot / 2`` pairs (fp64, radians per token) and the
    magnitude that goes with them, for ``rope`` and ``norm_rope``.

    ``scaling``: "plain"; for contexts stretched by ``factor`` "linear", "base",
    "by_pair" or "by_turns" (the last two: pairs that turn more than ``high``
    times in ``original`` tokens stay, those under ``low`` are slowed, those
    between in part, by their number or by their turns).  Computed on the host;
    with ``device`` the frequencies are copied there.
    """
    import torch
    rot = operator.index(rot)
    _int32(rot=rot)
    freqs = torch.empty(max(rot // 2, 0), dtype=torch.float64)
    magnitude = ctypes.c_double()
    st = lib().sgdn_rope_freqs(rot, _choice("scaling", scaling, ROPE_SCALINGS), float(base),
                               float(factor), float(original), float(low), float(high),
                               freqs.data_ptr(), ctypes.addressof(magnitude))
    if st != 0:
        raise SgdnError(st, "sgdn_rope_freqs")
    return (freqs if device is None else freqs.to(device)), magnitude.value


def _heads_view(t, name, device, dtype, shape):
    """[R, H, d] whose heads are contiguous: its row and head strides."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    row, head, e = t.stride()
    if e != 1 and t.shape[2] > 1:
        raise ValueError(f"each head of {name} must be contiguous, got strides {t.stride()}")
    return row, head


@functools.lru_cache(maxsize=256)
def _rope_shape(rows, n_q, n_k, d, rot, layout, dtype, w_dtype, *strides):
    _int32(rows=rows, n_q=n_q, n_k=n_k, d=d, rot=rot)
    return RopeShape(rows, n_q, n_k, d, rot, _choice("layout", layout, ROPE_LAYOUTS),
                     _ocode(dtype), _ocode(w_dtype), *(Strides(*s) for s in strides))


def _rope(name, q, k, weights, numbers, pos, freqs, layout, magnitude, pos_offset, q_out, k_out,
          stream):
    import torch
    x = k if q is None else q
    if x is None:
        raise ValueError("q or k must be given")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")
    if x.dim() != 3:
        raise ValueError(f"q and k must have three dimensions, got {tuple(x.shape)}")
    dev, dt = x.device, x.dtype
    rows, _, d = x.shape
    pos_offset = operator.index(pos_offset)
    _int32(pos_offset=pos_offset)
    if freqs.dim() != 1:
        raise ValueError(f"freqs must be [rot / 2], got {tuple(freqs.shape)}")
    w_dtype = torch.float32
    for w in weights:
        if w is not None:
            w_dtype = w.dtype
    _paged_check(dev, ("pos", pos, torch.int32, (rows,)), ("freqs", freqs, torch.float64, None),
                 *((n, w, w_dtype, (d,)) for n, w in zip(("q_weight", "k_weight"), weights)))
    on = _On(dev, stream)
    strides, n, outs = [], [], []
    for what, t, out in (("q", q, q_out), ("k", k, k_out)):
        if t is None:
            n.append(0)
            outs.append(None)
            strides += [(0, 0), (0, 0)]
            continue
        s = _heads_view(t, what, dev, dt, (rows, None, d))
        if out is None:
            out = on.empty(t.shape, dt)
        strides += [s, _heads_view(out, what + "_out", dev, dt, tuple(t.shape))]
        n.append(t.shape[1])
        outs.append(out)
    shape = _rope_shape(rows, n[0], n[1], d, 2 * freqs.numel(), layout, dt, w_dtype,
                        strides[0], strides[2], strides[1], strides[3])
    on.call(name, ctypes.byref(shape), _optional(q), _optional(k), *numbers, pos.data_ptr(),
            pos_offset, freqs.data_ptr(), float(magnitude), _optional(outs[0]), _optional(outs[1]),
            hold=(q, k, *weights, pos, freqs, *outs))
    return tuple(outs)


def rope(q, k, pos, freqs, layout="half", magnitude=1.0, pos_offset=0, q_out=None, k_out=None,
         stream=None):
    """Rotary positions of queries [R, Hq, d] and keys [R, Hk, d] (either may be
    None); returns (q, k).

    Row r stands at ``pos[r] + pos_offset``; a negative place leaves the row out
    (its outputs are not written), so that ``paged_plan``'s ``row_len`` can be
    given with ``pos_offset`` -1.  The first 2 ``freqs.numel()`` elements of each
    head are turned (``rope_freqs`` makes the frequencies and the magnitude),
    the rest is copied.  ``layout``: pairs (i, i + rot/2) ("half") or
    (2i, 2i + 1) ("interleaved").  q and k may be strided views whose heads are
    contiguous; ``q_out`` and ``k_out`` may be q and k themselves.
    """
    return _rope("sgdn_rope", q, k, (), (), pos, freqs, layout, magnitude, pos_offset, q_out,
                 k_out, stream)


def norm_rope(q, k, q_weight, k_weight, pos, freqs, layout="half", magnitude=1.0, eps=1e-6,
              weight_offset=0.0, pos_offset=0, q_out=None, k_out=None, stream=None):
    """``rope`` of heads that are normed first: x / sqrt(mean x^2 + eps) times
    (weight + ``weight_offset``), weights [d] of one type (None: zeros)."""
    weights = (q_weight, k_weight)
    return _rope("sgdn_norm_rope", q, k, weights,
                 (_optional(q_weight), _optional(k_weight), float(weight_offset), float(eps)), pos,
                 freqs, layout, magnitude, pos_offset, q_out, k_out, stream)


@functools.lru_cache(maxsize=256)
def _chunk_bytes(*sizes):
    return paged_chunk_workspace_bytes(_paged(*sizes))


def paged_chunk_workspace_bytes(shape: Paged) -> int:
    """Workspace of paged_attend_chunk."""
    return int(lib().sgdn_paged_chunk_workspace_bytes(ctypes.byref(shape)))


def paged_attend_chunk(q, k_cache, v_cache, table, cu, lens, scale=None, max_len=None, o=None,
                       out_dtype=None, want_lse=False, lse=None, workspace=None, stream=None):
    """``paged_attend`` for steps in which requests have many new tokens; returns (o, lse).

    Rows ``cu[b]`` .. ``cu[b + 1] - 1`` are the last tokens of request b, which
    has ``lens[b]`` with them (``cu`` and ``lens`` of ``paged_plan``): each sees
    the tokens up to its own.  Rows of no request give 0 (lse -inf).  The other
    arguments are those of ``paged_attend``.
    """
    import torch
    dev, dt, i32 = k_cache.device, k_cache.dtype, torch.int32
    if k_cache.dim() != 4:
        raise ValueError("the caches must be [n_pages, Hkv, page, d]")
    d = k_cache.shape[3]
    ldq = _row_view(q, "q", dev, dt, (None, None, d))
    rows, n_q, _ = q.shape
    B, W = _table_shape(table)
    max_len = None if max_len is None else operator.index(max_len)
    if o is not None:
        out_dtype = o.dtype
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    _paged_check(dev, ("k_cache", k_cache, None, None), ("v_cache", v_cache, dt, k_cache.shape),
                 ("table", table, i32, None), ("cu", cu, i32, (B + 1,)), ("lens", lens, i32, (B,)),
                 ("o", o, None, (rows, n_q, d)), ("lse", lse, torch.float32, (rows, n_q)),
                 ("workspace", workspace, None, None))
    sizes = (rows, n_q, k_cache.shape, dt, out_dtype, B, W, max_len)
    shape = _paged(*sizes)
    on = _On(dev, stream)
    nbytes = _chunk_bytes(*sizes)
    if nbytes == 0:
        raise SgdnError(-2, "sgdn_paged_chunk_workspace_bytes")
    if workspace is None:
        workspace = on.empty(nbytes, torch.uint8)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    if o is None:
        o = on.empty((rows, n_q, d), out_dtype)
    if want_lse and lse is None:
        lse = on.empty((rows, n_q), torch.float32)
    on.call("sgdn_paged_attend_chunk", ctypes.byref(shape), q.data_ptr(), ldq, k_cache.data_ptr(),
            v_cache.data_ptr(), table.data_ptr(), cu.data_ptr(), lens.data_ptr(),
            d ** -0.5 if scale is None else float(scale), o.data_ptr(), _optional(lse),
            workspace.data_ptr(), nbytes,
            hold=(q, k_cache, v_cache, table, cu, lens, o, lse, workspace))
    return o, lse
