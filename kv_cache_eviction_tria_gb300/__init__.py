"""Python binding of the TriAttention KV-cache eviction library (``libtria.so``).

Argument marshalling only: every step of the pass runs in the CUDA kernels of
``libtria.so``; the functions here turn tensors and Python values into the C
structs of ``include/tria.h`` and call the entry point of the same name. There
is no CPU fallback: if the library cannot be loaded, every call raises.

PyTorch supplies device memory and streams. Device arguments are CUDA
tensors; host arguments are sequences of ints / numpy arrays.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtria.so")

TRIA_MAX_SEQS = 128
F32, F16, Q8_0, Q4_0, BF16 = range(5)
DTYPES = {"f32": F32, "f16": F16, "q8_0": Q8_0, "q4_0": Q4_0}   # types of the cache's planes
ROPE_LAYOUTS = {"half": 0, "interleaved": 1, "interleaved_to_half": 2}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

STATUS = {
    0: "TRIA_OK", 1: "TRIA_ERR_INVALID_ARG", 2: "TRIA_ERR_UNSUPPORTED", 3: "TRIA_ERR_BUDGET",
    4: "TRIA_ERR_CUDA", 5: "TRIA_ERR_WORKSPACE", 6: "TRIA_ERR_TIMEOUT", 7: "TRIA_ERR_DEVICE_ARG",
    8: "TRIA_ERR_KEEP_LIST", 9: "TRIA_ERR_CAPACITY",
}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_BUDGET, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT, \
    ERR_DEVICE_ARG, ERR_KEEP_LIST, ERR_CAPACITY = range(10)
TRIGGER_LENGTH, TRIGGER_INTERVAL = 0, 1
NO_PASS = 2 ** 31 - 1

EXPORTS = (
    "tria_gate_check", "tria_gate_describe", "tria_budget_rows", "tria_should_evict", "tria_load_stats", "tria_free_stats",
    "tria_workspace_size", "tria_workspace_init", "tria_score", "tria_select", "tria_compact",
    "tria_evict", "tria_evict_staged", "tria_evict_model", "tria_evict_model_fused", "tria_model_workspace_size",
    "tria_evict_layers",
    "tria_evict_profiled", "tria_evict_marked", "tria_select_noalloc", "tria_device_status", "tria_selftest_bounded_wait",
    "tria_calib_accumulate", "tria_calib_finish", "tria_append", "tria_schedule_check", "tria_seq_init",
    "tria_seq_prefill", "tria_seq_decode", "tria_schedule_plan", "tria_schedule_passed",
    "tria_shared_combine", "tria_shared_select",
    "tria_status_string", "tria_version", "tria_workspace_score_offset",
    "tria_rope_frequencies", "tria_load_rope", "tria_free_rope", "tria_rotate", "tria_append_qkv",
    "tria_attend_workspace_size", "tria_attend", "tria_attend_prefix_workspace_size", "tria_attend_prefix",
    "tria_beam_select_workspace_size", "tria_beam_select", "tria_reorder_workspace_size", "tria_reorder",
)


class TriaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


# --------------------------------------------------------------------------- C structs

class _StatsDesc(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("rope_theta", ctypes.c_double),
        ("omega", ctypes.POINTER(ctypes.c_double)), ("q_mean", ctypes.POINTER(ctypes.c_float)),
        ("q_abs", ctypes.POINTER(ctypes.c_float)), ("kv_of_q", ctypes.POINTER(ctypes.c_int32)),
        ("offsets", ctypes.POINTER(ctypes.c_int64)), ("n_offsets", ctypes.c_int32),
        ("layer_head_dim", ctypes.POINTER(ctypes.c_int32)), ("layer_rope_theta", ctypes.POINTER(ctypes.c_double)),
        ("nonrot_dim", ctypes.c_int32), ("q_nonrot", ctypes.POINTER(ctypes.c_float)),
    ]


class _LayerCache(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("k_type", ctypes.c_int32), ("v_type", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("n_live", ctypes.c_void_p),
        ("seq_row0", ctypes.POINTER(ctypes.c_int64)), ("capacity", ctypes.POINTER(ctypes.c_int32)),
    ]


class _Policy(ctypes.Structure):
    _fields_ = [
        ("budget_frac", ctypes.c_double), ("n_ctx", ctypes.POINTER(ctypes.c_int32)),
        ("budget_rows", ctypes.POINTER(ctypes.c_int32)), ("window", ctypes.c_int32),
        ("sink", ctypes.c_int32), ("interval", ctypes.c_int32),
        ("cur_pos", ctypes.POINTER(ctypes.c_int64)), ("sink_rows", ctypes.POINTER(ctypes.c_int32)),
    ]


class _Schedule(ctypes.Structure):
    _fields_ = [
        ("trigger", ctypes.c_int32), ("count_prompt_tokens", ctypes.c_int32),
        ("protect_prefill", ctypes.c_int32), ("sink", ctypes.c_int32), ("window", ctypes.c_int32),
        ("pad", ctypes.c_int32), ("kv_budget", ctypes.c_int64), ("divide_length", ctypes.c_int64),
        ("budget_frac", ctypes.c_double), ("n_ctx", ctypes.c_int64),
    ]


class _SeqState(ctypes.Structure):
    _fields_ = [
        ("capacity", ctypes.c_int64), ("rows", ctypes.c_int64), ("counted", ctypes.c_int64),
        ("prompt_rows", ctypes.c_int64), ("next_pos", ctypes.c_int64), ("decode_steps", ctypes.c_int64),
        ("passes", ctypes.c_int64), ("due", ctypes.c_int32), ("pad", ctypes.c_int32),
    ]


class _RopeDesc(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("nonrot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("scaling", ctypes.c_int32), ("theta", ctypes.c_double), ("omega", ctypes.POINTER(ctypes.c_double)),
        ("factor", ctypes.c_double), ("orig_ctx", ctypes.c_int64), ("low", ctypes.c_double),
        ("high", ctypes.c_double), ("mscale", ctypes.c_double),
    ]


class _Heads(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("norm", ctypes.c_void_p), ("n_heads", ctypes.c_int32),
        ("pad", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
    ]


class _Qkv(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_held", ctypes.c_void_p), ("v_held", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("q_out_stride", ctypes.c_int64), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
        ("eps", ctypes.c_double), ("pos", ctypes.c_void_p), ("tok0", ctypes.c_void_p), ("n_before", ctypes.c_void_p),
    ]


class _Attention(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("pos", ctypes.c_void_p),
        ("tok0", ctypes.c_void_p), ("scale", ctypes.c_double), ("window", ctypes.c_int32), ("sink", ctypes.c_int32),
        ("round_keys", ctypes.c_int32), ("pad", ctypes.c_int32),
    ]


class _Beams(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("seq0", ctypes.c_void_p), ("vocab", ctypes.c_int32),
        ("n_out", ctypes.c_int32), ("logits", ctypes.c_void_p), ("stride", ctypes.c_int64), ("total", ctypes.c_void_p),
        ("ended", ctypes.c_void_p), ("end_token", ctypes.c_int32), ("in_place", ctypes.c_int32), ("total_out", ctypes.c_void_p),
        ("parent_out", ctypes.c_void_p), ("token_out", ctypes.c_void_p), ("ended_out", ctypes.c_void_p),
    ]


_lib = None


def load_library(path: str | None = None):
    """Load ``libtria.so`` (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} not found: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.tria_gate_check.argtypes = [i32, i32, i32, i32]
    lib.tria_gate_check.restype = i32
    lib.tria_gate_describe.argtypes = [i32, i32, i32, i32, i32, ctypes.c_char_p, sz]
    lib.tria_gate_describe.restype = i32
    lib.tria_budget_rows.argtypes = [ctypes.c_double, i64]
    lib.tria_budget_rows.restype = i64
    lib.tria_should_evict.argtypes = [i64, i64, i64]
    lib.tria_should_evict.restype = i32
    lib.tria_load_stats.argtypes = [ctypes.POINTER(_StatsDesc), ctypes.POINTER(vp), vp]
    lib.tria_load_stats.restype = i32
    lib.tria_free_stats.argtypes = [vp]
    lib.tria_free_stats.restype = None
    lib.tria_workspace_size.argtypes = [ctypes.POINTER(_LayerCache), i32]
    lib.tria_workspace_size.restype = sz
    lib.tria_workspace_init.argtypes = [vp, sz, vp]
    lib.tria_workspace_init.restype = i32
    lib.tria_score.argtypes = [vp, i32, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, vp, vp, sz, vp]
    lib.tria_score.restype = i32
    lib.tria_select.argtypes = [vp, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, vp, sz, vp]
    lib.tria_select.restype = i32
    lib.tria_select_noalloc.argtypes = [vp, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, vp]
    lib.tria_select_noalloc.restype = i32
    lib.tria_compact.argtypes = [ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, vp, sz, vp]
    lib.tria_compact.restype = i32
    lib.tria_evict.argtypes = [vp, i32, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, sz, vp]
    lib.tria_evict.restype = i32
    lib.tria_evict_staged.argtypes = [vp, i32, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, sz, vp]
    lib.tria_evict_staged.restype = i32
    lib.tria_model_workspace_size.argtypes = [ctypes.POINTER(_LayerCache), i32, i32]
    lib.tria_model_workspace_size.restype = sz
    lib.tria_evict_model.argtypes = [vp, ctypes.POINTER(i32), i32, ctypes.POINTER(_LayerCache),
                                     ctypes.POINTER(_Policy), vp, vp, sz, vp]
    lib.tria_evict_model.restype = i32
    lib.tria_evict_model_fused.argtypes = [vp, ctypes.POINTER(i32), i32, ctypes.POINTER(_LayerCache)]
    lib.tria_evict_model_fused.restype = i32
    lib.tria_evict_layers.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy),
                                      vp, sz, vp]
    lib.tria_evict_layers.restype = i32
    lib.tria_evict_profiled.argtypes = [vp, i32, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, sz,
                                        vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i32)]
    lib.tria_evict_profiled.restype = i32
    lib.tria_evict_marked.argtypes = [vp, i32, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, sz, vp,
                                      ctypes.POINTER(vp)]
    lib.tria_evict_marked.restype = i32
    lib.tria_device_status.argtypes = [vp, vp]
    lib.tria_device_status.restype = i32
    lib.tria_selftest_bounded_wait.argtypes = [i32, vp, sz, vp]
    lib.tria_selftest_bounded_wait.restype = i32
    lib.tria_calib_accumulate.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp]
    lib.tria_calib_accumulate.restype = i32
    lib.tria_calib_finish.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, vp]
    lib.tria_calib_finish.restype = i32
    lib.tria_shared_combine.argtypes = [vp, i64, i32, ctypes.POINTER(_LayerCache), vp, vp, sz, vp]
    lib.tria_shared_combine.restype = i32
    lib.tria_shared_select.argtypes = [vp, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Policy), vp, vp, sz, vp]
    lib.tria_shared_select.restype = i32
    lib.tria_append.argtypes = [ctypes.POINTER(_LayerCache), vp, vp, vp, vp, vp, i32, vp, sz, vp]
    lib.tria_append.restype = i32
    sch_p, st_p, i32_p = ctypes.POINTER(_Schedule), ctypes.POINTER(_SeqState), ctypes.POINTER(i32)
    lib.tria_schedule_check.argtypes = [sch_p]
    lib.tria_schedule_check.restype = i32
    lib.tria_seq_init.argtypes = [st_p, i64]
    lib.tria_seq_init.restype = i32
    lib.tria_seq_prefill.argtypes = [sch_p, st_p, i64]
    lib.tria_seq_prefill.restype = i32
    lib.tria_seq_decode.argtypes = [sch_p, st_p]
    lib.tria_seq_decode.restype = i32
    lib.tria_schedule_plan.argtypes = [sch_p, st_p, i32, i32_p, i32_p, ctypes.POINTER(i64), i32_p]
    lib.tria_schedule_plan.restype = i32
    lib.tria_schedule_passed.argtypes = [sch_p, st_p, i32]
    lib.tria_schedule_passed.restype = i32
    lib.tria_rope_frequencies.argtypes = [ctypes.POINTER(_RopeDesc), ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(ctypes.c_double)]
    lib.tria_rope_frequencies.restype = i32
    lib.tria_load_rope.argtypes = [ctypes.POINTER(_RopeDesc), ctypes.POINTER(vp)]
    lib.tria_load_rope.restype = i32
    lib.tria_free_rope.argtypes = [vp]
    lib.tria_free_rope.restype = None
    lib.tria_rotate.argtypes = [vp, i32, ctypes.POINTER(_Heads), i32, i32, vp, ctypes.c_double, vp]
    lib.tria_rotate.restype = i32
    lib.tria_append_qkv.argtypes = [vp, ctypes.POINTER(_LayerCache), ctypes.POINTER(_Qkv), vp, sz, vp]
    lib.tria_append_qkv.restype = i32
    lib.tria_attend_workspace_size.argtypes = [ctypes.POINTER(_LayerCache), i32, vp]
    lib.tria_attend_workspace_size.restype = sz
    lib.tria_attend.argtypes = [ctypes.POINTER(_LayerCache), ctypes.POINTER(_Attention), vp, sz, vp]
    lib.tria_attend.restype = i32
    cache_p = ctypes.POINTER(_LayerCache)
    lib.tria_attend_prefix_workspace_size.argtypes = [cache_p, cache_p, vp, i32, vp]
    lib.tria_attend_prefix_workspace_size.restype = sz
    lib.tria_attend_prefix.argtypes = [cache_p, cache_p, vp, ctypes.POINTER(_Attention), vp, sz, vp]
    lib.tria_attend_prefix.restype = i32
    lib.tria_beam_select_workspace_size.argtypes = [vp, i32, i32, i32]
    lib.tria_beam_select_workspace_size.restype = sz
    lib.tria_beam_select.argtypes = [ctypes.POINTER(_Beams), vp, sz, vp]
    lib.tria_beam_select.restype = i32
    lib.tria_reorder_workspace_size.argtypes = [cache_p, i32, vp, i32]
    lib.tria_reorder_workspace_size.restype = sz
    lib.tria_reorder.argtypes = [cache_p, i32, vp, i32, vp, vp, sz, vp]
    lib.tria_reorder.restype = i32
    lib.tria_status_string.argtypes = [i32]
    lib.tria_status_string.restype = ctypes.c_char_p
    lib.tria_workspace_score_offset.argtypes = [ctypes.POINTER(_LayerCache)]
    lib.tria_workspace_score_offset.restype = sz
    lib.tria_version.argtypes = []
    lib.tria_version.restype = i32
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != OK:
        raise TriaError(status, where)


_raw_stream = None


def _current_stream() -> int:
    """Address of torch's current stream on the current device."""
    global _raw_stream
    import torch
    if _raw_stream is None:
        fast = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = (lambda: fast(torch.cuda.current_device())) if fast else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream_handle(stream):
    if stream is None:
        return ctypes.c_void_p(_current_stream())
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not t.is_cuda:
        raise ValueError("device argument must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("device argument must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _host_array(values, dtype, ctype):
    if values is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(values, dtype=dtype))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctype))


# --------------------------------------------------------------------------- host-only helpers

def gate_check(n_q_heads: int, n_kv_heads: int, head_dim: int, nonrot_dim: int = 0) -> int:
    return load_library().tria_gate_check(n_q_heads, n_kv_heads, head_dim, nonrot_dim)


def gate_describe(n_q_heads: int, n_kv_heads: int, head_dim: int, k_type: str = "q8_0",
                  nonrot_dim: int = 0) -> tuple:
    """tria_gate_describe: (status, the gate log line)."""
    buf = ctypes.create_string_buffer(256)
    st = load_library().tria_gate_describe(n_q_heads, n_kv_heads, head_dim, nonrot_dim, DTYPES[k_type], buf, 256)
    return st, buf.value.decode()


def budget_rows(budget_frac: float, n_ctx: int) -> int:
    return load_library().tria_budget_rows(budget_frac, n_ctx)


def should_evict(n_live: int, budget: int, interval: int) -> bool:
    return bool(load_library().tria_should_evict(n_live, budget, interval))


def status_string(status: int) -> str:
    return load_library().tria_status_string(status).decode()


def version() -> int:
    return load_library().tria_version()


# --------------------------------------------------------------------------- stats

class Stats:
    """Device-resident calibration statistics (``tria_load_stats``)."""

    def __init__(self, q_mean, q_abs, *, n_kv_heads: int, head_dim: int = 0, rope_theta: float = 0.0,
                 omega=None, kv_of_q=None, offsets=None, layer_head_dim=None, layer_rope_theta=None,
                 nonrot_dim: int = 0, q_nonrot=None, stream=None):
        """Uniform models: q_mean [L][n_q][rot/2][2], q_abs [L][n_q][rot/2] (or None),
        rot = hd - nonrot_dim the rotary dims; q_nonrot [L][n_q][nonrot_dim] the
        mean non-rotary query (or None: no content term).
        Hybrid models (layer_head_dim given): q_mean / q_abs / omega are lists with
        one array per layer, packed here layer after layer."""
        lib = load_library()
        if layer_head_dim is not None:
            n_layers, n_q = len(q_mean), len(q_mean[0])
            q_mean = np.concatenate([np.asarray(x, np.float32).ravel() for x in q_mean])
            if q_abs is not None:
                q_abs = np.concatenate([np.asarray(x, np.float32).ravel() for x in q_abs])
            if omega is not None:
                omega = np.concatenate([np.asarray(x, np.float64).ravel() for x in omega])
        else:
            q_mean = np.ascontiguousarray(np.asarray(q_mean, dtype=np.float32))
            n_layers, n_q = q_mean.shape[0], q_mean.shape[1]
        self._keep = []
        qm_arr, qm_p = _host_array(q_mean, np.float32, ctypes.c_float)
        qa_arr, qa_p = _host_array(q_abs, np.float32, ctypes.c_float)
        om_arr, om_p = _host_array(omega, np.float64, ctypes.c_double)
        kv_arr, kv_p = _host_array(kv_of_q, np.int32, ctypes.c_int32)
        of_arr, of_p = _host_array(offsets, np.int64, ctypes.c_int64)
        lh_arr, lh_p = _host_array(layer_head_dim, np.int32, ctypes.c_int32)
        lt_arr, lt_p = _host_array(layer_rope_theta, np.float64, ctypes.c_double)
        qn_arr, qn_p = _host_array(q_nonrot, np.float32, ctypes.c_float)
        self._keep += [qm_arr, qa_arr, om_arr, kv_arr, of_arr, lh_arr, lt_arr, qn_arr]
        desc = _StatsDesc(n_layers, n_q, n_kv_heads, head_dim, float(rope_theta), om_p, qm_p, qa_p,
                          kv_p, of_p, 0 if of_arr is None else len(of_arr), lh_p, lt_p, int(nonrot_dim), qn_p)
        handle = ctypes.c_void_p()
        _check(lib.tria_load_stats(ctypes.byref(desc), ctypes.byref(handle), _stream_handle(stream)),
               "tria_load_stats")
        self.handle = handle
        self.n_layers, self.n_q_heads, self.n_kv_heads, self.head_dim = n_layers, n_q, n_kv_heads, head_dim
        self.nonrot_dim = int(nonrot_dim)
        self.group = n_q // n_kv_heads

    def close(self):
        if self.handle:
            load_library().tria_free_stats(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def load_stats(q_mean, q_abs, **kw) -> Stats:
    return Stats(q_mean, q_abs, **kw)


# --------------------------------------------------------------------------- cache / policy

class LayerCache:
    """One layer's cache (``tria_layer_cache``): device tensors + host layout."""

    _made = None       # what c_ref() keeps: how to ask the planes, their addresses, the C struct

    def __init__(self, *, k, v, pos, n_live, seq_row0, capacity, head_dim: int, n_kv_heads: int,
                 k_type: str = "f16", v_type: str = "f16", k_scale=None, v_scale=None):
        self.k, self.v, self.pos, self.n_live = k, v, pos, n_live
        self.k_scale, self.v_scale = k_scale, v_scale
        self.head_dim, self.n_kv_heads = head_dim, n_kv_heads
        self.k_type, self.v_type = DTYPES[k_type], DTYPES[v_type]
        self.seq_row0 = np.ascontiguousarray(np.asarray(seq_row0, dtype=np.int64))
        self.capacity = np.ascontiguousarray(np.asarray(capacity, dtype=np.int32))

    def c_struct(self) -> _LayerCache:
        return _LayerCache(
            len(self.seq_row0), self.n_kv_heads, self.head_dim, self.k_type, self.v_type,
            _ptr(self.k), _ptr(self.k_scale), _ptr(self.v), _ptr(self.v_scale), _ptr(self.pos),
            _ptr(self.n_live), self.seq_row0.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
            self.capacity.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))

    def __setattr__(self, name, value):
        object.__setattr__(self, "_made", None)
        object.__setattr__(self, name, value)

    def __getstate__(self):
        """For copy and pickle: all but the C struct, whose addresses belong to this object."""
        return {name: value for name, value in self.__dict__.items() if name != "_made"}

    def c_ref(self):
        """A reference to the C struct, made anew only when a field or a plane's address has changed since the last
        call (a decode step calls this for every layer)."""
        made = self._made
        if made is not None:
            address, whole, at, ref, _ = made
            if [f() for f in address] == at:
                if False in [f() for f in whole]:            # restrided in place
                    raise ValueError("device argument must be contiguous")
                return ref
        c = self.c_struct()
        planes = [t for t in (self.k, self.v, self.pos, self.n_live, self.k_scale, self.v_scale)
                  if t is not None and not isinstance(t, int)]
        address = [t.data_ptr for t in planes]
        made = (address, [t.is_contiguous for t in planes], [f() for f in address], ctypes.byref(c), c)
        object.__setattr__(self, "_made", made)
        return made[3]


class Policy:
    """Eviction policy (``tria_policy``)."""

    def __init__(self, *, budget_frac: float = 0.0, n_ctx=None, budget_rows=None, window: int = 512,
                 sink: int = 0, interval: int = 128, cur_pos=None, sink_rows=None):
        self.budget_frac, self.window, self.sink, self.interval = budget_frac, window, sink, interval
        self.n_ctx, self._n_ctx_p = _host_array(n_ctx, np.int32, ctypes.c_int32)
        self.budget_rows, self._br_p = _host_array(budget_rows, np.int32, ctypes.c_int32)
        self.cur_pos, self._cp_p = _host_array(cur_pos, np.int64, ctypes.c_int64)
        self.sink_rows, self._sr_p = _host_array(sink_rows, np.int32, ctypes.c_int32)

    def c_struct(self) -> _Policy:
        return _Policy(float(self.budget_frac), self._n_ctx_p, self._br_p, self.window, self.sink,
                       self.interval, self._cp_p, self._sr_p)


# --------------------------------------------------------------------------- the pass

def workspace_size(cache: LayerCache, group: int) -> int:
    c = cache.c_struct()
    n = load_library().tria_workspace_size(ctypes.byref(c), group)
    if n == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_workspace_size")
    return n


def workspace_scores(ws, cache: LayerCache):
    """tria_workspace_score_offset: the workspace's float view of the z-max
    scores the staged evict path selected with (valid after evict_staged for
    the live rows of segments above their budget)."""
    c = cache.c_struct()
    off = load_library().tria_workspace_score_offset(ctypes.byref(c))
    if off == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_workspace_score_offset")
    rows = int(max(r0 + cache.n_kv_heads * cp for r0, cp in zip(cache.seq_row0, cache.capacity)))
    return ws[off:off + 4 * rows].view(__import__("torch").float32)


def workspace_init(ws, stream=None):
    _check(load_library().tria_workspace_init(_ptr(ws), ws.numel() * ws.element_size(),
                                              _stream_handle(stream)), "tria_workspace_init")


def _ws(ws):
    return _ptr(ws), ws.numel() * ws.element_size()


def score(stats: Stats, layer: int, cache: LayerCache, policy: Policy, score_out, raw_out=None,
          *, ws, stream=None):
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_score(stats.handle, layer, ctypes.byref(c), ctypes.byref(p),
                                     _ptr(score_out), _ptr(raw_out), wp, wb, _stream_handle(stream)),
           "tria_score")


def select(score_in, cache: LayerCache, policy: Policy, keep_out, *, ws, stream=None):
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_select(_ptr(score_in), ctypes.byref(c), ctypes.byref(p), _ptr(keep_out),
                                      wp, wb, _stream_handle(stream)), "tria_select")


def select_noalloc(score_in, cache: LayerCache, policy: Policy, keep_out, *, stream=None):
    """tria_select_noalloc: tria_select with the library's fixed scratch array
    instead of a workspace (for callers that cannot allocate)."""
    c, p = cache.c_struct(), policy.c_struct()
    _check(load_library().tria_select_noalloc(_ptr(score_in), ctypes.byref(c), ctypes.byref(p), _ptr(keep_out),
                                              _stream_handle(stream)), "tria_select_noalloc")


def compact(cache: LayerCache, policy: Policy, keep, *, ws, stream=None):
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_compact(ctypes.byref(c), ctypes.byref(p), _ptr(keep), wp, wb,
                                       _stream_handle(stream)), "tria_compact")


def evict(stats: Stats, layer: int, cache: LayerCache, policy: Policy, *, ws, stream=None):
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_evict(stats.handle, layer, ctypes.byref(c), ctypes.byref(p), wp, wb,
                                     _stream_handle(stream)), "tria_evict")


def evict_staged(stats: Stats, layer: int, cache: LayerCache, policy: Policy, *, ws, stream=None):
    """tria_evict_staged: the pass as three kernels (score, select, compact)."""
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_evict_staged(stats.handle, layer, ctypes.byref(c), ctypes.byref(p), wp, wb,
                                            _stream_handle(stream)), "tria_evict_staged")


def model_workspace_size(cache: LayerCache, n_layers: int, group: int) -> int:
    c = cache.c_struct()
    n = load_library().tria_model_workspace_size(ctypes.byref(c), n_layers, group)
    if n == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_model_workspace_size")
    return n


def evict_model(stats: Stats, layers, caches, policy: Policy, *, ws, score_out=None, stream=None):
    """tria_evict_model: one pass over several layers (caches[i] is the cache
    of layer layers[i]); score_out (optional device float tensor) receives the
    z-max scores of the compacted segments' live rows, [n_layers][layer rows]."""
    if len(caches) != len(layers) or not caches:
        raise ValueError("one cache per layer")
    structs = (_LayerCache * len(caches))(*[c.c_struct() for c in caches])
    arr, ptr = _host_array(layers, np.int32, ctypes.c_int32)
    p = policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_evict_model(stats.handle, ptr, len(layers), structs, ctypes.byref(p),
                                           _ptr(score_out) if score_out is not None else None, wp, wb,
                                           _stream_handle(stream)), "tria_evict_model")


def evict_model_fused(stats: Stats, layers, caches) -> bool:
    """tria_evict_model_fused: whether tria_evict_model (without score_out)
    runs these layers as one fused kernel (True) or as the staged kernels per
    layer (False). Host only."""
    if len(caches) != len(layers) or not caches:
        raise ValueError("one cache per layer")
    structs = (_LayerCache * len(caches))(*[c.c_struct() for c in caches])
    arr, ptr = _host_array(layers, np.int32, ctypes.c_int32)
    r = load_library().tria_evict_model_fused(stats.handle, ptr, len(layers), structs)
    if r < 0:
        raise TriaError(ERR_INVALID_ARG, "tria_evict_model_fused")
    return r == 1


def evict_layers(stats: Stats, layer_of_seq, cache: LayerCache, policy: Policy, *, ws, stream=None):
    """tria_evict_layers: one pass over sequences of several layers (sequence s
    scored with the statistics of layer layer_of_seq[s])."""
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    arr, ptr = _host_array(layer_of_seq, np.int32, ctypes.c_int32)
    if arr is None or len(arr) != len(cache.seq_row0):
        raise ValueError("one layer per sequence")
    _check(load_library().tria_evict_layers(stats.handle, ptr, ctypes.byref(c), ctypes.byref(p), wp, wb,
                                            _stream_handle(stream)), "tria_evict_layers")


def evict_profiled(stats: Stats, layer: int, cache: LayerCache, policy: Policy, *, ws, stream=None):
    """tria_evict_profiled: returns ({stage: ms}, kernels launched); synchronises."""
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    ms = (ctypes.c_float * 5)()
    nl = ctypes.c_int32()
    _check(load_library().tria_evict_profiled(stats.handle, layer, ctypes.byref(c), ctypes.byref(p), wp, wb,
                                              _stream_handle(stream), ms, ctypes.byref(nl)),
           "tria_evict_profiled")
    names = ("score", "zscore", "select", "compact", "total")
    return dict(zip(names, list(ms))), nl.value


def evict_marked(stats: Stats, layer: int, cache: LayerCache, policy: Policy, events, *, ws, stream=None):
    """tria_evict_marked: the pass with four torch.cuda.Event (timing) recorded
    before, between and after its kernels; no synchronisation (capturable)."""
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    if len(events) != 4:
        raise ValueError("four events")
    handles = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(int(e.cuda_event)) for e in events])
    _check(load_library().tria_evict_marked(stats.handle, layer, ctypes.byref(c), ctypes.byref(p), wp, wb,
                                            _stream_handle(stream), handles), "tria_evict_marked")


def device_status(ws, stream=None) -> int:
    return load_library().tria_device_status(_ptr(ws), _stream_handle(stream))


def selftest_bounded_wait(spin_limit: int, ws, stream=None) -> int:
    wp, wb = _ws(ws)
    return load_library().tria_selftest_bounded_wait(spin_limit, wp, wb, _stream_handle(stream))


def calib_accumulate(q, acc, *, nonrot_dim: int = 0, stream=None):
    """tria_calib_accumulate: add the sums of a batch of pre-RoPE queries
    q[tokens][heads][head_dim] (float32 or float16 CUDA tensor) to acc
    (float64 CUDA tensor [heads][head_dim/2][3], zeroed before the first batch);
    the last nonrot_dim dims of each head are the non-rotary ones."""
    import torch
    if q.dim() != 3:
        raise ValueError("q must be [tokens][heads][head_dim]")
    t, h, hd = q.shape
    qt = {torch.float32: F32, torch.float16: F16}.get(q.dtype)
    if qt is None:
        raise ValueError("q must be float32 or float16")
    if acc.dtype != torch.float64 or tuple(acc.shape) != (h, hd // 2, 3):
        raise ValueError("acc must be float64 [heads][head_dim/2][3]")
    qp = _ptr(q) if t > 0 else None
    _check(load_library().tria_calib_accumulate(qp, qt, t, h, hd, nonrot_dim, _ptr(acc), _stream_handle(stream)),
           "tria_calib_accumulate")


def calib_finish(acc, n_tokens: int, *, nonrot_dim: int = 0, stream=None):
    """tria_calib_finish: (q_mean [heads][rot/2][2], q_abs [heads][rot/2]) float32
    CUDA tensors, rot = head_dim - nonrot_dim; with nonrot_dim > 0 also the mean
    non-rotary query [heads][nonrot_dim] as a third element."""
    import torch
    h, fc, _ = acc.shape
    fcr = fc - nonrot_dim // 2
    q_mean = torch.empty((h, fcr, 2), dtype=torch.float32, device=acc.device)
    q_abs = torch.empty((h, fcr), dtype=torch.float32, device=acc.device)
    q_nonrot = torch.empty((h, nonrot_dim), dtype=torch.float32, device=acc.device) if nonrot_dim else None
    _check(load_library().tria_calib_finish(_ptr(acc), n_tokens, h, 2 * fc, nonrot_dim, _ptr(q_mean), _ptr(q_abs),
                                            _ptr(q_nonrot) if q_nonrot is not None else None,
                                            _stream_handle(stream)), "tria_calib_finish")
    return (q_mean, q_abs) if not nonrot_dim else (q_mean, q_abs, q_nonrot)


# --------------------------------------------------------------------------- shared-slot variant

def shared_combine(scores, cache: LayerCache, combined, *, ws, stream=None):
    """tria_shared_combine: scores float32 CUDA tensor [layers][rows] (tria_score output per layer)."""
    rows = int(max(r0 + cache.n_kv_heads * c for r0, c in zip(cache.seq_row0, cache.capacity)))
    if scores.dim() != 2 or scores.stride(1) != 1 or scores.shape[1] < rows:
        raise ValueError("scores must be [layers][rows] (rows contiguous, at least the cache layout's rows)")
    c = cache.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_shared_combine(_ptr(scores), scores.stride(0), scores.shape[0], ctypes.byref(c),
                                              _ptr(combined), wp, wb, _stream_handle(stream)),
           "tria_shared_combine")


def shared_select(combined, cache: LayerCache, policy: Policy, keep_out, *, ws, stream=None):
    """tria_shared_select: one keep list per sequence, written to every KV head's slot."""
    c, p = cache.c_struct(), policy.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_shared_select(_ptr(combined), ctypes.byref(c), ctypes.byref(p), _ptr(keep_out),
                                             wp, wb, _stream_handle(stream)), "tria_shared_select")


# --------------------------------------------------------------------------- rows in, rows out

def _rope_desc(head_dim, theta, nonrot_dim, layout, scaling, omega, factor, orig_ctx, low, high, mscale):
    om_arr, om_p = _host_array(omega, np.float64, ctypes.c_double)
    if om_arr is not None and om_arr.size != (head_dim - nonrot_dim) // 2:
        raise ValueError("omega must hold (head_dim - nonrot_dim) / 2 frequencies")
    desc = _RopeDesc(int(head_dim), int(nonrot_dim), ROPE_LAYOUTS[layout], ROPE_SCALINGS[scaling], float(theta), om_p,
                     float(factor), int(orig_ctx), float(low), float(high), float(mscale))
    return desc, om_arr


def rope_frequencies(*, head_dim: int, theta: float = 0.0, nonrot_dim: int = 0, layout: str = "half",
                     scaling: str = "none", omega=None, factor: float = 1.0, orig_ctx: int = 0, low: float = 0.0,
                     high: float = 0.0, mscale: float = 0.0):
    """tria_rope_frequencies: (omega float64 [rot/2] as Stats takes it, the factor on the rotated dims). Host only."""
    desc, _keep = _rope_desc(head_dim, theta, nonrot_dim, layout, scaling, omega, factor, orig_ctx, low, high, mscale)
    out = np.zeros(max((head_dim - nonrot_dim) // 2, 1), np.float64)
    m = ctypes.c_double()
    _check(load_library().tria_rope_frequencies(ctypes.byref(desc), out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                                ctypes.byref(m)), "tria_rope_frequencies")
    return out, m.value


class Rope:
    """Device-resident rotation (``tria_load_rope``); arguments as rope_frequencies."""

    def __init__(self, *, head_dim: int, theta: float = 0.0, nonrot_dim: int = 0, layout: str = "half",
                 scaling: str = "none", omega=None, factor: float = 1.0, orig_ctx: int = 0, low: float = 0.0,
                 high: float = 0.0, mscale: float = 0.0):
        self.handle = ctypes.c_void_p()
        desc, _keep = _rope_desc(head_dim, theta, nonrot_dim, layout, scaling, omega, factor, orig_ctx, low, high, mscale)
        handle = ctypes.c_void_p()
        _check(load_library().tria_load_rope(ctypes.byref(desc), ctypes.byref(handle)), "tria_load_rope")
        self.handle = handle
        self.head_dim, self.nonrot_dim = int(head_dim), int(nonrot_dim)

    def close(self):
        if self.handle:
            load_library().tria_free_rope(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_ACT, _INT32 = {}, ()       # torch's types, filled at the first call


def _fill_types():
    global _INT32
    import torch
    _ACT.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    _INT32 = (torch.int32,)


def _act_type(t) -> int:
    if not _ACT:
        _fill_types()
    kind = _ACT.get(t.dtype)
    if kind is None:
        raise ValueError("activations must be float32, float16 or bfloat16")
    return kind


def _rows3(t, name: str, n_tokens: int, head_dim: int, like=None):
    """(address, values between tokens) of [tokens][heads][head_dim], heads of a token consecutive."""
    try:
        n, heads, hd = t.shape
    except ValueError:
        n = -1
    if n != n_tokens or hd != head_dim or (like is not None and t.dtype is not like):
        raise ValueError(f"{name} must be [{n_tokens}][heads][{head_dim}] of the call's type")
    if not t.is_cuda:
        raise ValueError("device argument must be a CUDA tensor")
    s0, s1, s2 = t.stride()
    if n and (s2 != 1 or (heads > 1 and s1 != hd)):
        raise ValueError(f"{name}: the heads of a token must be consecutive")
    return t.data_ptr(), s0 if n > 1 else max(s0, heads * hd)


def _pos32(pos, n_tokens: int) -> int:
    if pos.numel() != n_tokens or pos.dtype not in _INT32 or not pos.is_contiguous() or not pos.is_cuda:
        raise ValueError(f"pos must be a contiguous int32 CUDA tensor of {n_tokens} positions")
    return pos.data_ptr()


def _vec32(t, n: int, name: str):
    if t is None:
        return None
    if t.numel() != n or _ACT.get(t.dtype) != F32 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {n} values")
    return t.data_ptr()


def _tokens0(tok0, n_seqs: int, n_tokens: int):
    """Host token offsets [n_seqs + 1]; None: the same number of tokens for every sequence."""
    if tok0 is None:
        if n_tokens % n_seqs:
            raise ValueError("tok0 is needed when the sequences' tokens differ")
        return np.arange(n_seqs + 1, dtype=np.int32) * (n_tokens // n_seqs)
    if not (isinstance(tok0, np.ndarray) and tok0.dtype == np.int32 and tok0.flags.c_contiguous):
        tok0 = np.ascontiguousarray(np.asarray(tok0, dtype=np.int32))
    if len(tok0) != n_seqs + 1 or tok0[n_seqs] != n_tokens:
        raise ValueError("tok0 must hold n_seqs + 1 offsets, the last one the number of tokens")
    return tok0


def rotate(rope: Rope, parts, pos, *, eps: float = 1e-6, stream=None):
    """tria_rotate: per-head norm and rotation of one or two sets of heads. parts: [(x, out, norm or None)],
    x / out [tokens][heads][head_dim] (slices of a joint projection are fine), norm float32 [head_dim];
    pos int32 [tokens]."""
    n = pos.numel()
    structs = (_Heads * len(parts))()
    kind, act = parts[0][0].dtype, _act_type(parts[0][0])
    for h, (x, out, norm) in zip(structs, parts):
        h.x, h.x_stride = _rows3(x, "x", n, rope.head_dim, kind)
        h.out, h.out_stride = _rows3(out, "out", n, rope.head_dim, kind)
        if x.shape[1] != out.shape[1]:
            raise ValueError("x and out must have the same heads")
        h.norm, h.n_heads = _vec32(norm, rope.head_dim, "norm"), x.shape[1]
    _check(load_library().tria_rotate(rope.handle, act, structs, len(parts), n, _pos32(pos, n),
                                      float(eps), _stream_handle(stream)), "tria_rotate")


def append_qkv(rope: Rope, cache: LayerCache, q, k, v, pos, *, ws, q_out=None, tok0=None, n_before=None, q_norm=None,
               k_norm=None, eps: float = 1e-6, k_held=None, v_held=None, stream=None):
    """tria_append_qkv: norm and rotation of queries and keys, the new tokens' rows into the cache in its types,
    n_live = rows before + new rows. q (or None) / k / v [tokens][heads][head_dim], pos int32 [tokens], tok0 host
    offsets of the sequences' tokens (None: equally many each), n_before int32 [n_seqs] live rows before the call
    (None: n_live); k_held / v_held receive the values that the cache now holds for the tokens."""
    n, hd, n_seqs = pos.numel(), cache.head_dim, len(cache.seq_row0)
    kind = k.dtype
    a = _Qkv()
    a.type = _act_type(k)
    a.k, a.k_stride = _rows3(k, "k", n, hd, kind)
    a.v, a.v_stride = _rows3(v, "v", n, hd, kind)
    if k.shape[1] != cache.n_kv_heads or v.shape[1] != cache.n_kv_heads:
        raise ValueError("k and v must have the cache's KV heads")
    if q is not None:
        if q_out is None or q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        a.q, a.q_stride = _rows3(q, "q", n, hd, kind)
        a.q_out, a.q_out_stride = _rows3(q_out, "q_out", n, hd, kind)
        a.n_q_heads = q.shape[1]
    for name, t in (("k_held", k_held), ("v_held", v_held)):
        if t is not None:
            if not t.is_contiguous() or t.shape != k.shape:
                raise ValueError(f"{name} must be contiguous [tokens][n_kv_heads][head_dim]")
            setattr(a, name, _rows3(t, name, n, hd, kind)[0])
    a.q_norm, a.k_norm, a.eps = _vec32(q_norm, hd, "q_norm"), _vec32(k_norm, hd, "k_norm"), float(eps)
    a.pos = _pos32(pos, n)
    tok0 = _tokens0(tok0, n_seqs, n)
    a.tok0 = tok0.ctypes.data
    if n_before is not None:
        a.n_before = _pos32(n_before, n_seqs)
    wp, wb = _ws(ws)
    st = load_library().tria_append_qkv(rope.handle, cache.c_ref(), ctypes.byref(a), wp, wb, _stream_handle(stream))
    if st:
        _check(st, "tria_append_qkv")


def attend_workspace_size(cache: LayerCache, n_q_heads: int, tok0) -> int:
    """tria_attend_workspace_size: tok0 host offsets of the sequences' tokens, or the tokens of every sequence."""
    n_seqs = len(cache.seq_row0)
    if np.ndim(tok0) == 0:
        tok0 = np.arange(n_seqs + 1, dtype=np.int32) * int(tok0)
    tok0 = _tokens0(tok0, n_seqs, int(tok0[-1]))
    c = cache.c_struct()
    n = load_library().tria_attend_workspace_size(ctypes.byref(c), n_q_heads, tok0.ctypes.data)
    if n == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_attend_workspace_size")
    return n


def _attention(q, out, pos, lse, head_dim: int, n_seqs: int, tok0, scale, window, sink, round_keys):
    """(tria_attention, what it points to on the host)."""
    n = pos.numel()
    a = _Attention()
    a.type, a.n_q_heads = _act_type(q), q.shape[1]
    a.q, a.q_stride = _rows3(q, "q", n, head_dim)
    a.out, a.out_stride = _rows3(out, "out", n, head_dim, q.dtype)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    a.lse = _vec32(lse, n * q.shape[1], "lse")
    a.pos = _pos32(pos, n)
    tok0 = _tokens0(tok0, n_seqs, n)
    a.tok0, a.scale, a.window, a.sink = tok0.ctypes.data, float(scale), int(window), int(sink)
    a.round_keys = int(round_keys)
    return a, tok0


def attend(cache: LayerCache, q, out, pos, *, ws, tok0=None, lse=None, scale: float = 0.0, window: int = 0, sink: int = 0,
           round_keys: bool = False, stream=None):
    """tria_attend: attention of new tokens over the cache. q / out [tokens][n_q_heads][head_dim], pos int32
    [tokens], tok0 host offsets of the sequences' tokens (None: equally many each), lse float32
    [tokens][n_q_heads] or None; scale 0: 1 / sqrt(head_dim); window 0: none; sink first rows stay visible;
    round_keys: prompts over quantised keys take them rounded to fp16 (faster), in out and in lse."""
    a, _keep = _attention(q, out, pos, lse, cache.head_dim, len(cache.seq_row0), tok0, scale, window, sink, round_keys)
    wp, wb = _ws(ws)
    st = load_library().tria_attend(cache.c_ref(), ctypes.byref(a), wp, wb, _stream_handle(stream))
    if st:
        _check(st, "tria_attend")


# --------------------------------------------------------------------------- several continuations of one prompt

def _groups(seq0, n_seqs: int, n_groups: int | None = None):
    """Host offsets of the groups' sequences; None: one group, or equally many sequences in each of n_groups."""
    if seq0 is None:
        g = 1 if n_groups is None else n_groups
        if g < 1 or n_seqs % g:
            raise ValueError("seq0 is needed when the groups' sequences differ")
        return np.arange(g + 1, dtype=np.int32) * (n_seqs // g)
    if not (isinstance(seq0, np.ndarray) and seq0.dtype == np.int32 and seq0.flags.c_contiguous):
        seq0 = np.ascontiguousarray(np.asarray(seq0, dtype=np.int32))
    if seq0.ndim != 1 or len(seq0) < 2 or seq0[-1] != n_seqs or (n_groups is not None and len(seq0) != n_groups + 1):
        raise ValueError("seq0 must hold the groups' first sequences and, last, the number of sequences")
    return seq0


def attend_prefix_workspace_size(prefix: LayerCache, cache: LayerCache, n_q_heads: int, tok0, seq0=None) -> int:
    """tria_attend_prefix_workspace_size: tok0 host offsets of the sequences' tokens, or the tokens of every sequence."""
    n_seqs = len(cache.seq_row0)
    if np.ndim(tok0) == 0:
        tok0 = np.arange(n_seqs + 1, dtype=np.int32) * int(tok0)
    tok0 = _tokens0(tok0, n_seqs, int(tok0[-1]))
    seq0 = _groups(seq0, n_seqs, len(prefix.seq_row0))
    n = load_library().tria_attend_prefix_workspace_size(prefix.c_ref(), cache.c_ref(), seq0.ctypes.data, n_q_heads, tok0.ctypes.data)
    if n == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_attend_prefix_workspace_size")
    return n


def attend_prefix(prefix: LayerCache, cache: LayerCache, q, out, pos, *, ws, seq0=None, tok0=None, lse=None, scale: float = 0.0,
                  window: int = 0, sink: int = 0, round_keys: bool = False, stream=None):
    """tria_attend_prefix: attention of new tokens over the rows of their sequence's prefix, held once for the sequences
    seq0[i] .. seq0[i + 1] - 1 that continue prefix i (host offsets; None: equally many each), and over the sequence's
    own rows in cache. The other arguments as attend; sink: first rows of the prefix alone (a shorter prefix has fewer)."""
    a, _keep = _attention(q, out, pos, lse, cache.head_dim, len(cache.seq_row0), tok0, scale, window, sink, round_keys)
    seq0 = _groups(seq0, len(cache.seq_row0), len(prefix.seq_row0))
    wp, wb = _ws(ws)
    st = load_library().tria_attend_prefix(prefix.c_ref(), cache.c_ref(), seq0.ctypes.data, ctypes.byref(a), wp, wb, _stream_handle(stream))
    if st:
        _check(st, "tria_attend_prefix")


def beam_select_workspace_size(seq0, vocab: int, n_out: int) -> int:
    """tria_beam_select_workspace_size: seq0 host offsets of the groups' beams."""
    seq0 = np.ascontiguousarray(np.asarray(seq0, dtype=np.int32))
    n = load_library().tria_beam_select_workspace_size(seq0.ctypes.data, len(seq0) - 1, vocab, n_out)
    if n == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_beam_select_workspace_size")
    return n


def beam_select(logits, total, total_out, parent, token, *, ws, seq0=None, ended=None, ended_out=None, end_token: int = -1,
                in_place: bool = False, stream=None):
    """tria_beam_select: the best continuations of groups of beams. logits [beams][vocab] (float32, float16 or bfloat16,
    a row's values consecutive), total float32 [beams]; total_out float32, parent and token int32 [groups][n_out];
    seq0 host offsets of the groups' beams (None: equally many each); ended / ended_out int32 [beams] / [groups][n_out]
    or None. in_place: every surviving beam's best continuation in the beam's own place."""
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor [beams][vocab], a row's values consecutive")
    if parent.dim() != 2:
        raise ValueError("parent must be [groups][n_out]")
    n, vocab = logits.shape
    n_groups, n_out = parent.shape
    b = _Beams()
    b.type, b.n_groups, b.vocab, b.n_out = _act_type(logits), n_groups, vocab, n_out
    seq0 = _groups(seq0, n, n_groups)
    b.seq0 = seq0.ctypes.data
    b.logits, b.stride = logits.data_ptr(), logits.stride(0) if n > 1 else max(logits.stride(0), vocab)
    b.total, b.total_out = _vec32(total, n, "total"), _vec32(total_out, n_groups * n_out, "total_out")
    for name, t, field, count in (("parent", parent, "parent_out", n_groups * n_out), ("token", token, "token_out", n_groups * n_out),
                                  ("ended", ended, "ended", n), ("ended_out", ended_out, "ended_out", n_groups * n_out)):
        if t is not None:
            if t.numel() != count or t.dtype not in _INT32 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {count} values")
            setattr(b, field, t.data_ptr())
    b.end_token, b.in_place = int(end_token), int(in_place)
    wp, wb = _ws(ws)
    st = load_library().tria_beam_select(ctypes.byref(b), wp, wb, _stream_handle(stream))
    if st:
        _check(st, "tria_beam_select")


def _layers(caches):
    if not caches:
        raise ValueError("at least one layer")
    return (_LayerCache * len(caches))(*[c.c_ref()._obj for c in caches])


def reorder_workspace_size(caches, seq0=None) -> int:
    """tria_reorder_workspace_size."""
    structs = _layers(caches)
    seq0 = _groups(seq0, len(caches[0].seq_row0))
    n = load_library().tria_reorder_workspace_size(structs, len(caches), seq0.ctypes.data, len(seq0) - 1)
    if n == 0:
        raise TriaError(ERR_INVALID_ARG, "tria_reorder_workspace_size")
    return n


def reorder(caches, parent, *, ws, seq0=None, stream=None):
    """tria_reorder: in every layer (caches: one LayerCache each), sequence s takes the live rows and n_live of sequence
    parent[s] (int32 CUDA tensor, one per sequence) of its group; seq0 host offsets of the groups' sequences (None: all
    sequences are one group)."""
    structs = _layers(caches)
    n_seqs = len(caches[0].seq_row0)
    seq0 = _groups(seq0, n_seqs)
    if not _ACT:
        _fill_types()
    if parent.numel() != n_seqs or parent.dtype not in _INT32 or not parent.is_contiguous() or not parent.is_cuda:
        raise ValueError(f"parent must be a contiguous int32 CUDA tensor of {n_seqs} sequences")
    wp, wb = _ws(ws)
    st = load_library().tria_reorder(structs, len(caches), seq0.ctypes.data, len(seq0) - 1, parent.data_ptr(), wp, wb, _stream_handle(stream))
    if st:
        _check(st, "tria_reorder")


# --------------------------------------------------------------------------- decode-loop lifecycle

def append(cache: LayerCache, k_new, v_new, pos_new, *, ws, k_scale_new=None, v_scale_new=None, stream=None):
    """tria_append: rows k_new / v_new [n_seqs][n_kv_heads][n_tokens][...] (cache dtypes) and
    pos_new int32 [n_seqs][n_tokens] after the live rows of every segment; n_live += n_tokens."""
    n_seqs = len(cache.seq_row0)
    if pos_new.dim() != 2 or pos_new.shape[0] != n_seqs or pos_new.dtype.itemsize != 4:
        raise ValueError("pos_new must be int32 [n_seqs][n_tokens]")
    n_tokens = int(pos_new.shape[-1])
    half_bytes = {F32: 8, F16: 4, Q8_0: 2, Q4_0: 1}
    for name, t, dt in (("k_new", k_new, cache.k_type), ("v_new", v_new, cache.v_type)):
        want = n_seqs * cache.n_kv_heads * n_tokens * cache.head_dim * half_bytes[dt] // 2
        if t is None or not t.is_contiguous() or t.numel() * t.element_size() != want:
            raise ValueError(f"{name} must be contiguous [n_seqs][n_kv_heads][n_tokens][head_dim] rows of the cache type")
    c = cache.c_struct()
    wp, wb = _ws(ws)
    _check(load_library().tria_append(ctypes.byref(c), _ptr(k_new), _ptr(k_scale_new), _ptr(v_new),
                                      _ptr(v_scale_new), _ptr(pos_new), n_tokens, wp, wb,
                                      _stream_handle(stream)), "tria_append")


class Schedule:
    """Decode-loop schedule (``tria_schedule``)."""

    def __init__(self, *, trigger: int = TRIGGER_LENGTH, kv_budget: int = 0, divide_length: int = 128,
                 count_prompt_tokens: bool = True, protect_prefill: bool = True, sink: int = 0,
                 window: int = 0, budget_frac: float = 0.0, n_ctx: int = 0):
        self.c = _Schedule(int(trigger), int(bool(count_prompt_tokens)), int(bool(protect_prefill)), int(sink),
                           int(window), 0, int(kv_budget), int(divide_length), float(budget_frac), int(n_ctx))
        _check(load_library().tria_schedule_check(ctypes.byref(self.c)), "tria_schedule_check")

    @property
    def window(self) -> int:
        return self.c.window


class Sequences:
    """The ``tria_seq_state`` of every sequence of a loop (host memory)."""

    def __init__(self, schedule: Schedule, capacity):
        self.schedule = schedule
        self.n = len(capacity)
        self.st = (_SeqState * self.n)()
        for s, cap in enumerate(capacity):
            _check(load_library().tria_seq_init(ctypes.byref(self.st[s]), int(cap)), "tria_seq_init")

    def prefill(self, s: int, n_tokens: int):
        _check(load_library().tria_seq_prefill(ctypes.byref(self.schedule.c), ctypes.byref(self.st[s]),
                                               int(n_tokens)), "tria_seq_prefill")

    def decode(self, s: int) -> bool:
        _check(load_library().tria_seq_decode(ctypes.byref(self.schedule.c), ctypes.byref(self.st[s])),
               "tria_seq_decode")
        return bool(self.st[s].due)

    def plan(self):
        """tria_schedule_plan: (budget_rows, sink_rows, cur_pos, n_due)."""
        b = np.zeros(self.n, np.int32)
        k = np.zeros(self.n, np.int32)
        p = np.zeros(self.n, np.int64)
        nd = ctypes.c_int32()
        i32p = ctypes.POINTER(ctypes.c_int32)
        _check(load_library().tria_schedule_plan(ctypes.byref(self.schedule.c), self.st, self.n,
                                                 b.ctypes.data_as(i32p), k.ctypes.data_as(i32p),
                                                 p.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                                 ctypes.byref(nd)), "tria_schedule_plan")
        return b, k, p, nd.value

    def policy(self) -> tuple:
        """(Policy of the planned pass, sequences due)."""
        b, k, p, nd = self.plan()
        return Policy(budget_rows=b, sink_rows=k, cur_pos=p, window=self.schedule.window,
                      sink=self.schedule.c.sink), nd

    def passed(self):
        _check(load_library().tria_schedule_passed(ctypes.byref(self.schedule.c), self.st, self.n),
               "tria_schedule_passed")

    def state(self, s: int) -> dict:
        return {name: getattr(self.st[s], name) for name, _ in _SeqState._fields_ if name != "pad"}


def raw_call(name: str, *args):
    """Call an entry point by name with ctypes arguments (used by the host tests)."""
    return getattr(load_library(), name)(*args)
