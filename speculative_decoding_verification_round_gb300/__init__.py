"""Python binding of the verify-round library (libspecverify.so, sm_103a).

Argument marshalling only: every step of the verify round runs in the CUDA
kernels behind the C ABI declared in ``include/spec_verify.h``.  torch is used
for device memory and streams.  There is no CPU fallback: if the compiled
library is missing, loading fails loudly.

Functions keep the C names (``spec_linear_q``, ``spec_verify_round``, ...);
tensors are passed as device pointers, streams as ``torch.cuda.Stream`` (or
None for torch's current stream).
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libspecverify.so")

SPEC_OK = 0
SPEC_E_INVALID = -1
SPEC_E_SHAPE = -2
SPEC_E_CUDA = -3
SPEC_E_OOM = -4
SPEC_E_UNSUPPORTED = -5
SPEC_E_TIMEOUT = -6
SPEC_Q4, SPEC_Q6, SPEC_Q8 = 4, 6, 8
SPEC_MAX_NT = 16
SPEC_MAX_TREE = 64
SPEC_FILTERED = -3.4028234663852886e38
SPEC_ST_SLOT, SPEC_ST_PAGE, SPEC_ST_SHARED, SPEC_ST_FULL, SPEC_ST_TREE, SPEC_ST_TIMEOUT, SPEC_ST_BLOCK = (
    1, 2, 4, 8, 16, 32, 64)
SPEC_PROF_QKV, SPEC_PROF_O, SPEC_PROF_GATE_UP, SPEC_PROF_DOWN = 0, 1, 2, 3
SPEC_PROF_LM_HEAD, SPEC_PROF_ALL_GEMMS, SPEC_PROF_ATTN = 4, 5, 6

EXPORTED = ["spec_last_error", "spec_qmat_create", "spec_qmat_destroy", "spec_linear_q",
            "spec_linear_q_tc", "spec_model_set_tc_min_seqs",
            "spec_model_create", "spec_model_destroy", "spec_model_kv_cache", "spec_kv_fill",
            "spec_kv_read", "spec_model_debug_read",
            "spec_state_set", "spec_state_get", "spec_error_check", "spec_model_set_graphs",
            "spec_model_set_wait_budget", "spec_model_profile", "spec_model_profile_read",
            "spec_verify_attn", "spec_lm_head", "spec_accept_greedy",
            "spec_accept_stochastic", "spec_accept_stochastic_noalloc", "spec_verify_round",
            "spec_verify_round_host", "spec_depth_params_default", "spec_depth_ctl_create",
            "spec_depth_ctl_destroy", "spec_depth_ctl_next", "spec_depth_ctl_observe",
            "spec_depth_ctl_estimates", "spec_model_pages", "spec_pages_copy", "spec_pages_fork",
            "spec_pages_extend", "spec_pages_commit", "spec_pages_free", "spec_tree_attn",
            "spec_tree_attn_workspace", "spec_accept_tree", "spec_sample",
            "spec_sample_workspace", "spec_tree_set_wait_budget", "spec_pages_q4_copy",
            "spec_pages_q4_fork", "spec_pages_q4_extend", "spec_pages_q4_free", "spec_pages_q4_commit",
            "spec_pages_q4_read", "spec_tree_attn_q4", "spec_tree_attn_q4_workspace",
            "spec_block_digest", "spec_block_digest_q4", "spec_block_scores", "spec_block_select",
            "spec_block_attn", "spec_block_attn_q4"]

P = ctypes.c_void_p
I32 = ctypes.c_int32
U64 = ctypes.c_uint64
I64 = ctypes.c_int64
SZ = ctypes.c_size_t


class SpecError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"spec error {code}: {msg}")
        self.code = code


class spec_qweight(ctypes.Structure):
    _fields_ = [("qtype", I32), ("N", I32), ("K", I32), ("qs", P), ("qh", P), ("scales", P)]


class spec_model_desc(ctypes.Structure):
    _fields_ = [("n_layers", I32), ("hidden", I32), ("n_q_heads", I32), ("n_kv_heads", I32),
                ("head_dim", I32), ("ffn", I32), ("vocab", I32), ("max_ctx", I32),
                ("max_nt", I32), ("max_seqs", I32), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("use_rope", I32)]


class spec_model_weights(ctypes.Structure):
    _fields_ = [("embed", P), ("norm_w", P), ("wqkv", ctypes.POINTER(spec_qweight)),
                ("wo", ctypes.POINTER(spec_qweight)), ("wgu", ctypes.POINTER(spec_qweight)),
                ("wd", ctypes.POINTER(spec_qweight)), ("lm_head", spec_qweight)]


class spec_depth_params(ctypes.Structure):
    _fields_ = [("d_min", I32), ("d_max", I32), ("prior_accept", ctypes.c_double),
                ("prior_reject", ctypes.c_double), ("decay", ctypes.c_double),
                ("hysteresis", ctypes.c_double), ("cost_window", I32)]


class spec_pages(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("layer_stride", I64), ("n_layers", I32), ("n_pages", I32),
                ("n_kv_heads", I32), ("page_size", I32), ("head_dim", I32), ("n_slots", I32),
                ("max_pages", I32), ("table", P), ("refs", P), ("len", P)]


class spec_pages_q4(ctypes.Structure):
    _fields_ = [("k_qs", P), ("v_qs", P), ("k_scales", P), ("v_scales", P), ("layer_stride", I64),
                ("n_layers", I32), ("n_pages", I32), ("n_kv_heads", I32), ("page_size", I32),
                ("head_dim", I32), ("n_slots", I32), ("max_pages", I32), ("table", P), ("refs", P), ("len", P)]


class spec_digest(ctypes.Structure):
    _fields_ = [("data", P), ("layer_stride", I64), ("n_layers", I32), ("n_pages", I32), ("n_kv_heads", I32),
                ("page_size", I32), ("head_dim", I32), ("block", I32), ("n_slots", I32), ("max_pages", I32),
                ("table", P), ("len", P)]


class spec_tree(ctypes.Structure):
    _fields_ = [("n_seq", I32), ("nt", I32), ("n_q_heads", I32), ("window", I32), ("sinks", I32),
                ("scale", ctypes.c_float), ("slots", P), ("parents", P), ("n_nodes", P)]


class spec_sampling(ctypes.Structure):
    _fields_ = [("greedy", I32), ("temperature", ctypes.c_float), ("seed", U64)]


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            sig = {
                "spec_last_error": (None, [ctypes.c_char_p, ctypes.c_size_t]),
                "spec_qmat_create": (I32, [ctypes.POINTER(spec_qweight), I32, P, ctypes.POINTER(P)]),
                "spec_qmat_destroy": (I32, [P]),
                "spec_linear_q": (I32, [P, P, I32, P, P]),
                "spec_linear_q_tc": (I32, [P, P, I32, P, P]),
                "spec_model_set_tc_min_seqs": (I32, [P, I32]),
                "spec_model_create": (I32, [ctypes.POINTER(spec_model_desc),
                                            ctypes.POINTER(spec_model_weights), P, ctypes.POINTER(P)]),
                "spec_model_destroy": (I32, [P]),
                "spec_model_kv_cache": (I32, [P, I32, ctypes.POINTER(P), ctypes.POINTER(P)]),
                "spec_kv_fill": (I32, [P, I32, I32, I32, I32, P, P, P]),
                "spec_kv_read": (I32, [P, I32, I32, I32, I32, P, P, P]),
                "spec_model_debug_read": (I32, [P, I32, P, ctypes.c_size_t, P]),
                "spec_state_set": (I32, [P, I32, P, P, P, P]),
                "spec_state_get": (I32, [P, I32, P, P, P, P]),
                "spec_error_check": (I32, [P, P, ctypes.POINTER(ctypes.c_uint32)]),
                "spec_model_set_graphs": (I32, [P, I32]),
                "spec_model_set_wait_budget": (I32, [P, I32]),
                "spec_model_profile": (I32, [P, I32]),
                "spec_model_profile_read": (I32, [P, I32, ctypes.POINTER(ctypes.c_double),
                                                  ctypes.POINTER(ctypes.c_int64),
                                                  ctypes.POINTER(ctypes.c_double),
                                                  ctypes.POINTER(ctypes.c_double)]),
                "spec_verify_attn": (I32, [P, I32, I32, P, I32, P, P, P, P, P]),
                "spec_lm_head": (I32, [P, P, I32, P, P, P]),
                "spec_accept_greedy": (I32, [P, P, I32, I32, P, P, P]),
                "spec_accept_stochastic": (I32, [P, P, P, I32, I32, I32, ctypes.c_float, U64,
                                                 P, P, P, P, P]),
                "spec_accept_stochastic_noalloc": (I32, [P, P, P, I32, I32, I32, ctypes.c_float,
                                                         U64, P, P, P, P, P]),
                "spec_verify_round": (I32, [P, I32, P, P, I32, P, ctypes.POINTER(spec_sampling),
                                            P, P, P, P]),
                "spec_verify_round_host": (I32, [P, I32, P, P, I32, P,
                                                 ctypes.POINTER(spec_sampling), P, P, P]),
                "spec_depth_params_default": (None, [ctypes.POINTER(spec_depth_params)]),
                "spec_depth_ctl_create": (I32, [ctypes.POINTER(spec_depth_params),
                                                ctypes.POINTER(P)]),
                "spec_depth_ctl_destroy": (I32, [P]),
                "spec_depth_ctl_next": (I32, [P, ctypes.POINTER(I32)]),
                "spec_depth_ctl_observe": (I32, [P, I32, I32, P, ctypes.c_double,
                                                 ctypes.POINTER(I32)]),
                "spec_depth_ctl_estimates": (I32, [P, P, P]),
                "spec_model_pages": (I32, [P, ctypes.POINTER(spec_pages)]),
                "spec_pages_copy": (I32, [P, I32, P, P, P, P, P]),
                "spec_pages_fork": (I32, [P, I32, P, P, P, P]),
                "spec_pages_extend": (I32, [P, I32, P, P, P, P, P]),
                "spec_pages_commit": (I32, [P, I32, P, I32, P, P, I64, P, P, P, P, P]),
                "spec_pages_free": (I32, [P, I32, P, P, P]),
                "spec_tree_attn": (I32, [P, I32, P, P, I64, P, P, I64, P, P, SZ, P, P]),
                "spec_tree_attn_workspace": (I32, [P, I32, I32, I32, P]),
                "spec_accept_tree": (I32, [P, P, P, P, I32, I32, P, P, P, P]),
                "spec_sample": (I32, [P, I32, I32, I64, P, P, P, P, P, P, P, P, I64, P, SZ, P]),
                "spec_sample_workspace": (I32, [I32, I32, P]),
                "spec_tree_set_wait_budget": (I32, [I32]),
                "spec_pages_q4_copy": (I32, [P, I32, P, P, P, P, P]),
                "spec_pages_q4_fork": (I32, [P, I32, P, P, P, P]),
                "spec_pages_q4_extend": (I32, [P, I32, P, P, P, P, P]),
                "spec_pages_q4_free": (I32, [P, I32, P, P, P]),
                "spec_pages_q4_commit": (I32, [P, I32, P, I32, P, P, I64, P, P, P, P, P]),
                "spec_pages_q4_read": (I32, [P, I32, P, I32, P, P, P, P, I64, P, P]),
                "spec_tree_attn_q4": (I32, [P, I32, P, P, I64, P, P, I64, P, P, SZ, P, P]),
                "spec_tree_attn_q4_workspace": (I32, [P, I32, I32, I32, P]),
                "spec_block_digest": (I32, [P, P, I32, P, P, P, P]),
                "spec_block_digest_q4": (I32, [P, P, I32, P, P, P, P]),
                "spec_block_scores": (I32, [P, I32, I32, P, I32, P, I32, P, I64, P, I64, P, P]),
                "spec_block_select": (I32, [P, I32, I32, I32, P, I32, P, I32, P, I64, I32, I32, I32, P, P, P]),
                "spec_block_attn": (I32, [P, I32, P, I32, I32, P, P, I64, P, P, I64, P, P, P]),
                "spec_block_attn_q4": (I32, [P, I32, P, I32, I32, P, P, I64, P, P, I64, P, P, P]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def last_error() -> str:
    buf = ctypes.create_string_buffer(1024)
    lib().spec_last_error(buf, 1024)
    return buf.value.decode(errors="replace")


def _check(rc: int):
    if rc != SPEC_OK:
        raise SpecError(rc, last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


_cuda_device = _cuda_raw_stream = None  # torch's current device, and its stream there as an address


def _init_cuda():
    global _cuda_device, _cuda_raw_stream
    import torch
    torch.cuda.current_stream()  # (initialises CUDA)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _cuda_raw_stream = raw or (lambda d: torch.cuda.current_stream(d).cuda_stream)
    _cuda_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here(stream):
    """The current device, and a stream as an address (None: torch's current one)."""
    if _cuda_device is None:
        _init_cuda()
    d = _cuda_device()
    return d, _cuda_raw_stream(d) if stream is None else stream.cuda_stream


def _stream(stream):
    return _here(None)[1] if stream is None else stream.cuda_stream


def _dev(t, device: int):
    """A tensor's address for a kernel on `device`: it has to be there, or in
    pinned host memory."""
    if t is None:
        return None
    if t.get_device() != device and (t.is_cuda or not t.is_pinned()):
        raise ValueError(f"a tensor on {t.device}: the current device's (or pinned host memory) is required")
    return t.data_ptr()


def _qweight(w: dict) -> spec_qweight:
    """dict(qtype, N, K, qs, qh, scales) of device tensors -> spec_qweight."""
    return spec_qweight(int(w["qtype"]), int(w["N"]), int(w["K"]), w["qs"].data_ptr(),
                        None if w.get("qh") is None else w["qh"].data_ptr(),
                        w["scales"].data_ptr())


# ---------------------------------------------------------------------------
# packed matrices and the verify GEMM
# ---------------------------------------------------------------------------
class QMat:
    """A block-quantised matrix repacked on the device (spec_qmat)."""

    def __init__(self, w: dict, max_rows: int = SPEC_MAX_NT, stream=None):
        self.handle = P()
        self.N, self.K, self.qtype = int(w["N"]), int(w["K"]), int(w["qtype"])
        qw = _qweight(w)
        _check(lib().spec_qmat_create(ctypes.byref(qw), int(max_rows), _stream(stream),
                                      ctypes.byref(self.handle)))

    def close(self):
        if self.handle:
            lib().spec_qmat_destroy(self.handle)
            self.handle = P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def spec_qmat_create(w: dict, max_rows: int = SPEC_MAX_NT, stream=None) -> QMat:
    return QMat(w, max_rows, stream)


def spec_linear_q(w: QMat, x, nt: int, y, stream=None):
    """y[nt][N] fp32 = W x[nt][K] (fp16); all device tensors."""
    _check(lib().spec_linear_q(w.handle, _ptr(x), int(nt), _ptr(y), _stream(stream)))


def spec_linear_q_tc(w: QMat, x, R: int, y, stream=None):
    """The same product on the tensor-core GEMM of multi-sequence rounds."""
    _check(lib().spec_linear_q_tc(w.handle, _ptr(x), int(R), _ptr(y), _stream(stream)))


# ---------------------------------------------------------------------------
# the decoder model
# ---------------------------------------------------------------------------
class Model:
    """spec_model: repacked weights, KV cache, per-sequence state."""

    def __init__(self, desc: dict, weights: dict, stream=None):
        d = spec_model_desc(int(desc["n_layers"]), int(desc["hidden"]),
                            int(desc.get("n_q_heads", 1)), int(desc.get("n_kv_heads", 1)),
                            int(desc.get("head_dim", 128)), int(desc.get("ffn", 32)),
                            int(desc["vocab"]), int(desc.get("max_ctx", 1)),
                            int(desc.get("max_nt", SPEC_MAX_NT)), int(desc.get("max_seqs", 1)),
                            float(desc.get("rms_eps", 1e-6)),
                            float(desc.get("rope_theta", 10000.0)),
                            int(desc.get("use_rope", 1)))
        self.desc = d
        L = d.n_layers
        arr = lambda key: (spec_qweight * max(L, 1))(*[_qweight(w) for w in weights.get(key, [])])
        self._keep = [arr("wqkv"), arr("wo"), arr("wgu"), arr("wd")]
        W = spec_model_weights(
            None if weights.get("embed") is None else weights["embed"].data_ptr(),
            weights["norm_w"].data_ptr(), self._keep[0], self._keep[1], self._keep[2],
            self._keep[3], _qweight(weights["lm_head"]))
        self.handle = P()
        _check(lib().spec_model_create(ctypes.byref(d), ctypes.byref(W), _stream(stream),
                                       ctypes.byref(self.handle)))

    def close(self):
        if self.handle:
            lib().spec_model_destroy(self.handle)
            self.handle = P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def kv_cache(self, layer: int):
        """(k, v) device pointers (ints) of one layer's cache
        [max_seqs][n_kv_heads][max_ctx][head_dim] fp16."""
        k, v = P(), P()
        _check(lib().spec_model_kv_cache(self.handle, int(layer), ctypes.byref(k), ctypes.byref(v)))
        return k.value, v.value

    def set_graphs(self, enable: bool):
        _check(lib().spec_model_set_graphs(self.handle, int(bool(enable))))

    def set_tc_min_seqs(self, min_seqs: int):
        """Rounds of at least min_seqs sequences use the tensor-core GEMM (0: never)."""
        _check(lib().spec_model_set_tc_min_seqs(self.handle, int(min_seqs)))

    def profile(self, enable: bool):
        """In-round kernel timing on (raw launches, events around each GEMM and
        attention launch) or off; clears the totals."""
        _check(lib().spec_model_profile(self.handle, int(bool(enable))))

    def profile_read(self, kind: int) -> dict:
        """Totals of one kernel class since the last profile() call."""
        t, b, f = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
        n = ctypes.c_int64()
        _check(lib().spec_model_profile_read(self.handle, int(kind), ctypes.byref(t),
                                             ctypes.byref(n), ctypes.byref(b), ctypes.byref(f)))
        return dict(seconds=t.value, launches=n.value, bytes=b.value, flops=f.value)

    def set_wait_budget(self, tries: int):
        """Test hook: try budget of each GEMM CTA's first copy wait (see the header)."""
        _check(lib().spec_model_set_wait_budget(self.handle, int(tries)))


def spec_kv_fill(m: Model, layer: int, seq: int, pos0: int, n_pos: int, k, v, stream=None):
    """k, v: fp16 tensors [n_kv_heads][n_pos][head_dim] (device or pinned host)."""
    _check(lib().spec_kv_fill(m.handle, int(layer), int(seq), int(pos0), int(n_pos), _ptr(k),
                              _ptr(v), _stream(stream)))


def spec_kv_read(m: Model, layer: int, seq: int, pos0: int, n_pos: int, k, v, stream=None):
    """Copies cache rows out into k, v: fp16 tensors [n_kv_heads][n_pos][head_dim]."""
    _check(lib().spec_kv_read(m.handle, int(layer), int(seq), int(pos0), int(n_pos), _ptr(k),
                              _ptr(v), _stream(stream)))


def spec_model_debug_read(m: Model, which: int, dst, stream=None):
    """Copies an internal activation buffer of the last pass into dst."""
    _check(lib().spec_model_debug_read(m.handle, int(which), _ptr(dst),
                                       dst.numel() * dst.element_size(), _stream(stream)))


def _host_array(values, ctype):
    if values is None:
        return None
    vals = [int(v) for v in values]
    return (ctype * len(vals))(*vals)


def spec_state_set(m: Model, seq_ids, n_past=None, emit_idx=None, anchor=None):
    n = len(seq_ids)
    _check(lib().spec_state_set(m.handle, n, _host_array(seq_ids, ctypes.c_int32),
                                _host_array(n_past, ctypes.c_int32),
                                _host_array(emit_idx, ctypes.c_uint64),
                                _host_array(anchor, ctypes.c_int32)))


def spec_state_get(m: Model, seq_ids):
    n = len(seq_ids)
    a = (ctypes.c_int32 * n)()
    b = (ctypes.c_uint64 * n)()
    c = (ctypes.c_int32 * n)()
    _check(lib().spec_state_get(m.handle, n, _host_array(seq_ids, ctypes.c_int32), a, b, c))
    return list(a), list(b), list(c)


def spec_error_check(m: Model | None = None, stream=None) -> int:
    """Synchronises, returns and clears the device error bits (0 = none)."""
    bits = ctypes.c_uint32(0)
    rc = lib().spec_error_check(None if m is None else m.handle, _stream(stream),
                                ctypes.byref(bits))
    if rc not in (SPEC_OK, SPEC_E_INVALID):
        _check(rc)
    return int(bits.value)


def spec_verify_attn(m: Model, layer: int, n_seq: int, seq_ids, nt: int, q, k_new, v_new, out,
                     stream=None):
    _check(lib().spec_verify_attn(m.handle, int(layer), int(n_seq), _ptr(seq_ids), int(nt),
                                  _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), _stream(stream)))


def spec_lm_head(m: Model, x, R: int, logits=None, argmax=None, stream=None):
    _check(lib().spec_lm_head(m.handle, _ptr(x), int(R), _ptr(logits), _ptr(argmax),
                              _stream(stream)))


def spec_accept_greedy(argmax, draft, n_seq: int, d: int, n_acc, emitted, stream=None):
    _check(lib().spec_accept_greedy(_ptr(argmax), _ptr(draft), int(n_seq), int(d), _ptr(n_acc),
                                    _ptr(emitted), _stream(stream)))


def spec_accept_stochastic(p_logits, q_logits, draft, n_seq: int, d: int, V: int,
                           temperature: float, seed: int, seq_ids, emit_idx, n_acc, emitted,
                           stream=None):
    _check(lib().spec_accept_stochastic(_ptr(p_logits), _ptr(q_logits), _ptr(draft), int(n_seq),
                                        int(d), int(V), float(temperature), int(seed),
                                        _ptr(seq_ids), _ptr(emit_idx), _ptr(n_acc),
                                        _ptr(emitted), _stream(stream)))


def spec_accept_stochastic_noalloc(p_logits, q_logits, draft, n_seq: int, d: int, V: int,
                                   temperature: float, seed: int, seq_ids, emit_idx, n_acc,
                                   emitted, stream=None):
    """spec_accept_stochastic without any allocation (fixed scratch; see the header)."""
    _check(lib().spec_accept_stochastic_noalloc(_ptr(p_logits), _ptr(q_logits), _ptr(draft),
                                                int(n_seq), int(d), int(V), float(temperature),
                                                int(seed), _ptr(seq_ids), _ptr(emit_idx),
                                                _ptr(n_acc), _ptr(emitted), _stream(stream)))


def spec_verify_round(m: Model, n_seq: int, seq_ids, draft, d: int, q_logits=None,
                      greedy: bool = True, temperature: float = 1.0, seed: int = 0,
                      n_acc=None, emitted=None, logits_out=None, stream=None):
    sp = spec_sampling(int(bool(greedy)), float(temperature), int(seed))
    _check(lib().spec_verify_round(m.handle, int(n_seq), _ptr(seq_ids), _ptr(draft), int(d),
                                   _ptr(q_logits), ctypes.byref(sp), _ptr(n_acc), _ptr(emitted),
                                   _ptr(logits_out), _stream(stream)))


def _host_i32(a, n, name):
    """a as a C-contiguous int32 numpy array of at least n elements (no copy
    when it already is one)."""
    import numpy as np
    if not (type(a) is np.ndarray and a.dtype == np.int32 and a.flags.c_contiguous):
        a = np.ascontiguousarray(a, dtype=np.int32)
    if a.size < n:
        raise ValueError(f"{name}: {n} int32 values required, got {a.size}")
    return a


def spec_verify_round_host(m: Model, n_seq: int, seq_ids, draft, d: int, q_logits=None,
                           greedy: bool = True, temperature: float = 1.0, seed: int = 0,
                           n_acc=None, emitted=None, stream=None):
    """spec_verify_round with host (numpy int32) seq_ids, draft, n_acc and emitted;
    q_logits a device tensor, a (pinned) host tensor or a float32 numpy array.
    Returns (n_acc, emitted); they are valid on return (the call synchronises).
    n_acc / emitted, when given, must be C-contiguous int32 arrays (written in
    place)."""
    import numpy as np
    sid = _host_i32(seq_ids, n_seq, "seq_ids")
    dr = _host_i32(draft, n_seq * d, "draft") if d > 0 else None
    if n_acc is None:
        n_acc = np.empty(n_seq, np.int32)
    if emitted is None:
        emitted = np.empty((n_seq, d + 1), np.int32)
    for a, n, name in ((n_acc, n_seq, "n_acc"), (emitted, n_seq * (d + 1), "emitted")):
        if not (type(a) is np.ndarray and a.dtype == np.int32 and a.flags.c_contiguous
                and a.size >= n):
            raise ValueError(f"{name}: a C-contiguous int32 numpy array of {n} values is required")
    sp = spec_sampling(int(bool(greedy)), float(temperature), int(seed))
    if type(q_logits) is np.ndarray:  # host q_logits: copied by the library
        if not (q_logits.dtype == np.float32 and q_logits.flags.c_contiguous):
            raise ValueError("q_logits: a C-contiguous float32 array is required")
        qp = ctypes.c_void_p(q_logits.ctypes.data)
    else:
        qp = _ptr(q_logits)
    _check(lib().spec_verify_round_host(m.handle, int(n_seq), sid.ctypes.data,
                                        None if dr is None else dr.ctypes.data, int(d),
                                        qp, ctypes.byref(sp), n_acc.ctypes.data,
                                        emitted.ctypes.data, _stream(stream)))
    return n_acc, emitted


class DepthController:
    """The library's adaptive draft-depth controller (host only; rules in
    include/spec_verify.h).  Keyword arguments override the defaults."""

    def __init__(self, **kw):
        prm = spec_depth_params()
        lib().spec_depth_params_default(ctypes.byref(prm))
        for k, v in kw.items():
            setattr(prm, k, v)
        self.params = prm
        h = P()
        _check(lib().spec_depth_ctl_create(ctypes.byref(prm), ctypes.byref(h)))
        self.handle = h

    def next_depth(self) -> int:
        d = I32()
        _check(lib().spec_depth_ctl_next(self.handle, ctypes.byref(d)))
        return d.value

    def observe(self, d: int, n_acc, round_seconds: float) -> int:
        import numpy as np
        a = np.ascontiguousarray(n_acc, dtype=np.int32)
        nd = I32()
        _check(lib().spec_depth_ctl_observe(self.handle, int(d), int(a.size),
                                            a.ctypes.data if a.size else None,
                                            float(round_seconds), ctypes.byref(nd)))
        return nd.value

    def estimates(self):
        """(p[0..d_max], r[0..d_max]) as lists of floats."""
        n = self.params.d_max + 1
        p = (ctypes.c_double * n)()
        r = (ctypes.c_double * n)()
        _check(lib().spec_depth_ctl_estimates(self.handle, p, r))
        return list(p), list(r)

    def close(self):
        if self.handle:
            lib().spec_depth_ctl_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# drafted trees
# ---------------------------------------------------------------------------
class KVPages:
    """A paged KV cache (spec_pages) over the caller's tensors, which it keeps
    alive: k, v fp16 [n_layers][n_pages][n_kv_heads][page_size][head_dim]
    (a layer's pages contiguous), table int32 [n_slots][max_pages], lens
    int32 [n_slots], refs int32 [n_pages] (None: pages fixed to their slots).
    Without a table only spec_pages_copy takes it."""

    def __init__(self, k, v, table=None, lens=None, refs=None):
        n_layers, n_pages, n_kv_heads, page_size, head_dim = k.shape
        self.device = k.get_device()  # of a call; -1: any
        for t, name in ((v, "v"), (table, "table"), (lens, "lens"), (refs, "refs")):
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"{name}: a tensor on {t.device} beside a cache on {k.device}")
        if not all(t is None or t.is_cuda or t.is_pinned() for t in (k, v, table, lens, refs)):
            self.device = -2  # no kernel can read them
        for t, name in ((k, "k"), (v, "v")):
            if tuple(t.shape) != tuple(k.shape) or t.element_size() != 2 or not t[0].is_contiguous() or (
                    t.is_floating_point() and str(t.dtype) != "torch.float16"):
                raise ValueError(f"{name}: an fp16 tensor [n_layers][n_pages][n_kv_heads][page_size]"
                                 "[head_dim] with contiguous layers is required")
        if k.stride(0) != v.stride(0):
            raise ValueError("k and v must have the same layer stride")
        n_slots, max_pages = (0, 0) if table is None else table.shape
        for t, n, name in ((table, n_slots * max_pages, "table"), (lens, n_slots, "lens"),
                           (refs, n_pages, "refs")):
            if t is not None and (t.element_size() != 4 or t.is_floating_point()
                                  or not t.is_contiguous() or t.numel() != n):
                raise ValueError(f"{name}: a contiguous int32 tensor of {n} values is required")
        self._keep = (k, v, table, lens, refs)
        self.pages = spec_pages(k.data_ptr(), v.data_ptr(), k.stride(0), n_layers, n_pages,
                                n_kv_heads, page_size, head_dim, n_slots, max_pages,
                                None if table is None else table.data_ptr(),
                                None if refs is None else refs.data_ptr(),
                                None if lens is None else lens.data_ptr())
        self.ref = ctypes.byref(self.pages)

    def at(self, device: int):
        """The struct for a call on `device`."""
        if self.device != device and self.device != -1:
            raise ValueError("pages on another device than the current one" if self.device >= 0 else
                             "pages in host memory that is not pinned")
        return self.ref

    @classmethod
    def of_model(cls, m: Model) -> "KVPages":
        """The model's own slot cache (spec_model_pages): page id = slot."""
        self = cls.__new__(cls)
        self._keep = (m,)
        self.device = -1  # (the model's; not known here)
        self.pages = spec_pages()
        self.ref = ctypes.byref(self.pages)
        _check(lib().spec_model_pages(m.handle, self.ref))
        return self


def spec_model_pages(m: Model) -> KVPages:
    return KVPages.of_model(m)


def spec_pages_copy(kv: KVPages, n: int, src, dst, status, n_pos=None, stream=None):
    """Page src[i] to page dst[i], all layers; n_pos: only its first positions."""
    d, st = _here(stream)
    _check(lib().spec_pages_copy(kv.at(d), int(n), _dev(src, d), _dev(dst, d), _dev(n_pos, d), _dev(status, d),
                                 st))


def spec_pages_fork(kv: KVPages, n: int, src, dst, status, stream=None):
    """Slot dst[i] becomes a branch of slot src[i], sharing its pages."""
    d, st = _here(stream)
    _check(lib().spec_pages_fork(kv.at(d), int(n), _dev(src, d), _dev(dst, d), _dev(status, d), st))


def spec_pages_extend(kv: KVPages, n: int, slots, n_new, copies, status, stream=None):
    """Room for n_new[i] more positions of slot slots[i] (copy on write)."""
    d, st = _here(stream)
    _check(lib().spec_pages_extend(kv.at(d), int(n), _dev(slots, d), _dev(n_new, d), _dev(copies, d),
                                   _dev(status, d), st))


def spec_pages_commit(kv: KVPages, n: int, slots, nt: int, k_new, v_new, path, n_path, status,
                      new_len=None, new_layer_stride: int = 0, stream=None):
    """Rows path[i][:n_path[i]] of k_new / v_new [n_layers][n][nt][n_kv_heads]
    [head_dim] behind the committed positions of slot slots[i], all layers."""
    d, st = _here(stream)
    _check(lib().spec_pages_commit(kv.at(d), int(n), _dev(slots, d), int(nt), _dev(k_new, d), _dev(v_new, d),
                                   int(new_layer_stride), _dev(path, d), _dev(n_path, d), _dev(new_len, d),
                                   _dev(status, d), st))


def spec_pages_free(kv: KVPages, n: int, slots, status, stream=None):
    """Gives back every page of the slots."""
    d, st = _here(stream)
    _check(lib().spec_pages_free(kv.at(d), int(n), _dev(slots, d), _dev(status, d), st))


def spec_tree_attn_workspace(kv: KVPages, n_seq: int, nt: int, n_q_heads: int) -> int:
    """Bytes of workspace that spec_tree_attn needs for trees of this size."""
    b = SZ()
    _check(lib().spec_tree_attn_workspace(kv.ref, int(n_seq), int(nt), int(n_q_heads),
                                          ctypes.byref(b)))
    return b.value


def spec_tree_attn(kv: KVPages, layer: int, n_seq: int, slots, nt: int, n_q_heads: int, q, k_new,
                   v_new, out, workspace, status, parents=None, n_nodes=None, window: int = 0,
                   sinks: int = 0, scale: float = 0.0, q_stride: int = 0, kv_stride: int = 0,
                   stream=None):
    """Attention of n_seq trees of up to nt nodes over the pages of `layer`
    and over their own nodes (rules in include/spec_verify.h)."""
    d, st = _here(stream)
    t = spec_tree(n_seq, nt, n_q_heads, window, sinks, scale, _dev(slots, d), _dev(parents, d), _dev(n_nodes, d))
    _check(lib().spec_tree_attn(kv.at(d), int(layer), ctypes.byref(t), _dev(q, d), int(q_stride),
                                _dev(k_new, d), _dev(v_new, d), int(kv_stride), _dev(out, d),
                                _dev(workspace, d), workspace.numel() * workspace.element_size(),
                                _dev(status, d), st))


def spec_tree_set_wait_budget(tries: int):
    """Test hook: the budget of each CTA's first wait in this thread's later
    spec_tree_attn calls (0: it gives up at once; normally 131072)."""
    _check(lib().spec_tree_set_wait_budget(int(tries)))


def spec_accept_tree(argmax, tokens, parents, n_nodes, n_seq: int, nt: int, path, n_path, emitted,
                     stream=None):
    """Greedy acceptance along the trees; n_nodes None: nt each."""
    d, st = _here(stream)
    _check(lib().spec_accept_tree(_dev(argmax, d), _dev(tokens, d), _dev(parents, d), _dev(n_nodes, d),
                                  int(n_seq), int(nt), _dev(path, d), _dev(n_path, d), _dev(emitted, d),
                                  st))


def spec_sample_workspace(R: int, V: int) -> int:
    """Bytes of workspace that spec_sample needs for R rows of V logits (0: none)."""
    b = SZ()
    _check(lib().spec_sample_workspace(int(R), int(V), ctypes.byref(b)))
    return b.value


def spec_sample(logits, R: int, V: int, u, token, temperature=None, top_k=None, top_p=None,
                min_p=None, n_kept=None, filtered=None, ld: int = 0, ld_filtered: int = 0,
                workspace=None, stream=None):
    """One token per row from the random words u after temperature, top-k,
    top-p and min-p; filtered: the logits that stayed (SPEC_FILTERED elsewhere).
    workspace: a tensor of spec_sample_workspace bytes (None: taken from
    torch's allocator for the call where one is needed)."""
    d, st = _here(stream)
    at = _dev(logits, d)
    n = 0
    if workspace is not None:
        n = workspace.numel() * workspace.element_size()
    elif R * V > 2000000:  # (below, no call needs one)
        n = spec_sample_workspace(R, V)
        if n > 0:
            import contextlib
            import torch
            # (of the allocator's pool of the call's stream: behind that stream's work only)
            with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                workspace = torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", d))
    _check(lib().spec_sample(at, int(R), int(V), int(ld), _dev(u, d), _dev(temperature, d),
                             _dev(top_k, d), _dev(top_p, d), _dev(min_p, d), _dev(token, d), _dev(n_kept, d),
                             _dev(filtered, d), int(ld_filtered), _dev(workspace, d), n, st))


# ---------------------------------------------------------------------------
# long contexts: a cache in 4 bits
# ---------------------------------------------------------------------------
def _check_book(table, lens, refs, n_pages):
    """(n_slots, max_pages) of a cache's bookkeeping."""
    n_slots, max_pages = (0, 0) if table is None else table.shape
    for t, n, name in ((table, n_slots * max_pages, "table"), (lens, n_slots, "lens"), (refs, n_pages, "refs")):
        if t is not None and (t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous()
                              or t.numel() != n):
            raise ValueError(f"{name}: a contiguous int32 tensor of {n} values is required")
    return n_slots, max_pages


def _one_device(first, others):
    """The device of tensors that belong together (-2: no kernel can read them)."""
    device = first.get_device()
    for t, name in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{name}: a tensor on {t.device} beside one on {first.device}")
    return device if all(t is None or t.is_cuda or t.is_pinned() for t in (first, *(t for t, _ in others))) else -2


def _struct(x, kinds, device=None):
    """The struct of a cache or digest of one of `kinds` (another's has other
    fields), for a call on `device`."""
    if not isinstance(x, kinds):
        names = " or ".join(k.__name__ for k in (kinds if isinstance(kinds, tuple) else (kinds,)))
        raise TypeError(f"{type(x).__name__}: {names} is required")
    if device is not None and x.device not in (device, -1):
        raise ValueError("pages on another device than the current one" if x.device >= 0 else
                         "pages in host memory that is not pinned")
    return x.ref if isinstance(x, KVPages) else x._ref


class KVPagesQ4:
    """A paged KV cache in 4 bits (spec_pages_q4) over the caller's tensors,
    which it keeps alive: codes uint8 [n_layers][n_pages][n_kv_heads][page_size]
    [head_dim / 32][16] and scales fp16 [n_layers][n_pages][n_kv_heads]
    [page_size][head_dim / 32] (a layer's pages contiguous), table, lens and
    refs as in KVPages."""

    def __init__(self, k_qs, v_qs, k_scales, v_scales, table=None, lens=None, refs=None):
        n_layers, n_pages, n_kv_heads, page_size, blocks = k_scales.shape
        self.device = _one_device(k_qs, ((v_qs, "v_qs"), (k_scales, "k_scales"), (v_scales, "v_scales"),
                                         (table, "table"), (lens, "lens"), (refs, "refs")))
        rows = n_pages * n_kv_heads * page_size
        for t, name, bytes_, shape in ((k_qs, "k_qs", 1, (*k_scales.shape, 16)), (v_qs, "v_qs", 1, (*k_scales.shape, 16)),
                                       (k_scales, "k_scales", 2, k_scales.shape), (v_scales, "v_scales", 2, k_scales.shape)):
            if tuple(t.shape) != tuple(shape) or t.element_size() != bytes_ or not t[0].is_contiguous() or (
                    t.is_floating_point() and str(t.dtype) != "torch.float16"):
                raise ValueError(f"{name}: a tensor {tuple(shape)} of {bytes_}-byte values with contiguous layers is "
                                 "required")
        strides = {k_qs.stride(0) / (16 * blocks), v_qs.stride(0) / (16 * blocks), k_scales.stride(0) / blocks,
                   v_scales.stride(0) / blocks} if n_layers > 1 else {float(rows)}
        if len(strides) != 1 or not next(iter(strides)).is_integer():
            raise ValueError("codes and scales must have the same layer stride, in rows")
        n_slots, max_pages = _check_book(table, lens, refs, n_pages)
        self._keep = (k_qs, v_qs, k_scales, v_scales, table, lens, refs)
        self.pages = spec_pages_q4(k_qs.data_ptr(), v_qs.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                   int(strides.pop()), n_layers, n_pages, n_kv_heads, page_size, 32 * blocks,
                                   n_slots, max_pages, _ptr(table), _ptr(refs), _ptr(lens))
        self._ref = ctypes.byref(self.pages)


def spec_pages_q4_copy(kv: KVPagesQ4, n: int, src, dst, status, n_pos=None, stream=None):
    """spec_pages_copy for a cache in 4 bits."""
    d, st = _here(stream)
    _check(lib().spec_pages_q4_copy(_struct(kv, KVPagesQ4, d), int(n), _dev(src, d), _dev(dst, d), _dev(n_pos, d),
                                    _dev(status, d), st))


def spec_pages_q4_fork(kv: KVPagesQ4, n: int, src, dst, status, stream=None):
    """spec_pages_fork for a cache in 4 bits."""
    d, st = _here(stream)
    _check(lib().spec_pages_q4_fork(_struct(kv, KVPagesQ4, d), int(n), _dev(src, d), _dev(dst, d), _dev(status, d),
                                    st))


def spec_pages_q4_extend(kv: KVPagesQ4, n: int, slots, n_new, copies, status, stream=None):
    """spec_pages_extend for a cache in 4 bits."""
    d, st = _here(stream)
    _check(lib().spec_pages_q4_extend(_struct(kv, KVPagesQ4, d), int(n), _dev(slots, d), _dev(n_new, d),
                                      _dev(copies, d), _dev(status, d), st))


def spec_pages_q4_free(kv: KVPagesQ4, n: int, slots, status, stream=None):
    """spec_pages_free for a cache in 4 bits."""
    d, st = _here(stream)
    _check(lib().spec_pages_q4_free(_struct(kv, KVPagesQ4, d), int(n), _dev(slots, d), _dev(status, d), st))


def spec_pages_q4_commit(kv: KVPagesQ4, n: int, slots, nt: int, k_new, v_new, path, n_path, status,
                         new_len=None, new_layer_stride: int = 0, stream=None):
    """spec_pages_commit into a cache in 4 bits: fp16 rows are quantised on their way."""
    d, st = _here(stream)
    _check(lib().spec_pages_q4_commit(_struct(kv, KVPagesQ4, d), int(n), _dev(slots, d), int(nt), _dev(k_new, d),
                                      _dev(v_new, d), int(new_layer_stride), _dev(path, d), _dev(n_path, d), _dev(new_len, d),
                                      _dev(status, d), st))


def spec_pages_q4_read(kv: KVPagesQ4, n: int, slots, nt: int, pos0, n_pos, k, v, status,
                       layer_stride: int = 0, stream=None):
    """Positions pos0[i] + j, j < n_pos[i], of slot slots[i] as fp16 into row j of
    entry i of k and v [n_layers][n][nt][n_kv_heads][head_dim]."""
    d, st = _here(stream)
    _check(lib().spec_pages_q4_read(_struct(kv, KVPagesQ4, d), int(n), _dev(slots, d), int(nt), _dev(pos0, d),
                                    _dev(n_pos, d), _dev(k, d), _dev(v, d), int(layer_stride), _dev(status, d), st))


def spec_tree_attn_q4_workspace(kv: KVPagesQ4, n_seq: int, nt: int, n_q_heads: int) -> int:
    """Bytes of workspace that spec_tree_attn_q4 needs for trees of this size."""
    b = SZ()
    _check(lib().spec_tree_attn_q4_workspace(_struct(kv, KVPagesQ4), int(n_seq), int(nt), int(n_q_heads),
                                             ctypes.byref(b)))
    return b.value


def spec_tree_attn_q4(kv: KVPagesQ4, layer: int, n_seq: int, slots, nt: int, n_q_heads: int, q, k_new,
                      v_new, out, workspace, status, parents=None, n_nodes=None, window: int = 0,
                      sinks: int = 0, scale: float = 0.0, q_stride: int = 0, kv_stride: int = 0,
                      stream=None):
    """spec_tree_attn over a cache in 4 bits."""
    d, st = _here(stream)
    t = spec_tree(n_seq, nt, n_q_heads, window, sinks, scale, _dev(slots, d), _dev(parents, d), _dev(n_nodes, d))
    _check(lib().spec_tree_attn_q4(_struct(kv, KVPagesQ4, d), int(layer), ctypes.byref(t), _dev(q, d), int(q_stride),
                                   _dev(k_new, d), _dev(v_new, d), int(kv_stride), _dev(out, d),
                                   _dev(workspace, d), workspace.numel() * workspace.element_size(),
                                   _dev(status, d), st))


# ---------------------------------------------------------------------------
# long contexts: attention over selected blocks
# ---------------------------------------------------------------------------
class KVDigest:
    """The digests of a cache's blocks (spec_digest) over the caller's tensors,
    which it keeps alive: data fp16 [n_layers][n_pages][n_kv_heads]
    [page_size / block][2][head_dim] (a layer's contiguous), the cache's table
    and lens."""

    def __init__(self, data, block: int, table, lens):
        n_layers, n_pages, n_kv_heads, per, two, head_dim = data.shape
        self.device = _one_device(data, ((table, "table"), (lens, "lens")))
        if two != 2 or data.element_size() != 2 or not data[0].is_contiguous() or (
                data.is_floating_point() and str(data.dtype) != "torch.float16"):
            raise ValueError("data: an fp16 tensor [n_layers][n_pages][n_kv_heads][page_size / block][2][head_dim] "
                             "with contiguous layers is required")
        n_slots, max_pages = _check_book(table, lens, None, n_pages)
        self._keep = (data, table, lens)
        self.pages = spec_digest(data.data_ptr(), data.stride(0), n_layers, n_pages, n_kv_heads, per * int(block),
                                 head_dim, int(block), n_slots, max_pages, _ptr(table), _ptr(lens))
        self._ref = ctypes.byref(self.pages)


def spec_block_digest(dg: KVDigest, kv, n: int, slots, status, pos0=None, stream=None):
    """Digests of the blocks that hold positions [pos0[i], len) of slot slots[i],
    every layer; kv: a KVPages or KVPagesQ4 (spec_block_digest_q4)."""
    d, st = _here(stream)
    call = lib().spec_block_digest_q4 if isinstance(kv, KVPagesQ4) else lib().spec_block_digest
    _check(call(_struct(dg, KVDigest, d), _struct(kv, (KVPagesQ4, KVPages), d), int(n), _dev(slots, d),
                _dev(pos0, d), _dev(status, d), st))


def spec_block_digest_q4(dg: KVDigest, kv: KVPagesQ4, n: int, slots, status, pos0=None, stream=None):
    """spec_block_digest of a cache in 4 bits."""
    _struct(kv, KVPagesQ4)
    spec_block_digest(dg, kv, n, slots, status, pos0, stream)


def _rows_of_scores(scores):
    if scores.element_size() != 4 or not scores.is_floating_point() or not scores.is_contiguous():
        raise ValueError("scores: a contiguous fp32 tensor [n_seq][nt][n_kv_heads][blocks] is required")
    return scores.size(-1)


def spec_block_scores(dg: KVDigest, layer: int, n_seq: int, slots, nt: int, n_q_heads: int, q, scores,
                      status, n_nodes=None, q_stride: int = 0, stream=None):
    """Every block's score for each node's query: scores fp32 [n_seq][nt][n_kv_heads][ld]."""
    d, st = _here(stream)
    _check(lib().spec_block_scores(_struct(dg, KVDigest, d), int(layer), int(n_seq), _dev(slots, d), int(nt),
                                   _dev(n_nodes, d), int(n_q_heads), _dev(q, d), int(q_stride), _dev(scores, d),
                                   _rows_of_scores(scores), _dev(status, d), st))


def spec_block_select(lens, block: int, n_seq: int, slots, nt: int, n_kv_heads: int, scores, n_keep: int,
                      blocks, status, n_nodes=None, n_first: int = 1, n_last: int = 1, stream=None):
    """The first n_first, the last n_last and the largest-scored others of a row's
    blocks, ascending, -1 behind: blocks int32 [n_seq][nt][n_kv_heads][n_keep]."""
    d, st = _here(stream)
    if lens.element_size() != 4 or lens.is_floating_point() or not lens.is_contiguous():
        raise ValueError("lens: a contiguous int32 tensor is required")
    _check(lib().spec_block_select(_dev(lens, d), lens.numel(), int(block), int(n_seq), _dev(slots, d), int(nt),
                                   _dev(n_nodes, d), int(n_kv_heads), _dev(scores, d), _rows_of_scores(scores),
                                   int(n_keep), int(n_first), int(n_last), _dev(blocks, d), _dev(status, d), st))


def spec_block_attn(kv, layer: int, n_seq: int, slots, nt: int, n_q_heads: int, block: int, n_keep: int,
                    blocks, q, k_new, v_new, out, status, parents=None, n_nodes=None, scale: float = 0.0,
                    q_stride: int = 0, kv_stride: int = 0, stream=None):
    """Attention of the trees' nodes over the blocks of each node's and kv head's
    list and over themselves; kv: a KVPages or KVPagesQ4 (spec_block_attn_q4);
    status int32 [n_seq][nt][n_kv_heads]."""
    d, st = _here(stream)
    t = spec_tree(n_seq, nt, n_q_heads, 0, 0, scale, _dev(slots, d), _dev(parents, d), _dev(n_nodes, d))
    call = lib().spec_block_attn_q4 if isinstance(kv, KVPagesQ4) else lib().spec_block_attn
    _check(call(_struct(kv, (KVPagesQ4, KVPages), d), int(layer), ctypes.byref(t), int(block), int(n_keep),
                _dev(blocks, d), _dev(q, d), int(q_stride), _dev(k_new, d), _dev(v_new, d), int(kv_stride), _dev(out, d), _dev(status, d), st))


def spec_block_attn_q4(kv: KVPagesQ4, *args, **kw):
    """spec_block_attn over a cache in 4 bits."""
    _struct(kv, KVPagesQ4)
    spec_block_attn(kv, *args, **kw)
