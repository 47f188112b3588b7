"""kv_shared_b200 -- Python binding of libhs2, the B200 HySparse2 hybrid-block library.

Argument marshalling only: every function below forwards torch tensors (device
memory) and the current CUDA stream to the C ABI declared in include/hs2.h, with
the same names, and raises HS2Error on a non-OK status (through ctypes; the calls
around the block, some of which run for a few microseconds, through csrc/calls.c).  All computation runs in
the CUDA kernels of libhs2.so, on the current device; there is no fallback.  Build the library with
``python -m kv_shared_b200.build`` (or ``__graft_entry__.build()``).
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhs2.so")

HS2_F32, HS2_BF16, HS2_E4M3 = 0, 1, 2
HS2_OK, HS2_ERR_INVALID_ARG, HS2_ERR_UNSUPPORTED, HS2_ERR_WORKSPACE, HS2_ERR_CUDA, \
    HS2_ERR_TIMEOUT, HS2_ERR_INDEX = range(7)

EXPORTS = ("hs2_workspace_size", "hs2_workspace_init", "hs2_full_attn_select", "hs2_full_attn_launches",
           "hs2_topk_select",
           "hs2_sparse_attn", "hs2_sparse_attn_noalloc", "hs2_kv_bridge_proj", "hs2_kv_quantize_fp8", "hs2_last_status",
           "hs2_status_string", "hs2_qk_norm_rope", "hs2_window_workspace_size", "hs2_window_attn",
           "hs2_weight_accum_workspace_size", "hs2_weight_accum", "hs2_kv_evict")


class hs2_attn_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("window", ctypes.c_int32), ("budget", ctypes.c_int32),
                ("q_dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("idx_stride", ctypes.c_int32),
                ("kv_capacity", ctypes.c_int64), ("max_ctx", ctypes.c_int64)]


class hs2_rope_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n", "heads", "head_dim", "rot_dim", "interleaved",
                                              "normalize", "in_dtype", "kv_dtype")] + \
        [("eps", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("q_row", "k_row", "v_row", "kv_capacity")]


class hs2_evict_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "head_dim", "kv_dtype", "sinks", "window", "budget")] + \
        [("kv_capacity", ctypes.c_int64), ("out_capacity", ctypes.c_int64)]


class HS2Error(RuntimeError):
    def __init__(self, fn, status, why=""):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} ({status})" + (f": {why}" if why else ""))


_lib = None


def lib():
    """The loaded libhs2.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m kv_shared_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        dp = ctypes.POINTER(hs2_attn_desc)
        L.hs2_workspace_size.argtypes = [dp, i32]
        L.hs2_workspace_size.restype = sz
        L.hs2_workspace_init.argtypes = [vp, vp]
        L.hs2_full_attn_select.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.hs2_full_attn_launches.argtypes = [dp]
        L.hs2_topk_select.argtypes = [dp, vp, i64, vp, i32, vp, vp, vp, sz, vp]
        L.hs2_sparse_attn.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.hs2_sparse_attn_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.hs2_kv_bridge_proj.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, i64, vp, vp, vp, vp, vp]
        L.hs2_kv_quantize_fp8.argtypes = [vp, i64, i32, vp, vp, vp]
        L.hs2_last_status.argtypes = [vp, vp]
        L.hs2_status_string.argtypes = [ctypes.c_int]
        L.hs2_status_string.restype = ctypes.c_char_p
        rp, ep, f32 = ctypes.POINTER(hs2_rope_desc), ctypes.POINTER(hs2_evict_desc), ctypes.c_float
        L.hs2_qk_norm_rope.argtypes = [rp] + [vp] * 15
        L.hs2_window_workspace_size.argtypes = [dp, i32]
        L.hs2_window_workspace_size.restype = sz
        L.hs2_window_attn.argtypes = [dp, i32] + [vp] * 10 + [sz, vp]
        L.hs2_weight_accum_workspace_size.argtypes = [dp]
        L.hs2_weight_accum_workspace_size.restype = sz
        L.hs2_weight_accum.argtypes = [dp] + [vp] * 6 + [f32] + [vp] * 3 + [sz, vp]
        L.hs2_kv_evict.argtypes = [ep] + [vp] * 14
        for name in EXPORTS:
            if not name.endswith("workspace_size") and name != "hs2_status_string":
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


_bound = None


def _fast():
    """The calls around the block as functions that take tensors (csrc/calls.c); raises if it has not been built."""
    global _bound
    if _bound is None:
        L = lib()
        try:
            from kv_shared_b200 import _calls as m
        except ImportError as e:
            raise RuntimeError("kv_shared_b200/_calls.so is missing: build it with `python -m kv_shared_b200.build`") from e
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                 for f in (L.hs2_qk_norm_rope, L.hs2_window_attn, L.hs2_weight_accum, L.hs2_kv_evict)))
        _bound = m
    return _bound


# Addresses go over as plain integers (the argument types make pointers of them).
def _p(t):
    return None if t is None else t.data_ptr()


def _current_stream_getter(c):
    """A function that gives the current stream's handle (of the current device, d if the caller knows
    it): torch's own two calls below torch.cuda.current_stream() where `c` (torch._C) has them (0.1 us
    against 1), else that."""
    raw, device = getattr(c, "_cuda_getCurrentRawStream", None), getattr(c, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda d=None: torch.cuda.current_stream().cuda_stream
    return lambda d=None: raw(device() if d is None else d)


_current_stream = _current_stream_getter(torch._C)


def _stream(stream=None):
    return _current_stream() if stream is None else stream.cuda_stream


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_here(fn, stream, t):
    """_stream for a call around the block.  Its kernels run on the current device, where another device's
    or the host's memory is a fault, so one tensor of the call, t, is looked at (all of them would cost a
    single token's call a tenth of its time).  Beside a given stream only another device is refused."""
    if stream is None:
        here = _device()
        try:
            if t.get_device() != here:
                raise HS2Error(fn, HS2_ERR_INVALID_ARG, "a tensor is not on the current device")
        except AttributeError:                 # None, or an object that has an address alone
            pass
        return _current_stream(here)
    d = getattr(t, "get_device", lambda: -1)()
    if d >= 0 and (d != _device() or d != getattr(stream, "device_index", d)):
        raise HS2Error(fn, HS2_ERR_INVALID_ARG, "a tensor or the stream is not on the current device")
    return stream.cuda_stream


def _check(fn, status):
    if status != HS2_OK:
        raise HS2Error(fn, status)


def status_string(status):
    return lib().hs2_status_string(int(status)).decode()


def make_desc(batch, n_q, heads, head_dim, window=128, budget=1024, q_dtype=HS2_BF16,
              kv_dtype=HS2_BF16, softmax_scale=0.0, idx_stride=None, kv_capacity=None, max_ctx=None):
    d = hs2_attn_desc()
    d.batch, d.n_q, d.heads, d.head_dim = batch, n_q, heads, head_dim
    d.window, d.budget, d.q_dtype, d.kv_dtype = window, budget, q_dtype, kv_dtype
    d.softmax_scale = softmax_scale
    d.idx_stride = window + budget if idx_stride is None else idx_stride
    d.max_ctx = max_ctx
    d.kv_capacity = max_ctx if kv_capacity is None else kv_capacity
    return d


# ------------------------------------------------------------------ C-ABI calls
def hs2_workspace_size(desc, scores_in_workspace=True):
    return int(lib().hs2_workspace_size(ctypes.byref(desc), int(bool(scores_in_workspace))))


def hs2_full_attn_launches(desc):
    """Kernels one hs2_full_attn_select call with `desc` enqueues (host query)."""
    return int(lib().hs2_full_attn_launches(ctypes.byref(desc)))


def hs2_workspace_init(workspace, stream=None):
    _check("hs2_workspace_init", lib().hs2_workspace_init(_p(workspace), _stream(stream)))


def hs2_full_attn_select(desc, q, k, v, k_scale, v_scale, q_pos0, o, lse, idx, cnt, scores,
                         workspace, stream=None):
    st = lib().hs2_full_attn_select(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(k_scale), _p(v_scale),
                                    _p(q_pos0), _p(o), _p(lse), _p(idx), _p(cnt), _p(scores),
                                    _p(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check("hs2_full_attn_select", st)


def hs2_topk_select(desc, scores, score_row_stride, q_pos0, block_size, idx, cnt, workspace, stream=None):
    st = lib().hs2_topk_select(ctypes.byref(desc), _p(scores), int(score_row_stride), _p(q_pos0),
                               int(block_size), _p(idx), _p(cnt), _p(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check("hs2_topk_select", st)


def hs2_sparse_attn(desc, q, k, v, k_scale, v_scale, idx, cnt, o, lse, workspace, stream=None):
    st = lib().hs2_sparse_attn(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(k_scale), _p(v_scale),
                               _p(idx), _p(cnt), _p(o), _p(lse), _p(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check("hs2_sparse_attn", st)


def hs2_sparse_attn_noalloc(desc, q, k, v, k_scale, v_scale, idx, cnt, o, lse, stream=None):
    """hs2_sparse_attn without a workspace: for callers that cannot allocate device memory
    where they call us; scratch is a fixed array inside the library (see include/hs2.h)."""
    st = lib().hs2_sparse_attn_noalloc(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(k_scale), _p(v_scale),
                                       _p(idx), _p(cnt), _p(o), _p(lse), _stream(stream))
    _check("hs2_sparse_attn_noalloc", st)


def hs2_kv_bridge_proj(hidden, w_kv, batch, n, d_model, head_dim, pos0, kv_capacity, k, v,
                       kv_dtype=HS2_BF16, k_scale=None, v_scale=None, stream=None):
    st = lib().hs2_kv_bridge_proj(_p(hidden), _p(w_kv), batch, n, d_model, head_dim, _p(pos0),
                                  int(kv_dtype), int(kv_capacity), _p(k), _p(v), _p(k_scale), _p(v_scale),
                                  _stream(stream))
    _check("hs2_kv_bridge_proj", st)


def hs2_kv_quantize_fp8(src, rows, head_dim, codes, scales, stream=None):
    st = lib().hs2_kv_quantize_fp8(_p(src), int(rows), int(head_dim), _p(codes), _p(scales), _stream(stream))
    _check("hs2_kv_quantize_fp8", st)


def make_rope_desc(batch, n, heads, head_dim, rot_dim=None, interleaved=False, normalize=True, in_dtype=HS2_BF16,
                   kv_dtype=HS2_BF16, eps=1e-6, q_row=None, k_row=None, v_row=None, kv_capacity=None):
    d = hs2_rope_desc()
    d.batch, d.n, d.heads, d.head_dim = batch, n, heads, head_dim
    d.rot_dim = head_dim if rot_dim is None else rot_dim
    d.interleaved, d.normalize = int(bool(interleaved)), int(bool(normalize))
    d.in_dtype, d.kv_dtype, d.eps = in_dtype, kv_dtype, eps
    d.q_row = heads * head_dim if q_row is None else q_row
    d.k_row = head_dim if k_row is None else k_row
    d.v_row = head_dim if v_row is None else v_row
    d.kv_capacity = n if kv_capacity is None else kv_capacity
    return d


def make_evict_desc(batch, head_dim, kv_dtype=HS2_BF16, sinks=0, window=128, budget=1024, kv_capacity=None,
                    out_capacity=None):
    d = hs2_evict_desc()
    d.batch, d.head_dim, d.kv_dtype = batch, head_dim, kv_dtype
    d.sinks, d.window, d.budget = sinks, window, budget
    d.kv_capacity = kv_capacity
    d.out_capacity = sinks + window + budget if out_capacity is None else out_capacity
    return d


def hs2_qk_norm_rope(desc, q, k, v, q_weight, k_weight, inv_freq, row0, pos, n_rows, q_out, k_cache, v_cache,
                     k_scale=None, v_scale=None, stream=None):
    st = _fast().qk_norm_rope(desc, q, k, v, q_weight, k_weight, inv_freq, row0, pos, n_rows, q_out, k_cache, v_cache,
                              k_scale, v_scale, _stream_here("hs2_qk_norm_rope", stream, row0))
    _check("hs2_qk_norm_rope", st)


def hs2_window_workspace_size(desc, sinks=0):
    return int(lib().hs2_window_workspace_size(ctypes.byref(desc), int(sinks)))


def hs2_window_attn(desc, sinks, q, k, v, k_scale, v_scale, q_pos0, n_rows, o, lse, workspace, stream=None):
    st = _fast().window_attn(desc, int(sinks), q, k, v, k_scale, v_scale, q_pos0, n_rows, o, lse, workspace,
                             workspace.numel() * workspace.element_size(), _stream_here("hs2_window_attn", stream, q_pos0))
    _check("hs2_window_attn", st)


def hs2_weight_accum_workspace_size(desc):
    return int(lib().hs2_weight_accum_workspace_size(ctypes.byref(desc)))


def hs2_weight_accum(desc, q, k, k_scale, lse, q_pos0, n_rows, decay, acc_in, acc_out, workspace, stream=None):
    st = _fast().weight_accum(desc, q, k, k_scale, lse, q_pos0, n_rows, decay, acc_in, acc_out, workspace,
                              workspace.numel() * workspace.element_size(), _stream_here("hs2_weight_accum", stream, q_pos0))
    _check("hs2_weight_accum", st)


def hs2_kv_evict(desc, len_, acc, k, v, k_scale, v_scale, k_out, v_out, k_scale_out, v_scale_out, acc_out, idx,
                 new_len, stream=None):
    st = _fast().kv_evict(desc, len_, acc, k, v, k_scale, v_scale, k_out, v_out, k_scale_out, v_scale_out, acc_out, idx,
                          new_len, _stream_here("hs2_kv_evict", stream, len_))
    _check("hs2_kv_evict", st)


def hs2_last_status(workspace, stream=None):
    """Waits for the stream and returns (and clears) the device status word."""
    return int(lib().hs2_last_status(_p(workspace), _stream(stream)))


# ------------------------------------------------------------------ allocation helpers (plumbing)
def _alloc(fn, n, device):
    if n == 0:
        raise HS2Error(fn, HS2_ERR_INVALID_ARG)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    hs2_workspace_init(ws)
    return ws


def alloc_workspace(desc, scores_in_workspace=True, device="cuda"):
    return _alloc("hs2_workspace_size", hs2_workspace_size(desc, scores_in_workspace), device)


def alloc_window_workspace(desc, sinks=0, device="cuda"):
    return _alloc("hs2_window_workspace_size", hs2_window_workspace_size(desc, sinks), device)


def alloc_accum_workspace(desc, device="cuda"):
    return _alloc("hs2_weight_accum_workspace_size", hs2_weight_accum_workspace_size(desc), device)


__all__ = ["hs2_attn_desc", "hs2_rope_desc", "hs2_evict_desc", "HS2Error", "make_desc", "make_rope_desc",
           "make_evict_desc", "lib", "status_string", "alloc_workspace", "alloc_window_workspace",
           "alloc_accum_workspace",
           "HS2_F32", "HS2_BF16", "HS2_E4M3", "EXPORTS"] + list(EXPORTS)
