"""Thin ctypes binding of libdsa (include/dsa.h) with the same names.

Argument marshalling only: every step of both passes runs in the CUDA kernels
of libdsa.so.  Tensors are torch CUDA tensors; their data pointers and the
current CUDA stream are handed to the C ABI.  There is no fallback: if the
library is missing or no GPU is present, the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

DSA_OK = 0
DSA_ERR_INVALID_ARG = -1
DSA_ERR_UNSUPPORTED = -2
DSA_ERR_WORKSPACE_TOO_SMALL = -3
DSA_ERR_CUDA = -4
DSA_ERR_DEVICE_TIMEOUT = -5
DSA_ERR_BAD_INDEX = -6
DSA_ERR_NONFINITE = -7
DSA_ERR_SCRATCH_LIMIT = -8

# size of the library-held scratch array of dsa_select_static_scratch
DSA_SELECT_STATIC_SCRATCH_BYTES = 16 << 20

# smallest workspace of the operators that need only the status header
WORKSPACE_HEADER_BYTES = 4096

# every symbol include/dsa.h declares
EXPORTED = ("dsa_select", "dsa_sparse_attn", "dsa_select_workspace_size",
            "dsa_sparse_workspace_size", "dsa_workspace_init", "dsa_get_status",
            "dsa_strerror", "dsa_kernels_per_call", "dsa_select_launches", "dsa_version",
            "dsa_select_static_scratch",
            "dsa_merge_attn", "dsa_sparse_kernel",
            "dsa_qk_norm_rope", "dsa_window_attn", "dsa_window_workspace_size",
            "dsa_window_launches", "dsa_kv4_store", "dsa_kv4_load", "dsa_kv4_attn",
            "dsa_kv4_workspace_size", "dsa_kv4_launches")


class DsaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} (code {code})")
        self.code = code


class dsa_dims(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("B", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("page", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("kmax", ctypes.c_int32),
                ("n_phys", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("sm_limit", ctypes.c_int32), ("lse_out", ctypes.c_void_p),
                ("head_budget", ctypes.c_int32), ("active", ctypes.c_void_p),
                ("prefix_o_cache", ctypes.c_void_p), ("prefix_lse_cache", ctypes.c_void_p),
                ("early_gather", ctypes.c_int32)]


class dsa_rope(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("inv_freq", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("n_new", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


class dsa_window(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("n_new", ctypes.c_void_p)]


class dsa_kv4(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libdsa.so (raises if it has not been built); the binding's functions use
    the first library loaded."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = open_library(path)
    return _lib


def open_library(path: str):
    """A libdsa build at `path` with the C ABI's signatures declared, independent of
    the one the binding's functions use (e.g. a test build of the same sources)."""
    if not os.path.exists(path):
        raise RuntimeError(f"libdsa.so not built ({path}); run "
                           "`python -m block_sparse_attention_27_b200.build`")
    lib = ctypes.CDLL(path)
    vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dims_p = ctypes.POINTER(dsa_dims)
    lib.dsa_select.restype = ci
    lib.dsa_select.argtypes = [vp, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, dims_p, vp, vp, sz]
    lib.dsa_select_static_scratch.restype = ci
    lib.dsa_select_static_scratch.argtypes = [vp, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp,
                                              dims_p, vp, vp]
    lib.dsa_merge_attn.restype = ci
    lib.dsa_merge_attn.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int64, ctypes.c_int32, vp]
    lib.dsa_sparse_attn.restype = ci
    lib.dsa_sparse_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, dims_p, vp, vp, vp, sz]
    lib.dsa_select_workspace_size.restype = sz
    lib.dsa_select_workspace_size.argtypes = [dims_p]
    lib.dsa_sparse_workspace_size.restype = sz
    lib.dsa_sparse_workspace_size.argtypes = [dims_p]
    lib.dsa_workspace_init.restype = ci
    lib.dsa_workspace_init.argtypes = [vp, sz, vp]
    lib.dsa_get_status.restype = ci
    lib.dsa_get_status.argtypes = [vp, vp]
    lib.dsa_strerror.restype = ctypes.c_char_p
    lib.dsa_strerror.argtypes = [ci]
    lib.dsa_version.restype = ci
    lib.dsa_version.argtypes = []
    lib.dsa_kernels_per_call.restype = ci
    lib.dsa_kernels_per_call.argtypes = [ci]
    lib.dsa_select_launches.restype = ci
    lib.dsa_select_launches.argtypes = [dims_p]
    rope_p, win_p = ctypes.POINTER(dsa_rope), ctypes.POINTER(dsa_window)
    kv4_p = ctypes.POINTER(dsa_kv4)
    lib.dsa_qk_norm_rope.restype = ci
    lib.dsa_qk_norm_rope.argtypes = [vp] * 9 + [dims_p, rope_p, vp, vp, sz]
    lib.dsa_window_attn.restype = ci
    lib.dsa_window_attn.argtypes = [vp] * 7 + [dims_p, win_p, vp, vp, sz]
    lib.dsa_window_workspace_size.restype = sz
    lib.dsa_window_workspace_size.argtypes = [dims_p]
    lib.dsa_window_launches.restype = ci
    lib.dsa_window_launches.argtypes = [dims_p, win_p]
    lib.dsa_kv4_store.restype = ci
    lib.dsa_kv4_store.argtypes = [vp, vp, kv4_p, vp, dims_p, vp, vp, vp, sz]
    lib.dsa_kv4_load.restype = ci
    lib.dsa_kv4_load.argtypes = [kv4_p, vp, vp, vp, dims_p, vp, vp, vp, sz]
    lib.dsa_kv4_attn.restype = ci
    lib.dsa_kv4_attn.argtypes = [vp, kv4_p, vp, vp, vp, vp, vp, dims_p, vp, vp, vp, vp, sz]
    lib.dsa_kv4_workspace_size.restype = sz
    lib.dsa_kv4_workspace_size.argtypes = [dims_p]
    lib.dsa_kv4_launches.restype = ci
    lib.dsa_kv4_launches.argtypes = [dims_p, ctypes.c_int32]
    lib.dsa_sparse_kernel.restype = ci
    lib.dsa_sparse_kernel.argtypes = [dims_p]
    return lib


def kernels_per_call(pass_: int) -> int:
    """Kernel launches per call: 0 = dsa_select (groups in one launch), 1 = dsa_sparse_attn,
    2 = dsa_merge_attn, 3 = dsa_qk_norm_rope, 4 = dsa_kv4_store, 5 = dsa_kv4_load."""
    return int(load().dsa_kernels_per_call(int(pass_)))


def select_launches(dims: dsa_dims) -> int:
    """Kernel launches of one dsa_select call with these dims on the current device."""
    rc = int(load().dsa_select_launches(ctypes.byref(dims)))
    if rc < 0:
        raise DsaError(rc, "dsa_select_launches")
    return rc


def sparse_kernel(dims: dsa_dims) -> int:
    """1 = streaming sparse kernel, 1 + C = the all-keys-resident kernel in clusters of
    C CTAs, for these dims on the current device."""
    rc = int(load().dsa_sparse_kernel(ctypes.byref(dims)))
    if rc < 0:
        raise DsaError(rc, "dsa_sparse_kernel")
    return rc


def strerror(code: int) -> str:
    return load().dsa_strerror(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_dims(S, B, Hq, Hkv, d, page, max_pages, kmax, n_phys, page_table=None,
              sm_limit=0, head_budget=0, early_gather=0) -> dsa_dims:
    return dsa_dims(S, B, Hq, Hkv, d, page, max_pages, kmax, n_phys,
                    None if page_table is None else page_table.data_ptr(), int(sm_limit), None,
                    int(head_budget), None, None, None, int(early_gather))


def _with_lse(dims: dsa_dims, lse_out) -> dsa_dims:
    """dims for one call, with its optional log-sum-exp output (fp32 [S, B, Hq])."""
    if lse_out is None:
        return dims
    _check(lse_out, "lse_out", torch.float32)
    d = dsa_dims.from_buffer_copy(dims)
    d.lse_out = lse_out.data_ptr()
    return d


def dims_for(q_blk, k_cache, max_pages, kmax, page_table=None, sm_limit=0,
             head_budget=0, early_gather=0) -> dsa_dims:
    S, B, Hq, d = q_blk.shape
    n_phys, Hkv, page, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("q_blk and k_cache disagree on the head dimension")
    return make_dims(S, B, Hq, Hkv, d, page, max_pages, kmax, n_phys, page_table, sm_limit,
                     head_budget, early_gather)


def _check(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


class Workspace:
    """Device workspace for one stream of calls (zeroed header, sticky status word)."""

    def __init__(self, nbytes: int, device=None, stream=None):
        self.nbytes = int(nbytes)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        rc = load().dsa_workspace_init(_ptr(self.buf), self.nbytes, _stream(stream))
        if rc != DSA_OK:
            raise DsaError(rc, "dsa_workspace_init")

    def status(self, stream=None) -> int:
        return int(load().dsa_get_status(_ptr(self.buf), _stream(stream)))


def select_workspace_size(dims: dsa_dims) -> int:
    return int(load().dsa_select_workspace_size(ctypes.byref(dims)))


def sparse_workspace_size(dims: dsa_dims) -> int:
    return int(load().dsa_sparse_workspace_size(ctypes.byref(dims)))


def dsa_select(q_blk, k_cache, v_cache, n_ctx, page, topk, idx_out, o_out, stream=None, *,
               dims: dsa_dims, cnt_out, workspace: Workspace, lse_out=None):
    """Selection pass (see include/dsa.h).  All tensors on the GPU; raises DsaError."""
    _check(q_blk, "q_blk", torch.bfloat16, 4)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(n_ctx, "n_ctx", torch.int32)
    _check(topk, "topk", torch.int32)
    _check(idx_out, "idx_out", torch.int32)
    _check(o_out, "o_out", torch.bfloat16)
    _check(cnt_out, "cnt_out", torch.int32)
    dims = _with_lse(dims, lse_out)
    rc = load().dsa_select(_ptr(q_blk), _ptr(k_cache), _ptr(v_cache), _ptr(n_ctx), int(page),
                           _ptr(topk), _ptr(idx_out), _ptr(o_out), _stream(stream),
                           ctypes.byref(dims), _ptr(cnt_out), _ptr(workspace.buf), workspace.nbytes)
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_select")


def dsa_select_static_scratch(q_blk, k_cache, v_cache, n_ctx, page, topk, idx_out, o_out,
                              stream=None, *, dims: dsa_dims, cnt_out, status):
    """Selection pass with the library's static scratch instead of a workspace (see
    include/dsa.h).  `status` is a device int32/uint32 tensor of one element that
    holds 0 before the first call; read it with status_word().  Raises DsaError."""
    _check(q_blk, "q_blk", torch.bfloat16, 4)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(n_ctx, "n_ctx", torch.int32)
    _check(topk, "topk", torch.int32)
    _check(idx_out, "idx_out", torch.int32)
    _check(o_out, "o_out", torch.bfloat16)
    _check(cnt_out, "cnt_out", torch.int32)
    if status.dtype == torch.uint32:  # the same 4-byte word either way
        status = status.view(torch.int32)
    _check(status, "status", torch.int32)
    rc = load().dsa_select_static_scratch(_ptr(q_blk), _ptr(k_cache), _ptr(v_cache), _ptr(n_ctx),
                                          int(page), _ptr(topk), _ptr(idx_out), _ptr(o_out),
                                          _stream(stream), ctypes.byref(dims), _ptr(cnt_out),
                                          _ptr(status))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_select_static_scratch")


def status_word(status, stream=None) -> int:
    """dsa_get_status() of a caller-owned status word (synchronises `stream`)."""
    return int(load().dsa_get_status(_ptr(status), _stream(stream)))


def dsa_sparse_attn(q_blk, k_cache, v_cache, idx, blk_k, blk_v, o_out, stream=None, *,
                    dims: dsa_dims, n_ctx, idx_cnt, workspace: Workspace, lse_out=None,
                    active=None, prefix_o_cache=None, prefix_lse_cache=None):
    """Sparse pass (see include/dsa.h).  All tensors on the GPU; raises DsaError.
    active (uint8 [S, B]) with prefix_o_cache (bf16 [S, B, Hq, d]) and prefix_lse_cache
    (fp32 [S, B, Hq]): reuse of the prefix part for stable tokens."""
    _check(q_blk, "q_blk", torch.bfloat16, 4)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(idx, "idx", torch.int32)
    _check(blk_k, "blk_k", torch.bfloat16, 4)
    _check(blk_v, "blk_v", torch.bfloat16, 4)
    _check(o_out, "o_out", torch.bfloat16)
    _check(n_ctx, "n_ctx", torch.int32)
    _check(idx_cnt, "idx_cnt", torch.int32)
    dims = _with_lse(dims, lse_out)
    if active is not None:
        _check(active, "active", torch.uint8)
        _check(prefix_o_cache, "prefix_o_cache", torch.bfloat16)
        _check(prefix_lse_cache, "prefix_lse_cache", torch.float32)
        dims = dsa_dims.from_buffer_copy(dims)
        dims.active = active.data_ptr()
        dims.prefix_o_cache = prefix_o_cache.data_ptr()
        dims.prefix_lse_cache = prefix_lse_cache.data_ptr()
    rc = load().dsa_sparse_attn(_ptr(q_blk), _ptr(k_cache), _ptr(v_cache), _ptr(idx), _ptr(blk_k),
                                _ptr(blk_v), _ptr(o_out), _stream(stream), ctypes.byref(dims),
                                _ptr(n_ctx), _ptr(idx_cnt), _ptr(workspace.buf), workspace.nbytes)
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_sparse_attn")


def dsa_merge_attn(o_a, lse_a, o_b, lse_b, o_out, lse_out=None, stream=None):
    """Merge of two attention results over disjoint key sets (see include/dsa.h).
    o_*: bf16 [..., d] with the same leading shape; lse_*: fp32 over the leading shape."""
    for t, n in ((o_a, "o_a"), (o_b, "o_b"), (o_out, "o_out")):
        _check(t, n, torch.bfloat16)
    for t, n in ((lse_a, "lse_a"), (lse_b, "lse_b")):
        _check(t, n, torch.float32)
    if lse_out is not None:
        _check(lse_out, "lse_out", torch.float32)
    d = o_a.shape[-1]
    rows = o_a.numel() // d
    if o_b.shape != o_a.shape or o_out.shape != o_a.shape or lse_a.numel() != rows or lse_b.numel() != rows:
        raise ValueError("dsa_merge_attn: shapes disagree")
    rc = load().dsa_merge_attn(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(o_out),
                               _ptr(lse_out), rows, d, _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_merge_attn")


# ------------------------------------------- operators beside the two passes ----
def _int32(x) -> int:
    """A window or a count of sinks as 32 bits hold it: past them it is past every position, and one
    below zero stays so (ctypes would keep the low bits)."""
    return max(-1, min(int(x), 2 ** 31 - 1))


# A call's host time counts where its kernel takes a few microseconds: each tensor is checked
# in one expression, and the reason is worked out only where that fails.
def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, name, dtype, shape=None, dev=None):
    """Address of a contiguous tensor of that type and shape on the current device."""
    if dev is None:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        dev = torch.cuda.current_device()
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.get_device() != dev
            or (shape is not None and t.shape != shape) or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _ws(workspace, dev):
    buf = workspace.buf
    return _arg(buf, "workspace", torch.uint8, None, dev)


def _raw_stream(stream, dev):
    # (torch.cuda.current_stream() builds a Stream object, which takes as long as the call itself)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _call(rc, what):
    if rc != DSA_OK:
        raise DsaError(rc, what)


def rope_inv_freq(rot, base=10000.0, *, scaling=None, device="cuda"):
    """(inv_freq fp32 [rot/2], scale) of dsa_qk_norm_rope: radians per position of each pair,
    base ** (-2i / rot), computed in fp64, and the factor on cos and sin.

    scaling, for contexts longer than the trained one:
      None
      ("linear", f)      every position divided by f
      ("ntk", f)         the base raised so that the slowest pair is stretched f times
      ("yarn", f, n0)    the method of that name (Peng et al., 2023): pairs that turn more than 32
                         times within the trained length n0 are kept, those that turn less than
                         once are stretched f times, a linear ramp over the pair index between
                         (its ends rounded outwards); cos and sin times 0.1 ln f + 1
    """
    if rot < 8 or rot % 8:
        raise ValueError("rot must be a positive multiple of 8")
    if not base > 1:
        raise ValueError("the base must be greater than 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    freq, scale = float(base) ** (-2 * i / rot), 1.0
    if scaling is not None:
        kind, f = scaling[0], float(scaling[1])
        if f < 1:
            raise ValueError("the scaling factor must be at least 1")
        if kind == "linear":
            freq = freq / f
        elif kind == "ntk":
            freq = (float(base) * f ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == "yarn":
            n0 = float(scaling[2])

            def pair(turns):  # index of the pair that turns that often within n0 positions
                return rot * math.log(n0 / (turns * 2 * math.pi)) / (2 * math.log(base))

            lo = max(0.0, float(math.floor(pair(32.0))))
            hi = min(rot - 1.0, float(math.ceil(pair(1.0))))  # (past the last pair if all turn more than once)
            ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
            freq = freq * (1 - ramp) + freq / f * ramp
            scale = 0.1 * math.log(f) + 1.0
        else:
            raise ValueError(f"unknown scaling {kind!r}")
    return freq.to(torch.float32).to(device), scale


class Rope:
    """What dsa_qk_norm_rope needs of a layer: frequencies, layout and norm weights
    (include/dsa.h, dsa_rope).  Keeps the tensors alive."""

    def __init__(self, inv_freq, rot, *, interleaved=False, scale=1.0, eps=1e-6, q_norm=None,
                 k_norm=None):
        self.inv_freq, self.q_norm, self.k_norm = inv_freq, q_norm, k_norm
        self.rot, self.scale, self.eps = int(rot), float(scale), float(eps)
        self.interleaved = int(bool(interleaved))
        _arg(inv_freq, "inv_freq", torch.float32, (self.rot // 2,))
        for w, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if w is not None:
                _arg(w, name, torch.bfloat16)
                if w.dim() != 1:
                    raise ValueError(f"{name} must have one dimension")
        self.device = inv_freq.get_device()
        self.c = dsa_rope(self.rot, self.interleaved, self.eps, self.scale, inv_freq.data_ptr(), None,
                          None if q_norm is None else q_norm.data_ptr(),
                          None if k_norm is None else k_norm.data_ptr())


def _projection(t, name, S, B, H, d, dev):
    """Address and token stride of a projection [S, B, H, d] whose tokens may be a view into a
    packed row."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.get_device() != dev or t.shape != (S, B, H, d):
        _refuse(t, name, torch.bfloat16, (S, B, H, d), dev)
    st = t.stride()
    token = st[1] if B > 1 else st[0] if S > 1 else H * d
    if st[3] != 1 or (H > 1 and st[2] != d) or (S > 1 and st[0] != B * token):
        raise ValueError(f"{name}: a token's heads must be contiguous and the tokens evenly spaced")
    return t.data_ptr(), token


def dsa_qk_norm_rope(q, k, v, q_out, k_out=None, v_out=None, stream=None, *, dims: dsa_dims,
                     rope: Rope, n_ctx=None, workspace: Workspace, positions=None, n_new=None,
                     k_cache=None, v_cache=None):
    """Norm of each head's query and key, rotation by position, and append to the paged cache in
    one pass (see include/dsa.h).  q, k, v: bf16 [S, B, H, d], possibly views into a packed
    projection; k and v go to k_out / v_out (contiguous) and / or the cache."""
    S, B, Hq, Hkv, d = dims.S, dims.B, dims.Hq, dims.Hkv, dims.d
    bf, dev = torch.bfloat16, torch.cuda.current_device()
    for w in (rope.q_norm, rope.k_norm):
        if w is not None and w.numel() != d:
            raise ValueError(f"norm weights must have {d} elements")
    if rope.device != dev:
        raise ValueError(f"rope is on cuda:{rope.device}, the current device is cuda:{dev}")
    r = dsa_rope.from_buffer_copy(rope.c)
    if positions is not None:
        r.positions = _arg(positions, "positions", torch.int32, (S, B), dev)
    if n_new is not None:
        r.n_new = _arg(n_new, "n_new", torch.int32, (S,), dev)
    pq = pk = pv = None
    if q is not None:
        pq, r.q_stride = _projection(q, "q", S, B, Hq, d, dev)
    if k is not None:
        pk, r.k_stride = _projection(k, "k", S, B, Hkv, d, dev)
    if v is not None:
        pv, r.v_stride = _projection(v, "v", S, B, Hkv, d, dev)
    cache = (dims.n_phys, Hkv, dims.page, d)
    _call(load().dsa_qk_norm_rope(
        pq, pk, pv, _opt(q_out, "q_out", bf, (S, B, Hq, d), dev), _opt(k_out, "k_out", bf, (S, B, Hkv, d), dev),
        _opt(v_out, "v_out", bf, (S, B, Hkv, d), dev), _opt(k_cache, "k_cache", bf, cache, dev),
        _opt(v_cache, "v_cache", bf, cache, dev), _raw_stream(stream, dev), ctypes.byref(dims), ctypes.byref(r),
        _opt(n_ctx, "n_ctx", torch.int32, (S,), dev), _ws(workspace, dev), workspace.nbytes), "dsa_qk_norm_rope")


def window_workspace_size(dims: dsa_dims) -> int:
    return int(load().dsa_window_workspace_size(ctypes.byref(dims)))


def window_launches(dims: dsa_dims, window, sinks=0, causal=False) -> int:
    rc = int(load().dsa_window_launches(ctypes.byref(dims), ctypes.byref(dsa_window(
        _int32(window), _int32(sinks), int(bool(causal)), None))))
    if rc < 0:
        raise DsaError(rc, "dsa_window_launches")
    return rc


def dsa_window_attn(q_blk, k_cache, v_cache, blk_k, blk_v, o_out, stream=None, *, dims: dsa_dims,
                    window, sinks=0, causal=False, n_ctx, workspace: Workspace, n_new=None,
                    lse_out=None):
    """Attention with a sliding window and `sinks` first tokens that stay visible (see
    include/dsa.h).  blk_k = blk_v = None: the prefix alone."""
    S, B, Hq, Hkv, d = dims.S, dims.B, dims.Hq, dims.Hkv, dims.d
    bf, dev = torch.bfloat16, torch.cuda.current_device()
    cache, blk = (dims.n_phys, Hkv, dims.page, d), (S, B, Hkv, d)
    w = dsa_window(_int32(window), _int32(sinks), int(bool(causal)), _opt(n_new, "n_new", torch.int32, (S,), dev))
    dims = _with_lse_out(dims, lse_out, dev)
    _call(load().dsa_window_attn(
        _arg(q_blk, "q_blk", bf, (S, B, Hq, d), dev), _arg(k_cache, "k_cache", bf, cache, dev),
        _arg(v_cache, "v_cache", bf, cache, dev), _opt(blk_k, "blk_k", bf, blk, dev), _opt(blk_v, "blk_v", bf, blk, dev),
        _arg(o_out, "o_out", bf, (S, B, Hq, d), dev), _raw_stream(stream, dev), ctypes.byref(dims), ctypes.byref(w),
        _arg(n_ctx, "n_ctx", torch.int32, (S,), dev), _ws(workspace, dev), workspace.nbytes), "dsa_window_attn")


def _with_lse_out(dims: dsa_dims, lse_out, dev) -> dsa_dims:
    """dims for one call with its log-sum-exp output: that of the argument, else none (an address
    left in dims stands for a tensor that nobody has checked for this call)."""
    if lse_out is None and not dims.lse_out:
        return dims
    d = dsa_dims.from_buffer_copy(dims)
    d.lse_out = _opt(lse_out, "lse_out", torch.float32, (dims.S, dims.B, dims.Hq), dev)
    return d


class Kv4Cache:
    """A paged cache in 4 bits (include/dsa.h, dsa_kv4): k, v uint8 [n_phys, Hkv, page, d/2],
    k_scale, v_scale bf16 [n_phys, Hkv, page, d/32]."""

    GROUP = 32

    def __init__(self, k, v, k_scale, v_scale):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must have 4 dimensions")
        n_phys, Hkv, page, half = k.shape
        codes, scales = tuple(k.shape), (n_phys, Hkv, page, 2 * half // self.GROUP)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.shape = (n_phys, Hkv, page, 2 * half)
        self.c = dsa_kv4(_arg(k, "k", torch.uint8, codes), _arg(v, "v", torch.uint8, codes),
                         _arg(k_scale, "k_scale", torch.bfloat16, scales),
                         _arg(v_scale, "v_scale", torch.bfloat16, scales))

    @classmethod
    def zeros(cls, n_phys, Hkv, page, d, device=None):
        dev = device or "cuda"
        codes = [torch.zeros((n_phys, Hkv, page, d // 2), dtype=torch.uint8, device=dev) for _ in range(2)]
        scales = [torch.zeros((n_phys, Hkv, page, d // cls.GROUP), dtype=torch.bfloat16, device=dev) for _ in range(2)]
        return cls(*codes, *scales)

    def _fits(self, dims, dev):
        if self.shape != (dims.n_phys, dims.Hkv, dims.page, dims.d):
            raise ValueError(f"the 4-bit cache holds {self.shape}, dims say "
                             f"{(dims.n_phys, dims.Hkv, dims.page, dims.d)}")
        if self.k.get_device() != dev:
            raise ValueError(f"the 4-bit cache is on {self.k.device}, the current device is cuda:{dev}")
        return ctypes.byref(self.c)


def dsa_kv4_store(blk_k, blk_v, cache: Kv4Cache, stream=None, *, dims: dsa_dims, n_ctx,
                  workspace: Workspace, n_new=None):
    """Appends the block's keys and values to the 4-bit cache at n_ctx[s] + b (see include/dsa.h)."""
    bf, blk, dev = torch.bfloat16, (dims.S, dims.B, dims.Hkv, dims.d), torch.cuda.current_device()
    _call(load().dsa_kv4_store(
        _arg(blk_k, "blk_k", bf, blk, dev), _arg(blk_v, "blk_v", bf, blk, dev), cache._fits(dims, dev), _raw_stream(stream, dev),
        ctypes.byref(dims), _arg(n_ctx, "n_ctx", torch.int32, (dims.S,), dev),
        _opt(n_new, "n_new", torch.int32, (dims.S,), dev), _ws(workspace, dev), workspace.nbytes), "dsa_kv4_store")


def dsa_kv4_load(cache: Kv4Cache, k_out, v_out, stream=None, *, dims: dsa_dims, start,
                 workspace: Workspace, n_new=None):
    """Reads tokens start[s] + b of the 4-bit cache back in bf16 (see include/dsa.h)."""
    bf, blk, dev = torch.bfloat16, (dims.S, dims.B, dims.Hkv, dims.d), torch.cuda.current_device()
    _call(load().dsa_kv4_load(
        cache._fits(dims, dev), _arg(k_out, "k_out", bf, blk, dev), _arg(v_out, "v_out", bf, blk, dev), _raw_stream(stream, dev),
        ctypes.byref(dims), _arg(start, "start", torch.int32, (dims.S,), dev),
        _opt(n_new, "n_new", torch.int32, (dims.S,), dev), _ws(workspace, dev), workspace.nbytes), "dsa_kv4_load")


def kv4_workspace_size(dims: dsa_dims) -> int:
    return int(load().dsa_kv4_workspace_size(ctypes.byref(dims)))


def kv4_launches(dims: dsa_dims, sparse: bool) -> int:
    rc = int(load().dsa_kv4_launches(ctypes.byref(dims), int(bool(sparse))))
    if rc < 0:
        raise DsaError(rc, "dsa_kv4_launches")
    return rc


def dsa_kv4_attn(q_blk, cache: Kv4Cache, idx, blk_k, blk_v, o_out, stream=None, *, dims: dsa_dims,
                 n_ctx, workspace: Workspace, idx_cnt=None, n_new=None, lse_out=None):
    """The sparse pass over a 4-bit cache: the pages idx names, or every page where idx is None,
    and the block's own tokens (see include/dsa.h; dsa_select itself reads a bf16 cache only)."""
    S, B, Hq, Hkv, d = dims.S, dims.B, dims.Hq, dims.Hkv, dims.d
    bf, blk, dev = torch.bfloat16, (S, B, Hkv, d), torch.cuda.current_device()
    dims = _with_lse_out(dims, lse_out, dev)
    _call(load().dsa_kv4_attn(
        _arg(q_blk, "q_blk", bf, (S, B, Hq, d), dev), cache._fits(dims, dev),
        _opt(idx, "idx", torch.int32, (S, Hkv, dims.kmax), dev), _opt(blk_k, "blk_k", bf, blk, dev),
        _opt(blk_v, "blk_v", bf, blk, dev), _arg(o_out, "o_out", bf, (S, B, Hq, d), dev), _raw_stream(stream, dev),
        ctypes.byref(dims), _arg(n_ctx, "n_ctx", torch.int32, (S,), dev),
        _opt(idx_cnt, "idx_cnt", torch.int32, (S, Hkv), dev), _opt(n_new, "n_new", torch.int32, (S,), dev),
        _ws(workspace, dev), workspace.nbytes), "dsa_kv4_attn")


class DeviceWorkload:
    """A workload's tensors on the GPU plus the dims, outputs and workspaces of both passes."""

    def __init__(self, w, device="cuda", sm_limit=0, head_budget=0, early_gather=0):
        """head_budget=1: one budget of Hkv*kp pages per sequence shared by its KV heads;
        idx rows then hold up to min(max_pages, Hkv*kp) pages.  early_gather=1: sparse steps
        gather their pages before waiting for the kernel ahead of them (include/dsa.h)."""
        self.w = w
        dev = torch.device(device)
        self.q1 = w.q1.to(dev)
        self.k_cache = w.k_cache.to(dev)
        self.v_cache = w.v_cache.to(dev)
        self.blk_k1 = w.blk_k1.to(dev)
        self.blk_v1 = w.blk_v1.to(dev)
        self.n_ctx = w.n_ctx.to(dev)
        self.topk = w.topk.to(dev)
        self.page_table = None if w.page_table is None else w.page_table.to(dev)
        kmax = min(w.max_pages, w.Hkv * w.kmax) if head_budget else w.kmax
        self.kmax = kmax
        self.dims = dims_for(self.q1, self.k_cache, w.max_pages, kmax, self.page_table, sm_limit,
                             head_budget, early_gather)
        S, Hkv = w.S, w.Hkv
        self.idx = torch.full((S, Hkv, kmax), -1, dtype=torch.int32, device=dev)
        self.cnt = torch.zeros((S, Hkv), dtype=torch.int32, device=dev)
        self.o_sel = torch.zeros_like(self.q1)
        self.o_sp = torch.zeros_like(self.q1)
        self.ws_sel = Workspace(select_workspace_size(self.dims), dev)
        self.ws_sp = Workspace(sparse_workspace_size(self.dims), dev)

    def select(self, q=None, stream=None, lse_out=None):
        dsa_select(self.q1 if q is None else q, self.k_cache, self.v_cache, self.n_ctx,
                   self.w.P, self.topk, self.idx, self.o_sel, stream, dims=self.dims,
                   cnt_out=self.cnt, workspace=self.ws_sel, lse_out=lse_out)
        return self.idx, self.cnt, self.o_sel

    def sparse(self, q, blk_k, blk_v, idx=None, cnt=None, stream=None, out=None, lse_out=None,
               active=None, cache=None):
        """cache = (prefix_o_cache, prefix_lse_cache), used with `active`."""
        o = self.o_sp if out is None else out
        dsa_sparse_attn(q, self.k_cache, self.v_cache, self.idx if idx is None else idx, blk_k,
                        blk_v, o, stream, dims=self.dims, n_ctx=self.n_ctx,
                        idx_cnt=self.cnt if cnt is None else cnt, workspace=self.ws_sp,
                        lse_out=lse_out, active=active,
                        prefix_o_cache=None if cache is None else cache[0],
                        prefix_lse_cache=None if cache is None else cache[1])
        return o
