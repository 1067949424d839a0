"""Python binding of the int4g C ABI (libfl_int4g.so, declared in include/fl_int4g.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  The library
is loaded lazily and a missing library is an error: there is no fallback.

Function names match the C entry points.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

from . import _build

__all__ = [
    "lib", "Int4gError", "FL_SOFTMAX", "FL_SIGMOID", "GROUP",
    "fl_strerror", "fl_int4g_version", "fl_int4g_status",
    "fl_int4g_quantize", "fl_int4g_repacked_bytes", "fl_int4g_repack", "fl_int4g_unrepack",
    "fl_int4g_linear_workspace", "fl_int4g_linear", "fl_int4g_linear_noalloc", "fl_int4g_linear_noalloc_status",
    "fl_int4g_linear_g", "fl_moe_int4g_g",
    "fl_int4g_test_withhold_cluster_arrival", "fl_int4g_test_decode_plan",
    "fl_moe_int4g_workspace", "fl_moe_int4g", "fl_moe_int4g_ptrs", "FlMoeRouting", "fl_int4g_mlp_workspace",
    "fl_moe_router_logits_workspace", "fl_moe_router_logits",
    "fl_int4g_mlp", "fl_int4g_mlp_fused",
    "FL_KV8_E4M3", "FL_KV8_INT8", "FlKv8Cache", "FlKv8Seqs",
    "fl_rmsnorm", "fl_rope", "fl_kv8_append", "fl_kv8_attention_workspace", "fl_kv8_attention",
    "fl_kv8_test_pages", "fl_kv8_test_units", "fl_kv8_test_plan",
]

GROUP = 128
FL_SOFTMAX = 0
FL_SIGMOID = 1
FL_ROPE_HALVES = 0
FL_ROPE_PAIRS = 1
FL_KV8_E4M3 = 0
FL_KV8_INT8 = 1

_c_size_p = ctypes.POINTER(ctypes.c_size_t)
_vp = ctypes.c_void_p
_i = ctypes.c_int
_l = ctypes.c_int64


class FlMoeRouting(ctypes.Structure):
    """struct fl_moe_routing (routing options of fl_moe_int4g_ex)."""
    _fields_ = [("scoring", ctypes.c_int), ("renorm", ctypes.c_int), ("score_bias", ctypes.c_void_p),
                ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int), ("routed_scale", ctypes.c_float)]


class FlKv8Cache(ctypes.Structure):
    """struct fl_kv8_cache (the 8-bit key/value cache)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int), ("block", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("format", ctypes.c_int)]


class FlKv8Seqs(ctypes.Structure):
    """struct fl_kv8_seqs (the sequences of one call)."""
    _fields_ = [("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("T", ctypes.c_int), ("B", ctypes.c_int), ("max_q", ctypes.c_int), ("max_blocks", ctypes.c_int)]


# C signatures: name -> (restype, argtypes)
SIGNATURES = {
    "fl_strerror": (ctypes.c_char_p, [_i]),
    "fl_int4g_version": (_i, []),
    "fl_int4g_status": (_i, [_vp, _vp, ctypes.POINTER(_i)]),
    "fl_int4g_quantize": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "fl_int4g_repacked_bytes": (_i, [_i, _i, _i, _c_size_p]),
    "fl_int4g_repack": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, ctypes.c_size_t, _vp]),
    "fl_int4g_unrepack": (_i, [_vp, ctypes.c_size_t, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "fl_int4g_linear_workspace": (_i, [_i, _i, _i, _c_size_p]),
    "fl_int4g_linear": (_i, [_vp, _i, _i, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_int4g_linear_g": (_i, [_vp, _i, _i, _vp, _i, _i, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_moe_int4g_g": (_i, [_vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(FlMoeRouting), _i, _vp, _vp, _vp, _vp,
                            _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_int4g_linear_noalloc": (_i, [_vp, _i, _i, _vp, _i, _vp, _vp]),
    "fl_int4g_linear_noalloc_status": (_i, [_vp, ctypes.POINTER(_i)]),
    "fl_int4g_test_withhold_cluster_arrival": (_i, [ctypes.c_longlong]),
    "fl_int4g_test_decode_plan": (_i, [_i, _i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_longlong)]),
    "fl_moe_int4g_workspace": (_i, [_i, _i, _i, _i, _i, _i, _c_size_p]),
    "fl_int4g_mlp_workspace": (_i, [_i, _i, _i, _c_size_p]),
    "fl_moe_router_logits_workspace": (_i, [_i, _i, _i, _c_size_p]),
    "fl_moe_router_logits": (_i, [_vp, _i, _i, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_int4g_mlp": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_int4g_mlp_fused": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_moe_int4g": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                          _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_moe_int4g_ex": (_i, [_vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(FlMoeRouting), _vp, _vp, _vp, _vp,
                             _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_moe_int4g_ptrs": (_i, [_vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(FlMoeRouting), _vp, _vp, _vp, _vp,
                               _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fl_rmsnorm": (_i, [_vp, _l, _vp, _l, _vp, ctypes.c_float, _i, _i, _i, _vp, _l, _vp, _l, _vp, _vp, _i, _vp]),
    "fl_rope": (_i, [_vp, _l, _i, _vp, _l, _i, _i, _i, _i, _i, _vp, _i, ctypes.POINTER(ctypes.c_int32), _vp,
                     _vp, _l, _vp, _l, _vp]),
    "fl_kv8_append": (_i, [_vp, _l, _vp, _l, _vp, _vp, _vp, _vp]),
    "fl_kv8_test_pages": (_i, [ctypes.POINTER(FlKv8Seqs), _i, _i, _i, _i, ctypes.POINTER(ctypes.c_longlong)]),
    "fl_kv8_test_units": (_i, [_i, _i, _i, _i, _i, ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)]),
    "fl_kv8_test_plan": (_i, [_i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_longlong)]),
    "fl_kv8_attention_workspace": (_i, [_i, _i, _i, _i, _i, _c_size_p]),
    "fl_kv8_attention": (_i, [_vp, _l, _i, _vp, _vp, ctypes.c_float, _i, _vp, _l, _vp, _vp, ctypes.c_size_t, _vp]),
}

_LIB = None


class Int4gError(RuntimeError):
    def __init__(self, where, code):
        super().__init__(f"{where}: {fl_strerror(code)} (status {code})")
        self.code = code


def lib():
    """The loaded C library (ctypes.CDLL).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError(
                f"{_build.LIB} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
        L = ctypes.CDLL(_build.LIB)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _check(where, rc):
    if rc != 0:
        raise Int4gError(where, rc)


def _device():
    """The current device's index (CUDA is up: the caller has a tensor on it)."""
    get = getattr(_TORCH._C, "_cuda_getDevice", None)
    return get() if get is not None else _TORCH.cuda.current_device()


def _stream(stream=None):
    torch = _torch()
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:   # the current stream's handle without building a Stream object
        return ctypes.c_void_p(raw(_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


_WS = {}
_OUTGROWN = []   # workspaces that a larger one has replaced: a captured graph may hold them


def _workspace(nbytes, device):
    """A zero-filled workspace per (device, stream), grown on demand.  One that
    is made while the stream is captured is zero-filled by the graph's replay
    alone, so it serves that one call."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    key = (device.index, raw(device.index) if raw is not None and device.index is not None
           else torch.cuda.current_stream(device).cuda_stream)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        if buf is not None:
            _OUTGROWN.append(buf)
            nbytes = max(nbytes, 2 * buf.numel())   # (so that those kept are smaller together than the last)
        buf = _WS[key] = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
    return buf


# ------------------------------------------------------------------ wrappers

def fl_strerror(code):
    return lib().fl_strerror(code).decode()


def fl_int4g_version():
    return lib().fl_int4g_version()


def fl_int4g_status(ws, stream=None):
    out = ctypes.c_int(0)
    _check("fl_int4g_status", lib().fl_int4g_status(_p(ws), _stream(stream), ctypes.byref(out)))
    return out.value


def fl_int4g_repacked_bytes(N, K, group=GROUP):
    out = ctypes.c_size_t(0)
    _check("fl_int4g_repacked_bytes", lib().fl_int4g_repacked_bytes(N, K, group, ctypes.byref(out)))
    return out.value


def fl_int4g_quantize(w, group=GROUP, check=True):
    """fp32 [N, K] CUDA tensor -> canonical (q uint8 [N, K/2], scales int16
    [N, G] holding fp16 bits, zeros uint8 [N, ceil(G/2)])."""
    torch = _torch()
    N, K = w.shape
    G = K // group
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, G), dtype=torch.int16, device=w.device)
    z = torch.empty((N, (G + 1) // 2), dtype=torch.uint8, device=w.device)
    st = torch.zeros(4, dtype=torch.int32, device=w.device)
    _check("fl_int4g_quantize", lib().fl_int4g_quantize(_p(w), N, K, group, _p(q), _p(s), _p(z), _p(st), _stream()))
    if check:
        _check("fl_int4g_quantize (device)", fl_int4g_status(st))
    return q, s, z


def fl_int4g_repack(q, s, z, N, K, group=GROUP):
    torch = _torch()
    nbytes = fl_int4g_repacked_bytes(N, K, group)
    w = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check("fl_int4g_repack",
           lib().fl_int4g_repack(_p(q), _p(s), _p(z), N, K, group, _p(w), nbytes, _stream()))
    return w


def fl_int4g_unrepack(w, N, K, group=GROUP):
    torch = _torch()
    G = K // group
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, G), dtype=torch.int16, device=w.device)
    z = torch.empty((N, (G + 1) // 2), dtype=torch.uint8, device=w.device)
    _check("fl_int4g_unrepack",
           lib().fl_int4g_unrepack(_p(w), w.numel(), N, K, group, _p(q), _p(s), _p(z), _stream()))
    return q, s, z


def fl_int4g_linear_workspace(M, N, K):
    out = ctypes.c_size_t(0)
    _check("fl_int4g_linear_workspace", lib().fl_int4g_linear_workspace(M, N, K, ctypes.byref(out)))
    return out.value


def fl_int4g_linear(x, w, N, y=None, ws=None, group=GROUP):
    """y[M, N] bf16 = x[M, K] bf16 . deq(W)^T, W given in the interleaved
    layout of groups of `group` (128 and 256 share one layout; 64 adds the
    side array: fl_int4g_linear_g)."""
    torch = _torch()
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if ws is None:   # (a caller's workspace is checked for size by the library)
        ws = _workspace(fl_int4g_linear_workspace(M, N, K), x.device)
    if group == GROUP:
        _check("fl_int4g_linear",
               lib().fl_int4g_linear(_p(x), M, K, _p(w), N, _p(y), _p(ws), ws.numel(), _stream()))
    else:
        _check("fl_int4g_linear_g",
               lib().fl_int4g_linear_g(_p(x), M, K, _p(w), N, int(group), _p(y), _p(ws), ws.numel(), _stream()))
    return y


def fl_int4g_linear_noalloc(x, w, N, y=None):
    """Decode linear (M <= 32) with no workspace: for callers that cannot
    allocate device memory where they call.  The library keeps the scratch in
    a fixed device array shared by all calls (do not overlap calls on the GPU);
    make the first call on a device before any stream capture."""
    torch = _torch()
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check("fl_int4g_linear_noalloc", lib().fl_int4g_linear_noalloc(_p(x), M, K, _p(w), N, _p(y), _stream()))
    return y


def fl_int4g_linear_noalloc_status(stream=None):
    """Reads and clears the status block of fl_int4g_linear_noalloc's
    library-held array on the current device (synchronizes the stream)."""
    out = ctypes.c_int(0)
    _check("fl_int4g_linear_noalloc_status", lib().fl_int4g_linear_noalloc_status(_stream(stream), ctypes.byref(out)))
    return out.value


def fl_int4g_test_withhold_cluster_arrival(ns):
    """Test hook: ns >= 0 makes the cluster reductions of later decode
    launches withhold one arrival, so their bounded wait runs out after ns
    nanoseconds and FL_ERR_TIMEOUT is recorded; ns < 0 turns it off."""
    lib().fl_int4g_test_withhold_cluster_arrival(int(ns))


def fl_int4g_test_decode_plan(M, N, K, sms, group=GROUP, glu=False, minb=0, max_cs=8):
    """Test hook: the decode kernel's plan for one shape, computed on the
    host without a GPU.  A dict of T, G, P, csize, stages, stage_bytes, smem,
    xr_stride, xr_off, red_off and zrow_off, or None when the kernel does not
    take the shape."""
    out = (ctypes.c_longlong * 11)()
    rc = lib().fl_int4g_test_decode_plan(M, N, K, sms, group, int(bool(glu)), minb, max_cs, out)
    if rc != 0:
        return None
    keys = ("T", "G", "P", "csize", "stages", "stage_bytes", "smem", "xr_stride", "xr_off", "red_off", "zrow_off")
    return dict(zip(keys, list(out)))


def fl_int4g_mlp_workspace(M, H, I):
    out = ctypes.c_size_t(0)
    _check("fl_int4g_mlp_workspace", lib().fl_int4g_mlp_workspace(M, H, I, ctypes.byref(out)))
    return out.value


def fl_int4g_mlp(x, w_gate, w_up, w_down, I, y=None, ws=None, one_launch=False):
    """Decode MLP block (M <= 8): y = D . (silu(G x) * (U x)), the three
    matrices in the interleaved layout (G, U: [I, H]; D: [H, I]).
    one_launch: the cooperative single-launch form (fl_int4g_mlp_fused)."""
    torch = _torch()
    M, H = x.shape
    if y is None:
        y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    nb = fl_int4g_mlp_workspace(M, H, I)
    if ws is None:
        ws = _workspace(nb, x.device)
    name = "fl_int4g_mlp_fused" if one_launch else "fl_int4g_mlp"
    _check(name, getattr(lib(), name)(_p(x), M, H, I, _p(w_gate), _p(w_up), _p(w_down), _p(y), _p(ws),
                                      ws.numel(), _stream()))
    return y


def fl_moe_int4g_workspace(M, E, k, H, I, has_shared):
    out = ctypes.c_size_t(0)
    _check("fl_moe_int4g_workspace",
           lib().fl_moe_int4g_workspace(M, E, k, H, I, int(bool(has_shared)), ctypes.byref(out)))
    return out.value


def fl_moe_int4g(x, logits, k, I, w13, w2, scoring=FL_SOFTMAX, renorm=True, shared_w13=None, shared_w2=None,
                 y=None, topk_ids=None, topk_w=None, expert_offsets=None, perm=None, ws=None,
                 score_bias=None, n_group=1, topk_group=1, routed_scale=1.0, group=GROUP):
    """Routed MoE layer.  w13 / w2: uint8 CUDA tensors holding the E
    interleaved expert matrices back to back.  Optional routing outputs are
    written when given.  score_bias (fp32 [E] CUDA tensor), n_group /
    topk_group and routed_scale are the routing options of fl_moe_int4g_ex;
    with their defaults this is fl_moe_int4g."""
    torch = _torch()
    M, H = x.shape
    E = logits.shape[1]
    if y is None:
        y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    has_shared = shared_w13 is not None
    nb = fl_moe_int4g_workspace(M, E, k, H, I, has_shared)
    if ws is None:
        ws = _workspace(nb, x.device)
    if group != GROUP:
        r = FlMoeRouting(scoring, int(bool(renorm)), _p(score_bias), int(n_group), int(topk_group),
                         float(routed_scale))
        _check("fl_moe_int4g_g",
               lib().fl_moe_int4g_g(_p(x), _p(logits), M, H, E, k, I, ctypes.byref(r), int(group),
                                    _p(w13), _p(w2), _p(shared_w13), _p(shared_w2), _p(y),
                                    _p(topk_ids), _p(topk_w), _p(expert_offsets), _p(perm),
                                    _p(ws), ws.numel(), _stream()))
        return y
    if score_bias is None and n_group <= 1 and routed_scale == 1.0:
        _check("fl_moe_int4g",
               lib().fl_moe_int4g(_p(x), _p(logits), M, H, E, k, I, scoring, int(bool(renorm)),
                                  _p(w13), _p(w2), _p(shared_w13), _p(shared_w2), _p(y),
                                  _p(topk_ids), _p(topk_w), _p(expert_offsets), _p(perm),
                                  _p(ws), ws.numel(), _stream()))
        return y
    r = FlMoeRouting(scoring, int(bool(renorm)), _p(score_bias), int(n_group), int(topk_group), float(routed_scale))
    _check("fl_moe_int4g_ex",
           lib().fl_moe_int4g_ex(_p(x), _p(logits), M, H, E, k, I, ctypes.byref(r),
                                 _p(w13), _p(w2), _p(shared_w13), _p(shared_w2), _p(y),
                                 _p(topk_ids), _p(topk_w), _p(expert_offsets), _p(perm),
                                 _p(ws), ws.numel(), _stream()))
    return y


def fl_moe_int4g_ptrs(x, logits, k, I, w13_list, w2_list, scoring=FL_SOFTMAX, renorm=True, shared_w13=None,
                      shared_w2=None, y=None, topk_ids=None, topk_w=None, expert_offsets=None, perm=None, ws=None,
                      score_bias=None, n_group=1, topk_group=1, routed_scale=1.0, tables=None):
    """Routed MoE layer with each expert's matrices in its own CUDA tensor
    (w13_list[e]: interleaved [2I, H], w2_list[e]: interleaved [H, I]).  The
    device tables of expert pointers are built here (int64 CUDA tensors) or
    taken from `tables` = (w13_table, w2_table) when given."""
    torch = _torch()
    M, H = x.shape
    E = logits.shape[1]
    if y is None:
        y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    if tables is None:
        tables = (torch.tensor([t.data_ptr() for t in w13_list], dtype=torch.int64, device=x.device),
                  torch.tensor([t.data_ptr() for t in w2_list], dtype=torch.int64, device=x.device))
    nb = fl_moe_int4g_workspace(M, E, k, H, I, shared_w13 is not None)
    if ws is None:
        ws = _workspace(nb, x.device)
    r = FlMoeRouting(scoring, int(bool(renorm)), _p(score_bias), int(n_group), int(topk_group), float(routed_scale))
    _check("fl_moe_int4g_ptrs",
           lib().fl_moe_int4g_ptrs(_p(x), _p(logits), M, H, E, k, I, ctypes.byref(r),
                                   _p(tables[0]), _p(tables[1]), _p(shared_w13), _p(shared_w2), _p(y),
                                   _p(topk_ids), _p(topk_w), _p(expert_offsets), _p(perm),
                                   _p(ws), ws.numel(), _stream()))
    return y


def fl_moe_router_logits_workspace(M, H, E):
    out = ctypes.c_size_t(0)
    _check("fl_moe_router_logits_workspace", lib().fl_moe_router_logits_workspace(M, H, E, ctypes.byref(out)))
    return out.value


def fl_moe_router_logits(x, w_router, logits=None, ws=None):
    """fp32 [M, E] router logits = x[M, H] . w_router[E, H]^T (bf16 inputs)."""
    torch = _torch()
    M, H = x.shape
    E = w_router.shape[0]
    if logits is None:
        logits = torch.empty((M, E), dtype=torch.float32, device=x.device)
    nb = fl_moe_router_logits_workspace(M, H, E)
    if ws is None:
        ws = _workspace(nb, x.device)
    _check("fl_moe_router_logits", lib().fl_moe_router_logits(_p(x), M, H, _p(w_router), E, _p(logits), _p(ws),
                                                               ws.numel(), _stream()))
    return logits


# ------------------------------------------------- decoder-layer operators
# These calls sit between the linears of a decode step, where the host's time
# for a call counts: pointers go as plain integers, and the two structures of a
# cache call as packed bytes.

_KV8_CACHE = struct.Struct("PPPPiiiii")   # struct fl_kv8_cache
_KV8_SEQS = struct.Struct("PPPiiii")      # struct fl_kv8_seqs


def _raise(name, what):
    raise ValueError(f"{name}: {what}")


def _ptr(t, dtype, name):
    """Address of a contiguous CUDA tensor of the given type."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        _raise(name, f"expected a contiguous {dtype} CUDA tensor, got {t.dtype}, strides {t.stride()}, on {t.device}")
    return t.data_ptr()


def _tokens(t, name):
    """(address, token stride) of bf16 [tokens, heads, width], or [tokens,
    width], whose heads are packed; tokens may be rows of a wider projection."""
    st, sh = t.stride(), t.shape
    if t.dtype is not _TORCH.bfloat16 or not t.is_cuda:
        _raise(name, f"expected a bfloat16 CUDA tensor, got {t.dtype} on {t.device}")
    if len(sh) == 3:
        n, h, w = sh
        if (st[2] != 1 and w > 1) or (st[1] != w and h > 1):
            _raise(name, "the heads of a token must be packed")
        return t.data_ptr(), st[0] if n > 1 else h * w   # (the stride of a single token means nothing)
    n, w = sh
    if st[1] != 1 and w > 1:
        _raise(name, "the columns of a row must be packed")
    return t.data_ptr(), st[0] if n > 1 else w


def fl_rmsnorm(x, weight=None, eps=1e-6, residual=None, y=None, residual_out=None, out8=False, group=0, need_y=True):
    """RMS norm of bf16 x [M, H] or [M, heads, H] (each row of H by itself) with
    the residual's addition.  Returns a dict: "y" (bf16, unless need_y is
    False), "residual" (bf16(x + residual), with a residual), and with out8
    "codes" (uint8, e4m3 bits) and "scales" (fp32 [..., H / group], or [..., 1]
    for group 0).  y and residual_out may be given, and may be x or residual."""
    torch = _torch()
    shape = x.shape
    if len(shape) == 2:
        M, H = shape
        heads = 1
    elif len(shape) == 3:
        M, heads, H = shape
    else:
        _raise("fl_rmsnorm", "x is [M, H] or [M, heads, H]")
    xp, xs = _tokens(x, "x")
    out = {}
    rp, rs, op, os_, yp, ys, cp, sp, wp = None, 0, None, 0, None, 0, None, None, None
    if residual is not None:
        if residual.shape != shape:
            _raise("fl_rmsnorm", "residual and x differ in shape")
        rp, rs = _tokens(residual, "residual")
        if residual_out is None:
            residual_out = out["residual"] = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
            op, os_ = residual_out.data_ptr(), heads * H
    if y is None:
        if need_y:
            y = out["y"] = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
            yp, ys = y.data_ptr(), heads * H
    else:
        if y.shape != shape:
            _raise("fl_rmsnorm", "y and x differ in shape")
        yp, ys = _tokens(y, "y")
        out["y"] = y
    if residual_out is not None and op is None:
        if residual_out.shape != shape:
            _raise("fl_rmsnorm", "residual_out and x differ in shape")
        op, os_ = _tokens(residual_out, "residual_out")
        out["residual"] = residual_out
    if out8:
        codes = out["codes"] = torch.empty(shape, dtype=torch.uint8, device=x.device)
        scales = out["scales"] = torch.empty((*shape[:-1], H // group if group else 1), dtype=torch.float32,
                                             device=x.device)
        cp, sp = codes.data_ptr(), scales.data_ptr()
    if weight is not None:
        if weight.numel() != H:
            _raise("fl_rmsnorm", "weight is [H]")
        wp = _ptr(weight, torch.bfloat16, "weight")
    _check("fl_rmsnorm", lib().fl_rmsnorm(xp, xs, rp, rs, wp, eps, M, heads, H, yp, ys, op, os_, cp, sp,
                                          group if out8 else 0, _stream()))
    return out


@functools.lru_cache(maxsize=256)
def _sections(sections):
    return (ctypes.c_int32 * len(sections))(*sections)


def fl_rope(q, k, positions, inv_freq, sections=None, halves=True, q_out=None, k_out=None):
    """Rotary positions of bf16 q [T, Hq, D] and k [T, Hk, D] (or None).
    positions: int32 [T] or [n_axes, T]; inv_freq: float64 [rot / 2]; sections:
    with several axes, how many consecutive pairs turn by each.  halves: pair i
    is elements i and i + rot / 2, else 2i and 2i + 1.  Returns (q_out, k_out);
    they may be q and k themselves."""
    torch = _torch()
    T, Hq, D = q.shape
    qp, qs = _tokens(q, "q")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
        qop, qos = q_out.data_ptr(), Hq * D
    elif q_out.shape != q.shape:
        _raise("fl_rope", "q_out and q differ in shape")
    else:
        qop, qos = _tokens(q_out, "q_out")
    kp, ks, kop, kos, Hk = None, 0, None, 0, 0
    if k is not None:
        Tk, Hk, Dk = k.shape
        if Tk != T or Dk != D:
            _raise("fl_rope", "q and k differ in tokens or width")
        kp, ks = _tokens(k, "k")
        if k_out is None:
            k_out = torch.empty((T, Hk, D), dtype=torch.bfloat16, device=q.device)
            kop, kos = k_out.data_ptr(), Hk * D
        elif k_out.shape != k.shape:
            _raise("fl_rope", "k_out and k differ in shape")
        else:
            kop, kos = _tokens(k_out, "k_out")
    psh = positions.shape
    axes = psh[0] if len(psh) == 2 else 1
    if len(psh) not in (1, 2) or psh[-1] != T or (sections is not None and len(sections) != axes):
        _raise("fl_rope", "positions are [n_axes, T], sections [n_axes]")
    _check("fl_rope", lib().fl_rope(qp, qs, Hq, kp, ks, Hk, T, D, 2 * inv_freq.numel(),
                                    FL_ROPE_HALVES if halves else FL_ROPE_PAIRS,
                                    _ptr(positions, torch.int32, "positions"), axes,
                                    _sections(tuple(sections)) if sections is not None else None,
                                    _ptr(inv_freq, torch.float64, "inv_freq"), qop, qos, kop, kos, _stream()))
    return q_out, k_out


def _kv8(where, T, heads, dim, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q, max_q, fmt):
    """The two structures of a cache call, from its tensors, and B and kv_heads."""
    torch = _TORCH
    shape = k_cache.shape
    nb, hk, block, d = shape
    if v_cache.shape != shape or k_scale.shape != shape[:2] or v_scale.shape != shape[:2]:
        _raise(where, "the caches are [blocks, kv_heads, block, head_dim], their scales [blocks, kv_heads]")
    if d != dim or (heads is not None and heads != hk):
        _raise(where, "the tokens and the cache differ in heads or width")
    B = kv_lens.numel()
    rows, most = block_table.shape
    if rows != B or (cu_q is not None and cu_q.numel() != B + 1):
        _raise(where, "block_table is [B, max_blocks], kv_lens [B], cu_q [B + 1]")
    if max_q is None:
        max_q = T // B if cu_q is None else T
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    return (_KV8_CACHE.pack(_ptr(k_cache, u8, "k_cache"), _ptr(v_cache, u8, "v_cache"), _ptr(k_scale, f32, "k_scale"),
                            _ptr(v_scale, f32, "v_scale"), nb, block, hk, d, fmt),
            _KV8_SEQS.pack(_ptr(cu_q, i32, "cu_q") if cu_q is not None else 0, _ptr(kv_lens, i32, "kv_lens"),
                           _ptr(block_table, i32, "block_table"), T, B, max_q, most), B, hk)


def fl_kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q=None, max_q=None,
                  fmt=FL_KV8_E4M3, status=None):
    """Writes bf16 k, v [T, kv_heads, head_dim] into the 8-bit cache (uint8
    [blocks, kv_heads, block, head_dim], scales fp32 [blocks, kv_heads]).
    Sequence b's rows cu_q[b] .. cu_q[b+1]-1 (None: T / B each) are the last of
    its kv_lens[b] tokens; token j lives in block block_table[b][j // block].
    max_q: at least the rows of every sequence; it may be larger.  A sequence
    whose lists name rows, or tokens past its table, that are not there is left
    out: nothing of it is written, and the status block says so.
    status: the status block to record device-side errors in (an int32 or uint8
    CUDA tensor of 16 bytes or a workspace; None: this stream's workspace, whose
    status nobody reads)."""
    _torch()
    T, h, d = k.shape
    if v.shape != k.shape:
        _raise("fl_kv8_append", "k and v differ in shape")
    kp, ks = _tokens(k, "k")
    vp, vs = _tokens(v, "v")
    c, s, _, _ = _kv8("fl_kv8_append", T, h, d, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q, max_q, fmt)
    if status is None:
        status = _workspace(256, k.device)
    elif status.numel() * status.element_size() < 16:
        _raise("fl_kv8_append", "the status block has 16 bytes")
    _check("fl_kv8_append", lib().fl_kv8_append(kp, ks, vp, vs, c, s, _p(status), _stream()))


def fl_kv8_test_pages(kv_lens, table, T, num_blocks, block, b, cu_q=None, max_q=None, window=0):
    """Test hook: what the cache kernels make of sequence b, from Python lists
    and without a GPU: a dict of start, rows, kv, write and read, the last two
    (first page, pages, pages without a block)."""
    def arr(v):
        return (ctypes.c_int32 * max(1, len(v)))(*v)
    B, flat = len(kv_lens), [i for row in table for i in row]
    lens, tab, cu = arr(kv_lens), arr(flat), arr(cu_q) if cu_q is not None else None

    def at(a):
        return ctypes.cast(a, ctypes.c_void_p) if a is not None else None
    s = FlKv8Seqs(at(cu), at(lens), at(tab), T, B, T if max_q is None else max_q, len(table[0]))
    out = (ctypes.c_longlong * 9)()
    _check("fl_kv8_test_pages", lib().fl_kv8_test_pages(ctypes.byref(s), num_blocks, block, window, b, out))
    return {"start": out[0], "rows": out[1], "kv": out[2], "write": tuple(out[3:6]), "read": tuple(out[6:9])}


def fl_kv8_test_units(n, kv, group, u=-1, window=0):
    """Test hook: (items, units) of a kv head in the attention of many rows, and
    for unit u also (item, index, units, first tile, last token + 1, first token)."""
    out = (ctypes.c_longlong * 8)()
    _check("fl_kv8_test_units", lib().fl_kv8_test_units(n, kv, group, 1, window, u, out))
    return tuple(out[:2]) if u < 0 else tuple(out[2:])


def fl_kv8_test_plan(T, B, max_q, Hq, kv_heads, head_dim):
    """Test hook: (rows, many, few, bytes): the bound on a sequence's rows, the
    attention kernels launched for it and the workspace bytes they reach."""
    out = (ctypes.c_longlong * 4)()
    _check("fl_kv8_test_plan", lib().fl_kv8_test_plan(T, B, max_q, Hq, kv_heads, head_dim, out))
    return tuple(out)


def fl_kv8_attention_workspace(T, B, Hq, kv_heads, head_dim):
    out = ctypes.c_size_t(0)
    _check("fl_kv8_attention_workspace",
           lib().fl_kv8_attention_workspace(T, B, Hq, kv_heads, head_dim, ctypes.byref(out)))
    return out.value


@functools.lru_cache(maxsize=4096)
def _kv8_workspace(device_index, T, B, Hq, kv_heads, head_dim):
    return fl_kv8_attention_workspace(T, B, Hq, kv_heads, head_dim)


def fl_kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q=None, max_q=None,
                     fmt=FL_KV8_E4M3, scale=None, window=0, out=None, return_lse=False, ws=None):
    """Attention of bf16 q [T, Hq, head_dim] over the 8-bit cache (tensors as
    for fl_kv8_append; kv_lens count the tokens already written, the rows of q
    among them).  Row i of a sequence sees the tokens up to its own position,
    with window > 0 only the last `window`.  scale: 1 / sqrt(head_dim) by
    default.  Returns out [T, Hq, head_dim], or (out, lse [T, Hq] fp32); out may
    not lie over q.  Rows of no sequence, or of one that is left out as in
    fl_kv8_append, are not written.
    ws: a workspace of the caller's, zero-filled before its first use; give one
    to calls that are captured in a graph (without one each captured call whose
    stream has none yet fills its own with zeros at every replay)."""
    torch = _torch()
    T, Hq, d = q.shape
    qp, qs = _tokens(q, "q")
    c, s, B, hk = _kv8("fl_kv8_attention", T, None, d, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_q,
                       max_q, fmt)
    device = q.device
    if out is None:
        out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=device)
        op, os_ = out.data_ptr(), Hq * d
    elif out.shape != q.shape:
        _raise("fl_kv8_attention", "out and q differ in shape")
    else:
        op, os_ = _tokens(out, "out")
    lse = torch.empty((T, Hq), dtype=torch.float32, device=device) if return_lse else None
    if ws is None:
        ws = _workspace(_kv8_workspace(device.index, T, B, Hq, hk, d), device)
    _check("fl_kv8_attention",
           lib().fl_kv8_attention(qp, qs, Hq, c, s, d ** -0.5 if scale is None else scale, window, op, os_,
                                  lse.data_ptr() if return_lse else None, _p(ws), ws.numel(), _stream()))
    return (out, lse) if return_lse else out
