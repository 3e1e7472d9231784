"""Thin Python binding of liblsrm_nsa.so (the C ABI declared in include/lsrm_nsa.h).

Argument marshalling only: every function has the name of the C entry point it
calls, takes torch tensors that already live on the GPU (or None), passes their
device pointers and the current CUDA stream, and raises NsaError when the call
returns a status other than LSRM_OK.  All computation happens in the CUDA
kernels behind the ABI; there is no CPU path.  Importing works anywhere, but the
first call loads the library and fails loudly if it has not been built or no
GPU is present.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblsrm_nsa.so")

LSRM_OK = 0
STATUS = {0: "LSRM_OK", 1: "LSRM_ERR_INVALID_ARG", 2: "LSRM_ERR_UNSUPPORTED", 3: "LSRM_ERR_CUDA",
          4: "LSRM_ERR_TIMEOUT", 5: "LSRM_ERR_BOUNDS", 6: "LSRM_ERR_WORKSPACE"}
ROUTE_GIVEN, ROUTE_SCORE, ROUTE_GEOMETRIC, ROUTE_ALL = 0, 1, 2, 3

# every symbol include/lsrm_nsa.h declares
EXPORTS = ("lsrm_nsa_workspace_size", "lsrm_nsa_workspace_init", "lsrm_nsa_compress", "lsrm_route_score_topk",
           "lsrm_route_geometric", "lsrm_route_geometric_noalloc", "lsrm_route_camera", "lsrm_route_pooled_topk", "lsrm_nsa_cmp_attn", "lsrm_nsa_select_attn",
           "lsrm_nsa_window_attn", "lsrm_nsa_gate_combine", "lsrm_nsa_attend", "lsrm_nsa_mixture", "lsrm_nsa_forward", "lsrm_nsa_backward",
           "lsrm_relpos_workspace_size", "lsrm_relpos_workspace_init", "lsrm_relpos_log_buckets",
           "lsrm_relpos_forward", "lsrm_relpos_backward",
           "lsrm_layer_norm_forward", "lsrm_layer_norm_workspace_size", "lsrm_layer_norm_backward",
           "lsrm_nsa_last_device_status", "lsrm_status_string", "lsrm_diag_exp2_poly")


class NsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class Desc(ctypes.Structure):
    """lsrm_nsa_desc (host struct)."""
    _fields_ = [("n_tokens", ctypes.c_int64), ("n_blocks", ctypes.c_int32), ("max_block_len", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("pooled_q", ctypes.c_int32), ("n_gates", ctypes.c_int32), ("n_forced", ctypes.c_int32),
                ("forced_blocks", ctypes.c_void_p)]


def make_desc(n_tokens, n_blocks, max_block_len, n_q_heads, n_kv_heads, head_dim, top_k, window, scale=0.0,
              pooled_q=False, n_gates=3, forced: Optional[torch.Tensor] = None) -> Desc:
    if forced is not None and forced.numel() > 0:
        _check(forced, torch.int32, "forced")
        nf, fp = forced.numel(), forced.data_ptr()
    else:
        nf, fp = 0, None
    return Desc(int(n_tokens), int(n_blocks), int(max_block_len), int(n_q_heads), int(n_kv_heads), int(head_dim),
                int(top_k), int(window), float(scale), int(bool(pooled_q)), int(n_gates), nf, fp)


class RelposDesc(ctypes.Structure):
    """lsrm_relpos_desc (host struct)."""
    _fields_ = [("n_q_tokens", ctypes.c_int64), ("n_k_tokens", ctypes.c_int64), ("n_segs", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("n_buckets", ctypes.c_int32), ("max_distance", ctypes.c_int32),
                ("scale", ctypes.c_float)]


def make_relpos_desc(n_q_tokens, n_k_tokens, n_segs, n_q_heads, n_kv_heads, head_dim, n_axes, n_buckets,
                     max_distance, scale=0.0) -> RelposDesc:
    return RelposDesc(int(n_q_tokens), int(n_k_tokens), int(n_segs), int(n_q_heads), int(n_kv_heads), int(head_dim),
                      int(n_axes), int(n_buckets), int(max_distance), float(scale))


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblsrm_nsa.so; raise if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m block_sparse_gqa_nsa_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(Desc)
    R = ctypes.POINTER(RelposDesc)
    sigs = {
        "lsrm_nsa_workspace_size": ([D], sz),
        "lsrm_nsa_workspace_init": ([D, vp, sz, vp], ctypes.c_int),
        "lsrm_nsa_compress": ([D, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_route_score_topk": ([D, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_route_geometric": ([D, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_route_geometric_noalloc": ([D, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_route_pooled_topk": ([D, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_cmp_attn": ([D, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_select_attn": ([D, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_window_attn": ([D, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_gate_combine": ([D, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_attend": ([D, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_mixture": ([D, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_route_camera": ([D, vp, vp, i32, i32, vp, i32, i32, i32, vp, i32, i32, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_forward": ([D, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_nsa_backward": ([D, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_relpos_workspace_size": ([R], sz),
        "lsrm_relpos_workspace_init": ([R, vp, sz, vp], ctypes.c_int),
        "lsrm_relpos_log_buckets": ([i32, i32, vp], ctypes.c_int),
        "lsrm_relpos_forward": ([R] + [vp] * 12 + [sz, vp], ctypes.c_int),
        "lsrm_relpos_backward": ([R] + [vp] * 17 + [sz, vp], ctypes.c_int),
        "lsrm_layer_norm_forward": ([i64, i32, i32, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp], ctypes.c_int),
        "lsrm_layer_norm_workspace_size": ([i64, i32], sz),
        "lsrm_layer_norm_backward": ([i64, i32, i32] + [vp] * 9 + [sz, vp], ctypes.c_int),
        "lsrm_nsa_last_device_status": ([vp, vp], ctypes.c_int),
        "lsrm_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "lsrm_diag_exp2_poly": ([vp, vp, ctypes.c_int64, vp], ctypes.c_int),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _check(t: Optional[torch.Tensor], dtype, name: str, cuda: bool = True):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _call(name: str, *args):
    rc = getattr(load_library(), name)(*args)
    if rc != LSRM_OK:
        raise NsaError(name, rc)


def lsrm_nsa_workspace_size(desc: Desc) -> int:
    return int(load_library().lsrm_nsa_workspace_size(ctypes.byref(desc)))


def workspace(desc: Desc, device=None, stream=None) -> torch.Tensor:
    """Allocate (through torch) and zero the workspace the calls of this descriptor need."""
    n = lsrm_nsa_workspace_size(desc)
    if n == 0:
        raise NsaError("lsrm_nsa_workspace_size", 1)
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    lsrm_nsa_workspace_init(desc, ws, stream)
    return ws


def lsrm_nsa_workspace_init(desc: Desc, ws: torch.Tensor, stream=None):
    _check(ws, torch.uint8, "ws")
    _call("lsrm_nsa_workspace_init", ctypes.byref(desc), ws.data_ptr(), ws.numel(), _stream(stream))


def lsrm_nsa_compress(desc, off, q, k, v, kc32=None, kc=None, vc32=None, vc=None, qc32=None, qc=None, ws=None,
                      stream=None):
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (kc32, "kc32", torch.float32), (kc, "kc", torch.bfloat16),
                     (vc32, "vc32", torch.float32), (vc, "vc", torch.bfloat16), (qc32, "qc32", torch.float32),
                     (qc, "qc", torch.bfloat16)):
        _check(t, dt, n)
    _call("lsrm_nsa_compress", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(k), _ptr(v), _ptr(kc32), _ptr(kc),
          _ptr(vc32), _ptr(vc), _ptr(qc32), _ptr(qc), _ptr(ws), _stream(stream))


def lsrm_route_score_topk(desc, off, q, kc32, idx, score=None, ws=None, stream=None):
    _check(off, torch.int32, "off"); _check(q, torch.bfloat16, "q"); _check(kc32, torch.float32, "kc32")
    _check(idx, torch.int32, "idx"); _check(score, torch.float32, "score")
    _call("lsrm_route_score_topk", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(kc32), _ptr(idx), _ptr(score),
          _ptr(ws), _stream(stream))


def lsrm_route_geometric(desc, off, coords, idx, ws, stream=None):
    _check(off, torch.int32, "off"); _check(coords, torch.int32, "coords"); _check(idx, torch.int32, "idx")
    _call("lsrm_route_geometric", ctypes.byref(desc), _ptr(off), _ptr(coords), _ptr(idx), _ptr(ws),
          _stream(stream))


def lsrm_route_geometric_noalloc(desc, off, coords, idx, status=None, stream=None):
    """Geometric routing without a workspace, for callers that cannot allocate device memory
    (its scratch is a fixed array inside the library; at most 16384 blocks; calls that
    overlap on the GPU race).  `status` is an optional one-element device tensor that receives
    the bounds bit.  The C entry point declares it uint32_t*; torch has no unsigned 32-bit
    tensor type, so it is passed as torch.int32, which has the same size and layout (the bit
    LSRM_ERR_BOUNDS sets, 1 << 4, reads the same in either type)."""
    _check(off, torch.int32, "off"); _check(coords, torch.int32, "coords"); _check(idx, torch.int32, "idx")
    _check(status, torch.int32, "status")
    _call("lsrm_route_geometric_noalloc", ctypes.byref(desc), _ptr(off), _ptr(coords), _ptr(idx), _ptr(status),
          _stream(stream))


def lsrm_route_pooled_topk(desc, qc, kc, idx, ws, stream=None, qc32=None, kc32=None):
    """Speed3R routing from the bf16 pooled tensors; with the fp32 means qc32 / kc32 the ranking is
    that of the fp32 means (the exact mode)."""
    _check(qc, torch.bfloat16, "qc"); _check(kc, torch.bfloat16, "kc"); _check(idx, torch.int32, "idx")
    _check(qc32, torch.float32, "qc32"); _check(kc32, torch.float32, "kc32")
    _call("lsrm_route_pooled_topk", ctypes.byref(desc), _ptr(qc), _ptr(kc), _ptr(qc32), _ptr(kc32), _ptr(idx),
          _ptr(ws), _stream(stream))


def lsrm_nsa_cmp_attn(desc, off, q, kc, vc, o_cmp, lse=None, ws=None, stream=None):
    _check(off, torch.int32, "off"); _check(q, torch.bfloat16, "q"); _check(kc, torch.bfloat16, "kc")
    _check(vc, torch.bfloat16, "vc"); _check(o_cmp, torch.float32, "o_cmp"); _check(lse, torch.float32, "lse")
    _call("lsrm_nsa_cmp_attn", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(kc), _ptr(vc), _ptr(o_cmp), _ptr(lse),
          _ptr(ws), _stream(stream))


def lsrm_nsa_select_attn(desc, off, q, k, v, idx, idx_heads, o_slc, lse=None, ws=None, stream=None):
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (idx, "idx", torch.int32), (o_slc, "o_slc", torch.float32),
                     (lse, "lse", torch.float32)):
        _check(t, dt, n)
    _call("lsrm_nsa_select_attn", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(k), _ptr(v), _ptr(idx),
          int(idx_heads), _ptr(o_slc), _ptr(lse), _ptr(ws), _stream(stream))


def lsrm_nsa_window_attn(desc, off, q, k, v, o_win, lse=None, ws=None, stream=None):
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (o_win, "o_win", torch.float32), (lse, "lse", torch.float32)):
        _check(t, dt, n)
    _call("lsrm_nsa_window_attn", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(k), _ptr(v), _ptr(o_win),
          _ptr(lse), _ptr(ws), _stream(stream))


def lsrm_nsa_gate_combine(desc, o_cmp, o_slc, o_win, gates, out, stream=None):
    for t, n, dt in ((o_cmp, "o_cmp", torch.float32), (o_slc, "o_slc", torch.float32),
                     (o_win, "o_win", torch.float32), (gates, "gates", torch.bfloat16), (out, "out", torch.bfloat16)):
        _check(t, dt, n)
    _call("lsrm_nsa_gate_combine", ctypes.byref(desc), _ptr(o_cmp), _ptr(o_slc), _ptr(o_win), _ptr(gates),
          _ptr(out), _stream(stream))


def lsrm_nsa_attend(desc, off, q, k, v, kc, vc, gates, idx, idx_heads, route_all, out, lse=None, ws=None,
                    stream=None):
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (kc, "kc", torch.bfloat16), (vc, "vc", torch.bfloat16),
                     (gates, "gates", torch.bfloat16), (idx, "idx", torch.int32), (out, "out", torch.bfloat16),
                     (lse, "lse", torch.float32)):
        _check(t, dt, n)
    _call("lsrm_nsa_attend", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(k), _ptr(v), _ptr(kc), _ptr(vc),
          _ptr(gates), _ptr(idx), int(idx_heads), int(route_all), _ptr(out), _ptr(lse), _ptr(ws), _stream(stream))


def lsrm_route_camera(desc, off, coords, n_vol_blocks, proj, tile_block, tile_px, radius, k_vol, idx, ws,
                      stream=None):
    """Camera-projection routing: proj int32 [V][3][4], tile_block int32 [V][tiles_y][tiles_x]
    (device); idx int32 [B][top_k] = k_vol volume blocks, then top_k - k_vol image blocks."""
    for t, n, dt in ((off, "off", torch.int32), (coords, "coords", torch.int32), (proj, "proj", torch.int32),
                     (tile_block, "tile_block", torch.int32), (idx, "idx", torch.int32)):
        _check(t, dt, n)
    V, ty, tx = tile_block.shape
    if tuple(proj.shape) != (V, 3, 4):
        raise ValueError("proj: expected [views][3][4]")
    _call("lsrm_route_camera", ctypes.byref(desc), _ptr(off), _ptr(coords), int(n_vol_blocks), int(V), _ptr(proj),
          int(tx), int(ty), int(tile_px), _ptr(tile_block), int(radius), int(k_vol), _ptr(idx), _ptr(ws),
          _stream(stream))


def lsrm_nsa_mixture(desc, off, n_blocks_x, q, k, v, gates, out, lse=None, ws=None, stream=None):
    """Self/cross gated mixture: blocks [0, n_blocks_x) are one stream, the rest the other;
    gates [N][Hq][2] = (self, cross); lse (optional) fp32 [N][Hq][2]."""
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (gates, "gates", torch.bfloat16), (out, "out", torch.bfloat16),
                     (lse, "lse", torch.float32)):
        _check(t, dt, n)
    _call("lsrm_nsa_mixture", ctypes.byref(desc), _ptr(off), int(n_blocks_x), _ptr(q), _ptr(k), _ptr(v),
          _ptr(gates), _ptr(out), _ptr(lse), _ptr(ws), _stream(stream))


def lsrm_nsa_forward(desc, off, q, k, v, gates, coords, route_mode, out, idx=None, lse=None, ws=None, stream=None,
                     obr=None):
    """obr: optional bf16 [N][Hq][n_gates][d] that receives the per-branch outputs for the backward."""
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (gates, "gates", torch.bfloat16), (coords, "coords", torch.int32),
                     (out, "out", torch.bfloat16), (idx, "idx", torch.int32), (lse, "lse", torch.float32),
                     (obr, "obr", torch.bfloat16)):
        _check(t, dt, n)
    _call("lsrm_nsa_forward", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(k), _ptr(v), _ptr(gates), _ptr(coords),
          int(route_mode), _ptr(out), _ptr(idx), _ptr(lse), _ptr(obr), _ptr(ws), _stream(stream))


def lsrm_nsa_backward(desc, off, q, k, v, gates, idx, idx_heads, lse, dout, dq, dk, dv, dgates, ws, stream=None,
                      obr=None):
    """obr: the forward's saved per-branch outputs (optional); with them each branch is streamed once."""
    for t, n, dt in ((off, "off", torch.int32), (q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (gates, "gates", torch.bfloat16), (idx, "idx", torch.int32),
                     (lse, "lse", torch.float32), (dout, "dout", torch.bfloat16), (dq, "dq", torch.bfloat16),
                     (dk, "dk", torch.bfloat16), (dv, "dv", torch.bfloat16), (dgates, "dgates", torch.bfloat16),
                     (obr, "obr", torch.bfloat16)):
        _check(t, dt, n)
    _call("lsrm_nsa_backward", ctypes.byref(desc), _ptr(off), _ptr(q), _ptr(k), _ptr(v), _ptr(gates), _ptr(idx),
          int(idx_heads), _ptr(lse), _ptr(obr), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dgates), _ptr(ws),
          _stream(stream))


def lsrm_nsa_last_device_status(ws: torch.Tensor, stream=None) -> int:
    return int(load_library().lsrm_nsa_last_device_status(ws.data_ptr(), _stream(stream)))


def lsrm_status_string(status: int) -> str:
    return load_library().lsrm_status_string(int(status)).decode()


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)


def lsrm_diag_exp2_poly(x, y, stream=None):
    """y = 2^x through the attention kernels' FMA-pipe polynomial (a diagnostic)."""
    _check(x, torch.float32, "x"); _check(y, torch.float32, "y")
    if x.numel() != y.numel():
        raise ValueError("x and y differ in size")
    _call("lsrm_diag_exp2_poly", _ptr(x), _ptr(y), ctypes.c_int64(x.numel()), _stream(stream))


# ---- relative position bias and layer norm ---------------------------------------------------------
# These calls check shapes as well, and run on the tensors' own device (its current stream unless
# one is given), whichever device is current.

def _check_all(items) -> int:
    """The type, shape, contiguity and device that the call needs of each (tensor, name, dtype, shape);
    returns the device index.  Kept lean: small calls are bound by the host."""
    index = items[0][0].get_device()
    for t, name, dtype, shape in items:
        if t.dtype is not dtype:
            raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: expected {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if t.get_device() != index:
            raise ValueError(f"{name}: on {t.device}, expected {items[0][0].device}")
    return index


# the raw handle of a device's current stream, without making a stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call_on(index: int, name: str, stream, *args):
    if index < 0:
        raise ValueError(f"{name}: needs CUDA tensors")
    if stream is not None:
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(index)
    else:
        handle = torch.cuda.current_stream(index).cuda_stream
    if index == torch.cuda.current_device():
        _call(name, *args, handle)
    else:
        with torch.cuda.device(index):
            _call(name, *args, handle)


def lsrm_relpos_workspace_size(desc: RelposDesc) -> int:
    return int(load_library().lsrm_relpos_workspace_size(ctypes.byref(desc)))


def lsrm_relpos_workspace_init(desc: RelposDesc, ws: torch.Tensor, stream=None):
    _check(ws, torch.uint8, "ws")
    _call_on(ws.get_device(), "lsrm_relpos_workspace_init", stream, ctypes.byref(desc), ws.data_ptr(), ws.numel())


def relpos_workspace(desc: RelposDesc, device=None, stream=None) -> torch.Tensor:
    """Allocate (through torch) and initialise the workspace the relpos calls of this descriptor need."""
    n = lsrm_relpos_workspace_size(desc)
    if n == 0:
        raise NsaError("lsrm_relpos_workspace_size", 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)
    lsrm_relpos_workspace_init(desc, ws, stream)
    return ws


def lsrm_relpos_log_buckets(n_buckets: int, max_distance: int) -> torch.Tensor:
    """Logarithmic buckets of the clamped distances -D..D: int32 [2 D + 1] on the host."""
    out = torch.empty(2 * max(int(max_distance), 0) + 1, dtype=torch.int32)
    _call("lsrm_relpos_log_buckets", int(n_buckets), int(max_distance), out.data_ptr())
    return out


def _relpos_checks(desc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v):
    bf, i32 = torch.bfloat16, torch.int32
    qs = (desc.n_q_tokens, desc.n_q_heads, desc.head_dim)
    ks = (desc.n_k_tokens, desc.n_kv_heads, desc.head_dim)
    segs = (desc.n_segs + 1,)
    return qs, ks, [(off_q, "off_q", i32, segs), (off_k, "off_k", i32, segs),
                    (pos_q, "pos_q", i32, (desc.n_q_tokens, desc.n_axes)),
                    (pos_k, "pos_k", i32, (desc.n_k_tokens, desc.n_axes)),
                    (bucket_of, "bucket_of", i32, (2 * desc.max_distance + 1,)),
                    (table, "table", bf, (desc.n_axes, desc.n_buckets, desc.n_q_heads)),
                    (q, "q", bf, qs), (k, "k", bf, ks), (v, "v", bf, ks)]


def lsrm_relpos_forward(desc: RelposDesc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, out, lse=None,
                        ws=None, stream=None):
    """Attention over ragged segments with a learned relative position bias by buckets; lse (optional)
    fp32 [Nq][Hq] is what the backward needs."""
    qs, ks, items = _relpos_checks(desc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v)
    items.append((out, "out", torch.bfloat16, qs))
    if lse is not None:
        items.append((lse, "lse", torch.float32, qs[:2]))
    if ws is not None:
        items.append((ws, "ws", torch.uint8, ws.shape))
    _call_on(_check_all(items), "lsrm_relpos_forward", stream, ctypes.byref(desc), *map(_ptr, (off_q, off_k, pos_q,
             pos_k, bucket_of, table, q, k, v, out, lse, ws)), 0 if ws is None else ws.numel())


def lsrm_relpos_backward(desc: RelposDesc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, out, lse, dout,
                         dq, dk, dv, dtable, ws, stream=None):
    """Gradients of lsrm_relpos_forward with respect to q, k, v and the bias table."""
    bf = torch.bfloat16
    qs, ks, items = _relpos_checks(desc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v)
    items += ((out, "out", bf, qs), (lse, "lse", torch.float32, qs[:2]), (dout, "dout", bf, qs), (dq, "dq", bf, qs),
              (dk, "dk", bf, ks), (dv, "dv", bf, ks), (dtable, "dtable", bf, table.shape),
              (ws, "ws", torch.uint8, ws.shape))
    _call_on(_check_all(items), "lsrm_relpos_backward", stream, ctypes.byref(desc), *map(_ptr, (off_q, off_k, pos_q,
             pos_k, bucket_of, table, q, k, v, out, lse, dout, dq, dk, dv, dtable, ws)), ws.numel())


_LN_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _ln_rows(x):
    if x.dtype not in _LN_DTYPES:
        raise TypeError(f"x: expected torch.bfloat16 or torch.float32, got {x.dtype}")
    shape = x.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("x: needs rows of at least one element")
    return x.numel() // shape[-1], shape[-1]


def lsrm_layer_norm_forward(x, gamma, beta, eps, y, mean=None, rstd=None, stream=None):
    """Layer norm over the last axis of x; gamma / beta (or None) of x's type; mean / rstd (optional)
    fp32, one per row, are what the backward needs.  y may be x."""
    rows, width = _ln_rows(x)
    dtype, per_row = x.dtype, (rows,)
    items = [(x, "x", dtype, x.shape), (y, "y", dtype, x.shape)]
    if gamma is not None:
        items.append((gamma, "gamma", dtype, (width,)))
    if beta is not None:
        items.append((beta, "beta", dtype, (width,)))
    if mean is not None:
        items.append((mean, "mean", torch.float32, per_row))
    if rstd is not None:
        items.append((rstd, "rstd", torch.float32, per_row))
    _call_on(_check_all(items), "lsrm_layer_norm_forward", stream, rows, width, _LN_DTYPES[dtype], _ptr(x),
             _ptr(gamma), _ptr(beta), eps, _ptr(y), _ptr(mean), _ptr(rstd))


def lsrm_layer_norm_workspace_size(rows: int, width: int) -> int:
    return int(load_library().lsrm_layer_norm_workspace_size(int(rows), int(width)))


def layer_norm_workspace(rows: int, width: int, device=None) -> torch.Tensor:
    """Allocate (through torch) the workspace lsrm_layer_norm_backward needs."""
    n = lsrm_layer_norm_workspace_size(rows, width)
    if n == 0:
        raise NsaError("lsrm_layer_norm_workspace_size", 1)
    return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)


def lsrm_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, stream=None):
    """Gradients of lsrm_layer_norm_forward; dgamma / dbeta may be None.  dx may be dy or x."""
    rows, width = _ln_rows(x)
    dtype, columns = x.dtype, (width,)
    items = [(x, "x", dtype, x.shape), (dy, "dy", dtype, x.shape), (dx, "dx", dtype, x.shape),
             (mean, "mean", torch.float32, (rows,)), (rstd, "rstd", torch.float32, (rows,)),
             (ws, "ws", torch.uint8, ws.shape)]
    if gamma is not None:
        items.append((gamma, "gamma", dtype, columns))
    if dgamma is not None:
        items.append((dgamma, "dgamma", dtype, columns))
    if dbeta is not None:
        items.append((dbeta, "dbeta", dtype, columns))
    _call_on(_check_all(items), "lsrm_layer_norm_backward", stream, rows, width, _LN_DTYPES[dtype], _ptr(dy), _ptr(x),
             _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(ws), ws.numel())
