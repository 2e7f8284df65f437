"""Thin Python binding of libfa3.so (the C ABI declared in include/fa3.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  If the
library has not been built, every call raises; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading
from collections import OrderedDict
from typing import Optional

import torch

from . import build as _build

_lib = None

FA3_DEVERR_POS = 1
FA3_DEVERR_LENS = 2
FA3_DEVERR_TIMEOUT = 4
FA3_DEVERR_PAGE = 8
FA3_DEVERR_CALIB = 16


class FA3Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {lib().fa3_status_string(status).decode()} (status {status})")
        self.status = status


_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_D = ctypes.c_double

_SIGS = {
    "fa3_status_string": (ctypes.c_char_p, [_I]),
    "fa3_version": (_I, []),
    "fa3_set_kernel_timing": (_I, [_P, _P]),
    "fa3_calibrate_workspace_size": (_SZ, [_I]),
    "fa3_calibrate_perhead": (_I, [_P, _I64, _I, _I64, _I64, _I64, _D, _P, _P, _P, _SZ, _P]),
    "fa3_qparams": (_I, [_P, _P, _P, _I, _P]),
    "fa3_range_merge": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "fa3_calibrate_f32_workspace_size": (_SZ, [_I]),
    "fa3_calibrate_perhead_f32": (_I, [_P, _I64, _I, _I64, _I64, _I64, _D, _P, _P, _P, _SZ, _P, _P]),
    "fa3_qparams_channel": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "fa3_calibrate_perchannel": (_I, [_P, _I64, _I, _I64, _I, _I64, _I64, _I64, _D, _P, _P, _P]),
    "fa3_quantize_append_channel": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "fa3_quantize_append": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P]),
    "fa3_mla_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "fa3_decode_attn_mla": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P]),
    "fa3_gqa_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "fa3_decode_attn_gqa": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P]),
    "fa3_decode_attn_gqa_channel": (_I, [_P] * 11 + [_I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P]),
    "fa3_prefill_attn_gqa": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P]),
    "fa3_quantize_append_paged": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P]),
    "fa3_decode_attn_mla_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _SZ,
                                       _P, _P]),
    "fa3_decode_attn_gqa_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                       _SZ, _P, _P]),
    "fa3_norm_rope": (_I, [_P] * 4 + [_F, _P, _I, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I] + [_I64] * 12
                      + [_P, _P]),
    "fa3_rope_append_gqa_paged": (_I, [_P] * 5 + [_F, _P, _I, _I, _I] + [_P] * 9 + [_I] * 5 + [_I64] * 3 + [_I] * 3
                                  + [_P, _P]),
    "fa3_chunk_workspace_size": (_SZ, [_I] * 5),
    "fa3_prefill_attn_gqa_paged": (_I, [_P] * 10 + [_I] * 8 + [_F, _P, _SZ, _P, _P]),
    "fa3_cross_attn_gqa": (_I, [_P] * 9 + [_I] * 6 + [_F, _P, _SZ, _P, _P]),
    "fa3_call": (_I, [_I, ctypes.c_char_p, _I]),
}

# fa3_call: number of the call, packer of its arguments, their number.  ctypes converts one by one what this
# packs at once.
_CALLS = {name: (i, struct.Struct("=" + "".join("d" if a is _F else "q" for a in _SIGS[name][1])).pack,
                 len(_SIGS[name][1]))
          for i, name in enumerate(("fa3_norm_rope", "fa3_rope_append_gqa_paged", "fa3_prefill_attn_gqa_paged",
                                    "fa3_cross_attn_gqa"))}


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded libfa3.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libfa3.so is not built ({path}); run __graft_entry__.build()")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise FA3Error(fn, status)


def _need(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of dtype {dtype}")


def _need_contig(t: torch.Tensor, dtype, name: str):
    _need(t, dtype, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# Cached scratch buffers, one per (call kind, device, stream), at most
# _WS_PER_KIND streams per (call kind, device): the least recently used entry is
# dropped when another stream needs one.  Callers that manage memory themselves
# pass workspace= explicitly and the cache is never touched.  Host threads may call
# at once, also on one stream (their calls then share a buffer, and the library
# enqueues the kernels of a call together): the cache is looked up under a lock.  A
# buffer dropped while another thread still enqueues work on it goes back to
# the stream it was allocated on, behind that work.
_ws_cache: "OrderedDict" = OrderedDict()
_ws_lock = threading.RLock()
_WS_PER_KIND = 4


def _ws_key(key, device, stream=None):
    dev = device.index if device.index is not None else torch.cuda.current_device()
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return (key, dev, s.cuda_stream), s


def _workspace(key, nbytes: int, device, zero: bool = False, stream=None) -> Optional[torch.Tensor]:
    """A cached scratch buffer per (call kind, device, stream): calls that share a
    workspace must not overlap, and calls on one stream never do.  It is allocated
    (and zeroed) on that stream, so its first use is ordered after the fill."""
    if nbytes == 0:
        return None
    k, s = _ws_key(key, device, stream)
    with _ws_lock:
        ws = _ws_cache.get(k)
        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(s):
                ws = (torch.zeros if zero else torch.empty)(nbytes, dtype=torch.uint8, device=device)
            _ws_cache[k] = ws
            same = [c for c in _ws_cache if c[:2] == k[:2]]
            for old in same[:-_WS_PER_KIND]:
                if old != k:
                    del _ws_cache[old]
        _ws_cache.move_to_end(k)
    return ws


def _forget_workspace(key, device, stream=None) -> None:
    with _ws_lock:
        _ws_cache.pop(_ws_key(key, device, stream)[0], None)


# --------------------------------------------------------------------- calls
def set_kernel_timing(start: Optional["torch.cuda.Event"], stop: Optional["torch.cuda.Event"]):
    """fa3_set_kernel_timing: later decode / calibration calls record these events
    around their main kernel (None, None turns it off).  The events must have been
    recorded once, so that their CUDA handles exist."""
    a = None if start is None else ctypes.c_void_p(start.cuda_event)
    b = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check("fa3_set_kernel_timing", lib().fa3_set_kernel_timing(a, b))


def calibrate_workspace_size(H: int) -> int:
    return int(lib().fa3_calibrate_workspace_size(H))


def calibrate_perhead(x: torch.Tensor, ratio: float, min_io: torch.Tensor, max_io: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Per-head Recall-Window calibration of one batch; updates min_io/max_io in place.

    x: bf16 (B, H, S, D) with (S, D) contiguous, or (H, N) with N contiguous.
    """
    _need(x, torch.bfloat16, "x")
    _need_contig(min_io, torch.float32, "min_io")
    _need_contig(max_io, torch.float32, "max_io")
    if x.dim() == 4:
        B, H, S, D = x.shape
        if x.stride(3) != 1 or x.stride(2) != D:
            raise ValueError("x must have contiguous (S, D) planes")
        L, sb, sh = S * D, x.stride(0), x.stride(1)
    elif x.dim() == 2:
        H, L = x.shape
        if x.stride(1) != 1:
            raise ValueError("x rows must be contiguous")
        B, sb, sh = 1, 0, x.stride(0)
    else:
        raise ValueError("x must be (B, H, S, D) or (H, N)")
    if min_io.numel() != H or max_io.numel() != H:
        raise ValueError("min_io/max_io must hold H values")
    nbytes = calibrate_workspace_size(H)
    cached = workspace is None
    if cached:
        workspace = _workspace("calib", nbytes, x.device, zero=True, stream=stream)
    st = lib().fa3_calibrate_perhead(_ptr(x), B, H, L, sb, sh, float(ratio), _ptr(min_io), _ptr(max_io),
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    if st != 0 and cached:
        # The key counts may not have been cleared: never hand this buffer out again.
        _forget_workspace("calib", x.device, stream)
    _check("fa3_calibrate_perhead", st)


def calibrate_perhead_f32(x: torch.Tensor, ratio: float, min_io: torch.Tensor, max_io: torch.Tensor,
                          workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """Per-head Recall-Window calibration of float32 activations, (B, H, S, D) with
    (S, D) contiguous or (H, N); updates min_io / max_io in place."""
    _need(x, torch.float32, "x")
    _need_contig(min_io, torch.float32, "min_io")
    _need_contig(max_io, torch.float32, "max_io")
    if x.dim() == 4:
        B, H, S, D = x.shape
        if x.stride(3) != 1 or x.stride(2) != D:
            raise ValueError("x must have contiguous (S, D) planes")
        L, sb, sh = S * D, x.stride(0), x.stride(1)
    elif x.dim() == 2:
        H, L = x.shape
        if x.stride(1) != 1:
            raise ValueError("x rows must be contiguous")
        B, sb, sh = 1, 0, x.stride(0)
    else:
        raise ValueError("x must be (B, H, S, D) or (H, N)")
    if min_io.numel() != H or max_io.numel() != H:
        raise ValueError("min_io/max_io must hold H values")
    nbytes = int(lib().fa3_calibrate_f32_workspace_size(H))
    cached = workspace is None
    if cached:
        workspace = _workspace("calib_f32", nbytes, x.device, zero=True, stream=stream)
    st = lib().fa3_calibrate_perhead_f32(_ptr(x), B, H, L, sb, sh, float(ratio), _ptr(min_io), _ptr(max_io),
                                         _ptr(workspace), workspace.numel(), _ptr(dev_err), _stream(stream))
    if st != 0 and cached:
        _forget_workspace("calib_f32", x.device, stream)
    _check("fa3_calibrate_perhead_f32", st)


def range_merge(mins: torch.Tensor, maxs: torch.Tensor, min_io: torch.Tensor, max_io: torch.Tensor,
                stream=None) -> None:
    """Folds R ranges mins/maxs [R][H] into the running range min_io/max_io [H] (in place)."""
    _need_contig(mins, torch.float32, "mins")
    _need_contig(maxs, torch.float32, "maxs")
    _need_contig(min_io, torch.float32, "min_io")
    _need_contig(max_io, torch.float32, "max_io")
    H = min_io.numel()
    if mins.dim() != 2 or mins.shape != maxs.shape or mins.shape[1] != H or max_io.numel() != H:
        raise ValueError("mins/maxs must be [R][H] with H = min_io.numel()")
    st = lib().fa3_range_merge(_ptr(mins), _ptr(maxs), mins.shape[0], H, _ptr(min_io), _ptr(max_io),
                               _stream(stream))
    _check("fa3_range_merge", st)


def calibrate_perhead_sharded(batches, ratio: float, min_io: torch.Tensor, max_io: torch.Tensor,
                              group=None, stream=None) -> None:
    """Recall-Window calibration with the batches sharded over the ranks of a
    torch.distributed group: each rank calibrates its own batches into a local
    range (fa3_calibrate_perhead), the ranks all-gather their [H] ranges (the one
    exchange step), and every rank folds them into min_io/max_io
    (fa3_range_merge).  Step 3 is associative, so the result is bit-identical to
    one process accumulating every batch in any order."""
    import torch.distributed as dist
    H = min_io.numel()
    dev = min_io.device
    loc_mn = torch.full((H,), float("inf"), dtype=torch.float32, device=dev)
    loc_mx = torch.full((H,), float("-inf"), dtype=torch.float32, device=dev)
    for x in batches:
        calibrate_perhead(x, ratio, loc_mn, loc_mx, stream=stream)
    world = dist.get_world_size(group)
    mins = torch.empty(world, H, dtype=torch.float32, device=dev)
    maxs = torch.empty(world, H, dtype=torch.float32, device=dev)
    ctx = torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()
    with ctx:                                   # the collective is ordered on the calls' stream
        dist.all_gather(list(mins.unbind(0)), loc_mn, group=group)    # rows of mins / maxs
        dist.all_gather(list(maxs.unbind(0)), loc_mx, group=group)
    range_merge(mins, maxs, min_io, max_io, stream=stream)


def qparams(min_v: torch.Tensor, max_v: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    _need_contig(min_v, torch.float32, "min")
    _need_contig(max_v, torch.float32, "max")
    H = min_v.numel()
    if out is None:
        out = torch.empty(H, dtype=torch.float32, device=min_v.device)
    st = lib().fa3_qparams(_ptr(min_v), _ptr(max_v), _ptr(out), H, _stream(stream))
    _check("fa3_qparams", st)
    return out


def calibrate_perchannel(x: torch.Tensor, ratio: float, min_io: torch.Tensor, max_io: torch.Tensor,
                         stream=None) -> None:
    """Recall-Window calibration per (head, channel) of one batch x bf16 (B, H, S, D)
    (D contiguous); updates min_io / max_io [H][D] in place."""
    _need(x, torch.bfloat16, "x")
    _need_contig(min_io, torch.float32, "min_io")
    _need_contig(max_io, torch.float32, "max_io")
    if x.dim() != 4 or x.stride(3) != 1:
        raise ValueError("x must be (B, H, S, D) with D contiguous")
    B, H, S, D = x.shape
    if min_io.numel() != H * D or max_io.numel() != H * D:
        raise ValueError("min_io / max_io must hold H * D values")
    st = lib().fa3_calibrate_perchannel(_ptr(x), B, H, S, D, x.stride(0), x.stride(1), x.stride(2), float(ratio),
                                        _ptr(min_io), _ptr(max_io), _stream(stream))
    _check("fa3_calibrate_perchannel", st)


def qparams_channel(min_v: torch.Tensor, max_v: torch.Tensor, asymmetric: bool, stream=None):
    """Per-(head, channel) scale and offset from per-channel ranges [H][D]; returns (scale, offset)."""
    _need_contig(min_v, torch.float32, "min")
    _need_contig(max_v, torch.float32, "max")
    if min_v.shape != max_v.shape:
        raise ValueError("min and max must have the same shape")
    scale = torch.empty_like(min_v)
    offset = torch.empty_like(min_v)
    st = lib().fa3_qparams_channel(_ptr(min_v), _ptr(max_v), min_v.numel(), int(bool(asymmetric)), _ptr(scale),
                                   _ptr(offset), _stream(stream))
    _check("fa3_qparams_channel", st)
    return scale, offset


def quantize_append_channel(kv: torch.Tensor, scale: torch.Tensor, offset: Optional[torch.Tensor], asymmetric: bool,
                            cache: torch.Tensor, pos: torch.Tensor, dev_err: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """kv bf16 [B][T_new][H][D] -> cache int8 [B][T_max][H][D] at pos[b], per-channel scale/offset [H][D]."""
    _need_contig(kv, torch.bfloat16, "kv")
    _need_contig(scale, torch.float32, "scale")
    if asymmetric:
        _need_contig(offset, torch.float32, "offset")
    _need_contig(cache, torch.int8, "cache")
    _need_contig(pos, torch.int32, "pos")
    B, T_new, H, D = kv.shape
    if cache.dim() != 4 or cache.shape[0] != B or cache.shape[2] != H or cache.shape[3] != D:
        raise ValueError("cache must be [B][T_max][H][D]")
    if scale.numel() != H * D or (asymmetric and offset.numel() != H * D):
        raise ValueError("scale / offset must hold H * D values")
    st = lib().fa3_quantize_append_channel(_ptr(kv), _ptr(scale), _ptr(offset) if asymmetric else None,
                                           int(bool(asymmetric)), _ptr(cache), _ptr(pos), B, T_new, H, D,
                                           cache.shape[1], _ptr(dev_err), _stream(stream))
    _check("fa3_quantize_append_channel", st)


def quantize_append(kv: torch.Tensor, scale: torch.Tensor, cache: torch.Tensor, pos: torch.Tensor,
                    rope_src: Optional[torch.Tensor] = None, rope_cache: Optional[torch.Tensor] = None,
                    dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """kv bf16 [B][T_new][H][D] -> cache int8 [B][T_max][H][D] at pos[b]."""
    _need_contig(kv, torch.bfloat16, "kv")
    _need_contig(scale, torch.float32, "scale")
    _need_contig(cache, torch.int8, "cache")
    _need_contig(pos, torch.int32, "pos")
    B, T_new, H, D = kv.shape
    if cache.dim() != 4 or cache.shape[0] != B or cache.shape[2] != H or cache.shape[3] != D:
        raise ValueError("cache must be [B][T_max][H][D]")
    Dr = 0
    if rope_src is not None:
        _need_contig(rope_src, torch.bfloat16, "rope_src")
        _need_contig(rope_cache, torch.bfloat16, "rope_cache")
        Dr = rope_src.shape[-1]
    st = lib().fa3_quantize_append(_ptr(kv), _ptr(scale), _ptr(cache), _ptr(pos), B, T_new, H, D, cache.shape[1],
                                   _ptr(rope_src), _ptr(rope_cache), Dr, _ptr(dev_err), _stream(stream))
    _check("fa3_quantize_append", st)


def mla_workspace_size(B: int, H: int, Dl: int, T_max: int) -> int:
    return int(lib().fa3_mla_workspace_size(B, H, Dl, T_max))


def decode_attn_mla(q: torch.Tensor, ckv: torch.Tensor, krope: torch.Tensor, q_scale: torch.Tensor,
                    kv_scale: torch.Tensor, lens: torch.Tensor, softmax_scale: float,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Absorbed-MLA decode: q bf16 [B][H][Dl+Dr], ckv int8 [B][T_max][Dl], krope bf16 [B][T_max][Dr]."""
    _need_contig(q, torch.bfloat16, "q")
    _need_contig(ckv, torch.int8, "ckv")
    _need_contig(krope, torch.bfloat16, "krope")
    _need_contig(q_scale, torch.float32, "q_scale")
    _need_contig(kv_scale, torch.float32, "kv_scale")
    _need_contig(lens, torch.int32, "lens")
    B, H, Dqk = q.shape
    T_max, Dl = ckv.shape[1], ckv.shape[2]
    Dr = krope.shape[2]
    if Dqk != Dl + Dr:
        raise ValueError("q last dim must be Dl + Dr")
    if out is None:
        out = torch.empty(B, H, Dl, dtype=torch.float32, device=q.device)
    nbytes = mla_workspace_size(B, H, Dl, T_max)
    if workspace is None:
        workspace = _workspace("mla", nbytes, q.device, stream=stream)
    st = lib().fa3_decode_attn_mla(_ptr(q), _ptr(ckv), _ptr(krope), _ptr(q_scale), _ptr(kv_scale), _ptr(lens),
                                   _ptr(out), B, H, Dl, Dr, T_max, float(softmax_scale), _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _ptr(dev_err), _stream(stream))
    _check("fa3_decode_attn_mla", st)
    return out


def gqa_workspace_size(B: int, Hq: int, Hkv: int, D: int, T_max: int) -> int:
    return int(lib().fa3_gqa_workspace_size(B, Hq, Hkv, D, T_max))


def decode_attn_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
                    k_scale: torch.Tensor, v_scale: torch.Tensor, lens: torch.Tensor, softmax_scale: float,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """GQA decode: q int8 [B][Hq][D], k/v int8 [B][T_max][Hkv][D] -> bf16 [B][Hq][D]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_contig(t, torch.int8, n)
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _need_contig(t, torch.float32, n)
    _need_contig(lens, torch.int32, "lens")
    B, Hq, D = q.shape
    T_max, Hkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=q.device)
    nbytes = gqa_workspace_size(B, Hq, Hkv, D, T_max)
    if workspace is None:
        workspace = _workspace("gqa", nbytes, q.device, stream=stream)
    st = lib().fa3_decode_attn_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale),
                                   _ptr(lens), _ptr(out), B, Hq, Hkv, D, T_max, float(softmax_scale),
                                   _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                   _ptr(dev_err), _stream(stream))
    _check("fa3_decode_attn_gqa", st)
    return out


def decode_attn_gqa_channel(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
                            q_offset: torch.Tensor, k_scale: torch.Tensor, k_offset: torch.Tensor,
                            v_scale: torch.Tensor, v_offset: torch.Tensor, lens: torch.Tensor, softmax_scale: float,
                            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """GQA decode with per-channel scales / offsets ([heads][D] each): q int8 [B][Hq][D],
    k/v int8 [B][T_max][Hkv][D] -> bf16 [B][Hq][D]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_contig(t, torch.int8, n)
    for t, n in ((q_scale, "q_scale"), (q_offset, "q_offset"), (k_scale, "k_scale"), (k_offset, "k_offset"),
                 (v_scale, "v_scale"), (v_offset, "v_offset")):
        _need_contig(t, torch.float32, n)
    _need_contig(lens, torch.int32, "lens")
    B, Hq, D = q.shape
    T_max, Hkv = k.shape[1], k.shape[2]
    if q_scale.numel() != Hq * D or k_scale.numel() != Hkv * D or v_scale.numel() != Hkv * D:
        raise ValueError("per-channel parameters must be [heads][D]")
    if out is None:
        out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=q.device)
    nbytes = gqa_workspace_size(B, Hq, Hkv, D, T_max)
    if workspace is None:
        workspace = _workspace("gqa", nbytes, q.device, stream=stream)
    st = lib().fa3_decode_attn_gqa_channel(_ptr(q), _ptr(k), _ptr(v), _ptr(q_scale), _ptr(q_offset), _ptr(k_scale),
                                           _ptr(k_offset), _ptr(v_scale), _ptr(v_offset), _ptr(lens), _ptr(out), B,
                                           Hq, Hkv, D, T_max, float(softmax_scale), _ptr(workspace),
                                           0 if workspace is None else workspace.numel(), _ptr(dev_err),
                                           _stream(stream))
    _check("fa3_decode_attn_gqa_channel", st)
    return out


def prefill_attn_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
                     k_scale: torch.Tensor, v_scale: torch.Tensor, q_lens: torch.Tensor, kv_lens: torch.Tensor,
                     softmax_scale: float, out: Optional[torch.Tensor] = None,
                     dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal prefill: q int8 [B][S][Hq][D], k/v int8 [B][T][Hkv][D] -> bf16 [B][S][Hq][D].

    Rows i >= q_lens[b] of ``out`` are left untouched (zero-filled when ``out`` is
    allocated here)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_contig(t, torch.int8, n)
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _need_contig(t, torch.float32, n)
    _need_contig(q_lens, torch.int32, "q_lens")
    _need_contig(kv_lens, torch.int32, "kv_lens")
    B, S, Hq, D = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.zeros(B, S, Hq, D, dtype=torch.bfloat16, device=q.device)
    _need_contig(out, torch.bfloat16, "out")
    st = lib().fa3_prefill_attn_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale),
                                    _ptr(q_lens), _ptr(kv_lens), _ptr(out), B, S, T, Hq, Hkv, D,
                                    float(softmax_scale), _ptr(dev_err), _stream(stream))
    _check("fa3_prefill_attn_gqa", st)
    return out


# ------------------------------------------------------------- paged cache
def _block_table(block_table: torch.Tensor, B: int) -> int:
    _need_contig(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B][max_pages]")
    return block_table.shape[1]


def quantize_append_paged(kv: torch.Tensor, scale: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                          pos: torch.Tensor, rope_src: Optional[torch.Tensor] = None,
                          rope_cache: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """kv bf16 [B][T_new][H][D] -> page pool int8 [num_pages][page_size][H][D] at pos[b]."""
    _need_contig(kv, torch.bfloat16, "kv")
    _need_contig(scale, torch.float32, "scale")
    _need_contig(cache, torch.int8, "cache")
    _need_contig(pos, torch.int32, "pos")
    B, T_new, H, D = kv.shape
    if cache.dim() != 4 or cache.shape[2] != H or cache.shape[3] != D:
        raise ValueError("cache must be [num_pages][page_size][H][D]")
    num_pages, page_size = cache.shape[0], cache.shape[1]
    max_pages = _block_table(block_table, B)
    Dr = 0
    if rope_src is not None:
        _need_contig(rope_src, torch.bfloat16, "rope_src")
        _need_contig(rope_cache, torch.bfloat16, "rope_cache")
        Dr = rope_src.shape[-1]
    st = lib().fa3_quantize_append_paged(_ptr(kv), _ptr(scale), _ptr(cache), _ptr(block_table), _ptr(pos), B, T_new,
                                         H, D, num_pages, page_size, max_pages, _ptr(rope_src), _ptr(rope_cache), Dr,
                                         _ptr(dev_err), _stream(stream))
    _check("fa3_quantize_append_paged", st)


def decode_attn_mla_paged(q: torch.Tensor, ckv: torch.Tensor, krope: torch.Tensor, q_scale: torch.Tensor,
                          kv_scale: torch.Tensor, lens: torch.Tensor, block_table: torch.Tensor, softmax_scale: float,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Absorbed-MLA decode over page pools: ckv int8 [num_pages][page_size][Dl], krope bf16 [...][Dr]."""
    _need_contig(q, torch.bfloat16, "q")
    _need_contig(ckv, torch.int8, "ckv")
    _need_contig(krope, torch.bfloat16, "krope")
    _need_contig(q_scale, torch.float32, "q_scale")
    _need_contig(kv_scale, torch.float32, "kv_scale")
    _need_contig(lens, torch.int32, "lens")
    B, H, Dqk = q.shape
    num_pages, page_size, Dl = ckv.shape
    Dr = krope.shape[2]
    if Dqk != Dl + Dr:
        raise ValueError("q last dim must be Dl + Dr")
    max_pages = _block_table(block_table, B)
    if out is None:
        out = torch.empty(B, H, Dl, dtype=torch.float32, device=q.device)
    nbytes = mla_workspace_size(B, H, Dl, max_pages * page_size)
    if workspace is None:
        workspace = _workspace("mla", nbytes, q.device, stream=stream)
    st = lib().fa3_decode_attn_mla_paged(_ptr(q), _ptr(ckv), _ptr(krope), _ptr(q_scale), _ptr(kv_scale), _ptr(lens),
                                         _ptr(block_table), _ptr(out), B, H, Dl, Dr, num_pages, page_size, max_pages,
                                         float(softmax_scale), _ptr(workspace),
                                         0 if workspace is None else workspace.numel(), _ptr(dev_err),
                                         _stream(stream))
    _check("fa3_decode_attn_mla_paged", st)
    return out


def decode_attn_gqa_paged(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
                          k_scale: torch.Tensor, v_scale: torch.Tensor, lens: torch.Tensor, block_table: torch.Tensor,
                          softmax_scale: float, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """GQA decode over page pools: k/v int8 [num_pages][page_size][Hkv][D] -> bf16 [B][Hq][D]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_contig(t, torch.int8, n)
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _need_contig(t, torch.float32, n)
    _need_contig(lens, torch.int32, "lens")
    B, Hq, D = q.shape
    num_pages, page_size, Hkv = k.shape[0], k.shape[1], k.shape[2]
    max_pages = _block_table(block_table, B)
    if out is None:
        out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=q.device)
    nbytes = gqa_workspace_size(B, Hq, Hkv, D, max_pages * page_size)
    if workspace is None:
        workspace = _workspace("gqa", nbytes, q.device, stream=stream)
    st = lib().fa3_decode_attn_gqa_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale),
                                         _ptr(lens), _ptr(block_table), _ptr(out), B, Hq, Hkv, D, num_pages,
                                         page_size, max_pages, float(softmax_scale), _ptr(workspace),
                                         0 if workspace is None else workspace.numel(), _ptr(dev_err),
                                         _stream(stream))
    _check("fa3_decode_attn_gqa_paged", st)
    return out


# ------------------------------------- attention input and packed new rows
_BF16, _F32, _I32, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, device="cuda",
               inv_freq: Optional[torch.Tensor] = None) -> torch.Tensor:
    """float32 [n_pos][rot_dim] of cos, then sin, of position * inv_freq, computed in
    float64 (angles of far positions lose their fraction in float32); inv_freq
    [rot_dim / 2] defaults to base^(-2i / rot_dim)."""
    if n_pos <= 0 or rot_dim <= 0 or rot_dim % 2:
        raise ValueError("n_pos must be positive and rot_dim positive and even")
    if inv_freq is None:
        inv_freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    elif inv_freq.numel() != rot_dim // 2:
        raise ValueError("inv_freq must hold rot_dim / 2 values")
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * inv_freq.to(device, torch.float64)[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


# The calls below are made once a layer and step with little work behind them, so their checks are one
# expression each; what is wrong is worked out only when something is.
def _wrong(t, dtype, name: str):
    _need_contig(t, dtype, name)
    raise ValueError("all tensors must be on one device")


def _here(dev: int, stream):
    """(raw stream of the call, context to enter for its launches and allocations or None)."""
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError("stream must be on the tensors' device")
        return stream.cuda_stream, torch.cuda.stream(stream)
    ctx = torch.cuda.device(dev) if torch._C._cuda_getDevice() != dev else None
    return torch._C._cuda_getCurrentRawStream(dev), ctx


def _rows4(t: torch.Tensor, name: str, out: bool = False):
    """Strides (b, s, h) of head rows [B][S][H][D] or [n][H][D]; 0 where there is one index."""
    st = t.stride()
    if len(st) == 4 and st[3] == 1 and st[0] and st[1] and st[2] and not (st[0] | st[1] | st[2]) & 3:
        return st[:3]                                        # nothing below would change or refuse it
    sh = t.shape
    if len(sh) == 3:
        st, sh = (0,) + st, (1,) + tuple(sh)
    if len(sh) != 4:
        raise ValueError(f"{name} must be [B][S][H][D] or [n][H][D]")
    if st[3] != 1 and sh[3] > 1:
        raise ValueError(f"{name} must have contiguous head rows")
    sb, ss, hs = st[0] if sh[0] > 1 else 0, st[1] if sh[1] > 1 else 0, st[2] if sh[2] > 1 else 0
    if out and ((sb == 0 and sh[0] > 1) or (ss == 0 and sh[1] > 1) or (hs == 0 and sh[2] > 1)):
        raise ValueError(f"{name} must not be an expanded tensor")
    return sb, ss, hs


def norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
              pos: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
              q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, dev_err: Optional[torch.Tensor] = None, stream=None):
    """Per-head RMS norm (with q_weight / k_weight bf16 [D]) and position rotation of q and k in one pass.

    q bf16 [B][S][Hq][D] or [n][Hq][D] and k likewise with Hkv heads (or None): any strides
    with contiguous head rows, so slices of one projection need no copy.  cos_sin float32
    [table_len][rot_dim] (rope_table; None: no rotation), pos int32 of one position a token.
    Results are bf16 or float32: contiguous, or in q_out / k_out of q's / k's shape and any
    such strides (a transposed view lays them out (B, H, S, D) for calibrate_perhead; q and
    k themselves are allowed).  Returns (q_out, k_out)."""
    _need(q, _BF16, "q")
    sh = q.shape
    qs = _rows4(q, "q")
    B, S, Hq, D = sh if len(sh) == 4 else (1,) + tuple(sh)
    dev = q.get_device()
    Hkv, ks, kos, kp, kop = 0, (0, 0, 0), (0, 0, 0), 0, 0
    if k is not None:
        if not (isinstance(k, torch.Tensor) and k.dtype is _BF16 and k.get_device() == dev):
            _need(k, _BF16, "k")
            raise ValueError("all tensors must be on one device")
        ks = _rows4(k, "k")
        ksh = k.shape
        Hkv = ksh[-2]
        if len(ksh) != len(sh) or ksh[0] != sh[0] or ksh[-1] != D or (len(sh) == 4 and ksh[1] != S):
            raise ValueError("k must have q's tokens and head size")
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight go together")
        kp = k.data_ptr()
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    table_len, rot, cp, pp = 0, 0, 0, 0
    if cos_sin is not None:
        table_len, rot, cp = _table(cos_sin, D, dev)
        if pos is None:
            raise ValueError("pos must be given with cos_sin")
        if not (pos.dtype is _I32 and pos.get_device() == dev and pos.is_contiguous()):
            _wrong(pos, _I32, "pos")
        if pos.numel() != B * S:
            raise ValueError("pos must hold one position for each token")
        pp = pos.data_ptr()
    qw = 0 if q_weight is None else _vector(q_weight, D, _BF16, "q_weight", dev)
    kw = 0 if k_weight is None else _vector(k_weight, D, _BF16, "k_weight", dev)
    ep = 0 if dev_err is None else _error_word(dev_err, dev)
    raw, ctx = _here(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        t = out_dtype if q_out is None else q_out.dtype
        if t is not _BF16 and t is not _F32:
            raise TypeError("results are bfloat16 or float32")
        if q_out is None:
            q_out = torch.empty(sh, dtype=t, device=q.device)
        elif q_out.shape != sh or q_out.get_device() != dev:
            raise ValueError("q_out must have the input's shape and device")
        qos = _rows4(q_out, "q_out", True)
        if k is not None:
            if k_out is None:
                k_out = torch.empty(ksh, dtype=t, device=q.device)
            elif k_out.dtype is not t or k_out.shape != ksh or k_out.get_device() != dev:
                raise ValueError("k_out must have the input's shape and device and q_out's type")
            kos, kop = _rows4(k_out, "k_out", True), k_out.data_ptr()
        if B * S and D:                                      # a q without heads is refused by the call
            i, pack, count = _CALLS["fa3_norm_rope"]
            st = lib().fa3_call(i, pack(q.data_ptr(), kp, qw, kw, eps, cp, table_len, rot, bool(interleaved), pp,
                                        q_out.data_ptr(), kop, t is _F32, B, S, Hq, Hkv, D, *qs, *ks, *qos, *kos, ep,
                                        raw), count)
            if st:
                raise FA3Error("fa3_norm_rope", st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    return q_out, k_out


def _table(cos_sin: torch.Tensor, D: int, dev: int):
    if not (cos_sin.dtype is _F32 and cos_sin.get_device() == dev and cos_sin.is_contiguous()):
        _wrong(cos_sin, _F32, "cos_sin")
    sh = cos_sin.shape
    if len(sh) != 2 or sh[1] > D:
        raise ValueError("cos_sin must be [table_len][rot_dim] with rot_dim <= D")
    return sh[0], sh[1], cos_sin.data_ptr()


def _vector(t: Optional[torch.Tensor], n: int, dtype, name: str, dev: int):
    """The address of n contiguous values, or 0."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
        _wrong(t, dtype, name)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values")
    return t.data_ptr()


def _error_word(t: Optional[torch.Tensor], dev: int):
    if t is None:
        return 0
    if not (t.dtype is _I32 and t.get_device() == dev and t.numel() >= 1):
        _need(t, _I32, "dev_err")
        raise ValueError("dev_err must hold one value on the tensors' device")
    return t.data_ptr()


def _lens(q_start: torch.Tensor, lens: torch.Tensor, lens_name: str, dev: int) -> int:
    if not (lens.dtype is _I32 and lens.get_device() == dev and lens.is_contiguous()):
        _wrong(lens, _I32, lens_name)
    B = lens.numel()
    if B == 0:
        raise ValueError(f"{lens_name} must not be empty")
    if not (q_start.dtype is _I32 and q_start.get_device() == dev and q_start.is_contiguous()):
        _wrong(q_start, _I32, "q_start")
    if q_start.numel() != B + 1:
        raise ValueError(f"q_start must hold one value more than {lens_name}")
    return B


def _packed_rows(t: torch.Tensor, H: int, D: int, n: int, name: str, dev: int) -> int:
    """Row stride of packed rows [n][H][D] with contiguous rows of heads."""
    if not (t.dtype is _BF16 and t.get_device() == dev):
        _need(t, _BF16, name)
        raise ValueError("all tensors must be on one device")
    if t.shape != (n, H, D):
        raise ValueError(f"{name} must be [n][H][D]")
    st = t.stride()
    if (D > 1 and st[2] != 1) or (H > 1 and st[1] != D):
        raise ValueError(f"{name} must have contiguous rows of heads")
    return 0 if n == 1 else st[0]


def _pool_shape(k: torch.Tensor, v: torch.Tensor, dev: int):
    for t, name in ((k, "the k pool"), (v, "the v pool")):
        if not (t.dtype is _I8 and t.get_device() == dev and t.is_contiguous()):
            _wrong(t, _I8, name)
    sh = k.shape
    if len(sh) != 4 or sh != v.shape:
        raise ValueError("the k and v pools must both be [num_pages][page_size][Hkv][D]")
    return sh


def _pages(block_table: torch.Tensor, B: int, dev: int) -> int:
    if not (block_table.dtype is _I32 and block_table.get_device() == dev and block_table.is_contiguous()):
        _wrong(block_table, _I32, "block_table")
    sh = block_table.shape
    if len(sh) != 2 or sh[0] != B:
        raise ValueError("block_table must be [B][max_pages]")
    return sh[1]


def rope_append_gqa_paged(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                          cos_sin: Optional[torch.Tensor], q_scale: Optional[torch.Tensor], k_scale: torch.Tensor,
                          v_scale: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_table: torch.Tensor, q_start: torch.Tensor, kv_lens: torch.Tensor,
                          q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                          dev_err: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """The input step of a GQA layer over the paged INT8 cache, in one launch: k (normed if k_weight is
    given, and rotated) and v are quantized into their pools; q (or None) likewise to INT8 codes.

    q bf16 [n][Hq][D], k, v bf16 [n][Hkv][D] with any row stride (slices of one projection): rows
    q_start[b] .. q_start[b+1] - 1 are the last tokens of sequence b's kv_lens[b]-token context.
    k_cache, v_cache int8 [num_pages][page_size][Hkv][D].  Returns the query's codes int8
    [n][Hq][D] (zero outside the sequences' rows when allocated here)."""
    _need(k, _BF16, "k")
    dev = k.get_device()
    num_pages, page_size, Hkv, D = _pool_shape(k_cache, v_cache, dev)
    B = _lens(q_start, kv_lens, "kv_lens", dev)
    n = k.shape[0]
    ks, vs = _packed_rows(k, Hkv, D, n, "k", dev), _packed_rows(v, Hkv, D, n, "v", dev)
    ksc, vsc = _vector(k_scale, Hkv, _F32, "k_scale", dev), _vector(v_scale, Hkv, _F32, "v_scale", dev)
    qw, kw = _vector(q_weight, D, _BF16, "q_weight", dev), _vector(k_weight, D, _BF16, "k_weight", dev)
    table_len, rot, cp = _table(cos_sin, D, dev) if cos_sin is not None else (0, 0, 0)
    max_pages = _pages(block_table, B, dev)
    ep = _error_word(dev_err, dev)
    Hq, qs, qsc, qp, qop = 0, 0, 0, 0, 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [n][H][D]")
        Hq = q.shape[1]
        qs, qsc, qp = _packed_rows(q, Hq, D, n, "q", dev), _vector(q_scale, Hq, _F32, "q_scale", dev), q.data_ptr()
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    raw, ctx = _here(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        if q is not None:
            if q_out is None:
                q_out = torch.zeros(n, Hq, D, dtype=_I8, device=q.device)
            elif not (q_out.dtype is _I8 and q_out.get_device() == dev and q_out.is_contiguous()):
                _wrong(q_out, _I8, "q_out")
            elif q_out.shape != (n, Hq, D):
                raise ValueError("q_out must be [n][Hq][D]")
            qop = q_out.data_ptr()
        if n:
            i, pack, count = _CALLS["fa3_rope_append_gqa_paged"]
            st = lib().fa3_call(i, pack(
                qp, k.data_ptr(), v.data_ptr(), qw, kw, eps, cp, table_len, rot, bool(interleaved), qsc, ksc, vsc, qop,
                k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), q_start.data_ptr(),
                kv_lens.data_ptr(), n, B, Hq, Hkv, D, qs, ks, vs, num_pages, page_size, max_pages, ep, raw), count)
            if st:
                raise FA3Error("fa3_rope_append_gqa_paged", st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    return q_out


def chunk_workspace_size(n: int, B: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().fa3_chunk_workspace_size(n, B, Hq, Hkv, D))


def _chunk_workspace(nbytes: int, device, stream, dev: int, raw: int):
    # A captured call takes its buffer from the graph's own pool: replays of two graphs
    # (or of a graph and eager calls) then never share one.
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = ("chunk", dev, raw)                                # _ws_key's, without asking for the stream again
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is not None and ws.numel() >= nbytes:
            _ws_cache.move_to_end(key)
            return ws
        return _workspace("chunk", nbytes, device, stream=stream)


def _packed_attn(name, q, k, v, q_scale, k_scale, v_scale, q_start, lens, B, Hkv, sizes, table, softmax_scale, out,
                 workspace, dev_err, stream, dev):
    if not (q.dtype is _I8 and q.get_device() == dev and q.is_contiguous()):
        _wrong(q, _I8, "q")
    sh = q.shape
    D = k.shape[3]
    if len(sh) != 3 or sh[2] != D:
        raise ValueError("q must be [n][Hq][D] with k's head size")
    n, Hq = sh[0], sh[1]
    qsc = _vector(q_scale, Hq, _F32, "q_scale", dev)
    ksc, vsc = _vector(k_scale, Hkv, _F32, "k_scale", dev), _vector(v_scale, Hkv, _F32, "v_scale", dev)
    ep = _error_word(dev_err, dev)
    raw, ctx = _here(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        if out is None:
            out = torch.zeros(sh, dtype=_BF16, device=q.device)
        elif not (out.dtype is _BF16 and out.get_device() == dev and out.is_contiguous()):
            _wrong(out, _BF16, "out")
        elif out.shape != sh:
            raise ValueError("out must have q's shape")
        if n:
            L = lib()
            if workspace is None:
                nbytes = L.fa3_chunk_workspace_size(n, B, Hq, Hkv, D)
                workspace = _chunk_workspace(nbytes, q.device, stream, dev, raw) if nbytes else None
            elif workspace.get_device() != dev or not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous and on the tensors' device")
            wp, wn = (0, 0) if workspace is None else (workspace.data_ptr(),
                                                       workspace.numel() * workspace.element_size())
            i, pack, count = _CALLS[name]
            st = L.fa3_call(i, pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), qsc, ksc, vsc, q_start.data_ptr(),
                                    lens.data_ptr(), *table, out.data_ptr(), n, B, *sizes(Hq), softmax_scale, wp, wn, ep,
                                    raw), count)
            if st:
                raise FA3Error(name, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    return out


def prefill_attn_gqa_paged(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
                           k_scale: torch.Tensor, v_scale: torch.Tensor, q_start: torch.Tensor, kv_lens: torch.Tensor,
                           block_table: torch.Tensor, softmax_scale: float, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Causal attention of a chunk of new tokens over page pools: q int8 [n][Hq][D] packed by q_start,
    k/v int8 [num_pages][page_size][Hkv][D] (holding the new tokens already) -> bf16 [n][Hq][D].

    Rows outside the sequences are left as they were (zero when ``out`` is allocated here)."""
    _need(k, _I8, "k")
    dev = k.get_device()
    num_pages, page_size, Hkv, D = _pool_shape(k, v, dev)
    B = _lens(q_start, kv_lens, "kv_lens", dev)
    max_pages = _pages(block_table, B, dev)
    return _packed_attn("fa3_prefill_attn_gqa_paged", q, k, v, q_scale, k_scale, v_scale, q_start, kv_lens, B, Hkv,
                        lambda Hq: (Hq, Hkv, D, num_pages, page_size, max_pages), (block_table.data_ptr(),),
                        softmax_scale, out, workspace, dev_err, stream, dev)


def cross_attn_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor, k_scale: torch.Tensor,
                   v_scale: torch.Tensor, q_start: torch.Tensor, enc_lens: torch.Tensor, softmax_scale: float,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of q int8 [n][Hq][D] (packed by q_start) to all enc_lens[b] encoder states k/v int8
    [B][T][Hkv][D] of its sequence -> bf16 [n][Hq][D]; zero rows where there is no state."""
    _need_contig(k, _I8, "k")
    dev = k.get_device()
    if not (v.dtype is _I8 and v.get_device() == dev and v.is_contiguous()):
        _wrong(v, _I8, "v")
    B = _lens(q_start, enc_lens, "enc_lens", dev)
    sh = k.shape
    if len(sh) != 4 or sh != v.shape or sh[0] != B:
        raise ValueError("k and v must both be [B][T][Hkv][D]")
    T, Hkv, D = sh[1], sh[2], sh[3]
    return _packed_attn("fa3_cross_attn_gqa", q, k, v, q_scale, k_scale, v_scale, q_start, enc_lens, B, Hkv,
                        lambda Hq: (T, Hq, Hkv, D), (), softmax_scale, out, workspace, dev_err, stream, dev)
