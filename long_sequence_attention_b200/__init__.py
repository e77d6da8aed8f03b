"""Python binding of the DiT joint-attention library for B200 (sm_100a).

Argument marshalling only: every computation runs in the CUDA kernels of
``libdit_attn.so`` (built in-tree by ``long_sequence_attention_b200/build.py``).  The C
functions keep their names here (``dit_attn_fwd``, ``dit_attn_fwd_chunk``,
``dit_attn_merge``, ``dit_quant_fp8`` ...); tensors may be passed as torch CUDA tensors or
as raw device addresses (ints).  A non-zero status raises ``DitError``.

Importing this package fails loudly (ImportError) when the library has not been built:
there is no fallback implementation.

The few ``attention`` / ``attention_chunk`` / ``merge`` / ``quantize_fp8`` helpers below
only allocate outputs with torch and call the C entry points.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdit_attn.so")

DIT_BF16, DIT_FP8_E4M3, DIT_FP32 = 0, 1, 2
DIT_OK, DIT_ERR_INVALID_ARG, DIT_ERR_UNSUPPORTED, DIT_ERR_MISALIGNED, DIT_ERR_CUDA, DIT_ERR_TIMEOUT = range(6)


class DitError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where} failed: {status_str(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python long_sequence_attention_b200/build.py` "
                          "(nvcc, sm_100a). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
    sz, ull = ctypes.c_size_t, ctypes.c_ulonglong
    lib.dit_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp]
    lib.dit_attn_fwd_chunk.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, vp, vp]
    lib.dit_attn_merge.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), i, vp, vp, i, i, i, i, i, i, vp]
    lib.dit_attn_fwd_chunk_acc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp, vp]
    lib.dit_attn_acc_init.argtypes = [vp, vp, i, i, i, i, vp]
    lib.dit_quant_fp8_workspace_bytes.argtypes = [ll]
    lib.dit_quant_fp8_workspace_bytes.restype = sz
    lib.dit_quant_fp8.argtypes = [vp, vp, vp, ll, vp, sz, vp]
    lib.dit_quant_fp8_noalloc.argtypes = [vp, vp, vp, ll, vp]
    lib.dit_quant_fp8_noalloc.restype = ctypes.c_int
    lib.dit_device_status.argtypes = [ctypes.POINTER(i), i]
    lib.dit_set_wait_timeout_us.argtypes = [ull]
    lib.dit_selftest_wait_timeout.argtypes = [ull, vp]
    lib.dit_set_sm_reserve.argtypes = [i]
    lib.dit_quant_fp8_blocks.argtypes = [vp, vp, vp, i, i, i, i, vp]
    lib.dit_attn_fwd_seg.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, vp]
    lib.dit_swap01_chunks.argtypes = [vp, vp, ll, ll, ll, vp]
    lib.dit_na3d_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp]
    lib.dit_na3d_plan.argtypes = [i, i, i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(ll), ctypes.POINTER(ll)]
    lib.dit_attn_fwd_parts.argtypes = [ctypes.POINTER(vp), i, ctypes.POINTER(vp), ctypes.POINTER(vp), i,
                                       ctypes.POINTER(vp), ctypes.POINTER(vp), i, i, i, i, i, i, f, vp]
    lib.dit_ipc_export.argtypes = [vp, vp, ctypes.POINTER(ll)]
    lib.dit_ipc_import.argtypes = [vp, ll, ctypes.POINTER(vp), ctypes.POINTER(vp)]
    lib.dit_ipc_close.argtypes = [vp]
    lib.dit_attn_fwd_fp8_blocks.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
    lib.dit_rms_norm.argtypes = [vp, ll, vp, vp, vp, vp, vp, ll, i, f, i, i, i, vp]
    lib.dit_rope_qk.argtypes = [vp, vp, ctypes.POINTER(ll), ctypes.POINTER(ll), vp, vp, f, vp, ll, vp, ctypes.POINTER(i),
                                i, i, i, f, vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.dit_attn_masked_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.dit_attn_masked_workspace_bytes.restype = sz
    lib.dit_attn_fwd_masked.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, f, vp, i, vp, vp, vp, vp, vp, sz, vp]
    lib.dit_status_str.argtypes = [i]
    lib.dit_status_str.restype = ctypes.c_char_p
    lib.dit_version.argtypes = []
    for name in ("dit_attn_fwd", "dit_attn_fwd_chunk", "dit_attn_fwd_chunk_acc", "dit_attn_acc_init",
                 "dit_attn_merge", "dit_quant_fp8", "dit_device_status",
                 "dit_set_wait_timeout_us", "dit_selftest_wait_timeout", "dit_version"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


def status_str(status: int) -> str:
    return lib.dit_status_str(int(status)).decode()


def _check(rc: int, where: str) -> None:
    if rc != DIT_OK:
        raise DitError(rc, where)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# --------------------------------------------------------------------------- C entry points

def dit_attn_fwd(q, k, v, out, lse, B: int, H: int, S: int, D: int, scale: float,
                 dtype: int = DIT_BF16, descale_qkv=None, stream=None) -> None:
    _check(lib.dit_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D, float(scale),
                            dtype, _ptr(descale_qkv), _stream(stream)), "dit_attn_fwd")


def dit_attn_fwd_chunk(q, k, v, out, lse, B: int, H: int, S_q: int, S_kv: int, D: int, k0: int, k1: int,
                       scale: float, dtype: int = DIT_BF16, out_dtype: int = DIT_FP32, descale_qkv=None,
                       stream=None) -> None:
    _check(lib.dit_attn_fwd_chunk(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S_q, S_kv, D, k0, k1,
                                  float(scale), dtype, out_dtype, _ptr(descale_qkv), _stream(stream)),
           "dit_attn_fwd_chunk")


def dit_attn_fwd_chunk_acc(q, k, v, acc_out, acc_lse, B: int, H: int, S_q: int, S_kv: int, D: int, k0: int,
                           k1: int, scale: float, dtype: int = DIT_BF16, descale_qkv=None, stream=None) -> None:
    _check(lib.dit_attn_fwd_chunk_acc(_ptr(q), _ptr(k), _ptr(v), _ptr(acc_out), _ptr(acc_lse), B, H, S_q, S_kv, D,
                                      k0, k1, float(scale), dtype, _ptr(descale_qkv), _stream(stream)),
           "dit_attn_fwd_chunk_acc")


def dit_attn_acc_init(acc_out, acc_lse, B: int, H: int, S: int, D: int, stream=None) -> None:
    _check(lib.dit_attn_acc_init(_ptr(acc_out), _ptr(acc_lse), B, H, S, D, _stream(stream)), "dit_attn_acc_init")


def dit_attn_merge(outs: Sequence, lses: Sequence, out, lse, B: int, H: int, S: int, D: int,
                   in_dtype: int = DIT_FP32, out_dtype: int = DIT_BF16, stream=None) -> None:
    n = len(outs)
    arr_o = (ctypes.c_void_p * n)(*[_ptr(o) for o in outs])
    arr_l = (ctypes.c_void_p * n)(*[_ptr(x) for x in lses])
    _check(lib.dit_attn_merge(arr_o, arr_l, n, _ptr(out), _ptr(lse), B, H, S, D, in_dtype, out_dtype,
                              _stream(stream)), "dit_attn_merge")


def dit_quant_fp8_workspace_bytes(n: int) -> int:
    return int(lib.dit_quant_fp8_workspace_bytes(int(n)))


def dit_quant_fp8(x_bf16, x_fp8, descale, n: int, workspace, workspace_bytes: int, stream=None) -> None:
    _check(lib.dit_quant_fp8(_ptr(x_bf16), _ptr(x_fp8), _ptr(descale), int(n), _ptr(workspace),
                             int(workspace_bytes), _stream(stream)), "dit_quant_fp8")


def dit_attn_fwd_seg(q, k, v, out, lse, B: int, H: int, S: int, D: int, seg: int, scale: float,
                     dtype: int = 0, out_dtype: int = 0, descale_qkv=None, stream=None) -> None:
    _check(lib.dit_attn_fwd_seg(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D, seg, float(scale),
                                dtype, out_dtype, _ptr(descale_qkv), _stream(stream)), "dit_attn_fwd_seg")


def dit_attn_fwd_parts(q_parts: Sequence, k_parts: Sequence, v_parts: Sequence, out_parts: Sequence,
                       lse_parts: Optional[Sequence], B: int, part_H: int, h0: int, H: int, part_rows: int, D: int,
                       scale: float, stream=None) -> None:
    """Query blocks q_parts (outputs out_parts, lse_parts) and key blocks k_parts / v_parts;
    the counts are the lengths of the lists."""
    def arr(xs):
        return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])
    lse_arr = None if lse_parts is None else ctypes.cast(arr(lse_parts), ctypes.POINTER(ctypes.c_void_p))
    _check(lib.dit_attn_fwd_parts(arr(q_parts), len(q_parts), arr(k_parts), arr(v_parts), len(k_parts),
                                  arr(out_parts), lse_arr, B, part_H, h0, H, part_rows, D, float(scale),
                                  _stream(stream)), "dit_attn_fwd_parts")


def dit_ipc_export(ptr) -> Tuple[bytes, int]:
    """(64-byte CUDA IPC handle of the allocation holding ptr, byte offset of ptr in it)."""
    h = ctypes.create_string_buffer(64)
    off = ctypes.c_longlong(0)
    _check(lib.dit_ipc_export(_ptr(ptr), h, ctypes.byref(off)), "dit_ipc_export")
    return h.raw, off.value


def dit_ipc_import(handle: bytes, offset: int) -> Tuple[int, int]:
    """(device address, mapped allocation base) of a buffer exported by another process."""
    p, b = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib.dit_ipc_import(ctypes.create_string_buffer(handle, 64), int(offset), ctypes.byref(p), ctypes.byref(b)),
           "dit_ipc_import")
    return p.value, b.value


def dit_ipc_close(base: int) -> None:
    _check(lib.dit_ipc_close(base), "dit_ipc_close")


def dit_na3d_fwd(q, k, v, out, lse, B: int, H: int, T: int, Y: int, X: int, D: int, Kt: int, Ky: int, Kx: int,
                 scale: float, stream=None) -> None:
    _check(lib.dit_na3d_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, T, Y, X, D, Kt, Ky, Kx,
                            float(scale), _stream(stream)), "dit_na3d_fwd")


def dit_na3d_plan(T: int, Y: int, X: int, Kt: int, Ky: int, Kx: int):
    """The neighborhood kernel's tiling for a grid and window (host only): dict with the Q
    brick (t, y, x), the pairing axis, units and KV steps per head."""
    qb = (ctypes.c_int * 4)()
    units, steps = ctypes.c_longlong(0), ctypes.c_longlong(0)
    _check(lib.dit_na3d_plan(T, Y, X, Kt, Ky, Kx, qb, ctypes.byref(units), ctypes.byref(steps)), "dit_na3d_plan")
    return {"q_brick": (qb[0], qb[1], qb[2]), "pair_axis": qb[3], "units_per_head": units.value,
            "steps_per_head": steps.value}


def neighborhood_attention(q, k, v, grid, kernel, scale: Optional[float] = None, with_lse: bool = True,
                           stream=None):
    """(out bf16, lse fp32 or None) of 3-D neighborhood attention; q, k, v [B,H,T*Y*X,D] bf16,
    grid = (T, Y, X), kernel = (Kt, Ky, Kx)."""
    import torch
    B, H, S, D = _dims(q)
    scale = (1.0 / D ** 0.5) if scale is None else scale
    out = torch.empty_like(q)
    lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device) if with_lse else None
    dit_na3d_fwd(q, k, v, out, lse, B, H, *grid, D, *kernel, scale, stream)
    return out, lse


def dit_swap01_chunks(src, dst, d0: int, d1: int, chunk_bytes: int, stream=None) -> None:
    _check(lib.dit_swap01_chunks(_ptr(src), _ptr(dst), int(d0), int(d1), int(chunk_bytes), _stream(stream)),
           "dit_swap01_chunks")


def dit_quant_fp8_blocks(x_bf16, x_fp8, descales, B: int, H: int, S: int, D: int, stream=None) -> None:
    _check(lib.dit_quant_fp8_blocks(_ptr(x_bf16), _ptr(x_fp8), _ptr(descales), B, H, S, D, _stream(stream)),
           "dit_quant_fp8_blocks")


def dit_attn_fwd_fp8_blocks(q8, k8, v8, dq_blk, dk_blk, dv_blk, out, lse, B: int, H: int, S_q: int, S_kv: int,
                            D: int, k0: int, k1: int, scale: float, out_dtype: int = 0, stream=None) -> None:
    _check(lib.dit_attn_fwd_fp8_blocks(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(dq_blk), _ptr(dk_blk), _ptr(dv_blk),
                                       _ptr(out), _ptr(lse), B, H, S_q, S_kv, D, k0, k1, float(scale), out_dtype,
                                       _stream(stream)), "dit_attn_fwd_fp8_blocks")


def dit_quant_fp8_noalloc(x_bf16, x_fp8, descale, n: int, stream=None) -> None:
    """dit_quant_fp8 without a workspace, for callers that cannot allocate device memory
    (the scratch is a small array inside the library's device data; see the header)."""
    _check(lib.dit_quant_fp8_noalloc(_ptr(x_bf16), _ptr(x_fp8), _ptr(descale), int(n), _stream(stream)),
           "dit_quant_fp8_noalloc")


def dit_rms_norm(x, x_stride: int, residual, weight, out, stream_out, descales, rows: int, C: int, eps: float,
                 dtype: int = DIT_BF16, out_dtype: int = DIT_BF16, group: int = 0, stream=None) -> None:
    _check(lib.dit_rms_norm(_ptr(x), x_stride, _ptr(residual), _ptr(weight), _ptr(out), _ptr(stream_out),
                            _ptr(descales), rows, C, eps, dtype, out_dtype, group, _stream(stream)), "dit_rms_norm")


def dit_rope_qk(q, k, q_strides: Sequence[int], k_strides: Optional[Sequence[int]], q_weight, k_weight, eps: float, pos,
                pos_batch_stride: int, freqs, axis_pairs: Sequence[int], rot: int, interleaved: bool, magnitude: float,
                q_out, k_out, dq_blk, dk_blk, B: int, S: int, H: int, H_kv: int, D: int, out_dtype: int = DIT_BF16,
                stream=None) -> None:
    qs = (ctypes.c_longlong * 3)(*q_strides)
    ks = None if k_strides is None else (ctypes.c_longlong * 3)(*k_strides)
    _check(lib.dit_rope_qk(_ptr(q), _ptr(k), qs, ks, _ptr(q_weight), _ptr(k_weight), eps, _ptr(pos), pos_batch_stride,
                           _ptr(freqs), (ctypes.c_int * len(axis_pairs))(*axis_pairs), len(axis_pairs), rot,
                           1 if interleaved else 0, magnitude, _ptr(q_out), _ptr(k_out), _ptr(dq_blk), _ptr(dk_blk),
                           B, S, H, H_kv, D, out_dtype, _stream(stream)), "dit_rope_qk")


def dit_attn_masked_workspace_bytes(B: int, H: int, H_kv: int, S_q: int, S_kv: int, D: int, documents: bool) -> int:
    return int(lib.dit_attn_masked_workspace_bytes(B, H, H_kv, S_q, S_kv, D, 1 if documents else 0))


def dit_attn_fwd_masked(q, k, v, out, lse, B: int, H: int, H_kv: int, S_q: int, S_kv: int, D: int, scale: float,
                        softcap: float = 0.0, slopes=None, causal: bool = False, q_start=None, prefix=None, q_doc=None,
                        kv_doc=None, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(lib.dit_attn_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, H_kv, S_q, S_kv, D, scale,
                                   softcap, _ptr(slopes), 1 if causal else 0, _ptr(q_start), _ptr(prefix), _ptr(q_doc),
                                   _ptr(kv_doc), _ptr(workspace), workspace_bytes, _stream(stream)),
           "dit_attn_fwd_masked")


def dit_device_status(clear: bool = True) -> int:
    st = ctypes.c_int(0)
    _check(lib.dit_device_status(ctypes.byref(st), 1 if clear else 0), "dit_device_status")
    return st.value


def dit_set_wait_timeout_us(us: int) -> None:
    _check(lib.dit_set_wait_timeout_us(int(us)), "dit_set_wait_timeout_us")


def dit_set_sm_reserve(n_sms: int) -> None:
    _check(lib.dit_set_sm_reserve(int(n_sms)), "dit_set_sm_reserve")


def dit_selftest_wait_timeout(timeout_us: int, stream=None) -> None:
    _check(lib.dit_selftest_wait_timeout(int(timeout_us), _stream(stream)), "dit_selftest_wait_timeout")


def dit_version() -> int:
    return int(lib.dit_version())


# --------------------------------------------------------------------------- torch helpers

def _dims(q):
    if q.dim() != 4:
        raise ValueError("expected a [B, H, S, D] tensor")
    return tuple(int(x) for x in q.shape)


def attention(q, k, v, scale: Optional[float] = None, with_lse: bool = True, descale_qkv=None,
              stream=None) -> Tuple[object, Optional[object]]:
    """out (bf16) and lse (fp32) of full attention; q/k/v bf16 or uint8 E4M3 codes."""
    import torch
    B, H, S, D = _dims(q)
    fp8 = q.dtype == torch.uint8
    scale = (1.0 / D ** 0.5) if scale is None else scale
    out = torch.empty((B, H, S, D), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device) if with_lse else None
    dit_attn_fwd(q, k, v, out, lse, B, H, S, D, scale, DIT_FP8_E4M3 if fp8 else DIT_BF16, descale_qkv, stream)
    return out, lse


def attention_chunk(q, k, v, k0: int, k1: int, scale: Optional[float] = None, out_dtype=None,
                    descale_qkv=None, stream=None):
    """Partial (out, lse) over keys [k0, k1); out fp32 unless out_dtype is torch.bfloat16."""
    import torch
    B, H, S_q, D = _dims(q)
    S_kv = int(k.shape[2])
    fp8 = q.dtype == torch.uint8
    scale = (1.0 / D ** 0.5) if scale is None else scale
    od = torch.float32 if out_dtype is None else out_dtype
    out = torch.empty((B, H, S_q, D), dtype=od, device=q.device)
    lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    dit_attn_fwd_chunk(q, k, v, out, lse, B, H, S_q, S_kv, D, k0, k1, scale,
                       DIT_FP8_E4M3 if fp8 else DIT_BF16, DIT_FP32 if od == torch.float32 else DIT_BF16,
                       descale_qkv, stream)
    return out, lse


def ring_attention(q, k, v, bounds: Sequence, scale: Optional[float] = None, descale_qkv=None, stream=None):
    """Attention accumulated over the KV ranges in `bounds` with fused ring steps:
    (out fp32, lse) = exact attention over the union of the ranges."""
    import torch
    B, H, S_q, D = _dims(q)
    S_kv = int(k.shape[2])
    fp8 = q.dtype == torch.uint8
    scale = (1.0 / D ** 0.5) if scale is None else scale
    out = torch.empty((B, H, S_q, D), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    dit_attn_acc_init(out, lse, B, H, S_q, D, stream)
    for k0, k1 in bounds:
        dit_attn_fwd_chunk_acc(q, k, v, out, lse, B, H, S_q, S_kv, D, k0, k1, scale,
                               DIT_FP8_E4M3 if fp8 else DIT_BF16, descale_qkv, stream)
    return out, lse


def merge(outs: Sequence, lses: Sequence, out_dtype=None, stream=None):
    """Merged (out, lse) of chunk partials; out bf16 unless out_dtype is torch.float32."""
    import torch
    B, H, S, D = _dims(outs[0])
    od = torch.bfloat16 if out_dtype is None else out_dtype
    out = torch.empty((B, H, S, D), dtype=od, device=outs[0].device)
    lse = torch.empty((B, H, S), dtype=torch.float32, device=outs[0].device)
    in_dt = DIT_FP32 if outs[0].dtype == torch.float32 else DIT_BF16
    dit_attn_merge(outs, lses, out, lse, B, H, S, D, in_dt, DIT_FP32 if od == torch.float32 else DIT_BF16, stream)
    return out, lse


def quantize_fp8_blocks(x, stream=None):
    """(codes uint8 [B,H,S,D], descales fp32 [B,H,ceil(S/128)]) of a bf16 [B,H,S,D] tensor."""
    import torch
    B, H, S, D = _dims(x)
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    ds = torch.empty((B, H, (S + 127) // 128), dtype=torch.float32, device=x.device)
    dit_quant_fp8_blocks(x, codes, ds, B, H, S, D, stream)
    return codes, ds


def attention_fp8_blocks(q8, k8, v8, dq, dk, dv, scale: Optional[float] = None, k0: int = 0, k1: Optional[int] = None,
                         out_dtype=None, stream=None):
    """(out, lse) of E4M3 inputs with per-block descales over keys [k0, k1)."""
    import torch
    B, H, S_q, D = _dims(q8)
    S_kv = int(k8.shape[2])
    k1 = S_kv if k1 is None else k1
    scale = (1.0 / D ** 0.5) if scale is None else scale
    odt = torch.bfloat16 if out_dtype is None else out_dtype
    out = torch.empty((B, H, S_q, D), dtype=odt, device=q8.device)
    lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q8.device)
    dit_attn_fwd_fp8_blocks(q8, k8, v8, dq, dk, dv, out, lse, B, H, S_q, S_kv, D, k0, k1, scale,
                            DIT_FP32 if odt == torch.float32 else DIT_BF16, stream)
    return out, lse


def quantize_fp8(x, stream=None):
    """(codes uint8 same shape, descale fp32 [1]) of a bf16 tensor; per-tensor absmax scale."""
    import torch
    n = x.numel()
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    descale = torch.empty((1,), dtype=torch.float32, device=x.device)
    ws_bytes = dit_quant_fp8_workspace_bytes(n)
    ws = torch.empty((ws_bytes // 4,), dtype=torch.float32, device=x.device)
    dit_quant_fp8(x, codes, descale, n, ws, ws_bytes, stream)
    return codes, descale


# ------------------------------------------------- a block's other operators: norm, rotary positions, masks

class _Place:
    """The device and stream of a call that are not the current ones: within it they are, so that
    outputs and scratch belong to the stream that uses them."""

    def __init__(self, device, stream):
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        self.inside = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for c in self.inside:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.inside):
            c.__exit__(*exc)


def _raw_stream(index: int) -> int:
    """Address of a device's current stream (what torch.cuda.current_stream holds, without the object)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


@functools.lru_cache(maxsize=1024)
def _host_array(kind, *values):
    """A small array of host numbers for a call to read (by value: the same numbers share one)."""
    return (kind * len(values))(*values)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _like(t, name: str, dtype, shape, device) -> None:
    """t is a dense tensor of this type, shape and device."""
    if not (t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {list(shape)} on {device}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")


def _out_code(out_dtype):
    import torch
    codes = {torch.bfloat16: DIT_BF16, torch.float32: DIT_FP32, torch.uint8: DIT_FP8_E4M3}
    _need(out_dtype in codes, "out_dtype: torch.bfloat16, torch.float32 or torch.uint8 (E4M3 codes)")
    return codes[out_dtype]


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, out_dtype=None, group: int = 0, inplace: bool = False,
             stream=None):
    """(y, stream, descales) of a row-wise root-mean-square norm of h = x + residual over x's last dimension.

    x, weight, residual: all bf16 or all fp32.  y: x's type unless out_dtype says otherwise; torch.uint8 gives
    E4M3 codes with fp32 descales [..., 1], or [..., ceil(C/128)] with group = 128 (else descales is None).
    stream: h in x's type, written over residual where inplace is true; None without a residual."""
    import torch
    dt, dev, shape = x.dtype, x.device, x.shape
    bf16 = dt is torch.bfloat16
    if not (dev.type == "cuda" and (bf16 or dt is torch.float32) and shape and shape[-1]):
        raise ValueError("x: a CUDA tensor of bf16 or fp32")
    if stream is not None or dev.index != torch.cuda.current_device():
        with _Place(dev, stream):
            return rms_norm(x, weight, residual, eps, out_dtype, group, inplace)
    C = ldx = shape[-1]
    dense = x.is_contiguous()
    if not dense:
        _need(len(shape) == 2 and x.stride(1) == 1 and x.stride(0) >= C,
              "x: a contiguous tensor, or a matrix whose rows are dense")
        ldx = x.stride(0)
    wp = rp = hp = dp = h = ds = None
    if weight is not None:
        if weight.dtype is not dt or weight.shape != (C,) or weight.device != dev or not weight.is_contiguous():
            _like(weight, "weight", dt, (C,), dev)
        wp = weight.data_ptr()
    if residual is not None:
        if residual.dtype is not dt or residual.shape != shape or residual.device != dev or not residual.is_contiguous():
            _like(residual, "residual", dt, shape, dev)
        rp = residual.data_ptr()
        h = residual if inplace else torch.empty_like(residual)
        hp = h.data_ptr()
    elif inplace:
        raise ValueError("inplace needs a residual")
    if out_dtype is None or out_dtype is dt:
        code = DIT_BF16 if bf16 else DIT_FP32
        out = torch.empty_like(x) if dense else x.new_empty(shape)
    else:
        code = _out_code(out_dtype)
        out = x.new_empty(shape, dtype=out_dtype)
        if code == DIT_FP8_E4M3:
            ds = x.new_empty((*shape[:-1], (C + 127) // 128 if group else 1), dtype=torch.float32)
            dp = ds.data_ptr()
    rc = lib.dit_rms_norm(x.data_ptr(), ldx, rp, wp, out.data_ptr(), hp, dp, x.numel() // C, C, eps,
                          DIT_BF16 if bf16 else DIT_FP32, code, group, _raw_stream(dev.index))
    if rc:
        raise DitError(rc, "dit_rms_norm")
    return out, h, ds


def rope_frequencies(rot: int, theta: float = 10000.0, axis_pairs: Optional[Sequence[int]] = None,
                     scaling: str = "none", factor: float = 1.0, original_length: int = 0, fast_turns: float = 32.0,
                     slow_turns: float = 1.0, device=None):
    """(freqs, magnitude) for rope_qk: fp64 radians per position of the rot / 2 pairs.

    Pair i of an axis of n pairs turns by theta^(-i / n) per position (axis_pairs: the pairs of each
    axis; one axis unless given).  scaling stretches them `factor`-fold for contexts longer than trained on:
    "linear" divides every frequency; "ntk" raises theta so that the slowest pair is divided and the fastest
    kept; "by_parts" keeps pairs that turn more than fast_turns times within original_length, divides those
    that turn less than slow_turns times, mixes in between, and gives the magnitude 0.1 ln(factor) + 1
    (1 otherwise)."""
    import math

    import torch
    _need(rot >= 2 and rot % 2 == 0, "rot: an even number of elements")
    per = [rot // 2] if axis_pairs is None else list(axis_pairs)
    _need(sum(per) == rot // 2 and all(n >= 0 for n in per), "axis_pairs: counts that sum to rot / 2")
    _need(scaling in ("none", "linear", "ntk", "by_parts"), "scaling: none, linear, ntk or by_parts")
    _need(theta > 0 and factor >= 1, "theta > 0 and factor >= 1")
    freqs, magnitude = [], 1.0
    for n in per:
        base = theta
        if scaling == "ntk" and n > 1:
            base = theta * factor ** (n / (n - 1))
        for i in range(n):
            f = base ** (-i / n)
            if scaling == "linear":
                f /= factor
            elif scaling == "by_parts":
                turns = original_length * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - slow_turns) / (fast_turns - slow_turns)))
                f = f * keep + f / factor * (1.0 - keep)
            freqs.append(f)
    if scaling == "by_parts":
        _need(original_length > 0 and fast_turns > slow_turns, "by_parts: original_length and fast_turns > slow_turns")
        magnitude = 0.1 * math.log(factor) + 1.0
    return torch.tensor(freqs, dtype=torch.float64, device=device), magnitude


def rope_qk(q, k, pos, freqs, q_weight=None, k_weight=None, eps: float = 1e-6, axis_pairs: Optional[Sequence[int]] = None,
            interleaved: bool = False, magnitude: float = 1.0, out_dtype=None, stream=None):
    """(q_out, k_out, dq, dk): rotary positions of q [B, S, H, D] and k [B, S, H_kv, D] (bf16, any strides that are
    multiples of 8 with a dense head; k may be None), normed per head first where weights [D] are given, in the
    [B, heads, S, D] layout of the attention calls.

    pos: int32 [B or 1, S, axes] (or [B or 1, S] for one axis); freqs: fp64 [rot / 2] on the device, see
    rope_frequencies; axis_pairs: the pairs of each axis.  out_dtype torch.uint8 gives E4M3 codes in 128-row blocks
    and their descales dq, dk, as attention_fp8_blocks takes them (otherwise dq and dk are None)."""
    import torch
    bf16 = torch.bfloat16
    dev, shape = q.device, q.shape
    if not (dev.type == "cuda" and len(shape) == 4 and q.dtype is bf16):
        raise ValueError("q: a CUDA bf16 tensor [B, S, H, D]")
    if stream is not None or dev.index != torch.cuda.current_device():
        with _Place(dev, stream):
            return rope_qk(q, k, pos, freqs, q_weight, k_weight, eps, axis_pairs, interleaved, magnitude, out_dtype)
    B, S, H, D = shape
    qs, ks, H_kv, kp = q.stride(), (0, 0, 0, 1), 0, None
    if k is not None:
        H_kv, ks, kp = k.shape[2] if k.dim() == 4 else 0, k.stride(), k.data_ptr()
        _need(k.dtype is bf16 and k.device == dev and k.shape == (B, S, H_kv, D),
              "k: a bf16 tensor [B, S, H_kv, D] on q's device")
    _need(qs[3] == 1 and ks[3] == 1, "q, k: dense heads (stride 1 along D)")
    qw = kw = None
    if q_weight is not None:
        _like(q_weight, "q_weight", bf16, (D,), dev)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _like(k_weight, "k_weight", bf16, (D,), dev)
        kw = k_weight.data_ptr()
    ps, fs = pos.shape, freqs.shape
    axes = ps[2] if len(ps) == 3 else 1
    if not (pos.dtype is torch.int32 and pos.device == dev and len(ps) in (2, 3) and (ps[0] == B or ps[0] == 1)
            and ps[1] == S and pos.is_contiguous()):
        raise ValueError("pos: contiguous int32 [B or 1, S, axes] on q's device")
    if not (freqs.dtype is torch.float64 and freqs.device == dev and len(fs) == 1 and freqs.is_contiguous()):
        raise ValueError("freqs: a contiguous fp64 vector on q's device")
    pairs = fs[0]
    per = (pairs,) if axis_pairs is None else axis_pairs
    _need(len(per) == axes and axes <= 3, "axis_pairs: one count for each axis of pos, at most three")
    if out_dtype is None:
        out_dtype = bf16
    code = _out_code(out_dtype)
    q_out = q.new_empty((B, H, S, D), dtype=out_dtype)
    k_out = dq = dk = kop = dqp = dkp = None
    if k is not None:
        k_out = q.new_empty((B, H_kv, S, D), dtype=out_dtype)
        kop = k_out.data_ptr()
    if code == DIT_FP8_E4M3:
        dq = q.new_empty((B, H, (S + 127) // 128), dtype=torch.float32)
        dqp = dq.data_ptr()
        if k is not None:
            dk = q.new_empty((B, H_kv, (S + 127) // 128), dtype=torch.float32)
            dkp = dk.data_ptr()
    ll = ctypes.c_longlong
    rc = lib.dit_rope_qk(q.data_ptr(), kp, _host_array(ll, *qs[:3]), None if k is None else _host_array(ll, *ks[:3]), qw, kw,
                         eps, pos.data_ptr(),
                         S * axes if B > 1 and ps[0] == B else 0, freqs.data_ptr(), _host_array(ctypes.c_int, *per), axes, 2 * pairs,
                         1 if interleaved else 0, magnitude, q_out.data_ptr(), kop, dqp, dkp, B, S, H, H_kv, D, code,
                         _raw_stream(dev.index))
    if rc:
        raise DitError(rc, "dit_rope_qk")
    return q_out, k_out, dq, dk


def masked_attention(q, k, v, scale: Optional[float] = None, softcap: float = 0.0, slopes=None, causal: bool = False,
                     q_start=None, prefix=None, q_doc=None, kv_doc=None, with_lse: bool = True, stream=None):
    """(out bf16, lse fp32 or None) of attention with capped scores (softcap > 0), a distance bias (slopes fp32 [H]),
    causal, prefix (int32 [B], with causal) and document masks (int32 [B, S_q] and [B, S_kv], negative: padding).

    q [B, H, S_q, D], k and v [B, H_kv, S_kv, D] bf16 with H a multiple of H_kv.  q_start int32 [B]: position of each
    sequence's first query among the keys (S_kv - S_q unless given)."""
    import torch
    bf16 = torch.bfloat16
    dev, shape, kshape = q.device, q.shape, k.shape
    if not (dev.type == "cuda" and len(shape) == 4 and len(kshape) == 4):
        raise ValueError("q, k: CUDA tensors [B, H, S_q, D] and [B, H_kv, S_kv, D]")
    if stream is not None or dev.index != torch.cuda.current_device():
        with _Place(dev, stream):
            return masked_attention(q, k, v, scale, softcap, slopes, causal, q_start, prefix, q_doc, kv_doc, with_lse)
    B, H, S_q, D = shape
    H_kv, S_kv = kshape[1], kshape[2]
    if not (q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16 and k.device == dev and v.device == dev
            and v.shape == kshape and kshape[0] == B and kshape[3] == D and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous()):
        raise ValueError("q, k, v: contiguous bf16 tensors [B, H, S_q, D], [B, H_kv, S_kv, D] twice, on one device")
    slp = stp = prp = qdp = kdp = lp = wp = None
    if slopes is not None:
        _like(slopes, "slopes", torch.float32, (H,), dev)
        slp = slopes.data_ptr()
    if q_start is not None:
        _like(q_start, "q_start", torch.int32, (B,), dev)
        stp = q_start.data_ptr()
    if prefix is not None:
        _like(prefix, "prefix", torch.int32, (B,), dev)
        prp = prefix.data_ptr()
    if q_doc is not None or kv_doc is not None:
        _need(q_doc is not None and kv_doc is not None, "q_doc, kv_doc: both or neither")
        _like(q_doc, "q_doc", torch.int32, (B, S_q), dev)
        _like(kv_doc, "kv_doc", torch.int32, (B, S_kv), dev)
        qdp, kdp = q_doc.data_ptr(), kv_doc.data_ptr()
    out, lse = torch.empty_like(q), None
    if with_lse:
        lse = q.new_empty((B, H, S_q), dtype=torch.float32)
        lp = lse.data_ptr()
    n = lib.dit_attn_masked_workspace_bytes(B, H, H_kv, S_q, S_kv, D, 0 if q_doc is None else 1)
    if n:
        ws = q.new_empty((n,), dtype=torch.uint8)
        wp = ws.data_ptr()
    rc = lib.dit_attn_fwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp, B, H, H_kv, S_q, S_kv, D,
                                 1.0 / D ** 0.5 if scale is None else scale, softcap, slp, 1 if causal else 0, stp, prp,
                                 qdp, kdp, wp, n, _raw_stream(dev.index))
    if rc:
        raise DitError(rc, "dit_attn_fwd_masked")
    return out, lse
