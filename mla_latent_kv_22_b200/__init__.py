"""Python binding of libmla.so: absorbed Multi-head Latent Attention decode on B200.

Argument marshalling only.  Every function takes torch tensors, checks dtype,
shape, device and contiguity, and passes raw pointers, sizes and the current CUDA
stream to the C ABI of the same name (include/mla.h); every step of the
computation runs in the library's CUDA kernels.  Importing fails loudly when the
library has not been built (``python mla_latent_kv_22_b200/build.py``); there is
no fallback.  The short calls go through a compiled extension first where one is built
for the running torch and Python; without it they make the same call through ctypes.
"""
from __future__ import annotations

import ctypes
import importlib.util
import operator
import os
import types
import warnings

import torch

from .build import binding_path

__all__ = [
    "MlaError", "mla_decode", "mla_decode_multi", "mla_decode_noalloc", "mla_absorb_q", "mla_absorb_o", "mla_append",
    "mla_decode_window", "mla_decode_window_workspace_size", "mla_decode_shared", "mla_decode_shared_workspace_size",
    "mla_workspace_size", "mla_set_workspace",
    "mla_get_device_error", "mla_status_string", "mla_set_knob", "mla_get_knob", "mla_selected_decode_kernel",
    "mla_timing_enable",
    "mla_timing_read", "lib", "LIB_PATH", "KNOB", "STATUS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla.so")

STATUS = {
    0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE", 4: "MLA_ERR_CUDA",
    5: "MLA_ERR_DEVICE_BAD_PAGE", 6: "MLA_ERR_DEVICE_TIMEOUT", 7: "MLA_ERR_DEVICE_BAD_POSITION",
}
KNOB = {"num_workers": 0, "min_pages": 1, "decode_kernel": 2, "wait_limit": 3, "withhold_arrive": 4, "split_policy": 5,
        "piece_cost": 6, "row_tile": 7}

D_LATENT, D_ROPE, D_QK, PAGE, D_NOPE, D_V, MAX_HEADS = 512, 64, 576, 64, 128, 128, 128


class MlaError(RuntimeError):
    def __init__(self, status: int, message: str = ""):
        self.status = status
        self.name = STATUS.get(status, f"status {status}")
        super().__init__(f"{self.name}: {message}" if message else self.name)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python mla_latent_kv_22_b200/build.py` "
                          "(nvcc, sm_100a); there is no fallback implementation")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    i64 = ctypes.c_int64
    sig = {
        "mla_decode": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp], i32),
        "mla_decode_multi": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp], i32),
        "mla_decode_noalloc": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp], i32),
        "mla_absorb_q": ([vp, vp, vp, vp, i32, i32, vp], i32),
        "mla_absorb_o": ([vp, vp, vp, i32, i32, vp], i32),
        "mla_absorb_o_bf16": ([vp, vp, vp, i32, i32, vp], i32),
        "mla_append": ([vp] * 10 + [i64] * 6 + [i32] * 7 + [vp], i32),
        "mla_decode_window": ([vp] * 6 + [i32] * 7 + [f32, vp, sz, vp], i32),
        "mla_decode_window_workspace_size": ([i32, i32, i32], sz),
        "mla_decode_shared": ([vp] * 8 + [i32] * 6 + [f32, vp, sz, vp], i32),
        "mla_decode_shared_workspace_size": ([i32, i32, i32], sz),
        "mla_workspace_size": ([i32, i32, i32], sz),
        "mla_set_workspace": ([vp, sz], i32),
        "mla_get_device_error": ([vp], i32),
        "mla_status_string": ([i32], ctypes.c_char_p),
        "mla_last_error_message": ([], ctypes.c_char_p),
        "mla_set_knob": ([i32, i32], i32),
        "mla_get_knob": ([i32], i32),
        "mla_selected_decode_kernel": ([i32], i32),
        "mla_timing_enable": ([i32], i32),
        "mla_timing_read": ([ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = _load()


def _load_binding():
    """The quick path of the short calls (csrc/binding.cpp), or, where it has not been built for
    this torch and Python, functions that hand every call back to the code below."""
    path, why = binding_path(), "is missing"
    if os.path.exists(path):
        try:
            spec = importlib.util.spec_from_file_location(__name__ + "._binding", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            return module
        except ImportError as e:
            why = f"does not load ({e})"
    warnings.warn(f"{path} {why}: the same kernels run, but short calls take longer on the host; build it with "
                  "`python mla_latent_kv_22_b200/build.py`", RuntimeWarning, stacklevel=3)
    decline = lambda *args: NotImplemented
    return types.SimpleNamespace(decode_window=decline, decode_shared=decline, append=decline, absorb_o=decline)


_binding = _load_binding()


def _check(status: int) -> None:
    if status != 0:
        raise MlaError(status, lib.mla_last_error_message().decode(errors="replace"))


# The current stream's handle without a Stream object (0.1 against 3 us, of the 5 us that a
# small call's launch takes on the host); torch's own generated code takes it the same way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev: int | None = None) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if dev is None else dev)
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple | None = None) -> None:
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and (shape is None or t.shape == shape) and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cache_args(kv_cache, block_table, B):
    if block_table is None:
        _need(kv_cache, "kv_cache", torch.bfloat16)
        if kv_cache.dim() != 3 or kv_cache.shape[0] != B or kv_cache.shape[2] != D_QK or kv_cache.shape[1] % PAGE:
            raise ValueError("contiguous kv_cache must be [B, Tcap, 576] with Tcap % 64 == 0")
        return int(kv_cache.shape[1]) // PAGE, 0, None
    _need(block_table, "block_table", torch.int32)
    _need(kv_cache, "kv_cache", torch.bfloat16)
    if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (PAGE, D_QK):
        raise ValueError("paged kv_cache must be [num_pages, 64, 576]")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    return int(block_table.shape[1]), int(kv_cache.shape[0]), block_table.data_ptr()


def mla_decode(q, kv_cache, block_table, cache_seqlens, out, lse, softmax_scale: float, stream=None) -> None:
    """Absorbed decode (see include/mla.h).  q [B,H,576] bf16; kv_cache paged
    [num_pages,64,576] with block_table [B,max_blocks] int32, or contiguous
    [B,Tcap,576] with block_table None; cache_seqlens [B] int32; out [B,H,512] fp32;
    lse [B,H] fp32."""
    if q.dim() == 4 and q.shape[1] == 1:  # [B, 1, H, 576] (s_q = 1)
        q = q.view(q.shape[0], q.shape[2], q.shape[3])
    B, H = int(q.shape[0]), int(q.shape[1])
    _need(q, "q", torch.bfloat16, (B, H, D_QK))
    _need(cache_seqlens, "cache_seqlens", torch.int32, (B,))
    _need(out, "out", torch.float32, (B, H, D_LATENT))
    _need(lse, "lse", torch.float32, (B, H))
    max_blocks, num_pages, bt = _cache_args(kv_cache, block_table, B)
    _check(lib.mla_decode(q.data_ptr(), kv_cache.data_ptr(), bt, cache_seqlens.data_ptr(), out.data_ptr(),
                          lse.data_ptr(), B, H, num_pages, max_blocks, float(softmax_scale), _stream(stream)))


def mla_decode_multi(q, kv_cache, block_table, cache_seqlens, out, lse, softmax_scale: float, stream=None) -> None:
    """Decode of s_q causal query tokens per sequence (see include/mla.h).
    q [B,s_q,H,576] bf16; out [B,s_q,H,512] fp32; lse [B,s_q,H] fp32; the cache
    arguments are those of mla_decode."""
    if q.dim() != 4:
        raise ValueError("q must be [B, s_q, H, 576]")
    B, SQ, H = int(q.shape[0]), int(q.shape[1]), int(q.shape[2])
    _need(q, "q", torch.bfloat16, (B, SQ, H, D_QK))
    _need(cache_seqlens, "cache_seqlens", torch.int32, (B,))
    _need(out, "out", torch.float32, (B, SQ, H, D_LATENT))
    _need(lse, "lse", torch.float32, (B, SQ, H))
    max_blocks, num_pages, bt = _cache_args(kv_cache, block_table, B)
    _check(lib.mla_decode_multi(q.data_ptr(), kv_cache.data_ptr(), bt, cache_seqlens.data_ptr(), out.data_ptr(),
                                lse.data_ptr(), B, SQ, H, num_pages, max_blocks, float(softmax_scale),
                                _stream(stream)))


def _noalloc_args(q, kv_cache, block_table, cache_seqlens, out, lse):
    if q.dim() == 4 and q.shape[1] == 1:  # [B, 1, H, 576] (s_q = 1)
        q = q.view(q.shape[0], q.shape[2], q.shape[3])
    B, H = int(q.shape[0]), int(q.shape[1])
    _need(q, "q", torch.bfloat16, (B, H, D_QK))
    _need(cache_seqlens, "cache_seqlens", torch.int32, (B,))
    _need(out, "out", torch.float32, (B, H, D_LATENT))
    _need(lse, "lse", torch.float32, (B, H))
    if block_table is None:
        _need(kv_cache, "kv_cache", torch.bfloat16)
        if kv_cache.dim() != 3 or kv_cache.shape[0] != B or kv_cache.shape[2] != D_QK or kv_cache.shape[1] % PAGE:
            raise ValueError("contiguous kv_cache must be [B, Tcap, 576] with Tcap % 64 == 0")
        max_blocks, num_pages, bt = int(kv_cache.shape[1]) // PAGE, 0, None
    else:
        _need(block_table, "block_table", torch.int32)
        _need(kv_cache, "kv_cache", torch.bfloat16)
        if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (PAGE, D_QK):
            raise ValueError("paged kv_cache must be [num_pages, 64, 576]")
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_blocks]")
        max_blocks, num_pages, bt = int(block_table.shape[1]), int(kv_cache.shape[0]), block_table.data_ptr()
    return (q.data_ptr(), kv_cache.data_ptr(), bt, cache_seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H,
            num_pages, max_blocks)


def mla_decode_noalloc(q, kv_cache, block_table, cache_seqlens, out, lse, softmax_scale: float,
                       stream=None) -> None:
    """mla_decode for callers that cannot allocate device memory: same arguments and
    results, scratch from the library's static 32 MiB device array (see include/mla.h)."""
    args = _noalloc_args(q, kv_cache, block_table, cache_seqlens, out, lse)
    _check(lib.mla_decode_noalloc(*args, float(softmax_scale), _stream(stream)))


def mla_absorb_q(q_nope, q_rope, w_uk, q_out, stream=None) -> None:
    """q_out[b,h] = [q_nope[b,h] W_UK[h] | q_rope[b,h]] (bf16, fp32 accumulate)."""
    B, H = int(q_nope.shape[0]), int(q_nope.shape[1])
    _need(q_nope, "q_nope", torch.bfloat16, (B, H, D_NOPE))
    _need(q_rope, "q_rope", torch.bfloat16, (B, H, D_ROPE))
    _need(w_uk, "w_uk", torch.bfloat16, (H, D_NOPE, D_LATENT))
    _need(q_out, "q_out", torch.bfloat16, (B, H, D_QK))
    _check(lib.mla_absorb_q(q_nope.data_ptr(), q_rope.data_ptr(), w_uk.data_ptr(), q_out.data_ptr(), B, H,
                            _stream(stream)))


def mla_absorb_o(out_latent, w_uv, out, stream=None) -> None:
    """out[b,h] = bf16(out_latent[b,h]) W_UV[h] (fp32 accumulate, fp32 out).  out_latent is
    mla_decode's fp32, or the bf16 of mla_decode_window and mla_decode_shared (then
    mla_absorb_o_bf16 of the C ABI runs)."""
    if stream is None and _quick(_binding.absorb_o(out_latent, w_uv, out)):
        return
    B, H = int(out_latent.shape[0]), int(out_latent.shape[1])
    if out_latent.dtype == torch.bfloat16:
        dev = torch.cuda.current_device()
        _check(lib.mla_absorb_o_bf16(_here(out_latent, "out_latent", torch.bfloat16, (B, H, D_LATENT), dev),
                                     _here(w_uv, "w_uv", torch.bfloat16, (H, D_LATENT, D_V), dev),
                                     _here(out, "out", torch.float32, (B, H, D_V), dev), B, H, _stream(stream, dev)))
        return
    _need(out_latent, "out_latent", torch.float32, (B, H, D_LATENT))
    _need(w_uv, "w_uv", torch.bfloat16, (H, D_LATENT, D_V))
    _need(out, "out", torch.float32, (B, H, D_V))
    _check(lib.mla_absorb_o(out_latent.data_ptr(), w_uv.data_ptr(), out.data_ptr(), B, H, _stream(stream)))


def _quick(status) -> bool:
    """Whether the compiled binding made the call (raising what the library reported); if it
    did not, the arguments are for the code that follows to accept or to refuse."""
    if status is None:
        return True
    if status is NotImplemented:
        return False
    _check(status)
    return True


def _here(t, name, dtype, shape, dev: int) -> int:
    """_need for a tensor that must also live on the current device ``dev``, where the
    library launches; returns its address.  One pass of cheap tests, messages on failure."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")


def _rows_view(t, name, shape, dev: int):
    """Address and strides of a bf16 tensor of ``shape`` on device ``dev`` whose last
    dimension is dense; other strides are free."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    st = t.stride()
    if st[-1] != 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be dense")
    return t.data_ptr(), st


def _cache_here(kv_cache, block_table, B: int, dev: int):
    """_cache_args on the current device: (cache address, max_blocks, num_pages, table address)."""
    kv = _here(kv_cache, "kv_cache", torch.bfloat16, None, dev)
    if block_table is None:
        return (kv, *_cache_args(kv_cache, None, B))
    bt = _here(block_table, "block_table", torch.int32, None, dev)
    if kv_cache.dim() != 3 or kv_cache.shape[1] != PAGE or kv_cache.shape[2] != D_QK:
        raise ValueError("paged kv_cache must be [num_pages, 64, 576]")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    return kv, block_table.shape[1], kv_cache.shape[0], bt


def mla_append(c_kv, k_rope, kv_cache, block_table, cache_seqlens, cos_sin, cu_tokens=None, q_rope=None, q_out=None,
               pos_offset=None, interleaved: bool = True, stream=None) -> None:
    """Write new tokens' rows [c_kv | rotated k_rope] into the cache and rotate q_rope into
    q_out (see include/mla.h).  c_kv [N,512], k_rope [N,64], q_rope and q_out [N,H,64] bf16
    (views with other strides are taken, the last dimension dense); kv_cache and
    block_table as in mla_decode; cache_seqlens [B] int32, lengths with the new tokens;
    cos_sin [max_pos,64] fp32; cu_tokens [B+1] int32, or None for N / B tokens per
    sequence; pos_offset [B] int32 or None."""
    if stream is None and _quick(_binding.append(c_kv, k_rope, kv_cache, block_table, cache_seqlens, cos_sin, cu_tokens, q_rope,
                                                 q_out, pos_offset, interleaved)):
        return
    if c_kv.dim() != 2:
        raise ValueError("c_kv must be [N, 512]")
    dev = torch.cuda.current_device()
    N, B = c_kv.shape[0], cache_seqlens.shape[0]
    p_c, s_c = _rows_view(c_kv, "c_kv", (N, D_LATENT), dev)
    p_k, s_k = _rows_view(k_rope, "k_rope", (N, D_ROPE), dev)
    lens = _here(cache_seqlens, "cache_seqlens", torch.int32, (B,), dev)
    table = _here(cos_sin, "cos_sin", torch.float32, None, dev)
    if cos_sin.dim() != 2 or cos_sin.shape[1] != D_ROPE:
        raise ValueError("cos_sin must be [max_pos, 64]")
    cu = None if cu_tokens is None else _here(cu_tokens, "cu_tokens", torch.int32, (B + 1,), dev)
    off = None if pos_offset is None else _here(pos_offset, "pos_offset", torch.int32, (B,), dev)
    if (q_rope is None) != (q_out is None):
        raise ValueError("q_rope and q_out go together")
    H, p_q, p_o, s_q, s_o = 0, None, None, (0, 0), (0, 0)
    if q_rope is not None:
        if q_rope.dim() != 3:
            raise ValueError("q_rope must be [N, H, 64]")
        H = q_rope.shape[1]
        p_q, s_q = _rows_view(q_rope, "q_rope", (N, H, D_ROPE), dev)
        p_o, s_o = _rows_view(q_out, "q_out", (N, H, D_ROPE), dev)
    kv, max_blocks, num_pages, bt = _cache_here(kv_cache, block_table, B, dev)
    _check(lib.mla_append(p_c, p_k, p_q, p_o, table, cu, lens, off, bt, kv, s_c[0], s_k[0], s_q[0], s_q[1], s_o[0], s_o[1], N,
                          B, H, num_pages, max_blocks, cos_sin.shape[0], 1 if interleaved else 0, _stream(stream, dev)))


def _query_shape(q):
    """(B, s_q, H) of q [B,H,576] or [B,s_q,H,576], and the shape of the rows it asks for."""
    if q.dim() == 3:
        return (q.shape[0], 1, q.shape[1]), (q.shape[0], q.shape[1])
    if q.dim() == 4:
        rows = tuple(q.shape[:3])
        return rows, rows
    raise ValueError("q must be [B, H, 576] or [B, s_q, H, 576]")


def _workspace(workspace, size, stream, device, dev):
    """A caller's workspace, or one from torch's allocator that the call alone uses: taken
    on the launching stream, so its reuse is ordered after this call."""
    if workspace is not None:
        _here(workspace, "workspace", torch.uint8, None, dev)
        return workspace
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    with torch.cuda.stream(s):
        return torch.empty(size, dtype=torch.uint8, device=device)


def mla_decode_window(q, kv_cache, block_table, cache_seqlens, out, lse, softmax_scale: float, window: int,
                      sinks: int = 0, workspace=None, stream=None) -> None:
    """Decode over the last ``window`` tokens and the first ``sinks`` (see include/mla.h).
    q [B,H,576] or [B,s_q,H,576] bf16; out like q with 512, bf16; lse fp32; the cache
    arguments are those of mla_decode.  ``workspace``: a CUDA uint8 tensor of at least
    mla_decode_window_workspace_size(B, s_q, H) bytes, or None to take one from torch's
    allocator for this call.  ``window`` and ``sinks`` may be larger than any sequence."""
    if workspace is None and stream is None and _quick(_binding.decode_window(
            q, kv_cache, block_table, cache_seqlens, out, lse, softmax_scale, window, sinks)):
        return
    (B, SQ, H), rows = _query_shape(q)
    dev = torch.cuda.current_device()
    p_q = _here(q, "q", torch.bfloat16, rows + (D_QK,), dev)
    lens = _here(cache_seqlens, "cache_seqlens", torch.int32, (B,), dev)
    p_o = _here(out, "out", torch.bfloat16, rows + (D_LATENT,), dev)
    p_l = _here(lse, "lse", torch.float32, rows, dev)
    kv, max_blocks, num_pages, bt = _cache_here(kv_cache, block_table, B, dev)
    window, sinks = (max(-1, min(operator.index(n), 2**31 - 1)) for n in (window, sinks))  # as 32-bit integers
    ws = _workspace(workspace, lib.mla_decode_window_workspace_size(B, SQ, H), stream, q.device, dev)
    _check(lib.mla_decode_window(p_q, kv, bt, lens, p_o, p_l, B, SQ, H, num_pages, max_blocks, window, sinks, softmax_scale,
                                 ws.data_ptr(), ws.numel(), _stream(stream, dev)))


def mla_decode_window_workspace_size(batch: int, s_q: int, heads: int) -> int:
    return int(lib.mla_decode_window_workspace_size(batch, s_q, heads))


def mla_decode_shared(q, kv_cache, prefix_table, prefix_len, block_table, cache_seqlens, out, lse, softmax_scale: float,
                      workspace=None, stream=None) -> None:
    """Decode of a batch that shares a cached prefix (see include/mla.h).  prefix_table
    [prefix_blocks] int32 and prefix_len [1] int32 describe it, block_table
    [B,max_blocks] and cache_seqlens [B] int32 each sequence's own tokens; q, out, lse,
    workspace as in mla_decode_window (mla_decode_shared_workspace_size)."""
    if workspace is None and stream is None and _quick(_binding.decode_shared(
            q, kv_cache, prefix_table, prefix_len, block_table, cache_seqlens, out, lse, softmax_scale)):
        return
    (B, SQ, H), rows = _query_shape(q)
    dev = torch.cuda.current_device()
    p_q = _here(q, "q", torch.bfloat16, rows + (D_QK,), dev)
    ptab = _here(prefix_table, "prefix_table", torch.int32, None, dev)
    if prefix_table.dim() != 1:
        raise ValueError("prefix_table must be [prefix_blocks]")
    plen = _here(prefix_len, "prefix_len", torch.int32, (1,), dev)
    lens = _here(cache_seqlens, "cache_seqlens", torch.int32, (B,), dev)
    p_o = _here(out, "out", torch.bfloat16, rows + (D_LATENT,), dev)
    p_l = _here(lse, "lse", torch.float32, rows, dev)
    if block_table is None:
        raise ValueError("block_table is needed: the shared prefix and the own tokens are pages of one cache")
    kv, max_blocks, num_pages, bt = _cache_here(kv_cache, block_table, B, dev)
    ws = _workspace(workspace, lib.mla_decode_shared_workspace_size(B, SQ, H), stream, q.device, dev)
    _check(lib.mla_decode_shared(p_q, kv, ptab, plen, bt, lens, p_o, p_l, B, SQ, H, num_pages, prefix_table.shape[0],
                                 max_blocks, softmax_scale, ws.data_ptr(), ws.numel(), _stream(stream, dev)))


def mla_decode_shared_workspace_size(batch: int, s_q: int, heads: int) -> int:
    return int(lib.mla_decode_shared_workspace_size(batch, s_q, heads))


def mla_workspace_size(batch: int, heads: int, max_blocks: int) -> int:
    return int(lib.mla_workspace_size(batch, heads, max_blocks))


def mla_set_workspace(buf: torch.Tensor | None) -> None:
    """Use ``buf`` (a CUDA uint8 tensor the caller keeps alive) as the workspace, or None."""
    if buf is None:
        _check(lib.mla_set_workspace(None, 0))
    else:
        _need(buf, "workspace", torch.uint8)
        _check(lib.mla_set_workspace(buf.data_ptr(), buf.numel()))


def mla_get_device_error(stream=None) -> int:
    """Synchronise and return (and clear) the device error status code (0 = none)."""
    return int(lib.mla_get_device_error(_stream(stream)))


def mla_status_string(status: int) -> str:
    return lib.mla_status_string(status).decode()


def mla_set_knob(name: str, value: int) -> None:
    _check(lib.mla_set_knob(KNOB[name], int(value)))


def mla_get_knob(name: str) -> int:
    return int(lib.mla_get_knob(KNOB[name]))


def mla_selected_decode_kernel(heads: int) -> int:
    """2 = dim-split pair kernel, 3 = head-split pair kernel (what mla_decode runs for ``heads`` now)."""
    return int(lib.mla_selected_decode_kernel(int(heads)))


def mla_timing_enable(enable: bool = True) -> None:
    _check(lib.mla_timing_enable(1 if enable else 0))


def mla_timing_read() -> tuple[list[float], int]:
    """Summed milliseconds of (schedule, decode, combine) since enabling, and the call count."""
    ms = (ctypes.c_float * 3)()
    calls = ctypes.c_int()
    _check(lib.mla_timing_read(ms, ctypes.byref(calls)))
    return [ms[0], ms[1], ms[2]], calls.value
