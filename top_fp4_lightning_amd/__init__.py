"""fp4idx: FP4 lightning-indexer hot path for MI355X (gfx950).

Thin ctypes binding over ``libfp4idx.so`` (C ABI in ``include/fp4idx.h``). Each function has
the name of the C entry point it calls and only marshals arguments: torch tensors supply device
memory and the current stream; every step of the indexer runs in the HIP kernels. There is no
CPU or eager fallback: importing fails if the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4idx.so")

IDX_OK, IDX_EINVAL, IDX_EALIGN, IDX_EUNSUPPORTED, IDX_EHIP, IDX_EWORKSPACE = 0, -1, -2, -3, -4, -5
IDX_OP_BUILD_POOL, IDX_OP_TOPK, IDX_OP_ATTEND, IDX_OP_DISTILL, IDX_OP_ATTEND_LOCAL = 1, 2, 3, 4, 5
HEADS, DIM, BLOCK = 32, 128, 8

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with top_fp4_lightning_amd.build.build_library() "
                      "(or __graft_entry__.build()); the indexer has no fallback path")

_P, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_f32, _f64 = ctypes.c_float, ctypes.c_double
lib = ctypes.CDLL(LIB_PATH)
lib.idx_abi_version.restype = _i32
lib.idx_last_error.restype = ctypes.c_char_p
lib.idx_workspace_size.argtypes = [_i32, _i32, _i64, _i32]
lib.idx_workspace_size.restype = _sz
lib.idx_quantize_q.argtypes = [_P, _i64, _P, _P, _P, _P]
lib.idx_score_full.argtypes = [_P, _P, _P, _P, _i32, _i32, _i64, _P, _P, _P, _P, _i64, _P, _i64, _P, _P]
lib.idx_build_pool.argtypes = [_P, _i64, _P, _i32, _i64, _i32, _i32, _P, _i64, _P, _P, _sz, _P]
lib.idx_build_pool_noalloc.argtypes = [_P, _i64, _P, _i32, _i64, _i32, _i32, _P, _i64, _P, _P]
lib.idx_top_blocks.argtypes = [_P, _i64, _P, _i32, _i64, _i32, _i32, _P, _i64, _P, _P, _sz, _P]
lib.idx_score_pool_gather.argtypes = [_P, _P, _P, _P, _i32, _P, _i64, _P, _i32, _i32, _P, _P, _P, _P, _i64, _P, _P]
lib.idx_topk.argtypes = [_P, _i64, _P, _i32, _i64, _i32, _P, _i64, _i32, _P, _i64, _P, _P, _sz, _P]
lib.idx_quantize_kv.argtypes = [_P, _i64, _P, _P, _P]
lib.idx_gather_kv.argtypes = [_P, _P, _P, _P, _i32, _P, _i64, _i32, _P, _P]
lib.idx_mask_pool.argtypes = [_P, _i64, _P, _i32, _i64, _P, _i64, _P, _i32, _i32, _P]
lib.idx_topk_pool.argtypes = [_P, _i64, _P, _i32, _i64, _P, _i64, _P, _i32, _i32, _i32, _i32, _P, _i64, _P, _P]
lib.idx_rope_freqs.argtypes = [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _P, _P]
lib.idx_rope.argtypes = [_P, _i32, _i64, _i32, _i32, _i64, _i64, _P, _P, _i32, _i32, _i32, _f32, _i32, _P, _i64, _i64, _P]
lib.idx_attend.argtypes = [_P, _i32, _i32, _P, _P, _i64, _P, _P, _i64, _i32, _i32, _P, _P, _i64, _i64, _P, _i64, _i32,
                           _f32, _P, _P, _P, _sz, _P]
lib.idx_attend_weights.argtypes = [_P, _i32, _i32, _P, _P, _i64, _P, _P, _i64, _i32, _i32, _P, _P, _i64, _P, _i64, _i32,
                                   _f32, _P, _P, _i64, _P]
lib.idx_distill.argtypes = [_P, _i64, _P, _i32, _i64, _P, _P, _i64, _i32, _f32, _P, _P, _P, _P, _sz, _P]
lib.idx_distill_bwd.argtypes = [_P, _i64, _P, _i32, _i64, _P, _P, _i64, _i32, _f32, _P, _P, _P, _P, _i64, _P]
lib.idx_write_rows.argtypes = [_i32, _P, _i32, _i64, _i64, _i32, _P, _f64, _P, _P, _i32, _i32, _i32, _f64, _P, _P, _P, _i64,
                               _P, _P, _i64, _i32, _i32, _P, _P, _i64, _i64, _P]
lib.idx_write_rows_kept.argtypes = [*lib.idx_write_rows.argtypes[:-1], _P, _P]
lib.idx_read_rows.argtypes = [_i32, _P, _P, _i64, _P, _P, _i64, _i32, _i32, _P, _P, _i64, _i64, _i64, _P, _P, _i32, _i32,
                              _i32, _f64, _i32, _P, _i32, _i64, _P]
lib.idx_attend_local.argtypes = [_P, _i32, _i32, _i32, _P, _P, _i64, _P, _P, _i64, _i32, _i32, _P, _P, _i64, _i64, _i64, _f32,
                                 _P, _P, _P, _P, _i32, _i32, _i32, _f64, _P, _P, _P, _sz, _P]
lib.idx_attend_local_strided.argtypes = [*lib.idx_attend_local.argtypes[:13], _i64, *lib.idx_attend_local.argtypes[13:]]
for _f in ("idx_quantize_q", "idx_score_full", "idx_build_pool", "idx_build_pool_noalloc", "idx_top_blocks",
           "idx_score_pool_gather", "idx_topk",
           "idx_quantize_kv", "idx_gather_kv", "idx_mask_pool", "idx_topk_pool", "idx_rope_freqs", "idx_rope",
           "idx_attend", "idx_attend_weights", "idx_distill", "idx_distill_bwd", "idx_write_rows", "idx_read_rows",
           "idx_attend_local", "idx_attend_local_strided", "idx_write_rows_kept"):
    getattr(lib, _f).restype = _i32

EXPORTS = ("idx_abi_version", "idx_last_error", "idx_workspace_size", "idx_quantize_q", "idx_score_full",
           "idx_build_pool", "idx_build_pool_noalloc", "idx_top_blocks", "idx_score_pool_gather", "idx_topk",
           "idx_quantize_kv",
           "idx_gather_kv", "idx_mask_pool", "idx_topk_pool", "idx_rope_freqs", "idx_rope", "idx_attend",
           "idx_attend_weights", "idx_distill", "idx_distill_bwd", "idx_write_rows", "idx_read_rows", "idx_attend_local",
           "idx_attend_local_strided", "idx_write_rows_kept")
MKV_DIM = 512


class IdxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"fp4idx status {status}: {msg}")
        self.status = status


def _check(status: int) -> None:
    if status != IDX_OK:
        raise IdxError(status, lib.idx_last_error().decode())


_recording: list | None = None


def _call(fn, *args) -> None:
    """Run one library call and raise on a failed status, or, inside record(), only keep it."""
    if _recording is not None:
        _recording.append((fn, args))
        return
    _check(fn(*args))


class Recorded:
    """A fixed sequence of library calls with their arguments marshalled once (tensor checks,
    pointers, strides and the stream resolved when recorded): replaying costs the host one foreign
    call per launch. The tensors the calls name must keep their storage while it is in use."""

    def __init__(self, calls: list):
        self.calls = list(calls)

    def __call__(self) -> None:
        for fn, args in self.calls:
            status = fn(*args)
            if status != IDX_OK:
                raise IdxError(status, lib.idx_last_error().decode())


@contextlib.contextmanager
def record():
    """Collect the library calls made inside the block, without running them: yields a list that
    holds them afterwards (wrap it in Recorded to replay)."""
    global _recording
    if _recording is not None:
        raise RuntimeError("record() does not nest")
    calls: list = []
    _recording = calls
    try:
        yield calls
    finally:
        _recording = None


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp4idx tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("fp4idx tensors must be contiguous")
    return t.data_ptr()


def _rows_ptr(t: torch.Tensor | None) -> int | None:
    """A 2-D argument the library reads through its own row stride: each row contiguous."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp4idx tensors must live on the GPU")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("fp4idx row arguments must be 2-D with contiguous rows")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without the Stream object in between (2.7 us of a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """An output that a call on `stream` writes. Memory that was free on the current stream may still be read there by
    work queued before it was freed, so the output comes from the stream that writes it; and it goes back only behind
    the work queued on the current stream by then, where the caller reads it after a wait."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = _stream(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    if stream != here:
        out.record_stream(here)
    return out


def _need(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def abi_version() -> int:
    return int(lib.idx_abi_version())


def workspace_size(op: int, nq: int, max_n: int, k: int) -> int:
    return int(lib.idx_workspace_size(op, nq, max_n, k))


def workspace(op: int, nq: int, max_n: int, k: int, device="cuda") -> torch.Tensor:
    """Zero-filled workspace; the library restores its counters after every call."""
    n = workspace_size(op, nq, max_n, k)
    if n == 0:
        raise ValueError("invalid workspace request")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def idx_quantize_q(x: torch.Tensor, signs: torch.Tensor, codes: torch.Tensor | None = None,
                   scales: torch.Tensor | None = None, stream=None):
    """Rotate + MXFP4-quantise bf16 rows [..., 128] -> (codes [..., 64] u8, scales [..., 4] u8)."""
    _need(x, torch.bfloat16, "x")
    _need(signs, torch.int8, "signs")
    lead = x.shape[:-1]
    rows = x.numel() // DIM
    if codes is None:
        codes = _empty((*lead, 64), torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty((*lead, 4), torch.uint8, x.device, stream)
    _call(lib.idx_quantize_q, _ptr(x), rows, _ptr(signs), _ptr(codes), _ptr(scales), _stream(stream))
    return codes, scales


def idx_score_full(k_codes, k_scales, k_base, n_vis, q_codes, q_scales, w, max_n: int, group: int = 1,
                   scores=None, block_max=None, head_dots=None, stream=None):
    """Full-layer scan. Returns (scores, block_max, head_dots) as passed (None where not requested)."""
    nq = n_vis.shape[0]
    _need(k_base, torch.int64, "k_base")
    _need(n_vis, torch.int32, "n_vis")
    _need(w, torch.float32, "w")
    ss = scores.stride(0) if scores is not None else (head_dots.shape[-1] if head_dots is not None else 0)
    bs = block_max.stride(0) if block_max is not None else 0
    _call(lib.idx_score_full, _ptr(k_codes), _ptr(k_scales), _ptr(k_base), _ptr(n_vis), nq, group, max_n,
          _ptr(q_codes), _ptr(q_scales), _ptr(w),
          _ptr(scores) if head_dots is not None else _rows_ptr(scores), ss,
          _rows_ptr(block_max), bs, _ptr(head_dots), _stream(stream))
    return scores, block_max, head_dots


def idx_build_pool(block_max, n_vis, max_n: int, pool_blocks, pool_count, ws, topk_blocks: int = 2048,
                   block: int = BLOCK, stream=None):
    nq = n_vis.shape[0]
    _need(block_max, torch.float32, "block_max")
    _need(pool_blocks, torch.int32, "pool_blocks")
    _call(lib.idx_build_pool, _rows_ptr(block_max), block_max.stride(0), _ptr(n_vis), nq, max_n, topk_blocks, block,
          _ptr(pool_blocks), pool_blocks.stride(0), _ptr(pool_count), _ptr(ws), ws.numel(),
          _stream(stream))
    return pool_blocks, pool_count


def idx_build_pool_noalloc(block_max, n_vis, max_n: int, pool_blocks, pool_count, topk_blocks: int = 2048,
                           block: int = BLOCK, stream=None):
    """idx_build_pool without a workspace (the library's fixed per-GPU scratch); allocates nothing."""
    nq = n_vis.shape[0]
    _need(block_max, torch.float32, "block_max")
    _need(pool_blocks, torch.int32, "pool_blocks")
    _call(lib.idx_build_pool_noalloc, _rows_ptr(block_max), block_max.stride(0), _ptr(n_vis), nq, max_n, topk_blocks,
          block, _ptr(pool_blocks), pool_blocks.stride(0), _ptr(pool_count),
          _stream(stream))
    return pool_blocks, pool_count


def idx_top_blocks(block_max, n_vis, max_n: int, k: int, blocks, count, ws, block: int = BLOCK, stream=None):
    """Top-k blocks by raw block maxima (no pin): ascending ids [nq, >= k] and counts [nq]."""
    nq = n_vis.shape[0]
    _need(block_max, torch.float32, "block_max")
    _need(blocks, torch.int32, "blocks")
    _call(lib.idx_top_blocks, _rows_ptr(block_max), block_max.stride(0), _ptr(n_vis), nq, max_n, k, block,
          _rows_ptr(blocks), blocks.stride(0), _ptr(count), _ptr(ws), ws.numel(), _stream(stream))
    return blocks, count


def idx_score_pool_gather(k_codes, k_scales, k_base, n_vis, blocks, block_count, max_blocks: int, q_codes,
                          q_scales, w, scores, head_dots=None, block: int = BLOCK, stream=None):
    nq = n_vis.shape[0]
    _need(scores, torch.float32, "scores")
    _call(lib.idx_score_pool_gather, _ptr(k_codes), _ptr(k_scales), _ptr(k_base), _ptr(n_vis), nq, _rows_ptr(blocks),
          blocks.stride(0), _ptr(block_count), max_blocks, block, _ptr(q_codes),
          _ptr(q_scales), _ptr(w),
          _ptr(scores) if head_dots is not None else _rows_ptr(scores), scores.stride(0),
          _ptr(head_dots),
          _stream(stream))
    return scores


def idx_topk(scores, max_n: int, k: int, out_idx, ws, n_valid=None, out_val=None, blocks=None, block: int = BLOCK,
             stream=None):
    nq = scores.shape[0]
    _need(scores, torch.float32, "scores")
    _need(out_idx, torch.int32, "out_idx")
    _call(lib.idx_topk, _rows_ptr(scores), scores.stride(0), _ptr(n_valid), nq, max_n, k, _rows_ptr(blocks),
          blocks.stride(0) if blocks is not None else 0, block, _ptr(out_idx), out_idx.stride(0),
          _ptr(out_val), _ptr(ws), ws.numel(), _stream(stream))
    return out_idx, out_val


def idx_quantize_kv(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                    stream=None):
    """Main-KV rows bf16 [..., 512] -> (codes [..., 256] u8, E4M3 scales [..., 32] u8)."""
    _need(x, torch.bfloat16, "x")
    lead = x.shape[:-1]
    rows = x.numel() // MKV_DIM
    if codes is None:
        codes = _empty((*lead, MKV_DIM // 2), torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty((*lead, MKV_DIM // 16), torch.uint8, x.device, stream)
    _call(lib.idx_quantize_kv, _ptr(x), rows, _ptr(codes), _ptr(scales), _stream(stream))
    return codes, scales


def idx_gather_kv(codes, scales, kv_base, n_vis, idx, out=None, k: int | None = None, stream=None):
    """Selected main-KV entries dequantised: idx int32 [nq, >= k] -> bf16 [nq, k, 512]."""
    _need(kv_base, torch.int64, "kv_base")
    _need(n_vis, torch.int32, "n_vis")
    _need(idx, torch.int32, "idx")
    nq = idx.shape[0]
    k = idx.shape[1] if k is None else k
    if out is None:
        out = _empty((nq, k, MKV_DIM), torch.bfloat16, idx.device, stream)
    _need(out, torch.bfloat16, "out")
    _call(lib.idx_gather_kv, _ptr(codes), _ptr(scales), _ptr(kv_base), _ptr(n_vis), nq, _ptr(idx), idx.stride(0), k,
          _ptr(out), _stream(stream))
    return out


def idx_mask_pool(scores, n_vis, max_n: int, pool_blocks, pool_count, group: int = 1, block: int = BLOCK,
                  stream=None):
    """In place: -inf at every visible position outside the pooled blocks (the pool's training
    form); score row t uses pool row t // group."""
    _need(scores, torch.float32, "scores")
    _need(pool_blocks, torch.int32, "pool_blocks")
    nq = n_vis.shape[0]
    _call(lib.idx_mask_pool, _rows_ptr(scores), scores.stride(0), _ptr(n_vis), nq, max_n, _rows_ptr(pool_blocks),
          pool_blocks.stride(0), _ptr(pool_count), group, block, _stream(stream))
    return scores


def idx_topk_pool(scores, n_vis, max_n: int, pool_blocks, pool_count, max_blocks: int, k: int, out_idx,
                  out_val=None, group: int = 1, block: int = BLOCK, stream=None):
    """Top-k of full score rows over the pooled positions only (equal to idx_mask_pool then
    idx_topk, without writing the mask); score row t uses pool row t // group."""
    _need(scores, torch.float32, "scores")
    _need(pool_blocks, torch.int32, "pool_blocks")
    _need(out_idx, torch.int32, "out_idx")
    nq = n_vis.shape[0]
    _call(lib.idx_topk_pool, _rows_ptr(scores), scores.stride(0), _ptr(n_vis), nq, max_n, _rows_ptr(pool_blocks),
          pool_blocks.stride(0), _ptr(pool_count), max_blocks, group, block, k, _ptr(out_idx),
          out_idx.stride(0), _ptr(out_val), _stream(stream))
    return out_idx, out_val


def _arg(t: torch.Tensor, dtype: torch.dtype, shape: tuple | None, name: str) -> int:
    """Address of a contiguous argument of this type and shape (None: any; its place is checked by _same_gpu)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows_arg(t: torch.Tensor, dtype: torch.dtype, rows: int, width: int, name: str) -> tuple:
    """(address, row stride) of a 2-D argument of at least `width` columns, each row contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < width:
        raise ValueError(f"{name} must be [{rows}, >= {width}], got {tuple(shape)}")
    stride, one = t.stride()
    columns = shape[1]
    if one != 1 and columns > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), stride if rows > 1 else max(stride, columns)


def _same_gpu(*tensors) -> None:
    """The arguments lie together on the current device (the library launches there)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"fp4idx tensors must live on one GPU, got {tensors[0].device} and {t.device}")
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"fp4idx tensors must live on the current GPU, got {tensors[0].device}")


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_freqs(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, original: float = 4096.0,
               fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Rotation per position of each pair, fp64 [rot / 2] on `device`, and the factor (mscale) that goes with
    it; scaling stretches a context of `original` positions by `factor` (see idx_rope_freqs in the header)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    freq = torch.empty(max(rot, 0) // 2, dtype=torch.float64)
    mscale = _f32()
    _check(lib.idx_rope_freqs(rot, base, ROPE_SCALINGS[scaling], factor, original, fast, slow, freq.data_ptr(),
                              ctypes.addressof(mscale)))
    return freq.to(device), mscale.value


def idx_rope(x: torch.Tensor, pos: torch.Tensor, freq: torch.Tensor, offset: int | None = None, layout: str = "half",
             mscale: float = 1.0, inverse: bool = False, out: torch.Tensor | None = None, stream=None):
    """Rotate the values offset .. offset + 2 * len(freq) - 1 (default: the last ones) of rows x [tokens, heads,
    dim] (bf16 or fp32, consecutive values, any strides) by pos [tokens] (int64) * freq. out may be x itself;
    inverse=True is the gradient."""
    dtype = x.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {dtype}")
    if x.dim() != 3 or (x.shape[2] > 1 and x.stride(2) != 1):
        raise ValueError("x must be [tokens, heads, dim] with consecutive values")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    if out is None:
        out = _empty(x.shape, dtype, x.device, stream)
    elif out.dtype is not dtype:
        raise TypeError(f"out must be {dtype}, got {out.dtype}")
    elif out.shape != x.shape or (out.shape[2] > 1 and out.stride(2) != 1):
        raise ValueError("out must have x's shape and consecutive values")
    tokens, heads, dim = x.shape
    half = freq.numel()
    pos_ptr = _arg(pos, torch.int64, (tokens,), "pos")
    freq_ptr = _arg(freq, torch.float64, (half,), "freq")
    _same_gpu(x, pos, freq, out)
    x_token, x_head, _ = x.stride()
    out_token, out_head, _ = out.stride()
    _call(lib.idx_rope, x.data_ptr(), 0 if dtype is torch.bfloat16 else 1, tokens, heads, dim, x_token, x_head, pos_ptr,
          freq_ptr, 2 * half, dim - 2 * half if offset is None else offset, ROPE_LAYOUTS[layout], mscale, int(inverse),
          out.data_ptr(), out_token, out_head, _stream(stream))
    return out


def _attend_where(q, codes, scales, n_vis, max_n, kv_base, pages, page_size, seq, idx) -> tuple:
    """Checks shared by the attention calls: the arguments from q to n_vis, and those of the list."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != MKV_DIM:
        raise ValueError(f"q must be [nq, heads, {MKV_DIM}], got {tuple(shape)}")
    nq, heads, _ = shape
    rows, rest = divmod(codes.numel(), MKV_DIM // 2)
    if rest or scales.numel() != rows * (MKV_DIM // 16):
        raise ValueError("codes and scales must hold 256 and 32 bytes for each cache row")
    q_ptr = _arg(q, torch.bfloat16, None, "q")
    codes_ptr = _arg(codes, torch.uint8, None, "codes")
    scales_ptr = _arg(scales, torch.uint8, None, "scales")
    nv_ptr = _arg(n_vis, torch.int32, (nq,), "n_vis")
    base_ptr = pages_ptr = seq_ptr = idx_ptr = None
    pages_stride = nseq = idx_stride = k = 0
    if kv_base is not None:
        base_ptr = _arg(kv_base, torch.int64, (nq,), "kv_base")
    if pages is not None:
        nseq = pages.shape[0]
        pages_ptr, pages_stride = _rows_arg(pages, torch.int32, nseq, 0, "pages")
        if pages.shape[1] * page_size < max_n:
            raise ValueError(f"pages must cover max_n={max_n} positions: {pages.shape[1]} pages of {page_size}")
        pages_ptr = pages_ptr or nv_ptr  # no column: a table all the same, never read
    if seq is not None:
        seq_ptr = _arg(seq, torch.int32, (nq,), "seq")
    if idx is not None:
        idx_ptr, idx_stride = _rows_arg(idx, torch.int32, nq, 0, "idx")
        idx_ptr = idx_ptr or nv_ptr  # no slot: a list all the same, never read
        k = idx.shape[1]
    return ((q_ptr, nq, heads, codes_ptr, scales_ptr, rows, base_ptr, pages_ptr, pages_stride, nseq, page_size, seq_ptr,
             nv_ptr), (idx_ptr, idx_stride, k))


def idx_attend(q, codes, scales, n_vis, max_n: int, scale: float, out, ws, lse=None, window: int = 0, kv_base=None,
               pages=None, page_size: int = 0, seq=None, idx=None, stream=None):
    """Core attention of q [nq, heads, 512] over the FP4 main-KV cache: all visible positions (or the last
    `window`), or those of idx [nq, k]. Rows lie at kv_base [nq] + position, or in pages [nseq, ...] of
    page_size positions (seq [nq] names each query's page row). ws: workspace(IDX_OP_ATTEND, nq, entries, heads),
    or another call's: in a smaller one the queries are cut into fewer parts."""
    where, lst = _attend_where(q, codes, scales, n_vis, max_n, kv_base, pages, page_size, seq, idx)
    out_ptr = _arg(out, torch.bfloat16, q.shape, "out")
    lse_ptr = None if lse is None else _arg(lse, torch.float32, q.shape[:2], "lse")
    ws_ptr = _arg(ws, torch.uint8, None, "ws")
    _same_gpu(q, codes, scales, n_vis, kv_base, pages, seq, idx, out, lse, ws)
    _call(lib.idx_attend, *where, max_n, window, *lst, scale, out_ptr, lse_ptr, ws_ptr, ws.numel(), _stream(stream))
    return out, lse


def idx_attend_weights(q, codes, scales, n_vis, max_n: int, scale: float, lse, weights, kv_base=None, pages=None,
                       page_size: int = 0, seq=None, idx=None, stream=None):
    """The attention's probability of each entry (idx slot, or visible position), mean over the heads, from the
    saved lse [nq, heads], into weights [nq, >= k] (or [nq, >= max_n])."""
    where, lst = _attend_where(q, codes, scales, n_vis, max_n, kv_base, pages, page_size, seq, idx)
    lse_ptr = _arg(lse, torch.float32, q.shape[:2], "lse")
    w_ptr, w_stride = _rows_arg(weights, torch.float32, q.shape[0], max_n if idx is None else lst[2], "weights")
    _same_gpu(q, codes, scales, n_vis, kv_base, pages, seq, idx, lse, weights)
    _call(lib.idx_attend_weights, *where, max_n, *lst, scale, lse_ptr, w_ptr, w_stride, _stream(stream))
    return weights


def _distill_rows(scores, n_vis, max_n, t_idx, t_logit) -> tuple:
    """Checks shared by the two directions: the arguments from scores to k."""
    nq = n_vis.shape[0]
    s_ptr, s_stride = _rows_arg(scores, torch.float32, nq, max_n, "scores")
    nv_ptr = _arg(n_vis, torch.int32, (nq,), "n_vis")
    i_ptr, i_stride = _rows_arg(t_idx, torch.int32, nq, 0, "t_idx")
    if t_logit.shape != t_idx.shape:
        raise ValueError(f"t_logit must have t_idx's shape {tuple(t_idx.shape)}, got {tuple(t_logit.shape)}")
    l_ptr, l_stride = _rows_arg(t_logit, torch.float32, nq, 0, "t_logit")
    k = t_idx.shape[1]
    if nq > 1 and i_stride != l_stride:
        raise ValueError("t_idx and t_logit must have the same row stride")
    return s_ptr, s_stride, nv_ptr, nq, max_n, i_ptr, l_ptr, i_stride if nq > 1 else k, k


def idx_distill(scores, n_vis, max_n: int, t_idx, t_logit, loss, lse, t_lse, ws, inv_temp: float = 1.0, stream=None):
    """KL divergence of score rows [nq, >= max_n] from a teacher's top logits (t_idx, t_logit [nq, k]): writes
    loss, lse and t_lse [nq]. ws: workspace(IDX_OP_DISTILL, nq, max_n, 1)."""
    rows = _distill_rows(scores, n_vis, max_n, t_idx, t_logit)
    each = (rows[3],)
    outs = (_arg(loss, torch.float32, each, "loss"), _arg(lse, torch.float32, each, "lse"),
            _arg(t_lse, torch.float32, each, "t_lse"), _arg(ws, torch.uint8, None, "ws"))
    _same_gpu(scores, n_vis, t_idx, t_logit, loss, lse, t_lse, ws)
    _call(lib.idx_distill, *rows, inv_temp, *outs, ws.numel(), _stream(stream))
    return loss


def idx_distill_bwd(scores, n_vis, max_n: int, t_idx, t_logit, lse, t_lse, dloss, dscores, inv_temp: float = 1.0,
                    stream=None):
    """Gradient of idx_distill with dloss [nq], from its lse and t_lse, into dscores [nq, >= max_n] (visible
    positions only; may be scores itself)."""
    rows = _distill_rows(scores, n_vis, max_n, t_idx, t_logit)
    each = (rows[3],)
    ins = (_arg(lse, torch.float32, each, "lse"), _arg(t_lse, torch.float32, each, "t_lse"),
           _arg(dloss, torch.float32, each, "dloss"))
    d_ptr, d_stride = _rows_arg(dscores, torch.float32, rows[3], max_n, "dscores")
    _same_gpu(scores, n_vis, t_idx, t_logit, lse, t_lse, dloss, dscores)
    _call(lib.idx_distill_bwd, *rows, inv_temp, *ins, d_ptr, d_stride, _stream(stream))
    return dscores


# format: its number, values of a row, code bytes, scale bytes
ROW_FORMATS = {"main": (0, MKV_DIM, MKV_DIM // 2, MKV_DIM // 16), "local": (1, MKV_DIM, MKV_DIM, MKV_DIM // 32),
               "key": (2, DIM, DIM // 2, DIM // 32)}


# (The helpers below ask for a tensor's properties in place, a few tenths of a microsecond less for each than through _arg,
# and leave it to _arg to say what is wrong: the calls of a decode step cost the host more than the card.)
_U8, _I32, _I64, _F32, _F64, _BF16 = torch.uint8, torch.int32, torch.int64, torch.float32, torch.float64, torch.bfloat16


def _row_format(format, codes, scales) -> tuple:
    """(number, values of a row, address of codes, of scales, rows) of a cache in a format"""
    found = ROW_FORMATS.get(format)
    if found is None:
        raise ValueError(f"format must be one of {sorted(ROW_FORMATS)}, got {format!r}")
    if codes.dtype is not _U8 or scales.dtype is not _U8 or not codes.is_contiguous() or not scales.is_contiguous():
        _arg(codes, _U8, None, "codes"), _arg(scales, _U8, None, "scales")
    number, dim, width, groups = found
    size = codes.numel()
    rows = size // width
    if size != rows * width or scales.numel() != rows * groups:
        raise ValueError(f"codes and scales must hold {width} and {groups} bytes for each cache row")
    return number, dim, codes.data_ptr(), scales.data_ptr(), rows


def _places(n, max_n, ring, kv_base, pages, page_size, seq, strided: bool = False) -> tuple:
    """The arguments from kv_base to seq; n: how many kv_base and seq name. strided: seq's numbers may lie apart."""
    base_ptr = pages_ptr = seq_ptr = None
    stride = nseq = 0
    if kv_base is not None:
        if kv_base.dtype is not _I64 or kv_base.shape != (n,) or not kv_base.is_contiguous():
            _arg(kv_base, _I64, (n,), "kv_base")
        base_ptr = kv_base.data_ptr()
    if pages is not None:
        nseq = pages.shape[0]
        pages_ptr, stride = _rows_arg(pages, _I32, nseq, 0, "pages")
        most = min(max_n, ring) if ring else max_n
        if pages.shape[1] * page_size < most:
            raise ValueError(f"pages must cover {most} places: {pages.shape[1]} pages of {page_size}")
        if pages_ptr == 0:  # no column: every place lies outside
            raise ValueError("pages must not be empty")
    if seq is not None:
        if seq.dtype is not _I32 or seq.shape != (n,) or not (strided or seq.is_contiguous()):
            _arg(seq, _I32, (n,), "seq")
        seq_ptr = seq.data_ptr()
    return base_ptr, pages_ptr, stride, nseq, page_size, seq_ptr


def _turn(pos, freq, n, dim, offset, layout) -> tuple:
    """The arguments pos, freq, rot, offset and layout (freq None: no rotation)"""
    if freq is None:
        return None, None, 0, 0, 0
    number = ROPE_LAYOUTS.get(layout)
    if number is None:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    pairs = freq.numel()
    if freq.dtype is not _F64 or freq.dim() != 1 or not freq.is_contiguous():
        _arg(freq, _F64, (pairs,), "freq")
    pos_ptr = None
    if pos is not None:
        if pos.dtype is not _I64 or pos.shape != (n,) or not pos.is_contiguous():
            _arg(pos, _I64, (n,), "pos")
        pos_ptr = pos.data_ptr()
    return pos_ptr, freq.data_ptr(), 2 * pairs, dim - 2 * pairs if offset is None else offset, number


def _value_rows(x, tokens, dim, name) -> tuple:
    """(address, type, row stride) of rows [tokens, dim] of consecutive values"""
    dtype = x.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {dtype}")
    if x.shape != (tokens, dim) or x.stride(1) != 1:
        raise ValueError(f"{name} must be [{tokens}, {dim}] with consecutive values, got {tuple(x.shape)}")
    return x.data_ptr(), 0 if dtype is _BF16 else 1, x.stride(0) if tokens > 1 else dim


def idx_write_rows(format: str, x, codes, scales, at, max_n: int, kv_base=None, pages=None, page_size: int = 0, seq=None,
                   ring: int = 0, gamma=None, eps: float | None = None, pos=None, freq=None, offset: int | None = None,
                   layout: str = "half", mscale: float = 1.0, signs=None, keep=None, stream=None):
    """Rows x [tokens, 512] (keys: 128; bf16 or fp32, any row stride), normalised (with eps; times gamma), turned by
    pos (default: at) * freq, quantised in the cache's format ("main", "local" or "key") and stored in codes and scales
    at entries at [tokens] (int64) below max_n: rows kv_base [tokens] + entry, or of pages [nseq, ...] of page_size
    (seq [tokens] names the page row); with ring, entry % ring takes the entry's place. Tokens with keep [tokens] (int64)
    below 0 are left out."""
    number, dim, codes_ptr, scales_ptr, rows = _row_format(format, codes, scales)
    if at.dtype is not _I64 or at.dim() != 1 or not at.is_contiguous():
        _arg(at, _I64, (at.numel(),), "at")
    tokens = at.numel()
    x_ptr, dtype, stride = _value_rows(x, tokens, dim, "x")
    where = _places(tokens, max_n, ring, kv_base, pages, page_size, seq)
    turn = _turn(pos, freq, tokens, dim, offset, layout)
    if gamma is not None and eps is None:
        raise ValueError("gamma needs eps")
    gamma_ptr = None if gamma is None else _arg(gamma, _F32, (dim,), "gamma")
    signs_ptr = None if signs is None else _arg(signs, torch.int8, (DIM,), "signs")
    fn, kept = lib.idx_write_rows, ()
    if keep is not None:
        fn, kept = lib.idx_write_rows_kept, (_arg(keep, _I64, (tokens,), "keep"),)
    _same_gpu(codes, scales, x, at, kv_base, pages, seq, pos, freq, gamma, signs, keep)
    _call(fn, number, x_ptr, dtype, tokens, stride, int(eps is not None), gamma_ptr, eps or 0.0, *turn, mscale, signs_ptr,
          codes_ptr, scales_ptr, rows, *where, at.data_ptr(), max_n, ring, *kept, _stream(stream))
    return codes, scales


def idx_read_rows(format: str, codes, scales, at, max_n: int, kv_base=None, pages=None, page_size: int = 0, seq=None,
                  ring: int = 0, pos=None, freq=None, offset: int | None = None, layout: str = "half",
                  mscale: float = 1.0, inverse: bool = False, out=None, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The stored rows of entries at [tokens] as values [tokens, 512] (keys: 128) of `dtype` or in out; with freq,
    turned by pos (default: at) as by idx_rope. The other arguments as for idx_write_rows; entries that are not there
    give zeros."""
    number, dim, codes_ptr, scales_ptr, rows = _row_format(format, codes, scales)
    if at.dtype is not _I64 or at.dim() != 1 or not at.is_contiguous():
        _arg(at, _I64, (at.numel(),), "at")
    tokens = at.numel()
    where = _places(tokens, max_n, ring, kv_base, pages, page_size, seq)
    turn = _turn(pos, freq, tokens, dim, offset, layout)
    if out is None:
        out = _empty((tokens, dim), dtype, at.device, stream)
    out_ptr, number_out, stride = _value_rows(out, tokens, dim, "out")
    if stride < dim:
        raise ValueError("out's rows may not overlap")
    _same_gpu(codes, scales, at, kv_base, pages, seq, pos, freq, out)
    _call(lib.idx_read_rows, number, codes_ptr, scales_ptr, rows, *where, at.data_ptr(), max_n, ring, tokens, *turn, mscale,
          int(inverse), out_ptr, number_out, stride, _stream(stream))
    return out


def idx_attend_local(q, codes, scales, n_vis, max_n: int, scale: float, out, ws, lse=None, window: int = 0, ring: int = 0,
                     group: int = 1, kv_base=None, pages=None, page_size: int = 0, seq=None, other=None, other_lse=None,
                     pos=None, freq=None, offset: int | None = None, layout: str = "half", mscale: float = 1.0,
                     stream=None):
    """Attention of q [nq, heads, 512] over the FP8 cache of local positions (IDX_ROWS_LOCAL rows): the last `window`
    visible entries or all of them, joined with `other` (out and lse of the attention over other entries) and, with freq,
    turned back by pos [nq]. Runs of `group` queries are of one sequence; kv_base or seq [nq / group] names its rows, as for
    idx_write_rows; seq may be a view of any stride (seq[::group] of the queries' sequences).
    ws: workspace(IDX_OP_ATTEND_LOCAL, nq, entries, heads), or another call's."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != MKV_DIM:
        raise ValueError(f"q must be [nq, heads, {MKV_DIM}], got {tuple(shape)}")
    nq, heads, _ = shape
    if group < 1 or nq % group:
        raise ValueError(f"group={group} must divide nq={nq}")
    if q.dtype is not _BF16 or not q.is_contiguous():
        _arg(q, _BF16, None, "q")
    if n_vis.dtype is not _I32 or n_vis.shape != (nq,) or not n_vis.is_contiguous():
        _arg(n_vis, _I32, (nq,), "n_vis")
    if out.dtype is not _BF16 or out.shape != shape or not out.is_contiguous():
        _arg(out, _BF16, shape, "out")
    if ws.dtype is not _U8 or not ws.is_contiguous():
        _arg(ws, _U8, None, "ws")
    _, _, codes_ptr, scales_ptr, rows = _row_format("local", codes, scales)
    where = _places(nq // group, max_n, ring, kv_base, pages, page_size, seq, strided=True)
    fn = lib.idx_attend_local
    if seq is not None and nq > group and seq.stride(0) != 1:
        fn, where = lib.idx_attend_local_strided, (*where, seq.stride(0))
    other_ptr = None if other is None else _arg(other, _BF16, shape, "other")
    other_lse_ptr = None if other_lse is None else _arg(other_lse, _F32, (nq, heads), "other_lse")
    turn = _turn(pos, freq, nq, MKV_DIM, offset, layout)
    lse_ptr = None if lse is None else _arg(lse, _F32, (nq, heads), "lse")
    _same_gpu(q, codes, scales, n_vis, kv_base, pages, seq, other, other_lse, pos, freq, out, lse, ws)
    _call(fn, q.data_ptr(), nq, heads, group, codes_ptr, scales_ptr, rows, *where, n_vis.data_ptr(), max_n,
          window, ring, scale, other_ptr, other_lse_ptr, *turn, mscale, out.data_ptr(), lse_ptr, ws.data_ptr(), ws.numel(),
          _stream(stream))
    return out, lse
