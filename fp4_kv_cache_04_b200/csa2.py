"""Python binding of libcsa2.so (ctypes).  Argument marshalling only: every step of the
CSA2 path runs in the library's CUDA kernels.  Tensors are torch CUDA tensors (torch is
used for device memory and streams); each function has the name of its C entry point
without the ``csa2_`` prefix.  Errors raise ``Csa2Error`` with the library's status.

There is no fallback: if the shared library is missing or fails to load, importing this
module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libcsa2.so not built at {LIB_PATH}; run __graft_entry__.build() "
                      "or python -m fp4_kv_cache_04_b200.build")
_lib = ctypes.CDLL(LIB_PATH)

# Constants mirrored from include/csa2.h
D = 512
GROUP = 16
ROW_CODES = 256
ROW_SCALES = 32
HEADS = 16
IDX_HEADS = 4
IDX_DIM = 64
TOPK = 512
WINDOW = 128
POOL_BLOCKS = 2048
POOL_BLOCK = 8
MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2
CACHE_OFF, CACHE_FILL, CACHE_USE = 0, 1, 2
SWA_BF16, SWA_FP8 = 0, 1
Q_BF16, Q_NVFP4 = 0, 1

T_BF16, T_F16, T_F32 = 0, 1, 2
ROPE_NORM, ROPE_INVERSE, ROPE_HALF = 1, 2, 4
TYPES = {torch.bfloat16: T_BF16, torch.float16: T_F16, torch.float32: T_F32}

OK = 0
STATUS_NAMES = {0: "CSA2_OK", 1: "CSA2_ERR_INVALID_ARG", 2: "CSA2_ERR_UNSUPPORTED",
                3: "CSA2_ERR_WORKSPACE", 4: "CSA2_ERR_CUDA", 5: "CSA2_ERR_TIMEOUT",
                6: "CSA2_ERR_DEVICE"}

EXPORTED = ["csa2_status_string", "csa2_last_error", "csa2_abi_version",
            "csa2_kernel_launches", "csa2_quantize_kv", "csa2_append_kv",
            "csa2_index_score", "csa2_topk", "csa2_pool_workspace_size", "csa2_build_pool",
            "csa2_build_pool_noalloc",
            "csa2_workspace_size", "csa2_attend", "csa2_check_device_status", "csa2_set_wait_limit",
            "csa2_norm_rope", "csa2_append_rope", "csa2_dequantize_kv", "csa2_cache_workspace_size",
            "csa2_attend_cache"]


class Csa2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = _lib.csa2_last_error().decode() if status == 4 else ""
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} {detail}".strip())


class IndexArgs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_per_seq", ctypes.c_int32),
                ("ratio", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("max_n", ctypes.c_int64), ("kv_offsets", ctypes.c_void_p),
                ("q_pos", ctypes.c_void_p), ("idx_q", ctypes.c_void_p),
                ("idx_w", ctypes.c_void_p), ("idx_k", ctypes.c_void_p),
                ("idx_kscale", ctypes.c_void_p), ("pool_blocks", ctypes.c_void_p)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("q_per_seq", ctypes.c_int32), ("ratio", ctypes.c_int32),
                ("want_pool", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("max_n", ctypes.c_int64), ("total_n", ctypes.c_int64),
                ("kv_offsets", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("idx_q", ctypes.c_void_p),
                ("idx_w", ctypes.c_void_p), ("idx_k", ctypes.c_void_p),
                ("idx_kscale", ctypes.c_void_p), ("pool_blocks", ctypes.c_void_p),
                ("topk_idx", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("swa_kv", ctypes.c_void_p), ("swa_rows", ctypes.c_int64),
                ("sm_scale", ctypes.c_float), ("reserved1", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("sel_cache", ctypes.c_void_p),
                ("sel_cache_mode", ctypes.c_int32), ("swa_format", ctypes.c_int32),
                ("ev_index_begin", ctypes.c_void_p), ("ev_index_end", ctypes.c_void_p),
                ("swa_kv8", ctypes.c_void_p), ("swa_kscale", ctypes.c_void_p),
                ("pool_k", ctypes.c_void_p), ("pool_kscale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("page_rows", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("q_format", ctypes.c_int32),
                ("reserved2", ctypes.c_int32), ("ev_pool", ctypes.c_void_p)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("in_type", ctypes.c_int32), ("out_type", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("x_row_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("eps", ctypes.c_float), ("reserved0", ctypes.c_int32)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("batch", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("idx_rope_dim", ctypes.c_int32), ("in_type", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("eps", ctypes.c_float), ("latent_stride", ctypes.c_int64), ("idx_stride", ctypes.c_int64),
                ("total_rows", ctypes.c_int64), ("latent", ctypes.c_void_p), ("idx_proj", ctypes.c_void_p),
                ("seq", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("kv_offsets", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("page_rows", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
                ("idx_inv_freq", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("idx_k", ctypes.c_void_p), ("idx_kscale", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p)]


class CacheArgs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_per_seq", ctypes.c_int32), ("ratio", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("max_n", ctypes.c_int64), ("total_n", ctypes.c_int64),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("kv_offsets", ctypes.c_void_p),
                ("q_pos", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("sm_scale", ctypes.c_float), ("reserved0", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("page_rows", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_lib.csa2_status_string.restype = ctypes.c_char_p
_lib.csa2_status_string.argtypes = [_i32]
_lib.csa2_last_error.restype = ctypes.c_char_p
_lib.csa2_abi_version.restype = _i32
_lib.csa2_kernel_launches.restype = ctypes.c_uint64
_lib.csa2_quantize_kv.restype = _i32
_lib.csa2_quantize_kv.argtypes = [_vp, _i64, _i32, _vp, _vp, _vp, _vp]
_lib.csa2_append_kv.restype = _i32
_lib.csa2_append_kv.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.csa2_index_score.restype = _i32
_lib.csa2_index_score.argtypes = [ctypes.POINTER(IndexArgs), _vp, _i64, _vp]
_lib.csa2_topk.restype = _i32
_lib.csa2_topk.argtypes = [_vp, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _vp]
_lib.csa2_pool_workspace_size.restype = _sz
_lib.csa2_pool_workspace_size.argtypes = [_i32, _i64]
_lib.csa2_build_pool.restype = _i32
_lib.csa2_build_pool.argtypes = [_vp, _i64, _vp, _i32, _i64, _vp, _vp, _sz, _vp]
_lib.csa2_build_pool_noalloc.restype = _i32
_lib.csa2_build_pool_noalloc.argtypes = [_vp, _i64, _vp, _i32, _i64, _vp, _vp]
_lib.csa2_workspace_size.restype = _sz
_lib.csa2_workspace_size.argtypes = [ctypes.POINTER(LayerArgs)]
_lib.csa2_attend.restype = _i32
_lib.csa2_attend.argtypes = [ctypes.POINTER(LayerArgs), _vp]
_lib.csa2_norm_rope.restype = _i32
_lib.csa2_norm_rope.argtypes = [ctypes.POINTER(RopeArgs), _vp]
_lib.csa2_append_rope.restype = _i32
_lib.csa2_append_rope.argtypes = [ctypes.POINTER(AppendArgs), _vp]
_lib.csa2_dequantize_kv.restype = _i32
_lib.csa2_dequantize_kv.argtypes = [_vp, _vp, _i64, _vp, _i64, _vp, _vp]
_lib.csa2_cache_workspace_size.restype = _sz
_lib.csa2_cache_workspace_size.argtypes = [ctypes.POINTER(CacheArgs)]
_lib.csa2_attend_cache.restype = _i32
_lib.csa2_attend_cache.argtypes = [ctypes.POINTER(CacheArgs), _vp]
_lib.csa2_check_device_status.restype = _i32
_lib.csa2_check_device_status.argtypes = [_vp, _vp]
_lib.csa2_set_wait_limit.restype = _i32
_lib.csa2_set_wait_limit.argtypes = [_vp, ctypes.c_uint32, _vp]


def lib() -> ctypes.CDLL:
    return _lib


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libcsa2 takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libcsa2 takes contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str) -> None:
    if status != OK:
        raise Csa2Error(status, where)


def abi_version() -> int:
    return _lib.csa2_abi_version()


def kernel_launches() -> int:
    return _lib.csa2_kernel_launches()


def status_string(status: int) -> str:
    return _lib.csa2_status_string(status).decode()


def quantize_kv(x: torch.Tensor, ratio: int, codes: torch.Tensor, scales: torch.Tensor,
                dst_row: torch.Tensor | None = None, stream=None) -> None:
    """bf16 rows [n][512] -> codes [rows][256] u8 + scales [rows][32] u8 (see csa2.h)."""
    assert x.dtype == torch.bfloat16 and codes.dtype == torch.uint8 and scales.dtype == torch.uint8
    _check(_lib.csa2_quantize_kv(_ptr(x), x.shape[0] if x.dim() else 0, ratio, _ptr(dst_row),
                                 _ptr(codes), _ptr(scales), _stream(stream)), "csa2_quantize_kv")


def append_kv(latent: torch.Tensor, idx_proj: torch.Tensor, dst_row: torch.Tensor, codes: torch.Tensor,
              scales: torch.Tensor, idx_k: torch.Tensor, idx_kscale: torch.Tensor, stream=None) -> None:
    """New decode positions: bf16 latent [n][512] and fp32 indexer values [n][64] ->
    FP4 main-KV rows and FP8 indexer-K rows (+ fp32 scales) at rows dst_row."""
    _check(_lib.csa2_append_kv(_ptr(latent), _ptr(idx_proj), latent.shape[0], _ptr(dst_row), _ptr(codes),
                               _ptr(scales), _ptr(idx_k), _ptr(idx_kscale), _stream(stream)), "csa2_append_kv")


def _index_args(batch, q_per_seq, ratio, max_n, kv_offsets, q_pos, idx_q, idx_w, idx_k,
                idx_kscale, pool_blocks) -> IndexArgs:
    return IndexArgs(batch, q_per_seq, ratio, 0, max_n, _ptr(kv_offsets), _ptr(q_pos),
                     _ptr(idx_q), _ptr(idx_w), _ptr(idx_k), _ptr(idx_kscale), _ptr(pool_blocks))


def index_score(*, batch, q_per_seq, max_n, kv_offsets, idx_q, idx_w, idx_k, idx_kscale,
                scores, ratio=1, q_pos=None, pool_blocks=None, stream=None) -> None:
    a = _index_args(batch, q_per_seq, ratio, max_n, kv_offsets, q_pos, idx_q, idx_w, idx_k,
                    idx_kscale, pool_blocks)
    _check(_lib.csa2_index_score(ctypes.byref(a), _ptr(scores), scores.stride(0), _stream(stream)),
           "csa2_index_score")


def topk(scores: torch.Tensor, n_cols: int, k: int, idx_out: torch.Tensor,
         pool_blocks: torch.Tensor | None = None, q_per_seq: int = 1, stream=None) -> None:
    _check(_lib.csa2_topk(_ptr(scores), scores.stride(0), n_cols, scores.shape[0], k,
                          _ptr(pool_blocks), q_per_seq, _ptr(idx_out), _stream(stream)),
           "csa2_topk")


def pool_workspace_size(batch: int, max_n: int) -> int:
    return _lib.csa2_pool_workspace_size(batch, max_n)


def build_pool(scores: torch.Tensor, kv_offsets: torch.Tensor, max_n: int,
               pool_blocks: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _check(_lib.csa2_build_pool(_ptr(scores), scores.stride(0), _ptr(kv_offsets), scores.shape[0],
                                max_n, _ptr(pool_blocks), _ptr(workspace), workspace.numel(),
                                _stream(stream)), "csa2_build_pool")


NOALLOC_POOL_SCRATCH_BYTES = 8 << 20


def build_pool_noalloc(scores: torch.Tensor, kv_offsets: torch.Tensor, max_n: int,
                       pool_blocks: torch.Tensor, stream=None) -> None:
    _check(_lib.csa2_build_pool_noalloc(_ptr(scores), scores.stride(0), _ptr(kv_offsets),
                                        scores.shape[0], max_n, _ptr(pool_blocks),
                                        _stream(stream)), "csa2_build_pool_noalloc")


def layer_args(*, mode, batch, q_per_seq, max_n, kv_offsets, codes, scales, topk_idx, q, swa_kv,
               out, workspace=None, ratio=1, want_pool=False, q_pos=None, idx_q=None, idx_w=None,
               idx_k=None, idx_kscale=None, pool_blocks=None, swa_rows=None, sm_scale=1.0,
               ev_index_begin=None, ev_index_end=None, total_n=None, sel_cache=None,
               sel_cache_mode=0, swa_kv8=None, swa_kscale=None, pool_k=None, pool_kscale=None,
               page_table=None, page_rows=0, q_nvfp4=False, ev_pool=None) -> LayerArgs:
    """swa_kv: bf16 [B][rows][512]; or pass swa_kv=None with swa_kv8 (E4M3 [B][rows][512])
    and swa_kscale (fp32 [B][rows]) for the FP8 SWA format.  pool_k (uint8 [B][16384][64])
    and pool_kscale (fp32 [B][16384]): the HSI pool's rows, contiguous (written by a FULL
    call with want_pool, streamed by REINDEX calls).  page_table (int32 [B][pages]) with
    page_rows: a paged cache (row of position p of sequence b = page_table[b][p // page_rows]
    * page_rows + p % page_rows).  q_nvfp4: the block-scaled FP4 query variant
    (CSA2_Q_NVFP4).  ev_pool (torch.cuda.Event): a FULL call with want_pool records it
    instead of joining its pool work into the stream; a REINDEX call waits for it."""
    swa_format = SWA_FP8 if swa_kv8 is not None else SWA_BF16
    if swa_rows is None:
        swa_rows = (swa_kv8 if swa_kv8 is not None else swa_kv).shape[1]
    if total_n is None:
        total_n = codes.shape[0]           # rows of the packed caches
    return LayerArgs(mode, batch, q_per_seq, ratio, int(bool(want_pool)), 0, max_n, total_n,
                     _ptr(kv_offsets), _ptr(q_pos), _ptr(codes), _ptr(scales), _ptr(idx_q),
                     _ptr(idx_w), _ptr(idx_k), _ptr(idx_kscale), _ptr(pool_blocks),
                     _ptr(topk_idx), _ptr(q), _ptr(swa_kv), swa_rows, sm_scale, 0, _ptr(out),
                     _ptr(workspace), workspace.numel() if workspace is not None else 0,
                     _ptr(sel_cache), sel_cache_mode, swa_format, _event(ev_index_begin),
                     _event(ev_index_end), _ptr(swa_kv8), _ptr(swa_kscale), _ptr(pool_k), _ptr(pool_kscale),
                     _ptr(page_table), int(page_rows), 0 if page_table is None else page_table.shape[1],
                     Q_NVFP4 if q_nvfp4 else Q_BF16, 0, _event(ev_pool))


def _event(ev) -> int | None:
    """torch.cuda.Event -> its cudaEvent_t handle (the event is created if needed)."""
    if ev is None:
        return None
    if isinstance(ev, int):
        return ev
    if ev.cuda_event == 0:
        ev.record()                      # torch creates the CUDA event lazily
        torch.cuda.current_stream().synchronize()
    return ev.cuda_event


def workspace_size(args: LayerArgs) -> int:
    return _lib.csa2_workspace_size(ctypes.byref(args))


def alloc_workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zeroed workspace (the device error word starts cleared)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def attend(args: LayerArgs, stream=None) -> None:
    _check(_lib.csa2_attend(ctypes.byref(args), _stream(stream)), "csa2_attend")


def attend_status(args: LayerArgs, stream=None) -> int:
    """csa2_attend returning the raw status instead of raising (for validation tests)."""
    return _lib.csa2_attend(ctypes.byref(args), _stream(stream))


def check_device_status(workspace: torch.Tensor, stream=None) -> int:
    return _lib.csa2_check_device_status(_ptr(workspace), _stream(stream))


def set_wait_limit(workspace: torch.Tensor, polls: int, stream=None) -> None:
    """Bound (in polls) of the device-side waits of later calls with this workspace; 0 =
    the library default."""
    _check(_lib.csa2_set_wait_limit(_ptr(workspace), int(polls), _stream(stream)), "csa2_set_wait_limit")


# ------------------------------------------------------------------ dense use of the cache
#
# rope_args, append_args and cache_args check their tensors and hold them: 6 to 10 us on the host,
# where a call on a block takes 3.  A loop keeps its blocks, and writes each step's inputs into the
# tensors that they name.


# torch's own calls behind torch.cuda.current_device() and current_stream().cuda_stream, without
# the objects those make (absent in a torch built without CUDA, where nothing is launched)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(f"libcsa2: {what}")


def _same_device(args, *tensors) -> None:
    """The tensors' device goes with the argument block: a call from another current device
    would launch there on this one's pointers."""
    devs = {t.device for t in tensors if t is not None}
    _need(len(devs) == 1, f"tensors on different devices: {sorted(map(str, devs))}")
    args.device = devs.pop().index
    args.tensors = tensors                     # alive as long as the block that points at them


def _launch(fn, args, stream, where: str) -> None:
    """Calls fn(args, stream); the current device must be the one the block's tensors are on."""
    dev = _current_device()
    if dev != args.device:
        raise ValueError(f"libcsa2: {where}: the tensors are on cuda:{args.device}, the current device is cuda:{dev}")
    status = fn(args, _stream(stream) if stream is not None else _raw_stream(dev))
    if status:
        raise Csa2Error(status, where)


def _cache_rows(codes: torch.Tensor, scales: torch.Tensor) -> int:
    """Rows of a cache: the first dimension of two matrices, also of a paged one (pages in turn)."""
    _need(codes.dtype == torch.uint8 and scales.dtype == torch.uint8 and codes.dim() == 2 and scales.dim() == 2 and
          codes.shape[1] == ROW_CODES and scales.shape[1] == ROW_SCALES and codes.shape[0] == scales.shape[0],
          "codes uint8 [rows][256] and scales uint8 [rows][32]")
    return codes.shape[0]


def _vec(t: torch.Tensor | None, dtype, n: int, what: str) -> int | None:
    if t is None:
        return None
    _need(t.dtype == dtype and t.numel() == n, f"{what}: {n} values of {dtype} expected, got {t.numel()} of {t.dtype}")
    return _ptr(t)


def _strided(t: torch.Tensor, what: str) -> int:
    """Device pointer of a tensor whose last dimension is contiguous."""
    if not t.is_cuda:
        raise ValueError("libcsa2 takes CUDA tensors")
    _need(t.dtype in TYPES, f"{what}: bf16, f16 or fp32 expected, got {t.dtype}")
    _need(t.shape[-1] <= 1 or t.stride(-1) == 1, f"{what}: the last dimension must be contiguous")
    return t.data_ptr()


def _step(t: torch.Tensor, dim: int) -> int:
    """Stride of a dimension; 0 where it has one element, whatever torch says there."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


def rope_args(*, x: torch.Tensor, out: torch.Tensor, pos: torch.Tensor | None = None,
              inv_freq: torch.Tensor | None = None, weight: torch.Tensor | None = None, norm: bool = True,
              eps: float = 1e-6, inverse: bool = False, half: bool = False) -> RopeArgs:
    """Arguments of norm_rope.  x, out: [rows][heads][dim] (any row and head strides, last
    dimension contiguous; bf16 / f16 / fp32 each); out may be x.  pos int64 [rows] and
    inv_freq fp32 [r/2] rotate the last r channels of each vector (both None: no rotation);
    weight fp32 [dim] or None with norm.  inverse turns back, half pairs (i, i + r/2).  Keep the
    block for the calls to come (it costs more than the call)."""
    _need(x.dim() == 3 and out.shape == x.shape, "x and out are [rows][heads][dim] of one shape")
    rows, heads, dim = x.shape
    _need((pos is None) == (inv_freq is None), "pos and inv_freq go together")
    r = 0 if inv_freq is None else 2 * inv_freq.numel()
    flags = (ROPE_NORM if norm else 0) | (ROPE_INVERSE if inverse else 0) | (ROPE_HALF if half else 0)
    a = RopeArgs(rows, heads, dim, r, TYPES.get(x.dtype, -1), TYPES.get(out.dtype, -1), flags, _step(x, 0), _step(x, 1),
                 _step(out, 0), _step(out, 1), _strided(x, "x"), _strided(out, "out"),
                 _vec(pos, torch.int64, rows, "pos"), _vec(inv_freq, torch.float32, r // 2, "inv_freq"),
                 _vec(weight, torch.float32, dim, "weight"), eps, 0)
    _same_device(a, x, out, pos, inv_freq, weight)
    return a


def norm_rope(args: RopeArgs, stream=None) -> None:
    """Head norm and rotary positions in one pass (csa2_norm_rope)."""
    _launch(_lib.csa2_norm_rope, args, stream, "csa2_norm_rope")


def append_args(*, latent: torch.Tensor, pos: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                seq: torch.Tensor | None = None, kv_offsets: torch.Tensor | None = None,
                page_table: torch.Tensor | None = None, page_rows: int = 0, weight: torch.Tensor | None = None,
                norm: bool = True, eps: float = 1e-6, inv_freq: torch.Tensor | None = None, half: bool = False,
                idx_proj: torch.Tensor | None = None, idx_inv_freq: torch.Tensor | None = None,
                idx_k: torch.Tensor | None = None, idx_kscale: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> AppendArgs:
    """Arguments of append_rope.  latent [n][512] (bf16 / f16 / fp32, any row stride), pos
    int64 [n] (-1: padding), seq int32 [n] or None (token i belongs to sequence i); the cache
    packed by kv_offsets or paged; idx_proj fp32 [n][64] with idx_k / idx_kscale adds the
    indexer rows.  Keep the block for the calls to come."""
    n = latent.shape[0]
    _need(latent.dim() == 2 and latent.shape[1] == D, "latent is [n][512]")
    total = _cache_rows(codes, scales)
    _need((kv_offsets is None) != (page_table is None), "either kv_offsets or page_table")
    if page_table is not None:
        _need(page_table.dtype == torch.int32 and page_table.dim() == 2, "page_table is int32 [batch][pages]")
        batch, pages = page_table.shape
    else:
        _need(kv_offsets.dtype == torch.int64 and kv_offsets.numel() >= 2, "kv_offsets is int64 [batch+1]")
        batch, pages = kv_offsets.numel() - 1, 0
    if idx_proj is not None:
        _need(idx_proj.dtype == torch.float32 and tuple(idx_proj.shape) == (n, IDX_DIM), "idx_proj is fp32 [n][64]")
        _need(idx_k is not None and idx_kscale is not None and idx_k.dtype == torch.uint8 and
              tuple(idx_k.shape) == (total, IDX_DIM), "idx_k uint8 [rows][64] and idx_kscale fp32 [rows] with idx_proj")
    r = 0 if inv_freq is None else 2 * inv_freq.numel()
    ri = 0 if idx_inv_freq is None else 2 * idx_inv_freq.numel()
    _need(workspace is None or workspace.numel() >= 256, "workspace of 256 bytes or more")
    a = AppendArgs(n, batch, r, ri, TYPES.get(latent.dtype, -1), (ROPE_NORM if norm else 0) | (ROPE_HALF if half else 0),
                   eps, _step(latent, 0) if n > 1 else D, 0 if idx_proj is None else _step(idx_proj, 0) if n > 1 else IDX_DIM, total,
                   _strided(latent, "latent"), None if idx_proj is None else _strided(idx_proj, "idx_proj"),
                   _vec(seq, torch.int32, n, "seq"), _vec(pos, torch.int64, n, "pos"), _ptr(kv_offsets), _ptr(page_table),
                   int(page_rows) if page_table is not None else 0, pages, _vec(inv_freq, torch.float32, r // 2, "inv_freq"),
                   _vec(idx_inv_freq, torch.float32, ri // 2, "idx_inv_freq"), _vec(weight, torch.float32, D, "weight"),
                   _ptr(codes), _ptr(scales), _ptr(idx_k),
                   None if idx_kscale is None else _vec(idx_kscale, torch.float32, total, "idx_kscale"), _ptr(workspace))
    _same_device(a, latent, pos, codes, scales, seq, kv_offsets, page_table, weight, inv_freq, idx_proj, idx_inv_freq,
                 idx_k, idx_kscale, workspace)
    return a


def append_rope(args: AppendArgs, stream=None) -> None:
    """Cache append with norm and rotation on the way (csa2_append_rope)."""
    _launch(_lib.csa2_append_rope, args, stream, "csa2_append_rope")


def dequantize_kv(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, src_row: torch.Tensor | None = None,
                  stream=None) -> None:
    """Cache rows (src_row int64 [n], or rows 0 .. n-1) -> bf16 out [n][512]."""
    n, d = out.shape
    rows, wide = codes.shape
    if (codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8 or out.dtype is not torch.bfloat16 or d != D or
            wide != ROW_CODES or scales.shape != (rows, ROW_SCALES)):
        raise ValueError("libcsa2: codes uint8 [rows][256], scales uint8 [rows][32], out bf16 [n][512]")
    dev = _current_device()
    if (codes.get_device() != dev or scales.get_device() != dev or out.get_device() != dev or not codes.is_contiguous() or
            not scales.is_contiguous() or not out.is_contiguous()):
        raise ValueError("libcsa2: dequantize_kv takes contiguous tensors on the current device")
    src = None
    if src_row is not None:
        if src_row.dtype is not torch.int64 or src_row.numel() != n or src_row.get_device() != dev or not src_row.is_contiguous():
            raise ValueError("libcsa2: src_row is contiguous int64 [n] on the current device")
        src = src_row.data_ptr()
    status = _lib.csa2_dequantize_kv(codes.data_ptr(), scales.data_ptr(), rows, src, n, out.data_ptr(),
                                     _stream(stream) if stream is not None else _raw_stream(dev))
    if status:
        raise Csa2Error(status, "csa2_dequantize_kv")


def cache_args(*, batch: int, max_n: int, kv_offsets: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
               q: torch.Tensor, out: torch.Tensor, q_per_seq: int = 1, q_pos: torch.Tensor | None = None, ratio: int = 1,
               window: int = 0, sinks: int = 0, sm_scale: float = 1.0, lse: torch.Tensor | None = None,
               page_table: torch.Tensor | None = None, page_rows: int = 0,
               workspace: torch.Tensor | None = None) -> CacheArgs:
    """Arguments of attend_cache.  q bf16 and out (bf16 or fp32) [batch * q_per_seq][16][512];
    window 0: every visible position, else the last `window` and the first `sinks` ones; lse
    fp32 [rows][16] or None; a paged cache as in layer_args.  Keep the block (and the
    workspace) for the calls to come."""
    rows = batch * q_per_seq
    _need(q.dtype == torch.bfloat16 and q.numel() == rows * HEADS * D, "q is bf16 [batch * q_per_seq][16][512]")
    _need(out.numel() == rows * HEADS * D, "out is [batch * q_per_seq][16][512]")
    _cache_rows(codes, scales)
    _need(page_table is None or (page_table.dtype == torch.int32 and page_table.dim() == 2 and
                                 page_table.shape[0] == batch), "page_table is int32 [batch][pages]")
    a = CacheArgs(batch, q_per_seq, ratio, TYPES.get(out.dtype, -1), max_n, codes.shape[0], window, sinks,
                  _vec(kv_offsets, torch.int64, batch + 1, "kv_offsets"), _vec(q_pos, torch.int64, batch, "q_pos"),
                  _ptr(codes), _ptr(scales), _ptr(q), sm_scale, 0, _ptr(out),
                  _vec(lse, torch.float32, rows * HEADS, "lse"), _ptr(page_table), int(page_rows) if page_table is not None else 0,
                  0 if page_table is None else page_table.shape[1], _ptr(workspace),
                  workspace.numel() if workspace is not None else 0)
    _same_device(a, kv_offsets, codes, scales, q, out, q_pos, lse, page_table, workspace)
    return a


def cache_workspace_size(args: CacheArgs) -> int:
    """Bytes of workspace; one for the largest batch, max_n and window serves smaller calls."""
    return _lib.csa2_cache_workspace_size(ctypes.byref(args))


def attend_cache(args: CacheArgs, stream=None) -> None:
    """Attention over the whole cache or a window of it (csa2_attend_cache)."""
    _launch(_lib.csa2_attend_cache, args, stream, "csa2_attend_cache")
