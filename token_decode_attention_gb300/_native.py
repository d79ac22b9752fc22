"""ctypes binding of libdattn (include/dattn.h).

Argument marshalling only: every function here checks dtypes, devices, shapes
and contiguity of torch tensors, passes raw device pointers and the current
CUDA stream to the C ABI, and turns a non-zero status into ``DattnError``.
All arithmetic runs in the library's CUDA kernels.  There is no fallback: if
``libdattn.so`` is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

_LIB = None


class DattnError(RuntimeError):
    """A libdattn entry point returned a non-zero status."""

    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {status_name(status)}: {message}")


class Plan(ctypes.Structure):
    _fields_ = [("partitions", ctypes.c_int), ("heads_per_cta", ctypes.c_int),
                ("head_groups", ctypes.c_int), ("stage_positions", ctypes.c_int),
                ("stages", ctypes.c_int), ("threads_per_cta", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
                ("sm_count", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t),
                ("cluster_size", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class RopeParams(ctypes.Structure):
    """struct dattn_rope_params."""
    _fields_ = [("rope_dims", ctypes.c_int), ("traditional", ctypes.c_int),
                ("rope_base", ctypes.c_double), ("scaling", ctypes.c_int),
                ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


# status codes (enum dattn_status)
(OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT,
 ERR_BAD_PAGE, ERR_BAD_POSITION) = (0, -1, -2, -3, -4, -5, -6, -7, -8)

# enum dattn_dtype, dattn_kv_type, dattn_rope_scaling
_DTYPES = {torch.float16: 1, torch.bfloat16: 2, torch.float32: 3}
_KV_TYPES = {torch.float8_e4m3fn: 1, torch.int8: 2}
_ROPE_SCALINGS = {"linear": 1, "base": 2, "by_parts": 3}

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_ROPE = ctypes.POINTER(RopeParams)
_SIGNATURES = {
    "dattn_version": ([], _I),
    "dattn_status_string": ([_I], ctypes.c_char_p),
    "dattn_last_error": ([], ctypes.c_char_p),
    "dattn_decode_plan": ([_I, _I, _I, _I, _I, ctypes.POINTER(Plan)], _I),
    "dattn_decode_paged_plan": ([_I, _I, _I, _I, _I, ctypes.c_longlong, _I, ctypes.POINTER(Plan)],
                                _I),
    "dattn_decode_workspace_bytes": ([_I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)], _I),
    "dattn_decode_f16_ex": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, ctypes.c_size_t, _I, _P],
                            _I),
    "dattn_decode_f16": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "dattn_decode_paged_f16": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_longlong, _P, _P, _P,
                                ctypes.c_size_t, _I, _P], _I),
    "dattn_decode_f16_noalloc": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "dattn_qk_f16": ([_P, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "dattn_pv_f16": ([_P, _P, _P, _I, _I, _I, _I, _P], _I),
    "dattn_device_error": ([_I], _I),
    "dattn_selftest_wait_timeout": ([_P], _I),
    "dattn_softmax_f32": ([_P, _P, ctypes.c_longlong, _I, _P], _I),
    "dattn_rope_append_f16": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_double, _I,
                               _P, _P], _I),
    "dattn_rope_append_paged_f16": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                     ctypes.c_longlong, _P, _I, ctypes.c_double, _I, _P, _P], _I),
    "dattn_rope": ([_P, _P, _I, _L, _I, _I, _L, _L, _P, _ROPE, _I, _P], _I),
    "dattn_rope_append_q8": ([_P] * 8 + [_I, _I, _I, _I, _P, _L, _L, _L, _I, _I, _I, _I, _ROPE, _P,
                                         _P], _I),
    "dattn_rope_append_paged_q8": ([_P] * 8 + [_I, _I, _I, _I, _P, _L, _L, _L, _I, _I, _I, _I, _I,
                                               _L, _P, _ROPE, _P, _P], _I),
    "dattn_decode_q8_plan": ([_I] * 6 + [ctypes.POINTER(Plan)], _I),
    "dattn_decode_q8_workspace_bytes": ([_I] * 6 + [ctypes.POINTER(ctypes.c_size_t)], _I),
    "dattn_decode_q8": ([_P] * 6 + [_I] * 7 + [_P, _P, ctypes.c_size_t, _I, _P], _I),
    "dattn_decode_paged_q8": ([_P] * 6 + [_I] * 8 + [_L, _P, _P, _P, ctypes.c_size_t, _I, _P], _I),
    "dattn_attend_workspace_bytes": ([_I] * 9 + [ctypes.POINTER(ctypes.c_size_t)], _I),
    "dattn_attend": ([_P] * 4 + [_I, _I, _I, _P, _L] + [_I] * 6 + [_P, _P, ctypes.c_size_t, _P], _I),
    "dattn_attend_paged": ([_P] * 4 + [_I, _I, _I, _P, _L] + [_I] * 5
                           + [_L, _P, _I, _I, _P, _P, ctypes.c_size_t, _P], _I),
    "dattn_decode_shared_workspace_bytes": ([_I] * 6 + [ctypes.POINTER(ctypes.c_size_t)], _I),
    "dattn_decode_shared": ([_P] * 6 + [_I, _I, _L] + [_I] * 5 + [_P, _P, ctypes.c_size_t, _P], _I),
    "dattn_decode_shared_paged": ([_P] * 4 + [_I, _I, _L] + [_I] * 5
                                  + [_L, _P, _I, _P, _P, ctypes.c_size_t, _P], _I),
    "dattn_batch_begin": ([_P], _I),
    "dattn_batch_end": ([_P, ctypes.POINTER(ctypes.c_void_p)], _I),
    "dattn_batch_launch": ([_P, _P], _I),
    "dattn_batch_nodes": ([_P], ctypes.c_longlong),
    "dattn_batch_destroy": ([_P], _I),
}


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Open libdattn and declare every exported signature."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"libdattn is not built ({p} missing); run "
                           "__graft_entry__.build() or python -m "
                           "token_decode_attention_gb300.build")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _LIB = lib
    return lib


def status_name(status: int) -> str:
    return load().dattn_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise DattnError(status, where, load().dattn_last_error().decode())


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _tensor(t: torch.Tensor, name: str, shape=None, dtype=torch.float16) -> int:
    """Raw pointer of a CUDA tensor, or of a pinned (page-locked) CPU tensor: with
    unified addressing pinned host memory has the same address on the device, and
    the kernels read or write it over the CPU-GPU link."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (call .contiguous() first)")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _cur_pos(t: torch.Tensor, B: int) -> int:
    if t.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32)):
        raise TypeError(f"current_pos must be int32 or uint32, got {t.dtype}")
    return _tensor(t, "current_pos", (B,), t.dtype)


def _qkv_dims(q, k):
    if q.dim() != 3 or k.dim() != 4:
        raise ValueError("Q must be [batch, n_heads, head_dim] and K/V "
                         "[batch, seq_len, n_heads, head_dim]")
    B, H, D = q.shape
    S = k.shape[1]
    return int(B), int(H), int(D), int(S)


# ----------------------------------------------------------- C-ABI mirrors

def dattn_version() -> int:
    return int(load().dattn_version())


def dattn_decode_plan(batch: int, n_heads: int, head_dim: int, seq_len: int,
                      num_partitions: int = 0) -> dict:
    plan = Plan()
    _check(load().dattn_decode_plan(batch, n_heads, head_dim, seq_len, num_partitions,
                                    ctypes.byref(plan)), "dattn_decode_plan")
    return plan.as_dict()


def dattn_decode_paged_plan(batch: int, n_heads: int, head_dim: int, page_size: int,
                            max_pages: int, num_pages: int, num_partitions: int = 0) -> dict:
    plan = Plan()
    _check(load().dattn_decode_paged_plan(batch, n_heads, head_dim, page_size, max_pages,
                                          num_pages, num_partitions, ctypes.byref(plan)),
           "dattn_decode_paged_plan")
    return plan.as_dict()


def dattn_decode_workspace_bytes(batch: int, n_heads: int, head_dim: int, seq_len: int,
                                 num_partitions: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(load().dattn_decode_workspace_bytes(batch, n_heads, head_dim, seq_len, num_partitions,
                                               ctypes.byref(n)),
           "dattn_decode_workspace_bytes")
    return int(n.value)


def dattn_decode_f16_ex(q, k, v, out, current_pos, workspace=None, num_partitions: int = 0,
                        stream=None) -> None:
    B, H, D, S = _qkv_dims(q, k)
    args = (_tensor(q, "Q", (B, H, D)), _tensor(k, "K_cache", (B, S, H, D)),
            _tensor(v, "V_cache", (B, S, H, D)), _tensor(out, "out", (B, H, D)))
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _tensor(workspace, "workspace", None, workspace.dtype)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().dattn_decode_f16_ex(*args, B, H, D, S, _cur_pos(current_pos, B), ws_ptr,
                                      ws_bytes, num_partitions, _stream_handle(stream)),
           "dattn_decode_f16_ex")


def dattn_decode_paged_f16(q, k_pages, v_pages, out, block_table, current_pos, workspace=None,
                           num_partitions: int = 0, stream=None) -> None:
    if q.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("Q must be [batch, n_heads, head_dim], pages [num_pages, page_size, "
                         "n_heads, head_dim], block_table [batch, max_pages]")
    B, H, D = (int(x) for x in q.shape)
    num_pages, page_size = int(k_pages.shape[0]), int(k_pages.shape[1])
    max_pages = int(block_table.shape[1])
    args = (_tensor(q, "Q", (B, H, D)), _tensor(k_pages, "K_pages", (num_pages, page_size, H, D)),
            _tensor(v_pages, "V_pages", (num_pages, page_size, H, D)),
            _tensor(out, "out", (B, H, D)))
    table = _tensor(block_table, "block_table", (B, max_pages), torch.int32)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _tensor(workspace, "workspace", None, workspace.dtype)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().dattn_decode_paged_f16(*args, B, H, D, page_size, max_pages, num_pages, table,
                                         _cur_pos(current_pos, B), ws_ptr, ws_bytes,
                                         num_partitions, _stream_handle(stream)),
           "dattn_decode_paged_f16")


def dattn_decode_f16(q, k, v, out, current_pos, stream=None) -> None:
    B, H, D, S = _qkv_dims(q, k)
    _check(load().dattn_decode_f16(_tensor(q, "Q", (B, H, D)), _tensor(k, "K_cache", (B, S, H, D)),
                                   _tensor(v, "V_cache", (B, S, H, D)),
                                   _tensor(out, "out", (B, H, D)), B, H, D, S,
                                   _cur_pos(current_pos, B), _stream_handle(stream)),
           "dattn_decode_f16")


def dattn_qk_f16(q, k, scores, current_pos, stream=None) -> None:
    B, H, D, S = _qkv_dims(q, k)
    _check(load().dattn_qk_f16(_tensor(q, "Q", (B, H, D)), _tensor(k, "K_cache", (B, S, H, D)),
                               _tensor(scores, "scores", (B, H, S)), B, H, D, S,
                               _cur_pos(current_pos, B), _stream_handle(stream)),
           "dattn_qk_f16")


def dattn_pv_f16(scores, v, out, stream=None) -> None:
    if scores.dim() != 3 or v.dim() != 4:
        raise ValueError("scores must be [batch, n_heads, seq_len], V [batch, seq_len, n_heads, "
                         "head_dim]")
    B, H, S = (int(x) for x in scores.shape)
    D = int(v.shape[3])
    _check(load().dattn_pv_f16(_tensor(scores, "scores", (B, H, S)),
                               _tensor(v, "V_cache", (B, S, H, D)),
                               _tensor(out, "out", (B, H, D)), B, H, D, S,
                               _stream_handle(stream)), "dattn_pv_f16")


def dattn_device_error(clear: bool = True) -> int:
    """Status of the device error word (DATTN_OK, or the TIMEOUT, BAD_PAGE or
    BAD_POSITION it records); never raises on those, so callers can assert on it."""
    st = int(load().dattn_device_error(1 if clear else 0))
    if st not in (OK, ERR_TIMEOUT, ERR_BAD_PAGE, ERR_BAD_POSITION):
        _check(st, "dattn_device_error")
    return st


def dattn_softmax_f32(x, out, stream=None) -> None:
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    rows, cols = (int(v) for v in x.shape)
    _check(load().dattn_softmax_f32(_tensor(x, "x", (rows, cols), torch.float32),
                                    _tensor(out, "out", (rows, cols), torch.float32), rows, cols,
                                    _stream_handle(stream)), "dattn_softmax_f32")


def softmax(x, out=None, stream=None):
    """Row softmax over the last dimension of a float32 [rows, cols] tensor."""
    if out is None:
        out = torch.empty_like(x)
    dattn_softmax_f32(x, out, stream)
    return out


def dattn_rope_append_f16(q_new, k_new, v_new, q_out, k_cache, v_cache, current_pos,
                          rope_dims: int = 0, rope_base: float = 10000.0,
                          traditional: bool = False, stream=None) -> None:
    if q_new.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q_new must be [batch, n_heads, head_dim], the cache [batch, seq_len, "
                         "n_heads, head_dim]")
    B, H, D = (int(x) for x in q_new.shape)
    S = int(k_cache.shape[1])
    new = [_tensor(t, n, (B, H, D)) for t, n in ((q_new, "q_new"), (k_new, "k_new"),
                                                 (v_new, "v_new"), (q_out, "q_out"))]
    _check(load().dattn_rope_append_f16(*new, _tensor(k_cache, "K_cache", (B, S, H, D)),
                                        _tensor(v_cache, "V_cache", (B, S, H, D)), B, H, D, S,
                                        rope_dims or D, float(rope_base), int(bool(traditional)),
                                        _cur_pos(current_pos, B), _stream_handle(stream)),
           "dattn_rope_append_f16")


def dattn_rope_append_paged_f16(q_new, k_new, v_new, q_out, k_pages, v_pages, block_table,
                                current_pos, rope_dims: int = 0, rope_base: float = 10000.0,
                                traditional: bool = False, stream=None) -> None:
    if q_new.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q_new must be [batch, n_heads, head_dim], pages [num_pages, page_size, "
                         "n_heads, head_dim], block_table [batch, max_pages]")
    B, H, D = (int(x) for x in q_new.shape)
    num_pages, page_size = int(k_pages.shape[0]), int(k_pages.shape[1])
    max_pages = int(block_table.shape[1])
    new = [_tensor(t, n, (B, H, D)) for t, n in ((q_new, "q_new"), (k_new, "k_new"),
                                                 (v_new, "v_new"), (q_out, "q_out"))]
    _check(load().dattn_rope_append_paged_f16(
        *new, _tensor(k_pages, "K_pages", (num_pages, page_size, H, D)),
        _tensor(v_pages, "V_pages", (num_pages, page_size, H, D)), B, H, D, page_size, max_pages,
        num_pages, _tensor(block_table, "block_table", (B, max_pages), torch.int32),
        rope_dims or D, float(rope_base), int(bool(traditional)), _cur_pos(current_pos, B),
        _stream_handle(stream)), "dattn_rope_append_paged_f16")


def rope_append(q_new, k_new, v_new, k_cache, v_cache, current_pos, rope_dims: int = 0,
                rope_base: float = 10000.0, traditional: bool = False, block_table=None,
                q_out=None, stream=None):
    """Rotate the new token's q and k at current_pos[b] and append k, v to the cache
    (dense, or paged when ``block_table`` is given); returns the rotated q."""
    if q_out is None:
        q_out = torch.empty_like(q_new)
    if block_table is None:
        dattn_rope_append_f16(q_new, k_new, v_new, q_out, k_cache, v_cache, current_pos,
                              rope_dims, rope_base, traditional, stream)
    else:
        dattn_rope_append_paged_f16(q_new, k_new, v_new, q_out, k_cache, v_cache, block_table,
                                    current_pos, rope_dims, rope_base, traditional, stream)
    return q_out


def dattn_selftest_wait_timeout(stream=None) -> None:
    _check(load().dattn_selftest_wait_timeout(_stream_handle(stream)),
           "dattn_selftest_wait_timeout")


class Batch:
    """Calls recorded between dattn_batch_begin and dattn_batch_end on a stream,
    replayed as one submission (see include/dattn.h)."""

    def __init__(self, handle: int):
        self.handle = handle

    def launch(self, stream=None) -> None:
        _check(load().dattn_batch_launch(self.handle, _stream_handle(stream)),
               "dattn_batch_launch")

    @property
    def nodes(self) -> int:
        return int(load().dattn_batch_nodes(self.handle))

    def close(self) -> None:
        if self.handle:
            _check(load().dattn_batch_destroy(self.handle), "dattn_batch_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_RECORDING: set[int] = set()  # streams between dattn_batch_begin and dattn_batch_end


def dattn_batch_begin(stream) -> None:
    handle = _stream_handle(stream)
    _check(load().dattn_batch_begin(handle), "dattn_batch_begin")
    _RECORDING.add(handle)


def dattn_batch_end(stream) -> Batch:
    h = ctypes.c_void_p(0)
    handle = _stream_handle(stream)
    _RECORDING.discard(handle)
    _check(load().dattn_batch_end(handle, ctypes.byref(h)), "dattn_batch_end")
    return Batch(h.value)


# ------------------------------------------------------- convenience forms

def decode(q, k, v, current_pos, num_partitions: int = 0, out=None, workspace=None, stream=None):
    """Fused decode attention; allocates ``out`` and the workspace with torch if not given."""
    B, H, D, S = _qkv_dims(q, k)
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        n = dattn_decode_workspace_bytes(B, H, D, S, num_partitions)
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=q.device)
    dattn_decode_f16_ex(q, k, v, out, current_pos, workspace, num_partitions, stream)
    return out


def decode_paged(q, k_pages, v_pages, block_table, current_pos, num_partitions: int = 0,
                 out=None, workspace=None, stream=None):
    """Fused decode over a paged cache; allocates ``out`` and the workspace if not given."""
    B, H, D = (int(x) for x in q.shape)
    S = int(k_pages.shape[1]) * int(block_table.shape[1])
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        n = dattn_decode_workspace_bytes(B, H, D, S, num_partitions)
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=q.device)
    dattn_decode_paged_f16(q, k_pages, v_pages, out, block_table, current_pos, workspace,
                           num_partitions, stream)
    return out


def qk(q, k, current_pos, scores=None, stream=None):
    B, H, D, S = _qkv_dims(q, k)
    if scores is None:
        scores = torch.empty((B, H, S), dtype=torch.float16, device=q.device)
    dattn_qk_f16(q, k, scores, current_pos, stream)
    return scores


def pv(scores, v, out=None, stream=None):
    B, H, S = (int(x) for x in scores.shape)
    if out is None:
        out = torch.empty((B, H, int(v.shape[3])), dtype=torch.float16, device=v.device)
    dattn_pv_f16(scores, v, out, stream)
    return out


# ------------------------------------- rotary positions and the 8-bit KV cache
#
# A step of one token takes the GPU 2 to 8 us, less than a check of every argument
# by itself would take the host.  The calls below first test what an ordinary call
# looks like (CUDA tensors of the current device, right types and shapes) in one
# expression of attribute reads; only where it does not hold do the checks run
# that name what is wrong, or accept pinned host memory.

_F16, _F32 = torch.float16, torch.float32
_INDEX = (torch.int32, getattr(torch, "uint32", torch.int32))


# The current stream's handle, without the Stream object that torch.cuda.current_stream()
# builds (3 us) where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(dev: int, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _device() -> int:
    """The current device, or -2 (no tensor's device) where there is none."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


class RopeScaling:
    """Frequencies of a rotation scaled for long contexts (enum dattn_rope_scaling):
    ``kind`` "linear", "base" or "by_parts" (which takes ``original_len``,
    ``low_turns`` and ``high_turns``); ``magnitude`` multiplies the rotated
    channels.  Immutable; make it once and pass it to every call."""

    __slots__ = ("kind", "factor", "original_len", "low_turns", "high_turns", "magnitude",
                 "_hash")

    def __init__(self, kind: str, factor: float, original_len: float = 0.0,
                 low_turns: float = 1.0, high_turns: float = 32.0, magnitude: float = 1.0):
        if kind not in _ROPE_SCALINGS:
            raise ValueError(f"kind must be one of {sorted(_ROPE_SCALINGS)}, got {kind!r}")
        for name, v in (("kind", kind), ("factor", float(factor)),
                        ("original_len", float(original_len)), ("low_turns", float(low_turns)),
                        ("high_turns", float(high_turns)), ("magnitude", float(magnitude))):
            object.__setattr__(self, name, v)
        object.__setattr__(self, "_hash", hash(self._key()))

    def __setattr__(self, name, value):
        raise AttributeError("RopeScaling is immutable")

    def _key(self):
        return (self.kind, self.factor, self.original_len, self.low_turns, self.high_turns,
                self.magnitude)

    def __eq__(self, other):
        return isinstance(other, RopeScaling) and self._key() == other._key()

    def __hash__(self):
        return self._hash

    def __reduce__(self):  # how copies and pickles make it
        return RopeScaling, self._key()

    def __repr__(self):
        return "RopeScaling(" + ", ".join(f"{n}={getattr(self, n)!r}" for n in self.__slots__[:-1]) + ")"


_ROPE_PARAMS: dict[tuple, RopeParams] = {}  # read only once made; a program uses a few


def _rope_params(head_dim: int, rope_dims: int, rope_base: float, traditional: bool,
                 scaling) -> RopeParams:
    key = (rope_dims or head_dim, traditional, rope_base, scaling)
    p = _ROPE_PARAMS.get(key)
    if p is None:
        if scaling is None:
            extra = (0, 1.0, 0.0, 0.0, 0.0, 1.0)
        elif isinstance(scaling, RopeScaling):
            extra = (_ROPE_SCALINGS[scaling.kind], scaling.factor, scaling.original_len,
                     scaling.low_turns, scaling.high_turns, scaling.magnitude)
        else:
            raise TypeError(f"scaling must be a RopeScaling, got {type(scaling).__name__}")
        p = RopeParams(rope_dims or head_dim, 1 if traditional else 0, rope_base, *extra)
        if len(_ROPE_PARAMS) < 256:
            _ROPE_PARAMS[key] = p
    return p


def _on_device(named, dev: int) -> None:
    """Every CUDA tensor on the current device, whose stream the call goes to."""
    for name, t in named:
        if t.is_cuda and t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is "
                             f"cuda:{dev}")


def _like(t, stream, shape=None, dtype=None):
    """A tensor (as `t`, or of that shape and type) from the pool of the stream that
    the call goes to; on the current device where `t` lies in pinned host memory."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _like(t, None, shape, dtype)
    if not t.is_cuda and t.is_pinned():
        return torch.empty(shape or t.shape, dtype=dtype or t.dtype, device="cuda")
    if shape is None:
        if t.is_contiguous():
            return torch.empty_like(t)
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return torch.empty(shape, dtype=dtype, device=t.device)


_forward_ad = torch.autograd.forward_ad


def _follows_tangents() -> bool:
    """Whether a level of forward-mode differentiation has been entered."""
    return getattr(_forward_ad, "_current_level", 0) >= 0


def _has_tangent(t) -> bool:
    return _forward_ad.unpack_dual(t).tangent is not None


_grad_enabled = torch.is_grad_enabled


def _no_derivative(**named) -> None:
    """Refuse a tensor whose derivative torch would follow and this call would lose."""
    grad, dual = _grad_enabled(), _follows_tangents()
    for name, t in named.items():
        if isinstance(t, torch.Tensor) and (grad and t.requires_grad or dual and _has_tangent(t)):
            raise ValueError(f"{name} requires a gradient or has a tangent, which this call does "
                             "not follow: detach it, or call under torch.no_grad()")


# The kernels write through raw pointers: what a call was given to write counts as changed in
# place, so that torch notices where a graph keeps the tensor for a gradient.
_written = torch.autograd.graph.increment_version


def _not_recorded(stream, name: str) -> None:
    """A batch that is being recorded on `stream` cannot own a fresh output."""
    if _RECORDING and _current_stream(_device(), stream) in _RECORDING:
        raise ValueError(f"a recorded call needs an output that outlives the batch: pass {name}")


def _index32(t, name: str, shape) -> None:
    if isinstance(t, torch.Tensor) and t.dtype not in _INDEX:
        raise TypeError(f"{name} must be int32 or uint32, got {t.dtype}")
    _tensor(t, name, shape, getattr(t, "dtype", torch.int32))


def _tokens(t, name: str, dtype, shape=None) -> None:
    """Check a [tokens, heads, head_dim] tensor whose tokens are dense inside and may
    lie apart (a slice of a fused projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous, strides are {t.stride()}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _token_stride(t) -> int:
    n, h, d = t.shape
    return t.stride(0) if n > 1 else h * d


def _rope(x, out, positions, rope_dims, rope_base, traditional, scaling, gradient, stream) -> None:
    dev = _device()
    try:
        dtype, shape = x.dtype, x.shape
        n, h, d = shape
        xs = os_ = h * d
        ordinary = (dtype in _DTYPES and out.dtype is dtype and out.shape == shape
                    and x.is_contiguous() and out.is_contiguous() and positions.dtype in _INDEX
                    and positions.shape == (n,) and positions.is_contiguous()
                    and x.get_device() == dev == out.get_device()
                    and positions.get_device() == dev)
    except (AttributeError, TypeError, ValueError):  # not tensors, or not of three dimensions
        ordinary = False
    if not ordinary:
        _all_tensors(x=x, out=out, positions=positions)
        dtype = x.dtype
        if dtype not in _DTYPES:
            raise TypeError(f"x must be float16, bfloat16 or float32, got {dtype}")
        _tokens(x, "x", dtype)
        _tokens(out, "out", dtype, x.shape)
        _index32(positions, "positions", x.shape[:1])
        _on_device((("x", x), ("out", out), ("positions", positions)), dev)
        n, h, d = x.shape
        xs, os_ = _token_stride(x), _token_stride(out)
    st = load().dattn_rope(x.data_ptr(), out.data_ptr(), _DTYPES[dtype], n, h, d, xs, os_,
                           positions.data_ptr(),
                           _rope_params(d, rope_dims, rope_base, traditional, scaling),
                           1 if gradient else 0, _current_stream(dev, stream))
    if st != OK:
        _check(st, "dattn_rope")


def dattn_rope(x, out, positions, rope_dims: int = 0, rope_base: float = 10000.0,
               traditional: bool = False, scaling=None, gradient: bool = False,
               stream=None) -> None:
    _no_derivative(x=x, out=out)
    _rope(x, out, positions, rope_dims, rope_base, traditional, scaling, gradient, stream)
    _written(out)


def _captured(t) -> bool:
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


def _refuse_capture(t) -> None:
    """Neither pass of torch's graph is captured: a backward pass that is captured while an
    eager graph of the same leaves lives can end the process."""
    if _captured(t):
        raise ValueError("x requires a gradient, which a captured call does not follow: capture "
                         "the call without it and the one with gradient=True")


class _RopeOfGraph(torch.autograd.Function):
    """The rotation as a node of torch's graph.  The map is linear: a tangent is rotated as
    the tensor is, and the gradient is the call with the other ``gradient``; both are nodes
    again where torch asks for one."""

    @staticmethod
    def forward(ctx, x, positions, options):
        ctx.save_for_backward(positions)
        ctx.save_for_forward(positions)
        ctx.options = options
        out = _like(x, None)
        _rope(x, out, positions, *options, None)
        return out

    @staticmethod
    def backward(ctx, g):
        _refuse_capture(g)
        positions, = ctx.saved_tensors
        *options, gradient = ctx.options
        return rope(_dense(g), positions, *options, gradient=not gradient), None, None

    @staticmethod
    def jvp(ctx, tangent, *_):
        positions, = ctx.saved_tensors
        *options, gradient = ctx.options
        return rope(_dense(tangent), positions, *options, gradient=gradient)


def _dense(g):
    """A derivative as torch hands it over (a broadcast sum's, a slice, zeros that are not
    stored) as rows that the kernel takes."""
    at = g.data_ptr()
    if at == 0 or at % 16 or not g.is_contiguous():
        return g.clone(memory_format=torch.contiguous_format)
    return g


def rope(x, positions, rope_dims: int = 0, rope_base: float = 10000.0, traditional: bool = False,
         scaling=None, gradient: bool = False, out=None, stream=None):
    """Rotate x [tokens, heads, head_dim] (f16, bf16 or f32) at ``positions``; with
    ``gradient`` the gradient of the rotated tensor into that of the tensor.  Where x
    requires a gradient or carries a forward-mode tangent, torch follows it through this
    call (without ``out`` and ``stream``, and not while a graph is captured)."""
    if isinstance(x, torch.Tensor) and (x.requires_grad and torch.is_grad_enabled()
                                        or _follows_tangents() and _has_tangent(x)):
        if out is not None or stream is not None:
            raise ValueError("x requires a gradient or has a tangent: out and stream cannot be given")
        _not_recorded(stream, "out")
        _refuse_capture(x)
        return _RopeOfGraph.apply(x, positions, (rope_dims, rope_base, traditional, scaling, gradient))
    if out is not None:
        dattn_rope(x, out, positions, rope_dims, rope_base, traditional, scaling, gradient, stream)
        return out
    _not_recorded(stream, "out")
    out = _like(x, stream)
    _rope(x, out, positions, rope_dims, rope_base, traditional, scaling, gradient, stream)
    return out


def _q8_checks(k, v, k_scale, v_scale, scale_block, block_table, batch, current_pos) -> None:
    """Name what is wrong with an 8-bit cache, its table or the positions."""
    if not isinstance(k, torch.Tensor) or k.dtype not in _KV_TYPES:
        raise TypeError("the cache must be float8_e4m3fn or int8, got "
                        f"{getattr(k, 'dtype', type(k).__name__)}")
    if k.dim() != 4:
        raise ValueError("the cache must be [batch, seq_len, n_kv_heads, head_dim] or [num_pages, "
                         "page_size, n_kv_heads, head_dim]")
    if scale_block < 1:
        raise ValueError(f"scale_block={scale_block} must be positive")
    lead, rows, hk, d = k.shape
    if block_table is None and lead != batch:
        raise ValueError(f"the cache holds {lead} sequences, the batch {batch}")
    sshape = (lead, -(-rows // scale_block), hk)
    _tensor(k, "K cache", k.shape, k.dtype)
    _tensor(v, "V cache", k.shape, k.dtype)
    _tensor(k_scale, "K_scale", sshape, _F32)
    _tensor(v_scale, "V_scale", sshape, _F32)
    if block_table is not None:
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise ValueError("block_table must be [batch, max_pages]")
        _tensor(block_table, "block_table", (batch, block_table.shape[1]), torch.int32)
    _index32(current_pos, "current_pos", (batch,))


def _q8_ordinary(k, v, k_scale, v_scale, scale_block, block_table, batch, current_pos, dev, shape) -> bool:
    """Whether the cache, of that shape, and its companions are what an ordinary call brings."""
    dtype = k.dtype
    lead = shape[0]
    scales = (lead, -(-shape[1] // scale_block), shape[2])
    return (dtype in _KV_TYPES and v.dtype is dtype and v.shape == shape and k_scale.dtype is _F32
            and v_scale.dtype is _F32 and k_scale.shape == scales and v_scale.shape == scales
            and k.is_contiguous() and v.is_contiguous() and k_scale.is_contiguous()
            and v_scale.is_contiguous() and k.get_device() == dev == v.get_device()
            and k_scale.get_device() == dev == v_scale.get_device()
            and current_pos.dtype in _INDEX and current_pos.shape == (batch,)
            and current_pos.is_contiguous() and current_pos.get_device() == dev
            and scale_block > 0
            and (lead == batch if block_table is None else
                 (block_table.dtype is torch.int32 and block_table.ndim == 2
                  and block_table.shape[0] == batch and block_table.is_contiguous()
                  and block_table.get_device() == dev)))


def _all_tensors(**named) -> None:
    for name, t in named.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _meets(lo: int, hi: int, at: int, n: int, step: int, row: int) -> bool:
    """Whether the bytes [lo, hi) hold one of n tokens of `row` bytes, `step` apart from `at`."""
    i = max(0, (lo - row - at) // step + 1)   # the first token that ends past lo
    return i < n and at + i * step < hi


def dattn_rope_append_q8(q_new, k_new, v_new, q_out, k_cache, v_cache, k_scale, v_scale,
                         current_pos, scale_block: int, token_offsets=None, rope_dims: int = 0,
                         rope_base: float = 10000.0, traditional: bool = False, scaling=None,
                         block_table=None, stream=None) -> None:
    """The dense call, or the paged one when ``block_table`` is given."""
    dev = _device()
    try:
        batch, = current_pos.shape
        n, h, d = shape = q_new.shape
        lead, rows, hk, dc = cache = k_cache.shape
        new = (n, hk, dc)
        qs = h * d
        ks = vs = hk * dc
        ordinary = (_q8_ordinary(k_cache, v_cache, k_scale, v_scale, scale_block, block_table,
                                 batch, current_pos, dev, cache)
                    and not (_grad_enabled()
                             and (q_new.requires_grad or k_new.requires_grad or v_new.requires_grad
                                  or q_out.requires_grad or k_cache.requires_grad
                                  or v_cache.requires_grad or k_scale.requires_grad
                                  or v_scale.requires_grad))
                    and getattr(_forward_ad, "_current_level", 0) < 0
                    and q_new.dtype is _F16 and k_new.dtype is _F16 and v_new.dtype is _F16
                    and q_out.dtype is _F16 and q_out.shape == shape and d == dc
                    and k_new.shape == new and v_new.shape == new and q_new.is_contiguous()
                    and k_new.is_contiguous() and v_new.is_contiguous() and q_out.is_contiguous()
                    and q_new.get_device() == dev == k_new.get_device()
                    and v_new.get_device() == dev == q_out.get_device()
                    and (n == batch if token_offsets is None else
                         (token_offsets.dtype is torch.int32
                          and token_offsets.shape == (batch + 1,)
                          and token_offsets.is_contiguous()
                          and token_offsets.get_device() == dev)))
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        ordinary = False
    if not ordinary:
        named = {"q_new": q_new, "k_new": k_new, "v_new": v_new, "q_out": q_out,
                 "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale}
        _all_tensors(**named, current_pos=current_pos)
        _no_derivative(**named)
        batch = current_pos.shape[0] if current_pos.ndim == 1 else -1
        _q8_checks(k_cache, v_cache, k_scale, v_scale, scale_block, block_table, batch, current_pos)
        _tokens(q_new, "q_new", _F16)
        n, h, d = q_new.shape
        lead, rows, hk, dc = k_cache.shape
        if d != dc:
            raise ValueError(f"q_new has head_dim {d}, the cache {dc}")
        _tokens(k_new, "k_new", _F16, (n, hk, d))
        _tokens(v_new, "v_new", _F16, (n, hk, d))
        _tensor(q_out, "q_out", q_new.shape)
        if token_offsets is not None:
            _tensor(token_offsets, "token_offsets", (batch + 1,), torch.int32)
        elif n != batch:
            raise ValueError(f"without token_offsets each sequence brings one token: {n} tokens, "
                             f"{batch} sequences")
        _on_device([(name, t) for name, t in
                    (("q_new", q_new), ("k_new", k_new), ("v_new", v_new), ("q_out", q_out),
                     ("K cache", k_cache), ("V cache", v_cache), ("K_scale", k_scale),
                     ("V_scale", v_scale), ("current_pos", current_pos),
                     ("token_offsets", token_offsets), ("block_table", block_table))
                    if t is not None], dev)
        qs, ks, vs = _token_stride(q_new), _token_stride(k_new), _token_stride(v_new)
    kp, vp, qo = k_new.data_ptr(), v_new.data_ptr(), q_out.data_ptr()
    end, row = qo + 2 * n * h * d, 2 * hk * d
    if (qo < kp + 2 * n * ks and kp < end and _meets(qo, end, kp, n, 2 * ks, row)
            or qo < vp + 2 * n * vs and vp < end and _meets(qo, end, vp, n, 2 * vs, row)):
        raise ValueError("q_out overlaps k_new or v_new")
    args = (q_new.data_ptr(), kp, vp, qo,
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            _KV_TYPES[k_cache.dtype], scale_block, batch, n,
            None if token_offsets is None else token_offsets.data_ptr(), qs, ks, vs, h, hk, d, rows)
    rp = _rope_params(d, rope_dims, rope_base, traditional, scaling)
    if block_table is None:
        st = load().dattn_rope_append_q8(*args, rp, current_pos.data_ptr(),
                                         _current_stream(dev, stream))
        if st != OK:
            _check(st, "dattn_rope_append_q8")
    else:
        st = load().dattn_rope_append_paged_q8(*args, block_table.shape[1], lead,
                                               block_table.data_ptr(), rp, current_pos.data_ptr(),
                                               _current_stream(dev, stream))
        if st != OK:
            _check(st, "dattn_rope_append_paged_q8")
    _written((q_out, k_cache, v_cache, k_scale, v_scale))


def rope_append_q8(q_new, k_new, v_new, k_cache, v_cache, k_scale, v_scale, current_pos,
                   scale_block: int, token_offsets=None, rope_dims: int = 0,
                   rope_base: float = 10000.0, traditional: bool = False, scaling=None,
                   block_table=None, q_out=None, stream=None):
    """Rotate the new tokens' q and k and append k, v to an 8-bit cache (dense, or
    paged when ``block_table`` is given): one token per sequence, or the ragged
    ``token_offsets`` [batch + 1].  ``current_pos`` holds the position of each
    sequence's last new token.  Returns the rotated q."""
    if q_out is None:
        _not_recorded(stream, "q_out")
        q_out = _like(q_new, stream)
    dattn_rope_append_q8(q_new, k_new, v_new, q_out, k_cache, v_cache, k_scale, v_scale,
                         current_pos, scale_block, token_offsets, rope_dims, rope_base, traditional,
                         scaling, block_table, stream)
    return q_out


def dattn_decode_q8_plan(batch: int, n_heads: int, n_kv_heads: int, head_dim: int, seq_len: int,
                         num_partitions: int = 0) -> dict:
    plan = Plan()
    _check(load().dattn_decode_q8_plan(batch, n_heads, n_kv_heads, head_dim, seq_len,
                                       num_partitions, ctypes.byref(plan)), "dattn_decode_q8_plan")
    return plan.as_dict()


_Q8_WORKSPACE: dict[tuple, int] = {}  # the size depends on the shape and the device only


def _q8_workspace(*key) -> int:
    n = _Q8_WORKSPACE.get(key)
    if n is None:
        size = ctypes.c_size_t(0)
        _check(load().dattn_decode_q8_workspace_bytes(*key[1:], ctypes.byref(size)),
               "dattn_decode_q8_workspace_bytes")
        if len(_Q8_WORKSPACE) >= 1024:  # a program that never repeats a shape
            _Q8_WORKSPACE.clear()
        n = _Q8_WORKSPACE[key] = int(size.value)
    return n


def dattn_decode_q8_workspace_bytes(batch: int, n_heads: int, n_kv_heads: int, head_dim: int,
                                    seq_len: int, num_partitions: int = 0) -> int:
    return _q8_workspace(_device(), batch, n_heads, n_kv_heads, head_dim,
                         seq_len, num_partitions)


def _decode_q8(q, k, v, k_scale, v_scale, block_table, current_pos, scale_block, num_partitions,
               out, workspace, stream, allocate):
    dev = _device()
    fresh = out is None and allocate
    try:
        b, h, d = shape = q.shape
        lead, rows, hk, dc = cache = k.shape
        ordinary = (_q8_ordinary(k, v, k_scale, v_scale, scale_block, block_table, b, current_pos,
                                 dev, cache)
                    and not (_grad_enabled()
                             and (q.requires_grad or k.requires_grad or v.requires_grad
                                  or k_scale.requires_grad or v_scale.requires_grad
                                  or not fresh and out.requires_grad))
                    and getattr(_forward_ad, "_current_level", 0) < 0
                    and q.dtype is _F16 and d == dc and q.is_contiguous() and q.get_device() == dev
                    and (fresh or (out.dtype is _F16 and out.shape == shape
                                   and out.is_contiguous() and out.get_device() == dev)))
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        ordinary = False
    if not ordinary:
        named = {"Q": q, "k_cache": k, "v_cache": v, "k_scale": k_scale, "v_scale": v_scale}
        if not fresh:
            named["out"] = out
        _all_tensors(**named, current_pos=current_pos)
        _no_derivative(**named)
        if q.dim() != 3:
            raise ValueError("Q must be [batch, n_heads, head_dim]")
        b, h, d = q.shape
        _q8_checks(k, v, k_scale, v_scale, scale_block, block_table, b, current_pos)
        lead, rows, hk, dc = k.shape
        if d != dc:
            raise ValueError(f"Q has head_dim {d}, the cache {dc}")
        _tensor(q, "Q")
        named = [("Q", q), ("K cache", k), ("V cache", v), ("K_scale", k_scale),
                 ("V_scale", v_scale), ("current_pos", current_pos)]
        if not fresh:
            _tensor(out, "out", q.shape)
            named.append(("out", out))
        if block_table is not None:
            named.append(("block_table", block_table))
        _on_device(named, dev)
    handle = _current_stream(dev, stream)
    wp, wn = None, 0
    if workspace is not None:
        wp = _tensor(workspace, "workspace", None, getattr(workspace, "dtype", None))
        _on_device((("workspace", workspace),), dev)
        wn = workspace.numel() * workspace.element_size()
    elif allocate:
        wn = _q8_workspace(dev, b, h, hk, d,
                           rows if block_table is None else rows * block_table.shape[1],
                           num_partitions)
    if _RECORDING and handle in _RECORDING and (fresh or (wn and wp is None)) and allocate:
        raise ValueError("a recorded decode needs buffers that outlive the batch: pass out and "
                         "workspace (dattn_decode_q8_workspace_bytes)")
    if wn and wp is None:
        workspace = _like(k, stream, (wn,), torch.uint8)
        wp = workspace.data_ptr()
    if fresh:
        out = _like(q, stream)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            out.data_ptr(), _KV_TYPES[k.dtype], scale_block, b, h, hk, d, rows)
    if block_table is None:
        st = load().dattn_decode_q8(*args, current_pos.data_ptr(), wp, wn, num_partitions, handle)
        if st != OK:
            _check(st, "dattn_decode_q8")
    else:
        st = load().dattn_decode_paged_q8(*args, block_table.shape[1], lead, block_table.data_ptr(),
                                          current_pos.data_ptr(), wp, wn, num_partitions, handle)
        if st != OK:
            _check(st, "dattn_decode_paged_q8")
    if not fresh:
        _written(out)
    return out


def dattn_decode_q8(q, k, v, k_scale, v_scale, out, current_pos, scale_block: int, workspace=None,
                    num_partitions: int = 0, block_table=None, stream=None) -> None:
    """The dense call, or the paged one when ``block_table`` is given."""
    _decode_q8(q, k, v, k_scale, v_scale, block_table, current_pos, scale_block, num_partitions,
               out, workspace, stream, False)


def decode_q8(q, k, v, k_scale, v_scale, current_pos, scale_block: int, num_partitions: int = 0,
              out=None, workspace=None, stream=None):
    """Fused decode over an 8-bit cache [batch, seq_len, n_kv_heads, head_dim]
    (float8_e4m3fn or int8) with scales [batch, ceil(seq_len / scale_block),
    n_kv_heads]; allocates ``out`` and the workspace if not given."""
    return _decode_q8(q, k, v, k_scale, v_scale, None, current_pos, scale_block, num_partitions,
                      out, workspace, stream, True)


def decode_paged_q8(q, k_pages, v_pages, k_scale, v_scale, block_table, current_pos,
                    scale_block: int, num_partitions: int = 0, out=None, workspace=None,
                    stream=None):
    """Fused decode over a paged 8-bit cache [num_pages, page_size, n_kv_heads,
    head_dim] with scales [num_pages, page_size / scale_block, n_kv_heads]."""
    return _decode_q8(q, k_pages, v_pages, k_scale, v_scale, block_table, current_pos, scale_block,
                      num_partitions, out, workspace, stream, True)


# ------------------------------------------- attention over a 16-bit cache
#
# As above: an ordinary call is recognised by attribute reads alone.

_BF16 = torch.bfloat16


_ATTEND_WORKSPACE: dict[tuple, int] = {}  # the size depends on the shape and the device only


def _attend_workspace(key: tuple) -> int:
    """Bytes for (device, shared, the arguments of the size query); `shared` tells the two
    queries apart."""
    size = ctypes.c_size_t(0)
    query = "dattn_decode_shared_workspace_bytes" if key[1] else "dattn_attend_workspace_bytes"
    _check(getattr(load(), query)(*key[2:], ctypes.byref(size)), query)
    if len(_ATTEND_WORKSPACE) >= 1024:  # a program that never repeats a shape
        _ATTEND_WORKSPACE.clear()
    n = _ATTEND_WORKSPACE[key] = int(size.value)
    return n


def dattn_attend_workspace_bytes(batch: int, tokens: int, ragged: bool, n_heads: int, n_kv_heads: int,
                                 head_dim: int, seq_len: int, window: int = 0, sinks: int = 0) -> int:
    return _attend_workspace((_device(), False, batch, tokens, 1 if ragged else 0, n_heads, n_kv_heads,
                              head_dim, seq_len, window, sinks))


def dattn_decode_shared_workspace_bytes(batch: int, n_heads: int, n_kv_heads: int, head_dim: int,
                                        shared_len: int, own_len: int) -> int:
    return _attend_workspace((_device(), True, batch, n_heads, n_kv_heads, head_dim, shared_len, own_len))


def _attend(name, q, prefix, k, v, block_table, current_pos, token_offsets, shared_len, window, sinks,
            out, workspace, stream, allocate):
    """Checks and marshalling of dattn_attend and dattn_decode_shared (`prefix`: a pair of
    tensors, or `shared_len` positions of the first sequence's pages)."""
    if window >> 31 or sinks >> 31 or (shared_len or 0) >> 31:
        raise ValueError(f"window={window}, sinks={sinks} and shared_len={shared_len} must be from 0 to 2^31 - 1")
    dev = _device()
    fresh = out is None and allocate
    kp, vp = prefix or (None, None)
    shared = prefix is not None or shared_len is not None
    try:
        batch, = current_pos.shape
        n, h, d = shape = q.shape
        lead, rows, hk, dc = cache = k.shape
        dtype = q.dtype
        qs = h * d
        ordinary = ((dtype is _F16 or dtype is _BF16) and k.dtype is dtype and v.dtype is dtype
                    and v.shape == cache and d == dc and q.is_contiguous() and k.is_contiguous()
                    and v.is_contiguous() and q.get_device() == dev == k.get_device()
                    and v.get_device() == dev
                    and not (_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                                  or not fresh and out.requires_grad
                                                  or kp is not None and (kp.requires_grad or vp.requires_grad)))
                    and getattr(_forward_ad, "_current_level", 0) < 0
                    and (fresh or (out.dtype is dtype and out.shape == shape and out.is_contiguous()
                                   and out.get_device() == dev))
                    and current_pos.dtype in _INDEX and current_pos.is_contiguous()
                    and current_pos.get_device() == dev
                    and (n == batch if token_offsets is None else
                         (token_offsets.dtype is torch.int32 and token_offsets.shape == (batch + 1,)
                          and token_offsets.is_contiguous() and token_offsets.get_device() == dev))
                    and (lead == batch if block_table is None else
                         (block_table.dtype is torch.int32 and block_table.ndim == 2
                          and block_table.shape[0] == batch and block_table.is_contiguous()
                          and block_table.get_device() == dev))
                    and (prefix is None or
                         (kp.dtype is dtype and vp.dtype is dtype and kp.shape == vp.shape
                          and kp.ndim == 3 and kp.shape[1:] == cache[2:] and kp.is_contiguous()
                          and vp.is_contiguous() and kp.get_device() == dev == vp.get_device())))
    except (AttributeError, TypeError, ValueError):
        ordinary = False
    if not ordinary:
        named = {"Q": q, "k_cache": k, "v_cache": v}
        if prefix is not None:
            named.update(k_prefix=kp, v_prefix=vp)
        if not fresh:
            named["out"] = out
        _all_tensors(**named, current_pos=current_pos)
        _no_derivative(**named)
        dtype = q.dtype
        if dtype not in (_F16, _BF16):
            raise TypeError(f"Q must be float16 or bfloat16, got {dtype}")
        _tokens(q, "Q", dtype)
        n, h, d = q.shape
        if k.dim() != 4:
            raise ValueError("the cache must be [batch, seq_len, n_kv_heads, head_dim] or [num_pages, "
                             "page_size, n_kv_heads, head_dim]")
        lead, rows, hk, dc = k.shape
        if d != dc:
            raise ValueError(f"Q has head_dim {d}, the cache {dc}")
        _tensor(k, "K cache", None, dtype)
        _tensor(v, "V cache", k.shape, dtype)
        batch = current_pos.shape[0] if current_pos.ndim == 1 else -1
        _index32(current_pos, "current_pos", (batch,))
        if block_table is None and lead != batch:
            raise ValueError(f"the cache holds {lead} sequences, the batch {batch}")
        named = [("Q", q), ("K cache", k), ("V cache", v), ("current_pos", current_pos)]
        if token_offsets is not None:
            _tensor(token_offsets, "token_offsets", (batch + 1,), torch.int32)
            named.append(("token_offsets", token_offsets))
        elif n != batch:
            raise ValueError(f"without token_offsets each sequence brings one token: {n} tokens, "
                             f"{batch} sequences")
        if block_table is not None:
            if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
                raise ValueError("block_table must be [batch, max_pages]")
            _tensor(block_table, "block_table", (batch, block_table.shape[1]), torch.int32)
            named.append(("block_table", block_table))
        if prefix is not None:
            if kp.dim() != 3:
                raise ValueError("the prefix must be [shared_len, n_kv_heads, head_dim]")
            _tensor(kp, "k_prefix", (kp.shape[0], hk, d), dtype)
            _tensor(vp, "v_prefix", kp.shape, dtype)
            named += [("k_prefix", kp), ("v_prefix", vp)]
        if not fresh:
            _tensor(out, "out", q.shape, dtype)
            named.append(("out", out))
        _on_device(named, dev)
        qs = _token_stride(q)
    handle = _current_stream(dev, stream)
    if prefix is not None:
        shared_len = kp.shape[0]
    table_pages = 0 if block_table is None else block_table.shape[1]
    wp, wn = None, 0
    if workspace is not None:
        wp = _tensor(workspace, "workspace", None, getattr(workspace, "dtype", None))
        _on_device((("workspace", workspace),), dev)
        _apart_from_caches(workspace, k, v)
        wn = workspace.numel() * workspace.element_size()
    elif allocate:
        capacity = rows * table_pages if table_pages else rows
        if shared:
            key = (dev, True, batch, h, hk, d, shared_len,
                   capacity if prefix is not None else max(0, capacity - shared_len))
        else:
            key = (dev, False, batch, n, 0 if token_offsets is None else 1, h, hk, d, capacity, window, sinks)
        wn = _ATTEND_WORKSPACE.get(key)
        if wn is None:
            wn = _attend_workspace(key)
    if _RECORDING and handle in _RECORDING and (fresh or (wn and wp is None)) and allocate:
        raise ValueError(f"a recorded call needs buffers that outlive the batch: pass out and "
                         f"workspace (dattn_{name}_workspace_bytes)")
    if wn and wp is None:
        workspace = _like(k, stream, (wn,), torch.uint8)
        wp = workspace.data_ptr()
    if fresh:
        out = _like(q, stream)
    kind = 1 if dtype is _F16 else 2
    lib = load()
    if shared:
        if block_table is None:
            st = lib.dattn_decode_shared(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), k.data_ptr(),
                                         v.data_ptr(), out.data_ptr(), kind, batch, qs, h, hk, d,
                                         shared_len, rows, current_pos.data_ptr(), wp, wn, handle)
        else:
            st = lib.dattn_decode_shared_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                               kind, batch, qs, h, hk, d, rows, table_pages, lead,
                                               block_table.data_ptr(), shared_len,
                                               current_pos.data_ptr(), wp, wn, handle)
    else:
        at = None if token_offsets is None else token_offsets.data_ptr()
        if block_table is None:
            st = lib.dattn_attend(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), kind, batch,
                                  n, at, qs, h, hk, d, rows, window, sinks, current_pos.data_ptr(), wp,
                                  wn, handle)
        else:
            st = lib.dattn_attend_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), kind,
                                        batch, n, at, qs, h, hk, d, rows, table_pages, lead,
                                        block_table.data_ptr(), window, sinks, current_pos.data_ptr(),
                                        wp, wn, handle)
    if st != OK:
        _check(st, f"dattn_{name}" if block_table is None else f"dattn_{name}_paged")
    if not fresh:
        _written(out)
    return out


def dattn_attend(q, k_cache, v_cache, out, current_pos, window: int = 0, sinks: int = 0,
                 token_offsets=None, block_table=None, workspace=None, stream=None) -> None:
    """The dense call, or the paged one when ``block_table`` is given."""
    _attend("attend", q, None, k_cache, v_cache, block_table, current_pos, token_offsets, None, window,
            sinks, out, workspace, stream, False)


def attend(q, k_cache, v_cache, current_pos, window: int = 0, sinks: int = 0, token_offsets=None,
           block_table=None, out=None, workspace=None, stream=None):
    """Attention of q [tokens, n_heads, head_dim] (f16 or bf16) over a cache [batch,
    seq_len, n_kv_heads, head_dim] of that type (paged when ``block_table`` is given):
    one token per sequence, or the ragged ``token_offsets`` [batch + 1] of a prompt or a
    mixed step.  A token sees the positions up to its own, with ``window`` the last
    ``window`` of them and the first ``sinks``.  ``current_pos`` holds the position of
    each sequence's last new token, whose row is in the cache already.  Allocates ``out``
    and the workspace if not given."""
    return _attend("attend", q, None, k_cache, v_cache, block_table, current_pos, token_offsets, None,
                   window, sinks, out, workspace, stream, True)


def dattn_decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, out, current_pos, workspace=None,
                        stream=None) -> None:
    _attend("decode_shared", q, (k_prefix, v_prefix), k_cache, v_cache, None, current_pos, None, None, 0,
            0, out, workspace, stream, False)


def dattn_decode_shared_paged(q, k_pages, v_pages, out, block_table, current_pos, shared_len: int,
                              workspace=None, stream=None) -> None:
    _attend("decode_shared", q, None, k_pages, v_pages, _table(block_table), current_pos, None,
            _length(shared_len), 0, 0, out, workspace, stream, False)


def decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, current_pos, out=None, workspace=None,
                  stream=None):
    """Decode attention of a batch that shares a prefix [shared_len, n_kv_heads, head_dim],
    read once for all sequences; the cache [batch, seq_len, n_kv_heads, head_dim] and
    ``current_pos`` count what follows it.  Allocates ``out`` and the workspace if not given."""
    return _attend("decode_shared", q, (k_prefix, v_prefix), k_cache, v_cache, None, current_pos, None,
                   None, 0, 0, out, workspace, stream, True)


def decode_shared_paged(q, k_pages, v_pages, block_table, current_pos, shared_len: int, out=None,
                        workspace=None, stream=None):
    """Decode attention over a paged cache whose sequences share their first ``shared_len``
    positions, which are read once, through the first sequence's row of ``block_table``."""
    return _attend("decode_shared", q, None, k_pages, v_pages, _table(block_table), current_pos, None,
                   _length(shared_len), 0, 0, out, workspace, stream, True)


def _apart_from_caches(workspace, k, v) -> None:
    """The C entry compares the workspace with everything but the caches."""
    at = workspace.data_ptr()
    end = at + workspace.numel() * workspace.element_size()
    for name, t in (("K", k), ("V", v)):
        if at < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < end:
            raise ValueError(f"the workspace overlaps the {name} cache")


def _table(block_table):
    if block_table is None:
        raise TypeError("block_table must be a torch.Tensor")
    return block_table


def _length(shared_len):
    if shared_len is None:  # without it _attend is the call that shares nothing
        raise TypeError("shared_len must be an int")
    return shared_len
