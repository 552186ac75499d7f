"""ctypes binding of ``libpagedkv.so`` (declared in ``include/pagedkv.h``).

Argument marshalling only: every function takes torch tensors that already
live on the current CUDA device, passes their data pointers, sizes and the
current stream to the C ABI function of the same name, and raises
:class:`PagedKVError` on a non-zero status.  There is no CPU path: without
the built library every call fails.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB

_lib = None

DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
FP8_E4M3 = 3
FP8_POOL_DTYPES = (torch.uint8, torch.float8_e4m3fn)  # one E4M3 code per element
INT8 = 4  # pools of 8-bit rows, a scale for each row

DEVERR_BLOCK_ID = 0x1
DEVERR_SLOT = 0x2
DEVERR_LENGTH = 0x4
DEVERR_PAIR = 0x8
DEVERR_TIMEOUT = 0x10
DEVERR_POSITION = 0x20

ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}

EXPORTED = (
    "pkv_status_string",
    "pkv_last_cuda_error",
    "pkv_reshape_and_cache",
    "pkv_reshape_and_cache_fp8",
    "pkv_copy_blocks",
    "pkv_swap_blocks",
    "pkv_paged_attention_decode",
    "pkv_paged_attention_decode_fp8",
    "pkv_paged_attention_decode_step",
    "pkv_paged_attention_decode_step_fp8",
    "pkv_paged_attention_decode_static_scratch",
    "pkv_decode_workspace_size",
    "pkv_decode_partition_size",
    "pkv_paged_attention_prefill_chunk",
    "pkv_paged_attention_prefill_chunk_fp8",
    "pkv_prefill_fp8_workspace_size",
    "pkv_paged_attention_decode_multi",
    "pkv_paged_attention_decode_multi_step",
    "pkv_decode_multi_partition_size",
    "pkv_get_device_error",
    "pkv_set_wait_limit_ns",
    "pkv_rope_table",
    "pkv_rope_and_cache",
    "pkv_rope_and_cache_fp8",
    "pkv_rope_and_cache_int8",
    "pkv_int8_block_bytes",
    "pkv_reshape_and_cache_int8",
    "pkv_read_cache_int8",
    "pkv_paged_attention_decode_int8",
    "pkv_paged_attention_decode_step_int8",
    "pkv_paged_attention_prefill_chunk_int8",
)


class RopeSpec(ctypes.Structure):
    """``pkv_rope_spec``."""
    _fields_ = [("base", ctypes.c_double), ("factor", ctypes.c_double), ("alpha", ctypes.c_double),
                ("beta", ctypes.c_double), ("attention_factor", ctypes.c_double),
                ("original_max_position", ctypes.c_int64), ("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)]


class PagedKVError(RuntimeError):
    def __init__(self, what: str, status: int):
        lib = _lib
        msg = lib.pkv_status_string(status).decode() if lib else str(status)
        extra = lib.pkv_last_cuda_error().decode() if lib else ""
        super().__init__(f"{what}: {msg} ({status}){' - ' + extra if extra and status == -4 else ''}")
        self.status = status


def library_path() -> str:
    return LIB


def load_library():
    """Load ``libpagedkv.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError(f"{LIB} is missing: build it with `python -m paged_kv_cache_409_b200.build`")
    lib = ctypes.CDLL(LIB)
    P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.pkv_status_string.argtypes = [I]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_last_cuda_error.argtypes = []
    lib.pkv_last_cuda_error.restype = ctypes.c_char_p
    lib.pkv_reshape_and_cache.argtypes = [P, P, P, P, P, I64, I, I, I, I64, I, P]
    lib.pkv_reshape_and_cache_fp8.argtypes = [P, P, P, P, P, I64, I, I, I, I64, I, F, F, P]
    lib.pkv_paged_attention_decode_fp8.argtypes = [P, P, P, P, P, P, F, F, F, I, I, I, I, I, I, I64, I, I, I, P, SZ,
                                                   P]
    lib.pkv_copy_blocks.argtypes = [P, P, I, P, I64, I64, I64, P]
    lib.pkv_swap_blocks.argtypes = [P, P, P, P, P, I64, I64, I64, I64, P]
    lib.pkv_paged_attention_decode.argtypes = [P, P, P, P, P, P, F, I, I, I, I, I, I, I64, I, I, I, P, SZ, P]
    lib.pkv_decode_workspace_size.argtypes = [I, I, I, I, I]
    lib.pkv_decode_workspace_size.restype = SZ
    lib.pkv_decode_partition_size.argtypes = [I, I, I, I, I, I, I64, I]
    lib.pkv_paged_attention_prefill_chunk.argtypes = [P, P, P, P, P, P, P, I, I64, I, F, I, I, I, I, I, I64, I, P]
    lib.pkv_paged_attention_decode_multi.argtypes = [P, P, P, P, P, P, P, I, I64, I, I, F, I, I, I, I, I, I64, I, I,
                                                     P, SZ, P]
    lib.pkv_paged_attention_decode_multi_step.argtypes = [P, P, P, I64, P, P, P, P, P, P, P, I, I64, I, I, F, I, I,
                                                          I, I, I, I64, I, I, P, SZ, P]
    lib.pkv_decode_multi_partition_size.argtypes = [I, I, I, I]
    lib.pkv_paged_attention_prefill_chunk_fp8.argtypes = [P, P, P, P, P, P, P, I, I64, I, F, F, F, I, I, I, I, I,
                                                          I64, I, P, SZ, P]
    lib.pkv_prefill_fp8_workspace_size.argtypes = [I, I, I, I, I, I64, I, I]
    lib.pkv_prefill_fp8_workspace_size.restype = SZ
    lib.pkv_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), P]
    lib.pkv_paged_attention_decode_step.argtypes = [P, P, P, I64, P, P, P, P, P, P, F, I, I, I, I, I, I, I64, I, I,
                                                    I, P, SZ, P]
    lib.pkv_paged_attention_decode_step_fp8.argtypes = [P, P, P, I64, P, P, P, P, P, P, F, F, F, I, I, I, I, I, I,
                                                        I64, I, I, I, P, SZ, P]
    lib.pkv_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.pkv_rope_table.argtypes = [P, I64, I64, ctypes.POINTER(RopeSpec), P]
    rope = [P, P, P, P, I64, I64, I64, P, P, F, P, I64, I, I, P, P, P, P, I64, I, I, I, I, I64, I]
    lib.pkv_rope_and_cache.argtypes = rope + [P]
    lib.pkv_rope_and_cache_fp8.argtypes = rope + [F, F, P]
    lib.pkv_rope_and_cache_int8.argtypes = rope + [P]
    lib.pkv_int8_block_bytes.argtypes = [I, I, I]
    lib.pkv_int8_block_bytes.restype = I64
    lib.pkv_reshape_and_cache_int8.argtypes = [P, P, P, P, P, I64, I, I, I, I64, I, P]
    lib.pkv_paged_attention_decode_int8.argtypes = lib.pkv_paged_attention_decode.argtypes
    lib.pkv_paged_attention_decode_step_int8.argtypes = lib.pkv_paged_attention_decode_step.argtypes
    lib.pkv_paged_attention_prefill_chunk_int8.argtypes = lib.pkv_paged_attention_prefill_chunk.argtypes
    lib.pkv_read_cache_int8.argtypes = [P, P, P, P, P, I64, I, I, I, I64, I, P]
    for name in ("pkv_reshape_and_cache", "pkv_reshape_and_cache_fp8", "pkv_paged_attention_decode_fp8",
                 "pkv_copy_blocks", "pkv_swap_blocks", "pkv_paged_attention_decode",
                 "pkv_decode_partition_size", "pkv_paged_attention_prefill_chunk", "pkv_get_device_error",
                 "pkv_paged_attention_prefill_chunk_fp8", "pkv_paged_attention_decode_multi",
                 "pkv_paged_attention_decode_multi_step",
                 "pkv_decode_multi_partition_size", "pkv_paged_attention_decode_step",
                 "pkv_paged_attention_decode_step_fp8", "pkv_set_wait_limit_ns", "pkv_rope_table",
                 "pkv_rope_and_cache", "pkv_rope_and_cache_fp8", "pkv_rope_and_cache_int8",
                 "pkv_reshape_and_cache_int8", "pkv_read_cache_int8", "pkv_paged_attention_decode_int8",
                 "pkv_paged_attention_decode_step_int8", "pkv_paged_attention_prefill_chunk_int8"):
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _stream(stream) -> int:
    if stream is None:  # the current stream's handle, without building a Stream object around it
        return torch._C._cuda_getCurrentRawStream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_INT32, _INT64, _UINT8, _FLOAT32 = torch.int32, torch.int64, torch.uint8, torch.float32
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _device(t: torch.Tensor, name: str) -> int:
    """Device index of a call's first tensor, which must be the current device."""
    dev = t.get_device()
    if dev < 0:
        _dev(t, name)  # not a CUDA tensor
    elif dev != _current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return dev


def _at(t: torch.Tensor, name: str, dev: int) -> int:
    """Pointer of a contiguous tensor on device ``dev``."""
    if t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the call's other tensors, not on {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _code(t: torch.Tensor) -> int:
    try:
        return DTYPE_CODE[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def _ok(rc: int, what: str):
    if rc != 0:
        raise PagedKVError(what, rc)


def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, stream=None):
    """Write ``key``/``value`` ``[T, Hkv, D]`` into pool slots ``slot_mapping`` (int64, -1 = skip)."""
    lib = load_library()
    T, Hkv, D = key.shape
    NB, B = key_cache.shape[:2]
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    rc = lib.pkv_reshape_and_cache(_dev(key, "key"), _dev(value, "value"), _dev(key_cache, "key_cache"),
                                   _dev(value_cache, "value_cache"), _dev(slot_mapping, "slot_mapping"), T, Hkv,
                                   D, B, NB, _code(key), _stream(stream))
    _ok(rc, "reshape_and_cache")


def _fp8_pool(t: torch.Tensor, name: str) -> int:
    if t.dtype not in FP8_POOL_DTYPES:
        raise ValueError(f"{name} must be a uint8 or float8_e4m3fn pool of E4M3 codes")
    return _dev(t, name)


def reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale, stream=None):
    """Quantise ``key``/``value`` ``[T, Hkv, D]`` (fp32/fp16/bf16) by ``1/k_scale``, ``1/v_scale`` into the
    E4M3 pools' slots ``slot_mapping`` (int64, -1 = skip)."""
    lib = load_library()
    T, Hkv, D = key.shape
    NB, B = key_cache.shape[:2]
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    rc = lib.pkv_reshape_and_cache_fp8(_dev(key, "key"), _dev(value, "value"), _fp8_pool(key_cache, "key_cache"),
                                       _fp8_pool(value_cache, "value_cache"), _dev(slot_mapping, "slot_mapping"), T,
                                       Hkv, D, B, NB, _code(key), float(k_scale), float(v_scale), _stream(stream))
    _ok(rc, "reshape_and_cache_fp8")


def copy_blocks(key_caches, value_caches, src_dst_pairs, stream=None):
    """Copy block src over block dst in every layer's K and V pool (``src_dst_pairs`` int64 ``[P, 2]``)."""
    lib = load_library()
    L = len(key_caches)
    if L != len(value_caches):
        raise ValueError("key_caches and value_caches differ in length")
    if L == 0:
        return
    kp = (ctypes.c_void_p * L)(*[_dev(c, "key_caches[i]") for c in key_caches])
    vp = (ctypes.c_void_p * L)(*[_dev(c, "value_caches[i]") for c in value_caches])
    NB = key_caches[0].shape[0]
    block_bytes = key_caches[0].numel() // NB * key_caches[0].element_size()
    if src_dst_pairs.dtype != torch.int64:
        raise ValueError("src_dst_pairs must be int64")
    npairs = src_dst_pairs.numel() // 2
    rc = lib.pkv_copy_blocks(kp, vp, L, _dev(src_dst_pairs, "src_dst_pairs") if npairs else None, npairs,
                             block_bytes, NB, _stream(stream))
    _ok(rc, "copy_blocks")


def swap_blocks(src_key, src_value, dst_key, dst_value, src_dst_pairs, stream=None):
    """Move blocks ``src -> dst`` between two pools (device and/or pinned host tensors)."""
    lib = load_library()
    for t, name in ((src_key, "src_key"), (src_value, "src_value"), (dst_key, "dst_key"), (dst_value, "dst_value"),
                    (src_dst_pairs, "src_dst_pairs")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if src_dst_pairs.dtype != torch.int64:
        raise ValueError("src_dst_pairs must be int64")
    block_bytes = src_key[0].numel() * src_key.element_size()
    if dst_key[0].numel() * dst_key.element_size() != block_bytes:
        raise ValueError("pools differ in block size")
    rc = lib.pkv_swap_blocks(src_key.data_ptr(), src_value.data_ptr(), dst_key.data_ptr(), dst_value.data_ptr(),
                             src_dst_pairs.data_ptr(), src_dst_pairs.numel() // 2, block_bytes, src_key.shape[0],
                             dst_key.shape[0], _stream(stream))
    _ok(rc, "swap_blocks")


def decode_workspace_size(num_seqs, num_q_heads, head_dim, max_context_len, partition_size) -> int:
    return int(load_library().pkv_decode_workspace_size(num_seqs, num_q_heads, head_dim, max_context_len,
                                                         partition_size))


def decode_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, dtype,
                          total_context_tokens=0) -> int:
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    rc = load_library().pkv_decode_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                  max_context_len, int(total_context_tokens), code)
    if rc < 0:
        raise PagedKVError("decode_partition_size", rc)
    return rc


def paged_attention_decode(out, query, key_cache, value_cache, block_tables, context_lens, scale, max_context_len,
                           partition_size=None, workspace=None, stream=None, total_context_tokens=0):
    """Decode attention; ``out``/``query`` ``[S, Hq, D]``, pools ``[NB, B, Hkv, D]``.

    ``partition_size`` None picks the library's recommendation (given the
    optional host-side ``total_context_tokens``); a workspace is allocated
    here when one is needed and none is given.
    """
    lib = load_library()
    S, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    MB = block_tables.shape[1] if block_tables.dim() == 2 else 1
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if partition_size is None:
        partition_size = decode_partition_size(S, Hq, Hkv, D, B, max_context_len, query.dtype, total_context_tokens)
    need = decode_workspace_size(S, Hq, D, max_context_len, partition_size) if partition_size else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = _dev(workspace, "workspace") if (need and workspace is not None) else None
    ws_bytes = workspace.numel() * workspace.element_size() if ws_ptr else 0
    rc = lib.pkv_paged_attention_decode(_dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"),
                                        _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables"),
                                        _dev(context_lens, "context_lens"), float(scale), S, Hq, Hkv, D, B, MB, NB,
                                        int(max_context_len), int(partition_size), _code(query), ws_ptr, ws_bytes,
                                        _stream(stream))
    _ok(rc, "paged_attention_decode")
    return out


def paged_attention_decode_fp8(out, query, key_cache, value_cache, block_tables, context_lens, scale, k_scale,
                               v_scale, max_context_len, partition_size=None, workspace=None, stream=None,
                               total_context_tokens=0):
    """Decode attention over E4M3 pools (values ``k_scale * code``, ``v_scale * code``); ``out``/``query``
    ``[S, Hq, D]`` in fp16 or bf16."""
    lib = load_library()
    S, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    MB = block_tables.shape[1] if block_tables.dim() == 2 else 1
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if partition_size is None:
        partition_size = decode_partition_size(S, Hq, Hkv, D, B, max_context_len, FP8_E4M3, total_context_tokens)
    need = decode_workspace_size(S, Hq, D, max_context_len, partition_size) if partition_size else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = _dev(workspace, "workspace") if (need and workspace is not None) else None
    ws_bytes = workspace.numel() * workspace.element_size() if ws_ptr else 0
    rc = lib.pkv_paged_attention_decode_fp8(_dev(out, "out"), _dev(query, "query"), _fp8_pool(key_cache, "key_cache"),
                                            _fp8_pool(value_cache, "value_cache"), _dev(block_tables, "block_tables"),
                                            _dev(context_lens, "context_lens"), float(scale), float(k_scale),
                                            float(v_scale), S, Hq, Hkv, D, B, MB, NB, int(max_context_len),
                                            int(partition_size), _code(query), ws_ptr, ws_bytes, _stream(stream))
    _ok(rc, "paged_attention_decode_fp8")
    return out


def _decode_workspace(S, Hq, Hkv, D, B, max_context_len, dtype_code, partition_size, workspace, device,
                      total_context_tokens):
    """(partition_size, workspace pointer, workspace bytes) of a decode call; allocates a workspace when one
    is needed and none (or too small a one) is given."""
    if partition_size is None:
        partition_size = decode_partition_size(S, Hq, Hkv, D, B, max_context_len, dtype_code, total_context_tokens)
    need = decode_workspace_size(S, Hq, D, max_context_len, partition_size) if partition_size else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    ws_ptr = _dev(workspace, "workspace") if (need and workspace is not None) else None
    ws_bytes = workspace.numel() * workspace.element_size() if ws_ptr else 0
    return int(partition_size), ws_ptr, ws_bytes


def paged_attention_decode_step(new_keys, new_values, slot_mapping, out, query, key_cache, value_cache, block_tables,
                                context_lens, scale, max_context_len, partition_size=None, workspace=None,
                                stream=None, total_context_tokens=0):
    """One decode step: ``reshape_and_cache(new_keys, new_values, ..., slot_mapping)`` then
    ``paged_attention_decode`` in one call (the decode launched as the append's programmatic dependent)."""
    lib = load_library()
    S, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    MB = block_tables.shape[1] if block_tables.dim() == 2 else 1
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    part, ws_ptr, ws_bytes = _decode_workspace(S, Hq, Hkv, D, B, max_context_len, _code(query), partition_size,
                                               workspace, query.device, total_context_tokens)
    rc = lib.pkv_paged_attention_decode_step(_dev(new_keys, "new_keys"), _dev(new_values, "new_values"),
                                             _dev(slot_mapping, "slot_mapping"), new_keys.shape[0], _dev(out, "out"),
                                             _dev(query, "query"), _dev(key_cache, "key_cache"),
                                             _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables"),
                                             _dev(context_lens, "context_lens"), float(scale), S, Hq, Hkv, D, B, MB,
                                             NB, int(max_context_len), part, _code(query), ws_ptr, ws_bytes,
                                             _stream(stream))
    _ok(rc, "paged_attention_decode_step")
    return out


def paged_attention_decode_step_fp8(new_keys, new_values, slot_mapping, out, query, key_cache, value_cache,
                                    block_tables, context_lens, scale, k_scale, v_scale, max_context_len,
                                    partition_size=None, workspace=None, stream=None, total_context_tokens=0):
    """The decode step over E4M3 pools: ``reshape_and_cache_fp8`` then ``paged_attention_decode_fp8``."""
    lib = load_library()
    S, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    MB = block_tables.shape[1] if block_tables.dim() == 2 else 1
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    part, ws_ptr, ws_bytes = _decode_workspace(S, Hq, Hkv, D, B, max_context_len, FP8_E4M3, partition_size,
                                               workspace, query.device, total_context_tokens)
    rc = lib.pkv_paged_attention_decode_step_fp8(_dev(new_keys, "new_keys"), _dev(new_values, "new_values"),
                                                 _dev(slot_mapping, "slot_mapping"), new_keys.shape[0],
                                                 _dev(out, "out"), _dev(query, "query"),
                                                 _fp8_pool(key_cache, "key_cache"),
                                                 _fp8_pool(value_cache, "value_cache"),
                                                 _dev(block_tables, "block_tables"),
                                                 _dev(context_lens, "context_lens"), float(scale), float(k_scale),
                                                 float(v_scale), S, Hq, Hkv, D, B, MB, NB, int(max_context_len), part,
                                                 _code(query), ws_ptr, ws_bytes, _stream(stream))
    _ok(rc, "paged_attention_decode_step_fp8")
    return out


def set_wait_limit_ns(limit_ns: int):
    """Limit of the kernels' main-loop waits for later launches (0 = give up at the first blocking wait; a
    test setting).  The default is one second."""
    _ok(load_library().pkv_set_wait_limit_ns(int(limit_ns)), "set_wait_limit_ns")


DEFAULT_WAIT_LIMIT_NS = 1_000_000_000


def paged_attention_prefill_chunk(out, query, key_cache, value_cache, block_tables, seq_lens, query_start_loc,
                                  max_q_len, scale, stream=None):
    """Causal chunked prefill; ``out``/``query`` packed ``[sum n_r, Hq, D]``."""
    lib = load_library()
    Tq, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    R = seq_lens.numel()
    MB = block_tables.shape[1]
    for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (query_start_loc, "query_start_loc")):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    rc = lib.pkv_paged_attention_prefill_chunk(_dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"),
                                               _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables"),
                                               _dev(seq_lens, "seq_lens"), _dev(query_start_loc, "query_start_loc"),
                                               R, Tq, int(max_q_len), float(scale), Hq, Hkv, D, B, MB, NB,
                                               _code(query), _stream(stream))
    _ok(rc, "paged_attention_prefill_chunk")
    return out


def prefill_fp8_workspace_size(num_chunks, max_blocks_per_seq, block_size, num_kv_heads, head_dim, total_q_tokens,
                               num_q_heads, dtype) -> int:
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().pkv_prefill_fp8_workspace_size(num_chunks, max_blocks_per_seq, block_size,
                                                             num_kv_heads, head_dim, int(total_q_tokens),
                                                             num_q_heads, code))


def paged_attention_prefill_chunk_fp8(out, query, key_cache, value_cache, block_tables, seq_lens, query_start_loc,
                                      max_q_len, scale, k_scale, v_scale, workspace=None, stream=None):
    """Causal chunked prefill over E4M3 pools (values ``k_scale * code``, ``v_scale * code``)."""
    lib = load_library()
    Tq, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    R = seq_lens.numel()
    MB = block_tables.shape[1]
    for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (query_start_loc, "query_start_loc")):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    need = prefill_fp8_workspace_size(R, MB, B, Hkv, D, Tq, Hq, query.dtype)
    if workspace is None or workspace.numel() * workspace.element_size() < need or workspace.data_ptr() % 256:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=query.device)
    rc = lib.pkv_paged_attention_prefill_chunk_fp8(
        _dev(out, "out"), _dev(query, "query"), _fp8_pool(key_cache, "key_cache"),
        _fp8_pool(value_cache, "value_cache"), _dev(block_tables, "block_tables"), _dev(seq_lens, "seq_lens"),
        _dev(query_start_loc, "query_start_loc"), R, Tq, int(max_q_len), float(scale), float(k_scale),
        float(v_scale), Hq, Hkv, D, B, MB, NB, _code(query), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _ok(rc, "paged_attention_prefill_chunk_fp8")
    return out


def decode_multi_partition_size(num_chunks, num_kv_heads, block_size, max_seq_len) -> int:
    rc = load_library().pkv_decode_multi_partition_size(num_chunks, num_kv_heads, block_size, max_seq_len)
    if rc < 0:
        raise PagedKVError("decode_multi_partition_size", rc)
    return rc


def paged_attention_decode_multi(out, query, key_cache, value_cache, block_tables, seq_lens, query_start_loc,
                                 max_q_len, max_seq_len, scale, partition_size=None, workspace=None, stream=None):
    """Multi-token decode (a few causal query tokens per sequence); arguments as for
    :func:`paged_attention_prefill_chunk` plus the host bound ``max_seq_len``."""
    lib = load_library()
    Tq, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    R = seq_lens.numel()
    MB = block_tables.shape[1]
    for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (query_start_loc, "query_start_loc")):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if partition_size is None:
        partition_size = decode_multi_partition_size(R, Hkv, B, max_seq_len)
    need = decode_workspace_size(Tq, Hq, D, max_seq_len, partition_size) if partition_size else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = _dev(workspace, "workspace") if (need and workspace is not None) else None
    ws_bytes = workspace.numel() * workspace.element_size() if ws_ptr else 0
    rc = lib.pkv_paged_attention_decode_multi(_dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"),
                                              _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables"),
                                              _dev(seq_lens, "seq_lens"), _dev(query_start_loc, "query_start_loc"),
                                              R, Tq, int(max_q_len), int(max_seq_len), float(scale), Hq, Hkv, D, B,
                                              MB, NB, int(partition_size), _code(query), ws_ptr, ws_bytes,
                                              _stream(stream))
    _ok(rc, "paged_attention_decode_multi")
    return out


def paged_attention_decode_multi_step(new_keys, new_values, slot_mapping, out, query, key_cache, value_cache,
                                      block_tables, seq_lens, query_start_loc, max_q_len, max_seq_len, scale,
                                      partition_size=None, workspace=None, stream=None):
    """One verification step: ``reshape_and_cache(new_keys, new_values, ..., slot_mapping)`` then
    ``paged_attention_decode_multi`` in one call (the attention launched as the append's
    programmatic dependent)."""
    lib = load_library()
    Tq, Hq, D = query.shape
    NB, B, Hkv, _ = key_cache.shape
    R = seq_lens.numel()
    MB = block_tables.shape[1]
    for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (query_start_loc, "query_start_loc")):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if partition_size is None:
        partition_size = decode_multi_partition_size(R, Hkv, B, max_seq_len)
    need = decode_workspace_size(Tq, Hq, D, max_seq_len, partition_size) if partition_size else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=query.device)
    ws_ptr = _dev(workspace, "workspace") if (need and workspace is not None) else None
    ws_bytes = workspace.numel() * workspace.element_size() if ws_ptr else 0
    rc = lib.pkv_paged_attention_decode_multi_step(
        _dev(new_keys, "new_keys"), _dev(new_values, "new_values"), _dev(slot_mapping, "slot_mapping"),
        new_keys.shape[0], _dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"),
        _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables"), _dev(seq_lens, "seq_lens"),
        _dev(query_start_loc, "query_start_loc"), R, Tq, int(max_q_len), int(max_seq_len), float(scale), Hq, Hkv, D,
        B, MB, NB, int(partition_size), _code(query), ws_ptr, ws_bytes, _stream(stream))
    _ok(rc, "paged_attention_decode_multi_step")
    return out


# ---------------------------------------------------------------- rotary positions, and pools of 8-bit rows
def rope_table(cos_sin, base=10000.0, first_position=0, scaling="none", factor=1.0, alpha=1.0, beta=32.0,
               original_max_position=1, attention_factor=1.0, stream=None):
    """Fill ``cos_sin`` (fp32 ``[positions, rotary_dim]``) with the rotary table's rows from ``first_position`` on:
    the cosines, then the sines, of ``position * theta_i``, times ``attention_factor``.  ``scaling``: "none",
    "linear", "ntk" or "by_parts" (see ``pkv_rope_table``)."""
    lib = _lib or load_library()
    if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32:
        raise ValueError("cos_sin must be a float32 [positions, rotary_dim] tensor")
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    n, rotary_dim = cos_sin.shape
    spec = RopeSpec(base, factor, alpha, beta, attention_factor, int(original_max_position), rotary_dim,
                    ROPE_SCALING[scaling])
    rc = lib.pkv_rope_table(_at(cos_sin, "cos_sin", _device(cos_sin, "cos_sin")), int(first_position), n, ctypes.byref(spec),
                            _stream(stream))
    _ok(rc, "rope_table")
    return cos_sin


# The calls below sit between a layer's kernels, where a few microseconds of host time count: what holds of correct
# arguments is tested in one expression, and only a call that fails it looks for the reason.
def _rope_refusal(query_out, query, key, value, cos_sin, positions, dev, pool_shape, slot_mapping, weights):
    T, Hq, D = query.shape
    NB, B, Hkv, Dp = pool_shape
    if Dp != D or query_out.shape != query.shape:
        return "query and query_out must be [tokens, num_q_heads, head_dim] of the pools"
    if key.shape != (T, Hkv, D) or value.shape != (T, Hkv, D):
        return "key and value must be [tokens, num_kv_heads, head_dim] of the query's tokens and the pools"
    if not query_out.dtype == query.dtype == key.dtype == value.dtype:
        return "query_out, query, key and value must have one dtype"
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        return "slot_mapping must be int64 [tokens]"
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32:
            return "cos_sin must be a float32 [positions, rotary_dim] tensor"
        if positions is None or positions.dtype != torch.int64 or positions.shape != (T,):
            return "positions must be int64 [tokens]"
    for w in weights:
        if w is not None and (w.dtype != query.dtype or w.shape != (D,)):
            return "a norm weight must be [head_dim] in the query's dtype"
    for name, t in (("query_out", query_out), ("query", query), ("key", key), ("value", value), ("cos_sin", cos_sin),
                    ("positions", positions), ("slot_mapping", slot_mapping), ("q_norm_weight", weights[0]),
                    ("k_norm_weight", weights[1])):
        if t is None or name == "positions" and cos_sin is None:
            continue
        if t.get_device() != dev:
            return f"{name} must be on the device of the call's other tensors, not on {t.device}"
        if name in ("query", "key", "value"):
            if T and (t.stride(2) != 1 or t.stride(1) != D and t.shape[1] > 1):
                return f"{name}'s heads must be contiguous within a token"
        elif not t.is_contiguous():
            return f"{name} must be contiguous"
    return None


def _rope_and_cache(fn, query_out, query, key, value, cos_sin, positions, dev, kc, vc, pool_shape, slot_mapping, interleaved,
                    qw, kw, eps, scales, stream):
    shape = query.shape
    dtype = query.dtype
    T, Hq, D = shape
    NB, B, Hkv, Dp = pool_shape
    rows = (T, Hkv, D)
    qs, qh, qe = query.stride()
    ks, kh, ke = key.stride()
    vs, vh, ve = value.stride()
    max_position = rotary_dim = 0
    table = pos = None
    fine = (Dp == D and query_out.shape == shape and key.shape == rows and value.shape == rows
            and query_out.dtype == dtype and key.dtype == dtype and value.dtype == dtype
            and slot_mapping.dtype == _INT64 and slot_mapping.shape == (T,)
            and qe == 1 and ke == 1 and ve == 1 and (qh == D or Hq == 1) and (kh == D and vh == D or Hkv == 1)
            and query_out.get_device() == dev and query.get_device() == dev and key.get_device() == dev
            and value.get_device() == dev and slot_mapping.get_device() == dev
            and query_out.is_contiguous() and slot_mapping.is_contiguous())
    if fine and cos_sin is not None:
        fine = (cos_sin.dtype == _FLOAT32 and cos_sin.dim() == 2 and cos_sin.get_device() == dev and cos_sin.is_contiguous()
                and positions is not None and positions.dtype == _INT64 and positions.shape == (T,)
                and positions.get_device() == dev and positions.is_contiguous())
    if fine and qw is not None:
        fine = qw.dtype == dtype and qw.shape == (D,) and qw.get_device() == dev and qw.is_contiguous()
    if fine and kw is not None:
        fine = kw.dtype == dtype and kw.shape == (D,) and kw.get_device() == dev and kw.is_contiguous()
    if not fine:  # (an empty batch whose rows have odd strides has no reason)
        why = _rope_refusal(query_out, query, key, value, cos_sin, positions, dev, pool_shape, slot_mapping, (qw, kw))
        if why:
            raise ValueError(why)
    if cos_sin is not None:
        max_position, rotary_dim = cos_sin.shape
        table, pos = cos_sin.data_ptr(), positions.data_ptr()
    if qw is not None:
        qw = qw.data_ptr()
    if kw is not None:
        kw = kw.data_ptr()
    if T <= 1:  # a single row's token stride says nothing
        qs, ks = Hq * D, Hkv * D
        vs = ks
    rc = fn(query_out.data_ptr(), query.data_ptr(), key.data_ptr(), value.data_ptr(), qs, ks, vs, qw, kw, float(eps), table,
            max_position, rotary_dim, 1 if interleaved else 0, pos, kc, vc, slot_mapping.data_ptr(), T, Hq, Hkv, D, B, NB,
            DTYPE_CODE.get(dtype, -1), *scales, _stream(stream))
    if rc:
        raise PagedKVError(fn.__name__[4:], rc)
    return query_out


def rope_and_cache(query_out, query, key, value, cos_sin, positions, key_cache, value_cache, slot_mapping,
                   interleaved=False, q_norm_weight=None, k_norm_weight=None, eps=1e-6, stream=None):
    """Norm of every query and key head (weights ``[D]``, or None), rotary positions (rows ``positions`` of
    ``cos_sin``, or None) and the append, in one pass: queries ``[T, Hq, D]`` to ``query_out``, keys and values
    ``[T, Hkv, D]`` to the pools' slots.  Query, key and value may be slices of one projection's output."""
    shape = key_cache.shape
    if key_cache.dtype != query.dtype or value_cache.dtype != query.dtype or value_cache.shape != shape:
        raise ValueError("the pools must have the query's dtype and one shape")
    dev = _device(query, "query")
    return _rope_and_cache((_lib or load_library()).pkv_rope_and_cache, query_out, query, key, value, cos_sin, positions,
                           dev, _at(key_cache, "key_cache", dev), _at(value_cache, "value_cache", dev), shape, slot_mapping,
                           interleaved, q_norm_weight, k_norm_weight, eps, (), stream)


def rope_and_cache_fp8(query_out, query, key, value, cos_sin, positions, key_cache, value_cache, slot_mapping, k_scale,
                       v_scale, interleaved=False, q_norm_weight=None, k_norm_weight=None, eps=1e-6, stream=None):
    """:func:`rope_and_cache` into E4M3 pools."""
    shape = key_cache.shape
    if value_cache.shape != shape or key_cache.dtype not in FP8_POOL_DTYPES or value_cache.dtype not in FP8_POOL_DTYPES:
        raise ValueError("the pools must be uint8 or float8_e4m3fn pools of E4M3 codes, of one shape")
    dev = _device(query, "query")
    return _rope_and_cache((_lib or load_library()).pkv_rope_and_cache_fp8, query_out, query, key, value, cos_sin,
                           positions, dev, _at(key_cache, "key_cache", dev), _at(value_cache, "value_cache", dev), shape,
                           slot_mapping, interleaved, q_norm_weight, k_norm_weight, eps, (float(k_scale), float(v_scale)),
                           stream)


def rope_and_cache_int8(query_out, query, key, value, cos_sin, positions, key_cache, value_cache, slot_mapping,
                        interleaved=False, q_norm_weight=None, k_norm_weight=None, eps=1e-6, stream=None):
    """:func:`rope_and_cache` into int8 pools."""
    shape, dev, k, v = _int8_pools(key_cache, value_cache)
    return _rope_and_cache((_lib or load_library()).pkv_rope_and_cache_int8, query_out, query, key, value, cos_sin,
                           positions, dev, k, v, shape, slot_mapping, interleaved, q_norm_weight, k_norm_weight, eps, (),
                           stream)


def int8_block_bytes(block_size, num_kv_heads, head_dim) -> int:
    """Bytes of one block of an int8 pool, ``block_size * num_kv_heads * (head_dim + 4)``."""
    rc = int(load_library().pkv_int8_block_bytes(block_size, num_kv_heads, head_dim))
    if rc < 0:
        raise PagedKVError("int8_block_bytes", rc)
    return rc


def int8_pool_views(pool):
    """``(codes, scales)`` of an int8 pool, uint8 ``[NB, B, Hkv, D + 4]``, as views of it: the codes uint8
    ``[NB, B, Hkv, D]`` (zero point 128) and the scales float32 ``[NB, Hkv, B]``."""
    NB, B, H, W = pool.shape
    flat = pool.view(NB, B * H * W)
    n = B * H * (W - 4)
    return flat[:, :n].view(NB, B, H, W - 4), flat.view(torch.float32)[:, n // 4:].view(NB, H, B)


def _int8_pools(key_cache, value_cache):
    """((NB, B, Hkv, D), device, key pointer, value pointer) of two int8 pools."""
    shape = key_cache.shape
    if len(shape) != 4 or shape[3] <= 4 or key_cache.dtype != _UINT8 or value_cache.dtype != _UINT8 \
            or value_cache.shape != shape:
        raise ValueError("key_cache and value_cache must be uint8 [blocks, block_size, num_kv_heads, head_dim + 4] "
                         "pools of one shape")
    dev = _device(key_cache, "key_cache")
    NB, B, H, W = shape
    return (NB, B, H, W - 4), dev, _at(key_cache, "key_cache", dev), _at(value_cache, "value_cache", dev)


def _int8_rows(fn, key, value, key_cache, value_cache, slot_mapping, stream):
    (NB, B, H, D), dev, k, v = _int8_pools(key_cache, value_cache)
    T = slot_mapping.numel()
    rows, dtype = (T, H, D), key.dtype
    if slot_mapping.dtype != _INT64:
        raise ValueError("slot_mapping must be int64")
    if key.shape != rows or value.shape != rows or value.dtype != dtype:
        raise ValueError("the rows must be [tokens, num_kv_heads, head_dim] of the pools, in one dtype")
    rc = fn(_at(key, "the key rows", dev), _at(value, "the value rows", dev), k, v, _at(slot_mapping, "slot_mapping", dev), T,
            H, D, B, NB, DTYPE_CODE.get(dtype, -1), _stream(stream))
    if rc:
        raise PagedKVError(fn.__name__[4:], rc)


def reshape_and_cache_int8(key, value, key_cache, value_cache, slot_mapping, stream=None):
    """Quantise ``key``/``value`` ``[T, Hkv, D]`` (fp32/fp16/bf16) row by row into the int8 pools' slots
    ``slot_mapping`` (int64, -1 = skip)."""
    _int8_rows((_lib or load_library()).pkv_reshape_and_cache_int8, key, value, key_cache, value_cache, slot_mapping, stream)


def read_cache_int8(key_out, value_out, key_cache, value_cache, slot_mapping, stream=None):
    """The rows of ``slot_mapping``'s slots of two int8 pools as values, into ``key_out``/``value_out``
    ``[T, Hkv, D]`` (fp32/fp16/bf16); the rows of negative slots are left as they were."""
    _int8_rows((_lib or load_library()).pkv_read_cache_int8, key_out, value_out, key_cache, value_cache, slot_mapping, stream)
    return key_out, value_out


def _int8_decode_args(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len, partition_size,
                      workspace, total_context_tokens, stream):
    """The arguments shared by the int8 decode and its step: the device, (out, query, pools, tables) pointers, the
    sizes, the partition and the workspace."""
    (NB, B, Hkv, D), dev, k, v = _int8_pools(key_cache, value_cache)
    shape, tables = query.shape, block_tables.shape
    S, Hq, Dq = shape
    dtype = query.dtype
    if Dq != D or out.shape != shape or out.dtype != dtype:
        raise ValueError("out and query must be [num_seqs, num_q_heads, head_dim] of the pools, in one dtype")
    if block_tables.dtype != _INT32 or context_lens.dtype != _INT32:
        raise ValueError("block_tables and context_lens must be int32")
    if len(tables) != 2 or tables[0] != S or context_lens.shape != (S,):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq] and context_lens [num_seqs]")
    max_context_len = int(max_context_len)
    ws_ptr, ws_bytes = None, 0
    if partition_size is None:
        partition_size = _lib.pkv_decode_partition_size(S, Hq, Hkv, D, B, max_context_len, int(total_context_tokens), INT8)
        if partition_size < 0:
            raise PagedKVError("decode_partition_size", partition_size)
    if partition_size:
        need = decode_workspace_size(S, Hq, D, max_context_len, partition_size)
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            if stream is None:
                workspace = torch.empty(need, dtype=_UINT8, device=query.device)
            else:  # from the pool of the stream that uses it: this one may hand it out again as soon as it is freed
                with torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream), device=query.device)):
                    workspace = torch.empty(need, dtype=_UINT8, device=query.device)
        if need:
            ws_ptr, ws_bytes = _at(workspace, "workspace", dev), workspace.numel() * workspace.element_size()
    return (dev, (_at(out, "out", dev), _at(query, "query", dev), k, v, _at(block_tables, "block_tables", dev),
                  _at(context_lens, "context_lens", dev)),
            (S, Hq, Hkv, D, B, tables[1], NB, max_context_len, partition_size, DTYPE_CODE.get(dtype, -1), ws_ptr, ws_bytes))


def paged_attention_decode_int8(out, query, key_cache, value_cache, block_tables, context_lens, scale,
                                max_context_len, partition_size=None, workspace=None, stream=None,
                                total_context_tokens=0):
    """Decode attention over int8 pools (uint8 ``[NB, B, Hkv, D + 4]``); ``out``/``query`` ``[S, Hq, D]`` in fp16 or
    bf16, the other arguments as for :func:`paged_attention_decode`."""
    lib = _lib or load_library()
    _, ptrs, sizes = _int8_decode_args(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len,
                                       partition_size, workspace, total_context_tokens, stream)
    rc = lib.pkv_paged_attention_decode_int8(*ptrs, float(scale), *sizes, _stream(stream))
    if rc:
        raise PagedKVError("paged_attention_decode_int8", rc)
    return out


def paged_attention_decode_step_int8(new_keys, new_values, slot_mapping, out, query, key_cache, value_cache,
                                     block_tables, context_lens, scale, max_context_len, partition_size=None,
                                     workspace=None, stream=None, total_context_tokens=0):
    """The decode step over int8 pools: ``reshape_and_cache_int8`` then ``paged_attention_decode_int8``."""
    load_library()
    dev, ptrs, sizes = _int8_decode_args(out, query, key_cache, value_cache, block_tables, context_lens,
                                         max_context_len, partition_size, workspace, total_context_tokens, stream)
    T = slot_mapping.numel()
    rows = (T, sizes[2], sizes[3])
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if new_keys.shape != rows or new_values.shape != rows or not new_keys.dtype == new_values.dtype == query.dtype:
        raise ValueError("new_keys and new_values must be [tokens, num_kv_heads, head_dim] in the query's dtype")
    rc = _lib.pkv_paged_attention_decode_step_int8(_at(new_keys, "new_keys", dev), _at(new_values, "new_values", dev),
                                                   _at(slot_mapping, "slot_mapping", dev), T, *ptrs, float(scale),
                                                   *sizes,
                                                   _stream(stream))
    _ok(rc, "paged_attention_decode_step_int8")
    return out


def paged_attention_prefill_chunk_int8(out, query, key_cache, value_cache, block_tables, seq_lens, query_start_loc,
                                       max_q_len, scale, stream=None):
    """Causal chunked prefill over int8 pools (uint8 ``[NB, B, Hkv, D + 4]``); ``out``/``query`` packed
    ``[sum n_r, Hq, D]`` in fp16 or bf16."""
    (NB, B, Hkv, D), dev, k, v = _int8_pools(key_cache, value_cache)
    Tq, Hq, Dq = query.shape
    R = seq_lens.numel()
    if Dq != D or out.shape != query.shape or out.dtype != query.dtype:
        raise ValueError("out and query must be [tokens, num_q_heads, head_dim] of the pools, in one dtype")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or query_start_loc.dtype != torch.int32:
        raise ValueError("block_tables, seq_lens and query_start_loc must be int32")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != R or query_start_loc.numel() != R + 1:
        raise ValueError("block_tables must be [chunks, max_blocks_per_seq] and query_start_loc [chunks + 1]")
    rc = (_lib or load_library()).pkv_paged_attention_prefill_chunk_int8(
        _at(out, "out", dev), _at(query, "query", dev), k, v, _at(block_tables, "block_tables", dev),
        _at(seq_lens, "seq_lens", dev), _at(query_start_loc, "query_start_loc", dev), R, Tq, int(max_q_len), float(scale), Hq, Hkv, D,
        B, tables[1], NB, _code(query), _stream(stream))
    _ok(rc, "paged_attention_prefill_chunk_int8")
    return out


def get_device_error(stream=None) -> int:
    """Read and clear the device error word (PKV_DEVERR_* bits); synchronises the stream."""
    lib = load_library()
    v = ctypes.c_uint32(0)
    _ok(lib.pkv_get_device_error(ctypes.byref(v), _stream(stream)), "get_device_error")
    return int(v.value)
