"""Python binding of the C ABI: argument marshalling only.

Every function takes CUDA tensors, checks their shapes and dtypes, and calls
the same-named entry point of ``libpa.so`` on the current (or given) stream.
All computation happens in the library's kernels; nothing here falls back to
PyTorch or the CPU.  PyTorch provides device memory and streams.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import itertools
import operator
from typing import Iterator, NamedTuple, Optional, Sequence, Tuple

import torch

from . import native
from .native import CacheDesc, PaError

DTYPE_CODE = {torch.float32: native.PA_F32, torch.float16: native.PA_F16, torch.bfloat16: native.PA_BF16}


# The current stream's raw handle without building a Stream object (a few
# microseconds per call saved; decode is called once per layer per step).
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_current_stream is not None:
        return ctypes.c_void_p(_raw_current_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check_cuda(*tensors: torch.Tensor) -> None:
    for t in tensors:
        _require(t.is_cuda, "tensors must be on a CUDA device")
        _require(t.is_contiguous(), "tensors must be contiguous")


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    _require(k_cache.dim() == 4, "a pool is [num_blocks][num_kv_heads][block_size][head_dim]")
    _require(k_cache.dtype in DTYPE_CODE, f"unsupported cache dtype {k_cache.dtype}")
    nb, hkv, bs, d = k_cache.shape
    return CacheDesc(nb, hkv, bs, d, DTYPE_CODE[k_cache.dtype])


def _raise(status: int, what: str) -> None:
    if status != native.PA_OK:
        raise PaError(status, what)


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write key/value [T][Hkv][d] into the pools at slot_mapping[t] (< 0: skip)."""
    lib = native.load()
    _check_cuda(key, value, k_cache, v_cache, slot_mapping)
    _require(k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype, "K and V pools must match")
    _require(key.dtype == k_cache.dtype and value.dtype == k_cache.dtype, "key/value dtype must match the pools")
    _require(key.dim() == 3 and key.shape == value.shape, "key/value are [num_tokens][num_kv_heads][head_dim]")
    _require(tuple(key.shape[1:]) == (k_cache.shape[1], k_cache.shape[3]), "key/value heads or head_dim mismatch")
    _require(slot_mapping.dtype == torch.int64 and slot_mapping.numel() == key.shape[0], "slot_mapping is int64 [T]")
    desc = cache_desc(k_cache)
    _raise(lib.pa_reshape_and_cache(key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                    slot_mapping.data_ptr(), key.shape[0], ctypes.byref(desc),
                                    _stream_ptr(stream)), "pa_reshape_and_cache")


class PreparedCacheWrite:
    """A pa_reshape_and_cache call whose arguments are checked and marshalled
    once: for a serving loop that writes each step's new tokens from the same
    buffers (new contents, same tensors) into the same pools.  Each call is
    then one C-ABI call.  The tensors are kept referenced; their shapes,
    dtypes, devices and storage must not change while the object is used."""

    def __init__(self, key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slot_mapping: torch.Tensor):
        self._lib = native.load()
        _check_cuda(key, value, k_cache, v_cache, slot_mapping)
        _require(k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype, "K and V pools must match")
        _require(key.dtype == k_cache.dtype and value.dtype == k_cache.dtype, "key/value dtype must match the pools")
        _require(key.dim() == 3 and key.shape == value.shape, "key/value are [num_tokens][num_kv_heads][head_dim]")
        _require(tuple(key.shape[1:]) == (k_cache.shape[1], k_cache.shape[3]), "key/value heads or head_dim mismatch")
        _require(slot_mapping.dtype == torch.int64 and slot_mapping.numel() == key.shape[0],
                 "slot_mapping is int64 [T]")
        self._desc = cache_desc(k_cache)
        self._keep = (key, value, k_cache, v_cache, slot_mapping)
        self._args = (key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                      slot_mapping.data_ptr(), key.shape[0], ctypes.byref(self._desc))

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        _raise(self._lib.pa_reshape_and_cache(*self._args, _stream_ptr(stream)), "pa_reshape_and_cache")


def decode_workspace_size(num_seqs: int, num_heads: int, max_context_len: int, partition_size: int = 0,
                          head_dim: int = 128) -> int:
    return int(native.load().pa_decode_workspace_size(num_seqs, num_heads, max_context_len, partition_size,
                                                      head_dim))


def decode(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
           context_lens: torch.Tensor, scale: float, *, num_kv_heads: Optional[int] = None,
           out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
           max_context_len: Optional[int] = None, partition_size: int = 0,
           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode attention; returns out [S][H][d].

    ``max_context_len`` is a host-side upper bound of context_lens; when None
    the table capacity (max_blocks_per_seq * block_size) is used, which needs
    no device sync but may size a larger workspace."""
    lib = native.load()
    _check_cuda(query, k_cache, v_cache, block_tables, context_lens)
    _require(query.dim() == 3, "query is [num_seqs][num_heads][head_dim]")
    s, h, d = query.shape
    desc = cache_desc(k_cache)
    _require(k_cache.shape == v_cache.shape and v_cache.dtype == k_cache.dtype, "K and V pools must match")
    _require(query.dtype == k_cache.dtype and d == desc.head_dim, "query dtype/head_dim must match the pools")
    _require(block_tables.dtype == torch.int32 and block_tables.dim() == 2 and block_tables.shape[0] == s,
             "block_tables is int32 [num_seqs][max_blocks]")
    _require(context_lens.dtype == torch.int32 and context_lens.numel() == s, "context_lens is int32 [num_seqs]")
    hkv = desc.num_kv_heads if num_kv_heads is None else num_kv_heads
    max_blocks = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = max_blocks * desc.block_size
    if out is None:
        out = torch.empty((s, h, d), dtype=out_dtype, device=query.device)
    _check_cuda(out)
    _require(out.shape == (s, h, d) and out.dtype in DTYPE_CODE, "out is [num_seqs][num_heads][head_dim]")
    if workspace is None:
        need = decode_workspace_size(s, h, max_context_len, partition_size, d)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=query.device)
    _check_cuda(workspace)
    _raise(lib.pa_decode(out.data_ptr(), DTYPE_CODE[out.dtype], query.data_ptr(), k_cache.data_ptr(),
                         v_cache.data_ptr(), ctypes.byref(desc), block_tables.data_ptr(), max_blocks,
                         context_lens.data_ptr(), s, int(max_context_len), h, hkv, float(scale),
                         int(partition_size), workspace.data_ptr(), workspace.numel(), _stream_ptr(stream)),
           "pa_decode")
    return out


class PreparedDecode:
    """A pa_decode call whose arguments are checked and marshalled once: for a
    serving loop that decodes the same buffers every step (new contents, same
    tensors), each call is then one C-ABI call with no per-call argument
    checks.  The tensors are kept referenced; their shapes, dtypes, devices and
    storage must not change while the object is used."""

    def __init__(self, query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *, out: torch.Tensor,
                 max_context_len: int, workspace: Optional[torch.Tensor] = None,
                 num_kv_heads: Optional[int] = None, partition_size: int = 0):
        self._lib = native.load()
        _check_cuda(query, k_cache, v_cache, block_tables, context_lens, out)
        _require(query.dim() == 3, "query is [num_seqs][num_heads][head_dim]")
        s, h, d = query.shape
        self._desc = cache_desc(k_cache)
        _require(k_cache.shape == v_cache.shape and v_cache.dtype == k_cache.dtype, "K and V pools must match")
        _require(query.dtype == k_cache.dtype and d == self._desc.head_dim, "query dtype/head_dim must match the pools")
        _require(block_tables.dtype == torch.int32 and block_tables.dim() == 2 and block_tables.shape[0] == s,
                 "block_tables is int32 [num_seqs][max_blocks]")
        _require(context_lens.dtype == torch.int32 and context_lens.numel() == s, "context_lens is int32 [num_seqs]")
        _require(out.shape == (s, h, d) and out.dtype in DTYPE_CODE, "out is [num_seqs][num_heads][head_dim]")
        hkv = self._desc.num_kv_heads if num_kv_heads is None else num_kv_heads
        if workspace is None:
            need = decode_workspace_size(s, h, max_context_len, partition_size, d)
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=query.device)
        _check_cuda(workspace)
        self._keep = (query, k_cache, v_cache, block_tables, context_lens, out, workspace)
        self.out = out
        self._args = (out.data_ptr(), DTYPE_CODE[out.dtype], query.data_ptr(), k_cache.data_ptr(),
                      v_cache.data_ptr(), ctypes.byref(self._desc), block_tables.data_ptr(), block_tables.shape[1],
                      context_lens.data_ptr(), s, int(max_context_len), h, hkv, ctypes.c_float(float(scale)),
                      int(partition_size), workspace.data_ptr(), workspace.numel())

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        _raise(self._lib.pa_decode(*self._args, _stream_ptr(stream)), "pa_decode")
        return self.out


def prefill(query: torch.Tensor, query_start_loc: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
            block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, max_query_len: int, *,
            num_kv_heads: Optional[int] = None, out: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.float32, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Prompt-phase attention of new tokens over a cached prefix; returns
    out [T][H][d].

    Sequence s owns query rows query_start_loc[s] .. query_start_loc[s+1]-1,
    the last n_s of its context_lens[s] cached tokens; row i attends to
    positions 0 .. context_lens[s] - n_s + i.  ``max_query_len`` is a host-side
    upper bound of every n_s."""
    lib = native.load()
    _check_cuda(query, query_start_loc, k_cache, v_cache, block_tables, context_lens)
    _require(query.dim() == 3, "query is [num_tokens][num_heads][head_dim]")
    t, h, d = query.shape
    desc = cache_desc(k_cache)
    _require(k_cache.shape == v_cache.shape and v_cache.dtype == k_cache.dtype, "K and V pools must match")
    _require(query.dtype == k_cache.dtype and d == desc.head_dim, "query dtype/head_dim must match the pools")
    _require(block_tables.dtype == torch.int32 and block_tables.dim() == 2, "block_tables is int32 [S][max_blocks]")
    s = block_tables.shape[0]
    _require(context_lens.dtype == torch.int32 and context_lens.numel() == s, "context_lens is int32 [num_seqs]")
    _require(query_start_loc.dtype == torch.int32 and query_start_loc.numel() == s + 1,
             "query_start_loc is int32 [num_seqs + 1]")
    hkv = desc.num_kv_heads if num_kv_heads is None else num_kv_heads
    if out is None:
        out = torch.empty((t, h, d), dtype=out_dtype, device=query.device)
    _check_cuda(out)
    _require(out.shape == (t, h, d) and out.dtype in DTYPE_CODE, "out is [num_tokens][num_heads][head_dim]")
    _raise(lib.pa_prefill(out.data_ptr(), DTYPE_CODE[out.dtype], query.data_ptr(), query_start_loc.data_ptr(), t,
                          int(max_query_len), k_cache.data_ptr(), v_cache.data_ptr(), ctypes.byref(desc),
                          block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), s, h, hkv,
                          float(scale), _stream_ptr(stream)), "pa_prefill")
    return out


def _require_here(*tensors: torch.Tensor) -> None:
    """The library works on the current device: tensors of another one are refused."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:  # -1 for a CPU tensor
            raise ValueError("tensors must be on the current CUDA device")


def _empty(shape: Sequence[int], dtype: torch.dtype, device: torch.device,
           stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """An output that the call makes, from the memory of the stream that it is written on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements from one token's row of heads to the next; the heads of a token are contiguous."""
    tokens, heads, d = t.shape
    by_token, by_head, by_elem = t.stride()
    if tokens > 1 and by_elem == 1 and by_head == d and by_token >= heads * d:
        return by_token
    if (by_elem != 1 and d > 1) or (by_head != d and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if tokens <= 1:
        return heads * d
    if by_token < heads * d:
        raise ValueError(f"{name}: rows of tokens must not overlap")
    return by_token


def rotary_and_cache(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                     cos_sin: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, *, interleaved: bool = False, query_out: Optional[torch.Tensor] = None,
                     key_out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rotate the first rotary_dim elements of every query and key head by the
    angles of positions[t], write the keys and values to slot_mapping[t] (< 0:
    not cached) and return the rotated query [T][H][d]; the rotated keys too go
    to ``key_out`` where that is given.  ``cos_sin`` is float32
    [positions][rotary_dim], cosines then sines.  A token at a negative position
    is padding: nothing of it is written (a new query_out is undefined there).
    The rows may be slices of a fused projection's rows, and query_out / key_out
    the query / key themselves."""
    lib = native.load()
    _require(query.dim() == 3 and key.dim() == 3, "rows are [tokens][heads][head_dim]")
    t, h, d = query.shape
    desc = cache_desc(k_cache)
    dtype = k_cache.dtype
    _require(k_cache.shape == v_cache.shape and v_cache.dtype is dtype and k_cache.is_contiguous()
             and v_cache.is_contiguous(), "K and V pools must match and be contiguous")
    _require(key.shape == (t, desc.num_kv_heads, d) and value.shape == key.shape and d == desc.head_dim,
             "key/value are [num_tokens][num_kv_heads][head_dim] of the pools")
    _require(query.dtype is dtype and key.dtype is dtype and value.dtype is dtype,
             "query, key and value share the pools' dtype")
    _require(positions.dtype is torch.int32 and positions.shape == (t,) and positions.is_contiguous()
             and slot_mapping.dtype is torch.int64 and slot_mapping.shape == (t,) and slot_mapping.is_contiguous(),
             "positions is int32 [T], slot_mapping int64 [T]")
    _require(cos_sin.dtype is torch.float32 and cos_sin.dim() == 2 and cos_sin.is_contiguous(),
             "cos_sin is float32 [positions][rotary_dim]")
    if query_out is None:
        query_out = _empty((t, h, d), dtype, query.device, stream)
    _require(query_out.shape == query.shape and query_out.dtype is dtype, "query_out is like query")
    _require_here(query, key, value, positions, cos_sin, slot_mapping, k_cache, v_cache, query_out)
    key_ptr, key_stride = None, 0
    if key_out is not None:
        _require(key_out.shape == key.shape and key_out.dtype == key.dtype, "key_out is like key")
        _require_here(key_out)
        key_ptr, key_stride = key_out.data_ptr(), _token_stride(key_out, "key_out")
    _raise(lib.pa_rotary_and_cache(query_out.data_ptr(), _token_stride(query_out, "query_out"), key_ptr, key_stride,
                                   query.data_ptr(), _token_stride(query, "query"), key.data_ptr(),
                                   _token_stride(key, "key"), value.data_ptr(), _token_stride(value, "value"),
                                   positions.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1],
                                   1 if interleaved else 0, k_cache.data_ptr(), v_cache.data_ptr(),
                                   slot_mapping.data_ptr(), t, h, ctypes.byref(desc), _stream_ptr(stream)),
           "pa_rotary_and_cache")
    return query_out


class StepPlan(NamedTuple):
    """What plan_step makes (device tensors)."""
    context_lens: torch.Tensor      # int32 [S] after the step
    free_state: torch.Tensor        # int32 [2] first free entry of the ring, free blocks
    query_start_loc: torch.Tensor   # int32 [S + 1]
    slot_mapping: torch.Tensor      # int64 [max_tokens], -1 behind the last token
    positions: torch.Tensor         # int32 [max_tokens], -1 behind the last token


def plan_step(new_lens: torch.Tensor, context_lens: torch.Tensor, free_ring: torch.Tensor, free_state: torch.Tensor,
              block_tables: torch.Tensor, block_size: int, max_tokens: int, num_blocks: int, *,
              out: Optional[StepPlan] = None, stream: Optional[torch.cuda.Stream] = None) -> StepPlan:
    """Plan a step on the GPU: take blocks for the new_lens[s] tokens that each
    sequence gains (-1: finished, its blocks go back; 0: idle), write them into
    block_tables, and return the lengths after the step, the free blocks left,
    the start rows and every new token's slot and position.

    ``free_ring`` int32 holds the free block ids from entry free_state[0] on,
    free_state[1] of them, wrapping around.  ``out`` may reuse buffers, the
    inputs context_lens and free_state among them (a captured step that advances
    in place).  A step that does not fit is refused whole (get_device_error)."""
    lib = native.load()
    s = new_lens.numel()
    i32 = torch.int32
    _require(max_tokens >= 0, "max_tokens must not be negative")
    _require(new_lens.dtype is i32 and context_lens.dtype is i32 and free_state.dtype is i32
             and free_ring.dtype is i32 and block_tables.dtype is i32, "lengths, blocks and tables are int32")
    _require(new_lens.shape == (s,) and context_lens.shape == (s,) and free_state.shape == (2,)
             and free_ring.dim() == 1 and block_tables.dim() == 2 and block_tables.shape[0] == s,
             "new_lens and context_lens are [num_seqs], free_state [2], free_ring [ring_size], block_tables "
             "[num_seqs][max_blocks]")
    _require(new_lens.is_contiguous() and context_lens.is_contiguous() and free_state.is_contiguous()
             and free_ring.is_contiguous() and block_tables.is_contiguous(), "tensors must be contiguous")
    if out is None:
        dev, empty = new_lens.device, torch.empty
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            out = StepPlan(empty((s,), dtype=i32, device=dev), empty((2,), dtype=i32, device=dev),
                           empty((s + 1,), dtype=i32, device=dev), empty((max_tokens,), dtype=torch.int64, device=dev),
                           empty((max_tokens,), dtype=i32, device=dev))
    else:
        for t, n, dt in zip(out, (s, 2, s + 1, max_tokens, max_tokens),
                            (torch.int32, torch.int32, torch.int32, torch.int64, torch.int32)):
            _require(t.dtype == dt and t.dim() == 1 and t.numel() == n and t.is_contiguous(),
                     "out is (context_lens [S], free_state [2], query_start_loc [S + 1], slot_mapping int64 [T], "
                     "positions [T])")
    _require_here(new_lens, context_lens, free_ring, free_state, block_tables, *out)
    _raise(lib.pa_plan_step(new_lens.data_ptr(), context_lens.data_ptr(), out[0].data_ptr(), s, free_ring.data_ptr(),
                            free_ring.numel(), free_state.data_ptr(), out[1].data_ptr(), int(num_blocks),
                            int(block_size), block_tables.data_ptr(), block_tables.shape[1], out[2].data_ptr(),
                            out[3].data_ptr(), out[4].data_ptr(), int(max_tokens), _stream_ptr(stream)),
           "pa_plan_step")
    return out


def prompt_attention_workspace_size(num_seqs: int, num_tokens: int, num_heads: int, num_kv_heads: int) -> int:
    return int(native.load().pa_prompt_attention_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads))


def prompt_attention(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, query_start_loc: torch.Tensor,
                     scale: float, *, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention of whole packed prompts over themselves; returns
    out [T][H][d] in the inputs' type (f16 or bf16).

    Sequence s owns rows query_start_loc[s] .. query_start_loc[s+1]-1 of query
    [T][H][d], key and value [T][Hkv][d]; its token i attends to its tokens
    0 .. i.  The rows may be slices of a fused projection's rows (a token's
    heads contiguous, the token stride a multiple of d).  Rows outside every
    sequence are neither used nor written: a given ``out`` keeps them."""
    lib = native.load()
    _require(query.dim() == 3 and key.dim() == 3, "query is [num_tokens][num_heads][head_dim], key its KV heads")
    t, h, d = query.shape
    hkv = key.shape[1]
    dtype = query.dtype
    _require(key.shape == (t, hkv, d) and value.shape == key.shape,
             "key/value are [num_tokens][num_kv_heads][head_dim]")
    _require(dtype in DTYPE_CODE and key.dtype is dtype and value.dtype is dtype,
             "query, key and value share one dtype")
    _require(query_start_loc.dtype is torch.int32 and query_start_loc.dim() == 1 and query_start_loc.numel() > 0
             and query_start_loc.is_contiguous(), "query_start_loc is int32 [num_seqs + 1]")
    if out is None:
        out = _empty((t, h, d), dtype, query.device, stream)
    _require(out.shape == query.shape and out.dtype is dtype and out.is_contiguous(),
             "out is contiguous [num_tokens][num_heads][head_dim] of the inputs' dtype")
    if workspace is None:
        need = lib.pa_prompt_attention_workspace_size(query_start_loc.numel() - 1, t, h, hkv)
        workspace = _empty((max(need, 256),), torch.uint8, query.device, stream)
    _require(workspace.dtype is torch.uint8 and workspace.is_contiguous(), "workspace is bytes")
    _require_here(query, key, value, query_start_loc, out, workspace)
    _raise(lib.pa_prompt_attention(out.data_ptr(), query.data_ptr(), _token_stride(query, "query"), key.data_ptr(),
                                   _token_stride(key, "key"), value.data_ptr(), _token_stride(value, "value"),
                                   query_start_loc.data_ptr(), query_start_loc.numel() - 1, t, h, hkv, d,
                                   DTYPE_CODE[dtype], float(scale), workspace.data_ptr(), workspace.numel(),
                                   _stream_ptr(stream)),
           "pa_prompt_attention")
    return out


# The calls of drafted trees come once per layer or step, next to kernels of a few
# microseconds: their checks are single expressions, and the device is asked for once.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_here(stream: Optional[torch.cuda.Stream], device: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_current_stream is not None:
        return _raw_current_stream(device)
    return torch.cuda.current_stream().cuda_stream


def _refuse_elsewhere(cond: bool) -> None:
    if not cond:
        raise ValueError("tensors must be on the current CUDA device")


class TreePlan(NamedTuple):
    """What plan_tree makes (device tensors)."""
    positions: torch.Tensor  # int32 [T], -1 for rows of no sequence
    tree_mask: torch.Tensor  # int64 [T][ceil(max_nodes / 64)]: bit j of a row, node j of its sequence


def plan_tree(parents: torch.Tensor, query_start_loc: torch.Tensor, context_lens: torch.Tensor, max_nodes: int, *,
              out: Optional[TreePlan] = None, stream: Optional[torch.cuda.Stream] = None) -> TreePlan:
    """Positions and ancestor masks of drafted trees.

    Sequence s owns rows query_start_loc[s] .. query_start_loc[s+1]-1, the last
    ones of its context_lens[s] cached tokens (plan_step with new_lens[s] nodes);
    ``parents`` int32 [T] holds each node's parent as an index in its sequence,
    less than its own (-1: none).  ``max_nodes`` is a host-side upper bound of the
    nodes of a sequence.  Positions are the depths behind the cached tokens; they
    and the slots of plan_step go to rotary_and_cache, the masks to tree_attention."""
    i32 = torch.int32
    _require(max_nodes >= 1, "max_nodes must be positive")
    words = (max_nodes + 63) // 64
    _require(parents.dtype is i32 and parents.dim() == 1 and parents.is_contiguous(), "parents is int32 [T]")
    _require(context_lens.dtype is i32 and context_lens.dim() == 1 and context_lens.is_contiguous(),
             "context_lens is int32 [num_seqs]")
    t, s = parents.numel(), context_lens.numel()
    _require(query_start_loc.dtype is i32 and query_start_loc.dim() == 1 and query_start_loc.numel() == s + 1
             and query_start_loc.is_contiguous(), "query_start_loc is int32 [num_seqs + 1]")
    if out is None:
        positions = _empty((t,), i32, parents.device, stream)
        mask = _empty((t, words), torch.int64, parents.device, stream)
        out = TreePlan(positions, mask)
    else:
        positions, mask = out
        _require(positions.dtype is i32 and positions.shape == (t,) and positions.is_contiguous()
                 and mask.dtype is torch.int64 and mask.shape == (t, words) and mask.is_contiguous(),
                 "out is (positions int32 [T], tree_mask int64 [T][words])")
    dev = _current_device()
    _refuse_elsewhere(parents.get_device() == query_start_loc.get_device() == context_lens.get_device()
                      == positions.get_device() == mask.get_device() == dev)
    status = native.load().pa_plan_tree(parents.data_ptr(), query_start_loc.data_ptr(), context_lens.data_ptr(), s, t,
                                        positions.data_ptr(), mask.data_ptr(), words, _stream_here(stream, dev))
    if status:
        raise PaError(status, "pa_plan_tree")
    return out


def tree_attention_workspace_size(num_tokens: int, mask_words: int, num_heads: int, num_kv_heads: int,
                                  head_dim: int) -> int:
    return int(native.load().pa_tree_attention_workspace_size(num_tokens, mask_words, num_heads, num_kv_heads,
                                                              head_dim))


def tree_attention(query: torch.Tensor, query_start_loc: torch.Tensor, tree_mask: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   context_lens: torch.Tensor, scale: float, *, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the nodes of drafted trees over the paged cache; returns
    out [T][H][d] in the pools' type (f16 or bf16).

    Sequence s owns rows query_start_loc[s] .. query_start_loc[s+1]-1 of query
    [T][H][d], the last n_s of its context_lens[s] cached tokens, their K/V in the
    pools.  A row attends to every position before its tree and to the nodes whose
    bit of its row of ``tree_mask`` (plan_tree's, or any other mask; int64
    [T][words]) is set; to nothing: 0.  The query may be a slice of a fused
    projection's rows.  Rows outside every sequence are not written."""
    _require(query.dim() == 3, "query is [num_tokens][num_heads][head_dim]")
    t, h, d = query.shape
    dtype, i32 = k_cache.dtype, torch.int32
    desc = cache_desc(k_cache)
    _require(v_cache.shape == k_cache.shape and v_cache.dtype is dtype and k_cache.is_contiguous()
             and v_cache.is_contiguous(), "K and V pools must match and be contiguous")
    _require(query.dtype is dtype and d == desc.head_dim, "query dtype/head_dim must match the pools")
    _require(block_tables.dtype is i32 and block_tables.dim() == 2 and block_tables.is_contiguous(),
             "block_tables is int32 [num_seqs][max_blocks]")
    s, max_blocks = block_tables.shape
    _require(context_lens.dtype is i32 and context_lens.dim() == 1 and context_lens.numel() == s
             and context_lens.is_contiguous(), "context_lens is int32 [num_seqs]")
    _require(query_start_loc.dtype is i32 and query_start_loc.dim() == 1 and query_start_loc.numel() == s + 1
             and query_start_loc.is_contiguous(), "query_start_loc is int32 [num_seqs + 1]")
    _require(tree_mask.dtype is torch.int64 and tree_mask.dim() == 2 and tree_mask.is_contiguous()
             and tree_mask.shape[0] == t, "tree_mask is int64 [num_tokens][words]")
    words, hkv = tree_mask.shape[1], desc.num_kv_heads
    if out is None:
        out = _empty((t, h, d), dtype, query.device, stream)
    else:
        _require(out.shape == query.shape and out.dtype is dtype and out.is_contiguous(),
                 "out is contiguous [num_tokens][num_heads][head_dim] of the pools' dtype")
    lib = native.load()
    if workspace is None:
        size = max(lib.pa_tree_attention_workspace_size(t, words, h, hkv, d), 256)
        workspace = _empty((size,), torch.uint8, query.device, stream)
    else:
        size = workspace.numel()
        _require(workspace.dtype is torch.uint8 and workspace.is_contiguous(), "workspace is bytes")
    dev = _current_device()
    _refuse_elsewhere(query.get_device() == query_start_loc.get_device() == tree_mask.get_device()
                      == k_cache.get_device() == v_cache.get_device() == block_tables.get_device()
                      == context_lens.get_device() == out.get_device() == workspace.get_device() == dev)
    status = lib.pa_tree_attention(out.data_ptr(), query.data_ptr(), _token_stride(query, "query"),
                                   query_start_loc.data_ptr(), t, tree_mask.data_ptr(), words, k_cache.data_ptr(),
                                   v_cache.data_ptr(), desc, block_tables.data_ptr(), max_blocks,
                                   context_lens.data_ptr(), s, h, hkv, float(scale), workspace.data_ptr(), size,
                                   _stream_here(stream, dev))
    if status:
        raise PaError(status, "pa_tree_attention")
    return out


class TreeVerdict(NamedTuple):
    """What verify_tree makes (device tensors)."""
    accepted_lens: torch.Tensor  # int32 [S] accepted nodes, node 0 among them
    path: torch.Tensor           # int32 [T] each sequence's accepted nodes from its first row on, then -1
    next_tokens: torch.Tensor    # int32 [S]


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements from one row of probabilities to the next; a row is contiguous."""
    rows, width = t.shape
    _require(width == 1 or t.stride(1) == 1, f"{name}: a row must be contiguous")
    stride = t.stride(0) if rows > 1 else width
    _require(stride >= width, f"{name}: rows must not overlap")
    return stride


def verify_tree(tokens: torch.Tensor, parents: torch.Tensor, query_start_loc: torch.Tensor,
                target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor], accept_uniforms: torch.Tensor,
                sample_uniforms: torch.Tensor, *, out: Optional[TreeVerdict] = None,
                stream: Optional[torch.cuda.Stream] = None) -> TreeVerdict:
    """Which nodes of drafted trees the target accepts, and the token that follows.

    ``target_probs`` and ``draft_probs`` [T][vocab] (f32, f16 or bf16; rows may be
    padded): row i is the distribution of the token after node i, the draft's the
    one that i's children were drawn from independently; None for tokens that were
    not drawn (a lookup's).  ``accept_uniforms`` [T] and ``sample_uniforms`` [S]
    float32 in [0, 1).  Children are tried in order, a refused one leaves the
    residual distribution to the next, and the last token is drawn from what is
    left: the accepted tokens are distributed as the target's own."""
    i32, f32 = torch.int32, torch.float32
    t = tokens.numel()
    _require(tokens.dtype is i32 and tokens.dim() == 1 and tokens.is_contiguous() and parents.dtype is i32
             and parents.dim() == 1 and parents.numel() == t and parents.is_contiguous(),
             "tokens and parents are int32 [T]")
    _require(query_start_loc.dtype is i32 and query_start_loc.dim() == 1 and query_start_loc.is_contiguous()
             and query_start_loc.numel() > 0, "query_start_loc is int32 [num_seqs + 1]")
    s = query_start_loc.numel() - 1
    dtype = target_probs.dtype
    _require(target_probs.dim() == 2 and target_probs.shape[0] == t and dtype in DTYPE_CODE,
             "target_probs is [T][vocab] of f32, f16 or bf16")
    _require(accept_uniforms.dtype is f32 and accept_uniforms.dim() == 1 and accept_uniforms.numel() == t
             and accept_uniforms.is_contiguous() and sample_uniforms.dtype is f32 and sample_uniforms.dim() == 1
             and sample_uniforms.numel() == s and sample_uniforms.is_contiguous(),
             "accept_uniforms is float32 [T], sample_uniforms float32 [num_seqs]")
    if out is None:
        dev = tokens.device
        out = TreeVerdict(_empty((s,), i32, dev, stream), _empty((t,), i32, dev, stream),
                          _empty((s,), i32, dev, stream))
        accepted, path, following = out
    else:
        accepted, path, following = out
        for x, n in ((accepted, s), (path, t), (following, s)):
            _require(x.dtype is i32 and x.shape == (n,) and x.is_contiguous(),
                     "out is (accepted_lens int32 [S], path int32 [T], next_tokens int32 [S])")
    dev = _current_device()
    _refuse_elsewhere(tokens.get_device() == parents.get_device() == query_start_loc.get_device()
                      == target_probs.get_device() == accept_uniforms.get_device() == sample_uniforms.get_device()
                      == accepted.get_device() == path.get_device() == following.get_device() == dev)
    draft_ptr, draft_stride = None, 0
    if draft_probs is not None:
        _require(draft_probs.shape == target_probs.shape and draft_probs.dtype is dtype,
                 "draft_probs is like target_probs")
        _refuse_elsewhere(draft_probs.get_device() == dev)
        draft_ptr, draft_stride = draft_probs.data_ptr(), _row_stride(draft_probs, "draft_probs")
    status = native.load().pa_verify_tree(tokens.data_ptr(), parents.data_ptr(), query_start_loc.data_ptr(), s, t,
                                          target_probs.data_ptr(), _row_stride(target_probs, "target_probs"), draft_ptr,
                                          draft_stride, target_probs.shape[1], DTYPE_CODE[dtype],
                                          accept_uniforms.data_ptr(), sample_uniforms.data_ptr(), accepted.data_ptr(),
                                          path.data_ptr(), following.data_ptr(), _stream_here(stream, dev))
    if status:
        raise PaError(status, "pa_verify_tree")
    return out


_SHAPE, _DTYPE = operator.attrgetter("shape"), operator.attrgetter("dtype")


class TreeCommit(NamedTuple):
    """What commit_tree makes (device tensors)."""
    context_lens: torch.Tensor          # int32 [S] after the step
    free_state: Optional[torch.Tensor]  # int32 [2]; None without a ring


def commit_tree(k_caches: Sequence[torch.Tensor], v_caches: Sequence[torch.Tensor], query_start_loc: torch.Tensor,
                path: torch.Tensor, accepted_lens: torch.Tensor, context_lens: torch.Tensor,
                block_tables: torch.Tensor, *, free_ring: Optional[torch.Tensor] = None,
                free_state: Optional[torch.Tensor] = None, out: Optional[TreeCommit] = None,
                stream: Optional[torch.cuda.Stream] = None) -> TreeCommit:
    """Keep the accepted paths of drafted trees: move their K/V rows together in
    every layer's pools, cut the lengths to them, and give the blocks behind back to
    plan_step's ring (``free_ring`` and ``free_state``; None: the host's manager
    keeps the blocks).  A pool that several layers share is given once.  ``path`` and ``accepted_lens`` are verify_tree's.  ``out`` may
    reuse buffers, context_lens and free_state among them."""
    i32, n = torch.int32, len(k_caches)
    _require(n == len(v_caches) and n > 0, "one K and one V pool per layer")
    pools = [*k_caches, *v_caches]
    desc, first = cache_desc(pools[0]), pools[0]
    shape, dtype = first.shape, first.dtype
    # 64 pools and more: one pass of a C loop for each property
    _require(all(map(operator.eq, map(_SHAPE, pools), itertools.repeat(shape)))
             and all(map(operator.is_, map(_DTYPE, pools), itertools.repeat(dtype)))
             and all(map(torch.Tensor.is_contiguous, pools)), "all pools must match and be contiguous")
    s, t = context_lens.numel(), path.numel()
    _require(context_lens.dtype is i32 and context_lens.dim() == 1 and context_lens.is_contiguous()
             and accepted_lens.dtype is i32 and accepted_lens.dim() == 1 and accepted_lens.numel() == s
             and accepted_lens.is_contiguous(), "context_lens and accepted_lens are int32 [num_seqs]")
    _require(path.dtype is i32 and path.dim() == 1 and path.is_contiguous(), "path is int32 [T]")
    _require(query_start_loc.dtype is i32 and query_start_loc.dim() == 1 and query_start_loc.numel() == s + 1
             and query_start_loc.is_contiguous(), "query_start_loc is int32 [num_seqs + 1]")
    _require(block_tables.dtype is i32 and block_tables.dim() == 2 and block_tables.is_contiguous()
             and block_tables.shape[0] == s, "block_tables is int32 [num_seqs][max_blocks]")
    _require((free_ring is None) == (free_state is None), "free_ring and free_state come together")
    if out is None:
        where = context_lens.device
        out = TreeCommit(_empty((s,), i32, where, stream),
                         None if free_ring is None else _empty((2,), i32, where, stream))
    lens, state = out
    _require(lens.dtype is i32 and lens.dim() == 1 and lens.numel() == s and lens.is_contiguous(),
             "out is (context_lens int32 [S], free_state int32 [2] or None)")
    dev = _current_device()
    ring_ptr, ring_size, state_ptr, state_out = None, 0, None, None
    if free_ring is not None:
        _require(free_ring.dtype is i32 and free_ring.dim() == 1 and free_ring.is_contiguous()
                 and free_state.dtype is i32 and free_state.shape == (2,) and free_state.is_contiguous(),
                 "free_ring is int32 [ring_size], free_state int32 [2]")
        _require(state is not None and state.dtype is i32 and state.shape == (2,) and state.is_contiguous(),
                 "out is (context_lens int32 [S], free_state int32 [2])")
        _refuse_elsewhere(free_ring.get_device() == free_state.get_device() == state.get_device() == dev)
        ring_ptr, ring_size, state_ptr, state_out = (free_ring.data_ptr(), free_ring.numel(), free_state.data_ptr(),
                                                     state.data_ptr())
    _refuse_elsewhere(query_start_loc.get_device() == path.get_device() == accepted_lens.get_device()
                      == context_lens.get_device() == block_tables.get_device() == lens.get_device() == dev
                      and all(map(operator.eq, map(torch.Tensor.get_device, pools), itertools.repeat(dev))))
    ptrs = array.array("Q", map(torch.Tensor.data_ptr, pools))  # host array of both kinds of pools
    at = ptrs.buffer_info()[0]
    status = native.load().pa_commit_tree(at, at + 8 * n, n, desc, query_start_loc.data_ptr(), s, t, path.data_ptr(),
                                          accepted_lens.data_ptr(), context_lens.data_ptr(), lens.data_ptr(),
                                          block_tables.data_ptr(), block_tables.shape[1], ring_ptr, ring_size,
                                          state_ptr, state_out, _stream_here(stream, dev))
    if status:
        raise PaError(status, "pa_commit_tree")
    return out


def copy_blocks(k_caches: Sequence[torch.Tensor], v_caches: Sequence[torch.Tensor], src_dst_pairs: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy-on-write: copy K and V block pairs[i][0] -> pairs[i][1] in every layer."""
    lib = native.load()
    _require(len(k_caches) == len(v_caches) and len(k_caches) > 0, "one K and one V pool per layer")
    _check_cuda(*k_caches, *v_caches, src_dst_pairs)
    _require(src_dst_pairs.dtype == torch.int64 and src_dst_pairs.dim() == 2 and src_dst_pairs.shape[1] == 2,
             "src_dst_pairs is int64 [n][2]")
    desc = cache_desc(k_caches[0])
    for p in list(k_caches) + list(v_caches):
        _require(p.shape == k_caches[0].shape and p.dtype == k_caches[0].dtype, "all pools must match")
    n = len(k_caches)
    kp = (ctypes.c_void_p * n)(*[p.data_ptr() for p in k_caches])
    vp = (ctypes.c_void_p * n)(*[p.data_ptr() for p in v_caches])
    _raise(lib.pa_copy_blocks(kp, vp, n, src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], ctypes.byref(desc),
                              _stream_ptr(stream)), "pa_copy_blocks")


def swap_blocks(src_k: Sequence[torch.Tensor], src_v: Sequence[torch.Tensor], dst_k: Sequence[torch.Tensor],
                dst_v: Sequence[torch.Tensor], src_dst_pairs: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy blocks pairs[i][0] of the source pools to blocks pairs[i][1] of
    the destination pools, every layer, one launch: GPU <-> page-locked host
    (swap-out / swap-in).  Host pools must be pinned (``pin_memory()``)."""
    lib = native.load()
    n = len(src_k)
    _require(n > 0 and len(src_v) == n and len(dst_k) == n and len(dst_v) == n, "one pool per layer on each side")
    pools = list(src_k) + list(src_v) + list(dst_k) + list(dst_v)
    for p in pools:
        _require(p.is_contiguous(), "pools must be contiguous")
        _require(p.is_cuda or p.is_pinned(), "host pools must be in page-locked (pinned) memory")
        _require(p.dtype == src_k[0].dtype and tuple(p.shape[1:]) == tuple(src_k[0].shape[1:]),
                 "pools must share dtype and block shape")
    _require(src_dst_pairs.dtype == torch.int64 and src_dst_pairs.dim() == 2 and src_dst_pairs.shape[1] == 2,
             "src_dst_pairs is int64 [n][2]")
    _require(src_dst_pairs.is_cuda or src_dst_pairs.is_pinned(), "pairs must be on the GPU or pinned")
    _require(src_dst_pairs.is_contiguous(), "pairs must be contiguous")
    desc = cache_desc(src_k[0])
    arr = lambda ts: (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])
    _raise(lib.pa_swap_blocks(arr(src_k), arr(src_v), src_k[0].shape[0], arr(dst_k), arr(dst_v), dst_k[0].shape[0],
                              n, src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], ctypes.byref(desc),
                              _stream_ptr(stream)), "pa_swap_blocks")


def get_device_error(stream: Optional[torch.cuda.Stream] = None) -> Tuple[int, int]:
    """(status, PA_DEVERR_* mask); synchronises the stream and clears the word."""
    code = ctypes.c_int32(0)
    status = native.load().pa_get_device_error(_stream_ptr(stream), ctypes.byref(code))
    return int(status), int(code.value)


def decode_noalloc(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   context_lens: torch.Tensor, scale: float, *, out: torch.Tensor, max_context_len: int,
                   num_kv_heads: Optional[int] = None, partition_size: int = 0,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Decode attention through pa_decode_noalloc: for callers that must not
    allocate device memory.  ``out`` must be given (nothing is allocated
    here either); the workspace is the library's fixed array, so the batch must
    fit in it (PA_ERR_WORKSPACE otherwise) and calls that overlap on the GPU
    must be serialised by the caller."""
    lib = native.load()
    _check_cuda(query, k_cache, v_cache, block_tables, context_lens, out)
    s, h, d = query.shape
    desc = cache_desc(k_cache)
    _require(query.dtype == k_cache.dtype and d == desc.head_dim, "query dtype/head_dim must match the pools")
    _require(out.shape == (s, h, d) and out.dtype in DTYPE_CODE, "out is [num_seqs][num_heads][head_dim]")
    hkv = desc.num_kv_heads if num_kv_heads is None else num_kv_heads
    _raise(lib.pa_decode_noalloc(out.data_ptr(), DTYPE_CODE[out.dtype], query.data_ptr(), k_cache.data_ptr(),
                                 v_cache.data_ptr(), ctypes.byref(desc), block_tables.data_ptr(),
                                 block_tables.shape[1], context_lens.data_ptr(), s, int(max_context_len), h, hkv,
                                 float(scale), int(partition_size), _stream_ptr(stream)), "pa_decode_noalloc")
    return out


OPTIONS = {"debug_checks": native.OPT_DEBUG_CHECKS, "decode_kernel_simt": native.OPT_DECODE_KERNEL,
           "drop_first_fill": native.OPT_DROP_FIRST_FILL}


def set_option(name: str, value: bool) -> bool:
    """Set a process-wide library option (pa_set_option); returns the previous
    value.  ``debug_checks``: checked mode (precondition pre-passes that report
    violations through the error word); ``decode_kernel_simt``: CUDA-core
    decode for 16-bit pools; ``drop_first_fill``: test hook of the bounded
    waits."""
    prev = native.load().pa_set_option(OPTIONS[name], 1 if value else 0)
    if prev < 0:
        raise PaError(prev, "pa_set_option")
    return bool(prev)


def get_option(name: str) -> bool:
    value = native.load().pa_get_option(OPTIONS[name])
    if value < 0:
        raise PaError(value, "pa_get_option")
    return bool(value)


@contextlib.contextmanager
def option(name: str, value: bool = True) -> Iterator[None]:
    """``with api.option("debug_checks"):`` -- the option set for the block,
    restored afterwards."""
    prev = set_option(name, value)
    try:
        yield
    finally:
        set_option(name, prev)
