"""Python binding of the C ABI, with the same names.

Argument marshalling only: tensors become device pointers and element
strides, the current torch stream becomes the cudaStream_t, and every
non-zero status becomes a DecodeAttnError carrying the library's message.
Every step of the computation runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _native as N

_DT = {torch.float32: N.DA_F32, torch.float16: N.DA_F16, torch.bfloat16: N.DA_BF16,
       torch.float8_e4m3fn: N.DA_E4M3, torch.float8_e5m2: N.DA_E5M2}


class DecodeAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{N.STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


def _check(rc: int) -> None:
    if rc != N.DA_OK:
        raise DecodeAttnError(rc, decode_attn_last_error())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def dtype_code(dt: torch.dtype) -> int:
    if dt not in _DT:
        raise TypeError(f"unsupported dtype {dt}")
    return _DT[dt]


def make_args(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, scale: float, *,
              v_dim: Optional[int] = None, out_dtype: torch.dtype = torch.float32,
              force_splits: int = 0, flags: int = 0, timeout_us: int = 0) -> N.DaArgs:
    """Describe q [B, Hq, Dk] (one token per sequence) or [B, q_len, Hq, Dk]
    (q_len new tokens, causal among themselves) and caches [B, cap, Hkv, D]
    (any element strides) as a da_args_t. For MLA pass the same tensor as both
    caches and v_dim."""
    if q.dim() not in (3, 4) or k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("q must be [B, Hq, D] or [B, q_len, Hq, D] and caches [B, cap, Hkv, D]")
    if q.dim() == 3:
        (B, Hq, Dk), q_len = q.shape, 1
    else:
        B, q_len, Hq, Dk = q.shape
    a = N.DaArgs()
    a.batch, a.n_heads, a.n_kv_heads, a.head_dim = B, Hq, k_cache.shape[2], Dk
    a.q_len = q_len
    a.v_dim = int(v_dim) if v_dim is not None else v_cache.shape[3]
    a.capacity = k_cache.shape[1]
    ks, vs = k_cache.stride(), v_cache.stride()
    a.k_batch_stride, a.k_pos_stride, a.k_head_stride = ks[0], ks[1], ks[2]
    a.v_batch_stride, a.v_pos_stride, a.v_head_stride = vs[0], vs[1], vs[2]
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the last cache dimension must be contiguous")
    a.kv_dtype = dtype_code(k_cache.dtype)
    a.out_dtype = dtype_code(out_dtype)
    a.scale = float(scale)
    a.force_splits = int(force_splits)
    a.flags = int(flags)
    a.timeout_us = int(timeout_us)
    return a


def decode_attn_plan(args: N.DaArgs, seq_lens_host: Sequence[int], num_sms: int = 0) -> N.DaPlan:
    lens = (ctypes.c_int32 * max(1, args.batch))(*[int(x) for x in seq_lens_host])
    plan = N.DaPlan()
    _check(N.load().decode_attn_plan(ctypes.byref(args), ctypes.cast(lens, ctypes.c_void_p),
                                     int(num_sms), ctypes.byref(plan)))
    return plan


def decode_attn_workspace_bytes(plan: N.DaPlan) -> int:
    return int(N.load().decode_attn_workspace_bytes(ctypes.byref(plan)))


def new_workspace(plan: N.DaPlan, device=None) -> torch.Tensor:
    """Caller-owned workspace for one device (torch's allocator aligns to 512 bytes)."""
    return torch.empty(decode_attn_workspace_bytes(plan), dtype=torch.uint8,
                       device=device or "cuda")


def decode_attn_splitk_ex(args: N.DaArgs, plan: N.DaPlan, q: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                          stream=None) -> None:
    _check(N.load().decode_attn_splitk_ex(ctypes.byref(args), ctypes.byref(plan), _ptr(q),
                                          _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(stream)))


def decode_attn_combine(args: N.DaArgs, plan: N.DaPlan, workspace: torch.Tensor,
                        out: torch.Tensor, stream=None) -> None:
    _check(N.load().decode_attn_combine(ctypes.byref(args), ctypes.byref(plan), _ptr(workspace),
                                        _ptr(out), _stream(stream)))


def decode_attn_combine_ranks(args: N.DaArgs, plan: N.DaPlan, workspaces: torch.Tensor,
                              n_ranks: int, out: torch.Tensor, stream=None) -> None:
    """Merge the partials of n_ranks ranks that ran the same plan on their slices
    of the context; `workspaces` holds their workspaces back to back."""
    _check(N.load().decode_attn_combine_ranks(ctypes.byref(args), ctypes.byref(plan),
                                              _ptr(workspaces), int(n_ranks), _ptr(out),
                                              _stream(stream)))


def decode_attn_splitk(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       seq_lens: Sequence[int], n_heads: int, n_kv_heads: int, head_dim: int,
                       scale: float, out: torch.Tensor, stream=None) -> None:
    """Short form: batch 1, f32 everything, caches [L, Hkv, D] contiguous."""
    lens = (ctypes.c_int32 * 1)(int(seq_lens[0]))
    _check(N.load().decode_attn_splitk(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       ctypes.cast(lens, ctypes.c_void_p), int(n_heads),
                                       int(n_kv_heads), int(head_dim), float(scale), _ptr(out),
                                       _stream(stream)))


def decode_attn_splitk_noalloc(args: N.DaArgs, plan: N.DaPlan, q: torch.Tensor,
                               k_cache: torch.Tensor, v_cache: torch.Tensor, out: torch.Tensor,
                               stream=None) -> None:
    """decode_attn_splitk_ex without a workspace: the partials go to a 16 MiB
    array inside the library (for callers that cannot allocate). Calls that
    overlap on the GPU share that array and race."""
    _check(N.load().decode_attn_splitk_noalloc(ctypes.byref(args), ctypes.byref(plan), _ptr(q),
                                               _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                               _stream(stream)))


def make_paged_args(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, scale: float,
                    max_blocks_per_seq: int, *, v_dim: Optional[int] = None,
                    out_dtype: torch.dtype = torch.float32, force_splits: int = 0,
                    flags: int = 0, timeout_us: int = 0) -> N.DaArgs:
    """da_args_t for paged pools [num_blocks, block_size, Hkv, D]: the position and
    head strides come from the pools, the capacity is max_blocks_per_seq *
    block_size (the batch strides are not used for addressing). For MLA pass the
    latent pool as both pools and v_dim."""
    if k_pool.dim() != 4 or v_pool.dim() != 4:
        raise ValueError("pools must be [num_blocks, block_size, Hkv, D]")
    a = make_args(q, k_pool, v_pool, scale, v_dim=v_dim, out_dtype=out_dtype,
                  force_splits=force_splits, flags=flags, timeout_us=timeout_us)
    a.capacity = int(max_blocks_per_seq) * k_pool.shape[1]
    a.pools = _pools(k_pool, v_pool)      # (of this object alone, no field of the struct)
    return a


def make_dev(*, seq_lens: Optional[torch.Tensor] = None,
             block_table: Optional[torch.Tensor] = None, k_pool: Optional[torch.Tensor] = None,
             v_pool: Optional[torch.Tensor] = None) -> N.DaDev:
    """da_dev_t: device lengths (int32 [B] on the device) and, for paged caches, the
    block table (int32 [B, max_blocks] on the device) with the pools
    [num_blocks, block_size, Hkv, D]. The tensors must outlive every launch (and
    every replay of a captured launch) that uses them."""
    d = N.DaDev()
    if seq_lens is not None:
        if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
            raise TypeError("seq_lens must be an int32 CUDA tensor")
        d.seq_lens = seq_lens.data_ptr()
    if block_table is not None:
        if block_table.dtype != torch.int32 or not block_table.is_cuda or block_table.dim() != 2:
            raise TypeError("block_table must be a 2-D int32 CUDA tensor")
        if not block_table.is_contiguous():
            raise ValueError("block_table must be contiguous")
        if k_pool is None or v_pool is None:
            raise ValueError("a block table needs the K and V pools")
        d.block_table = block_table.data_ptr()
        d.max_blocks_per_seq = block_table.shape[1]
        d.block_size = k_pool.shape[1]
        d.num_blocks = k_pool.shape[0]
        d.k_block_stride = k_pool.stride(0)
        d.v_block_stride = v_pool.stride(0)
        d.pools = _pools(k_pool, v_pool)
    # (of this object alone, no fields of the struct: for decode_attn_splitk_8bit)
    given = [t for t in (seq_lens, block_table) if t is not None]
    if given:
        d.devices = [t.get_device() for t in given]
        d.batch = min(t.shape[0] if t.dim() == 2 else t.numel() for t in given)
    return d


def decode_attn_splitk_dev(args: N.DaArgs, plan: N.DaPlan, dev: N.DaDev, q: torch.Tensor,
                           k_cache: torch.Tensor, v_cache: torch.Tensor, out: torch.Tensor,
                           workspace: torch.Tensor, stream=None) -> None:
    """decode_attn_splitk_ex with lengths read on the device and, optionally,
    paged caches; capturable in a CUDA graph (no host decision depends on the
    current lengths)."""
    _check(N.load().decode_attn_splitk_dev(ctypes.byref(args), ctypes.byref(plan),
                                           ctypes.byref(dev), _ptr(q), _ptr(k_cache),
                                           _ptr(v_cache), _ptr(out), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(stream)))


def decode_attn_device_status(workspace: torch.Tensor, stream=None) -> None:
    _check(N.load().decode_attn_device_status(_ptr(workspace), _stream(stream)))


def decode_attn_last_error() -> str:
    return N.load().decode_attn_last_error().decode()


def decode_attn_release() -> None:
    N.load().decode_attn_release()


def decode_attn_version() -> str:
    return N.load().decode_attn_version().decode()


class DecodeAttention:
    """Plan once, run many times: holds the args, the plan and a workspace for
    fixed shapes and lengths (the plan/run split of the Kernel Level page)."""

    def __init__(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 seq_lens: Sequence[int], scale: Optional[float] = None, *,
                 v_dim: Optional[int] = None, out_dtype: torch.dtype = torch.float32,
                 force_splits: int = 0, flags: int = 0, num_sms: int = 0,
                 timeout_us: int = 0):
        sc = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
        self.args = make_args(q, k_cache, v_cache, sc, v_dim=v_dim, out_dtype=out_dtype,
                              force_splits=force_splits, flags=flags, timeout_us=timeout_us)
        self.plan = decode_attn_plan(self.args, list(seq_lens), num_sms)
        self.workspace = torch.empty(decode_attn_workspace_bytes(self.plan), dtype=torch.uint8,
                                     device=q.device)
        self.out_dtype = out_dtype

    def new_out(self, device) -> torch.Tensor:
        a = self.args
        shape = (a.batch, a.n_heads, a.v_dim) if a.q_len <= 1 else \
            (a.batch, a.q_len, a.n_heads, a.v_dim)
        return torch.empty(shape, dtype=self.out_dtype, device=device)

    def __call__(self, q, k_cache, v_cache, out=None, stream=None) -> torch.Tensor:
        if out is None:
            out = self.new_out(q.device)
        decode_attn_splitk_ex(self.args, self.plan, q, k_cache, v_cache, out, self.workspace,
                              stream)
        return out


def make_proj(w: torch.Tensor) -> N.DaProj:
    """da_proj_t for per-head projection weights w [n_heads, out_dim, v_dim]
    (f32 or bf16, on the device, last dimension contiguous). The tensor must
    outlive every launch that uses the descriptor."""
    if w.dim() != 3 or w.stride(2) != 1:
        raise ValueError("w must be [n_heads, out_dim, v_dim] with a contiguous last dimension")
    p = N.DaProj()
    p.w = w.data_ptr()
    p.w_dtype = dtype_code(w.dtype)
    p.out_dim = w.shape[1]
    p.head_stride, p.row_stride = w.stride(0), w.stride(1)
    return p


def decode_attn_combine_proj(args: N.DaArgs, plan: N.DaPlan, proj: N.DaProj,
                             workspaces: torch.Tensor, out: torch.Tensor, n_ranks: int = 1,
                             stream=None) -> None:
    """The merge of n_ranks workspaces (back to back) followed by the per-head
    projection: out [B, (q_len,) Hq, out_dim]."""
    _check(N.load().decode_attn_combine_proj(ctypes.byref(args), ctypes.byref(plan),
                                             ctypes.byref(proj), _ptr(workspaces),
                                             int(n_ranks), _ptr(out), _stream(stream)))


def decode_attn_splitk_proj(args: N.DaArgs, plan: N.DaPlan, proj: N.DaProj, q: torch.Tensor,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, out: torch.Tensor,
                            workspace: torch.Tensor, stream=None) -> None:
    """Split kernel, then the combine fused with the per-head projection."""
    _check(N.load().decode_attn_splitk_proj(ctypes.byref(args), ctypes.byref(plan),
                                            ctypes.byref(proj), _ptr(q), _ptr(k_cache),
                                            _ptr(v_cache), _ptr(out), _ptr(workspace),
                                            workspace.numel() * workspace.element_size(),
                                            _stream(stream)))


# ---- 8-bit paged caches ----------------------------------------------------------

# These calls take a few microseconds on the GPU, so their marshalling is kept lean: raw
# pointers and the raw current stream (3 us less than through a torch.cuda.Stream).

def _on(dev: torch.device, what: str, *tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"{what}: every tensor must be on {dev} (got one on {t.device})")


def _launch(dev: torch.device, stream, fn, *args) -> None:
    """fn(*args, stream handle) with `dev` current: by default on the current stream of
    the tensors' device, not of whichever device happens to be current."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev.index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev.index == torch._C._cuda_getDevice():    # (a CUDA tensor is there: initialised)
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        _check(rc)


def make_tables(seq_lens: torch.Tensor, block_table: torch.Tensor, free_list: torch.Tensor,
                state: torch.Tensor, block_size: int, *,
                seq_lens_out: Optional[torch.Tensor] = None,
                state_out: Optional[torch.Tensor] = None) -> N.DaTables:
    """da_tables_t: the device state of a batch's block tables, all int32 on one
    device: lengths [B], table [B, max_blocks], a stack of free blocks
    [num_blocks] and state [4] = {free blocks, status, 0, 0}. Lengths and state are
    updated in place unless *_out are given. The tensors must outlive every launch
    (and every replay of a captured launch) that uses them."""
    dev = seq_lens.device
    seq_lens_out = seq_lens if seq_lens_out is None else seq_lens_out
    state_out = state if state_out is None else state_out
    for name, t, dims in (("seq_lens", seq_lens, 1), ("block_table", block_table, 2),
                          ("free_list", free_list, 1), ("state", state, 1),
                          ("seq_lens_out", seq_lens_out, 1), ("state_out", state_out, 1)):
        if t.dtype != torch.int32 or not t.is_cuda or t.dim() != dims:
            raise TypeError(f"{name} must be a {dims}-D int32 CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _on(dev, "make_tables", block_table, free_list, state, seq_lens_out, state_out)
    B = seq_lens.shape[0]
    if block_table.shape[0] != B or seq_lens_out.shape[0] != B:
        raise ValueError("seq_lens, seq_lens_out and block_table must agree on the batch")
    if state.shape[0] != 4 or state_out.shape[0] != 4:
        raise ValueError("state must hold 4 words")
    t = N.DaTables()
    t.device = seq_lens.get_device()          # (of this object alone, no field of the struct)
    t.seq_lens, t.seq_lens_out = seq_lens.data_ptr(), seq_lens_out.data_ptr()
    t.block_table, t.free_list = block_table.data_ptr(), free_list.data_ptr()
    t.state, t.state_out = state.data_ptr(), state_out.data_ptr()
    t.batch, t.max_blocks_per_seq = B, block_table.shape[1]
    t.block_size, t.num_blocks = int(block_size), free_list.shape[0]
    return t


def decode_attn_grow_tables(tables: N.DaTables, new_lens: torch.Tensor,
                            slot_map: torch.Tensor, cu_new: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """Give sequence b new_lens[b] more tokens (int32 [B] on the device; negative:
    release it): takes the blocks, writes the tables, the slots of the new tokens
    (slot_map int64, -1 past the last) and their row offsets (cu_new int32 [B + 1])."""
    dev = new_lens.device
    if new_lens.dtype != torch.int32 or not new_lens.is_cuda or not new_lens.is_contiguous() \
            or new_lens.numel() != tables.batch:
        raise TypeError("new_lens must be a contiguous int32 CUDA tensor of the batch's size")
    if slot_map.dtype != torch.int64 or not slot_map.is_contiguous():
        raise TypeError("slot_map must be a contiguous int64 tensor")
    if cu_new is not None and (cu_new.dtype != torch.int32 or not cu_new.is_contiguous()
                               or cu_new.numel() != tables.batch + 1):
        raise TypeError("cu_new must be a contiguous int32 tensor of batch + 1 entries")
    _on(dev, "decode_attn_grow_tables", slot_map, cu_new)
    if getattr(tables, "device", dev.index) != dev.index:
        raise ValueError(f"the tables are on cuda:{tables.device}, new_lens on {dev}")
    _launch(dev, stream, N.load().decode_attn_grow_tables, ctypes.byref(tables),
            new_lens.data_ptr(), slot_map.data_ptr(), slot_map.numel(),
            0 if cu_new is None else cu_new.data_ptr())


def decode_attn_tables_status(state: torch.Tensor, stream=None) -> None:
    """Synchronises; raises if a decode_attn_grow_tables call on this state failed
    since the last check (and clears the status)."""
    if state.dtype != torch.int32 or not state.is_cuda or state.numel() != 4 \
            or not state.is_contiguous():
        raise TypeError("state must be a contiguous int32 CUDA tensor of 4 words")
    _launch(state.device, stream, N.load().decode_attn_tables_status, state.data_ptr())


def make_append(k_new: torch.Tensor, v_new: torch.Tensor, k_pool: torch.Tensor,
                v_pool: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor) -> N.DaAppend:
    """da_append_t for new rows [T, Hkv, D] (any token and head strides, e.g. the K and
    V parts of a fused projection), pools [num_blocks, block_size, Hkv, D] of
    float8_e4m3fn or float8_e5m2, and f32 scales [num_blocks, Hkv]."""
    if k_new.dim() != 3 or v_new.dim() != 3 or k_pool.dim() != 4 or v_pool.dim() != 4 \
            or k_scale.dim() != 2 or v_scale.dim() != 2:
        raise ValueError("new rows must be [T, Hkv, D], pools [num_blocks, block_size, Hkv, D] "
                         "and scales [num_blocks, Hkv]")
    if k_new.shape[:2] != v_new.shape[:2] or k_pool.shape[:3] != v_pool.shape[:3] \
            or k_new.dtype != v_new.dtype or k_pool.dtype != v_pool.dtype:
        raise ValueError("keys and values must agree in their tokens, heads, blocks and types")
    if k_new.shape[1:] != (k_pool.shape[2], k_pool.shape[3]) \
            or v_new.shape[1:] != (v_pool.shape[2], v_pool.shape[3]):
        raise ValueError("new rows and pools must agree in heads and width")
    want = (k_pool.shape[0], k_pool.shape[2])
    if tuple(k_scale.shape) != want or tuple(v_scale.shape) != want \
            or k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise ValueError("scales must be float32 [num_blocks, Hkv]")
    if any(t.stride(-1) != 1 for t in (k_new, v_new, k_pool, v_pool)):
        raise ValueError("the last dimension must be contiguous")
    a = N.DaAppend()
    a.n_tokens, a.n_kv_heads, a.head_dim = k_new.shape
    a.v_dim = v_new.shape[2]
    a.num_blocks, a.block_size = k_pool.shape[:2]
    a.src_dtype, a.code_dtype = dtype_code(k_new.dtype), dtype_code(k_pool.dtype)
    a.k_src_stride, a.k_src_head_stride = k_new.stride()[:2]
    a.v_src_stride, a.v_src_head_stride = v_new.stride()[:2]
    a.k_block_stride, a.k_pos_stride, a.k_head_stride = k_pool.stride()[:3]
    a.v_block_stride, a.v_pos_stride, a.v_head_stride = v_pool.stride()[:3]
    a.k_scale_block_stride, a.k_scale_head_stride = k_scale.stride()
    a.v_scale_block_stride, a.v_scale_head_stride = v_scale.stride()
    # (of this object alone, no field of the struct)
    a.tensors = (k_new.shape, k_new.stride(), v_new.shape, v_new.stride(), k_new.dtype,
                 v_new.dtype, k_pool.shape, k_pool.stride(), v_pool.shape, v_pool.stride(),
                 k_pool.dtype, v_pool.dtype, k_scale.shape, k_scale.stride(), v_scale.shape,
                 v_scale.stride(), k_scale.dtype, v_scale.dtype)
    return a


def decode_attn_append_8bit(append: N.DaAppend, k_new: torch.Tensor, v_new: torch.Tensor,
                            slot_map: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                            k_scale: torch.Tensor, v_scale: torch.Tensor, stream=None) -> None:
    """Quantise the new rows into the slots (int64 [T], negative: skip the row) of
    the pools, one power-of-two scale per (block, KV head). `append` describes
    tensors of these shapes and strides (make_append)."""
    if slot_map.dtype != torch.int64 or not slot_map.is_contiguous() \
            or slot_map.numel() != append.n_tokens:
        raise TypeError("slot_map must be a contiguous int64 tensor with a slot per row")
    index = k_pool.get_device()
    if index < 0:
        raise TypeError("the pools must be CUDA tensors")
    if not index == k_new.get_device() == v_new.get_device() == slot_map.get_device() \
            == v_pool.get_device() == k_scale.get_device() == v_scale.get_device():
        _on(k_pool.device, "decode_attn_append_8bit", k_new, v_new, slot_map, v_pool, k_scale,
            v_scale)
    if (k_new.shape, k_new.stride(), v_new.shape, v_new.stride(), k_new.dtype, v_new.dtype,
            k_pool.shape, k_pool.stride(), v_pool.shape, v_pool.stride(), k_pool.dtype,
            v_pool.dtype, k_scale.shape, k_scale.stride(), v_scale.shape, v_scale.stride(),
            k_scale.dtype, v_scale.dtype) != getattr(append, "tensors", None):
        # (a descriptor filled in by hand, or one for other tensors)
        if bytes(make_append(k_new, v_new, k_pool, v_pool, k_scale, v_scale)) != bytes(append):
            raise ValueError("append describes tensors of other shapes, strides or types")
    _append_8bit(append, k_new, v_new, slot_map, k_pool, v_pool, k_scale, v_scale, stream)


def _append_8bit(append, k_new, v_new, slot_map, k_pool, v_pool, k_scale, v_scale,
                 stream) -> None:
    _launch(k_pool.device, stream, N.load().decode_attn_append_8bit, ctypes.byref(append),
            k_new.data_ptr(), v_new.data_ptr(), slot_map.data_ptr(), k_pool.data_ptr(),
            v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())


def make_scales(k_scale: torch.Tensor, v_scale: torch.Tensor) -> N.DaScales:
    """da_scales_t for f32 scales [num_blocks, Hkv] (any strides). The tensors must
    outlive every launch that uses the descriptor."""
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or not t.is_cuda or t.dim() != 2:
            raise TypeError("scales must be 2-D float32 CUDA tensors")
    if k_scale.get_device() != v_scale.get_device():
        raise ValueError("scales must be on one device")
    s = N.DaScales()
    # (of this object alone, no fields of the struct: for decode_attn_splitk_8bit)
    s.devices = [k_scale.get_device()]
    s.blocks, s.heads = [min(n) for n in zip(k_scale.shape, v_scale.shape)]
    s.k_scale, s.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
    s.k_block_stride, s.k_head_stride = k_scale.stride()
    s.v_block_stride, s.v_head_stride = v_scale.stride()
    return s


def decode_attn_splitk_8bit(args: N.DaArgs, plan: N.DaPlan, dev: N.DaDev, scales: N.DaScales,
                            q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                            out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """decode_attn_splitk_dev over 8-bit pools with scales (make_paged_args,
    make_dev with a block table, make_scales). q, out and the pools are of the shapes and
    types that args and dev describe."""
    index = q.get_device()
    if index < 0:
        raise TypeError("q must be a CUDA tensor")
    if not index == k_pool.get_device() == v_pool.get_device() == out.get_device() \
            == workspace.get_device():
        _on(q.device, "decode_attn_splitk_8bit", k_pool, v_pool, out, workspace)
    if q.dtype != torch.float32 or not q.is_contiguous() or not out.is_contiguous():
        raise TypeError("q must be contiguous float32 and out contiguous")
    if _DT.get(out.dtype) != args.out_dtype:
        raise TypeError(f"out is {out.dtype}, not of the type that args were made for")
    rows = args.batch * args.n_heads * (args.q_len or 1)
    if q.numel() != rows * args.head_dim or out.numel() != rows * args.v_dim:
        raise ValueError(f"q and out must hold {rows} rows, as args describe")
    pools = _pools(k_pool, v_pool)
    if not pools == getattr(args, "pools", None) == getattr(dev, "pools", None):
        _check_pools(args, dev, k_pool, v_pool)
    _check_descriptors(index, args, dev, scales)
    _splitk_8bit(args, plan, dev, scales, q, k_pool, v_pool, out, workspace, stream)


def _check_descriptors(index: int, args: N.DaArgs, dev: N.DaDev, scales: N.DaScales) -> None:
    """Raises unless the tensors behind dev and scales are on the call's device and hold its
    batch and pages (of descriptors that make_dev and make_scales made)."""
    for what, x in (("lengths and table", dev), ("scales", scales)):
        if getattr(x, "devices", None) not in (None, [index], [index, index]):
            raise ValueError(f"the {what} must be on q's device, cuda:{index}")
    if getattr(dev, "batch", args.batch) < args.batch:
        raise ValueError(f"the lengths and table hold {dev.batch} sequences, q {args.batch}")
    if getattr(scales, "blocks", dev.num_blocks) < dev.num_blocks or \
            getattr(scales, "heads", args.n_kv_heads) < args.n_kv_heads:
        raise ValueError(f"the scales must be [{dev.num_blocks}, {args.n_kv_heads}]")


def _pools(k_pool: torch.Tensor, v_pool: torch.Tensor) -> tuple:
    return (k_pool.shape, k_pool.stride(), k_pool.dtype, v_pool.shape, v_pool.stride(),
            v_pool.dtype)


def _check_pools(args: N.DaArgs, dev: N.DaDev, k_pool: torch.Tensor, v_pool: torch.Tensor) -> None:
    """Raises unless the pools are what args and dev describe."""
    if _DT.get(k_pool.dtype) != args.kv_dtype or _DT.get(v_pool.dtype) != args.kv_dtype:
        raise TypeError("the pools are not of the type that args were made for")
    if not dev.block_table:
        return                # the library refuses the call
    n, rest = dev.num_blocks, (dev.block_size, args.n_kv_heads)
    if k_pool.shape[0] < n or k_pool.shape[1:] != rest + (args.head_dim,) or \
            v_pool.shape[0] < n or v_pool.shape[1:] != rest + (args.v_dim,):
        raise ValueError(f"the pools must be {(n, *rest)}, as args and dev describe")
    if k_pool.stride() != (dev.k_block_stride, args.k_pos_stride, args.k_head_stride, 1) or \
            v_pool.stride() != (dev.v_block_stride, args.v_pos_stride, args.v_head_stride, 1):
        raise ValueError("the pools' strides are not those of args and dev")


def _splitk_8bit(args, plan, dev, scales, q, k_pool, v_pool, out, workspace, stream) -> None:
    _launch(q.device, stream, N.load().decode_attn_splitk_8bit, ctypes.byref(args),
            ctypes.byref(plan), ctypes.byref(dev), ctypes.byref(scales), q.data_ptr(),
            k_pool.data_ptr(), v_pool.data_ptr(), out.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
