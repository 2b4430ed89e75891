"""A paged KV cache in 8 bits, and the decode step over it.

PagedCache8 owns the pools (float8 codes, one power-of-two scale per page and KV
head), the block tables and the free list of one layer, all on the device. A
step is three launches and the combine, in the order of a serving loop:

    cache.grow(new_lens)            blocks and slots of the new tokens
    cache.append(k_new, v_new)      the new rows, quantised into their slots
    out = step(q)                   attention over the pages (Step8)

None of them makes a host decision that depends on the current lengths, so a
whole step can be captured in a CUDA graph once and replayed while the contexts
grow ("The Kernel Level: Attention and MoE", the serving and CUDA-graph
sections).
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import api as A


def _init_tables(cache, max_batch: int, num_blocks: int, max_blocks_per_seq: int,
                 block_size: int, max_new: Optional[int], tables_of, device,
                 taken: int = 0) -> None:
    """Gives a cache with pools `k` its block tables, those of another cache (tables_of), or its
    own, whose free list leaves out the first `taken` blocks."""
    if tables_of is not None:
        t = tables_of
        if (t.block_size, t.free_list.numel(), getattr(t, "shared_blocks", 0)) != \
                (block_size, num_blocks - taken, taken):
            raise ValueError("caches that share tables need equal pages")
        if tuple(t.block_table.shape) != (max_batch, max_blocks_per_seq) \
                or max_new not in (None, t.slot_map.numel()):
            raise ValueError("caches that share tables need equal batches, widths and rows")
        if t.block_table.device != cache.k.device:
            raise ValueError(f"the tables are on {t.block_table.device}, not {cache.k.device}")
        for name in ("seq_lens", "block_table", "free_list", "state", "slot_map", "cu_new",
                     "tables"):
            setattr(cache, name, getattr(tables_of, name))
        return

    def ints(*size):
        return torch.zeros(*size, dtype=torch.int32, device=device)
    cache.seq_lens = ints(max_batch)
    cache.block_table = ints(max_batch, max_blocks_per_seq)
    # popped from the end: the lowest block first
    cache.free_list = torch.arange(num_blocks - 1, taken - 1, -1, dtype=torch.int32, device=device)
    cache.state = ints(4)
    cache.state[0] = num_blocks - taken
    cache.slot_map = torch.full((max_new or max_batch,), -1, dtype=torch.int64, device=device)
    cache.cu_new = ints(max_batch + 1)
    cache.tables = A.make_tables(cache.seq_lens, cache.block_table, cache.free_list, cache.state,
                                 block_size)


class PagedCache8:
    """One layer's 8-bit cache for up to `max_batch` sequences of up to
    `max_blocks_per_seq * block_size` positions in `num_blocks` shared pages.

    `max_new` is the number of new rows a step may bring (rows past the ones a
    step really has are skipped: their slot is -1). Layers of one model share
    the tables: pass the first layer's cache as `tables_of`, and grow only that one.
    """

    def __init__(self, max_batch: int, num_blocks: int, max_blocks_per_seq: int,
                 n_kv_heads: int, head_dim: int, *, block_size: int = 64,
                 max_new: Optional[int] = None, dtype: torch.dtype = torch.float8_e4m3fn,
                 tables_of: Optional["PagedCache8"] = None, device="cuda"):
        if dtype not in (torch.float8_e4m3fn, torch.float8_e5m2):
            raise TypeError("an 8-bit cache holds float8_e4m3fn or float8_e5m2 codes")
        shape = (num_blocks, block_size, n_kv_heads, head_dim)
        self.block_size = block_size
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)
        self.k_scale = torch.ones(num_blocks, n_kv_heads, device=device)
        self.v_scale = torch.ones(num_blocks, n_kv_heads, device=device)
        self.scales = A.make_scales(self.k_scale, self.v_scale)
        _init_tables(self, max_batch, num_blocks, max_blocks_per_seq, block_size, max_new,
                     tables_of, device)
        self.dev = A.make_dev(seq_lens=self.seq_lens, block_table=self.block_table,
                              k_pool=self.k, v_pool=self.v)
        self._append = None                  # of the last rows, and their shapes only

    def grow(self, new_lens: torch.Tensor, stream=None) -> torch.Tensor:
        """Give sequence b new_lens[b] tokens (int32 [max_batch] on the device, 0: none,
        negative: release it). Returns the slot map (this object's buffer)."""
        A.decode_attn_grow_tables(self.tables, new_lens, self.slot_map, self.cu_new, stream)
        return self.slot_map

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """Write the rows [T, Hkv, D] of the last grow() into their slots; T at most
        max_new, and at least the tokens that grow() gave (rows past them are skipped)."""
        if k_new.dim() != 3 or k_new.shape[0] > self.slot_map.numel():
            raise ValueError(f"new rows must be [T, Hkv, D] with T <= {self.slot_map.numel()}")
        shapes = (k_new.shape, v_new.shape, k_new.stride(), v_new.stride(), k_new.dtype,
                  v_new.dtype)
        append = self._append                # (another host thread's call may replace it)
        if append is None or append.shapes != shapes:
            append = A.make_append(k_new, v_new, self.k, self.v, self.k_scale, self.v_scale)
            append.shapes = shapes           # (of this object alone, no field of the struct)
            self._append = append
        if not k_new.device == v_new.device == self.k.device:
            raise ValueError(f"new rows must be on {self.k.device}")
        slots, n = self.slot_map, k_new.shape[0]
        A._append_8bit(append, k_new, v_new, slots if n == slots.numel() else slots[:n], self.k,
                       self.v, self.k_scale, self.v_scale, stream)

    def check(self, stream=None) -> None:
        """Synchronises; raises if a grow() since the last check could not be served."""
        A.decode_attn_tables_status(self.state, stream)


class Step8:
    """Attention of q [B, Hq, D] (or [B, q_len, Hq, D]) over a PagedCache8, B at most the
    cache's max_batch: plan and workspace for sequences of up to `max_lens` positions
    (default: the tables' width); the current lengths are the cache's, on the device.

    The work is split for max_lens, whatever the lengths are then: a bound near them is
    up to several times faster than the width of mostly empty tables. Positions past it
    are not attended to. Calls that overlap on the GPU need steps of their own (one
    workspace each)."""

    def __init__(self, cache: PagedCache8, q: torch.Tensor, scale: Optional[float] = None, *,
                 max_lens: Optional[Sequence[int]] = None,
                 out_dtype: torch.dtype = torch.float32, force_splits: int = 0, flags: int = 0,
                 timeout_us: int = 0):
        self.cache, self.out_dtype = cache, out_dtype
        width = cache.block_table.shape[1]
        if q.shape[0] > cache.seq_lens.numel():
            raise ValueError("q has more sequences than the cache")
        sc = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
        self.args = A.make_paged_args(q, cache.k, cache.v, sc, width, out_dtype=out_dtype,
                                      force_splits=force_splits, flags=flags,
                                      timeout_us=timeout_us)
        lens = [width * cache.block_size] * q.shape[0] if max_lens is None else list(max_lens)
        self.plan = A.decode_attn_plan(self.args, lens)
        self.shape = tuple(q.shape)
        self.workspace = A.new_workspace(self.plan, device=q.device)

    def __call__(self, q: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        if tuple(q.shape) != self.shape:
            raise ValueError(f"planned for q of shape {self.shape}")
        c = self.cache
        if q.dtype != torch.float32 or not q.is_contiguous() or q.device != c.k.device:
            raise TypeError(f"q must be contiguous float32 on {c.k.device}")
        if out is None:
            out = A._empty(self.shape, self.out_dtype, q.device, stream)
        elif tuple(out.shape) != self.shape or out.dtype != self.out_dtype \
                or not out.is_contiguous() or out.device != q.device:
            raise TypeError(f"out must be contiguous {self.out_dtype} of shape {self.shape} "
                            f"on {q.device}")
        A._splitk_8bit(self.args, self.plan, c.dev, c.scales, q, c.k, c.v, out,
                                  self.workspace, stream)
        return out
