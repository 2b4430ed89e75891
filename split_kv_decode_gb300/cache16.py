"""A paged KV cache in 16 bits, rotated on the way in, and scored attention over it.

PagedCache16 owns the pools (f16 or bf16), the block tables and the free list of one layer, all on
the device. A step is three launches and the combine, in the order of a serving loop:

    cache.grow(new_lens)                    blocks and slots of the new tokens
    q = cache.append(q, k, v, positions)    norms and rotary positions; k and v into their slots
    out = step(q)                           attention over the pages (ScoredStep)

None of them makes a host decision that depends on the current lengths, so a whole step can be
captured in a CUDA graph once and replayed while the contexts grow. A prefix that all sequences
share lies in blocks of its own (shared_blocks, append_shared) and is read once for all of them.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import _native as N
from . import api as A
from .cache8 import _init_tables


class PagedCache16:
    """One layer's 16-bit cache for up to `max_batch` sequences of up to
    `max_blocks_per_seq * block_size` positions in `num_blocks` shared pages, of which the first
    `shared_blocks` hold a prefix of all sequences.

    `max_new` is the number of new rows a step may bring (rows past the ones a step really has are
    skipped: their slot is -1). rope (make_rope; None: no rotation), eps and the weights are those
    of append(). Layers of one model share the tables: pass the first layer's cache as
    `tables_of`, and grow only that one.
    """

    def __init__(self, max_batch: int, num_blocks: int, max_blocks_per_seq: int,
                 n_kv_heads: int, head_dim: int, *, block_size: int = 64,
                 max_new: Optional[int] = None, dtype: torch.dtype = torch.bfloat16,
                 rope: Optional[N.DaRope] = None, eps: Optional[float] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 weight_offset: float = 0.0, shared_blocks: int = 0,
                 tables_of: Optional["PagedCache16"] = None, device="cuda"):
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("a 16-bit cache holds float16 or bfloat16")
        if not 0 <= shared_blocks <= num_blocks:
            raise ValueError(f"shared_blocks must be in [0, {num_blocks}]")
        shape = (num_blocks, block_size, n_kv_heads, head_dim)
        self.block_size, self.shared_blocks = block_size, shared_blocks
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        _init_tables(self, max_batch, num_blocks, max_blocks_per_seq, block_size, max_new,
                     tables_of, device, shared_blocks)
        self.shared_table = torch.arange(shared_blocks, dtype=torch.int32, device=device)
        # (made once: a slot map of a call's own would be written on torch's current stream, not on
        # the call's, and its memory given to others while the call is pending)
        self.shared_slots = torch.arange(shared_blocks * block_size, device=device)
        self.dev = A.make_dev(seq_lens=self.seq_lens, block_table=self.block_table,
                              k_pool=self.k, v_pool=self.v)
        self.rope = A.make_rope([], device=device) if rope is None else rope
        self._norm = dict(eps=eps, q_weight=q_weight, k_weight=k_weight,
                          weight_offset=weight_offset)
        self._prep = None                    # of the last rows; shapes, strides and types only

    def grow(self, new_lens: torch.Tensor, stream=None) -> torch.Tensor:
        """Give sequence b new_lens[b] tokens (int32 [max_batch] on the device, 0: none,
        negative: release it). Returns the slot map (this object's buffer)."""
        A.decode_attn_grow_tables(self.tables, new_lens, self.slot_map, self.cu_new, stream)
        return self.slot_map

    def append(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
               q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Normalise and rotate the rows q [T, Hq, D] and k [T, Hkv, D] of the last grow(), and write
        k and v into their slots; T at most max_new, and at least the tokens that grow() gave (rows
        past them are not cached). positions: int64 [T] or [axes, T]. Returns the rotated q (q_out,
        or a new tensor of q's type)."""
        if k.dim() != 3 or k.shape[0] > self.slot_map.numel():
            raise ValueError(f"new rows must be [T, Hkv, D] with T <= {self.slot_map.numel()}")
        return self._write(q, k, v, positions, self.slot_map[:k.shape[0]], q_out, stream)

    def append_shared(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      positions: torch.Tensor, first: int = 0,
                      q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The same for rows of the shared prefix: row t is its position first + t."""
        room = self.shared_blocks * self.block_size
        if k.dim() != 3 or not 0 <= first <= room - k.shape[0]:
            raise ValueError(f"the shared blocks hold {room} positions")
        return self._write(q, k, v, positions, self.shared_slots[first:first + k.shape[0]], q_out,
                           stream)

    def _write(self, q, k, v, positions, slots, q_out, stream) -> torch.Tensor:
        if q_out is None:
            q_out = A._empty(q.shape, q.dtype, q.device, stream)
        rows = (q, k, v, q_out, self.k, self.v)
        prep = self._prep                    # (another host thread's call may replace it)
        if prep is None or prep.tensors != A._prep_tensors(*rows):
            prep = self._prep = A.make_prep(*rows, self.rope, **self._norm)
        A.decode_attn_rope_append(prep, q, k, v, positions, slots, q_out, self.k, self.v, stream)
        return q_out

    def check(self, stream=None) -> None:
        """Synchronises; raises if a grow() since the last check could not be served."""
        A.decode_attn_tables_status(self.state, stream)


class ScoredStep:
    """Scored attention of q [B, Hq, D] (or [B, q_len, Hq, D]; f32 or of the cache's type) over a
    PagedCache16, B at most the cache's max_batch: plan and workspace for sequences of up to
    `max_lens` positions of their own (default: the tables' width); the current lengths are the
    cache's, on the device. softcap, slopes, window, keep, keep_lens and starts are make_score's
    (keep_lens needs keep, its upper bound); shared_len positions of the cache's shared blocks come
    before every sequence's own.

    The work is split for max_lens, whatever the lengths are then: a bound near them is up to three
    times faster than the width of mostly empty tables (a sequence of 4096 positions under a bound
    of 32 times that: 39 us instead of 12.5; 32 of them: 98 instead of 89). Positions past it are
    not attended to. Calls that overlap on the GPU need steps of their own (one workspace each). A
    new output is memory of the call's stream; the cache and the step are made on the current one,
    behind which another stream's first call has to be ordered."""

    def __init__(self, cache: PagedCache16, q: torch.Tensor, scale: Optional[float] = None, *,
                 max_lens: Optional[Sequence[int]] = None, out_dtype: Optional[torch.dtype] = None,
                 softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, window: int = 0,
                 keep: int = 0, keep_lens: Optional[torch.Tensor] = None,
                 starts: Optional[torch.Tensor] = None, shared_len: int = 0,
                 force_splits: int = 0, flags: int = 0, timeout_us: int = 0):
        self.cache, self.out_dtype = cache, out_dtype or cache.k.dtype
        width = cache.block_table.shape[1]
        if q.shape[0] > cache.seq_lens.numel():
            raise ValueError("q has more sequences than the cache")
        if keep_lens is not None and keep < 1:
            raise ValueError("keep_lens keeps nothing without keep, its upper bound")
        if shared_len > cache.shared_blocks * cache.block_size:
            raise ValueError("shared_len is more than the cache's shared blocks hold")
        sc = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
        self.args = A.make_paged_args(q, cache.k, cache.v, sc, width, out_dtype=self.out_dtype,
                                      force_splits=force_splits, flags=flags,
                                      timeout_us=timeout_us)
        self.score = A.make_score(q, softcap=softcap, slopes=slopes, window=window, keep=keep,
                                  keep_lens=keep_lens, starts=starts, shared_len=shared_len,
                                  shared_table=cache.shared_table if shared_len else None)
        lens = [width * cache.block_size] * q.shape[0] if max_lens is None else list(max_lens)
        self.plan = A.decode_attn_plan_scored(self.args, self.score, lens)
        self.shape, self.q_dtype = tuple(q.shape), q.dtype
        self.workspace = A.new_workspace(self.plan, device=q.device)

    def __call__(self, q: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        if tuple(q.shape) != self.shape or q.dtype != self.q_dtype:
            raise ValueError(f"planned for q of shape {self.shape} and type {self.q_dtype}")
        if out is None:
            out = A._empty(self.shape, self.out_dtype, q.device, stream)
        elif tuple(out.shape) != self.shape:
            raise ValueError(f"out must be of shape {self.shape}")
        A.decode_attn_splitk_scored(self.args, self.plan, self.cache.dev, self.score, q,
                                    self.cache.k, self.cache.v, out, self.workspace, stream)
        return out
