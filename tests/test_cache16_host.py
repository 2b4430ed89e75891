"""PagedCache16 and ScoredStep on the host: what a call does besides its launch (no GPU)."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300.cache16 import PagedCache16


class Ops(TorchDispatchMode):
    """The names of the torch operations that are called."""

    def __init__(self):
        super().__init__()
        self.names = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.append(func.overloadpacket.__name__)
        return func(*args, **(kwargs or {}))


@pytest.fixture
def appended(monkeypatch):
    """The arguments of the rotated appends."""
    got = []
    monkeypatch.setattr(A, "make_dev", lambda **kw: N.DaDev())
    monkeypatch.setattr(A, "make_tables", lambda *x: N.DaTables())
    monkeypatch.setattr(A, "decode_attn_rope_append", lambda *x: got.append(x))
    return got


def rows(n, hq=4, hkv=2, d=128):
    return [torch.zeros(n, h, d, dtype=torch.bfloat16) for h in (hq, hkv, hkv)]


def test_shared_rows_bring_no_work_of_their_own(appended):
    # a kernel that made the slots would run on the current stream, unordered with the call's, and
    # its result would be given back to the allocator while the call may still read it
    c = PagedCache16(2, 10, 4, 2, 128, block_size=16, shared_blocks=3, device="cpu")
    kept = {t.untyped_storage().data_ptr() for t in vars(c).values() if isinstance(t, torch.Tensor)}
    for first, n in ((5, 16), (0, 5), (21, 27), (0, 48), (48, 0)):
        q, k, v = rows(n)
        q_out, pos = torch.empty_like(q), torch.arange(first, first + n)
        with Ops() as ops:
            c.append_shared(q, k, v, pos, first, q_out=q_out, stream=1234)
        assert set(ops.names) <= {"slice", "view", "alias", "detach"}, ops.names
        slots, stream = appended[-1][5], appended[-1][-1]
        assert stream == 1234 and slots.dtype == torch.int64 and slots.is_contiguous()
        assert slots.tolist() == list(range(first, first + n))
        assert slots.untyped_storage().data_ptr() in kept
    for first, n in ((-1, 2), (47, 2), (49, 0)):
        q, k, v = rows(n)
        with pytest.raises(ValueError):
            c.append_shared(q, k, v, torch.arange(n), first)
