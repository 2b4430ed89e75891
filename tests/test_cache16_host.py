"""What calls of the caches and their steps do besides their launches (no GPU)."""
from contextlib import contextmanager
from types import SimpleNamespace

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300.cache8 import PagedCache8, Step8
from split_kv_decode_gb300.cache16 import PagedCache16, ScoredStep


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


@pytest.fixture
def streams(monkeypatch):
    """The streams that are made current, and on which of them torch.empty makes its tensors."""
    now, made, empty = [None], [], torch.empty

    @contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def new(*args, **kw):
        made.append(now[-1])
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("external", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", new)
    return made


def test_new_outputs_are_of_the_calls_stream(appended, streams, monkeypatch):
    # (of the current one's memory they could be written while earlier work there still uses it)
    cache = PagedCache16(2, 10, 4, 2, 128, block_size=16, shared_blocks=3, device="cpu")
    q, k, v = rows(2)
    pos = torch.arange(2)
    monkeypatch.setattr(A, "decode_attn_splitk_scored", lambda *x: None)
    monkeypatch.setattr(A, "_splitk_8bit", lambda *x: None)
    monkeypatch.setattr(A, "decode_attn_splitk_ex", lambda *x: None)
    scored = ScoredStep.__new__(ScoredStep)
    scored.shape, scored.q_dtype, scored.out_dtype = tuple(q.shape), q.dtype, torch.float32
    scored.cache = cache
    scored.args = scored.plan = scored.score = scored.workspace = None
    eight = Step8.__new__(Step8)
    eight.shape, eight.out_dtype = tuple(q.shape), torch.float16
    eight.cache = SimpleNamespace(k=k, v=v, dev=None, scales=None)
    eight.args = eight.plan = eight.workspace = None
    plain = A.DecodeAttention.__new__(A.DecodeAttention)
    plain.args, plain.out_dtype = SimpleNamespace(batch=2, n_heads=4, v_dim=128, q_len=0), torch.float32
    plain.plan = plain.workspace = None
    calls = [(lambda s: cache.append(q, k, v, pos, stream=s), q.dtype),
             (lambda s: cache.append_shared(q, k, v, pos, 7, stream=s), q.dtype),
             (lambda s: scored(q, stream=s), torch.float32),
             (lambda s: eight(q.float(), stream=s), torch.float16),
             (lambda s: plain(q, k, v, stream=s), torch.float32)]
    for call, dtype in calls:
        for given, used in ((None, None), (SimpleNamespace(cuda_stream=96), ("external", 96)),
                            (4096, ("external", 4096)), (0, "default"), (1, "default")):
            streams.clear()
            out = call(given)
            assert streams == [used] and out.shape == q.shape and out.dtype == dtype


@pytest.mark.parametrize("keep", [0, -1])
def test_kept_lengths_without_their_bound_are_refused(keep):
    # (they are bounded by keep, so that nothing would be kept)
    cache = SimpleNamespace(k=torch.zeros(4, 16, 2, 128), block_table=torch.zeros(2, 4),
                            seq_lens=torch.zeros(2))
    with pytest.raises(ValueError, match="keep_lens"):
        ScoredStep(cache, rows(2)[0], keep=keep, keep_lens=torch.zeros(2, dtype=torch.int32))


def test_a_call_keeps_its_descriptor_when_another_one_comes_between(appended, monkeypatch):
    # as another host thread's call does, between this one's look at the last descriptor and its launch
    few, more = rows(2), rows(3)
    pos = torch.arange(3)
    cache = PagedCache16(4, 10, 4, 2, 128, block_size=16, device="cpu")
    cache.append(*few, pos[:2])
    between, look = [], A._prep_tensors

    def look_and_meet(*x):
        got = look(*x)
        if between:
            between.pop()()
        return got

    monkeypatch.setattr(A, "_prep_tensors", look_and_meet)
    between.append(lambda: cache.append(*more, pos))
    appended.clear()
    cache.append(*few, pos[:2])
    assert sorted((x[0].n_tokens, x[1].shape[0]) for x in appended) == [(2, 2), (3, 3)]

    calls = []
    monkeypatch.setattr(A, "make_scales", lambda *x: N.DaScales())
    monkeypatch.setattr(A, "_append_8bit", lambda *x: calls.append((x[0].n_tokens, x[1].shape[0])))
    eight = PagedCache8(4, 10, 4, 2, 128, block_size=16, device="cpu")
    eight.append(*few[1:])

    class Meets:                                # (the slots are looked up behind the descriptor)
        def __get__(self, cache, _):
            if between:
                between.pop()()
            return torch.zeros(4, dtype=torch.int64)

    kept = eight.__dict__.pop("slot_map")
    monkeypatch.setattr(PagedCache8, "slot_map", Meets(), raising=False)
    calls.clear()

    def meet():
        # the first look at the slots is before the descriptor's
        between.append(lambda: eight.append(*more[1:]))

    between.append(meet)
    eight.append(*few[1:])
    assert kept.numel() == 4 and sorted(calls) == [(2, 2), (3, 3)]
