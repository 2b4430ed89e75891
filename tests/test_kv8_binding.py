"""Refusals of the 8-bit cache's binding (CPU): stand-ins for CUDA tensors carry a type, a
shape, strides and a device, and no call gets as far as a launch."""
from types import SimpleNamespace

import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300 import cache8 as C

CUDA = torch.device("cuda", 0)


class Fake:
    """What the binding looks at of a CUDA tensor."""

    def __init__(self, shape, dtype=torch.float32, stride=None, device=CUDA):
        self._t = torch.empty(0, dtype=dtype)
        full = []
        for n in reversed(shape):
            full.insert(0, full[0] * below if full else 1)
            below = n
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self._stride = tuple(stride or full)
        self._dense = tuple(full)
        self.is_cuda = device.type == "cuda"

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self._t.element_size()

    def is_contiguous(self):
        return self._stride == self._dense

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def launches(monkeypatch):
    """Launches that a call would make; none is made."""
    got = []
    monkeypatch.setattr(A, "_launch", lambda dev, stream, fn, *args: got.append((dev, args)))
    monkeypatch.setattr(N, "load", lambda: SimpleNamespace(
        decode_attn_splitk_8bit=None, decode_attn_append_8bit=None, decode_attn_grow_tables=None,
        decode_attn_tables_status=None))
    return got


E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
POOL = (40, 16, 2, 128)


def attend(q_shape=(3, 8, 128), out_dtype=torch.float32, pool=POOL, **kw):
    t = dict(q=Fake(q_shape), k=Fake(pool, E4), v=Fake(pool, E4), out=Fake(q_shape, out_dtype),
             lens=Fake((3,), torch.int32), table=Fake((3, 10), torch.int32),
             ks=Fake(pool[::2][:2]), vs=Fake(pool[::2][:2]), ws=Fake((4096,), torch.uint8))
    a = A.make_paged_args(t["q"], t["k"], t["v"], 0.1, 10, out_dtype=out_dtype)
    dev = A.make_dev(seq_lens=t["lens"], block_table=t["table"], k_pool=t["k"], v_pool=t["v"])
    t.update(kw)
    A.decode_attn_splitk_8bit(a, N.DaPlan(), dev, A.make_scales(t["ks"], t["vs"]), t["q"], t["k"],
                              t["v"], t["out"], t["ws"])


@pytest.mark.parametrize("q_shape", [(3, 8, 128), (3, 2, 8, 128)])
@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
def test_attention_takes_what_it_was_made_for(launches, q_shape, out):
    attend(q_shape, out)
    assert len(launches) == 1 and launches[0][0] == CUDA
    attend(q_shape, out, out=Fake((torch.Size(q_shape).numel(),), out))   # any shape of that size
    assert len(launches) == 2


@pytest.mark.parametrize("kw", [
    dict(out=Fake((3, 8, 128), torch.bfloat16)), dict(out=Fake((2, 8, 128))),
    dict(out=Fake((3, 8, 64))), dict(q=Fake((2, 8, 128))), dict(q=Fake((3, 8, 256))),
    dict(q=Fake((3, 8, 128), torch.float16)), dict(k=Fake(POOL, E5)), dict(v=Fake(POOL, E5)),
    dict(k=Fake(POOL, torch.float16)), dict(v=Fake((39, 16, 2, 128), E4)),
    dict(k=Fake((40, 32, 2, 128), E4)), dict(k=Fake((40, 16, 1, 128), E4)),
    dict(v=Fake((40, 16, 2, 256), E4)), dict(k=Fake(POOL, E4, (4096, 128, 2048, 1))),
    dict(out=Fake((3, 8, 128), device=torch.device("cpu")))])
def test_attention_refuses_other_tensors_than_described(launches, kw):
    with pytest.raises((TypeError, ValueError)):
        attend(**kw)
    assert not launches


def step(q_shape=(3, 8, 128), out_dtype=torch.float32):
    s = C.Step8.__new__(C.Step8)
    s.cache = SimpleNamespace(k=Fake(POOL, E4), v=Fake(POOL, E4), dev=N.DaDev(), scales=N.DaScales())
    s.shape, s.out_dtype, s.args, s.plan = q_shape, out_dtype, N.DaArgs(), N.DaPlan()
    s.workspace = Fake((4096,), torch.uint8)
    return s


def test_a_step_takes_its_own_shapes_alone(launches):
    s = step()
    s(Fake((3, 8, 128)), Fake((3, 8, 128)))
    assert len(launches) == 1
    for q, out in ((Fake((2, 8, 128)), None), (Fake((3, 8, 128), torch.float16), None),
                   (Fake((3, 8, 128), device=torch.device("cuda", 1)), None),
                   (Fake((3, 8, 128)), Fake((3, 8, 128), torch.bfloat16)),
                   (Fake((3, 8, 128)), Fake((2, 8, 128))),
                   (Fake((3, 8, 128)), Fake((3, 8, 128), stride=(1, 3, 24))),
                   (Fake((3, 8, 128)), Fake((3, 8, 128), device=torch.device("cpu")))):
        with pytest.raises((TypeError, ValueError)):
            s(q, out)
    assert len(launches) == 1


def append(new=(5, 2, 128), pool=POOL, src=torch.bfloat16, **kw):
    t = dict(k_new=Fake(new, src), v_new=Fake(new, src), k=Fake(pool, E4), v=Fake(pool, E4),
             ks=Fake(pool[::2][:2]), vs=Fake(pool[::2][:2]), slots=Fake(new[:1], torch.int64))
    a = A.make_append(t["k_new"], t["v_new"], t["k"], t["v"], t["ks"], t["vs"])
    t.update(kw)
    A.decode_attn_append_8bit(t.get("append", a), t["k_new"], t["v_new"], t["slots"], t["k"],
                              t["v"], t["ks"], t["vs"])
    return a


def test_append_takes_what_it_was_made_for(launches):
    a = append()
    by_hand = N.DaAppend.from_buffer_copy(a)
    append(append=by_hand)
    assert len(launches) == 2
    with pytest.raises(ValueError):
        append(append=by_hand, k_new=Fake((5, 2, 128), torch.float32))


@pytest.mark.parametrize("kw", [
    dict(k_new=Fake((4, 2, 128), torch.bfloat16)), dict(v_new=Fake((5, 2, 64), torch.bfloat16)),
    dict(k_new=Fake((5, 2, 128), torch.float32), v_new=Fake((5, 2, 128), torch.float32)),
    dict(k_new=Fake((5, 2, 128), torch.bfloat16, (512, 128, 1))),
    dict(k=Fake((39, 16, 2, 128), E4)), dict(v=Fake(POOL, E5)), dict(k=Fake(POOL, E5), v=Fake(POOL, E5)),
    dict(ks=Fake((39, 2))), dict(vs=Fake((40, 2), torch.float16)), dict(vs=Fake((40, 2), stride=(1, 40))),
    dict(slots=Fake((4,), torch.int64)), dict(slots=Fake((5,), torch.int32)),
    dict(ks=Fake((40, 2), device=torch.device("cuda", 1)))])
def test_append_refuses_other_tensors_than_described(launches, kw):
    with pytest.raises((TypeError, ValueError)):
        append(**kw)
    assert not launches


def test_a_cache_appends_rows_of_its_device_alone(launches):
    c = C.PagedCache8.__new__(C.PagedCache8)
    c.k, c.v, c.k_scale, c.v_scale = Fake(POOL, E4), Fake(POOL, E4), Fake((40, 2)), Fake((40, 2))
    c.slot_map, c._shapes, c._append = Fake((5,), torch.int64), None, None
    rows = [Fake((5, 2, 128), torch.float16, device=torch.device("cuda", i)) for i in (0, 0, 1)]
    c.append(rows[0], rows[1])
    assert len(launches) == 1
    for k, v in ((rows[0], rows[2]), (rows[2], rows[0])):
        with pytest.raises(ValueError):
            c.append(k, v)
    assert len(launches) == 1


@pytest.mark.parametrize("kw", [
    dict(lens=Fake((2,), torch.int32)), dict(table=Fake((2, 10), torch.int32)),
    dict(ks=Fake((39, 2))), dict(vs=Fake((40, 1)))])
def test_attention_refuses_descriptors_that_hold_too_little(launches, kw):
    t = dict(lens=Fake((3,), torch.int32), table=Fake((3, 10), torch.int32), ks=Fake((40, 2)),
             vs=Fake((40, 2)))
    t.update(kw)
    q, k, v, out = Fake((3, 8, 128)), Fake(POOL, E4), Fake(POOL, E4), Fake((3, 8, 128))
    a = A.make_paged_args(q, k, v, 0.1, 10)
    dev = A.make_dev(seq_lens=t["lens"], block_table=t["table"], k_pool=k, v_pool=v)
    with pytest.raises(ValueError):
        A.decode_attn_splitk_8bit(a, N.DaPlan(), dev, A.make_scales(t["ks"], t["vs"]), q, k, v,
                                  out, Fake((4096,), torch.uint8))
    assert not launches


OTHER = torch.device("cuda", 1)


@pytest.mark.parametrize("kw", [
    dict(lens=Fake((3,), torch.int32, device=OTHER)),
    dict(table=Fake((3, 10), torch.int32, device=OTHER)),
    dict(lens=Fake((3,), torch.int32, device=OTHER), table=Fake((3, 10), torch.int32, device=OTHER)),
    dict(ks=Fake((40, 2), device=OTHER), vs=Fake((40, 2), device=OTHER)),
    dict(vs=Fake((40, 2), device=OTHER))])
def test_attention_refuses_descriptors_of_another_device(launches, kw):
    t = dict(lens=Fake((3,), torch.int32), table=Fake((3, 10), torch.int32), ks=Fake((40, 2)),
             vs=Fake((40, 2)))
    t.update(kw)
    q, k, v, out = Fake((3, 8, 128)), Fake(POOL, E4), Fake(POOL, E4), Fake((3, 8, 128))
    a = A.make_paged_args(q, k, v, 0.1, 10)
    dev = A.make_dev(seq_lens=t["lens"], block_table=t["table"], k_pool=k, v_pool=v)
    with pytest.raises(ValueError):
        A.decode_attn_splitk_8bit(a, N.DaPlan(), dev, A.make_scales(t["ks"], t["vs"]), q, k, v,
                                  out, Fake((4096,), torch.uint8))
    assert not launches


def test_tables_of_another_device_are_refused(launches):
    t = A.make_tables(Fake((3,), torch.int32), Fake((3, 10), torch.int32),
                      Fake((40,), torch.int32), Fake((4,), torch.int32), 16)
    A.decode_attn_grow_tables(t, Fake((3,), torch.int32), Fake((9,), torch.int64))
    assert len(launches) == 1
    with pytest.raises(ValueError):
        A.decode_attn_grow_tables(t, Fake((3,), torch.int32, device=OTHER),
                                  Fake((9,), torch.int64, device=OTHER))
    assert len(launches) == 1


class Shared:
    """A cache whose tables another shares, as far as the other looks at it."""

    def __init__(self, device=torch.device("cpu"), batch=3, width=10, rows=6):
        self.block_size = 16
        self.free_list = torch.zeros(40, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.block_table = torch.zeros(batch, width, dtype=torch.int32, device=device)
        self.slot_map = torch.zeros(rows, dtype=torch.int64, device=device)
        self.state, self.cu_new, self.tables = None, None, None


def share(of, **kw):
    """A cache on the CPU, as far as its tables; make_dev and make_scales refuse CPU tensors."""
    args = dict(max_batch=3, num_blocks=40, max_blocks_per_seq=10, n_kv_heads=2, head_dim=128,
                block_size=16, device="cpu")
    args.update(kw)
    return C.PagedCache8(tables_of=of, **args)


@pytest.mark.parametrize("kw,of", [
    (dict(max_batch=4), {}), (dict(max_blocks_per_seq=9), {}), (dict(max_new=5), {}),
    (dict(block_size=32), {}), (dict(num_blocks=41), {}), ({}, dict(device="meta"))])
def test_caches_that_share_tables_agree_in_them(monkeypatch, kw, of):
    monkeypatch.setattr(A, "make_dev", lambda **kw: N.DaDev())
    monkeypatch.setattr(A, "make_scales", lambda *x: N.DaScales())
    for right in ({}, dict(max_new=6)):
        assert share(Shared(), **right).slot_map.numel() == 6
    with pytest.raises(ValueError):
        share(Shared(**of), **kw)


@pytest.mark.parametrize("state", [Fake((2,), torch.int32), Fake((8,), torch.int32, (2,)),
                                   Fake((4,), torch.int32, (2,)), Fake((4,), torch.int64),
                                   Fake((4,), torch.int32, device=torch.device("cpu"))])
def test_the_status_wants_a_state_of_four_words(launches, state):
    with pytest.raises((TypeError, ValueError)):
        A.decode_attn_tables_status(state)
    assert not launches
    A.decode_attn_tables_status(Fake((4,), torch.int32))
    assert len(launches) == 1
