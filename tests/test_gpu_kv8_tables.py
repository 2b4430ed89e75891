"""Block tables and slot maps grown on the GPU (decode_attn_grow_tables), against
Python lists: random loads of growing, idle and released sequences, exhaustion,
overflows, in place and beside, large batches of prompts, captured and replayed."""
import random

import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from tests.kv8_util import Blocks

pytestmark = pytest.mark.gpu


class Device:
    def __init__(self, batch, num_blocks, width, page, capacity):
        def ints(*s):
            return torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.lens, self.table = ints(batch), ints(batch, width)
        self.free = torch.arange(num_blocks - 1, -1, -1, dtype=torch.int32, device="cuda")
        self.state = ints(4)
        self.state[0] = num_blocks
        self.slots = torch.full((capacity,), 77, dtype=torch.int64, device="cuda")
        self.cu = torch.full((batch + 1,), 77, dtype=torch.int32, device="cuda")
        self.t = A.make_tables(self.lens, self.table, self.free, self.state, page)

    def grow(self, new):
        new = torch.tensor(new, dtype=torch.int32, device="cuda")
        A.decode_attn_grow_tables(self.t, new, self.slots, self.cu)

    def check(self, ref, slots, cu, status=0):
        assert self.state.tolist() == [len(ref.free), status, 0, 0]
        assert self.lens.tolist() == ref.lens
        assert self.slots.tolist() == slots
        assert self.cu.tolist() == cu
        assert self.free[:len(ref.free)].tolist() == ref.free
        table = self.table.tolist()
        for b, r in enumerate(ref.rows):
            assert table[b][:len(r)] == r


@pytest.mark.parametrize("batch,num_blocks,width,page,capacity,most", [
    (1, 3, 3, 16, 5, 5), (7, 40, 9, 16, 64, 20), (32, 500, 20, 1, 300, 12),
    (256, 4000, 30, 64, 4000, 100), (33, 3000, 200, 48, 20000, 900),
    (5, 2, 8, 1000, 40, 10)])
def test_random_loads(batch, num_blocks, width, page, capacity, most):
    rng = random.Random(batch)
    ref, dev = Blocks(batch, num_blocks, width, page), Device(batch, num_blocks, width, page,
                                                              capacity)
    seen = set()
    for step in range(40):
        new = [rng.choice([0, 1, 1, rng.randint(0, most), rng.randint(0, most), -1])
               for _ in range(batch)]
        if step == 39:
            new = [-3] * batch                    # everything goes back
        status, slots, cu = ref.grow(new, capacity)
        dev.grow(new)
        dev.check(ref, slots, cu, status)
        seen.add(status)
        if status:
            with pytest.raises(A.DecodeAttnError) as e:
                A.decode_attn_tables_status(dev.state)
            assert e.value.status == status
        A.decode_attn_tables_status(dev.state)    # read once, then clear
    assert len(ref.free) == num_blocks and sorted(ref.free) == list(range(num_blocks))


@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("shift", [0, 1])
def test_prompts_of_a_full_batch(page, shift):
    # over 155,648 slots a lane takes several; with an odd start they are stored one by one
    rng = random.Random(page)
    ref, dev = Blocks(256, 100000, 700, page), Device(256, 100000, 700, page, 200001)
    room = torch.full((200004,), 77, dtype=torch.int64, device="cuda")
    dev.slots = room[shift:shift + 200001]
    for step in range(3):
        new = [rng.choice([0, 1, 2, rng.randint(0, 700), rng.randint(400, 2000)]) for _ in range(256)]
        if step == 1:
            new = [-1 if b % 3 == 0 else 1 for b in range(256)]
        status, slots, cu = ref.grow(new, 200001)
        dev.grow(new)
        dev.check(ref, slots, cu, status)
    assert room[200001 + shift:].eq(77).all() and room[:shift].eq(77).all()


def test_the_first_failure_is_kept_and_nothing_changes():
    ref, dev = Blocks(3, 4, 8, 16), Device(3, 4, 8, 16, 200)
    status, slots, cu = ref.grow([20, 5, 0], 200)
    dev.grow([20, 5, 0])
    dev.check(ref, slots, cu)
    dev.grow([0, 0, 40])                          # three blocks, one left
    dev.check(ref, [-1] * 200, [0] * 4, N.DA_ENOSPACE)
    dev.grow([0, 0, 500])                         # too many rows: the first status stays
    dev.check(ref, [-1] * 200, [0] * 4, N.DA_ENOSPACE)
    status, slots, cu = ref.grow([1, 1, 1], 200)  # a later call that can be served is
    dev.grow([1, 1, 1])
    dev.check(ref, slots, cu, N.DA_ENOSPACE)
    with pytest.raises(A.DecodeAttnError):
        A.decode_attn_tables_status(dev.state)
    A.decode_attn_tables_status(dev.state)


@pytest.mark.parametrize("state,lens", [([99, 0, 0, 0], 0), ([-1, 0, 0, 0], 0), ([4, 0, 0, 0], -7)])
def test_a_state_that_is_not_one_is_refused_on_the_device(state, lens):
    dev = Device(3, 4, 8, 16, 9)
    dev.state.copy_(torch.tensor(state))
    dev.lens[1] = lens
    before = dev.table.clone(), dev.free.clone()
    dev.grow([1, 1, 1])
    assert dev.slots.tolist() == [-1] * 9 and dev.state[1].item() == N.DA_EINVAL
    assert torch.equal(before[0], dev.table) and torch.equal(before[1], dev.free)


def test_lengths_at_the_int32_limit_do_not_wrap():
    # 2^31 - 3 positions in pages of 2^24: one more token is the last that fits
    page, width = 1 << 24, 200
    dev = Device(1, 3, width, page, 8)
    dev.lens[0] = 2 ** 31 - 3
    dev.grow([5])
    assert dev.state[1].item() == N.DA_EINVAL and dev.slots.tolist() == [-1] * 8
    dev.state[1] = 0
    dev.table[0, 127] = 2
    dev.grow([2])
    assert dev.lens.item() == 2 ** 31 - 1 and dev.state[1].item() == 0
    assert dev.slots.tolist()[:2] == [2 * page + page - 3, 2 * page + page - 2]


def test_slots_past_32_bits():
    page = 1 << 20
    dev = Device(2, 5000, 4, page, 4)
    dev.free[4999] = 4999                         # the top of the stack: the pool's last block
    dev.grow([2, 0])
    assert dev.slots.tolist() == [4999 * page, 4999 * page + 1, -1, -1]


def test_beside_the_old_lengths_it_can_be_asked_again():
    lens = torch.tensor([5, 16, 0], dtype=torch.int32, device="cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda").reshape(3, 4).contiguous()
    free = torch.arange(20, 40, dtype=torch.int32, device="cuda")
    state = torch.tensor([20, 0, 0, 0], dtype=torch.int32, device="cuda")
    lens_out, state_out = torch.zeros_like(lens), torch.zeros_like(state)
    t = A.make_tables(lens, table, free, state, 16, seq_lens_out=lens_out, state_out=state_out)
    slots = torch.empty(100000, dtype=torch.int64, device="cuda")   # many CTAs
    new = torch.tensor([30, 1, -1], dtype=torch.int32, device="cuda")
    got = []
    for _ in range(2):
        A.decode_attn_grow_tables(t, new, slots)
        got.append([x.clone() for x in (table, free, lens_out, state_out, slots)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert lens.tolist() == [5, 16, 0] and state.tolist() == [20, 0, 0, 0]
    assert lens_out.tolist() == [35, 17, 0] and state_out.tolist() == [17, 0, 0, 0]
    assert table[0, 1:3].tolist() == [39, 38] and table[1, 1].item() == 37


def test_released_blocks_are_taken_before_the_stack_in_one_call():
    ref, dev = Blocks(4, 12, 6, 4), Device(4, 12, 6, 4, 64)
    for new in ([9, 7, 3, 0], [-1, 2, -1, 13], [5, -2, 0, 0], [-1, 20, -1, -1]):
        status, slots, cu = ref.grow(new, 64)
        dev.grow(new)
        dev.check(ref, slots, cu, status)


def test_captured_once_and_replayed():
    ref, dev = Blocks(8, 300, 16, 16), Device(8, 300, 16, 16, 200)
    new = torch.zeros(8, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.decode_attn_grow_tables(dev.t, new, dev.slots, dev.cu)
    rng = random.Random(3)
    for _ in range(12):
        want = [rng.choice([0, 1, 3, 17, -1]) for _ in range(8)]
        new.copy_(torch.tensor(want))
        g.replay()
        status, slots, cu = ref.grow(want, 200)
        dev.check(ref, slots, cu, status)


def test_without_slots_or_offsets():
    dev = Device(3, 9, 4, 16, 0)
    A.decode_attn_grow_tables(dev.t, torch.tensor([0, -1, 0], dtype=torch.int32, device="cuda"),
                              dev.slots)
    assert dev.state.tolist() == [9, 0, 0, 0]
    dev.grow([1, 0, 0])                           # a token, and no slot for it
    assert dev.state.tolist() == [9, N.DA_EINVAL, 0, 0] and dev.lens.tolist() == [0, 0, 0]


def test_refusals():
    dev = Device(3, 9, 4, 16, 8)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        A.decode_attn_grow_tables(dev.t, new.long(), dev.slots)
    with pytest.raises(TypeError):
        A.decode_attn_grow_tables(dev.t, new[:2], dev.slots)
    with pytest.raises(TypeError):
        A.decode_attn_grow_tables(dev.t, new, dev.slots.int())
    with pytest.raises(TypeError):
        A.decode_attn_grow_tables(dev.t, new, dev.slots, dev.cu[:3])
    with pytest.raises(ValueError):
        A.decode_attn_grow_tables(dev.t, new, dev.slots.cpu())
    with pytest.raises(ValueError):
        A.make_tables(dev.lens[:2], dev.table, dev.free, dev.state, 16)
    with pytest.raises(ValueError):
        A.make_tables(dev.lens, dev.table.t(), dev.free, dev.state, 16)
    with pytest.raises(TypeError):
        A.make_tables(dev.lens.cpu(), dev.table, dev.free, dev.state, 16)
    bad = A.make_tables(dev.lens, dev.table, dev.free, dev.state, 0)
    with pytest.raises(A.DecodeAttnError) as e:
        A.decode_attn_grow_tables(bad, new, dev.slots)
    assert e.value.status == N.DA_EINVAL and "block_size" in e.value.message
