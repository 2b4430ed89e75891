"""Rotated appends (decode_attn_rope_append) against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from tests.prep_util import bound, normed, rotated

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    """New rows as parts of a fused projection, pools full of a pattern, slots in any order."""

    def __init__(self, T, hq, hkv, d, *, dv=None, page=16, src="bf16", cache="bf16", q_out="bf16",
                 rot=None, axes=None, interleaved=False, factor=1.0, norm=True, weights="row",
                 offset=0.0, w="f32", far=4096, lo=0, seed=0, slots=None, strided_pool=False,
                 theta=10000.0):
        g = torch.Generator().manual_seed(seed)
        dv = dv or d
        rot = d if rot is None else rot
        self.names = src, cache, q_out
        fused = torch.randn(T, hq * d + hkv * d + hkv * dv, generator=g) * 1.5
        fused = fused.to(DT[src]).cuda()
        self.q = fused[:, :hq * d].unflatten(1, (hq, d))
        self.k = fused[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        self.v = fused[:, (hq + hkv) * d:].unflatten(1, (hkv, dv))
        half = rot // 2
        self.inv_freq = [theta ** (-i / max(half, 1)) for i in range(half)]
        self.axes = axes or [0] * half
        self.n_axes = max(self.axes, default=0) + 1
        self.pos = torch.randint(lo, far, (self.n_axes, T), generator=g)
        self.interleaved, self.factor, self.norm, self.offset = interleaved, factor, norm, offset
        self.eps = 1e-5 if norm else None
        self.qw = self.kw = None
        if norm and weights != "none":
            shape = {"row": lambda h: (d,), "heads": lambda h: (h, d)}[weights]
            self.qw = (torch.randn(shape(hq), generator=g) * 0.3 + 1 - offset).to(DT[w]).cuda()
            self.kw = (torch.randn(shape(hkv), generator=g) * 0.3 + 1 - offset).to(DT[w]).cuda()
        nb = -(-T // page) + 2
        self.page, self.nb = page, nb
        if slots is None:
            slots = torch.randperm(nb * page, generator=g)[:T].tolist()
        self.slots = slots
        if strided_pool:                          # head-major pages, padded rows
            room = torch.zeros(2, nb, hkv, page + 1, max(d, dv) + 8, dtype=DT[cache], device="cuda")
            self.kp = room[0][:, :, :page, :d].permute(0, 2, 1, 3)
            self.vp = room[1][:, :, :page, :dv].permute(0, 2, 1, 3)
        else:
            self.kp = torch.zeros(nb, page, hkv, d, dtype=DT[cache], device="cuda")
            self.vp = torch.zeros(nb, page, hkv, dv, dtype=DT[cache], device="cuda")
        self.kp.fill_(7.0)
        self.vp.fill_(-3.0)
        self.qo = torch.full((T, hq, d), 5.0, dtype=DT[q_out], device="cuda")
        self.rope = A.make_rope(self.inv_freq, axes=axes, interleaved=interleaved, factor=factor)

    def prep(self):
        return A.make_prep(self.q, self.k, self.v, self.qo, self.kp, self.vp, self.rope,
                           q_weight=self.qw, k_weight=self.kw, eps=self.eps,
                           weight_offset=self.offset)

    def run(self, stream=None):
        slots = None if self.slots is None else \
            torch.tensor(self.slots, dtype=torch.int64, device="cuda")
        A.decode_attn_rope_append(self.prep(), self.q, self.k, self.v, self.pos.cuda(), slots,
                                  self.qo, self.kp, self.vp, stream)
        torch.cuda.synchronize()

    def want(self, x, w):
        y = x.double().cpu().numpy()
        if self.norm:
            y = normed(y, None if w is None else w.double().cpu().numpy(), self.eps, self.offset)
        return rotated(y, self.pos.tolist(), self.inv_freq, self.axes, self.interleaved,
                       self.factor)

    def check(self):
        src, cache, q_out = self.names
        zq, mq = self.want(self.q, self.qw)
        zk, mk = self.want(self.k, self.kw)
        v = self.v.to(DT[cache]).double().cpu().numpy()
        self.run()
        near(self.qo.double().cpu().numpy(), zq, mq, q_out)
        k, vv = self.kp.double().cpu().numpy(), self.vp.double().cpu().numpy()
        left = np.ones((self.nb, self.page), bool)
        slots = range(len(zk)) if self.slots is None else self.slots
        for t, s in enumerate(slots):
            if 0 <= s < self.nb * self.page:
                blk, at = divmod(s, self.page)
                near(k[blk, at], zk[t], mk[t], cache)
                np.testing.assert_array_equal(vv[blk, at], v[t])
                left[blk, at] = False
        assert (k[left] == 7.0).all() and (vv[left] == -3.0).all()


def near(got, want, mag, dtype):
    err, tol = np.abs(got - want), bound(want, mag, dtype)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (float((err / tol).max()), np.unravel_index((err / tol).argmax(),
                                                                        err.shape))


@pytest.mark.parametrize("cache", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,hq,hkv,d", [(1, 8, 2, 128), (33, 4, 4, 256), (7, 3, 1, 64)])
def test_types(T, hq, hkv, d, src, cache):
    Case(T, hq, hkv, d, src=src, cache=cache, q_out={"f32": "f16", "f16": "bf16", "bf16": "f32"}[src],
         seed=T).check()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (256, 64), (80, 80), (80, 32), (96, 16),
                                   (8, 0), (16, 16), (192, 128), (248, 240), (128, 0)])
def test_widths_and_partial_rotation(d, rot, interleaved):
    Case(19, 5, 2, d, rot=rot, interleaved=interleaved, src="f32", cache="f32", q_out="f32",
         seed=d + rot).check()


@pytest.mark.parametrize("T,hq,hkv,d,dv,rot,kw", [
    (1301, 2, 1, 256, 256, 256, dict(src="f16", cache="f16", q_out="f16")),
    (1216, 1, 3, 256, 256, 0, dict(src="bf16", cache="f32", q_out="f32", norm=False)),
    (1250, 1, 1, 208, 256, 16, dict(src="f16", cache="bf16", q_out="f32", w="bf16", offset=1.0)),
    (2435, 3, 2, 128, 128, 64, dict(interleaved=True, cache="bf16", q_out="f32", weights="heads")),
    (4901, 2, 1, 48, 64, 32, dict(src="f16", cache="f32", q_out="bf16", weights="none")),
    (4870, 1, 1, 56, 56, 48, dict(src="f16", cache="f16", q_out="f16")),   # half a lane over: narrow
])
def test_long_prompts(T, hq, hkv, d, dv, rot, kw):
    # enough rows of 16 bits that a lane takes 16 columns
    slots = torch.randperm(T + 32, generator=torch.Generator().manual_seed(T))[:T].tolist()
    slots[T // 2] = -1
    Case(T, hq, hkv, d, dv=dv, rot=rot, slots=slots, seed=rot, **kw).check()


@pytest.mark.parametrize("norm,weights,offset,w", [(False, "none", 0.0, "f32"),
                                                   (True, "none", 1.0, "f32"),
                                                   (True, "row", 1.0, "bf16"),
                                                   (True, "heads", 0.0, "f16"),
                                                   (True, "heads", 1.0, "f32")])
def test_norms(norm, weights, offset, w):
    Case(21, 6, 3, 128, norm=norm, weights=weights, offset=offset, w=w, src="f16", cache="f16",
         q_out="f32").check()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [[0] * 8 + [1] * 12 + [2] * 12, [i % 3 for i in range(32)],
                                  [7 - i // 4 for i in range(32)], [1] * 32])
def test_axes(axes, interleaved):
    Case(40, 4, 2, 128, rot=64, axes=axes, interleaved=interleaved, factor=1.25, src="f32",
         cache="f32", q_out="f32").check()


@pytest.mark.parametrize("lo,far", [(1 << 20, (1 << 20) + 50), (-70000, -1), ((1 << 24) - 3, 1 << 24)])
def test_far_and_negative_positions(lo, far):
    # (the reference's own products are exact to 2^-29 of a turn up to 2^24 positions)
    Case(16, 2, 1, 128, lo=lo, far=far, src="f32", cache="f32", q_out="f32").check()


def test_positions_past_32_bits():
    # frequencies that are whole fractions of a turn, so that the angle is known exactly
    c = Case(4, 2, 1, 64, rot=16, norm=False, src="f32", cache="f32", q_out="f32")
    c.pos = torch.tensor([[(1 << 40) + 1, 3 - (1 << 36), (1 << 50) + 2, 1 << 33]])
    c.rope.table.copy_(torch.tensor([1 << (61 - i) for i in range(8)]))
    c.run()
    x, z = c.q.double().cpu().numpy(), c.qo.double().cpu().numpy()
    for t, p in enumerate(c.pos[0].tolist()):
        for i in range(8):
            angle = 2 * math.pi * ((p << (61 - i)) % (1 << 64)) / 2.0 ** 64
            a, b = x[t, :, i], x[t, :, i + 8]
            tol = 8 * 2.0 ** -24 * (np.abs(a) + np.abs(b))
            assert (np.abs(z[t, :, i] - (a * math.cos(angle) - b * math.sin(angle))) <= tol).all()
            assert (np.abs(z[t, :, i + 8] - (b * math.cos(angle) + a * math.sin(angle))) <= tol).all()


@pytest.mark.parametrize("T,hq,hkv,d,page", [(1, 1, 1, 128, 16), (2, 128, 8, 128, 64),
                                             (300, 1, 1, 16, 5), (257, 2, 1, 8, 48),
                                             (1000, 16, 4, 256, 64), (4096, 4, 1, 128, 100)])
def test_sizes(T, hq, hkv, d, page):
    Case(T, hq, hkv, d, page=page, rot=min(d, 16) if d > 8 else 0, seed=T).check()


def test_skipped_rows_leave_the_pools_and_still_give_q():
    page, nb = 16, 3
    slots = [5, -1, 17, nb * page, 1 << 40, -(1 << 40), nb * page - 1, 0, -1]
    Case(len(slots), 4, 2, 128, page=page, slots=slots).check()


def test_values_of_another_width_and_strided_pools():
    Case(50, 4, 2, 128, dv=64, strided_pool=True).check()
    Case(50, 4, 2, 64, dv=128, strided_pool=True, src="f32", cache="f32").check()


def test_q_in_place():
    c = Case(37, 8, 2, 128, src="bf16", q_out="bf16")
    zq, mq = c.want(c.q, c.qw)
    c.qo = c.q
    c.run()
    near(c.q.double().cpu().numpy(), zq, mq, "bf16")


def test_q_in_place_of_a_long_prompt():
    c = Case(2433, 3, 1, 128, src="f16", q_out="f16")
    zq, mq = c.want(c.q, c.qw)
    c.qo = c.q
    c.run()
    near(c.q.double().cpu().numpy(), zq, mq, "f16")


def test_without_a_slot_map_rows_go_to_plain_buffers():
    c = Case(32, 4, 2, 128, page=32)
    c.slots = None
    c.check()


def test_rows_that_are_no_numbers_stay_with_their_heads():
    c = Case(6, 4, 2, 128, src="f32", cache="f32", q_out="f32")
    c.q[2, 1, 5] = math.nan
    c.k[3, 0, 7] = math.inf
    c.v[4, 1, 9] = -math.inf
    c.run()
    good = torch.isfinite(c.qo).all(-1)
    assert not good[2, 1] and good.sum() == good.numel() - 1
    k = c.kp.reshape(-1, 2, 128)[c.slots]
    ok = torch.isfinite(k).all(-1)
    assert not ok[3, 0] and ok.sum() == ok.numel() - 1
    v = c.vp.reshape(-1, 2, 128)[c.slots]
    assert v[4, 1, 9] == -math.inf and torch.isfinite(v).sum() == v.numel() - 1


def test_a_row_of_zeros():
    c = Case(3, 2, 1, 64, src="f32", cache="f32", q_out="f32")
    c.q.zero_()
    c.run()
    assert (c.qo == 0).all()


def test_streams_and_graphs():
    c = Case(64, 8, 2, 128)
    s = torch.cuda.Stream()
    prep, pos = c.prep(), c.pos.cuda()
    slots = torch.tensor(c.slots, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    call = lambda: A.decode_attn_rope_append(prep, c.q, c.k, c.v, pos, slots, c.qo, c.kp, c.vp)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    first = c.qo.clone(), c.kp.clone(), c.vp.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    # new rows, positions and slots in the same buffers
    c.q.mul_(1.5)
    pos.add_(3)
    slots.copy_(slots.flip(0))
    for t in (c.qo, c.kp, c.vp):
        t.fill_(2.0)
    g.replay()
    torch.cuda.synchronize()
    replayed = c.qo.clone(), c.kp.clone(), c.vp.clone()
    for t in (c.qo, c.kp, c.vp):
        t.fill_(2.0)
    call()
    torch.cuda.synchronize()
    for a, b, f in zip(replayed, (c.qo, c.kp, c.vp), first):
        assert torch.equal(a, b) and not torch.equal(a, f)


def test_no_tokens():
    c = Case(1, 2, 1, 64)
    c.q, c.k, c.v, c.qo = c.q[:0], c.k[:0], c.v[:0], c.qo[:0]
    c.pos, c.slots = c.pos[:, :0].contiguous(), []
    c.run()
    assert (c.kp == 7.0).all()
