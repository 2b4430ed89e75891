"""Scored attention (decode_attn_splitk_scored) against its formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from tests.scored_util import Case, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache,q", [("bf16", "same"), ("bf16", "f32"), ("f16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("d", [128, 256])
def test_plain_scores_of_every_type(d, cache, q, out):
    Case([300], 8, 2, d, cache=cache, q=q, out=out).check()


@pytest.mark.parametrize("L", [1, 2, 15, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_lengths(d, L, out):
    Case([L], 4, 2, d, out=out, page=0 if L % 2 else 32, seed=L).check()


@pytest.mark.parametrize("hq,hkv,q_len", [(1, 1, 1), (3, 1, 1), (8, 8, 1), (12, 1, 1), (24, 4, 4),
                                          (32, 1, 4), (33, 1, 3), (64, 1, 2), (2, 1, 64), (6, 2, 5)])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("cache,q,out", [("bf16", "same", "bf16"), ("bf16", "f32", "f32"),
                                         ("f16", "f32", "f16")])
def test_head_layouts_and_new_tokens(d, hq, hkv, q_len, cache, q, out):
    Case([q_len, 200 + q_len, 97 + q_len], hq, hkv, d, q_len=q_len, cache=cache, q=q, out=out).check()


@pytest.mark.parametrize("page", [0, 16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("d", [128, 256])
def test_pages(d, page):
    Case([519, 1, 260, 64, 16], 4, 2, d, page=page, cache="f16", q="f32").check()


@pytest.mark.parametrize("page", [0, 48])
def test_head_major_caches(page):
    Case([300, 77], 8, 2, 128, page=page, head_major=True).check()


@pytest.mark.parametrize("splits", [1, 2, 3, 7])
@pytest.mark.parametrize("q_len", [1, 3])
def test_forced_splits(splits, q_len):
    Case([777, 130, 5], 8, 2, 128, q_len=q_len, force_splits=splits, cap=20.0).check()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
@pytest.mark.parametrize("cap,spread", [(1.0, 3.0), (30.0, 1.0), (50.0, 8.0), (0.25, 0.1)])
def test_softcap(cap, spread, cache, out):
    Case([400, 33], 8, 2, 128, cap=cap, spread=spread, cache=cache, q="f32", out=out).check()


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("d", [128, 256])
def test_bias_by_distance(d, cap, q_len):
    Case([700, 64, 129], 8, 2, d, slopes=True, cap=cap, q_len=q_len, cache="f16", q="f32").check()


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 129, 200, 500, 5000])
@pytest.mark.parametrize("q_len", [1, 4])
def test_windows(window, q_len):
    Case([700, 64, 129, 300], 8, 2, 128, window=window, q_len=q_len, out="f32").check()


@pytest.mark.parametrize("window,keep", [(1, 1), (64, 64), (100, 4), (100, 300), (130, 130), (0, 50),
                                         (33, 128), (500, 1000)])
@pytest.mark.parametrize("q_len", [1, 5])
@pytest.mark.parametrize("d", [128, 256])
def test_windows_with_kept_positions(window, keep, q_len, d):
    Case([900, 64, 129, 301], 4, 1, d, window=window, keep=keep, q_len=q_len).check()


@pytest.mark.parametrize("window,keep", [(0, 0), (64, 0), (64, 100), (1, 3), (0, 80)])
@pytest.mark.parametrize("q_len", [1, 4])
def test_starts_and_kept_lengths(window, keep, q_len):
    lens = [500, 300, 129, 64, 256, 200]
    c = Case(lens, 8, 2, 128, window=window, keep=keep, q_len=q_len,
             starts=[0, 250, 127, 64, 63, 1000], keep_lens=[keep, 1000, 5, 64, 0, 30])
    got = c.check()
    assert (got[3] == 0).all() and (got[5] == 0).all()        # nothing left to see


@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_kept_positions_that_are_causal(q_len):
    # as make_score says: with keep_lens of at most S - q_len + 1 and a window of q_len or more no token
    # sees past itself, and every one the first `keep` positions up to itself
    keep, window = 8, 16

    class Causal(Case):
        def sees(self, b, i):
            j, o = np.arange(self.lens[b]), self.lens[b] - self.q_len + i
            return (j <= o) & ((j < keep) | (j > o - window))

    lens = [q_len, q_len + 1, 8, 9, 10, 11, 12, 40, 300]
    Causal(lens, 8, 2, 128, q_len=q_len, window=window, keep=keep,
           keep_lens=[n - q_len + 1 for n in lens]).check()


def test_what_is_not_seen_may_hold_anything():
    # evicted positions between the kept ones and the window, padding before the start
    for kw, spoil in ((dict(window=70, keep=20), range(20, 300 - 70 - 3)),
                      (dict(starts=[100], window=150), list(range(100)) + list(range(100, 147))),
                      (dict(starts=[131]), range(131))):
        for value in (math.nan, math.inf, -math.inf):
            for page in (0, 16):
                c = Case([300], 8, 2, 128, q_len=4, page=page, **kw)
                for j in spoil:
                    at = (0, j) if page == 0 else (int(c.table[0, j // 16]), j % 16)
                    c.k[at], c.v[at] = value, value
                want = c.want()
                assert np.isfinite(want[0]).all()
                c.check()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("cache,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_rows_that_are_no_numbers_reach_the_tokens_that_see_them(d, cache, out):
    # three new tokens; the second one's key or value, or a value at a window's lower end, is
    # not a number: the tokens that do not see it are as if it were not there
    for what, j in (("v", 298), ("k", 298), ("v", 299), ("v", 199), ("v", 198)):
        for value in (math.nan, math.inf):
            c = Case([300], 8, 2, d, q_len=3, window=100, cache=cache, out=out)
            at = (int(c.table[0, j // 16]), j % 16)
            getattr(c, what)[at][1, 7] = value      # KV head 1, column 7
            got = c.run()
            sees = [c.sees(0, i)[j] for i in range(3)]
            assert any(sees) and not all(sees)
            with np.errstate(all="ignore"):
                want, mag, top = c.want()
            clean = Case([300], 8, 2, d, q_len=3, window=100, cache=cache, out=out)
            tol = clean.bound(*clean.want())
            for i in range(3):
                for h in range(8):
                    if not sees[i] or h < 4:
                        near(got[0, i, h], want[0, i, h], tol[0, i, h])
                    elif what == "v":
                        # that column alone
                        assert not np.isfinite(got[0, i, h, 7])
                        cols = np.arange(d) != 7
                        near(got[0, i, h, cols], want[0, i, h, cols], tol[0, i, h, cols])
                    elif math.isnan(value):
                        assert np.isnan(got[0, i, h]).all()


@pytest.mark.parametrize("hq,q_len", [(2, 3), (4, 10), (30, 3)])
@pytest.mark.parametrize("d,cache,out", [(128, "bf16", "bf16"), (128, "bf16", "f32"), (128, "f16", "f16"),
                                         (256, "bf16", "bf16"), (256, "f16", "f32")])
def test_rows_that_are_no_numbers_stay_with_their_sequence(d, cache, out, hq, q_len):
    # one CTA works on sequences one after the other, packed rows, rows in copies and one copy of the
    # rows: where an item's first tile (and that of its other warpgroup) starts its sums with a value
    # that some of the tokens see, the last item's results are still read from there
    lens = [260, 40, 129, 140, 64, 250, 33, 131, 70, 200] * 3
    kw = dict(q_len=q_len, cache=cache, out=out, num_sms=1, force_splits=1, seed=d + hq)
    clean = Case(lens, hq, 1, d, **kw)
    tol = clean.bound(*clean.want())
    for value in (math.nan, math.inf):
        c = Case(lens, hq, 1, d, **kw)
        for b, n in enumerate(lens):
            if b % 3 == 2:                      # (numbers all through: nothing reaches them)
                continue
            for j in {n - 1, max(n - q_len + 1, 0)}:
                c.v[int(c.table[b, j // 16]), j % 16, 0, (5 * b) % d] = value
        with np.errstate(all="ignore"):
            want = c.want()[0]
        fine = np.isfinite(want)
        assert not fine.all() and fine[2::3].all()
        for _ in range(4):
            got = c.run()
            assert np.array_equal(np.isfinite(got), fine), np.argwhere(np.isfinite(got) != fine)[:5]
            near(np.where(fine, got, 0.0), np.where(fine, want, 0.0), tol)


def test_device_lengths_below_the_plan_and_unused_places():
    for kw in (dict(), dict(window=64, keep=16), dict(slopes=True, cap=9.0)):
        for q_len in (1, 3):
            c = Case([0, 1, 2, 700, 129, 3], 8, 2, 128, q_len=q_len,
                     max_lens=[900, 64, 300, 1000, 129, 2048], **kw)
            got = c.check()
            assert (got[0] == 0).all()
            if q_len == 3:                       # tokens before the sequence's start
                assert (got[1, :2] == 0).all() and (got[1, 2] != 0).any()


def test_many_sequences():
    rng = np.random.default_rng(1)
    Case(rng.integers(1, 300, 256).tolist(), 2, 1, 128).check()
    Case(rng.integers(1, 200, 100).tolist(), 16, 16, 128, cache="f16", out="f16").check()


@pytest.mark.parametrize("bad", [-1, 10 ** 9, "num_blocks"])
@pytest.mark.parametrize("d,shared", [(128, 0), (256, 0), (128, 64)])
def test_blocks_that_do_not_exist_read_as_zeros(d, shared, bad):
    c = Case([300, 50], 8, 2, d, shared=shared)
    o = c.setup()
    if bad == "num_blocks":
        bad = o.k.shape[0]
    o.table[0, 3] = o.table[1, 1] = bad
    if shared:
        o.shared_table[2] = bad
    ws, out = A.new_workspace(o.plan), torch.empty(o.q.shape, device="cuda")
    A.decode_attn_splitk_scored(o.args, o.plan, o.dev, o.score, o.q, o.k, o.v, out, ws)
    A.decode_attn_device_status(ws)
    for b, i in ((0, 3), (1, 1)):
        c.k[int(c.table[b, i])], c.v[int(c.table[b, i])] = 0.0, 0.0
    if shared:
        c.k[int(c.shared_table[2])], c.v[int(c.shared_table[2])] = 0.0, 0.0
    want, mag, top = c.want()
    near(out.double().cpu().numpy()[:, None], want, c.bound(want, mag, top))


def test_bounds_that_reach_past_everything():
    top = 2 ** 31 - 1
    for kw in (dict(window=top, keep=top), dict(keep=top), dict(window=1, keep=top, keep_lens=[-5, 0, top]),
               dict(window=1), dict(starts=[top, 0, 299], window=5), dict(starts=[-top, 300, 0], keep=9)):
        c = Case([300, 301, 300], 8, 2, 128, q_len=2, **kw)
        c.check()


# ---- shared positions

@pytest.mark.parametrize("shared,page", [(16, 16), (64, 32), (128, 64), (144, 48), (1024, 16),
                                         (1280, 256)])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("cache,q,out", [("bf16", "same", "bf16"), ("bf16", "f32", "f32"),
                                         ("f16", "f32", "f16"), ("f16", "same", "f32")])
def test_shared_positions(d, shared, page, cache, q, out):
    Case([33, 1, 160, 64, 200], 8, 2, d, page=page, shared=shared, cache=cache, q=q, out=out).check()


@pytest.mark.parametrize("batch,hq,hkv,q_len", [(1, 4, 1, 1), (2, 64, 1, 1), (33, 8, 2, 1),
                                                (70, 12, 3, 1), (9, 32, 1, 4), (130, 8, 1, 2),
                                                (3, 128, 1, 1), (256, 2, 1, 1)])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("q", ["same", "f32"])
def test_shared_rows_of_every_number(batch, hq, hkv, q_len, d, q):
    rng = np.random.default_rng(batch)
    Case((q_len + rng.integers(0, 60, batch)).tolist(), hq, hkv, d, q_len=q_len, shared=320, page=64,
         q=q, out="bf16").check()


def test_shared_positions_with_cap_and_bias():
    for q_len in (1, 3):
        Case([50, 3, 129], 8, 2, 128, q_len=q_len, shared=384, slopes=True, cap=15.0).check()
        Case([50, 3, 129], 8, 2, 256, q_len=q_len, shared=384, slopes=True, out="bf16").check()


def test_shared_positions_and_unused_places():
    # a place of length 0 gives zeros, and so do tokens before a sequence's first own position
    c = Case([0, 5, 1, 40], 8, 2, 128, q_len=2, shared=256, max_lens=[100, 60, 20, 40])
    got = c.check()
    assert (got[0] == 0).all() and (got[2, 0] == 0).all() and (got[2, 1] != 0).any()


@pytest.mark.parametrize("splits", [1, 2, 5])
def test_shared_positions_in_forced_splits(splits):
    Case([300, 20], 8, 2, 128, shared=640, force_splits=splits).check()
    Case([300, 20] * 20, 8, 1, 128, shared=640, force_splits=splits, out="bf16").check()


@pytest.mark.parametrize("sms", [1, 2, 5])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("shared", [0, 320])
def test_many_items_of_every_kind_on_one_cta(shared, d, sms):
    # items of two row tiles, of one, of one tile, without tiles, one after the other
    lens = [5, 0, 300, 64, 1, 900] * 6 + [129]
    for splits in (0, 3):
        c = Case(lens, 16, 2, d, shared=shared, page=64, num_sms=sms, force_splits=splits,
                 out="bf16", max_lens=[max(n, 200) for n in lens])
        c.check()
    Case(lens, 16, 2, d, shared=shared, page=64, num_sms=sms, q="f32").check()


# ---- numerics

def test_a_dominating_position_leaves_the_others():
    # one key scores 11.5 / ln 2 more than 4000 others; its value is 0, so the output is the
    # others' mean times their share. Weights of 2^-16.6 of the largest
    for cache, out in (("f16", "f32"), ("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")):
        for where in (0, 2000, 3999):
            c = Case([4000], 4, 1, 128, cache=cache, out=out, scale=1.0)
            c.q.zero_()
            c.q[..., 0] = 1.0
            c.k[..., 0] = 0.0
            c.v.copy_(torch.rand(c.v.shape, generator=c.g) + 1)
            at = (int(c.table[0, where // 16]), where % 16)
            c.k[at][..., 0] = 11.5
            c.v[at] = 0.0
            got, (want, mag, top) = c.run(), c.want()
            # every other weight is 2^-16.6 = 1e-5 of the largest: two bf16 terms keep 2^-17 of
            # themselves, f16 terms a step of 2^-24 - OFF = 2^-31, which is 2^-15 of them
            eps = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[out]
            near(got, want, np.abs(want) * (2.0 ** -13 + eps) + 2.0 ** -25)


def test_scores_that_rise_and_fall():
    # every tile exceeds the last, so that references move in each; and the other way round
    for order in (1, -1):
        for out in ("f32", "bf16"):
            c = Case([1500], 4, 1, 128, out=out, scale=1.0)
            c.q.normal_(generator=c.g).mul_(0.1)
            c.q[..., 0] = 1.0
            for j in range(1500):
                at = (int(c.table[0, j // 16]), j % 16)
                c.k[at][..., 0] = (j if order > 0 else 1500 - j) / 8.0
            c.check()


@pytest.mark.parametrize("hq,q_len,shared", [(4, 1, 0), (20, 1, 0), (24, 4, 0), (4, 1, 512)])
@pytest.mark.parametrize("cache,out", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("d", [128, 256])
def test_references_that_move_in_some_tiles(d, cache, out, hq, q_len, shared):
    # the largest score of a tile jumps up and down by up to 60, for each half of the heads at other
    # tiles, so that every warpgroup raises references that the other one goes on with
    rng = np.random.default_rng(d + hq)
    for slopes in (False, True):
        c = Case([1100, 129], hq, 1, d, q_len=q_len, shared=shared, cache=cache, out=out, scale=1.0,
                 force_splits=1, slopes=slopes)
        c.q.normal_(generator=c.g).mul_(0.05)
        c.q[:, :, ::2, 0], c.q[:, :, 1::2, 0] = 1.0, 0.0
        c.q[:, :, 1::2, 1], c.q[:, :, ::2, 1] = 1.0, 0.0
        for column in (0, 1):
            height = rng.permutation(np.linspace(0, 60, 40))
            c.k[..., column] = 0.0
            for b, n in enumerate(c.lens):
                for j in range(n):
                    if rng.random() < 0.1:
                        at = (int(c.table[b, j // 16]), j % 16)
                        c.k[at][..., column] = float(height[j // 32 % 40])
            for j in range(0, shared, 9):
                c.k[int(c.shared_table[j // 16]), j % 16, :, column] = float(height[j // 32])
        c.check()


def test_negative_and_zero_scales():
    Case([300, 5], 4, 2, 128, scale=-0.1).check()
    Case([300, 5], 4, 2, 128, scale=0.0).check()
    Case([300, 5], 4, 2, 256, scale=-0.1, cap=3.0, q_len=3).check()


def test_large_and_tiny_queries_beside_f16():
    for s in (1e-30, 1e-6, 1e4, 1e20):
        c = Case([200], 4, 2, 128, cache="f16", q="f32", scale=128 ** -0.5 / s)
        c.q.mul_(s)
        c.check()


def test_equal_results_in_every_run():
    c = Case([3000, 40, 777], 8, 2, 128, shared=512)
    first = c.run()
    for _ in range(3):
        np.testing.assert_array_equal(c.run(), first)


@pytest.mark.parametrize("cache,out", [("f16", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("cap", [0.5, 4.0, 1000.0])
def test_caps_near_and_far_in_one_tile(cap, cache, out):
    # scores of 2^-20 to 2^3 of the cap, in one tile and in tiles of their own: the series and
    # the quotient on both sides of a quarter
    c = Case([520], 4, 1, 128, cap=cap, cache=cache, q="f32", out=out, scale=1.0)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k[..., 1:] = 0.0
    for j in range(520):
        at = (int(c.table[0, j // 16]), j % 16)
        step = j % 24 if j < 256 else (j // 64) % 8 * 3
        c.k[at][..., 0] = cap * 2.0 ** (step - 20) * (-1) ** j
    c.check()


@pytest.mark.parametrize("cap", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("cache,out", [("f16", "f32"), ("bf16", "bf16")])
def test_caps_of_every_size(cap, cache, out):
    # (the smallest leave no score, the largest all of them; a query of zeros has scores of zero)
    c = Case([300, 40], 4, 1, 128, cap=cap, cache=cache, q="f32", out=out)
    c.q[:, :, 0] = 0.0
    if cap > 1:                                 # within 2^-40 of none: of that call's precision
        got = c.run()
        c.cap = 0.0
        want, mag, top = c.want()
        near(got, want, c.bound(want, mag, top))
    else:
        c.check()


# ---- streams, graphs, errors

def test_captured_steps_follow_lengths_tables_and_inputs():
    c = Case([100, 200, 0], 8, 2, 128, window=128, keep=8, max_lens=[700, 700, 700], poison=False,
             cache="f16", out="f32")
    o = c.setup()
    nb = 3 * 44 + 3
    g = torch.Generator().manual_seed(5)
    o.k, o.v = (torch.randn(nb, 16, 2, 128, generator=g).half().cuda() for _ in range(2))
    o.table = torch.zeros(3, 46, dtype=torch.int32, device="cuda")
    o.args = A.make_paged_args(o.q, o.k, o.v, c.scale, 46)
    o.dev = A.make_dev(seq_lens=o.lens, block_table=o.table, k_pool=o.k, v_pool=o.v)
    ws, out = A.new_workspace(o.plan), torch.empty(o.q.shape, device="cuda")
    call = lambda: A.decode_attn_splitk_scored(o.args, o.plan, o.dev, o.score, o.q, o.k, o.v, out, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([100, 200, 0], [129, 700, 1], [0, 65, 433], [700, 700, 700]):
        o.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        o.table.copy_(torch.randperm(nb, generator=g)[:3 * 44].view(3, 44).int().cuda()
                      [:, [min(i, 43) for i in range(46)]])
        o.q.normal_()
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        c.lens, c.q = lens, o.q.cpu()[:, None]
        c.k, c.v, c.table = o.k.cpu(), o.v.cpu(), o.table.cpu()
        c.shared_table = torch.zeros(0, dtype=torch.int32)
        want, mag, top = c.want()
        near(out.double().cpu().numpy()[:, None], want, c.bound(want, mag, top))


def test_two_graphs_share_a_workspace():
    cs = [Case([500, 60], 8, 2, 256, seed=i, q_len=2) for i in range(2)]
    ons, outs, graphs = [c.setup() for c in cs], [], []
    ws = A.new_workspace(ons[0].plan)
    for o in ons:
        out = torch.empty(o.q.shape, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            A.decode_attn_splitk_scored(o.args, o.plan, o.dev, o.score, o.q, o.k, o.v, out, ws)
        outs.append(out), graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for c, out in zip(cs, outs):
        want, mag, top = c.want()
        near(out.double().cpu().numpy().reshape(want.shape), want, c.bound(want, mag, top))


def test_two_streams_with_workspaces_of_their_own():
    cs = [Case([900, 30], 8, 2, 128, seed=i, shared=256) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    ons, outs = [c.setup() for c in cs], []
    for o in ons:
        o.ws = A.new_workspace(o.plan)
        outs.append(torch.empty(o.q.shape, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(5):
        for o, out, s in zip(ons, outs, streams):
            A.decode_attn_splitk_scored(o.args, o.plan, o.dev, o.score, o.q, o.k, o.v, out, o.ws, s)
    torch.cuda.synchronize()
    for c, out in zip(cs, outs):
        want, mag, top = c.want()
        near(out.double().cpu().numpy()[:, None], want, c.bound(want, mag, top))


def test_contiguous_caches_without_a_descriptor():
    c = Case([300, 200], 8, 2, 128, page=0)
    o = c.setup()
    ws, out = A.new_workspace(o.plan), torch.empty(o.q.shape, device="cuda")
    A.decode_attn_splitk_scored(o.args, o.plan, None, o.score, o.q, o.k, o.v, out, ws)
    want, mag, top = c.want()
    near(out.double().cpu().numpy()[:, None], want, c.bound(want, mag, top))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("shared", [0, 256])
def test_a_wait_that_runs_out_is_reported(d, shared):
    c = Case([300, 40], 8, 2, d, flags=N.DA_FLAG_TEST_NO_TMA, timeout_us=2000, shared=shared)
    with pytest.raises(A.DecodeAttnError) as e:
        c.run()
    assert e.value.status == N.DA_ETIMEOUT and "scored" in e.value.message
    c.flags = 0
    c.timeout_us = 0
    c.check()                                    # the context and the next call are fine


def test_a_refused_launch_is_reported():
    c = Case([300], 8, 2, 128, flags=N.DA_FLAG_TEST_BAD_LAUNCH)
    with pytest.raises(A.DecodeAttnError) as e:
        c.run()
    assert e.value.status == N.DA_ELAUNCH and e.value.message.startswith("split")
