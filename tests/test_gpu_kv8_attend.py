"""Split-KV attention over 8-bit paged pools (decode_attn_splitk_8bit) against attention
in 64 bits over what the codes stand for.

Tolerance, per output element, from the arithmetic (u = 2^-24):
  * q is held to 2^-20 of itself for 16-bit outputs (four terms) and 2^-25 for f32 ones
    (five). A score is an f32 sum of at most 4 * 256 or 5 * 256 exact products, added 32 at
    a time, and four more f32 operations: |error of a score| <= (2^-20 + 44 u) * M or
    (2^-25 + 52 u) * M, M = scale * sum |q k|
    of the position, under 2^-18 * M (natural units). A weight is off by e^error - 1, the
    normalised output by twice that, times max |V|: 2^-17 M max|V|.
  * probabilities are held to 20 significant bits or more and 2^-26 of the largest, 2^x is good to
    2^-22, its f32 argument (at most 2^7 in size) to 2^-18: 2^-16.7 together; sums over
    positions and splits are f32, for the lengths here at most 2^-17: 2^-15 max|V|.
  * groups of more than 8 rows with a 16-bit output: probabilities of 15 significant bits. A
    term of 4 bits leaves half of its step, 2^-4 of the value's power of two; each further
    one, of a rest in the next lower power at most, 2^-5 of that: 2^-4, 2^-9, 2^-14 of a
    weight, of either sign, in the sum of weight times value: 2^-14 max|V|.
  * the output's rounding: half a step, eps / 2 of the value.
"""
import math

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from tests.kv8_util import TDT, attention_reference, code_values, gathered, paged_cache

pytestmark = pytest.mark.gpu

OUT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def queries(seed, B, T, hq, d, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, T, hq, d, generator=g) * std


def call(q, cache, page, scale, *, plan_lens, now=None, out="f32", splits=0, flags=0, num_sms=0,
         stream=None, combine=True):
    kp, vp, ks, vs, table = [t.cuda() for t in cache]
    x = q.cuda()
    x = x[:, 0].contiguous() if q.shape[1] == 1 else x
    args = A.make_paged_args(x, kp, vp, scale, table.shape[1], out_dtype=OUT[out],
                             force_splits=splits, flags=flags)
    plan = A.decode_attn_plan(args, plan_lens, num_sms)
    assert plan.kernel == N.DA_KERNEL_GQA_8BIT
    lens = None if now is None else torch.tensor(now, dtype=torch.int32, device="cuda")
    dev = A.make_dev(seq_lens=lens, block_table=table, k_pool=kp, v_pool=vp)
    sc = A.make_scales(ks, vs)
    ws = A.new_workspace(plan)
    ws.fill_(0xFF)                                # poisoned: every partial must be written
    o = torch.full(x.shape, math.nan, dtype=OUT[out], device="cuda")
    torch.cuda.synchronize()
    A.decode_attn_splitk_8bit(args, plan, dev, sc, x, kp, vp, o, ws, stream)
    torch.cuda.synchronize()
    A.decode_attn_device_status(ws)
    return o.double().cpu().numpy().reshape(q.shape)


def check(got, q, cache, lens, page, code, scale, out="f32", causal=True):
    kp, vp, ks, vs, table = cache
    k, v = gathered(kp, ks, table, lens, page, code), gathered(vp, vs, table, lens, page, code)
    ref, mag = attention_reference(q.double().numpy(), k, v, lens, scale, causal)
    assert np.all(np.isfinite(got))
    for b in range(len(lens)):
        vmax = np.abs(v[b]).max() if lens[b] else 0.0
        tol = vmax * (2.0 ** -17 * mag[b][..., None] + 2.0 ** -15)
        if out != "f32":
            tol = tol + (2.0 ** -14 * vmax if q.shape[1] * q.shape[2] // k[b].shape[1] > 8 else 0.0)
            tol = tol + torch.finfo(OUT[out]).eps / 2 * np.abs(ref[b])
            tol = tol + (6e-8 if out == "f16" else 0.0)      # half of f16's least step
        worst = (np.abs(got[b] - ref[b]) / np.maximum(tol, 1e-300)).max()
        assert worst <= 1, (b, worst, np.abs(got[b] - ref[b]).max(), vmax)
    return ref


def run_check(lens, page, hq, hkv, d, code, *, T=1, out="f32", seed=0, std=1.0, now=None,
              splits=0, num_sms=0, flags=0, **kw):
    cache = paged_cache(seed, lens if now is None else now, page, hkv, d, code,
                        width_extra=2 + max(lens) // page, **kw)
    q = queries(seed + 1, len(lens), T, hq, d, std)
    scale = 1 / math.sqrt(d)
    got = call(q, cache, page, scale, plan_lens=lens, now=now, out=out, splits=splits,
               num_sms=num_sms, flags=flags)
    at = lens if now is None else [min(max(n, 0), m) for n, m in zip(now, lens)]
    ref = check(got, q, cache, at, page, code, scale, out, not flags & N.DA_FLAG_NO_CAUSAL)
    return got, ref


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 256), (16, 4, 256), (32, 8, 128), (3, 3, 128),
                                      (10, 2, 128), (24, 4, 256), (7, 1, 256), (8, 1, 128)])
def test_groups_of_up_to_eight(hq, hkv, d, code):
    run_check([1500, 1, 129, 128, 700], 16, hq, hkv, d, code, seed=hq)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256, 400])
@pytest.mark.parametrize("d", [128, 256])
def test_page_sizes(page, d):
    run_check([2000, 17, 383], page, 8, 2, d, "e4m3", seed=page)


@pytest.mark.parametrize("rows", [9, 12, 16, 20, 25, 31, 32, 33, 48, 64, 96, 100, 128])
@pytest.mark.parametrize("d", [128, 256])
def test_large_groups(rows, d):
    run_check([900, 64], 64, rows, 1, d, "e4m3", seed=rows)


@pytest.mark.parametrize("T,hq,hkv,d", [(2, 8, 2, 256), (4, 24, 4, 256), (3, 5, 5, 128),
                                        (5, 16, 4, 128), (64, 2, 1, 128), (16, 8, 1, 256)])
def test_several_new_tokens(T, hq, hkv, d):
    # lengths down to the new tokens alone, and a causal limit that crosses tiles
    run_check([T, T + 1, 130, 515, 128 + T // 2 + 1], 16, hq, hkv, d, "e4m3", T=T, seed=T)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
def test_forced_splits(splits):
    run_check([4000, 260], 48, 8, 2, 128, "e4m3", splits=splits, seed=3)
    run_check([1000, 130], 48, 8, 2, 128, "e4m3", T=4, splits=splits, seed=4)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,d", [(12, 256), (3, 128), (16, 128), (24, 128), (24, 256), (44, 128),
                                  (64, 256)])
def test_output_types(out, hq, d):
    run_check([777, 300], 32, hq, 1, d, "e4m3", out=out, seed=9)
    run_check([200, 129], 32, hq // 2, 1, d, "e4m3", T=2, out=out, seed=10)


def test_few_ctas_walk_many_items():
    run_check([3000, 1, 500, 129, 2048], 16, 16, 4, 128, "e4m3", num_sms=3, splits=5, seed=5)
    run_check([600, 70], 64, 40, 2, 256, "e5m2", num_sms=2, splits=3, seed=6)


@pytest.mark.parametrize("rows", [3, 8, 16, 32])
@pytest.mark.parametrize("d", [128, 256])
def test_long_items(rows, d):
    # dozens of tiles an item, so that every slot of the ring is used again and again
    run_check([9000, 4000], 16, rows, 1, d, "e4m3", num_sms=2, splits=1, seed=rows + d)


def test_relative_accuracy_of_f32_output():
    # the 2-norm of the error: every source above averages over hundreds of positions;
    # 20-bit operands alone leave 2^-20 / sqrt(3) of the result
    got, ref = run_check([6000], 64, 16, 4, 256, "e4m3", seed=11)
    assert np.linalg.norm(got - ref) <= 2.0 ** -17 * np.linalg.norm(ref)


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 256), (8, 1, 128), (24, 1, 256), (40, 1, 128)])
def test_f32_output_is_as_good_as_f32_arithmetic(hq, hkv, d):
    # Five terms leave 2^-25 of q and of a weight, below the f32 roundings: a score's is at
    # most 2^-24 of M a step and far less on average, its shift and 2^x another 2^-22 each.
    # Their signs are random, so the 2-norm's ratio is one weight's error: under 2^-24 M + 2^-21.
    cache = paged_cache(31, [5000, 700], 64, hkv, d, "e4m3", width_extra=80)
    q = queries(32, 2, 1, hq, d)
    got = call(q, cache, 64, 1 / math.sqrt(d), plan_lens=[5000, 700])
    k, v = (gathered(p, s, cache[4], [5000, 700], 64, "e4m3") for p, s in
            ((cache[0], cache[2]), (cache[1], cache[3])))
    ref, mag = attention_reference(q.double().numpy(), k, v, [5000, 700], 1 / math.sqrt(d), True)
    for b in range(2):
        err = np.linalg.norm(got[b] - ref[b]) / np.linalg.norm(ref[b])
        assert err <= 2.0 ** -24 * mag[b].max() + 2.0 ** -21, (b, err, mag[b].max())


@pytest.mark.parametrize("now", [[0, 1000, 5], [1000, 0, 0], [16, 15, 17], [-4, 10 ** 6, 128]])
def test_device_lengths(now):
    # lengths of zero give zeros; lengths are kept within [0, the plan's]
    lens = [1000, 1000, 1000]
    at = [min(max(n, 0), 1000) for n in now]
    cache = paged_cache(2, at, 16, 2, 128, "e4m3", width_extra=64)
    q = queries(3, 3, 1, 8, 128)
    got = call(q, cache, 16, 0.1, plan_lens=lens, now=now)
    check(got, q, cache, at, 16, "e4m3", 0.1)
    for b in range(3):
        assert at[b] or np.all(got[b] == 0)


@pytest.mark.parametrize("now", [[0, 1, 2, 3, 200], [3, 0, 129, 4, 1]])
def test_new_tokens_before_the_start_give_zeros(now):
    cache = paged_cache(4, now, 16, 2, 128, "e4m3", width_extra=20)
    q = queries(5, 5, 4, 4, 128)
    got = call(q, cache, 16, 0.1, plan_lens=[256] * 5, now=now)
    check(got, q, cache, now, 16, "e4m3", 0.1)
    for b, n in enumerate(now):
        for i in range(4):
            assert n - 4 + 1 + i > 0 or np.all(got[b, i] == 0)


def test_every_new_token_sees_everything_without_the_causal_limit():
    run_check([300, 129], 16, 8, 2, 128, "e4m3", T=4, flags=N.DA_FLAG_NO_CAUSAL, seed=8)


def test_value_scales_that_differ_by_eighty_powers_of_two():
    run_check([2000, 300], 16, 8, 2, 128, "e4m3", uneven=True, seed=12)
    run_check([2000, 300], 16, 40, 2, 128, "e4m3", uneven=True, seed=13, splits=3)


def test_large_scores_and_a_rising_maximum():
    # scores up to about +-60, and a cache whose later pages score higher and higher
    run_check([3000], 16, 8, 2, 128, "e4m3", std=15.0, seed=14)
    cache = paged_cache(15, [2000], 16, 1, 128, "e4m3", spread=0.0)
    kp, vp, ks, vs, table = cache
    for j in range(125):
        ks[table[0, j]] *= 2.0 ** (j // 25)
    q = queries(16, 1, 1, 4, 128)
    got = call(q, cache, 16, 0.25, plan_lens=[2000], splits=1)
    check(got, q, cache, [2000], 16, "e4m3", 0.25)


def test_zero_scales_of_empty_pages():
    # pages of zeros under another quantiser's rule: scale 0
    cache = paged_cache(17, [500, 16], 16, 2, 128, "e4m3")
    kp, vp, ks, vs, table = cache
    for b, j in ((0, 3), (0, 7), (1, 0)):
        blk = int(table[b, j])
        kp.view(torch.uint8)[blk] = 0
        vp.view(torch.uint8)[blk] = 0
        ks[blk], vs[blk] = 0.0, 0.0
    q = queries(18, 2, 1, 8, 128)
    got = call(q, cache, 16, 0.1, plan_lens=[500, 16])
    check(got, q, cache, [500, 16], 16, "e4m3", 0.1)
    assert np.all(got[1] == 0)


def test_scales_that_are_no_powers_of_two():
    cache = paged_cache(19, [700], 32, 4, 256, "e4m3")
    kp, vp, ks, vs, table = cache
    g = torch.Generator().manual_seed(1)
    ks *= 1 + 0.9 * torch.rand(ks.shape, generator=g)
    vs *= 1 + 0.9 * torch.rand(vs.shape, generator=g)
    q = queries(20, 1, 1, 16, 256)
    got = call(q, cache, 32, 1 / 16, plan_lens=[700])
    check(got, q, cache, [700], 32, "e4m3", 1 / 16)


@pytest.mark.parametrize("code,nan", [("e4m3", 0x7F), ("e5m2", 0x7E), ("e5m2", 0x7C)])
@pytest.mark.parametrize("splits", [1, 3])
def test_nan_in_a_new_token_reaches_only_the_tokens_that_see_it(code, nan, splits):
    # (e5m2's infinity too: it is no number either once weighted against others)
    T, L, d = 4, 300, 128
    cache = paged_cache(21, [L], 16, 1, d, code)
    kp, vp, ks, vs, table = cache
    q = queries(22, 1, T, 2, d)
    clean = call(q, cache, 16, 0.1, plan_lens=[L], splits=splits)
    for pool, at, cols in ((vp, L - 2, [5]), (kp, L - 1, range(d))):
        pos, u = at, pool.view(torch.uint8)
        old = u[table[0, pos // 16], pos % 16, 0, 5].item()
        u[table[0, pos // 16], pos % 16, 0, 5] = nan
        kp_, vp_, ks_, vs_, t_ = [t.cuda() for t in cache]
        x = q.cuda()
        a = A.make_paged_args(x, kp_, vp_, 0.1, t_.shape[1], force_splits=splits)
        p = A.decode_attn_plan(a, [L])
        dv = A.make_dev(block_table=t_, k_pool=kp_, v_pool=vp_)
        ws, o = A.new_workspace(p), torch.empty_like(x)
        A.decode_attn_splitk_8bit(a, p, dv, A.make_scales(ks_, vs_), x, kp_, vp_, o, ws)
        got = o.double().cpu().numpy()
        sees = [i for i in range(T) if L - T + i >= at]
        blind = [i for i in range(T) if i not in sees]
        np.testing.assert_array_equal(got[0, blind], clean[0, blind])
        if nan != 0x7C or pool is vp:
            assert not np.any(np.isfinite(got[0][sees][..., list(cols)]))
        u[table[0, pos // 16], pos % 16, 0, 5] = old


def test_head_major_pools_and_strided_scales():
    lens, page, h, d = [500, 33], 16, 3, 128
    cache = paged_cache(23, lens, page, h, d, "e4m3")
    q = queries(24, 2, 1, 6, d)
    want = call(q, cache, page, 0.1, plan_lens=lens)
    kp, vp, ks, vs, table = cache
    room = torch.full((2, kp.shape[0], h, page + 1, d + 16), 0x7F, dtype=torch.uint8, device="cuda")
    pools = [r[:, :, :page, :d].permute(0, 2, 1, 3) for r in room]
    for r, x in zip(pools, (kp, vp)):
        r.copy_(x.view(torch.uint8))
    pools = [r.view(TDT["e4m3"]) for r in pools]
    scales = [s.t().contiguous().cuda().t() for s in (ks, vs)]
    x = q[:, 0].contiguous().cuda()
    t = table.cuda()
    a = A.make_paged_args(x, *pools, 0.1, t.shape[1])
    p = A.decode_attn_plan(a, lens)
    dv = A.make_dev(block_table=t, k_pool=pools[0], v_pool=pools[1])
    ws, o = A.new_workspace(p), torch.empty_like(x)
    A.decode_attn_splitk_8bit(a, p, dv, A.make_scales(*scales), x, *pools, o, ws)
    np.testing.assert_array_equal(o.double().cpu().numpy(), want[:, 0])


def test_the_same_page_in_two_sequences_and_twice_in_one():
    # a shared prefix, and a table that names a page again
    cache = paged_cache(25, [160, 100], 16, 2, 128, "e4m3", poison=False)
    table = cache[4]
    table[1, :4] = table[0, :4]
    table[0, 6] = table[0, 2]
    q = queries(26, 2, 1, 8, 128)
    got = call(q, cache, 16, 0.1, plan_lens=[160, 100])
    check(got, q, cache, [160, 100], 16, "e4m3", 0.1)


def test_table_entries_outside_the_pool_read_as_zeros():
    cache = paged_cache(27, [64], 16, 1, 128, "e4m3")
    table = cache[4]
    zero = [t.clone() for t in cache]
    for j, bad in ((1, -3), (2, 10 ** 9)):
        zero[0].view(torch.uint8)[table[0, j]] = 0
        zero[1].view(torch.uint8)[table[0, j]] = 0
        zero[3][table[0, j]] = 1.0
        table[0, j] = bad
    q = queries(28, 1, 1, 4, 128)
    got = call(q, cache, 16, 0.1, plan_lens=[64])
    check(got, q, zero, [64], 16, "e4m3", 0.1)


def test_pools_past_four_gigabytes():
    nb, page, h, d = 2100, 64, 128, 256
    kp = torch.zeros(nb, page, h, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vp = kp.clone()
    ks = torch.ones(nb, h, device="cuda")
    small = paged_cache(29, [100], page, h, d, "e4m3", spare=0)
    for pool, x in ((kp, small[0]), (vp, small[1])):
        pool.view(torch.uint8)[-2:] = x.view(torch.uint8).cuda()
    ks[-2:], vs = small[2].cuda(), ks.clone()
    vs[-2:] = small[3].cuda()
    table = (small[4][:, :2] + nb - 2).cuda()
    x = queries(30, 1, 1, h, d)
    a = A.make_paged_args(x[:, 0].cuda(), kp, vp, 1 / 16, 2)
    p = A.decode_attn_plan(a, [100])
    dv = A.make_dev(block_table=table, k_pool=kp, v_pool=vp)
    ws, o = A.new_workspace(p), torch.empty(1, h, d, device="cuda")
    xq = x[:, 0].contiguous().cuda()
    A.decode_attn_splitk_8bit(a, p, dv, A.make_scales(ks, vs), xq, kp, vp, o, ws)
    check(o.double().cpu().numpy()[:, None], x, small, [100], page, "e4m3", 1 / 16)


def test_a_long_context_sampled():
    # one (row, head) of a 131072-position context against 64 bits; the other bound on the
    # whole output: the same result from three times as many splits
    L, page, h, d = 131072, 64, 2, 128
    g = torch.Generator(device="cuda").manual_seed(31)
    nb = L // page
    codes = [(torch.randn(nb, page, h, d, generator=g, device="cuda") * 40).clamp(-448, 448)
             .to(torch.float8_e4m3fn) for _ in range(2)]
    sc = [torch.full((nb, h), 2.0 ** -5, device="cuda") for _ in range(2)]
    table = torch.randperm(nb, device="cuda", generator=g).int()[None].contiguous()
    x = torch.randn(1, 8, d, generator=g, device="cuda")
    outs = []
    for s in (0, 300):
        a = A.make_paged_args(x, *codes, d ** -0.5, nb, force_splits=s)
        p = A.decode_attn_plan(a, [L])
        dv = A.make_dev(block_table=table, k_pool=codes[0], v_pool=codes[1])
        ws, o = A.new_workspace(p), torch.empty_like(x)
        A.decode_attn_splitk_8bit(a, p, dv, A.make_scales(*sc), x, *codes, o, ws)
        outs.append(o.double())
    ids = table[0].long()
    k, v = [(c.view(torch.uint8)[ids].view(c.dtype).double() * 2.0 ** -5).reshape(L, h, d)
            for c in codes]
    for head in (0, 5):
        s = (k[:, head // 4] @ x[0, head].double()) * d ** -0.5
        ref = torch.softmax(s, 0) @ v[:, head // 4]
        assert (outs[0][0, head] - ref).norm() <= 2.0 ** -16 * ref.norm()
    assert (outs[0] - outs[1]).norm() <= 2.0 ** -15 * outs[0].norm()


def test_two_streams_at_once_and_captured():
    lens = [900, 200]
    caches = [paged_cache(s, lens, 16, 2, 128, "e4m3") for s in (32, 33)]
    q = queries(34, 2, 1, 8, 128)
    want = [call(q, c, 16, 0.1, plan_lens=lens) for c in caches]
    streams, states = [torch.cuda.Stream() for _ in caches], []
    x = q[:, 0].contiguous().cuda()
    for c in caches:
        kp, vp, ks, vs, t = [y.cuda() for y in c]
        a = A.make_paged_args(x, kp, vp, 0.1, t.shape[1])
        p = A.decode_attn_plan(a, lens)
        states.append((a, p, A.make_dev(block_table=t, k_pool=kp, v_pool=vp),
                       A.make_scales(ks, vs), x, kp, vp, torch.empty_like(x), A.new_workspace(p),
                       (t, ks, vs)))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s in zip(streams, states):
            A.decode_attn_splitk_8bit(*s[:9], stream=st)
    torch.cuda.synchronize()
    for w, s in zip(want, states):
        np.testing.assert_array_equal(s[7].double().cpu().numpy(), w[:, 0])
        s[7].fill_(math.nan)
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.decode_attn_splitk_8bit(*s[:9])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, s in zip(want, states):
        np.testing.assert_array_equal(s[7].double().cpu().numpy(), w[:, 0])


def test_partials_go_to_every_combine():
    lens, d = [1200, 300], 128
    cache = paged_cache(35, lens, 16, 2, d, "e4m3")
    q = queries(36, 2, 1, 8, d)
    want = call(q, cache, 16, 0.1, plan_lens=lens)[:, 0]
    kp, vp, ks, vs, t = [y.cuda() for y in cache]
    x = q[:, 0].contiguous().cuda()
    a = A.make_paged_args(x, kp, vp, 0.1, t.shape[1], flags=N.DA_FLAG_NO_COMBINE)
    p = A.decode_attn_plan(a, lens)
    dv = A.make_dev(block_table=t, k_pool=kp, v_pool=vp)
    ws, o = A.new_workspace(p), torch.empty_like(x)
    A.decode_attn_splitk_8bit(a, p, dv, A.make_scales(ks, vs), x, kp, vp, o, ws)
    A.decode_attn_combine(a, p, ws, o)
    np.testing.assert_array_equal(o.double().cpu().numpy(), want)
    # a second rank whose slice is empty changes nothing, with and without a projection
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    dz = A.make_dev(seq_lens=zero, block_table=t, k_pool=kp, v_pool=vp)
    n = A.decode_attn_workspace_bytes(p)
    both = torch.empty(2 * n, dtype=torch.uint8, device="cuda")
    both[:n] = ws
    A.decode_attn_splitk_8bit(a, p, dz, A.make_scales(ks, vs), x, kp, vp, o, both[n:])
    A.decode_attn_combine_ranks(a, p, both, 2, o)
    # the ranks' merge adds in another order: f32 sums of at most 20 partials
    np.testing.assert_allclose(o.double().cpu().numpy(), want, rtol=0, atol=2.0 ** -18 * 8)
    w = torch.randn(8, 64, d, generator=torch.Generator().manual_seed(2)).cuda() / d ** 0.5
    pr = torch.empty(2, 8, 64, device="cuda")
    A.decode_attn_combine_proj(a, p, A.make_proj(w), ws, pr)
    ref = np.einsum("hec,bhc->bhe", w.double().cpu().numpy(), want)
    np.testing.assert_allclose(pr.double().cpu().numpy(), ref, rtol=0, atol=2.0 ** -14)
    # two empty ranks: zeros
    both[:n] = both[n:]
    for r in (1, 2):
        A.decode_attn_combine_ranks(a, p, both, r, o.fill_(math.nan))
        assert torch.equal(o, torch.zeros_like(o))


def test_one_launch_is_accepted_and_bad_launches_are_reported():
    lens = [500]
    cache = paged_cache(37, lens, 16, 2, 128, "e4m3")
    q = queries(38, 1, 1, 8, 128)
    want = call(q, cache, 16, 0.1, plan_lens=lens)
    np.testing.assert_array_equal(
        call(q, cache, 16, 0.1, plan_lens=lens, flags=N.DA_FLAG_ONE_LAUNCH), want)
    with pytest.raises(A.DecodeAttnError) as e:
        call(q, cache, 16, 0.1, plan_lens=lens, flags=N.DA_FLAG_TEST_BAD_LAUNCH)
    assert e.value.status == N.DA_ELAUNCH and e.value.message.startswith("split")
    np.testing.assert_array_equal(call(q, cache, 16, 0.1, plan_lens=lens), want)


def test_codes_are_used_as_they_stand():
    # one position: the output is its value row, every code of the type among the columns
    for code in ("e4m3", "e5m2"):
        vals = code_values(code)
        finite = np.array([u for u in range(256) if np.isfinite(vals[u])], dtype=np.uint8)
        for lo in range(0, len(finite), 128):
            row = np.resize(finite[lo:lo + 128], 128)
            kp = torch.zeros(1, 16, 1, 128, dtype=torch.uint8)
            vp = torch.full((1, 16, 1, 128), 0x7F, dtype=torch.uint8)
            vp[0, 0, 0] = torch.from_numpy(row)
            cache = (kp.view(TDT[code]), vp.view(TDT[code]), torch.ones(1, 1),
                     torch.full((1, 1), 0.375), torch.zeros(1, 1, dtype=torch.int32))
            got = call(queries(1, 1, 1, 1, 128), cache, 16, 1.0, plan_lens=[1])
            np.testing.assert_allclose(got[0, 0, 0], vals[row] * 0.375, rtol=2.0 ** -19, atol=0)


@pytest.mark.parametrize("rows,d", [(4, 128), (8, 128), (16, 128), (24, 256), (32, 128)])
def test_a_wait_that_runs_out_is_reported(rows, d):
    # the copies are never issued; the next call on the same workspace is sound
    lens = [500, 2000]
    cache = paged_cache(39, lens, 16, 1, d, "e4m3")
    q = queries(40, 2, 1, rows, d)
    kp, vp, ks, vs, t = [y.cuda() for y in cache]
    x = q[:, 0].contiguous().cuda()
    dv = A.make_dev(block_table=t, k_pool=kp, v_pool=vp)
    ws = o = None
    for flags in (N.DA_FLAG_TEST_NO_TMA, 0):
        a = A.make_paged_args(x, kp, vp, 0.1, t.shape[1], flags=flags, timeout_us=20000)
        p = A.decode_attn_plan(a, lens)
        ws = A.new_workspace(p) if ws is None else ws
        o = torch.empty_like(x)
        A.decode_attn_splitk_8bit(a, p, dv, A.make_scales(ks, vs), x, kp, vp, o, ws)
        if flags:
            with pytest.raises(A.DecodeAttnError) as e:
                A.decode_attn_device_status(ws)
            assert e.value.status == N.DA_ETIMEOUT and "8 bits" in e.value.message
    A.decode_attn_device_status(ws)
    check(o.double().cpu().numpy()[:, None], q, cache, lens, 16, "e4m3", 0.1)


@pytest.mark.parametrize("rows", [4, 8, 16, 24])
@pytest.mark.parametrize("where", [(0,), (200,), (5, 140, 300)])
def test_a_nan_score_makes_the_row_nan(rows, where):
    # in the first tile, in the second (of the other warpgroups), in all of them; lengths
    # where a tile holds nothing but a NaN
    L, d = 301, 128
    cache = paged_cache(41, [L, 129], 16, 1, d, "e4m3")
    kp, table = cache[0].view(torch.uint8), cache[4]
    for pos in where:
        kp[table[0, pos // 16], pos % 16, 0, 3] = 0x7F
    kp[table[1, 8], 0, 0, 3] = 0x7F               # position 128: a tile of its own
    q = queries(42, 2, 1, rows, d)
    got = call(q, cache, 16, 0.1, plan_lens=[L, 129], splits=1)
    assert np.all(np.isnan(got))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("hq", [4, 24])
def test_a_query_that_is_no_number_spoils_its_own_row_alone(bad, hq):
    cache = paged_cache(43, [300], 16, 1, 128, "e4m3")
    q = queries(44, 1, 1, hq, 128)
    want = call(q, cache, 16, 0.1, plan_lens=[300])
    x = q.clone()
    x[0, 0, 2, 17] = bad
    got = call(x, cache, 16, 0.1, plan_lens=[300])
    assert np.all(np.isnan(got[0, 0, 2]))
    keep = [h for h in range(hq) if h != 2]
    np.testing.assert_array_equal(got[0, 0, keep], want[0, 0, keep])


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30])
def test_scales_of_the_scores(scale):
    cache = paged_cache(45, [500, 3], 16, 2, 128, "e4m3")
    q = queries(46, 2, 1, 8, 128)
    got = call(q, cache, 16, scale, plan_lens=[500, 3])
    check(got, q, cache, [500, 3], 16, "e4m3", abs(scale)) if scale >= 0 else \
        check(got, -q, cache, [500, 3], 16, "e4m3", -scale)


def test_queries_of_very_different_size():
    # rows from 1e-12 to 1e3: every row is scaled for itself
    cache = paged_cache(47, [400], 16, 1, 256, "e4m3")
    q = queries(48, 1, 1, 8, 256) * torch.tensor([1e-12, 1e-6, 1e-3, 0.1, 1.0, 10.0, 30.0, 0.0])[:, None]
    got = call(q, cache, 16, 1 / 16, plan_lens=[400])
    check(got, q, cache, [400], 16, "e4m3", 1 / 16)


def test_one_large_page_and_a_full_table():
    # a pool of a single page of 4096 positions, of which the table has one entry
    cache = paged_cache(49, [4096], 4096, 1, 128, "e4m3", spare=0, width_extra=0)
    q = queries(50, 1, 1, 8, 128)
    got = call(q, cache, 4096, 0.1, plan_lens=[4096])
    check(got, q, cache, [4096], 4096, "e4m3", 0.1)


def test_many_sequences():
    # the largest batch, a third of it empty
    lens = [(7 * b) % 200 if b % 3 else 0 for b in range(256)]
    cache = paged_cache(51, lens, 16, 1, 128, "e4m3")
    q = queries(52, 256, 1, 4, 128)
    got = call(q, cache, 16, 0.1, plan_lens=[max(1, n) for n in lens], now=lens)
    check(got, q, cache, lens, 16, "e4m3", 0.1)


def test_a_batch_that_is_empty():
    cache = paged_cache(53, [0, 0], 16, 2, 256, "e4m3")
    q = queries(54, 2, 1, 16, 256)
    got = call(q, cache, 16, 0.1, plan_lens=[20, 20], now=[0, 0])
    assert np.all(got == 0)


def test_refusals_of_the_binding():
    cache = [t.cuda() for t in paged_cache(55, [30], 16, 1, 128, "e4m3")]
    kp, vp, ks, vs, t = cache
    x = torch.randn(1, 4, 128, device="cuda")
    a = A.make_paged_args(x, kp, vp, 0.1, t.shape[1])
    p = A.decode_attn_plan(a, [30])
    dv, sc = A.make_dev(block_table=t, k_pool=kp, v_pool=vp), A.make_scales(ks, vs)
    ws, o = A.new_workspace(p), torch.empty_like(x)
    for q_, o_ in ((x.half(), o), (x.cpu(), o), (x.transpose(1, 2), o), (x, o.transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            A.decode_attn_splitk_8bit(a, p, dv, sc, q_, kp, vp, o_, ws)
    with pytest.raises(ValueError):
        A.decode_attn_splitk_8bit(a, p, dv, sc, x, kp.cpu(), vp, o, ws)
    with pytest.raises(TypeError):
        A.make_scales(ks.half(), vs)
    with pytest.raises(A.DecodeAttnError) as e:
        A.decode_attn_splitk_8bit(a, p, A.make_dev(), sc, x, kp, vp, o, ws)
    assert e.value.status == N.DA_EINVAL and "block_table" in e.value.message


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,T", [(8, 2, 1), (16, 2, 1), (5, 1, 4), (40, 1, 1), (24, 1, 2),
                                      (32, 1, 1)])
def test_one_split_a_sequence_writes_the_same_bits_as_the_combine(hq, hkv, T, out):
    # lengths of zero, and tokens before the start, among them
    now = [40, 0, 129, 2, 128, 0, 300, 1]
    cache = paged_cache(57, now, 16, hkv, 128, "e4m3", width_extra=20)
    kp, vp, ks, vs, t = [y.cuda() for y in cache]
    x = queries(58, 8, T, hq, 128).cuda()
    x = x[:, 0].contiguous() if T == 1 else x
    lens = torch.tensor(now, dtype=torch.int32, device="cuda")
    dv, sc = A.make_dev(seq_lens=lens, block_table=t, k_pool=kp, v_pool=vp), A.make_scales(ks, vs)
    got = []
    for flags in (0, N.DA_FLAG_NO_COMBINE):
        a = A.make_paged_args(x, kp, vp, 0.1, t.shape[1], out_dtype=OUT[out], force_splits=1,
                              flags=flags)
        p = A.decode_attn_plan(a, [320] * 8, 3)   # 3 CTAs: many items each
        assert p.max_splits == 1
        ws, o = A.new_workspace(p), torch.full(x.shape, math.nan, dtype=OUT[out], device="cuda")
        ws.fill_(0xFF)
        A.decode_attn_splitk_8bit(a, p, dv, sc, x, kp, vp, o, ws)
        if flags:
            A.decode_attn_combine(a, p, ws, o)
        got.append(o.view(torch.int32 if out == "f32" else torch.int16).clone())
    assert torch.equal(*got)
    check(o.double().cpu().numpy().reshape(8, T, hq, 128), queries(58, 8, T, hq, 128), cache, now,
          16, "e4m3", 0.1, out)
