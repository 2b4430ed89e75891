"""Attention over 8-bit pages where weights and page scales span many powers of two: rows
that one position dominates, and value scales from one end of the range to the other.

Tolerances, from the arithmetic (test_gpu_kv8_attend derives the first line):
  * a weight is good to (2^-17 M + 2^-15) of itself, M = scale * sum |q k|, the sums
    included; here that is of the positions that contribute, tau (their probability) max|V|.
  * the sum of values takes weights in steps: half a step is 2^-25 (four terms) or 2^-30
    (f32 outputs, five) where the largest weight of a tile of 128 positions is at least 2^-10
    or 2^-8, and 2^2 when it set the row's reference. The others' weights here are alike: on
    average within 2^3 of their tile's largest, so at least 2^-13 or 2^-11, and off by
    2^-12 or 2^-19 of themselves. In the tile of the dominating position 128 half steps are
    2^-20 or 2^-25 of its weight.
  * the output's rounding: half a step, eps / 2 of the value.
"""
import math

import numpy as np
import pytest
import torch

from tests.kv8_util import attention_reference, code_values, gathered, paged_cache
from tests.test_gpu_kv8_attend import OUT, call, check, queries

pytestmark = pytest.mark.gpu

ONE = {"e4m3": 0x38, "e5m2": 0x3C}


def peaked(seed, n, rows, d, code, where, odds, value):
    """A cache of one head whose positions `where` have the odds `odds` (a row at a time) each
    against all others together, and values of `value` times the others' size. Column 0 of
    the keys is theirs alone, values are positive. Returns cache, queries."""
    assert code_values(code)[ONE[code]] == 1.0
    cache = paged_cache(seed, [n], 64, 1, d, code)
    kp, vp, ks, vs, table = cache
    k8, v8 = kp.view(torch.uint8), vp.view(torch.uint8)
    live = table[0, :-(-n // 64)].long()
    ks[live], vs[live] = 2.0 ** -7, 2.0 ** -7       # as the random pages' are, near enough
    k8[live, :, :, 0] = 0
    v8[live] &= 0x7F
    if n % 64:
        v8[table[0, n // 64], n % 64:] = 0x7F
    q = queries(seed + 1, 1, 1, rows, d)
    q[..., 1:] *= 0.3                             # the others' scores: N(0, 0.3)
    for r in range(rows):
        q[0, 0, r, 0] = math.log(odds[r] * n) * math.sqrt(d) / 2.0 ** -7
    for pos in where:
        blk = table[0, pos // 64]
        k8[blk, pos % 64, 0, 0] = ONE[code]
        if value == 0:
            v8[blk, pos % 64] = 0
        else:                                     # codes of the same type, `value` times 1
            v8[blk, pos % 64] = torch.tensor([value]).to(vp.dtype).view(torch.uint8)[0]
    return cache, q


def check_peaked(got, q, cache, n, d, code, where, out):
    kp, vp, ks, vs, table = cache
    k, v = gathered(kp, ks, table, [n], 64, code), gathered(vp, vs, table, [n], 64, code)
    ref, mag = attention_reference(q.double().numpy(), k, v, [n], d ** -0.5)
    five = out == "f32"
    rest = np.ones(n, bool)
    rest[where] = False
    vmax, vpeak = np.abs(v[0][rest]).max(), np.abs(v[0][where]).max()
    s = (k[0][:, 0] @ q[0, 0].double().numpy().T) * d ** -0.5
    p = np.exp(s - s.max(0))
    tau = (p[rest].sum(0) / p.sum(0))[:, None]
    rel = 2.0 ** -17 * mag[0, 0][:, None] + 2.0 ** -15 + 2.0 ** (-19 if five else -12)
    tol = (tau * vmax + (1 - tau) * vpeak) * rel + 2.0 ** (-25 if five else -20) * vmax
    if not five:
        tol = tol + torch.finfo(OUT[out]).eps / 2 * np.abs(ref[0, 0])
        tol = tol + (6e-8 if out == "f16" else 0.0)
    err = np.abs(got[0, 0] - ref[0, 0])
    assert np.all(np.isfinite(got))
    assert (err / tol).max() <= 1, ((err / tol).max(), np.linalg.norm(err) / np.linalg.norm(ref))


@pytest.mark.parametrize("rows,d,out", [(4, 128, "f32"), (8, 128, "f32"), (24, 128, "f32"),
                                        (3, 256, "bf16"), (8, 128, "f16"), (16, 128, "bf16"),
                                        (24, 256, "bf16"), (32, 128, "f16"), (40, 128, "bf16")])
@pytest.mark.parametrize("n,where,value,splits", [
    (16384, [0], 0.0, 0), (16384, [0], 0.1, 1), (65536, [0], 0.0, 1), (20000, [77, 9000], 0.0, 1),
    (20000, [19999], 0.0, 0), (3000, [130], 0.02, 1)])
def test_a_dominating_position_leaves_the_others(rows, d, out, n, where, value, splits):
    code = "e5m2" if rows in (3, 32) else "e4m3"
    odds = [10 ** (1 + 2 * r / max(1, rows - 1)) for r in range(rows)]     # 10 to 1000
    cache, q = peaked(60 + rows, n, rows, d, code, where, odds, value)
    got = call(q, cache, 64, d ** -0.5, plan_lens=[n], out=out, splits=splits)
    check_peaked(got, q, cache, n, d, code, where, out)


@pytest.mark.parametrize("rows,out", [(4, "f32"), (8, "bf16"), (16, "bf16"), (24, "f32"),
                                      (32, "f16")])
def test_scores_that_rise_and_fall_from_tile_to_tile(rows, out):
    # pages whose keys are 1 to 32 times as large, in runs of three: scores up to +-60
    n, page = 5000, 16
    cache = paged_cache(70, [n], page, 1, 128, "e4m3")
    kp, vp, ks, vs, table = cache
    for j in range(-(-n // page)):
        ks[table[0, j]] *= 2.0 ** ((j // 3 * 7) % 6)
    q = queries(71, 1, 1, rows, 128)
    got = call(q, cache, page, 128 ** -0.5, plan_lens=[n], out=out, splits=1)
    check(got, q, cache, [n], page, "e4m3", 128 ** -0.5, out)


def scaled(seed, n, d, power, zero=()):
    """A cache of pages of 16, page j's value scale times 2^power(j); pages in `zero` hold zero
    values under the scale 2^-100, as an append writes them."""
    cache = paged_cache(seed, [n], 16, 1, d, "e4m3")
    kp, vp, ks, vs, table = cache
    for j in range(-(-n // 16)):
        blk = int(table[0, j])
        if j in zero:
            keep = vp.view(torch.uint8)[blk, n - 16 * j:].clone() if n < 16 * j + 16 else None
            vp.view(torch.uint8)[blk] = 0
            if keep is not None:
                vp.view(torch.uint8)[blk, n - 16 * j:] = keep
            vs[blk] = 2.0 ** -100
        else:
            vs[blk] = 2.0 ** (power(j) + round(math.log2(float(vs[blk, 0]))))
    return cache


SHAPES = [(4, 128, "f32"), (8, 128, "f32"), (8, 256, "bf16"), (16, 128, "bf16"), (24, 256, "f32")]


@pytest.mark.parametrize("rows,d,out", SHAPES)
@pytest.mark.parametrize("splits", [1, 5])
@pytest.mark.parametrize("power", [122, -92, 40])
def test_value_scales_at_the_ends_of_their_range(rows, d, out, splits, power):
    # pages of random values have scales about 2^-7: 2^115, 2^-99 and 2^33
    n = 3000
    cache = scaled(80, n, d, lambda j: power)
    q = queries(81, 1, 1, rows, d, 2.0)
    got = call(q, cache, 16, d ** -0.5, plan_lens=[n], out=out, splits=splits)
    check(got, q, cache, [n], 16, "e4m3", d ** -0.5, out)


@pytest.mark.parametrize("rows,d,out", SHAPES)
@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("zero", ["first", "last", "odd tiles", "even tiles", "all but one"])
@pytest.mark.parametrize("power", [37, 47, 120])
def test_pages_of_zeros_beside_large_ones(rows, d, out, splits, zero, power):
    # pages of zeros hold their share of the probabilities whatever the others' scales are
    n, pages = 2048, 128
    half = {"first": range(pages // 2), "last": range(pages // 2, pages),
            "odd tiles": [j for j in range(pages) if j // 8 % 2],
            "even tiles": [j for j in range(pages) if j // 8 % 2 == 0],
            "all but one": [j for j in range(pages) if j != 70]}[zero]
    cache = scaled(82, n, d, lambda j: power, set(half))
    q = queries(83, 1, 1, rows, d)
    got = call(q, cache, 16, d ** -0.5, plan_lens=[n], out=out, splits=splits)
    check(got, q, cache, [n], 16, "e4m3", d ** -0.5, out)


@pytest.mark.parametrize("rows,d,out", SHAPES)
@pytest.mark.parametrize("splits", [1, 4])
def test_value_scales_anywhere_in_their_range(rows, d, out, splits):
    n = 2500
    rng = np.random.default_rng(84)
    powers = rng.integers(-92, 122, size=-(-n // 16))
    cache = scaled(85, n, d, lambda j: int(powers[j]))
    q = queries(86, 1, 1, rows, d)
    got = call(q, cache, 16, d ** -0.5, plan_lens=[n], out=out, splits=splits)
    check(got, q, cache, [n], 16, "e4m3", d ** -0.5, out)
