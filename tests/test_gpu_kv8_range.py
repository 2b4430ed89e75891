"""Attention over 8-bit pages whose value scales lie anywhere in their range, against
attention in 64 bits. Tolerances as derived in test_gpu_kv8_attend.
"""
import math

import numpy as np
import pytest
import torch

from tests.kv8_util import paged_cache
from tests.test_gpu_kv8_attend import call, check, queries

pytestmark = pytest.mark.gpu

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
