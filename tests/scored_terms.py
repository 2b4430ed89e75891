"""Inputs of scored attention in which every 16-bit term of q or of the weights shows in the output, and
what the output is without the last of them."""
import math

import numpy as np
import torch

from tests.scored_util import DT, EPS, Case

# cache, output and terms of an f32 q and of a weight
TYPES = [("f16", "f32", 2), ("f16", "f16", 2), ("bf16", "f16", 2), ("bf16", "bf16", 2),
         ("bf16", "f32", 3)]
# those in which a term of the weights is more than half a step of the output
WEIGHT_TYPES = [("f16", "f32", 2), ("bf16", "f16", 2), ("bf16", "f32", 3)]
# lengths, query heads and shared positions: rows that are packed, in four copies, in two and in one;
# and behind shared positions, in one row tile and in several
LAYOUTS = [((32,), 4, 0), ((32,), 12, 0), ((32,), 20, 0), ((32,), 40, 0), ((32,), 100, 0),
           ((32,) * 5, 4, 32), ((32,) * 3, 100, 64)]
# half a step of that many terms: 11 bits each, or 8
TERMS = {("f16", 2): 2.0 ** -22, ("bf16", 2): 2.0 ** -16, ("bf16", 3): 2.0 ** -24}


def in_terms(x, cache, n):
    """x as the sum of n terms of the cache's type, each the nearest to what is left."""
    left = np.asarray(x, dtype=np.float64).copy()
    total = np.zeros_like(left)
    for _ in range(n):
        t = torch.tensor(left, dtype=torch.float32).to(DT[cache]).double().numpy()
        total, left = total + t, left - t
    return total


def query_case(cache, out, terms, layout, d):
    """Half of the positions score what only the last term of q holds, 1/8, the others 0; their
    values are 1 and 0, so that the output is the logistic function of that score."""
    lens, hq, shared = layout
    if cache == "f16":
        q, top = (1 + 2.0 ** -13, -1.0), 2.0 ** 10
    elif terms == 2:
        q, top = (1 + 2.0 ** -9, -1.0), 2.0 ** 6
    else:
        q, top = (1 + 2.0 ** -9 + 2.0 ** -18, -1.0, -2.0 ** -9), 2.0 ** 15
    c = Case(lens, hq, 1, d, cache=cache, q="f32", out=out, scale=1.0, shared=shared, page=32,
             poison=False)
    c.q.zero_()
    c.q[..., :len(q)] = torch.tensor(q)
    c.k.zero_()
    c.k[:, ::2, :, :len(q)] = top
    c.v.zero_()
    c.v[:, ::2] = 1.0
    # an MMA a term: three products and the sum so far, cut off at the 24th bit of the largest each
    c.score_error = 4 * terms * top * 2.0 ** -23
    return c


def query_bound(c, terms):
    """The score's error moves the logistic function by a quarter of it. A weight is off by half a step
    of its terms and the exponential's 2^-22; 12 MMAs at most cut off 16 products and a sum at their
    24th bit; then half a step of the output, which is below 1."""
    return c.score_error / 4 + TERMS[c.cache, terms] + 2.0 ** -22 + 12 * 17 * 2.0 ** -23 + EPS[c.out] / 4


# scores (exact in 16 bits) whose weights lose much without their last term
DELTA = {("f16", 2): 1.34375, ("bf16", 2): 1.359375, ("bf16", 3): 1.25}


def weight_case(cache, out, terms, layout, d):
    """Every eighth position scores 0, the others -delta. One of those, of a sequence's own and of the
    shared ones each, has a value of 1, all others have 0."""
    lens, hq, shared = layout
    c = Case(lens, hq, 1, d, cache=cache, out=out, scale=1.0, shared=shared, page=32, poison=False)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k.zero_()
    c.k[..., 0] = -DELTA[cache, terms]
    c.k[:, ::8, :, 0] = 0.0
    c.v.zero_()
    c.v[c.table[:, 0].long(), 13] = 1.0
    if shared:
        c.v[int(c.shared_table[0]), 13] = 1.0
    return c


def weight_share(c, terms, used):
    """The output of weight_case where the weights that multiply values have `used` terms."""
    w = math.exp(-DELTA[c.cache, terms])
    n = c.lens[0] + c.shared
    return (1 + (c.shared > 0)) * float(in_terms(w, c.cache, used)) / (n / 8 + n * 7 / 8 * w)


def weight_bound(c, terms):
    """Relative: half a step of the weights' terms; an MMA a term, of one product and the sum so far
    (the others are 0), cut off at their 24th bit; the exponential and its exponent, 2^-22 + 2^-23 of a
    weight, of which the sum takes two thirds back; f32 sums of up to 96 weights, 16 in a row at
    most and joined in four steps more; the quotient, the product and the combine's four steps; half a
    step of the output."""
    return TERMS[c.cache, terms] + 2 * terms * 2.0 ** -23 + 2.0 ** -23 + (20 + 6) * 2.0 ** -24 \
        + EPS[c.out] / 2
