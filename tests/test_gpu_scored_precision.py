"""The precision that scored attention promises, where a term or a bound that is lost would show."""
import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import api as A
from tests import scored_terms as S
from tests.scored_util import DT, near

pytestmark = pytest.mark.gpu


def attend(q, k, v, out, shared=0, page=64, **kw):
    """The call on one context [L, D], or on three short ones behind it as a shared prefix, by one CTA
    in as few splits as may be; and the formula in 64 bits."""
    L, d = k.shape
    out_t = DT[out]
    if shared:
        n = q.shape[0]
        pool = [x.reshape(-1, page, 1, d) for x in (k, v)]
        own = L // page - n                              # the last blocks are the sequences' own
        front = torch.arange(own, dtype=torch.int32, device="cuda")
        table = (own + torch.arange(n, dtype=torch.int32, device="cuda"))[:, None].contiguous()
        lens = torch.full((n,), page, dtype=torch.int32, device="cuda")
        args = A.make_paged_args(q, *pool, d ** -0.5, 1, out_dtype=out_t, force_splits=1)
        dev = A.make_dev(seq_lens=lens, block_table=table, k_pool=pool[0], v_pool=pool[1])
        score = A.make_score(q, shared_len=own * page, shared_table=front)
        plan = A.decode_attn_plan_scored(args, score, [page] * n, 1)
    else:
        pool, dev, n = [x[None, :, None] for x in (k, v)], None, 1
        args = A.make_args(q, *pool, d ** -0.5, out_dtype=out_t, force_splits=1)
        score = A.make_score(q)
        plan = A.decode_attn_plan_scored(args, score, [L], 1)
    ws, got = A.new_workspace(plan), torch.empty(q.shape, dtype=out_t, device="cuda")
    A.decode_attn_splitk_scored(args, plan, dev, score, q, pool[0], pool[1], got, ws)
    A.decode_attn_device_status(ws)
    want = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b in range(n):
        y = (q[b].double() @ k.double().T) * d ** -0.5   # [.., Hq, L]
        j = torch.arange(L, device="cuda")
        if shared:
            seen = (j < own * page) | ((j >= (own + b) * page) & (j < (own + b + 1) * page))
            y = y.masked_fill(~seen, -torch.inf)
        elif q.dim() == 4:
            y = y.masked_fill((j > L - q.shape[1] + torch.arange(q.shape[1], device="cuda")[:, None])
                              [:, None], -torch.inf)
        want[b] = torch.softmax(y, -1) @ v.double()
    return got.double(), want


@pytest.mark.parametrize("shape,shared", [((1, 6, 16), 0), ((1, 64), 0), ((1, 8), 0), ((3, 100), 1)])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
def test_long_items_beside_16_bit_outputs(cache, d, shape, shared):
    # values of one sign, so that every addition that is cut off at its 24th bit takes something away:
    # 1024 of them at most, 2^-23 each, and the merges of partials; the weights' terms and their
    # exponents, 2^-16 and 2^-20 of a weight, are as often too large as too small but counted in
    # full on both sides of the quotient; then half a step of f16 below 2
    g = torch.Generator(device="cuda").manual_seed(d + len(shape))
    L = 131072
    k = torch.randn(L, d, generator=g, device="cuda").to(DT[cache])
    v = (torch.rand(L, d, generator=g, device="cuda") * 0.1 + 1.9).to(DT[cache])
    q = torch.randn(*shape, d, generator=g, device="cuda").to(DT[cache])
    got, want = attend(q, k, v, "f16", shared)
    tol = 2.0 * (1024 * 2.0 ** -23 + 2 * (2.0 ** -16 + 2.0 ** -20)) + 2.0 ** -11
    assert (got - want).abs().max() <= tol, ((got - want).abs().max(), tol)


@pytest.mark.parametrize("layout", S.LAYOUTS)
@pytest.mark.parametrize("cache,out,terms", S.TYPES)
@pytest.mark.parametrize("d", [128, 256])
def test_every_term_of_a_query_counts(d, cache, out, terms, layout):
    c = S.query_case(cache, out, terms, layout, d)
    want = c.want()[0]
    near(c.run(), want, np.full_like(want, S.query_bound(c, terms)))


@pytest.mark.parametrize("layout", S.LAYOUTS)
@pytest.mark.parametrize("cache,out,terms", S.WEIGHT_TYPES)
@pytest.mark.parametrize("d", [128, 256])
def test_every_term_of_a_weight_counts(d, cache, out, terms, layout):
    c = S.weight_case(cache, out, terms, layout, d)
    want = c.want()[0]
    near(c.run() / want, np.ones_like(want), np.full_like(want, S.weight_bound(c, terms)))
