"""The inputs of tests/scored_terms.py tell a kernel that leaves a term out (no GPU)."""
import numpy as np
import pytest
import torch

from tests import scored_terms as S


@pytest.mark.parametrize("layout", S.LAYOUTS)
@pytest.mark.parametrize("cache,out,terms", S.TYPES)
def test_a_query_without_its_last_term_is_told(cache, out, terms, layout):
    c = S.query_case(cache, out, terms, layout, 128)
    want, tol = c.want()[0], S.query_bound(c, terms)
    q = c.q.numpy()
    for used, told in ((terms, False), (terms - 1, True)):
        c.q = torch.tensor(S.in_terms(q, cache, used), dtype=torch.float32)
        err = np.abs(c.want()[0] - want)
        assert (err > 2 * tol).all() if told else (err == 0).all(), (used, err.max(), tol)


@pytest.mark.parametrize("layout", S.LAYOUTS)
@pytest.mark.parametrize("cache,out,terms", S.WEIGHT_TYPES)
def test_a_weight_without_its_last_term_is_told(cache, out, terms, layout):
    c = S.weight_case(cache, out, terms, layout, 128)
    want, tol = c.want()[0], S.weight_bound(c, terms)
    for used, told in ((terms, False), (terms - 1, True)):
        err = np.abs(S.weight_share(c, terms, used) / want - 1)
        assert (err > 2 * tol).all() if told else (err < S.TERMS[cache, terms] + 1e-12).all(), \
            (used, err.max(), tol)
