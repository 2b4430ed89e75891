"""The combines over an 8-bit plan whose split kernel writes the output itself (CPU)."""
import ctypes

import pytest

from split_kv_decode_gb300 import _native as N
from tests.test_kv8_host import FAKE, P, args, lib, plan  # noqa: F401


@pytest.mark.parametrize("flags,status", [(0, N.DA_EINVAL), (N.DA_FLAG_ONE_LAUNCH, N.DA_EINVAL)])
@pytest.mark.parametrize("dt", [N.DA_E4M3, N.DA_E5M2])
def test_one_split_leaves_no_partials_to_combine(lib, flags, status, dt):  # noqa: F811
    a = args(8, 8, 128, dt, cap=64, batch=2)
    a.force_splits, a.flags = 1, flags
    rc, p = plan(lib, a, [40, 64])
    assert rc == 0 and p.max_splits == 1
    r = ctypes.byref
    pj = N.DaProj()
    pj.w, pj.out_dim = 1 << 20, 64
    for rc in (lib.decode_attn_combine(r(a), r(p), FAKE, FAKE, None),
               lib.decode_attn_combine_ranks(r(a), r(p), FAKE, 2, FAKE, None),
               lib.decode_attn_combine_proj(r(a), r(p), r(pj), FAKE, 1, FAKE, None)):
        assert rc == status
        assert b"DA_FLAG_NO_COMBINE" in lib.decode_attn_last_error()


def test_a_plan_that_has_partials_is_taken(lib):  # noqa: F811
    # (as far as the next check: a workspace that is misaligned)
    for flags, splits, dt in ((N.DA_FLAG_NO_COMBINE, 1, N.DA_E4M3), (0, 2, N.DA_E4M3)):
        a = args(8, 8, 128, dt, cap=512, batch=1)
        a.force_splits, a.flags = splits, flags
        rc, p = plan(lib, a, [512])
        assert rc == 0 and p.max_splits == splits
        assert lib.decode_attn_combine(ctypes.byref(a), ctypes.byref(p), P((1 << 20) + 8), FAKE,
                                       None) == N.DA_EINVAL
        assert b"misaligned" in lib.decode_attn_last_error()
