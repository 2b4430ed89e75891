"""Host side of the 8-bit cache calls (CPU): struct layouts, plans, refusals, and the
references the GPU tests compare with."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import build as B
from tests.kv8_util import MAX, TDT, Blocks, append_reference, code_values, page_exponent, round_to

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE = P(1 << 20)                                 # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def test_struct_layouts_match_the_c_compiler():
    structs = {"da_tables_t": N.DaTables, "da_append_t": N.DaAppend, "da_scales_t": N.DaScales}
    body = "".join(f'printf("%zu ", sizeof({c}));' + "".join(
        f'printf("%zu ", offsetof({c}, {f}));' for f, _ in s._fields_)
        for c, s in structs.items())
    src = f'#include <stdio.h>\n#include <stddef.h>\n#include "split_kv_decode.h"\n' \
          f'int main(void) {{ {body} return 0; }}'
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    want = []
    for s in structs.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert [int(x) for x in got] == want


def args(hq=16, hkv=4, d=256, dt=N.DA_E4M3, cap=4096, batch=1, q_len=1):
    a = N.DaArgs()
    a.batch, a.n_heads, a.n_kv_heads, a.head_dim, a.v_dim = batch, hq, hkv, d, d
    a.capacity, a.kv_dtype, a.out_dtype, a.scale, a.q_len = cap, dt, N.DA_F32, 0.1, q_len
    a.k_pos_stride = a.v_pos_stride = hkv * d
    a.k_head_stride = a.v_head_stride = d
    a.k_batch_stride = a.v_batch_stride = cap * hkv * d
    return a


def plan(lib, a, lens):
    p, ls = N.DaPlan(), (ctypes.c_int32 * len(lens))(*lens)
    return lib.decode_attn_plan(ctypes.byref(a), ctypes.cast(ls, P), 152, ctypes.byref(p)), p


def test_plans(lib):
    for dt in (N.DA_E4M3, N.DA_E5M2):
        for hq, hkv, d, q_len in ((16, 4, 256, 1), (8, 8, 128, 1), (128, 1, 128, 1), (10, 2, 256, 5)):
            a = args(hq, hkv, d, dt, cap=200000, batch=2, q_len=q_len)
            rc, p = plan(lib, a, [150000, q_len])
            assert rc == 0 and p.kernel == N.DA_KERNEL_GQA_8BIT
            assert all(c % p.tile == 0 for c in p.chunk[:2])
            assert p.n_items % p.total_splits == 0 and p.grid <= 152
            assert p.workspace_bytes == lib.decode_attn_workspace_bytes(ctypes.byref(p))


def test_plan_cost_is_the_makespan_of_items_by_size(lib):
    # sequences by the length of their items, the longest first; item i is the (i % grid)-th
    # of its round, odd rounds go from the last CTA to the first
    import random
    rnd = random.Random(12)
    for _ in range(60):
        batch, hkv = rnd.choice([1, 2, 5, 16, 64, 256]), rnd.choice([1, 2, 4, 8])
        lens = [int(2 ** rnd.uniform(0, rnd.choice([6, 13, 17]))) for _ in range(batch)]
        a = args(hkv * 4, hkv, 128, cap=max(lens), batch=batch)
        a.force_splits = rnd.choice([0, 0, 0, 7])
        rc, p = plan(lib, a, lens)
        assert rc == 0
        load, i = [0] * p.grid, 0
        for b in sorted(range(batch), key=lambda b: -min(p.chunk[b], lens[b])):
            for s in range(p.n_splits[b]):
                for _ in range(hkv):
                    j = i % p.grid if i // p.grid % 2 == 0 else p.grid - 1 - i % p.grid
                    load[j] += min(p.chunk[b], lens[b] - s * p.chunk[b]) + 4 * p.tile
                    i += 1
        assert i == p.n_items and p.est_cost == max(load)


@pytest.mark.parametrize("lens,hkv,splits", [([256], 4, 1), ([300] * 4, 2, 1), ([713], 2, 6),
                                             ([4096], 2, 32), ([1024] * 8, 8, 1)])
def test_plans_count_the_combine(lib, lens, hkv, splits):
    # four tiles for the combine that a plan of several splits needs
    a = args(4 * hkv, hkv, 128, cap=max(lens), batch=len(lens))
    rc, p = plan(lib, a, lens)
    assert rc == 0 and p.max_splits == splits
    a.flags = N.DA_FLAG_NO_COMBINE           # the partials are wanted: no call is saved
    rc, p = plan(lib, a, lens)
    assert rc == 0 and p.max_splits > 1


def test_plans_of_ragged_batches_are_balanced(lib):
    lens = [2999, 17, 1500, 3500, 64, 2048, 777, 1]
    rc, p = plan(lib, args(16, 16, 128, cap=4096, batch=8), lens)
    assert rc == 0 and p.est_cost <= 1.3 * (sum(lens) * 16 / 152 + 4 * p.tile)


@pytest.mark.parametrize("change,status", [
    (dict(d=64), N.DA_EUNSUPPORTED), (dict(d=576), N.DA_EUNSUPPORTED),
    (dict(hq=129, hkv=1, d=128), N.DA_EUNSUPPORTED), (dict(hq=66, hkv=1, q_len=2), N.DA_EUNSUPPORTED)])
def test_plan_refusals(lib, change, status):
    assert plan(lib, args(**change), [100])[0] == status
    assert b"8-bit" in lib.decode_attn_last_error()


def test_plan_refuses_unaligned_strides_and_8bit_outputs(lib):
    a = args()
    a.v_pos_stride += 8
    assert plan(lib, a, [100])[0] == N.DA_EUNSUPPORTED
    for dt in (N.DA_E4M3, N.DA_E5M2, 5):
        a = args(dt=N.DA_F16)
        a.out_dtype = dt
        assert plan(lib, a, [100])[0] == N.DA_EINVAL


def test_an_mla_shape_is_refused(lib):
    a = args(96, 1, 576)
    a.v_dim = 512
    assert plan(lib, a, [100])[0] == N.DA_EUNSUPPORTED


def test_calls_without_scales_refuse_an_8bit_cache(lib):
    a = args()
    rc, p = plan(lib, a, [100])
    assert rc == 0
    r = ctypes.byref
    d, pj = N.DaDev(), N.DaProj()
    pj.w, pj.out_dim = 1 << 20, 64
    tail = (FAKE, FAKE, FAKE, FAKE, FAKE, p.workspace_bytes, None)
    for rc in (lib.decode_attn_splitk_ex(r(a), r(p), *tail),
               lib.decode_attn_splitk_dev(r(a), r(p), r(d), *tail),
               lib.decode_attn_splitk_proj(r(a), r(p), r(pj), *tail)):
        assert rc == N.DA_EUNSUPPORTED
        assert b"decode_attn_splitk_8bit" in lib.decode_attn_last_error()


def _dev(a, page=16, width=300, blocks=40):
    d = N.DaDev()
    d.block_table, d.max_blocks_per_seq, d.block_size, d.num_blocks = 1 << 20, width, page, blocks
    d.k_block_stride = d.v_block_stride = page * a.k_pos_stride
    return d


def _scales():
    s = N.DaScales()
    s.k_scale = s.v_scale = 1 << 20
    s.k_block_stride = s.v_block_stride = 4
    s.k_head_stride = s.v_head_stride = 1
    return s


@pytest.mark.parametrize("spoil,status", [
    (lambda a, d, s: setattr(d, "block_table", None), N.DA_EINVAL),
    (lambda a, d, s: setattr(d, "block_table", (1 << 20) + 2), N.DA_EINVAL),
    (lambda a, d, s: setattr(d, "seq_lens", (1 << 20) + 2), N.DA_EINVAL),
    (lambda a, d, s: setattr(d, "block_size", 24), N.DA_EUNSUPPORTED),
    (lambda a, d, s: setattr(d, "num_blocks", 0), N.DA_EINVAL),
    (lambda a, d, s: setattr(d, "max_blocks_per_seq", 6), N.DA_EINVAL),
    (lambda a, d, s: setattr(d, "k_block_stride", 100), N.DA_EUNSUPPORTED),
    (lambda a, d, s: setattr(s, "v_scale", None), N.DA_EINVAL),
    (lambda a, d, s: setattr(s, "k_scale", (1 << 20) + 1), N.DA_EINVAL),
    (lambda a, d, s: setattr(s, "k_head_stride", 0), N.DA_EINVAL),
    (lambda a, d, s: setattr(a, "kv_dtype", N.DA_F16), N.DA_EUNSUPPORTED),
    (lambda a, d, s: setattr(a, "n_heads", 15), N.DA_EINVAL),
])
def test_attention_refusals(lib, spoil, status):
    a = args()
    rc, p = plan(lib, a, [100])
    d, s = _dev(a), _scales()
    spoil(a, d, s)
    r = ctypes.byref
    assert lib.decode_attn_splitk_8bit(r(a), r(p), r(d), r(s), FAKE, FAKE, FAKE, FAKE, FAKE,
                                       p.workspace_bytes, None) == status
    assert lib.decode_attn_last_error()


def test_attention_refuses_null_misaligned_and_small(lib):
    a = args()
    rc, p = plan(lib, a, [100])
    d, s, r, n = _dev(a), _scales(), ctypes.byref, p.workspace_bytes
    f = lib.decode_attn_splitk_8bit
    assert f(r(a), r(p), None, r(s), FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == N.DA_EINVAL
    assert f(r(a), r(p), r(d), None, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == N.DA_EINVAL
    for i in range(5):
        ptrs = [FAKE] * 5
        ptrs[i] = None
        assert f(r(a), r(p), r(d), r(s), *ptrs, n, None) == N.DA_EINVAL
        ptrs[i] = P((1 << 20) + 8)
        assert f(r(a), r(p), r(d), r(s), *ptrs, n, None) == N.DA_EINVAL
    assert f(r(a), r(p), r(d), r(s), *[FAKE] * 5, n - 1, None) == N.DA_ENOSPACE
    p.chunk[0] += 8
    assert f(r(a), r(p), r(d), r(s), *[FAKE] * 5, n, None) == N.DA_EINVAL


def _tables(**kw):
    t = N.DaTables()
    for f in ("seq_lens", "seq_lens_out", "block_table", "free_list", "state", "state_out"):
        setattr(t, f, 1 << 20)
    t.batch, t.max_blocks_per_seq, t.block_size, t.num_blocks = 4, 8, 16, 32
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=257), dict(block_size=0),
                                dict(max_blocks_per_seq=0), dict(num_blocks=0),
                                dict(batch=256, max_blocks_per_seq=1 << 24), dict(state=None),
                                dict(seq_lens=None), dict(free_list=(1 << 20) + 2)])
def test_tables_refusals(lib, kw):
    t = _tables(**kw)
    assert lib.decode_attn_grow_tables(ctypes.byref(t), FAKE, FAKE, 8, FAKE, None) == N.DA_EINVAL
    assert lib.decode_attn_last_error()


def test_tables_refuse_null_and_sizes(lib):
    t, f = _tables(), lib.decode_attn_grow_tables
    r = ctypes.byref(t)
    assert f(None, FAKE, FAKE, 8, None, None) == N.DA_EINVAL
    assert f(r, None, FAKE, 8, None, None) == N.DA_EINVAL
    assert f(r, FAKE, None, 8, None, None) == N.DA_EINVAL
    assert f(r, FAKE, FAKE, -1, None, None) == N.DA_EINVAL
    assert f(r, FAKE, FAKE, 1 << 31, None, None) == N.DA_EINVAL
    assert f(r, FAKE, P((1 << 20) + 4), 8, None, None) == N.DA_EINVAL
    assert lib.decode_attn_tables_status(None, None) == N.DA_EINVAL


def _append(**kw):
    a = N.DaAppend()
    a.n_tokens, a.n_kv_heads, a.head_dim, a.v_dim, a.block_size, a.num_blocks = 4, 2, 128, 128, 16, 8
    a.src_dtype, a.code_dtype = N.DA_BF16, N.DA_E4M3
    for f, _ in N.DaAppend._fields_:
        if f.endswith("stride"):
            setattr(a, f, 256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(n_tokens=-1), dict(n_tokens=(1 << 30) + 1),
                                dict(n_kv_heads=0), dict(head_dim=24),
                                dict(head_dim=0), dict(v_dim=1040), dict(block_size=0),
                                dict(num_blocks=0), dict(src_dtype=N.DA_E4M3), dict(src_dtype=9),
                                dict(code_dtype=N.DA_F16), dict(k_src_stride=4),
                                dict(v_src_head_stride=-8), dict(k_pos_stride=8),
                                dict(v_head_stride=0), dict(k_scale_block_stride=0),
                                dict(block_size=1 << 26, v_dim=1024)])
def test_append_refusals(lib, kw):
    a = _append(**kw)
    assert lib.decode_attn_append_8bit(ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                       None) == N.DA_EINVAL
    assert lib.decode_attn_last_error()


def test_append_refuses_null_and_misaligned_and_takes_no_rows(lib):
    a, f = _append(), lib.decode_attn_append_8bit
    for i in range(7):
        ptrs = [FAKE] * 7
        ptrs[i] = None
        assert f(ctypes.byref(a), *ptrs, None) == N.DA_EINVAL
        ptrs[i] = P((1 << 20) + 2)
        assert f(ctypes.byref(a), *ptrs, None) == N.DA_EINVAL
    assert f(None, *[FAKE] * 7, None) == N.DA_EINVAL
    none = _append(n_tokens=0)
    assert f(ctypes.byref(none), *[None] * 7, None) == N.DA_OK


# ---- the references ----------------------------------------------------------------

@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
def test_code_values_and_rounding_are_torchs(code):
    u = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(code_values(code), u.view(TDT[code]).double().numpy())
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 3
    x = torch.cat([x, torch.exp2(torch.linspace(-20, 8.7, 5000)), torch.tensor([0.0, -0.0, 2.0 ** -10])])
    np.testing.assert_array_equal(round_to(x.double().numpy(), code), x.to(TDT[code]).double().numpy())
    assert round_to(np.array([np.inf, -1e9, np.nan]), code)[0] == MAX[code]


def test_page_exponent_is_the_least():
    rng = np.random.default_rng(0)
    for code in ("e4m3", "e5m2"):
        for a in np.exp(rng.uniform(-60, 80, 300)):
            e = page_exponent(a, code)
            assert a <= MAX[code] * 2.0 ** e and (e == -100 or a > MAX[code] * 2.0 ** (e - 1))


def test_append_reference_by_hand():
    val, sc = np.zeros((2, 4, 1, 1)), np.ones((2, 1))
    val[0, 0], sc[0] = 448.0, 1.0
    append_reference(np.array([[[900.0]], [[3.0]], [[0.5]]]), [1, 2, 4], val, sc, 4, "e4m3")
    assert sc.tolist() == [[4.0], [2.0 ** -9]]    # 900 <= 448 * 4; 0.5 <= 448 * 2^-9 = 0.875
    assert val[0, :3, 0, 0].tolist() == [112.0, 224.0, 0.75] and val[1, 0, 0, 0] == 256.0


def test_blocks_reference_by_hand():
    b = Blocks(2, 4, 3, 2)
    assert b.grow([3, 1], 6) == (0, [0, 1, 2, 4, -1, -1], [0, 3, 4])
    assert b.grow([0, 4], 6)[0] == 3              # two blocks, one left
    assert b.grow([-1, 4], 6) == (0, [5, 2, 3, 0, -1, -1], [0, 0, 4])
    assert b.free == [3] and b.lens == [0, 5]
