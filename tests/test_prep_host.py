"""Refusals of decode_attn_rope_append and its binding, and the angles' table (no GPU)."""
import ctypes
import math
import os
import subprocess
import tempfile
from fractions import Fraction

import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def shapes(**kw):
    a = N.DaPrep()
    a.n_tokens, a.n_heads, a.n_kv_heads, a.head_dim, a.v_dim = 4, 8, 2, 128, 128
    a.block_size, a.num_blocks = 16, 3
    a.src_dtype, a.q_dtype, a.cache_dtype, a.w_dtype = N.DA_BF16, N.DA_F32, N.DA_F16, N.DA_F32
    a.norm, a.eps = 1, 1e-6
    for s in "qkv":
        setattr(a, f"{s}_src_stride", 12 * 128)
        setattr(a, f"{s}_src_head_stride", 128)
    a.q_out_stride, a.q_out_head_stride = 8 * 128, 128
    for s in "kv":
        setattr(a, f"{s}_block_stride", 16 * 256)
        setattr(a, f"{s}_pos_stride", 256)
        setattr(a, f"{s}_head_stride", 128)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def rope(**kw):
    r = N.DaRope()
    r.turns, r.rot_dim, r.n_axes, r.factor = 4096, 128, 1, 1.0
    for k, v in kw.items():
        setattr(r, k, v)
    return r


P = 1 << 20     # an aligned address that no call below reaches


def call(lib, a, r, ptrs=None):
    x = dict(q=P, k=P, v=P, positions=P, slot_map=P, q_out=P, k_pool=P, v_pool=P)
    x.update(ptrs or {})
    rc = lib.decode_attn_rope_append(ctypes.byref(a), ctypes.byref(r), *x.values(), None)
    return rc, lib.decode_attn_last_error().decode()


@pytest.mark.parametrize("field,value,word", [
    ("n_tokens", -1, "n_tokens"), ("n_tokens", (1 << 30) + 1, "n_tokens"),
    ("n_heads", 0, "n_heads"), ("n_kv_heads", 0, "n_kv_heads"), ("n_heads", 70000, "n_heads"),
    ("head_dim", 0, "head_dim"), ("head_dim", 132, "head_dim"), ("head_dim", 264, "head_dim"),
    ("v_dim", 4, "v_dim"), ("block_size", 0, "block_size"), ("num_blocks", 0, "num_blocks"),
    ("src_dtype", N.DA_E4M3, "types"), ("q_dtype", 9, "types"), ("cache_dtype", N.DA_E5M2, "types"),
    ("norm", 2, "norm"), ("eps", -1.0, "eps"), ("eps", math.nan, "eps"), ("eps", math.inf, "eps"),
    ("weight_offset", math.nan, "weight_offset"),
    ("q_src_stride", 12 * 128 + 1, "source"), ("v_src_head_stride", -8, "source"),
    ("q_out_stride", 0, "q_out"), ("q_out_head_stride", 126, "q_out"),
    ("k_pos_stride", 0, "pool"), ("v_block_stride", 16 * 256 + 4, "pool"),
])
def test_refuses_shapes(lib, field, value, word):
    rc, msg = call(lib, shapes(**{field: value}), rope())
    assert rc == N.DA_EINVAL and word in msg and msg.startswith("rope_append:"), msg


@pytest.mark.parametrize("kw,word", [
    (dict(rot_dim=-16), "rot_dim"), (dict(rot_dim=24), "rot_dim"), (dict(rot_dim=144), "rot_dim"),
    (dict(n_axes=0), "n_axes"), (dict(n_axes=9), "n_axes"), (dict(factor=math.nan), "factor"),
    (dict(factor=math.inf), "factor"), (dict(turns=0), "turns"), (dict(turns=4), "aligned"),
])
def test_refuses_rotations(lib, kw, word):
    rc, msg = call(lib, shapes(), rope(**kw))
    assert rc == N.DA_EINVAL and word in msg, msg


def test_refuses_an_axis_past_the_last(lib):
    r = rope(n_axes=2)
    r.axis[63] = 2
    rc, msg = call(lib, shapes(), r)
    assert rc == N.DA_EINVAL and "axis" in msg
    r.rot_dim = 64                       # (entries past the pairs are not looked at)
    rc, msg = call(lib, shapes(n_tokens=0), r)
    assert rc == N.DA_OK, msg


@pytest.mark.parametrize("kw,word", [
    (dict(q_weight=P + 8), "weights"), (dict(q_weight=P, w_dtype=7), "w_dtype"),
    (dict(k_weight=P, k_weight_head_stride=-4), "weight strides"),
    (dict(k_weight=P, k_weight_head_stride=2), "weight strides"),
])
def test_refuses_weights(lib, kw, word):
    rc, msg = call(lib, shapes(**kw), rope())
    assert rc == N.DA_EINVAL and word in msg, msg


@pytest.mark.parametrize("name", ["q", "k", "v", "q_out", "k_pool", "v_pool", "positions"])
def test_refuses_pointers(lib, name):
    rc, msg = call(lib, shapes(), rope(), {name: 0})
    assert rc == N.DA_EINVAL and "NULL" in msg
    rc, msg = call(lib, shapes(), rope(), {name: P + 4})
    assert rc == N.DA_EINVAL and "aligned" in msg
    rc, msg = call(lib, shapes(), rope(), {"slot_map": P + 4})
    assert rc == N.DA_EINVAL and "aligned" in msg


def test_null_structs_and_no_tokens(lib):
    assert lib.decode_attn_rope_append(None, ctypes.byref(rope()), *[P] * 8, None) == N.DA_EINVAL
    assert lib.decode_attn_rope_append(ctypes.byref(shapes()), None, *[P] * 8, None) == N.DA_EINVAL
    rc, msg = call(lib, shapes(n_tokens=0), rope(), dict(q=0, k=0))
    assert rc == N.DA_OK, msg


def test_struct_layout_matches_the_c_compiler():
    fields = [f"offsetof(da_rope_t, {n})" for n, _ in N.DaRope._fields_] + \
             [f"offsetof(da_prep_t, {n})" for n, _ in N.DaPrep._fields_] + \
             ["sizeof(da_rope_t)", "sizeof(da_prep_t)"]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "split_kv_decode.h"\nint main(void) {\n' \
        + "".join(f'  printf("%zu ", {f});\n' for f in fields) + "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    want = [getattr(N.DaRope, n).offset for n, _ in N.DaRope._fields_] + \
           [getattr(N.DaPrep, n).offset for n, _ in N.DaPrep._fields_] + \
           [ctypes.sizeof(N.DaRope), ctypes.sizeof(N.DaPrep)]
    assert got == want


def two_pi():
    """2 pi as a fraction, by Machin's formula in whole numbers."""
    one = 10 ** 60

    def arctan_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return Fraction(2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 2.0])
def test_turns_are_the_frequencies_in_whole_numbers(theta):
    freqs = [theta ** (-i / 32) for i in range(32)] + [0.0, -0.25, 7.5, 100.0, 1e-9, 6.25, -6.5, 3.0]
    r = A.make_rope(torch.tensor(freqs, dtype=torch.float64), device="cpu")
    for f, t in zip(freqs, r.table.tolist()):
        exact = (Fraction(f) / two_pi() * 2 ** 64) % 2 ** 64
        off = abs(exact - t % 2 ** 64)
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 20)


def test_make_rope_refuses():
    with pytest.raises(ValueError, match="multiple of 8"):
        A.make_rope([1.0] * 7, device="cpu")
    with pytest.raises(ValueError, match="multiple of 8"):
        A.make_rope([1.0] * 136, device="cpu")
    with pytest.raises(ValueError, match="finite"):
        A.make_rope([math.inf] * 8, device="cpu")
    for axes in ([0] * 7, [0] * 7 + [8], [-1] * 8):
        with pytest.raises(ValueError, match="axes"):
            A.make_rope([1.0] * 8, axes=axes, device="cpu")


def rows(T=4, hq=8, hkv=2, d=128, dt=torch.bfloat16):
    return [torch.zeros(T, h, d, dtype=dt) for h in (hq, hkv, hkv, hq)] + \
        [torch.zeros(3, 16, hkv, d, dtype=dt) for _ in range(2)]


def test_make_prep_refuses():
    r = A.make_rope([1.0] * 64, device="cpu")
    q, k, v, qo, kp, vp = rows()
    A.make_prep(q, k, v, qo, kp, vp, r, eps=1e-6, q_weight=torch.ones(128))
    bad = [
        ((q[0], k, v, qo, kp, vp), {}, "rows must be"),
        ((q, k, v, qo[:3], kp, vp), {}, "agree"),
        ((q, k[:3], v[:3], qo, kp, vp), {}, "agree"),
        ((q, k, v[:, :1], qo, kp, vp), {}, "agree"),
        ((q, k, v, qo, kp[:, :, :1], vp[:, :, :1]), {}, "heads and width"),
        ((q, k.float(), v, qo, kp, vp), {}, "one type"),
        ((q, k, v, qo, kp, vp.float()), {}, "of one"),
        ((q.transpose(1, 2).contiguous().transpose(1, 2), k, v, qo, kp, vp), {}, "contiguous"),
        ((q, k, v, qo, kp, vp), dict(q_weight=torch.ones(128)), "eps"),
        ((q, k, v, qo, kp, vp), dict(eps=1e-6, q_weight=torch.ones(64)), "q_weight"),
        ((q, k, v, qo, kp, vp), dict(eps=1e-6, k_weight=torch.ones(8, 128)), "k_weight"),
        ((q, k, v, qo, kp, vp), dict(eps=1e-6, q_weight=torch.ones(128),
                                     k_weight=torch.ones(128).half()), "one type"),
    ]
    for args, kw, word in bad:
        with pytest.raises(ValueError, match=word):
            A.make_prep(*args, r, **kw)


def test_the_call_refuses_tensors_of_other_shapes():
    r = A.make_rope([1.0] * 64, axes=[0] * 32 + [1] * 32, device="cpu")
    q, k, v, qo, kp, vp = rows()
    prep = A.make_prep(q, k, v, qo, kp, vp, r)
    pos, slots = torch.zeros(2, 4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)
    for p in (pos[0], pos.int(), pos[:, :3], torch.zeros(4, 2, dtype=torch.int64).t()):
        with pytest.raises(TypeError, match="positions"):
            A.decode_attn_rope_append(prep, q, k, v, p, slots, qo, kp, vp)
    for s in (slots[:3], slots.int(), torch.zeros(8, dtype=torch.int64)[::2]):
        with pytest.raises(TypeError, match="slot_map"):
            A.decode_attn_rope_append(prep, q, k, v, pos, s, qo, kp, vp)
    with pytest.raises(TypeError, match="CUDA"):
        A.decode_attn_rope_append(prep, q, k, v, pos, slots, qo, kp, vp)
