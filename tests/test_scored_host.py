"""Plans and refusals of scored attention and its binding (no GPU)."""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20      # an aligned address that no call below reaches
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def args(batch=2, hq=8, hkv=2, d=128, cap=4096, q_len=0, kv=N.DA_BF16, out=N.DA_BF16, **kw):
    a = N.DaArgs()
    a.batch, a.n_heads, a.n_kv_heads, a.head_dim, a.v_dim = batch, hq, hkv, d, d
    a.capacity, a.q_len, a.kv_dtype, a.out_dtype, a.scale = cap, q_len, kv, out, d ** -0.5
    for s in "kv":
        setattr(a, f"{s}_pos_stride", hkv * d)
        setattr(a, f"{s}_head_stride", d)
        setattr(a, f"{s}_batch_stride", cap * hkv * d)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def score(**kw):
    s = N.DaScore()
    s.q_dtype = N.DA_BF16
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def dev(lib, block_size=16, num_blocks=64, max_blocks=256, a=None, **kw):
    x = N.DaDev()
    x.block_table, x.max_blocks_per_seq = P, max_blocks
    x.block_size, x.num_blocks = block_size, num_blocks
    a = a or args()
    x.k_block_stride = x.v_block_stride = block_size * a.n_kv_heads * a.head_dim
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def plan(lib, a, s, lens, sms=152):
    p = N.DaScoredPlan()
    x = (ctypes.c_int32 * max(1, len(lens)))(*lens)
    rc = lib.decode_attn_plan_scored(ref(a), ref(s), ctypes.cast(x, ctypes.c_void_p), sms, ref(p))
    return rc, p


def run(lib, a, p, s, d=None, q=P, k=P, v=P, out=P, ws=P, nbytes=None):
    rc = lib.decode_attn_splitk_scored(ref(a), ref(p), None if d is None else ref(d), ref(s), q, k,
                                       v, out, ws, p.workspace_bytes if nbytes is None else nbytes,
                                       None)
    return rc, lib.decode_attn_last_error().decode()


@pytest.mark.parametrize("kw,word", [
    (dict(kv=N.DA_F32), "f16 and bf16"), (dict(kv=N.DA_E4M3), "f16 and bf16"),
    (dict(d=64), "128 or 256"), (dict(d=192), "128 or 256"), (dict(v_dim=256), "128 or 256"),
    (dict(hq=129, hkv=1), "128 rows"), (dict(hq=64, hkv=1, q_len=3), "128 rows"),
    (dict(k_pos_stride=260), "16 bytes"), (dict(v_head_stride=132), "16 bytes"),
    (dict(k_batch_stride=4096 * 256 + 4), "16 bytes"),
    (dict(flags=N.DA_FLAG_ONE_LAUNCH), "flags"), (dict(flags=N.DA_FLAG_NO_COMBINE), "flags"),
    (dict(cap=(1 << 30) + 8), "2^30"),
])
def test_refuses_arguments(lib, kw, word):
    a = args(**kw)
    a.v_dim = kw.get("v_dim", a.head_dim)
    rc, _ = plan(lib, a, score(q_dtype=a.kv_dtype), [8, 8])
    assert rc != N.DA_OK and word in lib.decode_attn_last_error().decode(), \
        lib.decode_attn_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(q_dtype=N.DA_F16), "q_dtype"), (dict(q_dtype=9), "q_dtype"),
    (dict(softcap=-1.0), "softcap"), (dict(softcap=math.nan), "softcap"),
    (dict(softcap=math.inf), "softcap"), (dict(window=-1), "window"), (dict(keep=-1), "keep"),
    (dict(shared_len=-16), "shared_len"), (dict(shared_len=16), "shared_table"),
    (dict(shared_len=(1 << 30) + 16, shared_table=P), "shared_len"),
    (dict(shared_len=16, shared_table=P, window=5), "window"),
    (dict(shared_len=16, shared_table=P, keep=5), "keep"),
    (dict(shared_len=16, shared_table=P, starts=P), "starts"),
    (dict(shared_len=16, shared_table=P, keep_lens=P), "starts"),
    (dict(slopes=P + 2), "aligned"), (dict(starts=P + 2), "aligned"),
    (dict(keep_lens=P + 1), "aligned"), (dict(shared_table=P + 2), "aligned"),
])
def test_refuses_scores(lib, kw, word):
    rc, _ = plan(lib, args(), score(**kw), [8, 8])
    assert rc != N.DA_OK and word in lib.decode_attn_last_error().decode(), \
        lib.decode_attn_last_error()


@pytest.mark.parametrize("cap,fine", [
    (0.0, True), (2.0 ** -60, True), (2.0 ** 60, True), (30.0, True), (-0.0, True),
    (2.0 ** -61, False), (1e-39, False), (2.0 ** 61, False), (3e38, False)])
def test_caps_whose_products_leave_the_range_are_refused(lib, cap, fine):
    # (times log2 e 3e38 is infinite, and so is a score over 1e-39)
    rc, _ = plan(lib, args(), score(softcap=cap), [8, 8])
    assert (rc == N.DA_OK) == fine
    assert fine or "softcap" in lib.decode_attn_last_error().decode()


def test_refuses_lengths_and_null(lib):
    for lens in ([0, 8], [8, 4097], [-1, 8]):
        assert plan(lib, args(), score(), lens)[0] == N.DA_EINVAL
    assert plan(lib, args(q_len=4), score(), [3, 8])[0] == N.DA_EINVAL
    p = N.DaScoredPlan()
    x = (ctypes.c_int32 * 2)(8, 8)
    for a, s, lens, to in ((None, score(), x, p), (args(), None, x, p), (args(), score(), None, p),
                           (args(), score(), x, None)):
        rc = lib.decode_attn_plan_scored(a and ref(a), s and ref(s),
                                         lens and ctypes.cast(lens, ctypes.c_void_p), 152,
                                         to and ref(to))
        assert rc == N.DA_EINVAL


@pytest.mark.parametrize("kw", [dict(), dict(d=256, hq=24, hkv=4, q_len=4), dict(out=N.DA_F32),
                                dict(d=256, hq=16, hkv=2, out=N.DA_F32), dict(hq=128, hkv=1)])
@pytest.mark.parametrize("skw", [dict(), dict(window=300, keep=20), dict(slopes=P, softcap=30.0),
                                 dict(shared_len=1024, shared_table=P), dict(q_dtype=N.DA_F32),
                                 dict(q_dtype=N.DA_F32, shared_len=5120, shared_table=P)])
@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("sms", [7, 152])
def test_plans_cover_what_is_visible(lib, kw, skw, splits, sms):
    a, s = args(batch=5, cap=70000, **kw), score(**skw)
    a.force_splits = splits
    lens = [70000, 4, 1000, 129, 333]
    rc, p = plan(lib, a, s, lens, sms)
    assert rc == N.DA_OK, lib.decode_attn_last_error()
    T = p.tile
    assert T in (64, 128) and p.kernel == N.DA_KERNEL_GQA_SCORED and p.batch == 5
    assert 1 <= p.grid <= min(sms, p.n_items)
    base = 0
    for b, n in enumerate(lens):
        assert p.seq_lens[b] == n and p.split_base[b] == base
        tiles = -(-n // T)
        if s.window:
            tiles = min(tiles, -(-s.keep // T) + -(-(s.window + max(a.q_len, 1) - 1) // T) + 1)
        own = p.n_splits[b] - p.shared_splits
        assert p.chunk[b] % T == 0 and p.chunk[b] > 0 and own >= 1
        assert (own - 1) * p.chunk[b] < tiles * T <= own * p.chunk[b]
        base += p.n_splits[b]
    assert p.total_splits == base and p.max_splits == max(p.n_splits[:5])
    assert p.shared_len == s.shared_len
    if s.shared_len:
        assert p.shared_splits >= 1 and p.shared_chunk % T == 0
        assert (p.shared_splits - 1) * p.shared_chunk < s.shared_len <= \
            p.shared_splits * p.shared_chunk
    else:
        assert p.shared_splits == 0
    # f32 outputs add a lane's accumulator up at most 48 times a partial (of a window's one row group
    # of few rows, in copies): no slice is longer than all additions of a lane allow
    if a.out_dtype == N.DA_F32:
        assert max(p.chunk[:5]) // 16 <= 48 * 2 * 4


GEOMETRY = r"""
#include <cstdio>
#include "scored.h"
int main()
{
    int d, q, w, own;
    long long shared;
    while (std::scanf("%d %d %d %d %lld", &d, &q, &w, &own, &shared) == 5) {
        const skv::ScoredGeometry g = skv::scored_geometry(d, q, w, own, shared);
        std::printf("%d %d %d\n", g.tile_rows, g.rpad, g.kind == skv::kScoredPacked);
    }
    return 0;
}
"""


def test_no_accumulator_takes_more_additions_than_its_output_bears(lib):
    # the longest slices that the planner makes: one CTA, one split wanted, long contexts. A lane adds a
    # term of 16 positions at a time; copies of its row share a tile's positions, the two
    # accumulators of 128 columns the tiles, and packed rows' terms lie in lanes of their own
    cases = [(d, kv, out, q, rows, shared)
             for d in (128, 256) for kv in (N.DA_F16, N.DA_BF16)
             for out in (N.DA_F32, N.DA_F16, N.DA_BF16) for q in (N.DA_F32, kv)
             for rows, shared in ((1, 0), (8, 0), (9, 0), (16, 0), (20, 0), (33, 0), (40, 0), (65, 0),
                                  (100, 0), (128, 0), (4, 1), (40, 1), (128, 1))]
    batch, cap = 3, 1 << 20
    given, plans = "", []
    for d, kv, out, q, rows, shared in cases:
        a = args(batch=batch, hq=rows, hkv=1, d=d, cap=cap, kv=kv, out=out, force_splits=1)
        s = score(q_dtype=q, shared_len=cap * shared, shared_table=P)
        rc, p = plan(lib, a, s, [cap, 5, cap], 1)
        assert rc == N.DA_OK, lib.decode_attn_last_error()
        plans.append(p)
        terms = 3 if kv == N.DA_BF16 and out == N.DA_F32 else 2
        given += f"{d} {terms if q == N.DA_F32 else 1} {terms} {rows} {batch * rows * shared}\n"
    with tempfile.TemporaryDirectory() as folder:
        c, exe = os.path.join(folder, "t.cpp"), os.path.join(folder, "t")
        open(c, "w").write(GEOMETRY)
        subprocess.run([B._nvcc(), "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", B.SRC, c,
                        "-o", exe], check=True)
        lines = subprocess.run([exe], input=given, capture_output=True, text=True,
                               check=True).stdout.splitlines()
    assert len(lines) == len(cases)
    for (d, kv, out, q, rows, shared), p, line in zip(cases, plans, lines):
        tile_rows, rpad, packed = map(int, line.split())
        terms = 3 if kv == N.DA_BF16 and out == N.DA_F32 else 2
        assert p.tile == (128 if d == 128 and terms == 2 else 64)

        def additions(positions, of):
            of = min(of, tile_rows)
            span = 32 if of <= 32 else 64 if of <= 64 else 128
            copies = 1 if of > 128 else max(1, rpad // span)
            own = 2 if d == 128 and of <= 128 else 1     # accumulators that take the tiles in turn
            tiles = -(-(positions // p.tile) // own)
            return tiles * max(1, p.tile // 16 * (1 if packed else terms) // copies)

        most = {N.DA_F32: 48, N.DA_F16: 1024, N.DA_BF16: 8192}[out]
        slices = [(p.chunk[0], rows)] + [(p.shared_chunk, batch * rows)] * shared
        for positions, of in slices:
            n = additions(positions, of)
            # (and not far fewer, so that long contexts are not cut up for nothing)
            assert most // 3 < n <= most, (d, kv, out, q, rows, shared, positions, n)


def test_refuses_plans_of_other_arguments(lib):
    a, s = args(), score()
    rc, p = plan(lib, a, s, [4000, 100])
    assert rc == N.DA_OK
    for other_a, other_s in ((args(batch=3), s), (args(hq=16), s), (args(hq=64), s),
                             (args(d=256), s), (a, score(window=100)), (args(q_len=2), s),
                             (a, score(shared_len=16, shared_table=P))):
        rc, msg = run(lib, other_a, p, other_s)
        assert rc != N.DA_OK and "plan" in msg, msg
    for field, value in (("grid", 0), ("grid", p.n_items + 1), ("n_items", p.n_items + 1),
                         ("total_splits", 0), ("workspace_bytes", 256), ("tile", 32), ("kernel", 1),
                         ("max_splits", 99), ("shared_splits", 1), ("shared_len", 16)):
        q = N.DaScoredPlan.from_buffer_copy(p)
        setattr(q, field, value)
        rc, msg = run(lib, a, q, s, nbytes=1 << 30)
        assert rc == N.DA_EINVAL and "plan" in msg, (field, msg)
    for field in ("chunk", "n_splits", "split_base"):
        # (a chunk past the sequence's 100 positions is one split, as is the plan's)
        for value in (-128, 0, 64) + (() if field == "chunk" else (1 << 20,)):
            q = N.DaScoredPlan.from_buffer_copy(p)
            if getattr(q, field)[1] == value:
                continue
            getattr(q, field)[1] = value
            rc, msg = run(lib, a, q, s, nbytes=1 << 30)
            assert rc == N.DA_EINVAL, (field, value, msg)


def test_refuses_pointers_workspaces_and_tables(lib):
    a, s = args(), score()
    _, p = plan(lib, a, s, [4000, 100])
    for name in ("q", "k", "v", "out", "ws"):
        rc, msg = run(lib, a, p, s, **{name: 0})
        assert rc == N.DA_EINVAL, (name, msg)
        rc, msg = run(lib, a, p, s, **{name: P + 8})
        assert rc == N.DA_EINVAL and "align" in msg, (name, msg)
    rc, msg = run(lib, a, p, s, nbytes=p.workspace_bytes - 1)
    assert rc == N.DA_ENOSPACE, msg
    rc, msg = run(lib, a, p, s, dev(lib, block_table=0, seq_lens=P + 2))
    assert rc == N.DA_EINVAL and "seq_lens" in msg, msg
    for kw in (dict(block_size=0), dict(num_blocks=0), dict(max_blocks_per_seq=3), dict(block_size=24),
               dict(k_block_stride=12), dict(block_table=P + 2)):
        rc, msg = run(lib, a, p, s, dev(lib, **kw))
        assert rc != N.DA_OK, (kw, msg)
    s = score(shared_len=40, shared_table=P)
    _, p = plan(lib, a, s, [4000, 100])
    rc, msg = run(lib, a, p, s)
    assert rc == N.DA_EINVAL and "block_table" in msg, msg
    rc, msg = run(lib, a, p, s, dev(lib))
    assert rc == N.DA_EINVAL and "multiple" in msg, msg


def test_other_entry_points_refuse_scored_plans(lib):
    a, s = args(), score()
    for splits in (1, 3):
        a.force_splits = splits
        _, p = plan(lib, a, s, [4000, 100])
        pj = N.DaProj()
        pj.w, pj.out_dim = P, 64
        for rc in (lib.decode_attn_combine(ref(a), ref(p), P, P, None),
                   lib.decode_attn_combine_ranks(ref(a), ref(p), P, 2, P, None),
                   lib.decode_attn_combine_proj(ref(a), ref(p), ref(pj), P, 1, P, None),
                   lib.decode_attn_splitk_ex(ref(a), ref(p), P, P, P, P, P, p.workspace_bytes, None)):
            assert rc == N.DA_EINVAL and b"plan" in lib.decode_attn_last_error()
    b = args()
    other = N.DaPlan()
    x = (ctypes.c_int32 * 2)(4000, 100)
    assert lib.decode_attn_plan(ref(b), ctypes.cast(x, ctypes.c_void_p), 152, ref(other)) == N.DA_OK
    q = N.DaScoredPlan()
    ctypes.memmove(ref(q), ref(other), ctypes.sizeof(other))
    rc, msg = run(lib, b, q, s)
    assert rc == N.DA_EINVAL and "plan" in msg


def test_struct_layout_matches_the_c_compiler():
    fields = [f"offsetof(da_score_t, {n})" for n, _ in N.DaScore._fields_] + \
             [f"offsetof(da_scored_plan_t, {n})" for n, _ in N.DaScoredPlan._fields_] + \
             ["offsetof(da_scored_plan_t, base)", "sizeof(da_score_t)", "sizeof(da_scored_plan_t)"]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "split_kv_decode.h"\nint main(void) {\n' \
        + "".join(f'  printf("%zu ", {f});\n' for f in fields) + "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    want = [getattr(N.DaScore, n).offset for n, _ in N.DaScore._fields_] + \
           [getattr(N.DaScoredPlan, n).offset for n, _ in N.DaScoredPlan._fields_] + \
           [0, ctypes.sizeof(N.DaScore), ctypes.sizeof(N.DaScoredPlan)]
    assert got == want


ORDER = r"""
#include <cassert>
#include <vector>
#include "scored.h"
int main()
{
    using namespace skv;
    for (int grid : {1, 2, 3, 7, 152})
        for (int all : {0, 1, 2, 5, 6, 7, 14, 128, 152, 153, 300, 304})
            for (int lead : {1, 2, 3, 5, 1024})
                for (int own : {1, 4, 64, 500, 2048}) {
                    const ScoredOrder o = {grid, all, lead};
                    const int n = all + own;
                    std::vector<int> seen(n, 0);
                    for (int c = 0; c < grid; ++c)
                        for (int r = 0;; ++r) {
                            const int64_t i = o.item(c, r);
                            assert(i >= 0);
                            if (i >= n) { // and none behind it
                                for (int k = 1; k < 6; ++k) assert(o.item(c, r + k) >= n);
                                break;
                            }
                            ++seen[i];
                            assert(o.cta(i) == c);
                        }
                    for (int x : seen) assert(x == 1);
                }
    return 0;
}
"""


def test_every_item_has_one_cta():
    nvcc = B._nvcc()
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.cpp"), os.path.join(d, "t")
        open(c, "w").write(ORDER)
        subprocess.run([nvcc, "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", B.SRC, c, "-o",
                        exe], check=True)
        subprocess.run([exe], check=True)


# ---- the binding

def test_make_score_refuses():
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    f, i = torch.zeros(8), torch.zeros(2, dtype=torch.int32)
    A.make_score(q, slopes=f, starts=i, keep_lens=i, keep=3)
    for kw in (dict(slopes=f.double()), dict(starts=i.long()), dict(slopes=torch.zeros(16)[::2]),
               dict(shared_len=16, shared_table=i.view(1, 2)), dict(keep_lens=f[:2])):
        with pytest.raises(TypeError):
            A.make_score(q, **kw)
    for kw in (dict(slopes=f[:7]), dict(starts=i[:1]), dict(shared_len=16)):
        with pytest.raises(ValueError):
            A.make_score(q, **kw)
    with pytest.raises(ValueError):
        A.make_score(q[0])
    with pytest.raises(TypeError):
        A.make_score(q.to(torch.float64))


def test_plan_scored_wants_a_length_each(lib):
    with pytest.raises(ValueError):
        A.decode_attn_plan_scored(args(), score(), [8])
    with pytest.raises(A.DecodeAttnError):
        A.decode_attn_plan_scored(args(), score(), [8, 0])


def test_the_call_wants_cuda_tensors(lib):
    a, s = args(), score()
    p = A.decode_attn_plan_scored(a, s, [8, 8], 152)
    x = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        A.decode_attn_splitk_scored(a, p, None, s, x, x, x, x, torch.zeros(8))
