"""Quantised append (decode_attn_append_8bit) against the page rule in 64 bits: codes
and scales are compared bit for bit (the rule rounds every value once, so there is one
right code)."""
import math

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import _native as N
from split_kv_decode_gb300 import api as A
from tests.kv8_util import MAX, TDT, append_reference, decode

pytestmark = pytest.mark.gpu

SRC = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def pools(nb, page, hkv, dk, dv, code, seed=0, strided=False):
    """Random codes (every finite one) and power-of-two scales."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for d in (dk, dv):
        u = torch.randint(0, 256, (nb, page, hkv, d), generator=g, dtype=torch.uint8)
        u[(u & 127) > (126 if code == "e4m3" else 123)] = 0x11
        if strided:                               # head-major pages, padded rows
            room = torch.zeros(nb, hkv, page + 1, d + 16, dtype=torch.uint8, device="cuda")
            view = room[:, :, :page, :d].permute(0, 2, 1, 3)
            view.copy_(u)
            u = view
        out.append(u.cuda() if not strided else u)
    scales = [torch.exp2(torch.randint(-9, 3, (nb, hkv), generator=g).float()).cuda()
              for _ in range(2)]
    if strided:
        scales = [torch.stack([s.t().contiguous(), torch.zeros_like(s.t())])[0].t() for s in scales]
    return [x.view(TDT[code]) for x in out], scales


def run(kn, vn, slots, kp, vp, ks, vs, stream=None):
    a = A.make_append(kn, vn, kp, vp, ks, vs)
    A.decode_attn_append_8bit(a, kn, vn, torch.as_tensor(slots, dtype=torch.int64, device="cuda"),
                              kp, vp, ks, vs, stream)
    torch.cuda.synchronize()


def check(kn, vn, slots, page, code, strided=False, nb=12, seed=0):
    (kp, vp), (ks, vs) = pools(nb, page, kn.shape[1], kn.shape[2], vn.shape[2], code, seed, strided)
    want = []
    for x, p, s in ((kn, kp, ks), (vn, vp, vs)):
        val, sc = decode(p, code), s.double().cpu().numpy().copy()
        append_reference(x.double().cpu().numpy(), slots, val, sc, page, code)
        want += [(val, sc)]
    run(kn, vn, slots, kp, vp, ks, vs)
    for (val, sc), p, s in zip(want, (kp, vp), (ks, vs)):
        np.testing.assert_array_equal(s.double().cpu().numpy(), sc)
        np.testing.assert_array_equal(decode(p, code), val)


def rows(T, hkv, d, src, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, d, generator=g) * torch.exp(spread * torch.randn(T, hkv, 1, generator=g))
    return x.to(SRC[src]).cuda()


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page,hkv,d", [(16, 8, 128), (64, 4, 256), (48, 1, 128), (1, 2, 16),
                                        (5, 3, 80), (256, 2, 256), (100, 1, 1024), (33, 2, 48)])
def test_runs_of_every_kind(page, hkv, d, src, code):
    # into a fresh page, into a page that goes on, over two and three pages, one row, the
    # last row of a page, skipped rows, and a block past the pool
    nb = 12
    runs = [(0, 0, page), (1, page // 3, 1), (2, page - 1, 1), (4, 0, max(1, page // 2)),
            (6, page // 2, page - page // 2)]
    slots = []
    for blk, p0, n in runs:
        slots += [blk * page + p0 + i for i in range(n)]
        slots += [-1]
    slots += [nb * page, nb * page + 1, (1 << 40), -5]
    slots += list(range(7 * page + page // 4, 9 * page + page // 2 + 1))
    kn, vn = rows(len(slots), hkv, d, src, 5), rows(len(slots), hkv, d, src, 6)
    check(kn, vn, slots, page, code, nb=nb, seed=page)


def test_many_single_rows_as_a_decode_step_writes_them():
    slots = [b * 16 + (7 * b) % 16 for b in range(200)]
    kn, vn = rows(200, 8, 128, "bf16", 1), rows(200, 8, 128, "bf16", 2)
    check(kn, vn, slots, 16, "e4m3", nb=200)


def test_a_long_prompt():
    slots = list(range(37, 37 + 5000))
    kn, vn = rows(5000, 2, 128, "f16", 1), rows(5000, 2, 128, "f16", 2)
    check(kn, vn, slots, 64, "e4m3", nb=80)


def test_keys_and_values_of_different_width_from_a_fused_projection():
    T, h, dk, dv = 45, 2, 192, 128
    fused = torch.randn(T, h, dk + dv, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    check(fused[:, :, :dk], fused[:, :, dk:], list(range(3, 48)), 16, "e4m3")


def test_strided_pools_and_scales():
    kn, vn = rows(40, 3, 128, "f32", 1), rows(40, 3, 128, "f32", 2)
    check(kn, vn, list(range(9, 49)), 16, "e4m3", strided=True)


def test_scales_at_the_borders():
    # the largest value exactly at MAX * 2^e keeps e; the next float32 above it takes e + 1
    for code in ("e4m3", "e5m2"):
        for e in (-20, 0, 7):
            for up in (False, True):
                x = torch.zeros(1, 1, 16)
                x[0, 0, 3] = MAX[code] * 2.0 ** e
                if up:
                    x = torch.nextafter(x, torch.tensor(float("inf"))) * (x > 0)
                (kp, vp), (ks, vs) = pools(2, 4, 1, 16, 16, code)
                run(x.cuda(), x.cuda(), [4], kp, vp, ks, vs)
                assert ks[1].item() == 2.0 ** (e + up)


def test_zeros_tiny_and_huge_values():
    for v, e in ((0.0, -100), (1e-38, -100), (1e-45, -100), (3.4e38, 120), (2.0 ** 127, 119)):
        x = torch.full((1, 1, 16), v)
        (kp, vp), (ks, vs) = pools(2, 4, 1, 16, 16, "e4m3")
        run(x.cuda(), -x.cuda(), [0], kp, vp, ks, vs)
        want = append_case(x, 4, e)
        assert ks[0].item() == 2.0 ** e and vs[0].item() == 2.0 ** e
        assert np.array_equal(decode(kp, "e4m3")[0, 0, 0], want)


def append_case(x, page, e):
    from tests.kv8_util import round_to
    return round_to(x.double().numpy()[0, 0] / 2.0 ** e, "e4m3")


def test_zeros_then_values_in_one_page():
    # a page that began with zeros takes its scale from the first values
    z, x = torch.zeros(3, 1, 32).cuda(), rows(2, 1, 32, "f32", 3)
    (kp, vp), (ks, vs) = pools(1, 8, 1, 32, 32, "e4m3")
    run(z, z, [0, 1, 2], kp, vp, ks, vs)
    assert ks.item() == 2.0 ** -100
    run(x, x, [3, 4], kp, vp, ks, vs)
    assert ks.item() > 2.0 ** -12 and np.all(decode(kp, "e4m3")[0, :3] == 0)


def test_non_finite_rows():
    x = torch.randn(4, 2, 32, generator=torch.Generator().manual_seed(2))
    x[0, 0, 5], x[1, 0, 6], x[2, 1, 7] = math.inf, -math.inf, math.nan
    x[3, 1] = math.nan                            # no finite value in the row
    for src in ("f32", "f16", "bf16"):
        for code in ("e4m3", "e5m2"):
            check(x.to(SRC[src]).cuda(), x.to(SRC[src]).cuda(), [3, 4, 5, 8], 8, code)
    only = torch.full((1, 1, 16), math.nan).cuda()
    (kp, vp), (ks, vs) = pools(1, 4, 1, 16, 16, "e4m3")
    run(only, only, [0], kp, vp, ks, vs)
    assert ks.item() == 2.0 ** -100 and np.all(np.isnan(decode(kp, "e4m3")[0, 0]))


def test_growing_step_by_step_equals_writing_at_once_where_no_code_is_subnormal():
    # power-of-two scales: rescaling loses nothing but subnormal codes
    g = torch.Generator().manual_seed(9)
    x = torch.randn(16, 2, 64, generator=g)
    x = torch.sign(x) * x.abs().clamp(0.5, 4) * torch.exp2(torch.arange(16) / 16.0)[:, None, None]
    x = x.cuda()
    a, b = pools(1, 16, 2, 64, 64, "e4m3"), pools(1, 16, 2, 64, 64, "e4m3")
    run(x, x, list(range(16)), *a[0], *a[1])
    for i in range(16):
        run(x[i:i + 1], x[i:i + 1], [i], *b[0], *b[1])
    assert torch.equal(a[1][0], b[1][0])
    assert torch.equal(a[0][0].view(torch.uint8), b[0][0].view(torch.uint8))


def test_a_page_with_another_quantisers_scale_goes_on_with_it():
    x = rows(2, 1, 32, "f32", 3) * 0.01
    (kp, vp), (ks, vs) = pools(1, 8, 1, 32, 32, "e4m3")
    ks.fill_(0.3), vs.fill_(0.7)
    old = decode(kp, "e4m3")[0, :5].copy()
    run(x, x, [5, 6], kp, vp, ks, vs)
    assert ks.item() == np.float32(0.3)
    np.testing.assert_array_equal(decode(kp, "e4m3")[0, :5], old)
    from tests.kv8_util import round_to
    # the f32 quotient, rounded to a code
    quotient = x.cpu() / torch.full((), 0.3, dtype=torch.float32)
    want = round_to(quotient.double().numpy(), "e4m3")
    np.testing.assert_array_equal(decode(kp, "e4m3")[0, 5:7], want)


def test_no_rows_and_only_skipped_rows_change_nothing():
    (kp, vp), (ks, vs) = pools(2, 8, 1, 32, 32, "e4m3")
    before = [t.view(torch.uint8).clone() for t in (kp, vp)] + [ks.clone(), vs.clone()]
    run(rows(0, 1, 32, "f32", 1), rows(0, 1, 32, "f32", 1), [], kp, vp, ks, vs)
    run(rows(3, 1, 32, "f32", 1), rows(3, 1, 32, "f32", 1), [-1, -1, 16], kp, vp, ks, vs)
    after = [t.view(torch.uint8) for t in (kp, vp)] + [ks, vs]
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_on_another_stream_and_captured():
    x, y = rows(6, 2, 128, "bf16", 1), rows(6, 2, 128, "bf16", 2)
    want = pools(3, 16, 2, 128, 128, "e4m3")
    run(x, y, list(range(13, 19)), *want[0], *want[1])
    st = torch.cuda.Stream()
    got = pools(3, 16, 2, 128, 128, "e4m3")
    torch.cuda.synchronize()
    run(x, y, list(range(13, 19)), *got[0], *got[1], stream=st)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want[0], got[0]))
    (kp, vp), (ks, vs) = pools(3, 16, 2, 128, 128, "e4m3")
    slots = torch.full((6,), -1, dtype=torch.int64, device="cuda")
    a = A.make_append(x, y, kp, vp, ks, vs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.decode_attn_append_8bit(a, x, y, slots, kp, vp, ks, vs)
    slots.copy_(torch.arange(13, 19))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip(want[0], (kp, vp))) and torch.equal(want[1][0], ks)


def test_pools_past_four_gigabytes():
    # offsets of the last blocks pass 2^32 bytes
    nb, page, h, d = 2100, 64, 128, 256
    kp = torch.zeros(nb, page, h, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks = torch.ones(nb, h, device="cuda")
    x = rows(2, h, d, "bf16", 3)
    run(x, x, [(nb - 1) * page + 62, (nb - 1) * page + 63], kp, kp.clone(), ks, ks.clone())
    val, sc = np.zeros((1, page, h, d)), np.ones((1, h))
    append_reference(x.double().cpu().numpy(), [62, 63], val, sc, page, "e4m3")
    np.testing.assert_array_equal(decode(kp[-1:], "e4m3"), val)
    np.testing.assert_array_equal(ks[-1:].double().cpu().numpy(), sc)
    assert int(kp.view(torch.uint8)[:-1].any()) == 0


def test_refusals():
    (kp, vp), (ks, vs) = pools(2, 8, 2, 32, 32, "e4m3")
    x = rows(3, 2, 32, "f32", 1)
    a = A.make_append(x, x, kp, vp, ks, vs)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        A.decode_attn_append_8bit(a, x, x, slots.int(), kp, vp, ks, vs)
    with pytest.raises(TypeError):
        A.decode_attn_append_8bit(a, x, x, slots[:2], kp, vp, ks, vs)
    with pytest.raises(ValueError):
        A.decode_attn_append_8bit(a, x.cpu(), x, slots, kp, vp, ks, vs)
    with pytest.raises(ValueError):
        A.make_append(x, x, kp, vp, ks[:1], vs)
    with pytest.raises(ValueError):
        A.make_append(x, x.half(), kp, vp, ks, vs)
    with pytest.raises(ValueError):
        A.make_append(x[:, :1], x[:, :1], kp, vp, ks, vs)
    odd = torch.zeros(3, 2, 33, device="cuda")[:, :, :32]   # rows not 16-byte aligned
    with pytest.raises(A.DecodeAttnError) as e:
        A.decode_attn_append_8bit(A.make_append(odd, odd, kp, vp, ks, vs), odd, odd, slots, kp,
                                  vp, ks, vs)
    assert e.value.status == N.DA_EINVAL and "16 bytes" in e.value.message
