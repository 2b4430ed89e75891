"""The operators as a serving loop runs them (PagedCache16, ScoredStep): requests come, grow, are
released and replaced. Every step's rows in the cache are compared with norm and rotation in 64
bits, its output with attention in 64 bits over what the cache holds, eagerly and replayed from
one captured graph."""
import math
import random

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300.cache8 import PagedCache8, Step8
from split_kv_decode_gb300.cache16 import PagedCache16, ScoredStep
from tests import prep_util as P
from tests.kv8_util import Blocks
from tests.scored_util import DT, Case, near

pytestmark = pytest.mark.gpu


def frequencies(n):
    return [10000.0 ** (-i / n) for i in range(n)]


def view(cache, step, q, **kw):
    """A Case of what the cache and the step hold now."""
    c = Case.__new__(Case)
    names = {v: k for k, v in DT.items()}
    c.lens = cache.seq_lens.tolist()[:q.shape[0]]
    c.page, c.hkv, c.d = cache.block_size, cache.k.shape[2], cache.k.shape[3]
    c.q = (q if q.dim() == 4 else q[:, None]).cpu()
    c.q_len, c.hq = c.q.shape[1:3]
    c.cache, c.qt, c.out = names[cache.k.dtype], names[q.dtype], names[step.out_dtype]
    c.k, c.v, c.table = cache.k.cpu(), cache.v.cpu(), cache.block_table.cpu()
    c.scale = c.d ** -0.5
    c.cap, c.window, c.keep = kw.get("softcap", 0.0), kw.get("window", 0), kw.get("keep", 0)
    c.keep_lens = c.starts = None
    c.slopes = kw["slopes"].cpu() if kw.get("slopes") is not None else None
    c.shared = kw.get("shared_len", 0)
    c.shared_table = cache.shared_table[:c.shared // c.page].cpu()
    return c


def check_rows(cache, rows, slots, weights, eps, freqs, positions, shared=False):
    """The rows q, k, v in the cache's slots and q's copy."""
    q, k, v, q_out = (x.double().cpu().numpy() for x in rows)
    names = {v: k for k, v in DT.items()}
    ok = [i for i, s in enumerate(slots) if s >= 0]
    for x, w, got, dt in ((q, weights[0], q_out, rows[3].dtype), (k, weights[1], None, cache.k.dtype)):
        y = P.normed(x, w.double().cpu().numpy(), eps)
        z, mag = P.rotated(y, [positions], freqs, [0] * len(freqs), False)
        tol = P.bound(z, mag, names[dt])
        if got is None:
            got = cache.k.reshape(-1, *cache.k.shape[2:])[[slots[i] for i in ok]].double().cpu().numpy()
            z, tol = z[ok], tol[ok]
        near(got, z, tol)
    got = cache.v.reshape(-1, *cache.v.shape[2:])[[slots[i] for i in ok]]
    assert torch.equal(got, rows[2][ok].to(cache.v.dtype))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,page,cache,kw", [
    (1, 8, 2, 128, 16, "bf16", dict(window=70, keep=5)),
    (1, 8, 4, 256, 64, "f16", dict(softcap=20.0)),
    (3, 12, 2, 128, 48, "bf16", dict(slopes=True)),
    (1, 8, 2, 128, 32, "bf16", dict(shared_len=256)),
    (2, 8, 2, 256, 64, "f16", dict(shared_len=320, softcap=9.0)),
])
def test_a_serving_loop(T, hq, hkv, d, page, cache, kw, graph):
    B, width, blocks, rows = 5, 20, 70, 5 * 40
    rng, gen = random.Random(T + d), torch.Generator().manual_seed(d + T)
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.exp2(-torch.arange(1, hq + 1).float() / 2).cuda()
    front = kw.get("shared_len", 0)
    taken = front // page
    freqs = frequencies(d // 2)
    weights = [(torch.rand(d, generator=gen) + 0.5).cuda() for _ in range(2)]
    pages = PagedCache16(B, blocks + taken, width, hkv, d, block_size=page, max_new=rows,
                         dtype=DT[cache], rope=A.make_rope(freqs), eps=1e-5, q_weight=weights[0],
                         k_weight=weights[1], shared_blocks=taken)
    make = lambda n, h: torch.randn(n, h, d, generator=gen).to(DT[cache]).cuda()
    if front:                                        # the prefix, in two parts
        for first, n in ((0, front - 7), (front - 7, 7)):
            q, k, v = make(n, hq), make(n, hkv), make(n, hkv)
            pos = torch.arange(first, first + n, device="cuda")
            q_out = pages.append_shared(q, k, v, pos, first)
            check_rows(pages, (q, k, v, q_out), list(range(first, first + n)), weights, 1e-5, freqs,
                       pos.tolist())
    b = Blocks(B, blocks, width, page)
    shape = (B, hq, d) if T == 1 else (B, T, hq, d)
    q, k, v = make(rows, hq), make(rows, hkv), make(rows, hkv)
    positions = torch.zeros(rows, dtype=torch.int64, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    q_out, now = torch.empty_like(q), torch.zeros(shape, dtype=DT[cache], device="cuda")
    step = ScoredStep(pages, now, **kw)
    out = torch.empty(shape, dtype=DT[cache], device="cuda")

    def once():
        pages.grow(new)
        pages.append(q, k, v, positions, q_out)
        step(now, out)

    if graph:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
            once()
    for i in range(10):
        want = [rng.choice([-1, 0, T, T, T, rng.randint(T, 40)]) for _ in range(B)]
        if i == 0:
            want = [40, T, 17, 0, T]
        want = [n if n < 0 or L + n <= width * page else -1 for n, L in zip(want, b.lens)]
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen))
        before = list(b.lens)
        status, slots, cu = b.grow(want, rows)
        assert status == 0
        pos = [0] * rows
        for s, n in enumerate(want):
            for e in range(max(n, 0)):
                pos[cu[s] + e] = front + before[s] + e
        positions.copy_(torch.tensor(pos))
        now.copy_(torch.randn(shape, generator=gen))
        new.copy_(torch.tensor(want))
        out.fill_(math.nan)
        g.replay() if graph else once()
        pages.check()
        A.decode_attn_device_status(step.workspace)
        slots = [s if s < 0 else s + taken * page for s in slots]
        assert pages.seq_lens.tolist() == b.lens and pages.slot_map.tolist() == slots
        check_rows(pages, (q, k, v, q_out), slots, weights, 1e-5, freqs, pos)
        c = view(pages, step, now, **kw)
        want_out, mag, top = c.want()
        got = out.double().cpu().numpy().reshape(want_out.shape)
        near(got, want_out, c.bound(want_out, mag, top))


def test_the_8_bit_cache_takes_rotated_rows():
    # norm and rotation into plain rows (a row's slot is its number), quantised into the pages from
    # there: as if torch had made the rows
    gen = torch.Generator().manual_seed(3)
    B, hq, hkv, d = 3, 8, 2, 128
    cache = PagedCache8(B, 12, 4, hkv, d, block_size=16, max_new=B)
    rope = A.make_rope(frequencies(d // 2))
    q, k, v = (torch.randn(B, h, d, generator=gen).bfloat16().cuda() for h in (hq, hkv, hkv))
    rows = torch.zeros(2, 1, B, hkv, d, device="cuda")
    q_out = torch.empty(B, hq, d, device="cuda")
    positions = torch.tensor([0, 7, 100000], device="cuda")
    prep = A.make_prep(q, k, v, q_out, rows[0], rows[1], rope)
    A.decode_attn_rope_append(prep, q, k, v, positions, None, q_out, rows[0], rows[1])
    cache.grow(torch.ones(B, dtype=torch.int32, device="cuda"))
    cache.append(rows[0, 0], rows[1, 0])
    other = PagedCache8(B, 12, 4, hkv, d, block_size=16, max_new=B)
    z, mag = P.rotated(k.double().cpu().numpy(), [positions.tolist()], frequencies(d // 2),
                       [0] * (d // 2), False)
    near(rows[0, 0].double().cpu().numpy(), z, P.bound(z, mag, "f32"))
    other.grow(torch.ones(B, dtype=torch.int32, device="cuda"))
    other.append(rows[0, 0].clone(), v.float())
    assert torch.equal(Step8(cache, q_out)(q_out), Step8(other, q_out)(q_out))


def test_shared_rows_on_a_stream_beside_a_busy_one():
    # the call's stream is ordered behind its inputs alone, and the current one has work for longer
    gen = torch.Generator().manual_seed(4)
    c = PagedCache16(2, 10, 4, 2, 128, block_size=16, shared_blocks=4)
    side = torch.cuda.Stream()
    parts, at = [], 0
    for n in (7, 20, 1, 36):
        q, k, v = (torch.randn(n, h, 128, generator=gen).bfloat16().cuda() for h in (4, 2, 2))
        parts.append((at, q, k, v, torch.arange(at, at + n, device="cuda"), torch.empty_like(q)))
        at += n
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    for first, q, k, v, pos, q_out in parts:
        c.append_shared(q, k, v, pos, first, q_out, stream=side)
        torch.full((n,), 9, device="cuda")           # (takes what a call gave back)
    side.synchronize()
    got = [x.clone() for x in (c.k, c.v)]
    torch.cuda.synchronize()
    for x, i in zip(got, (2, 3)):
        assert torch.equal(x.view(-1, 2, 128)[:64], torch.cat([p[i] for p in parts]))
        assert (x[4:] == 0).all()
    assert all(torch.equal(p[5], p[1]) for p in parts)


@pytest.mark.parametrize("handle", [False, True])
def test_new_outputs_on_a_stream_beside_a_busy_one(handle):
    # memory that the current stream has given back but still writes is not what a call on another
    # stream gets for its output
    gen = torch.Generator().manual_seed(6)
    c = PagedCache16(2, 10, 4, 2, 128, block_size=16, max_new=32)
    q, k, v = (torch.randn(32, h, 128, generator=gen).bfloat16().cuda() for h in (512, 2, 2))
    c.grow(torch.tensor([20, 12], dtype=torch.int32, device="cuda"))
    pos = torch.arange(32, device="cuda")
    c.append(q, k, v, pos)
    now = q[:2].contiguous()
    step = ScoredStep(c, now[:, :8].contiguous(), out_dtype=torch.float32)
    one = now[:, :8].contiguous()
    want = step(one)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.empty_like(q), torch.empty_like(want)]
    torch.cuda._sleep(50_000_000)
    for x in held:
        x.fill_(math.nan)
    x = None
    del held
    on = side.cuda_stream if handle else side
    rotated, got = c.append(q, k, v, pos, stream=on), step(one, stream=on)
    torch.cuda.synchronize()
    assert torch.equal(rotated, q) and torch.equal(got, want)


def test_layers_share_the_tables():
    kw = dict(block_size=16, max_new=8, shared_blocks=2)
    a = PagedCache16(2, 10, 4, 2, 128, **kw)
    b = PagedCache16(2, 10, 4, 2, 128, tables_of=a, **kw)
    a.grow(torch.tensor([3, 5], dtype=torch.int32, device="cuda"))
    x, q = (torch.randn(8, h, 128, device="cuda").bfloat16() for h in (2, 4))
    pos = torch.arange(8, device="cuda")
    for c in (a, b):
        out = c.append(q, x, 2 * x, pos)
        assert torch.equal(out, q)               # neither a norm nor a rotation
        c.append_shared(q, x, x, pos)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and a.slot_map.min() == 2 * 16
    one = q[:2].contiguous()
    assert torch.equal(ScoredStep(a, one, shared_len=16)(one),
                       ScoredStep(b, one, shared_len=16, max_lens=[64, 64])(one))
    for other in (dict(kw, block_size=32), dict(kw, shared_blocks=1)):
        with pytest.raises(ValueError):
            PagedCache16(2, 10, 4, 2, 128, tables_of=a, **other)


def test_steps_without_rows():
    c = PagedCache16(2, 10, 4, 2, 128, block_size=16, max_new=4)
    none = torch.zeros(0, 2, 128, device="cuda").bfloat16()
    c.grow(torch.zeros(2, dtype=torch.int32, device="cuda"))
    q = c.append(torch.zeros(0, 4, 128, device="cuda").bfloat16(), none, none,
                 torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert q.shape == (0, 4, 128) and (c.k == 0).all()
    one = torch.randn(2, 4, 128, device="cuda").bfloat16()
    assert (ScoredStep(c, one)(one) == 0).all()  # nothing to see


def test_refusals():
    with pytest.raises(TypeError):
        PagedCache16(2, 10, 4, 2, 128, dtype=torch.float32)
    with pytest.raises(ValueError):
        PagedCache16(2, 10, 4, 2, 128, shared_blocks=11)
    c = PagedCache16(2, 10, 4, 2, 128, block_size=16, max_new=4, shared_blocks=2)
    q, x = (torch.randn(5, h, 128, device="cuda").bfloat16() for h in (4, 2))
    pos = torch.arange(5, device="cuda")
    with pytest.raises(ValueError):
        c.append(q, x, x, pos)                   # more rows than max_new
    for first in (-1, 28):
        with pytest.raises(ValueError):
            c.append_shared(q, x, x, pos, first)
    with pytest.raises(TypeError):
        c.append_shared(q, x, x, pos[:4])
    one = q[:2].contiguous()
    with pytest.raises(ValueError):
        ScoredStep(c, q)                         # more sequences than the cache
    with pytest.raises(ValueError):
        ScoredStep(c, one, shared_len=48)
    step = ScoredStep(c, one)
    with pytest.raises(ValueError):
        step(one.float())
    with pytest.raises(ValueError):
        step(one[:1])
    with pytest.raises(ValueError):
        step(one, torch.empty(2, 4, 64, device="cuda").bfloat16())
    with pytest.raises(TypeError):
        step(one, torch.empty(2, 4, 128, device="cuda"))
