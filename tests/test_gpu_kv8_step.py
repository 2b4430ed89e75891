"""The three operators as a serving loop runs them (PagedCache8, Step8): requests come,
grow, are released and replaced; every step's output is compared with attention in
64 bits over a quantised cache kept by the reference rules, eagerly and replayed from
one captured graph."""
import math
import random

import numpy as np
import pytest
import torch

from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300.cache8 import PagedCache8, Step8
from tests.kv8_util import TDT, Blocks, append_reference, attention_reference

pytestmark = pytest.mark.gpu


class Reference:
    def __init__(self, batch, blocks, width, page, hkv, d, code):
        self.b = Blocks(batch, blocks, width, page)
        self.page, self.code = page, code
        self.val = [np.zeros((blocks, page, hkv, d)) for _ in range(2)]
        self.sc = [np.ones((blocks, hkv)) for _ in range(2)]

    def step(self, new, k, v, rows):
        status, slots, _ = self.b.grow(new, rows)
        assert status == 0
        for x, val, sc in zip((k, v), self.val, self.sc):
            append_reference(x, slots, val, sc, self.page, self.code)

    def kv(self):
        out = []
        for val, sc in zip(self.val, self.sc):
            y = val * sc[:, None, :, None]
            out.append([y[r].reshape(-1, *y.shape[2:])[:n] if r else y[:0].reshape(0, *y.shape[2:])
                        for r, n in zip(self.b.rows, self.b.lens)])
        return out


def tolerance(v, mag, lens):
    # derived in test_gpu_kv8_attend
    vmax = np.array([np.abs(x).max() if n else 0.0 for x, n in zip(v, lens)])
    return vmax[:, None, None, None] * (2.0 ** -17 * mag[..., None] + 2.0 ** -15) + 1e-300


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,page,code", [(1, 8, 2, 128, 16, "e4m3"),
                                                  (3, 8, 4, 256, 64, "e4m3"),
                                                  (1, 12, 1, 128, 48, "e5m2")])
def test_a_serving_loop(T, hq, hkv, d, page, code, graph):
    B, width, blocks, rows = 5, 20, 60, 5 * 40
    rng, gen = random.Random(T + d), torch.Generator().manual_seed(d + T)
    ref = Reference(B, blocks, width, page, hkv, d, code)
    cache = PagedCache8(B, blocks, width, hkv, d, block_size=page, max_new=rows, dtype=TDT[code])
    q = torch.zeros((B, hq, d) if T == 1 else (B, T, hq, d), device="cuda")
    k, v = [torch.zeros(rows, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    step = Step8(cache, q)
    out = torch.empty_like(q)

    def once():
        cache.grow(new)
        cache.append(k, v)
        step(q, out)

    if graph:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
            once()
    for i in range(14):
        want = [rng.choice([-1, 0, T, T, T, rng.randint(T, 40)]) for _ in range(B)]
        if i == 0:
            want = [40, T, 17, 0, T]
        want = [n if n < 0 or L + n <= width * page else -1 for n, L in zip(want, ref.b.lens)]
        kn, vn = [torch.randn(rows, hkv, d, generator=gen).mul_(2.0 ** rng.randint(-4, 3)).bfloat16()
                  for _ in range(2)]
        qn = torch.randn(q.shape, generator=gen)
        k.copy_(kn), v.copy_(vn), q.copy_(qn)
        new.copy_(torch.tensor(want))
        g.replay() if graph else once()
        cache.check()
        A.decode_attn_device_status(step.workspace)
        ref.step(want, kn.double().numpy(), vn.double().numpy(), rows)
        keys, values = ref.kv()
        lens = ref.b.lens
        assert cache.seq_lens.tolist() == lens
        r, mag = attention_reference(qn.double().numpy().reshape(B, T, hq, d), keys, values, lens,
                                     d ** -0.5)
        got = out.double().cpu().numpy().reshape(r.shape)
        assert np.all(np.abs(got - r) <= tolerance(values, mag, lens)), i


def test_layers_share_the_tables():
    a = PagedCache8(2, 10, 4, 2, 128, block_size=16, max_new=8)
    b = PagedCache8(2, 10, 4, 2, 128, block_size=16, tables_of=a)
    a.grow(torch.tensor([3, 5], dtype=torch.int32, device="cuda"))
    x = torch.randn(8, 2, 128, device="cuda")
    for c in (a, b):
        c.append(x, 2 * x)
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))
    q = torch.randn(2, 4, 128, device="cuda")
    assert torch.equal(Step8(a, q)(q), Step8(b, q, max_lens=[64, 64])(q))
    with pytest.raises(ValueError):
        PagedCache8(2, 10, 4, 2, 128, block_size=32, tables_of=a)


def test_rows_of_changing_shapes_strides_and_types():
    cache = PagedCache8(3, 24, 8, 2, 128, block_size=16, max_new=12)
    fused = torch.randn(9, 5, 2, 128, device="cuda")
    rows = [(fused[:, 0], fused[:, 1]), (fused[:, 1], fused[:, 3]),
            (fused[:, 2].contiguous(), fused[:, 4].contiguous()),
            (fused[:3, 0].half(), fused[:3, 1].half()), (fused[:3, 2], fused[:3, 0]),
            (fused[:3, 0].bfloat16(), fused[:3, 1].bfloat16()),
            (torch.cat([fused, fused[:3]])[:, 0], torch.cat([fused, fused[:3]])[:, 1])]
    want = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    for k, v in rows:
        n = k.shape[0] // 3
        slots = cache.grow(torch.full((3,), n, dtype=torch.int32, device="cuda"))
        cache.append(k, v)
        A.decode_attn_append_8bit(A.make_append(k, v, *want), k, v, slots[:3 * n].clone(), *want)
        for got, ref in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    with pytest.raises(ValueError):
        cache.append(rows[0][0], rows[0][1][:3])
    with pytest.raises(ValueError):
        cache.append(fused[:, 0, :, ::2], fused[:, 1, :, ::2])


def test_a_step_that_finds_no_blocks_leaves_the_cache_as_it_was():
    c = PagedCache8(2, 3, 4, 1, 128, block_size=16, max_new=64)
    x = torch.randn(64, 1, 128, device="cuda")
    q = torch.randn(2, 2, 128, device="cuda")
    step = Step8(c, q)
    c.grow(torch.tensor([20, 10], dtype=torch.int32, device="cuda"))
    c.append(x, x)
    before, codes = step(q).clone(), c.k.view(torch.uint8).clone()
    c.grow(torch.tensor([1, 30], dtype=torch.int32, device="cuda"))
    c.append(-x, -x)                              # every slot is -1
    assert torch.equal(step(q), before) and torch.equal(c.k.view(torch.uint8), codes)
    with pytest.raises(A.DecodeAttnError):
        c.check()
    c.check()


def test_refusals():
    with pytest.raises(TypeError):
        PagedCache8(2, 3, 4, 1, 128, dtype=torch.bfloat16)
    c = PagedCache8(2, 3, 4, 1, 128, block_size=16, max_new=4)
    x = torch.randn(5, 1, 128, device="cuda")
    with pytest.raises(ValueError):
        c.append(x, x)
    q = torch.randn(2, 2, 128, device="cuda")
    with pytest.raises(ValueError):
        Step8(c, torch.randn(3, 2, 128, device="cuda"))
    with pytest.raises(ValueError):
        Step8(c, q)(q[:1])
