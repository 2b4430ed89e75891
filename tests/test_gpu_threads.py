"""Calls from host threads other than the main one."""
import threading

import pytest
import torch

from split_kv_decode_gb300 import api as A
from split_kv_decode_gb300.cache8 import PagedCache8, Step8
from tests.scored_util import DT, Case, near

pytestmark = pytest.mark.gpu


def in_a_new_thread(call):
    """call() in a thread that has made no CUDA call; raises what it raises."""
    failed = []

    def body():
        try:
            call()
        except Exception as e:                  # (to the thread that waits)
            failed.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("shared", [0, 32])
def test_a_threads_first_call_is_scored(page, shared):
    if shared and not page:
        return
    c = Case([300, 41], 8, 2, 128, page=page, shared=shared)
    o = c.setup()
    ws, out = A.new_workspace(o.plan), torch.empty(o.q.shape, device="cuda")
    in_a_new_thread(lambda: A.decode_attn_splitk_scored(o.args, o.plan, o.dev, o.score, o.q, o.k,
                                                        o.v, out, ws))
    want, mag, top = c.want()
    near(out.double().cpu().numpy().reshape(want.shape), want, c.bound(want, mag, top))


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_threads_first_call_of_the_other_kernels(dt, hq):
    g = torch.Generator().manual_seed(hq)
    q = torch.randn(2, hq, 128, generator=g).cuda()
    k, v = (torch.randn(2, 500, 1, 128, generator=g).to(dt).cuda() for _ in range(2))
    da = A.DecodeAttention(q, k, v, [500, 77])
    out = da.new_out("cuda")
    in_a_new_thread(lambda: da(q, k, v, out))
    assert torch.equal(out, da(q, k, v))


def test_a_threads_first_call_is_over_an_8_bit_cache():
    g = torch.Generator().manual_seed(3)
    cache = PagedCache8(2, 12, 4, 2, 128, block_size=16, max_new=40)
    q, k, v = (torch.randn(n, h, 128, generator=g).cuda() for n, h in ((2, 8), (40, 2), (40, 2)))
    cache.grow(torch.tensor([30, 10], dtype=torch.int32, device="cuda"))
    cache.append(k, v)
    step, out = Step8(cache, q), torch.empty_like(q)
    in_a_new_thread(lambda: step(q, out))
    assert torch.equal(out, step(q))


def at_once(calls, times):
    """Each call in a thread of its own, `times` times; raises what one of them raised."""
    start, failed = threading.Barrier(len(calls)), []

    def loop(call, stream):
        start.wait()
        try:
            for i in range(times):
                call(stream)
                if i % 500 == 499:
                    stream.synchronize()
        except Exception as e:                  # (to the thread that waits)
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(c, torch.cuda.Stream())) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("d", [128, 256])
def test_scored_calls_of_other_rows_and_splits(d):
    # 20 and 100 rows of a sequence take rings of other lengths, 4 and 40 splits other combines
    cs = [Case([300], 20, 1, d, out="bf16", num_sms=4, force_splits=1),
          Case([300], 100, 1, d, out="bf16", num_sms=4, force_splits=1),
          Case([400], 4, 1, d, out="bf16", force_splits=4),
          Case([6000], 4, 1, d, out="bf16", force_splits=40)]
    calls, outs = [], []
    for c in cs:
        o = c.setup()
        ws, out = A.new_workspace(o.plan), torch.empty(o.q.shape, dtype=DT[c.out], device="cuda")
        calls.append(lambda s, o=o, ws=ws, out=out: A.decode_attn_splitk_scored(
            o.args, o.plan, o.dev, o.score, o.q, o.k, o.v, out, ws, s))
        outs.append(out)
    at_once(calls, 5000)
    for c, out in zip(cs, outs):
        want, mag, top = c.want()
        near(out.double().cpu().numpy().reshape(want.shape), want, c.bound(want, mag, top))


@pytest.mark.parametrize("out_dims", [(16, 256), (256, 8)])
def test_tensor_core_and_projected_calls_of_other_rows(out_dims):
    # 8 and 128 rows of a KV head, and projections of other widths behind other numbers of splits
    g = torch.Generator().manual_seed(7)
    calls, outs, want = [], [], []
    for (hq, splits), width in zip(((8, 40), (128, 4)), out_dims):
        q = torch.randn(1, hq, 128, generator=g).cuda()
        k, v = (torch.randn(1, 6000, 1, 128, generator=g).bfloat16().cuda() for _ in range(2))
        w = torch.randn(hq, width, 128, generator=g).cuda()
        da = A.DecodeAttention(q, k, v, [6000], force_splits=splits)
        proj, out = A.make_proj(w), torch.empty(1, hq, width, device="cuda")
        call = lambda s, da=da, proj=proj, q=q, k=k, v=v, w=w, out=out: A.decode_attn_splitk_proj(
            da.args, da.plan, proj, q, k, v, out, da.workspace, s)
        call(None)
        calls.append(call), outs.append(out), want.append(out.clone())
    for out in outs:
        out.zero_()
    at_once(calls, 5000)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
