"""What the serving operators over an 8-bit paged KV cache are measured on.

Three operators that a decode loop calls one after the other:

  tables  block tables and slot maps of a batch, grown on the GPU from the
          request lengths (decode_attn_grow_tables)
  append  new K/V rows quantised into the pages their slots name, with one
          power-of-two scale per (page, KV head) (decode_attn_append_8bit)
  attend  split-KV decode attention over those pages
          (decode_attn_splitk_8bit)

`run` with `own` false computes them in elementary torch operations; with `own`
true it makes the library's calls.
"""
import math
import random

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
CODE_MAX = {"e4m3": 448.0, "e5m2": 57344.0}     # 1.75 * 2^TOP_EXP
TOP_EXP = {"e4m3": 8, "e5m2": 15}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LEAST_EXP = {"e4m3": -6, "e5m2": -14}           # of a normal code
MIN_EXP = -100                                  # a page of zeros has the scale 2^-100
NAN_CODE = 0x7F
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases

def _attend(name, lens, hq, hkv, dim, page, q_len=1, code="e4m3", out="f32"):
    return {"name": name, "op": "attend", "lens": lens, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "q_len": q_len, "code": code, "out": out}


def _append(name, lens, new, hkv, dim, page, src="bf16", code="e4m3", pad=0):
    return {"name": name, "op": "append", "lens": lens, "new": new, "hkv": hkv, "dim": dim,
            "page": page, "src": src, "code": code, "pad": pad}


def _tables(name, batch, page, lo, hi, new_lo, new_hi, release, seed):
    return {"name": name, "op": "tables", "batch": batch, "page": page, "lo": lo, "hi": hi,
            "new_lo": new_lo, "new_hi": new_hi, "release": release, "seed": seed}


def _text(xs):
    return ",".join(str(int(x)) for x in xs)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _ragged(batch, lo, hi, seed):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(batch)]


def listed():
    return [
        # a chat's first answers: one request, a few hundred tokens; latency counts
        _attend("attend_short", "713", 8, 2, 128, 16),
        # the benchmark's smallest geometry (8/2 heads of 256, 4096 positions)
        _attend("attend_8x2_4k", "4096", 8, 2, 256, 64),
        # its long single context (16/4 heads of 256, 151552 positions)
        _attend("attend_16x4_152k", "151552", 16, 4, 256, 64),
        # its ragged batch of 32 (32/8 heads of 128), pages of 16, bf16 output: the largest
        _attend("attend_ragged32", _text(_ragged(32, 1024, 131072, 1238)), 32, 8, 128, 16,
                out="bf16"),
        # its 24/4-head batch, with four new tokens a sequence (a draft being verified): 24 rows
        _attend("attend_24x4_draft4", "8192,20480,61440,131072", 24, 4, 256, 128, q_len=4,
                out="bf16"),
        # every query head with its own KV head, e5m2 codes, odd pages, f16 output
        _attend("attend_mha_e5m2", "2999,17,1500,3500,64,2048,777,1", 16, 16, 128, 48,
                code="e5m2", out="f16"),
        # one decode step of a batch of 32: a row each
        _append("append_step32", _text(_ragged(32, 1024, 131072, 1238)), _text([1] * 32), 8, 128,
                16),
        # a small batch of drafts of ragged lengths in f32, rows padded to a fixed count
        _append("append_draft7", "100,63,64,65,4095,1,0", "4,2,5,1,8,3,7", 4, 256, 64, src="f32",
                pad=2),
        # one long prompt in one call
        _append("append_prompt32k", "0", "32768", 4, 256, 64, src="f16"),
        # a batch of prompts of ragged lengths, some continuing a page
        _append("append_prompts8", "0,5,0,1000,31,0,77,4096",
                "16001,20480,9999,16,30000,131,24576,28673", 8, 128, 16),
        # the tables of one decode step of 32 requests, two of them done
        _tables("tables_step32", 32, 16, 1024, 131072, 1, 1, 2, 7),
        # the tables of a full batch of prompts arriving at once
        _tables("tables_prompts256", 256, 16, 0, 64, 1, 16384, 0, 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "tables"])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([128, 256])
    code = rng.choice(["e4m3", "e4m3", "e4m3", "e5m2"])
    if op == "attend":
        batch = _log(rng, 1, 32)
        q_len = rng.choice([1, 1, 1, 2, 3, 5])
        group = rng.choice([1, 2, 4, 6, 8, 12])
        hi = _log(rng, 64, max(65, min(131072, (1 << 28) // (batch * hkv * dim))))
        lens = [max(q_len, _log(rng, max(1, hi // 16), hi)) for _ in range(batch)]
        return {"op": "attend", "lens": _text(lens), "hq": hkv * group, "hkv": hkv, "dim": dim,
                "page": page, "q_len": q_len, "code": code,
                "out": rng.choice(["f32", "f16", "bf16"])}
    if op == "append":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, min(16384, (1 << 26) // (batch * hkv * dim))))
        return {"op": "append", "lens": _text([rng.choice([0, _log(rng, 1, 2000)])
                                               for _ in range(batch)]),
                "new": _text([_log(rng, 1, hi) for _ in range(batch)]), "hkv": hkv, "dim": dim,
                "page": page, "src": rng.choice(["f32", "f16", "bf16"]), "code": code,
                "pad": rng.choice([0, 0, 3])}
    batch = _log(rng, 1, 256)
    return {"op": "tables", "batch": batch, "page": page, "lo": 0, "hi": _log(rng, 1, 16384),
            "new_lo": rng.choice([0, 1]), "new_hi": _log(rng, 1, 8192),
            "release": rng.randint(0, batch // 4), "seed": rng.randint(1, 1 << 20)}


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pow2(e):
    """2^e in 32 bits, from its bits (-126 <= e <= 127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _page_exp(amax, code):
    """The least e with amax <= CODE_MAX * 2^e, at least MIN_EXP (amax >= 0, finite)."""
    m, x = torch.frexp(amax)                     # amax = m * 2^x, m in [0.5, 1)
    e = torch.where(m <= 0.875, x - 1 - TOP_EXP[code], x - TOP_EXP[code])
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _fill_pool(g, blocks, page, hkv, dim, code):
    """A pool of random pages, quantised page by page: N(0, s) values, s differing from page to
    page and head to head as a layer's keys and values do. Returns codes (uint8) and scales."""
    pool = torch.empty(blocks, page, hkv, dim, dtype=torch.uint8, device="cuda")
    scale = torch.empty(blocks, hkv, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (page * hkv * dim))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn(n, page, hkv, dim, generator=g, device="cuda")
        x *= torch.exp(0.3 * torch.randn(n, 1, hkv, 1, generator=g, device="cuda"))
        s = _pow2(_page_exp(x.abs().amax((1, 3)), code))
        scale[i:i + n] = s
        pool[i:i + n] = (x / s[:, None, :, None]).to(F8[code]).view(torch.uint8)
    return pool, scale


def _tables_for(g, lens, page, blocks, width):
    """A block table [B, width] whose used entries are a random choice of the pool's blocks."""
    order = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at:at + k]
        at += k
    return table, order[at:]


def _ragged_new(case):
    r = random.Random(case["seed"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    for b in r.sample(range(case["batch"]), case["release"]):
        new[b] = -1
    return lens, new


def prepare(case, seed):
    g = _gen(seed)
    op, page = case["op"], case["page"]
    s = {"case": case}
    if op == "attend":
        lens = _ints(case["lens"])
        hkv, dim, code = case["hkv"], case["dim"], case["code"]
        blocks = sum(-(-n // page) for n in lens) + 3
        for name in ("k", "v"):
            pool, scale = _fill_pool(g, blocks, page, hkv, dim, code)
            s[name], s[name + "_scale"] = pool, scale
        width = max(-(-n // page) for n in lens) + 1
        s["table"], _ = _tables_for(g, lens, page, blocks, width)
        for b, n in enumerate(lens):              # slots past a length: never written
            if n % page:
                blk = s["table"][b, n // page].long()
                s["k"][blk, n % page:] = NAN_CODE
                s["v"][blk, n % page:] = NAN_CODE
        s["k"], s["v"] = s["k"].view(F8[code]), s["v"].view(F8[code])
        shape = (len(lens), case["hq"], dim)
        if case["q_len"] > 1:
            shape = (len(lens), case["q_len"], case["hq"], dim)
        s["q"] = torch.randn(shape, generator=g, device="cuda")
        s["host_lens"] = lens
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    elif op == "append":
        lens, new = _ints(case["lens"]), _ints(case["new"])
        hkv, dim, code = case["hkv"], case["dim"], case["code"]
        # the pages that the old rows' last page and the new rows need, and a few more
        first = [n // page for n in lens]
        pages = [-(-(n + m) // page) - f for n, m, f in zip(lens, new, first)]
        blocks = sum(pages) + 4
        order = torch.randperm(blocks, generator=g, device="cuda")
        for name in ("k", "v"):
            pool, scale = _fill_pool(g, blocks, page, hkv, dim, code)
            s[name], s[name + "_scale"] = pool.view(F8[code]), scale
        slots, at = [], 0
        for n, m, f, k in zip(lens, new, first, pages):
            pos = torch.arange(n, n + m, device="cuda")
            slots.append(order[at + pos // page - f] * page + pos % page)
            at += k
        slots.append(torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda"))
        s["slots"] = torch.cat(slots)
        rows = s["slots"].numel()
        # K and V of a fused projection: rows of [K heads | V heads]
        fused = torch.randn(rows, 2 * hkv, dim, generator=g, device="cuda")
        fused *= torch.exp(0.3 * torch.randn(rows, 2 * hkv, 1, generator=g, device="cuda"))
        fused = fused.to(TYPES[case["src"]])
        s["new_k"], s["new_v"] = fused[:, :hkv], fused[:, hkv:]
    else:
        lens, new = _ragged_new(case)
        batch = case["batch"]
        ends = [n + max(m, 0) for n, m in zip(lens, new)]
        width = max(1, max(-(-e // page) for e in ends)) + 2
        blocks = sum(-(-e // page) for e in ends) + 5
        s["table"], free = _tables_for(g, lens, page, blocks, width)
        s["free"] = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        s["free"][:free.numel()] = free
        s["state"] = torch.tensor([free.numel(), 0, 0, 0], dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        # a call's outputs; lengths and state come out beside the old ones, so that a pass
        # can be made again on the same ones
        s["lens_out"], s["state_out"] = torch.empty_like(s["lens"]), torch.zeros_like(s["state"])
        s["cu"] = torch.empty(batch + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(sum(max(m, 0) for m in new) + 3, dtype=torch.int64, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_attend(s):
    c = s["case"]
    page, hkv, dim, t = c["page"], c["hkv"], c["dim"], c["q_len"]
    batch, top = len(s["host_lens"]), max(s["host_lens"])
    q = s["q"].reshape(batch, t, hkv, c["hq"] // hkv, dim)
    pos = torch.arange(top, device="cuda")
    there = pos < s["lens"][:, None]                                       # [B, L]
    blk = torch.where(there, s["table"][:, :-(-top // page)].long()
                      .repeat_interleave(page, 1)[:, :top], 0)
    off = (pos % page).expand(batch, top)

    def values(pool, scale):
        x = pool.view(torch.uint8)[blk, off].view(pool.dtype).float()      # [B, L, H, D]
        x = x * scale[blk][..., None]
        return torch.where(there[:, :, None, None], x, 0.0)

    k = values(s["k"], s["k_scale"])
    score = torch.einsum("bthgd,blhd->bhtgl", q, k) / math.sqrt(dim)
    del k
    sees = pos[None, None] <= (s["lens"][:, None] - t + torch.arange(t, device="cuda"))[..., None]
    score = score.masked_fill(~sees[:, None, :, None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m)
    del score
    norm = p.sum(-1)
    v = values(s["v"], s["v_scale"])
    out = torch.einsum("bhtgl,blhd->bthgd", p, v) / norm.permute(0, 2, 1, 3)[..., None]
    return out.reshape(s["q"].shape).to(TYPES[c["out"]])


def _plain_append(s):
    c = s["case"]
    page, hkv, code = c["page"], c["hkv"], c["code"]
    blocks = s["k"].shape[0]
    slot = s["slots"]
    real = slot >= 0
    # rows without a slot go to a page past the pool's last, which is dropped
    blk = torch.where(real, slot // page, blocks)
    off = torch.where(real, slot % page, 0)
    first = torch.full((blocks + 1,), page, device="cuda").scatter_reduce(0, blk, off, "amin")
    first = first[:blocks]
    old_row = torch.arange(page, device="cuda") < first[:, None]           # [blocks, page]
    touched = first < page
    for new, pool, scale in ((s["new_k"], s["k"], s["k_scale"]), (s["new_v"], s["v"], s["v_scale"])):
        x = new.float()
        a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)           # [rows, H]
        amax = torch.zeros(blocks + 1, hkv, device="cuda").scatter_reduce(
            0, blk[:, None].expand(-1, hkv), a, "amax")[:blocks]
        need = _pow2(_page_exp(amax, code))
        grown = torch.where((first > 0)[:, None], torch.maximum(need, scale), need)
        grown = torch.where(touched[:, None], grown, scale)
        old = pool.float() * (scale / grown)[:, None, :, None]
        changes = old_row & touched[:, None]
        pool.copy_(torch.where(changes[:, :, None, None], old, pool.float()).to(F8[code]))
        top = CODE_MAX[code]
        padded = torch.cat([grown, grown.new_ones(1, hkv)])
        y = (x / padded[blk][..., None]).clamp(-top, top).to(F8[code]).view(torch.uint8)
        bytes_ = torch.cat([pool.view(torch.uint8), y.new_zeros(1, *pool.shape[1:])])
        bytes_[blk, off] = y
        pool.view(torch.uint8).copy_(bytes_[:blocks])
        scale.copy_(grown)
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _plain_tables(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    lens, new, count = s["lens"].long(), s["new"].long(), s["state"][0].long()
    batch, width = table.shape
    gone = new < 0
    add = new.clamp(min=0)
    have = (lens + page - 1) // page
    need = torch.where(gone, 0, (lens + add + page - 1) // page - have)
    given = torch.where(gone, have, 0)
    total, back, rows = need.sum(), given.sum(), add.sum()
    fits = ((lens + add <= width * page) & (lens >= 0)).all() & (rows <= s["slots"].numel())
    enough = total <= count + back
    ok = fits & enough
    # the blocks of released sequences, in the order of the sequences and of their tables
    col = torch.arange(width, device="cuda")
    pushed = torch.zeros(batch * width + 1, dtype=torch.int64, device="cuda")
    at = (given.cumsum(0) - given)[:, None] + col
    mine = gone[:, None] & (col < have[:, None])
    pushed[torch.where(mine, at, batch * width)] = table.long()
    # taken from the top of the stack: the last pushed first
    k = (need.cumsum(0) - need)[:, None] + col - have[:, None]
    takes = (col >= have[:, None]) & (col < (have + need)[:, None]) & ok
    k = torch.where(takes, k, 0)
    from_free = free.long()[(count - 1 - (k - back)).clamp(0, free.numel() - 1)]
    block = torch.where(k < back, pushed[(back - 1 - k).clamp(min=0)], from_free)
    table.copy_(torch.where(takes, block, table.long()))
    i = torch.arange(free.numel(), device="cuda")
    left = (back - total).clamp(min=0)
    puts = (i >= count) & (i < count + left) & ok
    free.copy_(torch.where(puts, pushed[(i - count).clamp(0, batch * width)], free.long()))
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)]) * ok
    j = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(cu, j, right=True).clamp(max=batch) - 1
    pos = lens[b] + j - cu[b]
    block = table.long()[b, (pos // page).clamp(0, width - 1)]
    s["slots"].copy_(torch.where(j < cu[-1], block * page + pos % page, -1))
    s["cu"].copy_(cu)
    s["lens_out"].copy_(torch.where(ok, torch.where(gone, 0, lens + add), lens))
    s["state_out"][0] = torch.where(ok, count + back - total, count)
    code = torch.where(ok, 0, torch.where(fits, 3, 1))
    s["state_out"][1] = torch.where(s["state"][1] != 0, s["state"][1].long(), code)
    return {k: s[k] for k in ("table", "free", "slots", "cu", "lens_out", "state_out")}


# ------------------------------------------------------------------ the library's calls

def _own_attend(s):
    from split_kv_decode_gb300 import api as A
    c = s["case"]
    out = torch.empty(s["q"].shape, dtype=TYPES[c["out"]], device="cuda")
    if "plan" not in s:       # what a serving loop makes once for its lengths
        args = A.make_paged_args(s["q"], s["k"], s["v"], 1.0 / math.sqrt(c["dim"]),
                                 s["table"].shape[1], out_dtype=out.dtype)
        plan = A.decode_attn_plan(args, s["host_lens"])
        dev = A.make_dev(seq_lens=s["lens"], block_table=s["table"], k_pool=s["k"], v_pool=s["v"])
        scales = A.make_scales(s["k_scale"], s["v_scale"])
        s["plan"] = args, plan, dev, scales, A.new_workspace(plan)
    args, plan, dev, scales, workspace = s["plan"]
    A.decode_attn_splitk_8bit(args, plan, dev, scales, s["q"], s["k"], s["v"], out, workspace)
    return out


def _own_append(s):
    from split_kv_decode_gb300 import api as A
    if "append" not in s:
        s["append"] = A.make_append(s["new_k"], s["new_v"], s["k"], s["v"], s["k_scale"],
                                    s["v_scale"])
    A.decode_attn_append_8bit(s["append"], s["new_k"], s["new_v"], s["slots"], s["k"], s["v"],
                              s["k_scale"], s["v_scale"])
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _own_tables(s):
    from split_kv_decode_gb300 import api as A
    if "tables" not in s:
        s["tables"] = A.make_tables(s["lens"], s["table"], s["free"], s["state"],
                                    s["case"]["page"], seq_lens_out=s["lens_out"],
                                    state_out=s["state_out"])
    A.decode_attn_grow_tables(s["tables"], s["new"], s["slots"], s["cu"])
    return {k: s[k] for k in ("table", "free", "slots", "cu", "lens_out", "state_out")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "tables": _own_tables}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "tables": _plain_tables}[op](state)


# ------------------------------------------------------------------ work, and 64 bits

def work(case):
    page = case["page"]
    if case["op"] == "attend":
        lens = _ints(case["lens"])
        rows, total = len(lens) * case["q_len"] * case["hq"], sum(lens)
        pages = sum(-(-n // page) for n in lens)
        return {"bytes": 2 * total * case["hkv"] * case["dim"] + pages * (8 * case["hkv"] + 4)
                + rows * case["dim"] * (4 + SIZE[case["out"]]),
                "flops": 4 * case["q_len"] * case["hq"] * case["dim"] * total}
    if case["op"] == "append":
        lens, new = _ints(case["lens"]), _ints(case["new"])
        pages = sum(-(-(n + m) // page) - n // page for n, m in zip(lens, new))
        values = 2 * sum(new) * case["hkv"] * case["dim"]
        return {"bytes": values * (SIZE[case["src"]] + 1) + 8 * sum(new)
                + 2 * 4 * pages * case["hkv"], "flops": 3 * values}
    lens, new = _ragged_new(case)
    rows = sum(max(m, 0) for m in new)
    moved = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(lens, new) if m > 0)
    moved += sum(-(-n // page) for n, m in zip(lens, new) if m < 0)
    return {"bytes": 8 * (rows + 3) + 8 * moved + 16 * case["batch"], "flops": 0}


def _power(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _decoded(codes, code):
    """What 8-bit codes stand for, in 64 bits, from their bits."""
    u = codes.view(torch.uint8).long()
    man, bias = MANTISSA[code], 1 - LEAST_EXP[code]
    e, m = (u & 127) >> man, u & ((1 << man) - 1)
    x = torch.where(e > 0, (m + (1 << man)).double() * _power(e - bias - man),
                    m.double() * 2.0 ** (1 - bias - man))
    return torch.where(u > 127, -x, x)


def _rounded(x, code):
    """x rounded to the nearest value of the code, ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    quantum = _power((e - 1).clamp(min=LEAST_EXP[code]) - MANTISSA[code])
    return torch.round(x / quantum) * quantum


def exact(case, seed):
    if case["op"] == "tables":
        return None                                # whole numbers only
    s = prepare(case, seed)
    page, hkv, dim, code = case["page"], case["hkv"], case["dim"], case["code"]
    if case["op"] == "attend":
        t, group = case["q_len"], case["hq"] // case["hkv"]
        out = []
        for b, n in enumerate(s["host_lens"]):
            pages = s["table"][b, :-(-n // page)].long()
            q = s["q"][b].double().reshape(t, hkv, group, dim)
            k = (_decoded(s["k"].view(torch.uint8)[pages], code)
                 * s["k_scale"][pages].double()[:, None, :, None]).reshape(-1, hkv, dim)[:n]
            score = torch.stack([q[:, h].reshape(-1, dim) @ k[:, h].T for h in range(hkv)])
            del k
            score = score.reshape(hkv, t, group, n) * dim ** -0.5
            late = torch.arange(n, device="cuda") > (n - t + torch.arange(t, device="cuda"))[:, None]
            p = torch.softmax(score.masked_fill(late[None, :, None], -math.inf), -1)
            del score
            v = (_decoded(s["v"].view(torch.uint8)[pages], code)
                 * s["v_scale"][pages].double()[:, None, :, None]).reshape(-1, hkv, dim)[:n]
            o = torch.stack([p[h].reshape(-1, n) @ v[:, h] for h in range(hkv)])
            out.append(o.reshape(hkv, t, group, dim).transpose(0, 1).reshape(s["q"][b].shape))
        return torch.stack(out)
    # append: page by page of each sequence's run, in the order of the slots
    slot = s["slots"][s["slots"] >= 0]
    rows = slot.numel()
    blk, off = slot // page, slot % page
    starts = torch.ones(rows, dtype=torch.bool, device="cuda")
    starts[1:] = blk[1:] != blk[:-1]
    run_of = starts.cumsum(0) - 1                 # each page's new rows are one run
    heads = torch.nonzero(starts)[:, 0]
    page_of, from_row = blk[heads], off[heads]
    got = []
    for new, pool, scale in ((s["new_k"], s["k"], s["k_scale"]), (s["new_v"], s["v"], s["v_scale"])):
        x = new[:rows].double()
        top = torch.zeros(len(heads), hkv, dtype=torch.float64, device="cuda").scatter_reduce(
            0, run_of[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        e = torch.ceil(torch.log2(top / CODE_MAX[code])).clamp(min=MIN_EXP)
        # a logarithm next to a whole number is settled by the definition itself
        e = torch.where(top <= CODE_MAX[code] * _power(e - 1), e - 1, e).clamp(min=MIN_EXP)
        e = torch.where(top > CODE_MAX[code] * _power(e), e + 1, e)
        was = scale[page_of].double()
        now = torch.where(from_row[:, None] > 0, torch.maximum(_power(e), was), _power(e))
        value = torch.cat([_decoded(c, code) for c in pool.view(torch.uint8).split(1024)])
        for lo in range(0, len(heads), 512):      # old rows of pages that go on
            at = slice(lo, lo + 512)
            keep = torch.arange(page, device="cuda") < from_row[at, None]
            old = value[page_of[at]]
            moved = _rounded(old * (was[at] / now[at])[:, None, :, None], code)
            value[page_of[at]] = torch.where(keep[:, :, None, None], moved, old)
        value[blk, off] = _rounded(x / now[run_of][..., None], code)
        scales = scale.double()
        scales[page_of] = now
        got.append((value, scales))
    return got[0][0], got[1][0], got[0][1], got[1][1]
