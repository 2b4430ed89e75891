"""What three operators of a serving step over a 16-bit KV cache are measured on.

  prep    the new tokens' queries and keys normalised head by head, rotated to their
          positions (one axis or several), and the keys and values written into the
          slots of the cache (decode_attn_rope_append)
  scored  split-KV decode attention whose scores are capped by a tanh, biased by the
          distance, or limited to a window, a kept prefix or a document
          (decode_attn_splitk_scored)
  shared  the same over sequences that continue one long common prefix, which is read
          and multiplied once for all of them (the same call with a shared table)

`run` with `own` false computes them in elementary torch operations; with `own`
true it makes the library's calls.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases

def _prep(name, tokens, hq, hkv, dim, page, src="bf16", cache="bf16", q_out="bf16", rot=0,
          axes="", pairs="halves", norm=True, far=1 << 17, pad=0):
    return {"name": name, "op": "prep", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "src": src, "cache": cache, "q_out": q_out, "rot": rot or dim,
            "axes": axes, "pairs": pairs, "norm": norm, "far": far, "pad": pad}


def _scored(name, lens, hq, hkv, dim, page, q_len=1, cache="bf16", q="bf16", out="bf16",
            cap=0.0, slopes=False, window=0, keep=0, starts=False):
    return {"name": name, "op": "scored", "lens": lens, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "q_len": q_len, "cache": cache, "q": q, "out": out, "cap": cap,
            "slopes": slopes, "window": window, "keep": keep, "starts": starts, "prefix": 0}


def _shared(name, prefix, lens, hq, hkv, dim, page, q_len=1, cache="bf16", q="bf16", out="bf16",
            cap=0.0, slopes=False):
    return {"name": name, "op": "shared", "prefix": prefix, "lens": lens, "hq": hq, "hkv": hkv,
            "dim": dim, "page": page, "q_len": q_len, "cache": cache, "q": q, "out": out,
            "cap": cap, "slopes": slopes, "window": 0, "keep": 0, "starts": False}


def _text(xs):
    return ",".join(str(x) for x in xs)


def _ints(s):
    return [int(x) for x in s.split(",")] if s else []


def _ragged(batch, lo, hi, seed):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(batch)]


def listed():
    return [
        # one decode step of a batch of 32 (32/8 heads of 128): a row each
        _prep("prep_step32", 32, 32, 8, 128, 16),
        # a long prompt in one call (16/4 heads of 256), f16 throughout
        _prep("prep_prompt32k", 32768, 16, 4, 256, 64, src="f16", cache="f16", q_out="f16"),
        # frames of a video among text: time, height and width on their own frequencies, half
        # of each head rotated in neighbouring pairs, f32 projections, a padded batch
        _prep("prep_video3", 9999, 8, 2, 128, 48, src="f32", q_out="f32", rot=64, axes="8,12,12",
              pairs="neighbours", far=20000, pad=17),
        # a chat's first answers: one request of a few hundred tokens; latency counts
        _scored("scored_short", "713", 8, 2, 128, 16, cap=50.0),
        # the benchmark's long single context (16/4 heads of 256, f16), capped scores
        _scored("scored_cap_152k", "151552", 16, 4, 256, 0, cache="f16", q="f32", out="f32",
                cap=30.0),
        # its ragged batch of 32 (32/8 heads of 128) on a layer with a window, whose first
        # positions stay visible
        _scored("scored_window32", _text(_ragged(32, 1024, 131072, 1238)), 32, 8, 128, 16,
                window=4096, keep=64),
        # four draft tokens a sequence under a bias by distance (24/4 heads of 256): 24 rows
        _scored("scored_bias_draft4", "8192,20480,61440,131072", 24, 4, 256, 128, q_len=4,
                slopes=True),
        # every query head with its own KV head, odd pages, padding on the left
        _scored("scored_docs_mha", "2999,17,1500,3500,64,2048,777,1", 16, 16, 128, 48,
                cache="f16", q="f32", out="f16", starts=True),
        # four samples of one short prompt; latency counts
        _shared("shared_best4", 1024, "33,7,160,64", 8, 2, 128, 16),
        # 32 requests (32/8 heads of 128) behind one long document
        _shared("shared_doc32", 32768, _text(_ragged(32, 16, 2048, 5)), 32, 8, 128, 64),
        # a full batch behind a system prompt: as many rows as a prompt has
        _shared("shared_system256", 8192, _text(_ragged(256, 1, 1024, 6)), 32, 8, 128, 16),
        # drafts of four tokens behind a long prefix (24/4 heads of 256)
        _shared("shared_draft4", 61440, _text(_ragged(16, 4, 4096, 7)), 24, 4, 256, 64, q_len=4,
                cache="f16", q="f32", out="f16", cap=50.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "scored", "scored", "shared"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([128, 256])
    group = rng.choice([1, 2, 4, 6, 8, 12])
    cache = rng.choice(["bf16", "f16"])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    if op == "prep":
        tokens = _log(rng, 1, max(2, (1 << 27) // (hkv * (group + 2) * dim)))
        rot = rng.choice([dim, dim, dim // 2])
        axes = rng.choice(["", "", "two", "three"])
        if axes == "two":
            axes = _text([rot // 8, rot // 2 - rot // 8])
        elif axes == "three":
            axes = _text([rot // 8, rot // 8 + 5, rot // 4 - 5])
        return {"op": "prep", "tokens": tokens, "hq": hkv * group, "hkv": hkv, "dim": dim,
                "page": page, "src": rng.choice(["f32", "f16", "bf16"]),
                "cache": rng.choice(["f32", "f16", "bf16"]),
                "q_out": rng.choice(["f32", "f16", "bf16"]), "rot": rot, "axes": axes,
                "pairs": rng.choice(["halves", "neighbours"]), "norm": rng.choice([True, True, False]),
                "far": _log(rng, 64, 1 << 20), "pad": rng.choice([0, 0, 3])}
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    case = {"op": op, "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page, "q_len": q_len,
            "cache": cache, "q": rng.choice(["f32", cache]),
            "out": rng.choice(["f32", "f16", "bf16"]), "cap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "slopes": rng.choice([False, False, True]), "window": 0, "keep": 0, "starts": False,
            "prefix": 0}
    if op == "scored":
        batch = _log(rng, 1, 32)
        hi = _log(rng, 64, max(65, min(131072, (1 << 27) // (batch * hkv * dim))))
        case["page"] = rng.choice([0, page, page])
        case["window"] = rng.choice([0, 0, _log(rng, 16, 8192)])
        case["keep"] = rng.choice([0, 0, _log(rng, 1, 300)])
        case["starts"] = rng.choice([False, False, True])
    else:
        batch = _log(rng, 2, 256)
        hi = _log(rng, 16, max(17, min(4096, (1 << 25) // (batch * hkv * dim))))
        top = max(2, min(65536, (1 << 25) // (hkv * dim),
                         (1 << 29) // (batch * q_len * hkv * group))) // page
        case["prefix"] = page * _log(rng, 1, max(2, top))
    case["lens"] = _text([max(q_len, _log(rng, max(1, hi // 16), hi)) for _ in range(batch)])
    return case


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype, spread=1.0):
    """N(0, spread), made a few million numbers at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(spread))
    return out


def _prepare_prep(s, g, case):
    n, hq, hkv, dim, page = (case[k] for k in ("tokens", "hq", "hkv", "dim", "page"))
    rows = n + case["pad"]
    # q, k and v of one fused projection: rows of [Q heads | K heads | V heads]
    fused = _randn(g, rows, hq + 2 * hkv, dim, dtype=TYPES[case["src"]], spread=1.5)
    s["q"], s["k"], s["v"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    axes = max(1, len(_ints(case["axes"])))
    if axes == 1:                                   # runs of positions, as sequences have them
        start = torch.randint(0, case["far"], (1,), generator=g, device="cuda")
        pos = (start + torch.arange(rows, device="cuda"))[None]
        if n <= 256:                                # a decode step: any position each
            pos = torch.randint(0, case["far"], (1, rows), generator=g, device="cuda")
    else:
        pos = torch.randint(0, case["far"], (axes, rows), generator=g, device="cuda")
    s["positions"] = pos.contiguous()
    half = case["rot"] // 2
    s["inv_freq"] = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).cuda()
    s["axis"] = [i for i, m in enumerate(_ints(case["axes"])) for _ in range(m)] or [0] * half
    s["q_weight"] = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    s["k_weight"] = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    blocks = -(-n // page) + 3
    order = torch.randperm(blocks, generator=g, device="cuda")
    i = torch.arange(n, device="cuda")
    s["slots"] = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    s["slots"][:n] = order[i // page] * page + i % page
    for name in ("k_pool", "v_pool"):
        s[name] = torch.zeros(blocks, page, hkv, dim, dtype=TYPES[case["cache"]], device="cuda")
    s["q_rot"] = torch.empty(rows, hq, dim, dtype=TYPES[case["q_out"]], device="cuda")


def _prepare_attend(s, g, case):
    lens, prefix, page = _ints(case["lens"]), case["prefix"], case["page"]
    hkv, dim, dt = case["hkv"], case["dim"], TYPES[case["cache"]]
    batch, top = len(lens), max(lens)
    if page == 0:                                   # contiguous caches with some room
        s["k"] = _randn(g, batch, top + 37, hkv, dim, dtype=dt)
        s["v"] = _randn(g, batch, top + 37, hkv, dim, dtype=dt)
        for b, n in enumerate(lens):                # past a length: never written
            s["k"][b, n:], s["v"][b, n:] = math.nan, math.nan
    else:
        used = [-(-n // page) for n in lens]
        ahead = prefix // page
        blocks = ahead + sum(used) + 3
        s["k"] = _randn(g, blocks, page, hkv, dim, dtype=dt)
        s["v"] = _randn(g, blocks, page, hkv, dim, dtype=dt)
        order = torch.randperm(blocks, generator=g, device="cuda").int()
        s["shared_table"] = order[:ahead].clone()
        s["table"] = torch.zeros(batch, max(used) + 1, dtype=torch.int32, device="cuda")
        at = ahead
        for b, n in enumerate(lens):
            s["table"][b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            if n % page:
                last = order[at - 1].long()
                s["k"][last, n % page:], s["v"][last, n % page:] = math.nan, math.nan
    shape = (batch, case["hq"], dim)
    if case["q_len"] > 1:
        shape = (batch, case["q_len"], case["hq"], dim)
    s["q"] = _randn(g, *shape, dtype=TYPES[case["q"]], spread=2.0)
    s["host_lens"] = lens
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    h = torch.arange(1, case["hq"] + 1, device="cuda")
    s["slopes"] = torch.exp2(-8.0 * h / case["hq"]) if case["slopes"] else None
    s["starts"] = None
    if case["starts"]:                              # the first position of each one's document
        s["starts"] = (torch.rand(batch, generator=g, device="cuda") * 0.6 * s["lens"]).int()


def prepare(case, seed):
    s = {"case": case}
    {"prep": _prepare_prep}.get(case["op"], _prepare_attend)(s, _gen(seed), case)
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_prep(s):
    c = s["case"]
    dim, rot = c["dim"], c["rot"]
    half = rot // 2
    axis = torch.tensor(s["axis"], device="cuda")
    angle = s["positions"].double()[axis].T * s["inv_freq"]                 # [rows, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotated(x, weight, cos, sin):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
        if c["pairs"] == "halves":
            a, b = y[..., :half], y[..., half:rot]
            return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1)
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([z, y[..., rot:]], -1)

    s["q_rot"].copy_(rotated(s["q"], s["q_weight"], cos, sin))
    # rows without a slot come after the others
    n = c["tokens"]
    blk, off = s["slots"][:n] // c["page"], s["slots"][:n] % c["page"]
    k = rotated(s["k"][:n], s["k_weight"], cos[:n], sin[:n])
    s["k_pool"][blk, off] = k.to(s["k_pool"].dtype)
    s["v_pool"][blk, off] = s["v"][:n].to(s["v_pool"].dtype)
    return s["q_rot"], s["k_pool"], s["v_pool"]


def _plain_attend(s):
    c = s["case"]
    page, hkv, dim, t, prefix = c["page"], c["hkv"], c["dim"], c["q_len"], c["prefix"]
    batch, top = len(s["host_lens"]), max(s["host_lens"])
    group = c["hq"] // hkv
    q = s["q"].float().reshape(batch, t, hkv, group, dim)
    j = torch.arange(top, device="cuda")
    there = j < s["lens"][:, None]                                          # [B, L]
    at = s["lens"][:, None].long() - t + torch.arange(t, device="cuda")     # [B, T] of the tokens
    sees = j <= at[..., None]                                               # [B, T, L]
    if c["window"]:
        sees &= j > at[..., None] - c["window"]
    sees |= j < c["keep"]
    sees &= there[:, None]
    if s["starts"] is not None:
        sees &= (j >= s["starts"][:, None])[:, None]

    def own_rows(x):
        if page == 0:
            x = x[:, :top]
        else:
            blk = torch.where(there, s["table"][:, :-(-top // page)].long()
                              .repeat_interleave(page, 1)[:, :top], 0)
            x = x[blk, (j % page).expand(batch, top)]                       # [B, L, H, D]
        return torch.where(there[..., None, None], x.float(), 0.0)

    def score(raw, distance):                       # [B, H, T, G, n], [B, T, n]
        y = raw / math.sqrt(dim)
        if c["cap"]:
            y = c["cap"] * torch.tanh(y / c["cap"])
        if c["slopes"]:
            slope = s["slopes"].view(1, hkv, 1, group, 1)
            y = y - slope * distance.float()[:, None, :, None]
        return y

    y = score(torch.einsum("bthgd,blhd->bhtgl", q, own_rows(s["k"])), (at[..., None] - j).abs())
    y = y.masked_fill(~sees[:, None, :, None, :], -math.inf)
    m = y.amax(-1, keepdim=True)
    if prefix:
        def front_rows(x):
            return x[s["shared_table"].long()].float().reshape(prefix, hkv, dim)
        i = torch.arange(prefix, device="cuda")
        z = score(torch.einsum("bthgd,lhd->bhtgl", q, front_rows(s["k"])),
                  prefix + at[..., None] - i)
        m = torch.maximum(m, z.amax(-1, keepdim=True))
    m = m.clamp(min=-1e30)                          # a token that sees nothing gives zeros
    p = torch.exp(y - m)
    norm = p.sum(-1)
    out = torch.einsum("bhtgl,blhd->bthgd", p, own_rows(s["v"]))
    if prefix:
        p = torch.exp(z - m)
        norm = norm + p.sum(-1)
        out = out + torch.einsum("bhtgl,lhd->bthgd", p, front_rows(s["v"]))
    norm = norm.permute(0, 2, 1, 3)[..., None]
    out = torch.where(norm > 0, out / norm, 0.0)
    return out.reshape(s["q"].shape).to(TYPES[c["out"]])


# ------------------------------------------------------------------ the library's calls

def _own_prep(s):
    from split_kv_decode_gb300 import api as A
    c = s["case"]
    if "rope" not in s:       # what a serving loop makes once for its model and its buffers
        s["rope"] = A.make_rope(s["inv_freq"], axes=s["axis"],
                                interleaved=c["pairs"] == "neighbours")
        weights = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": 1e-6}
        s["prep"] = A.make_prep(s["q"], s["k"], s["v"], s["q_rot"], s["k_pool"], s["v_pool"],
                                s["rope"], **(weights if c["norm"] else {}))
    A.decode_attn_rope_append(s["prep"], s["q"], s["k"], s["v"], s["positions"], s["slots"],
                              s["q_rot"], s["k_pool"], s["v_pool"])
    return s["q_rot"], s["k_pool"], s["v_pool"]


def _own_attend(s):
    from split_kv_decode_gb300 import api as A
    c = s["case"]
    out = torch.empty(s["q"].shape, dtype=TYPES[c["out"]], device="cuda")
    if "plan" not in s:       # what a serving loop makes once for its lengths
        scale = 1.0 / math.sqrt(c["dim"])
        if c["page"]:
            args = A.make_paged_args(s["q"], s["k"], s["v"], scale, s["table"].shape[1],
                                     out_dtype=out.dtype)
            dev = A.make_dev(seq_lens=s["lens"], block_table=s["table"], k_pool=s["k"],
                             v_pool=s["v"])
        else:
            args = A.make_args(s["q"], s["k"], s["v"], scale, out_dtype=out.dtype)
            dev = A.make_dev(seq_lens=s["lens"])
        score = A.make_score(s["q"], softcap=c["cap"], slopes=s["slopes"], window=c["window"],
                             keep=c["keep"], starts=s["starts"], shared_len=c["prefix"],
                             shared_table=s["shared_table"] if c["prefix"] else None)
        plan = A.decode_attn_plan_scored(args, score, s["host_lens"])
        s["plan"] = args, plan, dev, score, A.new_workspace(plan)
    args, plan, dev, score, workspace = s["plan"]
    A.decode_attn_splitk_scored(args, plan, dev, score, s["q"], s["k"], s["v"], out, workspace)
    return out


def run(state):
    prep = state["case"]["op"] == "prep"
    if own:
        return _own_prep(state) if prep else _own_attend(state)
    return _plain_prep(state) if prep else _plain_attend(state)


# ------------------------------------------------------------------ work, and 64 bits

def work(case):
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "prep":
        n, rows = case["tokens"], case["tokens"] + case["pad"]
        axes = max(1, len(_ints(case["axes"])))
        return {"bytes": rows * hq * dim * (SIZE[case["src"]] + SIZE[case["q_out"]])
                + 2 * n * hkv * dim * (SIZE[case["src"]] + SIZE[case["cache"]])
                + rows * 8 * (1 + axes),
                "flops": rows * (hq + hkv) * dim * (6 if case["norm"] else 3)}
    lens, t = _ints(case["lens"]), case["q_len"]
    near = case["window"] + t - 1 if case["window"] else 1 << 30
    spans = [min(n, near + min(case["keep"], max(0, n - near))) for n in lens]
    if case["starts"]:                              # 0.3 of a length lies before it, on average
        spans = [max(1, int(0.7 * n)) for n in spans]
    rows = len(lens) * t * hq
    return {"bytes": 2 * 2 * (sum(spans) + case["prefix"]) * hkv * dim
            + rows * dim * (SIZE[case["q"]] + SIZE[case["out"]]),
            "flops": 4 * t * hq * dim * (sum(spans) + len(lens) * case["prefix"])}


def _exact_prep(s, case):
    dim, rot, page, n = case["dim"], case["rot"], case["page"], case["tokens"]
    half = rot // 2
    first = torch.arange(half, device="cuda")
    if case["pairs"] == "halves":
        second = first + half
    else:
        first, second = 2 * first, 2 * first + 1

    def turned(x, weight, positions):
        y = x.double()
        if case["norm"]:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / dim + 1e-6) * weight.double()
        phase = torch.stack([positions[a].double() * f for a, f in zip(s["axis"], s["inv_freq"])],
                            -1)
        unit = torch.polar(torch.ones_like(phase), phase)[:, None]
        z = torch.complex(y[..., first], y[..., second]) * unit
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q = torch.cat([turned(a, s["q_weight"], p) for a, p in
                   zip(s["q"].split(4096), s["positions"].split(4096, 1))])
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    slot = s["slots"][:n]
    k_pool.view(-1, *k_pool.shape[2:])[slot] = torch.cat(
        [turned(a, s["k_weight"], p) for a, p in
         zip(s["k"][:n].split(4096), s["positions"][:, :n].split(4096, 1))])
    v_pool.view(-1, *v_pool.shape[2:])[slot] = s["v"][:n].double()
    return q, k_pool, v_pool


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prep":
        return _exact_prep(s, case)
    page, hkv, dim, t, prefix = (case[k] for k in ("page", "hkv", "dim", "q_len", "prefix"))
    group = case["hq"] // hkv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for h in range(hkv):
        front = [x[s["shared_table"].long(), :, h].double().reshape(prefix, dim)
                 if prefix else None for x in (s["k"], s["v"])]
        for b, n in enumerate(s["host_lens"]):
            if page:
                pages = s["table"][b, :-(-n // page)].long()
                k, v = (x[pages, :, h].reshape(-1, dim)[:n].double() for x in (s["k"], s["v"]))
            else:
                k, v = (x[b, :n, h].double() for x in (s["k"], s["v"]))
            if prefix:
                k, v = torch.cat([front[0], k]), torch.cat([front[1], v])
            heads = slice(h * group, (h + 1) * group)
            q = s["q"][b].double().reshape(t, -1, dim)[:, heads]
            y = (q.reshape(-1, dim) @ k.T).reshape(t, group, -1) * dim ** -0.5
            if case["cap"]:
                y = case["cap"] * torch.tanh(y / case["cap"])
            where = torch.arange(prefix + n, device="cuda")
            token = prefix + n - t + torch.arange(t, device="cuda")[:, None]
            if case["slopes"]:
                y = y - s["slopes"][heads].double()[:, None] * (token - where).abs()[:, None]
            hidden = where > token
            if case["window"]:
                hidden |= where <= token - case["window"]
            hidden &= where >= case["keep"]
            if s["starts"] is not None:
                hidden |= where < s["starts"][b]
            y = y.masked_fill(hidden[:, None], -math.inf)
            p = torch.softmax(y, -1)
            p = torch.where(hidden.all(-1)[:, None, None], 0.0, p)
            o = (p.reshape(t * group, -1) @ v).reshape(t, group, dim)
            out[b].view(t, -1, dim)[:, heads] = o
    return out
