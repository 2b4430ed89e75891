"""Scored attention in 64 bits and plain loops, and its inputs. Shares no code with the library."""
import math

import numpy as np
import torch

from split_kv_decode_gb300 import api as A

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}


class Case:
    """Inputs of a call, on the CPU, and the call. Slots past the lengths, unused blocks and table
    entries hold what must not matter: NaN, and blocks that do not exist."""

    def __init__(self, lens, hq, hkv, d, *, page=16, q_len=1, cache="bf16", q="same", out="f32",
                 cap=0.0, slopes=False, window=0, keep=0, keep_lens=None, starts=None, shared=0,
                 scale=None, seed=0, spread=1.5, force_splits=0, max_lens=None, flags=0,
                 timeout_us=0, poison=True, num_sms=0, head_major=False):
        g = torch.Generator().manual_seed(seed)
        self.g = g
        self.lens, self.hq, self.hkv, self.d, self.page = list(lens), hq, hkv, d, page
        self.q_len, self.cache, self.out, self.cap = q_len, cache, out, cap
        self.window, self.keep, self.keep_lens, self.starts = window, keep, keep_lens, starts
        self.shared, self.force_splits, self.flags = shared, force_splits, flags
        self.timeout_us, self.num_sms = timeout_us, num_sms
        self.max_lens = list(max_lens) if max_lens else [max(n, q_len) for n in lens]
        self.qt = cache if q == "same" else q
        self.scale = d ** -0.5 if scale is None else scale
        B, dt = len(self.lens), DT[cache]
        self.q = (torch.randn(B, q_len, hq, d, generator=g) * spread).to(DT[self.qt])
        self.slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq) if slopes else None
        top = max(self.max_lens)
        if page == 0:
            cap_len = top + 5
            shape = (B, hkv, cap_len, d) if head_major else (B, cap_len, hkv, d)
            self.k, self.v = (torch.randn(shape, generator=g).to(dt) for _ in range(2))
            if head_major:
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
            if poison:
                for b, n in enumerate(self.lens):
                    self.k[b, n:], self.v[b, n:] = math.nan, math.nan
            self.table = self.shared_table = None
        else:
            used = [-(-n // page) for n in self.lens]
            ahead = shared // page
            nb = ahead + sum(used) + 2
            shape = (nb, hkv, page, d) if head_major else (nb, page, hkv, d)
            self.k, self.v = (torch.randn(shape, generator=g).to(dt) for _ in range(2))
            if head_major:
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
            order = torch.randperm(nb, generator=g).int()
            self.shared_table = order[:ahead].clone()
            self.table = torch.full((B, -(-top // page) + 2), 10 ** 9, dtype=torch.int32)
            self.table[:, 1::2] = -7
            at = ahead
            for b, n in enumerate(self.lens):
                self.table[b, :used[b]] = order[at:at + used[b]]
                at += used[b]
                if poison and n % page:
                    last = int(order[at - 1])
                    self.k[last, n % page:], self.v[last, n % page:] = math.nan, math.nan
            if poison:
                for i in order[at:].tolist():
                    self.k[i], self.v[i] = math.nan, math.nan

    # ---- the reference
    def rows_of(self, b):
        """Own keys and values [S, Hkv, D] of sequence b, and the shared ones, in float64."""
        n = self.lens[b]
        if self.page == 0:
            own = [x[b, :n].double().numpy() for x in (self.k, self.v)]
            return own, [np.zeros((0,) + x.shape[1:]) for x in own]
        ids = self.table[b, :-(-n // self.page)].long()
        own = [x[ids].reshape(-1, self.hkv, self.d)[:n].double().numpy() for x in (self.k, self.v)]
        ids = self.shared_table.long()
        front = [x[ids].reshape(-1, self.hkv, self.d).double().numpy() for x in (self.k, self.v)]
        return own, front

    def sees(self, b, i):
        """Which own positions token i of sequence b sees."""
        n = self.lens[b]
        o = n - self.q_len + i
        j = np.arange(n)
        if o < 0:
            return j < 0
        keep = self.keep if self.keep_lens is None else min(self.keep_lens[b], self.keep)
        near = (j <= o) & ((j > o - self.window) if self.window else True)
        return ((j < keep) | near) & (j >= (self.starts[b] if self.starts is not None else 0))

    def want(self):
        """Outputs [B, q_len, Hq, D], and per output the largest |q| . |k| scale and the largest |v|
        among what it sees."""
        B, T, G = len(self.lens), self.q_len, self.hq // self.hkv
        out = np.zeros((B, T, self.hq, self.d))
        mag, top = np.zeros((B, T, self.hq)), np.zeros((B, T, self.hq))
        q = self.q.double().numpy()
        for b in range(B):
            (k, v), (fk, fv) = self.rows_of(b)
            for i in range(T):
                o = self.lens[b] - T + i
                if o < 0:
                    continue
                see = self.sees(b, i)
                dist = np.concatenate([self.shared + o - np.arange(len(fk)),
                                       np.abs(o - np.arange(self.lens[b]))[see]])
                for h in range(self.hq):
                    kk = np.concatenate([fk[:, h // G], k[see, h // G]])
                    vv = np.concatenate([fv[:, h // G], v[see, h // G]])
                    if not len(kk):
                        continue
                    with np.errstate(all="ignore"):
                        y = kk @ q[b, i, h] * float(np.float32(self.scale))
                        if self.cap:
                            y = self.cap * np.tanh(y / self.cap)
                        if self.slopes is not None:
                            y = y - float(self.slopes[h]) * dist
                        p = np.exp(y - y.max())
                        out[b, i, h] = p @ vv / p.sum()
                        mag[b, i, h] = (np.abs(kk) @ np.abs(q[b, i, h])).max() * abs(self.scale)
                        top[b, i, h] = np.abs(vv).max()
        return out, mag, top

    # ---- the call
    def setup(self, device="cuda"):
        dev = lambda t: None if t is None else t.to(device)
        ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=device)
        c = self.on = type("On", (), {})()
        c.q, c.table, c.shared_table = dev(self.q), dev(self.table), dev(self.shared_table)
        c.k, c.v = ((x.transpose(1, 2).contiguous().to(device).transpose(1, 2)
                     if not x.is_contiguous() else x.to(device)) for x in (self.k, self.v))
        if self.q_len == 1:
            c.q = c.q[:, 0].contiguous()
        c.lens = ints(self.lens)
        c.slopes, c.starts, c.keep_lens = dev(self.slopes), ints(self.starts), ints(self.keep_lens)
        kw = dict(out_dtype=DT[self.out], force_splits=self.force_splits, flags=self.flags,
                  timeout_us=self.timeout_us)
        if self.page:
            c.args = A.make_paged_args(c.q, c.k, c.v, self.scale, self.table.shape[1], **kw)
            c.dev = A.make_dev(seq_lens=c.lens, block_table=c.table, k_pool=c.k, v_pool=c.v)
        else:
            c.args = A.make_args(c.q, c.k, c.v, self.scale, **kw)
            c.dev = A.make_dev(seq_lens=c.lens)
        c.score = A.make_score(c.q, softcap=self.cap, slopes=c.slopes, window=self.window,
                               keep=self.keep, keep_lens=c.keep_lens, starts=c.starts,
                               shared_len=self.shared,
                               shared_table=c.shared_table if self.shared else None)
        c.plan = A.decode_attn_plan_scored(c.args, c.score, self.max_lens, self.num_sms)
        return c

    def run(self, stream=None):
        c = self.setup()
        c.ws = A.new_workspace(c.plan)
        c.ws.fill_(255)
        c.out = torch.full(c.q.shape, math.nan, dtype=DT[self.out], device="cuda")
        A.decode_attn_splitk_scored(c.args, c.plan, c.dev, c.score, c.q, c.k, c.v, c.out, c.ws,
                                    stream)
        A.decode_attn_device_status(c.ws, stream)
        return c.out.double().cpu().numpy().reshape(len(self.lens), self.q_len, self.hq, self.d)

    def bound(self, want, mag, top):
        """What an output may be off by.

        Scores: the product's f32 sum has D terms of relative error 2^-23 each at most (the MMA
        may round its partial sums down), so 2^-23 D mag; an f32 q of 16 bits (two bf16 terms) adds
        2^-17 mag, of 22 (two f16 terms) or 24 (three) 2^-22. Scaling, cap and bias: 2^-22 of mag and
        8 * 2^-23 of the cap (its quotient and exponential, of 2 units each), and 2^-22 of
        slope times distance, which weighs nothing where it is large: 64 of it.
        Weights: their exponent's error, the exponential's 2^-22, and their own terms' 2^-16 (two
        bf16 terms: half a step of 16 bits), 2^-22 or 2^-24. A relative error e of every
        weight moves the quotient by 2 e max |v| at most; the sums add 2^-20.
        Then the output's rounding."""
        f32q = self.qt == "f32"
        two_bf16 = self.cache == "bf16" and self.out != "f32"
        score = 2.0 ** -23 * self.d * mag + 2.0 ** -22 * mag
        score = score + ((2.0 ** -17 if two_bf16 else 2.0 ** -22) * mag if f32q else 0.0)
        score = score + 8 * 2.0 ** -23 * self.cap + (64 * 2.0 ** -22 if self.slopes is not None else 0)
        weight = np.expm1(score) + 2.0 ** -22 + (2.0 ** -16 if two_bf16 else 2.0 ** -22) + 2.0 ** -20
        err = 2 * (weight * top)[..., None]
        return err + (np.abs(want) + err) * EPS[self.out] / 2 + 2.0 ** -25

    def check(self, stream=None):
        got = self.run(stream)
        want, mag, top = self.want()
        assert np.isfinite(want).all(), "a reference without numbers"
        near(got, want, self.bound(want, mag, top))
        return got


def near(got, want, tol):
    err = np.abs(got - want)
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:5]
    worst = np.unravel_index((err / tol).argmax(), err.shape)
    assert (err <= tol).all(), (worst, float(err[worst]), float(tol[worst]))
