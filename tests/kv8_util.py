"""References for the 8-bit paged cache, in 64 bits and plain loops: what a code
stands for, the rounding to a code, the page rule of the append, the stack of free
blocks, and attention over dequantised pages. Shares no code with the library."""
import math

import numpy as np
import torch

TDT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MAX = {"e4m3": 448.0, "e5m2": 57344.0}
_MAN = {"e4m3": 3, "e5m2": 2}
_EMIN = {"e4m3": -6, "e5m2": -14}


def code_values(code):
    """The 256 values of a code, indexed by its bits (float64)."""
    out = np.empty(256)
    man, emin = _MAN[code], _EMIN[code]
    for u in range(256):
        e, m = (u & 127) >> man, u & ((1 << man) - 1)
        x = math.ldexp(m + (1 << man), e - 1 + emin - man) if e else math.ldexp(m, emin - man)
        if code == "e4m3" and (u & 127) == 127:
            x = math.nan
        if code == "e5m2" and e == 31:
            x = math.inf if m == 0 else math.nan
        out[u] = -x if u > 127 else x
    return out


def decode(codes, code):
    """uint8 (or float8) tensor -> float64 numpy."""
    return code_values(code)[codes.view(torch.uint8).cpu().numpy()]


def round_to(x, code):
    """x (float64 numpy) to the nearest value of the code, ties to even, saturating."""
    x = np.asarray(x, dtype=np.float64)
    top = MAX[code]
    _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    quantum = np.ldexp(1.0, np.maximum(e - 1, _EMIN[code]) - _MAN[code])
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.rint(x / quantum) * quantum
        return np.where(np.isnan(x), np.nan, np.clip(y, -top, top))


def page_exponent(amax, code):
    """Least e >= -100 with amax <= MAX * 2^e."""
    if amax <= 0:
        return -100
    e = math.floor(math.log2(amax / MAX[code])) - 1
    while amax > math.ldexp(MAX[code], e):
        e += 1
    return max(e, -100)


def append_reference(x, slots, values, scale, page, code):
    """The page rule, slot by slot. x [T, H, D] float64, values [NB, page, H, D] (what the
    codes stand for, without the scale) and scale [NB, H] float64; both are updated."""
    t, T = 0, len(slots)
    while t < T:
        s = int(slots[t])
        blk, p0 = divmod(s, page) if s >= 0 else (-1, 0)
        if blk < 0 or blk >= values.shape[0]:
            t += 1
            continue
        n = 1
        while t + n < T and p0 + n < page and int(slots[t + n]) == s + n:
            n += 1
        for h in range(x.shape[1]):
            rows = x[t:t + n, h]
            fin = np.abs(rows[np.isfinite(rows)])
            new = 2.0 ** page_exponent(float(fin.max()) if fin.size else 0.0, code)
            if p0 > 0:
                new = max(new, scale[blk, h])
                if new > scale[blk, h]:
                    values[blk, :p0, h] = round_to(values[blk, :p0, h] * (scale[blk, h] / new), code)
            with np.errstate(invalid="ignore"):
                values[blk, p0:p0 + n, h] = round_to(rows / new, code)
            scale[blk, h] = new
        t += n


class Blocks:
    """The free list and tables, as Python lists."""

    def __init__(self, batch, num_blocks, width, page):
        self.free = list(range(num_blocks - 1, -1, -1))
        self.rows = [[] for _ in range(batch)]
        self.lens = [0] * batch
        self.width, self.page = width, page

    def grow(self, new, capacity):
        """-> (status, slots, cu)"""
        P = self.page
        want = [0 if n < 0 else -(-(L + n) // P) - -(-L // P) for L, n in zip(self.lens, new)]
        back = sum(len(r) for r, n in zip(self.rows, new) if n < 0)
        fits = all(L + max(n, 0) <= self.width * P for L, n in zip(self.lens, new)) \
            and sum(max(n, 0) for n in new) <= capacity
        if not fits or sum(want) > len(self.free) + back:
            return (3 if fits else 1), [-1] * capacity, [0] * (len(new) + 1)
        for b, n in enumerate(new):
            if n < 0:
                self.free += self.rows[b]
                self.rows[b], self.lens[b] = [], 0
        slots, cu = [], [0]
        for b, n in enumerate(new):
            if n > 0:
                self.rows[b] += [self.free.pop() for _ in range(want[b])]
                for pos in range(self.lens[b], self.lens[b] + n):
                    slots.append(self.rows[b][pos // P] * P + pos % P)
                self.lens[b] += n
            cu.append(len(slots))
        return 0, slots + [-1] * (capacity - len(slots)), cu


def attention_reference(q, k, v, lens, scale, causal=True):
    """q [B, T, Hq, D], k and v lists of [L_b, Hkv, D], all float64 numpy. Token i of T
    sees positions below L - T + 1 + i; a token that sees none gives zeros. NaN in keys
    or values a token does not see has no effect. Returns ([B, T, Hq, D], per-element
    error scale [B, T, Hq, D]: max over the seen positions of sum |q k| * scale)."""
    B, T, Hq, D = q.shape
    out, mag = np.zeros_like(q), np.zeros((B, T, Hq))
    for b in range(B):
        L = lens[b]
        for i in range(T):
            n = max(0, L - T + 1 + i) if causal else L
            if n == 0:
                continue
            for h in range(Hq):
                kv = h // (Hq // k[b].shape[1])
                s = k[b][:n, kv] @ q[b, i, h] * scale
                p = np.exp(s - s.max())
                out[b, i, h] = (p / p.sum()) @ v[b][:n, kv]
                mag[b, i, h] = (np.abs(k[b][:n, kv]) @ np.abs(q[b, i, h])).max() * scale
    return out, mag


def paged_cache(seed, lens, page, hkv, dim, code, *, spread=0.3, spare=3, poison=True,
                uneven=False, width_extra=2):
    """A random 8-bit paged cache on the CPU: N(0, s) values, s differing by page and head,
    quantised page by page with a power-of-two scale. Slots past the lengths, unused pages
    and their scales hold NaN (poison); table entries past a length point anywhere.
    uneven: value scales of the pages spread over 2^-40 .. 2^40."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    nb = sum(used) + spare
    pools, scales = [], []
    for i in range(2):
        x = torch.randn(nb, page, hkv, dim, generator=g, dtype=torch.float64).numpy()
        x = x * np.exp(spread * rng.standard_normal((nb, 1, hkv, 1)))
        if uneven and i == 1:
            x = x * np.exp2(rng.integers(-40, 40, size=(nb, 1, hkv, 1)).astype(float))
        amax = np.abs(x).max((1, 3))
        s = np.array([[2.0 ** page_exponent(a, code) for a in r] for r in amax])
        y = torch.from_numpy(round_to(x / s[:, None, :, None], code)).float().to(TDT[code])
        pools.append(y)
        scales.append(torch.from_numpy(s).float())
    order = torch.randperm(nb, generator=g).tolist()
    table = torch.full((len(lens), max(max(used), 1) + width_extra), 10 ** 9, dtype=torch.int32)
    table[:, 1::2] = -5
    at = 0
    for b, n in enumerate(lens):
        for j in range(used[b]):
            table[b, j] = order[at]
            at += 1
    if poison:
        live = set(order[:at])
        for x, s in zip(pools, scales):
            u = x.view(torch.uint8)
            for blk in range(nb):
                if blk not in live:
                    u[blk] = 0x7F
                    s[blk] = math.nan
            for b, n in enumerate(lens):
                if n % page:
                    u[table[b, n // page], n % page:] = 0x7F
    return pools[0], pools[1], scales[0], scales[1], table


def gathered(pool, scale, table, lens, page, code):
    """Per sequence [L, H, D] float64: what its pages stand for."""
    out = []
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // page)].long()
        x = decode(pool.view(torch.uint8)[ids], code)
        x = x * scale[ids].double().numpy()[:, None, :, None]
        out.append(x.reshape(-1, *x.shape[2:])[:n])
    return out
