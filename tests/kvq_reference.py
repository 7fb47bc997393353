"""Plain 64-bit forms of the 8-bit cache's operators, written from include/sq.h
(torch on the CPU, one request and block at a time), and caches to call them on."""
import math

import numpy as np
import torch

TOP = {"int8": 127.0, "e4m3": 448.0}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # e4m3: 0 .. 448, code by code


def code_values(u, fmt):
    return u.double() - 128.0 if fmt == "int8" else u.contiguous().view(torch.float8_e4m3fn).double()


def codes(x, s, fmt):
    """Bytes of float32 values x at the float32 scale s: nearest, half to even, infinities to the largest."""
    y = torch.nan_to_num(x.double(), 0.0, math.inf, -math.inf) / float(s)
    if fmt == "int8":
        return (torch.round(y.clamp(-127, 127)) + 128).to(torch.uint8)
    a = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(GRID, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = GRID[hi] - a, a - GRID[lo]
    i = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (i + 128 * torch.signbit(y)).to(torch.uint8)


def values(u, s, fmt):
    """fl32(c s)"""
    return (code_values(u, fmt) * float(s)).float()


class Cache:
    """Codes, scales and which positions hold tokens; everything else holds rubbish."""

    def __init__(self, pages, H, P, d, fmt, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.P, self.H, self.d, self.pages = fmt, P, H, d, pages
        self.k = torch.randint(0, 256, (pages, H, P, d), generator=g, dtype=torch.uint8)
        self.v = torch.randint(0, 256, (pages, H, P // 16, d, 16), generator=g, dtype=torch.uint8)
        self.k[:, :, ::3] = 0xff  # a NaN of e4m3
        self.v[..., ::5] = 0x7f
        bad = torch.tensor([math.nan, math.inf, -1.0, 3e38, 0.0])
        self.scales = bad[torch.randint(0, 5, (pages, H, P // 16, 2), generator=g)]
        self.held = torch.zeros(pages, P, dtype=torch.bool)

    def gpu(self, sq):
        f = {"int8": sq.SQ_KVQ_INT8, "e4m3": sq.SQ_KVQ_E4M3}[self.fmt]
        return sq.SqKvqCache(self.k.cuda(), self.v.cuda(), self.scales.cuda(), f)

    def append(self, k, v, ctx, cu, table):
        """k, v float tensors [N][H][d]; lists; a numpy table."""
        for r, start in enumerate(ctx):
            if start < 0:
                continue
            end = start + cu[r + 1] - cu[r]
            for b in range(start // 16 * 16, end, 16):
                if b // self.P >= table.shape[1] or not 0 <= table[r, b // self.P] < self.pages:
                    continue
                pg, blk, at = int(table[r, b // self.P]), b % self.P // 16, b % self.P
                lo, hi = max(start - b, 0), min(end - b, 16)
                t0 = cu[r] + b + lo - start
                for h in range(self.H):
                    for i, x in ((0, k), (1, v)):
                        new = x[t0:t0 + hi - lo, h].float()
                        fin = new[torch.isfinite(new)].abs()
                        most = float(fin.max()) if fin.numel() else 0.0
                        s = max(np.float32(most / TOP[self.fmt]), np.float32(2.0 ** -100))
                        old = np.float32(self.scales[pg, h, blk, i])
                        c = self.k[pg, h, at:at + 16] if i == 0 else self.v[pg, h, blk].T  # views [16][d]
                        if lo > 0 and s > old:
                            c[:lo] = codes(values(c[:lo], old, self.fmt), s, self.fmt)
                        elif lo > 0:
                            s = old
                        self.scales[pg, h, blk, i] = float(s)
                        c[lo:hi] = codes(new, s, self.fmt)
                self.held[pg, at + lo:at + hi] = True

    def at(self, x, which):
        """The values [n][H][d] of (page, place) pairs x, float32."""
        out = []
        for pg, p in x:
            c = self.k[pg, :, p] if which == 0 else self.v[pg, :, p // 16, :, p % 16]
            s = self.scales[pg, :, p // 16, which].double()[:, None]
            out.append((code_values(c, self.fmt) * s).float())
        return torch.stack(out) if out else torch.zeros(0, self.H, self.d)

    def same(self, c):
        """A GPU cache holds the same tokens: bytes, and scales of the blocks that have any."""
        held = self.held[:, None, :, None].expand_as(self.k)
        assert torch.equal(c.k.cpu()[held], self.k[held])
        held = self.held.view(self.pages, 1, self.P // 16, 1, 16).expand_as(self.v)
        assert torch.equal(c.v.cpu()[held], self.v[held])
        some = self.held.view(self.pages, 1, self.P // 16, 16).any(-1).expand(-1, self.H, -1)
        assert torch.equal(c.scales.cpu()[some], self.scales[some])
        # keys past the tokens, and blocks without any, are as they were
        assert torch.equal(c.k.cpu()[~self.held[:, None, :, None].expand_as(self.k)],
                           self.k[~self.held[:, None, :, None].expand_as(self.k)])
        assert torch.equal(c.v.cpu()[~some], self.v[~some])
        assert torch.equal(c.scales.cpu()[~some].view(torch.int32), self.scales[~some].view(torch.int32))


def tables(lens, P, g, spare=2, cols=1):
    """Pages for requests of these lengths, anywhere in a pool; unused entries are -1."""
    need = [-(-x // P) for x in lens]
    ids = torch.randperm(sum(need) + spare, generator=g).tolist()
    table = np.full((len(lens), max(need + [0]) + cols), -1, np.int32)
    for r, n in enumerate(need):
        table[r, :n] = [ids.pop() for _ in range(n)]
    return table, sum(need) + spare


def filled(lens, P, H, d, fmt, seed, spread=1.0):
    """A cache that holds tokens of random codes and scales 2^(+-spread) / 64 for these requests."""
    g = torch.Generator().manual_seed(seed)
    table, pages = tables(lens, P, g)
    c = Cache(pages, H, P, d, fmt, seed)
    for r, n in enumerate(lens):
        for b in range(0, n, 16):
            pg, blk, m = int(table[r, b // P]), b % P // 16, min(16, n - b)
            if fmt == "int8":
                new = torch.randint(1, 256, (2, H, 16, d), generator=g, dtype=torch.uint8)
            else:
                new = (32 * torch.randn(2, H, 16, d, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c.k[pg, :, b % P:b % P + m] = new[0, :, :m]
            c.v[pg, :, blk, :, :m] = new[1, :, :m].transpose(-1, -2)
            c.scales[pg, :, blk] = torch.exp2(spread * (2 * torch.rand(H, 2, generator=g) - 1)) / 64
            c.held[pg, b % P:b % P + m] = True
    return c, table


def attention(c, q, table, lens, cu, scale, window, most=2 ** 31):
    """o, lse, sum p |v|, the largest scale sum |q k| and (tokens x largest value) of every row, in 64 bits.
    q [nq][Hq][d]."""
    nq, Hq, d = q.shape
    G = Hq // c.H
    o, lse = torch.zeros(nq, Hq, d, dtype=torch.float64), torch.full((nq, Hq), -math.inf, dtype=torch.float64)
    mag, size = torch.zeros(nq, Hq, d, dtype=torch.float64), torch.zeros(nq, Hq, dtype=torch.float64)
    top = torch.zeros(nq, Hq, dtype=torch.float64)
    for r, n in enumerate(lens):
        m = cu[r + 1] - cu[r]
        if m <= 0 or n <= 0:
            continue
        pos = np.arange(n)
        there = np.array([x // c.P < table.shape[1] and 0 <= table[r, x // c.P] < c.pages for x in range(0, n, 16)])
        pos = torch.from_numpy(pos[np.repeat(there, 16)[:n]])
        pos = pos[pos < most]
        if not len(pos):
            continue
        pg, pl = torch.from_numpy(table[r].astype(np.int64))[pos // c.P], pos % c.P
        K = code_values(c.k[pg, :, pl], c.fmt) * c.scales[pg, :, pl // 16, 0].double()[..., None]
        V = code_values(c.v[pg, :, pl // 16, :, pl % 16], c.fmt) * c.scales[pg, :, pl // 16, 1].double()[..., None]
        own = n - m + torch.arange(m)
        seen = pos[None] <= own[:, None]
        if window:
            seen &= pos[None] > own[:, None] - window
        for h in range(Hq):
            qq = q[cu[r]:cu[r + 1], h].double()
            x = (qq @ K[:, h // G].T) * scale
            x = torch.where(seen, x, -math.inf)
            l = torch.logsumexp(x, -1)
            p = torch.where(seen, torch.exp(x - torch.where(l == -math.inf, 0.0, l)[:, None]), 0.0)
            o[cu[r]:cu[r + 1], h] = p @ V[:, h // G]
            mag[cu[r]:cu[r + 1], h] = p @ V[:, h // G].abs()
            lse[cu[r]:cu[r + 1], h] = l
            size[cu[r]:cu[r + 1], h] = torch.where(seen, abs(scale) * (qq.abs() @ K[:, h // G].abs().T), 0.0).amax(-1)
            top[cu[r]:cu[r + 1], h] = (seen * (TOP[c.fmt] * c.scales[pg, h // G, pl // 16, 1].double())).amax(-1) * seen.sum(-1)
    return o, lse, mag, size, top


def limits(w, dtype):
    """How far o and lse may be off.  A score's error is that of fp32 products and of q's 22 bits, some
    2^-21 of the sum of its terms' magnitudes (`size`, nats), and moves p by as much; p is rounded to 11
    bits (bfloat16 outputs) or 22; fp32 sums over a few hundred steps add 2^-14 of the magnitudes; the output
    is rounded once.  Far below the largest probability of a row, p has the last place of float16 and not
    its 11 bits: numbers under 2^-14 are multiples of 2^-24, rounded by 2^-25 at most, and p is kept as 32 p
    (times a value scale over at most the largest), so each token may be off by 2^-25 / 32 = 2^-30 of the
    largest value (the sum they are divided by is 1 at least, the largest p itself).  A value scale below 2^-100
    may count as that: codes are 448 at most."""
    o, lse, mag, size, top = w
    near = 2.0 ** -20 * (1 + size) + 2.0 ** -14
    half = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    p = {"bf16": 2.0 ** -11, "f32": 2.0 ** -21}[dtype]
    return (near + p)[..., None] * mag + half * o.abs() + 2.0 ** -30 * top[..., None] + 448 * 2.0 ** -100, near + 2.0 ** -22 * torch.where(lse.isinf(), 0.0, lse.abs())
