"""Plain 64-bit implementation of the operators over a paged cache, on the host,
from their definitions (no code of the package), and the inputs of their tests."""
import math

import numpy as np
import torch

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


class Case:
    """Inputs of one test, on the CPU: pools, table, lengths, q, mask and dense views."""

    def __init__(self, seed, lens, T, Hkv, G, d, page, dtype, kv, n=None, spare=2, extra=0, scale=2.0,
                 junk=True):
        rng = np.random.default_rng(seed)
        self.lens, self.T, self.Hkv, self.G, self.d, self.page = lens, T, Hkv, G, d, page
        self.n = [T] * len(lens) if n is None else n
        self.B, self.dtype, self.kv = len(lens), DT[dtype], kv
        self.MP = max(-(-(max(l + t for l, t in zip(lens, self.n))) // page), 1) + extra
        self.pages = self.B * self.MP + spare
        self.table = torch.from_numpy(rng.permutation(self.pages)[:self.B * self.MP].astype(
            np.int32)).view(self.B, self.MP)
        shape = (self.pages, Hkv, page, d)

        def draw(*shape):
            return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32))

        off = 2 * draw(Hkv, 1, d)
        self.pool = {}
        for name, x in (("k", draw(*shape) + off), ("v", draw(*shape) + draw(Hkv, 1, d))):
            if kv == "e4m3":
                self.pool[name], self.pool[name + "_scale"] = codes(x.to(self.dtype))
            else:
                self.pool[name] = x.to(self.dtype)
        if junk:   # rows that no slot in use names hold NaN
            used = torch.zeros(self.pages, page, dtype=torch.bool)
            for b in range(self.B):
                for s in range(lens[b] + self.n[b]):
                    used[self.table[b, s // page], s % page] = True
            for name in "kv":
                raw = self.pool[name].view(torch.uint8 if kv == "e4m3" else torch.int16)
                raw.masked_fill_(~used[:, None, :, None], 0x7f if kv == "e4m3" else 0x7fff)
                if kv == "e4m3":
                    self.pool[name + "_scale"].masked_fill_(~used[:, None, :], math.nan)
        self.q = (scale * draw(self.B, Hkv * G, T, d) + draw(Hkv * G, 1, d)).to(self.dtype)
        m = np.zeros((self.B, T, T), bool)
        for b in range(self.B):
            for i in range(T):
                p = int(rng.integers(max(-1, i - 5), i)) if i else -1
                if p >= 0:
                    m[b, i] |= m[b, p]
                m[b, i, i] = True
        self.mask = torch.from_numpy(m)
        self.sm = 1.0 / math.sqrt(d)

    def cuda(self):
        self.c = {n: t.cuda() for n, t in self.pool.items()}
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        return dict(q=self.q.cuda(), cache=self.c, table=self.table.cuda(), lens=i32(self.lens),
                    n=i32(self.n), mask=self.mask.cuda())

    def dense(self, name, b, h, length):
        """Rows 0..length-1 of sequence b, head h, in 64 bits."""
        return dense(self.pool, self.table, self.page, name, b, h, length)


def codes(x):
    """e4m3 rows and scales by the definition: every fp32 operation rounded once."""
    x = x.double()
    a = x.abs().amax(-1)
    scale = torch.where(a > 0, a / 448.0, 0.0).float()
    inv = torch.where(a > 0, 448.0 / a, 0.0).float().double()
    return (x * inv[..., None]).float().to(torch.float8_e4m3fn), scale


def dense(pool, table, page, name, b, h, length):
    out = torch.zeros(length, pool[name].shape[-1], dtype=torch.float64)
    for s0 in range(0, length, page):
        p, k = int(table[b, s0 // page]), min(page, length - s0)
        x = pool[name][p, h, :k].to(torch.float64)
        if name + "_scale" in pool:
            x = x * pool[name + "_scale"][p, h, :k, None].double()
        out[s0:s0 + k] = x
    return out


def attend(c: Case, mask=True):
    """(o, lse, mag): outputs in 64 bits and, for the tolerance, sum_s w_s |V_s|."""
    B, Hq = c.B, c.Hkv * c.G
    o = torch.zeros(B, Hq, c.T, c.d, dtype=torch.float64)
    mag = torch.zeros_like(o)
    lse = torch.full((B, Hq, c.T), -math.inf, dtype=torch.float64)
    for b in range(B):
        ln, n = c.lens[b], c.n[b]
        m = c.mask[b] if mask is True else (torch.ones(c.T, c.T).tril().bool() if mask is None else mask[b])
        for h in range(c.Hkv):
            K, V = c.dense("k", b, h, ln + n), c.dense("v", b, h, ln + n)
            for g in range(c.G):
                for i in range(n):
                    at = torch.cat([torch.arange(ln), ln + torch.nonzero(m[i, :n])[:, 0]])
                    if not len(at):
                        continue
                    x = K[at] @ c.q[b, h * c.G + g, i].double() * c.sm
                    z = torch.logsumexp(x, 0)
                    w = torch.exp(x - z)
                    o[b, h * c.G + g, i] = w @ V[at]
                    mag[b, h * c.G + g, i] = w @ V[at].abs()
                    lse[b, h * c.G + g, i] = z
    return o, lse, mag


def weights(c: Case, lse, mask=True):
    """What one call adds to the tally, [B, Hkv, slots], in 64 bits."""
    acc = torch.zeros(c.B, c.Hkv, c.MP * c.page, dtype=torch.float64)
    for b in range(c.B):
        ln, n = c.lens[b], c.n[b]
        m = c.mask[b] if mask is True else torch.ones(c.T, c.T).tril().bool()
        for h in range(c.Hkv):
            K = c.dense("k", b, h, ln + n)
            for g in range(c.G):
                for i in range(n):
                    z = lse[b, h * c.G + g, i].double()
                    if z == -math.inf:
                        continue
                    at = torch.cat([torch.arange(ln), ln + torch.nonzero(m[i, :n])[:, 0]])
                    x = K[at] @ c.q[b, h * c.G + g, i].double() * c.sm
                    acc[b, h, at] += torch.exp(x - z)
    return acc


def choose(acc, ln, keep, sinks, recent):
    """The kept slots of one head, ascending."""
    if ln <= keep:
        return list(range(ln))
    mid = range(sinks, ln - recent)
    val = lambda s: -math.inf if math.isnan(acc[s]) else float(acc[s])
    best = sorted(mid, key=lambda s: (-val(s), s))[:keep - sinks - recent]
    return sorted(list(range(sinks)) + best + list(range(ln - recent, ln)))
