"""The operators over a paged cache on the GPU against their 64-bit definitions
(tests/cache_ref.py).

Tolerances, derived from the arithmetic:
 - Scores: products of 16-bit (or e4m3) values are exact in fp32; a sum of d of them
   in fp32, whatever the order, is off by at most d 2^-23 sum|q k| (a rounding or
   truncation a term); SCORE takes that bound with sum|q k| <= |q||k| from the
   data, in units of the logit, plus the roundings of the scaling (4 2^-24 |x|) and of
   ex2 (2^-22 relative).
 - o: with logits off by at most e each weight is off by a factor exp(+-2e); P
   is rounded to 16 bits (half a step, 2^-8 bf16 or 2^-11 fp16 relative, plus
   2^-25 absolute in fp16 where P is subnormal; the fp32 scale of an e4m3 V adds
   4 2^-24), all relative to sum w|V|; then the output rounding of half a step.
 - lse: off by at most e, plus 2^-22 (|lse| + 1) for the fp32 sum and logarithm.
 - weights: a factor exp(+-e) on each, and the fp32 sum of R terms (R 2^-24).
"""
import math

import numpy as np
import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qa():
    from quantized_attention_04_b200 import build
    build.build()
    import quantized_attention_04_b200 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.lib()
    assert m.sage2_check_device_error() == 0
    return m


def logit_error(c):
    """Bound on |logit - exact| over the case."""
    qn = c.q.double().norm(dim=-1).max().item()
    kn = max(c.dense("k", b, h, c.lens[b] + c.n[b]).norm(dim=-1).max().item()
             for b in range(c.B) for h in range(c.Hkv) if c.lens[b] + c.n[b])
    x = qn * kn * c.sm
    return x * (c.d * 2.0 ** -23 + 4 * 2.0 ** -24) + 2.0 ** -22


def check_tree(c, o, lse, want, odt):
    wo, wl, mag = want
    e = logit_error(c)
    p16 = 2.0 ** -8 if c.dtype == torch.bfloat16 and c.kv != "e4m3" else 2.0 ** -11
    out = 0.0 if odt == torch.float32 else torch.finfo(odt).eps / 2
    keys = max(x + y for x, y in zip(c.lens, c.n))
    vmax = max([c.dense("v", b, h, c.lens[b] + c.n[b]).abs().max().item()
                for b in range(c.B) for h in range(c.Hkv) if c.lens[b] + c.n[b]] + [0.0])
    rel = math.expm1(2 * e) + p16 + 4 * 2.0 ** -24 + keys * 2.0 ** -24
    sub = 0.0 if p16 == 2.0 ** -8 else 2.0 ** -25 * keys * vmax
    tol = rel * mag + sub
    tol = tol + out * (wo.abs() + tol) + 1e-30
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all()
    bad = (o - wo).abs() > tol
    assert not bad.any(), ("o", bad.nonzero()[:5].tolist(), ((o - wo).abs() / tol).max().item())
    none = wl == -math.inf
    assert torch.equal(lse == -math.inf, none)
    assert (o[none] == 0).all()
    ltol = e + 2.0 ** -22 * (wl[~none].abs() + 1) + keys * 2.0 ** -24
    assert ((lse[~none] - wl[~none]).abs() <= ltol).all(), (lse[~none] - wl[~none]).abs().max()


# (lens, T, Hkv, G, d, page, dtype, kv, n)
TREE = [
    ([1], 1, 1, 1, 128, 16, "bf16", "same", None),
    ([0], 1, 2, 1, 64, 16, "fp16", "same", None),
    ([0, 5, 16, 17], 1, 2, 4, 128, 16, "fp16", "same", None),
    ([63, 64, 65, 0], 1, 1, 8, 128, 32, "bf16", "e4m3", None),
    ([130, 1, 700], 3, 2, 4, 128, 16, "bf16", "same", [3, 0, 2]),
    ([33, 257], 5, 1, 3, 64, 64, "fp16", "e4m3", [5, 1]),
    ([500, 77], 4, 2, 5, 128, 128, "bf16", "same", None),
    ([200, 31, 90], 7, 2, 4, 64, 16, "bf16", "e4m3", [7, 3, 6]),
    ([1000], 16, 1, 2, 128, 32, "fp16", "e4m3", None),
    ([129, 640], 17, 2, 2, 128, 64, "bf16", "same", [17, 9]),
    ([411], 61, 1, 4, 128, 32, "bf16", "same", None),
    ([300, 0], 64, 1, 4, 128, 64, "bf16", "e4m3", [64, 33]),
    ([150], 40, 2, 7, 64, 16, "fp16", "same", None),
    ([77, 300], 33, 1, 8, 64, 128, "bf16", "e4m3", [33, 33]),
    ([900, 10], 100, 1, 1, 128, 16, "fp16", "same", [100, 70]),
    ([2500], 1, 1, 1, 128, 16, "bf16", "e4m3", None),
    ([1, 0, 2, 127, 128, 129, 255, 60], 20, 2, 2, 128, 16, "bf16", "same", [20, 0, 1, 7, 20, 3, 2, 11]),
    ([3, 0, 90, 127, 128, 130, 255, 64], 30, 3, 5, 64, 32, "fp16", "e4m3", [30, 20, 0, 1, 30, 5, 12, 30]),
    ([1, 70, 0, 300], 33, 5, 1, 128, 16, "fp16", "e4m3", [33, 1, 0, 20]),
    ([40, 700], 200, 1, 2, 64, 64, "bf16", "same", [200, 77]),
    ([0], 1024, 1, 1, 64, 128, "fp16", "same", None),
]
ids = lambda c: "-".join(str(x) for x in c[1:8])


@pytest.mark.parametrize("case", TREE, ids=map(ids, TREE))
@pytest.mark.parametrize("masked", [True, False])
def test_tree(qa, case, masked):
    lens, T, Hkv, G, d, page, dtype, kv, n = case
    c = R.Case(7, lens, T, Hkv, G, d, page, dtype, kv, n)
    x = c.cuda()
    if not masked:
        x["mask"] = None
    want = R.attend(c, True if masked else None)
    for odt in (c.dtype, torch.float32):
        o, lse = qa.sage2_attn_tree(out_dtype=odt, **x)
        assert qa.sage2_check_device_error() == 0
        check_tree(c, o, lse, want, odt)


def attend_gpu(c, x):
    """(o, lse, mag) as cache_ref.attend gives them, in 64 bits with torch on the GPU."""
    B, Hq = c.B, c.Hkv * c.G
    o = torch.zeros(B, Hq, c.T, c.d, dtype=torch.float64, device="cuda")
    lse, mag = torch.full((B, Hq, c.T), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros_like(o)
    for b in range(B):
        ln, n = c.lens[b], c.n[b]
        bar = torch.zeros(n, ln + n, dtype=torch.float64, device="cuda")
        bar[:, ln:][~x["mask"][b, :n, :n]] = -math.inf
        for h in range(c.Hkv):
            K, V = (c.dense(w, b, h, ln + n).cuda() for w in "kv")
            for g in range(c.G):
                s = x["q"][b, h * c.G + g, :n].double() @ K.T * c.sm + bar
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - z[:, None])
                o[b, h * c.G + g, :n], mag[b, h * c.G + g, :n] = w @ V, w @ V.abs()
                lse[b, h * c.G + g, :n] = z
    return o.cpu(), lse.cpu(), mag.cpu()


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("T, G, d, dtype", [(1, 1, 128, "bf16"), (3, 7, 64, "fp16"), (9, 4, 128, "fp16"),
                                            (33, 3, 64, "bf16"), (48, 4, 128, "bf16"), (64, 8, 64, "fp16")])
def test_tree_long_runs(qa, T, G, d, dtype, kv):
    """Enough keys that every block walks many tiles and crosses from one sequence's to the next's."""
    lens = [9000, 1, 3333, 6400, 0, 777, 8191, 2048, 5, 4095]
    c = R.Case(17, lens, T, 4, G, d, 64, dtype, kv, [T - (b % T) // 2 for b in range(len(lens))], junk=False)
    x = c.cuda()
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    check_tree(c, o, lse, attend_gpu(c, x), torch.float32)
    o2, lse2 = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("T, G, d", [(5, 3, 128), (7, 4, 64), (40, 2, 128), (40, 4, 64), (33, 6, 128)])
def test_not_finite_in_masked_places(qa, T, G, d, kv):
    """An infinity or NaN in a drafted token's K or V reaches the tokens that attend it, no others."""
    c = R.Case(13, [150, 3], T, 1, G, d, 32, "bf16", kv)
    clean = R.attend(c)
    x = c.cuda()
    hit = torch.zeros(2, T, dtype=torch.bool)
    for b, j, name in ((0, 2, "v"), (0, 4, "k"), (1, 1, "v"), (1, 3, "k"), (1, 4, "v")):
        s = c.lens[b] + j
        p, r = int(c.table[b, s // 32]), s % 32
        if kv == "e4m3" and j != 2:
            x["cache"][name + "_scale"][p, 0, r] = math.nan
        elif kv == "e4m3":
            x["cache"][name].view(torch.uint8)[p, 0, r, 5] = 0xff
        else:
            x["cache"][name][p, 0, r, 3] = math.inf if name == "v" and b else math.nan
        hit[b] |= c.mask[b, :, j]
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    assert 0 < hit.sum() < hit.numel()
    at = hit[:, None].expand(2, G, T)
    assert torch.isnan(o.cpu()[at]).all()
    o[at.cuda()], lse[at.cuda()] = clean[0][at].float().cuda(), clean[1][at].float().cuda()
    check_tree(c, o, lse, clean, torch.float32)


@pytest.mark.parametrize("case", TREE, ids=map(ids, TREE))
def test_weights(qa, case):
    lens, T, Hkv, G, d, page, dtype, kv, n = case
    c = R.Case(8, lens, T, Hkv, G, d, page, dtype, kv, n)
    x = c.cuda()
    _, lse, _ = R.attend(c)
    lse = lse.float()
    want = R.weights(c, lse)
    acc = torch.full((c.B, Hkv, c.MP * page + 3), 0.5, device="cuda")
    got = qa.sage2_cache_weights(x["q"], lse.cuda(), x["cache"], x["table"], x["lens"], acc,
                                 mask=x["mask"], n=x["n"])
    assert got is acc and qa.sage2_check_device_error() == 0
    got = acc.double().cpu()
    assert (got[:, :, c.MP * page:] == 0.5).all()
    got = got[:, :, :c.MP * page]
    e = logit_error(c) + 2.0 ** -22 * (lse[lse > -math.inf].abs().max().item() + 1 if (lse > -math.inf).any() else 1)
    tol = want * (math.expm1(e) + (G * T + 4) * 2.0 ** -24) + 2.0 ** -24 * (want + 0.5)
    assert ((got - 0.5 - want).abs() <= tol).all(), ((got - 0.5 - want).abs() / (tol + 1e-30)).max()
    # slots that nothing attends keep their value bit for bit
    assert (got[want == 0] == 0.5).all()


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("T, G, d, dtype", [(1, 1, 128, "bf16"), (9, 4, 64, "fp16"), (48, 4, 128, "bf16"),
                                            (64, 8, 64, "bf16"), (37, 7, 128, "fp16")])
def test_weights_long_runs(qa, T, G, d, dtype, kv):
    """Many tiles a block, pieces that end inside a block's run, more rows than one unit holds; each
    weight in 64 bits on the GPU."""
    lens = [9000, 1, 3333, 0, 777, 8191]
    c = R.Case(18, lens, T, 3, G, d, 16, dtype, kv, [T - (b % T) // 2 for b in range(len(lens))], junk=False)
    x = c.cuda()
    lse = attend_gpu(c, x)[1].float()
    acc = torch.full((c.B, 3, c.MP * 16), 0.25, device="cuda")
    qa.sage2_cache_weights(x["q"], lse.cuda(), x["cache"], x["table"], x["lens"], acc, mask=x["mask"], n=x["n"])
    assert qa.sage2_check_device_error() == 0
    want = torch.zeros(acc.shape, dtype=torch.float64, device="cuda")
    for b in range(c.B):
        ln, n = c.lens[b], c.n[b]
        bar = torch.zeros(n, ln + n, dtype=torch.float64, device="cuda")
        bar[:, ln:][~x["mask"][b, :n, :n]] = -math.inf
        for h in range(3):
            K = c.dense("k", b, h, ln + n).cuda()
            for g in range(G):
                s = x["q"][b, h * G + g, :n].double() @ K.T * c.sm + bar
                want[b, h, :ln + n] += torch.exp(s - lse[b, h * G + g, :n, None].double().cuda()).sum(0)
    e = logit_error(c) + 2.0 ** -22 * (lse[lse > -math.inf].abs().max().item() + 1)
    tol = want * (math.expm1(e) + (G * T + 4) * 2.0 ** -24) + 2.0 ** -24 * (want + 0.25)
    assert ((acc.double() - 0.25 - want).abs() <= tol).all(), ((acc.double() - 0.25 - want).abs() / tol).max()


def pools_after_append(c, k, v):
    """The pools after writing k, v [B, Hkv, T, d] behind lens, by the definition."""
    out = {n: t.clone() for n, t in c.pool.items()}
    for b in range(c.B):
        for t in range(c.n[b]):
            s = c.lens[b] + t
            p, r = int(c.table[b, s // c.page]), s % c.page
            for name, x in (("k", k), ("v", v)):
                if c.kv == "e4m3":
                    code, out[name + "_scale"][p, :, r] = R.codes(x[b, :, t])
                    out[name].view(torch.uint8)[p, :, r] = code.view(torch.uint8)
                else:
                    out[name][p, :, r] = x[b, :, t]
    return out


def same_bits(a, b):
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.cpu().contiguous().view(raw), b.cpu().contiguous().view(raw))


@pytest.mark.parametrize("case", TREE, ids=map(ids, TREE))
@pytest.mark.parametrize("strided", [False, True])
def test_append(qa, case, strided):
    lens, T, Hkv, G, d, page, dtype, kv, n = case
    c = R.Case(9, lens, T, Hkv, G, d, page, dtype, kv, n)
    x = c.cuda()
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(c.B, Hkv, T, d, generator=g).to(c.dtype) * 3 for _ in range(2))
    if kv == "e4m3":
        k[0, 0, 0] = 0                          # a row of zeros
        v[0, 0, 0, 1:] = 0                      # a row of one value
        k[-1, -1, -1] *= 2.0 ** -9
    want = pools_after_append(c, k, v)
    kd, vd = k.cuda(), v.cuda()
    if strided:                                 # [B, T, Hkv, 2, d]: what a fused projection returns
        both = torch.stack([kd, vd], 3).transpose(1, 2).contiguous()
        kd, vd = both[:, :, :, 0].transpose(1, 2), both[:, :, :, 1].transpose(1, 2)
    qa.sage2_cache_append(kd, vd, x["cache"], x["table"], x["lens"], n=x["n"])
    assert qa.sage2_check_device_error() == 0
    for name, t in want.items():
        assert same_bits(x["cache"][name], t), name


def test_append_rows_that_are_not_finite(qa):
    """Zero below 2^-100, NaN scale for a row with an infinity or NaN, the other rows untouched."""
    c = R.Case(1, [4], 6, 1, 1, 128, 16, "bf16", "e4m3")
    x = c.cuda()
    k = torch.ones(1, 1, 6, 128, dtype=torch.bfloat16)
    k[0, 0, 1, 5], k[0, 0, 2, 127], k[0, 0, 3, 0] = math.inf, math.nan, -math.inf
    k[0, 0, 4] = 2.0 ** -101
    qa.sage2_cache_append(k.cuda(), k.cuda(), x["cache"], x["table"], x["lens"])
    p = int(c.table[0, 0])
    for name in "kv":
        s = x["cache"][name + "_scale"][p, 0, 4:10].cpu()
        assert torch.isnan(s[1:4]).all() and s[4] == 0
        assert s[0] == s[5] == torch.tensor(1.0) / 448
        codes = x["cache"][name].view(torch.uint8)[p, 0, 4:10].cpu()
        assert (codes[4] == 0).all() and (codes[0] == 0x7e).all() and (codes[5] == 0x7e).all()


def pools_after_move(pool, table, out_table, page, idx, count, base):
    out = {n: t.clone() for n, t in pool.items()}
    for b in range(table.shape[0]):
        for h in range(idx.shape[1]):
            for i in range(count[b]):
                s, t = int(idx[b, h, i]), base[b] + i
                sp, sr, dp, dr = int(table[b, s // page]), s % page, int(out_table[b, t // page]), t % page
                for name in pool:
                    raw = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                    raw(out[name])[dp, h, dr] = raw(pool[name])[sp, h, sr]
    return out


MOVE = [([300, 40, 1], 2, 128, 16, "bf16", "same"), ([700, 513], 3, 64, 64, "fp16", "e4m3"),
        ([1500], 1, 64, 32, "fp16", "same"), ([260, 999], 2, 128, 128, "bf16", "e4m3")]


@pytest.mark.parametrize("case", MOVE, ids=lambda c: f"{c[2]}-{c[3]}-{c[5]}")
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(qa, case, in_place):
    lens, Hkv, d, page, dtype, kv = case
    c = R.Case(5, lens, 1, Hkv, 1, d, page, dtype, kv, junk=False)
    x = c.cuda()
    g = torch.Generator().manual_seed(4)
    S = c.MP * page
    acc = torch.rand(c.B, Hkv, S, generator=g)
    acc[:, :, ::3] = 0.25                       # many equal ones
    acc[0, 0, 5:9] = torch.tensor([math.inf, math.nan, 0.0, -0.0])
    for keep, sinks, recent in ((256, 4, 31), (37, 0, 0), (64, 32, 32), (64, 64, 0), (1, 0, 1), (2000, 1, 1)):
        keep = min(keep, c.MP * page)
        sinks, recent = min(sinks, keep), min(recent, keep)
        x = c.cuda()
        out_table, pool, ot = None, dict(c.pool), c.table
        if not in_place:                        # pages behind the ones of the sequences
            MO = -(-keep // page)
            pool = {n: torch.cat([(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t),
                                  torch.zeros(c.B * MO, *t.shape[1:], dtype=t.dtype).view(
                                      torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype)]).view(t.dtype)
                    for n, t in c.pool.items()}
            ot = (c.pages + torch.arange(c.B * MO, dtype=torch.int32)).view(c.B, MO)
            out_table = ot.cuda()
        cache = {n: t.cuda() for n, t in pool.items()}
        idx, new, kept = qa.sage2_cache_evict(cache, x["table"], x["lens"], acc.cuda(), keep, sinks,
                                              recent, out_table=out_table)
        assert qa.sage2_check_device_error() == 0
        count = [min(keep, l) for l in lens]
        assert new.tolist() == count
        want = torch.full((c.B, Hkv, keep), -1, dtype=torch.int32)
        wacc = torch.zeros(c.B, Hkv, keep)
        for b in range(c.B):
            for h in range(Hkv):
                got = torch.tensor(R.choose(acc[b, h], lens[b], keep, sinks, recent))
                want[b, h, :count[b]], wacc[b, h, :count[b]] = got, acc[b, h, got]
        assert torch.equal(idx.cpu(), want)
        assert same_bits(kept, wacc)
        after = pools_after_move(pool, c.table, ot, page, want, count, [0] * c.B)
        for name, t in after.items():
            assert same_bits(cache[name], t), (name, keep, sinks, recent)


@pytest.mark.parametrize("case", MOVE, ids=lambda c: f"{c[2]}-{c[3]}-{c[5]}")
def test_compact_path_in_place(qa, case):
    """An accepted path of a tree moves behind the context, the same for all heads."""
    lens, Hkv, d, page, dtype, kv = case
    T = 30
    c = R.Case(6, lens, T, Hkv, 1, d, page, dtype, kv, junk=False)
    x = c.cuda()
    path = torch.tensor([0, 1, 4, 5, 11, 29])
    count = [(6, 3, 0)[b % 3] for b in range(c.B)]
    idx = torch.stack([path + l for l in lens]).to(torch.int32)[:, None].expand(c.B, Hkv, 6)
    want = pools_after_move(c.pool, c.table, c.table, page, idx, count, lens)
    S = c.MP * page
    acc = torch.rand(c.B, Hkv, S)
    wacc = acc.clone()
    for b in range(c.B):
        for i in range(count[b]):
            wacc[b, :, lens[b] + i] = acc[b, :, lens[b] + path[i]]
    accd = acc.cuda()
    qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda(), torch.tensor(count, dtype=torch.int32).cuda(),
                           base=x["lens"], acc=accd)
    assert qa.sage2_check_device_error() == 0
    for name, t in want.items():
        assert same_bits(x["cache"][name], t), name
    assert same_bits(accd, wacc)


def test_compact_repeats_in_place(qa):
    """In place a row may be taken more than once, in any order that moves towards the front."""
    c = R.Case(6, [900], 1, 2, 1, 128, 16, "bf16", "e4m3", junk=False)
    x = c.cuda()
    g = torch.Generator().manual_seed(1)
    i = torch.arange(700)
    idx = torch.stack([i + (torch.rand(700, generator=g) * (900 - i)).long() for _ in range(2)])[None]
    idx = idx.to(torch.int32)
    want = pools_after_move(c.pool, c.table, c.table, 16, idx, [700], [0])
    qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda())
    assert qa.sage2_check_device_error() == 0
    for name, t in want.items():
        assert same_bits(x["cache"][name], t), name


def test_serving_run(qa):
    """The operators together: prompt, tree, accepted path, tally and eviction, then a decode step,
    in both cache types, against the same steps on the host."""
    for kv in ("same", "e4m3"):
        lens, T, Hkv, G, d, page = [70, 41], 6, 2, 2, 64, 16
        c = R.Case(11, lens, T, Hkv, G, d, page, "bf16", kv, extra=2)
        x = c.cuda()
        g = torch.Generator().manual_seed(2)
        table, cache = x["table"], x["cache"]
        # prompt (the shorter one padded), then the tree's tokens
        P = max(lens)
        k, v = (torch.randn(2, Hkv, P, d, generator=g).to(c.dtype) for _ in range(2))
        zero = torch.zeros(2, dtype=torch.int32, device="cuda")
        qa.sage2_cache_append(k.cuda(), v.cuda(), cache, table, zero, n=x["lens"])
        kt, vt = (torch.randn(2, Hkv, T, d, generator=g).to(c.dtype) for _ in range(2))
        qa.sage2_cache_append(kt.cuda(), vt.cuda(), cache, table, x["lens"])
        c.pool = {n: t.cpu() for n, t in cache.items()}
        ref = {"k": [torch.cat([k[b, :, :lens[b]], kt[b]], 1) for b in range(2)]}
        if kv == "same":
            for b in range(2):
                assert torch.equal(c.dense("k", b, 1, lens[b] + T), ref["k"][b][1].double())
        o, lse = qa.sage2_attn_tree(x["q"], cache, table, x["lens"], mask=x["mask"])
        check_tree(c, o, lse, R.attend(c), c.dtype)
        acc = torch.zeros(2, Hkv, c.MP * page, device="cuda")
        qa.sage2_cache_weights(x["q"], lse, cache, table, x["lens"], acc, mask=x["mask"])
        # every attended weight is in the tally: G*T rows a head, each of weight 1
        # (lse and the weight are each off by the error of a logit, the sums by 2^-24 a term)
        total = acc.double().sum(-1).cpu()
        rel = math.expm1(2 * logit_error(c)) + (G * T + max(lens) + T) * 2.0 ** -23
        assert (total - G * T).abs().max() <= G * T * rel
        path = torch.tensor([[0, 3, 5], [0, 1, 2]], dtype=torch.int32)
        took = torch.tensor([3, 2], dtype=torch.int32)
        idx = (path + torch.tensor(lens, dtype=torch.int32)[:, None])[:, None].expand(2, Hkv, 3)
        qa.sage2_cache_compact(cache, table, idx.cuda(), took.cuda(), base=x["lens"], acc=acc)
        now = x["lens"] + took.cuda()
        idx, new, _ = qa.sage2_cache_evict(cache, table, now, acc, 48, sinks=2, recent=8, acc_out=acc)
        assert new.tolist() == [48, 43]
        # one more token
        k1, v1 = (torch.randn(2, Hkv, 1, d, generator=g).to(c.dtype) for _ in range(2))
        qa.sage2_cache_append(k1.cuda(), v1.cuda(), cache, table, new)
        c2 = R.Case(12, [48, 43], 1, Hkv, G, d, page, "bf16", kv, junk=False)
        c2.pool, c2.table = {n: t.cpu() for n, t in cache.items()}, c.table
        o, lse = qa.sage2_attn_tree(c2.q.cuda(), cache, table, new)
        assert qa.sage2_check_device_error() == 0
        check_tree(c2, o, lse, R.attend(c2), c2.dtype)


def bad_index(qa):
    from quantized_attention_04_b200 import Sage2Error
    status = qa.sage2_check_device_error()
    assert qa.sage2_check_device_error() == 0        # reading clears it
    return status == 8


@pytest.mark.parametrize("T, G", [(3, 2), (40, 4)])
@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_device_integers_out_of_range(qa, T, G, kv):
    """Lengths, counts, pages and indices out of range set the error word; the sequences beside them and all
    rows that nothing names keep what they hold."""
    c = R.Case(19, [100, 37], T, 2, G, 64, 16, "bf16", kv, junk=False)
    want = R.attend(c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cap = c.MP * 16
    for what, v in (("lens", [cap - T + 1, 37]), ("lens", [-1, 37]), ("lens", [2 ** 31 - 1, 37]), ("n", [T + 1, T]),
                    ("n", [-5, T]), ("page", c.pages), ("page", -1), ("page", 2 ** 31 - 1)):
        x = c.cuda()
        if what == "page":
            x["table"][0, 1] = v
        else:
            x[what] = i32(v)
        before = {n: t.clone() for n, t in x["cache"].items()}
        o, lse = qa.sage2_attn_tree(**x)
        assert bad_index(qa), (what, v)
        acc = torch.ones(2, 2, cap, device="cuda")
        qa.sage2_cache_weights(x["q"], want[1].float().cuda(), x["cache"], x["table"], x["lens"], acc,
                               mask=x["mask"], n=x["n"])
        assert bad_index(qa), (what, v)
        for n, t in x["cache"].items():
            assert same_bits(t, before[n])
        one = type(c)(19, [37], T, 2, G, 64, 16, "bf16", kv, junk=False)
        one.pool, one.table, one.q, one.mask, one.MP = c.pool, c.table[1:], c.q[1:], c.mask[1:], c.MP
        check_tree(one, o[1:], lse[1:], tuple(w[1:] for w in want), c.dtype)
        k = torch.ones(2, 2, T, 64, dtype=c.dtype, device="cuda")
        other = set(range(c.pages)) - set(c.table.flatten().tolist())
        qa.sage2_cache_append(k, k, x["cache"], x["table"], x["lens"], n=x["n"])
        if what != "page" or v == c.pages:
            bad_index(qa)                            # only if a row of the bad page is written
        for n, t in x["cache"].items():
            for p in other:
                assert same_bits(t[p], before[n][p])
    x = c.cuda()
    before = {n: t.clone() for n, t in x["cache"].items()}
    idx = torch.tensor([3, 0, 200000, -1], dtype=torch.int32, device="cuda").expand(2, 2, 4).contiguous()
    qa.sage2_cache_compact(x["cache"], x["table"], idx)   # slot 1 from slot 0 would move back
    assert bad_index(qa)
    after = pools_after_move(c.pool, c.table, c.table, 16, torch.full((2, 2, 1), 3), [1, 1], [0, 0])
    for n, t in x["cache"].items():
        assert same_bits(t, after[n]), n


def test_refusals(qa):
    c = R.Case(20, [40], 3, 2, 2, 64, 16, "bf16", "same")
    x = c.cuda()
    q, cache, table, lens, mask = x["q"], x["cache"], x["table"], x["lens"], x["mask"]
    acc = torch.zeros(1, 2, 64, device="cuda")
    err = (ValueError, qa.Sage2Error)
    with pytest.raises(err):
        qa.sage2_attn_tree(q.float(), cache, table, lens)
    with pytest.raises(err):
        qa.sage2_attn_tree(q.half(), cache, table, lens)                 # a 16-bit cache takes its own type
    with pytest.raises(err):
        qa.sage2_attn_tree(q[:, :3], cache, table, lens)                 # heads no multiple of the cache's
    with pytest.raises(err):
        qa.sage2_attn_tree(q, cache, table.long(), lens)
    with pytest.raises(err):
        qa.sage2_attn_tree(q, cache, table, lens.cpu())
    with pytest.raises(err):
        qa.sage2_attn_tree(q, cache, table, lens, mask=mask[:, :2])
    with pytest.raises(err):
        qa.sage2_attn_tree(q, cache, table, lens, sm_scale=-1.0)
    with pytest.raises(err):
        qa.sage2_attn_tree(q, {"k": cache["k"], "v": cache["v"].transpose(1, 2)}, table, lens)
    with pytest.raises(err):
        qa.sage2_attn_tree(q.transpose(2, 3), cache, table, lens)
    with pytest.raises(err):
        qa.sage2_cache_weights(q, torch.zeros(1, 4, 2, device="cuda"), cache, table, lens, acc)
    with pytest.raises(err):
        qa.sage2_cache_weights(q, torch.zeros(1, 4, 3, device="cuda"), cache, table, lens, acc.double())
    with pytest.raises(err):
        qa.sage2_cache_evict(cache, table, lens, acc, 8, sinks=5, recent=4)
    with pytest.raises(err):
        qa.sage2_cache_evict(cache, table, lens, acc, 8, out_table=table.clone(), acc_out=acc)
    with pytest.raises(err):
        qa.sage2_cache_compact(cache, table, torch.zeros(1, 3, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(err):
        qa.sage2_cache_append(q[:, :2], q[:, :2], cache, table, lens, n=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert qa.sage2_check_device_error() == 0


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_streams_and_graphs(qa, kv):
    """The calls on another stream than the default one, and captured: two graphs replayed at the same
    time on two streams give what eager calls give."""
    cs = [R.Case(s, [700, 90, 0], T, 2, 4, 128, 32, "bf16", kv, junk=False) for s, T in ((21, 2), (22, 30))]
    want = []
    for c in cs:
        x = c.cuda()
        o, lse = qa.sage2_attn_tree(**x)
        acc = torch.zeros(3, 2, c.MP * 32, device="cuda")
        qa.sage2_cache_weights(x["q"], lse, x["cache"], x["table"], x["lens"], acc, mask=x["mask"], n=x["n"])
        idx, new, kept = qa.sage2_cache_evict(x["cache"], x["table"], x["lens"], acc, 64, 2, 8)
        want.append([o, lse, acc, idx, new, kept, *x["cache"].values()])
    torch.cuda.synchronize()
    runs = []
    for c in cs:
        x = c.cuda()
        start = {n: t.clone() for n, t in x["cache"].items()}
        acc, kept = torch.zeros(3, 2, c.MP * 32, device="cuda"), torch.zeros(3, 2, 64, device="cuda")
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            for n, t in x["cache"].items():
                t.view(torch.uint8).copy_(start[n].view(torch.uint8))
            acc.zero_()
            kept.zero_()
            o, lse = qa.sage2_attn_tree(**x)
            qa.sage2_cache_weights(x["q"], lse, x["cache"], x["table"], x["lens"], acc, mask=x["mask"], n=x["n"])
            idx, new, _ = qa.sage2_cache_evict(x["cache"], x["table"], x["lens"], acc, 64, 2, 8, acc_out=kept)
        # x and start stay alive: the graph reads them
        runs.append((st, g, [o, lse, acc, idx, new, kept, *x["cache"].values()], x, start))
    for _ in range(3):
        for st, g, *_ in runs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, got, *_), w in zip(runs, want):
            for a, b in zip(got, w):
                assert same_bits(a, b)
    assert qa.sage2_check_device_error() == 0
    # eager, on a stream of its own, while the graphs live
    c, w = cs[1], want[1]
    st = torch.cuda.Stream()
    x = c.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        o, lse = qa.sage2_attn_tree(**x)
    st.synchronize()
    assert same_bits(o, w[0]) and same_bits(lse, w[1])


@pytest.mark.parametrize("T, G", [(1, 4), (20, 4), (50, 4)])
def test_strided_queries_and_masks(qa, T, G):
    """q as a fused projection lays it out, one mask for all, a mask per sequence apart, out and lse given."""
    c = R.Case(23, [300, 41], T, 2, G, 64, 16, "fp16", "e4m3")
    c.mask[1] = c.mask[0]
    x = c.cuda()
    want = R.attend(c)
    wide = torch.zeros(2, T, 2 * G, 3, 64, dtype=c.dtype, device="cuda")
    wide[:, :, :, 1] = x["q"].transpose(1, 2)
    x["q"] = wide[:, :, :, 1].transpose(1, 2)
    far = torch.zeros(2, 3, T, T, dtype=torch.bool, device="cuda")
    far[:, 1] = x["mask"]
    for mask in (x["mask"][0].clone(), far[:, 1]):
        x["mask"] = mask
        out, lse = torch.empty(2, 2 * G, T, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 2 * G, T, device="cuda")
        o, l = qa.sage2_attn_tree(out=out, lse=lse, **x)
        assert o is out and l is lse and qa.sage2_check_device_error() == 0
        check_tree(c, o, l, want, torch.bfloat16)


def test_pools_past_32_bits(qa):
    """Rows whose offset in the pools passes 2^32 bytes (and 2^31 values)."""
    pages, Hkv, page, d = 70000, 8, 64, 128                   # 4.6 GB each of k and v
    cache = qa.sage2_cache_alloc(pages, Hkv, page, d, torch.float8_e4m3fn)
    near = qa.sage2_cache_alloc(8, Hkv, page, d, torch.float8_e4m3fn)
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn(1, Hkv, 200, d, device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(1, 4 * Hkv, 40, d, device="cuda", generator=g, dtype=torch.bfloat16)
    far = torch.arange(pages - 4, pages, dtype=torch.int32, device="cuda")[None]
    tables = (far, torch.arange(4, dtype=torch.int32, device="cuda")[None])
    zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 160, dtype=torch.int32, device="cuda")
    got = []
    for c, t in ((cache, tables[0]), (near, tables[1])):
        qa.sage2_cache_append(k, v, c, t, zero)
        res = [qa.sage2_attn_tree(q[:, :, :T].contiguous(), c, t, lens) for T in (1, 8, 20, 40)]
        acc = torch.zeros(1, Hkv, 256, device="cuda")
        qa.sage2_cache_weights(q, res[-1][1], c, t, lens, acc)
        idx, new, kept = qa.sage2_cache_evict(c, t, lens, acc, 70, 1, 5)
        rows = [x[t[0].long()].contiguous() for x in (c["k"].view(torch.uint8), c["v"].view(torch.uint8), c["k_scale"])]
        got.append([*(y for r in res for y in r), acc, idx, kept, *rows])
    assert qa.sage2_check_device_error() == 0
    for a, b in zip(*got):
        assert same_bits(a, b)


@pytest.mark.parametrize("S", [53999, 54001, 80000])
def test_evict_long_tallies(qa, S):
    """Tallies on both sides of what the choice holds in shared memory, with many equal ones."""
    c = R.Case(24, [S, 30000], 1, 2, 1, 64, 128, "bf16", "e4m3", junk=False)
    x = c.cuda()
    g = torch.Generator().manual_seed(6)
    S = c.MP * 128
    acc = (torch.rand(2, 2, S, generator=g) * 500).floor() / 64
    keep, sinks, recent = 5001, 3, 77
    out_table = torch.arange(c.B * 40, dtype=torch.int32).view(2, 40) + c.pages
    cache = {n: torch.cat([t.view(torch.uint8), torch.zeros(c.B * 40, *t.shape[1:], dtype=torch.uint8)]).view(t.dtype).cuda()
             if t.dtype == torch.float8_e4m3fn else torch.cat([t, torch.zeros(c.B * 40, *t.shape[1:])]).cuda()
             for n, t in c.pool.items()}
    idx, new, kept = qa.sage2_cache_evict(cache, x["table"], x["lens"], acc.cuda(), keep, sinks, recent,
                                          out_table=out_table.cuda())
    assert qa.sage2_check_device_error() == 0 and new.tolist() == [keep, keep]
    for b in range(2):
        ln = c.lens[b]
        for h in range(2):
            mid = np.arange(sinks, ln - recent)
            best = mid[np.lexsort((mid, -acc[b, h, mid].double().numpy()))[:keep - sinks - recent]]
            want = np.sort(np.concatenate([np.arange(sinks), best, np.arange(ln - recent, ln)]))
            assert (idx[b, h].cpu().numpy() == want).all()
            assert torch.equal(kept[b, h].cpu(), acc[b, h, torch.from_numpy(want)])
            at = torch.from_numpy(want)
            src = c.pool["k"].view(torch.uint8)[c.table[b].long()[at // 128], h, at % 128]
            i = torch.arange(keep)
            assert torch.equal(cache["k"].view(torch.uint8).cpu()[out_table[b].long()[i // 128], h, i % 128], src)


@pytest.mark.parametrize("kv, d", [("same", 128), ("e4m3", 128), ("e4m3", 64)])
def test_compact_in_place_many_heads(qa, kv, d):
    """So many heads that a block walks whole rows; indices with repeats and rows that stay."""
    c = R.Case(25, [200 - b for b in range(30)], 1, 6, 1, d, 16, "bf16", kv, junk=False)
    x = c.cuda()
    g = torch.Generator().manual_seed(7)
    M = 150
    i = torch.arange(M)
    idx = (i + (torch.rand(30, 6, M, generator=g) ** 4 * (170 - i).clamp(min=0)).long()).to(torch.int32)
    count = [(M, 0, 1, 77)[b % 4] for b in range(30)]
    acc = torch.rand(30, 6, c.MP * 16, generator=g)
    want = pools_after_move(c.pool, c.table, c.table, 16, idx, count, [0] * 30)
    wacc = acc.clone()
    for b in range(30):
        for h in range(6):
            wacc[b, h, :count[b]] = acc[b, h, idx[b, h, :count[b]].long()]
    accd = acc.cuda()
    qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda(), torch.tensor(count, dtype=torch.int32).cuda(), acc=accd)
    assert qa.sage2_check_device_error() == 0
    for name, t in want.items():
        assert same_bits(x["cache"][name], t), name
    assert same_bits(accd, wacc)
    with pytest.raises((ValueError, qa.Sage2Error)):
        qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda(), acc=acc.cuda(),
                               acc_out=torch.zeros(30, 1, 160, device="cuda").expand(30, 6, 160))
