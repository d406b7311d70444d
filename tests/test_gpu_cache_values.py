"""Attention over a paged cache where its values are far apart: value rows of very different sizes, scores that
climb late, sums of many keys.  Against 64-bit definitions; tolerances as derived in tests/test_gpu_cache.py,
but for P's absolute rounding to fp16.  With an e4m3 cache P times a key's value scale is packed relative to the
largest such product among the keys that the row attends (at most: a reference that lags is below it), so that
each key is off by 2^-25 of that largest product, times its code of 448 at most.  With a 16-bit one P is packed
relative to the largest weight at most: a key of less than 2^-14 of it is off by 2^-25 of it, times its value.
"""
import math

import pytest
import torch

from tests import cache_ref as R
from tests.test_gpu_cache import logit_error

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


def attend(c):
    """(o, lse, mag, top): outputs in 64 bits, sum_s w_s |V_s|, and the values that P's rounding by 2^-25 meets."""
    B, Hq = c.B, c.Hkv * c.G
    o = torch.zeros(B, Hq, c.T, c.d, dtype=torch.float64)
    lse, mag = torch.full((B, Hq, c.T), -math.inf, dtype=torch.float64), torch.zeros_like(o)
    top = torch.zeros(B, Hq, c.T, dtype=torch.float64)
    for b in range(B):
        ln, n = c.lens[b], c.n[b]
        bar = torch.zeros(n, ln + n, dtype=torch.float64)
        bar[:, ln:][~c.mask[b, :n, :n]] = -math.inf
        for h in range(c.Hkv):
            K, V = (c.dense(w, b, h, ln + n) for w in "kv")
            size = V.abs().amax(-1) / 448
            for g in range(c.G):
                r = h * c.G + g
                s = c.q[b, r, :n].double() @ K.T * c.sm + bar
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - z[:, None])
                o[b, r, :n], mag[b, r, :n], lse[b, r, :n] = w @ V, w @ V.abs(), z
                if c.kv == "e4m3":
                    top[b, r, :n] = (w * size).amax(-1) * 448 * (ln + n)
                else:
                    most = w.amax(-1, keepdim=True)
                    top[b, r, :n] = ((w < most * 2.0 ** -13).double() @ V.abs().amax(-1)) * most[:, 0]
    return o, lse, mag, top


def check(c, o, lse, want):
    """o in fp32."""
    wo, wl, mag, top = want
    e = logit_error(c)
    keys = max(x + y for x, y in zip(c.lens, c.n))
    bf = c.dtype == torch.bfloat16 and c.kv != "e4m3"
    # an exponential against a reference r away is off by 2^-24 |x - r|, counted in logit_error by |x|
    rel = math.expm1(2 * e) + (2.0 ** -8 if bf else 2.0 ** -11) + 4 * 2.0 ** -24 + keys * 2.0 ** -24
    tol = rel * mag + 1e-30
    if not bf:
        tol = tol + 2.0 ** -25 * top[..., None]
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all()
    err = (o - wo).abs()
    assert (err <= tol).all(), ("o", (err > tol).nonzero()[:5].tolist(), (err / tol).max().item())
    ltol = e + 2.0 ** -22 * (wl.abs() + 1) + keys * 2.0 ** -24
    assert ((lse - wl).abs() <= ltol).all(), ("lse", (lse - wl).abs().max().item())


def cell(c, b, slot):
    return int(c.table[b, slot // c.page]), slot % c.page


# rows of a head: up to 48 one kernel, more the other (up to 128 and above)
ROWS = [(1, 1, 128), (4, 4, 64), (9, 5, 128), (50, 1, 128), (31, 4, 64), (64, 4, 128), (64, 8, 64)]


@pytest.mark.parametrize("up", [12, 20, 40, 60])
@pytest.mark.parametrize("T, G, d", ROWS)
def test_large_value_rows_that_weigh_nothing(qa, T, G, d, up):
    """A drafted token's value row of 2^up times the others' size leaves the rows that do not attend it alone,
    and a context token's counts for no more than its weight."""
    c = R.Case(31, [200, 75], T, 2, G, d, 16, "bf16", "e4m3")
    if T > 1:                                    # token 1 is attended by itself alone
        c.mask[:, :, 1] = False
        c.mask[:, 1, 1] = True
    base = torch.randn(2 * G, 1, d, generator=torch.Generator().manual_seed(5))
    c.q = (c.q + 4 * base).to(c.dtype)
    for b in range(2):
        if T > 1:
            p, r = cell(c, b, c.lens[b] + 1)
            c.pool["v_scale"][p, :, r] *= 2.0 ** up
        for slot in (3, 70):                     # keys that point away from the queries of the first head
            p, r = cell(c, b, slot)
            for h in range(2):
                far = -base[h * G, 0] / base[h * G, 0].norm() * 30
                c.pool["k"].view(torch.uint8)[p, h, r], c.pool["k_scale"][p, h, r] = (
                    x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in R.codes(far))
                c.pool["v_scale"][p, h, r] *= 2.0 ** (up - 4)
    x = c.cuda()
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    check(c, o, lse, attend(c))


@pytest.mark.parametrize("T, G, d", ROWS)
def test_infinite_value_scale_of_a_context_token(qa, T, G, d):
    """Every token attends it: o is not finite, and lse is what the keys alone make it."""
    c = R.Case(32, [100], T, 2, G, d, 16, "bf16", "e4m3")
    want = attend(c)[1]
    p, r = cell(c, 0, 40)
    c.pool["v_scale"][p, 1, r] = math.inf
    x = c.cuda()
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    assert torch.isfinite(o[:, :G]).all() and not torch.isfinite(o[:, G:]).any()
    e = logit_error(c)
    tol = e + 2.0 ** -22 * (want.abs() + 1) + (100 + T) * 2.0 ** -24
    assert ((lse.double().cpu() - want).abs() <= tol).all()


def two_levels(kv, d, page, slots, B, G, rise, v):
    """B sequences of `slots` slots (the last a drafted token) over two pages in turn: all keys of the first have
    the score 0, of the second `rise` log2 units; all values are v.  (arguments of the call, lse)"""
    dt = torch.bfloat16
    pool = {}
    for name, rows in (("k", (0.0, 1.0)), ("v", (v, v))):
        x = torch.tensor(rows, dtype=torch.float64)[:, None, None, None].expand(2, 1, page, d).to(dt)
        if kv == "e4m3":
            pool[name], pool[name + "_scale"] = R.codes(x)
        else:
            pool[name] = x.clone(memory_format=torch.contiguous_format)
    key = float(R.codes(torch.ones(1, d))[1]) * 448 if kv == "e4m3" else 1.0
    MP = slots // page
    table = (torch.arange(MP, dtype=torch.int32) % 2).expand(B, MP).contiguous().cuda()
    sm = rise * math.log(2.0) / d
    x = dict(q=torch.ones(B, G, 1, d, dtype=dt, device="cuda"), cache={n: t.cuda() for n, t in pool.items()},
             table=table, lens=torch.full((B,), slots - 1, dtype=torch.int32, device="cuda"), sm_scale=sm)
    high = (MP // 2) * page
    lse = math.log((slots - high) + high * math.exp(key * d * sm))
    return x, lse


@pytest.mark.parametrize("G", [1, 33, 64, 160])
def test_sums_of_keys_without_values(qa, G):
    """Many keys whose value rows are zero, their scores rising by less than moves the reference: lse is finite."""
    slots, rise = 20_000_000 // 256 * 256, 13.9
    x, want = two_levels("e4m3", 64, 128, slots, 1, G, rise, 0.0)
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    assert (o == 0).all()
    # logits and their exponentials as in logit_error; a thread adds the keys of its block at most
    x = rise * math.log(2.0)
    tol = x * (64 * 2.0 ** -23 + 4 * 2.0 ** -24) + 2.0 ** -22 * (want + 2) + (slots / 148 + 1024) * 2.0 ** -24
    assert ((lse.double() - want).abs() <= tol).all(), (lse.min().item(), lse.max().item(), want)


@pytest.mark.parametrize("G", [1, 16, 64, 160])
@pytest.mark.parametrize("rise", [23.5, 13.5])
def test_large_values_of_many_keys(qa, G, rise):
    """16-bit caches: values just below 2^100, 8192 keys a sequence, scores that rise in the middle of a run."""
    v = float(torch.tensor(2.0 ** 99.9).to(torch.bfloat16))
    x, want = two_levels("same", 128, 64, 8192, 16, G, rise, v)
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    t = rise * math.log(2.0)
    e = t * (128 * 2.0 ** -23 + 4 * 2.0 ** -24) + 2.0 ** -22
    assert ((lse.double() - want).abs() <= e + 2.0 ** -22 * (want + 1) + 8192 * 2.0 ** -24).all()
    # equal weights among equal scores, values alike: o is v but for P's rounding and the sums'
    rel = math.expm1(2 * e) + 2.0 ** -8 + 4 * 2.0 ** -24 + 8192 * 2.0 ** -24
    assert ((o.double() / v - 1).abs() <= rel).all(), (o.min().item() / v, o.max().item() / v)


def set_rows(c, name, b, h, first, x):
    """Rows `first`.. of sequence b, head h become x [n, d]."""
    if c.kv == "e4m3":
        code, scale = R.codes(x.to(c.dtype))
    for i in range(len(x)):
        p, r = cell(c, b, first + i)
        if c.kv == "e4m3":
            c.pool[name].view(torch.uint8)[p, h, r] = code[i].view(torch.uint8)
            c.pool[name + "_scale"][p, h, r] = scale[i]
        else:
            c.pool[name][p, h, r] = x[i].to(c.dtype)


# (T, G, d, dtype): rows of a head below and above each kernel's limits
CLIMB = [(1, 1, 128, "bf16"), (1, 8, 64, "fp16"), (3, 5, 128, "fp16"), (6, 8, 64, "bf16"), (30, 2, 128, "bf16"),
         (25, 4, 64, "fp16"), (50, 4, 128, "fp16"), (50, 4, 64, "bf16"), (64, 5, 128, "bf16")]


@pytest.mark.parametrize("profile", ["climb", "steps", "values"])
@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("T, G, d, dtype", CLIMB)
def test_scores_that_climb(qa, T, G, d, dtype, kv, profile):
    """References that move in the middle of a run, by more than 2^14, sums and O with them.  climb: over each 300
    keys the scores rise by 60; steps: 100 keys, then 20 whose score is 14.5 log2 units higher, with values
    of 2^13 in the lower ones, so that what was added before a move is as much as what comes after it.  values: the
    scores alike, the values of 2^-20 in the 100 and 1 in the 20: with an e4m3 cache the reference moves all the same,
    and the keys before a move hold most of the sum."""
    lens, Hkv = [2600, 1111], 8
    c = R.Case(33, lens, T, Hkv, G, d, 32, dtype, kv, junk=False)
    g = torch.Generator().manual_seed(12)
    u = torch.randn(Hkv, d, generator=g)
    u /= u.norm(dim=-1, keepdim=True)
    # a query's part along u: the score of a key k u + noise is about k
    size = math.sqrt(1 / c.sm)
    q = 0.3 * torch.randn(2, Hkv, G, T, d, generator=g) + size * u[:, None, None]
    c.q = q.view(2, Hkv * G, T, d).to(c.dtype)
    for b in range(2):
        n = lens[b] + T
        s = torch.arange(n)
        if profile == "climb":
            score, val = (s % 300) / 300 * 60.0, torch.ones(n)
        elif profile == "values":
            score, val = torch.zeros(n), torch.where(s % 120 >= 100, 1.0, 2.0 ** -20)
        else:
            high = s % 120 >= 100
            score, val = torch.where(high, 14.5 * math.log(2.0), 0.0), torch.where(high, 1.0, 2.0 ** 13)
        for h in range(Hkv):
            set_rows(c, "k", b, h, 0, size * score[:, None] * u[h] + 0.3 * torch.randn(n, d, generator=g))
            set_rows(c, "v", b, h, 0, val[:, None] * torch.randn(n, d, generator=g).clamp(-3, 3))
    x = c.cuda()
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    check(c, o, lse, attend(c))
