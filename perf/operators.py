"""What is measured of the operators over a paged key/value cache.

A cache is a pool of pages, k and v [pages, Hkv, page, d], in 16 bits or in e4m3
with one fp32 scale a row; slot s of sequence b is row s % page of page
table[b, s // page].  `run` computes an operator in its plain form (elementary
torch operations, fp32) or, where `own` is set, through the package's calls.

Operators (the case's "op"):
  append   write the keys and values of new tokens behind each sequence's length
  tree     attention of drafted tokens (a tree, or one token) over cache and tree
  weights  add the attention weight that each cached token received to a tally
  evict    keep the tokens of the largest tally (and the first and last ones)
  compact  move given rows to the front of a region (an accepted path, a choice)
"""
import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases
def _case(name, op, B, Hq, Hkv, T, ctx, d, page, dtype, kv, keep=0):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "ctx": ctx, "d": d,
            "page": page, "dtype": dtype, "kv": kv, "keep": keep}


def listed():
    return [
        # one decoded token for two short sequences: latency of a step
        _case("tree_token_short", "tree", 2, 8, 8, 1, 2048, 128, 16, "f16", "same"),
        # one decoded token over a long 8-bit cache, grouped heads
        _case("tree_token_long", "tree", 1, 32, 8, 1, 32768, 128, 64, "bf16", "e4m3"),
        # a drafted tree of 61 nodes over ordinary contexts of unequal lengths
        _case("tree_61", "tree", 4, 32, 8, 61, 8192, 128, 32, "bf16", "same"),
        # a server's batch of trees over long 8-bit caches
        _case("tree_48_long", "tree", 16, 32, 8, 48, 32768, 128, 128, "bf16", "e4m3"),
        # tally of a small tree, a head for each query head, d = 64, an odd length
        _case("weights_13", "weights", 1, 24, 24, 13, 17776, 64, 16, "f16", "same"),
        # tally of a window of 48 queries over long 8-bit caches
        _case("weights_48_long", "weights", 8, 32, 8, 48, 32768, 128, 64, "bf16", "e4m3"),
        # a decode step's new token of 32 sequences: latency
        _case("append_token", "append", 32, 32, 8, 1, 2048, 128, 16, "bf16", "e4m3"),
        # a prompt written to an 8-bit cache
        _case("append_prompt", "append", 4, 32, 32, 8192, 0, 128, 64, "bf16", "e4m3"),
        # one long sequence cut to 4096 tokens a head
        _case("evict_one", "evict", 1, 24, 24, 0, 17776, 64, 16, "f16", "same", 4096),
        # a batch of long 8-bit caches cut to a quarter
        _case("evict_batch", "evict", 16, 32, 8, 0, 32768, 128, 64, "bf16", "e4m3", 8192),
        # the accepted path (7 nodes) of a tree moved behind the context
        _case("compact_path", "compact", 4, 32, 8, 61, 8192, 128, 32, "bf16", "same", 7),
        # a choice of half the tokens, by head, moved to the front
        _case("compact_half", "compact", 8, 32, 32, 0, 8192, 128, 128, "bf16", "same", 4096),
    ]


_MOST = {"tree": "tree_48_long", "weights": "weights_48_long", "append": "append_prompt",
         "evict": "evict_batch", "compact": "compact_half"}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "weights", "weights", "append", "evict", "compact"])
    most = work(next(c for c in listed() if c["name"] == _MOST[op]))
    while True:
        Hkv, G = rng.choice([1, 2, 4, 5, 8, 24, 32]), rng.choice([1, 1, 2, 3, 4, 7, 8])
        T, ctx, keep, B = 1, _log(rng, 1, 40000), 0, _log(rng, 1, 32)
        if op in ("tree", "weights"):
            T = rng.choice([1, 1, 2, 5, _log(rng, 3, 64), _log(rng, 8, 64), 64])
        if op == "append":
            T, ctx = rng.choice([1, _log(rng, 2, 64), _log(rng, 64, 8192)]), _log(rng, 1, 4096)
        if op == "evict":
            T, ctx, keep = 0, _log(rng, 200, 40000), 0
            keep = _log(rng, 64, max(65, ctx))
        if op == "compact":
            if rng.random() < 0.5:
                T = _log(rng, 4, 64)
                keep = rng.randint(1, max(1, T // 3))
            else:
                T, ctx = 0, _log(rng, 64, 16000)
                keep = rng.randint(1, ctx)
        c = _case("", op, B, Hkv * G, Hkv, T, ctx, rng.choice([64, 128, 128]),
                  rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16", "bf16"]),
                  rng.choice(["same", "e4m3"]), keep)
        del c["name"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and w["bytes"] > 2e5:
            return c


def _lens(c):
    """Tokens in the cache, by sequence: `ctx` for the first, up to a third fewer for the others."""
    return [c["ctx"] - (b * 977) % (c["ctx"] // 3 + 1) for b in range(c["B"])]


def _drafted(c):
    """Drafted tokens, by sequence: T for the first, some fewer for the others."""
    return [max(1, c["T"] - (b * 5) % (c["T"] // 4 + 1)) for b in range(c["B"])]


def _sinks_recent(c):
    return min(4, c["keep"] // 8), c["keep"] // 8


def work(case):
    c = case
    w = 2 if c["kv"] == "same" else 1
    row = c["d"] * w + (0 if c["kv"] == "same" else 4)  # bytes of one cached row of K or V
    B, Hq, Hkv, T, d = c["B"], c["Hq"], c["Hkv"], c["T"], c["d"]
    lens = _lens(c)
    if c["op"] in ("tree", "weights"):
        n = _drafted(c)
        keys = sum(x + y for x, y in zip(lens, n))
        dots = sum(y * (x + y) for x, y in zip(lens, n)) * Hq
        q = B * Hq * T * d * 2
        if c["op"] == "tree":
            return {"bytes": 2 * q + B * Hq * T * 4 + 2 * Hkv * keys * row + B * T * T,
                    "flops": 4.0 * dots * d}
        return {"bytes": q + B * Hq * T * 4 + Hkv * keys * (row + 8) + B * T * T,
                "flops": 2.0 * dots * d}
    if c["op"] == "append":
        return {"bytes": 2.0 * B * Hkv * T * (2 * d + row), "flops": 0.0}
    if c["op"] == "evict":
        kept = sum(min(c["keep"], x) for x in lens) * Hkv
        return {"bytes": sum(lens) * Hkv * 4.0 + kept * (4 * row + 12), "flops": 0.0}
    moved = sum(min(c["keep"], x) if T == 0 else c["keep"] for x in lens) * Hkv
    return {"bytes": moved * (4.0 * row + 4), "flops": 0.0}


# -------------------------------------------------------------------- inputs
def _cuts(x):
    """Rows of `x` in e4m3 and their scales: scale = amax / 448, code = x * (448 / amax)."""
    x = x.float()
    amax = x.abs().amax(-1)
    top = torch.full_like(amax, 448.0)
    some = amax > 0
    scale = torch.where(some, torch.div(amax, top), 0.0)
    inv = torch.where(some, torch.div(top, amax), 0.0)
    return (x * inv[..., None]).to(torch.float8_e4m3fn), scale


def _tree(g, T):
    """Which drafted tokens a drafted token attends: itself and its ancestors in a random tree."""
    m = np.eye(T, dtype=bool)
    for i in range(1, T):
        p = int(g.integers(max(-1, i - 9), i))
        if p >= 0:
            m[i] |= m[p]
    return m


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(seed)
    ng = np.random.default_rng(seed)
    dev, dt = "cuda", _DT[c["dtype"]]
    B, Hq, Hkv, T, d, page = c["B"], c["Hq"], c["Hkv"], c["T"], c["d"], c["page"]
    MP = -(-(c["ctx"] + T) // page)
    rows = 2 if c["op"] == "evict" else 1  # the eviction writes to pages of its own
    MO = -(-c["keep"] // page) if rows == 2 else 0
    pages = B * (MP + MO)
    perm = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    s = {"op": c["op"], "d": d, "page": page, "sm": 1.0 / math.sqrt(d),
         "table": perm[:B * MP].view(B, MP).contiguous(),
         "lens": torch.tensor(_lens(c), dtype=torch.int32, device=dev), "slots": MP * page}

    def rand(*shape):
        return torch.randn(*shape, device=dev, generator=g, dtype=dt)

    def keys(shape):
        # an offset a channel and four channels of a larger spread, as keys have
        spread = torch.ones(Hkv, 1, d, device=dev, dtype=dt)
        spread[:, :, torch.randperm(d, device=dev, generator=g)[:4]] = 3
        return rand(*shape) * spread + 2 * rand(Hkv, 1, d)

    if c["op"] == "append":
        s["k"], s["v"] = keys((B, Hkv, T, d)), rand(B, Hkv, T, d) + rand(Hkv, 1, d)
        if c["kv"] == "same":
            s["cache"] = {n: torch.zeros(pages, Hkv, page, d, dtype=dt, device=dev) for n in "kv"}
        else:
            s["cache"] = {n: torch.zeros(pages, Hkv, page, d, dtype=torch.float8_e4m3fn, device=dev)
                          for n in "kv"}
            for n in "kv":
                s["cache"][n + "_scale"] = torch.zeros(pages, Hkv, page, device=dev)
        return s

    k, v = keys((pages, Hkv, page, d)), rand(pages, Hkv, page, d) + rand(Hkv, 1, d)
    if c["kv"] == "same":
        s["cache"] = {"k": k, "v": v}
    else:
        s["cache"] = {}
        for n, x in (("k", k), ("v", v)):
            codes, scales = zip(*(_cuts(p) for p in x.split(max(1, 2 ** 28 // (Hkv * page * d)))))
            s["cache"][n], s["cache"][n + "_scale"] = torch.cat([t.view(torch.uint8) for t in codes]).view(
                torch.float8_e4m3fn), torch.cat(scales)
    del k, v
    if c["op"] in ("tree", "weights"):
        s["q"] = 3 * rand(B, Hq, T, d) + rand(Hq, 1, d)
        s["n"] = torch.tensor(_drafted(c), dtype=torch.int32, device=dev)
        s["mask"] = torch.from_numpy(np.stack([_tree(ng, T) for _ in range(B)])).to(dev)
    if c["op"] == "weights":
        s["lse"] = _attend(s)[1]  # what the attention before has returned
    if c["op"] in ("weights", "evict"):
        # few tokens hold most of it; its mean is that of a tally of some steps
        s["acc"] = torch.rand(B, Hkv, s["slots"], device=dev, generator=g) ** 8 * (
            9.0 * max(1, T) * (Hq // Hkv) / c["ctx"])
    if c["op"] == "evict":
        s["keep"], s["out_table"] = c["keep"], perm[B * MP:].view(B, MO).contiguous()
        s["sinks"], s["recent"] = _sinks_recent(c)
    if c["op"] == "compact":
        M = c["keep"]
        if T:  # a path of M nodes, the same for all heads
            idx = np.stack([np.sort(ng.choice(T, M, replace=False)) + x for x in _lens(c)])[:, None]
            s["base"], count = s["lens"], [M] * B
        else:  # M tokens a head
            key = torch.rand(B, Hkv, s["slots"], device=dev, generator=g)
            at = torch.arange(s["slots"], device=dev)
            key = torch.where(at < s["lens"][:, None, None], key, 2.0)
            idx = torch.sort(torch.topk(key, M, dim=-1, largest=False).indices, -1).values.cpu().numpy()
            s["base"], count = torch.zeros(B, dtype=torch.int32, device=dev), [min(M, x) for x in _lens(c)]
        s["idx"] = torch.from_numpy(np.ascontiguousarray(idx)).to(torch.int32).to(dev).expand(
            B, Hkv, M)
        s["count"] = torch.tensor(count, dtype=torch.int32, device=dev)
    return s


# --------------------------------------------------------------- plain forms
def _dense(s, n):
    """K or V of each sequence in slot order, [B, Hkv, slots, d] in fp32."""
    t = s["table"].long()
    x = s["cache"][n]
    if x.dtype == torch.float8_e4m3fn:
        x = x.view(torch.uint8)[t].view(torch.float8_e4m3fn).float()
        x = x * s["cache"][n + "_scale"][t][..., None]
    else:
        x = x[t].float()
    return x.transpose(1, 2).flatten(2, 3)


def _allowed(s):
    """[B, 1, T, slots]: which slot each drafted token attends."""
    T = s["q"].shape[2]
    at = torch.arange(s["slots"], device="cuda")
    ln, n = s["lens"].long()[:, None], s["n"].long()[:, None]
    j = at - ln
    inside = s["mask"].gather(2, j.clamp(0, T - 1)[:, None].expand(-1, T, -1))
    a = (j < 0)[:, None] | (inside & ((j >= 0) & (j < n))[:, None])
    return (a & (torch.arange(T, device="cuda") < n)[:, :, None])[:, None]


def _scores(s):
    """Scaled scores [B, Hkv, G, T, slots], -inf where a token is not attended."""
    q = s["q"].float()
    B, Hq, T, d = q.shape
    k = _dense(s, "k")
    Hkv = k.shape[1]
    x = (q.view(B, Hkv, -1, d) @ k.transpose(2, 3)).mul_(s["sm"]).view(B, Hkv, Hq // Hkv, T, -1)
    return x.masked_fill_(~_allowed(s)[:, :, None], -math.inf)


def _attend(s):
    x = _scores(s)
    B, Hkv, G, T, S = x.shape
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * T, S) @ _dense(s, "v")).view(B, Hkv, G, T, -1)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    return o.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(B, Hkv * G, T)


def _weights(s):
    x = _scores(s)
    lse = s["lse"].view(x.shape[:4])[..., None]
    x = x.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    s["acc"] += x.sum((2, 3))
    return s["acc"]


def _append(s):
    B, Hkv, T, d = s["k"].shape
    slot = s["lens"].long()[:, None] + torch.arange(T, device="cuda")
    at = s["table"].long().gather(1, slot // s["page"])
    at = (at[:, None] * Hkv + torch.arange(Hkv, device="cuda")[:, None]) * s["page"] + (slot % s["page"])[:, None]
    for n in "kv":
        pool = s["cache"][n]
        if pool.dtype == torch.float8_e4m3fn:
            codes, scale = _cuts(s[n])
            pool.view(torch.uint8).view(-1, d)[at] = codes.view(torch.uint8)
            s["cache"][n + "_scale"].view(-1)[at] = scale
        else:
            pool.view(-1, d)[at] = s[n]
    return s["cache"]


def _move(s, idx, base, count, table):
    """Slot base + i of `table` takes slot idx[.., i], i < count; the others go to themselves."""
    B, Hkv, M = idx.shape
    page, d = s["page"], s["d"]
    i = torch.arange(M, device="cuda")
    live = (i < count.long()[:, None])[:, None]
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    first = torch.where(live, idx.long(), idx[:, :, :1].long())
    into = torch.where(live, (base.long()[:, None] + i)[:, None].expand(-1, Hkv, -1), base.long()[:, None, None])

    def rows(t, slot):
        return (t.long()[:, None].expand(-1, Hkv, -1).gather(2, slot // page) * Hkv + h) * page + slot % page

    # a row that is not live repeats the first one
    src, dst = rows(s["table"], first), rows(table, into)
    for n, pool in s["cache"].items():
        flat = pool.view(torch.uint8).view(-1, d) if pool.dtype == torch.float8_e4m3fn else \
            pool.view(-1, d) if pool.dim() == 4 else pool.view(-1)
        flat[dst] = flat[src]


def _evict(s):
    B, Hkv, S = s["acc"].shape
    keep, sinks, recent = s["keep"], s["sinks"], s["recent"]
    at = torch.arange(S, device="cuda")
    ln = s["lens"].long()[:, None, None]
    new = torch.minimum(s["lens"], torch.full_like(s["lens"], keep))
    key = torch.where((at < sinks) | ((at >= ln - recent) & (at < ln)), math.inf, s["acc"])
    key = torch.where(at < ln, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    live = (torch.arange(keep, device="cuda") < new[:, None])[:, None]
    idx = torch.sort(torch.where(live, order, S), dim=-1).values
    idx = torch.where(live, idx, -1).to(torch.int32)
    acc = torch.where(live, s["acc"].gather(2, idx.long().clamp(min=0)), 0.0)
    _move(s, idx, torch.zeros_like(new), new, s["out_table"])
    return {"idx": idx, "lens": new, "acc": acc, "cache": s["cache"]}


def run(state):
    s = state
    op = s["op"]
    if own:
        import quantized_attention_04_b200 as qa
        if op == "tree":
            return qa.sage2_attn_tree(s["q"], s["cache"], s["table"], s["lens"], mask=s["mask"],
                                      n=s["n"], sm_scale=s["sm"])
        if op == "weights":
            return qa.sage2_cache_weights(s["q"], s["lse"], s["cache"], s["table"], s["lens"],
                                          s["acc"], mask=s["mask"], n=s["n"], sm_scale=s["sm"])
        if op == "append":
            return qa.sage2_cache_append(s["k"], s["v"], s["cache"], s["table"], s["lens"])
        if op == "evict":
            idx, lens, acc = qa.sage2_cache_evict(s["cache"], s["table"], s["lens"], s["acc"],
                                                  s["keep"], sinks=s["sinks"], recent=s["recent"],
                                                  out_table=s["out_table"])
            return {"idx": idx, "lens": lens, "acc": acc, "cache": s["cache"]}
        return qa.sage2_cache_compact(s["cache"], s["table"], s["idx"], s["count"], base=s["base"])
    if op == "tree":
        return _attend(s)
    if op == "weights":
        return _weights(s)
    if op == "append":
        return _append(s)
    if op == "evict":
        return _evict(s)
    _move(s, s["idx"], s["base"], s["count"], s["table"])
    return s["cache"]


# ------------------------------------------------------------------- 64 bits
def _sequence(s, n, b, h, length, dt=torch.float64):
    """K or V of one head of one sequence, `length` slots, in 64 bits."""
    pages = s["table"][b, :-(-length // s["page"])].long()
    pool = s["cache"][n]
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).to(dt)
        x = x * s["cache"][n + "_scale"][pages, h].to(dt)[..., None]
    else:
        x = pool[pages, h].to(dt)
    return x.reshape(-1, s["d"])[:length]


def _exact_rows(s, want_o):
    """For each (sequence, head): its rows' logits in 64 bits, with what they make of them."""
    q, sm = s["q"].double(), s["sm"]
    B, Hq, T, d = q.shape
    Hkv = s["cache"]["k"].shape[1]
    G = Hq // Hkv
    lens, drafted = s["lens"].tolist(), s["n"].tolist()
    o = torch.zeros_like(q)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if not want_o else None
    for b in range(B):
        ln, n = lens[b], drafted[b]
        bar = torch.zeros(n, ln + n, dtype=torch.float64, device="cuda")
        bar[:, ln:][~s["mask"][b, :n, :n]] = -math.inf
        for h in range(Hkv):
            rows = q[b, h * G:(h + 1) * G, :n].reshape(G * n, d)
            x = torch.einsum("rd,sd->rs", rows, _sequence(s, "k", b, h, ln + n)) * sm
            x = x.view(G, n, -1) + bar
            if want_o:
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[..., None])
                o[b, h * G:(h + 1) * G, :n] = torch.einsum("gts,sd->gtd", w, _sequence(s, "v", b, h, ln + n))
                lse[b, h * G:(h + 1) * G, :n] = z
            else:
                z = s["lse"][b, h * G:(h + 1) * G, :n].double()
                acc[b, h, :ln + n] += torch.exp(x - z[..., None]).sum((0, 1))
    return (o, lse) if want_o else acc


def _exact_codes(x):
    """The rows' codes and scales, with the roundings that the stored form is defined by."""
    x = x.double()
    a = x.abs().amax(-1)
    scale = torch.where(a > 0, a / 448.0, 0.0).float()
    inv = torch.where(a > 0, 448.0 / a, 0.0).float().double()
    return (x * inv[..., None]).float().to(torch.float8_e4m3fn), scale


def exact(case, seed):
    s = prepare(case, seed)
    op, page = s["op"], s["page"]
    if op == "tree":
        return _exact_rows(s, True)
    if op == "weights":
        return _exact_rows(s, False)
    out = {n: t.clone() for n, t in s["cache"].items()}
    table, lens = s["table"].long(), s["lens"].tolist()
    B = len(lens)

    def pool(t):
        return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t

    if op == "append":
        T = s["k"].shape[2]
        for b in range(B):
            slot = torch.arange(lens[b], lens[b] + T, device="cuda")
            p, r = table[b][slot // page], slot % page
            for n in "kv":
                x = s[n][b].transpose(0, 1)
                if out[n].dtype == torch.float8_e4m3fn:
                    codes, out[n + "_scale"][p, :, r] = _exact_codes(x)
                    pool(out[n])[p, :, r] = codes.view(torch.uint8)
                else:
                    out[n][p, :, r] = x
        return out

    Hkv = s["cache"]["k"].shape[1]
    if op == "evict":
        keep, sinks, recent = s["keep"], s["sinks"], s["recent"]
        tally = s["acc"].cpu().numpy()
        idx = np.full((B, Hkv, keep), -1, np.int32)
        acc = np.zeros((B, Hkv, keep))
        for b in range(B):
            for h in range(Hkv):
                ln, a = lens[b], tally[b, h].astype(np.float64)
                if ln <= keep:
                    got = np.arange(ln)
                else:
                    mid = np.arange(sinks, ln - recent)
                    best = mid[np.lexsort((mid, -a[mid]))[:keep - sinks - recent]]
                    got = np.sort(np.concatenate([np.arange(sinks), best, np.arange(ln - recent, ln)]))
                idx[b, h, :len(got)], acc[b, h, :len(got)] = got, a[got]
        count, base, to = [min(keep, x) for x in lens], [0] * B, s["out_table"].long()
    else:
        idx, count, base, to = s["idx"].cpu().numpy(), s["count"].tolist(), s["base"].tolist(), table
    for b in range(B):
        src = torch.from_numpy(idx[b, :, :count[b]].astype(np.int64)).to("cuda")
        dst = torch.arange(base[b], base[b] + count[b], device="cuda")
        h = torch.arange(Hkv, device="cuda")
        for n in out:
            out_n, in_n = pool(out[n]), pool(s["cache"][n])
            out_n[to[b][dst // page][None], h[:, None], (dst % page)[None]] = in_n[
                table[b][src // page], h[:, None], src % page]
    if op == "compact":
        return out
    return {"idx": idx, "lens": np.array(count, np.int32), "acc": acc, "cache": out}
