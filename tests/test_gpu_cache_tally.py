"""The tally of attention weight over a sequence's life: what eviction and moves leave of it."""
import math

import pytest
import torch

from tests import cache_ref as R
from tests.test_gpu_cache import logit_error, same_bits

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


@pytest.mark.parametrize("where", ["in place", "in place, apart", "another table"])
@pytest.mark.parametrize("kv, keep", [("same", 48), ("e4m3", 48), ("same", 1), ("e4m3", 300), ("same", 700)])
def test_eviction_clears_the_tally_behind_the_kept(qa, where, kv, keep):
    """Slots from the new length on have a tally of 0, whatever acc_out held, and no slot before them changes but
    as the choice says."""
    lens = [700, 48, 47, 0, 333, 2]
    c = R.Case(41, lens, 1, 3, 1, 64, 16, "bf16", kv, extra=3, spare=6 * 48, junk=False)
    x = c.cuda()
    S = c.MP * 16
    acc = torch.rand(6, 3, S, generator=torch.Generator().manual_seed(8)) + 0.5
    out, table = None, None
    if where == "in place":
        accd = out = acc.cuda()
    else:
        accd, out = acc.cuda(), torch.full((6, 3, S + 5), 7.0, device="cuda")
        if where == "another table":
            other = sorted(set(range(c.pages)) - set(c.table.flatten().tolist()))
            table = torch.tensor(other[:6 * 44], dtype=torch.int32).view(6, 44).cuda()
    idx, new, got = qa.sage2_cache_evict(x["cache"], x["table"], x["lens"], accd, keep, min(2, keep - 1),
                                         min(7, keep - 1) if keep > 8 else 0, out_table=table, acc_out=out)
    assert qa.sage2_check_device_error() == 0 and got is out
    assert new.tolist() == [min(keep, l) for l in lens]
    want = torch.zeros(out.shape)
    for b in range(6):
        for h in range(3):
            at = idx[b, h, :new[b]].cpu().long()
            want[b, h, :len(at)] = acc[b, h, at]
    assert same_bits(out, want)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_rounds_of_drafting_and_eviction(qa, kv):
    """The loop of a server, three times over: append, attention, tally, accepted path,
    and an eviction in each.  The tally of every token is the weight that it has received since it was written (in
    64 bits on the host), and slots without a token have none."""
    B, Hkv, G, T, d, page, keep, sinks, recent = 2, 2, 2, 6, 64, 16, 40, 2, 8
    dt, rng = torch.bfloat16, torch.Generator().manual_seed(9)
    Hq, sm = Hkv * G, 1.0 / math.sqrt(d)
    cache = qa.sage2_cache_alloc(2 * 8, Hkv, page, d, torch.float8_e4m3fn if kv == "e4m3" else dt)
    table = torch.randperm(16, generator=rng).to(torch.int32).view(2, 8).cuda()
    acc = torch.zeros(B, Hkv, 8 * page, device="cuda")
    slots = torch.arange(8 * page, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def rows(x):                       # what the cache holds of rows x
        if kv == "same":
            return x.double()
        code, scale = R.codes(x)
        return code.double() * scale.double()[..., None]

    # on the host: by sequence and head, the keys of its tokens in slot order, and their tallies
    keys = [[torch.zeros(0, d, dtype=torch.float64) for _ in range(Hkv)] for _ in range(B)]
    tally = [[torch.zeros(0, dtype=torch.float64) for _ in range(Hkv)] for _ in range(B)]
    err = 0.0                          # bound on what a tally may be off by

    def draft(k, v, q, mask):
        nonlocal err
        qa.sage2_cache_append(k.cuda(), v.cuda(), cache, table, lens)
        o, lse = qa.sage2_attn_tree(q.cuda(), cache, table, lens, mask=mask.cuda())
        qa.sage2_cache_weights(q.cuda(), lse, cache, table, lens, acc, mask=mask.cuda())
        lse, t, most = lse.double().cpu(), k.shape[2], 0.0
        for b in range(B):
            for h in range(Hkv):
                K = keys[b][h] = torch.cat([keys[b][h], rows(k[b, h])])
                ln = len(K) - t
                add = torch.zeros(len(K), dtype=torch.float64)
                for g in range(G):
                    s = q[b, h * G + g].double() @ K.T * sm
                    s[:, ln:][~mask[b]] = -math.inf
                    add += torch.exp(s - lse[b, h * G + g, :, None]).sum(0)
                tally[b][h] = torch.cat([tally[b][h], torch.zeros(t, dtype=torch.float64)]) + add
                x = q[b].double().norm(dim=-1).max().item() * K.norm(dim=-1).max().item() * sm
                e = x * (d * 2.0 ** -23 + 4 * 2.0 ** -24) + 2.0 ** -22 * (lse.abs().max().item() + 2)
                most = max(most, (add * (math.expm1(e) + (G * t + 4) * 2.0 ** -24)).max().item()
                           + 2.0 ** -24 * tally[b][h].max().item())
        err += most

    def compare():
        assert qa.sage2_check_device_error() == 0
        got, ln = acc.double().cpu(), lens.tolist()
        for b in range(B):
            for h in range(Hkv):
                assert ln[b] == len(keys[b][h])
                assert ((got[b, h, :ln[b]] - tally[b][h]).abs() <= err).all()
            assert (got[b, :, ln[b]:] == 0).all()

    new = lambda *s: torch.randn(*s, d, generator=rng).to(dt)
    P = 50                             # the prompt: its queries too, as one chain
    draft(new(B, Hkv, P), new(B, Hkv, P), 2 * new(B, Hq, P), torch.ones(B, P, P).tril().bool())
    lens += P
    compare()
    for step in range(3):
        mask = torch.eye(T).bool().expand(B, T, T).clone()
        for b in range(B):
            for i in range(1, T):
                mask[b, i] |= mask[b, int(torch.randint(0, i, (1,), generator=rng))]
        draft(new(B, Hkv, T), new(B, Hkv, T), 2 * new(B, Hq, T), mask)
        # the accepted path: the ancestors of a node
        took = [int(torch.nonzero(mask[b, T - 1 - b]).numel()) for b in range(B)]
        path = torch.zeros(B, T, dtype=torch.int32)
        for b in range(B):
            path[b, :took[b]] = torch.nonzero(mask[b, T - 1 - b])[:, 0].to(torch.int32)
        path_slots = (lens[:, None] + path.cuda())[:, None].expand(B, Hkv, T)
        n = torch.tensor(took, dtype=torch.int32, device="cuda")
        qa.sage2_cache_compact(cache, table, path_slots, n=n, base=lens, acc=acc)
        lens = lens + n
        acc.masked_fill_(slots >= lens[:, None, None], 0)
        for b in range(B):
            for h in range(Hkv):
                ln = len(keys[b][h]) - T
                at = torch.cat([torch.arange(ln), ln + path[b, :took[b]].long()])
                keys[b][h], tally[b][h] = keys[b][h][at], tally[b][h][at]
        compare()
        before = acc.cpu()
        old = lens.tolist()
        idx, lens, acc = qa.sage2_cache_evict(cache, table, lens, acc, keep, sinks, recent, acc_out=acc)
        assert lens.tolist() == [min(keep, x) for x in old]
        for b in range(B):
            for h in range(Hkv):
                at = torch.tensor(R.choose(before[b, h], old[b], keep, sinks, recent))
                assert torch.equal(idx[b, h, :len(at)].cpu().long(), at)
                keys[b][h], tally[b][h] = keys[b][h][at], tally[b][h][at]
        compare()


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("T, G, d, dtype", [(1, 1, 128, "bf16"), (9, 4, 64, "fp16"), (40, 8, 128, "bf16")])
@pytest.mark.parametrize("query", [False, True])
def test_rows_whose_lse_is_not_a_number(qa, T, G, d, dtype, kv, query):
    """Such a row (an attended key or its own query was not finite) reaches the tallies of the slots that it
    attends, all of them, and no others; with an infinity in its query too."""
    c = R.Case(42, [300, 20], T, 2, G, d, 16, dtype, kv)
    _, lse, _ = R.attend(c)
    lse = lse.float()
    i = min(2, T - 1)
    lse[0, G, i] = math.nan                                  # a row of sequence 0, head 1
    want = R.weights(c, lse)                                 # of finite q: NaN where the row attends
    if query:
        c.q[0, G, i, 5] = math.inf
    x = c.cuda()
    acc = torch.zeros(2, 2, c.MP * 16, device="cuda")
    qa.sage2_cache_weights(x["q"], lse.cuda(), x["cache"], x["table"], x["lens"], acc, mask=x["mask"], n=x["n"])
    assert qa.sage2_check_device_error() == 0
    got = acc.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    c.q[0, G, i, 5] = 0
    fine = torch.isfinite(lse)
    e = logit_error(c) + 2.0 ** -22 * (lse[fine].abs().max().item() + 1)
    some = ~torch.isnan(want)
    assert ((got - want).abs() <= want * (math.expm1(e) + (G * T + 8) * 2.0 ** -24))[some].all()


def test_tallies_in_other_layouts(qa):
    """Heads before sequences, slots of a wider buffer, a sequence's tally apart: as the contiguous one."""
    c = R.Case(43, [150, 99, 20], 4, 2, 2, 64, 16, "bf16", "same", junk=False)
    x = c.cuda()
    _, lse = qa.sage2_attn_tree(**x)
    S = c.MP * 16
    got = []
    for make in (lambda: torch.zeros(3, 2, S, device="cuda"), lambda: torch.zeros(2, 3, S, device="cuda").transpose(0, 1),
                 lambda: torch.zeros(3, 2, 2 * S, device="cuda")[:, :, S:], lambda: torch.zeros(2, 5, S, device="cuda")[:, 1:4].transpose(0, 1)):
        acc, y = make(), c.cuda()
        qa.sage2_cache_weights(x["q"], lse, x["cache"], x["table"], x["lens"], acc, mask=x["mask"])
        one = acc.clone()
        idx, new, out = qa.sage2_cache_evict(y["cache"], y["table"], y["lens"], acc, 64, 2, 8, acc_out=acc)
        got.append((one, idx, new, out))
    assert qa.sage2_check_device_error() == 0
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert same_bits(a, b)


@pytest.mark.parametrize("in_place", [True, False])
def test_moves_outside_of_the_tally(qa, in_place):
    """A row whose tally, taken or written, has no place in acc or acc_out sets the error word; the rows move and the
    other tallies with them."""
    c = R.Case(44, [200], 1, 2, 1, 64, 16, "bf16", "e4m3", spare=13, junk=False)
    other = sorted(set(range(c.pages)) - set(c.table.flatten().tolist()))
    table = None if in_place else torch.tensor(other, dtype=torch.int32)[None].cuda()
    idx = torch.arange(40, 60, dtype=torch.int32).expand(1, 2, 20)
    for S, SO in ((50, 100), (100, 7), (100, 100)):
        x = c.cuda()
        acc = torch.rand(1, 2, S, device="cuda")
        out = torch.full((1, 2, SO), 3.0, device="cuda")
        qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda(), out_table=table, acc=acc, acc_out=out)
        assert qa.sage2_check_device_error() == (0 if S == SO else 8)
        n = min(S - 40, SO, 20)
        assert torch.equal(out[:, :, :n], acc[:, :, 40:40 + n])
        assert (out[:, :, 20:] == 3).all()
        to = c.table[0] if in_place else table[0].cpu()
        for i in range(20):
            p, r, q, t = int(c.table[0, (40 + i) // 16]), (40 + i) % 16, int(to[i // 16]), i % 16
            assert same_bits(x["cache"]["k"].view(torch.uint8)[q, :, t], c.pool["k"].view(torch.uint8)[p, :, r])
            assert same_bits(x["cache"]["v_scale"][q, :, t], c.pool["v_scale"][p, :, r])
