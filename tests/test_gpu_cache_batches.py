"""Attention and tally over a paged cache for more sequences than a warp looks up at a time, device integers out of
range for an append, and equal calls.  Tolerances as in tests/test_gpu_cache.py."""
import math

import pytest
import torch

from tests import cache_ref as R
from tests.test_gpu_cache import bad_index, check_tree, logit_error, pools_after_append, same_bits

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


# (B, longest, T, Hkv, G, d, kv): both attention kernels and both joins of pieces; 148 SMs
BATCH = [(33, 900, 1, 1, 1, 128, "same"), (33, 900, 50, 1, 1, 64, "e4m3"), (64, 300, 2, 2, 3, 64, "e4m3"),
         (100, 150, 3, 2, 2, 128, "same"), (97, 120, 25, 1, 3, 128, "e4m3"), (65, 130, 40, 1, 4, 64, "same"),
         (32, 500, 1, 2, 2, 128, "e4m3")]


@pytest.mark.parametrize("case", BATCH, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("empty", [False, True])
def test_many_sequences(qa, case, empty):
    """empty: the second 32 sequences ask for nothing, and of the others every fifth."""
    B, longest, T, Hkv, G, d, kv = case
    lens = [(b * 7919) % longest for b in range(B)]
    lens[0], lens[-1] = longest, 1
    n = [(T, max(1, T // 2), 1)[b % 3] for b in range(B)]
    if empty:
        n = [0 if 32 <= b < 64 or b % 5 == 2 else n[b] for b in range(B)]
    c = R.Case(61, lens, T, Hkv, G, d, 16, "bf16", kv, n, junk=False)
    x = c.cuda()
    want = R.attend(c)
    o, lse = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    assert qa.sage2_check_device_error() == 0
    check_tree(c, o, lse, want, torch.float32)
    acc = torch.full((B, Hkv, c.MP * 16), 0.5, device="cuda")
    known = want[1].float()
    args = (x["q"], known.cuda(), x["cache"], x["table"], x["lens"])
    qa.sage2_cache_weights(*args, acc, mask=x["mask"], n=x["n"])
    assert qa.sage2_check_device_error() == 0
    add = R.weights(c, known)
    e = logit_error(c) + 2.0 ** -22 * (known[known > -math.inf].abs().max().item() + 1)
    tol = add * (math.expm1(e) + (G * T + 4) * 2.0 ** -24) + 2.0 ** -24 * (add + 0.5)
    got = acc.double().cpu() - 0.5
    assert ((got - add).abs() <= tol).all()
    assert (got[add == 0] == 0).all()
    # equal calls give equal bits
    o2, lse2 = qa.sage2_attn_tree(out_dtype=torch.float32, **x)
    again = torch.full_like(acc, 0.5)
    qa.sage2_cache_weights(*args, again, mask=x["mask"], n=x["n"])
    assert same_bits(o, o2) and same_bits(lse, lse2) and same_bits(acc, again)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_equal_evictions(qa, kv):
    """The choice counts with atomics: equal calls choose and move alike."""
    c = R.Case(62, [3000, 2999], 1, 4, 1, 64, 32, "bf16", kv, junk=False)
    acc = (torch.rand(2, 4, c.MP * 32, generator=torch.Generator().manual_seed(3)) * 40).floor()
    got = []
    for _ in range(3):
        x = c.cuda()
        idx, new, out = qa.sage2_cache_evict(x["cache"], x["table"], x["lens"], acc.cuda(), 1001, 4, 100)
        got.append([idx, new, out, *x["cache"].values()])
    assert qa.sage2_check_device_error() == 0
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert same_bits(a, b)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_append_with_integers_out_of_range(qa, kv):
    """The error word is set; the sequence beside the bad one is written, its context and all other pages stay."""
    T = 3
    c = R.Case(63, [100, 37], T, 2, 1, 64, 16, "bf16", kv, junk=False)
    cap = c.MP * 16
    k, v = (torch.randn(2, 2, T, 64, generator=torch.Generator().manual_seed(i)).to(c.dtype) for i in (1, 2))
    good = pools_after_append(c, k, v)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    own = set(c.table[0].tolist())                      # pages of the bad sequence
    for what, val, kept in (("lens", [-1, 37], 0), ("lens", [2 ** 31 - 1, 37], 0), ("lens", [cap - 1, 37], 1),
                            ("n", [T + 1, T], 0), ("n", [-5, T], 0), ("page", c.pages, 0), ("page", -1, 0),
                            ("page", 2 ** 31 - 1, 0)):
        x = c.cuda()
        if what == "page":
            x["table"][0, 100 // 16] = val              # the page that its tokens go to
        else:
            x[what] = i32(val)
        qa.sage2_cache_append(k.cuda(), v.cuda(), x["cache"], x["table"], x["lens"], n=x["n"])
        assert bad_index(qa), (what, val)
        for name, t in x["cache"].items():
            for p in range(c.pages):
                if p not in own:
                    assert same_bits(t[p], good[name][p]), (what, val, name)
                elif not kept:                          # nothing of the bad sequence is written
                    assert same_bits(t[p], c.pool[name][p]), (what, val, name)
    # a bad page that no token goes to is not looked at
    x = c.cuda()
    x["table"][0, 0] = c.pages
    qa.sage2_cache_append(k.cuda(), v.cuda(), x["cache"], x["table"], x["lens"], n=x["n"])
    assert qa.sage2_check_device_error() == 0
    for name, t in x["cache"].items():
        assert same_bits(t, good[name])
