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
