"""Padded batches: more tokens or indices a sequence than its table has slots, of which n[b] are in use."""
import pytest
import torch

from tests import cache_ref as R
from tests.test_gpu_cache import pools_after_append, pools_after_move, same_bits

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


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_padded_prompt(qa, kv):
    c = R.Case(51, [0, 3, 60], 200, 2, 1, 64, 16, "bf16", kv, n=[64, 10, 0], junk=False)
    assert c.MP * 16 == 64
    x = c.cuda()
    k, v = (torch.randn(3, 2, 200, 64, generator=torch.Generator().manual_seed(i)).to(c.dtype) for i in (1, 2))
    want = pools_after_append(c, k, v)
    qa.sage2_cache_append(k.cuda(), v.cuda(), x["cache"], x["table"], x["lens"], n=x["n"])
    assert qa.sage2_check_device_error() == 0
    for name, t in want.items():
        assert same_bits(x["cache"][name], t), name
    with pytest.raises(qa.Sage2Error):
        qa.sage2_cache_append(k.cuda(), v.cuda(), x["cache"], x["table"], x["lens"])


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_padded_indices(qa, kv):
    c = R.Case(52, [60, 30], 1, 2, 1, 128, 16, "bf16", kv, junk=False)
    x = c.cuda()
    idx = torch.full((2, 2, 300), -1, dtype=torch.int32)
    idx[:, :, :20] = torch.arange(20) + 5
    want = pools_after_move(c.pool, c.table, c.table, 16, idx, [20, 7], [0, 2])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda(), i32([20, 7]), base=i32([0, 2]))
    assert qa.sage2_check_device_error() == 0
    for name, t in want.items():
        assert same_bits(x["cache"][name], t), name
    with pytest.raises(qa.Sage2Error):
        qa.sage2_cache_compact(x["cache"], x["table"], idx.cuda())
