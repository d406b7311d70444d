"""Host-side refusals of the cache entries (no GPU needed): argument checks return their status
before anything touches CUDA, and the binding raises on tensors it cannot pass on."""
import ctypes

import pytest
import torch

P = 0x10000  # 16-byte aligned fake address: never dereferenced by the checks


@pytest.fixture(scope="module")
def qa():
    from quantized_attention_04_b200 import build
    build.build()
    import quantized_attention_04_b200 as m
    m.lib()
    return m


def cache(qa, **kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, kv_dtype=3, pages=10, Hkv=2, page_size=16, d=64)
    a.update(kw)
    return ctypes.byref(qa._Cache(*[a[n] for n, _ in qa._Cache._fields_]))


BAD_CACHE = [(dict(k=0), 1), (dict(v=P + 8), 3), (dict(k_scale=0), 1), (dict(v_scale=P + 4), 3),
             (dict(kv_dtype=2), 1), (dict(kv_dtype=4), 1), (dict(pages=0), 1), (dict(Hkv=-1), 1),
             (dict(page_size=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2),
             (dict(page_size=256), 2), (dict(d=96), 2), (dict(Hkv=70000), 2),
             (dict(pages=2 ** 30, Hkv=2), 2)]


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def tree(qa, c=None, **kw):
    a = dict(q=P, dtype=1, qs=None, table=P, mp=4, lens=P, n=0, mask=0, ms=0, o=P, odt=1, lse=P, B=2,
             Hq=4, T=3, sm=0.1)
    a.update(kw)
    return qa.lib().sage2_attn_tree(a["q"], a["dtype"], a["qs"], c or cache(qa), a["table"], a["mp"],
                                    a["lens"], a["n"], a["mask"], a["ms"], a["o"], a["odt"], a["lse"],
                                    a["B"], a["Hq"], a["T"], a["sm"], None)


def weights(qa, c=None, **kw):
    a = dict(q=P, dtype=1, qs=None, lse=P, table=P, mp=4, lens=P, n=0, mask=0, ms=0, acc=P,
             st=strides(128, 64), S=64, B=2, Hq=4, T=3, sm=0.1)
    a.update(kw)
    return qa.lib().sage2_cache_weights(a["q"], a["dtype"], a["qs"], a["lse"], c or cache(qa), a["table"],
                                        a["mp"], a["lens"], a["n"], a["mask"], a["ms"], a["acc"], a["st"],
                                        a["S"], a["B"], a["Hq"], a["T"], a["sm"], None)


def append(qa, c=None, **kw):
    a = dict(k=P, v=P, dtype=1, ks=None, vs=None, table=P, mp=4, lens=P, n=0, B=2, T=3)
    a.update(kw)
    return qa.lib().sage2_cache_append(a["k"], a["v"], a["dtype"], a["ks"], a["vs"], c or cache(qa),
                                       a["table"], a["mp"], a["lens"], a["n"], a["B"], a["T"], None)


def compact(qa, c=None, **kw):
    a = dict(table=P, mp=4, ot=0, om=0, idx=P, ist=None, n=0, base=0, acc=0, ast=None, S=0, ao=0,
             aost=None, SO=0, B=2, M=5)
    a.update(kw)
    return qa.lib().sage2_cache_compact(c or cache(qa), a["table"], a["mp"], a["ot"], a["om"], a["idx"],
                                        a["ist"], a["n"], a["base"], a["acc"], a["ast"], a["S"], a["ao"],
                                        a["aost"], a["SO"], a["B"], a["M"], None)


def evict(qa, c=None, **kw):
    a = dict(table=P, mp=4, ot=0, om=0, lens=P, acc=P, ast=strides(128, 64), S=64, ao=P,
             aost=strides(128, 64), SO=64, B=2, keep=5, sinks=1, recent=1, idx=P, new=P)
    a.update(kw)
    return qa.lib().sage2_cache_evict(c or cache(qa), a["table"], a["mp"], a["ot"], a["om"], a["lens"],
                                      a["acc"], a["ast"], a["S"], a["ao"], a["aost"], a["SO"], a["B"],
                                      a["keep"], a["sinks"], a["recent"], a["idx"], a["new"], None)


@pytest.mark.parametrize("call", [tree, weights, append, compact, evict])
def test_bad_caches(qa, call):
    for kw, want in BAD_CACHE:
        assert call(qa, cache(qa, **kw)) == want, kw
    for kw, want in [(dict(table=0), 1), (dict(table=P + 2), 3), (dict(mp=0), 1), (dict(B=0), 1),
                     (dict(B=70000), 2), (dict(mp=2 ** 30), 2)]:
        assert call(qa, **kw) == want, kw


@pytest.mark.parametrize("call", [tree, weights])
def test_bad_queries(qa, call):
    for kw, want in [(dict(q=0), 1), (dict(q=P + 8), 3), (dict(dtype=2), 1), (dict(dtype=3), 1),
                     (dict(Hq=0), 1), (dict(Hq=3), 1), (dict(T=0), 1), (dict(T=1025), 2),
                     (dict(sm=0.0), 1), (dict(sm=float("nan")), 1), (dict(sm=float("inf")), 1),
                     (dict(lens=0), 1), (dict(lens=P + 1), 3), (dict(n=P + 2), 3), (dict(ms=-1), 1),
                     (dict(qs=strides(-8, 64, 64)), 1), (dict(qs=strides(768, 65, 64)), 3)]:
        assert call(qa, **kw) == want, kw
    # a 16-bit cache takes queries of its own type
    assert call(qa, cache(qa, kv_dtype=0, k_scale=0, v_scale=0), dtype=1) == 1


def test_bad_others(qa):
    for kw, want in [(dict(o=0), 1), (dict(o=P + 8), 3), (dict(odt=3), 1), (dict(odt=-1), 1),
                     (dict(lse=P + 2), 3)]:
        assert tree(qa, **kw) == want, kw
    for kw, want in [(dict(lse=0), 1), (dict(acc=0), 1), (dict(acc=P + 2), 3), (dict(S=0), 1),
                     (dict(st=None), 1), (dict(st=strides(-1, 64)), 1)]:
        assert weights(qa, **kw) == want, kw
    for kw, want in [(dict(k=0), 1), (dict(v=P + 8), 3), (dict(dtype=2), 1), (dict(T=0), 1),
                     (dict(T=65), 1), (dict(lens=0), 1), (dict(n=P + 1), 3),
                     (dict(ks=strides(8, 8, 4)), 3), (dict(vs=strides(8, -8, 8)), 1)]:
        assert append(qa, **kw) == want, kw
    assert append(qa, cache(qa, kv_dtype=0, k_scale=0, v_scale=0), dtype=1) == 1
    for kw, want in [(dict(M=-1), 1), (dict(M=65), 1), (dict(M=0), 0), (dict(idx=0), 1),
                     (dict(idx=P + 2), 3), (dict(n=P + 2), 3), (dict(base=P + 1), 3), (dict(acc=P), 1),
                     (dict(ao=P), 1), (dict(acc=P, ao=P, S=64, SO=64), 1), (dict(ot=2 * P, om=0), 1),
                     (dict(ot=P + 2, om=4), 3), (dict(ist=strides(-1, 0)), 1)]:
        assert compact(qa, **kw) == want, kw
    for kw, want in [(dict(keep=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1),
                     (dict(sinks=3, recent=3), 1), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 1),
                     (dict(acc=0), 1), (dict(ao=0), 1), (dict(idx=0), 1), (dict(new=0), 1),
                     (dict(new=P + 2), 3), (dict(lens=0), 1), (dict(SO=4), 1), (dict(keep=65, SO=65), 1)]:
        assert evict(qa, **kw) == want, kw


def test_status_string(qa):
    assert "range" in qa.sage2_status_string(8) and qa.STATUS[8] == "SAGE2_ERR_BAD_INDEX"


def test_binding_refuses_host_tensors(qa):
    c = qa.sage2_cache_alloc(4, 2, 16, 64, torch.float8_e4m3fn, device="cpu")
    assert set(c) == {"k", "v", "k_scale", "v_scale"} and c["k_scale"].shape == (4, 2, 16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        qa.sage2_cache_append(x, x, c, table, lens)
    with pytest.raises(ValueError):
        qa.sage2_attn_tree(x, c, table, lens)
    with pytest.raises(ValueError):
        qa.sage2_cache_alloc(4, 2, 16, 64, torch.float32, device="cpu")
