"""Host-side refusals of tallies and lengths that a call would write to twice or read while it writes them (no GPU
needed: the checks come before anything touches CUDA)."""
import pytest

from tests.test_cache_abi import P, append, cache, compact, evict, qa, strides, tree, weights  # noqa: F401


def test_lengths_are_not_written_over(qa):
    assert evict(qa, new=P, lens=P) == 1


@pytest.mark.parametrize("st", [(128, 63), (127, 64), (64, 64), (64, 128 - 1), (63, 128), (0, 64), (128, 0), (2 ** 62, 1),
                                (1, 2 ** 62)])
def test_tallies_that_overlap(qa, st):
    """Two heads of a written tally share a slot: 2 sequences of 2 heads, 64 slots each."""
    assert weights(qa, st=strides(*st)) == 1
    assert evict(qa, aost=strides(*st), ao=2 * P, new=2 * P) == 1
    assert compact(qa, acc=P, ao=2 * P, ast=strides(128, 64), aost=strides(*st), S=64, SO=64) == 1


def test_tallies_moved_onto_themselves(qa):
    """acc_out may be acc in place and laid out alike, nowhere else."""
    a = dict(acc=P, ao=P, ast=strides(128, 64), S=64, SO=64)
    assert compact(qa, aost=strides(64, 128), **a) == 1
    assert compact(qa, aost=strides(128, 64), ot=2 * P, om=4, **a) == 1
    assert evict(qa, aost=strides(64, 128), new=2 * P) == 1
    assert evict(qa, ot=2 * P, om=4, new=2 * P) == 1


def test_error_word_of_the_device_asked_for(qa, monkeypatch):
    """The error word is the current device's in the library: the binding makes the device that is asked for
    current around the call, as the cache entries do for the device of their tensors."""
    import torch
    now, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = torch.device(dev).index

        def __enter__(self):
            self.old, now[0] = now[0], self.dev

        def __exit__(self, *a):
            now[0] = self.old

    class Lib:
        def sage2_check_device_error(self, st):
            seen.append((now[0], st.value))
            return 8

    class Stream:
        def __init__(self, dev):
            self.cuda_stream = 100 + torch.device(dev).index

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(qa, "lib", Lib)
    assert qa.sage2_check_device_error("cuda:1") == 8 and qa.sage2_check_device_error() == 8
    assert seen == [(1, 101), (0, 100)] and now == [0]
