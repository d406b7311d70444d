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
