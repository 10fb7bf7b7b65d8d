"""Inputs that tests seed with hash() of their parameters are the same in each run,
texts among the parameters or not."""
import pytest
import torch


def gen(*key):
    return torch.Generator().manual_seed(hash(key) & 0x7FFFFFFF)


@pytest.mark.parametrize("key,seed", [((64, "skewed"), 1502262164), ((64, 5000, "uniform"), 1577092809), (("one",), 1349677485)])
def test_texts_among_the_parameters(key, seed):
    assert gen(*key).initial_seed() == seed


def test_numbers_keep_the_seeds_they_had():
    for key in ((1,), (3, 4096), (5000, 35, 93, 3, 1)):
        assert gen(*key).initial_seed() == key.__hash__() & 0x7FFFFFFF
