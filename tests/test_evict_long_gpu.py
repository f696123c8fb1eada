"""Eviction in tables of more rows than the select keeps keys of (49,152): sequences on both
sides of that in one batch."""
import pytest
import torch

from paged_util import DEV, gen
from test_evict_gpu import Cache, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,planes,in_place", [([300, 49152, 49153, 60, 65536, 5000], 2, True), ([49153, 400], 1, False),
                                                     ([49151, 65535, 7], 3, True)])
def test_sequences_on_both_sides(cuda_lib, lengths, planes, in_place):
    g = gen(len(lengths))
    # few different masses, so that the last place is a tie of many
    mass = torch.randint(0, 9, (planes, len(lengths), 8192 * 8 + 2), generator=g, device=DEV).float()
    c = Cache(lengths, 8, planes, ik=False, max_pages=8192, mass=mass)
    c.run(cuda_lib, 250, 290, 3, 20, in_place=in_place)
    status(cuda_lib)
    c.check()


def test_keep_more_than_the_keys_kept(cuda_lib):
    c = Cache([65000, 50001, 49999], 8, 1, True, max_pages=8192)
    c.run(cuda_lib, 50000, 50000, 1, 1)
    status(cuda_lib)
    c.check()


def test_many_sequences_a_block(cuda_lib):
    """More sequences than SMs, long and short in turn on each."""
    c = Cache([49200 if b % 40 == 0 else 30 + b % 50 for b in range(400)], 8, 1, True, False, max_pages=6200)
    c.run(cuda_lib, 24, 33, 2, 5)
    status(cuda_lib)
    c.check()
