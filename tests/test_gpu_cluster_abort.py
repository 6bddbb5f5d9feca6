"""A cluster whose CTAs add their partial sums stores nothing once one of them has given up."""
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4


@pytest.mark.gpu
def test_every_cta_sees_one_that_gave_up():
    status = torch.full((9,), -1, dtype=torch.int32, device=G.DEV)
    for rank in range(-1, 8):
        status.fill_(-1)
        nv4.nv4_selftest_cluster(rank, status)
        assert status.tolist() == [0 if rank < 0 else nv4.FLAG_TIMEOUT] * 8 + [-1]


def test_refusals():
    from nvfp4_block_numerics_b200.build import build_library

    build_library()
    L = nv4.lib()
    assert L.nv4_selftest_cluster(8, 0x1000, None) == 6 and L.nv4_selftest_cluster(-2, 0x1000, None) == 6
    assert L.nv4_selftest_cluster(0, None, None) == 1
