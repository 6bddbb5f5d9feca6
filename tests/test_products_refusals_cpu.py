"""Further refusals of the products on FP4 weights (no GPU: the checks come before any launch)."""
import pytest

FAKE = 0x1000


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_numerics_b200 import binding
    from nvfp4_block_numerics_b200.build import build_library

    build_library()
    return binding.lib()


def test_linear_w4a16_scale_pointer(L):
    """d_s2 is read as a float: refused where that would be misaligned, as the experts' scales are."""
    for T in (4, 40):
        for off in (1, 2, 3):
            assert L.nv4_linear_w4a16(FAKE, 0, T, 64, 64, FAKE, FAKE, FAKE + off, 8, 0, FAKE, 8, None, None) == 3
