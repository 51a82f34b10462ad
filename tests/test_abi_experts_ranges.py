"""Expert ranges that the row order refuses on the host (CPU only)."""
import pytest

import nvfp4_block_scaled_07_amd as nv
from tests.test_abi_experts import FAKE, NULL, SHAPE, UNSUPPORTED, _sort

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("first,E", [(TOP, 2), (TOP, 8), (TOP - 6, 8), (TOP - 65533, 65535), (TOP, TOP), (2, TOP)])
def test_ranges_past_the_largest_id(first, E):
    # id - first wraps: -2^31 - (2^31 - 1) is 1, and would count as an expert of the range
    assert (-2 ** 31 - TOP) % 2 ** 32 == 1
    assert _sort(first=first, E=E) == SHAPE and "first" in nv.nvfp4_last_error()


def test_ranges_up_to_the_largest_id():
    # the largest that is taken: checks go on to what comes next
    for first, E in ((TOP - 7, 8), (TOP, 1), (TOP - 65534, 65535), (0, 65535)):
        assert _sort(first=first, E=E, ids=None) == NULL
        assert min((-2 ** 31 - first) % 2 ** 32, (-1 - first) % 2 ** 32) >= E
    assert _sort(first=1, E=TOP) == UNSUPPORTED
