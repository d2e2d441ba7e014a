"""GPU parity of the paged attention in every instantiation: each width of the kernels (and D between
two of them) with each block of heads (one, up to four, eight and sixteen, and two blocks), as a cluster a unit,
as equal stretches of the tiles with joined parts, and with several units to a CTA, whose queries then take one
another's place. Bounds as in test_parity_paged_attention."""
import pytest

from tests import gpu_util as gu
from tests.test_parity_paged_attention import LINE, TYPES, check

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

GROUPS = [1, 3, 5, 8, 9, 12, 16, 17]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 80, 96, 128, 160, 192, 200, 256])
@pytest.mark.parametrize("group", GROUPS)
def test_clusters_and_joined_parts(dtype, D, group):
    check([130, 1, 77], 2 * group, 2, D, 16, dtype)
    check([130, 1, 77], 2 * group, 2, D, 16, dtype, width=LINE)
    check([700], group, 1, D, 24, dtype, layout="heads", window=301)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 80, 96, 128, 160, 192, 200, 256])
@pytest.mark.parametrize("group", GROUPS)
def test_several_units_to_a_cta(dtype, D, group):
    # 1000 units at least, for 456 CTAs at most
    check([1 + i * 7 % 40 for i in range(1000)], group, 1, D, 16, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [63, 131, 190, 255])
@pytest.mark.parametrize("group", [1, 8, 9, 16])
def test_heads_off_16_bytes(dtype, D, group):
    check([130, 0, 77], 2 * group, 2, D, 16, dtype)
    check([130, 0, 77] + [9] * 300, 2 * group, 2, D, 16, dtype)
