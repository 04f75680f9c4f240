"""Norm and rotation of many tokens at every number of heads that a lane takes at a time (needs a GB300)."""
import pytest

from test_gpu_norm_rope import Q, test_matches_the_oracle as _matches  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu


# eight groups of lanes for heads of 128: 2, 3, 4, 5, 6, 7, 8, 9 heads a lane, and two CTAs a token
@pytest.mark.parametrize("heads", [(14, 2), (17, 7), (28, 4), (32, 8), (40, 3), (52, 4), (56, 5), (64, 8), (96, 8)])
def test_heads_of_a_lane(Q, heads):  # noqa: F811
    tokens = 2 * 16 * 152 * 8 // sum(heads)
    _matches(Q, (min(tokens, 1400), *heads, 128, 128), False, False, True)


@pytest.mark.parametrize("dim,heads", [(64, (33, 5)), (256, (16, 8))])
def test_other_head_sizes(Q, dim, heads):  # noqa: F811
    _matches(Q, (900, *heads, dim, dim // 2), True, True, True)
