"""The scales that sq_paged_attention refuses, before anything touches a GPU: those
whose product with log2 e is not finite."""
import math

import pytest

from test_decoder_abi import A, INVALID, OK, lib  # noqa: F401  (a fixture)


@pytest.mark.parametrize("scale,want", [
    (2.0 ** 127 * (1 + 2.0 ** -23), INVALID), (-3.4e38, INVALID), (math.inf, INVALID),
    (-math.inf, INVALID), (math.nan, INVALID), (2.0 ** 127, OK), (-2.0 ** 127, OK), (0.0, OK),
    (1e-45, OK),
])
def test_scales(lib, scale, want):  # noqa: F811
    # (no tokens: a scale that is not refused ends the call there)
    assert lib.sq_paged_attention(A, 512, 0, 8, 4, 64, A, A, 0, 8, 16, A, 4, A, A, 2, 1, None, 0,
                                  scale, A, A, 1 << 30, None) == want
