"""The cache's oracle against its contract, value by value (CPU)."""
import numpy as np

from oracle import cache_oracle as O


def test_a_quotient_past_float32_saturates_and_only_x_makes_nan():
    """y = x / scale; a scale is at most 448, a code at most 6; a group with a NaN or an infinity among
    its x, and no other, has a NaN scale."""
    x = np.zeros((4, 16))
    x[0, :3] = 3.3e38, -3.3e38, 1.0
    x[1, :2] = np.inf, 1.0
    x[2, :2] = np.nan, 1.0
    x[3, :2] = 2688.0, 448.0
    for scale in (1.0, 0.25, 2.0**-90):
        codes, s8 = O.encode(x.reshape(1, 64), scale)
        codes = codes.reshape(4, 16)
        assert list(s8[0, 1:3]) == [0x7F, 0x7F] and not codes[1:3].any()
        assert s8[0, 0] == 126 and list(codes[0, :2]) == [7, 15]
        assert s8[0, 3] == 126 and codes[3, 0] == 7
    assert codes[0, 2] == 7 and O.encode(x.reshape(1, 64), 1.0)[0].reshape(4, 16)[3, 1] == 2
