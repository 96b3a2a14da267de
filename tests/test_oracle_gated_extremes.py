"""The gated block's oracle at infinities and NaN.  CPU only."""
import numpy as np

from oracle import gated as OG


def test_relu():
    x = np.array([-np.inf, -1e300, -0.0, 0.0, 1e300, np.inf, np.nan])
    a, da = OG.act(x, "relu")
    assert np.array_equal(a, [0, 0, 0, 0, 1e300, np.inf, np.nan], equal_nan=True)
    assert np.array_equal(da, [0, 0, 0, 0, 1, 1, 0])
