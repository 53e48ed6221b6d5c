"""The oracle's clipping factor at the ends of its range."""
import math

from oracle import ops


def test_factor_at_the_limits():
    inf, nan = math.inf, math.nan
    for norm, limit, eps, want in [(inf, inf, 1e-6, 1.0), (inf, 1.0, 1e-6, 0.0), (inf, 0.0, 1e-6, 0.0), (0.0, 0.0, 0.0, 1.0),
                                   (0.0, 0.0, 1e-6, 0.0), (0.0, 1.0, 0.0, 1.0), (5.0, inf, 1e-6, 1.0),
                                   (4.0, 2.0, 0.0, 0.5)]:
        assert ops.clip_factor(norm, limit, eps) == want, (norm, limit, eps)
    assert all(math.isnan(ops.clip_factor(nan, limit)) for limit in (0.0, 1.0, inf))
