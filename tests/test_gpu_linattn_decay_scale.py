"""Scales far from one, at every strength of decay: the result is linear in
the scale, so the bounds are those of test_gpu_linattn_decay.py.
"""
import numpy as np
import pytest

from test_gpu_linattn_decay import Case, check_backward, check_forward, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** 34, -1e12, 2.0 ** 60, 2.0 ** -60])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,M", [(1, 64, 64), (1, 128, 128), (40, 64, 64)])
def test_large_and_small_scales(B, D, M, dtype, scale):
    decay = [-2.23, -2.2, -1.5, -0.3, -0.001, -2.3, -30.0, 0.0]  # 31 positions of the first two: just above 2^-100
    c = Case(D + M, B, 300, len(decay), D, M, dtype, state=True, decay=decay)
    c.scale = scale
    out = check_forward(c)
    assert np.all(np.isfinite(host(out)))
    check_backward(c)
