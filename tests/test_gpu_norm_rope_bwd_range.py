"""The gradients of Q/K RMSNorm + 3D rotation far from values of order one, without
an epsilon that would hide it: groups whose root mean square is very small or very
large.  r^3 alone leaves float32 there (above 7e12 and below 1e-13), the gradient
does not: r u w and x r^3 mean(x u w) are both of the size of r u.

Bounds: those of test_gpu_norm_rope_bwd.py.  They are relative to the terms'
magnitudes, and a float32's relative rounding is the same at every size that is
neither denormal nor infinite.  At |x| of 1e-17 and 1e17 the squares are some 1e-34
and 1e34, and so is r^2 mean(x u w) r at the other end; of a group's smallest elements
a square below 1e-38 is denormal, and loses less than 1e-45 next to a sum above 1e-34."""
import pytest
import torch

from tests.gpu_util import watchdog_clear
from tests.test_gpu_norm_rope_bwd import _check_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    watchdog_clear()


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("x_scale", [1e-17, 1e-14, 1e-12, 1e13, 1e15, 1e17])
def test_small_and_large_groups_without_eps(x_scale, per_token):
    _check_norm(1, (3, 5, 6), 2, 128, (44, 42, 42), 256 if per_token else 128, eps=0.0, x_scale=x_scale)
