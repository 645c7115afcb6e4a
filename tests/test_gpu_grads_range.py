"""Clipping of gradients so large that the factor lies below fp32's normal range."""
import pytest
import torch

from conftest import announce_case
from test_gpu_grads import check_scaled, clip, close_norm, tensors, true_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("max_norm", [1.0, 1e-6, 1e-30])
@pytest.mark.parametrize("std", [1e25, 1e33, 1e36])
@pytest.mark.parametrize("offset", [0, 1])
def test_factors_below_the_normal_range(std, max_norm, offset):
    src, _ = tensors([1000, 7, 8200], ["f32", "bf16"], 3, std, offset)
    src[0][5], src[0][6] = std * 1e-6, 1e-20  # (small elements beside them)
    want = true_norm(src)
    assert want < 3e38
    dst = [torch.empty_like(t) for t in src]
    norm = clip(src, dst, max_norm)
    assert close_norm(norm[0], want)
    check_scaled(src, dst, max_norm / want)
    clip(src, dst, max_norm, norm)
    check_scaled(src, dst, max_norm / float(norm))
    zero = [torch.ones_like(t) for t in src]
    clip(src, zero, 0.0)
    assert all(int(t.count_nonzero()) == 0 for t in zero)
