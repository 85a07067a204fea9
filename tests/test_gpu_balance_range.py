"""Balance loss of sigmoid scores far below zero: shares of the sum stay right
where the sigmoids themselves leave fp32's range."""
import numpy as np
import pytest

from tests.test_gpu_block_ops import check_balance

pytestmark = pytest.mark.gpu


# the single block and the three kernels, vectors and single scores, one token and several to a warp
@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (30, 255, 3), (3000, 12, 2), (2000, 64, 6), (700, 190, 4), (1500, 256, 8)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("top", [-16.0, -21.0, -40.0, -54.0, -60.0, -90.0])
def test_sigmoid_scores_far_below_zero(T, E, k, dt, top):
    """Each token's largest score near top, the others down to 60 below it; experts chosen without regard to them, so
    that the loss is a sum of small shares, too."""
    r = np.random.default_rng([T, E, int(-top)])
    z = top - 60 * r.random((T, E))
    z[np.arange(T), r.integers(0, E, T)] = top
    topk = np.argsort(z, 1)[:, :k].astype(np.int32)   # the smallest
    check_balance(z, topk, k, score="sigmoid", dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_far_and_ordinary_tokens_side_by_side(dt):
    """Tokens of one warp, some far below zero and some not, do not disturb each other."""
    r = np.random.default_rng(7)
    for T, E in ((64, 16), (5000, 12), (5000, 16)):
        z = r.standard_normal((T, E))
        z[r.random(T) < 0.4] -= 60.0
        z[r.random(T) < 0.1] = -np.inf
        topk = r.integers(0, E, (T, 2)).astype(np.int32)
        check_balance(z, topk, 2, score="sigmoid", dt=dt)
