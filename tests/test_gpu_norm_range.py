"""Layer norm at the ends of fp32's range: statistics of rows whose sums are
infinite, and gradients of rows far from zero."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe
from oracle import block_ops as ob
from tests.test_gpu_block_ops import dev, norm_tol, np64, run_norm, within

pytestmark = pytest.mark.gpu

INF = float("inf")
# widths of every layout: lanes of a warp, several warps, two chunks a thread, one by one, above 8192
WIDTHS = [8, 24, 31, 256, 300, 640, 1037, 1100, 4096, 4104, 8192, 9001, 9004, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_statistics_of_infinite_sums(d, x, many):
    """many: rows enough for two to a group of threads, where that form exists."""
    if many and d > 4096:
        pytest.skip("one row a group whatever the number")
    r = np.random.default_rng([d, 31])
    rows = (1776 * max(1, 2048 // d) + 9) if many else 9
    h = r.standard_normal((rows, d))
    h[1, 3], h[3, d - 1] = INF, -INF            # one infinite element
    h[4, 0], h[4, d - 1] = INF, -INF            # two of different signs
    h[5, d // 2] = np.nan
    h[6] = 1e20 * (1 - 2.0 * (np.arange(d) % 2))   # finite, squared deviations past the range
    h[7] = 3e38                                 # finite, the sum past the range
    G, B = dev(1 + r.standard_normal(d) * 0.3), dev(r.standard_normal(d))
    X, out, _, mean, rstd = run_norm(h, G, B, x=x, y="f32")
    h = np64(X)
    y, mu, rs = np64(out), np64(mean), np64(rstd)
    assert mu[1] == INF and mu[3] == -INF and np.isnan(mu[[4, 5]]).all()
    assert np.isnan(rs[[1, 3, 4, 5]]).all() and np.isnan(y[[1, 3, 4, 5]]).all()
    assert rs[6] == 0 and np.array_equal(y[6], np64(B))
    assert mu[7] == INF and rs[7] == 0 and np.isnan(y[7]).all()
    fine = np.setdiff1d(np.arange(rows), [1, 3, 4, 5, 6, 7])
    ry, rmu, rrs = ob.layer_norm(h[fine], np64(G), np64(B))
    tol, e_mu, e_rs = norm_tol(h[fine], ry, rmu, rrs, np64(G), np64(B), "f32")
    within(y[fine], ry, tol, "y")
    within(mu[fine], rmu, e_mu + 2.0 ** -24 * np.abs(rmu), "mean")
    within(rs[fine], rrs, e_rs + 2.0 ** -22 * rrs, "rstd")


@pytest.mark.parametrize("eps", [1.4e-45, 4.2e-45, 1e-44, 1e-40, 1e-38, 1e-5, 1e30])
def test_rstd_of_constant_rows_is_the_root_of_eps(eps):
    """Subnormal eps among them; each rstd to the few roundings of the root."""
    eps = float(np.float32(eps))
    cfg = moe.make_norm_config(5, 96, eps, x="f32")
    X, Y = torch.full((5, 96), 0.75, device="cuda"), torch.empty(5, 96, device="cuda")
    mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    moe.moe_layer_norm_forward(cfg, X, None, None, Y, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    assert bool((mean == 0.75).all()) and not Y.any()
    within(rstd, np.full(5, eps ** -0.5), 8 * 2.0 ** -24 * eps ** -0.5, "rstd")
