"""Layer norm with one operand at a time off the alignment of the others, under
the element-wise bounds of the suite: vectors, single elements and whole-row
copies at widths of every layout, above 8192 columns too."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe
from oracle import block_ops as ob
from tests.test_gpu_block_ops import DT, HALF, TINY, U, dev, norm_bwd_tol, norm_tol, np64, within, ws_of

pytestmark = pytest.mark.gpu

ROWS = 19
WIDTHS = [64, 260, 512, 1037, 4096, 5120, 8192, 9000, 9001, 16384]
OFFS = [1, 2, 4, 8]
TYPES = [("f32", "bf16", "f32"), ("bf16", "f32", "bf16"), ("f16", "f16", "f16")]   # x (and sum, dx), y or dy, weights


def shifted(t, off):
    """A copy that starts off elements into its buffer, whose start is aligned to 256 bytes."""
    buf = torch.zeros(t.numel() + off, dtype=t.dtype, device=t.device)
    buf[off:].copy_(t.reshape(-1))
    return buf[off:].view(t.shape)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("x,y,w", TYPES)
@pytest.mark.parametrize("name", ["x", "add", "gamma", "beta", "y", "sum", "mean", "rstd", "all"])
def test_forward(d, x, y, w, name):
    r = np.random.default_rng([d, 41])
    t = dict(x=dev(r.standard_normal((ROWS, d)) * 2 + 1, DT[x]), add=dev(r.standard_normal((ROWS, d)), DT[y]),
             gamma=dev(1 + 0.3 * r.standard_normal(d), DT[w]), beta=dev(r.standard_normal(d), DT[w]),
             y=torch.zeros(ROWS, d, device="cuda", dtype=DT[y]), sum=torch.zeros(ROWS, d, device="cuda", dtype=DT[x]),
             mean=torch.zeros(ROWS, device="cuda"), rstd=torch.zeros(ROWS, device="cuda"))
    cfg = moe.make_norm_config(ROWS, d, x=x, y=y, w=w, add=y)
    h0 = np64(t["x"]) + np64(t["add"])
    for off in OFFS:
        s = {k: shifted(v, off) if name in (k, "all") else v.clone() for k, v in t.items()}
        moe.moe_layer_norm_forward(cfg, s["x"], s["gamma"], s["beta"], s["y"], add=s["add"], sum=s["sum"],
                                   mean=s["mean"], rstd=s["rstd"])
        torch.cuda.synchronize()
        within(s["sum"], h0, HALF[x] * np.abs(h0) * (1 + 2 * U) + U * np.abs(h0) + TINY[x], "sum")
        h = np64(s["sum"])
        ref, mu, rs = ob.layer_norm(h, np64(t["gamma"]), np64(t["beta"]))
        tol, e_mu, e_rs = norm_tol(h, ref, mu, rs, np64(t["gamma"]), np64(t["beta"]), y)
        within(s["y"], ref, tol, "y")
        within(s["mean"], mu, e_mu + U * np.abs(mu), "mean")
        within(s["rstd"], rs, e_rs + 4 * U * rs, "rstd")


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("x,dy,w", TYPES)
@pytest.mark.parametrize("name", ["dy", "x", "mean", "rstd", "gamma", "dsum", "dx", "dgamma", "dbeta", "all"])
def test_backward(d, x, dy, w, name):
    r = np.random.default_rng([d, 42])
    X = dev(r.standard_normal((ROWS, d)) * 2 + 1, DT[x])
    _, mu, rs = ob.layer_norm(np64(X))
    t = dict(dy=dev(r.standard_normal((ROWS, d)) * 0.1, DT[dy]), x=X, mean=dev(mu), rstd=dev(rs),
             gamma=dev(1 + 0.3 * r.standard_normal(d), DT[w]), dsum=dev(r.standard_normal((ROWS, d)) * 0.1, DT[x]),
             dx=torch.zeros(ROWS, d, device="cuda", dtype=DT[x]), dgamma=torch.zeros(d, device="cuda"),
             dbeta=torch.zeros(d, device="cuda"))
    mu, rs, g, ds, dyn = (np64(t[k]) for k in ("mean", "rstd", "gamma", "dsum", "dy"))
    rdx, rdg, rdb = ob.layer_norm_backward(dyn, np64(X), mu, rs, g, ds)
    xh = (np64(X) - mu[:, None]) * rs[:, None]
    tdx, tdg, tdb = norm_bwd_tol(dyn, xh, rs, g, ds, rdx, x, ROWS + 16)
    cfg = moe.make_norm_config(ROWS, d, x=x, w=w, dy=dy)
    ws = ws_of(moe.moe_layer_norm_workspace_size(cfg))
    for off in OFFS:
        s = {k: shifted(v, off) if name in (k, "all") else v.clone() for k, v in t.items()}
        moe.moe_layer_norm_backward(cfg, s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], s["dx"], s["dgamma"],
                                    s["dbeta"], ws, dsum=s["dsum"])
        torch.cuda.synchronize()
        within(s["dx"], rdx, tdx, "dx")
        within(s["dgamma"], rdg, tdg + U * np.abs(rdg), "dgamma")
        within(s["dbeta"], rdb, tdb + U * np.abs(rdb), "dbeta")
