"""The failure path of the bounded waits in the layer norm's backward, reached
without a GPU fault: the test hook moe_testing_set_norm_wait keeps rounds of
rows from being copied, with a 1 ms limit on the waits for them.  The call must
return, say so (MOE_DEV_TIMEOUT where there are stats; NaN in what it missed
with and without them) and leave the context usable."""
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe

pytestmark = pytest.mark.gpu


def make(rows, d, x):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[x]
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + d)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
    X, DY, DS, G = rnd(rows, d).to(dt), rnd(rows, d), rnd(rows, d).to(dt), 1 + 0.2 * rnd(d)
    mean, rstd = X.float().mean(1), torch.rsqrt(X.float().var(1, unbiased=False) + 1e-5)
    cfg = moe.make_norm_config(rows, d, x=x)
    ws = torch.empty(moe.moe_layer_norm_workspace_size(cfg), dtype=torch.uint8, device="cuda")

    def run(stats=None):
        dx = torch.full((rows, d), 7.0, device="cuda").to(dt)
        dg, db = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
        moe.moe_layer_norm_backward(cfg, DY, X, mean, rstd, G, dx, dg, db, ws, dsum=DS, stats=stats)
        torch.cuda.synchronize()
        return dx, dg, db
    return run


# one and two chunks a thread, one and several rows a block, a layout that is filled, one that is not, an odd width
@pytest.mark.parametrize("rows,d", [(12000, 256), (20000, 100), (2000, 1037), (1500, 4096), (1500, 520), (700, 8192),
                                    (5, 64)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("kept", [0, 1])
def test_rows_that_never_come(rows, d, x, kept):
    run = make(rows, d, x)
    want = run()
    assert all(torch.isfinite(t).all() for t in want)
    stats = torch.zeros(moe.STATS_BYTES, dtype=torch.uint8, device="cuda")
    moe.moe_testing_set_norm_wait(1_000_000, kept)
    try:
        told, silent = run(stats), run()
    finally:
        moe.moe_testing_set_norm_wait(0, -1)
    # rows of even widths that are no whole 16-byte pieces are read by plain loads: no copies, nothing to wait for
    waits = d % 4 != 0 or d * (4 if x == "f32" else 2) % 16 == 0
    lost = 0
    for dx, dg, db in (told, silent):
        bad = torch.isnan(dx).all(1)
        lost = int(bad.sum())
        assert torch.equal(torch.isnan(dx).any(1), bad)            # a row is lost as a whole
        assert torch.equal(dx[~bad], want[0][~bad])                # or right
        if lost:
            assert torch.isnan(dg).all() and torch.isnan(db).all()
        else:
            assert torch.equal(dg, want[1]) and torch.equal(db, want[2])
    if not waits or (kept == 1 and rows == 5):
        assert lost == 0
    else:
        assert lost == rows if kept == 0 else 0 < lost < rows
    assert moe.read_stats(stats)["status"] == (moe.MOE_DEV_TIMEOUT if lost else 0)
    for a, b in zip(run(stats), want):   # the limits back to the defaults: a clean call
        assert torch.equal(a, b)


def test_hook_rejects_bad_values():
    with pytest.raises(moe.MoeError):
        moe.moe_testing_set_norm_wait(61 * 10**9, -1)
    with pytest.raises(moe.MoeError):
        moe.moe_testing_set_norm_wait(0, -2)
    moe.moe_testing_set_norm_wait(0, -1)
