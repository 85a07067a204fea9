"""Layer norm, balance loss and AdamW step on the device against the float64
oracle (oracle/block_ops.py).

Tolerances are element by element, from the roundings on the way: u = 2^-24
per fp32 operation, at most N of them in a chain (a sum's length along one
thread, its tree, and the formula's steps), and half a step of the output's
type at the end (2^-8 bf16, 2^-11 fp16 of the value; fp16 also 2^-25 where it is
subnormal)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def dev(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dt)


def np64(t):
    return t.detach().cpu().double().numpy()


def ws_of(n):
    return torch.full((max(n, 256),), 0xA5, dtype=torch.uint8, device="cuda")


def within(got, ref, tol, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    err = np.where(np.isnan(ref), 0, np.abs(got - ref))
    over = err - np.broadcast_to(tol, err.shape)
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[i] <= 0, f"{what} at {i}: {got[i]} for {ref[i]}, off by {err[i]:.3e} > {np.broadcast_to(tol, err.shape)[i]:.3e}"


# ------------------------------------------------------------------ layer norm
def run_norm(h, gamma, beta, add=None, x="f32", y=None, w="f32", at="f32", eps=1e-5, stats=True, into_x=False):
    rows, d = h.shape
    cfg = moe.make_norm_config(rows, d, eps, x=x, y=y, w=w, add=at)
    X = dev(h, DT[x])
    out = torch.full((rows, d), float("nan"), device="cuda", dtype=DT[y or x])
    S = None if add is None else (X if into_x else torch.empty_like(X))
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2)) if stats else (None, None)
    moe.moe_layer_norm_forward(cfg, X, gamma, beta, out, add=add, sum=S, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    return X, out, S, mean, rstd


def norm_tol(h, y, mu, r, gamma, beta, yt):
    """N = 128 roundings at most on a path through a row's sums."""
    N = 128 * U
    e_mu = N * np.abs(h).mean(1, keepdims=True)
    c = h - mu[:, None]
    r = r[:, None]
    xh = np.abs(c * r)
    g = 1.0 if gamma is None else np.abs(gamma)
    e = r * e_mu + xh * (N + (e_mu * r) ** 2)
    b = 0.0 if beta is None else np.abs(beta)
    fp = e * g + 4 * U * (xh * g + b)
    return fp + HALF[yt] * (np.abs(y) + fp) + TINY[yt], e_mu[:, 0], np.abs(r[:, 0]) * (N + (e_mu[:, 0] * r[:, 0]) ** 2)


NORMS = [(1, 1), (1, 7), (3, 8), (2, 31), (5, 64), (9, 100), (33, 256), (17, 257), (4, 512), (2, 1000), (3, 1024),
         (2, 2048), (300, 96), (1, 4096), (2, 4097), (6, 4100), (7, 5120), (2, 9004), (2, 7168), (2, 8192), (1, 11111), (2, 16384),
         (1500, 520)]


@pytest.mark.parametrize("rows,d", NORMS)
@pytest.mark.parametrize("x,y,w,at", [("f32", "bf16", "f32", "f32"), ("bf16", "bf16", "bf16", None),
                                      ("f16", "f32", "f32", "f16"), ("bf16", "f16", "f16", "f32")])
def test_norm_forward(rows, d, x, y, w, at):
    r = np.random.default_rng([rows, d])
    h = np64(dev(r.standard_normal((rows, d)) * r.uniform(0.2, 4, (rows, 1)) + r.standard_normal((rows, 1)) * 5, DT[x]))
    G, B = dev(1 + r.standard_normal(d) * 0.3, DT[w]), dev(r.standard_normal(d), DT[w])
    A = None if at is None else dev(r.standard_normal((rows, d)), DT[at])
    X, out, S, mean, rstd = run_norm(h, G, B, A, x, y, w, at or "f32")
    if at is not None:
        within(S, h + np64(A), HALF[x] * np.abs(h + np64(A)) * (1 + 2 * U) + U * np.abs(h + np64(A)) + TINY[x], "sum")
        h = np64(S)   # what is stored is what is normalised
    ref, mu, rs = ob.layer_norm(h, np64(G), np64(B))
    tol, e_mu, e_rs = norm_tol(h, ref, mu, rs, np64(G), np64(B), y)
    within(out, ref, tol, "y")
    within(mean, mu, e_mu + U * np.abs(mu), "mean")
    within(rstd, rs, e_rs + 4 * U * rs, "rstd")


@pytest.mark.parametrize("rows,d", [(1777, 4096), (1779, 2057), (1777, 1100), (14209, 300), (28417, 65), (113665, 24)])
@pytest.mark.parametrize("x,y,w", [("bf16", "bf16", "bf16"), ("f32", "f16", "f32")])
def test_norm_forward_of_many_rows(rows, d, x, y, w):
    """Without an addend, and enough rows for two to a group of threads (an odd one is left over)."""
    r = np.random.default_rng([rows, d, 2])
    h = np64(dev(r.standard_normal((rows, d)) * r.uniform(0.2, 4, (rows, 1)) + r.standard_normal((rows, 1)) * 5, DT[x]))
    G, B = dev(1 + r.standard_normal(d) * 0.3, DT[w]), dev(r.standard_normal(d), DT[w])
    _, out, _, mean, rstd = run_norm(h, G, B, None, x, y, w)
    ref, mu, rs = ob.layer_norm(h, np64(G), np64(B))
    tol, e_mu, e_rs = norm_tol(h, ref, mu, rs, np64(G), np64(B), y)
    within(out, ref, tol, "y")
    within(mean, mu, e_mu + U * np.abs(mu), "mean")
    within(rstd, rs, e_rs + 4 * U * rs, "rstd")


def test_norm_without_weights_and_in_place_sum():
    r = np.random.default_rng(1)
    h, a = np64(dev(r.standard_normal((6, 640)))), dev(r.standard_normal((6, 640)))
    X, out, S, _, _ = run_norm(h, None, None, a, into_x=True, stats=False)
    h2 = np64(X)
    within(X, h + np64(a), U * np.abs(h + np64(a)), "sum in place")
    ref, mu, rs = ob.layer_norm(h2)
    within(out, ref, norm_tol(h2, ref, mu, rs, None, None, "f32")[0], "y")


def test_norm_of_constant_and_huge_offset_rows():
    h = np.full((3, 520), 7.0)
    h[1] = 4096.0 + np.arange(520) % 2      # variance 1/4 on an offset of 2^12
    h[2] = 0.0
    _, out, _, mean, rstd = run_norm(h, None, None)
    ref, mu, rs = ob.layer_norm(h)
    within(out, ref, norm_tol(h, ref, mu, rs, None, None, "f32")[0], "y")
    assert np64(out)[0].any() == False and np64(out)[2].any() == False   # noqa: E712 (exact: the mean is)


def test_norm_keeps_a_bad_row_to_itself():
    r = np.random.default_rng(2)
    for d in (24, 640, 4104):
        h = r.standard_normal((5, d))
        h[1, 3], h[3, d - 1] = np.nan, np.inf
        _, out, _, _, _ = run_norm(h, None, None)
        got = np64(out)
        assert np.isnan(got[[1, 3]]).all() and np.isfinite(got[[0, 2, 4]]).all()


def norm_bwd_tol(dy, xh, rs, gamma, dsum, dx, odt, depth):
    N = 128 * U
    g = dy if gamma is None else dy * gamma
    r = rs[:, None]
    a, b = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    fp = np.abs(r) * (8 * U * (np.abs(g) + a + np.abs(xh) * b) + N * a + np.abs(xh) * N * b)
    if dsum is not None:
        fp = fp + U * (np.abs(dx) + np.abs(dsum))
    n = depth * U
    return fp + HALF[odt] * (np.abs(dx) + fp) + TINY[odt], (n + 4 * U) * np.abs(dy * xh).sum(0), n * np.abs(dy).sum(0)


@pytest.mark.parametrize("rows,d", NORMS + [(4000, 24), (3000, 512), (700, 2048)])
@pytest.mark.parametrize("x,dy,w,dx,res", [("f32", "f32", "f32", "f32", True), ("bf16", "bf16", "bf16", "bf16", False),
                                           ("bf16", "f32", "f32", "f32", True), ("f16", "f16", "f16", "f16", True)])
def test_norm_backward(rows, d, x, dy, w, dx, res):
    r = np.random.default_rng([rows, d, 1])
    X, DY = dev(r.standard_normal((rows, d)) * 2 + 1, DT[x]), dev(r.standard_normal((rows, d)) * 0.1, DT[dy])
    G, DS = dev(1 + r.standard_normal(d) * 0.3, DT[w]), dev(r.standard_normal((rows, d)) * 0.1, DT[dx]) if res else None
    _, mu, rs = ob.layer_norm(np64(X))
    mean, rstd = dev(mu), dev(rs)
    mu, rs = np64(mean), np64(rstd)
    cfg = moe.make_norm_config(rows, d, x=x, w=w, dy=dy, dx=dx)
    out = torch.full((rows, d), float("nan"), device="cuda", dtype=DT[dx])
    dg, db = (torch.full((d,), float("nan"), device="cuda") for _ in range(2))
    moe.moe_layer_norm_backward(cfg, DY, X, mean, rstd, G, out, dg, db, ws_of(moe.moe_layer_norm_workspace_size(cfg)),
                                dsum=DS)
    torch.cuda.synchronize()
    dyn, g = np64(DY), np64(G)
    ds = None if DS is None else np64(DS)
    rdx, rdg, rdb = ob.layer_norm_backward(dyn, np64(X), mu, rs, g, ds)
    xh = (np64(X) - mu[:, None]) * rs[:, None]
    # a column's sum: at most every row one after the other
    tdx, tdg, tdb = norm_bwd_tol(dyn, xh, rs, g, ds, rdx, dx, rows + 16)
    within(out, rdx, tdx, "dx")
    within(dg, rdg, tdg + U * np.abs(rdg) + TINY["f32"], "dgamma")
    within(db, rdb, tdb + U * np.abs(rdb) + TINY["f32"], "dbeta")


def test_norm_backward_in_place_and_partial_outputs():
    r = np.random.default_rng(3)
    for rows, d in ((40, 72), (9, 1030)):
        cfg = moe.make_norm_config(rows, d, x="f32", dy="f32", dx="f32")
        X, DY, DS = (dev(r.standard_normal((rows, d))) for _ in range(3))
        _, mu, rs = ob.layer_norm(np64(X))
        mean, rstd = dev(mu), dev(rs)
        ws = ws_of(moe.moe_layer_norm_workspace_size(cfg))
        full = [torch.empty(rows, d, device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
        moe.moe_layer_norm_backward(cfg, DY, X, mean, rstd, None, *full, ws, dsum=DS)
        over_dsum, over_dy = DS.clone(), DY.clone()
        moe.moe_layer_norm_backward(cfg, DY, X, mean, rstd, None, over_dsum, dsum=over_dsum)   # no weights, no ws
        only = torch.empty(d, device="cuda")
        moe.moe_layer_norm_backward(cfg, over_dy, X, mean, rstd, None, over_dy, None, only, ws, dsum=DS)
        torch.cuda.synchronize()
        assert torch.equal(over_dsum, full[0]) and torch.equal(over_dy, full[0]) and torch.equal(only, full[2])


def test_norm_of_no_rows_clears_the_weights_gradient():
    cfg = moe.make_norm_config(0, 40, x="f32")
    e = torch.empty(0, 40, device="cuda")
    dg, db = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    moe.moe_layer_norm_forward(cfg, e, None, None, e)
    z = torch.empty(0, device="cuda")
    moe.moe_layer_norm_backward(cfg, e, e, z, z, None, e, dg, db, ws_of(moe.moe_layer_norm_workspace_size(cfg)))
    assert not dg.any() and not db.any()


@pytest.mark.parametrize("d", [64, 512, 4096])
def test_norm_takes_any_alignment_and_repeats_exactly(d):
    """Operands that start one element into a buffer give the bits of aligned ones, and so does a second call."""
    r = np.random.default_rng(4)
    rows = 37
    cfg = moe.make_norm_config(rows, d, x="bf16", y="f32", w="bf16", dy="bf16", dx="bf16")
    h, dy = r.standard_normal((rows, d)), r.standard_normal((rows, d))
    got = []
    for off in (0, 0, 1, 3, 4):
        cut = lambda a, dt, off=off: torch.cat([torch.zeros(off, device="cuda", dtype=dt), dev(a, dt).view(-1)])[off:]  # noqa: E731, E501
        X, DY, G = cut(h, torch.bfloat16), cut(dy, torch.bfloat16), cut(np.linspace(0.5, 2, d), torch.bfloat16)
        Y, DX = cut(h * 0, torch.float32), cut(h * 0, torch.bfloat16)
        mean, rstd, dg, db = (torch.empty(n, device="cuda") for n in (rows, rows, d, d))
        moe.moe_layer_norm_forward(cfg, X, G, None, Y, mean=mean, rstd=rstd)
        moe.moe_layer_norm_backward(cfg, DY, X, mean, rstd, G, DX, dg, db, ws_of(moe.moe_layer_norm_workspace_size(cfg)))
        got.append([t.clone() for t in (Y, mean, rstd, DX, dg, db)])
    for a, b in zip(got[0], got[1]):
        assert torch.equal(a, b)
    for other in got[2:]:   # another order of the sums: the same values to a few roundings
        for a, b in zip(got[0], other):
            assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(a.float().abs().max())


# ---------------------------------------------------------------- balance loss
def run_balance(z, topk, k, S=1, off=None, mask=None, score="softmax", dt="f32", coef=None, counts=None, grad=True):
    T, E = z.shape
    cfg = moe.make_balance_config(T, E, k, S, score, dt)
    given = counts is not None
    C = dev(counts, torch.int32) if given else torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    loss, dz = torch.full((1,), -7.0, device="cuda"), torch.full((T, E), -7.0, device="cuda").to(DT[dt])
    stats = torch.zeros(moe.STATS_BYTES, dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(cfg, dev(z, DT[dt]), None if given else dev(topk, torch.int32), C, loss,
                         ws_of(moe.moe_balance_workspace_size(cfg)),
                         seq_offsets=None if off is None else dev(off, torch.int32),
                         mask=None if mask is None else dev(mask, torch.uint8),
                         coef=None if coef is None else torch.tensor(coef, device="cuda"),
                         dscores=dz if grad else None, stats=stats)
    torch.cuda.synchronize()
    return float(loss), C.cpu().numpy().reshape(S, E), np64(dz), moe.read_stats(stats)["status"]


def check_balance(z, topk, k, S=1, off=None, mask=None, score="softmax", dt="f32", coef=0.3, counts=None):
    T, E = z.shape
    z = np64(dev(z, DT[dt])).reshape(T, E)
    loss, C, dz, status = run_balance(z, topk, k, S, off, mask, score, dt, coef, counts)
    rl, rc, rdz = ob.balance(z, topk, k, E, off, mask, score, float(np.float32(coef)), counts)
    assert status == 0 and np.array_equal(C, rc)
    # p: the exponent's argument is off by u times its size, exp and its sum by a chain of at most 64 roundings
    fin = np.where(np.isfinite(z), z, 0)
    live = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    span = np.abs(fin[live]).max() * 2 if live.any() else 0.0
    n = (span + 64) * U
    assert abs(loss - rl) <= 4 * n * abs(rl) + 1e-30, (loss, rl)
    tol = np.zeros((T, E))
    offs = np.array([0, T]) if off is None else np.asarray(off)
    keep = [np.arange(offs[s], offs[s + 1])[live[offs[s]:offs[s + 1]]] for s in range(S)]
    G = max(1, sum(len(u) > 0 for u in keep))
    for s, u in enumerate(keep):
        if len(u) and rc[s].sum():
            p, f = ob.probabilities(z[u], score), E * rc[s] / rc[s].sum()
            slope = 1.0 if score == "softmax" else 1 / (1 + np.exp(np.minimum(z[u], 700)))
            tol[u] = 4 * n * coef / (G * len(u)) * p * (f + (p @ f)[:, None]) * slope
    # sums of terms below the smallest normal number lose at most its step; exp flushes there
    within(dz, rdz, tol + HALF[dt] * (np.abs(rdz) + tol) + 2.0 ** -126 * E, "dscores")
    return loss, C, dz


def router(r, T, E, k):
    z = r.standard_normal((T, E)) * 1.5 - 0.4 * np.log1p(np.arange(E))
    return z, np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (5, 3, 1), (17, 5, 3), (100, 8, 2), (257, 16, 4),
                                   (300, 31, 5), (129, 32, 2), (500, 33, 6), (1000, 64, 6), (333, 65, 1),
                                   (400, 100, 8), (600, 128, 8), (200, 200, 7), (2049, 255, 2), (777, 256, 8),
                                   (20000, 12, 2)])
@pytest.mark.parametrize("score,dt", [("softmax", "f32"), ("sigmoid", "bf16"), ("sigmoid", "f32"), ("softmax", "bf16")])
def test_balance(T, E, k, score, dt):
    r = np.random.default_rng([T, E])
    check_balance(*router(r, T, E, k), k, score=score, dt=dt)


@pytest.mark.parametrize("T,E,k", [(80000, 16, 2), (80001, 12, 2), (80000, 10, 2), (80003, 13, 1), (40000, 24, 3),
                                   (40000, 28, 3), (5000, 256, 8), (5001, 255, 8), (5000, 180, 4), (5003, 190, 3)])
@pytest.mark.parametrize("score,dt", [("softmax", "f32"), ("sigmoid", "bf16"), ("sigmoid", "f32"), ("softmax", "bf16")])
def test_balance_of_many_tokens(T, E, k, score, dt):
    """Tokens enough for every warp: up to 16 experts to a lane, few lanes to a token."""
    r = np.random.default_rng([T, E, 1])
    off = np.array([0, T // 3, T // 3, T - 7, T], np.int32)
    mask = (r.random(T) > 0.1).astype(np.uint8)
    check_balance(*router(r, T, E, k), k, S=4, off=off, mask=mask, score=score, dt=dt)


@pytest.mark.parametrize("T,E,k,S", [(40, 8, 2, 40), (64, 4, 1, 100), (1000, 16, 2, 7), (3000, 64, 6, 33),
                                     (5000, 20, 3, 900), (4096, 256, 8, 3)])
@pytest.mark.parametrize("score,dt", [("softmax", "f32"), ("sigmoid", "bf16")])
def test_balance_of_ragged_padded_sequences(T, E, k, S, score, dt):
    """Empty sequences, tokens before the first and behind the last one, sequences all of padding; what is masked
    or outside holds NaN scores and wild indices, which are not looked at."""
    r = np.random.default_rng([T, S])
    off = np.sort(r.integers(T // 10, T - T // 10, S + 1)).astype(np.int32)
    mask = (r.random(T) > 0.25).astype(np.uint8)
    for s in range(0, S, 3):
        mask[off[s]:off[s + 1]] = 0
    z, topk = router(r, T, E, k)
    dead = (mask == 0) | (np.arange(T) < off[0]) | (np.arange(T) >= off[-1])
    zz, tt = z.copy(), topk.copy()
    zz[dead], tt[dead] = np.nan, 1 << 30
    z[dead] = 0
    loss, C, dz = check_balance(z, topk, k, S, off, mask, score, dt)
    loss2, C2, dz2, status = run_balance(zz, tt, k, S, off, mask, score, dt, 0.3)
    assert status == 0 and loss2 == loss and np.array_equal(C, C2) and np.array_equal(dz, dz2)
    assert not dz[dead].any()


def test_balance_of_nothing():
    for T, mask in ((0, None), (50, np.zeros(50, np.uint8))):
        z, topk = np.zeros((T, 8)), np.zeros((T, 2), np.int32)
        loss, C, dz, status = run_balance(z, topk, 2, mask=mask)
        assert loss == 0 and not C.any() and not dz.any() and status == 0
    # counts that are given stay as they are
    loss, C, dz, _ = run_balance(np.zeros((0, 8)), None, 2, counts=np.arange(8)[None])
    assert loss == 0 and C.tolist() == [list(range(8))]


def test_balance_extreme_scores():
    big = 3.0e38
    for score in ("softmax", "sigmoid"):
        z = np.array([[0.0, -np.inf, 1.0, -np.inf], [-np.inf] * 4, [200.0, 199.0, 0.0, -200.0], [-big, -big, -big, 0.0],
                      [-90.0, -95.0, -100.0, -200.0], [-big, -big, -big, -big]], np.float32)
        topk = np.argsort(-z, 1, kind="stable")[:, :1].astype(np.int32)
        loss, C, dz, status = run_balance(z, topk, 1, score=score)
        rl, rc, rdz = ob.balance(z.astype(float), topk, 1, 4, score=score)
        # exp's argument is at most 400 here but where the result is 0 or 1
        assert status == 0 and np.array_equal(C, rc) and abs(loss - rl) <= 500 * 8 * U * rl
        within(dz, rdz, 500 * 8 * U * np.abs(rdz) + 500 * U * 4 / 6 * ob.probabilities(z.astype(float), score)
               + 2.0 ** -120, score)
        bad = np.zeros((3, 4), np.float32)
        bad[1, 2] = np.nan
        loss, _, dz, _ = run_balance(bad, np.zeros((3, 1), np.int32), 1, score=score)
        assert np.isnan(loss) and np.isnan(dz[1]).all() and np.isfinite(dz[[0, 2]]).all()


def test_balance_bad_indices_and_offsets_are_flagged():
    r = np.random.default_rng(8)
    z, topk = router(r, 60, 8, 2)
    topk[3, 1], topk[50, 0] = 8, -1
    loss, C, dz, status = run_balance(z, topk, 2)
    rl, rc, rdz = ob.balance(z, topk, 2, 8)
    assert status == moe.MOE_DEV_BOUNDS and np.array_equal(C, rc) and abs(loss - rl) < 1e-4
    topk = np.zeros((60, 2), np.int32)
    for off in ([0, 70], [5, 3, 60], [-4, 60], [0, -1, 60], [2 ** 31 - 1, -2 ** 31, 7, 60]):
        off = np.array(off, np.int32)
        assert run_balance(z, topk, 2, len(off) - 1, off)[3] == moe.MOE_DEV_BOUNDS


def test_balance_counts_of_two_ranks():
    """Counting alone, the counts added up, then the loss of each part on the common counts."""
    r = np.random.default_rng(9)
    parts = [router(r, T, 16, 2) for T in (300, 170)]
    total = np.zeros((1, 16), np.int64)
    for z, topk in parts:
        cfg = moe.make_balance_config(len(z), 16, 2)
        C = torch.empty(1, 16, dtype=torch.int32, device="cuda")
        moe.moe_balance_loss(cfg, None, dev(topk, torch.int32), C, None, ws_of(moe.moe_balance_workspace_size(cfg)))
        assert np.array_equal(C.cpu().numpy()[0], np.bincount(topk.reshape(-1), minlength=16))
        total += C.cpu().numpy()
    for z, topk in parts:
        check_balance(z, topk, 2, counts=total)


def test_balance_repeats_exactly_and_without_gradient():
    r = np.random.default_rng(10)
    z, topk = router(r, 9000, 64, 2)
    a, b = run_balance(z, topk, 2), run_balance(z, topk, 2)
    assert a[0] == b[0] and np.array_equal(a[2], b[2])
    assert run_balance(z, topk, 2, grad=False)[0] == a[0]


# ----------------------------------------------------------------------- AdamW
LR, B1, B2, EPS = 0.01, 0.9, 0.97, 1e-6


def adam_case(r, n, p, g, bits, master, decay, off=0):
    """One tensor on the device (off elements into its buffers) and its fp64 copies."""
    def cut(a, dt):
        return torch.cat([torch.zeros(off, device="cuda", dtype=dt), dev(a, torch.float32).to(dt)])[off:]
    level = np.repeat(10.0 ** r.uniform(-5, 1, ob.blocks(n)), ob.BLOCK)[:n]
    G = cut(r.standard_normal(n) * level * (r.random(n) > 0.1), DT[g])
    P32 = np.float32(r.standard_normal(n))
    M = cut(P32, torch.float32) if master else None
    Pm = cut(P32, DT[p])
    m0, v0 = np.float32(r.standard_normal(n) * level * 0.3), np.float32(r.random(n) * level ** 2)
    if bits == 32:
        m, v, ms, vs = cut(m0, torch.float32), cut(v0, torch.float32), None, None
        m64, v64 = np64(m), np64(v)
    else:
        (cm, sm), (cv, sv) = ob.encode_state(m0, False), ob.encode_state(np.sqrt(v0), True)
        code = lambda c: torch.cat([torch.zeros(off, dtype=torch.uint8), torch.from_numpy(c)]).cuda()[off:]  # noqa: E731
        m, v, ms, vs = code(cm), code(cv), dev(sm), dev(sv)
        # the fp32 values that the kernel decodes: one rounded product, and its rounded square
        m64 = np.float32(ob.decode_state(cm, sm).astype(np.float32)).astype(float)
        v64 = (lambda q: (q * q).astype(float))(ob.decode_state(cv, sv).astype(np.float32))
    t = moe.adamw_tensor(Pm, G, m, v, m_scale=ms, v_scale=vs, master=M, weight_decay=decay)
    return t, dict(p=np64(M) if master else np64(Pm), g=np64(G), m=m64, v=v64)


def check_adam(t, s, step, gs=1.0, pt="f32", lr=LR):
    """The tensor t after the step against the fp64 step from s."""
    f = float(np.float32(gs))
    g = (np.float32(s["g"]) * np.float32(gs)).astype(float) if gs != 1.0 else s["g"]
    decay = float(np.float32(t["weight_decay"]))
    p, m, v = ob.adamw(s["p"], s["g"] * f, s["m"], s["v"], step, lr, B1, B2, EPS, decay)
    upd = np.abs(p - s["p"] * (1 - lr * decay))
    # m and v: constants rounded once, two products and a sum; the update: about a dozen roundings, and the bias
    # corrections' exponentials (a few u each)
    tm = 4 * U * (np.abs(B1 * s["m"]) + np.abs((1 - B1) * s["g"] * f)) + 2.0 ** -149
    tv = 5 * U * np.abs(v) + 2.0 ** -149
    rel_m = tm / np.maximum(np.abs(m), 1e-300)
    tp = 4 * U * (np.abs(s["p"]) + np.abs(p)) + upd * (32 * U + np.minimum(rel_m, 1.0)) + lr * 2.0 ** -149 / EPS
    if t["master"] is not None:
        within(t["master"], p, tp, "master")
        assert torch.equal(t["param"], t["master"].to(t["param"].dtype))
    else:
        within(t["param"], p, tp + HALF[pt] * (np.abs(p) + tp) + TINY[pt], "param")
    if t["m_scale"] is None:
        within(t["m"], m, tm, "m")
        within(t["v"], v, tv, "v")
        return
    # the codes are those of the fp32 steps, bit for bit
    m32, v32 = ob.adamw_f32_moments(np.float32(g), np.float32(s["m"]), np.float32(s["v"]), B1, B2)
    for name, x, root in (("m", m32, False), ("v", np.sqrt(v32), True)):
        c, sc = ob.encode_state(x, root)
        assert np.array_equal(t[name].view(torch.uint8).cpu().numpy(), c), name
        assert np.array_equal(t[name + "_scale"].cpu().numpy(), sc), name + "_scale"


def new_state(step=0):
    return torch.tensor([step, 0], dtype=torch.int32, device="cuda")


SIZES = [1, 2, 7, 8, 31, 255, 256, 257, 511, 2048, 2049, 5000, 70001]


@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("bf16", "f32", False), ("bf16", "f32", True), ("bf16", "bf16", False),
                                        ("f16", "f32", False), ("f16", "f16", True), ("f32", "bf16", False)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("off", [0, 1])
def test_adamw(p, g, master, bits, off):
    r = np.random.default_rng([bits, off])
    cases = [adam_case(r, n, p, g, bits, master, 0.1 * (i % 2), off) for i, n in enumerate(SIZES)]
    plan = moe.make_adamw_plan([t for t, _ in cases], lr=LR, beta1=B1, beta2=B2, eps=EPS)
    state, gs = new_state(6), 0.37
    moe.moe_adamw_step(plan, state, grad_scale=torch.tensor(gs, device="cuda"))
    torch.cuda.synchronize()
    assert state.tolist() == [7, 0]
    for t, s in cases:
        check_adam(t, s, 7, gs, p)


def test_adamw_many_tensors_of_mixed_kinds():
    """More tensors than one launch takes, empty ones among them, all types together."""
    r = np.random.default_rng(11)
    kinds = [("f32", "f32", 32, False), ("bf16", "f32", 8, True), ("bf16", "bf16", 8, False), ("f16", "f32", 32, True)]
    cases = [adam_case(r, int(r.integers(0, 700)) if i % 9 else 0, *kinds[i % 4][:3], kinds[i % 4][3], 0.01 * (i % 3),
                       off=i % 2) for i in range(1000)]
    plan = moe.make_adamw_plan([t for t, _ in cases], lr=LR, beta1=B1, beta2=B2, eps=EPS)
    state = new_state()
    moe.moe_adamw_step(plan, state)
    torch.cuda.synchronize()
    assert state.tolist() == [1, 0]
    for i, (t, s) in enumerate(cases):
        check_adam(t, s, 1, 1.0, kinds[i % 4][0])


@pytest.mark.parametrize("p,g,master", [("bf16", "f32", False), ("f16", "f32", False), ("bf16", "bf16", True)])
def test_adamw_several_tiles_a_block(p, g, master):
    """Tensors of more tiles than blocks, small ones between them, both kinds of states in one plan: a block goes on
    within a tensor and from one tensor to the next."""
    r = np.random.default_rng(17)
    kinds = [(1_300_000, 8, 0), (700, 8, 1), (900_123, 8, 0), (650_000, 32, 0), (256, 8, 0), (1_000_001, 8, 0), (3000, 32, 1)]
    cases = [adam_case(r, n, p, g, bits, master, 0.1, off) for n, bits, off in kinds]
    plan = moe.make_adamw_plan([t for t, _ in cases], lr=LR, beta1=B1, beta2=B2, eps=EPS)
    state = new_state(2)
    moe.moe_adamw_step(plan, state)
    torch.cuda.synchronize()
    assert state.tolist() == [3, 0]
    for t, s in cases:
        check_adam(t, s, 3, 1.0, p)


def test_adamw_from_zero_states_over_steps_and_in_a_graph():
    """Ten steps from new states, the last seven of them replays of one captured step with the rate on the device."""
    r = np.random.default_rng(12)
    n, rates = 3000, [0.01, 0.01, 0.01] + [0.01 / (i + 1) for i in range(7)]
    for bits in (8, 32):
        P = dev(r.standard_normal(n))
        p, m, v = np64(P), np.zeros(n), np.zeros(n)
        grad = torch.empty(n, device="cuda")
        mm, vv, ms, vs = moe.adamw_states(P, bits)
        t = moe.adamw_tensor(P, grad, mm, vv, m_scale=ms, v_scale=vs, weight_decay=0.1)
        plan = moe.make_adamw_plan([t], lr=LR, beta1=B1, beta2=B2, eps=EPS)
        state, lr = new_state(), torch.tensor(0.01, device="cuda")
        graph = None
        for i, rate in enumerate(rates):
            g = np64(dev(r.standard_normal(n) * 0.1))
            grad.copy_(dev(g))
            lr.fill_(rate)
            s = dict(p=np64(P), g=g, m=np64(mm) if bits == 32 else np.float32(ob.decode_state(
                mm.view(torch.uint8).cpu().numpy(), ms.cpu().numpy())).astype(float))
            if bits == 32:
                s["v"] = np64(vv)
            else:
                q = ob.decode_state(vv.view(torch.uint8).cpu().numpy(), vs.cpu().numpy()).astype(np.float32)
                s["v"] = (q * q).astype(float)
            if i < 2:
                moe.moe_adamw_step(plan, state, lr=lr)
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        moe.moe_adamw_step(plan, state, lr=lr)
                graph.replay()
            torch.cuda.synchronize()
            assert state.tolist() == [i + 1, 0]
            check_adam(t, s, i + 1, lr=float(np.float32(rate)))
            p, m, v = ob.adamw(p, g, m, v, i + 1, rate, B1, B2, EPS, 0.1)
        if bits == 32:
            assert np.abs(np64(P) - p).max() <= 10 * 64 * U * (np.abs(p).max() + 1)


def test_adamw_keeps_what_is_not_finite_to_its_element():
    r = np.random.default_rng(13)
    for bits in (8, 32):
        t, s = adam_case(r, 600, "f32", "f32", bits, False, 0.0)
        t["grad"][3], t["grad"][300] = float("nan"), float("inf")
        s["g"] = np64(t["grad"])
        plan = moe.make_adamw_plan([t], lr=LR, beta1=B1, beta2=B2, eps=EPS)
        moe.moe_adamw_step(plan, new_state(3))
        torch.cuda.synchronize()
        p = np64(t["param"])
        assert np.isnan(p[[3, 300]]).all() and np.isfinite(np.delete(p, [3, 300])).all()
        if bits == 8:
            assert t["m"].tolist()[3] == 0x7F and t["v"].tolist()[300] == 0x7F
            for name in ("m", "v"):
                keep = np.delete(np.arange(600), [3, 300])
                assert (t[name].cpu().numpy()[keep] & 0x7F != 0x7F).all() and torch.isfinite(t[name + "_scale"]).all()


def test_adamw_zero_and_tiny_gradients():
    """Zero gradients leave m and v at zero and the weights decayed; gradients whose squares underflow move nothing
    by more than the rate allows."""
    for bits in (8, 32):
        P = torch.linspace(-1, 1, 520, device="cuda")
        before = P.clone()
        g = torch.zeros(520, device="cuda")
        m, v, ms, vs = moe.adamw_states(P, bits)
        plan = moe.make_adamw_plan([moe.adamw_tensor(P, g, m, v, m_scale=ms, v_scale=vs, weight_decay=0.5)], lr=LR,
                                   beta1=B1, beta2=B2, eps=EPS)
        state = new_state()
        moe.moe_adamw_step(plan, state)
        assert not m.float().any() and not v.float().any()
        assert torch.allclose(P, before * (1 - LR * 0.5), rtol=4 * U, atol=0)
        g[::2] = 1e-30
        q = P.clone()
        moe.moe_adamw_step(plan, state)
        assert float((P - q * (1 - LR * 0.5)).abs().max()) <= 4 * U + LR * 1e-30 / EPS * 2


def test_adamw_of_nothing_counts_the_step():
    state = new_state(4)
    moe.moe_adamw_step(moe.make_adamw_plan([]), state)
    e = torch.empty(0, device="cuda")
    moe.moe_adamw_step(moe.make_adamw_plan([moe.adamw_tensor(e, e, e, e)]), state)
    assert state.tolist() == [6, 0]


# ----------------------------------------------------------- streams and graphs
def test_on_another_stream_and_in_graphs_that_share_a_workspace():
    r = np.random.default_rng(14)
    z, topk = router(r, 700, 16, 2)
    cfg = moe.make_balance_config(700, 16, 2)
    Z, K = dev(z), dev(topk, torch.int32)
    ws = ws_of(moe.moe_balance_workspace_size(cfg))
    want = run_balance(z, topk, 2)
    C = [torch.empty(1, 16, dtype=torch.int32, device="cuda") for _ in range(2)]
    loss, dz = [torch.empty(1, device="cuda") for _ in range(2)], [torch.empty(700, 16, device="cuda") for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_balance_loss(cfg, Z, K, C[i], loss[i], ws, dscores=dz[i])
        graphs.append(g)
    ws.fill_(0xFF)
    for i in (0, 1, 1, 0):
        dz[i].fill_(7.0)
        graphs[i].replay()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    l3, d3, C3 = torch.empty(1, device="cuda"), torch.empty(700, 16, device="cuda"), torch.empty_like(C[0])
    moe.moe_balance_loss(cfg, Z, K, C3, l3, ws, dscores=d3, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for l, d, c in ((loss[0], dz[0], C[0]), (loss[1], dz[1], C[1]), (l3, d3, C3)):
        assert float(l) == want[0] and np.array_equal(np64(d), want[2]) and np.array_equal(c.cpu().numpy(), want[1])


def test_calls_on_two_streams_at_once():
    """The same operators on two streams, each with its own workspace, give what they give one after the other."""
    T, E, d, n = 20000, 64, 1536, 900_000

    def make(seed):
        r = np.random.default_rng(seed)
        z, topk = router(r, T, E, 4)
        t, _ = adam_case(r, n, "bf16", "f32", 8, False, 0.1)
        return dict(z=dev(z), k=dev(topk, torch.int32), x=dev(r.standard_normal((3000, d)), torch.bfloat16),
                    dy=dev(r.standard_normal((3000, d))), t=t)

    def run(a, stream):
        out, ncfg, bcfg = {}, moe.make_norm_config(3000, d), moe.make_balance_config(T, E, 4)
        for name, shape, dt in (("y", (3000, d), torch.bfloat16), ("dx", (3000, d), torch.bfloat16), ("mean", 3000, None),
                                ("rstd", 3000, None), ("dg", d, None), ("db", d, None), ("loss", 1, None),
                                ("dz", (T, E), None), ("C", (1, E), torch.int32)):
            out[name] = torch.empty(shape, dtype=dt or torch.float32, device="cuda")
        t = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a["t"].items()}
        plan, state = moe.make_adamw_plan([t], lr=LR), new_state()
        ws1, ws2 = ws_of(moe.moe_layer_norm_workspace_size(ncfg)), ws_of(moe.moe_balance_workspace_size(bcfg))
        torch.cuda.synchronize()

        def go():
            for _ in range(5):
                moe.moe_layer_norm_forward(ncfg, a["x"], None, None, out["y"], mean=out["mean"], rstd=out["rstd"], stream=stream)
                moe.moe_layer_norm_backward(ncfg, a["dy"], a["x"], out["mean"], out["rstd"], None, out["dx"], out["dg"],
                                            out["db"], ws1, stream=stream)
                moe.moe_balance_loss(bcfg, a["z"], a["k"], out["C"], out["loss"], ws2, dscores=out["dz"], stream=stream)
                moe.moe_adamw_step(plan, state, stream=stream)
        return go, {**out, **{k: v for k, v in t.items() if isinstance(v, torch.Tensor)}, "state": state}

    both, streams = [make(1), make(2)], [torch.cuda.Stream() for _ in range(2)]
    want = []
    for a in both:
        go, out = run(a, streams[0])
        go()
        torch.cuda.synchronize()
        want.append(out)
    got = [run(a, s) for a, s in zip(both, streams)]
    for go, _ in got:
        go()
    torch.cuda.synchronize()
    for (_, out), ref in zip(got, want):
        for name in ref:
            assert torch.equal(out[name].view(torch.uint8), ref[name].view(torch.uint8)), name


def test_norm_in_a_graph():
    rows, d = 65, 384
    cfg = moe.make_norm_config(rows, d, x="bf16", dx="f32")
    x, dy = torch.randn(rows, d, device="cuda").bfloat16(), torch.randn(rows, d, device="cuda")
    gam, bet = torch.randn(d, device="cuda"), torch.randn(d, device="cuda")
    y, dx = torch.empty_like(x), torch.empty(rows, d, device="cuda")
    mean, rstd, dg, db = (torch.empty(n, device="cuda") for n in (rows, rows, d, d))
    ws = ws_of(moe.moe_layer_norm_workspace_size(cfg))

    def both():
        moe.moe_layer_norm_forward(cfg, x, gam, bet, y, mean=mean, rstd=rstd)
        moe.moe_layer_norm_backward(cfg, dy, x, mean, rstd, gam, dx, dg, db, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    x.copy_(torch.randn(rows, d, device="cuda"))
    g.replay()
    got = [t.clone() for t in (y, dx, mean, rstd, dg, db)]
    both()
    torch.cuda.synchronize()
    for a, b in zip(got, (y, dx, mean, rstd, dg, db)):
        assert torch.equal(a, b)
