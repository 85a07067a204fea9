"""The layer with its scores in the open, and a whole training step of a block:
residual addition and norm, the layer, the balance loss per sequence, both
backwards and the optimiser's step, on the device against float64."""
import numpy as np
import pytest
import torch

import moe_workloads as mw
import mixture_experts_layer_logit_b200 as moe
import oracle
from oracle import block_ops as bo
from oracle import moe_backward as mb
from oracle import moe_oracle as om
from tests.gpu_harness import DeviceLayer, to_np64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
W = mw.Workload
LAYERS = [
    W("s_relu", T=300, d=256, E=12, F=320, k=3, act=mw.RELU, dtype=mw.BF16, capacity_factor=1.1, seed=91),
    W("s_lam_bias", T=257, d=192, E=8, F=208, k=2, act=mw.SWIGLU, dtype=mw.BF16, lam=1.0, zipf_bias=True, seed=92),
    W("s_split", T=64, d=2048, E=64, F=176, k=6, act=mw.SWIGLU, dtype=mw.BF16, zipf_bias=True, seed=93),   # width cut
    W("s_split_lam", T=9, d=2048, E=33, F=64, k=2, act=mw.RELU, dtype=mw.BF16, lam=0.5, seed=94),
    W("s_many", T=130, d=64, E=256, F=64, k=8, act=mw.RELU, dtype=mw.BF16, seed=95),
    W("s_top9", T=140, d=64, E=20, F=64, k=9, act=mw.RELU, dtype=mw.BF16, lam=1.0, seed=96),              # k > 8
    W("s_fp32", T=200, d=64, E=5, F=96, k=2, act=mw.RELU, dtype=mw.F32, capacity_factor=1.0, seed=97),
    W("s_fp32_lam", T=77, d=32, E=6, F=40, k=3, act=mw.SWIGLU, dtype=mw.F32, lam=0.5, seed=98),
    W("s_E1", T=5, d=64, E=1, F=64, k=1, act=mw.RELU, dtype=mw.BF16, seed=99),
]


def zeros_stats():
    return torch.zeros(moe.STATS_BYTES, dtype=torch.uint8, device="cuda")


def forward_scores(L):
    n, lay = moe.moe_workspace_size(L.cfg)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.empty((L.T, L.w.d), device="cuda")
    scores = torch.full((L.T, L.w.E), float("nan"), device="cuda")
    stats = zeros_stats()
    moe.moe_layer_forward_scores(L.cfg, L.x, L.wg, L.bias, L.w1, L.w2, out, stats, scores, ws)
    torch.cuda.synchronize()
    assert moe.read_stats(stats)["status"] == 0
    return out, scores, ws, lay


def score_tolerance(x, wg, bias, z, s, lam):
    """z is a sum of d products in fp32 (any order); z_hat divides its deviation by the spread."""
    d, E = wg.shape[1], wg.shape[0]
    ez = (d + 16) * U * (np.abs(x) @ np.abs(wg).T + (0 if bias is None else np.abs(bias)))
    if lam <= 0:
        return ez
    worst = ez.max(1, keepdims=True)
    sd = z.std(1, keepdims=True)
    return lam * 2 * worst / sd * (1 + np.abs(s) / lam) + (E + 16) * U * (np.abs(s) + lam)


@pytest.mark.parametrize("w", LAYERS, ids=[w.name for w in LAYERS])
def test_scores(w):
    if w.E == 1 and w.lam > 0:
        pytest.skip("one expert has no spread")
    L = DeviceLayer(w)
    x, wg = mw.to_f64(L.inp.x), mw.to_f64(L.inp.wg)
    r = om.route(x, wg, L.inp.bias, oracle.LayerConfig.from_workload(w, L.T))
    z = om.gate_logits(x, wg, L.inp.bias)
    tol = score_tolerance(x, wg, L.inp.bias, z, r.s, w.lam)
    plain = L.forward()
    out, scores, ws, lay = forward_scores(L)
    err = np.abs(to_np64(scores) - r.s)
    assert (err <= tol).all(), (err - tol).max()
    assert torch.equal(out, plain["out"])
    # the step call: the same scores, and what moe_route gives
    idx, wt, gap, pm = L.route()
    idx2, wt2, gap2, pm2, s2 = (torch.empty_like(t) for t in (idx, wt, gap, pm, scores))
    moe.moe_route_scores(L.cfg, L.x, L.wg, L.bias, idx2, wt2, gap2, pm2, s2, L.scratch())
    torch.cuda.synchronize()
    for a, b in ((idx, idx2), (wt, wt2), (gap, gap2), (pm, pm2), (scores, s2)):
        assert torch.equal(a, b)


def backward(L, ws, dout, dscores, aux=0.0, zc=0.0, plain=False):
    w = L.w
    F1 = w.F if w.act == mw.RELU else 2 * w.F
    g = [torch.empty(s, device="cuda") for s in ((L.T, w.d), (w.E, w.d), (w.E,), (w.E, F1, w.d), (w.E, w.d, w.F),
                                                 (L.T, w.k))]
    bws = torch.full((moe.moe_backward_workspace_size(L.cfg),), 0xA5, dtype=torch.uint8, device="cuda")
    stats = zeros_stats()
    if plain:
        moe.moe_layer_backward(L.cfg, L.x, L.wg, L.bias, L.w1, L.w2, dout, aux, zc, ws, *g, stats, bws)
    else:
        moe.moe_layer_backward_scores(L.cfg, L.x, L.wg, L.bias, L.w1, L.w2, dout, dscores, aux, zc, ws, *g, stats, bws)
    torch.cuda.synchronize()
    assert moe.read_stats(stats)["status"] == 0
    return g


@pytest.mark.parametrize("w", LAYERS, ids=[w.name for w in LAYERS])
def test_gradient_of_the_scores_joins_the_gate(w):
    L = DeviceLayer(w)
    x, wg = mw.to_f64(L.inp.x), mw.to_f64(L.inp.wg)
    rng = np.random.default_rng(w.seed)
    dout = torch.from_numpy(rng.standard_normal((L.T, w.d)).astype(np.float32)).cuda()
    ds = rng.standard_normal((L.T, w.E)).astype(np.float32)
    _, _, ws, _ = forward_scores(L)
    base = backward(L, ws, dout, None, 0.05, 0.01)
    for a, b in zip(base, backward(L, ws, dout, None, 0.05, 0.01, plain=True)):
        assert torch.equal(a, b)   # without a gradient of the scores: the call that was there
    got = backward(L, ws, dout, torch.from_numpy(ds).cuda(), 0.05, 0.01)
    z = om.gate_logits(x, wg, L.inp.bias)
    dz = mb.normalise_backward(z, ds.astype(float), w.lam) if w.lam > 0 else ds.astype(float)
    for i in (3, 4, 5):   # the experts' gradients and that of the gate weights do not see it
        assert torch.equal(base[i], got[i])
    for i, add, mag in ((0, dz @ wg, np.abs(dz) @ np.abs(wg)), (1, dz.T @ x, np.abs(dz).T @ np.abs(x)),
                        (2, dz.sum(0), np.abs(dz).sum(0))):
        diff = to_np64(got[i]) - to_np64(base[i])
        # the scores' part is fp32 throughout: sums of at most T + E + d terms; its logits and, with lambda, their
        # spread are recomputed (1e-5 covers (d + 16) u of them over the spread); each total is rounded
        tol = ((L.T + w.E + w.d) * U + (1e-4 if w.lam > 0 else 0)) * mag + 8 * (L.T + w.E) * U * (
            np.abs(to_np64(base[i])) + np.abs(to_np64(got[i])) + mag)
        assert (np.abs(diff - add) <= tol + 1e-6 * np.abs(to_np64(base[i])).max()).all(), i


def close(got, ref, what, rel=1e-4):
    err, top = np.abs(to_np64(got) - ref).max(), np.abs(ref).max()
    assert err <= rel * top, f"{what}: {err:.3e} of {top:.3e}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step_of_a_block(score):
    """stream + add -> norm -> layer -> balance loss; back through the layer, the norm and the residual; AdamW.  The
    fp32 layer, held to the suite's 1e-4 of the largest value for every gradient and weight."""
    w = W("block", T=120, d=64, E=6, F=96, k=2, act=mw.SWIGLU, dtype=mw.F32, seed=55)
    rng = np.random.default_rng(3)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)   # noqa: E731
    L = DeviceLayer(w)
    T, d, E, F = w.T, w.d, w.E, w.F
    cu = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a)).cuda() if dt is None else torch.from_numpy(a).cuda().to(dt)  # noqa: E731, E501
    stream, add, gam, bet, dnext, dout = f(T, d), f(T, d), 1 + 0.2 * f(d), 0.2 * f(d), f(T, d), f(T, d)
    off = np.array([0, 30, 30, 95, 118], np.int32)
    mask = (rng.random(T) > 0.2).astype(np.uint8)
    coef = 0.5
    # ---- device
    ncfg = moe.make_norm_config(T, d, x="f32")
    X, Y, mean, rstd = cu(stream), torch.empty(T, d, device="cuda"), *(torch.empty(T, device="cuda") for _ in range(2))
    G, B = cu(gam), cu(bet)
    moe.moe_layer_norm_forward(ncfg, X, G, B, Y, add=cu(add), sum=X, mean=mean, rstd=rstd)
    L.x = Y
    _, scores, ws, lay = forward_scores(L)
    topk = ws[lay.topk_idx:lay.topk_idx + 4 * T * w.k].view(torch.int32).view(T, w.k)
    bcfg = moe.make_balance_config(T, E, w.k, S=4, score=score)
    counts, loss = torch.empty(4, E, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    ds = torch.empty(T, E, device="cuda")
    moe.moe_balance_loss(bcfg, scores, topk, counts, loss,
                         torch.empty(moe.moe_balance_workspace_size(bcfg), dtype=torch.uint8, device="cuda"),
                         seq_offsets=cu(off), mask=cu(mask), coef=torch.tensor(coef, device="cuda"), dscores=ds)
    without = backward(L, ws, cu(dout), None)
    dy, dwg, dbg, dw1, dw2, _ = backward(L, ws, cu(dout), ds)
    dX, dG, dB = torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    moe.moe_layer_norm_backward(ncfg, dy, X, mean, rstd, G, dX, dG, dB,
                                torch.empty(moe.moe_layer_norm_workspace_size(ncfg), dtype=torch.uint8, device="cuda"),
                                dsum=cu(dnext))
    weights = [(G, dG, 0.0), (B, dB, 0.0), (L.wg, dwg, 0.0), (L.w1, dw1, 0.1), (L.w2, dw2, 0.1)]
    old = [to_np64(p) for p, _, _ in weights]
    tensors, m0 = [], []
    for p, g, wd in weights:
        p.copy_(p)
        m, v, _, _ = moe.adamw_states(p)
        m.normal_(), v.uniform_(0.5, 1.5)   # a state in which the step is a smooth function of the gradient
        m0.append((to_np64(m), to_np64(v)))
        tensors.append(moe.adamw_tensor(p, g, m, v, weight_decay=wd))
    state = torch.tensor([9, 0], dtype=torch.int32, device="cuda")
    moe.moe_adamw_step(moe.make_adamw_plan(tensors, lr=0.02, beta1=0.9, beta2=0.95), state)
    torch.cuda.synchronize()
    # ---- float64
    wg, w1, w2 = (mw.to_f64(a) for a in (L.inp.wg, L.inp.w1, L.inp.w2))
    h = (stream + add).astype(float)
    y, mu, rs = bo.layer_norm(h, gam.astype(float), bet.astype(float))
    lc = oracle.LayerConfig.from_workload(w, T)
    fw = om.forward(y, wg, L.inp.bias, w1, w2, lc)
    assert (fw.routing.gap > 1e-4).all()
    rl, rc, rds = bo.balance(fw.routing.s, fw.routing.idx, w.k, E, off, mask, score, coef)
    g = mb.backward(y, wg, L.inp.bias, w1, w2, lc, dout.astype(float), 0.0, 0.0, fw=fw)
    dyr, dwgr, dbr = g.dx + rds @ wg, g.dwg + rds.T @ y, g.dbias + rds.sum(0)
    dxr, dgr, dber = bo.layer_norm_backward(dyr, h, mu, rs, gam.astype(float), dnext.astype(float))
    assert np.array_equal(counts.cpu().numpy(), rc) and abs(float(loss) - rl) <= 1e-4 * rl
    for a, b, n in ((Y, y, "y"), (ds, rds, "dscores"), (dwg, dwgr, "dWg"), (dbg, dbr, "db"), (dw1, g.dw1, "dW1"),
                    (dw2, g.dw2, "dW2"), (dX, dxr, "dx"), (dG, dgr, "dgamma"), (dB, dber, "dbeta")):
        close(a, b, n)
    # the balance loss's part of dWg alone: both totals are fp32 sums over T tokens of ds_te y_tc, of which only the
    # scores' gradient differs (itself held to 1e-4 above)
    part, mag = rds.T @ y, (np.abs(g.ds) + np.abs(rds)).T @ np.abs(y)
    diff = to_np64(dwg) - to_np64(without[1])
    assert (np.abs(diff - part) <= 1e-4 * np.abs(rds).max() * np.abs(y).sum(0) + 2 * (T + 16) * U * mag).all()
    for (p, _, wd), o, (m, v), gr in zip(weights, old, m0, (dgr, dber, dwgr, g.dw1, g.dw2)):
        ref = bo.adamw(o.reshape(-1), gr.reshape(-1), m, v, 10, 0.02, 0.9, 0.95, 1e-8, wd)[0]
        close(p.view(-1), ref, "updated weight")
