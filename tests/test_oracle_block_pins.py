"""Pins of the float64 oracle of the operators around the layer: its gradients
against central differences of its own forwards, closed forms, and the E4M3
codes against torch's conversion."""
import numpy as np
import pytest
import torch

from oracle import block_ops as ob

H = 1e-5   # step of the central differences: truncation H^2 f''' / 6, cancellation 2^-53 |f| / H, both near 1e-10
TOL = 1e-7


def numeric(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += H
        b[i] -= H
        g[i] = (f(a) - f(b)) / (2 * H)
    return g


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 2), (4, 7)])
def test_layer_norm_gradients(rows, d):
    r = np.random.default_rng([rows, d])
    h, dy, gam, bet, ds = (r.standard_normal(s) for s in [(rows, d), (rows, d), (d,), (d,), (rows, d)])
    eps = 0.1   # keeps the curvature of a nearly constant row moderate
    L = lambda h, gam, bet: (ob.layer_norm(h, gam, bet, eps)[0] * dy).sum() + (h * ds).sum()   # noqa: E731
    _, mu, rs = ob.layer_norm(h, gam, bet, eps)
    dh, dg, db = ob.layer_norm_backward(dy, h, mu, rs, gam, ds)
    assert np.abs(dh - numeric(lambda v: L(v, gam, bet), h)).max() < TOL
    assert np.abs(dg - numeric(lambda v: L(h, v, bet), gam)).max() < TOL
    assert np.abs(db - numeric(lambda v: L(h, gam, v), bet)).max() < TOL


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offsets,masked", [(None, False), ([0, 3, 3, 7, 9], True), ([1, 4, 8], True)])
def test_balance_gradient(score, offsets, masked):
    r = np.random.default_rng(5)
    T, E, k = 9, 5, 2
    z = r.standard_normal((T, E))
    topk = np.argsort(-z, 1)[:, :k]
    mask = (r.random(T) > 0.3) if masked else None
    f = lambda v: 0.7 * ob.balance(v, topk, k, E, offsets, mask, score)[0]   # noqa: E731
    _, counts, dz = ob.balance(z, topk, k, E, offsets, mask, score, coef=0.7)
    assert np.abs(dz - numeric(f, z)).max() < TOL
    if mask is not None:
        assert not dz[~mask].any()


def test_balance_of_a_uniform_router_is_one():
    z = np.zeros((8, 4))
    topk = np.arange(8)[:, None] % 4
    for score in ("softmax", "sigmoid"):
        loss, counts, dz = ob.balance(z, topk, 1, 4, score=score)
        assert abs(loss - 1.0) < 1e-12 and (counts == 2).all() and np.abs(dz).max() < 1e-15


def test_one_sequence_is_the_layers_aux_loss():
    from oracle import moe_oracle as om   # E sum_e f_e P_e over the whole batch
    r = np.random.default_rng(6)
    z = r.standard_normal((50, 6))
    topk = np.argsort(-z, 1)[:, :2]
    p = ob.probabilities(z)
    counts = np.bincount(topk.reshape(-1), minlength=6)
    assert abs(ob.balance(z, topk, 2, 6)[0] - 6 * ((counts / 100) * p.mean(0)).sum()) < 1e-12
    assert om is not None


def test_balance_skips_bad_indices_and_empty_rows():
    z = np.array([[0.0, 1.0], [-np.inf, -np.inf], [2.0, -np.inf]])
    topk = np.array([[1], [2 ** 31 - 1], [0]])
    for score in ("softmax", "sigmoid"):
        loss, counts, dz = ob.balance(z, topk, 1, 2, score=score)
        assert counts.tolist() == [[1, 1]] and np.isfinite(loss)
        assert not dz[1].any() and np.isfinite(dz).all()


def test_e4m3_codes_match_torch():
    r = np.random.default_rng(7)
    x = np.concatenate([r.standard_normal(4000) * 10.0 ** r.uniform(-4, 3, 4000), ob.e4m3_table(), -ob.e4m3_table(),
                        (ob.e4m3_table()[1:] + ob.e4m3_table()[:-1]) / 2, [0.0, -0.0, 448.0, 460.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ob.e4m3_encode(x), want)
    assert np.array_equal(ob.e4m3_decode(want), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_adamw_against_torch():
    r = np.random.default_rng(8)
    p0 = r.standard_normal(40)
    P = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([P], lr=0.01, betas=(0.9, 0.98), eps=1e-6, weight_decay=0.1)
    p, m, v = p0, np.zeros(40), np.zeros(40)
    for t in range(1, 6):
        g = r.standard_normal(40)
        P.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = ob.adamw(p, g, m, v, t, 0.01, 0.9, 0.98, 1e-6, 0.1)
        assert np.abs(p - P.detach().numpy()).max() < 1e-12


def test_8bit_state_error_is_half_a_step():
    r = np.random.default_rng(9)
    x = np.abs(r.standard_normal(700)) * 10.0 ** r.uniform(-3, 0, 700)
    x[5] = 0.0
    for root in (False, True):
        c, s = ob.encode_state(x, root)
        back, sc = ob.decode_state(c, s), np.repeat(s, ob.BLOCK)[:700].astype(float)
        # normal codes: 2^-4 of the value; below them the step is 2^-9 of the scale, and a root is lifted to one step
        assert (np.abs(back - x) <= x * 2.0 ** -4 * 1.0001 + sc * 2.0 ** -9 * (1.0 if root else 0.5001)).all()
        assert back[5] == 0 and (not root or (back[x > 0] > 0).all())
