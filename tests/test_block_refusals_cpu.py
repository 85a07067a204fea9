"""Refusals of the operators around the layer, before any device work: the C
ABI's status codes with stand-in pointers that are never dereferenced, and the
binding's checks of its tensors."""
import ctypes

import pytest
import torch

import mixture_experts_layer_logit_b200 as moe
from mixture_experts_layer_logit_b200 import build as moe_build

P = 1 << 20   # an aligned non-null stand-in
BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def norm(**kw):
    base = dict(rows=10, d=64, eps=1e-5, x="f32", w="f32")
    base.update(kw)
    return moe.make_norm_config(**base)


def fwd(L, c, x=P, add=None, gamma=P, beta=P, y=P, sum=None, mean=P, rstd=P):
    return L.moe_layer_norm_forward(BY(c) if c else None, x, add, gamma, beta, y, sum, mean, rstd, None)


def bwd(L, c, dy=P, x=P, mean=P, rstd=P, gamma=P, dsum=None, dx=P, dgamma=P, dbeta=P, stats=None, ws=P,
        n=1 << 30):
    return L.moe_layer_norm_backward(BY(c) if c else None, dy, x, mean, rstd, gamma, dsum, dx, dgamma, dbeta, stats,
                                     ws, n, None)


def test_struct_sizes(L):
    assert ctypes.sizeof(moe.moe_norm_config) == 36
    assert ctypes.sizeof(moe.moe_balance_config) == 24
    assert ctypes.sizeof(moe.moe_adamw_tensor) == 80
    assert ctypes.sizeof(moe.moe_adamw_hyper) == 32


@pytest.mark.parametrize("kw,code", [(dict(rows=-1), 1), (dict(d=0), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
                                     (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(d=16385), 2)])
def test_norm_config(L, kw, code):
    c = norm(**kw)
    assert moe.moe_layer_norm_workspace_size(c) == 0
    assert fwd(L, c) == code and bwd(L, c) == code
    assert fwd(L, None) == 1 and bwd(L, None) == 1


@pytest.mark.parametrize("field", ["x_dtype", "y_dtype", "w_dtype", "add_dtype", "dy_dtype", "dx_dtype"])
def test_norm_dtypes(L, field):
    c = norm()
    setattr(c, field, 3)
    assert fwd(L, c) == 1 and bwd(L, c) == 1


def test_norm_pointers(L):
    c = norm()
    assert fwd(L, c, x=None) == 1 and fwd(L, c, y=None) == 1
    assert fwd(L, c, sum=P) == 1                                   # a sum of nothing
    for name in ("x", "add", "gamma", "beta", "y", "mean", "rstd"):
        assert fwd(L, c, **{name: P + 2}) == 1, name               # half an fp32
    assert fwd(L, c, add=P, sum=P + 2) == 1
    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert bwd(L, c, **{name: None}) == 1, name
    for name in ("dy", "x", "mean", "rstd", "gamma", "dsum", "dx", "dgamma", "dbeta", "stats"):
        assert bwd(L, c, **{name: P + 2}) == 1, name
    h = norm(x="bf16", w="f16", add="bf16", dy="f16", dx="bf16")
    assert fwd(L, h, x=P + 1) == 1 and fwd(L, h, gamma=P + 1) == 1 and bwd(L, h, dy=P + 1) == 1


def test_norm_workspace(L):
    c = norm()
    n = moe.moe_layer_norm_workspace_size(c)
    assert n > 0 and n % 256 == 0
    assert bwd(L, c, ws=None) == 3 and bwd(L, c, ws=P + 16) == 3 and bwd(L, c, n=n - 1) == 3


def test_norm_of_no_rows(L):
    c = norm(rows=0)
    assert fwd(L, c, x=None, y=None) == 0
    assert bwd(L, c, None, None, None, None, dx=None, dgamma=None, dbeta=None, ws=None, n=0) == 0
    assert bwd(L, c, ws=None) == 3


def bal(**kw):
    base = dict(T=100, E=8, k=2, S=3)
    base.update(kw)
    return moe.make_balance_config(**base)


def loss(L, c, scores=P, topk=P, off=P, mask=None, coef=None, counts=P, out=P, dz=P, stats=None, ws=P, n=1 << 30):
    return L.moe_balance_loss(BY(c) if c else None, scores, topk, off, mask, coef, counts, out, dz, stats, ws, n,
                              None)


@pytest.mark.parametrize("kw,code", [(dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(S=0), 1),
                                     (dict(dtype="f16"), 1), (dict(E=257), 2), (dict(T=1 << 30), 2),
                                     (dict(S=1 << 28), 2)])
def test_balance_config(L, kw, code):
    c = bal(**kw)
    assert moe.moe_balance_workspace_size(c) == 0
    assert loss(L, c) == code
    assert loss(L, None) == 1


def test_balance_arguments(L):
    c = bal()
    bad = bal()
    bad.score = 2
    assert loss(L, bad) == 1
    assert loss(L, c, counts=None) == 1
    assert loss(L, c, off=None) == 1                               # three sequences need their offsets
    assert loss(L, c, scores=None) == 1                            # an output without scores
    assert loss(L, c, out=None, dz=None) == 1                      # scores without an output
    assert loss(L, c, scores=None, topk=None, out=None, dz=None) == 1
    for name in ("scores", "topk", "off", "coef", "counts", "out", "dz", "stats"):
        assert loss(L, c, **{name: P + 2}) == 1, name
    n = moe.moe_balance_workspace_size(c)
    assert n > 0 and loss(L, c, ws=None) == 3 and loss(L, c, n=n - 1) == 3 and loss(L, c, ws=P + 128) == 3


def tensor(**kw):
    t = dict(param=P, grad=P, master=None, m=P, v=P, m_scale=None, v_scale=None, n=10, param_dtype=0, grad_dtype=0,
             state_bits=32, weight_decay=0.0)
    t.update(kw)
    return moe.moe_adamw_tensor(**t)


def step(L, t, nt=1, hyper=(1e-3, 0.9, 0.99, 1e-8), lr=None, gs=None, state=P):
    h = moe.moe_adamw_hyper(*hyper) if hyper else None
    return L.moe_adamw_step(BY(t) if t is not None else None, nt, BY(h) if h else None, lr, gs, state, None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None),
                                dict(param_dtype=3), dict(grad_dtype=-1), dict(state_bits=16), dict(param=P + 2),
                                dict(grad=P + 2), dict(param=P + 1, param_dtype=1), dict(master=P + 2),
                                dict(m=P + 1), dict(v=P + 2), dict(state_bits=8),
                                dict(state_bits=8, m_scale=P, v_scale=P + 2), dict(weight_decay=float("nan"))])
def test_adamw_tensors(L, kw):
    assert step(L, tensor(**kw)) == 1


@pytest.mark.parametrize("hyper", [None, (float("nan"), 0.9, 0.99, 1e-8), (1e-3, 1.0, 0.99, 1e-8),
                                   (1e-3, -0.1, 0.99, 1e-8), (1e-3, 0.9, 1.0, 1e-8), (1e-3, 0.9, float("nan"), 1e-8),
                                   (1e-3, 0.9, 0.99, 0.0), (1e-3, 0.9, 0.99, 1e-60), (1e-3, 0.9, 0.99, float("inf"))])
def test_adamw_hyper(L, hyper):
    assert step(L, tensor(), hyper=hyper) == 1


def test_adamw_arguments(L):
    assert step(L, None) == 1 and step(L, tensor(), nt=-1) == 1
    assert step(L, tensor(), state=None) == 1 and step(L, tensor(), state=P + 2) == 1
    assert step(L, tensor(), lr=P + 1) == 1 and step(L, tensor(), gs=P + 2) == 1


def test_scores_entries_refuse_what_the_plain_ones_do(L):
    c = moe.make_config(100, 64, 8, 128, 2)
    assert L.moe_route_scores(BY(c), None, P, None, P, P, P, None, None, P, P, 1 << 30, None) == 1
    assert L.moe_route_scores(BY(c), P, P, None, P, P, P, None, None, P + 2, P, 1 << 30, None) == 1
    assert L.moe_layer_forward_scores(BY(c), P, P, None, P, P, P, P, P + 2, P, 1 << 30, None) == 1
    assert L.moe_layer_forward_scores(BY(c), P, P, None, P, P, P, P, P, P, 16, None) == 3
    args = [P, P, None, P, P, P, P + 2, ctypes.c_float(0), ctypes.c_float(0), P, 1 << 30, P, P, None, P, P, None, P, P,
            1 << 30, None]
    assert L.moe_layer_backward_scores(BY(c), *args) == 1
    args[6], args[10] = P, 16
    assert L.moe_layer_backward_scores(BY(c), *args) == 3


def test_binding_checks_its_tensors(L):
    t = torch.zeros(4, 6)
    ok = lambda t, dt=torch.float32, n=24: moe._arg("f", "t", t, -1, dt, n)   # noqa: E731 (-1: the CPU)
    assert ok(t) == t.data_ptr() and ok(None) is None and ok(P) == P
    for bad in (lambda: ok(t, torch.bfloat16), lambda: ok(t, n=23), lambda: ok(t.t()),
                lambda: moe._arg("f", "t", t, 0, torch.float32, 24)):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.code == 1 and "t is" in str(e.value) or "t has" in str(e.value)
    with pytest.raises(moe.MoeError):
        moe._workspace("f", t, 0)
    c = norm(rows=4, d=6)
    with pytest.raises(moe.MoeError):   # CPU tensors never reach the library
        moe.moe_layer_norm_forward(c, t, None, None, t)
    with pytest.raises(moe.MoeError):
        moe.make_adamw_plan([moe.adamw_tensor(t, t, t.clone(), t.clone())])


def test_new_states_are_zeros():
    p = torch.zeros(600, dtype=torch.bfloat16)
    m, v, ms, vs = moe.adamw_states(p, 8)
    assert m.numel() == v.numel() == 600 and ms.numel() == vs.numel() == 3 and m.dtype == torch.float8_e4m3fn
    m, v, ms, vs = moe.adamw_states(p, 32)
    assert m.dtype == v.dtype == torch.float32 and ms is None and vs is None
    with pytest.raises(ValueError):
        moe.adamw_states(p, 16)
