"""README's training step runs as it is written, and leaves what its calls give
when a user makes them one by one."""
import os
import re

import pytest
import torch

import mixture_experts_layer_logit_b200 as moe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, d, E, F, k, SEQ = 96, 128, 8, 192, 2, 3


def blocks():
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    return re.findall(r"```python\n(.*?)```", text, re.S)


def names(seed):
    """Everything that the text takes for granted: sizes, weights, inputs and buffers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
    buf = lambda *s: torch.full(s, float("nan"), device="cuda")   # noqa: E731
    raw = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")   # noqa: E731
    bf = torch.bfloat16
    cfg = moe.make_config(T, d, E, F, k, act="swiglu", dtype="bf16", capacity_factor=1.25)
    nbytes, layout = moe.moe_workspace_size(cfg)
    W1 = (rnd(E, 2 * F, d) * 0.1).to(bf)
    m, v, ms, vs = moe.adamw_states(W1, 8)
    return dict(
        moe=moe, torch=torch, T=T, d=d, E=E, F=F, k=k, sequences=SEQ, cfg=cfg, layout=layout, workspace=raw(nbytes),
        x=rnd(T, d).to(bf), stream=rnd(T, d), out_before=rnd(T, d), gamma=1 + 0.2 * rnd(d), beta=0.2 * rnd(d),
        y=buf(T, d).to(bf), mean=buf(T), rstd=buf(T), Wg=(rnd(E, d) * 0.1).to(bf), bg=0.1 * rnd(E), W1=W1,
        W2=(rnd(E, d, F) * 0.1).to(bf), out=buf(T, d), stats=torch.zeros(moe.STATS_BYTES, dtype=torch.uint8, device="cuda"),
        scores=buf(T, E), counts=torch.empty(SEQ, E, dtype=torch.int32, device="cuda"), loss=buf(1),
        bws=raw(moe.moe_balance_workspace_size(moe.make_balance_config(T, E, k, S=SEQ))),
        off=torch.tensor([0, 40, 70, T], dtype=torch.int32, device="cuda"),
        mask=(torch.rand(T, device="cuda", generator=g) > 0.2).to(torch.uint8), coef=torch.tensor(0.3, device="cuda"),
        ds=buf(T, E), dout=rnd(T, d), bwd_workspace=raw(moe.moe_backward_workspace_size(cfg)), dy=buf(T, d),
        dWg=buf(E, d), dbg=buf(E), dW1=buf(E, 2 * F, d), dW2=buf(E, d, F), dx=buf(T, d), dgamma=buf(d), dbeta=buf(d),
        nws=raw(moe.moe_layer_norm_workspace_size(moe.make_norm_config(T, d, x="f32", y="bf16"))), dstream=rnd(T, d),
        m=m, v=v, ms=ms, vs=vs, step_state=torch.zeros(2, dtype=torch.int32, device="cuda"))


def test_forward_runs():
    ns = names(1)
    exec(blocks()[0], ns)
    torch.cuda.synchronize()
    assert torch.isfinite(ns["out"]).all() and moe.read_stats(ns["stats"])["status"] == 0


def test_training_step_runs():
    ns, a = names(2), names(2)
    before = a["W1"].clone()
    exec(blocks()[1], ns)
    torch.cuda.synchronize()
    assert moe.read_stats(ns["stats"])["status"] == 0 and ns["step_state"].tolist() == [1, 0]
    ncfg, bcfg = moe.make_norm_config(T, d, x="f32", y="bf16"), moe.make_balance_config(T, E, k, S=SEQ)
    moe.moe_layer_norm_forward(ncfg, a["stream"], a["gamma"], a["beta"], a["y"], add=a["out_before"], sum=a["stream"],
                               mean=a["mean"], rstd=a["rstd"])
    w2 = moe.prepare_w2(a["cfg"], a["W2"])
    moe.moe_layer_forward_scores(a["cfg"], a["y"], a["Wg"], a["bg"], a["W1"], w2, a["out"], a["stats"], a["scores"],
                                 a["workspace"])
    at = a["layout"].topk_idx
    idx = a["workspace"][at:at + 4 * T * k].view(torch.int32)
    assert torch.equal(torch.sort(idx.view(T, k).long()).values, torch.sort(torch.topk(a["scores"], k).indices).values)
    moe.moe_balance_loss(bcfg, a["scores"], idx, a["counts"], a["loss"], a["bws"], seq_offsets=a["off"], mask=a["mask"],
                         coef=a["coef"], dscores=a["ds"])
    assert int(a["counts"].sum()) == k * int(a["mask"].sum())
    moe.moe_layer_backward_scores(a["cfg"], a["y"], a["Wg"], a["bg"], a["W1"], w2, a["dout"], a["ds"], 0.0, 0.0,
                                  a["workspace"], a["dy"], a["dWg"], a["dbg"], a["dW1"], a["dW2"], None, a["stats"],
                                  a["bwd_workspace"])
    moe.moe_layer_norm_backward(ncfg, a["dy"], a["stream"], a["mean"], a["rstd"], a["gamma"], a["dx"], a["dgamma"],
                                a["dbeta"], a["nws"], dsum=a["dstream"], stats=a["stats"])
    moe.moe_adamw_step(moe.make_adamw_plan([moe.adamw_tensor(a["W1"], a["dW1"], a["m"], a["v"], m_scale=a["ms"],
                                                             v_scale=a["vs"], weight_decay=0.1)], lr=3e-4), a["step_state"])
    torch.cuda.synchronize()
    for n in ("y", "out", "scores", "loss", "ds", "dy", "dWg", "dbg", "dW1", "dW2", "dx", "dgamma", "dbeta", "W1"):
        assert torch.isfinite(a[n]).all() and torch.equal(ns[n], a[n]), n
    assert not torch.equal(a["W1"], before)
