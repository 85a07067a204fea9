"""Timed cases of the operators around the MoE layer: layer norm (forward and
backward), the balance loss with its gradient, and the AdamW step.

Each case runs either the plain form below (elementary torch operations in
fp32) or, with ``own`` true, the library's kernels through its public calls.
Inputs are synthetic, drawn on the device from the seed alone.
"""
import math

import torch

own = False   # false: the plain forms; true: the library's kernels

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256          # elements per scale of an 8-bit state
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
FIRST_STEP = 10      # optimiser steps behind the prepared state


def listed():
    return [
        # pre-norm of one decoded token of the fine-grained layer: latency only
        dict(name="norm_decode", op="norm_fwd", rows=1, d=2048, x="bf16", y="bf16", w="bf16", add="", stats=False),
        # pre-norm of the Mixtral-shaped layer: the fp32 residual stream takes the last layer's fp32 output,
        # the norm of the sum goes to the next layer in bf16
        dict(name="norm_fwd_mixtral", op="norm_fwd", rows=16384, d=4096, x="f32", y="bf16", w="f32", add="f32",
             stats=True),
        # its backward in the FastMoE Transformer-XL layer: the layer's fp32 dx, the residual's gradient added
        dict(name="norm_bwd_fastmoe", op="norm_bwd", rows=8192, d=512, x="f32", dy="f32", w="f32", dx="f32",
             dsum=True),
        # a short batch of an odd width, everything in fp16
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1021, d=1037, x="f16", dy="f16", w="f16", dx="f16", dsum=False),
        # the Mixtral-shaped layer's backward
        dict(name="norm_bwd_mixtral", op="norm_bwd", rows=16384, d=4096, x="f32", dy="f32", w="f32", dx="f32",
             dsum=True),
        # the tiny fp32 layer's batch as one sequence
        dict(name="balance_tiny", op="balance", T=256, E=8, k=2, S=1, fn="softmax", z="f32", mask=False),
        # the FastMoE layer's batch: 16 ragged sequences with padded tokens
        dict(name="balance_fastmoe", op="balance", T=8192, E=64, k=2, S=16, fn="softmax", z="f32", mask=True),
        # a long batch over many experts with sigmoid scores held in bf16
        dict(name="balance_long", op="balance", T=131072, E=256, k=8, S=61, fn="sigmoid", z="bf16", mask=True),
        # every tensor of the tiny fp32 layer: launch latency
        dict(name="adamw_tiny", op="adamw", layers=1, d=64, E=8, F=128, F1=128, p="f32", g="f32", master=False,
             bits=32),
        # a deep stack of small layers: 160 tensors in one step, 8-bit states
        dict(name="adamw_stack", op="adamw", layers=32, d=256, E=8, F=352, F1=704, p="bf16", g="f32", master=False,
             bits=8),
        # the FastMoE layer: bf16 weights with fp32 master copies, 32-bit states
        dict(name="adamw_fastmoe", op="adamw", layers=1, d=512, E=64, F=1024, F1=1024, p="bf16", g="f32",
             master=True, bits=32),
        # the fine-grained layer, 0.55 G parameters: 8-bit states, no master copies
        dict(name="adamw_fine", op="adamw", layers=1, d=2048, E=64, F=1408, F1=2816, p="bf16", g="f32", master=False,
             bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance", "adamw"])
    any_type = lambda: rng.choice(["f32", "bf16", "f16"])   # noqa: E731
    if op in ("norm_fwd", "norm_bwd"):
        d = _log(rng, 32, 16384)
        d = d if rng.random() < 0.3 else max(32, d // 16 * 16)   # most widths are the layer's: multiples of 16
        rows = _log(rng, 1, max(1, min(65536, 16384 * 4096 // d)))
        x = any_type()
        if op == "norm_fwd":
            return dict(op=op, rows=rows, d=d, x=x, y=rng.choice([x, "bf16"]), w=rng.choice([x, "f32"]),
                        add=rng.choice(["", "f32", x]), stats=rng.random() < 0.5)
        return dict(op=op, rows=rows, d=d, x=x, dy=rng.choice([x, "f32"]), w=rng.choice([x, "f32"]),
                    dx=rng.choice([x, "f32"]), dsum=rng.random() < 0.5)
    if op == "balance":
        E = rng.choice([_log(rng, 2, 256), 8, 16, 64, 128, 256])
        T = _log(rng, 1, min(262144, 131072 * 256 // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=min(T, _log(rng, 1, 512)),
                    fn=rng.choice(["softmax", "sigmoid"]), z=rng.choice(["f32", "bf16"]), mask=rng.random() < 0.5)
    while True:
        d, E, F = 16 * _log(rng, 2, 160), _log(rng, 2, 128), 16 * _log(rng, 2, 160)
        F1 = F * rng.choice([1, 2])
        layers = _log(rng, 1, 32)
        if layers * E * d * (F + F1) <= 64 * 2048 * 1408 * 2:   # with the largest listed case at 12 bytes each
            break
    p = any_type()
    return dict(op=op, layers=layers, d=d, E=E, F=F, F1=F1, p=p, g=rng.choice(["f32", p]),
                master=p != "f32" and rng.random() < 0.5, bits=rng.choice([8, 32]))


# ------------------------------------------------------------------- inputs
def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(case, seed)
    return {"norm_fwd": _prepare_norm_fwd, "norm_bwd": _prepare_norm_bwd, "balance": _prepare_balance,
            "adamw": _prepare_adamw}[case["op"]](case, g)


def _norm_x(case, g):
    # a residual stream: rows of different size, a common offset, a few columns far larger than the rest
    x = _randn(g, case["rows"], case["d"]) * (0.5 + 2 * _rand(g, case["rows"], 1)) + 0.3
    x[:, :: max(1, case["d"] // 4)] *= 8.0
    return x.to(DT[case["x"]])


def _prepare_norm_fwd(case, g):
    rows, d, w = case["rows"], case["d"], DT[case["w"]]
    s = dict(case=case, x=_norm_x(case, g), gamma=(1 + 0.2 * _randn(g, d)).to(w), beta=(0.2 * _randn(g, d)).to(w))
    s["add"] = _randn(g, rows, d).to(DT[case["add"]]) if case["add"] else None
    s["y"] = torch.empty(rows, d, dtype=DT[case["y"]], device="cuda")
    s["sum"] = torch.empty_like(s["x"]) if case["add"] else None
    s["mean"] = torch.empty(rows, device="cuda") if case["stats"] else None
    s["rstd"] = torch.empty(rows, device="cuda") if case["stats"] else None
    return s


def _prepare_norm_bwd(case, g):
    rows, d, w = case["rows"], case["d"], DT[case["w"]]
    x = _norm_x(case, g)
    x32 = x.float()
    mean = x32.mean(1)
    rstd = torch.rsqrt((x32 - mean[:, None]).square_().mean(1) + EPS)   # what the forward has left
    del x32
    dy = _randn(g, rows, d).mul_(0.05 * _rand(g, rows, 1)).to(DT[case["dy"]])
    dsum = _randn(g, rows, d).mul_(0.02).to(DT[case["dx"]]) if case["dsum"] else None
    return dict(case=case, x=x, mean=mean, rstd=rstd, dy=dy, dsum=dsum, gamma=(1 + 0.2 * _randn(g, d)).to(w),
                dx=torch.empty(rows, d, dtype=DT[case["dx"]], device="cuda"),
                dgamma=torch.empty(d, device="cuda"), dbeta=torch.empty(d, device="cuda"))


def _prepare_balance(case, g):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    # a router with a skewed preference, per token noise
    z = _randn(g, T, E) * 1.2 - 0.5 * torch.log1p(torch.arange(E, device="cuda").float())
    z = z.to(DT[case["z"]])
    topk = torch.topk(z.float(), k, dim=1).indices.to(torch.int32)
    # ragged sequences; with a mask the last fifth of each and about a tenth of the rest is padding
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda", dtype=torch.int32)).values
    ends = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    off = torch.cat([ends[:1], cuts, ends[1:]]).contiguous()
    mask = None
    if case["mask"]:
        t = torch.arange(T, device="cuda")
        s = torch.searchsorted(off[1:].long(), t, right=True).clamp_(max=S - 1)
        lo, hi = off[s].long(), off[s + 1].long()
        mask = ((t - lo) * 5 < (hi - lo) * 4) & (_rand(g, T) > 0.1)
        mask = mask.to(torch.uint8)
    return dict(case=case, z=z, topk=topk, off=off, mask=mask, coef=torch.tensor(0.01, device="cuda"),
                counts=torch.empty(S, E, dtype=torch.int32, device="cuda"), loss=torch.empty(1, device="cuda"),
                dz=torch.empty_like(z))


def _sizes(case):
    """Element counts of the two groups: the experts' weights, and the norms and gates."""
    L, d, E, F, F1 = (case[n] for n in ("layers", "d", "E", "F", "F1"))
    return [E * F1 * d, E * d * F] * L, [d, d, E * d] * L


def _spans(sizes):
    """Places of the tensors in one flat buffer, each from a whole block on, and the buffer's length."""
    at, out = 0, []
    for n in sizes:
        out.append((at, n))
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return out, at


def _group(g, sizes, p, gr, master, bits, decay):
    spans, n = _spans(sizes)
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for at, m in spans:
        live[at:at + m] = True
    # gradients of different size from block to block, some blocks without any (experts that saw no token)
    level = 1e-3 * torch.exp(_randn(g, n // BLOCK, 1)) * (_rand(g, n // BLOCK, 1) > 0.1)
    grad = (_randn(g, n // BLOCK, BLOCK) * level).view(-1).mul_(live).to(DT[gr])
    p32 = (_randn(g, n) * 0.03).mul_(live)
    m = (_randn(g, n // BLOCK, BLOCK) * (0.3 * level)).view(-1).mul_(live)
    v = ((0.2 + _rand(g, n // BLOCK, BLOCK)) * level * level).view(-1).mul_(live)
    s = dict(param=p32.to(DT[p]), grad=grad, master=p32 if master else None, spans=spans, decay=decay, bits=bits)
    if bits == 32:
        s.update(m=m, v=v, ms=None, vs=None)
    else:
        s["m"], s["ms"] = _to_8bit(m, False)
        s["v"], s["vs"] = _to_8bit(v.sqrt_(), True)
    return s


def _prepare_adamw(case, g):
    big, small = _sizes(case)
    return dict(case=case, state=torch.tensor([FIRST_STEP, 0], dtype=torch.int32, device="cuda"),
                scale=torch.tensor(0.7, device="cuda"),   # gradient clipping's factor
                groups=[_group(g, big, case["p"], case["g"], case["master"], case["bits"], DECAY),
                        _group(g, small, "f32", "f32", False, 32, 0.0)])


# -------------------------------------------------------------- the operators
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "balance": _own_balance,
                "adamw": _own_adamw}[op](state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance,
            "adamw": _plain_adamw}[op](state)


def _plain_norm_fwd(s):
    h = s["x"].float()
    out = {}
    if s["add"] is not None:
        out["sum"] = (h + s["add"].float()).to(s["x"].dtype)
        h = out["sum"].float()
    mean = h.mean(1, keepdim=True)
    c = h - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    out["y"] = (c * rstd * s["gamma"].float() + s["beta"].float()).to(s["y"].dtype)
    if s["mean"] is not None:
        out["mean"], out["rstd"] = mean[:, 0], rstd[:, 0]
    return out


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    gy = dy * s["gamma"].float()
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["dx"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _plain_balance(s):
    case, z, off = s["case"], s["z"].float(), s["off"].long()
    T, E, S = case["T"], case["E"], case["S"]
    seq = torch.searchsorted(off[1:], torch.arange(T, device=z.device), right=True).clamp_(max=S - 1)
    live = s["mask"] != 0 if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=z.device)
    n = torch.zeros(S, device=z.device).index_add_(0, seq, live.float())
    slot = (seq[:, None] * E + s["topk"].long()).view(-1)
    counts = torch.zeros(S * E, dtype=torch.int32, device=z.device)
    counts.index_add_(0, slot, live[:, None].expand(-1, case["k"]).reshape(-1).to(torch.int32))
    counts = counts.view(S, E)
    f = E * counts.float() / counts.sum(1, keepdim=True).clamp(min=1).float()
    if case["fn"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        p, slope = e / e.sum(1, keepdim=True), 1.0
    else:
        q = 1 / (1 + torch.exp(-z))
        p, slope = q / q.sum(1, keepdim=True), 1 - q
    ft = f[seq]
    dot = (ft * p).sum(1, keepdim=True)
    weight = torch.where(live, 1 / (n[seq].clamp(min=1) * (n > 0).sum().clamp(min=1)), 0)[:, None]
    loss = (weight * dot).sum().view(1)
    dz = s["coef"] * weight * p * (ft - dot) * slope
    return {"loss": loss, "counts": counts, "dz": dz.to(s["z"].dtype)}


def _to_8bit(x, root):
    """E4M3 codes of x and the fp32 scale of each block of 256; a root that is not zero keeps a code that is not."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
    q = (b * (top.reciprocal() * 448.0)).clamp(-448.0, 448.0)
    if root:
        q = torch.where(b > 0, q.clamp(min=2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(-1), (top * (1.0 / 448.0)).view(-1)


def _from_8bit(q, scale):
    return (q.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _plain_group(s, scale, c1, c2):
    if s["bits"] == 8:
        m, r = _from_8bit(s["m"], s["ms"]), _from_8bit(s["v"], s["vs"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    g = s["grad"].float() * scale
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    p = s["master"] if s["master"] is not None else s["param"].float()
    p = p * (1 - LR * s["decay"]) - (LR / c1) * m / (root / torch.sqrt(c2) + ADAM_EPS)
    s["param"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if s["bits"] == 8:
        (qm, ms), (qv, vs) = _to_8bit(m, False), _to_8bit(root, True)
        s["m"].copy_(qm), s["ms"].copy_(ms), s["v"].copy_(qv), s["vs"].copy_(vs)
    else:
        s["m"].copy_(m), s["v"].copy_(v)


def _adamw_out(s):
    return [{n: x[n] for n in ("param", "master", "m", "v", "ms", "vs") if x[n] is not None} for x in s["groups"]]


def _plain_adamw(s):
    s["state"][0] += 1
    t = s["state"][0].double()
    c1, c2 = (1 - BETA1 ** t).float(), (1 - BETA2 ** t).float()
    _plain_group(s["groups"][0], s["scale"], c1, c2)
    _plain_group(s["groups"][1], s["scale"], c1, c2)
    return _adamw_out(s)


# ------------------------------------------------- the library's public calls
def _kept(s, make):
    """What a user's program makes once beside its buffers: the call's configuration, workspace or plan."""
    if "kept" not in s:
        s["kept"] = make(s)
    return s["kept"]


def _make_norm(s):
    import mixture_experts_layer_logit_b200 as moe
    c = s["case"]
    cfg = moe.make_norm_config(c["rows"], c["d"], eps=EPS, x=c["x"], y=c.get("y"), w=c["w"], add=c.get("add") or None,
                               dy=c.get("dy"), dx=c.get("dx"))
    ws = torch.empty(moe.moe_layer_norm_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    return moe, cfg, ws


def _own_norm_fwd(s):
    moe, cfg, _ = _kept(s, _make_norm)
    moe.moe_layer_norm_forward(cfg, s["x"], s["gamma"], s["beta"], s["y"], add=s["add"], sum=s["sum"],
                               mean=s["mean"], rstd=s["rstd"])
    return {n: s[n] for n in ("sum", "y", "mean", "rstd") if s[n] is not None}


def _own_norm_bwd(s):
    moe, cfg, ws = _kept(s, _make_norm)
    moe.moe_layer_norm_backward(cfg, s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], s["dx"], s["dgamma"],
                                s["dbeta"], ws, dsum=s["dsum"])
    return {n: s[n] for n in ("dx", "dgamma", "dbeta")}


def _make_balance(s):
    import mixture_experts_layer_logit_b200 as moe
    c = s["case"]
    cfg = moe.make_balance_config(c["T"], c["E"], c["k"], S=c["S"], score=c["fn"], dtype=c["z"])
    return moe, cfg, torch.empty(moe.moe_balance_workspace_size(cfg), dtype=torch.uint8, device="cuda")


def _own_balance(s):
    moe, cfg, ws = _kept(s, _make_balance)
    moe.moe_balance_loss(cfg, s["z"], s["topk"], s["counts"], s["loss"], ws, seq_offsets=s["off"], mask=s["mask"],
                         coef=s["coef"], dscores=s["dz"])
    return {"loss": s["loss"], "counts": s["counts"], "dz": s["dz"]}


def _make_adamw(s):
    import mixture_experts_layer_logit_b200 as moe
    tensors = []
    for x in s["groups"]:
        for at, n in x["spans"]:
            cut = lambda name: None if x[name] is None else x[name][at:at + n]   # noqa: E731
            block = lambda name: None if x[name] is None else x[name][at // BLOCK:(at + n + BLOCK - 1) // BLOCK]  # noqa: E731, E501
            tensors.append(moe.adamw_tensor(cut("param"), cut("grad"), cut("m"), cut("v"), m_scale=block("ms"),
                                            v_scale=block("vs"), master=cut("master"), weight_decay=x["decay"]))
    return moe, moe.make_adamw_plan(tensors, lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS)


def _own_adamw(s):
    moe, plan = _kept(s, _make_adamw)
    moe.moe_adamw_step(plan, s["state"], grad_scale=s["scale"])
    return _adamw_out(s)


# ------------------------------------------------------------------ the floor
def work(case):
    op = case["op"]
    if op == "norm_fwd":
        rows, d = case["rows"], case["d"]
        per = BYTES[case["x"]] + BYTES[case["y"]] + (BYTES[case["add"]] + BYTES[case["x"]] if case["add"] else 0)
        return {"bytes": rows * d * per + 2 * d * BYTES[case["w"]] + (8 * rows if case["stats"] else 0),
                "flops": 8 * rows * d}
    if op == "norm_bwd":
        rows, d = case["rows"], case["d"]
        per = BYTES[case["x"]] + BYTES[case["dy"]] + BYTES[case["dx"]] * (2 if case["dsum"] else 1)
        return {"bytes": rows * d * per + d * (BYTES[case["w"]] + 8) + 8 * rows, "flops": 14 * rows * d}
    if op == "balance":
        T, E = case["T"], case["E"]
        return {"bytes": 2 * T * E * BYTES[case["z"]] + 4 * T * case["k"] + (T if case["mask"] else 0)
                + 4 * case["S"] * (E + 1), "flops": 10 * T * E}
    big, small = (sum(v) for v in _sizes(case))
    per = BYTES[case["g"]] + (8 + BYTES[case["p"]] if case["master"] else 2 * BYTES[case["p"]])
    per += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": big * per + small * 28, "flops": 14 * (big + small)}


# ------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd, "balance": _exact_balance,
            "adamw": _exact_adamw}[case["op"]](s)


def _exact_norm_fwd(s):
    x, out = s["x"].double(), {}
    if s["add"] is not None:   # the stored sum is what is normalised: rounded to x's type
        x = x + s["add"].double()
        out["sum"], x = x, x.to(s["x"].dtype).double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False)
    rstd = (var + EPS) ** -0.5
    a = torch.outer(rstd, s["gamma"].double())
    out["y"] = (x - mean[:, None]) * a + s["beta"].double()
    if s["mean"] is not None:
        out["mean"], out["rstd"] = mean, rstd
    return out


def _exact_norm_bwd(s):
    # by the vector-Jacobian product of y = r (I - 11'/d) x: r P (I - xh xh'/d) P (gamma dy)
    d = s["case"]["d"]
    r, dy = s["rstd"].double()[:, None], s["dy"].double()
    xh = (s["x"].double() - s["mean"].double()[:, None]) * r
    dgamma, dbeta = torch.einsum("rc,rc->c", dy, xh), torch.einsum("rc->c", dy)
    gy = dy * s["gamma"].double()
    along = torch.einsum("rc,rc->r", gy, xh)[:, None] / d
    dx = gy.sub_(gy.sum(1, keepdim=True) / d).addcmul_(xh, along, value=-1).mul_(r)
    if s["dsum"] is not None:
        dx += s["dsum"].double()
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _exact_balance(s):
    c, off = s["case"], s["off"].cpu().long()
    E, S = c["E"], c["S"]
    z = s["z"].double()
    live = torch.ones(c["T"], dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"].bool()
    used = []   # per sequence: its live tokens
    for i in range(S):
        lo, hi = int(off[i]), int(off[i + 1])
        used.append(lo + torch.nonzero(live[lo:hi]).view(-1))
    G = sum(len(u) > 0 for u in used)
    counts = torch.zeros(S, E, dtype=torch.int32, device=z.device)
    dz, loss = torch.zeros_like(z), torch.zeros(1, dtype=torch.float64, device=z.device)
    for i, u in enumerate(used):
        if len(u) == 0:
            continue
        counts[i] = torch.bincount(s["topk"][u].reshape(-1).long(), minlength=E).to(torch.int32)
        f = counts[i].double() * (E / float(counts[i].sum()))
        if c["fn"] == "softmax":
            p, fall = torch.softmax(z[u], 1), 1.0
        else:
            q = torch.sigmoid(z[u])
            p, fall = q / q.sum(1, keepdim=True), torch.sigmoid(-z[u])
        dot = p @ f
        loss += dot.mean() / G
        dz[u] = p * (f - dot[:, None]) * fall * (float(s["coef"]) / (G * len(u)))
    return {"loss": loss, "counts": counts, "dz": dz}


def _exact_adamw(s):
    t, scale = FIRST_STEP + 1, float(s["scale"])
    return [_exact_group(x, t, scale) for x in s["groups"]]


def _exact_group(x, t, scale):
    if x["bits"] == 8:
        m = x["m"].double().view(-1, BLOCK) * x["ms"].double()[:, None]
        v = (x["v"].double().view(-1, BLOCK) * x["vs"].double()[:, None]) ** 2
        m, v = m.view(-1), v.view(-1)
    else:
        m, v = x["m"].double(), x["v"].double()
    g = x["grad"].double() * scale
    m.lerp_(g, 1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    del g
    p = (x["master"] if x["master"] is not None else x["param"]).double()
    denom = (v / (1 - BETA2 ** t)).sqrt_().add_(ADAM_EPS)
    p.mul_(1 - LR * x["decay"]).addcdiv_(m, denom, value=-LR / (1 - BETA1 ** t))
    del denom
    out = {"param": p}
    if x["master"] is not None:
        out["master"] = p
    if x["bits"] == 32:
        return {**out, "m": m, "v": v}
    # the codes themselves sit on a rounding border now and then; their scales are numbers
    root = v.sqrt_()
    return {**out, "m": None, "v": None, "ms": m.view(-1, BLOCK).abs().amax(1).clamp(min=2.0 ** -100) / 448,
            "vs": root.view(-1, BLOCK).amax(1).clamp(min=2.0 ** -100) / 448}
