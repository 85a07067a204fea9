"""Offsets past 32 bits and the largest row counts of the operators around the
layer: the end of a long operand gives what it gives on its own."""
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def ws(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")


def test_norm_of_more_than_2_to_the_31_elements():
    d, tail = 4096, 5
    rows = (1 << 31) // d + tail
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_()
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    g = torch.linspace(0.5, 1.5, d, device="cuda")
    cfg = moe.make_norm_config(rows, d, dy="bf16")
    moe.moe_layer_norm_forward(cfg, x, g, None, y, mean=mean, rstd=rstd)
    moe.moe_layer_norm_backward(cfg, x, x, mean, rstd, g, dx)
    end = moe.make_norm_config(tail, d, dy="bf16")
    y2, dx2 = (torch.empty(tail, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m2, r2 = torch.empty(tail, device="cuda"), torch.empty(tail, device="cuda")
    xt = x[-tail:].clone()
    moe.moe_layer_norm_forward(end, xt, g, None, y2, mean=m2, rstd=r2)
    moe.moe_layer_norm_backward(end, xt, xt, m2, r2, g, dx2)
    for a, b in ((y, y2), (dx, dx2), (mean, m2), (rstd, r2)):
        assert torch.equal(a[-tail:], b)
    assert bool(y[rows // 2].any()) and bool(dx[rows // 2].any())


def test_norm_of_almost_2_to_the_31_rows():
    rows = (1 << 31) - 3   # the last block's rows would be past 2^31
    x = torch.full((rows,), 2.0, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    cfg = moe.make_norm_config(rows, 1)
    moe.moe_layer_norm_forward(cfg, x, None, torch.full((1,), 0.75, device="cuda"), y)
    assert int((y != 0.75).sum()) == 0


def test_balance_of_more_than_2_to_the_31_scores():
    E, tail, k = 256, 300, 2
    T = (1 << 31) // E + tail
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z[-tail:].normal_()
    topk = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    topk[-tail:] = torch.topk(z[-tail:].float(), k).indices.int()
    off = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")

    def run(z, topk, S, off):
        cfg = moe.make_balance_config(z.shape[0], E, k, S, "softmax", "bf16")
        C, loss = torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
        dz = torch.ones_like(z)
        moe.moe_balance_loss(cfg, z, topk, C, loss, ws(moe.moe_balance_workspace_size(cfg)), seq_offsets=off,
                             dscores=dz, coef=torch.tensor(1024.0, device="cuda"))
        return C, float(loss), dz

    C, loss, dz = run(z, topk, 2, off)
    c, l, d = run(z[-tail:].clone(), topk[-tail:].clone(), 1, None)
    assert torch.equal(C[1:], c) and int(C[0, 0]) == (T - tail) * k
    # the long sequence is uniform: its loss is 1, and each sequence weighs half.  A token's experts may lie in another
    # number of lanes: sums of 64 roundings (2^-24) at most, of terms p f and dot <= max f, p <= 1, times
    # coef / (G n) = 1024 / 600; and half a bf16 step on each side
    f = E * c.max().item() / (tail * k)
    far = (dz[-tail:].float() - d.float() / 2).abs()
    assert abs(loss - (1 + l) / 2) < 1e-5
    assert bool((far <= 2.0 ** -7 * d.float().abs() / 2 + 2 * 64 * 2.0 ** -24 * 2 * f * 1024 / 600).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_of_more_than_2_to_the_31_elements(bits):
    tail = 1000
    n = (1 << 31) // 256 * 256 + tail
    p = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-tail:].normal_()
    small = moe.adamw_states(torch.empty(tail, device="cuda"), bits)
    big = moe.adamw_states(p, bits)
    q, gq = p[-tail:].clone(), g[-tail:].clone()
    for tensors in ((p, g, big), (q, gq, small)):
        t = moe.adamw_tensor(tensors[0], tensors[1], tensors[2][0], tensors[2][1], m_scale=tensors[2][2],
                             v_scale=tensors[2][3], weight_decay=0.1)
        moe.moe_adamw_step(moe.make_adamw_plan([t], lr=0.1), torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert torch.equal(p[-tail:], q)
    for a, b in zip(big[:2], small[:2]):
        assert torch.equal(a[-tail:].view(torch.uint8), b.view(torch.uint8))
    assert float(p[n // 2]) == float(p[0]) != 1.0
