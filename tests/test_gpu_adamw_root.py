"""The AdamW step's own square root is the correctly rounded one.  It shows in
the scales of 8-bit states: a block of 256 equal second moments v gets the
scale fl(root(v) / 448), which tells neighbouring roots apart wherever the
product stays in the root's binade (mantissas below 1.75).

Any v is reached exactly: with beta2 = 1/2, a state q^2 just below 2 v and a
gradient g with g^2 near 2 v - q^2, whose own rounding is far below half a step
of v."""
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe

pytestmark = pytest.mark.gpu

BLOCK = moe.MOE_ADAMW_BLOCK
CHUNK = 1 << 19   # blocks at a time: 134 M elements


def check(t):
    """t: fp32 second moments, one per block."""
    n = t.numel()
    t64 = t.double()
    q = torch.sqrt(2 * t64).float()
    q = torch.where(q.double() ** 2 > 2 * t64 * (1 - 2.0 ** -23), torch.nextafter(q, torch.zeros_like(q)), q)
    q = torch.nextafter(q, torch.zeros_like(q))
    left = 2 * t64 - (q * q).double()
    assert bool((left > 0).all()) and bool((left < 2 * t64 * 2.0 ** -20).all())
    g = torch.sqrt(left).float()
    grad = g.repeat_interleave(BLOCK)
    p = torch.zeros(n * BLOCK, dtype=torch.bfloat16, device="cuda")
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    m, v = torch.zeros(n * BLOCK, dtype=torch.uint8, device="cuda"), torch.full((n * BLOCK,), one, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(n, device="cuda"), q.clone()
    plan = moe.make_adamw_plan([moe.adamw_tensor(p, grad, m, v, m_scale=ms, v_scale=vs)], beta1=0.5, beta2=0.5)
    moe.moe_adamw_step(plan, torch.zeros(2, dtype=torch.int32, device="cuda"))
    # the construction: the kernel's fp32 steps give t itself
    assert torch.equal((q * q) * 0.5 + (g * g) * 0.5, t)
    want = torch.sqrt(t64).float() * torch.tensor(1.0 / 448, device="cuda")   # sqrt of a double rounds to fp32 only once
    off = torch.nonzero(vs.view(torch.int32) != want.view(torch.int32)).view(-1)
    assert off.numel() == 0, [(float(t[i]).hex(), float(vs[i]).hex(), float(want[i]).hex()) for i in off[:5]]


@pytest.mark.parametrize("exponent", [0, 1])
def test_every_mantissa(exponent):
    """All 2^23 mantissas of an even and of an odd exponent; others are these times a power of four."""
    for lo in range(0, 1 << 23, CHUNK):
        bits = torch.arange(lo, lo + CHUNK, dtype=torch.int32, device="cuda") + ((127 + exponent) << 23)
        check(bits.view(torch.float32))


@pytest.mark.parametrize("exponent", [-100, -99, -60, -21, 30, 63, 100, 125])
def test_ends_of_the_range(exponent):
    """From 2^-100 on, the smallest that the hand-written root takes, to near the largest float."""
    bits = torch.arange(0, 1 << 23, 997, dtype=torch.int32, device="cuda") + ((127 + exponent) << 23)
    check(bits.view(torch.float32))
