"""AdamW with one operand at a time off the alignment of the others, at every
step from one element to a whole vector, under the element-wise bounds and the
exact codes of the suite."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe
from tests.test_gpu_block_ops import B1, B2, EPS, LR, adam_case, check_adam, new_state

pytestmark = pytest.mark.gpu

SIZES = [3, 256, 2300, 9001]   # less than a block, one, more than a tile with a short last block


def shifted(t, off):
    """A copy that starts off elements into its buffer, whose start is aligned to 256 bytes."""
    buf = torch.zeros(t.numel() + off, dtype=t.dtype, device=t.device)
    buf[off:].copy_(t)
    return buf[off:]


@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("bf16", "f32", True), ("bf16", "bf16", False),
                                        ("f16", "f32", False), ("f32", "f16", False)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("name", ["param", "grad", "master", "m", "v", "all"])
def test_one_operand_off(p, g, master, bits, name):
    if name == "master" and not master:
        pytest.skip("no master copies")
    r = np.random.default_rng([bits, 21])
    cases = []
    for off in (1, 2, 4, 8, 16):
        for n in SIZES:
            t, s = adam_case(r, n, p, g, bits, master, 0.1)
            for k in ("param", "grad", "master", "m", "v") if name == "all" else (name,):
                if t[k] is not None:
                    t[k] = shifted(t[k], off)
                    assert (t[k].data_ptr() - off * t[k].element_size()) % 256 == 0
            cases.append((t, s))
    state = new_state(4)
    moe.moe_adamw_step(moe.make_adamw_plan([t for t, _ in cases], lr=LR, beta1=B1, beta2=B2, eps=EPS), state)
    torch.cuda.synchronize()
    for t, s in cases:
        check_adam(t, s, 5, 1.0, p)


@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_packed_in_one_buffer(bits):
    """Tensors whose gradients lie one after the other in a flat buffer, from 16-byte boundaries on, over several
    tiles a block; what lies between them is left alone and the same gradients on their own give the same bits."""
    r = np.random.default_rng([bits, 22])
    sizes = [5, 700_004, 256, 900_001, 12, 650_003]
    cases = [adam_case(r, n, "bf16", "f32", bits, True, 0.1) for n in sizes]
    twins = [{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in t.items()} for t, _ in cases]
    at, places = 0, []
    for n in sizes:
        at += 4 if (at // 4) % 2 == 0 else 0   # an odd multiple of four elements
        places.append(at)
        at += (n + 3) // 4 * 4
    flat = torch.full((at,), float("nan"), device="cuda")
    for (t, _), lo, n in zip(cases, places, sizes):
        flat[lo:lo + n].copy_(t["grad"])
        t["grad"] = flat[lo:lo + n]
        assert t["grad"].data_ptr() % 32 == 16
    before = flat.clone()
    states = [new_state(1), new_state(1)]
    for tensors, state in (([t for t, _ in cases], states[0]), (twins, states[1])):
        moe.moe_adamw_step(moe.make_adamw_plan(tensors, lr=LR, beta1=B1, beta2=B2, eps=EPS), state)
    torch.cuda.synchronize()
    assert torch.equal(flat.view(torch.int32), before.view(torch.int32))
    for (t, s), w in zip(cases, twins):
        check_adam(t, s, 2, 1.0, "bf16")
        for k in ("param", "master", "m", "v"):
            assert torch.equal(t[k].view(torch.uint8), w[k].view(torch.uint8)), k
