"""Balance loss with one operand at a time off the alignment of the others,
under the element-wise bounds of the suite."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_logit_b200 as moe
from tests.test_gpu_block_ops import check_balance, router

pytestmark = pytest.mark.gpu

NAMES = ["scores", "topk_idx", "counts", "loss", "seq_offsets", "mask", "coef", "dscores"]


def moved(t, off):
    """Room of t's size off elements into a buffer whose start is aligned to 256 bytes, with t's contents."""
    buf = torch.zeros(t.numel() + off, dtype=t.dtype, device=t.device)
    buf[off:].copy_(t.reshape(-1))
    return buf[off:].view(t.shape)


# the single block and the three kernels; experts in quads, filled or not
@pytest.mark.parametrize("T,E,k,S", [(60, 16, 2, 3), (90, 64, 4, 2), (4000, 24, 2, 5), (3000, 256, 8, 7)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("names", [[n] for n in NAMES] + [NAMES], ids=NAMES + ["all"])
def test_operands_off_their_alignment(monkeypatch, T, E, k, S, dt, off, names):
    r = np.random.default_rng([T, E, off])
    z, topk = router(r, T, E, k)
    cuts = np.sort(r.integers(0, T + 1, S + 1)).astype(np.int32)
    mask = (r.random(T) > 0.2).astype(np.uint8)
    plain = moe.moe_balance_loss

    def call(cfg, scores, topk_idx, counts, loss, ws, **kw):
        args = dict(scores=scores, topk_idx=topk_idx, counts=counts, loss=loss, ws=ws, **kw)
        for n in names:
            args[n] = moved(args[n], off)
        plain(cfg, **args)
        for n, t in (("counts", counts), ("loss", loss), ("dscores", kw["dscores"])):
            if n in names:
                t.copy_(args[n])

    monkeypatch.setattr(moe, "moe_balance_loss", call)
    check_balance(z, topk, k, S, cuts, mask, "softmax" if S % 2 else "sigmoid", dt)
