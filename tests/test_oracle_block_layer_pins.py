"""The balance oracle over one whole batch is the layer oracle's auxiliary loss."""
import numpy as np
import pytest

import moe_workloads as mw
import oracle
from oracle import block_ops as ob
from oracle import moe_oracle as om


@pytest.mark.parametrize("lam,k,cap", [(0.0, 2, 0.0), (1.0, 3, 1.0)])
def test_one_sequence_gives_the_layers_aux_loss(lam, k, cap):
    """Counts before the capacity drops, probabilities of the scores that the softmax takes: the same float64 sums in
    another order, some hundred terms of size one."""
    w = mw.Workload("aux_pin", T=150, d=24, E=7, F=16, k=k, act=mw.RELU, dtype=mw.F32, capacity_factor=cap, lam=lam,
                    zipf_bias=True, seed=12)
    inp = mw.generate(w)
    x, wg, w1, w2 = (mw.to_f64(a) for a in (inp.x, inp.wg, inp.w1, inp.w2))
    fw = om.forward(x, wg, inp.bias, w1, w2, oracle.LayerConfig.from_workload(w))
    loss, counts, _ = ob.balance(fw.routing.s, fw.routing.idx, k, w.E)
    assert np.array_equal(counts[0], fw.dispatch.counts)
    assert loss == pytest.approx(fw.dispatch.aux, rel=1e-12)
