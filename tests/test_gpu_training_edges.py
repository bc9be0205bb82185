"""The operators of a training step where a documented promise is easily lost: padding
beside infinite gradients. Against 64 bits, with bounds derived beside each test; on both builds."""
import numpy as np
import pytest
import torch

import precision_collective_reduction_gb300 as pcr
from test_gpu_training import DT, dev, f64, gen, lib, same  # noqa: F401 (lib: a fixture)

pytestmark = pytest.mark.gpu


# -- balance loss: padding ------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E", [(5, 8), (40, 65), (33, 256), (20, 384), (9, 1000)])
@pytest.mark.parametrize("dloss", [float("inf"), float("nan")])
def test_padding_has_no_gradient_whatever_the_loss_has(lib, dt, T, E, dloss):
    g = gen(T, E, 21)
    z = g.normal(size=(T, E))
    valid = np.arange(T) % 3 != 1
    z[~valid] = np.nan
    logits, v = dev(z, dt), torch.from_numpy(valid).cuda()
    counts = torch.from_numpy(np.append(np.arange(E) % 5, valid.sum()).astype(np.int32)).cuda()
    d = torch.full((1,), dloss, device="cuda")
    dz = torch.full((T, E), 7.0, device="cuda").to(DT[dt])
    pcr.expert_balance_backward(logits, counts, d, dz, valid=v)
    assert not dz[~v].any()
    assert not torch.isfinite(dz[v].float()).all()      # where there is a loss, it shows
    before = dev(g.normal(size=(T, E)), dt)
    more = before.clone()
    pcr.expert_balance_backward(logits, counts, d, more, valid=v, accumulate=True)
    assert same(more[~v], before[~v])
