"""The operators of a training step where a documented promise is easily lost: padding
beside infinite gradients, small probabilities. Against 64 bits, with bounds derived beside each test; on both builds."""
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


# -- balance loss: small probabilities ------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("E", [3, 64, 100, 256, 384, 1024])
@pytest.mark.parametrize("T", [1, 700])
def test_small_probabilities_have_all_their_digits(lib, dt, E, T):
    # One token that counts, with one logit 0 and all others from -40 to -100: the
    # softmax's sum is 1 in FP32 (and 1 + 1024 e^-40 = 1 + 5e-15 in truth), so every
    # probability is the exponential itself, whose argument is exact. expf is good to 2
    # ulp, at most 2 * 2^-23 of a normal value and 2 * 2^-149 below them; the sums over
    # tokens add zeros to it, and the division by 1 and the product with 1 are exact.
    at = T // 2 + T // 4
    z = np.full((T, E), 1.0)
    z[at] = np.linspace(-40.0, -100.0, E) - 0.0137
    z[at, E // 2] = 0.0
    logits = dev(z, dt)
    valid = np.arange(T) == at
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    loss, counts, sums = (torch.empty(1, device="cuda"),
                          torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                          torch.empty(E, device="cuda"))
    pcr.expert_balance(logits, ids, loss, counts, sums, valid=torch.from_numpy(valid).cuda())
    want = np.exp(f64(logits)[at])
    off = np.abs(f64(sums) - want)
    assert (off <= 2 * 2.0 ** -23 * want + 2 * 2.0 ** -149).all(), (off / want).max()
    assert counts.tolist() == [1] + [0] * (E - 1) + [1]
