"""The operators of a training step where a documented promise is easily lost: padding
beside infinite gradients, small probabilities, rows whose mean is large beside their
spread. Against 64 bits, with bounds derived beside each test; on both builds."""
import numpy as np
import pytest
import torch

import precision_collective_reduction_gb300 as pcr
import training_ref as ref
from test_gpu_training import DT, dev, f64, gen, lib, same, within  # noqa: F401 (lib: a fixture)

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


# -- norm gradients of rows far from zero ---------------------------------------

def far_rows(g, T, H, dt):
    """Rows whose mean is known exactly, in every order of summation: neighbouring
    columns lie the same step above and below it, the steps are multiples of one power
    of 2, and H is a power of 2."""
    mean, steps, unit = (1000.0, 2048, 2.0 ** -10) if dt == "f32" else (192.0, 63, 1.0)
    k = g.integers(1, steps + 1, size=(T, H // 2)) * unit
    x = np.empty((T, H))
    x[:, 0::2], x[:, 1::2] = mean + k, mean - k
    return x, mean


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(160, 8), (700, 256), (310, 1024), (160, 4096), (155, 8192),
                                 (155, 16384), (3, 512), (40, 4096)])
@pytest.mark.parametrize("dropout", [False, True])
def test_norm_gradients_of_rows_far_from_zero(lib, dt, T, H, dropout):
    # The row's mean m comes out exactly (far_rows), and so does x - m (both are multiples
    # of the unit, and the difference is shorter). Left are the errors of the squares'
    # sum and of r, of the products, and of the sums of q and q xh: none grows with m.
    # (Formed as r x - r m, xh would be off by half an ulp of r m, 1.2e-4 in FP32 here.)
    g = gen(T, H, 23)
    x, mean = far_rows(g, T, H, dt)
    xd = dev(x, dt)
    assert np.array_equal(f64(xd), x)
    eps = float(np.float32(1e-5))
    c = x - mean
    v = (c * c).mean(1, keepdims=True)
    r = 1 / np.sqrt(v + eps)
    xh = c * r
    er = 0.5 * (ref.DEEP + 10) * ref.U + 8 * ref.U      # the squares' sum; rsqrtf, 2 ulp
    exh = np.abs(xh) * (er + 3 * ref.U)
    # a gradient along xh, whose part in dx is what the mean's rounding would change; of
    # one token only, so that dw is that token's term itself
    at = T // 2
    dn = np.zeros((T, H))
    dn[at] = xh[at] + 0.25 * g.normal(size=H)
    dn = dev(dn, dt)
    q = f64(dn)
    dx, dh, dw, db = (torch.empty(T, H, device="cuda").to(DT[dt]), None,
                      torch.empty(H, device="cuda"), torch.empty(H, device="cuda"))
    keep, p = np.ones((T, H), bool), 0.0
    if dropout:
        p, rng = 0.3, torch.tensor([T, H], device="cuda")
        keep = ref.kept(T, H, T, H, p)
        dh = torch.empty_like(dx)
    aq, mq = np.abs(q).mean(1, keepdims=True), q.mean(1, keepdims=True)
    s = (q * xh).mean(1, keepdims=True)
    es = ((ref.DEEP + ref.OPS) * ref.U * 3 * aq * np.abs(xh).max(1, keepdims=True)
          + (np.abs(q) * exh).mean(1, keepdims=True))
    inner = q - mq - xh * s
    D = r * inner
    eD = (ref.OPS * ref.U * r * (np.abs(q) + aq + np.abs(xh * s))
          + r * ((ref.DEEP + ref.OPS) * ref.U * aq + exh * np.abs(s) + np.abs(xh) * es)
          + 2 * er * r * (np.abs(inner) + np.abs(xh * s)))
    want_dx = (D, ref.HALF_ULP[dt] * np.abs(D) * ref.SLACK + eD * ref.SLACK + ref.TINY)
    f = keep / (1 - float(np.float32(p)))
    want_dh = (D * f, ref.HALF_ULP[dt] * np.abs(D * f) * ref.SLACK
               + (eD + 3 * ref.U * np.abs(D)) * f * ref.SLACK + ref.TINY)
    e_dw = (np.abs(q) * exh + 2 * ref.U * np.abs(q * xh)).sum(0)
    want_dw = ((q * xh).sum(0), e_dw * ref.SLACK + ref.TINY)

    def check():
        within(dw, want_dw, "dw")
        assert np.array_equal(f64(db), q.sum(0))
    if dropout:
        kw = dict(eps=eps, dw=dw, db=db)
        pcr.residual_dropout_backward(torch.zeros_like(dx), dn, xd, dx, dh, rng, p, **kw)
        within(dx, want_dx, "dx")
        within(dh, want_dh, "dh")
        check()
        pcr.residual_dropout_backward(None, dn, xd, None, dh, rng, p, **kw)
        within(dh, want_dh, "dh alone")
        check()
        pcr.residual_dropout_backward(None, dn, xd, dx, None, rng, p, **kw)
        within(dx, want_dx, "dx alone")
    else:
        pcr.layer_norm_backward(dn, xd, dx, eps=eps, dw=dw, db=db)
        within(dx, want_dx, "dx")
        check()
        pcr.layer_norm_backward(dn, xd, None, eps=eps, dw=dw, db=db)
    check()


# -- embedding: ids of the shard --------------------------------------------------

@pytest.mark.parametrize("first", [1 << 63, -(1 << 63) - 1, 1 << 64])
def test_first_ids_that_are_no_64_bit_numbers_are_refused(first):
    # taken modulo 2^64 they would stand for other ids
    table, ids = torch.ones(4, 8, device="cuda"), torch.tensor([0, -(1 << 63)], device="cuda")
    out, d = torch.empty(2, 8, device="cuda"), torch.empty(4, 8, device="cuda")
    with pytest.raises(ValueError):
        pcr.token_embed(table, ids, out, first_id=first)
    with pytest.raises(ValueError):
        pcr.token_embed_backward(out, ids, d, first_id=first)


@pytest.mark.parametrize("kind", [int, np.int64, np.int32, torch.tensor])
def test_first_ids_of_every_integer_type(kind):
    table = torch.randn(4, 8, device="cuda")
    ids = torch.tensor([7, 9, 10, 11], device="cuda")
    out, d = torch.empty(4, 8, device="cuda"), torch.empty(4, 8, device="cuda")
    pcr.token_embed(table, ids, out, first_id=kind(7))
    assert same(out[:3], table[[0, 2, 3]]) and not out[3].any()
    pcr.token_embed_backward(table, ids, d, first_id=kind(7))
    assert same(d[[0, 2, 3]], table[:3]) and not d[1].any()
    with pytest.raises(TypeError):
        pcr.token_embed(table, ids, out, first_id=7.0)
