"""Corners of the operators around the collectives."""
import warnings

import numpy as np
import pytest
import torch

import layers_ref as ref
import precision_collective_reduction_gb300 as pcr
from test_gpu_layers import DT, Out, dev, f64, lib, norm_case, opt64, rng, within  # noqa: F401

pytestmark = pytest.mark.gpu


# -- barriers of teams whose last warp lacks columns -------------------------------

@pytest.mark.parametrize("T", [9, 700])
@pytest.mark.parametrize("dt,H", [("bf16", 1025), ("bf16", 2051), ("bf16", 4097), ("bf16", 2050),
                                  ("bf16", 1028), ("f32", 1025), ("f32", 2051), ("f32", 1026)])
def test_equal_rows_are_equal_in_every_team(lib, dt, T, H):  # noqa: F811
    # 9 rows: clusters; 700: several teams in a CTA (1025 to 1028 columns) or one, with
    # accesses of 2, 4 and 8 bytes. A sum read before all warps have written theirs
    # would make a row differ from the others, or from itself a run later.
    g, (h,), x, gate, wq, wp = norm_case(1, H, dt, "channel", True, True)
    dxo, dn = dev(g.normal(size=(1, H)), dt), dev(g.normal(size=(1, H)), dt)
    kw = dict(gate=gate, gate_kind="channel", w_post=wq, w_pre=wp, res_scale=0.9,
              branch_scale=0.7, eps=1e-5)
    hs, xs, dxs, dns = (t.expand(T, H).contiguous() for t in (h, x, dxo, dn))
    first = None
    for _ in range(15):
        xo, n, dx, dh = (torch.full_like(xs, float("nan")) for _ in range(4))
        dw = [torch.full((H,), float("nan"), device="cuda") for _ in range(3)]
        pcr.residual_norm(hs, xs, xo, n, **kw)
        pcr.residual_norm_backward(dxs, dns, hs, xs, dx, dh, dgate=dw[0], dw_post=dw[1],
                                   dw_pre=dw[2], **kw)
        for t in (xo, n, dx, dh):
            assert torch.equal(t, t[:1].expand(T, H))
        first = first or (xo, n, dx, dh, *dw)
        for a, b in zip(first, (xo, n, dx, dh, *dw)):
            assert torch.equal(a, b)
    a, b, eps = (float(np.float32(v)) for v in (0.9, 0.7, 1e-5))
    want = ref.residual_norm([f64(h)], f64(x), f64(gate), "channel", f64(wq), f64(wp), a, b, eps,
                             dt)
    within(xo[:1], want[0], "x_out")
    within(n[:1], want[1], "n_out")
    want = ref.residual_norm_backward(f64(dxo), f64(dn), f64(h), f64(x), f64(gate), "channel",
                                      f64(wq), f64(wp), a, b, eps, dt)
    within(dx[:1], want["dx"], "dx")
    within(dh[:1], want["dh"], "dh")


# -- a gate of one dimension where [T] and [H] are the same shape --------------

def test_gate_that_two_kinds_fit_is_reported():
    T = H = 6
    g, (h,), x, gate, wq, wp = norm_case(T, H, "f32", "token", True, True)
    out = [torch.empty_like(x) for _ in range(4)]
    dgate = torch.empty(T, device="cuda")
    kw = dict(gate=gate, w_post=wq, w_pre=wp)
    with pytest.warns(UserWarning, match="gate_kind"):
        pcr.residual_norm(h, x, out[0], out[1], **kw)
    with pytest.warns(UserWarning, match="gate_kind"):
        pcr.residual_norm_backward(x, x, h, out[0], out[2], out[3], dgate=dgate, **kw)
    a, b, eps = 1.0, 1.0, float(np.float32(1e-6))
    for kind in ("channel", "token"):
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            pcr.residual_norm(h, x, out[0], out[1], gate_kind=kind, **kw)
            pcr.residual_norm_backward(x, x, h, out[0], out[2], out[3], dgate=dgate,
                                       gate_kind=kind, **kw)
        want = ref.residual_norm([f64(h)], f64(x), f64(gate), kind, f64(wq), f64(wp), a, b, eps,
                                 "f32")
        within(out[0], want[0], "x_out, " + kind)
        within(out[1], want[1], "n_out, " + kind)
        want = ref.residual_norm_backward(f64(x), f64(x), f64(h), f64(out[0]), f64(gate), kind,
                                          f64(wq), f64(wp), a, b, eps, "f32")
        for got, name in ((out[2], "dx"), (out[3], "dh"), (dgate, "dgate")):
            within(got, want[name], name + ", " + kind)


def test_gate_that_one_kind_fits_is_not_reported():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for T, H in ((6, 5), (1, 1)):  # of one value both kinds are the same
            x, out = torch.ones(T, H, device="cuda"), torch.empty(T, H, device="cuda")
            for n in {T, H}:
                pcr.residual_norm(x, x, out, gate=torch.full((n,), 2.0, device="cuda"))
                assert bool((out == 3).all())
            pcr.residual_norm(x, x, out, gate=torch.full((T, H), 2.0, device="cuda"))
            assert bool((out == 3).all())


# -- the router's gradient far below the largest logit --------------------------

def test_route_gradient_of_small_probabilities(lib):  # noqa: F811
    # Logits are multiples of 1/8 below 128, so that z - max is exact. With one
    # choice m = w dw. Allowed for p m, p = e^d / S of E experts: expf 2 ulp = 4 u,
    # S (E - 1) u, its quotient, m and the last rounding u each, that is (E + 6) u,
    # or, where e^d is subnormal, 2 of its ulps of 2^-149; a factor 1 + 2^-8 covers
    # products of these.
    T, E = 4000, 8
    g = rng(T, E)
    z = -g.integers(160, 827, size=(T, E)) / 8.0     # e^-20 down to e^-103.25
    top = g.integers(0, E, size=T)
    z[np.arange(T), top] = 0.0
    out = Out()
    ids, w, dl = out(T, 1, dtype=torch.int32), out(T, 1), out(T, E)
    pcr.expert_route(dev(z), ids, w)
    assert np.array_equal(ids.cpu().numpy()[:, 0], top)
    dw = ((1 + g.random((T, 1))) * 2.0 ** 100).astype(np.float32)
    pcr.expert_route_backward(dev(z), ids, w, dev(dw), dl)
    p = np.exp(z) / np.exp(z).sum(1, keepdims=True)
    m = f64(w) * dw.astype(np.float64)
    bound = m * ((E + 6) * ref.U * p + 2.0 ** -148) * (1 + 2.0 ** -8) + ref.TINY
    rest = np.arange(E) != top[:, None]              # the chosen one cancels: not of interest
    got = f64(dl)
    off = np.abs(got + p * m)[rest]
    assert (off <= bound[rest]).all(), "worst %g times the bound" % (off / bound[rest]).max()
    assert out.intact()


# -- outputs without a gradient --------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,post", [(None, True), ("channel", True), ("token", False),
                                       ("full", True)])
@pytest.mark.parametrize("T,H", [(1, 7), (40, 768), (200, 1025)])
def test_norm_gradient_without_that_of_n_out(lib, dt, kind, post, T, H):  # noqa: F811
    # as if there were no second norm, whose weight's gradient is 0
    g, (h,), xo, gate, wq, wp = norm_case(T, H, dt, kind, post, True)
    dxo = dev(g.normal(size=(T, H)), dt)
    kw = dict(gate=gate, gate_kind=kind, w_post=wq, res_scale=0.9, branch_scale=0.7, eps=1e-5)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        out = Out()
        dx, dh = out(T, H, dtype=DT[dt]), out(T, H, dtype=DT[dt])
        grads = {}
        if kind:
            grads["dgate"] = (out(T, H, dtype=DT[dt]) if kind == "full"
                              else out(H if kind == "channel" else T))
        if post:
            grads["dw_post"] = out(H)
        same = [torch.empty_like(dx), torch.empty_like(dh),
                {k: torch.empty_like(v) for k, v in grads.items()}]
        pcr.residual_norm_backward(dxo, None, h, xo, same[0], same[1], **kw, **same[2])
        dw_pre = out(H)
        dw_pre.fill_(7.0)
        torch.cuda.synchronize()
        pcr.residual_norm_backward(dxo, None, h, xo, dx, dh, w_pre=wp, dw_pre=dw_pre,
                                   stream=stream, **kw, **grads)
        torch.cuda.synchronize()
        assert torch.equal(dx, same[0]) and torch.equal(dh, same[1])
        for k, v in grads.items():
            assert torch.equal(v, same[2][k]), k
        assert not bool(dw_pre.any())
        assert out.intact()
    want = ref.residual_norm_backward(f64(dxo), None, f64(h), f64(xo), opt64(gate), kind,
                                      opt64(wq), None, *(float(np.float32(v))
                                                         for v in (0.9, 0.7, 1e-5)), dt)
    within(dx, want["dx"], "dx")
    within(dh, want["dh"], "dh")


def test_norm_gradient_of_neither_output_is_refused():
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        pcr.residual_norm_backward(None, None, x, x, x, x, w_pre=w)


# -- rows of no elements ----------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_token_gate_of_rows_without_elements(lib, dt):  # noqa: F811
    # a sum over no channels is 0
    e = torch.empty(5, 0, dtype=DT[dt], device="cuda")
    gate = torch.ones(5, dtype=DT[dt], device="cuda")
    out = Out()
    dgate = out(5)
    dgate.fill_(7.0)
    pcr.residual_norm_backward(e, None, e, e, e, e, gate=gate, gate_kind="token", dgate=dgate)
    assert not bool(dgate.any())
    assert out.intact()
    misaligned = torch.zeros(6, device="cuda")[1:]
    with pytest.raises(pcr.LpcollError) as r:
        pcr.residual_norm_backward(e, None, e, e, e, e, gate=gate, gate_kind="token",
                                   dgate=misaligned)
    assert r.value.status == 2
