"""Seeded random configurations of the operators around the collectives against
their 64-bit forms (layers_ref.py, with the derived bounds), on the normal and
the bounds-checked build: types, gates, norms, ranks, capacities, dropped slots,
and sizes drawn over the logarithm of their range, odd ones among them.

LPCOLL_FUZZ_CONFIGS sets how many configurations run (default 900)."""
import os

import numpy as np
import pytest
import torch

import layers_ref as ref
import precision_collective_reduction_gb300 as pcr
from test_gpu_layers import DT, Out, dev, dev_i32, f64, lib, opt64, within  # noqa: F401

pytestmark = pytest.mark.gpu
OPS = ("route", "experts", "norm", "gradient")
MOST = 1 << 19  # elements of a matrix


def _log(g, lo, hi):
    return int(round(np.exp(g.uniform(np.log(lo), np.log(hi)))))


def _configs(count=int(os.environ.get("LPCOLL_FUZZ_CONFIGS", "900")), seed=4711):
    g = np.random.default_rng(seed)
    for i in range(count):
        c = dict(i=i, op=OPS[i % len(OPS)], dt=["f32", "bf16"][int(g.integers(2))])
        if c["op"] == "route":
            E = _log(g, 1, 1024)
            c.update(E=E, K=int(g.integers(1, min(E, 32) + 1)), T=_log(g, 1, 300),
                     renorm=bool(g.integers(2)))
        else:
            H = _log(g, 1, 16384)
            H = max(8, H // 64 * 64) if g.random() < 0.5 else H
            c.update(H=H, T=_log(g, 1, min(3000, max(1, MOST // H))))
        if c["op"] == "experts":
            c.update(K=int(g.integers(1, 9)), E=_log(g, 1, 300))
            c["T"] = max(1, min(c["T"], MOST // (c["H"] * c["K"]) + 1))
            c["capacity"] = int(g.choice([0, 0, 1, -(-c["T"] * c["K"] // c["E"])]))
            if c["capacity"] * c["E"] * c["H"] > 4 * MOST:
                c["capacity"] = 0
        if c["op"] in ("norm", "gradient"):
            c.update(kind=[None, "channel", "token", "full"][int(g.integers(4))],
                     post=bool(g.integers(4)), pre=bool(g.integers(4)),
                     ranks=int(g.choice([1, 1, 2, 5, 16])))
        yield c


def _route(c, g):
    T, E, K, dt = c["T"], c["E"], c["K"], c["dt"]
    z = g.normal(size=(T, E)) * 3
    z[g.random((T, E)) < 0.2] = -np.inf
    z[g.random((T, E)) < 0.1] = 1.25
    z = f64(dev(z, dt))
    out = Out()
    ids, w, dl = out(T, K, dtype=torch.int32), out(T, K), out(T, E, dtype=DT[dt])
    pcr.expert_route(dev(z, dt), ids, w, renormalize=c["renorm"])
    wi, ww, wb = ref.route(z, K, c["renorm"])
    assert np.array_equal(ids.cpu().numpy(), wi)
    within(w, (ww, wb), "weights")
    dw = g.normal(size=(T, K)).astype(np.float32)
    pcr.expert_route_backward(dev(z, dt), ids, w, dev(dw), dl, renormalize=c["renorm"])
    v, b = ref.route_backward(z, wi, ww, dw.astype(np.float64), c["renorm"])
    within(dl, (v, b + ref.HALF_ULP[dt] * np.abs(v) * (1 + 2 ** -8)), "dlogits")
    assert out.intact()


def _experts(c, g, oracle):
    T, K, E, H, dt, C = c["T"], c["K"], c["E"], c["H"], c["dt"], c["capacity"]
    ids = g.integers(-1, E, size=(T, K))
    out = Out()
    R = E * C or T * K
    i32 = torch.int32
    t = (out(T, K, dtype=i32), out(R, dtype=i32), out(E + 1, dtype=i32), out(E, dtype=i32))
    pcr.expert_sort(dev_i32(ids), E, *t, capacity=C)
    want = ref.sort(ids, E, C)
    for got, v in zip(t, want):
        assert np.array_equal(got.cpu().numpy(), v)
    slot_row, row_slot = want[:2]
    x = dev(g.normal(size=(T, H)), dt)
    rows = out(R, H, dtype=DT[dt])
    pcr.expert_dispatch(x, t[0], t[1], rows)
    used = torch.from_numpy(row_slot >= 0)
    sent = torch.zeros(R, H, dtype=DT[dt])
    sent[used] = x.cpu()[torch.from_numpy(row_slot // K)[used].long()]
    assert torch.equal(rows.cpu(), sent)
    codes, scales = out(R, H, dtype=torch.uint8), out(R, pcr.nblocks(H))
    pcr.expert_dispatch(x, t[0], t[1], block=128, codes=codes, scales=scales)
    host = sent.view(torch.int16).numpy().view(np.uint16) if dt == "bf16" else sent.numpy()
    pay = [oracle.quantize(host[r]) for r in range(R)]
    assert np.array_equal(codes.cpu().numpy(), np.stack([p[0] for p in pay]))
    assert np.array_equal(scales.cpu().numpy().view(np.uint32),
                          np.stack([p[1] for p in pay]).view(np.uint32))
    w = g.random((T, K)).astype(np.float32)
    y, z = out(T, H, dtype=DT[dt]), out(T, H, dtype=DT[dt])
    pcr.expert_combine(t[0], y, rows, weights=dev(w))
    within(y, ref.combine(f64(rows), slot_row, w, dt), "combined")
    pcr.expert_combine(t[0], z, weights=dev(w), block=128, codes=codes, scales=scales)
    vals = np.stack([oracle.dequantize(p[0], p[1]) for p in pay])
    within(z, ref.combine(vals, slot_row, w, dt), "combined from payloads")
    dy, drows, dw = dev(g.normal(size=(T, H)), dt), out(R, H, dtype=DT[dt]), out(T, K)
    pcr.expert_combine_backward(dy, t[0], t[1], drows, rows=rows, weights=dev(w), dweights=dw)
    wr, ww = ref.combine_backward(f64(dy), f64(rows), slot_row, w, R, dt)
    within(drows, wr, "drows")
    within(dw, ww, "dweights")
    assert out.intact()


def _norm_inputs(c, g, ranks):
    T, H, dt, kind = c["T"], c["H"], c["dt"], c["kind"]
    hs = [dev(g.normal(size=(T, H)) * 2, dt) for _ in range(ranks)]
    gate = None if kind is None else dev(
        g.normal(size={"channel": (H,), "token": (T,), "full": (T, H)}[kind]), dt)
    wq = dev(1 + 0.3 * g.normal(size=H), dt) if c["post"] else None
    wp = dev(1 + 0.3 * g.normal(size=H), dt) if c["pre"] else None
    a, b, eps = (float(np.float32(v)) for v in (0.9, -0.7, 1e-4))
    kw = dict(gate=gate, gate_kind=kind, w_post=wq, w_pre=wp, res_scale=a, branch_scale=b, eps=eps)
    return hs, dev(g.normal(size=(T, H)) * 3, dt), kw, (opt64(gate), kind, opt64(wq), opt64(wp), a,
                                                       b, eps, dt)


def _norm(c, g):
    T, H, dt = c["T"], c["H"], c["dt"]
    hs, x, kw, plain = _norm_inputs(c, g, c["ranks"])
    out = Out()
    xo, n, hsum = (out(T, H, dtype=DT[dt]) for _ in range(3))
    want_sum = hsum if g.random() < 0.5 else None
    pcr.residual_norm(hs, x, xo, n if c["pre"] else None, h_sum=want_sum, **kw)
    want = ref.residual_norm([f64(t) for t in hs], f64(x), *plain)
    within(xo, want[0], "x_out")
    if c["pre"]:
        within(n, want[1], "n_out")
    if want_sum is not None:
        within(hsum, want[2], "h_sum")
    assert out.intact()


def _gradient(c, g):
    T, H, dt, kind = c["T"], c["H"], c["dt"], c["kind"]
    (h,), xo, kw, plain = _norm_inputs(c, g, 1)
    dn = dev(g.normal(size=(T, H)), dt) if c["pre"] else None
    dxo = dev(g.normal(size=(T, H)), dt) if not c["pre"] or g.random() < 0.8 else None
    out = Out()
    got = dict(dx=out(T, H, dtype=DT[dt]), dh=out(T, H, dtype=DT[dt]))
    if kind:
        got["dgate"] = (out(T, H, dtype=DT[dt]) if kind == "full"
                        else out(H if kind == "channel" else T))
    if c["post"]:
        got["dw_post"] = out(H)
    if c["pre"]:
        got["dw_pre"] = out(H)
    pcr.residual_norm_backward(dxo, dn, h, xo, got["dx"], got["dh"], **kw, **{
        k: v for k, v in got.items() if k not in ("dx", "dh")})
    want = ref.residual_norm_backward(opt64(dxo), opt64(dn), f64(h), f64(xo), *plain)
    assert set(want) == set(got)
    for name in got:
        within(got[name], want[name], name)
    assert out.intact()


@pytest.mark.parametrize("c", list(_configs()), ids=lambda c: "%d-%s" % (c["i"], c["op"]))
def test_random_config(lib, oracle, c):  # noqa: F811
    g = np.random.default_rng([9, c["i"]])
    if c["op"] == "route":
        _route(c, g)
    elif c["op"] == "experts":
        _experts(c, g, oracle)
    elif c["op"] == "norm":
        _norm(c, g)
    else:
        _gradient(c, g)
