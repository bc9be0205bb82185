"""The operators around the collectives on the GPU against plain 64-bit forms
(layers_ref.py, with the derived bounds), at the sizes and inputs where they
can go wrong: one token, odd rows, slots and rows without a counterpart,
masked and empty rows, NaN and infinity in places that must not be read. Every
case runs on the bounds-checked build too."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import precision_collective_reduction_gb300 as pcr
from precision_collective_reduction_gb300 import _binding as B
from precision_collective_reduction_gb300 import build as lib_build
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(params=["normal", "checked"])
def lib(request):
    """Both builds of the library; the checked one must record nothing."""
    if request.param == "normal":
        lib_build.build()
        yield
        return
    with B.using_library(lib_build.build(debug_bounds=True)):
        B.debug_bounds_errors()
        yield
        st, bad = B.debug_bounds_errors()
        assert st == 0, "access outside the call's buffers (status %d, first 0x%x)" % (st, bad)


class Out:
    """Guarded result tensors: canaries behind each, which intact() checks."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=torch.float32):
        g = Guarded(int(np.prod(shape)), dtype)
        self.all.append(g)
        return g.t.view(*shape)

    def intact(self):
        return all(g.intact() for g in self.all)


def dev(a, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DT[dt]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, what):
    value, bound = want
    got = f64(got)
    assert got.shape == value.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(value)), what
    off = np.abs(got - value)
    bad = ~(off <= bound) & ~np.isnan(value)
    assert not bad.any(), "%s: %d of %d values outside, worst %g times the bound" % (
        what, bad.sum(), bad.size, np.nanmax(off / bound))


def rng(*key):
    return np.random.default_rng([7, *key])


# -- router -------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 64, 8), (5, 8, 8), (33, 60, 6), (40, 65, 4),
                                   (17, 128, 1), (20, 200, 10), (9, 384, 32), (6, 1000, 8),
                                   (3, 1024, 32)])
def test_route(lib, dt, renorm, T, E, K):
    g = rng(T, E, K, renorm)
    z = g.normal(size=(T, E)) * 2
    z[g.random((T, E)) < 0.15] = -np.inf       # experts switched off
    z[g.random((T, E)) < 0.1] = 0.5            # ties
    z[g.random((T, E)) < 0.05] = -0.0
    z[g.random((T, E)) < 0.05] = 0.0
    if T > 4:
        z[1] = -np.inf                         # none left
        z[2, 1:] = -np.inf                     # fewer than K left
        z[3] = 1.0                             # all the same
        z[4, : E // 2] = -3.0e38               # the types' lowest values
        z[4, 0] = torch.finfo(DT[dt]).min
    z = f64(dev(z, dt))
    out = Out()
    logits, ids, w = dev(z, dt), out(T, K, dtype=torch.int32), out(T, K)
    pcr.expert_route(logits, ids, w, renormalize=renorm)
    wi, ww, wb = ref.route(z, K, renorm)
    assert np.array_equal(ids.cpu().numpy(), wi)
    within(w, (ww, wb), "weights")
    dw = g.normal(size=(T, K)).astype(np.float32)
    dl = out(T, E, dtype=DT[dt])
    pcr.expert_route_backward(logits, ids, w, dev(dw), dl, renormalize=renorm)
    v, b = ref.route_backward(z, wi, ww, dw.astype(np.float64), renorm)
    within(dl, (v, b + ref.HALF_ULP[dt] * np.abs(v) * (1 + 2 ** -8)), "dlogits")
    torch.cuda.synchronize()
    assert out.intact()
    again = logits.clone()                     # in place
    pcr.expert_route_backward(again, ids, w, dev(dw), again, renormalize=renorm)
    assert torch.equal(again.view(torch.uint8), dl.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_nan_and_infinity(lib, dt, renorm):
    z = rng(1).normal(size=(4, 70))
    z[0, 40] = np.nan
    z[1, [3, 66]] = np.nan
    z[2, 12] = np.inf
    z[3, 5] = -np.inf
    z = f64(dev(z, dt))
    ids = torch.empty(4, 3, dtype=torch.int32, device="cuda")
    w = torch.empty(4, 3, device="cuda")
    pcr.expert_route(dev(z, dt), ids, w, renormalize=renorm)
    wi, ww, wb = ref.route(z, 3, renorm)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert wi[0, 0] == 40 and list(wi[1, :2]) == [3, 66] and wi[2, 0] == 12
    assert np.isnan(f64(w)[:3]).all() and np.isfinite(f64(w)[3]).all()
    within(w[3:], (ww[3:], wb[3:]), "weights beside")


@pytest.mark.parametrize("E", [8, 100, 256, 300, 1024])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_of_logits_that_agree_in_their_first_bits(lib, E, renorm):
    # FP32 logits one ulp apart, equal ones among them, in any order
    g = rng(E, 17)
    z = (1.0 + g.integers(0, 24, size=(60, E)) * 2.0 ** -23).astype(np.float32)
    z[20:40] *= -1
    z[40:] = np.where(g.random((20, E)) < 0.5, z[40:], g.normal(size=(20, E)))
    K = min(E, 9)
    ids = torch.empty(60, K, dtype=torch.int32, device="cuda")
    w = torch.empty(60, K, device="cuda")
    pcr.expert_route(dev(z), ids, w, renormalize=renorm)
    wi, ww, wb = ref.route(z, K, renorm)
    assert np.array_equal(ids.cpu().numpy(), wi)
    within(w, (ww, wb), "weights")


# -- sort ---------------------------------------------------------------------

def maps(T, K, E, capacity):
    out = Out()
    i32 = torch.int32
    t = (out(T, K, dtype=i32), out(E * capacity or T * K, dtype=i32), out(E + 1, dtype=i32),
         out(E, dtype=i32))
    return out, t


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 64), (7, 3, 5), (256, 8, 64), (257, 8, 1024),
                                   (683, 3, 7), (5000, 4, 128), (33000, 8, 200)])
@pytest.mark.parametrize("capacity", [0, 1, "even"])
@pytest.mark.parametrize("kind", ["some dropped", "one expert", "none"])
def test_sort(lib, T, K, E, capacity, kind):
    g = rng(T, K, E)
    capacity = -(-T * K // E) if capacity == "even" else capacity
    ids = g.integers(0, E, size=(T, K)) if kind != "one expert" else np.full((T, K), E - 1)
    if kind == "some dropped":
        ids[g.random((T, K)) < 0.2] = -1
        ids[g.random((T, K)) < 0.05] = E
        ids[g.random((T, K)) < 0.02] = 2 ** 31 - 1
    if kind == "none":
        ids[:] = -1
    out, t = maps(T, K, E, capacity)
    pcr.expert_sort(dev_i32(ids), E, *t, capacity=capacity)
    for got, want, what in zip(t, ref.sort(ids, E, capacity),
                               ("slot_row", "row_slot", "offsets", "counts")):
        assert np.array_equal(got.cpu().numpy(), want), what
    assert out.intact()


def dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def test_sort_of_nothing(lib):
    out, t = maps(0, 4, 6, 0)
    pcr.expert_sort(dev_i32(np.zeros((0, 4))), 6, *t)
    assert t[2].tolist() == [0] * 7 and t[3].tolist() == [0] * 6
    out, t = maps(0, 4, 6, 5)
    pcr.expert_sort(dev_i32(np.zeros((0, 4))), 6, *t, capacity=5)
    assert t[1].tolist() == [-1] * 30 and t[2].tolist() == list(range(0, 31, 5))
    assert t[3].tolist() == [0] * 6


# -- dispatch and combine -----------------------------------------------------

SIZES = [(1, 1, 1, 1), (1500, 2, 5, 512), (1300, 1, 3, 1024), (1, 8, 16, 8192), (3, 2, 4, 7), (5, 4, 6, 130), (9, 3, 8, 96),
         (20, 8, 32, 257), (33, 5, 7, 1000), (64, 32, 64, 128), (130, 2, 3, 2050), (11, 6, 8, 4100)]


def case(T, K, E, H, dt, capacity=0, dropped=0.15):
    g = rng(T, K, E, H)
    ids = g.integers(0, E, size=(T, K))
    ids[g.random((T, K)) < dropped] = -1
    slot_row, row_slot = ref.sort(ids, E, capacity)[:2]
    return g, slot_row, row_slot


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,E,H", SIZES)
@pytest.mark.parametrize("capacity", [0, 3])
def test_dispatch(lib, oracle, dt, T, K, E, H, capacity):
    g, slot_row, row_slot = case(T, K, E, H, dt, capacity)
    R = row_slot.size
    x = dev(g.normal(size=(T, H)) * np.exp(g.normal(size=(T, 1)) * 3), dt)
    x[0, 0] = 0.0
    out = Out()
    rows = out(R, H, dtype=DT[dt])
    pcr.expert_dispatch(x, dev_i32(slot_row), dev_i32(row_slot), rows)
    used = torch.from_numpy(row_slot >= 0)
    want = torch.zeros(R, H, dtype=DT[dt])
    want[used] = x.cpu()[torch.from_numpy(row_slot // K)[used].long()]
    assert torch.equal(rows.cpu(), want)
    codes, scales = out(R, H, dtype=torch.uint8), out(R, pcr.nblocks(H))
    pcr.expert_dispatch(x, dev_i32(slot_row), dev_i32(row_slot), block=128, codes=codes,
                        scales=scales)
    host = want.view(torch.int16).numpy().view(np.uint16) if dt == "bf16" else want.numpy()
    for r in range(R):
        c, s = oracle.quantize(host[r])
        assert np.array_equal(codes[r].cpu().numpy(), c), r
        assert np.array_equal(scales[r].cpu().numpy().view(np.uint32), s.view(np.uint32)), r
    assert out.intact()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,K,E,H", SIZES)
def test_combine(lib, oracle, dt, weighted, T, K, E, H):
    g, slot_row, row_slot = case(T, K, E, H, dt)
    slot_row[T // 2] = -1                       # a token without any row
    slot_row[0, 0] = row_slot.size              # an entry out of range counts as none
    R = row_slot.size
    rows = dev(g.normal(size=(R, H)), dt)
    w = g.random((T, K)).astype(np.float32) if weighted else None
    left = np.setdiff1d(np.arange(R), slot_row)  # rows that nobody asks for
    rows[torch.from_numpy(left).cuda()] = float("nan")
    out = Out()
    y = out(T, H, dtype=DT[dt])
    wt = None if w is None else dev(w)
    if w is not None:
        wt[torch.from_numpy((slot_row < 0) | (slot_row >= R)).cuda()] = float("nan")
    pcr.expert_combine(dev_i32(slot_row), y, rows, weights=wt)
    within(y, ref.combine(f64(rows), slot_row, w, dt), "combined")
    assert not f64(y)[T // 2].any()
    # from FP8 payloads, whose values the oracle gives
    host = torch.nan_to_num(rows.float().cpu()).numpy()
    pay = [oracle.quantize(host[r]) for r in range(R)]
    vals = np.stack([oracle.dequantize(c, s) for c, s in pay])
    z = out(T, H, dtype=DT[dt])
    pcr.expert_combine(dev_i32(slot_row), z, weights=wt, block=128,
                       codes=torch.from_numpy(np.stack([c for c, _ in pay])).cuda(),
                       scales=torch.from_numpy(np.stack([s for _, s in pay])).cuda())
    within(z, ref.combine(vals, slot_row, w, dt), "combined from payloads")
    assert out.intact()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,K,E,H", SIZES)
@pytest.mark.parametrize("capacity", [0, 3])
def test_combine_backward(lib, dt, weighted, T, K, E, H, capacity):
    g, slot_row, row_slot = case(T, K, E, H, dt, capacity)
    R = row_slot.size
    rows, dy = dev(g.normal(size=(R, H)), dt), dev(g.normal(size=(T, H)), dt)
    rows[torch.from_numpy(row_slot < 0).cuda()] = float("inf")
    w = g.random((T, K)).astype(np.float32) if weighted else None
    wt = None if w is None else dev(w)
    out = Out()
    drows, dw = out(R, H, dtype=DT[dt]), out(T, K)
    pcr.expert_combine_backward(dy, dev_i32(slot_row), dev_i32(row_slot), drows, rows=rows,
                                weights=wt, dweights=dw)
    wr, ww = ref.combine_backward(f64(dy), f64(rows), slot_row, w, R, dt)
    within(drows, wr, "drows")
    within(dw, ww, "dweights")
    assert not f64(drows)[row_slot < 0].any() and not f64(dw)[slot_row < 0].any()
    alone = out(R, H, dtype=DT[dt])            # without the weights' gradient
    pcr.expert_combine_backward(dy, dev_i32(slot_row), dev_i32(row_slot), alone, weights=wt)
    assert torch.equal(alone, drows)
    pcr.expert_combine_backward(dy, dev_i32(slot_row), dev_i32(row_slot), rows, rows=rows,
                                weights=wt, dweights=dw)  # in place
    assert torch.equal(rows, drows)
    within(dw, ww, "dweights of the call in place")
    assert out.intact()


def test_dispatch_and_its_gradient_are_adjoint(lib):
    # <dispatch(x), d> == <x, dispatch_backward(d)>, sums in 64 bits: FP32
    # products of one weight 1 are exact, the gradient's sums K - 1 roundings
    T, K, E, H = 50, 4, 9, 260
    g, slot_row, row_slot = case(T, K, E, H, "f32")
    x, d = dev(g.normal(size=(T, H))), dev(g.normal(size=(T * K, H)))
    rows, dx = torch.empty(T * K, H, device="cuda"), torch.empty(T, H, device="cuda")
    s, r = dev_i32(slot_row), dev_i32(row_slot)
    pcr.expert_dispatch(x, s, r, rows)
    pcr.expert_dispatch_backward(d, s, dx)
    lhs, rhs = (rows.double() * d.double()).sum(), (x.double() * dx.double()).sum()
    mag = (rows.double() * d.double()).abs().sum()
    assert abs(float(lhs - rhs)) <= K * ref.U * float(mag)


def test_empty_calls(lib):
    z = torch.empty(0, 16, device="cuda")
    i = dev_i32(np.zeros((0, 2)))
    rows = torch.full((3, 16), 5.0, device="cuda")
    pcr.expert_dispatch(z, i, dev_i32([-1, -1, -1]), rows)       # no tokens: only clears
    assert not rows.any()
    pcr.expert_combine(i, z, rows)
    y = torch.full((2, 16), 5.0, device="cuda")                  # no rows: zeros
    pcr.expert_combine(dev_i32([[-1, 0], [3, -1]]), y, torch.empty(0, 16, device="cuda"))
    assert not y.any()
    dw = torch.full((2, 2), 5.0, device="cuda")
    pcr.expert_combine_backward(y, dev_i32([[-1, -1], [-1, -1]]), dev_i32([]),
                                torch.empty(0, 16, device="cuda"), rows=torch.empty(
                                    0, 16, device="cuda"), dweights=dw)
    assert not dw.any()


# -- residual norm ------------------------------------------------------------

NORM_SIZES = [(1, 1), (1, 8192), (3, 7), (5, 96), (2, 130), (17, 257), (9, 1000), (400, 64),
              (2, 4100), (3, 5000), (2, 8191), (2, 16383), (2, 16384)]


def norm_case(T, H, dt, kind, post, pre, ranks=1):
    g = rng(T, H, ranks, post, pre)
    hs = [dev(g.normal(size=(T, H)) * 2, dt) for _ in range(ranks)]
    x = dev(g.normal(size=(T, H)) * np.exp(g.normal(size=H)), dt)
    gate = None
    if kind:
        gate = dev(g.normal(size={"channel": (H,), "token": (T,), "full": (T, H)}[kind]), dt)
    wq = dev(1 + 0.3 * g.normal(size=H), dt) if post else None
    wp = dev(1 + 0.3 * g.normal(size=H), dt) if pre else None
    return g, hs, x, gate, wq, wp


def opt64(t):
    return None if t is None else f64(t)


PARTS = [(None, True, True), ("channel", True, True), ("token", True, True), ("full", True, True),
         ("channel", False, True), ("token", False, False), (None, True, False), ("full", False, True)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("kind,post,pre", PARTS)
def test_residual_norm(lib, dt, T, H, kind, post, pre):
    a, b, eps = 0.9, 0.7, 1e-5
    for ranks in (1, 3):
        g, hs, x, gate, wq, wp = norm_case(T, H, dt, kind, post, pre, ranks)
        if T > 4:
            hs[0][1] = 0.0                     # a row of zeros
            for t in hs[1:]:
                t[1] = 0.0
            x[1] = 0.0
        out = Out()
        xo, n, hsum = (out(T, H, dtype=DT[dt]) for _ in range(3))
        kw = dict(gate=gate, w_post=wq, w_pre=wp, res_scale=a, branch_scale=b, eps=eps,
                  gate_kind=kind)
        pcr.residual_norm(hs, x, xo, n if pre else None, h_sum=hsum, **kw)
        a32, b32, e32 = np.float32(a), np.float32(b), np.float32(eps)
        want = ref.residual_norm([f64(t) for t in hs], f64(x), opt64(gate), kind, opt64(wq),
                                 opt64(wp), float(a32), float(b32), float(e32), dt)
        within(xo, want[0], "x_out")
        if pre:
            within(n, want[1], "n_out")
        within(hsum, want[2], "h_sum")
        assert out.intact()
        in_place = x.clone()
        pcr.residual_norm(hs, in_place, in_place, hs[0] if pre else None, **kw)
        assert torch.equal(in_place, xo) and (not pre or torch.equal(hs[0], n))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("kind,post,pre", PARTS)
def test_residual_norm_backward(lib, dt, T, H, kind, post, pre):
    a, b, eps = (float(np.float32(v)) for v in (0.9, 0.7, 1e-5))
    g, (h,), xo, gate, wq, wp = norm_case(T, H, dt, kind, post, pre)
    dxo = dev(g.normal(size=(T, H)), dt)
    dn = dev(g.normal(size=(T, H)), dt) if pre else None
    if T > 4:
        h[1] = 0.0
        xo[2] = 0.0
    for given in (dxo, None) if pre else (dxo,):
        out = Out()
        dx, dh = out(T, H, dtype=DT[dt]), out(T, H, dtype=DT[dt])
        got = dict(dx=dx, dh=dh)
        if kind:
            got["dgate"] = {"channel": lambda: out(H), "token": lambda: out(T),
                            "full": lambda: out(T, H, dtype=DT[dt])}[kind]()
        if post:
            got["dw_post"] = out(H)
        if pre:
            got["dw_pre"] = out(H)
        kw = dict(gate=gate, w_post=wq, w_pre=wp, res_scale=a, branch_scale=b, eps=eps,
                  gate_kind=kind)
        grads = {k: v for k, v in got.items() if k.startswith("d") and k not in ("dx", "dh")}
        pcr.residual_norm_backward(given, dn, h, xo, dx, dh, **kw, **grads)
        want = ref.residual_norm_backward(opt64(given), opt64(dn), f64(h), f64(xo), opt64(gate),
                                          kind, opt64(wq), opt64(wp), a, b, eps, dt)
        assert set(want) == set(got)
        for name in got:
            within(got[name], want[name], name)
        assert out.intact()
        alone = [torch.empty_like(dx), torch.empty_like(dh)]   # no sums over tokens wanted
        pcr.residual_norm_backward(given, dn, h, xo, *alone, **kw)
        assert torch.equal(alone[0], dx) and torch.equal(alone[1], dh)
    both = [dxo.clone(), None if dn is None else dn.clone()]
    hh = h.clone()
    pcr.residual_norm_backward(dxo, dn, h, xo, dx, dh, **kw)
    pcr.residual_norm_backward(both[0], both[1], hh, xo, both[0], hh, **kw)  # in place
    assert torch.equal(both[0], dx) and torch.equal(hh, dh)


def test_gate_of_one_dimension_where_both_fit():
    # as many tokens as channels: per channel, unless the kind says otherwise
    x = torch.ones(4, 4, device="cuda")
    gate = torch.arange(4.0, device="cuda")
    out = torch.empty_like(x)
    pcr.residual_norm(x, torch.zeros_like(x), out, gate=gate)
    assert torch.equal(out, gate.expand(4, 4))
    pcr.residual_norm(x, torch.zeros_like(x), out, gate=gate, gate_kind="token")
    assert torch.equal(out, gate[:, None].expand(4, 4))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(700, 1025), (1300, 130), (400, 1024), (310, 8704), (160, 16384),
                                 (5000, 64), (311, 2051), (160, 12288), (100, 6000),
                                 (100, 6100)])
@pytest.mark.parametrize("kind,post,pre", [("channel", True, True), ("token", False, True),
                                           ("full", True, True)])
def test_norms_of_many_tokens(lib, dt, T, H, kind, post, pre):
    # several rows per team, in a part of a CTA, a CTA and a cluster
    test_residual_norm(lib, dt, T, H, kind, post, pre)
    test_residual_norm_backward(lib, dt, T, H, kind, post, pre)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(3, 8192), (200, 4096), (40, 777), (2, 16384), (170, 768),
                                 (40, 768), (9, 1)])
@pytest.mark.parametrize("kind", [None, "full"])
def test_residual_norm_of_16_ranks(lib, dt, T, H, kind):
    a, b, eps = (float(np.float32(v)) for v in (0.9, 0.7, 1e-5))
    g, hs, x, gate, wq, wp = norm_case(T, H, dt, kind, True, True, 16)
    out = Out()
    xo, n, hsum = (out(T, H, dtype=DT[dt]) for _ in range(3))
    kw = dict(gate=gate, w_post=wq, w_pre=wp, res_scale=a, branch_scale=b, eps=eps, gate_kind=kind)
    pcr.residual_norm(hs, x, xo, n, h_sum=hsum, **kw)
    want = ref.residual_norm([f64(t) for t in hs], f64(x), opt64(gate), kind, opt64(wq), opt64(wp),
                             a, b, eps, dt)
    for got, w, what in zip((xo, n, hsum), want, ("x_out", "n_out", "h_sum")):
        within(got, w, what)
    assert out.intact()
    # h_sum is what the allreduce of the partial products gives, before rounding
    # to BF16 equal in FP32: the same sum in the same order
    total = torch.empty_like(x)
    pcr.dda_flat_sim([t.view(-1) for t in hs], [torch.empty_like(t).view(-1) for t in hs[1:]]
                     + [total.view(-1)], block=0)
    assert torch.equal(total, hsum)


def test_norm_gradient_of_no_tokens(lib):
    H = 40
    z = torch.empty(0, H, device="cuda")
    w = torch.ones(H, device="cuda")
    sums = [torch.full((H,), 7.0, device="cuda") for _ in range(3)]
    pcr.residual_norm(z, z, z, z, w_post=w, w_pre=w)
    pcr.residual_norm_backward(z, z, z, z, z, z, gate=w, gate_kind="channel", w_post=w, w_pre=w,
                               dgate=sums[0], dw_post=sums[1], dw_pre=sums[2])
    assert not any(bool(s.any()) for s in sums)


@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_norm_gradient_against_differences(kind):
    # the kernel's gradients along a random direction against central
    # differences of the 64-bit forward. Truncation is about step^2 = 1e-8 of
    # the loss' third derivative, the FP32 gradients a few 1e-7 of their
    # magnitudes: 1e-5 of the sum of magnitudes covers both.
    T, H = 6, 200
    a, b, eps = (float(np.float32(v)) for v in (0.9, 0.7, 1e-5))
    g, (h,), x, gate, wq, wp = norm_case(T, H, "f32", kind, True, True)
    th = dict(h=f64(h), x=f64(x), gate=f64(gate), w_post=f64(wq), w_pre=f64(wp))
    dxo, dn = dev(g.normal(size=(T, H))), dev(g.normal(size=(T, H)))

    def loss(v):
        xo, n = ref.forward(v["h"], v["x"], v["gate"], kind, v["w_post"], v["w_pre"], a, b, eps)
        return (xo * f64(dxo)).sum() + (n * f64(dn)).sum()
    xo, n = torch.empty_like(x), torch.empty_like(x)
    kw = dict(gate=gate, gate_kind=kind, w_post=wq, w_pre=wp, res_scale=a, branch_scale=b, eps=eps)
    pcr.residual_norm(h, x, xo, n, **kw)
    got = dict(x=torch.empty_like(x), h=torch.empty_like(x), gate=torch.empty_like(gate),
               w_post=torch.empty_like(wq), w_pre=torch.empty_like(wp))
    pcr.residual_norm_backward(dxo, dn, h, xo, got["x"], got["h"], dgate=got["gate"],
                               dw_post=got["w_post"], dw_pre=got["w_pre"], **kw)
    for name, v in th.items():
        d = g.normal(size=v.shape)
        step = 1e-4
        want = (loss({**th, name: v + step * d}) - loss({**th, name: v - step * d})) / (2 * step)
        terms = f64(got[name]) * d
        assert abs(terms.sum() - want) <= 1e-5 * np.abs(terms).sum() + 1e-7, name


# -- all of them --------------------------------------------------------------

def test_same_bits_again_and_on_another_stream():
    T, K, E, H = 700, 4, 24, 1032
    g = rng(9)
    logits, x = dev(g.normal(size=(T, E)), "bf16"), dev(g.normal(size=(T, H)), "bf16")
    w = dev(1 + 0.1 * g.normal(size=H), "bf16")

    def layer(stream=None):
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        ids, wt = e(T, K, dtype=torch.int32), e(T, K, dtype=torch.float32)
        m = (e(T, K, dtype=torch.int32), e(T * K, dtype=torch.int32), e(E + 1, dtype=torch.int32),
             e(E, dtype=torch.int32))
        rows, y, xo, n, drows, dwt = e(T * K, H), e(T, H), e(T, H), e(T, H), e(T * K, H), e(
            T, K, dtype=torch.float32)
        dx, dh, dp, dq = e(T, H), e(T, H), e(H, dtype=torch.float32), e(H, dtype=torch.float32)
        dl = e(T, E)
        torch.cuda.synchronize()
        pcr.expert_route(logits, ids, wt, stream=stream)
        pcr.expert_sort(ids, E, *m, stream=stream)
        pcr.expert_dispatch(x, m[0], m[1], rows, stream=stream)
        pcr.expert_combine(m[0], y, rows, weights=wt, stream=stream)
        pcr.residual_norm(y, x, xo, n, w_post=w, w_pre=w, stream=stream)
        pcr.residual_norm_backward(x, n, y, xo, dx, dh, w_post=w, w_pre=w, dw_post=dp, dw_pre=dq,
                                   stream=stream)
        pcr.expert_combine_backward(dh, m[0], m[1], drows, rows=rows, weights=wt, dweights=dwt,
                                    stream=stream)
        pcr.expert_route_backward(logits, ids, wt, dwt, dl, stream=stream)
        torch.cuda.synchronize()
        return [ids, wt, *m, rows, y, xo, n, dx, dh, dp, dq, drows, dwt, dl]
    first = layer()
    side = torch.cuda.Stream()
    for other in (layer(), layer(side), layer(side.cuda_stream)):
        for p, q in zip(first, other):
            assert torch.equal(p, q)
    with torch.cuda.stream(side):
        for p, q in zip(first, layer()):
            assert torch.equal(p, q)


def test_graph_capture():
    T, K, E, H = 32, 8, 64, 512
    g = rng(10)
    logits, x = dev(g.normal(size=(T, E)), "bf16"), dev(g.normal(size=(T, H)), "bf16")
    e = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    ids, wt = e(T, K, dtype=torch.int32), e(T, K, dtype=torch.float32)
    m = (e(T, K, dtype=torch.int32), e(T * K, dtype=torch.int32), e(E + 1, dtype=torch.int32),
         e(E, dtype=torch.int32))
    rows, y, xo, n, dx, dh = e(T * K, H), e(T, H), e(T, H), e(T, H), e(T, H), e(T, H)
    w, dw = torch.ones(H, dtype=torch.bfloat16, device="cuda"), e(H, dtype=torch.float32)

    def step():
        pcr.expert_route(logits, ids, wt, renormalize=True)
        pcr.expert_sort(ids, E, *m)
        pcr.expert_dispatch(x, m[0], m[1], rows)
        pcr.expert_combine(m[0], y, rows, weights=wt)
        pcr.residual_norm([y] * 9, x, xo, n, w_post=w, w_pre=w)
        pcr.residual_norm_backward(x, n, y, xo, dx, dh, w_post=w, w_pre=w, dw_post=dw)
    step()
    torch.cuda.synchronize()
    made = (ids, wt, *m, rows, y, xo, n, dx, dh, dw)
    want = [t.clone() for t in made]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in made:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, v in zip(made, want):
        assert torch.equal(t, v)


def test_scratch_memory_of_threads_and_streams():
    # gradients of different sizes from several threads, on the default stream
    # and on others, with and without a workspace: the same bits as alone
    import threading
    sizes = [(700, 1024), (40, 512), (1500, 264), (9, 4096)]
    cases, want = [], []
    for T, H in sizes:
        g = rng(T, H, 77)
        t = [dev(g.normal(size=(T, H)), "bf16") for _ in range(4)]
        w = dev(1 + 0.1 * g.normal(size=H), "bf16")
        cases.append((t, w))

    def run(i, stream=None, workspace=None):
        (d, n, h, x), w = cases[i]
        out = [torch.zeros_like(x), torch.zeros_like(x),
               *(torch.zeros(x.shape[1], device="cuda") for _ in range(2))]
        if stream is not None:
            torch.cuda.synchronize()
        pcr.residual_norm_backward(d, n, h, x, out[0], out[1], w_post=w, w_pre=w, dw_post=out[2],
                                   dw_pre=out[3], stream=stream, workspace=workspace)
        return out
    for i in range(len(sizes)):
        need = pcr.residual_norm_backward_workspace_bytes(*sizes[i], pcr.BF16)
        want.append(run(i, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            side = torch.cuda.Stream()
            for k in range(30):
                j = (i + k) % len(sizes)
                got = run(j, stream=side if k % 3 == 0 else None)
                torch.cuda.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[j])):
                    wrong.append((i, k))
        except Exception as e:  # reported by the main thread
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not wrong


def test_refusals():
    T, K, E, H = 4, 2, 3, 16
    f = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i = lambda *s: f(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError):
        pcr.expert_route(f(T, E, dtype=torch.float16), i(T, K), f(T, K))
    with pytest.raises(TypeError):
        pcr.expert_route(f(T, E), i(T, K).long(), f(T, K))
    with pytest.raises(ValueError):
        pcr.expert_route(f(T, E), i(T, K), f(T, K + 1))
    with pytest.raises(ValueError):
        pcr.expert_route(torch.zeros(T, E), i(T, K), f(T, K))            # host tensor
    with pytest.raises(ValueError):
        pcr.expert_route(f(E, T).t(), i(T, K), f(T, K))                  # not contiguous
    with pytest.raises(pcr.LpcollError) as e:
        pcr.expert_route(f(T, E), i(T, E + 1), f(T, E + 1))
    assert e.value.status == 1
    with pytest.raises(pcr.LpcollError) as e:                            # misaligned
        pcr.expert_route(f(T * E + 1)[1:].view(T, E), i(T, K), f(T, K))
    assert e.value.status == 2
    with pytest.raises(ValueError):
        pcr.expert_sort(i(T, K), E, i(T, K), i(T * K), i(E), i(E))
    with pytest.raises(ValueError):
        pcr.expert_sort(i(T, K), E, i(T, K), i(T * K), i(E + 1), i(E), capacity=-1)
    with pytest.raises(ValueError):
        pcr.expert_sort(i(4000, K), E, i(4000, K), i(4000 * K), i(E + 1), i(E),
                        workspace=f(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        pcr.expert_dispatch(f(T, H), i(T, K), i(T * K), block=128, codes=f(T * K, H,
                                                                           dtype=torch.uint8))
    with pytest.raises(pcr.LpcollError) as e:
        pcr.expert_dispatch(f(T, H), i(T, K), i(T * K), block=64,
                            codes=f(T * K, H, dtype=torch.uint8), scales=f(T * K, 1))
    assert e.value.status == 3
    with pytest.raises(TypeError):
        pcr.expert_combine(i(T, K), f(T, H), f(T * K, H, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        pcr.expert_combine_backward(f(T, H), i(T, K), i(T * K), f(T * K, H), dweights=f(T, K))
    x = f(T, H)
    with pytest.raises(ValueError):
        pcr.residual_norm(x, x, x, w_pre=f(H))                           # n_out missing
    with pytest.raises(ValueError):
        pcr.residual_norm(x, x, x, gate=f(H + 1))
    with pytest.raises(ValueError, match="gate_kind"):
        pcr.residual_norm(x, x, x, gate=f(H), gate_kind="row")
    with pytest.raises(ValueError):
        pcr.residual_norm(x, x, x, gate=f(T), gate_kind="channel")
    with pytest.raises(pcr.LpcollError) as e:
        pcr.residual_norm(f(1, 16388), f(1, 16388), f(1, 16388))
    assert e.value.status == 3
    with pytest.raises(pcr.LpcollError) as e:
        pcr.residual_norm(x, x, x, eps=0.0)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        pcr.residual_norm([x] * 0, x, x)
    with pytest.raises(ValueError):
        pcr.residual_norm_backward(x, x, x, x, x, x)                     # dn_out without w_pre
    with pytest.raises(ValueError):
        pcr.residual_norm_backward(x, None, x, x, x, x, dw_post=f(H))


def test_rows_past_2_31_elements():
    # 300,000 rows of 8192: element offsets pass 2^31 on both sides
    free, _ = torch.cuda.mem_get_info()
    if free < 24 * (1 << 30):
        pytest.skip("needs about 20 GB of free device memory")
    T, K, H = 300000, 1, 8192
    x = torch.randn(T, H, dtype=torch.bfloat16, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(3))
    perm = torch.randperm(T, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    slot_row = perm.int().view(T, K)
    row_slot = torch.empty(T, dtype=torch.int32, device="cuda")
    row_slot[perm] = torch.arange(T, dtype=torch.int32, device="cuda")
    rows = torch.empty_like(x)
    pcr.expert_dispatch(x, slot_row, row_slot, rows)
    back = torch.empty_like(x)
    pcr.expert_combine(slot_row, back, rows)
    assert torch.equal(back, x)
    at = torch.tensor([0, 1, 262143, 262144, 262145, T - 1], device="cuda")
    assert torch.equal(rows[perm[at]], x[at])
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    pcr.residual_norm(x, x, back, rows, w_post=w, w_pre=w)
    few = [torch.empty(6, H, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pcr.residual_norm(x[at].contiguous(), x[at].contiguous(), few[0], few[1], w_post=w, w_pre=w)
    assert torch.equal(back[at], few[0]) and torch.equal(rows[at], few[1])
