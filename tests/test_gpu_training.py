"""The operators of a training step on the GPU against plain 64-bit forms
(training_ref.py, with the derived bounds), at the sizes and inputs where they can
go wrong: one token, odd rows, clusters and teams, rows of one value, means that
are large beside the spread, dropped infinities, padding, ids of other shards,
frequent tokens. Every case runs on the bounds-checked build too."""
import numpy as np
import pytest
import torch

import precision_collective_reduction_gb300 as pcr
import training_ref as ref
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
    return None if t is None else t.double().cpu().numpy()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def within(got, want, what):
    value, bound = want
    got = f64(got)
    assert got.shape == value.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(value)), what
    off = np.abs(got - value)
    bad = ~(off <= bound) & ~np.isnan(value)
    assert not bad.any(), "%s: %d of %d values outside, worst %g times the bound" % (
        what, bad.sum(), bad.size, np.nanmax(off / bound))


def gen(*key):
    return np.random.default_rng([11, *key])


def words(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


EPS = float(np.float32(1e-5))
SIZES = [(1, 1), (1, 8192), (3, 7), (5, 96), (2, 130), (17, 257), (9, 1000), (400, 64), (2, 4100),
         (3, 5000), (2, 8191), (200, 2051), (2, 16383), (2, 16384), (160, 4096), (155, 8200)]


def stream_like(g, T, H):
    """Rows of a residual stream: channels of different loudness and level, and rows
    that are zeros, one value, or far from 0."""
    x = (g.normal(size=(T, H)) + g.normal(size=H)) * np.exp(g.normal(size=H))
    if T > 2:
        x[1] = 0.0
        x[2] = 7.25
    if T > 4:
        x[3] += 300.0
        x[4, 0] = 1e4  # one loud channel
    return x


# -- layer norm ---------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("has_w,has_b", [(True, True), (False, False), (True, False),
                                         (False, True)])
def test_layer_norm(lib, dt, T, H, has_w, has_b):
    g = gen(T, H, has_w, has_b)
    x = dev(stream_like(g, T, H), dt)
    w = dev(1 + 0.3 * g.normal(size=H), dt) if has_w else None
    b = dev(g.normal(size=H), dt) if has_b else None
    out = Out()
    y = out(T, H, dtype=DT[dt])
    assert pcr.layer_norm(x, y, w=w, b=b, eps=EPS) is y
    within(y, ref.layer_norm(f64(x), f64(w), f64(b), EPS, dt), "out")
    dout, dx, dw, db = dev(g.normal(size=(T, H)), dt), out(T, H, dtype=DT[dt]), out(H), out(H)
    pcr.layer_norm_backward(dout, x, dx, w=w, eps=EPS, dw=dw, db=db)
    want = ref.layer_norm_backward(f64(dout), f64(x), f64(w), EPS, dt)
    within(dx, want["dx"], "dx")
    within(dw, want["dw"], "dw")
    within(db, want["db"], "db")
    # the parts alone, and in place
    only_dx, only_db = out(T, H, dtype=DT[dt]), out(H)
    pcr.layer_norm_backward(dout, x, only_dx, w=w, eps=EPS)
    pcr.layer_norm_backward(dout, x, None, w=w, eps=EPS, db=only_db)
    assert same(only_dx, dx) and same(only_db, db)
    assert out.intact()
    pcr.layer_norm_backward(dout, x, dout, w=w, eps=EPS, dw=dw)
    assert same(dout, dx)
    pcr.layer_norm(x, x, w=w, b=b, eps=EPS)
    assert same(x, y)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(700, 256), (307, 768), (1001, 512), (331, 8192), (40, 2048),
                                 (459, 1280), (310, 6144), (170, 12288), (153, 16384),
                                 (154, 9001), (320, 4100), (609, 300), (320, 4098), (175, 4099)])
def test_norms_of_many_rows(lib, dt, T, H):
    # every form of the kernels for more rows than SMs: several at a time and a last one
    # alone, teams that share a CTA, clusters, long rows, lanes without columns
    g = gen(T, H, 9)
    x, dn, dxo = (dev(stream_like(g, T, H), dt) for _ in range(3))
    w, b = dev(1 + 0.3 * g.normal(size=H), dt), dev(g.normal(size=H), dt)
    out = Out()
    y, dx, dh, xo, n = (out(T, H, dtype=DT[dt]) for _ in range(5))
    dw, db = out(H), out(H)
    pcr.layer_norm(x, y, w=w, b=b, eps=EPS)
    within(y, ref.layer_norm(f64(x), f64(w), f64(b), EPS, dt), "out")
    pcr.layer_norm_backward(dn, x, dx, w=w, eps=EPS, dw=dw, db=db)
    want = ref.layer_norm_backward(f64(dn), f64(x), f64(w), EPS, dt)
    for name, t in dict(dx=dx, dw=dw, db=db).items():
        within(t, want[name], name)
    p, rng = 0.3, words(T, H)
    keep = ref.kept(T, H, T, H, p)
    pcr.residual_dropout_backward(dxo, dn, x, dx, dh, rng, p, w=w, eps=EPS, dw=dw, db=db)
    want = ref.layer_norm_backward(f64(dn), f64(x), f64(w), EPS, dt, f64(dxo),
                                   keep / (1 - float(np.float32(p))))
    for name, t in dict(dx=dx, dh=dh, dw=dw, db=db).items():
        within(t, want[name], name)
    for ranks in (1, 2, 16) if H <= 2048 else (1, 9):
        hs = [dev(g.normal(size=(T, H)), dt) for _ in range(ranks)]
        for res in (x, None):
            pcr.residual_dropout(hs, res, xo, rng, p, n_out=n, w=w, b=b, eps=EPS)
            want = ref.residual_dropout([f64(t) for t in hs], f64(res), keep, p, f64(w), f64(b),
                                        EPS, dt, True)
            within(xo, want[0], "x_out")
            within(n, want[1], "n_out")
    torch.cuda.synchronize()
    assert out.intact()


def test_layer_norm_of_rows_far_from_zero(lib):
    # values 1000 and one ulp's multiples: the squares about 0 would leave nothing
    g = gen(3)
    x = dev(1000.0 + g.integers(-8, 9, size=(6, 512)) * 2.0 ** -14)
    y = torch.empty_like(x)
    pcr.layer_norm(x, y, eps=1e-12)
    within(y, ref.layer_norm(f64(x), None, None, float(np.float32(1e-12)), "f32"), "out")
    # spread about the right variance: of +-8 steps, uniform, some 4.9 steps
    assert 0.9 < float(y.std()) < 1.1


def test_norm_rows_with_nan_and_infinity(lib):
    g = gen(4)
    x = dev(g.normal(size=(8, 300)))
    want = ref.layer_norm(f64(x), None, None, EPS, "f32")
    clean = [0, 1, 3, 4, 6, 7]
    x[2, 17] = float("nan")
    x[5, 299] = float("inf")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    pcr.layer_norm(x, y, eps=EPS)
    pcr.layer_norm_backward(torch.ones_like(x), x, dx, eps=EPS)
    within(y[clean], (want[0][clean], want[1][clean]), "rows beside")
    assert torch.isfinite(dx[clean]).all()
    for bad in (2, 5):
        assert torch.isnan(y[bad]).all() and torch.isnan(dx[bad]).all()


def test_layer_norm_without_tokens_or_columns(lib):
    dw, db = torch.full((32,), 5.0, device="cuda"), torch.full((32,), 5.0, device="cuda")
    z = torch.empty(0, 32, device="cuda")
    pcr.layer_norm(z, z)
    pcr.layer_norm_backward(z, z, z, dw=dw, db=db)
    assert not dw.any() and not db.any()
    z = torch.empty(4, 0, device="cuda")
    pcr.layer_norm(z, z)
    pcr.layer_norm_backward(z, z, z, dw=torch.empty(0, device="cuda"))


# -- residual_dropout ---------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("ranks,has_x,norm,p", [(1, True, True, 0.1), (3, True, True, 0.5),
                                                (1, False, True, 0.25), (2, True, False, 0.1),
                                                (1, False, False, 0.7), (1, True, True, 0.0),
                                                (2, False, False, 0.0)])
def test_residual_dropout(lib, dt, T, H, ranks, has_x, norm, p):
    g = gen(T, H, ranks, has_x, norm)
    seed, offset, first = -5 - T, 3 + H, 1 << 33
    rng = words(seed, offset) if p else None
    hs = [dev(g.normal(size=(T, H)) * 2, dt) for _ in range(ranks)]
    x = dev(stream_like(g, T, H), dt) if has_x else None
    w = dev(1 + 0.3 * g.normal(size=H), dt) if norm and ranks < 3 else None
    b = dev(g.normal(size=H), dt) if norm else None
    keep = ref.kept(T, H, seed, offset, p, first)
    out = Out()
    xo, n = out(T, H, dtype=DT[dt]), out(T, H, dtype=DT[dt]) if norm else None
    kw = dict(w=w, b=b, eps=EPS, first_row=first)
    pcr.residual_dropout(hs, x, xo, rng, p, n_out=n, **kw)
    want = ref.residual_dropout([f64(t) for t in hs], f64(x), keep, p, f64(w), f64(b), EPS, dt,
                                norm)
    within(xo, want[0], "x_out")
    if norm:
        within(n, want[1], "n_out")
    factor = keep / (1 - float(np.float32(p)))
    dxo = dev(g.normal(size=(T, H)), dt)
    dx, dh, dw, db = out(T, H, dtype=DT[dt]), out(T, H, dtype=DT[dt]), out(H), out(H)
    if norm:
        dn = dev(g.normal(size=(T, H)), dt)
        back = dict(w=w, eps=EPS, first_row=first)
        pcr.residual_dropout_backward(dxo, dn, xo, dx, dh, rng, p, dw=dw, db=db, **back)
        want = ref.layer_norm_backward(f64(dn), f64(xo), f64(w), EPS, dt, f64(dxo), factor)
        for name, t in dict(dx=dx, dh=dh, dw=dw, db=db).items():
            within(t, want[name], name)
        assert not f64(dh)[~keep].any()
        # the parts alone, and without a gradient of x_out
        d2, h2 = out(T, H, dtype=DT[dt]), out(T, H, dtype=DT[dt])
        pcr.residual_dropout_backward(dxo, dn, xo, d2, None, rng, p, **back)
        pcr.residual_dropout_backward(dxo, dn, xo, None, h2, rng, p, **back)
        within(d2, want["dx"], "dx alone")
        within(h2, want["dh"], "dh alone")
        assert not f64(h2)[~keep].any()
        pcr.residual_dropout_backward(dxo, dn, xo, d2, None, None, p, **back)  # no generator needed
        within(d2, want["dx"], "dx without a generator")
        pcr.residual_dropout_backward(None, dn, xo, d2, h2, rng, p, **back)
        want = ref.layer_norm_backward(f64(dn), f64(xo), f64(w), EPS, dt, None, factor)
        within(d2, want["dx"], "dx of the norm alone")
        within(h2, want["dh"], "dh of the norm alone")
        pcr.residual_dropout_backward(dxo, dn, xo, dn, dxo, rng, p, **back)   # in place
        assert same(dn, dx) and same(dxo, dh)
    else:
        pcr.residual_dropout_backward(dxo, None, None, dx, dh, rng, p, dw=dw, db=db,
                                      first_row=first)
        d = f64(dxo)
        assert same(dx, dxo) and not dw.any() and not db.any()
        v = np.where(keep, d, 0.0) / (1 - float(np.float32(p)))
        within(dh, (v, (ref.HALF_ULP[dt] + 3 * ref.U) * np.abs(v) * ref.SLACK + ref.TINY), "dh")
        pcr.residual_dropout_backward(dxo, None, None, None, dxo, rng, p, first_row=first)
        assert same(dxo, dh)
    assert out.intact()
    both = norm and has_x
    pcr.residual_dropout(hs, x, hs[0], rng, p, n_out=x if both else None,   # in place
                         **(kw if both else dict(first_row=first)))
    assert same(hs[0], xo) and (not both or same(x, n))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [64, 65, 66, 68, 2050])
def test_dropped_values_are_not_read_into_the_result(lib, dt, H):
    T, p = 6, 0.5
    keep = ref.kept(T, H, 1, 2, p)
    g = gen(H)
    h = g.normal(size=(T, H))
    loud = np.where(keep, h, np.where(g.random((T, H)) < 0.5, np.nan, np.inf))
    x, rng = dev(g.normal(size=(T, H)), dt), words(1, 2)
    outs = []
    for v in (h, loud):
        xo, n, plain, dh = (torch.empty(T, H, dtype=DT[dt], device="cuda") for _ in range(4))
        pcr.residual_dropout(dev(v, dt), x, xo, rng, p, n_out=n)
        pcr.residual_dropout(dev(v, dt), x, plain, rng, p)
        pcr.residual_dropout_backward(dev(v, dt), None, None, None, dh, rng, p)
        outs.append((xo, n, plain, dh))
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and same(a, b)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [50, 4097, 4098, 4100, 8200])
@pytest.mark.parametrize("tokens", [4, 160])
def test_all_bits_of_the_counters(lib, dt, H, tokens):
    # seeds and offsets with both halves, rows whose counters pass 2^32 and 2^64
    groups, p = (H + 3) // 4, 0.4
    assert groups & groups - 1
    one = torch.ones(tokens, H, device="cuda").to(DT[dt])
    for seed, offset, power in ((0x123456789, -7, 32), (-9, (5 << 40) + 3, 64), (1 << 62, 0, 32)):
        first = (1 << power) // groups - 1  # the second row passes the power
        keep = ref.kept(tokens, H, seed, offset, p, first)
        rng = words(seed, offset)
        for norm in (False, True):
            xo, n, dh = (torch.empty_like(one) for _ in range(3))
            pcr.residual_dropout(one, None, xo, rng, p, n_out=n if norm else None, first_row=first)
            assert np.array_equal(f64(xo) != 0, keep)
            pcr.residual_dropout_backward(one, torch.zeros_like(one) if norm else None,
                                          xo if norm else None, None, dh, rng, p, first_row=first)
            assert np.array_equal(f64(dh) != 0, keep)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(12, 96), (12, 97), (300, 130), (8, 4100), (12, 8192)])
def test_parts_of_the_rows_drop_what_the_whole_does(lib, dt, T, H):
    g = gen(T, H, 5)
    h, x, rng, p = dev(g.normal(size=(T, H)), dt), dev(g.normal(size=(T, H)), dt), words(9, 8), 0.3
    whole, parts = ([torch.empty(T, H, dtype=DT[dt], device="cuda") for _ in range(2)]
                    for _ in range(2))
    pcr.residual_dropout(h, x, whole[0], rng, p, n_out=whole[1], first_row=100)
    for lo, hi in ((0, 1), (1, 5), (5, T)):
        hp, xp = h[lo:hi].clone(), x[lo:hi].clone()
        o, n = torch.empty_like(hp), torch.empty_like(hp)
        pcr.residual_dropout(hp, xp, o, rng, p, n_out=n, first_row=100 + lo)
        plain = torch.empty_like(hp)
        pcr.residual_dropout(hp, xp, plain, rng, p, first_row=100 + lo)
        assert same(plain, o)
        parts[0][lo:hi], parts[1][lo:hi] = o, n
    assert same(parts[0], whole[0])
    # a part may be dealt out to other teams: sums in another order
    assert torch.allclose(parts[1].float(), whole[1].float(), rtol=2 ** -7, atol=1e-5)


def test_replayed_graph_takes_the_generator_as_it_stands():
    T, H, p = 20, 200, 0.4
    h, x, rng = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda"), words(3, 0)
    xo, n, dx, dh = (torch.empty(T, H, device="cuda") for _ in range(4))
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    d = torch.randn(T, H, device="cuda")

    def step():
        pcr.residual_dropout(h, x, xo, rng, p, n_out=n)
        pcr.residual_dropout_backward(d, d, xo, dx, dh, rng, p, dw=dw, db=db)
        rng[1] += 1
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng[1] = 0
    seen = []
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert int(rng[1]) == i + 1
        got = [t.clone() for t in (xo, n, dx, dh, dw, db)]
        rng[1] = i
        step()
        for a, b in zip(got, (xo, n, dx, dh, dw, db)):
            assert same(a, b)
        seen.append(got[0])
    assert not same(seen[0], seen[1]) and not same(seen[1], seen[2])


# -- balance loss -------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 64, 8), (5, 8, 8), (33, 60, 6), (40, 65, 4),
                                   (300, 128, 1), (1100, 200, 10), (9, 384, 32), (6, 1000, 8),
                                   (2500, 16, 2), (3, 1024, 32)])
@pytest.mark.parametrize("padded", [False, True])
def test_balance(lib, dt, T, E, K, padded):
    g = gen(T, E, K, padded)
    z = g.normal(size=(T, E)) * 2
    z[g.random((T, E)) < 0.1] = -np.inf
    if T > 4:
        z[1] = -np.inf                       # no expert left
        z[2, 1:] = -np.inf
        z[3] = 1.0
        z[4, 0] = torch.finfo(DT[dt]).min
    ids = np.stack([g.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    ids[g.random((T, K)) < 0.05] = -1
    ids[g.random((T, K)) < 0.02] = E + 3
    valid = None
    if padded:
        valid = (g.random(T) < 0.7).astype(np.uint8) * 3
        z[valid == 0] = np.nan               # padding is not read into anything
        ids[valid == 0] = 0
    logits, coef = dev(z, dt), 0.37
    z = f64(logits)
    i = torch.from_numpy(ids).cuda()
    v = None if valid is None else torch.from_numpy(valid).cuda()
    out = Out()
    loss, counts, sums, dz = out(1), out(E + 1, dtype=torch.int32), out(E), out(T, E, dtype=DT[dt])
    assert pcr.expert_balance(logits, i, loss, counts, sums, coef=coef, valid=v) is loss
    wl, wc, ws, probs, rate = ref.balance(np.where(np.isnan(z), 0.0, z), ids, valid, coef, E)
    assert np.array_equal(counts.cpu().numpy(), wc)
    within(sums, ws, "prob_sums")
    within(loss, (np.array([wl[0]]), np.array([wl[1]])), "loss")
    dloss = dev([1.7])
    pcr.expert_balance_backward(logits, counts, dloss, dz, coef=coef, valid=v)
    dl = float(np.float32(1.7))
    within(dz, ref.balance_backward(probs, wc[:E], rate, dl, dt), "dlogits")
    before = dev(g.normal(size=(T, E)) * 1e-3, dt)
    more = before.clone()
    pcr.expert_balance_backward(logits, counts, dloss, more, coef=coef, valid=v, accumulate=True)
    within(more, ref.balance_backward(probs, wc[:E], rate, dl, dt, f64(before)), "accumulated")
    if padded:
        pad = torch.from_numpy(valid == 0).cuda()
        assert not dz[pad].any() and same(more[pad], before[pad])
        as_bool = out(1)
        pcr.expert_balance(logits, i, as_bool, counts, sums, coef=coef, valid=v != 0)
        assert same(as_bool, loss)
    again = [torch.empty_like(t) for t in (loss, counts, sums)]
    pcr.expert_balance(logits, i, *again, coef=coef, valid=v)
    assert all(same(a, b) for a, b in zip(again, (loss, counts, sums)))
    assert out.intact()
    pcr.expert_balance_backward(logits, counts, dloss, logits, coef=coef, valid=v)   # in place
    assert same(logits, dz)


def test_balance_of_counts_from_several_ranks(lib):
    # each rank's gradient with the summed counts is its part of the whole batch's
    g = gen(6)
    T, E, K = 64, 24, 3
    z = dev(g.normal(size=(T, E)))
    ids = torch.from_numpy(np.stack([g.permutation(E)[:K] for _ in range(T)]).astype(np.int32)).cuda()
    dloss = torch.ones(1, device="cuda")

    def call(z, ids):
        loss, counts, sums = (torch.empty(1, device="cuda"),
                              torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                              torch.empty(E, device="cuda"))
        pcr.expert_balance(z, ids, loss, counts, sums, coef=0.1)
        return loss, counts, sums
    whole = call(z, ids)
    halves = [call(z[:32].clone(), ids[:32].clone()), call(z[32:].clone(), ids[32:].clone())]
    counts = halves[0][1] + halves[1][1]
    assert torch.equal(counts, whole[1])
    dz, part = torch.empty_like(z), torch.empty(32, E, device="cuda")
    pcr.expert_balance_backward(z, whole[1], dloss, dz, coef=0.1)
    for r in range(2):
        pcr.expert_balance_backward(z[32 * r:32 * r + 32].clone(), counts, dloss, part, coef=0.1)
        assert same(part, dz[32 * r:32 * r + 32])


def test_balance_without_valid_tokens_or_slots(lib):
    E = 12
    loss, counts, sums = (torch.full((1,), 5.0, device="cuda"),
                          torch.full((E + 1,), 5, dtype=torch.int32, device="cuda"),
                          torch.full((E,), 5.0, device="cuda"))
    dz = torch.full((3, E), 5.0, device="cuda")
    z = torch.zeros(3, E, device="cuda")
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    nobody = torch.zeros(3, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    pcr.expert_balance(z, ids, loss, counts, sums, valid=nobody)
    assert not loss.any() and not counts.any() and not sums.any()
    pcr.expert_balance_backward(z, counts, one, dz, valid=nobody)
    assert not dz.any()
    pcr.expert_balance(z, ids - 1, loss, counts, sums)      # no choice of any expert
    assert not loss.any() and counts.tolist() == [0] * E + [3] and sums.sum() > 2.9
    dz.fill_(5.0)
    pcr.expert_balance_backward(z, counts, one, dz)
    assert not dz.any()
    loss.fill_(5.0)
    counts.fill_(5)
    sums.fill_(5.0)
    empty = torch.empty(0, E, device="cuda")
    pcr.expert_balance(empty, ids[:0], loss, counts, sums)
    assert not loss.any() and not counts.any() and not sums.any()


def test_balance_nan_and_infinite_logits(lib):
    z = torch.zeros(4, 9, device="cuda")
    z[1, 3] = float("nan")
    ids = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    loss, counts, sums = (torch.empty(1, device="cuda"),
                          torch.empty(10, dtype=torch.int32, device="cuda"),
                          torch.empty(9, device="cuda"))
    dz = torch.empty_like(z)
    pcr.expert_balance(z, ids, loss, counts, sums)
    assert torch.isnan(loss).all() and torch.isnan(sums).all() and counts.tolist() == [4] + [0] * 8 + [4]
    pcr.expert_balance_backward(z, counts, torch.ones(1, device="cuda"), dz)
    assert torch.isnan(dz[1]).all() and torch.isfinite(dz[[0, 2, 3]]).all()


# -- embedding ----------------------------------------------------------------

def some_ids(g, T, V, first, kind):
    if kind == "same":
        return np.full(T, first + V // 2, np.int64)
    if kind == "none":
        return np.where(g.random(T) < 0.5, -1, first + V).astype(np.int64)
    ids = first + (g.random(T) ** 3 * (V + 3)).astype(np.int64) - 1   # some outside
    ids[g.random(T) < 0.05] = -1
    return ids


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 100, 4096), (7, 3, 5), (64, 700, 96),
                                   (33, 40, 129), (500, 1000, 66), (2100, 5000, 68),
                                   (5000, 300, 40), (70, 1024, 2051), (40, 50, 8200),
                                   (512, 90, 20), (513, 90, 20), (1100, 60, 12), (9000, 33, 8)])
@pytest.mark.parametrize("kind", ["mixed", "same", "none"])
def test_embed(lib, dt, T, V, H, kind):
    g = gen(T, V, H)
    first, scale = 1000, 1.5
    ids = some_ids(g, T, V, first, kind)
    table, dout = dev(g.normal(size=(V, H)), dt), dev(g.normal(size=(T, H)), dt)
    want, back = None, ref.embed_backward(f64(dout), ids, first, V, scale)
    base = dev(g.normal(size=(V, H)))
    added = ref.embed_backward(f64(dout), ids, first, V, scale, f64(base))
    touched = np.zeros(V, bool)
    touched[ids[(ids >= first) & (ids < first + V)] - first] = True
    results = []
    for it in (torch.int64, torch.int32):
        i = torch.from_numpy(ids).to(it).cuda()
        out = Out()
        y, d, more = out(T, H, dtype=DT[dt]), out(V, H), out(V, H)
        assert pcr.token_embed(table, i, y, first_id=first, scale=scale) is y
        want = want or ref.embed(f64(table), ids, first, scale, dt)
        within(y, want, "out")
        assert pcr.token_embed_backward(dout, i, d, first_id=first, scale=scale) is d
        within(d, back, "dtable")
        more.copy_(base)
        pcr.token_embed_backward(dout, i, more, first_id=first, scale=scale, accumulate=True)
        within(more, added, "accumulated")
        rest = torch.from_numpy(~touched).cuda()
        assert same(more[rest], base[rest]) and not d[rest].any()
        again = torch.full_like(d, 3.0)
        pcr.token_embed_backward(dout, i, again, first_id=first, scale=scale)
        assert same(again, d) and out.intact()
        results.append((y, d, more))
    for a, b in zip(*results):
        assert same(a, b)


@pytest.mark.parametrize("T,V", [(3000, 511), (3000, 512), (3000, 1 << 18), (3000, (1 << 18) + 1),
                                 (3000, 3_000_000), (8192, 40000), (8193, 40000), (65536, 700),
                                 (65537, 700), (70001, 300_000)])
def test_embed_gradient_at_the_sizes_of_the_sort(lib, T, V):
    g = gen(T, V)
    H = 4
    ids = g.integers(0, V, size=T)
    ids[:4] = [0, V - 1, V, -1]
    ids[100:400] = V - 1
    dout = dev(g.normal(size=(T, H)))
    d = torch.empty(V, H, device="cuda")
    pcr.token_embed_backward(dout, torch.from_numpy(ids).cuda(), d)
    rows = np.unique(ids[(ids >= 0) & (ids < V)])
    place = np.full(V + 2, -1)
    place[rows] = np.arange(len(rows))
    local = np.where((ids >= 0) & (ids < V), place[np.clip(ids, 0, V)], -1)
    value, bound = ref.embed_backward(f64(dout), local, 0, len(rows), 1.0)
    within(d[torch.from_numpy(rows).cuda()], (value, bound), "rows")
    d[torch.from_numpy(rows).cuda()] = 0
    assert not d.any()


def test_embed_ids_at_the_ends_of_their_type(lib):
    table = torch.randn(4, 8, device="cuda")
    lo, hi = -(1 << 63), (1 << 63) - 1
    for first in (lo, -2, 0, hi - 3):
        i = [lo, lo + 1, -1, 0, 1, hi - 1, hi, hi - 3, first, first + 3]
        ids = torch.tensor(i, dtype=torch.int64, device="cuda")
        y, d = torch.full((len(i), 8), 9.0, device="cuda"), torch.empty(4, 8, device="cuda")
        pcr.token_embed(table, ids, y, first_id=first)
        pcr.token_embed_backward(torch.ones_like(y), ids, d, first_id=first)
        n = [0] * 4
        for t, v in enumerate(i):
            inside = first <= v < first + 4
            assert torch.equal(y[t], table[v - first] if inside else torch.zeros(8, device="cuda"))
            if inside:
                n[v - first] += 1
        assert d[:, 0].tolist() == n


def test_embed_without_tokens_rows_or_columns(lib):
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    y = torch.full((3, 8), 5.0, device="cuda")
    pcr.token_embed(torch.empty(0, 8, device="cuda"), ids, y)          # no rows: zeros
    assert not y.any()
    d = torch.full((70, 8), 5.0, device="cuda")
    pcr.token_embed_backward(y[:0], ids[:0], d, accumulate=True)
    assert (d == 5).all()
    pcr.token_embed_backward(y[:0], ids[:0], d)                        # no tokens: zeros
    assert not d.any()
    pcr.token_embed(d, ids[:0], y[:0])
    pcr.token_embed_backward(y, ids, d[:0])
    pcr.token_embed(torch.empty(4, 0, device="cuda"), ids, torch.empty(3, 0, device="cuda"))
    pcr.token_embed_backward(torch.empty(3, 0, device="cuda"), ids, torch.empty(4, 0, device="cuda"))


def test_embed_gradient_of_infinite_values_stays_in_its_row(lib):
    ids = torch.tensor([2, 0, 2, 1, -1, 2], device="cuda")
    dout = torch.ones(6, 40, device="cuda")
    dout[3] = float("inf")
    dout[4] = float("nan")                                             # padding's
    d = torch.empty(4, 40, device="cuda")
    pcr.token_embed_backward(dout, ids, d)
    assert (d[0] == 1).all() and torch.isinf(d[1]).all() and (d[2] == 3).all() and not d[3].any()


# -- refusals of the binding --------------------------------------------------

def test_binding_refusals():
    f, b16 = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, device="cuda").bfloat16()
    with pytest.raises(TypeError):
        pcr.layer_norm(f, b16)
    with pytest.raises(ValueError):
        pcr.layer_norm(f, torch.empty(4, 63, device="cuda"))
    with pytest.raises(ValueError):
        pcr.layer_norm(f, f, w=torch.empty(63, device="cuda"))
    with pytest.raises(ValueError):
        pcr.layer_norm(torch.empty(64, 4, device="cuda").t(), f)       # not contiguous
    with pytest.raises(ValueError):
        pcr.layer_norm(f.cpu(), f)
    with pytest.raises(pcr.LpcollError):
        pcr.layer_norm(f, f, eps=0.0)
    with pytest.raises(TypeError):
        pcr.layer_norm(f.half(), f.half())
    with pytest.raises(ValueError):
        pcr.layer_norm_backward(f, f, f, dw=torch.empty(64, device="cuda"),
                                workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    rng = words(0, 0)
    with pytest.raises(pcr.LpcollError):
        pcr.residual_dropout(f, f, f, rng, 1.0)
    with pytest.raises(pcr.LpcollError):
        pcr.residual_dropout(f, f, f, None, 0.5)
    with pytest.raises(TypeError):
        pcr.residual_dropout(f, f, f, rng.int(), 0.5)
    with pytest.raises(ValueError):
        pcr.residual_dropout(f, f, f, rng, 0.5, w=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        pcr.residual_dropout([], f, f, rng, 0.5)
    with pytest.raises(ValueError):
        pcr.residual_dropout(f, f, f, rng, 0.5, first_row=-1)
    with pytest.raises(ValueError):
        pcr.residual_dropout_backward(None, None, f, f, f, rng, 0.5)
    with pytest.raises(ValueError):
        pcr.residual_dropout_backward(f, f, None, f, f, rng, 0.5)
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    one, n = torch.empty(1, device="cuda"), torch.empty(65, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pcr.expert_balance(f, ids, one, n[:64], torch.empty(64, device="cuda"))
    with pytest.raises(TypeError):
        pcr.expert_balance(f, ids.long(), one, n, torch.empty(64, device="cuda"))
    with pytest.raises(ValueError):
        pcr.expert_balance(f, ids, one, n, torch.empty(64, device="cuda"),
                           valid=torch.ones(3, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        pcr.expert_balance_backward(f, n, 1.0, f)
    with pytest.raises(TypeError):
        pcr.token_embed(f, torch.zeros(4, device="cuda"), f)
    with pytest.raises(ValueError):
        pcr.token_embed(f, torch.zeros(3, dtype=torch.int64, device="cuda"), f)
    with pytest.raises(TypeError):
        pcr.token_embed_backward(f, torch.zeros(4, dtype=torch.int64, device="cuda"), b16)


# -- calls at the same time -----------------------------------------------------

def test_calls_of_two_threads_on_their_own_streams():
    # each thread's results are those of the calls one after the other
    import threading
    T, H, V, E = 1500, 320, 700, 24

    def inputs(i):
        r = torch.Generator(device="cuda").manual_seed(i)
        x, d = (torch.randn(T, H, device="cuda", generator=r) for _ in range(2))
        return dict(x=x, d=d, ids=torch.randint(0, V, (T,), device="cuda", generator=r),
                    z=torch.randn(T, E, device="cuda", generator=r),
                    k=torch.randint(0, E, (T, 2), device="cuda", generator=r).int(),
                    rng=words(i, 1))

    def run(s):
        o = [torch.empty(T, H, device="cuda") for _ in range(5)]
        dw, db, dt_ = (torch.empty(H, device="cuda"), torch.empty(H, device="cuda"),
                       torch.empty(V, H, device="cuda"))
        loss, n, sums = (torch.empty(1, device="cuda"),
                         torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                         torch.empty(E, device="cuda"))
        for _ in range(10):
            pcr.residual_dropout(s["x"], s["d"], o[0], s["rng"], 0.2, n_out=o[1])
            pcr.residual_dropout_backward(s["d"], s["x"], o[0], o[2], o[3], s["rng"], 0.2, dw=dw, db=db)
            pcr.layer_norm_backward(o[2], o[0], o[4], dw=dw)
            pcr.token_embed_backward(o[4], s["ids"], dt_)
            pcr.expert_balance(s["z"], s["k"], loss, n, sums)
        return [*o, dw, db, dt_, loss, n, sums]
    sets = [inputs(i) for i in range(3)]
    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    got, errors = [None] * 3, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got[i] = run(sets[i])
            stream.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(same(x, y) for x, y in zip(a, b))
