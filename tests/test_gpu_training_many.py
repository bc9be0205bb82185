"""The operators of a training step at sizes where every loop of their kernels runs more
than once: teams that take many rows, rings that come round, second tokens of a pair,
rows cut over several CTAs, tiles of every length, counters of a row's later pieces.
Against plain 64-bit forms (torch on the GPU, with the bounds of training_ref.py), on
both builds of the library."""
import numpy as np
import pytest
import torch

import precision_collective_reduction_gb300 as pcr
import training_ref as ref
from layers_ref import HALF_ULP, TINY, U
from precision_collective_reduction_gb300 import _binding as B
from precision_collective_reduction_gb300 import build as lib_build
from training_ref import DEEP, OPS, SLACK

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = float(np.float32(1e-5))


def on_both_builds(check):
    """check() with the library, and with the bounds-checked one, which must record
    nothing."""
    lib_build.build()
    check()
    with B.using_library(lib_build.build(debug_bounds=True)):
        B.debug_bounds_errors()
        check()
        st, bad = B.debug_bounds_errors()
        assert st == 0, "access outside the call's buffers (status %d, first 0x%x)" % (st, bad)


def rand(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float64)


def within(got, want, what):
    value, bound = want
    off = (got.double() - value).abs()
    bad = ~(off <= bound)
    assert got.shape == value.shape and not bad.any(), \
        "%s: %d of %d values outside, worst %g times the bound, first at %s" % (
            what, int(bad.sum()), bad.numel(), float((off / bound).max()),
            bad.nonzero()[0].tolist())


def rounded(value, error, dt):
    return value, (HALF_ULP[dt] * value.abs() + error) * SLACK + TINY


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def poisoned(*tensors):
    for t in tensors:
        t.view(torch.uint8).fill_(0xA5)


# -- the norms ------------------------------------------------------------------

def row_mean(x):
    return x.mean(1, keepdim=True)


def stats(x, ex):
    """training_ref._stats in torch."""
    m = row_mean(x)
    c = x - m
    v = row_mean(c * c)
    r = 1 / torch.sqrt(v + EPS)
    em = (DEEP + 4) * U * row_mean(x.abs()) + row_mean(ex)
    ev = (DEEP + 10) * U * v + 2 * v.sqrt() * em + em ** 2 + 2 * row_mean(c.abs() * ex)
    er = 0.5 * ev / (v + EPS) + 8 * U
    xh = c * r
    return xh, r, r * (em + ex + U * c.abs()) + xh.abs() * er, er


def norm_form(x, w, b, dt, ex):
    xh, _, exh, _ = stats(x, ex)
    return rounded(xh * w + b, w.abs() * exh + OPS * U * ((xh * w).abs() + b.abs()), dt)


def gradient_form(dn, x, w, dt, dxo, factor):
    T = x.shape[0]
    xh, r, exh, er = stats(x, torch.zeros_like(x))
    q = dn * w
    mq, aq = row_mean(q), row_mean(q.abs())
    s = row_mean(q * xh)
    es = (DEEP + OPS) * U * 3 * aq * xh.abs().amax(1, keepdim=True) + row_mean(q.abs() * exh)
    inner = q - mq - xh * s
    D = r * inner + dxo
    size = r * (q.abs() + aq + (xh * s).abs()) + dxo.abs()
    eD = (OPS * U * size + r * ((DEEP + OPS) * U * aq + exh * s.abs() + xh.abs() * es)
          + 2 * er * r * (inner.abs() + (xh * s).abs()))
    return dict(dx=rounded(D, eD, dt),
                dh=rounded(D * factor, (eD + 3 * U * D.abs()) * factor, dt),
                dw=((dn * xh).sum(0), ((T + OPS) * U * (dn * xh).abs().sum(0)
                                       + (dn.abs() * exh).sum(0)) * SLACK + TINY),
                db=(dn.sum(0), (T + OPS) * U * dn.abs().sum(0) + TINY))


def dropped_form(hs, x, keep, p, dt):
    f = keep / (1 - p)
    d, habs = sum(hs) * f, sum(h.abs() for h in hs) * f
    xo = d if x is None else x + d
    ex = (len(hs) + 3) * U * habs + (0.0 if x is None else 2 * U * x.abs())
    return rounded(xo, ex, dt), xo, ex


# Turns of a team at these sizes, forward and back: 2 to 25 of them.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(45000, 256), (60000, 60), (15000, 768), (15000, 300),
                                 (30000, 97), (4000, 1280), (3000, 2050), (3000, 2051),
                                 (1000, 4096), (1000, 4098), (1000, 4099), (1000, 4100),
                                 (1000, 8192), (1000, 8191), (700, 12288), (700, 16384)])
def test_teams_that_take_many_rows(dt, T, H):
    g = rand(T + H)
    level, loud = normal(g, 1, H), normal(g, 1, H).exp()

    def stream():
        return ((normal(g, T, H) + level) * loud).to(DT[dt])
    x, dn, dxo, h2 = stream(), normal(g, T, H).to(DT[dt]), stream(), stream()
    x[T // 2] = 7.25
    w, b = (1 + 0.3 * normal(g, H)).to(DT[dt]), normal(g, H).to(DT[dt])
    p, first = float(np.float32(0.3)), (1 << 33) + 7
    rng = torch.tensor([T, H], device="cuda")
    keep = torch.from_numpy(ref.kept(T, H, T, H, p, first)).cuda()
    xd, wd, bd, dnd, dxod = x.double(), w.double(), b.double(), dn.double(), dxo.double()
    zero = torch.zeros_like(xd)
    want_y = norm_form(xd, wd, bd, dt, zero)
    want_g = gradient_form(dnd, xd, wd, dt, zero, 1.0)
    want_d = gradient_form(dnd, xd, wd, dt, dxod, keep / (1 - p))
    drops = []
    for hs, res in (([dxo], x), ([dxo, h2, dn], x), ([h2], None)):
        xo, exact, ex = dropped_form([h.double() for h in hs], None if res is None else xd, keep,
                                     p, dt)
        drops.append((hs, res, xo, norm_form(exact, wd, bd, dt, ex)))
    y, dx, dh = (torch.empty_like(x) for _ in range(3))
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")

    def check():
        poisoned(y, dx, dw, db)
        pcr.layer_norm(x, y, w=w, b=b, eps=EPS)
        within(y, want_y, "norm")
        pcr.layer_norm_backward(dn, x, dx, w=w, eps=EPS, dw=dw, db=db)
        for name, t in dict(dx=dx, dw=dw, db=db).items():
            within(t, want_g[name], name)
        poisoned(dx, dh, dw, db)
        pcr.layer_norm_backward(dn, x, None, w=w, eps=EPS, dw=dw)
        within(dw, want_g["dw"], "dw alone")
        kw = dict(w=w, eps=EPS, first_row=first)
        pcr.residual_dropout_backward(dxo, dn, x, dx, dh, rng, p, dw=dw, db=db, **kw)
        for name, t in dict(dx=dx, dh=dh, dw=dw, db=db).items():
            within(t, want_d[name], "dropout " + name)
        assert not dh[~keep].any()
        for hs, res, xo, n in drops:
            poisoned(y, dx)
            pcr.residual_dropout(hs, res, y, rng, p, n_out=dx, b=b, **kw)
            within(y, xo, "x_out")
            within(dx, n, "n_out")
    on_both_builds(check)


# Rows of more than 256 pieces in one CTA, and several short rows in one: 622592 pieces
# of 16 bytes and more.
@pytest.mark.parametrize("T,H,dt", [(700, 8200, "bf16"), (700, 4100, "f32"), (1300, 2051, "f32"),
                                    (1300, 4097, "bf16"), (1300, 4098, "bf16"),
                                    (80000, 40, "f32"), (90000, 60, "bf16"), (70000, 33, "f32")])
@pytest.mark.parametrize("ranks,has_x", [(1, True), (3, False)])
def test_dropout_without_norm_of_many_pieces(T, H, dt, ranks, has_x):
    assert T * -(-H * DT[dt].itemsize // 16) >= 152 * 16 * 256
    g = rand(T + H + ranks)
    hs = [normal(g, T, H).to(DT[dt]) for _ in range(ranks)]
    x = normal(g, T, H).to(DT[dt]) if has_x else None
    p, groups = float(np.float32(0.4)), -(-H // 4)
    first = (1 << 32) // groups - T // 2        # counters pass 2^32 in the middle
    rng = torch.tensor([-3, 1 << 40], device="cuda")
    keep = torch.from_numpy(ref.kept(T, H, -3, 1 << 40, p, first)).cuda()
    want = dropped_form([h.double() for h in hs], None if x is None else x.double(), keep, p, dt)[0]
    back = dropped_form([hs[0].double()], None, keep, p, dt)[0]
    xo, dx, dh = (torch.empty_like(hs[0]) for _ in range(3))

    def check():
        poisoned(xo, dx, dh)
        pcr.residual_dropout(hs, x, xo, rng, p, first_row=first)
        within(xo, want, "x_out")
        pcr.residual_dropout_backward(hs[0], None, None, dx, dh, rng, p, first_row=first)
        within(dh, back, "dh")
        assert same(dx, hs[0]) and torch.equal(dh != 0, keep & (hs[0] != 0))
    on_both_builds(check)


# -- balance loss -----------------------------------------------------------------

# One cluster that goes through its tokens several times; a second token beside the first
# (up to 256 experts) and second and third steps of the loops, forward (every 152 CTAs of
# 32 to 128 tokens) and back (1216 CTAs of 8 to 32).
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", [(512, 256, 8), (512, 100, 2), (12000, 256, 4), (21000, 200, 4),
                                   (45000, 16, 2), (80000, 16, 1), (30000, 128, 6),
                                   (12000, 384, 8), (10000, 1000, 3)])
@pytest.mark.parametrize("padded", [False, True])
def test_balance_of_many_tokens(dt, T, E, K, padded):
    g = rand(T + E + K + padded)
    z = 2 * normal(g, T, E)
    z[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -np.inf
    z[5] = -np.inf
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].int()
    ids[torch.rand(T, K, generator=g, device="cuda") < 0.03] = -1
    there, valid = torch.ones(T, dtype=torch.bool, device="cuda"), None
    if padded:
        valid = there = torch.rand(T, generator=g, device="cuda") < 0.7
        z[~valid] = np.nan
    logits, coef, dl = z.to(DT[dt]), 0.37, 1.7
    # the plain form, with training_ref's bounds
    z = torch.where(there[:, None], logits.double(), torch.tensor(-np.inf, device="cuda"))
    m = z.amax(1, keepdim=True)
    some = torch.isfinite(m)
    d = torch.where(some, z - m, torch.full_like(z, -np.inf))
    p = d.exp()
    p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    far = torch.where(torch.isfinite(d), -d, torch.zeros_like(d)).clamp_max(120.0)
    ep = (far + far.amax(1, keepdim=True) + DEEP + 32 + 12) * U * p + TINY * some
    mine = ids[there].flatten()
    n = torch.bincount(mine[mine >= 0], minlength=E).double()
    P = p.sum(0)
    S, V = float(n.sum()), float(there.sum())
    eP = ep.sum(0) + (T + DEEP) * U * P
    rate = float(np.float32(coef)) * E / (S * V)
    loss_form = (rate * (n * P).sum()[None],
                 (rate * ((n * eP).sum() + (E + DEEP) * U * (n * P).sum()) + TINY)[None])
    k = rate * float(np.float32(dl))
    mean = (p * n).sum(1, keepdim=True)
    emean = (ep * n).sum(1, keepdim=True) + (DEEP + 32) * U * mean
    grad = k * p * (n - mean)
    e = k * (ep * (n + mean) + p * emean + OPS * U * p * (n + mean))
    before = (1e-6 * normal(g, T, E)).to(DT[dt])
    added = grad + before.double()
    want = rounded(grad, e, dt)
    want_added = rounded(added, e + 2 * U * (added.abs() + before.double().abs()), dt)
    loss, sums, dloss = (torch.empty(1, device="cuda"), torch.empty(E, device="cuda"),
                         torch.full((1,), dl, device="cuda"))
    counts, dz = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty_like(logits)

    def check():
        poisoned(loss, sums, counts, dz)
        pcr.expert_balance(logits, ids, loss, counts, sums, coef=coef, valid=valid)
        assert torch.equal(counts[:E].double(), n) and int(counts[E]) == V
        within(sums, (P, eP + TINY), "prob_sums")
        within(loss, loss_form, "loss")
        pcr.expert_balance_backward(logits, counts, dloss, dz, coef=coef, valid=valid)
        within(dz, want, "dlogits")
        more = before.clone()
        pcr.expert_balance_backward(logits, counts, dloss, more, coef=coef, valid=valid,
                                    accumulate=True)
        within(more, want_added, "accumulated")
        assert same(more[~there], before[~there]) and not dz[~there].any()
    on_both_builds(check)


# -- embedding --------------------------------------------------------------------

# Four pieces a lane: many tokens, rows of several CTAs, of one, and several to a CTA.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", [(700, 300, 8200), (700, 300, 2051), (2500, 700, 2048),
                                   (1300, 400, 4098), (1300, 400, 4096), (3000, 90, 1025),
                                   (40000, 5000, 68), (40000, 5000, 33)])
@pytest.mark.parametrize("scale", [1.0, 1.5])
def test_embedded_rows_of_many_tokens(dt, T, V, H, scale):
    g = rand(T + H)
    table, first = normal(g, V, H).to(DT[dt]), 50
    ids = torch.randint(first - V // 8, first + V + V // 8, (T,), generator=g, device="cuda")
    local = ids - first
    inside = (local >= 0) & (local < V)
    value = table.double()[local.clamp(0, V - 1)] * scale * inside[:, None]
    out = torch.empty(T, H, device="cuda").to(DT[dt])

    def check():
        for index in (torch.int64, torch.int32):
            poisoned(out)
            pcr.token_embed(table, ids.to(index), out, first_id=first, scale=scale)
            if scale == 1.0:
                assert torch.equal(out.double(), value)
            within(out, (value, (HALF_ULP[dt] + U) * value.abs() * SLACK + TINY), "out")
            assert not out[~inside].view(torch.uint8).any()     # +0
    on_both_builds(check)


def embed_gradient(T, V, H, dt, ids, scale, seed):
    """The gradient against 64 bits, written and added to what stands there."""
    g = rand(seed)
    dout, first = normal(g, T, H).to(DT[dt]), 1000
    inside = (ids >= 0) & (ids < V)
    rows, where, n = ids[inside].unique(return_inverse=True, return_counts=True)
    value, size = (torch.zeros(len(rows), H, dtype=torch.float64, device="cuda") for _ in range(2))
    value.index_add_(0, where, dout[inside].double())
    size.index_add_(0, where, dout[inside].double().abs())
    value, size = value * scale, size * scale
    base = torch.randn(V, H, generator=g, device="cuda")
    at = base[rows].double()
    want = (value, (n[:, None] + 3) * U * size + TINY)
    want_added = (value + at, (n[:, None] + 3) * U * (size + at.abs()) + TINY)
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[rows] = False
    d = torch.empty(V, H, device="cuda")

    def check():
        poisoned(d)
        i = ids + first
        pcr.token_embed_backward(dout, i, d, first_id=first, scale=scale)
        within(d[rows], want, "rows")
        assert not d[rest].view(torch.uint8).any()
        again = torch.full_like(d, 3.0)
        pcr.token_embed_backward(dout, i.int(), again, first_id=first, scale=scale)
        assert same(again, d)
        d.copy_(base)
        pcr.token_embed_backward(dout, i, d, first_id=first, scale=scale, accumulate=True)
        within(d[rows], want_added, "accumulated")
        assert same(d[rest], base[rest])
    on_both_builds(check)


# Rows of the table that one CTA sums, and several; tables of which a part is cleared
# beside the sort and the rest beside the sums (up to 144 CTAs of 8 to 64 rows there).
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [700, 2100, 9000])
@pytest.mark.parametrize("V,H", [(10001, 1025), (5003, 2051), (2600, 4096), (1301, 8200),
                                 (60, 4096), (300, 8200), (2700, 4098)])
def test_embedding_gradient_of_wide_rows(dt, T, V, H):
    g = rand(T + H + V)
    ids = torch.randint(-2, V + 1, (T,), generator=g, device="cuda")
    ids[100:400] = V // 3               # several tiles, and next to another such run
    ids[400:500] = V // 3 + 1
    ids[0], ids[1] = 0, V - 1
    embed_gradient(T, V, H, dt, ids, 1.5, T + V)


# Sorted in one cluster of every size, and through memory, with tiles of 8 to 1024.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,H", [(20000, 5000, 300), (65536, 3000, 36), (66000, 3000, 36),
                                   (150000, 70000, 8), (300000, 2000, 20), (150001, 40, 5),
                                   (4400000, 30000, 4), (2000001, 9, 3)])
def test_embedding_gradient_of_many_tokens(dt, T, V, H):
    g = rand(T + V)
    ids = (torch.rand(T, generator=g, device="cuda", dtype=torch.float64) ** 4 * (V + 2)).long() - 1
    ids[T // 3:T // 2] = V // 2
    embed_gradient(T, V, H, dt, ids, 0.5, T)
