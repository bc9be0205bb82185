"""The operators of a training step without a GPU: refusals of the C entry points
(every call fails its checks before any launch), sizes of the workspaces, the
generator's published words, and the reference gradients against differences."""
import numpy as np
import pytest

import precision_collective_reduction_gb300 as pcr
import training_ref as ref
from precision_collective_reduction_gb300 import _binding as B
from precision_collective_reduction_gb300 import build as lib_build

OK, ARG, ALIGN, UNSUP, RANK = 0, 1, 2, 3, 4
A = 0x10000  # an aligned fake device address: never dereferenced in these calls
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return pcr.lib()


def test_layer_norm_refusals(L):
    def f(x=A, w=A, b=A, eps=1e-5, T=4, H=64, dt=0, out=A):
        return L.layer_norm(x, w, b, eps, T, H, dt, out, None)
    assert f(dt=2) == ARG and f(dt=-1) == ARG
    for eps in (0.0, -1.0, NAN, INF):
        assert f(eps=eps) == ARG
    assert f(H=16385) == UNSUP and f(T=1 << 31) == ARG
    assert f(T=0, x=None, out=None) == OK and f(H=0, x=None, out=None) == OK
    assert f(x=None) == ARG and f(out=None) == ARG
    assert f(x=A + 4, out=None) == ARG                      # NULL before alignment
    for name in ("x", "w", "b", "out"):
        assert f(**{name: A + 8}) == ALIGN
    need = L.layer_norm_backward_workspace_bytes(4, 64, 0)
    assert need > 0 and L.layer_norm_backward_workspace_bytes(0, 64, 0) == 0
    assert L.layer_norm_backward_workspace_bytes(4, 16385, 0) == 0
    assert L.layer_norm_backward_workspace_bytes(4, 64, 7) == 0

    def g(dout=A, x=A, w=A, eps=1e-5, T=4, H=64, dt=0, dx=A, dw=A, db=A, ws=A, n=need):
        return L.layer_norm_backward(dout, x, w, eps, T, H, dt, dx, dw, db, ws, n, None)
    assert g(dt=3) == ARG and g(eps=0.0) == ARG and g(H=1 << 20) == UNSUP
    assert g(n=need - 1) == ARG and g(ws=None) == ARG
    assert g(dout=None) == ARG and g(x=None) == ARG
    for name in ("dout", "x", "w", "dx", "dw", "db", "ws"):
        assert g(**{name: A + 4}) == ALIGN
    assert g(H=0, dout=None) == OK
    assert g(dx=None, dw=None, db=None, dout=None, ws=None, n=0) == OK  # nothing wanted


def test_residual_dropout_refusals(L):
    two = B.ptr_array([A, A])

    def f(h=two, n=2, x=A, rng=A, p=0.1, first=0, w=A, b=A, eps=1e-5, T=4, H=64, dt=0, xo=A,
          no=A):
        return L.residual_dropout(h, n, x, rng, p, first, w, b, eps, T, H, dt, xo, no, None)
    for p in (1.0, -0.1, 2.0, NAN, INF):
        assert f(p=p) == ARG
    assert f(dt=2) == ARG and f(n=0) == ARG and f(n=17) == ARG
    assert f(eps=0.0) == ARG and f(H=16385) == UNSUP
    assert f(T=1 << 31) == ARG and f(T=1 << 30, H=4096, no=None) == ARG
    assert f(T=1, H=(1 << 30) + 1, no=None) == ARG
    assert f(T=0, h=None, rng=None, xo=None) == OK and f(H=0, h=None) == OK
    assert f(h=None) == ARG and f(h=B.ptr_array([A, None])) == RANK
    assert f(rng=None) == ARG and f(xo=None) == ARG
    assert f(h=B.ptr_array([A, A + 8])) == ALIGN
    for name in ("x", "rng", "w", "b", "xo", "no"):
        assert f(**{name: A + 8}) == ALIGN
    need = L.residual_dropout_backward_workspace_bytes(4, 64, 0)
    assert need > 0 and L.residual_dropout_backward_workspace_bytes(4, 20000, 0) == 0

    def g(dxo=A, dn=A, xo=A, rng=A, p=0.1, first=0, w=A, eps=1e-5, T=4, H=64, dt=0, dx=A, dh=A,
          dw=A, db=A, ws=A, n=need):
        return L.residual_dropout_backward(dxo, dn, xo, rng, p, first, w, eps, T, H, dt, dx, dh,
                                           dw, db, ws, n, None)
    assert g(p=1.0) == ARG and g(p=NAN) == ARG and g(dt=2) == ARG and g(eps=0.0) == ARG
    assert g(H=16385) == UNSUP
    assert g(n=need - 1) == ARG and g(ws=None) == ARG
    assert g(xo=None) == ARG and g(rng=None) == ARG
    assert g(dxo=None, dn=None) == ARG
    for name in ("dxo", "dn", "xo", "rng", "w", "dx", "dh", "dw", "db", "ws"):
        assert g(**{name: A + 4}) == ALIGN
    assert g(H=0, dxo=None, dn=None) == OK
    assert g(dx=None, dh=None, dw=None, db=None, ws=None, n=0) == OK
    assert g(dn=None, T=0, dw=None, db=None, ws=None, n=0) == OK


def test_balance_refusals(L):
    need = L.expert_balance_workspace_bytes(4000, 8)
    assert need > 0 and L.expert_balance_workspace_bytes(4000, 0) == 0
    assert L.expert_balance_workspace_bytes(4, 1025) == 0
    assert L.expert_balance_workspace_bytes((1 << 31) - 1, 1024) <= 304 * 2049 * 4

    def f(z=A, dt=0, T=4000, E=8, ids=A, K=2, valid=None, coef=0.01, loss=A, counts=A, sums=A, ws=A,
          n=need):
        return L.expert_balance(z, dt, T, E, ids, K, valid, coef, loss, counts, sums, ws, n, None)
    assert f(dt=2) == ARG and f(E=0) == ARG and f(E=1025) == ARG and f(K=0) == ARG
    assert f(K=9) == ARG and f(E=64, K=33) == ARG and f(T=1 << 31) == ARG
    assert f(n=need - 1) == ARG and f(ws=None) == ARG
    for name in ("z", "ids", "loss", "counts", "sums"):
        assert f(**{name: None}) == ARG
    for name in ("z", "ids", "valid", "loss", "counts", "sums", "ws"):
        assert f(**{name: A + 4}) == ALIGN

    def g(z=A, dt=0, T=4, E=8, valid=None, counts=A, coef=0.01, dloss=A, acc=0, dz=A):
        return L.expert_balance_backward(z, dt, T, E, valid, counts, coef, dloss, acc, dz, None)
    assert g(dt=2) == ARG and g(E=0) == ARG and g(E=2000) == ARG
    assert g(T=0, z=None, counts=None, dloss=None, dz=None) == OK
    for name in ("z", "counts", "dloss", "dz"):
        assert g(**{name: None}) == ARG
    for name in ("z", "valid", "counts", "dloss", "dz"):
        assert g(**{name: A + 8}) == ALIGN


def test_embed_refusals(L):
    def f(table=A, V=16, ids=A, index=0, first=0, T=4, H=64, dt=0, scale=1.0, out=A):
        return L.token_embed(table, V, ids, index, first, T, H, dt, scale, out, None)
    assert f(dt=2) == ARG and f(index=2) == ARG and f(index=-1) == ARG
    assert f(T=1 << 31) == ARG and f(V=1 << 31) == ARG and f(T=1 << 30, H=4096) == ARG
    assert f(T=1, H=(1 << 30) + 1) == ARG
    assert f(T=0, table=None, ids=None, out=None) == OK and f(H=0, table=None) == OK
    assert f(table=None) == ARG and f(ids=None) == ARG and f(out=None) == ARG
    for name in ("table", "ids", "out"):
        assert f(**{name: A + 8}) == ALIGN
    need = L.token_embed_backward_workspace_bytes(4000, 16, 64)
    assert need > 0 and L.token_embed_backward_workspace_bytes(0, 16, 64) == 0
    assert L.token_embed_backward_workspace_bytes(1 << 31, 16, 64) == 0

    def g(dout=A, ids=A, index=0, first=0, T=4000, V=16, H=64, dt=0, scale=1.0, acc=0, dtable=A,
          ws=A, n=need):
        return L.token_embed_backward(dout, ids, index, first, T, V, H, dt, scale, acc, dtable,
                                      ws, n, None)
    assert g(dt=2) == ARG and g(index=5) == ARG and g(V=1 << 31) == ARG
    assert g(n=need - 1) == ARG and g(ws=None) == ARG
    assert g(dout=None) == ARG and g(ids=None) == ARG and g(dtable=None) == ARG
    for name in ("dout", "ids", "dtable", "ws"):
        assert g(**{name: A + 8}) == ALIGN
    assert g(V=0, dtable=None) == OK and g(H=0, dtable=None) == OK
    assert g(T=0, acc=1, dout=None, ids=None, dtable=None, ws=None, n=0) == OK
    # the partial rows of many tokens stay bounded
    assert L.token_embed_backward_workspace_bytes(1 << 22, 50000, 8192) < 1 << 30


def test_generator_words():
    # the words that the method's authors publish for ten rounds
    assert ref.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert ref.philox([ones] * 4, [ones] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]
                      ) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    # the array form, groups of four columns one counter apart
    seed, offset, first = 0x299F31D0A4093822, -3, (1 << 40) + 5
    keep = ref.kept(3, 10, seed, offset, 0.3, first)
    least = int(float(np.float32(0.3)) * 2 ** 32)
    for t in range(3):
        for c in range(10):
            n = (first + t) * 3 + c // 4
            o = offset & (1 << 64) - 1
            w = ref.philox([n & ones, n >> 32, o & ones, o >> 32], [seed & ones, seed >> 32])
            assert keep[t, c] == (w[c % 4] >= least)


def test_generator_rate():
    # 40000 draws: five standard deviations about the share that is kept
    for p in (0.1, 0.5, 0.9):
        keep = ref.kept(100, 400, 17, 4, p)
        assert abs(keep.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / keep.size)
    assert ref.kept(50, 33, 1, 2, 0.0).all()
    a, b = ref.kept(50, 40, 1, 2, 0.5), ref.kept(50, 40, 1, 3, 0.5)
    assert 0.4 < (a != b).mean() < 0.6
    assert np.array_equal(ref.kept(20, 40, 1, 2, 0.5, 30), a[30:])


def differences(loss, v, step=1e-6):
    want = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        up, dn = v.copy(), v.copy()
        up[i] += step
        dn[i] -= step
        want[i] = (loss(up) - loss(dn)) / (2 * step)
    return want


@pytest.mark.parametrize("weighted", [True, False])
def test_reference_norm_gradient_against_differences(weighted):
    g = np.random.default_rng([5, weighted])
    T, H, eps = 3, 6, 1e-3
    h, x, dxo, dn = (g.normal(size=(T, H)) for _ in range(4))
    w = 1 + g.normal(size=H) if weighted else None
    b = g.normal(size=H) if weighted else None
    keep = ref.kept(T, H, 5, 6, 0.25)

    def both(h, x, w, b):
        return ref.residual_dropout([h], x, keep, 0.25, w, b, eps, "f32", True)

    def loss(h, x, w, b):
        a, n = both(h, x, w, b)
        return (a[0] * dxo).sum() + (n[0] * dn).sum()
    xo = both(h, x, w, b)[0][0]
    got = ref.layer_norm_backward(dn, xo, w, eps, "f32", dxo, keep / 0.75)
    # central differences with a step of 1e-6: off by some 1e-9 of the loss's size
    near = dict(rtol=1e-6, atol=1e-7)
    assert np.allclose(got["dx"][0], differences(lambda v: loss(h, v, w, b), x), **near)
    assert np.allclose(got["dh"][0], differences(lambda v: loss(v, x, w, b), h), **near)
    if weighted:
        assert np.allclose(got["dw"][0], differences(lambda v: loss(h, x, v, b), w), **near)
        assert np.allclose(got["db"][0], differences(lambda v: loss(h, x, w, v), b), **near)


def test_reference_balance_gradient_against_differences():
    g = np.random.default_rng(8)
    T, E, K = 5, 6, 2
    z = g.normal(size=(T, E))
    z[0, 2] = -np.inf
    valid = np.array([1, 1, 0, 1, 1])
    ids = np.stack([g.permutation(E)[:K] for _ in range(T)])
    ids[3, 1] = -1
    _, counts, _, probs, rate = ref.balance(z, ids, valid, 0.5, E)
    got = ref.balance_backward(probs, counts[:E], rate, 1.7, "f32")[0]
    some = np.isfinite(z)

    def loss(v):
        return 1.7 * ref.balance(np.where(some, v, -np.inf), ids, valid, 0.5, E)[0][0]
    assert np.allclose(got, differences(loss, np.where(some, z, 0.0)), rtol=1e-6, atol=1e-8)
    assert not got[2].any() and got[0, 2] == 0


def test_reference_embedding_gradient_is_the_transpose():
    g = np.random.default_rng(9)
    V, H, T, first = 7, 3, 40, 11
    ids = g.integers(5, 25, size=T)
    table, dout = g.normal(size=(V, H)), g.normal(size=(T, H))
    out = ref.embed(table, ids, first, 1.5, "f32")[0]
    dtable = ref.embed_backward(dout, ids, first, V, 1.5)[0]
    assert np.isclose((out * dout).sum(), (table * dtable).sum(), rtol=1e-12)
