"""The operators around the collectives without a GPU: refusals of the C
entry points (every call fails its checks before any launch), sizes of the
workspaces, and the reference gradients of the GPU tests against differences."""
import numpy as np
import pytest

import layers_ref as ref
import precision_collective_reduction_gb300 as pcr
from precision_collective_reduction_gb300 import _binding as B
from precision_collective_reduction_gb300 import build as lib_build

OK, ARG, ALIGN, UNSUP, RANK = 0, 1, 2, 3, 4
A = 0x10000  # an aligned fake device address: never dereferenced in these calls
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return pcr.lib()


def test_route_refusals(L):
    f = L.expert_route
    assert f(A, 2, 4, 8, 2, 0, A, A, None) == ARG           # dtype
    assert f(A, 0, 4, 0, 1, 0, A, A, None) == ARG           # no experts
    assert f(A, 0, 4, 1025, 2, 0, A, A, None) == ARG
    assert f(A, 0, 4, 8, 0, 0, A, A, None) == ARG           # topk
    assert f(A, 0, 4, 8, 9, 0, A, A, None) == ARG           # more than experts
    assert f(A, 0, 4, 64, 33, 0, A, A, None) == ARG
    assert f(A, 0, 1 << 31, 8, 1, 0, A, A, None) == ARG     # slots past int32
    assert f(None, 0, 0, 8, 2, 0, None, None, None) == OK   # no tokens
    assert f(None, 0, 4, 8, 2, 0, A, A, None) == ARG
    assert f(A, 0, 4, 8, 2, 0, A + 4, None, None) == ARG    # NULL before alignment
    assert f(A, 0, 4, 8, 2, 0, A, A + 4, None) == ALIGN
    g = L.expert_route_backward
    assert g(A, 5, 4, 8, 2, 0, A, A, A, A, None) == ARG
    assert g(None, 0, 4, 8, 2, 0, A, A, A, A, None) == ARG  # the softmax needs the logits
    assert g(A, 0, 4, 8, 2, 1, A, A, None, A, None) == ARG
    assert g(A, 0, 4, 8, 2, 1, A, A, A, A + 8, None) == ALIGN
    assert g(None, 1, 0, 8, 2, 0, None, None, None, None, None) == OK


def test_sort_refusals(L):
    f = L.expert_sort
    assert f(A, 8, 0, 0, A, A, A, A, None, 0, None) == ARG
    assert f(A, 8, 1025, 0, A, A, A, A, None, 0, None) == ARG
    assert f(A, 1 << 31, 8, 0, A, A, A, A, A, 1 << 40, None) == ARG
    assert f(A, 8, 8, 1 << 29, A, A, A, A, None, 0, None) == ARG   # rows past int32
    need = L.expert_sort_workspace_bytes(5000, 16)
    assert need > 0 and L.expert_sort_workspace_bytes(2048, 16) == 0
    assert f(A, 5000, 16, 0, A, A, A, A, A, need - 1, None) == ARG
    assert f(A, 5000, 16, 0, A, A, A, A, None, need, None) == ARG
    assert f(A, 8, 8, 0, None, A, A, A, None, 0, None) == ARG
    assert f(A, 8, 8, 0, A, A, None, A, None, 0, None) == ARG
    assert f(A, 8, 8, 0, A, A + 4, A, A, None, 0, None) == ALIGN
    # the largest sort stays within its chunks
    assert L.expert_sort_workspace_bytes((1 << 31) - 1, 1024) <= 128 * 1024 * 4
    assert L.expert_sort_workspace_bytes(5000, 0) == 0


def test_rows_refusals(L):
    d, c, b = L.expert_dispatch, L.expert_combine, L.expert_combine_backward
    assert d(A, 4, 2, 8, 64, 3, 0, A, A, A, None, None, None) == ARG       # dtype
    assert d(A, 4, 0, 8, 64, 0, 0, A, A, A, None, None, None) == ARG       # topk
    assert d(A, 4, 33, 8, 64, 0, 0, A, A, A, None, None, None) == ARG
    assert d(A, 1 << 30, 2, 8, 64, 0, 0, A, A, A, None, None, None) == ARG
    assert d(A, 4, 2, 1 << 31, 64, 0, 0, A, A, A, None, None, None) == ARG
    assert d(A, 1 << 20, 2, 8, 1 << 20, 0, 0, A, A, A, None, None, None) == ARG  # grid
    assert d(A, 4, 2, 8, 64, 0, 64, A, A, A, A, A, None) == UNSUP          # block
    assert d(A, 4, 2, 8, 64, 0, 128, A, A, A, None, A, None) == ARG
    assert d(A, 4, 2, 8, 64, 0, 0, A, A, None, A, A, None) == ARG
    assert d(A, 4, 2, 8, 64, 0, 0, A, A + 4, A, None, None, None) == ALIGN
    assert d(None, 0, 2, 0, 64, 0, 0, None, None, None, None, None, None) == OK
    assert d(None, 4, 2, 8, 0, 0, 0, None, None, None, None, None, None) == OK
    assert c(A, None, None, 4, 2, 8, 64, 7, 0, A, A, A, None) == ARG
    assert c(A, None, None, 4, 2, 8, 64, 0, 32, A, A, A, None) == UNSUP
    assert c(None, None, None, 4, 2, 8, 64, 0, 0, A, A, A, None) == ARG
    assert c(A, None, A, 4, 2, 8, 64, 0, 128, A, A, A, None) == ARG
    assert c(A, None, None, 4, 2, 8, 64, 0, 0, None, A, A, None) == ARG
    assert c(A, None, None, 4, 2, 8, 64, 0, 0, A, A + 4, A, None) == ALIGN
    assert c(None, None, None, 0, 2, 8, 64, 0, 0, None, None, None, None) == OK
    assert b(A, A, 4, 2, 8, 64, 4, A, A, A, A, A, None) == ARG
    assert b(A, None, 4, 2, 8, 64, 0, A, A, A, A, A, None) == ARG          # dweights need rows
    assert b(A, A, 4, 2, 8, 64, 0, A, None, A, A, A, None) == ARG
    assert b(A, A, 4, 2, 8, 64, 0, A, A, A, A + 2, A, None) == ALIGN
    assert b(None, None, 0, 2, 0, 64, 0, None, None, None, None, None, None) == OK


def test_norm_refusals(L):
    two, f = B.ptr_array([A, A]), L.residual_norm

    def call(h=two, n=2, x=A, gate=None, kind=0, post=A, pre=A, eps=1e-5, T=4, H=64, dt=0, xo=A,
             no=A, hs=None):
        return f(h, n, x, gate, kind, post, pre, 1.0, 1.0, eps, T, H, dt, xo, no, hs, None)
    assert call(dt=2) == ARG and call(kind=4) == ARG and call(kind=-1) == ARG
    for eps in (0.0, -1.0, NAN, INF):
        assert call(eps=eps) == ARG
    assert call(n=0) == ARG and call(n=17) == ARG
    assert call(H=16385) == UNSUP and call(T=1 << 31) == ARG
    assert call(T=0, h=None, x=None, xo=None) == OK and call(H=0, h=None) == OK
    assert call(h=None) == ARG and call(h=B.ptr_array([A, None])) == RANK
    assert call(x=None) == ARG and call(xo=None) == ARG
    assert call(kind=1) == ARG and call(no=None) == ARG       # gate, n_out missing
    assert call(post=A + 2) == ALIGN and call(h=B.ptr_array([A, A + 8])) == ALIGN
    assert call(hs=A + 4) == ALIGN
    need = L.residual_norm_backward_workspace_bytes(4, 64, 0)
    assert need > 0 and L.residual_norm_backward_workspace_bytes(0, 64, 0) == 0
    assert L.residual_norm_backward_workspace_bytes(4, 16385, 0) == 0

    def back(dxo=A, dn=A, h=A, xo=A, gate=None, kind=0, post=A, pre=A, eps=1e-5, T=4, H=64, dt=0,
             dx=A, dh=A, dg=None, dq=A, dp=A, ws=A, n=need):
        return L.residual_norm_backward(dxo, dn, h, xo, gate, kind, post, pre, 1.0, 1.0, eps, T,
                                        H, dt, dx, dh, dg, dq, dp, ws, n, None)
    assert back(dt=2) == ARG and back(eps=0.0) == ARG and back(kind=9) == ARG
    assert back(H=20000) == UNSUP
    assert back(n=need - 1) == ARG and back(ws=None) == ARG
    assert back(dn=None) == ARG and back(dxo=None, pre=None) == ARG
    assert back(h=None) == ARG and back(xo=None) == ARG and back(dx=None) == ARG
    assert back(kind=2) == ARG and back(dh=A + 8) == ALIGN and back(dp=A + 4) == ALIGN
    assert back(H=0, h=None) == OK


@pytest.mark.parametrize("kind", [None, "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_reference_gradient_against_differences(kind, post, pre):
    g = np.random.default_rng([3, post, pre, ord((kind or "n")[0])])
    T, H = 3, 7
    th = dict(h=g.normal(size=(T, H)), x=g.normal(size=(T, H)))
    if kind:
        th["gate"] = g.normal(size={"channel": (H,), "token": (T,), "full": (T, H)}[kind])
    if post:
        th["w_post"] = 1 + g.normal(size=H)
    if pre:
        th["w_pre"] = 1 + g.normal(size=H)
    dx, dn = g.normal(size=(T, H)), g.normal(size=(T, H))
    a, b, eps = 0.9, 0.7, 1e-3

    def loss(v):
        xo, n = ref.forward(v["h"], v["x"], v.get("gate"), kind, v.get("w_post"), v.get("w_pre"),
                            a, b, eps)
        return (xo * dx).sum() + ((n * dn).sum() if pre else 0.0)
    xo = ref.forward(th["h"], th["x"], th.get("gate"), kind, th.get("w_post"), th.get("w_pre"), a,
                     b, eps)[0]
    got = ref.residual_norm_backward(dx, dn if pre else None, th["h"], xo, th.get("gate"), kind,
                                     th.get("w_post"), th.get("w_pre"), a, b, eps, "f32")
    for name, v in th.items():
        want = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            up, dn_ = dict(th), dict(th)
            up[name], dn_[name] = v.copy(), v.copy()
            up[name][i] += 1e-5
            dn_[name][i] -= 1e-5
            want[i] = (loss(up) - loss(dn_)) / 2e-5
        # central differences: truncation about 1e-10, rounding 1e-16 / 1e-5
        assert np.allclose(got["d" + name][0], want, rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_router_gradient_against_differences(renormalize):
    g = np.random.default_rng(5)
    z, K = g.normal(size=(4, 6)), 3
    z[1, 2] = -np.inf
    z[3] = -np.inf
    dw = g.normal(size=(4, K))
    ids, w, _ = ref.route(z, K, renormalize)
    assert (ids[3] == -1).all() and 2 not in ids[1]
    got = ref.route_backward(z, ids, w, dw, renormalize)[0]
    for i in np.ndindex(z.shape):
        if not np.isfinite(z[i]):
            assert got[i] == 0
            continue
        d = []
        for s in (1e-6, -1e-6):
            v = z.copy()
            v[i] += s
            i2, w2, _ = ref.route(v, K, renormalize)
            assert (i2 == ids).all()
            d.append((w2 * dw).sum())
        assert abs((d[0] - d[1]) / 2e-6 - got[i]) < 1e-8
