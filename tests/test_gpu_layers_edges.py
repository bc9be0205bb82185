"""Corners of the operators around the collectives."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import precision_collective_reduction_gb300 as pcr
from test_gpu_layers import dev, f64, lib, norm_case, within  # noqa: F401

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
