"""The expert-parallel block of examples/expert_block.py: the operators, the
all-to-all and torch's products together, against a plain 64-bit form of the
whole block and its gradients by autograd."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def load():
    path = os.path.join(os.path.dirname(HERE), "examples", "expert_block.py")
    spec = importlib.util.spec_from_file_location("expert_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rms(v, w, eps):
    return v / (v.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w


def plain(block, n, x, leaves):
    """The block in 64 bits, given which rows the router and the capacity kept."""
    every = []
    for r in range(block.ranks):
        me = block.rank[r]
        z = n[r] @ leaves[r]["router"]
        there = me.ids >= 0
        at = me.ids.clamp(min=0).long()
        w = torch.softmax(z.gather(1, at).masked_fill(~there, -torch.inf), 1)
        y = torch.zeros_like(n[r])
        for k in range(block.topk):
            kept = me.slot_row[:, k] >= 0
            for e in range(block.experts):
                t = torch.nonzero(kept & (at[:, k] == e))[:, 0]
                if len(t):
                    owner = leaves[e // block.local]
                    h = torch.nn.functional.silu(n[r][t] @ owner["w_in"][e % block.local])
                    y = y.index_add(0, t, w[t, k, None] * (h @ owner["w_out"][e % block.local]))
        eps = block.scales["eps"]
        xo = x[r] + leaves[r]["gate"] * rms(y, leaves[r]["w_post"], eps)
        every.append((xo, rms(xo, leaves[r]["w_pre"], eps)))
    return every


@pytest.mark.parametrize("ranks,tokens,hidden,experts,topk,capacity", [
    (1, 1, 16, 4, 2, 4), (2, 37, 64, 6, 3, None), (4, 50, 132, 8, 2, 9)])
def test_block_against_64_bits(ranks, tokens, hidden, experts, topk, capacity):
    m = load()
    block = m.ExpertBlock(ranks, tokens, hidden, experts, topk, capacity, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(5)
    n, x, dxo, dno = ([torch.randn(tokens, hidden, device="cuda", generator=g)
                       for _ in range(ranks)] for _ in range(4))
    out = [(a.clone(), b.clone()) for a, b in block.forward(n, x)]
    names = ("router", "w_in", "w_out", "gate", "w_post", "w_pre")
    leaves = [{k: getattr(r, k).double().requires_grad_() for k in names} for r in block.rank]
    n64 = [v.double().requires_grad_() for v in n]
    x64 = [v.double().requires_grad_() for v in x]
    want = plain(block, n64, x64, leaves)
    got = block.backward(n, dxo, dno)
    torch.autograd.backward([v for pair in want for v in pair],
                            [d.double() for pair in zip(dxo, dno) for d in pair])
    # FP32 products of up to 264 terms in a chain of five: 5 * 264 * 2^-24 of the
    # sums' magnitudes, which are some ten times the results': 1e-3 of the norm
    # leaves room, a wrong term does not pass
    def near(a, b, what):
        b = b.detach()
        assert float((a.double() - b).norm()) <= 1e-3 * float(b.norm()) + 1e-9, what
    for r in range(ranks):
        near(out[r][0], want[r][0], "x_out")
        near(out[r][1], want[r][1], "n_out")
        near(got[r]["dn"], n64[r].grad, "dn")
        near(got[r]["dx"], x64[r].grad, "dx")
        for k in names:
            near(got[r][k], leaves[r][k].grad, k)


def test_block_with_fp8_payloads():
    # each of the two exchanges rounds a value by at most 2^-4 of itself (E4M3),
    # on average far less: the block's branch stays within 10% in norm
    m = load()
    kw = dict(ranks=4, tokens=256, hidden=512, experts=16, topk=4, dtype=torch.float32)
    exact, low = m.ExpertBlock(**kw), m.ExpertBlock(low_precision=True, **kw)
    g = torch.Generator(device="cuda").manual_seed(6)
    n, x = ([torch.randn(256, 512, device="cuda", generator=g) for _ in range(4)] for _ in range(2))
    a, b = exact.forward(n, x), low.forward(n, x)
    for r in range(4):
        assert torch.equal(exact.rank[r].ids, low.rank[r].ids)
        off = (a[r][0] - b[r][0]).norm() / (a[r][0] - x[r]).norm()
        assert 0 < float(off) < 0.1
