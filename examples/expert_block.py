"""One expert-parallel block of a transformer, N ranks emulated on one GPU, with
the library's operators around its all-to-all:

    python examples/expert_block.py [--ranks 4] [--tokens 512] [--hidden 1024]
                                    [--experts 16] [--topk 4] [--low-precision]

Every rank holds its own tokens and 1/N of the experts. Forward, per rank:

    logits = n @ router            torch
    ids, weights                   expert_route
    slots sorted by expert         expert_sort, with a capacity: equal chunks
    rows of every expert           expert_dispatch (exact or FP8 payloads)
    rows to the experts' ranks     all_to_all_sim
    experts' products              torch, one batch over the local experts
    results back                   all_to_all_sim
    y = weighted sum of results    expert_combine
    norm, gate, residual, norm     residual_norm

and the gradients the same way back. In low precision the rows of both
exchanges are FP8 payloads: expert_dispatch quantizes a token once for all its
rows, and expert_combine reads the results' payload. (Rows that are not a whole
number of payload blocks are dispatched and combined exact, and all_to_all_sim
quantizes on its way.) The library runs on buffers that its caller provides, so a
block makes all of its own once.
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_collective_reduction_gb300 as pcr  # noqa: E402


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class _Rank:
    """What one rank keeps: its weights, and the buffers of a step."""

    def __init__(self, tokens, hidden, experts, local, topk, capacity, dtype, g):
        def normal(*shape, scale):
            return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)
        f32, i32 = torch.float32, torch.int32
        rows = experts * capacity
        self.router = normal(hidden, experts, scale=hidden ** -0.5)
        self.w_in = normal(local, hidden, 2 * hidden, scale=hidden ** -0.5)
        self.w_out = normal(local, 2 * hidden, hidden, scale=(2 * hidden) ** -0.5)
        self.gate = normal(hidden, scale=0.3)
        self.w_post = torch.ones(hidden, dtype=dtype, device="cuda")
        self.w_pre = torch.ones(hidden, dtype=dtype, device="cuda")
        self.ids, self.weights = _empty(tokens, topk, dtype=i32), _empty(tokens, topk, dtype=f32)
        self.slot_row, self.row_slot = _empty(tokens, topk, dtype=i32), _empty(rows, dtype=i32)
        self.offsets, self.counts = _empty(experts + 1, dtype=i32), _empty(experts, dtype=i32)
        # rows as sent, as received by the experts, and the results both ways
        self.sent, self.got, self.made, self.back = (
            _empty(rows, hidden, dtype=dtype) for _ in range(4))
        self.y, self.x_out, self.n_out, self.dx, self.dy, self.dn = (
            _empty(tokens, hidden, dtype=dtype) for _ in range(6))
        self.dweights, self.dlogits = _empty(tokens, topk, dtype=f32), _empty(tokens, experts,
                                                                              dtype=dtype)
        self.dgate, self.dw_post, self.dw_pre = (_empty(hidden, dtype=f32) for _ in range(3))


class ExpertBlock:
    """N emulated ranks of ``tokens`` tokens each; ``capacity`` rows per rank
    and expert (default: a quarter more than an even share)."""

    def __init__(self, ranks=4, tokens=512, hidden=1024, experts=16, topk=4, capacity=None,
                 dtype=torch.bfloat16, low_precision=False, seed=0):
        if experts % ranks:
            raise ValueError("the ranks share the experts evenly")
        self.ranks, self.tokens, self.hidden = ranks, tokens, hidden
        self.experts, self.local, self.topk = experts, experts // ranks, topk
        self.capacity = capacity or -(-tokens * topk * 5 // (experts * 4))
        self.block = pcr.BLOCK if low_precision else 0
        self.payloads = low_precision and hidden % pcr.BLOCK == 0
        self.scales = dict(res_scale=1.0, branch_scale=1.0, eps=1e-6)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rank = [_Rank(tokens, hidden, experts, self.local, topk, self.capacity, dtype, g)
                     for _ in range(ranks)]
        self.wire = {}
        if self.payloads:
            rows = experts * self.capacity
            for r in self.rank:
                # a rank's payload as sent and as received
                r.codes, r.codes_in = (_empty(rows, hidden, dtype=torch.uint8) for _ in range(2))
                r.scales, r.scales_in = (_empty(rows, pcr.nblocks(hidden), dtype=torch.float32)
                                         for _ in range(2))
        elif low_precision:
            n = experts * self.capacity * hidden
            chunk = self.local * self.capacity * hidden
            self.wire = dict(
                wire_codes=[_empty(n, dtype=torch.uint8) for _ in range(ranks)],
                wire_scales=[_empty(ranks * pcr.nblocks(chunk), dtype=torch.float32)
                             for _ in range(ranks)])

    def _exchange(self, src, dst, block):
        """Chunk j of every rank's rows to rank j."""
        pcr.all_to_all_sim([getattr(r, src).view(-1) for r in self.rank],
                           [getattr(r, dst).view(-1) for r in self.rank], block=block,
                           **(self.wire if block else {}))

    def _exchange_payloads(self):
        """The same for chunks of every rank's payload, which is there already: a copy
        does not look into what it moves, so four codes travel as one FP32 number."""
        for part in ("codes", "scales"):
            pcr.all_to_all_sim([getattr(r, part).view(-1).view(torch.float32) for r in self.rank],
                               [getattr(r, part + "_in").view(-1).view(torch.float32)
                                for r in self.rank], block=0)

    def _by_expert(self, rows):
        """Rows as received, [source rank, local expert, capacity] -> one batch
        of rows per local expert."""
        v = rows.view(self.ranks, self.local, self.capacity, self.hidden)
        return v.transpose(0, 1).reshape(self.local, -1, self.hidden)

    def _by_source(self, batch, out):
        v = batch.view(self.local, self.ranks, self.capacity, self.hidden)
        out.view(self.ranks, self.local, self.capacity, self.hidden).copy_(v.transpose(0, 1))

    @staticmethod
    def _experts(batch, w_in, w_out):
        return torch.bmm(torch.nn.functional.silu(torch.bmm(batch, w_in)), w_out)

    def forward(self, n, x):
        """n, x: the normed input and the residual of every rank, [T, H] each.
        Returns the ranks' (x_out, n_out)."""
        for r, nr in zip(self.rank, n):
            pcr.expert_route(nr @ r.router, r.ids, r.weights, renormalize=True)
            pcr.expert_sort(r.ids, self.experts, r.slot_row, r.row_slot, r.offsets, r.counts,
                            capacity=self.capacity)
            if self.payloads:
                pcr.expert_dispatch(nr, r.slot_row, r.row_slot, block=pcr.BLOCK, codes=r.codes,
                                    scales=r.scales)
            else:
                pcr.expert_dispatch(nr, r.slot_row, r.row_slot, r.sent)
        if self.payloads:
            self._exchange_payloads()
            for r in self.rank:
                pcr.lp_dequantize(r.codes_in.view(-1), r.scales_in.view(-1), r.got.view(-1))
        else:
            self._exchange("sent", "got", self.block)
        for r in self.rank:
            self._by_source(self._experts(self._by_expert(r.got), r.w_in, r.w_out), r.made)
        if self.payloads:
            for r in self.rank:
                pcr.lp_quantize(r.made.view(-1), r.codes.view(-1), r.scales.view(-1))
            self._exchange_payloads()
        else:
            self._exchange("made", "back", self.block)
        for r, xr in zip(self.rank, x):
            if self.payloads:
                pcr.expert_combine(r.slot_row, r.y, weights=r.weights, block=pcr.BLOCK,
                                   codes=r.codes_in, scales=r.scales_in)
            else:
                pcr.expert_combine(r.slot_row, r.y, r.back, weights=r.weights)
            pcr.residual_norm(r.y, xr, r.x_out, r.n_out, gate=r.gate, gate_kind="channel",
                              w_post=r.w_post, w_pre=r.w_pre, **self.scales)
        return [(r.x_out, r.n_out) for r in self.rank]

    def backward(self, n, dx_out, dn_out):
        """Gradients after forward(n, x) with exact payloads: per rank a dict of
        dx, dn and the weights' gradients. The gradients of rows travel exact."""
        for r, a, b in zip(self.rank, dx_out, dn_out):
            pcr.residual_norm_backward(a, b, r.y, r.x_out, r.dx, r.dy, gate=r.gate,
                                       gate_kind="channel", w_post=r.w_post, w_pre=r.w_pre,
                                       dgate=r.dgate, dw_post=r.dw_post, dw_pre=r.dw_pre,
                                       **self.scales)
            # the results combined are not wanted again: their gradient goes over them
            pcr.expert_combine_backward(r.dy, r.slot_row, r.row_slot, r.back, rows=r.back,
                                        weights=r.weights, dweights=r.dweights)
        self._exchange("back", "made", 0)
        out = []
        for r in self.rank:
            leaves = [t.detach().requires_grad_() for t in (self._by_expert(r.got), r.w_in,
                                                            r.w_out)]
            with torch.enable_grad():
                made = self._experts(*leaves)
            d_in, dw_in, dw_out = torch.autograd.grad(made, leaves, self._by_expert(r.made))
            self._by_source(d_in, r.got)
            out.append(dict(w_in=dw_in, w_out=dw_out))
        self._exchange("got", "sent", 0)
        for r, nr, o in zip(self.rank, n, out):
            pcr.expert_dispatch_backward(r.sent, r.slot_row, r.dn)
            logits = nr @ r.router
            pcr.expert_route_backward(logits, r.ids, r.weights, r.dweights, r.dlogits,
                                      renormalize=True)
            o.update(dx=r.dx, dn=r.dn + r.dlogits @ r.router.t(), router=nr.t() @ r.dlogits,
                     gate=r.dgate, w_post=r.dw_post, w_pre=r.dw_pre)
        return out


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("ranks", 4), ("tokens", 512), ("hidden", 1024), ("experts", 16),
                        ("topk", 4)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--low-precision", action="store_true", help="rows travel as FP8 payloads")
    a = p.parse_args()
    block = ExpertBlock(a.ranks, a.tokens, a.hidden, a.experts, a.topk,
                        low_precision=a.low_precision)
    make = lambda: [torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()  # noqa: E731
                    for _ in range(a.ranks)]
    n, x = make(), make()
    out = block.forward(n, x)
    kept = sum(int(r.counts.sum()) for r in block.rank)
    print("%d of %d slots within capacity; mean square of n_out %.4f" % (
        kept, a.ranks * a.tokens * a.topk,
        sum(float(v.float().square().mean()) for _, v in out) / a.ranks))
    if not a.low_precision:
        grads = block.backward(n, make(), make())
        print("gradient norms of rank 0: " + ", ".join(
            "%s %.3g" % (k, float(v.float().norm())) for k, v in grads[0].items()))


if __name__ == "__main__":
    main()
