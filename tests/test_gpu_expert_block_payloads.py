"""The low-precision expert block of examples/expert_block.py: its rows are
quantized by expert_dispatch and read as payloads by expert_combine."""
import pytest
import torch

import layers_ref as ref
import precision_collective_reduction_gb300 as pcr
from test_gpu_expert_block import load
from test_gpu_layers import DT, f64, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ranks,tokens,hidden,experts,topk,capacity", [
    (1, 1, 128, 4, 2, 4), (2, 37, 256, 6, 3, 5), (4, 100, 384, 8, 2, None)])
def test_payloads_from_dispatch_to_combine(monkeypatch, dt, ranks, tokens, hidden, experts, topk,
                                           capacity):
    m = load()
    blocks = []
    for name in ("expert_dispatch", "expert_combine"):
        def spy(*a, _call=getattr(pcr, name), _name=name, **kw):
            blocks.append((_name, kw.get("block", 0)))
            return _call(*a, **kw)
        monkeypatch.setattr(pcr, name, spy)
    b = m.ExpertBlock(ranks, tokens, hidden, experts, topk, capacity, dtype=DT[dt],
                      low_precision=True)
    g = torch.Generator(device="cuda").manual_seed(8)
    n, x = ([torch.randn(tokens, hidden, device="cuda", generator=g).to(DT[dt])
             for _ in range(ranks)] for _ in range(2))
    b.forward(n, x)
    assert blocks == [("expert_dispatch", 128)] * ranks + [("expert_combine", 128)] * ranks
    monkeypatch.undo()
    # what the experts got: the values that all_to_all_sim's own quantization of
    # the exact rows delivers
    rows = experts * b.capacity
    sent, got = ([torch.empty(rows, hidden, dtype=DT[dt], device="cuda") for _ in range(ranks)]
                 for _ in range(2))
    for r in range(ranks):
        me = b.rank[r]
        pcr.expert_dispatch(n[r], me.slot_row, me.row_slot, sent[r])
    chunk = b.local * b.capacity * hidden
    pcr.all_to_all_sim(
        [t.view(-1) for t in sent], [t.view(-1) for t in got], block=128,
        wire_codes=[torch.empty(rows * hidden, dtype=torch.uint8, device="cuda")
                    for _ in range(ranks)],
        wire_scales=[torch.empty(ranks * pcr.nblocks(chunk), device="cuda")
                     for _ in range(ranks)])
    for r in range(ranks):
        assert torch.equal(b.rank[r].got, got[r])
    # what came back: the results' payload, combined in FP32
    for r in range(ranks):
        me = b.rank[r]
        vals = torch.empty(rows, hidden, device="cuda")
        pcr.lp_dequantize(me.codes_in.view(-1), me.scales_in.view(-1), vals.view(-1))
        within(me.y, ref.combine(f64(vals), me.slot_row.cpu().numpy(), me.weights.cpu().numpy(),
                                 dt), "combined")


def test_rows_that_are_no_whole_payload_blocks():
    m = load()
    kw = dict(ranks=2, tokens=64, hidden=132, experts=4, topk=2, dtype=torch.float32)
    exact, low = m.ExpertBlock(**kw), m.ExpertBlock(low_precision=True, **kw)
    g = torch.Generator(device="cuda").manual_seed(9)
    n, x = ([torch.randn(64, 132, device="cuda", generator=g) for _ in range(2)] for _ in range(2))
    a, b = exact.forward(n, x), low.forward(n, x)
    for r in range(2):
        off = (a[r][0] - b[r][0]).norm() / (a[r][0] - x[r]).norm()
        assert 0 < float(off) < 0.1  # as with whole blocks
