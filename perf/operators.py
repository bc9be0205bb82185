"""The operators around the collectives of an expert-parallel transformer layer, as measurable cases: the router, tokens
sorted by expert and sent out as rows (exact or as FP8 payloads), the weighted way back with its gradient, and the norms
before and after a block fused with its gate and residual scale, with their gradients.

`prepare` makes the inputs, and the result buffers that a program keeps; `run` makes one pass, in plain torch operations in
32 bits or (with `own`) through the package; `exact` gives the results from the definitions in 64 bits."""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
BLOCK = 128      # elements per scale of an FP8 payload
EPS = 1e-5       # of the norms
RES_SCALE, BRANCH_SCALE = 0.9, 0.7


def listed():
    return [
        # the router at one decode step of a batch of 32, latency
        dict(name="route decode", op="route", tokens=32, experts=64, topk=8, dtype="bf16", renorm=True, masked=False, train=False),
        # the router of a training step, forward and backward, with experts switched off for some tokens
        dict(name="route train", op="route", tokens=32768, experts=256, topk=8, dtype="f32", renorm=False, masked=True, train=True),
        # a decode batch of 32 x hidden 8192 sorted to its experts, latency
        dict(name="dispatch decode", op="dispatch", tokens=32, topk=8, experts=64, hidden=8192, dtype="bf16", block=0, capacity=0, dropped=0.0),
        # prefill: rows laid out by expert for the experts' products, some slots without an expert
        dict(name="dispatch prefill", op="dispatch", tokens=8192, topk=4, experts=128, hidden=8192, dtype="bf16", block=0, capacity=0, dropped=0.05),
        # prefill in equal chunks for an all-to-all (rows of a full expert fall out), as FP8 payloads
        dict(name="dispatch prefill fp8", op="dispatch", tokens=8192, topk=4, experts=64, hidden=8192, dtype="bf16", block=128, capacity=640, dropped=0.0),
        # the experts' rows of a decode step back to their tokens, latency
        dict(name="combine decode", op="combine", tokens=32, topk=8, experts=64, hidden=8192, dtype="bf16", block=0, dropped=0.0),
        # the same for a prefill
        dict(name="combine prefill", op="combine", tokens=8192, topk=4, experts=128, hidden=8192, dtype="bf16", block=0, dropped=0.05),
        # gradients of rows and weights of a training step, a ragged batch of odd hidden size
        dict(name="combine gradient", op="combine_grad", tokens=4001, topk=8, experts=96, hidden=4100, dtype="f32", dropped=0.02),
        # end of a block at decode: the partial products of 8 ranks summed, normed, added, normed; latency
        dict(name="norm decode", op="norm", tokens=32, hidden=8192, dtype="bf16", ranks=8, gate="none", post=True, pre=True),
        # the same for a long prefill whose sum is there already, with a gate for each channel
        dict(name="norm prefill", op="norm", tokens=16384, hidden=8192, dtype="bf16", ranks=1, gate="channel", post=True, pre=True),
        # its gradients in a training step
        dict(name="norm gradient", op="norm_grad", tokens=8192, hidden=8192, dtype="bf16", gate="channel", post=True, pre=True),
        # gradients of a small odd-sized block in FP32 with one gate a token
        dict(name="norm gradient odd", op="norm_grad", tokens=1001, hidden=2051, dtype="f32", gate="token", post=True, pre=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "dispatch", "combine", "combine_grad", "norm", "norm_grad"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384])
        return dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, topk=rng.randint(1, min(10, experts)), dtype=dtype,
                    renorm=rng.random() < 0.5, masked=rng.random() < 0.5, train=rng.random() < 0.5)
    hidden = _log(rng, 96, 12288)
    if rng.random() < 0.75:
        hidden = max(64, hidden // 64 * 64)
    if op in ("norm", "norm_grad"):
        tokens = max(1, min(_log(rng, 1, 16384), (16384 if op == "norm" else 8192) * 8192 * 2 // (hidden * ES[dtype])))
        gate = rng.choice(["none", "channel", "token", "full"])
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        c = dict(op=op, tokens=tokens, hidden=hidden, dtype=dtype, gate=gate, post=post, pre=pre)
        if op == "norm":
            c["ranks"] = rng.choice([1, 1, 2, 4, 8])
            c["tokens"] = max(1, min(tokens, 16384 * 8192 * 4 // ((c["ranks"] + 3) * hidden * ES[dtype])))
        return c
    topk, experts = rng.randint(1, 8), rng.choice([8, 16, 60, 64, 128, 256])
    tokens = max(1, min(_log(rng, 1, 16384), 8192 * 4 * 8192 * 2 // (hidden * ES[dtype] * topk * (2 if op == "combine_grad" else 1))))
    c = dict(op=op, tokens=tokens, topk=topk, experts=experts, hidden=hidden, dtype=dtype, dropped=rng.choice([0.0, 0.03]))
    if op != "combine_grad":
        c["block"] = rng.choice([0, 0, 128])
    if op == "dispatch":
        room = max(1, -(-tokens * topk * 5 // (experts * 4)))
        c["capacity"] = rng.choice([0, 0, room if room * experts <= 2 * tokens * topk else 0])
    return c


# -- inputs ---------------------------------------------------------------------------------------------------------

def _blocks(n):
    return -(-n // BLOCK)


def _choices(c, g):
    """Experts of every slot: K different ones a token, some experts more popular, some slots without one (-1)."""
    T, K, E = c["tokens"], c["topk"], c["experts"]
    pull = torch.randn(E, device="cuda", generator=g) * 0.7
    z = pull - torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=g).clamp_(1e-9, 1 - 1e-7)))
    ids = z.topk(K, dim=1).indices.to(torch.int32)
    if c["dropped"]:
        ids[torch.rand(T, K, device="cuda", generator=g) < c["dropped"]] = -1
    return ids


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    T, dt = c["tokens"], DT[c["dtype"]]
    s = dict(c=c)

    def buf(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    if c["op"] == "route":
        E, K = c["experts"], c["topk"]
        z = torch.randn(T, E, device="cuda", generator=g) * 1.5 + torch.randn(E, device="cuda", generator=g)
        if c["masked"]:  # experts switched off for a token, and a few tokens with none left
            z[torch.rand(T, E, device="cuda", generator=g) < 0.2] = -math.inf
            z[torch.rand(T, device="cuda", generator=g) < 0.01] = -math.inf
        s |= dict(logits=z.to(dt), ids=buf(T, K, dtype=torch.int32), weights=buf(T, K, dtype=torch.float32))
        if c["train"]:
            s |= dict(dweights=_normal(g, T, K), dlogits=buf(T, E))
        return s
    H = c["hidden"]
    if c["op"] in ("dispatch", "combine", "combine_grad"):
        K, E = c["topk"], c["experts"]
        ids = _choices(c, g)
        if c["op"] == "dispatch":
            R = E * c["capacity"] or T * K
            spread = torch.exp(torch.randn(T, 1, device="cuda", generator=g))
            s |= dict(ids=ids, x=(torch.randn(T, H, device="cuda", generator=g) * spread).to(dt),
                      slot_row=buf(T, K, dtype=torch.int32), row_slot=buf(R, dtype=torch.int32),
                      offsets=buf(E + 1, dtype=torch.int32), counts=buf(E, dtype=torch.int32))
            if c["block"]:
                s |= dict(codes=buf(R, H, dtype=torch.uint8), scales=buf(R, _blocks(H), dtype=torch.float32))
            else:
                s |= dict(out=buf(R, H))
            return s
        R = T * K
        s["slot_row"], s["row_slot"] = _sorted(ids, E, 0)[:2]
        s["weights"] = torch.rand(T, K, device="cuda", generator=g) / K
        rows = _normal(g, R, H, dtype=dt)
        if c["op"] == "combine":
            s["out"] = buf(T, H)
            if c["block"]:
                s["codes"], s["scales"] = _payload(rows.float())
            else:
                s["rows"] = rows
        else:
            s |= dict(rows=rows, dout=_normal(g, T, H, dtype=dt, scale=0.05), drows=buf(R, H), dweights=buf(T, K, dtype=torch.float32))
        return s
    if c["gate"] == "channel":
        s["gate"] = _normal(g, H, dtype=dt, scale=0.3)
    elif c["gate"] == "token":
        s["gate"] = torch.rand(T, device="cuda", generator=g).to(dt)
    elif c["gate"] == "full":
        s["gate"] = torch.rand(T, H, device="cuda", generator=g).to(dt)
    else:
        s["gate"] = None
    s["w_post"] = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(dt) if c["post"] else None
    s["w_pre"] = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(dt) if c["pre"] else None
    loud = torch.exp(1.5 * torch.randn(H, device="cuda", generator=g).clamp_(-1, 2))  # channels of a residual stream differ
    if c["op"] == "norm":
        N = c["ranks"]
        s |= dict(h=[_normal(g, T, H, dtype=dt, scale=2 / math.sqrt(N)) for _ in range(N)],
                  x=(torch.randn(T, H, device="cuda", generator=g) * loud).to(dt),
                  x_out=buf(T, H), n_out=buf(T, H) if c["pre"] else None, h_sum=buf(T, H) if N > 1 else None)
    else:
        s |= dict(h=_normal(g, T, H, dtype=dt, scale=2.0), x_out=(torch.randn(T, H, device="cuda", generator=g) * loud).to(dt),
                  dx_out=_normal(g, T, H, dtype=dt, scale=0.05), dn_out=_normal(g, T, H, dtype=dt, scale=0.1) if c["pre"] else None,
                  dx=buf(T, H), dh=buf(T, H))
        s["dw_post"] = buf(H, dtype=torch.float32) if c["post"] else None
        s["dw_pre"] = buf(H, dtype=torch.float32) if c["pre"] else None
        s["dgate"] = {"none": None, "channel": buf(H, dtype=torch.float32) if c["gate"] == "channel" else None,
                      "token": buf(T, dtype=torch.float32) if c["gate"] == "token" else None,
                      "full": buf(T, H) if c["gate"] == "full" else None}[c["gate"]]
    return s


# -- one pass -------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    return (_own if own else _plain)(s["c"], s)


def _own(c, s):
    import precision_collective_reduction_gb300 as pcr
    if c["op"] == "route":
        pcr.expert_route(s["logits"], s["ids"], s["weights"], renormalize=c["renorm"])
        if not c["train"]:
            return [s["ids"], s["weights"]]
        pcr.expert_route_backward(s["logits"], s["ids"], s["weights"], s["dweights"], s["dlogits"], renormalize=c["renorm"])
        return [s["ids"], s["weights"], s["dlogits"]]
    if c["op"] == "dispatch":
        pcr.expert_sort(s["ids"], c["experts"], s["slot_row"], s["row_slot"], s["offsets"], s["counts"], capacity=c["capacity"])
        maps = [s["slot_row"], s["row_slot"], s["offsets"], s["counts"]]
        if c["block"]:
            pcr.expert_dispatch(s["x"], s["slot_row"], s["row_slot"], block=BLOCK, codes=s["codes"], scales=s["scales"])
            return maps + [s["codes"].view(torch.float8_e4m3fn), s["scales"]]
        pcr.expert_dispatch(s["x"], s["slot_row"], s["row_slot"], s["out"])
        return maps + [s["out"]]
    if c["op"] == "combine":
        if c["block"]:
            pcr.expert_combine(s["slot_row"], s["out"], weights=s["weights"], block=BLOCK, codes=s["codes"], scales=s["scales"])
        else:
            pcr.expert_combine(s["slot_row"], s["out"], s["rows"], weights=s["weights"])
        return [s["out"]]
    if c["op"] == "combine_grad":
        pcr.expert_combine_backward(s["dout"], s["slot_row"], s["row_slot"], s["drows"], rows=s["rows"], weights=s["weights"], dweights=s["dweights"])
        return [s["drows"], s["dweights"]]
    kw = dict(gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], res_scale=RES_SCALE, branch_scale=BRANCH_SCALE, eps=EPS)
    if c["op"] == "norm":
        pcr.residual_norm(s["h"], s["x"], s["x_out"], s["n_out"], h_sum=s["h_sum"], **kw)
        return [s["x_out"], s["n_out"], s["h_sum"]]
    pcr.residual_norm_backward(s["dx_out"], s["dn_out"], s["h"], s["x_out"], s["dx"], s["dh"], dgate=s["dgate"], dw_post=s["dw_post"],
                               dw_pre=s["dw_pre"], **kw)
    return [s["dx"], s["dh"], s["dgate"], s["dw_post"], s["dw_pre"]]


def _sorted(ids, E, capacity):
    """slot_row, row_slot, offsets, counts of a stable sort of the slots by expert."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, order = torch.sort(key, stable=True)
    each = (key[None, :] == torch.arange(E, device=key.device)[:, None]).sum(1)
    first = torch.cat([each.new_zeros(1), each.cumsum(0)])
    rank = torch.arange(n, device=key.device) - first[key]
    row = first[key] + rank
    kept = key < E
    rows = n
    if capacity:
        rows, each = E * capacity, each.clamp(max=capacity)
        row, kept = key * capacity + rank, kept & (rank < capacity)
        first = torch.arange(E + 1, device=key.device) * capacity
    slot_row = torch.empty(n, dtype=torch.long, device=key.device)
    slot_row[order] = torch.where(kept, row, -1)
    row_slot = torch.full((rows + 1,), -1, dtype=torch.long, device=key.device)
    row_slot[torch.where(kept, row, rows)] = order
    row_slot = row_slot[:rows]
    return slot_row.view(ids.shape).int(), row_slot.int(), first.int(), each.int()


def _payload(x):
    """FP8 codes and scales of every row's blocks of 128."""
    R, H = x.shape
    nb = _blocks(H)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - H)).view(R, nb, BLOCK)
    a = v.abs().amax(2)
    inv = 448.0 / a
    fine = torch.isfinite(inv)
    inv = torch.where(fine, inv, 0.0)
    codes = (v * inv[..., None]).to(torch.float8_e4m3fn).view(R, nb * BLOCK)[:, :H]
    return codes.contiguous().view(torch.uint8), torch.where(fine, a / 448.0, 0.0)


def _values(codes, scales):
    x = codes.view(torch.float8_e4m3fn).float()
    return x * scales.repeat_interleave(BLOCK, 1)[:, : x.shape[1]]


def _plain(c, s):
    dt = DT[c["dtype"]]
    if c["op"] == "route":
        K = c["topk"]
        z = s["logits"].float()
        top, ids = torch.sort(z, dim=1, descending=True, stable=True)
        top, ids = top[:, :K], ids[:, :K]
        there = top > -math.inf
        m = torch.where(there[:, :1], top[:, :1], 0.0)
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        chosen = torch.exp(top - m)
        over = chosen.sum(1, keepdim=True) if c["renorm"] else total
        w = torch.where(there, chosen / over, 0.0)
        ids = torch.where(there, ids, -1).int()
        if not c["train"]:
            return [ids, w]
        dw = s["dweights"]
        mean = (w * dw).sum(1, keepdim=True)
        at = torch.where(there, ids, 0).long()
        back = torch.zeros_like(z).scatter_add_(1, at, torch.where(there, w * (dw - mean if c["renorm"] else dw), 0.0))
        if not c["renorm"]:
            back -= torch.where(total > 0, e / total, 0.0) * mean
        return [ids, w, back.to(dt)]
    if c["op"] == "dispatch":
        maps = _sorted(s["ids"], c["experts"], c["capacity"])
        used = (maps[1] >= 0)[:, None]
        x = torch.where(used, s["x"].float()[maps[1].clamp(min=0).long() // c["topk"]], 0.0)
        if not c["block"]:
            return [*maps, x.to(dt)]
        codes, scales = _payload(x)
        return [*maps, codes.view(torch.float8_e4m3fn), scales]
    if c["op"] in ("combine", "combine_grad"):
        row = s["slot_row"].clamp(min=0).long()
        there = (s["slot_row"] >= 0)[..., None]
        w = s["weights"][..., None]
        if c["op"] == "combine":
            rows = _values(s["codes"], s["scales"]) if c["block"] else s["rows"].float()
            return [torch.where(there, rows[row] * w, 0.0).sum(1).to(dt)]
        dy = s["dout"].float()
        dw = torch.where(there, s["rows"].float()[row] * dy[:, None, :], 0.0).sum(2)
        slot = s["row_slot"].clamp(min=0).long()
        drows = dy[slot // c["topk"]] * s["weights"].reshape(-1)[slot][:, None]
        return [torch.where((s["row_slot"] >= 0)[:, None], drows, 0.0).to(dt), dw]
    gate = 1.0 if s["gate"] is None else s["gate"].float()[:, None] if c["gate"] == "token" else s["gate"].float()
    if c["op"] == "norm":
        h = torch.stack([p.float() for p in s["h"]]).sum(0)
        u = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w_post"].float() if c["post"] else h
        x = RES_SCALE * s["x"].float() + BRANCH_SCALE * gate * u
        n = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["w_pre"].float()).to(dt) if c["pre"] else None
        return [x.to(dt), n, h.to(dt) if c["ranks"] > 1 else None]
    h, x, d = s["h"].float(), s["x_out"].float(), s["dx_out"].float()
    dw_pre = dw_post = dgate = None
    if c["pre"]:
        dn = s["dn_out"].float()
        r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        xh, q = x * r, dn * s["w_pre"].float()
        dw_pre = (dn * xh).sum(0)
        d = d + r * (q - xh * (q * xh).mean(1, keepdim=True))
    u, hh = h, h
    if c["post"]:
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        hh = h * r
        u = hh * s["w_post"].float()
    if c["gate"] != "none":
        dgate = BRANCH_SCALE * u * d
        dgate = dgate.sum(0) if c["gate"] == "channel" else dgate.sum(1) if c["gate"] == "token" else dgate.to(dt)
    du = BRANCH_SCALE * gate * d
    if c["post"]:
        dw_post = (du * hh).sum(0)
        q = du * s["w_post"].float()
        du = r * (q - hh * (q * hh).mean(1, keepdim=True))
    return [(RES_SCALE * d).to(dt), du.to(dt), dgate, dw_post, dw_pre]


# -- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    c, es = case, ES[case["dtype"]]
    T = c["tokens"]
    if c["op"] == "route":
        E, K = c["experts"], c["topk"]
        n = T * E * es + 8 * T * K + ((T * E * es + 4 * T * K) if c["train"] else 0)
        return {"bytes": n, "flops": (8 if c["train"] else 4) * T * E}
    H = c["hidden"]
    row = H + 4 * _blocks(H) if c.get("block") else H * es
    if c["op"] == "dispatch":
        S = T * c["topk"]
        R = c["experts"] * c["capacity"] or S
        return {"bytes": 4 * S + 4 * S + 4 * R + 8 * c["experts"] + T * H * es + R * row, "flops": 3 * T * H if c["block"] else T * c["topk"]}
    if c["op"] in ("combine", "combine_grad"):
        S = T * c["topk"]
        used = int(S * (1 - c["dropped"]))
        if c["op"] == "combine":
            return {"bytes": 8 * S + used * row + T * H * es, "flops": 2 * used * H}
        return {"bytes": 16 * S + used * row + T * H * es + S * H * es, "flops": 3 * used * H}
    gate = {"none": 0, "channel": H, "token": T, "full": T * H}[c["gate"]] * es
    w = H * es * (c["post"] + c["pre"])
    if c["op"] == "norm":
        n = (c["ranks"] + 2 + c["pre"] + (c["ranks"] > 1)) * T * H * es + gate + w
        return {"bytes": n, "flops": (c["ranks"] + 8) * T * H}
    dgate = {"none": 0, "channel": 4 * H, "token": 4 * T, "full": T * H * es}[c["gate"]]
    return {"bytes": (5 + c["pre"]) * T * H * es + gate + dgate + w + 4 * H * (c["post"] + c["pre"]), "flops": 24 * T * H}


# -- the definitions in 64 bits -------------------------------------------------------------------------------------

def _rms(v, w):
    return v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w


def exact(case, seed):
    c, s = case, prepare(case, seed)
    T = c["tokens"]
    if c["op"] == "route":
        K = c["topk"]
        z = s["logits"].double().cpu().numpy()
        ids = np.argsort(-z, axis=1, kind="stable")[:, :K]
        there = np.take_along_axis(z, ids, 1) > -np.inf
        leaf = torch.from_numpy(z).requires_grad_()
        some = torch.from_numpy(there[:, :1])
        p = torch.softmax(torch.where(some, leaf, 0.0), 1)
        w = torch.where(torch.from_numpy(there), p.gather(1, torch.from_numpy(ids)), 0.0)
        if c["renorm"]:
            w = w / torch.where(some, w.sum(1, keepdim=True), 1.0)
        out = [torch.from_numpy(np.where(there, ids, -1).astype(np.int32)), w.detach()]
        if c["train"]:
            w.backward(s["dweights"].double().cpu())
            out.append(leaf.grad)
        return out
    H = c["hidden"]
    if c["op"] == "dispatch":
        K, E, C = c["topk"], c["experts"], c["capacity"]
        ids = s["ids"].cpu().numpy().reshape(-1)
        groups = [np.nonzero(ids == e)[0] for e in range(E)]
        if C:
            groups = [v[:C] for v in groups]
        counts = np.array([len(v) for v in groups], dtype=np.int32)
        offsets = np.arange(E + 1) * C if C else np.concatenate([[0], np.cumsum(counts)])
        R = E * C or T * K
        row_slot, slot_row = np.full(R, -1, np.int32), np.full(T * K, -1, np.int32)
        for e, v in enumerate(groups):
            row_slot[offsets[e]: offsets[e] + len(v)] = v
            slot_row[v] = offsets[e] + np.arange(len(v))
        out = [slot_row.reshape(T, K), row_slot, offsets.astype(np.int32), counts]
        token = torch.from_numpy(row_slot).cuda().long()
        x = torch.zeros(R, H, dtype=torch.float64, device="cuda")
        x[token >= 0] = s["x"].double()[token[token >= 0] // K]
        if not c["block"]:
            return out + [x]
        scale = torch.stack([b.abs().amax(1) for b in x.split(BLOCK, 1)], 1) / 448
        return out + [None, scale]
    if c["op"] in ("combine", "combine_grad"):
        rows = s["rows"].double() if "rows" in s else (s["codes"].view(torch.float8_e4m3fn).double()
                                                       * s["scales"].double().repeat_interleave(BLOCK, 1)[:, :H])
        w, y, got = s["weights"].double(), torch.zeros(T, H, dtype=torch.float64, device="cuda"), s["slot_row"].long()
        if c["op"] == "combine":
            for k in range(c["topk"]):
                t = torch.nonzero(got[:, k] >= 0)[:, 0]
                y[t] += w[t, k, None] * rows[got[t, k]]
            return [y]
        drows, dw, dy = torch.zeros_like(rows), torch.zeros_like(w), s["dout"].double()
        for k in range(c["topk"]):
            t = torch.nonzero(got[:, k] >= 0)[:, 0]
            dw[t, k] = torch.linalg.vecdot(rows[got[t, k]], dy[t])
            drows[got[t, k]] = w[t, k, None] * dy[t]
        return [drows, dw]
    if T * H > 40_000_000 and c["op"] == "norm_grad":  # autograd keeps many copies: let it go in parts
        parts = 4
    else:
        parts = 1
    leaf = {k: s[k].double().requires_grad_() for k in ("gate", "w_post", "w_pre") if s[k] is not None}
    per_row = c["gate"] in ("token", "full")

    def branch(h, lo, hi):
        u = _rms(h, leaf["w_post"]) if c["post"] else h
        if c["gate"] == "none":
            return u
        gate = leaf["gate"][lo:hi] if per_row else leaf["gate"]
        return u * (gate[:, None] if c["gate"] == "token" else gate)
    if c["op"] == "norm":
        with torch.no_grad():
            h = torch.zeros(T, H, dtype=torch.float64, device="cuda")
            for p in s["h"]:
                h += p.double()
            x = RES_SCALE * s["x"].double() + BRANCH_SCALE * branch(h, 0, T)
            return [x, _rms(x, leaf["w_pre"]) if c["pre"] else None, h if c["ranks"] > 1 else None]
    dx, dh = [], []
    step = -(-T // parts)
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        xo = s["x_out"][lo:hi].double().requires_grad_()
        h = s["h"][lo:hi].double().requires_grad_()
        d = s["dx_out"][lo:hi].double()
        if c["pre"]:
            n = _rms(xo, leaf["w_pre"])
            n.backward(s["dn_out"][lo:hi].double())
            d = d + xo.grad
            del n
        (BRANCH_SCALE * branch(h, lo, hi)).backward(d)
        dx.append((RES_SCALE * d).detach())
        dh.append(h.grad if h.grad is not None else torch.zeros_like(h))
    grad = {k: v.grad for k, v in leaf.items()}
    return [torch.cat(dx), torch.cat(dh), grad.get("gate"), grad.get("w_post"), grad.get("w_pre")]
