"""The operators of a training step around the collectives of a transformer's layers, as measurable cases: layer norm and
its gradients, the end of a block (partial products summed, dropout, residual, layer norm) and its gradients, the balance
loss of a router and its gradient, and the rows of a vocabulary shard with their gradient.

`prepare` makes the inputs, and the result buffers that a program keeps; `run` makes one pass, in plain torch operations in
32 bits or (with `own`) through the package; `exact` gives the results from the definitions in 64 bits."""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
IDS = {"i32": torch.int32, "i64": torch.int64}
EPS = 1e-5     # of the norms
COEF = 0.01    # of the balance loss
SCALE = 1.5    # of the embedding's rows
SKEW = 3.0     # of the tokens: id n of V as often as the n-th part of a power law


def listed():
    return [
        # the norm before a head at a decode batch of 32, latency
        dict(name="layer norm decode", op="ln", tokens=32, hidden=8192, dtype="bf16", affine=True),
        # the same for a long prefill
        dict(name="layer norm prefill", op="ln", tokens=16384, hidden=8192, dtype="bf16", affine=True),
        # its gradients in a training step
        dict(name="layer norm gradient", op="ln_grad", tokens=8192, hidden=8192, dtype="bf16", affine=True),
        # the same for a small ragged batch in FP32 of an odd hidden size
        dict(name="layer norm gradient odd", op="ln_grad", tokens=1001, hidden=2051, dtype="f32", affine=True),
        # end of a block in a training step: dropout, residual, next norm
        dict(name="dropout block", op="drop", tokens=16384, hidden=8192, dtype="bf16", ranks=1, residual=True, norm=True, p=0.1, first=0),
        # its gradients
        dict(name="dropout gradient", op="drop_grad", tokens=8192, hidden=8192, dtype="bf16", norm=True, p=0.1, first=0),
        # a small sequence-parallel shard: 4 ranks' partial products summed, rows of an odd size, no norm after it
        dict(name="dropout shard odd", op="drop", tokens=1001, hidden=2051, dtype="f32", ranks=4, residual=True, norm=False, p=0.25, first=2002),
        # the balance loss of a small padded batch, forward alone, latency
        dict(name="balance small", op="balance", tokens=512, experts=64, topk=8, dtype="bf16", padded=True, train=False),
        # the loss and its gradient in a training step
        dict(name="balance train", op="balance", tokens=32768, experts=256, topk=8, dtype="f32", padded=True, train=True),
        # the rows of a prefill from one of four shards of the vocabulary
        dict(name="embed shard", op="embed", tokens=16384, vocab=16000, hidden=8192, dtype="bf16", shards=4, ids="i64"),
        # the gradient of a whole table in a training step
        dict(name="embed gradient", op="embed_grad", tokens=16384, vocab=32000, hidden=8192, dtype="bf16", shards=1, ids="i64"),
        # the gradient of a shard of odd size for a small batch in FP32
        dict(name="embed gradient odd", op="embed_grad", tokens=777, vocab=4001, hidden=1025, dtype="f32", shards=4, ids="i32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln_grad", "drop", "drop_grad", "balance", "embed", "embed_grad"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op == "balance":
        experts = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384])
        return dict(op=op, tokens=max(1, min(_log(rng, 1, 32768), 32768 * 256 // experts)), experts=experts, topk=rng.randint(1, min(10, experts)),
                    dtype=dtype, padded=rng.random() < 0.5, train=rng.random() < 0.6)
    hidden = _log(rng, 96, 12288)
    if rng.random() < 0.75:
        hidden = max(64, hidden // 64 * 64)
    if op in ("embed", "embed_grad"):
        vocab = _log(rng, 500, 64000)
        if op == "embed":
            tokens = min(_log(rng, 1, 16384), 16384 * 8192 * 2 // (hidden * ES[dtype]))
            vocab = min(vocab, 32000 * 8192 * 2 // (hidden * ES[dtype]))
        else:
            tokens = min(_log(rng, 1, 16384), 16384 * 8192 * 2 // (hidden * ES[dtype]))
            vocab = min(vocab, 32000 * 8192 // hidden)
        return dict(op=op, tokens=max(1, tokens), vocab=max(1, vocab), hidden=hidden, dtype=dtype, shards=rng.choice([1, 1, 4, 8]),
                    ids=rng.choice(["i32", "i64"]))
    tokens = max(1, min(_log(rng, 1, 16384), (8192 if op.endswith("grad") else 16384) * 8192 * 2 // (hidden * ES[dtype])))
    c = dict(op=op, tokens=tokens, hidden=hidden, dtype=dtype)
    if op in ("ln", "ln_grad"):
        return c | dict(affine=rng.random() < 0.8)
    c |= dict(norm=rng.random() < 0.6, p=rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]), first=rng.choice([0, 0, 1001, 1 << 33]))
    if op == "drop":
        c |= dict(ranks=rng.choice([1, 1, 2, 4, 8]), residual=rng.random() < 0.8)
        c["tokens"] = max(1, min(tokens, 16384 * 8192 * 8 // ((c["ranks"] + 3) * hidden * ES[dtype])))
    return c


# -- inputs ---------------------------------------------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def _tokens(c, g):
    """Ids of a text: a few are frequent and many rare, spread over all shards; a few places are padding (-1)."""
    total = c["vocab"] * c["shards"]
    u = torch.rand(c["tokens"], device="cuda", generator=g, dtype=torch.float64)
    ids = (u.pow(SKEW) * total).long().clamp_(max=total - 1)
    step = next(s for s in (1000003, 999983, 999979) if math.gcd(s, total) == 1)
    ids = ids * step % total
    ids[torch.rand(c["tokens"], device="cuda", generator=g) < 0.02] = -1
    return ids.to(IDS[c["ids"]])


def _first_id(c):
    return c["shards"] // 2 * c["vocab"]


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    T, dt = c["tokens"], DT[c["dtype"]]
    s = dict(c=c)

    def buf(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    if c["op"] == "balance":
        E, K = c["experts"], c["topk"]
        z = torch.randn(T, E, device="cuda", generator=g) * 1.5 + torch.randn(E, device="cuda", generator=g)
        s |= dict(logits=z.to(dt), ids=z.topk(K, dim=1).indices.to(torch.int32), valid=None, loss=buf(1, dtype=torch.float32),
                  counts=buf(E + 1, dtype=torch.int32), prob_sums=buf(E, dtype=torch.float32))
        if c["padded"]:  # padding behind the sequences of a batch
            length = max(1, -(-T // 16))
            keep = (torch.rand(16, 1, device="cuda", generator=g) * 0.6 + 0.4) * length
            s["valid"] = (torch.arange(length, device="cuda") < keep).reshape(-1)[:T].to(torch.uint8)
        if c["train"]:
            s |= dict(dloss=torch.rand(1, device="cuda", generator=g) + 0.5, dlogits=buf(T, E))
        return s
    H = c["hidden"]
    if c["op"] in ("embed", "embed_grad"):
        s["ids"] = _tokens(c, g)
        if c["op"] == "embed":
            s |= dict(table=_normal(g, c["vocab"], H, dtype=dt, scale=0.02), out=buf(T, H))
        else:
            s |= dict(dout=_normal(g, T, H, dtype=dt, scale=0.05), dtable=buf(c["vocab"], H, dtype=torch.float32))
        return s
    loud = torch.exp(1.5 * torch.randn(H, device="cuda", generator=g).clamp_(-1, 2))  # channels of a residual stream differ
    level = 0.3 * torch.randn(H, device="cuda", generator=g)

    def stream():
        return ((torch.randn(T, H, device="cuda", generator=g) + level) * loud).to(dt)
    s["w"] = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(dt) if c.get("affine") or c.get("norm") else None
    s["b"] = _normal(g, H, dtype=dt, scale=0.2) if s["w"] is not None else None
    if c["op"] == "ln":
        return s | dict(x=stream(), out=buf(T, H))
    if c["op"] in ("drop", "drop_grad"):
        words = torch.randint(-1 << 62, 1 << 62, (2,), device="cuda", generator=g)
        s["rng"] = torch.stack([words[0], words[1].abs() % 100000])  # the seed, and which call of the step this is
    if c["op"] == "drop":
        N = c["ranks"]
        return s | dict(h=[_normal(g, T, H, dtype=dt, scale=2 / math.sqrt(N)) for _ in range(N)], x=stream() if c["residual"] else None,
                        x_out=buf(T, H), n_out=buf(T, H) if c["norm"] else None)
    s |= dict(dw=buf(H, dtype=torch.float32), db=buf(H, dtype=torch.float32)) if s["w"] is not None else dict(dw=None, db=None)
    if c["op"] == "ln_grad":
        return s | dict(x=stream(), dout=_normal(g, T, H, dtype=dt, scale=0.1), dx=buf(T, H))
    s |= dict(dx_out=_normal(g, T, H, dtype=dt, scale=0.05), dh=buf(T, H), x_out=None, dn_out=None, dx=None)
    if c["norm"]:
        s |= dict(x_out=stream(), dn_out=_normal(g, T, H, dtype=dt, scale=0.1), dx=buf(T, H))
    return s


# -- one pass -------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    return (_own if own else _plain)(s["c"], s)


def _own(c, s):
    import precision_collective_reduction_gb300 as pcr
    if c["op"] == "ln":
        pcr.layer_norm(s["x"], s["out"], w=s["w"], b=s["b"], eps=EPS)
        return [s["out"]]
    if c["op"] == "ln_grad":
        pcr.layer_norm_backward(s["dout"], s["x"], s["dx"], w=s["w"], eps=EPS, dw=s["dw"], db=s["db"])
        return [s["dx"], s["dw"], s["db"]]
    if c["op"] == "drop":
        pcr.residual_dropout(s["h"], s["x"], s["x_out"], s["rng"], c["p"], n_out=s["n_out"], w=s["w"], b=s["b"], eps=EPS, first_row=c["first"])
        return [s["x_out"], s["n_out"]]
    if c["op"] == "drop_grad":
        pcr.residual_dropout_backward(s["dx_out"], s["dn_out"], s["x_out"], s["dx"], s["dh"], s["rng"], c["p"], w=s["w"], eps=EPS, dw=s["dw"],
                                      db=s["db"], first_row=c["first"])
        return [s["dx"], s["dh"], s["dw"], s["db"]]
    if c["op"] == "balance":
        pcr.expert_balance(s["logits"], s["ids"], s["loss"], s["counts"], s["prob_sums"], coef=COEF, valid=s["valid"])
        out = [s["loss"], s["counts"], s["prob_sums"]]
        if c["train"]:
            pcr.expert_balance_backward(s["logits"], s["counts"], s["dloss"], s["dlogits"], coef=COEF, valid=s["valid"])
            out.append(s["dlogits"])
        return out
    if c["op"] == "embed":
        pcr.token_embed(s["table"], s["ids"], s["out"], first_id=_first_id(c), scale=SCALE)
        return [s["out"]]
    pcr.token_embed_backward(s["dout"], s["ids"], s["dtable"], first_id=_first_id(c), scale=SCALE)
    return [s["dtable"]]


_LOW = 0xFFFFFFFF


def _kept(c, rng):
    """The elements that dropout keeps: those whose random word (Philox4x32-10, four neighbouring columns from one counter) is
    not below p * 2^32."""
    T, H = c["tokens"], c["hidden"]
    groups = -(-H // 4)
    n = (torch.arange(T, device="cuda")[:, None] + c["first"]) * groups + torch.arange(groups, device="cuda")
    c0, c1 = n & _LOW, n >> 32 & _LOW
    c2, c3 = (rng[1] & _LOW).expand_as(n), (rng[1] >> 32 & _LOW).expand_as(n)
    k0, k1 = rng[0] & _LOW, rng[0] >> 32 & _LOW
    for i in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits are the product's, whatever its sign
        c0, c1, c2, c3 = (b >> 32 & _LOW) ^ c1 ^ k0, b & _LOW, (a >> 32 & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = k0 + 0x9E3779B9 & _LOW, k1 + 0xBB67AE85 & _LOW
    least = math.floor(float(np.float32(c["p"])) * 2.0 ** 32)
    return (torch.stack([c0, c1, c2, c3], 2) >= least).view(T, 4 * groups)[:, :H]


def _normed(x, w, b):
    d = x - x.mean(1, keepdim=True)
    y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    return y if w is None else y * w.float() + b.float()


def _normed_gradient(dy, x, w):
    d = x - x.mean(1, keepdim=True)
    r = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    xh = d * r
    q = dy if w is None else dy * w.float()
    dx = r * (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True))
    return (dx, None, None) if w is None else (dx, (dy * xh).sum(0), dy.sum(0))


def _plain(c, s):
    dt = DT[c["dtype"]]
    if c["op"] == "ln":
        return [_normed(s["x"].float(), s["w"], s["b"]).to(dt)]
    if c["op"] == "ln_grad":
        dx, dw, db = _normed_gradient(s["dout"].float(), s["x"].float(), s["w"])
        return [dx.to(dt), dw, db]
    if c["op"] == "drop":
        h = s["h"][0].float()
        for p in s["h"][1:]:
            h = h + p.float()
        if c["p"]:
            h = torch.where(_kept(c, s["rng"]), h * (1 / (1 - float(np.float32(c["p"])))), 0.0)
        x = h if s["x"] is None else s["x"].float() + h
        return [x.to(dt), _normed(x, s["w"], s["b"]).to(dt) if c["norm"] else None]
    if c["op"] == "drop_grad":
        d, dw, db = s["dx_out"].float(), None, None
        if c["norm"]:
            more, dw, db = _normed_gradient(s["dn_out"].float(), s["x_out"].float(), s["w"])
            d = d + more
        dh = torch.where(_kept(c, s["rng"]), d * (1 / (1 - float(np.float32(c["p"])))), 0.0) if c["p"] else d
        return [d.to(dt) if c["norm"] else None, dh.to(dt), dw, db]
    if c["op"] == "balance":
        E = c["experts"]
        z = s["logits"].float()
        e = torch.exp(z - z.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        hits = s["ids"].long()[:, :, None] == torch.arange(E, device="cuda")
        if s["valid"] is not None:
            there = s["valid"] != 0
            p = torch.where(there[:, None], p, 0.0)
            hits = hits & there[:, None, None]
            tokens = there.sum()
        else:
            tokens = torch.full((), c["tokens"], device="cuda")
        counts = hits.sum((0, 1))
        sums, slots = p.sum(0), counts.sum()
        rate = COEF * E / (slots.float() * tokens.float())
        out = [(rate * (counts.float() * sums).sum()).view(1), torch.cat([counts, tokens.view(1)]).int(), sums]
        if c["train"]:
            n = counts.float()
            out.append((s["dloss"] * rate * p * (n - (p * n).sum(1, keepdim=True))).to(dt))
        return out
    row = s["ids"].long() - _first_id(c)
    there = (row >= 0) & (row < c["vocab"])
    if c["op"] == "embed":
        return [torch.where(there[:, None], s["table"][torch.where(there, row, 0)].float() * SCALE, 0.0).to(dt)]
    table = torch.zeros(c["vocab"] + 1, c["hidden"], device="cuda")
    table.index_add_(0, torch.where(there, row, c["vocab"]), s["dout"].float())
    return [table[:-1] * SCALE]


# -- what a pass cannot do without ----------------------------------------------------------------------------------

def _different(c):
    """Rows of the shard that the tokens of a pass are expected to meet."""
    total = c["vocab"] * c["shards"]
    edges = (np.arange(total + 1) / total) ** (1 / SKEW)
    met = -np.expm1(c["tokens"] * 0.98 * np.log1p(-np.minimum(np.diff(edges), 1 - 1e-12))).sum()
    return int(met / c["shards"])


def work(case):
    c, es = case, ES[case["dtype"]]
    T = c["tokens"]
    if c["op"] == "balance":
        E, K = c["experts"], c["topk"]
        n = T * E * es + 4 * T * K + (T if c["padded"] else 0) + 8 * E
        return {"bytes": n + (T * E * es if c["train"] else 0), "flops": (9 if c["train"] else 4) * T * E}
    H = c["hidden"]
    all_ = T * H * es
    if c["op"] == "embed":
        return {"bytes": T * (4 if c["ids"] == "i32" else 8) + _different(c) * H * es + all_, "flops": T * H}
    if c["op"] == "embed_grad":
        used = T // c["shards"]
        return {"bytes": T * (4 if c["ids"] == "i32" else 8) + used * H * es + c["vocab"] * H * 4, "flops": used * H}
    if c["op"] == "ln":
        return {"bytes": 2 * all_ + (2 * H * es if c["affine"] else 0), "flops": 8 * T * H}
    if c["op"] == "ln_grad":
        return {"bytes": 3 * all_ + ((es + 8) * H if c["affine"] else 0), "flops": 14 * T * H}
    draws = 10 if c["p"] else 0  # integer operations of an element's random word
    if c["op"] == "drop":
        n = (c["ranks"] + 1 + c["residual"] + c["norm"]) * all_ + (2 * H * es if c["norm"] else 0)
        return {"bytes": n, "flops": (c["ranks"] + 1 + draws + (8 if c["norm"] else 0)) * T * H}
    return {"bytes": (5 * all_ + (es + 8) * H) if c["norm"] else 2 * all_, "flops": (1 + draws + (15 if c["norm"] else 0)) * T * H}


# -- the definitions in 64 bits -------------------------------------------------------------------------------------

def _product(a, m):
    """Both halves of the product of 32-bit numbers in an int64 tensor with a constant, from 16-bit parts."""
    lo, hi = (a & 0xFFFF) * m, (a >> 16) * m
    top = hi + (lo >> 16)
    return top >> 16, ((top & 0xFFFF) << 16) | (lo & 0xFFFF)


def _words(first, groups, rows, rng):
    """Philox4x32-10 of one group of four columns after the other: [rows, groups, 4]."""
    seed, offset = (int(v) & (1 << 64) - 1 for v in rng.tolist())
    start = torch.tensor([(first + t) * groups for t in range(rows)], dtype=torch.int64)
    x = (start[:, None] + torch.arange(groups)).cuda()
    word = [x % 2 ** 32, x // 2 ** 32, torch.full_like(x, offset % 2 ** 32), torch.full_like(x, offset >> 32)]
    key = [seed % 2 ** 32, seed >> 32]
    for _ in range(10):
        h0, l0 = _product(word[0], 0xD2511F53)
        h1, l1 = _product(word[2], 0xCD9E8D57)
        word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return torch.stack(word, -1)


def _factor(c, rng, lo, hi):
    """What dropout multiplies the rows lo..hi by: 0 or 1 / (1 - p)."""
    p, H = float(np.float32(c["p"])), c["hidden"]
    if p == 0:
        return torch.ones(hi - lo, H, dtype=torch.float64, device="cuda")
    words = _words(c["first"] + lo, -(-H // 4), hi - lo, rng).reshape(hi - lo, -1)[:, :H]
    return (words >= math.floor(p * 2.0 ** 32)).double() / (1 - p)


def _layer_norm(x, w, b):
    n = torch.var_mean(x, 1, correction=0, keepdim=True)
    y = (x - n[1]) / (n[0] + EPS).sqrt()
    return y if w is None else y * w + b


def exact(case, seed):
    c, s = case, prepare(case, seed)
    T = c["tokens"]
    if c["op"] == "balance":
        E = c["experts"]
        kept = np.ones(T, bool) if s["valid"] is None else s["valid"].cpu().numpy() != 0
        z = s["logits"].double().requires_grad_()
        p = torch.softmax(z[torch.from_numpy(kept).cuda()], 1)
        counts = np.bincount(s["ids"].cpu().numpy()[kept].reshape(-1), minlength=E)
        share = torch.from_numpy(counts / counts.sum()).cuda()
        loss = COEF * E * (share * p.mean(0)).sum()
        out = [loss.detach().view(1), torch.from_numpy(np.append(counts, kept.sum()).astype(np.int32)), p.detach().sum(0)]
        if c["train"]:
            loss.backward(s["dloss"].double()[0])
            out.append(z.grad)
        return out
    H = c["hidden"]
    if c["op"] in ("embed", "embed_grad"):
        ids, lo = s["ids"].cpu().numpy().astype(np.int64), _first_id(c)
        mine = np.nonzero((ids >= lo) & (ids < lo + c["vocab"]))[0]
        if c["op"] == "embed":
            out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
            out[torch.from_numpy(mine).cuda()] = s["table"][torch.from_numpy(ids[mine] - lo).cuda()].double() * SCALE
            return [out]
        mine = mine[np.argsort(ids[mine], kind="stable")]
        rows, first, count = np.unique(ids[mine] - lo, return_index=True, return_counts=True)
        total = torch.zeros(c["vocab"], H, dtype=torch.float64, device="cuda")
        one = torch.from_numpy(count == 1).cuda()
        at, of = torch.from_numpy(rows).cuda(), torch.from_numpy(mine[first]).cuda()
        total[at[one]] = s["dout"][of[one]].double()
        for r, f, n in zip(rows, first, count):
            if n > 1:
                total[r] = s["dout"][torch.from_numpy(mine[f: f + n]).cuda()].double().sum(0)
        return [total * SCALE]
    leaf = {k: s[k].double().requires_grad_() if s[k] is not None else None for k in ("w", "b")}
    parts = []
    step = max(1, -(-40_000_000 // H))  # autograd keeps many copies: rows go in parts
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        of = slice(lo, hi)
        if c["op"] == "ln":
            parts.append([_layer_norm(s["x"][of].double(), leaf["w"], leaf["b"]).detach()])
        elif c["op"] == "ln_grad":
            x = s["x"][of].double().requires_grad_()
            _layer_norm(x, leaf["w"], leaf["b"]).backward(s["dout"][of].double())
            parts.append([x.grad])
        elif c["op"] == "drop":
            h = sum(p[of].double() for p in s["h"]) * _factor(c, s["rng"], lo, hi)
            x = h if s["x"] is None else h + s["x"][of].double()
            parts.append([x] + ([_layer_norm(x, leaf["w"], leaf["b"]).detach()] if c["norm"] else []))
        else:
            d = s["dx_out"][of].double()
            if c["norm"]:
                x = s["x_out"][of].double().requires_grad_()
                _layer_norm(x, leaf["w"], leaf["b"]).backward(s["dn_out"][of].double())
                d = d + x.grad
            parts.append([d if c["norm"] else None, d * _factor(c, s["rng"], lo, hi)])
    out = [None if column[0] is None else torch.cat(column) for column in zip(*parts)]
    if c["op"] == "drop" and not c["norm"]:
        out.append(None)
    if c["op"].endswith("grad"):
        out += [leaf[k].grad if leaf[k] is not None else None for k in ("w", "b")]
    return out
