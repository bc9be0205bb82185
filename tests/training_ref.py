"""Plain 64-bit forms of the operators of a training step (numpy): layer norm,
residual_dropout, the router's balance loss and the embedding, with the bounds
that an FP32 evaluation has to keep. Conventions as in layers_ref.py: u = 2^-24,
a BF16 output adds half an ulp, every function returns (value, bound).

Sums. A row's sums are at most DEEP additions deep (16 columns of a thread, 5
steps in a warp, 5 over its CTA's warps, 8 CTAs, and the products), so a sum is
off by DEEP u times the sum of its terms' magnitudes.
"""
import numpy as np

from layers_ref import HALF_ULP, TINY, U

DEEP = 16 + 5 + 5 + 8 + 6
OPS = 12  # single operations between the sums and an output
SLACK = 1 + 2 ** -8  # of a bound's own first-order form


def f64(v):
    return None if v is None else np.asarray(v, np.float64)


# -- dropout's random words ---------------------------------------------------

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Four 32-bit words of one 128-bit counter (four words, lowest first) under
    a 64-bit key (two words), in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = M0 * c[0], M1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return c


def kept(T, H, seed, offset, p, first_row=0):
    """bool [T, H]: the elements that dropout keeps."""
    groups = -(-H // 4)
    least = int(float(np.float32(p)) * 2 ** 32)
    rows = np.array([(first_row + t) * groups & (1 << 64) - 1 for t in range(T)], np.uint64)
    n = rows[:, None] + np.arange(groups, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    seed, offset = seed & (1 << 64) - 1, offset & (1 << 64) - 1
    c = [n & low, n >> s32, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(M0), c[2] * np.uint64(M1)  # below 2^64
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s32) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return (np.stack(c, 2) >= np.uint64(least)).reshape(T, 4 * groups)[:, :H]


# -- layer norm ---------------------------------------------------------------

def _stats(x, ex, eps):
    """xh, r and the errors of xh and, relative, of r, for values that are off by
    ex before the norm."""
    m = x.mean(1, keepdims=True)
    c = x - m
    v = (c * c).mean(1, keepdims=True)
    r = 1 / np.sqrt(v + eps)
    # the mean: its sum, one product, and the values' own errors
    em = (DEEP + 4) * U * np.abs(x).mean(1, keepdims=True) + ex.mean(1, keepdims=True)
    # the squares: their sum; a mean that is off by em adds em^2 and, where warps
    # meet, 2 |m_w - m| em, at most 2 sqrt(v) em; the values' own errors
    ev = ((DEEP + 10) * U * v + 2 * np.sqrt(v) * em + em ** 2
          + 2 * (np.abs(c) * ex).mean(1, keepdims=True))
    er = 0.5 * ev / (v + eps) + 8 * U  # rsqrtf is good to 2 ulp, 4 u
    xh = c * r
    exh = r * (em + ex + U * np.abs(c)) + np.abs(xh) * er
    return xh, r, exh, er


def layer_norm(x, w, b, eps, dt, ex=None):
    """(out, bound); ex: errors of x before the norm."""
    x, w, b = f64(x), f64(w), f64(b)
    xh, _, exh, _ = _stats(x, np.zeros_like(x) if ex is None else ex, eps)
    w = 1.0 if w is None else w
    b = 0.0 if b is None else b
    y = xh * w + b
    e = np.abs(w) * exh + OPS * U * (np.abs(xh * w) + np.abs(b))
    return y, HALF_ULP[dt] * np.abs(y) * SLACK + e * SLACK + TINY


def layer_norm_backward(dn, x, w, eps, dt, dxo=None, factor=None):
    """{name: (gradient, bound)} of dx, dw, db and, with dropout's factor (0 or 1
    / (1 - p)), dh."""
    dn, x, w, dxo = f64(dn), f64(x), f64(w), f64(dxo)
    T = x.shape[0]
    xh, r, exh, er = _stats(x, np.zeros_like(x), eps)
    q = dn if w is None else dn * w
    mq, aq = q.mean(1, keepdims=True), np.abs(q).mean(1, keepdims=True)
    s = (q * xh).mean(1, keepdims=True)
    # terms about a warp's mean are at most three times the row's largest
    es = (DEEP + OPS) * U * 3 * aq * np.abs(xh).max(1, keepdims=True) + (np.abs(q) * exh).mean(
        1, keepdims=True)
    inner = q - mq - xh * s
    D = r * inner + (0.0 if dxo is None else dxo)
    size = r * (np.abs(q) + aq + np.abs(xh * s)) + (0.0 if dxo is None else np.abs(dxo))
    eD = (OPS * U * size + r * ((DEEP + OPS) * U * aq + exh * np.abs(s) + np.abs(xh) * es)
          + 2 * er * r * (np.abs(inner) + np.abs(xh * s)))
    out = {"dx": (D, HALF_ULP[dt] * np.abs(D) * SLACK + eD * SLACK + TINY)}
    if factor is not None:
        dh = D * factor
        out["dh"] = (dh, HALF_ULP[dt] * np.abs(dh) * SLACK
                     + (eD + 3 * U * np.abs(D)) * factor * SLACK + TINY)
    out["dw"] = ((dn * xh).sum(0), ((T + OPS) * U * np.abs(dn * xh).sum(0)
                                    + (np.abs(dn) * exh).sum(0)) * SLACK + TINY)
    out["db"] = (dn.sum(0), (T + OPS) * U * np.abs(dn).sum(0) + TINY)
    return out


def residual_dropout(hs, x, keep, p, w, b, eps, dt, norm):
    """[(x_out, bound), (n_out, bound) or None]"""
    hs, x = [f64(h) for h in hs], f64(x)
    # a dropped element is 0 whatever stands there
    h = np.where(keep, sum(hs), 0.0)
    habs = np.where(keep, sum(np.abs(v) for v in hs), 0.0)
    f = 1 / (1 - float(np.float32(p)))
    d, xabs = h * f, 0.0 if x is None else np.abs(x)
    xo = d if x is None else x + d
    ex = (len(hs) + 3) * U * habs * f + 2 * U * xabs
    out = [(xo, HALF_ULP[dt] * np.abs(xo) * SLACK + ex * SLACK + TINY), None]
    if norm:
        out[1] = layer_norm(xo, w, b, eps, dt, ex)
    return out


# -- balance loss -------------------------------------------------------------

def balance(logits, ids, valid, coef, E):
    """loss, counts (exact), prob_sums, each with its bound but the counts, and the
    probabilities with theirs."""
    z = f64(logits)
    T = z.shape[0]
    there = np.ones(T, bool) if valid is None else np.asarray(valid) != 0
    p, ep = np.zeros((T, E)), np.zeros((T, E))
    for t in np.nonzero(there)[0]:
        some = z[t] > -np.inf
        if not some.any() and not np.isnan(z[t]).any():
            continue
        m = z[t][some].max() if some.any() else 0.0
        with np.errstate(invalid="ignore"):
            e = np.exp(z[t] - m)
        p[t] = e / e.sum()
        # as the router's weights: the argument's rounding, exp (2 ulp), the sum
        far = np.minimum(np.where(np.isfinite(z[t]), np.abs(z[t] - m), 0.0), 120.0)
        ep[t] = (far + far.max() + DEEP + 32 + 12) * U * p[t] + TINY
    counts = np.zeros(E + 1, np.int64)
    for t in np.nonzero(there)[0]:
        for e in np.asarray(ids)[t]:
            if 0 <= e < E:
                counts[e] += 1
    counts[E] = there.sum()
    P = p.sum(0)
    eP = ep.sum(0) + (T + DEEP) * U * P
    S, V = counts[:E].sum(), counts[E]
    n = counts[:E].astype(np.float64)
    rate = 0.0 if S == 0 or V == 0 else float(np.float32(coef)) * E / (float(S) * float(V))
    loss = rate * (n * P).sum()
    eloss = abs(rate) * ((n * eP).sum() + (E + DEEP) * U * (n * P).sum()) + TINY
    return (loss, eloss), counts, (P, eP + TINY), (p, ep), rate


def balance_backward(probs, n, rate, dloss, dt, before=None):
    """(dlogits, bound) from the probabilities and their bounds."""
    p, ep = probs
    n = f64(n)
    mean = (p * n).sum(1, keepdims=True)
    g = float(dloss) * rate * p * (n - mean)
    k = abs(float(dloss) * rate)
    emean = (ep * n).sum(1, keepdims=True) + (DEEP + 32) * U * mean
    e = k * (ep * (n + mean) + p * emean + OPS * U * p * (n + mean))
    if before is not None:
        g = g + f64(before)
        e = e + 2 * U * (np.abs(g) + np.abs(f64(before)))
    return g, HALF_ULP[dt] * np.abs(g) * SLACK + e * SLACK + TINY


# -- embedding ----------------------------------------------------------------

def embed(table, ids, first, scale, dt):
    table = f64(table)
    V, H = table.shape
    out = np.zeros((len(ids), H))
    for t, i in enumerate(ids):
        if first <= i < first + V:
            out[t] = table[i - first] * scale
    return out, (HALF_ULP[dt] + U) * np.abs(out) * SLACK + TINY


def embed_backward(dout, ids, first, V, scale, before=None):
    dout = f64(dout)
    out, size, n = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros(V)
    for t, i in enumerate(ids):
        if first <= i < first + V:
            out[i - first] += dout[t]
            size[i - first] += np.abs(dout[t])
            n[i - first] += 1
    out, size = out * scale, size * abs(scale)
    if before is not None:
        out, size = out + before, size + np.abs(before)
    return out, (n[:, None] + 3) * U * size + TINY
