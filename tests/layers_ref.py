"""Plain 64-bit forms of the operators around the collectives (numpy), with
the bounds that an FP32 evaluation of them has to keep.

Bounds. u = 2^-24 is the unit roundoff of FP32; an output of BF16 (8
significant bits) adds half an ulp, 2^-8 of its value. A sum of n terms in
FP32, in any order, is off by at most (n - 1) u times the sum of the terms'
magnitudes. A chain of a few operations adds that many u to each term; every
function below says how many it allows and returns (value, bound) for each
output.
"""
import numpy as np

U = 2.0 ** -24
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 2.0 ** -126 * 2  # absolute: results below the normal range


def sort(ids, E, capacity=0):
    """slot_row, row_slot, offsets, counts, slot by slot."""
    flat = np.asarray(ids).reshape(-1)
    n = flat.size
    groups = [[] for _ in range(E)]
    for s, e in enumerate(flat):
        if 0 <= e < E and not (capacity and len(groups[e]) >= capacity):
            groups[e].append(s)
    rows = E * capacity if capacity else n
    slot_row, row_slot = np.full(n, -1, np.int32), np.full(rows, -1, np.int32)
    offsets, at = np.zeros(E + 1, np.int32), 0
    for e, g in enumerate(groups):
        at = e * capacity if capacity else at
        offsets[e] = at
        for i, s in enumerate(g):
            slot_row[s] = at + i
            row_slot[at + i] = s
        at += len(g)
    offsets[E] = rows if capacity else at
    return (slot_row.reshape(np.shape(ids)), row_slot, offsets,
            np.array([len(g) for g in groups], np.int32))


def route(logits, K, renormalize):
    """ids, weights and the weights' bound. NaN sorts above everything; -inf
    is never chosen."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    ids = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    bound = np.zeros((T, K))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (not np.isnan(z[t, e]), -z[t, e]
                                                if not np.isnan(z[t, e]) else 0.0, e))
        order = [e for e in order if not z[t, e] == -np.inf][:K]
        if not order:
            continue
        ids[t, :len(order)] = order
        m = z[t, order[0]]
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.exp(z[t] - m)
            total = p[order].sum() if renormalize else p.sum()
            w[t, :len(order)] = p[order] / total
            # exp's argument is rounded (|x - m| u), exp is good to 2 ulp (4 u),
            # the sum has E terms with the same errors, then one division
            far = np.where(np.isfinite(z[t]), np.abs(z[t] - m), 0.0)
            far = np.minimum(far, 120.0)  # below exp(-120) the result is under TINY
            bound[t, :len(order)] = ((far[order] + far.max() + E + 12) * U * w[t, :len(order)]
                                     + TINY)
    return ids, w, bound


def route_backward(logits, ids, w, dw, renormalize):
    """dlogits and its bound, from the 64-bit weights."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    dz, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        there = ids[t] >= 0
        mean = (w[t] * dw[t])[there].sum()
        amean = np.abs(w[t] * dw[t])[there].sum()
        if not there.any():
            continue
        if not renormalize:
            p = np.exp(z[t] - z[t][np.isfinite(z[t])].max())
            p /= p.sum()
            dz[t] = -p * mean
            mag[t] = p * amean
        for k in np.nonzero(there)[0]:
            e = ids[t, k]
            dz[t, e] += w[t, k] * (dw[t, k] - mean if renormalize else dw[t, k])
            mag[t, e] += w[t, k] * (abs(dw[t, k]) + amean)
    # the weights and p are off by (2 * 120 + E + 12) u at most as in route,
    # once in the term and once in the mean, plus K + 6 operations
    return dz, (2 * (240 + E + 12) + ids.shape[1] + 6) * U * mag + TINY


def combine(rows, slot_row, weights, dt):
    rows = np.asarray(rows, np.float64)
    T, K = slot_row.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for k in range(K):
            r = slot_row[t, k]
            if 0 <= r < rows.shape[0]:
                v = rows[r] * (1.0 if weights is None else float(weights[t, k]))
                y[t] += v
                mag[t] += np.abs(v)
    return y, HALF_ULP[dt] * np.abs(y) * (1 + 2 ** -8) + (K + 2) * U * mag * (1 + 2 ** -8) + TINY


def combine_backward(dy, rows, slot_row, weights, R, dt):
    dy = np.asarray(dy, np.float64)
    T, K = slot_row.shape
    H = dy.shape[1]
    drows, dw, mag = np.zeros((R, H)), np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = slot_row[t, k]
            if 0 <= r < R:
                drows[r] = dy[t] * (1.0 if weights is None else float(weights[t, k]))
                if rows is not None:
                    v = np.asarray(rows[r], np.float64) * dy[t]
                    dw[t, k], mag[t, k] = v.sum(), np.abs(v).sum()
    return (drows, (HALF_ULP[dt] + 2 * U) * np.abs(drows) + TINY), (dw, (H + 2) * U * mag + TINY)


# Roundings that the norms' formulas allow between the inputs and an output
# beside the long sums: products, the scale of the norm (whose sum of squares
# has only positive terms, at most SERIAL + 10 deep), the gate and residual.
SERIAL = 16
OPS = SERIAL + 10 + 40


def _f(v):
    return None if v is None else np.asarray(v, np.float64)


def _gate(gate, kind):
    g = _f(gate)
    return 1.0 if g is None else g[:, None] if kind == "token" else g


def residual_norm(hs, x, gate, kind, w_post, w_pre, a, b, eps, dt):
    """[(x_out, bound), (n_out, bound) or None, (h, bound)]"""
    hs, x, g, wq, wp = [_f(h) for h in hs], _f(x), _gate(gate, kind), _f(w_post), _f(w_pre)
    h, habs = sum(hs), sum(np.abs(v) for v in hs)
    eh = len(hs) * U * habs
    r1 = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps) if wq is not None else 1.0
    w = wq if wq is not None else 1.0
    u = h * r1 * w
    # h's own error moves r1 too: |dr1| / r1 <= r1^2 mean(|h| eh)
    eu = np.abs(w) * r1 * eh + OPS * U * np.abs(u)
    if wq is not None:
        eu = eu + np.abs(u) * r1 ** 2 * (np.abs(h) * eh).mean(1, keepdims=True)
    xo = a * x + b * g * u
    ex = OPS * U * (np.abs(a * x) + np.abs(b * g * u)) + np.abs(b * g) * eu
    out = [(xo, HALF_ULP[dt] * np.abs(xo) * (1 + 2 ** -8) + ex * (1 + 2 ** -8) + TINY), None]
    if wp is not None:
        r2 = 1 / np.sqrt((xo * xo).mean(1, keepdims=True) + eps)
        n = xo * r2 * wp
        en = (np.abs(wp) * r2 * ex + np.abs(n) * r2 ** 2 * (np.abs(xo) * ex).mean(1, keepdims=True)
              + OPS * U * np.abs(n))
        out[1] = (n, HALF_ULP[dt] * np.abs(n) * (1 + 2 ** -8) + en * (1 + 2 ** -8) + TINY)
    out.append((h, HALF_ULP[dt] * np.abs(h) * (1 + 2 ** -8) + eh * (1 + 2 ** -8) + TINY))
    return out


def residual_norm_backward(dxo, dn, h, xo, gate, kind, w_post, w_pre, a, b, eps, dt):
    """{name: (gradient, bound)} of dx, dh, dgate, dw_post, dw_pre."""
    dxo, dn, h, xo, g = _f(dxo), _f(dn), _f(h), _f(xo), _gate(gate, kind)
    wq, wp = _f(w_post), _f(w_pre)
    T, H = h.shape
    D = np.zeros((T, H)) if dxo is None else dxo
    Dabs = np.abs(D)  # the same with every term's magnitude
    out = {}
    half = HALF_ULP[dt]
    if wp is not None:
        r2 = 1 / np.sqrt((xo * xo).mean(1, keepdims=True) + eps)
        gw = dn * wp
        out["dw_pre"] = ((dn * xo * r2).sum(0), (T + OPS) * U * np.abs(dn * xo * r2).sum(0) + TINY)
        c2 = r2 ** 2 * (gw * xo).mean(1, keepdims=True)
        D = D + r2 * (gw - xo * c2)
        Dabs = Dabs + r2 * (np.abs(gw) + np.abs(xo) * r2 ** 2 * np.abs(gw * xo).mean(1, keepdims=True))
    out["dx"] = (a * D, half * np.abs(a * D) * (1 + 2 ** -8) + OPS * U * np.abs(a) * Dabs + TINY)
    r1 = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps) if wq is not None else 1.0
    w = wq if wq is not None else 1.0
    u = h * r1 * w
    if kind is not None:
        dg, dgabs = b * u * D, np.abs(b * u) * Dabs
        if kind == "full":
            out["dgate"] = (dg, half * np.abs(dg) * (1 + 2 ** -8) + OPS * U * dgabs + TINY)
        else:
            ax, n = (0, T) if kind == "channel" else (1, H)
            out["dgate"] = (dg.sum(ax), (min(n, SERIAL * 64) + OPS) * U * dgabs.sum(ax) + TINY)
            if kind == "channel":
                out["dgate"] = (dg.sum(0), (T + OPS) * U * dgabs.sum(0) + TINY)
    du, duabs = b * g * D, np.abs(b * g) * Dabs
    dh, dhabs = du, duabs
    if wq is not None:
        hh = h * r1
        out["dw_post"] = ((du * hh).sum(0), (T + OPS) * U * (duabs * np.abs(hh)).sum(0) + TINY)
        q, qabs = du * w, duabs * np.abs(w)
        dh = r1 * (q - hh * (q * hh).mean(1, keepdims=True))
        dhabs = r1 * (qabs + np.abs(hh) * (qabs * np.abs(hh)).mean(1, keepdims=True))
    # sums along a row are at most SERIAL + 10 deep, all within OPS
    out["dh"] = (dh, half * np.abs(dh) * (1 + 2 ** -8) + 2 * OPS * U * dhabs + TINY)
    return out


def forward(h, x, gate, kind, w_post, w_pre, a, b, eps):
    """x_out and n_out alone, for differences."""
    r = residual_norm([h], x, gate, kind, w_post, w_pre, a, b, eps, "f32")
    return r[0][0], None if r[1] is None else r[1][0]
