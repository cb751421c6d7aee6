"""CPU oracle of the operators around the expert layer: router, sorted rows,
block norms, and their gradients.

TEST INFRASTRUCTURE ONLY, numpy in 64 bits, written from the definitions
(one token after the other where that is plainest).  Functions that return
computed numbers return beside each the sum of the absolute values of the
terms it is made of, which a comparison's tolerance is proportional to.
"""
import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def clean_logits(x, pad=None):
    """NaN and -inf mask (-inf), +inf counts as the largest finite fp32."""
    x = np.array(x, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    x[x == np.inf] = FLT_MAX
    if pad is not None:
        x[np.asarray(pad) != 0] = -np.inf
    return x


def _scores(row, score):
    live = row > -np.inf
    s = np.zeros_like(row)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-row[live]))
    elif live.any():
        e = np.exp(row[live] - row[live].max())
        s[live] = e / e.sum()
    return s


def _best(keys, count):
    """Indices of the `count` largest keys above -inf, descending, ties by the
    lower index."""
    order = sorted((i for i in range(len(keys)) if keys[i] > -np.inf),
                   key=lambda i: (-keys[i], i))
    return order[:count]


def router_topk(x, k, score, bias=None, groups=1, topk_groups=1, group_top=1, renormalize=True,
                scale=1.0, pad=None):
    """(ids [T, k], weights [T, k])."""
    x = clean_logits(x, pad)
    T, E = x.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        s = _scores(x[t], score)
        live = x[t] > -np.inf
        key = x[t].copy()
        if bias is not None or group_top > 1:
            key[live] = s[live] + (np.asarray(bias, dtype=np.float64)[live]
                                   if bias is not None else 0.0)
        if groups > 1:
            size = E // groups
            value = []
            for g in range(groups):
                top = _best(key[g * size:(g + 1) * size], group_top)
                value.append(sum(key[g * size + i] for i in top) if top else -np.inf)
            keep = _best(value, topk_groups)
            for e in range(E):
                if e // size not in keep:
                    key[e] = -np.inf
        chosen = _best(key, k)
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if not renormalize:
            w[t, :len(chosen)] = s[chosen]
        elif score == "sigmoid":
            w[t, :len(chosen)] = s[chosen] / (s[chosen].sum() + 1e-20)
        else:
            e = np.exp(x[t, chosen] - x[t, chosen].max())
            w[t, :len(chosen)] = e / e.sum()
    return ids, w * scale


def router_topk_grad(x, ids, grad_w, score, renormalize=True, scale=1.0):
    """(grad of the logits [T, E], magnitude [T, E])."""
    x = clean_logits(x)
    T, E = x.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        js = [j for j, e in enumerate(ids[t]) if 0 <= e < E and x[t, e] > -np.inf]
        if not js:
            continue
        e = np.asarray(ids[t])[js]
        g = np.asarray(grad_w, dtype=np.float64)[t, js] * scale
        s = _scores(x[t], score)
        if score == "softmax":
            if renormalize:
                p = np.exp(x[t, e] - x[t, e].max())
                p = p / p.sum()
            else:
                p = s[e]
            dot, adot = (g * p).sum(), np.abs(g * p).sum()
            if not renormalize:
                out[t] -= s * dot
                mag[t] += s * adot
            for i, ei in enumerate(e):
                out[t, ei] += p[i] * (g[i] - (dot if renormalize else 0.0))
                mag[t, ei] += p[i] * (abs(g[i]) + (adot if renormalize else 0.0))
        else:
            with np.errstate(over="ignore"):
                ds = s[e] / (1.0 + np.exp(x[t, e]))      # 1 - s without cancellation
            D = s[e].sum() + 1e-20 if renormalize else 1.0
            dot = (g * s[e]).sum() / D if renormalize else 0.0
            adot = np.abs(g * s[e]).sum() / D if renormalize else 0.0
            for i, ei in enumerate(e):
                out[t, ei] += (g[i] - dot) / D * ds[i]
                mag[t, ei] += (abs(g[i]) + adot) / D * ds[i]
    return out, mag


def sort_slots(ids, E, pad=None):
    """(expert_offsets [E+1], slot_row [T, k], row_slot of the routed rows)."""
    ids = np.asarray(ids)
    T, k = ids.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        if pad is not None and pad[t]:
            continue
        for j in range(k):
            if 0 <= ids[t, j] < E:
                rows[ids[t, j]].append(t * k + j)
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    row_slot = np.array([s for r in rows for s in r], dtype=np.int64)
    slot_row = np.full(T * k, -1, dtype=np.int64)
    slot_row[row_slot] = np.arange(len(row_slot))
    return offsets, slot_row.reshape(T, k), row_slot


def combine(rows, slot_row, w=None):
    """(out [T, H], magnitude)."""
    T, k = slot_row.shape
    out, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < T * k:
                term = (1.0 if w is None else float(w[t, j])) * rows[r].astype(np.float64)
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_grad(grad_out, rows, slot_row, w=None):
    """({row: gradient}, grad_w [T, k], its magnitude)."""
    T, k = slot_row.shape
    grad_rows, gw, mag = {}, np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        g = grad_out[t].astype(np.float64)
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < T * k:
                grad_rows[int(r)] = g * (1.0 if w is None else float(w[t, j]))
                terms = g * rows[r].astype(np.float64)
                gw[t, j], mag[t, j] = terms.sum(), np.abs(terms).sum()
    return grad_rows, gw, mag


def _norm(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate(gate, kind, sigmoid):
    if gate is None:
        return np.float64(1.0)
    g = gate.astype(np.float64)
    if sigmoid:
        g = 1.0 / (1.0 + np.exp(-g))
    return g[:, None] if kind == "token" else g


def _weight(w, offset):
    return np.float64(1.0) if w is None else offset + w.astype(np.float64)


def block_norm(r, y=None, post_norm=False, w_post=None, gate=None, kind="none", sigmoid=False,
               w_pre=None, eps=1e-6, scale=1.0, offset=0.0):
    """{"residual_out", "normed"}: (value, magnitude) each."""
    r = r.astype(np.float64)
    mag, out = np.abs(r), {}
    if y is not None:
        n = y.astype(np.float64)
        if post_norm:
            n = n * _norm(n, eps) * _weight(w_post, offset)
        add = scale * _gate(gate, kind, sigmoid) * n
        r, mag = r + add, mag + np.abs(add)
        out["residual_out"] = (r, mag)
    s, w = _norm(r, eps), _weight(w_pre, offset)
    out["normed"] = (r * s * w, mag * s * np.abs(w))
    return out


def block_norm_grad(x, dh, dr_in=None, y=None, post_norm=False, w_post=None, gate=None,
                    kind="none", sigmoid=False, w_pre=None, eps=1e-6, scale=1.0, offset=0.0):
    """{name: (gradient, magnitude)} at the stored stream x."""
    x = x.astype(np.float64)
    dh = np.zeros_like(x) if dh is None else dh.astype(np.float64)
    dr_in = np.zeros_like(x) if dr_in is None else dr_in.astype(np.float64)
    w, xs = _weight(w_pre, offset), _norm(x, eps)
    e = dh * w
    D = dr_in + xs * e - x * xs ** 3 * (e * x).mean(axis=1, keepdims=True)
    Dm = (np.abs(dr_in) + xs * np.abs(e)
          + np.abs(x) * xs ** 3 * np.abs(e * x).mean(axis=1, keepdims=True))
    out = {"grad_residual": (D, Dm),
           "grad_pre_weight": ((dh * x * xs).sum(0), np.abs(dh * x * xs).sum(0))}
    if y is None:
        return out
    y = y.astype(np.float64)
    ys = _norm(y, eps) if post_norm else np.ones((len(y), 1))
    wp = _weight(w_post if post_norm else None, offset)
    g = _gate(gate, kind, sigmoid)
    n = y * ys * wp
    if gate is not None:
        slope = g * (1.0 - g) if sigmoid else np.float64(1.0)
        dg, dgm = scale * D * n * slope, np.abs(scale * n * slope) * Dm
        axis = {"token": 1, "channel": 0, "full": None}[kind]
        out["grad_gate"] = (dg, dgm) if axis is None else (dg.sum(axis), dgm.sum(axis))
    dn, dnm = scale * g * D, np.abs(scale * g) * Dm
    if post_norm:
        out["grad_post_weight"] = ((dn * y * ys).sum(0), (dnm * np.abs(y) * ys).sum(0))
        e, em = dn * wp, dnm * np.abs(wp)
        out["grad_y"] = (ys * e - y * ys ** 3 * (e * y).mean(axis=1, keepdims=True),
                         ys * em + np.abs(y) * ys ** 3
                         * (em * np.abs(y)).mean(axis=1, keepdims=True))
    else:
        out["grad_y"] = (dn, dnm)
    return out
