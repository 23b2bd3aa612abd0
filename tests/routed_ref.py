"""64-bit plain implementations of the scored router, its gradient, the combine's
gradient, MXFP4 rounding and the 4-bit product, for the CPU and GPU tests.  They
share no code with the library."""
import numpy as np

U = 2.0 ** -24  # unit roundoff of float32

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ----------------------------------------------------------------- router
def scores(l, score):
    l = np.asarray(l, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
    m = l.max(-1, keepdims=True)
    e = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
    s = e.sum(-1, keepdims=True)
    return np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0)


def route(l, k, bias, score, n_groups, topk_groups, group_score, normalize, scale):
    """ids, weights and the float32 bound on the weights, row by row."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    m = E // n_groups
    p = scores(l, score)
    ids = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    tol = np.zeros((T, k))
    for t in range(T):
        # without a bias, equal and unequal logits decide (a softmax may underflow to equal scores)
        key = p[t] + bias if bias is not None else p[t]
        tie = np.zeros(E) if bias is not None else l[t]
        order = sorted(range(E), key=lambda e: (-key[e], -tie[e], e))
        if topk_groups < n_groups:
            gs = []
            for g in range(n_groups):
                ks = sorted(key[g * m:(g + 1) * m], reverse=True)
                gs.append(ks[0] + (ks[1] if group_score == "top2" else 0.0))
            open_ = sorted(range(n_groups), key=lambda g: (-gs[g], g))[:topk_groups]
            order = [e for e in order if e // m in open_]
        ids[t] = order[:k]
        c = p[t, ids[t]]
        tot = c.sum()
        w[t] = scale * (c / tot if normalize and tot > 0 else c)
        # 64-bit scores that underflow next to each other: take the ratio from the logits
        lc = l[t, ids[t]]
        if normalize and np.isfinite(lc).any():
            base = np.minimum(lc, 0.0) if score == "sigmoid" else lc
            r = np.where(np.isneginf(lc), 0.0, np.exp(base - base.max()))
            if score == "sigmoid":
                r = r / (1.0 + np.exp(-np.abs(lc)))
            w[t] = scale * r / r.sum()
        fin = l[t][np.isfinite(l[t])]
        span = fin.max() - fin.min() if fin.size else 0.0
        tol[t] = (span + 16 + E + k) * U * np.abs(w[t]) + 2.0 ** -149
    return ids, w, tol


def route_grad(l, ids, g, score, normalize, scale, half_step):
    """dlogits and a bound on a float32 evaluation rounded once to a type of relative half step `half_step`."""
    l, g = np.asarray(l, np.float64), np.asarray(g, np.float64) * scale
    T, E = l.shape
    k = ids.shape[1]
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        p = scores(l[t:t + 1], score)[0]
        ok = (ids[t] >= 0) & (ids[t] < E)
        sel = ids[t][ok]
        gi = g[t][ok]
        s = p[sel]
        if score == "softmax" and not normalize:
            dot, adot = (gi * s).sum(), (np.abs(gi) * s).sum()
            gs, ag = np.zeros(E), np.zeros(E)
            np.add.at(gs, sel, gi)
            np.add.at(ag, sel, np.abs(gi))
            out[t] = p * (gs - dot)
            mag[t] = p * (ag + adot)
        else:
            if normalize:
                lc = l[t][sel]
                base = np.minimum(lc, 0.0) if score == "sigmoid" else lc
                if not np.isfinite(lc).any():
                    continue
                r = np.where(np.isneginf(lc), 0.0, np.exp(base - base.max()))
                if score == "sigmoid":
                    r = r / (1.0 + np.exp(-np.abs(lc)))
                q = r / r.sum()
                v, m = q * (gi - (gi * q).sum()), q * (np.abs(gi) + (np.abs(gi) * q).sum())
            else:
                v, m = gi * s, np.abs(gi) * s
            if score == "sigmoid":
                slope = scores(-l[t:t + 1], "sigmoid")[0][sel]
                v, m = v * slope, m * slope
            np.add.at(out[t], sel, v)
            np.add.at(mag[t], sel, m)
    fin = np.where(np.isfinite(l), l, 0.0)
    span = (fin.max(1) - fin.min(1))[:, None]
    # factors: each score within (span + 16 + E + k) u, products and differences a few u more
    rel = (3 * (span + 16 + E + k) + 16) * U
    return out, mag * rel * (1 + half_step) + np.abs(out) * half_step + 2.0 ** -24 * (half_step > U) * 0.5 + 2.0 ** -149


# ---------------------------------------------------------------- combine
def combine_grad(dy, dst, w):
    dy, dst, w = (np.asarray(a, np.float64) for a in (dy, dst, w))
    dw = np.einsum("tn,tkn->tk", dy, dst)
    mag = np.einsum("tn,tkn->tk", np.abs(dy), np.abs(dst))
    return dw, (dst.shape[-1] / 256 + 16) * U * mag + 2.0 ** -149, w[:, :, None] * dy[:, None, :]


# ------------------------------------------------------------------ MXFP4
def mx_round(x):
    """(values, scale bytes, codes) of rows [..., n] rounded to MXFP4 blocks of 32."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    _, e = np.frexp(amax)
    X = np.where(amax > 0, np.maximum(e - 1 - 2, -127) + 127, 0).astype(np.int64)
    r = np.abs(b) / np.exp2(X - 127.0)[..., None]
    d = np.abs(r[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    cand = d == best  # one code, or the two around a midpoint: the even one
    code = np.where(cand.sum(-1) > 1, np.argmax(cand & (np.arange(8) % 2 == 0), -1), np.argmax(cand, -1))
    sign = np.signbit(x.reshape(b.shape)) & ~bad[..., None]
    v = np.where(sign, -1.0, 1.0) * GRID[code] * np.exp2(X - 127.0)[..., None]
    v = np.where(bad[..., None], np.nan, v)
    return v.reshape(x.shape), np.where(bad, 255, X).astype(np.uint8), (code + 8 * sign).astype(np.uint8)


def mx_blocks(X, code):
    return np.concatenate([X[..., None], code[..., :16] | (code[..., 16:] << 4)], -1).astype(np.uint8)


def mx_weights(blocks):
    """64-bit values of MXFP4 blocks [..., nb, 17]."""
    b = np.asarray(blocks)
    code = np.concatenate([b[..., 1:] & 15, b[..., 1:] >> 4], -1)
    v = np.concatenate([GRID, -GRID])[code] * np.exp2(b[..., :1].astype(np.float64) - 127.0)
    return v.reshape(b.shape[:-2] + (-1,))


def mx_product(blocks, x, ids, per_slot):
    """(dst, sum of |terms|) of W[ids] . Q(x): blocks [E][n_out][nb][17], x [rows][n_in]."""
    W = mx_weights(blocks)
    q = mx_round(x)[0]
    T, k = ids.shape
    n_out = W.shape[1]
    out, mag = np.zeros((T, k, n_out)), np.zeros((T, k, n_out))
    for t in range(T):
        for s in range(k):
            r = q[t * k + s] if per_slot else q[t]
            with np.errstate(invalid="ignore"):
                out[t, s] = W[ids[t, s]] @ r
                mag[t, s] = np.abs(W[ids[t, s]]) @ np.abs(r)
    return out, mag
