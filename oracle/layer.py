"""fp64 definitions of the layer operators: attention over packed documents, the residual add with the
norms before and after a block, and log probabilities of given tokens, with their gradients.

Plain numpy on whole matrices, written from the formulas of include/lora_layer.h; the gradients are
checked against differences in tests/test_oracle_layer.py.
"""
from __future__ import annotations

import numpy as np


def visible(T, causal=True, window=0, cu_docs=None, prefix=None) -> np.ndarray:
    """(T, T) truth values: token i (row) sees token j (column)."""
    cu = [0, T] if cu_docs is None else [int(c) for c in cu_docs]
    see = np.zeros((T, T), dtype=bool)
    for m, (s, e) in enumerate(zip(cu, cu[1:])):
        pre = 0 if prefix is None else int(prefix[m])
        for i in range(s, e):
            for j in range(s, e):
                see[i, j] = (j <= i or not causal or j < s + pre) and (window == 0 or abs(i - j) < window)
    return see


def cross_visible(Tq, Tk, cu_q=None, cu_k=None, k_len=None) -> np.ndarray:
    """(Tq, Tk) truth values for attn_forward and attn_backward with keys of another tensor."""
    if cu_q is None:
        return np.ones((Tq, Tk), dtype=bool)
    see = np.zeros((Tq, Tk), dtype=bool)
    for m in range(len(cu_q) - 1):
        n = cu_k[m + 1] - cu_k[m] if k_len is None else min(k_len[m], cu_k[m + 1] - cu_k[m])
        see[cu_q[m]:cu_q[m + 1], cu_k[m]:cu_k[m] + n] = True
    return see


def _scores(q, k, see, scale, cap, slope):
    z = scale * (q @ k.T)
    t = np.tanh(z / cap) if cap else None
    s = cap * t if cap else z
    if slope:  # (of a token from another of the same tensor)
        n = np.arange(q.shape[0], dtype=np.float64)
        s = s - slope * np.abs(n[:, None] - n[None, :])
    bend = 1.0 - t * t if cap else np.ones_like(z)
    s = np.where(see, s, -np.inf)
    m = s.max(axis=1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.where(see, np.exp(s - m), 0.0)
    l = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return e / np.where(l > 0, l, 1.0), bend, lse


def attn_forward(q, k, v, see, scale, cap=0.0, slopes=None) -> dict:
    """q (T, hq, d), k and v (T, hk, d) -> O (T, hq, d), lse (hq, T)."""
    T, hq, _ = q.shape
    n = hq // k.shape[1]
    O, lse = np.zeros(q.shape), np.zeros((hq, T))
    for h in range(hq):
        P, _, lse[h] = _scores(q[:, h], k[:, h // n], see, scale, cap, 0.0 if slopes is None else slopes[h])
        O[:, h] = P @ v[:, h // n]
    return {"O": O, "lse": lse}


def attn_backward(q, k, v, dO, see, scale, cap=0.0, slopes=None) -> dict:
    T, hq, _ = q.shape
    n = hq // k.shape[1]
    dQ, dK, dV = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for h in range(hq):
        g = h // n
        P, bend, _ = _scores(q[:, h], k[:, g], see, scale, cap, 0.0 if slopes is None else slopes[h])
        dP = dO[:, h] @ v[:, g].T
        dz = scale * bend * P * (dP - (P * dP).sum(axis=1, keepdims=True))
        dV[:, g] += P.T @ dO[:, h]
        dQ[:, h] = dz @ k[:, g]
        dK[:, g] += dz.T @ q[:, h]
    return {"dQ": dQ, "dK": dK, "dV": dV}


def _norm(a, w, eps):
    r = 1.0 / np.sqrt((a * a).mean(axis=1, keepdims=True) + eps)
    return a * r * w, r


def _norm_back(g, a, r, w):
    """(gradient of a, of w) from that of a * r * w."""
    t = g * w
    return r * (t - a * r * r * (t * a).mean(axis=1, keepdims=True)), (g * a * r).sum(axis=0)


def addnorm_forward(h, y=None, w_in=None, w_post=None, gate=None, alpha=1.0, eps=1e-5, w_offset=0.0) -> dict:
    out = {"rstd_y": None, "rstd_h": None, "x": None}
    if y is not None:
        n = y
        if w_post is not None:
            n, r = _norm(y, w_post + w_offset, eps)
            out["rstd_y"] = r[:, 0]
        h = h + alpha * (1.0 if gate is None else gate) * n
    out["h"] = h
    if w_in is not None:
        out["x"], r = _norm(h, w_in + w_offset, eps)
        out["rstd_h"] = r[:, 0]
    return out


def addnorm_backward(h, y, dh_out, dx, w_in=None, w_post=None, gate=None, alpha=1.0, eps=1e-5, w_offset=0.0) -> dict:
    out = {"dy": None, "dw_in": None, "dw_post": None, "dgate": None}
    s = addnorm_forward(h, y, None, w_post, gate, alpha, eps, w_offset)["h"]
    g = np.zeros_like(s) if dh_out is None else dh_out
    if w_in is not None:
        _, r = _norm(s, w_in + w_offset, eps)
        gn, out["dw_in"] = _norm_back(dx, s, r, w_in + w_offset)
        g = g + gn
    out["dh"] = g
    if y is not None:
        dn = alpha * g * (1.0 if gate is None else gate)
        if w_post is None:
            out["dy"] = dn
        else:
            n, r = _norm(y, w_post + w_offset, eps)
            out["dy"], out["dw_post"] = _norm_back(dn, y, r, w_post + w_offset)
        if gate is not None:
            out["dgate"] = (alpha * g * (y if w_post is None else n)).sum(axis=0)
    return out


def logprob_forward(logits, targets, k=0, scale=1.0) -> dict:
    T, V = logits.shape
    x = scale * logits
    m = x.max(axis=1, keepdims=True)
    empty = np.isneginf(m)
    m0 = np.where(empty, 0.0, m)
    e = np.exp(x - m0)
    S = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = m0 + np.log(S)
        w = np.where(e > 0, e * (x - m0), 0.0).sum(axis=1, keepdims=True)
        ent = np.where(empty, 0.0, np.log(S) - w / S)[:, 0]
        lp = np.where(empty, -np.inf, x - lse)
    has = (targets >= 0) & (targets < V)
    logp = np.where(has, lp[np.arange(T), np.where(has, targets, 0)], 0.0)
    out = {"logp": logp, "entropy": ent, "lse": lse[:, 0], "top_ids": None, "top_logp": None}
    if k:
        key = np.where(np.isnan(logits), np.inf, logits)
        rank = np.lexsort((np.broadcast_to(np.arange(V), (T, V)), -key, ~np.isnan(logits)), axis=1)[:, :k]
        out["top_ids"] = rank.astype(np.int32)
        out["top_logp"] = np.take_along_axis(lp, rank, axis=1)
    return out


def logprob_backward(logits, targets, dlogp=None, dentropy=None, scale=1.0) -> np.ndarray:
    T, V = logits.shape
    f = logprob_forward(logits, targets, 0, scale)
    empty = np.isneginf(f["lse"])
    with np.errstate(invalid="ignore"):
        lp = scale * logits - f["lse"][:, None]
    p = np.where(empty[:, None], 0.0, np.exp(np.where(empty[:, None], 0.0, lp)))
    has = (targets >= 0) & (targets < V) & ~empty
    g = np.where(has, 0.0 if dlogp is None else dlogp, 0.0)
    d = -g[:, None] * p
    if dentropy is not None:
        with np.errstate(invalid="ignore"):
            d = d - np.where(p > 0, dentropy[:, None] * p * (lp + f["entropy"][:, None]), 0.0)
    d[np.arange(T)[has], targets[has]] += g[has]
    return scale * d


# ---------------------------------------------------------------------------------------------
# norms of query and key heads, rotation by position


def qkrope_angles(T, inv_freq, pos=None, axis=None) -> np.ndarray:
    """(T, pairs) angles in radians; pos (T,) or (axes, T), axis the row that turns each pair."""
    f = np.asarray(inv_freq, dtype=np.float64)
    p = np.arange(T)[None] if pos is None else np.atleast_2d(np.asarray(pos))
    which = np.zeros(f.size, dtype=int) if axis is None else np.clip(axis, 0, p.shape[0] - 1)
    return p[which].T.astype(np.float64) * f


def _pair_dims(pairs, interleaved):
    p = np.arange(pairs)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)


def qkrope_forward(x, angles=None, interleaved=False, factor=1.0, norm=False, w=None, eps=1e-6, w_offset=0.0) -> np.ndarray:
    """One side (queries or keys): x (T, h, d) -> the same."""
    y = np.array(x, dtype=np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * (1.0 if w is None else w + w_offset)
    if angles is None:
        return y
    i, j = _pair_dims(angles.shape[1], interleaved)
    c, s = factor * np.cos(angles)[:, None], factor * np.sin(angles)[:, None]
    out = y.copy()
    out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
    return out


def qkrope_backward(x, dy, angles=None, interleaved=False, factor=1.0, norm=False, w=None, eps=1e-6, w_offset=0.0):
    """(dx, dw) of one side; dw None without a weight."""
    g = np.array(dy, dtype=np.float64)
    if angles is not None:
        i, j = _pair_dims(angles.shape[1], interleaved)
        c, s = factor * np.cos(angles)[:, None], factor * np.sin(angles)[:, None]
        g[..., i], g[..., j] = dy[..., i] * c + dy[..., j] * s, dy[..., j] * c - dy[..., i] * s
    if not norm:
        return g, None
    T, h, d = g.shape
    flat = np.asarray(x, dtype=np.float64).reshape(T * h, d)
    wv = np.ones(d) if w is None else w + w_offset
    r = 1.0 / np.sqrt((flat * flat).mean(axis=1, keepdims=True) + eps)
    dx, dw = _norm_back(g.reshape(T * h, d), flat, r, wv)
    return dx.reshape(T, h, d), None if w is None else dw


# ---------------------------------------------------------------------------------------------
# distillation from a teacher's top logits


def _log_softmax_row(x):
    """(log softmax, log sum); a row of nothing but -inf has log sum -inf and no distribution (NaN)."""
    m = x.max(initial=-np.inf)
    if np.isneginf(m):
        return np.full(x.shape, np.nan), -np.inf
    l = np.log(np.exp(x - m).sum())
    return (x - m) - l, m + l  # (beside the lowest numbers of a type l is nothing)


def distill_forward(logits, ids, values, targets=None, scale=1.0, rest=False) -> dict:
    T, V = logits.shape
    out = {"kl": np.zeros(T), "lse": np.zeros(T), "logp": None if targets is None else np.zeros(T)}
    for t in range(T):
        lq, out["lse"][t] = _log_softmax_row(scale * logits[t])
        lq = np.where(np.isnan(lq) & ~np.isnan(logits[t]), -np.inf, lq)
        out["kl"][t] = sum(p * (lp - l) for p, lp, l in _outcomes(lq, ids[t], values[t], scale, rest) if p > 0)
        if targets is not None and 0 <= targets[t] < V:
            l1, s1 = _log_softmax_row(logits[t])
            out["logp"][t] = -np.inf if np.isneginf(s1) else l1[targets[t]]
    return out


def _entries(ids, values, V, scale, rest):
    """The row's entries as (id, log p)."""
    has = [(int(i), float(v)) for i, v in zip(ids, values) if 0 <= i < V]
    if rest or not has:
        return has
    lp, s = _log_softmax_row(scale * np.array([v for _, v in has]))
    return [] if np.isneginf(s) else [(i, l) for (i, _), l in zip(has, lp)]


def _outcomes(lq, ids, values, scale, rest):
    """(p, log p, log q) of every outcome."""
    e = _entries(ids, values, lq.size, scale, rest)
    res = [(np.exp(l), l, lq[i]) for i, l in e]
    if rest and e:
        left = max(0.0, 1.0 - sum(p for p, _, _ in res))
        others = _log_softmax_row(np.delete(lq, sorted({i for i, _ in e})))[1]
        if left > 0 and not np.isneginf(others):  # (no other token: no such outcome)
            res.append((left, np.log(left), others))
    return res


def distill_backward(logits, ids, values, dkl=None, targets=None, dlogp=None, scale=1.0, rest=False) -> np.ndarray:
    T, V = logits.shape
    d = np.zeros((T, V))
    for t in range(T):
        lq, s = _log_softmax_row(scale * logits[t])
        if np.isneginf(s):
            continue
        if dkl is not None and dkl[t] != 0:
            q, e = np.exp(lq), _entries(ids[t], values[t], V, scale, rest)
            p = np.zeros(V)
            for i, l in e:
                p[i] += np.exp(l)
            if rest and e:
                left, mine = max(0.0, 1.0 - p.sum()), np.zeros(V, dtype=bool)
                mine[[i for i, _ in e]] = True
                lo, so = _log_softmax_row(np.where(mine, -np.inf, scale * logits[t]))
                if np.isneginf(so):
                    left = 0.0
                else:  # (q / q_r where both may be tiny)
                    p = np.where(mine, p, left * np.exp(np.where(mine, 0.0, lo)))
                d[t] = scale * dkl[t] * (q * (p[mine].sum() + left) - p)
            elif e:
                d[t] = scale * dkl[t] * (q * p.sum() - p)
        if dlogp is not None and 0 <= targets[t] < V and dlogp[t] != 0:
            l1, _ = _log_softmax_row(logits[t])
            d[t] -= dlogp[t] * np.exp(l1)
            d[t, targets[t]] += dlogp[t]
    return d
