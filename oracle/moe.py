"""The mixture-of-experts MLP and the adapters beside a projection in fp64 (test infrastructure).

Formulas (N tokens, E experts, k choices for a token):
  * router: q = softmax of the logits over all experts ("softmax") or over the chosen ones ("topk"); the
    k largest logits are chosen, ties to the lowest index; -inf and NaN are masked and never chosen;
  * rows sorted by expert, tokens ascending inside an expert;
  * y_i = act(x[row_i] W_e); dx_i = act'(h_i) (dy_i W_e^T); dW_e = sum_i x[row_i]^T dy_i;
  * combine: y_n = sum_j w_nj u[slot_nj]; du[slot_nj] = w_nj dy_n; dw_nj = <dy_n, u[slot_nj]>;
  * logits: dl_i = q_i (dw_i - sum_j q_j dw_j), dw zero where an expert was not chosen;
  * adapters: y_n = x_n W + s_a (x_n A_a) B_a, a the token's adapter.
"""
from __future__ import annotations

import numpy as np

from .mlp import act_derivative, activate


def _clean(logits):
    v = np.array(logits, dtype=np.float64)
    v[np.isnan(v)] = -np.inf
    v[v == np.inf] = float(np.finfo(np.float32).max)
    return v


def _softmax(v):
    """Softmax along the last axis; a row of -inf gives zeros."""
    m = v.max(axis=-1, keepdims=True)
    e = np.where(np.isfinite(v), np.exp(v - np.where(np.isfinite(m), m, 0.0)), 0.0)
    s = e.sum(axis=-1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def choose(logits, k: int):
    """The chosen experts [N, k], -1 where fewer than k are left."""
    v = _clean(logits)
    order = np.argsort(-v, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(v, order, 1) == -np.inf, -1, order).astype(np.int32)


def gate_softmax(logits, expert, gate: str):
    """q [N, E]: what the weights are taken from."""
    v = _clean(logits)
    if gate == "topk":
        keep = np.zeros(v.shape, bool)
        for n, row in enumerate(expert):
            keep[n, row[row >= 0]] = True
        v = np.where(keep, v, -np.inf)
    return _softmax(v)


def sort_rows(expert, E: int, rest: bool = False):
    """(offsets, row_token, slot) of the entries sorted by expert; rest: the others follow as a last group."""
    N, k = expert.shape
    offsets, token = np.zeros(E + 1, np.int32), []
    slot = np.full((N, k), -1, np.int32)
    for e in list(range(E)) + ([None] if rest else []):
        for n in range(N):
            for j in range(k):
                if expert[n, j] == e or (e is None and not 0 <= expert[n, j] < E):
                    slot[n, j] = len(token)
                    token.append(n)
        if e is not None:
            offsets[e + 1] = len(token)
    return offsets, np.array(token, np.int32), slot


def route(logits, k: int, gate: str):
    expert = choose(logits, k)
    q = gate_softmax(logits, expert, gate)
    weight = np.where(expert >= 0, np.take_along_axis(q, np.maximum(expert, 0), 1), 0.0)
    offsets, row_token, slot = sort_rows(expert, np.shape(logits)[1])
    return {"expert": expert, "weight": weight, "offsets": offsets, "row_token": row_token, "slot": slot}


def route_backward(logits, expert, dweight, gate: str):
    q = gate_softmax(logits, expert, gate)
    dw = np.zeros_like(q)
    for n, row in enumerate(expert):
        for j, e in enumerate(row):
            if e >= 0:
                dw[n, e] += dweight[n, j]
    return q * (dw - (q * dw).sum(axis=1, keepdims=True))


def segments(offsets, R: int):
    """(first, end) of every segment as the library reads them: clamped to 0..R, never negative in length."""
    o = np.clip(np.asarray(offsets, np.int64), 0, R)
    return [(int(a), int(max(a, b))) for a, b in zip(o[:-1], o[1:])]


def rows_of(x, index, R: int):
    x = np.asarray(x, np.float64)
    if index is None:
        return x[:R]
    index = np.asarray(index)[:R]
    ok = (index >= 0) & (index < x.shape[0])
    return np.where(ok[:, None], x[np.where(ok, index, 0)], 0.0)


def ragged_products(x, index, offsets, R: int, w):
    """x[row_i] W_e for the rows of every segment; NaN in rows that belong to none. w [E, K, n]."""
    g = rows_of(x, index, R)
    out = np.full((R, w.shape[2]), np.nan)
    for e, (a, b) in enumerate(segments(offsets, R)):
        out[a:b] = g[a:b] @ np.asarray(w[e], np.float64)
    return out


def ragged_linear(x, index, offsets, R: int, w, act: str):
    return activate(ragged_products(x, index, offsets, R, w), act)


def activation_grad(h, dz, act: str):
    """act'(h) * dz; SwiGLU: h = [gate | up] and the result is [dgate | dup]."""
    if act == "swiglu":
        f = h.shape[-1] // 2
        g, u = h[..., :f], h[..., f:]
        s = 1.0 / (1.0 + np.exp(-g))
        return np.concatenate([dz * u * s * (1.0 + g * (1.0 - s)), dz * g * s], axis=-1)
    return dz * act_derivative(h, act)


def ragged_linear_dx(dy, offsets, R: int, w, act: str, h_pre):
    dz = ragged_products(dy, None, offsets, R, np.swapaxes(np.asarray(w, np.float64), 1, 2))
    return dz if act == "none" else activation_grad(np.asarray(h_pre, np.float64), dz, act)


def ragged_linear_dw(x, index, dy, offsets, R: int, E: int):
    g, dy = rows_of(x, index, R), np.asarray(dy, np.float64)
    out = np.zeros((E, g.shape[1], dy.shape[1]))
    for e, (a, b) in enumerate(segments(offsets, R)):
        out[e] = g[a:b].T @ dy[a:b]
    return out


def combine(u, weight, slot):
    u = np.asarray(u, np.float64)
    y = np.zeros((slot.shape[0], u.shape[1]))
    for j in range(slot.shape[1]):
        ok = (slot[:, j] >= 0) & (slot[:, j] < u.shape[0])
        w = 1.0 if weight is None else np.asarray(weight, np.float64)[ok, j, None]
        y[ok] += w * u[slot[ok, j]]
    return y


def combine_backward(dy, u, weight, slot):
    """(du with NaN in rows that no slot names, dweight)."""
    dy, u, weight = (np.asarray(v, np.float64) for v in (dy, u, weight))
    du = np.full(u.shape, np.nan)
    dweight = np.zeros(weight.shape)
    for j in range(slot.shape[1]):
        ok = (slot[:, j] >= 0) & (slot[:, j] < u.shape[0])
        du[slot[ok, j]] = weight[ok, j, None] * dy[ok]
        dweight[ok, j] = (dy[ok] * u[slot[ok, j]]).sum(axis=1)
    return du, dweight


def moe_mlp(x, logits, w_in, w_down, k: int, gate: str, act: str):
    """Forward pass of the whole MLP, nothing rounded."""
    r = route(logits, k, gate)
    R = len(r["row_token"])
    h = ragged_products(x, r["row_token"], r["offsets"], R, w_in)
    z = activate(h, act)
    u = ragged_products(z, None, r["offsets"], R, w_down)
    return {**r, "h": h, "z": z, "u": u, "y": combine(u, r["weight"], r["slot"])}


def moe_mlp_backward(x, logits, w_in, w_down, k: int, gate: str, act: str, dy):
    f = moe_mlp(x, logits, w_in, w_down, k, gate, act)
    R, E = len(f["row_token"]), w_in.shape[0]
    du, dweight = combine_backward(dy, f["u"], f["weight"], f["slot"])
    dh = ragged_linear_dx(du, f["offsets"], R, w_down, act, f["h"])
    dxr = ragged_linear_dx(dh, f["offsets"], R, w_in, "none", None)
    return {**f, "dw_down": ragged_linear_dw(f["z"], None, du, f["offsets"], R, E), "dh": dh,
            "dw_in": ragged_linear_dw(x, f["row_token"], dh, f["offsets"], R, E), "dx": combine(dxr, None, f["slot"]),
            "dweight": dweight, "dlogits": route_backward(logits, f["expert"], dweight, gate)}


def lora(x, w, a, b, scale, ids):
    """y [t, N, n/t]; w [t, k, n/t], a [L, k, rank], b [t, L, rank, n/t]."""
    x = np.asarray(x, np.float64)
    y = np.stack([x @ np.asarray(m, np.float64) for m in w])
    for n, i in enumerate(np.asarray(ids)):
        if 0 <= i < a.shape[0]:
            v = (1.0 if scale is None else float(scale[i])) * (x[n] @ np.asarray(a[i], np.float64))
            for r in range(y.shape[0]):
                y[r, n] += v @ np.asarray(b[r][i], np.float64)
    return y
