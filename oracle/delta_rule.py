"""fp64 oracle of the gated delta rule and of the head norms with rotation (test
infrastructure only; shares no code with the GPU path).

    S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,  out_t = scale S_t^T q_t

token by token and head by head, with S_{t-1} = 0 at a document start (token 0
starts one unless an initial state is given, then only where doc_start marks it);
value head h reads key head h // (Hv / Hk)."""

from __future__ import annotations

import numpy as np

CHUNK = 64


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def _starts(B, L, doc_start, initial_state):
    s = np.zeros((B, L), dtype=bool) if doc_start is None else np.asarray(doc_start) != 0
    s = s.copy()
    if initial_state is None and L:
        s[:, 0] = True
    return s


def gated_delta_rule(q, k, v, g, beta, scale=None, doc_start=None, initial_state=None):
    """(out, final_state, states): states (B, Hv, ceil(L / 64), K, V) enter tokens 0, 64, ..."""
    q, k, v, g, beta, initial_state = _f64(q, k, v, g, beta, initial_state)
    B, L, Hk, K = q.shape
    Hv, V = v.shape[2:]
    r = Hv // Hk
    scale = K ** -0.5 if scale is None else scale
    start = _starts(B, L, doc_start, initial_state)
    S = np.zeros((B, Hv, K, V)) if initial_state is None else initial_state.copy()
    out = np.zeros((B, L, Hv, V))
    states = np.zeros((B, Hv, -(-L // CHUNK), K, V))
    for t in range(L):
        if t % CHUNK == 0:
            states[:, :, t // CHUNK] = S
        kt, qt = np.repeat(k[:, t], r, 1), np.repeat(q[:, t], r, 1)
        decay = np.ones((B, Hv)) if g is None else np.exp(g[:, t])
        S = np.where(start[:, t, None, None, None], 0.0, decay[:, :, None, None] * S)
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhkv,bhk->bhv", S, kt))
        S = S + kt[..., None] * u[:, :, None, :]
        out[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, qt)
    return out, S, states


def gated_delta_rule_bwd(q, k, v, g, beta, dout, scale=None, doc_start=None, initial_state=None, d_final_state=None):
    """Gradients of sum(dout out) + sum(d_final_state final_state)."""
    q, k, v, g, beta, dout, initial_state, d_final_state = _f64(q, k, v, g, beta, dout, initial_state, d_final_state)
    B, L, Hk, K = q.shape
    Hv, V = v.shape[2:]
    r = Hv // Hk
    scale = K ** -0.5 if scale is None else scale
    start = _starts(B, L, doc_start, initial_state)
    S = np.zeros((B, Hv, K, V)) if initial_state is None else initial_state.copy()
    kept = []
    for t in range(L):
        kt = np.repeat(k[:, t], r, 1)
        decay = np.ones((B, Hv)) if g is None else np.exp(g[:, t])
        held = np.where(start[:, t, None, None, None], 0.0, decay[:, :, None, None] * S)
        miss = v[:, t] - np.einsum("bhkv,bhk->bhv", held, kt)
        S = held + kt[..., None] * (beta[:, t, :, None] * miss)[:, :, None, :]
        kept.append((decay, held, miss, S))
    dS = np.zeros((B, Hv, K, V)) if d_final_state is None else d_final_state.copy()
    dq, dk, dv = np.zeros((B, L, Hv, K)), np.zeros((B, L, Hv, K)), np.zeros((B, L, Hv, V))
    dg, dbeta = np.zeros((B, L, Hv)), np.zeros((B, L, Hv))
    for t in range(L - 1, -1, -1):
        decay, held, miss, S = kept[t]
        kt, qt, b, do = np.repeat(k[:, t], r, 1), np.repeat(q[:, t], r, 1), beta[:, t, :, None], scale * dout[:, t]
        dS = dS + qt[..., None] * do[:, :, None, :]
        dq[:, t] = np.einsum("bhkv,bhv->bhk", S, do)
        du = np.einsum("bhkv,bhk->bhv", dS, kt)
        dbeta[:, t] = (du * miss).sum(-1)
        dv[:, t] = b * du
        dk[:, t] = np.einsum("bhkv,bhv->bhk", dS, b * miss) - np.einsum("bhkv,bhv->bhk", held, b * du)
        dS = dS - kt[..., None] * (b * du)[:, :, None, :]
        dg[:, t] = (dS * held).sum((-1, -2))
        dS = np.where(start[:, t, None, None, None], 0.0, decay[:, :, None, None] * dS)
    res = {"dq": dq.reshape(B, L, Hk, r, K).sum(3), "dk": dk.reshape(B, L, Hk, r, K).sum(3), "dv": dv, "dg": dg,
           "dbeta": dbeta}
    if initial_state is not None:
        res["d_initial_state"] = dS
    return res


def _rotate(x, cos, sin, positions, interleaved):
    if cos is None:
        return x
    h = cos.shape[1]
    y = x.copy()
    first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    c, s = cos[positions][:, :, None], sin[positions][:, :, None]
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def head_norm(x, weight=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6, interleaved=False):
    """x (B, L, H, K) normed per head, weighted and rotated by the tables' rows of its positions (B, L)."""
    x, weight, cos, sin = _f64(x, weight, cos, sin)
    if cos is not None and positions is None:
        positions = np.broadcast_to(np.arange(x.shape[1]), x.shape[:2])
    size = (x * x).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1)
    y = x / np.sqrt(size + eps)
    return _rotate(y if weight is None else y * weight, cos, sin, positions, interleaved)


def head_norm_bwd(x, dy, weight=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6, interleaved=False):
    """(dx, dweight or None) of sum(dy head_norm(x))."""
    x, dy, weight, cos, sin = _f64(x, dy, weight, cos, sin)
    if cos is not None and positions is None:
        positions = np.broadcast_to(np.arange(x.shape[1]), x.shape[:2])
    n = x.shape[-1] if norm == "rms" else 1
    r = ((x * x).sum(-1, keepdims=True) / n + eps) ** -0.5
    d = _rotate(dy, cos, None if sin is None else -sin, positions, interleaved)
    dn = d if weight is None else d * weight
    dx = r * dn - x * r ** 3 * (dn * x).sum(-1, keepdims=True) / n
    return dx, None if weight is None else (d * x * r).sum((0, 1, 2))
