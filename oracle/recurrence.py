"""fp64 oracle of the gated linear recurrence and of the 8-bit activation
checkpoints (test infrastructure only; shares no code with the GPU path).

    r = sigmoid(gate_a), i = sigmoid(gate_x), log a = -c softplus(a_param) r
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,   out_t = h_t silu(z_t)

token by token, with h_{t-1} = 0 at a document start (token 0 starts one unless an
initial state is given, then only where doc_start marks it)."""

from __future__ import annotations

import numpy as np

CHUNK = 128
BLOCK = 64


def _sigmoid(v):
    with np.errstate(over="ignore"):   # e^-v = inf gives 0
        return 1.0 / (1.0 + np.exp(-v))


def _softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def _starts(shape, doc_start, initial_state):
    s = np.zeros(shape[:2], dtype=bool) if doc_start is None else np.asarray(doc_start) != 0
    s = s.copy()
    if initial_state is None and shape[1]:
        s[:, 0] = True
    return s


def _gates(x, gate_a, gate_x, a_param, c):
    r, i = _sigmoid(gate_a), _sigmoid(gate_x)
    log_a = -c * _softplus(a_param) * r
    return r, i, np.exp(log_a), np.sqrt(-np.expm1(2.0 * log_a)), i * x


def gated_recurrence(x, gate_a, gate_x, a_param, z=None, doc_start=None, c=8.0, initial_state=None):
    """(out, final_state, states): states (B, ceil(L / 128), D) enter tokens 0, 128, ..."""
    x, gate_a, gate_x, a_param, z, initial_state = _f64(x, gate_a, gate_x, a_param, z, initial_state)
    B, L, D = x.shape
    start = _starts(x.shape, doc_start, initial_state)
    _, _, a, w, v = _gates(x, gate_a, gate_x, a_param, c)
    h = np.zeros((B, D)) if initial_state is None else initial_state.copy()
    out = np.empty_like(x)
    states = np.empty((B, -(-L // CHUNK), D))
    for t in range(L):
        if t % CHUNK == 0:
            states[:, t // CHUNK] = h
        h = np.where(start[:, t, None], 0.0, a[:, t] * h) + w[:, t] * v[:, t]
        out[:, t] = h
    if z is not None:
        out = out * (z * _sigmoid(z))
    return out, h, states


def gated_recurrence_bwd(x, gate_a, gate_x, a_param, dout, z=None, doc_start=None, c=8.0, initial_state=None,
                         d_final_state=None, states=None):
    """Gradients of sum(dout * out) + sum(d_final_state * final_state).  With
    ``states`` the recurrence restarts from them every 128 tokens (their values are
    taken as the states there, the adjoint runs through)."""
    x, gate_a, gate_x, a_param, dout, z, initial_state, d_final_state, states = _f64(
        x, gate_a, gate_x, a_param, dout, z, initial_state, d_final_state, states)
    B, L, D = x.shape
    start = _starts(x.shape, doc_start, initial_state)
    r, i, a, w, v = _gates(x, gate_a, gate_x, a_param, c)
    h = np.zeros((B, D)) if initial_state is None else initial_state.copy()
    prev, cur = np.empty_like(x), np.empty_like(x)
    for t in range(L):
        if states is not None and t % CHUNK == 0:
            h = states[:, t // CHUNK]
        prev[:, t] = np.where(start[:, t, None], 0.0, h)
        h = a[:, t] * prev[:, t] + w[:, t] * v[:, t]
        cur[:, t] = h
    g = {}
    dy = dout
    if z is not None:
        sg = _sigmoid(z)
        g["dz"] = dout * cur * sg * (1.0 + z * (1.0 - sg))
        dy = dout * z * sg
    G = np.empty_like(x)
    e = np.zeros((B, D)) if d_final_state is None else d_final_state.copy()
    for t in range(L - 1, -1, -1):
        G[:, t] = dy[:, t] + e
        e = np.where(start[:, t, None], 0.0, a[:, t] * G[:, t])
    g["dx"] = G * w * i
    g["dgate_x"] = G * w * v * (1.0 - i)
    # d/d log a of w is -a^2 / w; its product with r stays finite where w -> 0
    rw = np.divide(r, w, out=np.zeros_like(w), where=w > 0)
    q = G * (r * a * prev - rw * a * a * v)
    g["dgate_a"] = -c * _softplus(a_param) * (1.0 - r) * q
    g["da_param"] = -c * _sigmoid(a_param) * q.sum((0, 1))
    if initial_state is not None:
        g["d_initial_state"] = e
    return g


def pack8(x):
    """Codes (..., D) int8 and scales (ceil(D / 64), ...) float32 of a float32 array: the
    format is defined in float32 arithmetic, every quotient and product rounded."""
    x = np.asarray(x, dtype=np.float32)
    D = x.shape[-1]
    q = np.zeros(x.shape, dtype=np.int8)
    scale = np.zeros((-(-D // BLOCK),) + x.shape[:-1], dtype=np.float32)
    for k in range(scale.shape[0]):
        xb = x[..., k * BLOCK:(k + 1) * BLOCK]
        with np.errstate(all="ignore"):
            m = np.maximum(np.abs(xb).max(-1), np.float32(2.0 ** -100))
            good = np.isfinite(xb).all(-1)
            inv = (np.float32(1.0) / m) * np.float32(127.0)
            scale[k] = np.where(good, m * (np.float32(1.0) / np.float32(127.0)), np.float32(np.nan))
            codes = np.rint(xb * inv[..., None])
        q[..., k * BLOCK:(k + 1) * BLOCK] = np.where(good[..., None], codes, 0).astype(np.int8)
    return q, scale


def unpack8(q, scale):
    """The values, float32."""
    D = q.shape[-1]
    s = np.moveaxis(scale, 0, -1).repeat(BLOCK, -1)[..., :D]
    return q.astype(np.float32) * s
