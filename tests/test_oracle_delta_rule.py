"""Pins of the delta rule's and the head norms' oracle: closed forms, finite
differences, split rows."""

import numpy as np
import pytest

import oracle.delta_rule as R


def draw(B=2, L=9, Hk=2, Hv=4, K=5, V=3, seed=0, docs=True):
    r = np.random.default_rng(seed)
    d = dict(q=r.standard_normal((B, L, Hk, K)), k=r.standard_normal((B, L, Hk, K)) / np.sqrt(K),
             v=r.standard_normal((B, L, Hv, V)), g=-r.uniform(0.0, 1.0, (B, L, Hv)), beta=r.uniform(0, 1, (B, L, Hv)))
    d["doc_start"] = (r.random((B, L)) < 0.25).astype(np.uint8) if docs else None
    d["initial_state"] = r.standard_normal((B, Hv, K, V))
    return d


def test_one_token_writes_its_value():
    """With beta = 1 and a unit key the state answers the key with the value."""
    d = draw(L=1)
    d["k"] /= np.linalg.norm(d["k"], axis=-1, keepdims=True)
    d["beta"][:] = 1.0
    d["q"] = d["k"]
    out, _, _ = R.gated_delta_rule(**d, scale=1.0)
    np.testing.assert_allclose(out, d["v"], atol=1e-12)


def test_orthogonal_keys_are_linear_attention():
    """Keys that do not overlap: nothing is erased, outputs are the decayed sum of beta (q.k) v."""
    K = 6
    d = draw(L=K, K=K, docs=False)
    d["initial_state"] = None
    d["k"] = np.broadcast_to(np.eye(K)[None, :, None], d["k"].shape)
    out, _, _ = R.gated_delta_rule(**d, scale=0.5)
    q, k = (np.repeat(d[n], 2, 2) for n in ("q", "k"))
    for t in range(K):
        ref = 0.0
        for s in range(t + 1):
            w = np.exp(d["g"][:, s + 1:t + 1].sum(1)) * d["beta"][:, s] * (q[:, t] * k[:, s]).sum(-1)
            ref = ref + w[..., None] * d["v"][:, s]
        np.testing.assert_allclose(out[:, t], 0.5 * ref, atol=1e-12)


def test_equal_keys_keep_the_last_value():
    """beta = 1 and one unit key: each token replaces what the last one wrote."""
    d = draw(L=130, K=4, docs=False)
    d["initial_state"], d["g"] = None, None
    d["k"][:] = 0.5
    d["q"][:] = 0.5
    d["beta"][:] = 1.0
    out, _, _ = R.gated_delta_rule(**d, scale=1.0)
    np.testing.assert_allclose(out, d["v"], atol=1e-10)


def test_split_rows_and_documents():
    d = draw(L=140)
    out, S, states = R.gated_delta_rule(**d)
    head = {n: d[n] if d[n].shape[1] != 140 else d[n][:, :64] for n in d}
    o1, S1, _ = R.gated_delta_rule(**head)
    tail = {n: d[n] if d[n].shape[1] != 140 else d[n][:, 64:] for n in d}
    o2, S2, _ = R.gated_delta_rule(**dict(tail, initial_state=S1))
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), out, atol=1e-12)
    np.testing.assert_allclose(S2, S, atol=1e-12)
    np.testing.assert_allclose(states[:, :, 1], S1, atol=1e-12)
    t = int(np.flatnonzero(d["doc_start"][0])[-1])     # the last document of row 0 on its own
    alone = {n: d[n][:1, t:] for n in ("q", "k", "v", "g", "beta")}
    o3, S3, _ = R.gated_delta_rule(**alone)
    np.testing.assert_allclose(o3[0], out[0, t:], atol=1e-12)
    np.testing.assert_allclose(S3[0], S[0], atol=1e-12)


@pytest.mark.parametrize("docs,carry,decay", [(True, True, True), (False, False, True), (True, True, False)])
def test_gradients_by_differences(docs, carry, decay):
    d = draw(docs=docs, seed=3)
    if not carry:
        d["initial_state"] = None
    if not decay:
        d["g"] = None
    r = np.random.default_rng(5)
    out, S, _ = R.gated_delta_rule(**d)
    do, dS = r.standard_normal(out.shape), r.standard_normal(S.shape)

    def loss(x):
        o, s, _ = R.gated_delta_rule(**x)
        return (o * do).sum() + (s * dS).sum()

    grads = R.gated_delta_rule_bwd(**d, dout=do, d_final_state=dS)
    names = {"q": "dq", "k": "dk", "v": "dv", "g": "dg", "beta": "dbeta", "initial_state": "d_initial_state"}
    for n, gn in names.items():
        if d[n] is None:
            continue
        for i in r.choice(d[n].size, min(40, d[n].size), replace=False):
            at = np.unravel_index(i, d[n].shape)
            up, down = d[n].copy(), d[n].copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            num = (loss(dict(d, **{n: up})) - loss(dict(d, **{n: down}))) / 2e-5
            assert abs(num - grads[gn][at]) <= 1e-7 * max(1.0, abs(num)), (n, at, num, grads[gn][at])


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_head_norm(norm, interleaved, weight):
    r = np.random.default_rng(1)
    x = r.standard_normal((2, 4, 3, 7))
    kw = dict(norm=norm, interleaved=interleaved, eps=1e-3)
    kw["weight"] = r.standard_normal(7) if weight else None
    ang = r.uniform(0, 6, (9, 2))
    kw["cos"], kw["sin"] = np.cos(ang), np.sin(ang)
    kw["positions"] = r.integers(0, 9, (2, 4))
    y = R.head_norm(x, **kw)
    if not weight:   # a rotation keeps the norm
        size = np.linalg.norm(x, axis=-1) / (np.sqrt(7) if norm == "rms" else 1)
        want = np.linalg.norm(x, axis=-1) / np.sqrt(size ** 2 + 1e-3)
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), want, rtol=1e-12)
    a, b = (0, 1) if interleaved else (0, 2)          # the first pair as a complex number
    un = R.head_norm(x, **dict(kw, cos=None, sin=None))
    z = (un[..., a] + 1j * un[..., b]) * np.exp(1j * ang[kw["positions"], 0])[..., None]
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-12)
    np.testing.assert_allclose(y[..., 4:], un[..., 4:])
    dy = r.standard_normal(y.shape)
    dx, dw = R.head_norm_bwd(x, dy, **kw)
    for i in range(x.size):
        at = np.unravel_index(i, x.shape)
        up, down = x.copy(), x.copy()
        up[at] += 1e-6
        down[at] -= 1e-6
        num = ((R.head_norm(up, **kw) - R.head_norm(down, **kw)) * dy).sum() / 2e-6
        assert abs(num - dx[at]) <= 1e-7 * max(1.0, abs(num))
    if weight:
        np.testing.assert_allclose(dw, [((R.head_norm(x, **dict(kw, weight=np.eye(7)[i]))) * dy).sum() for i in range(7)])
