"""Pins of the gated recurrence's fp64 oracle (CPU): closed forms, invariants and
central finite differences of every gradient."""

import numpy as np
import pytest

from oracle import recurrence as R


def inputs(B, L, D, seed=0, z=True):
    g = np.random.default_rng(seed)
    v = {k: g.standard_normal((B, L, D)) for k in ("x", "gate_a", "gate_x")}
    v["z"] = g.standard_normal((B, L, D)) if z else None
    v["a_param"] = g.uniform(-4.0, -1.0, D)
    return v


def call(v, **kw):
    return R.gated_recurrence(v["x"], v["gate_a"], v["gate_x"], v["a_param"], v["z"], **kw)


def test_one_token_and_unrolled():
    v = inputs(2, 5, 3, z=False)
    out, fin, states = call(v)
    sig = lambda t: 1 / (1 + np.exp(-t))  # noqa: E731
    a = np.exp(-8.0 * np.log1p(np.exp(v["a_param"])) * sig(v["gate_a"]))
    b = np.sqrt(1 - a * a) * sig(v["gate_x"]) * v["x"]
    for t in range(5):
        h = sum(np.prod(a[:, s + 1:t + 1], axis=1) * b[:, s] for s in range(t + 1))
        np.testing.assert_allclose(out[:, t], h, rtol=1e-13)
    np.testing.assert_allclose(fin, out[:, -1])
    assert states.shape == (2, 1, 3) and not states.any()


def test_no_decay_and_full_decay():
    v = inputs(1, 6, 4, z=False)
    v["gate_a"][:] = -2000.0                       # r = 0: a = 1, the input's weight 0
    h0 = np.arange(4.0)[None]
    out, fin, _ = call(v, initial_state=h0)
    np.testing.assert_array_equal(out, np.broadcast_to(h0[:, None], out.shape))
    v = inputs(1, 6, 4, z=False)
    v["a_param"][:] = 500.0                        # a = 0: each token stands alone
    out, _, _ = call(v, initial_state=h0)
    np.testing.assert_allclose(out, v["x"] / (1 + np.exp(-v["gate_x"])), rtol=1e-12)


def test_documents_split_and_carry():
    v = inputs(2, 300, 3)
    start = np.zeros((2, 300), np.uint8)
    start[0, 140] = start[1, 128] = 1
    out, fin, states = call(v, doc_start=start)
    cut = {k: (None if a is None else a[:1, 140:]) if k != "a_param" else a for k, a in v.items()}
    np.testing.assert_array_equal(call(cut)[0], out[:1, 140:])
    head = {k: (a[:, :200] if k != "a_param" else a) for k, a in v.items()}
    tail = {k: (a[:, 200:] if k != "a_param" else a) for k, a in v.items()}
    o1, h1, _ = call(head, doc_start=start[:, :200])
    o2, h2, _ = call(tail, doc_start=start[:, 200:], initial_state=h1)
    np.testing.assert_array_equal(np.concatenate([o1, o2], 1), out)
    np.testing.assert_array_equal(h2, fin)
    o3, _, _ = R.gated_recurrence(*(v[k][:, 128:] for k in ("x", "gate_a", "gate_x")), v["a_param"], v["z"][:, 128:],
                                  doc_start=start[:, 128:], initial_state=states[:, 1])
    np.testing.assert_array_equal(o3, out[:, 128:])


@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("carry", [False, True])
def test_gradients_by_differences(z, carry):
    B, L, D = 2, 7, 3
    v = inputs(B, L, D, seed=3, z=z)
    g = np.random.default_rng(4)
    dout = g.standard_normal((B, L, D))
    start = np.zeros((B, L), np.uint8)
    start[0, 3] = start[1, 0] = 1
    v["initial_state"] = g.standard_normal((B, D)) if carry else None
    dfin = g.standard_normal((B, D)) if carry else None

    def loss(v):
        out, fin, _ = call(v, doc_start=start, initial_state=v["initial_state"])
        return (dout * out).sum() + (0.0 if dfin is None else (dfin * fin).sum())

    grads = R.gated_recurrence_bwd(v["x"], v["gate_a"], v["gate_x"], v["a_param"], dout, v["z"], start,
                                   initial_state=v["initial_state"], d_final_state=dfin)
    for k, name in (("x", "dx"), ("gate_a", "dgate_a"), ("gate_x", "dgate_x"), ("a_param", "da_param"), ("z", "dz"),
                    ("initial_state", "d_initial_state")):
        if v[k] is None:
            assert name not in grads
            continue
        fd = np.empty_like(v[k])
        # central differences with step h: h^2 / 6 of the third derivative (O(10)) plus
        # rounding 1e-16 * |loss| / h: below 1e-8 at h = 1e-5
        for idx in np.ndindex(*v[k].shape):
            keep = v[k][idx]
            v[k][idx] = keep + 1e-5
            up = loss(v)
            v[k][idx] = keep - 1e-5
            fd[idx] = (up - loss(v)) / 2e-5
            v[k][idx] = keep
        np.testing.assert_allclose(grads[name], fd, rtol=1e-6, atol=1e-7)


def test_gradients_from_states_equal_the_whole_row():
    v = inputs(1, 300, 2, seed=5)
    dout = np.random.default_rng(6).standard_normal((1, 300, 2))
    start = np.zeros((1, 300), np.uint8)
    start[0, [128, 200]] = 1
    _, _, states = call(v, doc_start=start)
    args = (v["x"], v["gate_a"], v["gate_x"], v["a_param"], dout, v["z"], start)
    one, two = R.gated_recurrence_bwd(*args), R.gated_recurrence_bwd(*args, states=states)
    for k in one:
        np.testing.assert_array_equal(one[k], two[k])


def test_pack_format():
    g = np.random.default_rng(7)
    x = (g.standard_normal((5, 150)) * np.exp(g.uniform(-20, 20, (5, 1)))).astype(np.float32)
    x[1] = 0.0
    x[2, 3] = np.nan
    x[3, 70] = np.inf
    q, s = R.pack8(x)
    v = R.unpack8(q, s)
    assert q.shape == (5, 150) and s.shape == (3, 5)
    assert not v[1].any()
    assert np.isnan(v[2, :64]).all() and np.isfinite(v[2, 64:]).all()
    assert np.isnan(v[3, 64:128]).all() and np.isfinite(v[3, :64]).all()
    for r in (0, 4):
        for k in range(3):
            b = slice(64 * k, min(150, 64 * k + 64))
            assert np.abs(q[r, b]).max() == 127
            # half a step, plus the float32 roundings of the scale, its inverse and two products
            assert (np.abs(v[r, b] - x[r, b]) <= s[k, r] * (0.5 + 4 * 127 * 2.0 ** -24)).all()
