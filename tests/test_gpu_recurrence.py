"""Gated linear recurrence on the GPU against the fp64 oracle.

Tolerances, set from the arithmetic before the first run.  Every step of a channel
rounds a product and a sum (2 x 2^-24) and takes a decay that is off by a few
2^-24; an error lives as long as the state does (1 / (1 - a), some hundreds of
tokens here), so errors add to a few hundred times 2^-22 at worst and to the root
of that as they come: 1e-4 relative with a floor of 1e-4 of the output's rms, the
bound this library states for float32.  bf16 outputs round once more, by at most
2^-8 relative."""

import numpy as np
import pytest

import oracle.recurrence as R
from workloads import bf16_round
from workloads.device import to_dev, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    import torch

    import selective_state_space_23_amd as s
    if not torch.cuda.is_available():
        pytest.fail("no GPU")
    return s


def close(got, ref, dtype, what):
    got = to_host(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite"
    if got.size == 0:
        return
    floor = 1e-4 * np.sqrt(np.mean(ref ** 2))
    tol = (1e-4 + (2.0 ** -8 if dtype == "bf16" else 0.0)) * np.abs(ref) + floor
    err = np.abs(got - ref)
    i = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())} of {err.size} off, worst at {i}: {got[i]} for {ref[i]}"


def draw(B, L, D, dtype, z=True, docs=None, carry=False, seed=0, spread=1.0):
    g = np.random.default_rng(seed)
    rnd = bf16_round if dtype == "bf16" else (lambda a: a)
    v = {k: rnd((s * g.standard_normal((B, L, D))).astype(np.float32))
         for k, s in (("x", 1.0), ("gate_a", spread), ("gate_x", spread), ("z", 1.0), ("dout", 1.0))}
    if not z:
        v["z"] = None
    a1 = g.uniform(0.9, 0.999, D)                       # the decay at r = 1
    v["a_param"] = np.log(np.expm1(-np.log(a1) / 8.0)).astype(np.float32)
    v["doc_start"] = None
    if docs is not None:
        v["doc_start"] = (g.random((B, L)) < 1.0 / docs).astype(np.uint8)
        if L:
            v["doc_start"][::2, 0] = 1
    v["initial_state"] = g.standard_normal((B, D)).astype(np.float32) if carry else None
    v["d_final_state"] = g.standard_normal((B, D)).astype(np.float32) if carry else None
    return v


def dev(v, dtype):
    import torch

    up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    d = {k: None if v[k] is None else to_dev(v[k], dtype) for k in ("x", "gate_a", "gate_x", "z", "dout")}
    d.update({k: up(v[k]) for k in ("a_param", "doc_start", "initial_state", "d_final_state")})
    return d


def forward(ssm, d, **kw):
    return ssm.gated_recurrence_fwd(d["x"], d["gate_a"], d["gate_x"], d["a_param"], d["z"], d["doc_start"],
                                    initial_state=d["initial_state"], **kw)


def backward(ssm, d, **kw):
    return ssm.gated_recurrence_bwd(d["x"], d["gate_a"], d["gate_x"], d["a_param"], d["dout"], d["z"], d["doc_start"],
                                    initial_state=d["initial_state"], d_final_state=d["d_final_state"], **kw)


def oracle_fwd(v):
    return R.gated_recurrence(v["x"], v["gate_a"], v["gate_x"], v["a_param"], v["z"], v["doc_start"],
                              initial_state=v["initial_state"])


def oracle_bwd(v, **kw):
    return R.gated_recurrence_bwd(v["x"], v["gate_a"], v["gate_x"], v["a_param"], v["dout"], v["z"], v["doc_start"],
                                  initial_state=v["initial_state"], d_final_state=v["d_final_state"], **kw)


def equal(a, b):
    import torch

    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# lengths around the 128-token tile and the 4-token lanes, widths around the
# 64-channel tile and the quads, several rows
SHAPES = [(1, 1, 1), (2, 3, 4), (1, 127, 64), (2, 128, 68), (1, 129, 63), (3, 300, 70), (1, 700, 36), (2, 1025, 132),
          (5, 17, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("B,L,D", SHAPES)
def test_forward(ssm, B, L, D, z, dtype):
    for docs, carry in ((None, False), (40, True)):
        v = draw(B, L, D, dtype, z, docs, carry, seed=L + D)
        out, fin, kept = forward(ssm, dev(v, dtype), save="states")
        ref = oracle_fwd(v)
        close(out, ref[0], dtype, "out")
        close(fin, ref[1], "f32", "final_state")
        close(kept["states"], ref[2], "f32", "states")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("B,L,D", SHAPES)
def test_backward(ssm, B, L, D, z, dtype):
    for docs, carry in ((None, False), (40, True)):
        v = draw(B, L, D, dtype, z, docs, carry, seed=L + D + 1)
        d = dev(v, dtype)
        ref = oracle_bwd(v)
        g = backward(ssm, d)
        assert set(g) == set(ref)
        for k in ref:
            close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
        # from the forward's states: the same numbers, whoever computed the states
        kept = forward(ssm, d, save="states")[2]
        g2 = backward(ssm, d, states=kept["states"])
        for k in g:
            assert equal(g[k], g2[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,z", [(1, 1, 1, True), (2, 129, 63, True), (3, 300, 70, False), (1, 513, 200, True)])
def test_packed_training_step(ssm, B, L, D, z, dtype):
    v = draw(B, L, D, dtype, z, 50, True, seed=L)
    d = dev(v, dtype)
    out, fin, kept = forward(ssm, d, save="packed")
    plain = forward(ssm, d)
    assert equal(out, plain[0]) and equal(fin, plain[1])
    seen = dict(v)
    for k in ("x", "gate_a", "gate_x") + (("z",) if z else ()):
        q, s = R.pack8(v[k])
        assert np.array_equal(kept[k].q.cpu().numpy(), q) and np.array_equal(kept[k].scale.cpu().numpy(), s), k
        p = ssm.activation_pack(d[k])
        assert equal(p.q, kept[k].q) and equal(p.scale, kept[k].scale), k
        seen[k] = R.unpack8(q, s)
    dp = dict(d, **{k: kept.get(k) for k in ("x", "gate_a", "gate_x", "z")})
    for states in (kept["states"], None):
        ref = oracle_bwd(seen, states=None if states is None else states.cpu().numpy())
        g = backward(ssm, dp, states=states)
        assert set(g) == set(ref)
        for k in ref:
            close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
    if dtype == "f32":
        # float32 values of the checkpoints, given as tensors: the same gradients bit for bit
        du = dict(d, **{k: ssm.activation_unpack(kept[k], d["x"].dtype) for k in kept if k != "states"})
        a, b = backward(ssm, dp, states=kept["states"]), backward(ssm, du, states=kept["states"])
        for k in a:
            assert equal(a[k], b[k]), k


# widths: odd; quads whose rows do not lie on 16 bytes; rows that do
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("D", [701, 700, 704])
def test_more_tiles_than_workgroups(ssm, D, z, dtype):
    """594 tiles of 128 tokens and 64 channels: workgroups take several, one after the other."""
    B, L = 2, 3333
    v = draw(B, L, D, dtype, z, 300, True, seed=D)
    d = dev(v, dtype)
    out, fin, kept = forward(ssm, d, save="packed")
    ref = oracle_fwd(v)
    close(out, ref[0], dtype, "out")
    close(fin, ref[1], "f32", "final_state")
    close(kept["states"], ref[2], "f32", "states")
    plain = forward(ssm, d, save="states")
    assert equal(out, plain[0]) and equal(fin, plain[1]) and equal(kept["states"], plain[2]["states"])
    ref = oracle_bwd(v)
    g = backward(ssm, d)
    g2 = backward(ssm, d, states=kept["states"])
    for k in ref:
        close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
        assert equal(g[k], g2[k]), k
    seen = dict(v)
    for k in ("x", "gate_a", "gate_x") + (("z",) if z else ()):
        p = ssm.activation_pack(d[k])
        assert equal(p.q, kept[k].q) and equal(p.scale, kept[k].scale), k
        seen[k] = R.unpack8(*R.pack8(v[k]))
    ref = oracle_bwd(seen, states=kept["states"].cpu().numpy())
    dp = dict(d, **{k: kept.get(k) for k in ("x", "gate_a", "gate_x", "z")})
    g = backward(ssm, dp, states=kept["states"])
    for k in ref:
        close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
    ref = oracle_bwd(seen)
    g = backward(ssm, dp)
    for k in ref:
        close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_document_edges(ssm, dtype):
    """Starts on and around tile and lane edges, every token a start, and a start at token 0."""
    B, L, D = 3, 400, 12
    v = draw(B, L, D, dtype, True, 50, True, seed=9)
    v["doc_start"][:] = 0
    v["doc_start"][0, [0, 3, 4, 15, 16, 127, 128, 129, 255, 256, 383, 384, 399]] = 1
    v["doc_start"][1] = 1
    d = dev(v, dtype)
    out, fin, kept = forward(ssm, d, save="states")
    ref = oracle_fwd(v)
    close(out, ref[0], dtype, "out")
    close(fin, ref[1], "f32", "final")
    close(kept["states"], ref[2], "f32", "states")
    g, gr = backward(ssm, d, states=kept["states"]), oracle_bwd(v)
    for k in gr:
        close(g[k], gr[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
    assert not g["d_initial_state"][:2].any()                # token 0 starts a document there
    # any nonzero byte marks a start, and a bool mask is the same
    import torch
    other = dict(d, doc_start=d["doc_start"] * 255)
    assert equal(forward(ssm, other)[0], out)
    assert equal(forward(ssm, dict(d, doc_start=d["doc_start"].bool()))[0], out)
    assert d["doc_start"].dtype == torch.uint8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_values_stay_in_their_document(ssm, dtype):
    """A NaN or an infinity reaches no token of another document, forwards or backwards."""
    B, L, D = 1, 520, 8
    v = draw(B, L, D, dtype, True, None, True, seed=11)
    v["doc_start"] = np.zeros((B, L), np.uint8)
    v["doc_start"][0, [130, 300]] = 1
    d = dev(v, dtype)
    good_out, good_fin, kept = forward(ssm, d, save="states")
    good = backward(ssm, d)
    for bad in (float("inf"), float("nan")):
        e = {k: None if t is None else t.clone() for k, t in d.items()}
        e["x"][0, 200, 1] = bad
        e["gate_a"][0, 210, 2] = float("nan")
        e["dout"][0, 250, 3] = bad
        out, fin, _ = forward(ssm, e, save="states")
        assert equal(out[:, :130], good_out[:, :130]) and equal(out[:, 300:], good_out[:, 300:]) and equal(fin, good_fin)
        assert not out[0, 200:300, 1].float().isfinite().any() and not out[0, 210:300, 2].float().isfinite().any()
        g = backward(ssm, e)
        for k in ("dx", "dgate_a", "dgate_x", "dz"):
            assert equal(g[k][:, :130], good[k][:, :130]) and equal(g[k][:, 300:], good[k][:, 300:]), k
        assert equal(g["d_initial_state"], good["d_initial_state"])
        assert not g["dx"][0, 130:251, 3].float().isfinite().any()
        # the state entering the row, and the gradient entering it from the right
        e = dict(d, initial_state=torch_full_like(d["initial_state"], bad))
        e["doc_start"] = d["doc_start"].clone()
        e["doc_start"][0, 0] = 1
        assert forward(ssm, e)[0].float().isfinite().all()
        e = dict(d, d_final_state=torch_full_like(d["d_final_state"], bad))
        g = backward(ssm, e)
        for k in ("dx", "dgate_a", "dgate_x", "dz"):
            assert equal(g[k][:, :300], good[k][:, :300]), k


def torch_full_like(t, v):
    import torch

    return torch.full_like(t, v)


def test_saturated_gates(ssm):
    """Gates far out, decays at and near 0 and 1: no NaN, and what float32 can hold."""
    B, L, D = 1, 200, 64
    v = draw(B, L, D, "f32", True, None, True, seed=13, spread=12.0)
    v["a_param"][:8] = [-90.0, -40.0, -20.0, -10.0, 0.0, 5.0, 20.0, 60.0]
    v["gate_a"][0, :40] = np.float32(-60.0)
    v["gate_a"][0, 40:60] = np.float32(60.0)
    v["gate_a"][0, 60:70] = np.float32(-200.0)       # r = 0 in float32: nothing enters, nothing decays
    v["gate_x"][0, 50:90] = np.float32(-200.0)
    d = dev(v, "f32")
    out, fin, kept = forward(ssm, d, save="states")
    ref = oracle_fwd(v)
    close(out, ref[0], "f32", "out")
    close(fin, ref[1], "f32", "final")
    g, gr = backward(ssm, d), oracle_bwd(v)
    for k in ("dx", "dgate_a", "dgate_x", "dz", "d_initial_state"):
        close(g[k], gr[k], "f32", k)
    assert g["da_param"].isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 70])
def test_strides_and_alignment(ssm, dtype, D):
    """Slices of one projection, odd strides and unaligned buffers: the same bits as dense inputs."""
    import torch

    B, L = 2, 260
    v = draw(B, L, D, dtype, True, 60, True, seed=15)
    d = dev(v, dtype)
    want = forward(ssm, d, save="packed")
    grads = backward(ssm, d)
    names = ("x", "gate_a", "gate_x", "z", "dout")
    for pad in (0, 3, 4):
        proj = torch.randn(B, L, 5 * D + pad, device="cuda").to(d["x"].dtype)
        e = dict(d)
        for i, n in enumerate(names):
            e[n] = proj[..., i * D:(i + 1) * D]
            e[n].copy_(d[n])
        before = proj.clone()
        got = forward(ssm, e, save="packed")
        assert equal(got[0], want[0]) and equal(got[1], want[1]) and equal(got[2]["states"], want[2]["states"])
        for n in ("x", "gate_a", "gate_x", "z"):
            assert equal(got[2][n].q, want[2][n].q) and equal(got[2][n].scale, want[2][n].scale)
            p = ssm.activation_pack(e[n])
            assert equal(p.q, want[2][n].q) and equal(p.scale, want[2][n].scale)
        g = backward(ssm, e)
        for k in grads:
            assert equal(g[k], grads[k]), (pad, k)
        assert equal(proj, before)
    # buffers one element past an aligned address
    def shifted(t):
        if t is None:
            return None
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    e = {k: shifted(t) for k, t in d.items()}
    guard = torch.full((B * L * D + 8,), 7.0, dtype=d["x"].dtype, device="cuda")
    out = guard[3:3 + B * L * D].view(B, L, D)
    got = forward(ssm, e, out=out, save="packed")
    assert equal(out, want[0]) and equal(got[1], want[1])
    assert (guard[:3] == 7).all() and (guard[3 + B * L * D:] == 7).all()
    kept = {n: ssm.PackedActivation(shifted(p.q), shifted(p.scale)) for n, p in got[2].items() if n != "states"}
    g = backward(ssm, e, grads={k: shifted(torch.empty_like(t)) for k, t in grads.items()})
    for k in grads:
        assert equal(g[k], grads[k]), k
    a = backward(ssm, dict(d, **{n: want[2][n] for n in kept}), states=want[2]["states"])
    b = backward(ssm, dict(e, **kept), states=shifted(want[2]["states"]))
    for k in a:
        assert equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_behind_are_left_alone(ssm, dtype):
    """Calls on the first rows and channels of larger buffers write nothing behind them."""
    import torch

    B, L, D = 2, 130, 68
    v = draw(B, L, D, dtype, True, 60, True, seed=17)
    d = dev(v, dtype)
    bufs = {}

    def room(name, shape, dt):
        n = int(np.prod(shape))
        bufs[name] = (torch.full((n + 64,), 3.0, device="cuda").to(dt), n)
        return bufs[name][0][:n].view(shape)

    dt, f32 = d["x"].dtype, torch.float32
    nb = -(-D // 64)
    save = {"states": room("states", (B, 2, D), f32)}
    for n in ("x", "gate_a", "gate_x", "z"):
        save[n] = ssm.PackedActivation(room(n + "q", (B, L, D), torch.int8), room(n + "s", (nb, B, L), f32))
    forward(ssm, d, out=room("out", (B, L, D), dt), final_state=room("fin", (B, D), f32), save=save)
    grads = {k: room(k, (B, L, D), dt) for k in ("dx", "dgate_a", "dgate_x", "dz")}
    grads["da_param"] = room("da_param", (D,), f32)
    grads["d_initial_state"] = room("d_initial_state", (B, D), f32)
    backward(ssm, d, grads=grads)
    backward(ssm, dict(d, **{n: save[n] for n in ("x", "gate_a", "gate_x", "z")}), states=save["states"], grads=grads)
    for name, (t, n) in bufs.items():
        assert (t[n:].float() == 3.0).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_continues_the_prefill(ssm, dtype):
    import torch

    B, L, D = 3, 140, 70
    v = draw(B, L, D, dtype, True, 30, True, seed=19)
    d = dev(v, dtype)
    ref = oracle_fwd(v)
    n = 133
    head = dict(d, **{k: d[k][:, :n].contiguous() for k in ("x", "gate_a", "gate_x", "z", "doc_start")})
    state = forward(ssm, head)[1]
    for t in range(n, L):
        args = [d[k][:, t] for k in ("x", "gate_a", "gate_x")]       # rows L * D apart
        out = ssm.gated_recurrence_update(state, *args, d["a_param"], d["z"][:, t], reset=d["doc_start"][:, t].contiguous())
        close(out, ref[0][:, t], dtype, f"token {t}")
    close(state, ref[1], "f32", "state")
    # a reset row forgets even a NaN; the others keep theirs
    state[:] = float("nan")
    reset = torch.tensor([True, False, True], device="cuda")
    ssm.gated_recurrence_update(state, *[d[k][:, 0].contiguous() for k in ("x", "gate_a", "gate_x")], d["a_param"],
                                reset=reset)
    assert state[[0, 2]].isfinite().all() and state[1].isnan().all()


@pytest.mark.parametrize("B,D,dtype", [(1, 1, "f32"), (5, 63, "bf16"), (3, 260, "f32"), (1027, 1022, "f32"),
                                       (1029, 1026, "bf16"), (259, 4104, "bf16"), (65535, 17, "f32"), (8193, 128, "bf16")])
def test_update_of_many_rows(ssm, B, D, dtype):
    """Rows and widths that leave threads and groups of rows partly used, also of
    inputs sliced out of one tensor; a row's result does not depend on the others."""
    import torch

    v = draw(B, 1, D, dtype, True, None, True, seed=23)
    d = dev(v, dtype)
    ref = oracle_fwd(v)
    names = ("x", "gate_a", "gate_x", "z")
    dense = [d[n][:, 0] for n in names]
    sliced = torch.cat(dense, 1).split(D, 1)
    got = []
    for x, ga, gx, z in (dense, sliced):
        guard = torch.full((2 * B * D,), 5.0, device="cuda")
        state = guard[: B * D].view(B, D)
        state.copy_(d["initial_state"])
        out = ssm.gated_recurrence_update(state, x, ga, gx, d["a_param"], z)
        close(out, ref[0][:, 0], dtype, "out")
        close(state, ref[1], "f32", "state")
        assert (guard[B * D :] == 5.0).all()
        got.append((out, state))
    assert equal(got[0][0], got[1][0]) and equal(got[0][1], got[1][1])
    rows = [0, B // 2, B - 1]
    state = d["initial_state"][rows].contiguous()
    out = ssm.gated_recurrence_update(state, *[t[rows].contiguous() for t in dense[:3]], d["a_param"], dense[3][rows].contiguous())
    assert equal(out, got[0][0][rows]) and equal(state, got[0][1][rows])


def test_split_rows(ssm):
    """A row cut in two: states carried forwards, gradients backwards."""
    B, L, D, n = 2, 500, 40, 201
    v = draw(B, L, D, "f32", True, 80, True, seed=21)
    d = dev(v, "f32")
    cut = lambda s: dict(d, **{k: d[k][:, s].contiguous() for k in ("x", "gate_a", "gate_x", "z", "dout", "doc_start")})  # noqa: E731
    head, tail = cut(slice(0, n)), cut(slice(n, L))
    o1, h1 = forward(ssm, head)
    tail["initial_state"] = h1
    o2, h2 = forward(ssm, tail)
    ref, gr = oracle_fwd(v), oracle_bwd(v)
    close(o1, ref[0][:, :n], "f32", "head")
    close(o2, ref[0][:, n:], "f32", "tail")
    close(h2, ref[1], "f32", "final")
    g2 = backward(ssm, tail)
    head["d_final_state"] = g2["d_initial_state"]
    g1 = backward(ssm, head)
    for k in ("dx", "dgate_a", "dgate_x", "dz"):
        close(g1[k], gr[k][:, :n], "f32", k)
        close(g2[k], gr[k][:, n:], "f32", k)
    close(g1["da_param"] + g2["da_param"], gr["da_param"], "f32", "da_param")
    close(g1["d_initial_state"], gr["d_initial_state"], "f32", "d_initial_state")


def test_repeats_and_streams(ssm):
    """The same bits every time, with work on another stream than the default one and two calls at once."""
    import torch

    v = draw(2, 2000, 132, "bf16", True, 300, True, seed=23)
    d = dev(v, "bf16")

    def step():
        out, fin, kept = forward(ssm, d, save="packed")
        g = backward(ssm, dict(d, **{k: kept[k] for k in ("x", "gate_a", "gate_x", "z")}), states=kept["states"])
        return [out, fin, kept["states"], *g.values(), *backward(ssm, d).values()]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    for r in [step(), *got]:
        assert all(equal(a, b) for a, b in zip(r, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(1, 9000, 1), (1, 5000, 68), (3, 4200, 64), (1, 4096, 200)])
def test_few_long_chains(ssm, B, L, D, dtype):
    """Rows of 32 tiles and more over few channels: values handed on several tiles at a time."""
    v = draw(B, L, D, dtype, True, 2000, True, seed=L + D)
    d = dev(v, dtype)
    out, fin, kept = forward(ssm, d, save="packed")
    ref = oracle_fwd(v)
    close(out, ref[0], dtype, "out")
    close(fin, ref[1], "f32", "final_state")
    close(kept["states"], ref[2], "f32", "states")
    ref = oracle_bwd(v)
    g, g2 = backward(ssm, d), backward(ssm, d, states=kept["states"])
    for k in ref:
        close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
        assert equal(g[k], g2[k]), k
    dp = dict(d, **{k: kept[k] for k in ("x", "gate_a", "gate_x", "z")})
    seen = dict(v, **{k: R.unpack8(*R.pack8(v[k])) for k in ("x", "gate_a", "gate_x", "z")})
    ref = oracle_bwd(seen)
    g = backward(ssm, dp)
    for k in ref:
        close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)


def test_two_calls_at_once(ssm):
    """Calls with workspaces of their own, under way together on two streams and from
    two captured graphs, each larger than the card holds at a time."""
    import torch

    ds = [dev(draw(2, 3333, 704, "bf16", True, 300, True, seed=s), "bf16") for s in (31, 32)]

    def step(d):
        out, fin, kept = forward(ssm, d, save="packed")
        g = backward(ssm, dict(d, **{k: kept[k] for k in ("x", "gate_a", "gate_x", "z")}), states=kept["states"])
        return [out, fin, *g.values()]

    want = [step(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    graphs, held = [], []
    for s, d in zip(streams, ds):
        with torch.cuda.stream(s):
            step(d)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held.append(step(d))
        graphs.append(graph)
    for _ in range(3):
        got = []
        for s, d in zip(streams, ds):
            with torch.cuda.stream(s):
                got.append(step(d))
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, held):
            assert all(equal(p, q) for p, q in zip(a, b)) and all(equal(p, q) for p, q in zip(a, c))


def test_captured_training_step(ssm):
    """Forward, backward and a decode step in one graph, replayed on new inputs with eager work between."""
    import torch

    B, L, D = 2, 700, 96
    a, b = (dev(draw(B, L, D, "bf16", True, 90, True, seed=s), "bf16") for s in (25, 26))
    d = {k: t.clone() for k, t in a.items()}
    state = torch.zeros(B, D, device="cuda")

    def step(state):
        out, fin, kept = forward(ssm, d, save="packed")
        g = backward(ssm, dict(d, **{k: kept[k] for k in ("x", "gate_a", "gate_x", "z")}), states=kept["states"])
        last = ssm.gated_recurrence_update(state, *[d[k][:, 0] for k in ("x", "gate_a", "gate_x")], d["a_param"])
        return [out, fin, last, *g.values()]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(state.clone())
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(state)
    for src in (a, b, a, b):
        for k in d:
            d[k].copy_(src[k])
        state.copy_(src["initial_state"])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res] + [state.clone()]
        st = src["initial_state"].clone()
        want = step(st) + [st]
        torch.cuda.synchronize()
        assert all(equal(p, q) for p, q in zip(got, want))


def test_empty_calls(ssm):
    import torch

    v = draw(2, 0, 6, "f32", True, None, True)
    d = dev(v, "f32")
    out, fin, kept = forward(ssm, d, save="packed")
    assert out.shape == (2, 0, 6) and equal(fin, d["initial_state"]) and kept["states"].shape == (2, 0, 6)
    g = backward(ssm, d)
    assert equal(g["d_initial_state"], d["d_final_state"]) and not g["da_param"].any()
    d["initial_state"] = d["d_final_state"] = None
    assert not forward(ssm, d)[1].any()
    d = dev(draw(0, 5, 6, "f32", True), "f32")
    assert forward(ssm, d)[0].shape == (0, 5, 6)
    assert not backward(ssm, d)["da_param"].any()
    with pytest.raises(ValueError):
        ssm.gated_recurrence_fwd(torch.zeros(1, 2, 3), *[torch.zeros(1, 2, 3)] * 2, torch.zeros(3))


def test_refusals_of_the_binding(ssm):
    d = dev(draw(2, 20, 8, "f32", True, None, True), "f32")
    kept = forward(ssm, d, save="packed")[2]
    with pytest.raises(ValueError, match="all tensors or all"):
        backward(ssm, dict(d, x=kept["x"]))
    with pytest.raises(ValueError, match="save"):
        forward(ssm, d, save="everything")
    with pytest.raises(ValueError, match="together"):
        forward(ssm, d, save={"x": kept["x"]})
    with pytest.raises(ValueError, match="unknown"):
        forward(ssm, d, save={"y": kept["x"]})
    with pytest.raises(ssm.MambaArgumentError):
        ssm.gated_recurrence_fwd(d["x"], d["gate_a"], d["gate_x"], d["a_param"], c=0.0)
    with pytest.raises(ssm.MambaArgumentError):
        ssm.gated_recurrence_update(d["initial_state"], d["x"][:, 0], d["gate_a"][:, 0], d["gate_x"][:, 0],
                                    d["a_param"], out=d["initial_state"])
    with pytest.raises(ssm.MambaArgumentError, match="unsupported activation dtype"):
        ssm.gated_recurrence_fwd(*[d[k].double() for k in ("x", "gate_a", "gate_x")], d["a_param"])


def test_offsets_past_4_gib(ssm):
    """Tensors of 5.6 GB: a slice of the channels, run by itself, gives the same bits."""
    import torch

    B, L, D = 1, 140001, 20000
    g = torch.Generator(device="cuda").manual_seed(3)
    x, ga, gx = (torch.randn(B, L, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    ap = torch.full((D,), -4.0, device="cuda")
    out, fin, kept = ssm.gated_recurrence_fwd(x, ga, gx, ap, save="packed")
    grads = ssm.gated_recurrence_bwd(kept["x"], kept["gate_a"], kept["gate_x"], ap, out, states=kept["states"])
    s = slice(19968, 20000)                 # whole blocks of 64 up to the last, partial one
    part = [t[..., s] for t in (x, ga, gx)]
    o2, f2, k2 = ssm.gated_recurrence_fwd(*part, ap[s], save="packed")
    assert equal(o2, out[..., s]) and equal(f2, fin[..., s])
    for n in ("x", "gate_a", "gate_x"):
        assert equal(k2[n].q, kept[n].q[..., s]) and equal(k2[n].scale, kept[n].scale[312:])
    g2 = ssm.gated_recurrence_bwd(k2["x"], k2["gate_a"], k2["gate_x"], ap[s], o2, states=k2["states"])
    for k in g2:
        assert equal(g2[k], grads[k][..., s]), k


def nan_bits(t, index, sign):
    """Sets one element to a NaN with the given sign bit."""
    import torch

    if t.dtype == torch.bfloat16:
        t.view(torch.int16)[index] = -64 if sign else 0x7FC0
    else:
        t.view(torch.int32)[index] = -0x400000 if sign else 0x7FC00000


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [0, 1])
@pytest.mark.parametrize("z", [False, True])
def test_nan_gates_reach_their_document(ssm, dtype, sign, z):
    """A NaN decay, whatever its sign, spoils the gradients of the earlier tokens of its
    document, and of no other document: the oracle's finite elements are finite and
    close, the others are not."""
    B, L, D = 1, 520, 12
    v = draw(B, L, D, dtype, z, None, True, seed=41)
    v["doc_start"] = np.zeros((B, L), np.uint8)
    v["doc_start"][0, [130, 200, 300, 301, 381]] = 1
    d = dev(v, dtype)
    # in the lane of a start (behind, before, at it), inside a document, in a tile without
    # starts, in the row's last tile, and between two starts of one lane
    for c, t in enumerate((201, 199, 200, 210, 60, 519, 301, 300, 382, 383)):
        nan_bits(d["gate_a"], (0, t, c), sign)
        v["gate_a"][0, t, c] = np.nan
    states = forward(ssm, d, save="states")[2]["states"]
    ref = oracle_bwd(v)
    for kw in ({}, {"states": states}):
        g = backward(ssm, d, **kw)
        for k in ("dx", "dgate_a", "dgate_x", "d_initial_state", "da_param") + (("dz",) if z else ()):
            fine = np.isfinite(ref[k])
            assert np.array_equal(np.isfinite(to_host(g[k])), fine), k
            close(g[k][np_mask(fine, g[k])], ref[k][fine], dtype if g[k].dtype == d["x"].dtype else "f32", k)


def np_mask(m, like):
    import torch

    return torch.from_numpy(m).to(like.device)


def test_backward_of_many_short_rows(ssm):
    """4.26 million tiles of one token, more than one launch's 2^32 threads hold: the same bits
    as in calls of 4096 rows, and their da_param.

    x and dout are positive and no state enters, so that every term of da_param has one sign:
    a sum of 65535 of them, 4096 one after the other and 16 such sums, is off by at most
    4112 x 2^-24 of itself, the calls' own (256 and 16, 16 calls in 64 bits) by 272 x 2^-24."""
    import torch

    B, L, D = 65535, 1, 4160
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dout = (torch.rand(B, L, D, generator=g, device="cuda", dtype=torch.bfloat16) + 0.5 for _ in range(2))
    ga, gx = (torch.randn(B, L, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ap = torch.linspace(-5.0, -1.0, D, device="cuda")
    full = ssm.gated_recurrence_bwd(x, ga, gx, ap, dout)
    total = torch.zeros(D, dtype=torch.float64, device="cuda")
    for r in range(0, B, 4096):
        s = slice(r, r + 4096)
        part = ssm.gated_recurrence_bwd(x[s], ga[s], gx[s], ap, dout[s])
        for k in ("dx", "dgate_a", "dgate_x"):
            assert equal(full[k][s], part[k]), (r, k)
        total += part["da_param"].double()
    assert total.abs().min() > 0
    assert ((full["da_param"].double() - total).abs() <= 4400 * 2.0 ** -24 * total.abs()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1024, 1022])
def test_step_on_columns_of_long_rows(ssm, dtype, D):
    """One token of (B, L, D) tensors whose rows lie 2.1 million elements and more apart."""
    import torch

    B, L, t = 3, 2100, 2099
    v = draw(B, 1, D, dtype, True, None, True, seed=45)
    d = dev(v, dtype)
    names = ("x", "gate_a", "gate_x", "z")
    long = {n: torch.zeros(B, L, D, dtype=d["x"].dtype, device="cuda") for n in names}
    for n in names:
        long[n][:, t] = d[n][:, 0]
    got = []
    for x, ga, gx, z in ([d[n][:, 0] for n in names], [long[n][:, t] for n in names]):
        state = d["initial_state"].clone()
        got.append((ssm.gated_recurrence_update(state, x, ga, gx, d["a_param"], z), state))
    ref = oracle_fwd(v)
    close(got[1][0], ref[0][:, 0], dtype, "out")
    close(got[1][1], ref[1], "f32", "state")
    assert equal(got[0][0], got[1][0]) and equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 67])
def test_gradients_of_far_gates(ssm, dtype, D):
    """Gates of 10 to 16 and -16 to -10: every element of the gate gradients to its own size.

    Every token starts a document and there is no z, so that both gradients are products:
    dgate_x = dout w i x (1 - i), dgate_a = -c softplus (1 - r) r dout (-a^2 i x / w).  Their factors
    round some 2^-24 each, 30 of them at most, and an exponential of 16 log2(e) = 23
    (rounded by 2^-24 of it) is off by 23 x 0.7 x 2^-24, twice where both gates enter: 64 x 2^-24."""
    B, L = 2, 140
    v = draw(B, L, D, dtype, False, None, False, seed=43)
    g = np.random.default_rng(44)
    for n in ("gate_a", "gate_x"):
        far = (g.uniform(10, 16, (B, L, D)) * g.choice([-1.0, 1.0], (B, L, D))).astype(np.float32)
        v[n] = bf16_round(far) if dtype == "bf16" else far
    v["doc_start"] = np.ones((B, L), np.uint8)
    got, ref = backward(ssm, dev(v, dtype)), oracle_bwd(v)
    rtol = 64 * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    for k in ("dx", "dgate_x", "dgate_a"):
        err = np.abs(to_host(got[k]) - ref[k]) / np.abs(ref[k])
        assert err.max() <= rtol, f"{k}: off by {err.max()} of the element, {int((err > rtol).sum())} of {err.size}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sixteen_long_chains(ssm, dtype):
    """The most chains that hand values on eight tiles at a time, with more tiles than workgroups."""
    test_few_long_chains(ssm, 2, 4200, 500, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(4, 700, 128), (8, 300, 40), (4, 2600, 512)])
def test_eight_groups_of_chains(ssm, B, L, D, dtype):
    """Backward from checkpoints over rows times channel tiles that are a multiple of 8: tickets
    in eight groups (the last shape: more tiles than workgroups)."""
    v = draw(B, L, D, dtype, True, 200, True, seed=D)
    d = dev(v, dtype)
    kept = forward(ssm, d, save="packed")[2]
    dp = dict(d, **{k: kept[k] for k in ("x", "gate_a", "gate_x", "z")})
    seen = dict(v, **{k: R.unpack8(*R.pack8(v[k])) for k in ("x", "gate_a", "gate_x", "z")})
    for states in (kept["states"], None):
        ref = oracle_bwd(seen, states=None if states is None else states.cpu().numpy())
        g = backward(ssm, dp, states=states)
        for k in ref:
            close(g[k], ref[k], dtype if g[k].dtype != d["a_param"].dtype else "f32", k)
