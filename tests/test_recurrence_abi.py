"""Host-side checks of the gated recurrence's and the 8-bit checkpoints' entry
points: every call here is refused, or empty, before anything is launched."""

import ctypes

import pytest

from selective_state_space_23_amd import _lib

INVALID, UNSUPPORTED = _lib.MAMBA_ERR_INVALID_ARGUMENT, _lib.MAMBA_ERR_UNSUPPORTED
MISALIGNED, WORKSPACE = _lib.MAMBA_ERR_MISALIGNED, _lib.MAMBA_ERR_WORKSPACE
MB = 1 << 24                       # distance of two buffers that cannot overlap
AT = {n: MB * (i + 1) for i, n in enumerate(
    "x gate_a gate_x a_param z doc initial out final states ws dout dfinal dx dga dgx dap dz dh0 q0 q1 q2 q3 s0 s1 s2 "
    "s3 state reset".split())}    # addresses that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def dims(batch=2, seqlen=300, dim=64, dtype=1, c=8.0, **ld):
    lds = {k: 0 for k in ("ld_x", "ld_gate_a", "ld_gate_x", "ld_z", "ld_dout")}
    lds.update(ld)
    return _lib.RecurrenceDims(batch=batch, seqlen=seqlen, dim=dim, dtype=dtype, c=c, **lds)


def four(z=True, **kw):
    at = dict(AT, **kw)
    p = (_lib.Packed * 4)(*((at[f"q{i}"], at[f"s{i}"]) for i in range(4)))
    if not z:
        p[3].q = p[3].scale = None
    return p


def fwd(lib, d=None, save=None, ws_bytes=1 << 22, **kw):
    at = dict(AT, **kw)
    d = d or dims()
    return lib.mamba_gated_recurrence_fwd(ctypes.byref(d), at["x"], at["gate_a"], at["gate_x"], at["a_param"], at["z"],
                                          at["doc"], at["initial"], at["out"], at["final"], at["states"], save,
                                          at["ws"], ws_bytes, None)


def bwd(lib, d=None, packed=None, ws_bytes=1 << 22, **kw):
    at = dict(AT, **kw)
    d = d or dims()
    return lib.mamba_gated_recurrence_bwd(
        ctypes.byref(d), at["x"], at["gate_a"], at["gate_x"], at["a_param"], at["z"], at["doc"], at["initial"], packed,
        at["states"], at["dout"], at["dfinal"], at["dx"], at["dga"], at["dgx"], at["dap"], at["dz"], at["dh0"],
        at["ws"], ws_bytes, None)


def update(lib, d=None, **kw):
    at = dict(AT, **kw)
    d = d or dims(seqlen=1)
    return lib.mamba_gated_recurrence_update(ctypes.byref(d), at["state"], at["x"], at["gate_a"], at["gate_x"],
                                             at["a_param"], at["z"], at["reset"], at["out"], None)


BAD_DIMS = [
    (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(dim=-1), INVALID), (dict(batch=65536), INVALID),
    (dict(dtype=2), INVALID), (dict(c=0.0), INVALID), (dict(c=-1.0), INVALID), (dict(c=float("nan")), INVALID),
    (dict(c=float("inf")), INVALID), (dict(ld_x=63), INVALID), (dict(ld_gate_a=-64), INVALID),
    (dict(ld_dout=(1 << 21) + 4), UNSUPPORTED), (dict(dim=(1 << 21) + 4), UNSUPPORTED),
    (dict(seqlen=3000001), UNSUPPORTED), (dict(batch=400, seqlen=2560001), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_DIMS, ids=lambda v: str(v))
def test_dims(lib, kw, status):
    one = dict(kw, seqlen=1) if "seqlen" not in kw else None
    assert fwd(lib, dims(**kw)) == status
    assert bwd(lib, dims(**kw)) == status
    if one is not None:
        assert update(lib, dims(**one)) == status
    n = ctypes.c_size_t(7)
    assert lib.mamba_gated_recurrence_workspace_bytes(ctypes.byref(dims(**kw)), ctypes.byref(n)) == status
    assert lib.mamba_gated_recurrence_bwd_workspace_bytes(ctypes.byref(dims(**kw)), 0, ctypes.byref(n)) == status
    assert n.value == 0


def test_workspace(lib):
    n = ctypes.c_size_t(7)
    query = lib.mamba_gated_recurrence_workspace_bytes
    assert query(ctypes.byref(dims(seqlen=128)), ctypes.byref(n)) == 0 and n.value == 0
    assert query(ctypes.byref(dims(seqlen=129)), ctypes.byref(n)) == 0 and n.value > 0
    assert query(ctypes.byref(dims()), None) == INVALID
    assert query(None, ctypes.byref(n)) == INVALID
    query = lib.mamba_gated_recurrence_bwd_workspace_bytes
    assert query(ctypes.byref(dims(batch=0)), 0, ctypes.byref(n)) == 0 and n.value == 0
    assert query(ctypes.byref(dims()), 0, ctypes.byref(n)) == 0
    without = n.value
    assert query(ctypes.byref(dims()), 1, ctypes.byref(n)) == 0 and 0 < n.value < without
    assert fwd(lib, ws_bytes=0) == WORKSPACE and fwd(lib, ws=None) == WORKSPACE
    assert fwd(lib, ws=AT["ws"] + 64) == MISALIGNED
    assert bwd(lib, ws_bytes=n.value - 1) == WORKSPACE and bwd(lib, ws=None) == WORKSPACE
    assert bwd(lib, ws=AT["ws"] + 64) == MISALIGNED


def test_required_pointers(lib):
    for k in ("x", "gate_a", "gate_x", "a_param", "out"):
        assert fwd(lib, **{k: None}) == INVALID, k
    for k in ("x", "gate_a", "gate_x", "a_param", "dout", "dx", "dga", "dgx", "dap"):
        assert bwd(lib, **{k: None}) == INVALID, k
    for k in ("state", "x", "gate_a", "gate_x", "a_param", "out"):
        assert update(lib, **{k: None}) == INVALID, k
    assert bwd(lib, z=None) == INVALID and bwd(lib, dz=None) == INVALID      # dz exactly with z
    assert bwd(lib, initial=None) == INVALID                                 # d_initial_state without initial_state
    assert update(lib, dims(seqlen=2)) == INVALID and update(lib, dims(seqlen=0)) == INVALID


def test_alignment(lib):
    for k in ("x", "gate_a", "gate_x", "z", "out"):
        assert fwd(lib, **{k: AT[k] + 1}) == MISALIGNED, k
        assert fwd(lib, dims(dtype=0), **{k: AT[k] + 2}) == MISALIGNED, k
    for k in ("a_param", "initial", "final", "states"):
        assert fwd(lib, **{k: AT[k] + 2}) == MISALIGNED, k
    for k in ("x", "gate_a", "gate_x", "z", "dout", "dx", "dga", "dgx", "dz"):
        assert bwd(lib, **{k: AT[k] + 1}) == MISALIGNED, k
    for k in ("a_param", "initial", "states", "dfinal", "dap", "dh0"):
        assert bwd(lib, **{k: AT[k] + 2}) == MISALIGNED, k
    assert update(lib, state=AT["state"] + 2) == MISALIGNED
    assert fwd(lib, save=four(s1=AT["s1"] + 2)) == MISALIGNED


def test_overlap(lib):
    for k in ("x", "gate_a", "gate_x", "z", "initial", "doc", "a_param"):
        for o in ("out", "final", "states", "ws"):
            assert fwd(lib, **{k: AT[o]}) == INVALID, (k, o)
    assert fwd(lib, out=AT["states"]) == INVALID and fwd(lib, final=AT["ws"]) == INVALID
    # a strided input ends where its last token does, not at B L D elements
    assert fwd(lib, dims(ld_x=256), out=AT["x"] + 2 * 600 * 200) == INVALID
    for k in ("x", "dout", "states", "dfinal", "initial", "doc", "a_param", "z"):
        for o in ("dx", "dga", "dgx", "dz", "dap", "dh0", "ws"):
            assert bwd(lib, **{k: AT[o]}) == INVALID, (k, o)
    assert bwd(lib, dx=AT["dz"]) == INVALID
    assert update(lib, out=AT["state"]) == INVALID and update(lib, x=AT["state"]) == INVALID
    assert update(lib, reset=AT["out"]) == INVALID


def test_checkpoint_arguments(lib):
    assert fwd(lib, save=four(z=False)) == INVALID                # z without its checkpoint
    assert fwd(lib, z=None, save=four()) == INVALID               # a checkpoint without z
    assert fwd(lib, save=four(q0=None)) == INVALID and fwd(lib, save=four(s2=None)) == INVALID
    assert fwd(lib, save=four(q1=AT["out"])) == INVALID           # written twice
    assert bwd(lib, packed=four()) == INVALID                     # both forms of the inputs
    none = dict(x=None, gate_a=None, gate_x=None, z=None)
    assert bwd(lib, packed=four(z=False), **none) == INVALID      # dz without z
    assert bwd(lib, packed=four(q0=None), **none) == INVALID
    assert bwd(lib, packed=four(q2=AT["dx"]), **none) == INVALID
    assert bwd(lib, packed=four(s2=AT["ws"]), **none) == INVALID

    def pack(x=AT["x"], q=AT["q0"], s=AT["s0"], rows=100, dim=70, ld=0, dtype=1):
        return lib.mamba_activation_pack(x, q, s, rows, dim, ld, dtype, None)

    def unpack(q=AT["q0"], s=AT["s0"], out=AT["x"], rows=100, dim=70, dtype=1):
        return lib.mamba_activation_unpack(q, s, out, rows, dim, dtype, None)

    for f in (pack, unpack):
        assert f(rows=-1) == INVALID and f(dim=-1) == INVALID and f(dtype=5) == INVALID
        assert f(q=None) == INVALID and f(s=None) == INVALID and f(s=AT["s0"] + 1) == MISALIGNED
        assert f(dim=(1 << 21) + 1) == UNSUPPORTED and f(rows=1 << 41) == UNSUPPORTED
        assert f(rows=1 << 33, dim=64) == UNSUPPORTED
        assert f(q=AT["x"]) == INVALID and f(s=AT["x"] + 4) == INVALID
        assert f(q=None, s=None, rows=0) == 0 and f(q=None, s=None, dim=0) == 0
    assert pack(x=None) == INVALID and unpack(out=None) == INVALID and unpack(out=AT["x"] + 1) == MISALIGNED
    assert pack(ld=69) == INVALID and pack(ld=-70) == INVALID and pack(ld=(1 << 21) + 4) == UNSUPPORTED
    assert pack(q=AT["s0"]) == INVALID

    def conv(q=AT["q0"], s=AT["s0"], dx=AT["dx"], n=1 << 22, width=4):
        return lib.mamba_causal_conv1d_bwd_packed(q, s, AT["a_param"], None, AT["doc"], None, AT["dout"], dx,
                                                  AT["dap"], AT["dga"], None, 2, 100, 64, width, 1, 1, AT["ws"], n, None)

    assert conv(q=None) == INVALID and conv(s=None) == INVALID and conv(s=AT["s0"] + 2) == MISALIGNED
    assert conv(q=None, s=None) == INVALID
    assert conv(dx=AT["q0"]) == INVALID and conv(dx=AT["s0"]) == INVALID
    assert conv(n=0) == WORKSPACE and conv(width=3) == UNSUPPORTED


def test_empty_calls(lib):
    assert fwd(lib, dims(batch=0), x=None, out=None) == 0
    assert fwd(lib, dims(dim=0), x=None, out=None) == 0
    assert fwd(lib, dims(seqlen=0), final=None) == 0
    assert bwd(lib, dims(seqlen=0), dap=None, dh0=None) == 0
    assert update(lib, dims(seqlen=1, batch=0), state=None) == 0
    assert fwd(lib, dims(seqlen=0), final=AT["initial"]) == INVALID
    assert bwd(lib, dims(seqlen=0), dh0=AT["dfinal"]) == INVALID


def test_binding_strides():
    import torch

    from selective_state_space_23_amd import _strided

    cpu, f32 = torch.device("cpu"), torch.float32
    proj = torch.zeros(2, 5, 12)
    at = lambda t, shape=None: _strided(t, "x", cpu, f32, t.shape if shape is None else shape)  # noqa: E731
    assert at(proj) == (proj.data_ptr(), 0)
    assert at(proj[..., 4:8]) == (proj.data_ptr() + 16, 12)
    assert at(proj[:1, :, :4])[1] == 12 and at(proj[:, :1, :4])[1] == 60 and at(proj[:1, :1, :4])[1] == 0
    assert at(proj[:, 0, 4:8])[1] == 60                                      # rows of a (B, D) step
    assert _strided(None, "x", cpu, f32, (1,)) == (None, 0)
    with pytest.raises(ValueError, match="contiguous"):
        at(proj.transpose(1, 2))
    with pytest.raises(ValueError, match="one distance"):
        at(proj[:, :3, :4])                                                  # rows cut short
    with pytest.raises(ValueError, match="overlap"):
        at(proj[:1, :1].expand(2, 5, 12))
    with pytest.raises(ValueError, match="shape"):
        at(proj, (2, 5, 11))
    with pytest.raises(ValueError, match="must be"):
        at(proj.double())


def test_step_strides(lib):
    """The step's rows may lie further apart than a tile's tokens: refused for the missing
    state, not for the stride."""
    far = 1 << 22
    for k in ("ld_x", "ld_gate_a", "ld_gate_x", "ld_z"):
        assert update(lib, dims(seqlen=1, **{k: far}), state=None) == INVALID, k
        assert update(lib, dims(seqlen=1, **{k: (1 << 40) + 1})) == UNSUPPORTED, k
        assert update(lib, dims(seqlen=1, **{k: 63}), state=None) == INVALID, k
        assert fwd(lib, dims(seqlen=1, **{k: far})) == UNSUPPORTED and bwd(lib, dims(seqlen=1, **{k: far})) == UNSUPPORTED, k
    # an output inside the last, far row of an input
    assert update(lib, dims(seqlen=1, ld_x=far), out=AT["x"] + 2 * far) == INVALID
