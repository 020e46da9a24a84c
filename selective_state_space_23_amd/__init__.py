"""MI355X (gfx950) Mamba selective-scan forward path.

Python binding over libmamba_hip.so: argument marshalling only.  Every step of
the computation runs in the library's HIP kernels; PyTorch supplies device
memory and the current stream.  There is no CPU fallback: if the library is
missing or the tensors are not on a GPU the calls raise.

    u = causal_conv1d_fwd(x, weight, bias, doc_start)                  # (B, L, D)
    out, h = selective_scan_fwd(u, delta, A, B, C, D, z, delta_bias, doc_start)

    # gradients of sum(dout * out) for per-channel A (training), then through the conv
    g = selective_scan_bwd(u, delta, A, B, C, dout, D, z, delta_bias, doc_start)
    dx, dweight, dbias = causal_conv1d_bwd(x, weight, g["du"], bias, doc_start)

    # decode, one token per row, continuing the prefill above
    u_t = causal_conv1d_update(x_t, conv_state, weight, bias)          # (B, D)
    out_t = selective_state_update(h, u_t, delta_t, A, B_t, C_t, D, z_t, delta_bias)
    # or both in one launch
    out_t = conv_state_update(x_t, conv_state, weight, bias, h, delta_t, A, B_t, C_t, D, z_t, delta_bias)

    # gated linear recurrence; training keeps its inputs as 8-bit checkpoints
    out, h, kept = gated_recurrence_fwd(x, gate_a, gate_x, a_param, z, doc_start, save="packed")
    g = gated_recurrence_bwd(kept["x"], kept["gate_a"], kept["gate_x"], a_param, dout, kept["z"], doc_start,
                             states=kept["states"])
    out_t = gated_recurrence_update(h, x_t, gate_a_t, gate_x_t, a_param, z_t)

    # 8-bit checkpoints of any activation: the conv backward reads them as they are
    p = activation_pack(x)
    dx, dweight, dbias = causal_conv1d_bwd(p, weight, du, bias, doc_start)
    u = activation_unpack(activation_pack(u), torch.bfloat16)          # e.g. for selective_scan_bwd

    # queries and keys normed per head and rotated by their positions, for the delta rule
    q, k = qk_norm_rotary_fwd(q_in, k_in, cos=cos, sin=sin, positions=positions, norm="l2")
    grads = qk_norm_rotary_bwd(q_in, k_in, dq, dk, cos=cos, sin=sin, positions=positions, norm="l2")

    # gated delta rule: a K x V state per head, q and k (B, L, Hk, K), v (B, L, Hv, V), g and beta (B, L, Hv)
    out, S, kept = gated_delta_rule_fwd(q, k, v, g, beta, doc_start, save="states")
    grads = gated_delta_rule_bwd(q, k, v, g, beta, dout, doc_start, states=kept["states"])
    out_t = gated_delta_rule_update(S, q_t, k_t, v_t, g_t, beta_t)
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import _lib
from ._lib import MambaArgumentError, MambaError, ScanDims  # noqa: F401

__all__ = [
    "causal_conv1d_fwd",
    "selective_scan_fwd",
    "selective_scan_fwd_noalloc",
    "scan_workspace_bytes",
    "conv_scan_fwd",
    "causal_conv1d_update",
    "selective_state_update",
    "conv_state_update",
    "selective_scan_bwd",
    "scan_bwd_workspace_bytes",
    "causal_conv1d_bwd",
    "conv_bwd_workspace_bytes",
    "gated_recurrence_fwd",
    "gated_recurrence_bwd",
    "gated_recurrence_update",
    "gated_recurrence_workspace_bytes",
    "gated_recurrence_bwd_workspace_bytes",
    "PackedActivation",
    "activation_pack",
    "activation_unpack",
    "qk_norm_rotary_fwd",
    "qk_norm_rotary_bwd",
    "gated_delta_rule_fwd",
    "gated_delta_rule_bwd",
    "gated_delta_rule_update",
    "gated_delta_rule_workspace_bytes",
    "gated_delta_rule_bwd_workspace_bytes",
    "MambaError",
    "MambaArgumentError",
    "library_path",
    "version",
]


def library_path() -> str:
    return _lib.LIB_PATH


def version() -> str:
    v = _lib.load().mamba_version()
    return f"{v >> 16}.{(v >> 8) & 255}.{v & 255}"


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return _lib.MAMBA_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return _lib.MAMBA_DTYPE_BF16
    raise MambaArgumentError(_lib.MAMBA_ERR_INVALID_ARGUMENT, f"unsupported activation dtype {t.dtype}")


def _ptr(t, name, device, dtype=None, shape=None) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(device) -> int:
    """The current stream's handle.  (torch's own generated code asks for it by the
    first call, which makes no Stream object: 2 us less a launch.)"""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return raw(device.index)


def _launch(device, call, *args) -> int:
    """call(*args, stream) with the tensors' device current."""
    torch = _torch()
    if device.index is None or torch.cuda.current_device() == device.index:
        return call(*args, _stream(device))
    with torch.cuda.device(device):
        return call(*args, _stream(device))


def _check_device(x):
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU device (the library has no CPU path)")
    return x.device


def causal_conv1d_fwd(x, weight, bias=None, doc_start=None, apply_silu: bool = True, out=None, conv_state=None):
    """Depthwise causal conv1d (width 4) + SiLU; see mamba_causal_conv1d_fwd.

    x (B, L, D) float32/bfloat16; weight (D, 4) or (D, 1, 4) float32; bias (D,)
    float32; doc_start (B, L) uint8/bool; conv_state (B, D, 3) of x's dtype: the
    inputs before token 0 (token 0 then starts a document only where doc_start
    says so).  Returns out (B, L, D), x's dtype."""
    torch = _torch()
    dev = _check_device(x)
    if x.dim() != 3:
        raise ValueError("x must be (B, L, D)")
    Bt, L, Dm = x.shape
    if weight.dim() == 3:
        weight = weight.reshape(weight.shape[0], weight.shape[-1])
    W = weight.shape[-1]
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    if out is None:
        out = torch.empty_like(x)
    st = _lib.load().mamba_causal_conv1d_fwd(
        _ptr(x, "x", dev), _ptr(weight, "weight", dev, torch.float32, (Dm, W)),
        _ptr(bias, "bias", dev, torch.float32, (Dm,)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(conv_state, "conv_state", dev, x.dtype, (Bt, Dm, W - 1)),
        _ptr(out, "out", dev, x.dtype, (Bt, L, Dm)), Bt, L, Dm, W, _dtype_code(x), int(bool(apply_silu)),
        _stream(dev))
    _lib.check(st, "mamba_causal_conv1d_fwd")
    return out


def _scan_dims(Bt, L, Dm, N, nheads, dtype_code, softplus) -> ScanDims:
    return ScanDims(batch=Bt, seqlen=L, dim=Dm, dstate=N, nheads=nheads, ngroups=1, dtype=dtype_code,
                    delta_softplus=int(bool(softplus)))


def scan_workspace_bytes(batch, seqlen, dim, dstate, nheads=0, dtype="bf16") -> int:
    code = _lib.MAMBA_DTYPE_BF16 if dtype == "bf16" else _lib.MAMBA_DTYPE_F32
    dims = _scan_dims(batch, seqlen, dim, dstate, nheads, code, True)
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().mamba_selective_scan_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
               "mamba_selective_scan_workspace_bytes")
    return int(n.value)


def selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, doc_start=None,
                       delta_softplus: bool = True, out=None, final_state=True, workspace=None,
                       initial_state=None):
    """Selective scan forward; see mamba_selective_scan_fwd.

    u, z (B, L, D); delta (B, L, D) with A (D, N), or delta (B, L, H) with A (H,);
    B, C (B, L, N); D (D,), delta_bias (D,) or (H,), float32.  ``final_state``:
    True to allocate and return it, False/None to skip, or a (B, D, N) float32
    tensor to fill.  ``workspace``: optional uint8 device tensor of at least
    scan_workspace_bytes(...) bytes.  ``initial_state``: optional (B, D, N) float32
    state before token 0 (token 0 then resets only where doc_start[:, 0] is set).
    Returns (out, final_state or None)."""
    torch = _torch()
    dev = _check_device(u)
    if u.dim() != 3:
        raise ValueError("u must be (B, L, D)")
    Bt, L, Dm = u.shape
    N = B.shape[-1]
    nheads = A.shape[0] if A.dim() == 1 else 0
    nd = nheads if nheads else Dm
    code = _dtype_code(u)
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    if out is None:
        out = torch.empty_like(u)
    if final_state is True:
        final_state = torch.empty((Bt, Dm, N), dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    dims = _scan_dims(Bt, L, Dm, N, nheads, code, delta_softplus)
    lib = _lib.load()
    need = ctypes.c_size_t(0)
    _lib.check(lib.mamba_selective_scan_workspace_bytes(ctypes.byref(dims), ctypes.byref(need)),
               "mamba_selective_scan_workspace_bytes")
    if need.value and workspace is None:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=dev)
    ws_ptr = _ptr(workspace, "workspace", dev, torch.uint8) if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    st = lib.mamba_selective_scan_fwd(
        ctypes.byref(dims),
        _ptr(u, "u", dev, u.dtype, (Bt, L, Dm)),
        _ptr(delta, "delta", dev, u.dtype, (Bt, L, nd)),
        _ptr(A, "A", dev, torch.float32, (nheads,) if nheads else (Dm, N)),
        _ptr(B, "B", dev, u.dtype, (Bt, L, N)),
        _ptr(C, "C", dev, u.dtype, (Bt, L, N)),
        _ptr(D, "D", dev, torch.float32, (Dm,)),
        _ptr(z, "z", dev, u.dtype, (Bt, L, Dm)),
        _ptr(delta_bias, "delta_bias", dev, torch.float32, (nd,)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, torch.float32, (Bt, Dm, N)),
        _ptr(out, "out", dev, u.dtype, (Bt, L, Dm)),
        _ptr(final_state, "final_state", dev, torch.float32, (Bt, Dm, N)),
        ws_ptr, ws_bytes, _stream(dev))
    _lib.check(st, "mamba_selective_scan_fwd")
    return out, final_state


def selective_scan_fwd_noalloc(u, delta, A, B, C, out, D=None, z=None, delta_bias=None, doc_start=None,
                               delta_softplus: bool = True, final_state=None, initial_state=None):
    """Selective scan forward with no workspace; see mamba_selective_scan_fwd_noalloc.

    Arguments as selective_scan_fwd; ``out`` (B, L, D) and the optional
    ``final_state`` (B, D, N) float32 are caller-owned tensors the call fills
    (nothing is allocated here or in the library).  Returns (out, final_state)."""
    torch = _torch()
    dev = _check_device(u)
    if u.dim() != 3:
        raise ValueError("u must be (B, L, D)")
    Bt, L, Dm = u.shape
    N = B.shape[-1]
    nheads = A.shape[0] if A.dim() == 1 else 0
    nd = nheads if nheads else Dm
    if doc_start is not None and doc_start.dtype == torch.bool:
        raise ValueError("doc_start must be uint8 (a bool mask would need a converted copy)")
    dims = _scan_dims(Bt, L, Dm, N, nheads, _dtype_code(u), delta_softplus)
    st = _lib.load().mamba_selective_scan_fwd_noalloc(
        ctypes.byref(dims),
        _ptr(u, "u", dev, u.dtype, (Bt, L, Dm)),
        _ptr(delta, "delta", dev, u.dtype, (Bt, L, nd)),
        _ptr(A, "A", dev, torch.float32, (nheads,) if nheads else (Dm, N)),
        _ptr(B, "B", dev, u.dtype, (Bt, L, N)),
        _ptr(C, "C", dev, u.dtype, (Bt, L, N)),
        _ptr(D, "D", dev, torch.float32, (Dm,)),
        _ptr(z, "z", dev, u.dtype, (Bt, L, Dm)),
        _ptr(delta_bias, "delta_bias", dev, torch.float32, (nd,)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, torch.float32, (Bt, Dm, N)),
        _ptr(out, "out", dev, u.dtype, (Bt, L, Dm)),
        _ptr(final_state, "final_state", dev, torch.float32, (Bt, Dm, N)),
        _stream(dev))
    _lib.check(st, "mamba_selective_scan_fwd_noalloc")
    return out, final_state


def conv_scan_fwd(x, conv_weight, conv_bias, delta, A, B, C, D=None, z=None, delta_bias=None, doc_start=None,
                  delta_softplus: bool = True, initial_state=None, conv_state=None, u=True, out=None,
                  final_state=True, workspace=None):
    """Conv1d (width 4) + SiLU and the selective scan in one call; see mamba_conv_scan_fwd.

    Arguments as causal_conv1d_fwd (x, conv_weight, conv_bias, doc_start,
    conv_state) and selective_scan_fwd (the rest).  ``u``: a (B, L, D) tensor that
    receives the conv output, True (allocate one) or None (the conv output is not
    written).  Returns (u or None, out, final_state or None)."""
    torch = _torch()
    dev = _check_device(x)
    if x.dim() != 3:
        raise ValueError("x must be (B, L, D)")
    Bt, L, Dm = x.shape
    N = B.shape[-1]
    if conv_weight.dim() == 3:
        conv_weight = conv_weight.reshape(conv_weight.shape[0], conv_weight.shape[-1])
    nheads = A.shape[0] if A.dim() == 1 else 0
    nd = nheads if nheads else Dm
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    if u is True:
        u = torch.empty_like(x)
    elif u is False:
        u = None
    if out is None:
        out = torch.empty_like(x)
    if final_state is True:
        final_state = torch.empty((Bt, Dm, N), dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    dims = _scan_dims(Bt, L, Dm, N, nheads, _dtype_code(x), delta_softplus)
    lib = _lib.load()
    need = ctypes.c_size_t(0)
    _lib.check(lib.mamba_selective_scan_workspace_bytes(ctypes.byref(dims), ctypes.byref(need)),
               "mamba_selective_scan_workspace_bytes")
    if need.value and workspace is None:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=dev)
    ws_ptr = _ptr(workspace, "workspace", dev, torch.uint8) if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    st = lib.mamba_conv_scan_fwd(
        ctypes.byref(dims),
        _ptr(x, "x", dev, x.dtype, (Bt, L, Dm)),
        _ptr(conv_weight, "conv_weight", dev, torch.float32, (Dm, 4)),
        _ptr(conv_bias, "conv_bias", dev, torch.float32, (Dm,)),
        _ptr(conv_state, "conv_state", dev, x.dtype, (Bt, Dm, 3)),
        _ptr(delta, "delta", dev, x.dtype, (Bt, L, nd)),
        _ptr(A, "A", dev, torch.float32, (nheads,) if nheads else (Dm, N)),
        _ptr(B, "B", dev, x.dtype, (Bt, L, N)),
        _ptr(C, "C", dev, x.dtype, (Bt, L, N)),
        _ptr(D, "D", dev, torch.float32, (Dm,)),
        _ptr(z, "z", dev, x.dtype, (Bt, L, Dm)),
        _ptr(delta_bias, "delta_bias", dev, torch.float32, (nd,)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, torch.float32, (Bt, Dm, N)),
        _ptr(u, "u", dev, x.dtype, (Bt, L, Dm)),
        _ptr(out, "out", dev, x.dtype, (Bt, L, Dm)),
        _ptr(final_state, "final_state", dev, torch.float32, (Bt, Dm, N)),
        ws_ptr, ws_bytes, _stream(dev))
    _lib.check(st, "mamba_conv_scan_fwd")
    return u, out, final_state


def causal_conv1d_update(x, conv_state, weight, bias=None, reset=None, apply_silu: bool = True, out=None):
    """Causal conv1d (width 4) + SiLU for one token per row; see mamba_causal_conv1d_update.

    x (B, D); conv_state (B, D, 3) of x's dtype, updated in place (the last three
    inputs of each channel); weight (D, 4) float32; bias (D,); reset (B,)
    uint8/bool.  Returns out (B, D)."""
    torch = _torch()
    dev = _check_device(x)
    if x.dim() != 2:
        raise ValueError("x must be (B, D)")
    Bt, Dm = x.shape
    if weight.dim() == 3:
        weight = weight.reshape(weight.shape[0], weight.shape[-1])
    W = weight.shape[-1]
    if reset is not None and reset.dtype == torch.bool:
        reset = reset.to(torch.uint8)
    if out is None:
        out = torch.empty_like(x)
    st = _lib.load().mamba_causal_conv1d_update(
        _ptr(x, "x", dev), _ptr(conv_state, "conv_state", dev, x.dtype, (Bt, Dm, W - 1)),
        _ptr(weight, "weight", dev, torch.float32, (Dm, W)), _ptr(bias, "bias", dev, torch.float32, (Dm,)),
        _ptr(reset, "reset", dev, torch.uint8, (Bt,)), _ptr(out, "out", dev, x.dtype, (Bt, Dm)),
        Bt, Dm, W, _dtype_code(x), int(bool(apply_silu)), _stream(dev))
    _lib.check(st, "mamba_causal_conv1d_update")
    return out


def selective_state_update(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, reset=None,
                           delta_softplus: bool = True, out=None):
    """One recurrence step per row; see mamba_selective_state_update.

    state (B, D, N) float32, updated in place; u, z (B, D); delta (B, D) with A
    (D, N) or (B, H) with A (H,); B, C (B, N); reset (B,) uint8/bool.  Returns
    out (B, D)."""
    torch = _torch()
    dev = _check_device(u)
    if u.dim() != 2:
        raise ValueError("u must be (B, D)")
    Bt, Dm = u.shape
    N = B.shape[-1]
    nheads = A.shape[0] if A.dim() == 1 else 0
    nd = nheads if nheads else Dm
    if reset is not None and reset.dtype == torch.bool:
        reset = reset.to(torch.uint8)
    if out is None:
        out = torch.empty_like(u)
    dims = _scan_dims(Bt, 1, Dm, N, nheads, _dtype_code(u), delta_softplus)
    st = _lib.load().mamba_selective_state_update(
        ctypes.byref(dims), _ptr(state, "state", dev, torch.float32, (Bt, Dm, N)),
        _ptr(u, "u", dev, u.dtype, (Bt, Dm)), _ptr(delta, "delta", dev, u.dtype, (Bt, nd)),
        _ptr(A, "A", dev, torch.float32, (nheads,) if nheads else (Dm, N)),
        _ptr(B, "B", dev, u.dtype, (Bt, N)), _ptr(C, "C", dev, u.dtype, (Bt, N)),
        _ptr(D, "D", dev, torch.float32, (Dm,)), _ptr(z, "z", dev, u.dtype, (Bt, Dm)),
        _ptr(delta_bias, "delta_bias", dev, torch.float32, (nd,)), _ptr(reset, "reset", dev, torch.uint8, (Bt,)),
        _ptr(out, "out", dev, u.dtype, (Bt, Dm)), _stream(dev))
    _lib.check(st, "mamba_selective_state_update")
    return out


def scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, dtype="bf16", nheads=0) -> int:
    code = _lib.MAMBA_DTYPE_BF16 if dtype == "bf16" else _lib.MAMBA_DTYPE_F32
    dims = _scan_dims(batch, seqlen, dim, dstate, nheads, code, True)
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().mamba_selective_scan_bwd_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
               "mamba_selective_scan_bwd_workspace_bytes")
    return int(n.value)


def conv_state_update(x, conv_state, conv_weight, conv_bias, state, delta, A, B, C, D=None, z=None, delta_bias=None,
                      reset=None, delta_softplus: bool = True, out=None, u_out=None):
    """Both decode steps in one launch; see mamba_conv_state_update.  x (B, D);
    conv_state (B, D, 3) and state (B, D, N) updated in place; the rest as
    selective_state_update.  Returns out (B, D) (u is written to u_out if given)."""
    torch = _torch()
    dev = _check_device(x)
    if x.dim() != 2:
        raise ValueError("x must be (B, D)")
    Bt, Dm = x.shape
    N = B.shape[-1]
    nheads = A.shape[0] if A.dim() == 1 else 0
    nd = nheads if nheads else Dm
    if conv_weight.dim() == 3:
        conv_weight = conv_weight.reshape(conv_weight.shape[0], conv_weight.shape[-1])
    if reset is not None and reset.dtype == torch.bool:
        reset = reset.to(torch.uint8)
    if out is None:
        out = torch.empty_like(x)
    dims = _scan_dims(Bt, 1, Dm, N, nheads, _dtype_code(x), delta_softplus)
    st = _lib.load().mamba_conv_state_update(
        ctypes.byref(dims), _ptr(x, "x", dev), _ptr(conv_state, "conv_state", dev, x.dtype, (Bt, Dm, 3)),
        _ptr(conv_weight, "conv_weight", dev, torch.float32, (Dm, 4)),
        _ptr(conv_bias, "conv_bias", dev, torch.float32, (Dm,)),
        _ptr(state, "state", dev, torch.float32, (Bt, Dm, N)), _ptr(delta, "delta", dev, x.dtype, (Bt, nd)),
        _ptr(A, "A", dev, torch.float32, (nheads,) if nheads else (Dm, N)),
        _ptr(B, "B", dev, x.dtype, (Bt, N)), _ptr(C, "C", dev, x.dtype, (Bt, N)),
        _ptr(D, "D", dev, torch.float32, (Dm,)), _ptr(z, "z", dev, x.dtype, (Bt, Dm)),
        _ptr(delta_bias, "delta_bias", dev, torch.float32, (nd,)), _ptr(reset, "reset", dev, torch.uint8, (Bt,)),
        _ptr(u_out, "u_out", dev, x.dtype, (Bt, Dm)), _ptr(out, "out", dev, x.dtype, (Bt, Dm)), _stream(dev))
    _lib.check(st, "mamba_conv_state_update")
    return out


def selective_scan_bwd(u, delta, A, B, C, dout, D=None, z=None, delta_bias=None, doc_start=None,
                       delta_softplus: bool = True, workspace=None, grads=None, initial_state=None,
                       d_final_state=None):
    """Gradients of sum(dout * out) + sum(d_final_state * final_state) for the
    scan; see mamba_selective_scan_bwd.  Arguments as selective_scan_fwd (A
    (D, N) per channel, or (H,) for scalar-A heads with delta (B, L, H)) plus
    ``dout`` (B, L, D) and ``d_final_state`` (B, D, N) float32 or None.  Returns
    a dict with du, ddelta, dB, dC (u's dtype), dA (A's shape) float32 and, for
    each optional input given, dD, dz, ddelta_bias, d_initial_state (B, D, N)
    float32.  ``grads``: optional dict of preallocated outputs with the same
    keys."""
    torch = _torch()
    dev = _check_device(u)
    if u.dim() != 3 or A.dim() not in (1, 2):
        raise ValueError("u must be (B, L, D) and A (D, N) or (H,)")
    Bt, L, Dm = u.shape
    N = B.shape[-1]
    nheads = A.shape[0] if A.dim() == 1 else 0
    nd = nheads if nheads else Dm
    code = _dtype_code(u)
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    g = dict(grads) if grads else {}
    f32 = torch.float32
    shapes = {"du": ((Bt, L, Dm), u.dtype), "ddelta": ((Bt, L, nd), u.dtype), "dA": (tuple(A.shape), f32),
              "dB": ((Bt, L, N), u.dtype), "dC": ((Bt, L, N), u.dtype)}
    if D is not None:
        shapes["dD"] = ((Dm,), f32)
    if z is not None:
        shapes["dz"] = ((Bt, L, Dm), u.dtype)
    if delta_bias is not None:
        shapes["ddelta_bias"] = ((nd,), f32)
    if initial_state is not None:
        shapes["d_initial_state"] = ((Bt, Dm, N), f32)
    for k, (shape, dt) in shapes.items():
        if k not in g:
            g[k] = torch.empty(shape, dtype=dt, device=dev)
    dims = _scan_dims(Bt, L, Dm, N, nheads, code, delta_softplus)
    lib = _lib.load()
    need = ctypes.c_size_t(0)
    _lib.check(lib.mamba_selective_scan_bwd_workspace_bytes(ctypes.byref(dims), ctypes.byref(need)),
               "mamba_selective_scan_bwd_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(max(int(need.value), 1), dtype=torch.uint8, device=dev)
    out = lambda k: _ptr(g.get(k), k, dev, shapes[k][1], shapes[k][0]) if k in shapes else None  # noqa: E731
    st = lib.mamba_selective_scan_bwd(
        ctypes.byref(dims),
        _ptr(u, "u", dev, u.dtype, (Bt, L, Dm)),
        _ptr(delta, "delta", dev, u.dtype, (Bt, L, nd)),
        _ptr(A, "A", dev, f32, tuple(A.shape)),
        _ptr(B, "B", dev, u.dtype, (Bt, L, N)),
        _ptr(C, "C", dev, u.dtype, (Bt, L, N)),
        _ptr(D, "D", dev, f32, (Dm,)),
        _ptr(z, "z", dev, u.dtype, (Bt, L, Dm)),
        _ptr(delta_bias, "delta_bias", dev, f32, (nd,)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, f32, (Bt, Dm, N)),
        _ptr(dout, "dout", dev, u.dtype, (Bt, L, Dm)),
        _ptr(d_final_state, "d_final_state", dev, f32, (Bt, Dm, N)),
        out("du"), out("ddelta"), out("dA"), out("dB"), out("dC"), out("dD"), out("dz"), out("ddelta_bias"),
        out("d_initial_state"),
        _ptr(workspace, "workspace", dev, torch.uint8), workspace.numel(), _stream(dev))
    _lib.check(st, "mamba_selective_scan_bwd")
    return {k: g[k] for k in shapes}


def conv_bwd_workspace_bytes(batch, seqlen, dim) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().mamba_causal_conv1d_bwd_workspace_bytes(batch, seqlen, dim, ctypes.byref(n)),
               "mamba_causal_conv1d_bwd_workspace_bytes")
    return int(n.value)


def causal_conv1d_bwd(x, weight, du, bias=None, doc_start=None, apply_silu: bool = True, workspace=None,
                      dx=None, dweight=None, dbias=None, conv_state=None, d_conv_state=None):
    """Gradients of sum(du * u) for u = causal_conv1d_fwd(x, weight, bias, doc_start,
    conv_state, apply_silu); see mamba_causal_conv1d_bwd.  Returns (dx, dweight
    (D, 4) float32, dbias (D,) float32 or None when bias is None), and with a
    conv_state (B, D, 3) also d_conv_state (B, D, 3) float32 as a fourth item.
    ``x`` may be a PackedActivation: the gradients at the values it stands for, in
    du's dtype (mamba_causal_conv1d_bwd_packed)."""
    torch = _torch()
    packed = x if isinstance(x, PackedActivation) else None
    if packed is not None:
        x = du
    dev = _check_device(x)
    if x.dim() != 3:
        raise ValueError("x must be (B, L, D)")
    Bt, L, Dm = x.shape
    if weight.dim() == 3:
        weight = weight.reshape(weight.shape[0], weight.shape[-1])
    W = weight.shape[-1]
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    if dx is None:
        dx = torch.empty_like(x)
    if dweight is None:
        dweight = torch.empty((Dm, W), dtype=torch.float32, device=dev)
    if dbias is None and bias is not None:
        dbias = torch.empty((Dm,), dtype=torch.float32, device=dev)
    if d_conv_state is None and conv_state is not None:
        d_conv_state = torch.empty((Bt, Dm, 3), dtype=torch.float32, device=dev)
    lib = _lib.load()
    need = ctypes.c_size_t(0)
    _lib.check(lib.mamba_causal_conv1d_bwd_workspace_bytes(Bt, L, Dm, ctypes.byref(need)),
               "mamba_causal_conv1d_bwd_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(max(int(need.value), 1), dtype=torch.uint8, device=dev)
    if packed is None:
        call, name, xs = lib.mamba_causal_conv1d_bwd, "mamba_causal_conv1d_bwd", (_ptr(x, "x", dev),)
    else:
        call, name = lib.mamba_causal_conv1d_bwd_packed, "mamba_causal_conv1d_bwd_packed"
        xs = _packed_ptrs(packed, "x", dev, (Bt, L, Dm))
    st = _launch(
        dev, call, *xs, _ptr(weight, "weight", dev, torch.float32, (Dm, W)),
        _ptr(bias, "bias", dev, torch.float32, (Dm,)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(conv_state, "conv_state", dev, x.dtype, (Bt, Dm, 3)),
        _ptr(du, "du", dev, x.dtype, (Bt, L, Dm)), _ptr(dx, "dx", dev, x.dtype, (Bt, L, Dm)),
        _ptr(dweight, "dweight", dev, torch.float32, (Dm, W)), _ptr(dbias, "dbias", dev, torch.float32, (Dm,)),
        _ptr(d_conv_state, "d_conv_state", dev, torch.float32, (Bt, Dm, 3)),
        Bt, L, Dm, W, _dtype_code(x), int(bool(apply_silu)),
        _ptr(workspace, "workspace", dev, torch.uint8), workspace.numel())
    _lib.check(st, name)
    if conv_state is not None:
        return dx, dweight, dbias, d_conv_state
    return dx, dweight, dbias


class PackedActivation(NamedTuple):
    """An activation kept in 8 bits: ``q`` int8 codes (..., D) and ``scale`` float32
    (ceil(D / 64), ...), one per token and block of 64 channels; the values are
    q * scale.  A block that held a NaN or an infinity has a NaN scale."""

    q: object
    scale: object


def _packed_ptrs(p, name, dev, shape):
    torch = _torch()
    if not isinstance(p, PackedActivation):
        raise TypeError(f"{name} must be a PackedActivation")
    blocks = -(-shape[-1] // _lib.PACK_BLOCK)
    return (_ptr(p.q, f"{name}.q", dev, torch.int8, shape),
            _ptr(p.scale, f"{name}.scale", dev, torch.float32, (blocks,) + tuple(shape[:-1])))


def _packed_empty(shape, dev):
    torch = _torch()
    return PackedActivation(torch.empty(shape, dtype=torch.int8, device=dev),
                            torch.empty((-(-shape[-1] // _lib.PACK_BLOCK),) + tuple(shape[:-1]), dtype=torch.float32,
                                        device=dev))


def _strided(t, name, dev, dtype, shape):
    """(pointer, elements between two tokens) of a (..., D) tensor whose channels are
    contiguous and whose tokens lie at one distance: a dense tensor, or a slice of the
    channels of one.  (None, 0) for None."""
    if t is None:
        return None, 0
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    D = shape[-1]
    if D > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    ld, want = None, None   # distance of two tokens, of two steps of the dimension looked at
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if ld is None:
            ld = want = t.stride(i)
        if t.stride(i) != want:
            raise ValueError(f"{name}: tokens must lie at one distance")
        want *= shape[i]
    ld = D if ld is None else ld
    if ld < D:
        raise ValueError(f"{name}: tokens must not overlap")
    return t.data_ptr(), ld


def activation_pack(x, packed=None) -> PackedActivation:
    """The 8-bit checkpoint of x (..., D), float32/bfloat16; see mamba_activation_pack.
    x's channels are contiguous and its tokens lie at one distance.  ``packed``: an
    optional PackedActivation to fill."""
    dev = _check_device(x)
    if x.dim() < 1:
        raise ValueError("x must be (..., D)")
    code = _dtype_code(x)
    shape = tuple(x.shape)
    ptr, ld = _strided(x, "x", dev, x.dtype, shape)
    if packed is None:
        packed = _packed_empty(shape, dev)
    q, scale = _packed_ptrs(packed, "packed", dev, shape)
    rows = 1
    for n in shape[:-1]:
        rows *= n
    st = _launch(dev, _lib.load().mamba_activation_pack, ptr, q, scale, rows, shape[-1], ld, code)
    _lib.check(st, "mamba_activation_pack")
    return packed


def activation_unpack(packed, dtype=None, out=None):
    """The values a PackedActivation stands for, float32 or bfloat16 (``dtype``,
    bfloat16 if not given; or ``out``, a contiguous tensor of q's shape); see
    mamba_activation_unpack."""
    torch = _torch()
    if not isinstance(packed, PackedActivation):
        raise TypeError("packed must be a PackedActivation")
    dev = _check_device(packed.q)
    shape = tuple(packed.q.shape)
    if out is None:
        out = torch.empty(shape, dtype=dtype or torch.bfloat16, device=dev)
    elif dtype is not None and out.dtype != dtype:
        raise ValueError(f"out must be {dtype}, got {out.dtype}")
    q, scale = _packed_ptrs(packed, "packed", dev, shape)
    rows = 1
    for n in shape[:-1]:
        rows *= n
    st = _launch(dev, _lib.load().mamba_activation_unpack, q, scale, _ptr(out, "out", dev, out.dtype, shape), rows,
                 shape[-1], _dtype_code(out))
    _lib.check(st, "mamba_activation_unpack")
    return out


def _recurrence_dims(batch, seqlen, dim, code, c, lds=(0, 0, 0, 0, 0)) -> _lib.RecurrenceDims:
    return _lib.RecurrenceDims(batch, seqlen, dim, *lds, code, c)


def _recurrence_workspace(call, name, dev, *args):
    need = ctypes.c_size_t(0)
    _lib.check(call(*args, ctypes.byref(need)), name)
    return _torch().empty(int(need.value), dtype=_torch().uint8, device=dev) if need.value else None


def gated_recurrence_workspace_bytes(batch, seqlen, dim, dtype="bf16") -> int:
    dims = _recurrence_dims(batch, seqlen, dim, _lib.MAMBA_DTYPE_BF16 if dtype == "bf16" else _lib.MAMBA_DTYPE_F32, 8.0)
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().mamba_gated_recurrence_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
               "mamba_gated_recurrence_workspace_bytes")
    return int(n.value)


def gated_recurrence_bwd_workspace_bytes(batch, seqlen, dim, dtype="bf16", states=False) -> int:
    dims = _recurrence_dims(batch, seqlen, dim, _lib.MAMBA_DTYPE_BF16 if dtype == "bf16" else _lib.MAMBA_DTYPE_F32, 8.0)
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().mamba_gated_recurrence_bwd_workspace_bytes(ctypes.byref(dims), int(bool(states)),
                                                                      ctypes.byref(n)),
               "mamba_gated_recurrence_bwd_workspace_bytes")
    return int(n.value)


def gated_recurrence_fwd(x, gate_a, gate_x, a_param, z=None, doc_start=None, c: float = 8.0, initial_state=None,
                         final_state=True, out=None, save=None, workspace=None):
    """Gated linear recurrence; see mamba_gated_recurrence_fwd.

    x, gate_a, gate_x, z (B, L, D) float32/bfloat16, dense or slices of the channels
    of one projection's output; a_param (D,) float32; doc_start (B, L) uint8/bool;
    initial_state (B, D) float32.  ``final_state``: True to allocate and return it,
    False/None to skip, or a (B, D) float32 tensor to fill.  ``save``: None;
    "states" to keep the states the backward starts its chunks from; "packed" to
    keep them and 8-bit checkpoints of x, gate_a, gate_x and z; or a dict of such
    tensors to fill ("states" (B, ceil(L / 128), D) float32, and all or none of the
    PackedActivations "x", "gate_a", "gate_x" and, with a z, "z").  Returns (out,
    final_state or None), with ``save`` also the dict of what was kept."""
    torch = _torch()
    dev = _check_device(x)
    if x.dim() != 3:
        raise ValueError("x must be (B, L, D)")
    code, dt, f32 = _dtype_code(x), x.dtype, torch.float32
    shape = x.shape
    Bt, L, Dm = shape
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else torch.empty(shape, dtype=dt, device=dev)
    if final_state is True:
        final_state = torch.empty((Bt, Dm), dtype=f32, device=dev)
    elif final_state is False:
        final_state = None
    px, lx = _strided(x, "x", dev, dt, shape)
    pa, la = _strided(gate_a, "gate_a", dev, dt, shape)
    pg, lg = _strided(gate_x, "gate_x", dev, dt, shape)
    pz, lz = _strided(z, "z", dev, dt, shape)
    names = ("x", "gate_a", "gate_x") + (() if z is None else ("z",))
    kept, states, pk = None, None, None
    if save is not None:
        if isinstance(save, dict):
            kept = save
            unknown = set(kept) - {"states", "x", "gate_a", "gate_x", "z"}
            if unknown:
                raise ValueError(f"save: unknown entries {sorted(unknown)}")
            if any(n in kept for n in ("x", "gate_a", "gate_x", "z")) and \
                    {n for n in ("x", "gate_a", "gate_x", "z") if n in kept} != set(names):
                raise ValueError(f"save: checkpoints of {names} are kept together")
        elif save in ("states", "packed"):
            kept = {"states": torch.empty((Bt, -(-L // _lib.RECURRENCE_CHUNK), Dm), dtype=f32, device=dev)}
            if save == "packed":
                kept.update((n, _packed_empty((Bt, L, Dm), dev)) for n in names)
        else:
            raise ValueError('save must be None, "states", "packed" or a dict')
        states = kept.get("states")
        if "x" in kept:
            pk = (_lib.Packed * 4)(*(_packed_ptrs(kept[n], n, dev, (Bt, L, Dm)) for n in names))
    dims = _recurrence_dims(Bt, L, Dm, code, c, (lx, la, lg, lz, 0))
    lib = _lib.load()
    if workspace is None and L > _lib.RECURRENCE_CHUNK:
        workspace = _recurrence_workspace(lib.mamba_gated_recurrence_workspace_bytes,
                                          "mamba_gated_recurrence_workspace_bytes", dev, ctypes.byref(dims))
    st = _launch(
        dev, lib.mamba_gated_recurrence_fwd,
        ctypes.byref(dims), px, pa, pg, _ptr(a_param, "a_param", dev, f32, (Dm,)), pz,
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, f32, (Bt, Dm)),
        _ptr(out, "out", dev, dt, shape),
        _ptr(final_state, "final_state", dev, f32, (Bt, Dm)),
        _ptr(states, "states", dev, f32, (Bt, -(-L // _lib.RECURRENCE_CHUNK), Dm)), pk,
        _ptr(workspace, "workspace", dev, torch.uint8), 0 if workspace is None else workspace.numel())
    _lib.check(st, "mamba_gated_recurrence_fwd")
    return (out, final_state) if save is None else (out, final_state, kept)


def gated_recurrence_bwd(x, gate_a, gate_x, a_param, dout, z=None, doc_start=None, c: float = 8.0,
                         initial_state=None, d_final_state=None, states=None, workspace=None, grads=None):
    """Gradients of sum(dout * out) + sum(d_final_state * final_state) for the gated
    linear recurrence; see mamba_gated_recurrence_bwd.

    x, gate_a, gate_x and z as given to gated_recurrence_fwd, or all of them the
    PackedActivations it kept; ``states`` what it kept (or None: recomputed); dout
    (B, L, D), dense or a slice.  Returns a dict with dx, dgate_a, dgate_x (dout's
    dtype), da_param (D,) float32 and, for each optional input given, dz and
    d_initial_state (B, D) float32.  ``grads``: optional dict of preallocated outputs
    with the same keys."""
    torch = _torch()
    dev = _check_device(dout)
    if dout.dim() != 3:
        raise ValueError("dout must be (B, L, D)")
    code, dt, f32 = _dtype_code(dout), dout.dtype, torch.float32
    shape = dout.shape
    Bt, L, Dm = shape
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    inputs = (("x", x), ("gate_a", gate_a), ("gate_x", gate_x)) + ((("z", z),) if z is not None else ())
    is_packed = [isinstance(t, PackedActivation) for _, t in inputs]
    if any(is_packed) and not all(is_packed):
        raise ValueError("x, gate_a, gate_x and z must be all tensors or all PackedActivations")
    ptrs, lds, pk = [None] * 4, [0] * 4, None
    if all(is_packed):
        pk = (_lib.Packed * 4)(*(_packed_ptrs(t, n, dev, (Bt, L, Dm)) for n, t in inputs))
    else:
        for i, (n, t) in enumerate(inputs):
            ptrs[i], lds[i] = _strided(t, n, dev, dt, shape)
    po, lo = _strided(dout, "dout", dev, dt, shape)
    shapes = {"dx": ((Bt, L, Dm), dt), "dgate_a": ((Bt, L, Dm), dt), "dgate_x": ((Bt, L, Dm), dt),
              "da_param": ((Dm,), f32)}
    if z is not None:
        shapes["dz"] = ((Bt, L, Dm), dt)
    if initial_state is not None:
        shapes["d_initial_state"] = ((Bt, Dm), f32)
    g = dict(grads) if grads else {}
    for k, (sh, d) in shapes.items():
        if k not in g:
            g[k] = torch.empty(sh, dtype=d, device=dev)
    dims = _recurrence_dims(Bt, L, Dm, code, c, (*lds, lo))
    lib = _lib.load()
    if workspace is None:
        workspace = _recurrence_workspace(lib.mamba_gated_recurrence_bwd_workspace_bytes,
                                          "mamba_gated_recurrence_bwd_workspace_bytes", dev, ctypes.byref(dims),
                                          int(states is not None))
    res = lambda k: _ptr(g[k], k, dev, shapes[k][1], shapes[k][0]) if k in shapes else None  # noqa: E731
    st = _launch(
        dev, lib.mamba_gated_recurrence_bwd,
        ctypes.byref(dims), ptrs[0], ptrs[1], ptrs[2], _ptr(a_param, "a_param", dev, f32, (Dm,)), ptrs[3],
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, f32, (Bt, Dm)), pk,
        _ptr(states, "states", dev, f32, (Bt, -(-L // _lib.RECURRENCE_CHUNK), Dm)), po,
        _ptr(d_final_state, "d_final_state", dev, f32, (Bt, Dm)),
        res("dx"), res("dgate_a"), res("dgate_x"), res("da_param"), res("dz"), res("d_initial_state"),
        _ptr(workspace, "workspace", dev, torch.uint8), 0 if workspace is None else workspace.numel())
    _lib.check(st, "mamba_gated_recurrence_bwd")
    return {k: g[k] for k in shapes}


def gated_recurrence_update(state, x, gate_a, gate_x, a_param, z=None, reset=None, c: float = 8.0, out=None):
    """One step of the gated linear recurrence per row; see
    mamba_gated_recurrence_update.  state (B, D) float32, updated in place; x, gate_a,
    gate_x, z (B, D), dense or slices; reset (B,) uint8/bool.  Returns out (B, D)."""
    torch = _torch()
    dev = _check_device(x)
    if x.dim() != 2:
        raise ValueError("x must be (B, D)")
    dt, f32 = x.dtype, torch.float32
    shape = x.shape
    Bt, Dm = shape
    if reset is not None and reset.dtype == torch.bool:
        reset = reset.to(torch.uint8)
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else torch.empty(shape, dtype=dt, device=dev)
    px, lx = _strided(x, "x", dev, dt, shape)
    pa, la = _strided(gate_a, "gate_a", dev, dt, shape)
    pg, lg = _strided(gate_x, "gate_x", dev, dt, shape)
    pz, lz = _strided(z, "z", dev, dt, shape)
    dims = _recurrence_dims(Bt, 1, Dm, _dtype_code(x), c, (lx, la, lg, lz, 0))
    st = _launch(
        dev, _lib.load().mamba_gated_recurrence_update,
        ctypes.byref(dims), _ptr(state, "state", dev, f32, shape), px, pa, pg,
        _ptr(a_param, "a_param", dev, f32, (Dm,)), pz, _ptr(reset, "reset", dev, torch.uint8, (Bt,)),
        _ptr(out, "out", dev, dt, shape))
    _lib.check(st, "mamba_gated_recurrence_update")
    return out


def _heads(t, name, dev, dtype, shape):
    """(pointer, elements between two tokens) of a (..., H, D) tensor whose heads lie one
    behind the other and whose tokens lie at one distance: dense, or a slice of one
    projection's output.  (None, 0) for None."""
    if t is None:
        return None, 0
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous() and t.device == dev and t.dtype is dtype:
        return t.data_ptr(), 0
    H, D = shape[-2:]
    if (D > 1 and t.stride(-1) != 1) or (H > 1 and D > 0 and t.stride(-2) != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    flat = t.as_strided(tuple(shape[:-2]) + (H * D,), t.stride()[:-2] + (1,))
    return _strided(flat, name, dev, dtype, flat.shape)


def _delta_dims(q, k, v, lead, scale, code, lds=(0, 0, 0, 0)):
    """mamba_delta_dims_t of q, k (*lead, Hk, K) and v (*lead, Hv, V)."""
    Hk, K = q.shape[-2:]
    Hv, V = v.shape[-2:]
    batch, seqlen = lead if len(lead) == 2 else (lead[0], 1)
    if scale is None:
        scale = K ** -0.5 if K else 1.0   # (heads without channels: the library refuses them)
    return _lib.DeltaDims(batch, seqlen, Hk, Hv, K, V, *lds, code, scale)


def _any_strides(query, name, shape, dtype, *more):
    """Bytes that are enough for any strides of q and k: odd ones make the library copy them.  (Where it refuses copies
    as large, it refuses such strides.)"""
    code = _lib.MAMBA_DTYPE_BF16 if dtype == "bf16" else _lib.MAMBA_DTYPE_F32
    width = shape[2] * shape[4]
    odd = width | 1 if 0 < width < 2 ** 21 else 0
    n = ctypes.c_size_t(0)
    for ld in (odd, 0):
        dims = _lib.DeltaDims(*shape, ld, ld, 0, 0, code, 1.0)
        st = query(ctypes.byref(dims), *more, ctypes.byref(n))
        if st != _lib.MAMBA_ERR_UNSUPPORTED:
            break
    _lib.check(st, name)
    return int(n.value)


def gated_delta_rule_workspace_bytes(batch, seqlen, key_heads, value_heads, key_dim, value_dim, dtype="bf16") -> int:
    """Bytes of workspace that are enough for gated_delta_rule_fwd, q and k dense or slices of anything."""
    return _any_strides(_lib.load().mamba_gated_delta_rule_workspace_bytes, "mamba_gated_delta_rule_workspace_bytes",
                        (batch, seqlen, key_heads, value_heads, key_dim, value_dim), dtype)


def gated_delta_rule_fwd(q, k, v, g, beta, doc_start=None, scale=None, initial_state=None, final_state=True, out=None,
                         save=None, workspace=None):
    """Gated delta rule; see mamba_gated_delta_rule_fwd.

    q, k (B, L, Hk, K) and v (B, L, Hv, V) float32/bfloat16, dense or slices of one
    projection's output; g (or None: no decay) and beta (B, L, Hv) float32; doc_start
    (B, L) uint8/bool; ``scale``: K ** -0.5 if not given; initial_state (B, Hv, K, V)
    float32.  ``final_state``: True to allocate and return it, False/None to skip, or a
    tensor to fill.  ``save``: None; "states" to keep the states the backward
    starts its chunks from; or a dict of one such tensor to fill ("states" (B, Hv,
    ceil(L / 64), K, V) float32).  Returns (out (B, L, Hv, V), final_state or None),
    with ``save`` also the dict of what was kept."""
    torch = _torch()
    dev = _check_device(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be (B, L, Hk, K) and v (B, L, Hv, V)")
    code, dt, f32 = _dtype_code(q), q.dtype, torch.float32
    Bt, L, Hk, K = q.shape
    Hv, V = v.shape[-2:]
    state = (Bt, Hv, K, V)
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    if out is None:
        out = torch.empty((Bt, L, Hv, V), dtype=dt, device=dev)
    if final_state is True:
        final_state = torch.empty(state, dtype=f32, device=dev)
    elif final_state is False:
        final_state = None
    pq, lq = _heads(q, "q", dev, dt, q.shape)
    pk, lk = _heads(k, "k", dev, dt, q.shape)
    pv, lv = _heads(v, "v", dev, dt, (Bt, L, Hv, V))
    kept, states, saved = None, None, (Bt, Hv, -(-L // _lib.DELTA_CHUNK), K, V)
    if save is not None:
        if isinstance(save, dict):
            if set(save) - {"states"}:
                raise ValueError(f"save: unknown entries {sorted(set(save) - {'states'})}")
            kept = save
        elif save == "states":
            kept = {"states": torch.empty(saved, dtype=f32, device=dev)}
        else:
            raise ValueError('save must be None, "states" or a dict')
        states = kept.get("states")
    dims = _delta_dims(q, k, v, (Bt, L), scale, code, (lq, lk, lv, 0))
    lib = _lib.load()
    if workspace is None:
        workspace = _recurrence_workspace(lib.mamba_gated_delta_rule_workspace_bytes,
                                          "mamba_gated_delta_rule_workspace_bytes", dev, ctypes.byref(dims))
    st = _launch(
        dev, lib.mamba_gated_delta_rule_fwd, ctypes.byref(dims), pq, pk, pv,
        _ptr(g, "g", dev, f32, (Bt, L, Hv)), _ptr(beta, "beta", dev, f32, (Bt, L, Hv)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, f32, state), _ptr(out, "out", dev, dt, (Bt, L, Hv, V)),
        _ptr(final_state, "final_state", dev, f32, state), _ptr(states, "states", dev, f32, saved),
        _ptr(workspace, "workspace", dev, torch.uint8), 0 if workspace is None else workspace.numel())
    _lib.check(st, "mamba_gated_delta_rule_fwd")
    return (out, final_state) if save is None else (out, final_state, kept)


def gated_delta_rule_bwd_workspace_bytes(batch, seqlen, key_heads, value_heads, key_dim, value_dim, dtype="bf16",
                                         states=False) -> int:
    """The same for gated_delta_rule_bwd (``states``: with those that the forward kept)."""
    return _any_strides(_lib.load().mamba_gated_delta_rule_bwd_workspace_bytes,
                        "mamba_gated_delta_rule_bwd_workspace_bytes",
                        (batch, seqlen, key_heads, value_heads, key_dim, value_dim), dtype, int(bool(states)))


def gated_delta_rule_bwd(q, k, v, g, beta, dout, doc_start=None, scale=None, initial_state=None, d_final_state=None,
                         states=None, workspace=None, grads=None):
    """Gradients of sum(dout * out) + sum(d_final_state * final_state) for the gated
    delta rule; see mamba_gated_delta_rule_bwd.

    q ... initial_state as given to gated_delta_rule_fwd; ``states`` what it kept (or
    None: recomputed); dout (B, L, Hv, V), dense or a slice.  Returns a dict with dq, dk
    (summed over the value heads of a key head), dv (q's dtype), dbeta (B, L, Hv)
    float32 and, for each optional input given, dg (B, L, Hv) and d_initial_state
    (B, Hv, K, V) float32.  ``grads``: optional dict of preallocated outputs with the
    same keys."""
    torch = _torch()
    dev = _check_device(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be (B, L, Hk, K) and v (B, L, Hv, V)")
    code, dt, f32 = _dtype_code(q), q.dtype, torch.float32
    Bt, L, Hk, K = q.shape
    Hv, V = v.shape[-2:]
    state = (Bt, Hv, K, V)
    if doc_start is not None and doc_start.dtype == torch.bool:
        doc_start = doc_start.to(torch.uint8)
    pq, lq = _heads(q, "q", dev, dt, q.shape)
    pk, lk = _heads(k, "k", dev, dt, q.shape)
    pv, lv = _heads(v, "v", dev, dt, (Bt, L, Hv, V))
    po, lo = _heads(dout, "dout", dev, dt, (Bt, L, Hv, V))
    shapes = {"dq": ((Bt, L, Hk, K), dt), "dk": ((Bt, L, Hk, K), dt), "dv": ((Bt, L, Hv, V), dt)}
    if g is not None:
        shapes["dg"] = ((Bt, L, Hv), f32)
    shapes["dbeta"] = ((Bt, L, Hv), f32)
    if initial_state is not None:
        shapes["d_initial_state"] = (state, f32)
    res = dict(grads) if grads else {}
    for n, (sh, d) in shapes.items():
        if n not in res:
            res[n] = torch.empty(sh, dtype=d, device=dev)
    dims = _delta_dims(q, k, v, (Bt, L), scale, code, (lq, lk, lv, lo))
    lib = _lib.load()
    if workspace is None:
        workspace = _recurrence_workspace(lib.mamba_gated_delta_rule_bwd_workspace_bytes,
                                          "mamba_gated_delta_rule_bwd_workspace_bytes", dev, ctypes.byref(dims),
                                          int(states is not None))
    to = lambda n: _ptr(res[n], n, dev, shapes[n][1], shapes[n][0]) if n in shapes else None  # noqa: E731
    st = _launch(
        dev, lib.mamba_gated_delta_rule_bwd, ctypes.byref(dims), pq, pk, pv,
        _ptr(g, "g", dev, f32, (Bt, L, Hv)), _ptr(beta, "beta", dev, f32, (Bt, L, Hv)),
        _ptr(doc_start, "doc_start", dev, torch.uint8, (Bt, L)),
        _ptr(initial_state, "initial_state", dev, f32, state),
        _ptr(states, "states", dev, f32, (Bt, Hv, -(-L // _lib.DELTA_CHUNK), K, V)), po,
        _ptr(d_final_state, "d_final_state", dev, f32, state),
        to("dq"), to("dk"), to("dv"), to("dg"), to("dbeta"), to("d_initial_state"),
        _ptr(workspace, "workspace", dev, torch.uint8), 0 if workspace is None else workspace.numel())
    _lib.check(st, "mamba_gated_delta_rule_bwd")
    return {n: res[n] for n in shapes}


def gated_delta_rule_update(state, q, k, v, g, beta, reset=None, scale=None, out=None):
    """One step of the gated delta rule per row; see mamba_gated_delta_rule_update.
    state (B, Hv, K, V) float32, updated in place; q, k (B, Hk, K), v (B, Hv, V), dense
    or slices; g (or None) and beta (B, Hv) float32; reset (B,) uint8/bool.  Returns out
    (B, Hv, V)."""
    torch = _torch()
    dev = _check_device(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q must be (B, Hk, K) and v (B, Hv, V)")
    code, dt, f32 = _dtype_code(q), q.dtype, torch.float32
    Bt, Hk, K = q.shape
    Hv, V = v.shape[-2:]
    if reset is not None and reset.dtype == torch.bool:
        reset = reset.to(torch.uint8)
    if out is None:
        out = torch.empty((Bt, Hv, V), dtype=dt, device=dev)
    pq, lq = _heads(q, "q", dev, dt, q.shape)
    pk, lk = _heads(k, "k", dev, dt, q.shape)
    pv, lv = _heads(v, "v", dev, dt, (Bt, Hv, V))
    dims = _delta_dims(q, k, v, (Bt,), scale, code, (lq, lk, lv, 0))
    st = _launch(
        dev, _lib.load().mamba_gated_delta_rule_update, ctypes.byref(dims),
        _ptr(state, "state", dev, f32, (Bt, Hv, K, V)), pq, pk, pv, _ptr(g, "g", dev, f32, (Bt, Hv)),
        _ptr(beta, "beta", dev, f32, (Bt, Hv)), _ptr(reset, "reset", dev, torch.uint8, (Bt,)),
        _ptr(out, "out", dev, dt, (Bt, Hv, V)))
    _lib.check(st, "mamba_gated_delta_rule_update")
    return out


def _qk_norm_call(q, k, q_weight, k_weight, cos, sin, positions, norm, eps, interleaved, grads=()):
    """(dims, pointers of the inputs, device, lead, shapes of q and k) of a head norm's call; ``grads``: the gradients
    at the outputs."""
    torch = _torch()
    dev = _check_device(q)
    if q.dim() < 3:
        raise ValueError("q must be (B, L, Hq, D) or (B, Hq, D)")
    if norm not in _lib.NORMS:
        raise ValueError(f"norm must be one of {sorted(_lib.NORMS)}")
    code, dt, f32 = _dtype_code(q), q.dtype, torch.float32
    lead, (Hq, D) = q.shape[:-2], q.shape[-2:]
    if len(lead) > 2:
        raise ValueError("q must be (B, L, Hq, D) or (B, Hq, D)")
    Hk = 0 if k is None else k.shape[-2]
    shapes = (q.shape, None if k is None else lead + (Hk, D))
    pq, lq = _heads(q, "q", dev, dt, shapes[0])
    pk, lk = _heads(k, "k", dev, dt, shapes[1])
    lds, pg = [0, 0], [None, None]
    for i, (t, n) in enumerate(zip(grads, ("dq_out", "dk_out"))):
        if (t is None) != (shapes[i] is None):
            raise ValueError(f"{n} goes with its input")
        pg[i], lds[i] = _heads(t, n, dev, dt, shapes[i])
    rot, table = 0, None
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos must be (rows, R / 2)")
        table = cos.shape
        rot = 2 * table[1]
    elif sin is not None:
        raise ValueError("cos and sin go together")
    dims = _lib.QkNormDims(lead[0], lead[1] if len(lead) == 2 else 1, Hq, Hk, D, rot, 0 if table is None else table[0],
                           lq, lk, *lds, code, _lib.NORMS[norm], int(bool(interleaved)), eps)
    ptrs = (pq, pk, _ptr(q_weight, "q_weight", dev, f32, (D,)), _ptr(k_weight, "k_weight", dev, f32, (D,)),
            _ptr(cos, "cos", dev, f32, table), _ptr(sin, "sin", dev, f32, table),
            _ptr(positions, "positions", dev, torch.int32, lead))
    return dims, ptrs + tuple(pg[:len(grads)]), dev, shapes


def qk_norm_rotary_fwd(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6,
                       interleaved=False, q_out=None, k_out=None):
    """Norms of queries and keys for each head, with the position rotation; see
    mamba_qk_norm_rotary_fwd.

    q (B, L, Hq, D) and k (B, L, Hk, D), or (B, Hq, D) and (B, Hk, D) for one token of
    each row, float32/bfloat16, dense or slices of one projection's output; k may be None.
    q_weight, k_weight (D,) float32 or None; cos, sin (rows, R / 2) float32 or None: no
    rotation; positions (B, L) or (B,) int32 (None: a token's index in its row).  ``norm``:
    "rms" (mean of squares) or "l2" (their sum); ``interleaved``: pairs of neighbouring
    channels, else of the two halves.  Returns (q_out, k_out), dense."""
    torch = _torch()
    dims, ptrs, dev, shapes = _qk_norm_call(q, k, q_weight, k_weight, cos, sin, positions, norm, eps, interleaved)
    if q_out is None:
        q_out = torch.empty(shapes[0], dtype=q.dtype, device=dev)
    if k_out is None and k is not None:
        k_out = torch.empty(shapes[1], dtype=q.dtype, device=dev)
    st = _launch(dev, _lib.load().mamba_qk_norm_rotary_fwd, ctypes.byref(dims), *ptrs,
                 _ptr(q_out, "q_out", dev, q.dtype, shapes[0]), _ptr(k_out, "k_out", dev, q.dtype, shapes[1]))
    _lib.check(st, "mamba_qk_norm_rotary_fwd")
    return q_out, k_out


def qk_norm_rotary_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                       norm="rms", eps=1e-6, interleaved=False, workspace=None, grads=None):
    """Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) for qk_norm_rotary_fwd on
    the same arguments; see mamba_qk_norm_rotary_bwd.  dq_out, dk_out: shaped as q and k,
    dense or slices.  Returns a dict with dq, dk (with a k) and, for each weight given,
    dq_weight, dk_weight (D,) float32.  ``grads``: optional dict of preallocated outputs
    with the same keys."""
    torch = _torch()
    dims, ptrs, dev, shapes = _qk_norm_call(q, k, q_weight, k_weight, cos, sin, positions, norm, eps, interleaved,
                                            (dq_out, dk_out))
    want = {"dq": (shapes[0], q.dtype)}
    if k is not None:
        want["dk"] = (shapes[1], q.dtype)
    for n, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        if w is not None:
            want[n] = (q.shape[-1:], torch.float32)
    res = dict(grads) if grads else {}
    for n, (sh, d) in want.items():
        if n not in res:
            res[n] = torch.empty(sh, dtype=d, device=dev)
    lib = _lib.load()
    if workspace is None and len(want) > (1 if k is None else 2):
        workspace = _recurrence_workspace(lib.mamba_qk_norm_rotary_bwd_workspace_bytes,
                                          "mamba_qk_norm_rotary_bwd_workspace_bytes", dev, ctypes.byref(dims))
    to = lambda n: _ptr(res[n], n, dev, want[n][1], want[n][0]) if n in want else None  # noqa: E731
    st = _launch(dev, lib.mamba_qk_norm_rotary_bwd, ctypes.byref(dims), *ptrs, to("dq"), to("dk"), to("dq_weight"),
                 to("dk_weight"), _ptr(workspace, "workspace", dev, torch.uint8),
                 0 if workspace is None else workspace.numel())
    _lib.check(st, "mamba_qk_norm_rotary_bwd")
    return {n: res[n] for n in want}
