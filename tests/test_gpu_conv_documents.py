"""Conv backward: a NaN or an infinity at the head of a document reaches no gradient of
the document before it, nor the history that the row continues."""

import numpy as np
import pytest

from workloads import bf16_round, make_cotangent, make_custom
from workloads.device import to_dev, upload

pytestmark = pytest.mark.gpu

STARTS = (20, 46, 48, 49, 97, 110, 145)    # inside, at and around the 48-token tiles' edges


@pytest.fixture(scope="module")
def ssm():
    import torch

    import selective_state_space_23_amd as s
    if not torch.cuda.is_available():
        pytest.fail("no GPU")
    return s


def same_bits(a, b):
    import torch

    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [130, 63])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("silu", [True, False])
def test_bad_values_stay_in_their_document(ssm, dtype, D, packed, silu):
    import torch

    B, L = 2, 150
    inp = make_custom(B, L, D, 4, dtype=dtype, docs=40.0, seed=D)
    d = upload(inp)
    doc = torch.zeros(B, L, dtype=torch.uint8, device="cuda")
    doc[:, [0, *STARTS]] = 1
    du = to_dev(make_cotangent(B, L, D, dtype=dtype, seed=5), dtype)
    hist = to_dev(bf16_round(np.random.default_rng(6).standard_normal((B, D, 3)).astype(np.float32)), dtype)

    def run(x, du):
        if packed:
            x = ssm.activation_pack(x)
        return ssm.causal_conv1d_bwd(x, d["conv_w"], du, d["conv_b"], doc, apply_silu=silu, conv_state=hist)

    dx, _, _, dh = run(d["x"], du)
    assert not dh.any()                       # token 0 starts a document
    for bad in (float("nan"), float("inf")):
        for where in ("x", "du"):
            for k, (s, e) in enumerate(zip((0, *STARTS), (*STARTS, L))):
                for t in range(s, min(s + 3, e)):
                    x2, du2 = d["x"].clone(), du.clone()
                    (x2 if where == "x" else du2)[:, t, 1] = bad
                    got, _, _, gh = run(x2, du2)
                    what = (bad, where, s, t)
                    assert same_bits(got[:, :s], dx[:, :s]) and same_bits(got[:, e:], dx[:, e:]), what
                    assert not gh.any(), what
                    assert not got[:, t, 1].float().isfinite().any() or where == "x", what


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [130, 63])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("silu", [True, False])
def test_many_rows_as_each_alone(ssm, dtype, D, packed, silu):
    """2304 workgroups, which take tiles without a document start by a loop of their own:
    rows of the call give the same dx, bit for bit, as a call of one row, which does not."""
    import torch

    B, L = 64, 1700
    g = torch.Generator(device="cuda").manual_seed(D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, du = (torch.randn(B, L, D, generator=g, device="cuda").to(dt) for _ in range(2))
    hist = torch.randn(B, D, 3, generator=g, device="cuda").to(dt)
    w = torch.randn(D, 4, generator=g, device="cuda")
    bias = torch.randn(D, generator=g, device="cuda")
    doc = (torch.rand(B, L, generator=g, device="cuda") < 1 / 300).to(torch.uint8)
    doc[::2, 0] = 1
    doc[5] = 0
    pack = ssm.activation_pack if packed else lambda t: t
    dx, dw, db, dh = ssm.causal_conv1d_bwd(pack(x), w, du, bias, doc, silu, conv_state=hist)
    sw, sb = torch.zeros(D, 4, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for b in range(B):
        s = slice(b, b + 1)
        rx, rw, rb, rh = ssm.causal_conv1d_bwd(pack(x[s]), w, du[s], bias, doc[s], silu, conv_state=hist[s])
        assert same_bits(dx[s], rx) and same_bits(dh[s], rh), b
        sw += rw
        sb += rb
    # sums of 2304 parts, 72 of them one after the other: 88 roundings of 2^-24 of a partial sum, which
    # stays below 3 times the sum's own spread, sqrt(B L) |dw| per token (about 1 here; 4 for four taps)
    tol = 88 * 2.0 ** -24 * 3 * 4 * (B * L) ** 0.5
    assert (dw - sw).abs().max() <= tol and (db - sb).abs().max() <= tol
