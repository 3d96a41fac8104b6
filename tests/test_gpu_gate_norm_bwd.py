"""Gradients of the per-head RMSNorm and sigmoid gate against fp64 (tests/scan_ref.py derives the bounds)."""
import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from kda_testutil import guarded_empty

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, rows, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    o, ga, dy = (torch.randn((rows, 128), generator=g, device="cuda").clamp(-6, 6).to(dtype) for _ in range(3))
    return o, ga, dy, 1 + 0.3 * torch.randn(128, generator=g, device="cuda")


def check(o, ga, dy, w, r, eps=1e-6):
    d_o, oe, d_g, ge, d_w, we = scan_ref.gate_norm_bwd(o, ga, dy, w, eps)
    scan_ref.assert_within(r["d_o"], d_o, oe, "d_o")
    scan_ref.assert_within(r["d_gate"], d_g, ge, "d_gate")
    if r["d_norm_weight"] is not None:
        scan_ref.assert_within(r["d_norm_weight"], d_w, we, "d_norm_weight")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gout", [BF, F32])
@pytest.mark.parametrize("rows", [1, 2, 3, 15, 16, 17, 301, 5000])
@pytest.mark.parametrize("weight", [True, False])
def test_sizes(dtype, gout, rows, weight):
    o, ga, dy, w = inputs(rows, rows, dtype)
    w = w if weight else None
    check(o, ga, dy, w, kda.gate_norm_bwd(o, ga, dy, w, out_dtype=gout))


def test_many_rows_and_the_same_bits():
    o, ga, dy, w = inputs(5, 100_003, BF)
    a = kda.gate_norm_bwd(o, ga, dy, w)
    check(o, ga, dy, w, a)
    for _ in range(3):
        b = kda.gate_norm_bwd(o, ga, dy, w)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_scales_and_zero_rows():
    o, ga, dy, w = inputs(7, 64, F32)
    o[:16] *= 1e-4   # next to eps
    o[16:32] *= 1e4
    o[32:40] = 0
    check(o, ga, dy, w, kda.gate_norm_bwd(o, ga, dy, w))
    check(o, ga, dy, w, kda.gate_norm_bwd(o, ga, dy, w, eps=1e-2), eps=1e-2)


def test_gate_ends():
    """Gates so large that sigmoid is 0 or 1: finite gradients."""
    o, ga, dy, w = inputs(9, 8, F32)
    ga[:4], ga[4:] = 200.0, -200.0
    r = kda.gate_norm_bwd(o, ga, dy, w)
    assert (r["d_gate"] == 0).all() and (r["d_o"][4:] == 0).all() and torch.isfinite(r["d_o"]).all()


def test_layout_and_options():
    o, ga, dy, w = inputs(11, 60, BF)
    v = lambda t: t.view(2, 10, 3, 128)  # noqa: E731
    a, b = kda.gate_norm_bwd(o, ga, dy, w), kda.gate_norm_bwd(v(o), v(ga), v(dy), w, want_d_norm_weight=False)
    assert b["d_norm_weight"] is None and b["d_o"].shape == (2, 10, 3, 128)
    assert torch.equal(a["d_o"], b["d_o"].view(60, 128)) and torch.equal(a["d_gate"], b["d_gate"].view(60, 128))
    e = kda.gate_norm_bwd(o[:0], ga[:0], dy[:0], w)
    assert e["d_o"].shape == (0, 128) and (e["d_norm_weight"] == 0).all()


def test_against_differences_of_the_forward():
    """The gradient of sum(y dy) along a direction, against gate_norm's own outputs."""
    o, ga, dy, w = inputs(13, 40, F32)
    g = torch.Generator(device="cuda").manual_seed(1)
    do, dg = (torch.randn((40, 128), generator=g, device="cuda") for _ in range(2))
    r = kda.gate_norm_bwd(o, ga, dy, w)
    step = 2.0 ** -7
    f = lambda k: (kda.gate_norm(o + k * step * do, ga + k * step * dg, w).double() * dy.double()).sum()  # noqa: E731
    num = (8 * (f(1) - f(-1)) - (f(2) - f(-2))) / (12 * step)
    got = (r["d_o"].double() * do.double()).sum() + (r["d_gate"].double() * dg.double()).sum()
    # the difference's own error: step^4 times fifth derivatives of the terms (of their size), and each y's
    # rounding (32 of 2^-24) over the step, 5120 terms adding up like their root
    size = float((r["d_o"].double() * do.double()).abs().sum() + (r["d_gate"].double() * dg.double()).abs().sum())
    tol = 30 * step ** 4 * size + 4 * 32 * 2.0 ** -24 / step * float((dy.double() ** 2).sum().sqrt()) * 3
    assert abs(float(num - got)) <= tol, (float(num), float(got), tol)


def test_guards_stream_graph():
    o, ga, dy, w = inputs(17, 333, BF)
    want = kda.gate_norm_bwd(o, ga, dy, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = kda.gate_norm_bwd(o, ga, dy, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(want[k], r[k]) for k in want)
    so = torch.zeros_like(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = kda.gate_norm_bwd(so, ga, dy, w)
    so.copy_(o)
    g.replay()
    assert all(torch.equal(want[k], r[k]) for k in want)


def test_refusals():
    o, ga, dy, w = inputs(19, 4, BF)
    with pytest.raises(TypeError):
        kda.gate_norm_bwd(o, ga.float(), dy)
    with pytest.raises(ValueError):
        kda.gate_norm_bwd(o, ga[:2], dy)
    with pytest.raises(kda.KdaError):
        kda.gate_norm_bwd(o[:, :64].contiguous(), ga[:, :64].contiguous(), dy[:, :64].contiguous())
    with pytest.raises(ValueError):
        kda.gate_norm_bwd(o, ga, dy, w[:64])
    with pytest.raises(kda.KdaError):
        kda.gate_norm_bwd(o, ga, dy, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
