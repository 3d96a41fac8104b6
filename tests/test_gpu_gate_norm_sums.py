"""The gate norm's weight gradient and its ends: sums over more rows than one turn of the kernel's loop, eps = 0, gates
next to open (tests/scan_ref.py derives the bounds that are not derived here)."""
import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from test_gpu_gate_norm_bwd import check, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 3, 15, 301, 9473])
def test_eps_of_zero(dtype, rows):
    """Rows that no half warp has beside it: 1 / sqrt(0 + 0) of nothing must not reach the weight's sum."""
    o, ga, dy, w = inputs(rows + 100, rows, dtype)
    check(o, ga, dy, w, kda.gate_norm_bwd(o, ga, dy, w, eps=0.0), eps=0.0)


def weight_sum_bound(rows, terms_abs):
    """e (2^-24) times the roundings on a term's way: 45 of its factors (as scan_ref), one per row that a half warp
    walks (592 CTAs of 16 half warps at most), 16 half warps of a CTA, at most 19 partial sums per thread of the second
    kernel, 32 of those."""
    blocks = min(-(-rows // 16), 592)
    turns = -(-rows // (16 * blocks))
    return scan_ref.EPS * (45 + turns + 16 + 19 + 32) * terms_abs


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [5000, 9471, 9472, 9473, 18945, 100_003])
def test_weight_sums_of_every_turn(dtype, rows):
    """A half warp's rows of one turn or several, all CTAs' sums: no row is missing and none counted twice."""
    o, ga, dy, w = inputs(rows, rows, dtype)
    got = kda.gate_norm_bwd(o, ga, dy, w)["d_norm_weight"]
    terms = dy.double() * torch.sigmoid(ga.double()) * o.double() / (o.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
    bound = weight_sum_bound(rows, terms.abs().sum(0))
    scan_ref.assert_within(got, terms.sum(0), bound, "d_norm_weight")
    # a turn, a CTA's or a half warp's rows left out would be seen
    turn = slice(max(0, rows - 9472), rows)
    for part in (turn, slice(0, rows, 16)):
        assert ((terms[part].sum(0)).abs() > 2 * bound).float().mean() > 0.5


@pytest.mark.parametrize("gate", [7.0, 9.0, 12.0, 16.0, 30.0, 80.0])
def test_gradient_of_open_gates(gate):
    """1 - sigmoid keeps its digits where the sigmoid is next to 1.  e^-g is off by 2 + 1.173 g ulps (2 e each), the
    sigmoid beside it by 6 e, n by 11 e, products 4 e: relative to the value."""
    o, ga, dy, w = inputs(int(gate), 50, F32)
    ga = gate + 0.1 * ga
    got = kda.gate_norm_bwd(o, ga, dy, w)["d_gate"]
    o, ga, dy = (t.double() for t in (o, ga, dy))
    n = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    ref = dy * n * w.double() * torch.sigmoid(ga) * torch.sigmoid(-ga)
    scan_ref.assert_within(got, ref, scan_ref.EPS * (2 * (2 + 1.173 * ga) + 21) * ref.abs(), "d_gate")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_at_both_ends(dtype):
    """Shut gates and open ones, to infinity: zeros or what is left, no NaN; a NaN stays NaN."""
    o, ga, dy, w = inputs(3, 16, dtype)
    ends = torch.tensor([-float("inf"), -200.0, -88.5, -88.0, -87.0, 87.0, 200.0, float("inf")], device="cuda").to(dtype)
    ga = ends[torch.arange(ga.numel(), device="cuda") * 3 % 8].view_as(ga).clone()
    r = kda.gate_norm_bwd(o, ga, dy, w)
    assert all(torch.isfinite(r[k]).all() for k in r)
    assert (r["d_gate"].abs() <= 1e-36).all() and (r["d_gate"][torch.isinf(ga)] == 0).all()
    ga[2, 5] = float("nan")
    r = kda.gate_norm_bwd(o, ga, dy, w)
    assert torch.isnan(r["d_gate"][2, 5]) and torch.isnan(r["d_o"][2]).all()
    assert all(torch.isfinite(r[k][torch.arange(16, device="cuda") != 2]).all() for k in ("d_o", "d_gate"))
