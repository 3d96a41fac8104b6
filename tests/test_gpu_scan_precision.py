"""What the element-wise scan keeps of its digits where a rounding would show: gates next to open, states and gradients
handed from call to call, decays next to 1 (tests/scan_ref.py derives the bounds that are not derived here)."""
import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from test_gpu_scan import as_cu, inputs, ref_of, run_both

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("gate", [7.0, 9.0, 12.0, 16.0, 30.0])
def test_gate_gradient_of_open_gates(dtype, norm, gate):
    """dgate = G u (1 - s) = dx x (1 - s), 1 - s = e^-gate s.  dx's own bound holds 40 e of its G beside what G carries:
    enough for u's 36 as well.  e^-gate is off by 2 ulps (2 e each) of the hardware's 2^y and gate e of y's two
    roundings, s by 4 e, products 3 e: relative to 1 - s, a (12 + gate) / 40 part of that bound again.  The reference
    is dx x / (1 + e^gate): its own 1 - s of 64 bits is off by 2^-53 absolute, 1e-3 of the value at a gate of 30."""
    i = inputs(int(gate), 2, 150, 72, dtype)
    i["gate"] = (gate + 0.1 * i["gate"].float()).to(dtype)
    r = ref_of(i, True, norm, True, None, True)
    _, _, gr = run_both(i, True, norm)
    ga = i["gate"].double().cpu()
    rest = i["x"].double().cpu() * torch.sigmoid(-ga)
    scan_ref.assert_within(gr["dgate"], rest * r["dx"], rest.abs() * r["dx_e"] * (1 + (12 + ga) / 40), "dgate")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_of_infinity(dtype):
    """A shut gate lets exactly nothing through, also of huge values; an open one has no gradient; NaN stays."""
    i = inputs(5, 1, 60, 40, dtype)
    ends = torch.tensor([-float("inf"), -200.0, -89.0, 200.0, float("inf")], device="cuda").to(dtype)
    i["gate"] = ends[torch.arange(i["gate"].numel(), device="cuda") * 3 % 5].view_as(i["gate"]).clone()
    shut = i["gate"] < 0
    i["x"][shut] = 1e30
    _, _, gr = run_both(i, True, False)
    assert all(torch.isfinite(t).all() for t in gr.values())
    assert (gr["dx"][shut] == 0).all() and (gr["dgate"][i["gate"] == float("inf")] == 0).all()
    i["gate"][0, 30, 7] = float("nan")
    _, _, gr = run_both(i, True, False)
    assert torch.isnan(gr["dgate"][0, 30, 7]) and torch.isnan(gr["dx"][0, 30, 7])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays_are_not_one_sided(dtype):
    """Products of 16 decays of e^-0.12 to e^-0.02, forwards (a state of 1) and back (a gradient of 1).  A value has up
    to 32 roundings of half a step (e = 2^-24), either way: 6 of the mean's deviations over 4096 channels are
    6 e sqrt(32 / 3) / 64 = 0.31 e.  One way goes what a's series leaves out, d^6 / 720 a token: 16 of them come to
    1.1 e at d = 0.12 and to 0.2 e on average.  A decay off by e the same way at every token gives 16 e: so much, and
    twice, is allowed where tokens are bf16, whose decays are the hardware's 2^y (2 ulps; y's rounding 0.3 e)."""
    T, D = 16, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    la = -(0.02 + 0.1 * torch.rand((1, T, D), generator=g, device="cuda")).to(dtype)
    x, one = torch.zeros((1, T, D), device="cuda").to(dtype), torch.ones((1, D), device="cuda")
    h = kda.scan_fwd(x, la, one, out_dtype=F32)[0]
    dx = kda.scan_bwd(x, la, x, None, one)["dx"]
    sums = la.double().cumsum(1)
    for got, ref in ((h[:, -1], sums[:, -1].exp()), (dx[:, 0], (sums[:, -1] - la[:, 0].double()).exp())):
        mean = float((got.double() / ref - 1).mean())
        assert abs(mean) <= (0.6 if dtype == F32 else 16 * 2.3) * scan_ref.EPS, mean / scan_ref.EPS


def slow_channels(D, N, dtype):
    """Log-decays of -1e-5 to -2e-5, constant per sequence and channel."""
    g = torch.Generator(device="cuda").manual_seed(1)
    return (-1e-5 * (1 + torch.rand((N, D), generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1, 1, 1], [5, 5, 5], [16], [16, 21], [8, 3, 13]], ids=str)
def test_slow_decay_keeps_its_rate_from_call_to_call(dtype, lens):
    """Some 10000 tokens a sequence in short packed calls, the state handed on, and back, the gradient handed on: decays of
    1 - 1e-5 to 1 - 2e-5, whose own rounding would put a rate off by up to 2^-25 in 1e-5, 3e-3 of it (5e-4 of such a
    state over the channels).  As test_slow_decay_keeps_its_rate: two roundings a token of random sign add
    up to 2^-24 sqrt(2 T / 3) / sqrt(2), 3.5e-6 of a random walk's size for T = 10000, one more per call at most doubles
    their number; allowed is six times 2^-24 sqrt(4 T / 3) / sqrt(2) = 5e-6."""
    D, N, calls = 64, len(lens), 10000 // max(lens)
    cu = [sum(lens[:n]) for n in range(N + 1)]
    l = slow_channels(D, N, dtype)
    la = torch.cat([l[n:n + 1].expand(k, D) for n, k in enumerate(lens)])[None].contiguous()
    g = torch.Generator(device="cuda").manual_seed(4)
    xs = torch.randn((calls, 1, cu[-1], D), generator=g, device="cuda").to(dtype)
    state, grad = None, None
    for c in range(calls):
        state = kda.scan_fwd(xs[c], la, state, cu_seqlens=as_cu(cu))[1]
    zero = torch.zeros_like(la)
    for c in range(calls):
        grad = kda.scan_bwd(zero, la, xs[calls - 1 - c], None, grad, cu_seqlens=as_cu(cu))["d_initial_state"]
    for n, k in enumerate(lens):
        x = xs[:, 0, cu[n]:cu[n + 1]].reshape(calls * k, D).double()
        ago = torch.arange(calls * k, device="cuda", dtype=torch.float64)[:, None]
        fwd = (x * torch.exp(ago.flip(0) * l[n].double())).sum(0)
        bwd = (x * torch.exp((ago + 1) * l[n].double())).sum(0)
        for got, ref in ((state[n], fwd), (grad[n], bwd)):
            assert float((got.double() - ref).norm() / ref.norm()) < 3e-5, (n, k)
