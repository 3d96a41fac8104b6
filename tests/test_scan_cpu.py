"""What needs no GPU of the element-wise scan, the gate norm's gradient and the state pages: the reference's gradients
against differences, the workspace sizes and every refusal (none of these calls reaches CUDA)."""
import ctypes

import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from linear_attention_recurrence_06_b200 import build as kbuild

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 10]])
def test_reference_gradients_against_differences(gate, normalize, cu):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    B, T, D = (1, 10, 3) if cu else (2, 5, 3)
    N = len(cu) - 1 if cu else B
    x, la, dh = r(B, T, D), -torch.rand((B, T, D), generator=g, dtype=torch.float64) * 2 - 0.01, r(B, T, D)
    la[0, 1, 0] = 0.3  # above 0: clamped
    ga = r(B, T, D) if gate else None
    init, df = r(N, D), r(N, D)

    def loss(x=x, la=la, ga=ga, init=init):
        f = scan_ref.scan(x, la, ga, normalize, init, cu)
        return float((f["h"] * dh).sum() + (f["final"] * df).sum())

    ref = scan_ref.scan(x, la, ga, normalize, init, cu, dh, df)
    for name, t, key in (("x", x, "dx"), ("la", la, "dl"), ("ga", ga, "dgate"), ("init", init, "d_init")):
        if t is None:
            continue
        for k in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[k] = 1e-6
            d = d.reshape(t.shape)
            num = (loss(**{name: t + d}) - loss(**{name: t - d})) / 2e-6
            got = float(ref[key].reshape(-1)[k])
            if name == "la" and float(la.reshape(-1)[k]) > 0 and normalize:
                assert got == 0  # w = 0 on both sides of the step
            assert abs(num - got) <= 1e-6 * (1 + abs(num)), (name, k, num, got)


def test_reference_gate_norm_gradients():
    g = torch.Generator().manual_seed(6)
    o, ga, dy = (torch.randn((5, 128), generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.rand(128, generator=g, dtype=torch.float64) + 0.5
    o, ga, w = (t.requires_grad_() for t in (o, ga, w))
    y = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) * w * torch.sigmoid(ga)
    y.backward(dy)
    d_o, _, d_g, _, d_w, _ = scan_ref.gate_norm_bwd(o.detach(), ga.detach(), dy, w.detach())
    for got, ref in ((d_o, o.grad), (d_g, ga.grad), (d_w, w.grad)):
        assert torch.allclose(got, ref, rtol=1e-10, atol=1e-12)


def test_workspace_sizes(lib):
    assert kda.scan_bwd_workspace_size(1, 1, 5) == 256 + 20
    assert kda.scan_bwd_workspace_size(3, 60, 8) == 256 + 23 * 32  # a row for every 8 of 180 tokens
    assert kda.scan_bwd_workspace_size(2, 0, 8) == 256
    with pytest.raises(kda.KdaError):
        kda.scan_bwd_workspace_size(0, 64, 8)
    n = ctypes.c_size_t(0)
    assert lib.kda_gate_norm_bwd_workspace_size(1000, 128, ctypes.byref(n)) == 0 and n.value % 512 == 0
    assert lib.kda_gate_norm_bwd_workspace_size(1000, 64, ctypes.byref(n)) == -2
    assert lib.kda_gate_norm_bwd_workspace_size(-1, 128, ctypes.byref(n)) == -1


def test_scan_fwd_refusals(lib):
    def f(**o):
        a = dict(x=FAKE, la=FAKE, g=FAKE, s0=FAKE, h=FAKE, fs=FAKE, cs=FAKE, B=2, T=10, D=24, lx=0, ll=0, lg=0,
                 cu=None, N=0, idt=1, odt=1, norm=0, ws=None, wsb=0)
        a.update(o)
        return lib.kda_scan_fwd(*a.values(), None)
    assert f(x=None) == -1 and f(la=None) == -1 and f(h=None) == -1
    assert f(B=0) == -1 and f(T=-1) == -1 and f(D=0) == -1
    assert f(idt=2) == -1 and f(odt=-1) == -1
    assert f(lx=23) == -1 and f(ll=1) == -1 and f(lg=-24) == -1
    assert f(cu=FAKE, N=2) == -1             # packed sequences: B = 1
    assert f(cu=FAKE, B=1, N=0) == -1
    assert f(cu=FAKE, B=1, N=1, T=1 << 31) == -2
    assert f(T=1 << 41) == -2 and f(B=1 << 20, T=2048) == -2 and f(D=(1 << 28) + 1) == -2
    assert f(x=FAKE + 1) == -3 and f(la=FAKE + 2, idt=0) == -3
    assert f(s0=FAKE + 8) == -3 and f(h=FAKE + 2) == -3 and f(fs=FAKE + 4) == -3 and f(cs=FAKE + 4) == -3
    assert f(cu=FAKE + 2, B=1, N=1) == -3 and f(ws=FAKE, wsb=255) == -4 and f(ws=FAKE + 8, wsb=256) == -3


def test_scan_bwd_refusals(lib):
    def f(**o):
        a = dict(x=FAKE, la=FAKE, g=FAKE, s0=None, dh=FAKE, df=None, cs=FAKE, dx=FAKE, dl=FAKE, dg=FAKE, di=None, B=1,
                 T=10, D=24, lx=0, ll=0, lg=0, lh=0, cu=None, N=0, idt=1, odt=0, norm=1, ws=None, wsb=0)
        a.update(o)
        return lib.kda_scan_bwd(*a.values(), None)
    assert f(dh=None) == -1 and f(dx=None) == -1 and f(dl=None) == -1
    assert f(dg=None) == -1 and f(g=None) == -1    # a gate and its gradient come together
    assert f(lh=5) == -1
    assert f(cs=None) == -4 and f(cs=None, ws=FAKE, wsb=256) == -4
    assert f(dx=FAKE + 4) == -3 and f(di=FAKE + 4) == -3 and f(df=FAKE + 4) == -3 and f(dh=FAKE + 1) == -3
    assert f(odt=3) == -1


def test_scan_decode_refusals(lib):
    def f(**o):
        a = dict(state=FAKE, x=FAKE, la=FAKE, g=None, h=FAKE, slots=FAKE, P=4, n=1, Bd=4, D=8, idt=1, odt=1, norm=0,
                 ss=None)
        a.update(o)
        return lib.kda_scan_decode_steps(*a.values(), None)
    assert f(state=None) == -1 and f(x=None) == -1 and f(h=None) == -1
    assert f(n=-1) == -1 and f(Bd=-1) == -1 and f(D=0) == -1 and f(P=-1) == -1 and f(idt=9) == -1
    assert f(slots=None, P=3) == -1                # a state for every row
    assert f(Bd=65536) == -2
    assert f(slots=FAKE + 2) == -3 and f(state=FAKE + 8) == -3
    assert f(n=0) == 0 and f(Bd=0) == 0            # nothing to do, no launch


def test_paged_decode_refusals(lib):
    def f(**o):
        a = dict(state=FAKE, slots=FAKE, P=4, q=FAKE, k=FAKE, v=FAKE, la=FAKE, b=FAKE, o=FAKE, n=1, Bd=4, H=2, dk=128,
                 dv=128, idt=1, odt=1, scale=1.0, g=None, w=None, eps=1e-6, ss=None)
        a.update(o)
        return lib.kda_decode_steps_paged(*a.values(), None)
    assert f(slots=None) == -1 and f(P=-1) == -1 and f(q=None) == -1
    assert f(dk=64) == -2 and f(slots=FAKE + 2) == -3 and f(k=FAKE + 8) == -3
    assert f(Bd=0) == 0


def test_gate_norm_bwd_refusals(lib):
    def f(**o):
        a = dict(o=FAKE, g=FAKE, dy=FAKE, w=None, eps=1e-6, do=FAKE, dg=FAKE, dw=FAKE, rows=4, dv=128, idt=1, odt=1,
                 ws=FAKE, wsb=1 << 30)
        a.update(o)
        return lib.kda_gate_norm_bwd(*a.values(), None)
    assert f(o=None) == -1 and f(dy=None) == -1 and f(do=None) == -1 and f(rows=-1) == -1
    assert f(eps=-1.0) == -1 and f(eps=float("nan")) == -1 and f(idt=4) == -1
    assert f(dv=64) == -2 and f(dy=FAKE + 8) == -3
    assert f(ws=None) == -4 and f(wsb=4) == -4


def test_state_page_refusals(lib):
    def f(**o):
        a = dict(dst=FAKE, src=FAKE, L=1, page=64, P=4, Q=4, dl=0, sl=0, ds=FAKE, ss=FAKE, n=2)
        a.update(o)
        return lib.kda_state_copy(*a.values(), None)
    assert f(dst=None) == -1 and f(src=None) == -1 and f(ds=None) == -1 and f(ss=None) == -1
    assert f(page=0) == -1 and f(page=6) == -1 and f(n=-1) == -1 and f(P=-1) == -1
    assert f(n=65536) == -2 and f(L=65536, dl=256, sl=256) == -2
    assert f(dst=FAKE + 8) == -3 and f(ds=FAKE + 2) == -3 and f(ss=FAKE + 1) == -3
    assert f(src=FAKE + 64) == -1                  # overlaps without being the same pool
    assert f(src=FAKE + 64 * 3, Q=1) == -1
    assert f(L=2, dl=128, sl=256) == -1            # layers on top of one another
    assert f(L=2, dl=256, sl=320) == -1            # one pool under two strides
    assert f(n=0) == 0 and f(L=0) == 0
    assert lib.kda_state_alloc(None, 4, FAKE, 2, None) == -1
    assert lib.kda_state_alloc(FAKE, -1, FAKE, 2, None) == -1
    assert lib.kda_state_alloc(FAKE, 4, FAKE + 2, 2, None) == -3
    assert lib.kda_state_free(FAKE, 4, None, 2, None) == -1
    assert lib.kda_state_free(FAKE, 4, None, 0, None) == 0
    assert lib.kda_state_compact(FAKE, 4, None, FAKE, FAKE, FAKE, None) == -1
    assert lib.kda_state_compact(FAKE, -1, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert lib.kda_state_compact(FAKE, 4, FAKE, FAKE, FAKE, FAKE + 2, None) == -3


def test_binding_refuses_cpu_tensors():
    x, s, i = torch.zeros(1, 4, 8), torch.zeros(1, 8), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: kda.scan_fwd(x, x), lambda: kda.scan_bwd(x, x, x), lambda: kda.scan_decode_steps(s, x, x),
                 lambda: kda.gate_norm_bwd(torch.zeros(2, 128), torch.zeros(2, 128), torch.zeros(2, 128)),
                 lambda: kda.state_copy(s, i, s, i), lambda: kda.state_compact(torch.zeros(3, dtype=torch.uint8)),
                 lambda: kda.state_alloc(torch.zeros(3, dtype=torch.uint8), 1),
                 lambda: kda.state_free(torch.zeros(3, dtype=torch.uint8), i)):
        with pytest.raises(ValueError):
            call()


def test_token_rows():
    """What of a strided input the scan takes as it lies."""
    x = torch.zeros(2, 6, 4, 8)
    wide = torch.zeros(2, 6, 3, 4, 8)

    class Cuda(torch.Tensor):  # a host tensor that says it is on a GPU
        is_cuda = True
    c = lambda t: t.as_subclass(Cuda)  # noqa: E731
    assert kda._token_rows(c(x), c(x), "x") == 0
    assert kda._token_rows(c(x), c(wide[:, :, 1]), "x") == 96
    assert kda._token_rows(c(x[:1]), c(wide[:1, :, 2]), "x") == 96
    assert kda._token_rows(c(x[:, :1]), c(wide[:, :1, 1]), "x") == 6 * 96  # one token each: the batch's distance
    with pytest.raises(ValueError):
        kda._token_rows(c(x), c(torch.zeros(2, 6, 4, 16)[..., :8]), "x")            # heads apart
    with pytest.raises(ValueError):
        kda._token_rows(c(x), c(torch.zeros(2, 12, 4, 8)[:, :6]), "x")     # rows of a longer buffer
    with pytest.raises(ValueError):
        kda._token_rows(c(x), c(torch.zeros(2, 1, 4, 8).expand(2, 6, 4, 8)), "x")
    with pytest.raises(ValueError):
        kda._token_rows(c(x), c(torch.zeros(2, 6, 8, 4)), "x")
    with pytest.raises(TypeError):
        kda._token_rows(c(x), c(x.bfloat16()), "x")
