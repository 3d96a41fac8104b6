"""The element-wise gated scan on a GPU against its fp64 reference (tests/scan_ref.py, which derives the bounds)."""
import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from kda_testutil import guarded_empty

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, B, T, D, dtype, N=None, slow=True):
    """Decays from a memory of a token to one of thousands; gates within +-6."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rate = torch.exp(torch.rand(D, generator=g, device="cuda") * 8 - 7.5) if slow else torch.ones(D, device="cuda")
    N = B if N is None else N
    return dict(x=r(B, T, D).to(dtype), la=(-rate * torch.sigmoid(r(B, T, D)) * 2).to(dtype),
                gate=r(B, T, D).clamp(-6, 6).to(dtype), init=r(N, D), dh=r(B, T, D).to(dtype), dfin=r(N, D))


def cpu(t):
    return None if t is None else t.cpu()


def ref_of(i, gate, norm, init, cu=None, grads=False):
    return scan_ref.scan(cpu(i["x"]), cpu(i["la"]), cpu(i["gate"]) if gate else None, norm,
                         cpu(i["init"]) if init else None, cu, cpu(i["dh"]) if grads else None,
                         cpu(i["dfin"]) if grads and init else None)


def as_cu(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def in_sequences(cu, T):
    m = torch.zeros(T, dtype=torch.bool)
    m[cu[0]:cu[-1]] = True
    return m


def run_both(i, gate=True, norm=True, init=True, cu=None, out=None, gout=F32, given_states=True):
    g, s0, df = (i["gate"] if gate else None), (i["init"] if init else None), (i["dfin"] if init else None)
    c = as_cu(cu)
    h, fin, cs = kda.scan_fwd(i["x"], i["la"], s0, gate=g, normalize=norm, cu_seqlens=c, out_dtype=out,
                              chunk_states=True)
    gr = kda.scan_bwd(i["x"], i["la"], i["dh"], s0, df, gate=g, normalize=norm, cu_seqlens=c,
                      chunk_states=cs if given_states else None, out_dtype=gout)
    return h, fin, gr


def check(i, gate=True, norm=True, init=True, cu=None, out=None, gout=F32, given_states=True):
    h, fin, gr = run_both(i, gate, norm, init, cu, out, gout, given_states)
    r = ref_of(i, gate, norm, init, cu, True)
    rows = slice(None) if cu is None else slice(cu[0], cu[-1])
    cut = lambda t: t[:, rows]  # noqa: E731
    scan_ref.assert_within(cut(h), cut(r["h"]), cut(r["h_e"]), "h")
    scan_ref.assert_within(fin, r["final"], r["final_e"], "final state")
    for got, key in ((gr["dx"], "dx"), (gr["dlog_alpha"], "dl"), (gr["dgate"], "dgate")):
        if got is not None:
            scan_ref.assert_within(cut(got), cut(r[key]), cut(r[key + "_e"]), key)
    scan_ref.assert_within(gr["d_initial_state"], r["d_init"], r["d_init_e"], "d_initial_state")
    assert (gr["dgate"] is None) == (not gate)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (3, 1, 64), (1, 2, 7), (2, 63, 64), (1, 64, 65), (2, 65, 130), (1, 127, 8),
                                   (1, 128, 200), (3, 129, 72), (2, 200, 33), (1, 1000, 96), (5, 37, 256)])
def test_sizes(dtype, B, T, D):
    check(inputs(B * 1000 + T + D, B, T, D, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("init", [False, True])
def test_forms(dtype, gate, norm, init):
    check(inputs(7, 2, 150, 72, dtype), gate, norm, init)


@pytest.mark.parametrize("dtype,out,gout", [(BF, F32, BF), (F32, BF, BF), (BF, BF, F32)])
@pytest.mark.parametrize("D", [72, 67])
def test_output_types(dtype, out, gout, D):
    check(inputs(11, 2, 150, D, dtype), out=out, gout=gout)


CUS = [[0, 5], [0, 0, 5], [0, 1, 2, 3, 3, 3, 4], [0, 64, 128, 192], [0, 63, 65, 128, 129], [0, 300, 301, 301, 700],
       [0, 0, 0], [0, 128, 129, 257, 600, 600]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cu", CUS, ids=str)
@pytest.mark.parametrize("given_states", [True, False])
def test_packed(dtype, cu, given_states):
    T = max(cu[-1], 1)
    check(inputs(13 + len(cu), 1, T, 72, dtype, N=len(cu) - 1), cu=cu, given_states=given_states)


@pytest.mark.parametrize("D", [9, 64])
def test_many_short_sequences(D):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (700,), generator=g)
    cu = [0] + lens.cumsum(0).tolist()
    check(inputs(17, 1, cu[-1], D, BF, N=700), cu=cu)


@pytest.mark.parametrize("dtype,D", [(BF, 64), (F32, 40)])
def test_long(dtype, D):
    check(inputs(19, 1, 5003, D, dtype))


def test_longer_batch():
    check(inputs(23, 6, 700, 24, BF))


def from_lengths(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[211, 190, 0, 205, 201, 187, 1, 210, 199], [1500, 3, 40, 1, 77, 129], [5, 0, 31, 1301]],
                         ids=["even", "long first", "long last"])
def test_packed_over_clusters(dtype, lens):
    """CTAs of a cluster with sequences of their own, and with a long one together."""
    cu = from_lengths(lens)
    check(inputs(31, 1, cu[-1] + 9, 1020, dtype, N=len(lens)), cu=cu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1024] * 16, [8192] + [128] * 20, [128, 0, 6016, 256, 2048, 1920], [2048] * 6],
                         ids=["even", "one long", "mixed", "batch"])
def test_a_sequence_alone_gives_the_same_bits(dtype, lens):
    """However sequences are shared out: pieces are joined from left to right, tile by tile, and
    these begin where tiles do."""
    cu, D = from_lengths(lens), 4096
    i = inputs(32, 1, cu[-1], D, dtype, N=len(lens))
    together = run_both(i, cu=cu)
    if len(set(lens)) == 1:  # the same as a batch of equal lengths
        b = {k: v.view(len(lens), lens[0], D) if v.dim() == 3 else v for k, v in i.items()}
        h, fin, gr = run_both(b)
        assert torch.equal(h.view_as(together[0]), together[0]) and torch.equal(fin, together[1])
        for k, v in gr.items():
            assert torch.equal(v.view_as(together[2][k]), together[2][k]), k
    for n in range(len(lens)):
        s = slice(cu[n], cu[n + 1])
        one = {k: v[:, s].contiguous() if v.dim() == 3 else v[n:n + 1].contiguous() for k, v in i.items()}
        h, fin, gr = run_both(one)
        assert torch.equal(h, together[0][:, s]) and torch.equal(fin, together[1][n:n + 1]), n
        for k, v in gr.items():
            w = together[2][k]
            assert torch.equal(v, w[n:n + 1] if k == "d_initial_state" else w[:, s]), (n, k)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_behind_the_last_sequence_stay(dtype):
    cu, T, D = [0, 70, 150], 333, 72
    i = inputs(29, 1, T, D, dtype, N=2)
    for k in ("x", "la", "gate", "dh"):
        i[k][:, 150:] = float("nan")  # never looked at
    mark = 7.0
    h = torch.full((1, T, D), mark, dtype=dtype, device="cuda")
    fin = kda.scan_fwd(i["x"], i["la"], i["init"], gate=i["gate"], normalize=True, cu_seqlens=as_cu(cu), out=h)[1]
    r = ref_of(i, True, True, True, cu)
    scan_ref.assert_within(h[:, :150], r["h"][:, :150], r["h_e"][:, :150], "h")
    scan_ref.assert_within(fin, r["final"], r["final_e"], "final")
    assert (h[:, 150:] == mark).all()
    check(i, cu=cu)
    check(i, cu=cu, given_states=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,off", [(64, 0), (72, 8), (33, 1)])
@pytest.mark.parametrize("B", [1, 2])
def test_column_slices(dtype, D, off, B):
    T = 140
    i = inputs(31, B, T, D, dtype)
    wide = torch.full((B, T, 4 * (D + off)), float("nan"), dtype=dtype, device="cuda")
    j = dict(i)
    for k, name in enumerate(("x", "la", "gate", "dh")):
        at = k * (D + off) + off
        wide[:, :, at:at + D] = i[name]
        j[name] = wide[:, :, at:at + D]
    a, b = run_both(i), run_both(j)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for k in a[2]:
        assert torch.equal(a[2][k], b[2][k]), k


def test_head_layout():
    i = inputs(37, 2, 100, 96, BF)
    j = {k: (v.view(v.shape[:-1] + (3, 32))) for k, v in i.items()}
    a, b = run_both(i), run_both(j)
    assert b[0].shape == (2, 100, 3, 32) and b[1].shape == (2, 3, 32) and b[2]["d_initial_state"].shape == (2, 3, 32)
    assert torch.equal(a[0].view_as(b[0]), b[0]) and torch.equal(a[2]["dgate"].view_as(b[2]["dgate"]), b[2]["dgate"])


@pytest.mark.parametrize("norm", [False, True])
def test_border_decays(norm):
    """-inf restarts a channel, values above 0 count as 0 and have no gradient, 0 keeps the state."""
    i = inputs(41, 1, 200, 40, F32)
    la = i["la"]
    la[0, 50, :10] = float("-inf")
    la[0, 51, :10] = float("-inf")
    la[0, 60:70, 10:20] = 0.7
    la[0, 100:140, 20:30] = 0.0
    la[0, :, 30:35] = -100.0
    la[0, :, 35:40] = -1e-6
    if norm:  # the limit of the second term at 0 does not exist: it is left out
        check(i, norm=True)
    else:
        check(i, norm=False)
    _, _, gr = run_both(i, norm=norm)
    assert (gr["dlog_alpha"][0, 60:70, 10:20] == 0).all()
    assert (gr["dlog_alpha"][0, 50:52, :10] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
def test_open_and_shut_gates(dtype, norm):
    """sigmoid below 1e-19 (a gate below -44) may count as 0: what that can change is |x| <= 8 summed over 50 tokens."""
    i = inputs(27, 2, 50, 36, dtype)
    ends = torch.tensor([-float("inf"), -200.0, -88.0, -60.0, -44.0, -30.0, 30.0, 60.0, 200.0, float("inf")], device="cuda")
    i["gate"] = ends[torch.arange(i["gate"].numel(), device="cuda") * 7 % 10].view_as(i["gate"]).to(dtype)
    h, fin, gr = run_both(i, True, norm)
    r = ref_of(i, True, norm, True, None, True)
    tiny = 50 * 8 * 1e-19
    scan_ref.assert_within(h, r["h"], r["h_e"] + tiny, "h")
    scan_ref.assert_within(fin, r["final"], r["final_e"] + tiny, "final state")
    for key, ref in (("dx", "dx"), ("dlog_alpha", "dl"), ("dgate", "dgate")):
        scan_ref.assert_within(gr[key], r[ref], r[ref + "_e"] + 100 * tiny, key)


def test_what_a_restart_forgets():
    """After a_t = 0 nothing of a huge state is left, not even a rounding."""
    i = inputs(43, 1, 300, 64, F32)
    i["x"][0, :100] *= 1e30
    i["la"][0, 100] = float("-inf")
    h = kda.scan_fwd(i["x"], i["la"])[0]
    alone = kda.scan_fwd(i["x"][:, 100:].contiguous(), i["la"][:, 100:].contiguous())[0]
    scale = alone.abs().amax()
    assert torch.isfinite(h).all() and ((h[:, 100:] - alone).abs() <= 200 * 8 * scan_ref.EPS * scale).all()


def test_nan_stays_in_its_sequence_and_channel():
    cu = [0, 100, 101, 300, 450]
    i = inputs(47, 1, 450, 40, BF, N=4)
    clean = run_both(i, cu=cu)
    j = {k: v.clone() for k, v in i.items()}
    j["x"][0, 150, 3] = float("nan")
    j["x"][0, 20, 7] = float("inf")
    j["la"][0, 210, 5] = float("nan")
    h, fin, gr = run_both(j, cu=cu)
    same = torch.ones((1, 450, 40), dtype=torch.bool, device="cuda")
    same[0, 150:300, 3] = False
    same[0, 20:100, 7] = False
    same[0, 210:300, 5] = False
    assert torch.equal(h[same], clean[0][same])
    assert torch.isnan(h[0, 150:300, 3]).all() and torch.isnan(h[0, 210:300, 5]).all()
    assert not torch.isfinite(h[0, 20:30, 7]).any()
    ok = torch.ones_like(same)
    ok[0, :100, 7] = ok[0, 101:300, 3] = ok[0, 101:300, 5] = False
    for k in ("dx", "dlog_alpha", "dgate"):
        assert torch.equal(gr[k][ok], clean[2][k][ok]), k


def test_slow_decay_keeps_its_rate():
    """Decays of 1 - 1e-5 to 1 - 2e-5 over 20000 tokens.  Rounding a itself would put a channel's rate off by up to
    2^-25 in 1e-5 the same way at every token: 3e-4 of its state, 1e-4 over the channels.  Two roundings a token of
    random sign, 2^-24 / sqrt(3) each, add up to 2^-24 sqrt(2 T / 3) / sqrt(2) = 5e-6 of a random walk's size;
    allowed is six times that."""
    T, D = 20000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((1, T, D), generator=g, device="cuda")
    l = -1e-5 * (1 + torch.rand(D, generator=g, device="cuda"))
    fin = kda.scan_fwd(x, l.expand(1, T, D).contiguous())[1].double()
    k = torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.float64)[:, None]
    exact = (x[0].double() * torch.exp(k * l.double())).sum(0)
    assert float((fin[0] - exact).norm() / exact.norm()) < 3e-5


def test_guards_and_in_place_state():
    T, D = 130, 65
    i = inputs(53, 2, T, D, BF)
    h, ok_h = guarded_empty((2, T, D), BF)
    cs, ok_c = guarded_empty((-(-2 * T // kda.SCAN_CHUNK), D), F32)
    state, ok_s = guarded_empty((2, D), F32)
    state.copy_(i["init"])
    r = kda.scan_fwd(i["x"], i["la"], state, gate=i["gate"], out=h, final_state=state, chunk_states=cs)
    for f in (ok_h, ok_c, ok_s):
        f()
    a = kda.scan_fwd(i["x"], i["la"], i["init"], gate=i["gate"])
    assert torch.equal(h, a[0]) and torch.equal(state, a[1]) and r[1] is state


@pytest.mark.parametrize("cu,bad", [([0, 100, 200], False), ([0, 100, 150], False), ([0, 100, 201], True),
                                    ([0, 150, 100, 200], True), ([5, 100, 200], True), ([0, -7, 200], True),
                                    ([0, 1 << 30, 200], True)], ids=str)
def test_status_word(cu, bad):
    i = inputs(59, 1, 200, 72, BF, N=len(cu) - 1)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    h, ok = guarded_empty((1, 200, 72), BF)
    kda.scan_fwd(i["x"], i["la"], i["init"], gate=i["gate"], cu_seqlens=as_cu(cu), workspace=ws, out=h)
    ok()
    assert kda.query_status(ws) == (-7 if bad else 0)
    assert kda.query_status(ws) == 0
    n = kda.scan_bwd_workspace_size(1, 200, 72)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    kda.scan_bwd(i["x"], i["la"], i["dh"], i["init"], gate=i["gate"], cu_seqlens=as_cu(cu), workspace=ws)
    assert kda.query_status(ws) == (-7 if bad else 0)


def test_no_tokens():
    i = inputs(61, 2, 0, 40, BF)
    h, fin = kda.scan_fwd(i["x"], i["la"], i["init"])
    assert h.shape == (2, 0, 40) and torch.equal(fin, i["init"])
    assert (kda.scan_fwd(i["x"], i["la"])[1] == 0).all()
    cs = kda.scan_fwd(i["x"], i["la"], chunk_states=True)[2]
    for states in (None, cs):
        gr = kda.scan_bwd(i["x"], i["la"], i["dh"], i["init"], i["dfin"], chunk_states=states)
        assert torch.equal(gr["d_initial_state"], i["dfin"])


def test_same_bits_every_time():
    i = inputs(67, 3, 900, 200, BF)
    a = run_both(i)
    for _ in range(5):
        b = run_both(i)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert all(torch.equal(a[2][k], b[2][k]) for k in a[2])


def test_pieces_of_a_sequence():
    """A sequence in two calls, the state handed on, against the whole."""
    i = inputs(71, 1, 500, 72, F32)
    r = ref_of(i, True, True, True)
    cut = lambda k, a, b: i[k][:, a:b].contiguous()  # noqa: E731
    state = i["init"].clone()
    out = []
    for a, b in ((0, 190), (190, 191), (191, 500)):
        h, state = kda.scan_fwd(cut("x", a, b), cut("la", a, b), state, gate=cut("gate", a, b), normalize=True)
        out.append(h)
    scan_ref.assert_within(torch.cat(out, 1), r["h"], 2 * r["h_e"], "h")


def test_side_stream():
    i = inputs(73, 2, 300, 96, BF)
    a = run_both(i)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        h, fin, cs = kda.scan_fwd(i["x"], i["la"], i["init"], gate=i["gate"], normalize=True, chunk_states=True, stream=s)
        gr = kda.scan_bwd(i["x"], i["la"], i["dh"], i["init"], i["dfin"], gate=i["gate"], normalize=True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], h) and torch.equal(a[1], fin)
    assert all(torch.equal(a[2][k], gr[k]) for k in gr)


def test_two_streams_at_once():
    a, b = inputs(41, 2, 1000, 520, BF), inputs(42, 1, 1500, 1024, F32)
    cu = [0, 300, 300, 700, 1500]
    b["init"], b["dfin"] = b["init"].expand(4, -1).contiguous(), b["dfin"].expand(4, -1).contiguous()
    calls = [lambda: run_both(a), lambda: run_both(b, cu=cu, given_states=False)]
    alone = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(6):
        for f, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    for n, (h, fin, gr) in enumerate(got):
        h0, fin0, gr0 = alone[n % 2]
        assert torch.equal(h, h0) and torch.equal(fin, fin0)
        for k in gr:
            assert torch.equal(gr[k], gr0[k]), k


def test_captured_and_replayed():
    i = inputs(79, 2, 300, 96, BF)
    want = run_both(i)
    st = {k: torch.zeros_like(v) for k, v in i.items()}
    g = torch.cuda.CUDAGraph()
    run_both(st)
    with torch.cuda.graph(g):
        h, fin, gr = run_both(st, given_states=False)
    for _ in range(3):
        for k in st:
            st[k].copy_(i[k])
        g.replay()
        assert torch.equal(h, want[0]) and torch.equal(fin, want[1])
        assert all(torch.equal(gr[k], want[2][k]) for k in gr)
        for k in st:
            st[k].zero_()
        g.replay()


def test_binding_refusals():
    i = inputs(83, 2, 20, 40, BF)
    x, la = i["x"], i["la"]
    with pytest.raises(TypeError):
        kda.scan_fwd(x.half(), la.half())
    with pytest.raises(TypeError):
        kda.scan_fwd(x, la.float())
    with pytest.raises(ValueError):
        kda.scan_fwd(x, la[:, :10])
    with pytest.raises(ValueError):
        kda.scan_fwd(x, la, i["init"][:1])
    with pytest.raises(TypeError):
        kda.scan_fwd(x, la, i["init"].double())
    with pytest.raises(ValueError):
        kda.scan_fwd(x.transpose(0, 1), la.transpose(0, 1))
    with pytest.raises(ValueError):
        kda.scan_fwd(x, la, out=torch.empty((2, 20, 41), dtype=BF, device="cuda"))
    with pytest.raises(kda.KdaError):
        kda.scan_fwd(x, la, cu_seqlens=as_cu([0, 10, 20]))  # B = 2
    with pytest.raises(ValueError):
        kda.scan_bwd(x, la, i["dh"], chunk_states=torch.zeros((2, 40), device="cuda")[:, :40].t())
    with pytest.raises(kda.KdaError):
        kda.scan_bwd(x, la, i["dh"], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kda.scan_fwd(x, la, workspace=torch.empty(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        kda.scan_fwd(x, la, workspace=torch.empty((256, 2), dtype=torch.uint8, device="cuda")[:, 0])


# ------------------------------------------------------------------------------------------- single tokens

def decode_inputs(seed, n, Bd, D, dtype, P):
    i = inputs(seed, n, Bd, D, dtype)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return i, torch.randn((P, D), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,Bd,D", [(1, 1, 1), (1, 5, 8), (3, 4, 33), (1, 7, 1024), (9, 3, 130), (2, 300, 20), (4, 2, 2050)])
@pytest.mark.parametrize("gate,norm", [(True, True), (False, False), (True, False)])
def test_decode_against_the_scan(dtype, n, Bd, D, gate, norm):
    """n tokens of Bd sequences: the reference with sequences along the batch."""
    i, state = decode_inputs(89, n, Bd, D, dtype, Bd)
    j = {k: i[k].transpose(0, 1).contiguous() for k in ("x", "la", "gate")}
    r = scan_ref.scan(cpu(j["x"]), cpu(j["la"]), cpu(j["gate"]) if gate else None, norm, cpu(state))
    h, steps = kda.scan_decode_steps(state, i["x"], i["la"], gate=i["gate"] if gate else None, normalize=norm,
                                     step_states=True)
    scan_ref.assert_within(h.transpose(0, 1).contiguous(), r["h"], r["h_e"], "h")
    scan_ref.assert_within(steps.transpose(0, 1).contiguous(), r["h"], r["h_e"], "step states")
    scan_ref.assert_within(state, r["final"], r["final_e"], "state")
    assert torch.equal(steps[-1], state)


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("D", [40, 33])
def test_decode_slots(n, D):
    """Padding, slots out of range and a slot named twice; pages that no row names stay."""
    P, slots = 9, [3, -1, 0, 9, 3, 8, -5, 1 << 30, 5, 0]
    Bd = len(slots)
    i, pool = decode_inputs(97, n, Bd, D, BF, P)
    first = [b for b, s in enumerate(slots) if 0 <= s < P and slots.index(s) == b]
    padding = [b for b in range(Bd) if b not in first]
    for k in ("x", "la", "gate"):
        i[k][:, padding] = float("nan")
    before = pool.clone()
    rows = [slots[b] for b in first]
    own = before[rows].contiguous()
    sub = {k: i[k][:, first].contiguous() for k in ("x", "la", "gate")}
    want, want_steps = kda.scan_decode_steps(own, sub["x"], sub["la"], gate=sub["gate"], normalize=True, step_states=True)
    h, ok_h = guarded_empty((n, Bd, D), BF)
    steps, ok_s = guarded_empty((n, Bd, D), F32)
    kda.scan_decode_steps(pool, i["x"], i["la"], gate=i["gate"], normalize=True,
                          slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), out=h, step_states=steps)
    ok_h()
    ok_s()
    assert torch.equal(h[:, first], want) and torch.equal(steps[:, first], want_steps)
    assert (h[:, padding] == 0).all() and (steps[:, padding] == 0).all()
    assert torch.equal(pool[rows], own)
    rest = [p for p in range(P) if p not in rows]
    assert torch.equal(pool[rest], before[rest])


def test_decode_step_and_prefill_agree():
    i = inputs(101, 2, 40, 72, F32)
    h, fin = kda.scan_fwd(i["x"], i["la"], i["init"], gate=i["gate"], normalize=True)
    r = ref_of(i, True, True, True)
    state = i["init"].clone()
    for t in range(40):
        c = lambda k: i[k][:, t].contiguous()  # noqa: E731
        o = kda.scan_decode_step(state, c("x"), c("la"), gate=c("gate"), normalize=True)
        scan_ref.assert_within(o, r["h"][:, t], r["h_e"][:, t], f"token {t}")
    scan_ref.assert_within(state, r["final"], r["final_e"], "state")


def test_decode_refusals():
    i, state = decode_inputs(103, 1, 4, 40, BF, 4)
    with pytest.raises(TypeError):
        kda.scan_decode_steps(state, i["x"], i["la"], slots=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        kda.scan_decode_steps(state, i["x"], i["la"], slots=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kda.scan_decode_steps(state[:, :20].contiguous(), i["x"], i["la"])
    with pytest.raises(kda.KdaError):
        kda.scan_decode_steps(state[:3], i["x"], i["la"])
    with pytest.raises(TypeError):
        kda.scan_decode_steps(state.bfloat16(), i["x"], i["la"])
