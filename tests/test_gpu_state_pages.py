"""Pages of recurrent states on a GPU: copies against a list carried out one by one, plans against their definition,
decode through slots against decode on states side by side, and all of it together as a server runs it."""
import random

import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from kda_testutil import guarded_empty

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def one_by_one(dst, ds, src, ss):
    """dst, src: CPU [L, P, ...]; src may be dst."""
    for d, s in zip(ds, ss):
        if not 0 <= d < dst.shape[1] or (src is None and s >= 0) or (src is not None and s >= src.shape[1]):
            continue
        dst[:, d] = src[:, s].clone() if s >= 0 else 0
    return dst


@pytest.mark.parametrize("page", [(1,), (3,), (4,), (33,), (1, 128, 128), (2, 128, 128), (5001,)])
@pytest.mark.parametrize("layers", [0, 1, 3])
@pytest.mark.parametrize("how", ["apart", "tied", "two pools"])
def test_copy(page, layers, how):
    rng = random.Random(f"{page}{layers}{how}")
    P, Q = 17, 17 if how != "two pools" else 11
    shape = (layers, P) + page if layers else (P,) + page
    pool, ok = guarded_empty(shape, F32)
    pool.copy_(torch.randn(shape, device="cuda"))
    src = pool
    if how == "two pools":
        src = torch.randn(((layers, Q) if layers else (Q,)) + page, device="cuda")
    if how == "apart":   # destinations that nothing reads; some twice
        ds = [rng.randrange(9, 17) for _ in range(12)]
        ss = [rng.randrange(-2, 9) for _ in range(12)]
    else:                # chains, swaps, pages to themselves, slots out of range
        ds = [rng.randrange(-2, P + 2) for _ in range(25)]
        ss = [rng.randrange(-2, Q + 2) for _ in range(25)]
    up = lambda t: (t if layers else t[None]).cpu()  # noqa: E731
    want = up(pool).clone()
    want = one_by_one(want, ds, want if src is pool else up(src), ss)
    r = kda.state_copy(pool, i32(ds), src, i32(ss), layered=bool(layers))
    assert r is pool
    ok()
    assert torch.equal(up(pool), want)


@pytest.mark.parametrize("ds,ss", [([1, 2, 3, 4], [0, 1, 2, 3]), ([1, 0], [0, 1]), ([2, 0, 1], [0, 1, 2]), ([3, 3, 3], [0, 1, 2]),
                                   ([3, 4, 3], [0, 3, 1]), ([2, 2], [2, 0]), ([0], [0]), ([1, 1, 2], [0, -1, 1]),
                                   ([5, 0, 5], [1, 5, 2]), ([-1, -1], [-1, 3]), ([4, 2, 4, 0], [0, 4, 1, 2])], ids=str)
def test_copy_in_list_order(ds, ss):
    pool = torch.randn((6, 8192), device="cuda")
    want = one_by_one(pool[None].cpu().clone(), ds, None, ss) if all(s < 0 for s in ss) else None
    if want is None:
        want = pool[None].cpu().clone()
        want = one_by_one(want, ds, want, ss)
    kda.state_copy(pool, i32(ds), pool, i32(ss))
    assert torch.equal(pool.cpu(), want[0])


@pytest.mark.parametrize("seed", range(6))
def test_copy_long_lists(seed):
    rng = random.Random(seed)
    P, n = rng.choice([40, 3000]), 700
    pool = torch.randn((P, 40), device="cuda")
    ds, ss = ([rng.randrange(-1, P) for _ in range(n)] for _ in range(2))
    want = pool[None].cpu().clone()
    want = one_by_one(want, ds, want, ss)
    kda.state_copy(pool, i32(ds), pool, i32(ss))
    assert torch.equal(pool.cpu(), want[0])


def test_copy_of_layer_slices_and_other_types():
    """Some pages of a wider pool (layers at a distance), bf16 pages, and a list that clears only."""
    big = torch.randn((3, 20, 4, 33), device="cuda").to(BF)
    pool, src = big[:, :8], big[:, 10:]
    before = big.clone()
    with pytest.raises(kda.KdaError):  # the two share the range of one another's layers
        kda.state_copy(pool, i32([0, 1, 2]), src, i32([1, -1, 7]), layered=True)
    src = src.contiguous()
    kda.state_copy(pool, i32([0, 1, 2]), src, i32([1, -1, 7]), layered=True)
    before[:, 0], before[:, 1], before[:, 2] = before[:, 11], 0, before[:, 17]
    assert torch.equal(big, before)
    kda.state_copy(pool, i32([5, 99]), None, i32([-1, -1]), layered=True)
    before[:, 5] = 0
    assert torch.equal(big, before)
    with pytest.raises(ValueError):
        kda.state_copy(big[:, :, :2], i32([0]), big[:, :, :2], i32([1]), layered=True)
    with pytest.raises(ValueError):
        kda.state_copy(pool, i32([0]), src.float(), i32([1]), layered=True)
    with pytest.raises(TypeError):
        kda.state_copy(pool, i32([0]).long(), src, i32([1]).long(), layered=True)
    with pytest.raises(ValueError):
        kda.state_copy(pool, i32([0]), src, i32([1, 2]), layered=True)


def test_copy_past_32_bits():
    """Pages and layers whose distance passes 2^32 bytes."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 20 GB")
    pool = torch.zeros((2, 600, 2 << 20), dtype=F32, device="cuda")  # 8 MB pages, 5 GB layers
    pool[0, 1] = torch.arange(2 << 20, device="cuda")
    pool[1, 1] = 7 + torch.arange(2 << 20, device="cuda")
    kda.state_copy(pool, i32([599, 590]), pool, i32([1, 1]), layered=True)
    for layer in (0, 1):
        for p in (599, 590):
            assert torch.equal(pool[layer, p], pool[layer, 1])
    assert int(pool.count_nonzero(dim=2).ne(0).sum()) == 6


@pytest.mark.parametrize("P", [1, 2, 31, 32, 33, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.9, 1.0])
@pytest.mark.parametrize("kind", [torch.uint8, torch.bool])
def test_compact_plan(P, share, kind):
    g = torch.Generator().manual_seed(P)
    live = (torch.rand(P, generator=g) < share)
    lv = live.tolist()
    m = sum(lv)
    holes, tails = [p for p in range(m) if not lv[p]], [p for p in range(m, P) if lv[p]]
    new = [p if lv[p] and p < m else -1 for p in range(P)]
    for d, s in zip(holes, tails):
        new[s] = d
    d_live = live.to(kind).cuda()
    r = kda.state_compact(d_live)
    pad = [-1] * (P - len(holes))
    assert r["dst_slots"].tolist() == holes + pad and r["src_slots"].tolist() == tails + pad
    assert r["new_slots"].tolist() == new and r["n_live"].tolist() == [m]
    assert d_live.to(torch.uint8).tolist() == [1] * m + [0] * (P - m)


def test_alloc_and_free():
    P = 2100
    g = torch.Generator().manual_seed(2)
    live = (torch.rand(P, generator=g) < 0.6)
    free = [p for p in range(P) if not live[p]]
    d = live.to(torch.uint8).cuda()
    a = kda.state_alloc(d, 10)
    assert a.tolist() == free[:10]
    b = kda.state_alloc(d, len(free))
    assert b.tolist() == free[10:] + [-1] * 10
    assert int(d.sum()) == P
    kda.state_free(d, i32([5, 5, -1, P, 1 << 30, 2000]))
    assert kda.state_alloc(d, 3).tolist() == [5, 2000, -1]
    assert kda.state_alloc(d, 0).tolist() == []
    kda.state_free(d, i32([]))


# --------------------------------------------------------------------------------- decode through slots

def kda_tokens(seed, n, Bd, H, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    return dict(q=unit(r(n, Bd, H, 128)).to(dtype), k=unit(r(n, Bd, H, 128)).to(dtype), v=r(n, Bd, H, 128).to(dtype),
                log_alpha=(-torch.nn.functional.softplus(r(n, Bd, H, 128))).to(dtype),
                beta=torch.sigmoid(r(n, Bd, H)).to(dtype)), r(n, Bd, H, 128).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 3, 9])
@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("gated", [False, True])
def test_paged_decode(dtype, n, H, gated):
    P, slots = 7, [4, -1, 0, 7, 4, 6, -9]
    Bd = len(slots)
    first, padding = [0, 2, 5], [1, 3, 4, 6]
    tok, gate = kda_tokens(n * 10 + H, n, Bd, H, dtype)
    pool, ok_p = guarded_empty((P, H, 128, 128), F32)
    pool.copy_(0.1 * torch.randn((P, H, 128, 128), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    before = pool.clone()
    for t in list(tok.values()) + [gate]:
        t[:, padding] = float("nan")
    sub = {k: t[:, first].contiguous() for k, t in tok.items()}
    w = 1 + 0.1 * torch.randn(128, device="cuda")
    rows = [slots[b] for b in first]
    own = before[rows].contiguous()
    kw = dict(norm_weight=w if gated else None, out_dtype=F32, step_states=True)
    want, want_steps = kda.decode_steps(own, **sub, gate=gate[:, first].contiguous() if gated else None, **kw)
    o, ok_o = guarded_empty((n, Bd, H, 128), F32)
    steps, ok_s = guarded_empty((n, Bd, H, 128, 128), F32)
    kw["step_states"] = steps
    kda.decode_steps(pool, **tok, gate=gate if gated else None, slots=i32(slots), out=o, **kw)
    for f in (ok_p, ok_o, ok_s):
        f()
    if gated:  # whole heads in one CTA against halves and a second kernel: other orders of the same sums
        tol = lambda t: 64 * scan_ref.EPS * t.abs().amax()  # noqa: E731  (128-term dot products, 10 roundings deep)
        assert ((o[:, first] - want).abs() <= n * tol(want)).all()
        assert ((steps[:, first] - want_steps).abs() <= n * tol(want_steps)).all()
        assert ((pool[rows] - own).abs() <= n * tol(own)).all()
    else:
        assert torch.equal(o[:, first], want) and torch.equal(steps[:, first], want_steps) and torch.equal(pool[rows], own)
    assert (o[:, padding] == 0).all() and (steps[:, padding] == 0).all()
    rest = [p for p in range(P) if p not in rows]
    assert torch.equal(pool[rest], before[rest])


def test_paged_decode_step_is_decode_step():
    tok, gate = kda_tokens(3, 1, 5, 2, BF)
    one = {k: t[0] for k, t in tok.items()}
    pool = 0.1 * torch.randn((9, 2, 128, 128), device="cuda")
    slots = [8, 0, 3, 2, 7]
    own = pool[slots].contiguous()
    want = kda.decode_step(own, **one, gate=gate[0])
    got = kda.decode_step(pool, **one, gate=gate[0], slots=i32(slots))
    assert torch.equal(got, want) and torch.equal(pool[slots], own)
    with pytest.raises(ValueError):
        kda.decode_step(pool, **one, slots=i32(slots[:3]))
    with pytest.raises(ValueError):
        kda.decode_step(pool[:, :1].contiguous(), **one, slots=i32(slots))
    with pytest.raises(TypeError):
        kda.decode_step(pool, **one, slots=i32(slots).long())


def test_nothing_to_decode():
    pool = torch.ones((4, 2, 128, 128), device="cuda")
    tok, gate = kda_tokens(5, 3, 2, 2, BF)
    for cut in (lambda t: t[:, :0].contiguous(), lambda t: t[:0].contiguous()):
        none = {k: cut(t) for k, t in tok.items()}
        n, Bd = none["q"].shape[:2]
        o, steps = kda.decode_steps(pool, **none, gate=cut(gate), slots=i32([0, 1][:Bd]), step_states=True)
        assert o.shape == (n, Bd, 2, 128) and steps.shape == (n, Bd, 2, 128, 128)
        x = torch.zeros((n, Bd, 40), device="cuda")
        assert kda.scan_decode_steps(torch.zeros((4, 40), device="cuda"), x, x, slots=i32([0, 1][:Bd])).shape == x.shape
    assert (pool == 1).all()


def test_two_streams_at_once():
    """Two batches of one pool, pages of their own, and page moves of another pool, side by side."""
    pool = 0.1 * torch.randn((40, 4, 128, 128), device="cuda")
    want, other = pool.clone(), torch.randn((20, 1000), device="cuda")
    tok, gate = kda_tokens(6, 2, 16, 4, BF)
    slots = [i32(range(0, 32, 2)), i32(range(1, 33, 2))]
    moves = i32(range(10, 20)), i32(range(10))
    serial = [kda.decode_steps(want, **tok, gate=gate, slots=s) for s in slots for _ in range(3)]
    kda.state_copy(want_other := other.clone(), moves[0], other, moves[1])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(3):
        for n, s in enumerate(streams):
            got[n].append(kda.decode_steps(pool, **tok, gate=gate, slots=slots[n], stream=s))
            kda.state_copy(other, moves[0], other, moves[1], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(pool, want) and torch.equal(other, want_other)
    assert all(torch.equal(a, b) for a, b in zip(got[0] + got[1], serial))


def test_pool_larger_than_32_bits():
    """Pages behind 2^32 bytes of the pool."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 5 GB")
    P, H = 70000, 1
    pool = torch.zeros((P, H, 128, 128), device="cuda")
    tok, _ = kda_tokens(4, 1, 2, H, BF)
    own = torch.zeros((2, H, 128, 128), device="cuda")
    want = kda.decode_steps(own, **tok)
    got = kda.decode_steps(pool, **tok, slots=i32([P - 1, 3]))
    assert torch.equal(got, want) and torch.equal(pool[[P - 1, 3]], own)


def test_a_server_run():
    """Prefill two prompts, keep their states as pages, fork one prompt into three sequences, decode all in one padded
    captured batch, verify draft tokens and roll one sequence back, end one, compact, decode on: every sequence's
    outputs are those of the same sequence alone, its states side by side."""
    H, D, T, steps = 2, 256, 90, 4
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(r(2, T, H, 128)).to(BF), unit(r(2, T, H, 128)).to(BF), r(2, T, H, 128).to(BF)
    la, be = (-torch.nn.functional.softplus(r(2, T, H, 128))).to(BF), torch.sigmoid(r(2, T, H)).to(BF)
    x, sla, sg = r(2, T, D).to(BF), (-torch.rand((2, T, D), generator=g, device="cuda")).to(BF), r(2, T, D).to(BF)
    _, kda_state = kda.chunk_fwd(q, k, v, la, be)
    _, scan_state = kda.scan_fwd(x, sla, gate=sg, normalize=True)

    P = 6
    kpool, spool = torch.zeros((P, H, 128, 128), device="cuda"), torch.zeros((P, D), device="cuda")
    live = torch.zeros(P, dtype=torch.uint8, device="cuda")
    home = kda.state_alloc(live, 2)
    both = lambda ds, ks, ss, sl: (kda.state_copy(kpool, ds, ks, sl), kda.state_copy(spool, ds, ss, sl))  # noqa: E731
    both(home, kda_state, scan_state, i32([0, 1]))
    forks = kda.state_alloc(live, 2)
    both(forks, kpool, spool, home[:1].repeat(2))
    slots = torch.cat([home, forks, i32([-1])])
    assert slots.tolist() == [0, 1, 2, 3, -1]
    alone_k = kda_state[[0, 1, 0, 0]].contiguous()
    alone_s = scan_state[[0, 1, 0, 0]].contiguous()

    # a captured batch of 5 rows, its last one padding; other tokens for every replay
    tok, gate = kda_tokens(5, 1, 5, H, BF)
    sx, sl_, sgt = r(1, 5, D).to(BF), (-torch.rand((1, 5, D), generator=g, device="cuda")).to(BF), r(1, 5, D).to(BF)
    save = kpool.clone(), spool.clone()
    step = lambda: (kda.decode_steps(kpool, **tok, gate=gate, slots=slots),  # noqa: E731
                    kda.scan_decode_steps(spool, sx, sl_, gate=sgt, normalize=True, slots=slots))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, h = step()
    kpool.copy_(save[0])
    spool.copy_(save[1])
    for i in range(steps):
        new, ng = kda_tokens(100 + i, 1, 5, H, BF)
        for name in tok:
            tok[name].copy_(new[name])
        gate.copy_(ng)
        sx.copy_(r(1, 5, D))
        graph.replay()
        want = kda.decode_steps(alone_k, **{n: t[:, :4].contiguous() for n, t in tok.items()}, gate=gate[:, :4].contiguous())
        want_h = kda.scan_decode_steps(alone_s, sx[:, :4].contiguous(), sl_[:, :4].contiguous(),
                                       gate=sgt[:, :4].contiguous(), normalize=True)
        assert torch.equal(o[:, :4], want) and torch.equal(h[:, :4], want_h)
        assert (o[:, 4] == 0).all() and (h[:, 4] == 0).all()

    # three draft tokens, of which sequence 0 keeps one, 1 all, 2 two, 3 one
    tok, _ = kda_tokens(6, 3, 4, H, BF)
    sx, sl_ = r(3, 4, D).to(BF), (-torch.rand((3, 4, D), generator=g, device="cuda")).to(BF)
    keep = torch.tensor([1, 3, 2, 1], device="cuda", dtype=torch.int32)
    _, ks = kda.decode_steps(kpool, **tok, slots=slots[:4], step_states=True)
    _, ss = kda.scan_decode_steps(spool, sx, sl_, slots=slots[:4], step_states=True)
    at = (keep - 1) * 4 + i32([0, 1, 2, 3])
    kda.state_copy(kpool, slots[:4], ks.view((12,) + ks.shape[2:]), at)
    kda.state_copy(spool, slots[:4], ss.view(12, D), at)
    for b, n in enumerate(keep.tolist()):
        a = alone_k[b:b + 1]
        kda.decode_steps(a, **{m: t[:n, b:b + 1].clone() for m, t in tok.items()})
        kda.scan_decode_steps(alone_s[b:b + 1], sx[:n, b:b + 1].clone(), sl_[:n, b:b + 1].clone())
    assert torch.equal(kpool[:4], alone_k) and torch.equal(spool[:4], alone_s)

    # sequence 1 ends; its slot is filled from the end of the pool
    kda.state_free(live, slots[1:2])
    plan = kda.state_compact(live)
    both(plan["dst_slots"], kpool, spool, plan["src_slots"])
    assert plan["n_live"].item() == 3 and plan["new_slots"].tolist() == [0, -1, 2, 1, -1, -1]
    order = [0, 3, 2]
    tok, _ = kda_tokens(7, 1, 3, H, BF)
    rest = alone_k[order].contiguous()
    assert torch.equal(kpool[:3], rest) and torch.equal(spool[:3], alone_s[order])
    assert torch.equal(kda.decode_steps(kpool[:3], **tok), kda.decode_steps(rest, **tok))


def test_training_through_the_gate():
    """chunk_fwd, gate_norm and back: the loss's change along a direction of q, k, v, beta, log_alpha and the gate against
    differences of an fp64 token-by-token computation."""
    T, H = 70, 2
    tok, gate = kda_tokens(8, 1, T, H, F32)
    w = 1 + 0.1 * torch.randn(128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    dy = kda_tokens(9, 1, T, H, F32)[1]
    names = ("q", "k", "v", "log_alpha", "beta")
    o, _ = kda.chunk_fwd(*[tok[n] for n in names])
    gn = kda.gate_norm_bwd(o, gate, dy, w)
    gr = kda.chunk_bwd(*[tok[n] for n in names], gn["d_o"])

    leaf = {n: tok[n][0].double().cpu().requires_grad_() for n in names}
    lg, lw = gate[0].double().cpu().requires_grad_(), w.double().cpu().requires_grad_()
    S = torch.zeros((H, 128, 128), dtype=torch.float64)
    loss = 0.0
    for t in range(T):
        q, k, v, l, b = (leaf[n][t] for n in names)
        S = S * l.clamp(min=-5).exp()[..., None]
        S = S + (b[:, None, None] * k[..., None] * (v - torch.einsum("hkv,hk->hv", S, k))[:, None])
        o_t = torch.einsum("hkv,hk->hv", S, q)
        y = o_t * torch.rsqrt(o_t.square().mean(-1, keepdim=True) + 1e-6) * lw * torch.sigmoid(lg[t])
        loss = loss + (y * dy[0, t].double().cpu()).sum()
    loss.backward()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    # the chunk kernels round their products' operands to bf16 (2^-9 each, up to four in a row: their own tolerance
    # of 1e-2 over the recurrence); the norm's gradient takes o's relative error on twice, times its own conditioning
    # |d_o| r / |dn| of at most 2
    for n, key in zip(names, ("dq", "dk", "dv", "dlog_alpha", "dbeta")):
        assert rel(gr[key][0], leaf[n].grad) < 3e-2, key
    assert rel(gn["d_gate"][0], lg.grad) < 2e-2 and rel(gn["d_norm_weight"], lw.grad) < 2e-2
