"""Long lists of page moves, against the list carried out one by one on the host."""
import random

import pytest
import torch

import linear_attention_recurrence_06_b200 as kda

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def tags(P, Q=None):
    """Pools whose page p holds the number p (Q: a second pool, numbers from P + 1 on); 0 is a cleared page."""
    a = torch.arange(1, P + 1, dtype=torch.int32)
    return a, (a if Q is None else torch.arange(P + 1, P + Q + 1, dtype=torch.int32))


def one_by_one(dst, ds, src, ss):
    for d, s in zip(ds, ss):
        if 0 <= d < len(dst) and s < len(src):
            dst[d] = src[s] if s >= 0 else 0
    return dst


def check(P, ds, ss, Q=None, page=1):
    """Every page is `page` copies of its number."""
    a, b = tags(P, Q)
    want = a.tolist()
    want = one_by_one(want, ds, want if Q is None else b.tolist(), ss)
    dst = a[:, None].expand(P, page).contiguous().cuda()
    src = dst if Q is None else b[:, None].expand(Q, page).contiguous().cuda()
    kda.state_copy(dst, i32(ds), src, i32(ss))
    got = dst.cpu()
    assert (got == got[:, :1]).all() and got[:, 0].tolist() == want


@pytest.mark.parametrize("n", [2, 255, 256, 257, 4095, 4096, 4097, 12000])
def test_one_tied_pair_at_the_end(n):
    P = 2 * n + 2
    rng = random.Random(n)
    ds, ss = rng.sample(range(n + 1, 2 * n + 1), n), [rng.randrange(n) for _ in range(n)]
    ds[-2], ss[-2] = n, ss[-1]
    ss[-1] = n  # reads what the entry before it wrote
    check(P, ds, ss)


@pytest.mark.parametrize("page", [1, 5001])
def test_half_of_a_thousand_tied(page):
    rng = random.Random(page)
    ds, ss = list(range(1000, 1500)), [rng.randrange(0, 500) for _ in range(500)]
    for _ in range(500):  # a chain with repetitions among 40 pages
        ds.append(1600 + rng.randrange(40))
        ss.append(1600 + rng.randrange(-2, 40) if rng.random() < 0.9 else -1)
    check(1700, ds, ss, page=page)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("P,n", [(300, 5000), (70000, 3000), (200_000, 20000), (40000, 65535)])
def test_lists_of_any_order(P, n, seed):
    """Up to all entries tied; pools of more pages than a set has bits."""
    rng = random.Random(f"{P}{n}{seed}")
    ds, ss = ([rng.randrange(-1, P) for _ in range(n)] for _ in range(2))
    if seed == 1:  # pages that differ by a power of two only
        ds = [d % 100 + (1 << 17) * rng.randrange(2) for d in ds]
        ss = [s % 100 + (1 << 17) * rng.randrange(2) for s in ss]
    check(P, ds, ss, Q=P // 2 if seed == 2 else None)


def test_writers_of_one_page():
    """The last one stands, beside entries that are not tied, and from another pool as well."""
    ds = [7] * 300 + list(range(8, 20)) + [7]
    ss = list(range(300)) + [300 + k for k in range(12)] + [5]
    check(1000, [d + 500 for d in ds], ss)
    check(1000, ds, ss, Q=400)


def test_lists_longer_than_a_launch_takes():
    """The order holds over the pieces in which the binding passes a longer list."""
    P, n = 30000, 150_000
    rng = random.Random(3)
    check(P, [rng.randrange(P) for _ in range(n)], [rng.randrange(-1, P) for _ in range(n)])


def test_compaction_of_a_large_pool():
    P = 100_000
    g = torch.Generator().manual_seed(8)
    keep = torch.rand(P, generator=g) < 0.4
    pool = torch.arange(P, dtype=torch.int32, device="cuda")[:, None].contiguous()
    live = keep.to(torch.uint8).cuda()
    plan = kda.state_compact(live)
    kda.state_copy(pool, plan["dst_slots"], pool, plan["src_slots"])
    m = int(keep.sum())
    assert plan["n_live"].item() == m and live[:m].all() and not live[m:].any()
    old = keep.nonzero()[:, 0].cuda()
    assert torch.equal(pool[plan["new_slots"][old].long(), 0].long(), old)


@pytest.mark.parametrize("gated", [False, True])
def test_decode_in_a_pool_without_pages(gated):
    """Every row is padding: zeros."""
    n, Bd, H = 2, 3, 2
    t = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    tok = t(n, Bd, H, 128)
    kw = dict(slots=i32([0, -1, 5]), step_states=True)
    o, steps = kda.decode_steps(torch.empty((0, H, 128, 128), device="cuda"), tok, tok, tok, tok, t(n, Bd, H),
                                gate=tok if gated else None, **kw)
    assert (o == 0).all() and (steps == 0).all()
    x = t(n, Bd, 40)
    h, steps = kda.scan_decode_steps(torch.empty((0, 40), device="cuda"), x, x, gate=x if gated else None, **kw)
    assert (h == 0).all() and (steps == 0).all()


def test_free_of_the_longest_list():
    """2^31 - 100 slots (8.6 GB): the last CTA's numbers pass 31 bits."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 10 GB")
    n = (1 << 31) - 100
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[-1], slots[0] = 3, 5
    live = torch.ones(8, dtype=torch.uint8, device="cuda")
    kda.state_free(live, slots)
    assert live.tolist() == [1, 1, 1, 0, 1, 0, 1, 1]
