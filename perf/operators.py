"""The recurrent-state operators as they are used: the element-wise gated scan (forward, gradients, single tokens),
the gradient of the per-head RMSNorm and gate, the pages that hold recurrent states, and decode through a pool of them.

own = False computes each from elementary torch operations in 32 bits, own = True calls the library.
"""
import math

import torch

own = False

D_HEAD = 128
F32, F64 = torch.float32, torch.float64


def _dt(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the first tokens of one request through a narrow recurrent layer: latency only
        {"name": "scan first tokens", "kind": "scan", "lens": "fixed", "B": 1, "T": 64, "D": 256, "dtype": "bf16",
         "gate": False, "normalize": False, "init": True},
        # a packed serving prefill: 16 prompts of 512 to 16384 tokens, 32 heads of 128 channels
        {"name": "scan packed prefill", "kind": "scan", "lens": "packed", "N": 16, "lo": 512, "hi": 16384, "D": 4096,
         "dtype": "bf16", "gate": True, "normalize": True, "init": True},
        # one training step of the layer: forward, then the gradients, in bf16
        {"name": "scan training step", "kind": "train", "lens": "fixed", "B": 4, "T": 2048, "D": 4096, "dtype": "bf16",
         "gate": True, "normalize": True, "init": False},
        # gradients of packed documents of odd lengths (one token, none at all) in fp32, channels no multiple of a tile
        {"name": "scan ragged gradients", "kind": "scan_bwd", "lens": "packed", "N": 23, "lo": 0, "hi": 401, "D": 1000,
         "dtype": "fp32", "gate": True, "normalize": True, "init": True},
        # one token for each of 256 sequences whose states lie in a pool, a few rows of the batch being padding
        {"name": "scan decode in a pool", "kind": "scan_decode", "n": 1, "Bd": 256, "pad": 5, "P": 320, "D": 4096,
         "dtype": "bf16", "gate": True, "normalize": True},
        # checking five draft tokens of three sequences, fp32
        {"name": "scan draft tokens", "kind": "scan_decode", "n": 5, "Bd": 3, "pad": 0, "P": 8, "D": 1000,
         "dtype": "fp32", "gate": False, "normalize": False},
        # gradient of the output norm and gate over a prefill of 8192 tokens and 32 heads
        {"name": "gate norm gradient", "kind": "gate_norm_bwd", "rows": 8192 * 32, "dtype": "bf16", "grad": "bf16",
         "weight": True},
        # the same for 301 tokens of 2 heads in fp32, no weight
        {"name": "gate norm gradient small", "kind": "gate_norm_bwd", "rows": 602, "dtype": "fp32", "grad": "fp32",
         "weight": False},
        # 64 sequences forked from 8 cached prefixes, and 8 slots cleared for new ones: pages of 32 heads
        {"name": "fork pages", "kind": "pages", "L": 1, "P": 160, "H": 32, "moves": 64, "sources": 8, "clear": 8},
        # the pool of four layers after a third of the sequences ended: live pages moved to its front
        {"name": "compact pages", "kind": "compact", "L": 4, "P": 96, "H": 8, "live": 0.66},
        # one decode step of 256 sequences of 32 heads in a pool of 320 pages, 6 rows of padding
        {"name": "paged decode step", "kind": "decode", "n": 1, "Bd": 256, "pad": 6, "P": 320, "H": 32, "dtype": "bf16",
         "gate": False},
        # four draft tokens of nine sequences of 3 heads with the output gate
        {"name": "paged draft tokens", "kind": "decode", "n": 4, "Bd": 9, "pad": 1, "P": 12, "H": 3, "dtype": "bf16",
         "gate": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "train", "scan_bwd", "scan_decode", "gate_norm_bwd", "pages", "compact", "decode"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("scan", "train", "scan_bwd"):
        D = _log_int(rng, 64, 4096)
        D = D if rng.random() < 0.4 else max(8, D // 8 * 8)
        c = {"kind": kind, "D": D, "dtype": dtype, "gate": rng.random() < 0.6, "normalize": rng.random() < 0.6,
             "init": rng.random() < 0.5}
        # as many elements as the largest listed case of this direction at most
        most = (200_000_000 if kind == "scan" else 33_000_000) // D
        if rng.random() < 0.5:
            T = _log_int(rng, 1, min(32768, most))
            return {**c, "lens": "fixed", "B": _log_int(rng, 1, max(1, min(16, most // T))), "T": T}
        N = _log_int(rng, 1, 64)
        hi = _log_int(rng, 2, max(3, min(16384, most // N)))
        return {**c, "lens": "packed", "N": N, "lo": rng.choice([0, 1, hi // 4]), "hi": hi}
    if kind == "scan_decode":
        Bd, D = _log_int(rng, 1, 512), _log_int(rng, 64, 8192)
        pad = rng.randrange(0, Bd // 4 + 1)
        return {"kind": kind, "n": rng.choice([1, 1, 2, 3, 5, 8]), "Bd": Bd, "pad": pad, "P": Bd + rng.randrange(1, 64),
                "D": D if rng.random() < 0.4 else D // 8 * 8, "dtype": dtype, "gate": rng.random() < 0.6,
                "normalize": rng.random() < 0.6}
    if kind == "gate_norm_bwd":
        return {"kind": kind, "rows": _log_int(rng, 1, 262144), "dtype": dtype, "grad": rng.choice(["bf16", "fp32"]),
                "weight": rng.random() < 0.7}
    if kind == "pages":
        H, moves = _log_int(rng, 1, 32), _log_int(rng, 1, 64)
        sources = rng.randrange(1, moves + 1)
        clear = rng.randrange(0, 9)
        return {"kind": kind, "L": rng.choice([1, 1, 2, 3]), "P": moves + sources + clear + rng.randrange(0, 32), "H": H,
                "moves": moves, "sources": sources, "clear": clear}
    if kind == "compact":
        return {"kind": kind, "L": _log_int(rng, 1, 6), "P": _log_int(rng, 2, 128), "H": _log_int(rng, 1, 16),
                "live": round(rng.uniform(0.05, 0.98), 3)}
    Bd = _log_int(rng, 1, 256)
    H = _log_int(rng, 1, max(2, min(32, 8192 // Bd)))
    return {"kind": kind, "n": rng.choice([1, 1, 1, 2, 3, 4, 8]), "Bd": Bd, "pad": rng.randrange(0, Bd // 4 + 1),
            "P": Bd + rng.randrange(1, 64), "H": H, "dtype": dtype, "gate": rng.random() < 0.5}


# --------------------------------------------------------------------------------------------- inputs

def _randn(gen, shape, dtype=F32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32).to(dtype)


def _lengths(case, seed):
    """The case's lengths (their sum is the case's own), in an order of the seed's."""
    g = torch.Generator().manual_seed(case["N"] * 7919 + case["hi"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["N"],), generator=g)
    if int(lens.sum()) == 0:
        lens[0] = 1
    return lens[torch.randperm(case["N"], generator=torch.Generator().manual_seed(seed))].tolist()


def _scan_shape(case, seed):
    """(leading shape of the token tensors, number of sequences, lengths or None)"""
    if case["lens"] == "fixed":
        return (case["B"], case["T"]), case["B"], None
    lens = _lengths(case, seed)
    return (1, sum(lens)), len(lens), lens


def _decays(gen, lead, D, dtype):
    """Log-decays: each channel has its own rate, from a memory of a token to one of thousands, times a gate."""
    rate = torch.exp(torch.rand((D,), generator=gen, device="cuda") * math.log(3e3) - math.log(3e3 / 2.0))
    r = torch.randn(tuple(lead) + (D,), generator=gen, device="cuda")
    return r.sigmoid_().mul_(rate).neg_().to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k = case["kind"]
    s = {"case": dict(case)}
    if k in ("scan", "train", "scan_bwd"):
        dt, D = _dt(case["dtype"]), case["D"]
        lead, N, lens = _scan_shape(case, seed)
        s["x"] = _randn(gen, lead + (D,), dt)
        s["log_alpha"] = _decays(gen, lead, D, dt)
        s["gate"] = _randn(gen, lead + (D,), dt) if case["gate"] else None
        s["init"] = _randn(gen, (N, D)) if case["init"] else None
        s["cu"] = None
        if lens is not None:
            at = [0]
            at += torch.tensor(lens).cumsum(0).tolist()
            s["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
            s["max_seqlen"] = max(lens)
        if k != "scan":
            s["d_h"] = _randn(gen, lead + (D,), dt)
            s["d_final"] = _randn(gen, (N, D)) if case["init"] else None
    elif k == "scan_decode":
        dt, D, n, Bd = _dt(case["dtype"]), case["D"], case["n"], case["Bd"]
        s["pool"] = _randn(gen, (case["P"], D))
        s["slots"] = _slots(gen, case)
        s["x"], s["log_alpha"] = _randn(gen, (n, Bd, D), dt), _decays(gen, (n, Bd), D, dt)
        s["gate"] = _randn(gen, (n, Bd, D), dt) if case["gate"] else None
    elif k == "gate_norm_bwd":
        dt = _dt(case["dtype"])
        for name in ("o", "g", "d_y"):
            s[name] = _randn(gen, (case["rows"], D_HEAD), dt)
        s["w"] = 1.0 + 0.2 * _randn(gen, (D_HEAD,)) if case["weight"] else None
    elif k == "pages":
        s["pool"] = _randn(gen, (case["L"], case["P"], case["H"], D_HEAD, D_HEAD))
        order = torch.randperm(case["P"], generator=gen, device="cuda").to(torch.int32)
        m, q = case["moves"], case["sources"]
        pick = torch.randint(0, q, (m,), generator=gen, device="cuda")
        s["dst"] = order[q:q + m + case["clear"]].contiguous()
        s["src"] = torch.cat([order[:q][pick], torch.full((case["clear"],), -1, dtype=torch.int32, device="cuda")])
    elif k == "compact":
        s["pool"] = _randn(gen, (case["L"], case["P"], case["H"], D_HEAD, D_HEAD))
        s["live"] = (torch.rand((case["P"],), generator=gen, device="cuda") < case["live"]).to(torch.uint8)
    else:
        dt, n, Bd, H = _dt(case["dtype"]), case["n"], case["Bd"], case["H"]
        s["pool"] = 0.02 * _randn(gen, (case["P"], H, D_HEAD, D_HEAD))
        s["slots"] = _slots(gen, case)
        unit = lambda v: v / v.norm(dim=-1, keepdim=True)  # noqa: E731
        s["q"], s["k"] = (unit(_randn(gen, (n, Bd, H, D_HEAD))).to(dt) for _ in range(2))
        s["v"] = _randn(gen, (n, Bd, H, D_HEAD), dt)
        s["log_alpha"] = (-torch.nn.functional.softplus(_randn(gen, (n, Bd, H, D_HEAD)))).clamp_(min=-5).to(dt)
        s["beta"] = _randn(gen, (n, Bd, H)).sigmoid().to(dt)
        s["gate"] = _randn(gen, (n, Bd, H, D_HEAD), dt) if case["gate"] else None
    return s


def _slots(gen, case):
    """The pool page of each row of the batch; its last rows are padding and have none."""
    slots = torch.randperm(case["P"], generator=gen, device="cuda").to(torch.int32)[:case["Bd"]].contiguous()
    if case["pad"]:
        slots[case["Bd"] - case["pad"]:] = -1
    return slots


# ----------------------------------------------------------------------------------------------- runs

def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["kind"]](s, c)


def _library():
    import linear_attention_recurrence_06_b200 as kda
    return kda


def _own_scan(s, c):
    return _library().scan_fwd(s["x"], s["log_alpha"], s["init"], gate=s["gate"], normalize=c["normalize"],
                               cu_seqlens=s["cu"])


def _grads(g, c):
    out = {"dx": g["dx"], "dlog_alpha": g["dlog_alpha"], "dgate": g["dgate"]}
    if c["init"]:
        out["d_initial_state"] = g["d_initial_state"]
    return out


def _own_train(s, c):
    kda = _library()
    h, last, states = kda.scan_fwd(s["x"], s["log_alpha"], s["init"], gate=s["gate"], normalize=c["normalize"],
                                   cu_seqlens=s["cu"], chunk_states=True)
    g = kda.scan_bwd(s["x"], s["log_alpha"], s["d_h"], s["init"], s["d_final"], gate=s["gate"], normalize=c["normalize"],
                     cu_seqlens=s["cu"], chunk_states=states, out_dtype=s["x"].dtype, want_d_initial_state=c["init"])
    return {"h": h, "final_state": last, **_grads(g, c)}


def _own_scan_bwd(s, c):
    g = _library().scan_bwd(s["x"], s["log_alpha"], s["d_h"], s["init"], s["d_final"], gate=s["gate"],
                            normalize=c["normalize"], cu_seqlens=s["cu"], out_dtype=s["x"].dtype,
                            want_d_initial_state=c["init"])
    return _grads(g, c)


def _own_scan_decode(s, c):
    h = _library().scan_decode_steps(s["pool"], s["x"], s["log_alpha"], gate=s["gate"], normalize=c["normalize"],
                                     slots=s["slots"])
    return h, s["pool"]


def _own_gate_norm_bwd(s, c):
    return _library().gate_norm_bwd(s["o"], s["g"], s["d_y"], s["w"], out_dtype=_dt(c["grad"]))


def _own_pages(s, c):
    _library().state_copy(s["pool"], s["dst"], s["pool"], s["src"], layered=True)
    return s["pool"]


def _own_compact(s, c):
    kda = _library()
    live = s["live"].clone()  # the next pass finds the same sequences ended
    p = kda.state_compact(live)
    kda.state_copy(s["pool"], p["dst_slots"], s["pool"], p["src_slots"], layered=True)
    return {"pool": s["pool"], "live": live, "new_slots": p["new_slots"], "n_live": p["n_live"]}


def _own_decode(s, c):
    kda = _library()
    o = kda.decode_steps(s["pool"], s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], gate=s["gate"], slots=s["slots"])
    return o, s["pool"]


_own = {"scan": _own_scan, "train": _own_train, "scan_bwd": _own_scan_bwd, "scan_decode": _own_scan_decode,
        "gate_norm_bwd": _own_gate_norm_bwd, "pages": _own_pages, "compact": _own_compact, "decode": _own_decode}


# ------------------------------------------------------------------------------------- the plain forms

def _doubling(a, b, longest):
    """b_t + a_t (b_{t-1} + a_{t-1} (...)) along dim 1, by combining neighbours at distances 1, 2, 4, ..."""
    d = 1
    while d < longest:
        b = torch.cat([b[:, :d], torch.addcmul(b[:, d:], a[:, d:], b[:, :-d])], 1)
        if 2 * d < longest:
            a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _ends(s, T):
    """Packed sequences that have tokens: their numbers, first and last tokens."""
    cu = s["cu"].long()
    full = (cu[1:] > cu[:-1]).nonzero()[:, 0]
    return full, cu[:-1][full], cu[1:][full] - 1


def _terms(s, c):
    """Decay a, weight w, gate value g, input u: in fp32, or in fp64 where a state adds up so many tokens that the
    rounding of decays next to 1 would show."""
    wide = F64 if s.get("max_seqlen", s["x"].shape[1]) > 4096 else F32
    x, l = s["x"].to(wide), s["log_alpha"].to(wide).clamp(max=0)
    a = l.exp()
    w = (-torch.expm1(2 * l)).sqrt() if c["normalize"] else None
    g = torch.sigmoid(s["gate"].to(wide)) if s["gate"] is not None else None
    u = x if w is None else w * x
    u = u if g is None else u * g
    return x, a, w, g, u


def _forward(s, c, a, u):
    """All states in fp32, and the last of each sequence."""
    init, T = s["init"], u.shape[1]
    init = None if init is None else init.to(u.dtype)
    if s["cu"] is None:
        if init is not None:
            u = torch.cat([torch.addcmul(u[:, :1], a[:, :1], init[:, None]), u[:, 1:]], 1)
        h = _doubling(a, u, T)
        return h, h[:, -1].float()
    full, first, last = _ends(s, T)
    a0 = a.clone()
    if init is not None:
        u = u.clone()
        u[0, first] += a[0, first] * init[full]
    a0[0, first] = 0
    h = _doubling(a0, u, s["max_seqlen"])
    fin = u.new_zeros((s["cu"].numel() - 1, u.shape[2])) if init is None else init.clone()
    fin[full] = h[0, last]
    return h, fin.float()


def _plain_scan(s, c):
    _, a, _, _, u = _terms(s, c)
    h, fin = _forward(s, c, a, u)
    return h.to(s["x"].dtype), fin


def _backward(s, c, x, a, w, g, u, h):
    """Gradients from all states h, rounded once to the inputs' type."""
    dt, init, fin = s["x"].dtype, s["init"], s["d_final"]
    dh = s["d_h"].to(x.dtype, copy=True)
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    if s["cu"] is None:
        if fin is not None:
            dh[:, -1] += fin
        if init is not None:
            prev[:, 0] = init
        longest = x.shape[1]
    else:
        full, first, last = _ends(s, x.shape[1])
        nxt[0, last] = 0
        if fin is not None:
            dh[0, last] += fin[full]
        prev[0, first] = init[full].to(x.dtype) if init is not None else 0
        longest = s["max_seqlen"]
    G = _doubling(nxt.flip(1), dh.flip(1), longest).flip(1)
    dl = a * prev
    if w is not None:
        dl = dl - torch.where(w > 0, a * a * x * (1 if g is None else g) / w, 0)
    dx = G if w is None else G * w
    out = {"dx": (dx if g is None else dx * g).to(dt), "dlog_alpha": (G * dl).to(dt),
           "dgate": None if g is None else (G * u * (1 - g)).to(dt)}
    if init is not None:
        ag = a * G
        if s["cu"] is None:
            out["d_initial_state"] = ag[:, 0].float()
        else:
            out["d_initial_state"] = torch.zeros_like(init) if fin is None else fin.clone()
            out["d_initial_state"][full] = ag[0, first].float()
    return out


def _plain_train(s, c):
    t = _terms(s, c)
    h, fin = _forward(s, c, t[1], t[4])
    return {"h": h.to(s["x"].dtype), "final_state": fin, **_backward(s, c, *t, h)}


def _plain_scan_bwd(s, c):
    t = _terms(s, c)
    return _backward(s, c, *t, _forward(s, c, t[1], t[4])[0])


def _plain_scan_decode(s, c):
    n_live = c["Bd"] - c["pad"]
    rows = s["slots"][:n_live].long()
    _, a, _, _, u = _terms(s, c)
    h, out = s["pool"][rows], torch.zeros_like(u)
    for t in range(c["n"]):
        h = torch.addcmul(u[t, :n_live], a[t, :n_live], h)
        out[t, :n_live] = h
    s["pool"][rows] = h
    return out.to(s["x"].dtype), s["pool"]


def _plain_gate_norm_bwd(s, c):
    o, dy, g = s["o"].float(), s["d_y"].float(), torch.sigmoid(s["g"].float())
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-6)
    n = o * r
    dyn = dy * n * g
    dn = dy * g
    d_gate = dyn * (1 - g)
    if s["w"] is not None:
        dn, d_gate = dn * s["w"], d_gate * s["w"]
    dt = _dt(c["grad"])
    return {"d_o": (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(dt), "d_gate": d_gate.to(dt),
            "d_norm_weight": dyn.sum(0)}


def _plain_pages(s, c):
    m, pool = c["moves"], s["pool"]
    pool[:, s["dst"][:m].long()] = pool[:, s["src"][:m].long()]
    pool[:, s["dst"][m:].long()] = 0
    return pool


def _plain_compact(s, c):
    pool, live, P = s["pool"], s["live"].bool(), c["P"]
    n = live.sum()
    at = torch.arange(P, device=live.device)
    holes = ((~live) & (at < n)).nonzero()[:, 0]
    tail = (live & (at >= n)).nonzero()[:, 0]
    pool[:, holes] = pool[:, tail]
    new = torch.where(live, at, -1)
    new[tail] = holes
    return {"pool": pool, "live": (at < n).to(torch.uint8), "new_slots": new.int(), "n_live": n.int().reshape(1)}


def _plain_decode(s, c):
    n_live = c["Bd"] - c["pad"]
    rows = s["slots"][:n_live].long()
    S = s["pool"][rows]
    out = torch.zeros(s["v"].shape, device="cuda")
    for t in range(c["n"]):
        q, k, v, l, b = (s[name][t, :n_live].float() for name in ("q", "k", "v", "log_alpha", "beta"))
        S = S * l.clamp(min=-5).exp()[..., None]
        e = b[..., None] * (v - (S * k[..., None]).sum(-2))
        S = S + k[..., None] * e[..., None, :]
        o = (S * q[..., None]).sum(-2)
        if s["gate"] is not None:
            o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-6) * torch.sigmoid(s["gate"][t, :n_live].float())
        out[t, :n_live] = o
    s["pool"][rows] = S
    return out.to(s["v"].dtype), s["pool"]


_plain = {"scan": _plain_scan, "train": _plain_train, "scan_bwd": _plain_scan_bwd, "scan_decode": _plain_scan_decode,
          "gate_norm_bwd": _plain_gate_norm_bwd, "pages": _plain_pages, "compact": _plain_compact, "decode": _plain_decode}


# --------------------------------------------------------------------------------------- what it costs

def work(case):
    k = case["kind"]
    if k in ("scan", "train", "scan_bwd"):
        e = 2 if case["dtype"] == "bf16" else 4
        if case["lens"] == "fixed":
            tok, N = case["B"] * case["T"], case["B"]
        else:
            tok, N = sum(_lengths(case, 0)), case["N"]
        n, ins, states = tok * case["D"], 2 + case["gate"], N * case["D"] * 4
        fwd = n * e * (ins + 1) + states * (1 + case["init"])
        bwd = n * e * (ins + 1 + ins) + states * 3 * case["init"]
        return {"bytes": {"scan": fwd, "scan_bwd": bwd, "train": fwd + bwd}[k], "flops": n * {"scan": 8, "scan_bwd": 20, "train": 28}[k]}
    if k == "scan_decode":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["Bd"] - case["pad"]
        return {"bytes": rows * case["D"] * (8 + case["n"] * e * (2 + case["gate"])) + case["Bd"] * case["n"] * case["D"] * e,
                "flops": 8 * rows * case["D"] * case["n"]}
    if k == "gate_norm_bwd":
        e, f = (2 if case[x] == "bf16" else 4 for x in ("dtype", "grad"))
        return {"bytes": case["rows"] * D_HEAD * (3 * e + 2 * f), "flops": case["rows"] * D_HEAD * 20}
    page = case["H"] * D_HEAD * D_HEAD * 4
    if k == "pages":
        return {"bytes": case["L"] * page * (min(case["sources"], case["moves"]) + case["moves"] + case["clear"]), "flops": 0}
    if k == "compact":
        moved = max(0.25, case["P"] * case["live"] * (1 - case["live"]))
        return {"bytes": 2 * case["L"] * page * moved, "flops": 0}
    e, rows = (2 if case["dtype"] == "bf16" else 4), case["Bd"] - case["pad"]
    return {"bytes": rows * (2 * page + case["n"] * case["H"] * D_HEAD * e * (4 + case["gate"])) + case["n"] * case["Bd"] * case["H"] * D_HEAD * e,
            "flops": rows * case["n"] * case["H"] * D_HEAD * D_HEAD * 7}


# ------------------------------------------------------------------------------- the definition, 64 bits

def _each(s):
    """(row of the token tensors, first token, end) of every sequence."""
    if s["cu"] is None:
        return [(b, 0, s["x"].shape[1]) for b in range(s["x"].shape[0])]
    at = s["cu"].tolist()
    return [(0, i, j) for i, j in zip(at[:-1], at[1:])]


def _steps(s, c, x, l, gate, init):
    """The recurrence token by token, all sequences side by side, the longest first. Returns where each state belongs
    (row and token), the states in that order, and the last one of every sequence."""
    seqs = _each(s)
    order = sorted(range(len(seqs)), key=lambda n: seqs[n][1] - seqs[n][2])
    lens = torch.tensor([seqs[n][2] - seqs[n][1] for n in order])
    row = torch.tensor([seqs[n][0] for n in order], device="cuda")
    first = torch.tensor([seqs[n][1] for n in order], device="cuda")
    counts = (lens[None] > torch.arange(int(lens[0]))[:, None]).sum(1).tolist()  # sequences that have a token t
    i = torch.cat([row[:m] for m in counts]) if counts else row[:0]
    j = torch.cat([first[:m] + t for t, m in enumerate(counts)]) if counts else row[:0]
    lt, v = l[i, j].clamp(max=0), x[i, j]
    if c["normalize"]:
        v = v * (-torch.expm1(2 * lt)).sqrt()
    if gate is not None:
        v = v / (1 + (-gate[i, j]).exp())
    h = init[order] if init is not None else torch.zeros((len(seqs), x.shape[2]), dtype=F64, device="cuda")
    states, done = [], []
    for a, u in zip(lt.exp().split(counts), v.split(counts)):
        done.append(h[len(u):])
        h = a * h[:len(u)] + u
        states.append(h)
    last = torch.cat([h] + done[::-1])
    back = torch.empty(len(order), dtype=torch.long, device="cuda")
    back[torch.tensor(order, device="cuda")] = torch.arange(len(order), device="cuda")
    return i, j, torch.cat(states) if states else v, last[back]


def exact(case, seed):
    s, k = prepare(case, seed), case["kind"]
    c = s["case"]
    if k in ("scan", "train", "scan_bwd"):
        grad = k != "scan"
        if grad and s["x"].numel() > 40_000_000:
            return None
        wide = lambda v: None if v is None else v.to(F64).requires_grad_(grad)  # noqa: E731
        x, l, gate, init = wide(s["x"]), wide(s["log_alpha"]), wide(s["gate"]), wide(s["init"])
        with torch.set_grad_enabled(grad):
            i, j, states, last = _steps(s, c, x, l, gate, init)
            h = torch.empty(x.shape, dtype=F64, device="cuda")
            h[i, j] = states.detach()
            if not grad:
                return h, last
            total = (states * s["d_h"].to(F64)[i, j]).sum()
            if s["d_final"] is not None:
                total = total + (last * s["d_final"].to(F64)).sum()
            total.backward()
        out = {"dx": x.grad, "dlog_alpha": l.grad, "dgate": None if gate is None else gate.grad}
        if init is not None:
            out["d_initial_state"] = init.grad
        return {**out, "h": h, "final_state": last.detach()} if k == "train" else out
    if k == "scan_decode":
        pool, h = s["pool"].to(F64), torch.zeros(s["x"].shape, dtype=F64, device="cuda")
        for b, slot in enumerate(s["slots"].tolist()):
            for t in range(c["n"] if slot >= 0 else 0):
                lt, v = s["log_alpha"][t, b].to(F64).clamp(max=0), s["x"][t, b].to(F64)
                v = v * (1 - (2 * lt).exp()).sqrt() if c["normalize"] else v
                v = v * torch.sigmoid(s["gate"][t, b].to(F64)) if s["gate"] is not None else v
                pool[slot] = lt.exp() * pool[slot] + v
                h[t, b] = pool[slot]
        return h, pool
    if k == "gate_norm_bwd":
        o, g = (s[n].to(F64).requires_grad_() for n in ("o", "g"))
        w = (torch.ones(D_HEAD, device="cuda") if s["w"] is None else s["w"]).to(F64).requires_grad_()
        with torch.enable_grad():
            y = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w / (1 + (-g).exp())
            y.backward(s["d_y"].to(F64))
        return {"d_o": o.grad, "d_gate": g.grad, "d_norm_weight": w.grad}
    if k == "pages":
        pool = s["pool"].to(F64)
        for d, i in zip(s["dst"].tolist(), s["src"].tolist()):
            pool[:, d] = pool[:, i] if i >= 0 else 0
        return pool
    if k == "compact":
        live, pool, P = s["live"].tolist(), s["pool"].to(F64), c["P"]
        n = sum(live)
        new = [p if live[p] else -1 for p in range(P)]
        tail = [p for p in range(n, P) if live[p]]
        for hole in (p for p in range(n) if not live[p]):
            p = tail.pop(0)
            pool[:, hole] = pool[:, p]
            new[p] = hole
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"pool": pool, "live": i32([int(p < n) for p in range(P)]).to(torch.uint8), "new_slots": i32(new), "n_live": i32([n])}
    pool, out = s["pool"].to(F64), torch.zeros(s["v"].shape, dtype=F64, device="cuda")
    for b, slot in enumerate(s["slots"].tolist()):
        for t in range(c["n"] if slot >= 0 else 0):
            q, kk, v, l = (s[name][t, b].to(F64) for name in ("q", "k", "v", "log_alpha"))
            S = torch.exp(l.clamp(min=-5))[:, :, None] * pool[slot]
            err = v - torch.einsum("hkv,hk->hv", S, kk)
            S = S + s["beta"][t, b].to(F64)[:, None, None] * torch.einsum("hk,hv->hkv", kk, err)
            o = torch.einsum("hkv,hk->hv", S, q)
            if s["gate"] is not None:
                o = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt() * torch.sigmoid(s["gate"][t, b].to(F64))
            pool[slot], out[t, b] = S, o
    return out, pool
