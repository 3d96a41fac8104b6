"""fp64 reference of the element-wise gated scan and of its gradients, token by token, with a bound on
what fp32 arithmetic may be off by, element for element.

Bounds (e = 2^-24, half a step of fp32 relative to the value).  A step h = a h + u rounds at most twice, and a
itself is off by at most 5 e relative to 1 (the polynomial's six roundings scaled by |a - 1| < 1/4, or __expf's
2 + 1.173 |l| ulps times e^l <= 1): together 8 e H_t, where H is the recurrence of the absolute values.  u is off by
at most 36 e |u| for |gate| <= 6 (__expf 2 + 1.173 * 6 ulps of 2 e, the division 4 e, the sum 1 e, w 8 e, products 3 e).
Joining pieces of a sequence adds at most 10 e H per 8 tokens or more, which 8 e H per token covers.  Errors are
carried on by the recurrence itself:  E_t = a_t E_{t-1} + e (8 H_t + 36 |u_t|).  The gradient's walk is the same
with dh in u's place.  Products of these add their factors' relative errors; the constants are written beside them.
An output of fewer bits adds half a step of its type.
"""
import torch

EPS = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sequences(B, T, cu):
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return list(zip(cu[:-1], cu[1:]))


def scan(x, log_alpha, gate=None, normalize=False, init=None, cu=None, d_h=None, d_final=None):
    """All tensors on one device; x etc. [B, T, D], init [N, D], cu a list.  Returns a dict of fp64 tensors: h, final
    and their bounds h_e, final_e; with d_h also dx, dl, dgate, d_init and their bounds.  Tokens outside every
    sequence are NaN."""
    B, T, D = x.shape
    flat = lambda t: None if t is None else t.to(F64).reshape(B * T, D)  # noqa: E731
    x_, la, g_, dh = flat(x), flat(log_alpha), flat(gate), flat(d_h)
    l = torch.where(la > 0, torch.zeros_like(la), la)
    a = l.exp()
    s = torch.ones_like(x_) if g_ is None else torch.sigmoid(g_)
    n = -torch.expm1(2 * l)
    w = n.sqrt() if normalize else torch.ones_like(x_)
    u = w * s * x_
    nan = lambda: torch.full_like(x_, float("nan"))  # noqa: E731
    h, he, hp, hpe = nan(), nan(), nan(), nan()
    seqs = sequences(B, T, cu)
    z = torch.zeros(D, dtype=F64, device=x.device)
    fin, fine = [], []
    for k, (i, j) in enumerate(seqs):
        v = z if init is None else init[k].to(F64)
        H, E = v.abs(), z
        for t in range(i, j):
            hp[t], hpe[t] = v, E
            v = a[t] * v + u[t]
            H = a[t] * H + u[t].abs()
            E = a[t] * E + EPS * (8 * H + 36 * u[t].abs())
            h[t], he[t] = v, E
        fin.append(v)
        fine.append(E)
    stack = lambda r: torch.stack(r) if r else torch.zeros((0, D), dtype=F64, device=x.device)  # noqa: E731
    shaped = lambda t: t.reshape(B, T, D)  # noqa: E731
    r = dict(h=shaped(h), h_e=shaped(he), final=stack(fin), final_e=stack(fine))
    if dh is None:
        return r
    dx, dl, dg, dxe, dle, dge = nan(), nan(), nan(), nan(), nan(), nan()
    di, die = [], []
    q = a * a * s * x_ / w if normalize else torch.zeros_like(x_)
    q = torch.where(n < 1e-37, torch.zeros_like(q), q) if normalize else q
    for k, (i, j) in enumerate(seqs):
        c = z if d_final is None else d_final[k].to(F64)
        C, E = c.abs(), z
        for t in range(j - 1, i - 1, -1):
            G, Gm = dh[t] + c, dh[t].abs() + C
            Ge = E + EPS * Gm
            dx[t] = G * w[t] * s[t]
            dxe[t] = w[t] * s[t] * (Ge + 40 * EPS * Gm)                    # w s: 36, the product, spare 3
            dg[t] = G * u[t] * (1 - s[t])
            dge[t] = u[t].abs() * ((1 - s[t]) * (Ge + 40 * EPS * Gm) + 24 * EPS * Gm)  # 1 - s: 22 e absolute
            m = a[t] * hp[t].abs() + q[t].abs()
            dl[t] = torch.where(la[t] > 0, z, G * (a[t] * hp[t] - q[t]))
            dle[t] = Ge * m + Gm * (a[t] * hpe[t] + 64 * EPS * m)         # q: u 36, n 6, the division 4, a^2 10, products
            c = a[t] * G
            C = a[t] * Gm
            E = a[t] * Ge + EPS * 8 * Gm
        di.append(c)
        die.append(E)
    r.update(dx=shaped(dx), dx_e=shaped(dxe), dl=shaped(dl), dl_e=shaped(dle), dgate=shaped(dg), dgate_e=shaped(dge),
             d_init=stack(di), d_init_e=stack(die))
    return r


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type (of ref and of the bound), where ref is a number; NaN and
    infinities of ref have to be got's."""
    g = got.detach().to(F64).reshape(ref.shape).to(ref.device)
    tol = bound + half_step(got.dtype) * (ref.abs() + bound)
    fine = torch.isfinite(ref)
    bad = fine & ~((g - ref).abs() <= tol + 2.0 ** -126)
    worst = torch.where(fine, (g - ref).abs() / (tol + 2.0 ** -126), torch.zeros_like(ref)).nan_to_num(1e9)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, the worst "
                                 f"{float(worst.max()):.3g} times its own")
    odd = ~fine
    assert torch.equal(torch.isnan(g[odd]), torch.isnan(ref[odd])), f"{what}: NaN elsewhere"
    inf = torch.isinf(ref)
    assert torch.equal(g[inf], ref[inf]), f"{what}: infinities elsewhere"
    return float(worst.max()) if worst.numel() else 0.0


def gate_norm_bwd(o, g, dy, w=None, eps=1e-6):
    """d_o, d_gate, d_w in fp64 and their bounds (e as above).  sigmoid is off by 21 e for |g| <= 6, 1 - s by 22 e of s
    absolute, r by (9 roundings of the sum of squares + the mean and eps) / 2 + 4 = 10 e, a row's dot product by 16 e
    of the sum of its absolute terms besides its factors' 40 e; d_w adds one rounding per summed row."""
    o, g, dy = (t.to(F64).reshape(-1, 128) for t in (o, g, dy))
    wv = torch.ones(128, dtype=F64, device=o.device) if w is None else w.to(F64)
    r = 1 / (o.square().mean(-1, keepdim=True) + eps).sqrt()
    s, n = torch.sigmoid(g), o * r
    dn = dy * wv * s
    dot, dota = (dn * n).mean(-1, keepdim=True), (dn * n).abs().mean(-1, keepdim=True)
    d_o = r * (dn - n * dot)
    d_oe = EPS * r * (40 * dn.abs() + n.abs() * 80 * dota)
    d_g = dn * n * (1 - s)
    d_ge = EPS * (dn * n).abs() * (60 * (1 - s) + 24)
    terms = dy * n * s
    rows = o.shape[0]
    return d_o, d_oe, d_g, d_ge, terms.sum(0), EPS * (rows + 45) * terms.abs().sum(0)
