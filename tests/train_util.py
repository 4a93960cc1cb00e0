"""Plain 64-bit forms of the operators of a training step and the tolerances their tests use (the
conventions of ops_util: EPS32 and EPS16 are half a unit in the last place).

exp, 1 / x: the hardware's exponential of a product with log2(e) is off by at most (2 |z| + 4) EPS32 of
its value (the product's rounding grows with |z|), a reciprocal by 2 EPS32; RZ(z) below counts both and
the few roundings of the products around them.  Both give 0 for results below 2^-126, the smallest normal
number: a sigmoid s(z) of z < -87.3 is then off by up to FLUSH = 2^-126 beside its relative error, and what
it is multiplied with carries that on: |z| FLUSH for z s(z), (1 + |z|) FLUSH for the slope s (1 + z (1 - s)).
"""
import torch

from ops_util import EPS16, EPS32, F8, grouped_ref


FLUSH = 2.0 ** -126


def rz(z):
    return (4 * z.abs() + 24) * EPS32


def silu(z):
    return z * torch.sigmoid(z)


def gated_ref(rows64, w, offsets):
    """((h, tol), (gate_up, tol)), tolerances with the roundings of the results."""
    I = w.shape[1] // 2
    pre, t = grouped_ref(rows64, w, offsets)
    g, u, tg, tu = pre[:, :I], pre[:, I:], t[:, :I], t[:, I:]
    h = silu(g) * u
    # |silu'| <= 1.1
    th = 1.1 * tg * u.abs() + silu(g).abs() * tu + 1.1 * tg * tu + h.abs() * rz(g) + (g * u).abs() * FLUSH
    return (h, th + EPS16 * (h.abs() + th)), (pre, t + EPS16 * (pre.abs() + t))


def gated_grad_raw(dy, w, gate_up, offsets):
    """((d_gate_up, tol), (h, tol)) before their rounding to bf16; rows of no group NaN."""
    dh, t = grouped_ref(dy.to(F8), w.transpose(1, 2), offsets)
    I = dh.shape[1]
    g, u = gate_up[:, :I].to(F8), gate_up[:, I:].to(F8)
    s, n = torch.sigmoid(g), torch.sigmoid(-g)
    slope, mag = s * (1 + g * n), s * (1 + g.abs() * n)
    dg, du, h = dh * u * slope, dh * g * s, g * s * u
    td = torch.cat([t * (u * slope).abs() + (dh.abs() + t) * u.abs() * mag * rz(g),
                    t * (g * s).abs() + (dh.abs() + t) * (g * s).abs() * rz(g)], 1)
    far = (dh.abs() + t) * FLUSH
    td = td + torch.cat([far * u.abs() * (1 + g.abs()), far * g.abs()], 1)
    th = h.abs() * rz(g) + (g * u).abs() * FLUSH
    return (torch.cat([dg, du], 1), td), (torch.where(torch.isnan(dh), dh, h), th)


def gated_grad_ref(dy, w, gate_up, offsets):
    """((d_gate_up, tol), (h, tol)); rows of no group NaN."""
    (d, td), (h, th) = gated_grad_raw(dy, w, gate_up, offsets)
    return (d, td + EPS16 * (d.abs() + td)), (h, th + EPS16 * 1.01 * torch.nan_to_num(h).abs())


def feed_forward_grad_raw(dy, x64, w_gate_up, w_down, gate_up, offsets):
    """{name: (gradient, tol)} of a block before the results' rounding, nothing rounded between: products of fp32
    values whose sums take 2 EPS32 a term; x64 the grouped rows of x.  Rows of no group NaN."""
    (d, td), (h, th) = gated_grad_raw(dy, w_down, gate_up, offsets)
    (E, I2, K), H = w_gate_up.shape, w_down.shape[1]
    dx, tx = torch.full((len(dy), K), float("nan"), dtype=F8), torch.zeros(len(dy), K, dtype=F8)
    gu, tgu, dn, tdn = (torch.zeros(s, dtype=F8) for s in ((E, I2, K), (E, I2, K), (E, H, I2 // 2), (E, H, I2 // 2)))
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        n = r.stop - r.start
        if n <= 0:
            continue
        w, dd, a, y = w_gate_up[e].to(F8), d[r].abs() + td[r], x64[r].abs(), dy[r].to(F8)
        dx[r], tx[r] = d[r] @ w, td[r] @ w.abs() + 2 * EPS32 * I2 * (dd @ w.abs())
        gu[e], tgu[e] = d[r].t() @ x64[r], td[r].t() @ a + 2 * EPS32 * n * (dd.t() @ a)
        dn[e], tdn[e] = y.t() @ h[r], y.abs().t() @ (th[r] + 2 * EPS32 * n * (h[r].abs() + th[r]))
    return {"x": (dx, tx), "w_gate_up": (gu, tgu), "w_down": (dn, tdn)}


def invert_ref(perm, n, end):
    inv = torch.full((n,), -1, dtype=torch.int64)
    for p in range(min(end, len(perm)) - 1, -1, -1):  # the lowest row is written last
        a = int(perm[p])
        if 0 <= a < n:
            inv[a] = p
    return inv.int()


def combine_ref(y, inverse, k, weight=None, add=None):
    """(out, tol without the result's rounding)."""
    inv = inverse.long().view(-1, k)
    has = (inv >= 0) & (inv < y.shape[0])
    rows = y.to(F8)[inv.clamp(0, max(y.shape[0] - 1, 0))] if y.shape[0] else torch.zeros(*inv.shape, y.shape[1], dtype=F8)
    rows = torch.where(has[:, :, None], rows, torch.zeros((), dtype=F8))
    w = torch.ones(inv.shape, dtype=F8) if weight is None else torch.where(has, weight.to(F8), torch.zeros((), dtype=F8))
    t = w[:, :, None] * rows
    out, mag = t.sum(1), t.abs().sum(1)
    if add is not None:
        out, mag = out + add.to(F8), mag + add.to(F8).abs()
    return out, (k + 1) * EPS32 * mag


def dot_terms(H):
    """Roundings that a sum over H elements by one wave adds up: eight elements a lane and 512, then six
    steps of the wave, and the products' own."""
    return 8 * ((H + 511) // 512) + 8


def loss_ref(x, w, target, ignore=-100):
    """(loss, tol, lse, tol, logits, tol, valid)."""
    x, w = x.to(F8), w.to(F8)
    H, V = x.shape[1], w.shape[0]
    z = x @ w.t()
    tz = 2 * EPS32 * H * (x.abs() @ w.abs().t())
    lse = torch.logsumexp(z, 1)
    valid = (target >= 0) & (target < V) & (target != ignore)
    hit = z.gather(1, target.clamp(0, V - 1)[:, None])[:, 0]
    m = z.max(1).values
    # a sum of V positive terms: chains of 32 + 4 + 16 + V / 4096 additions; each term as exp above; the
    # logarithm and the sum with the maximum
    span = (m - z.min(1).values) + 2 * tz.max(1).values
    tl = tz.max(1).values + (2 * span + 80 + V / 4096) * EPS32 + 4 * EPS32 * (m.abs() + lse.abs() + 1)
    loss = torch.where(valid, lse - hit, torch.zeros((), dtype=F8))
    t = torch.where(valid, tl + tz.gather(1, target.clamp(0, V - 1)[:, None])[:, 0] + EPS32 * (lse.abs() + hit.abs()),
                    torch.zeros((), dtype=F8))
    return loss, t, lse, tl, z, tz, valid


def loss_grad_ref(d_loss, x, w, target, ignore=-100):
    """((dx, tol), (dw, tol)) without the results' roundings."""
    _, _, lse, tl, z, tz, valid = loss_ref(x, w, target, ignore)
    T, V = z.shape
    a = torch.where(valid, d_loss.to(F8), torch.zeros((), dtype=F8))
    p = torch.exp(z - lse[:, None])
    e = torch.zeros_like(p)
    rows = torch.nonzero(valid)[:, 0]
    e[rows, target[rows]] = 1.0
    # the kernel's d is p - e in bf16: p off by the logit's and the log-sum-exp's errors and its own
    # exponential, then a difference, then the rounding
    rel = tz + tl[:, None] + (2 * (z - lse[:, None]).abs() + 8) * EPS32
    u = torch.where(valid[:, None], p - e, torch.zeros((), dtype=F8))
    tu = torch.where(valid[:, None], p * rel * 1.01 + EPS32 * (p + e), torch.zeros((), dtype=F8))
    tu = tu + EPS16 * (u.abs() + tu)
    x, w = x.to(F8), w.to(F8)
    dx, dw = (a[:, None] * u) @ w, (a[:, None] * u).t() @ x
    tx = a.abs()[:, None] * (tu @ w.abs() + (2 * V + 2) * EPS32 * ((u.abs() + tu) @ w.abs()))
    # dw: rows x a / max |a|, two roundings of fp32 and one to bf16, which is none where all a are the same
    same = bool((a[valid].abs() == a.abs().max()).all()) if bool(valid.any()) else True
    row = a.abs()[:, None] * x.abs()
    tw = tu.t() @ row + ((0 if same else 1.01 * EPS16) + (2 * T + 4) * EPS32) * ((u.abs() + tu).t() @ row)
    return (dx, tx), (dw, tw)
