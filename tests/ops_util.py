"""Plain 64-bit forms of the operators in moe_ops.h and the tolerances their tests use.

Tolerances are per element, from the arithmetic alone.  EPS32 = 2^-24 and
EPS16 = 2^-8 are half a unit in the last place of fp32 and bf16, relative:
  - a sum of n fp32 products differs from the exact one by at most
    n * 2 * EPS32 * (sum of the products' magnitudes) (2 EPS32 a term: the
    matrix instructions may truncate where fp32 addition rounds);
  - every result is rounded once to its type: EPS32 or EPS16 of its magnitude.
"""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24
EPS16 = 2.0 ** -8
TINY = 1e-37  # below it fp32 and bf16 lose relative accuracy
F8 = torch.float64


def eps_of(dtype):
    return EPS16 if dtype == torch.bfloat16 else EPS32


def close(got, want, tol, what=""):
    """Every element within its tolerance; NaN only where expected."""
    got = got.detach().cpu().to(F8)
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} for {tuple(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN at the wrong places"
    err = torch.where(nan, torch.zeros((), dtype=F8), (got - want).abs())
    bad = err > torch.where(nan, torch.ones((), dtype=F8), tol + TINY)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {want[i]}, "
                             f"tolerance {tol.expand_as(err)[i] if torch.is_tensor(tol) else tol}")


def randn(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return o


def source_rows(rows, perm, top_k, x_rows):
    """Row of x for each grouped row; -1: a row of zeros."""
    if perm is None:
        return torch.arange(rows)
    p = perm.long()
    t = torch.div(p, top_k, rounding_mode="floor")
    return torch.where((p >= 0) & (t < x_rows), t, torch.full_like(t, -1))


def take(x, src):
    """Rows src of x in 64 bits, zeros for -1."""
    r = x.to(F8)[src.clamp(min=0)] if x.shape[0] else torch.zeros(len(src), x.shape[1], dtype=F8)
    return torch.where((src >= 0)[:, None], r, torch.zeros((), dtype=F8))


def grouped_ref(rows64, w, offsets):
    """(y, tolerance without the output's rounding) of rows64 [R, K] and w [E, N, K]; rows of no group NaN."""
    R, (E, N, K) = rows64.shape[0], w.shape
    y = torch.full((R, N), float("nan"), dtype=F8)
    mag = torch.zeros(R, N, dtype=F8)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            we = w[e].to(F8).t()
            y[a:b] = rows64[a:b] @ we
            mag[a:b] = rows64[a:b].abs() @ we.abs()
    return y, 2 * EPS32 * K * mag


def grad_input_ref(dy, w, offsets):
    return grouped_ref(dy.to(F8), w.transpose(1, 2), offsets)


def grad_weight_ref(rows64, dy, offsets):
    E = len(offsets) - 1
    N, K = dy.shape[1], rows64.shape[1]
    dw = torch.zeros(E, N, K, dtype=F8)
    tol = torch.zeros(E, N, K, dtype=F8)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            d = dy[a:b].to(F8).t()
            dw[e] = d @ rows64[a:b]
            tol[e] = 2 * EPS32 * (b - a) * (d.abs() @ rows64[a:b].abs())
    return dw, tol


def quantize_ref(x):
    """(codes, scale) in 64 bits; rows with an infinity or NaN: codes 0, scale that value."""
    x = x.to(F8)
    m = x.abs().amax(dim=1)
    m = torch.where(torch.isnan(x).any(dim=1), torch.full_like(m, float("nan")), m)
    ok = torch.isfinite(m) & (m > 0)
    q = torch.round(127.0 * x / torch.where(ok, m, torch.ones_like(m))[:, None])
    return torch.where(ok[:, None], q, torch.zeros((), dtype=F8)), m / 127.0


# ------------------------------------------------------------------ norms

def rms(v, w, eps):
    return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps) * w


def merge_ref(residual, y, w, eps, gate=None, scale=1.0):
    g = 1.0 if gate is None else torch.sigmoid(gate[:, None] if gate.dim() == 1 else gate)
    return residual + scale * g * rms(y, w, eps)


def rms_grad(d, v, w, eps):
    """Gradients of rms by the formula, and the magnitudes of their terms: (dv, dv_mag, dw terms)."""
    r = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)
    dn = d * w
    dv = r * dn - v * r ** 3 * (dn * v).mean(dim=1, keepdim=True)
    mag = (r * dn).abs() + v.abs() * r ** 3 * (dn * v).abs().mean(dim=1, keepdim=True)
    return dv, mag, d * v * r


def merge_grad_ref(d_out, d_h, y, w, eps, gate, scale, out, wn):
    """Gradients by the formulas in 64 bits and the magnitudes they come from, as
    {name: (value, magnitude)}; magnitudes bound what relative errors of 2^-24 in the terms do."""
    D, Dm = (torch.zeros_like(y), torch.zeros_like(y)) if d_out is None else (d_out, d_out.abs())
    res = {}
    if d_h is not None:
        dv, mag, t = rms_grad(d_h, out, wn, eps)
        D, Dm = D + dv, Dm + mag
        res["next_weight"] = (t.sum(0), t.abs().sum(0))
    res["residual"] = (D, Dm)
    g = torch.ones(1, 1, dtype=F8) if gate is None else torch.sigmoid(gate[:, None] if gate.dim() == 1 else gate)
    db, dbm = scale * g * D, abs(scale) * g * Dm
    dy, _, t = rms_grad(db, y, w, eps)
    _, dym, tm = rms_grad(dbm, y.abs(), w.abs(), eps)
    res["y"] = (dy, dym)
    res["weight"] = (t.sum(0), tm.abs().sum(0))
    if gate is not None:
        s = scale * g * torch.sigmoid(-(gate[:, None] if gate.dim() == 1 else gate))
        dg = s * D * rms(y, w, eps)
        dgm = s.abs() * Dm * rms(y, w, eps).abs()
        if gate.dim() == 1:
            dg, dgm = dg.sum(1), dgm.sum(1)
        res["gate"] = (dg, dgm)
    return res


def sum_terms(H):
    """Rounding errors a row statistic adds up, in units of EPS32: each of the fp32 sums over H terms
    runs in chains of at most H / 64 + 32 additions, its root and the few products after it add less
    than 32, a gate's exponential of |z| <= 16 less than 32."""
    return H / 64 + 96
