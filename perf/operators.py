"""Cases, plain forms and definitions of the operators around the MoE layer.

  grouped        y[p] = x[row(p)] . W_e^T over the rows p of each expert's group (ragged sizes)
  grouped_grad   the gradients of that product: rows (dx) and weights (dW)
  i8             product of tokens quantised to 8 bits (one scale a token) with int8 weights (one
                 scale a channel)
  i8_grouped     the same, grouped by expert
  norm           RMSNorm before a block
  merge          RMSNorm after a block, times its sigmoid gate and the residual scale, added to the
                 residual stream, with the next block's RMSNorm of the sum
  merge_grad     the gradients of every input of merge
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step through its eight experts' gate/up projections
        dict(name="grouped_1tok", op="grouped", tokens=1, top_k=8, experts=256, n=1024, k=2048, skew=0.0,
             gather=True, out="bf16"),
        # the gate/up projections of a 4096-token prefill: rows gathered through the routing permutation
        dict(name="grouped_4096tok", op="grouped", tokens=4096, top_k=8, experts=256, n=1024, k=2048, skew=0.0,
             gather=True, out="bf16"),
        # an odd batch with skewed routing and sizes off every tile, rows already grouped, fp32 result
        dict(name="grouped_skew_odd", op="grouped", tokens=2501, top_k=4, experts=60, n=1000, k=1416, skew=1.2,
             gather=False, out="fp32"),
        # a training step's backward through a wide expert projection
        dict(name="grad_8192tok", op="grouped_grad", tokens=8192, top_k=2, experts=16, n=2048, k=2048, skew=0.0,
             gather=True, out="bf16"),
        # the same for many small experts, skewed, with fp32 weight gradients
        dict(name="grad_skew_701tok", op="grouped_grad", tokens=701, top_k=4, experts=64, n=512, k=1032, skew=1.2,
             gather=True, out="fp32"),
        # a projection of one decoded token on 8-bit weights
        dict(name="i8_1tok", op="i8", tokens=1, n=4096, k=2048, bias=False, out="bf16"),
        # a wide projection of a 4096-token prefill on 8-bit weights
        dict(name="i8_4096tok", op="i8", tokens=4096, n=8192, k=4096, bias=True, out="bf16"),
        # 8-bit experts: the gate/up projections of a 4096-token prefill
        dict(name="i8_grouped_4096tok", op="i8_grouped", tokens=4096, top_k=8, experts=256, n=1024, k=2048, skew=0.0,
             gather=True, out="bf16"),
        # the norm before a block over an odd prefill
        dict(name="norm_4099tok", op="norm", tokens=4099, h=2048, stream="bf16"),
        # the merge after a block of one decoded token, one gate a token
        dict(name="merge_1tok", op="merge", tokens=1, h=2048, gate="token", stream="bf16"),
        # the merge of an 8192-token chunk, a gate for every element, fp32 residual stream
        dict(name="merge_8192tok", op="merge", tokens=8192, h=2048, gate="element", stream="fp32"),
        # its backward in training, bf16 residual stream
        dict(name="merge_grad_8191tok", op="merge_grad", tokens=8191, h=2048, gate="element", stream="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_grad", "i8", "i8_grouped", "norm", "merge", "merge_grad"])
    if op in ("grouped", "i8_grouped", "grouped_grad"):
        while True:
            experts = _log_int(rng, 4, 256)
            step = 16 if op == "i8_grouped" else 8
            c = dict(op=op, tokens=_log_int(rng, 1, 4096), top_k=rng.choice([t for t in (1, 2, 4, 8) if t <= experts]),
                     experts=experts, n=8 * _log_int(rng, 8, 256), k=step * _log_int(rng, 64 // step, 2048 // step),
                     skew=rng.choice([0.0, 1.2]), gather=rng.random() < 0.7, out=rng.choice(["bf16", "fp32"]))
            if c["tokens"] * c["top_k"] * c["n"] * c["k"] <= 2 ** 36 and experts * c["n"] * c["k"] <= 2 ** 29:
                return c
    if op == "i8":
        while True:
            c = dict(op=op, tokens=_log_int(rng, 1, 8192), n=8 * _log_int(rng, 8, 1024), k=16 * _log_int(rng, 4, 512),
                     bias=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]))
            if c["tokens"] * c["n"] * c["k"] <= 2 ** 37:
                return c
    while True:
        c = dict(op=op, tokens=_log_int(rng, 1, 16384), h=8 * _log_int(rng, 8, 2048),
                 stream=rng.choice(["bf16", "fp32"]))
        if op != "norm":
            c["gate"] = rng.choice(["none", "token", "element"])
        if c["tokens"] * c["h"] <= 2 ** 24:
            return c


# ------------------------------------------------------------------ inputs

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, device="cuda", dtype=dtype)
    return out.normal_(0.0, scale, generator=g)


def _route(case, g):
    """Top-k of random scores, grouped by expert in token order: offsets and the permutation that the
    layer's routing reports (perm[p] = token * top_k + slot)."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    # Gumbel scores: top-k of them draws k experts without replacement, probabilities (rank + 1)^-skew
    u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
    scores = -torch.log(-torch.log(u))
    if case["skew"]:
        rank = torch.randperm(E, device="cuda", generator=g)
        scores -= case["skew"] * torch.log1p(rank.float())
    ids = scores.topk(k, dim=1).indices.reshape(-1)
    perm = torch.sort(ids, stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, perm


def _i8_weights(g, *shape):
    w = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = w.reshape(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(_randn(g, part.numel(), scale=36.0, dtype=torch.float32).clamp_(-127, 127).round_())
    # channels of different size, as weights of N(0, 0.02^2) scaled by their own largest value have
    s = (torch.rand(shape[:-1], device="cuda", generator=g) + 0.5) * (0.02 / 36.0)
    return w, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("grouped", "grouped_grad", "i8_grouped"):
        T, k, E, N, K = case["tokens"], case["top_k"], case["experts"], case["n"], case["k"]
        offsets, perm = _route(case, g)
        st.update(offsets=offsets, bounds=offsets.tolist(), perm=perm if case["gather"] else None, top_k=k,
                  x=_randn(g, T if case["gather"] else T * k, K))
        if op == "i8_grouped":
            st["w"], st["ws"] = _i8_weights(g, E, N, K)
        else:
            st["w"] = _randn(g, E, N, K, scale=0.02)
        if op == "grouped_grad":
            st["dy"] = _randn(g, T * k, N)
    elif op == "i8":
        T, N, K = case["tokens"], case["n"], case["k"]
        st["x"] = _randn(g, T, K)
        st["w"], st["ws"] = _i8_weights(g, N, K)
        st["bias"] = _randn(g, N, dtype=torch.float32) if case["bias"] else None
    else:
        T, H = case["tokens"], case["h"]
        dt = _DT[case["stream"]]
        st["x"] = _randn(g, T, H, dtype=dt)
        st["w_next"] = _randn(g, H, scale=0.1) + 1.0
        if op != "norm":
            st["y"] = _randn(g, T, H, scale=0.5)
            st["w"] = _randn(g, H, scale=0.1) + 1.0
            st["gate"] = {"none": None, "token": _randn(g, T), "element": None}[case["gate"]]
            if case["gate"] == "element":
                st["gate"] = _randn(g, T, H)
            st["scale"] = 0.22
        if op == "merge_grad":
            # stands for the stream that the forward pass stored
            st["out"] = _randn(g, T, H, dtype=dt)
            st["d_out"] = _randn(g, T, H, dtype=dt)
            st["d_h"] = _randn(g, T, H)
    return st


# ------------------------------------------------------------------ one pass

def _rows(st):
    x = st["x"]
    return x if st["perm"] is None else x[(st["perm"] // st["top_k"]).long()]


def _plain_grouped(st):
    rows, w, b = _rows(st).float(), st["w"], st["bounds"]
    y = torch.empty(rows.shape[0], w.shape[1], device="cuda", dtype=torch.float32)
    for e in range(w.shape[0]):
        if b[e + 1] > b[e]:
            y[b[e]:b[e + 1]] = rows[b[e]:b[e + 1]] @ w[e].float().t()
    return y.to(_DT[st["case"]["out"]])


def _plain_grad(st):
    rows, w, dy, b = _rows(st).float(), st["w"], st["dy"].float(), st["bounds"]
    dx = torch.empty(rows.shape, device="cuda", dtype=torch.float32)
    dw = torch.zeros(w.shape, device="cuda", dtype=torch.float32)
    for e in range(w.shape[0]):
        if b[e + 1] > b[e]:
            d, r = dy[b[e]:b[e + 1]], rows[b[e]:b[e + 1]]
            dx[b[e]:b[e + 1]] = d @ w[e].float()
            dw[e] = d.t() @ r
    return dx.bfloat16(), dw.to(_DT[st["case"]["out"]])


def _plain_quant(x):
    # the codes in 64 bits: values next to a rounding border
    m = x.abs().amax(dim=1, keepdim=True).double()
    q = torch.where(m > 0, torch.round(x.double() * 127.0 / m), torch.zeros((), dtype=torch.float64, device="cuda"))
    return q.float(), m[:, 0].float() / 127.0


def _plain_i8(st):
    q, s = _plain_quant(st["x"])
    y = (q @ st["w"].float().t()) * (s[:, None] * st["ws"])
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(_DT[st["case"]["out"]])


def _plain_i8_grouped(st):
    q, s = _plain_quant(st["x"])
    if st["perm"] is not None:
        t = (st["perm"] // st["top_k"]).long()
        q, s = q[t], s[t]
    w, ws, b = st["w"], st["ws"], st["bounds"]
    y = torch.empty(q.shape[0], w.shape[1], device="cuda", dtype=torch.float32)
    for e in range(w.shape[0]):
        i, j = b[e], b[e + 1]
        if j > i:
            y[i:j] = (q[i:j] @ w[e].float().t()) * (s[i:j, None] * ws[e])
    return y.to(_DT[st["case"]["out"]])


def _plain_rms(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * w.float()


def _plain_gate(st):
    g = st["gate"]
    if g is None:
        return 1.0
    g = torch.sigmoid(g.float())
    return g[:, None] if g.dim() == 1 else g


def _plain_merge(st):
    x = st["x"]
    out = (x.float() + st["scale"] * _plain_gate(st) * _plain_rms(st["y"], st["w"])).to(x.dtype)
    return out, _plain_rms(out, st["w_next"]).bfloat16()


def _plain_rms_grad(d, x, w):
    """(dx, dw) of x * r * w, r = rsqrt(mean x^2 + eps)."""
    x, w = x.float(), w.float()
    r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    dn = d * w
    dx = r * dn - x * (r * r * r) * (dn * x).mean(dim=1, keepdim=True)
    return dx, (d * x * r).sum(dim=0)


def _plain_merge_grad(st):
    g = _plain_gate(st)
    dxn, dw_next = _plain_rms_grad(st["d_h"].float(), st["out"], st["w_next"])
    d = st["d_out"].float() + dxn
    dy, dw = _plain_rms_grad(st["scale"] * g * d, st["y"], st["w"])
    res = [d.to(st["x"].dtype), dy.bfloat16(), dw, dw_next]
    if st["gate"] is not None:
        dg = st["scale"] * d * _plain_rms(st["y"], st["w"]) * (g * (1 - g))
        res.append((dg.sum(dim=1) if st["gate"].dim() == 1 else dg).bfloat16())
    return res


def _run_own(st):
    from sparse_moe_router_amd import ops
    case = st["case"]
    op = case["op"]
    if op == "grouped":
        return ops.grouped_matmul(st["x"], st["w"], st["offsets"], perm=st["perm"], top_k=st["top_k"],
                                  out_dtype=_DT[case["out"]])
    if op == "grouped_grad":
        dx = ops.grouped_matmul_grad_input(st["dy"], st["w"], st["offsets"])
        dw = ops.grouped_matmul_grad_weight(st["x"], st["dy"], st["offsets"], perm=st["perm"], top_k=st["top_k"],
                                            out_dtype=_DT[case["out"]])
        return dx, dw
    if op == "i8":
        return ops.matmul_i8(st["x"], st["w"], st["ws"], bias=st["bias"], out_dtype=_DT[case["out"]])
    if op == "i8_grouped":
        return ops.grouped_matmul_i8(st["x"], st["w"], st["ws"], st["offsets"], perm=st["perm"], top_k=st["top_k"],
                                     out_dtype=_DT[case["out"]])
    if op == "norm":
        return ops.block_norm(st["x"], st["w_next"], EPS)
    if op == "merge":
        return ops.block_merge(st["x"], st["y"], st["w"], EPS, gate=st["gate"], scale=st["scale"],
                               next_weight=st["w_next"])
    g = ops.block_merge_grad(st["d_out"], st["y"], st["w"], EPS, gate=st["gate"], scale=st["scale"],
                             next_weight=st["w_next"], out=st["out"], d_h=st["d_h"])
    res = [g["residual"], g["y"], g["weight"], g["next_weight"]]
    if st["gate"] is not None:
        res.append(g["gate"])
    return res


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "grouped":
        return _plain_grouped(state)
    if op == "grouped_grad":
        return _plain_grad(state)
    if op == "i8":
        return _plain_i8(state)
    if op == "i8_grouped":
        return _plain_i8_grouped(state)
    if op == "norm":
        return _plain_rms(state["x"], state["w_next"]).bfloat16()
    if op == "merge":
        return _plain_merge(state)
    return _plain_merge_grad(state)


# ------------------------------------------------------------------ work

def _touched(case):
    """Experts with a row, in expectation."""
    E, k, T = case["experts"], case["top_k"], case["tokens"]
    p = [(i + 1.0) ** -case["skew"] for i in range(E)]
    tot = sum(p)
    return sum(1.0 - (1.0 - min(1.0, k * v / tot)) ** T for v in p)


def work(case):
    op = case["op"]
    ob = 4 if case.get("out") == "fp32" else 2
    if op in ("grouped", "i8_grouped", "grouped_grad"):
        T, k, E, N, K = case["tokens"], case["top_k"], case["experts"], case["n"], case["k"]
        R = T * k
        xb = (T if case["gather"] else R) * K * 2
        wb = _touched(case) * N * K
        if op == "grouped":
            return {"bytes": int(xb + 2 * wb + R * N * ob), "flops": 2 * R * N * K}
        if op == "i8_grouped":
            return {"bytes": int(xb + wb + R * N * ob), "flops": 2 * R * N * K}
        return {"bytes": int(xb + R * N * 2 + 2 * wb + R * K * 2 + E * N * K * ob), "flops": 4 * R * N * K}
    if op == "i8":
        T, N, K = case["tokens"], case["n"], case["k"]
        return {"bytes": T * K * 2 + N * K + 4 * N + T * N * ob, "flops": 2 * T * N * K}
    T, H = case["tokens"], case["h"]
    sb = 4 if case["stream"] == "fp32" else 2
    if op == "norm":
        return {"bytes": T * H * (sb + 2) + 2 * H, "flops": 4 * T * H}
    gb = {"none": 0, "token": 2 * T, "element": 2 * T * H}[case["gate"]]
    if op == "merge":
        return {"bytes": T * H * (2 * sb + 4) + gb + 4 * H, "flops": 12 * T * H}
    return {"bytes": T * H * (3 * sb + 6) + 2 * gb + 12 * H, "flops": 30 * T * H}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rms(v, w):
    return v / torch.sqrt(torch.mean(v ** 2, -1, keepdim=True) + EPS) * w


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    op = case["op"]
    if op in ("grouped", "grouped_grad", "i8_grouped"):
        R = case["tokens"] * case["top_k"]
        token = torch.arange(R, device="cuda") if st["perm"] is None else torch.div(
            st["perm"].to(torch.int64), st["top_k"], rounding_mode="floor")
        xd = st["x"].to(f8)
        if op == "i8_grouped":
            xd, scale = _exact_codes(xd)
        groups = [(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(st["bounds"][:-1], st["bounds"][1:])) if hi > lo]
        if op == "grouped_grad":
            dx = torch.zeros(R, case["k"], dtype=f8, device="cuda")
            dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=f8, device="cuda")
            for e, sl in groups:
                d = st["dy"][sl].to(f8)
                torch.mm(d, st["w"][e].to(f8), out=dx[sl])
                torch.mm(d.t().contiguous(), xd.index_select(0, token[sl]), out=dw[e])
            return dx, dw
        y = torch.zeros(R, case["n"], dtype=f8, device="cuda")
        for e, sl in groups:
            torch.mm(xd.index_select(0, token[sl]), st["w"][e].to(f8).t().contiguous(), out=y[sl])
            if op == "i8_grouped":
                y[sl] *= scale[token[sl]].unsqueeze(1)
                y[sl] *= st["ws"][e].to(f8).unsqueeze(0)
        return y
    if op == "i8":
        codes, scale = _exact_codes(st["x"].to(f8))
        y = torch.mm(codes, st["w"].to(f8).t().contiguous()) * torch.outer(scale, st["ws"].to(f8))
        return y if st["bias"] is None else y + st["bias"].to(f8).unsqueeze(0)
    xd, wn = st["x"].to(f8), st["w_next"].to(f8)
    if op == "norm":
        return _exact_rms(xd, wn)
    yd, w, a = st["y"].to(f8), st["w"].to(f8), st["scale"]
    g = torch.ones(case["tokens"], 1, dtype=f8, device="cuda")
    if st["gate"] is not None:
        z = st["gate"].to(f8).reshape(case["tokens"], -1)
        g = 1.0 / (1.0 + torch.exp(-z))
    if op == "merge":
        out = xd + a * g * _exact_rms(yd, w)
        # the next norm is of the stream as it is stored
        return out, _exact_rms(out.to(st["x"].dtype).to(f8), wn)
    # the gradients by automatic differentiation of the definition in 64 bits
    with torch.enable_grad():
        out = st["out"].to(f8).requires_grad_()
        wn = wn.requires_grad_()
        (_exact_rms(out, wn) * st["d_h"].to(f8)).sum().backward()
        d = st["d_out"].to(f8) + out.grad
        yv, wv = yd.requires_grad_(), w.requires_grad_()
        gv = None if st["gate"] is None else st["gate"].to(f8).requires_grad_()
        gate = 1.0 if gv is None else torch.sigmoid(gv.reshape(case["tokens"], -1))
        (a * gate * _exact_rms(yv, wv) * d).sum().backward()
    return [d, yv.grad, wv.grad, wn.grad] + ([] if gv is None else [gv.grad])


def _exact_codes(xd):
    big = torch.linalg.vector_norm(xd, ord=float("inf"), dim=1)
    codes = torch.round(127.0 * xd / torch.where(big > 0, big, torch.ones_like(big)).unsqueeze(1))
    return codes, big / 127.0
