"""The operators together, as a model uses them: a sandwich-normed MoE block built from routing, grouped
products and norms against the fused layer and against 64 bits; its backward; 8-bit experts; and the call
contract (graphs, streams, two calls at once)."""
import pytest
import torch

from ops_util import EPS32, F8, close, eps_of, merge_ref, randn, rms
from sparse_moe_router_amd import moe, ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def layer(M=300, H=256, E=16, k=4, I=128, seed=0):
    return dict(M=M, H=H, E=E, k=k, I=I, x=randn(seed, M, H).cuda(), router=randn(seed + 1, E, H, scale=0.05).cuda(),
                gu=randn(seed + 2, E, 2 * I, H, scale=0.05).cuda(), down=randn(seed + 3, E, H, I, scale=0.05).cuda(),
                w_in=(randn(seed + 4, H, scale=0.1) + 1).cuda(), w_out=(randn(seed + 5, H, scale=0.1) + 1).cuda(),
                w_next=(randn(seed + 6, H, scale=0.1) + 1).cuda(), gate=randn(seed + 7, M).cuda())


def route(p, h):
    M, E, k = p["M"], p["E"], p["k"]
    r = dict(topk_ids=torch.empty(M, k, dtype=torch.int32, device="cuda"),
             topk_w=torch.empty(M, k, dtype=F32, device="cuda"), offsets=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
             perm=torch.empty(M * k, dtype=torch.int32, device="cuda"))
    moe.route(h, p["router"], k, r, flags=moe.FLAG_FORCE_GEMM, I=p["I"])
    return r


def experts(p, h, r, gu=ops.grouped_matmul, down=ops.grouped_matmul):
    """The routed experts on the grouped order and their weighted sum per token."""
    I, k = p["I"], p["k"]
    a = gu(h, p["gu"], r["offsets"], perm=r["perm"], top_k=k, out_dtype=F32)
    act = (torch.nn.functional.silu(a[:, :I]) * a[:, I:]).to(BF16)
    y = down(act, p["down"], r["offsets"])
    slots = torch.empty(p["M"] * k, p["H"], device="cuda")
    slots[r["perm"].long()] = y.float()
    return a, act, y, (slots.view(p["M"], k, -1) * r["topk_w"][:, :, None]).sum(1).to(BF16)


def test_block_from_operators_is_the_fused_layer():
    p = layer()
    h = ops.block_norm(p["x"], p["w_in"], EPS)
    r = route(p, h)
    _, _, _, y = experts(p, h, r)
    packed = torch.cat([p["gu"].reshape(p["E"], -1), p["down"].reshape(p["E"], -1)], 1).contiguous()
    fused = moe.forward(h, p["router"], packed, None, p["k"], flags=moe.FLAG_FORCE_GEMM)
    # the two differ by roundings to bf16: of act and of each expert's row in both, and of the result
    scale = fused.float().abs().amax(dim=1, keepdim=True)
    assert ((y.float() - fused.float()).abs() <= 8 * 2.0 ** -8 * scale).all()
    out, hn = ops.block_merge(p["x"], y, p["w_out"], EPS, gate=p["gate"], scale=0.5, next_weight=p["w_next"])
    d = lambda t: t.cpu().to(F8)
    want = merge_ref(d(p["x"]), d(y), d(p["w_out"]), EPS, d(p["gate"]), 0.5)
    close(out, want, 100 * EPS32 * want.abs().amax() + eps_of(BF16) * want.abs())
    wh = rms(d(out), d(p["w_next"]), EPS)
    close(hn, wh, (100 * EPS32 + eps_of(BF16)) * wh.abs())


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_block_forward(M):
    """block_forward is its three parts, for every path of the layer, on the current and on a given
    stream, and blocks chained through the next norm."""
    p = layer(M=M)
    I, E = p["I"], p["E"]
    packed = torch.cat([p["gu"].reshape(E, -1), p["down"].reshape(E, -1)], 1).contiguous()
    shared = packed[0].clone()
    args = (p["router"], packed, shared, p["k"])
    out, hn = ops.block_forward(p["x"], *args, p["w_in"], p["w_out"], EPS, gate=p["gate"], scale=0.5,
                                next_weight=p["w_next"])
    h = ops.block_norm(p["x"], p["w_in"], EPS)
    want = ops.block_merge(p["x"], moe.forward(h, *args), p["w_out"], EPS, gate=p["gate"], scale=0.5,
                           next_weight=p["w_next"])
    assert torch.equal(out, want[0]) and torch.equal(hn, want[1])
    second = ops.block_forward(out, *args, None, p["w_out"], EPS, h=hn)
    assert torch.equal(second, ops.block_merge(out, moe.forward(hn, *args), p["w_out"], EPS))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = ops.block_forward(p["x"], *args, p["w_in"], p["w_out"], EPS, gate=p["gate"], scale=0.5, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    with pytest.raises(ValueError, match="norm_weight or h"):
        ops.block_forward(p["x"], *args, p["w_in"], p["w_out"], EPS, h=h)


def test_backward_of_the_block():
    """The gradients of a whole block through the operators' backward calls, against automatic
    differentiation of the block in 64 bits at the same routing."""
    p = layer(M=90, H=128, I=64, E=8, k=2)
    I, k, M = p["I"], p["k"], p["M"]
    h = ops.block_norm(p["x"], p["w_in"], EPS)
    r = route(p, h)
    a, act, y_rows, y = experts(p, h, r)
    out, hn = ops.block_merge(p["x"], y, p["w_out"], EPS, gate=p["gate"], scale=0.5, next_weight=p["w_next"])
    d_out, d_h = randn(20, M, p["H"]).cuda(), randn(21, M, p["H"]).cuda()
    g = ops.block_merge_grad(d_out, y, p["w_out"], EPS, gate=p["gate"], scale=0.5, next_weight=p["w_next"], out=out,
                             d_h=d_h)
    perm = r["perm"].long()
    wrow = r["topk_w"].reshape(-1)[perm][:, None]
    d_rows = (g["y"].float()[perm // k] * wrow).to(BF16)
    d_act = ops.grouped_matmul_grad_input(d_rows, p["down"], r["offsets"], out_dtype=F32)
    d_down = ops.grouped_matmul_grad_weight(act, d_rows, r["offsets"])
    s = torch.sigmoid(a[:, :I])
    d_a = torch.cat([d_act * a[:, I:] * s * (1 + a[:, :I] * (1 - s)), d_act * a[:, :I] * s], 1).to(BF16)
    d_copy = ops.grouped_matmul_grad_input(d_a, p["gu"], r["offsets"], out_dtype=F32)
    d_gu = ops.grouped_matmul_grad_weight(h, d_a, r["offsets"], perm=r["perm"], top_k=k)
    d_hin = torch.zeros(M, p["H"], device="cuda").index_add_(0, perm // k, d_copy).to(BF16)
    gn = ops.block_norm_grad(d_hin, p["x"], p["w_in"], EPS, d_add=g["residual"])

    v = {n: p[n].cpu().to(F8).requires_grad_() for n in ("x", "gu", "down", "w_in", "w_out", "w_next", "gate")}
    pc, off = perm.cpu(), r["offsets"].cpu()
    hh = rms(v["x"], v["w_in"], EPS)
    rows = []
    for e in range(p["E"]):
        t = pc[off[e]:off[e + 1]] // k
        z = hh[t] @ v["gu"][e].t()
        rows.append((torch.nn.functional.silu(z[:, :I]) * z[:, I:]) @ v["down"][e].t())
    yy = torch.zeros(M, p["H"], dtype=F8).index_add(0, pc // k, torch.cat(rows) * wrow.cpu().to(F8))
    oo = merge_ref(v["x"], yy, v["w_out"], EPS, v["gate"], 0.5)
    ((oo * d_out.cpu().to(F8)).sum() + (rms(oo, v["w_next"], EPS) * d_h.cpu().to(F8)).sum()).backward()
    # each stage rounds its rows to bf16, at most eight stages deep: an error of 8 * 2^-8 of a
    # tensor's own size in its norm
    for name, got in (("x", gn["x"]), ("w_in", gn["weight"]), ("gu", d_gu), ("down", d_down), ("w_out", g["weight"]),
                      ("w_next", g["next_weight"]), ("gate", g["gate"])):
        want = v[name].grad
        rel = (got.cpu().to(F8) - want).norm() / want.norm()
        assert rel <= 8 * 2.0 ** -8, (name, float(rel))


def quantized(w):
    s = w.float().abs().amax(dim=-1) / 127
    return torch.round(w.float() / s[..., None]).to(torch.int8), s


def test_eight_bit_experts():
    """Experts on 8-bit weights: within the error of the codes of the bf16 experts'."""
    p = layer()
    h = ops.block_norm(p["x"], p["w_in"], EPS)
    r = route(p, h)
    y = experts(p, h, r)[3].float()
    i8 = lambda x, w, off, **kw: ops.grouped_matmul_i8(x, *quantized(w), off, **kw)
    y8 = experts(p, h, r, gu=i8, down=i8)[3].float()
    # codes are off by at most half a step of 1/127 of the largest value: about 3 sigma / 254 a factor,
    # 1.2%, on both factors of two products, one of them under a gated activation (three factors)
    rel = (y8 - y).norm() / y.norm()
    assert 0 < rel < 5 * 1.2e-2


def every_call(p, few):
    """Every operator once on the tensors of p; returns all results in a list."""
    a = ops.grouped_matmul(p["x"], p["w"], p["off"], perm=p["perm"], top_k=2)
    b = ops.grouped_matmul_grad_input(p["dy"], p["w"], p["off"])
    c = ops.grouped_matmul_grad_weight(p["x"], p["dy"], p["off"], perm=p["perm"], top_k=2)
    d = ops.grouped_matmul_i8(p["x"], p["wq"], p["ws"], p["off"], perm=p["perm"], top_k=2)
    q = ops.quantize_i8(p["x"])
    e = ops.matmul_i8(p["x"], p["wq"][0], p["ws"][0])
    n = ops.block_norm(p["x"], p["nw"], EPS)
    o, h = ops.block_merge(p["x"], n, p["nw"], EPS, gate=p["gate"], next_weight=p["nw"])
    g = ops.block_merge_grad(p["x"], n, p["nw"], EPS, gate=p["gate"], next_weight=p["nw"], out=o, d_h=h)
    m = ops.block_norm_grad(h, p["x"], p["nw"], EPS)
    return [a, b, c, d, *q, e, n, o, h, *(g[k] for k in sorted(g)), m["x"], m["weight"]]


def call_inputs(few, seed=0):
    M, K, N, E = (4, 144, 80, 8) if few else (400, 272, 264, 5)
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:2] for _ in range(M)]).reshape(-1)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    return {n: t.cuda() for n, t in dict(
        x=randn(seed, M, K), w=randn(seed + 1, E, N, K), dy=randn(seed + 2, 2 * M, N), off=off,
        perm=torch.sort(ids, stable=True).indices.to(torch.int32), gate=randn(seed + 3, M, K), nw=randn(seed + 4, K),
        wq=torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8),
        ws=torch.rand(E, N, generator=g)).items()}


@pytest.mark.parametrize("few", [True, False])
def test_graph_replays(few):
    """A captured run of every operator, replayed on new inputs with eager work between."""
    p = call_inputs(few)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        every_call(p, few)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = every_call(p, few)
    for seed in (0, 50, 60, 0):
        for n, t in call_inputs(few, seed).items():
            p[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        want = every_call(p, few)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_replayed_at_once():
    """Two captured runs, each with its own inputs, replayed together on two streams."""
    ps = [call_inputs(False, s) for s in (0, 70)]
    want = [every_call(p, False) for p in ps]
    torch.cuda.synchronize()
    graphs, res = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(every_call(p, False))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r, w in zip(res, want):
            assert all(torch.equal(a, b) for a, b in zip(r, w))


def test_two_block_graphs_replayed_at_once():
    """Two captured blocks (the layer's workspace among their buffers) replayed together."""
    ps = [layer(M=200, seed=s) for s in (0, 40)]
    packed = [torch.cat([p["gu"].reshape(p["E"], -1), p["down"].reshape(p["E"], -1)], 1).contiguous() for p in ps]

    def block(i):
        p = ps[i]
        return ops.block_forward(p["x"], p["router"], packed[i], None, p["k"], p["w_in"], p["w_out"], EPS,
                                 gate=p["gate"], next_weight=p["w_next"])

    want = [block(0), block(1)]
    torch.cuda.synchronize()
    graphs, res = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(block(i))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r, w in zip(res, want):
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])


def test_other_streams():
    """Calls on a stream given as an argument and on the current one, two at once."""
    ps = [call_inputs(False, s) for s in (0, 70)]
    want = [every_call(p, False) for p in ps]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = every_call(ps[0], False)
        with torch.cuda.stream(s2):
            b = every_call(ps[1], False)
        c = ops.grouped_matmul_i8(ps[0]["x"], ps[0]["wq"], ps[0]["ws"], ps[0]["off"], perm=ps[0]["perm"], top_k=2,
                                  stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(a, want[0]))
        assert all(torch.equal(i, j) for i, j in zip(b, want[1]))
        assert torch.equal(c, want[0][3])
