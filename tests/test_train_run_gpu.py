"""The training operators together, as a training step uses them: routing, the experts' feed-forward block and its
combine, the loss against a vocabulary, all gradients and their clipping, against automatic differentiation in 64 bits;
and the call contract (graphs, streams, two calls at once)."""
import math

import pytest
import torch

import train_util as U
from ops_util import EPS16, EPS32, F8, close, eps_of, offsets_of, randn
from sparse_moe_router_amd import moe, ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def route(x, router, k, I):
    M, E = x.shape[0], router.shape[0]
    r = dict(topk_ids=torch.empty(M, k, dtype=torch.int32, device="cuda"),
             topk_w=torch.empty(M, k, dtype=F32, device="cuda"), offsets=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
             perm=torch.empty(M * k, dtype=torch.int32, device="cuda"))
    moe.route(x, router, k, r, flags=moe.FLAG_FORCE_GEMM, I=I)
    return r


def step(x, p, r, targets, k, max_norm):
    """One training step of x -> x + experts(x) -> loss: (loss, gradients by name, their norm)."""
    inv = ops.invert_permutation(r["perm"])
    kw = dict(perm=r["perm"], top_k=k)
    y, gate_up = ops.feed_forward(x, p["gu"], p["down"], r["offsets"], save=True, **kw)
    h = ops.combine(y, inv, k, weight=r["topk_w"], add=x)
    loss, lse = ops.cross_entropy(h, p["vocab"], targets)
    valid = ((targets >= 0) & (targets < p["vocab"].shape[0])).sum()
    g = ops.cross_entropy_grad(torch.ones_like(loss) / valid, h, p["vocab"], targets, lse)
    c = ops.combine_grad(g["x"], y, r["perm"], inv, r["topk_w"])
    f = ops.feed_forward_grad(c["y"], x, p["gu"], p["down"], gate_up, r["offsets"], dw_dtype=BF16, **kw)
    dx = ops.combine(f["x"], inv, k, add=g["x"])
    grads = dict(gu=f["w_gate_up"], down=f["w_down"], vocab=g["w"], x=dx, topk_w=c["weight"])
    before = {n: t.clone() for n, t in grads.items()}
    norm = ops.clip_grads(list(grads.values()), max_norm)
    return loss, before, norm, grads


def layer(M, H, E, k, I, V, seed=0):
    x = randn(seed, M, H).cuda()
    p = dict(gu=randn(seed + 2, E, 2 * I, H, scale=1 / H ** 0.5).cuda(), down=randn(seed + 3, E, H, I, scale=1 / I ** 0.5).cuda(),
             vocab=randn(seed + 4, V, H, scale=1 / H ** 0.5).cuda())
    r = route(x, randn(seed + 1, E, H, scale=0.05).cuda(), k, I)
    t = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(seed)).cuda()
    t[M // 2] = -100
    return x, p, r, t


@pytest.mark.parametrize("M,H,E,k,I,V", [(90, 128, 8, 2, 64, 500), (300, 256, 16, 4, 128, 1001)])
def test_training_step(M, H, E, k, I, V):
    x, p, r, t = layer(M, H, E, k, I, V)
    loss, g, norm, clipped = step(x, p, r, t, k, 0.01)
    v = {n: a.cpu().to(F8).requires_grad_() for n, a in dict(p, x=x, topk_w=r["topk_w"]).items()}
    pc, off = r["perm"].long().cpu(), r["offsets"].cpu()
    rows = []
    for e in range(E):
        z = v["x"][pc[off[e]:off[e + 1]] // k] @ v["gu"][e].t()
        rows.append((U.silu(z[:, :I]) * z[:, I:]) @ v["down"][e].t())
    y = torch.cat(rows) * v["topk_w"].reshape(-1)[pc][:, None]
    h = v["x"].index_add(0, pc // k, y)
    want = torch.nn.functional.cross_entropy(h @ v["vocab"].t(), t.cpu(), reduction="none", ignore_index=-100)
    (want.sum() / (M - 1)).backward()
    # h is rounded to bf16 three times on its way (act, rows, sum), each by at most 2^-8 of it: so is a logit, in
    # which 3 * 2^-8 of the magnitudes of its terms can add up
    mag = h.detach().abs() @ v["vocab"].detach().abs().t()
    assert ((loss.cpu().to(F8) - want.detach()).abs() <= 2 * 3 * EPS16 * mag.max(1).values).all()
    # at most ten roundings to bf16 follow each other on the way to a gradient: 10 * 2^-8 of its own size in its norm
    for n, a in g.items():
        rel = (a.cpu().to(F8) - v[n].grad).norm() / v[n].grad.norm()
        assert rel <= 10 * EPS16, (n, float(rel))
    exact = math.sqrt(sum(float((a.to(F8) ** 2).sum()) for a in g.values()))
    assert abs(norm.item() - exact) <= 1.01 * EPS32 * exact and exact > 0.02
    for n, a in clipped.items():
        s = g[n].cpu().to(F8) * (0.01 / (exact + 1e-6))
        close(a, s, (3.01 * EPS32 + eps_of(a.dtype)) * s.abs(), n)


def test_step_repeats_bit_for_bit():
    x, p, r, t = layer(500, 256, 16, 4, 128, 3001)
    a, b = (step(x, p, r, t, 4, 0.1) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    assert all(torch.equal(a[3][n], b[3][n]) for n in a[3])


def test_combined_experts_are_the_fused_layer():
    x, p, r, _ = layer(300, 256, 16, 4, 128, 8)
    y = ops.feed_forward(x, p["gu"], p["down"], r["offsets"], perm=r["perm"], top_k=4)
    out = ops.combine(y, ops.invert_permutation(r["perm"]), 4, weight=r["topk_w"])
    router = randn(1, 16, 256, scale=0.05).cuda()
    packed = torch.cat([p["gu"].reshape(16, -1), p["down"].reshape(16, -1)], 1).contiguous()
    fused = moe.forward(x, router, packed, None, 4, flags=moe.FLAG_FORCE_GEMM)
    # both round act, each expert's row and the result to bf16
    scale = fused.float().abs().amax(dim=1, keepdim=True)
    assert ((out.float() - fused.float()).abs() <= 8 * EPS16 * scale).all()


# ------------------------------------------------------------------ the call contract

def every_call(p):
    """Every training operator once on the tensors of p; returns all results in a list."""
    kw = dict(perm=p["perm"], top_k=2)
    h, gu = ops.gated_matmul(p["x"], p["gu"], p["off"], save=True, **kw)
    a = ops.gated_matmul_grad(p["dy"], p["down"], gu, p["off"])
    f = ops.feed_forward_grad(p["dy"], p["x"], p["gu"], p["down"], gu, p["off"], **kw)
    inv = ops.invert_permutation(p["perm"])
    out = ops.combine(p["dy"], inv, 2, weight=p["weight"], add=p["x"])
    c = ops.combine_grad(out, p["dy"], p["perm"], inv, p["weight"])
    loss, lse = ops.cross_entropy(out, p["vocab"], p["targets"])
    g = ops.cross_entropy_grad(p["d_loss"], out, p["vocab"], p["targets"], lse)
    grads = [f["w_gate_up"], f["w_down"], g["w"]]
    n = ops.grad_norm(grads)
    into = [torch.empty_like(t) for t in grads]
    m = ops.clip_grads(grads, 0.5, out=into)
    return [h, gu, a["gate_up"], a["h"], f["x"], *grads, inv, out, c["y"], c["weight"], loss, lse, g["x"], n, m, *into]


def call_inputs(few, seed=0):
    M, K, I, E, V = (4, 144, 40, 8, 300) if few else (700, 264, 136, 5, 1100)
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:2] for _ in range(M)]).reshape(-1)
    return {n: t.cuda() for n, t in dict(
        x=randn(seed, M, K), gu=randn(seed + 1, E, 2 * I, K, scale=0.1), down=randn(seed + 2, E, K, I, scale=0.1),
        dy=randn(seed + 3, 2 * M, K), off=offsets_of(torch.bincount(ids, minlength=E).tolist()),
        perm=torch.sort(ids, stable=True).indices.to(torch.int32), weight=torch.rand(M, 2, generator=g),
        vocab=randn(seed + 4, V, K, scale=0.1), targets=torch.randint(-1, V, (M,), generator=g),
        d_loss=torch.rand(M, generator=g)).items()}


@pytest.mark.parametrize("few", [True, False])
def test_graph_replays(few):
    """A captured run of every operator, replayed on new inputs with eager work between."""
    p = call_inputs(few)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        every_call(p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = every_call(p)
    for seed in (0, 50, 60, 0):
        for n, t in call_inputs(few, seed).items():
            p[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        want = every_call(p)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_replayed_at_once():
    """Two captured runs, each with its own inputs, replayed together on two streams."""
    ps = [call_inputs(False, s) for s in (0, 70)]
    want = [every_call(p) for p in ps]
    torch.cuda.synchronize()
    graphs, res = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(every_call(p))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r, w in zip(res, want):
            assert all(torch.equal(a, b) for a, b in zip(r, w))


def test_other_streams():
    """Calls on a stream given as an argument and on the current one, two at once."""
    ps = [call_inputs(False, s) for s in (0, 70)]
    want = [every_call(p) for p in ps]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = every_call(ps[0])
        with torch.cuda.stream(s2):
            b = every_call(ps[1])
        p = ps[0]
        c = ops.cross_entropy(want[0][9], p["vocab"], p["targets"], stream=s2)
        d = ops.clip_grads(want[0][5:8], 0.5, out=[torch.empty_like(t) for t in want[0][5:8]], stream=s2)
        y = ops.feed_forward(p["x"], p["gu"], p["down"], p["off"], perm=p["perm"], top_k=2, stream=s1)
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(a, want[0]))
        assert all(torch.equal(i, j) for i, j in zip(b, want[1]))
        assert torch.equal(c[0], want[0][12]) and torch.equal(c[1], want[0][13]) and torch.equal(d, want[0][16])
        assert torch.equal(y, ops.grouped_matmul(want[0][0], p["down"], p["off"]))


def test_given_workspaces():
    """A workspace of the needed size, filled with other bytes, changes nothing; a smaller one is refused."""
    p = call_inputs(False)
    lib = ops.lib()
    x, w, t = p["x"], p["vocab"], p["targets"]
    d = ops.MoeLoss(x.shape[0], x.shape[1], w.shape[0], x.shape[1], -100)
    f = ops.MoeFeedForward(p["dy"].shape[0], x.shape[0], x.shape[1], x.shape[1], 5, 136, x.shape[1], x.shape[1], 2,
                           p["off"].data_ptr(), p["perm"].data_ptr())
    h, gu = ops.gated_matmul(x, p["gu"], p["off"], save=True, perm=p["perm"], top_k=2)
    lse = ops.cross_entropy(x, w, t)[1]
    tensors = (ops.MoeTensor * 2)(*(ops.MoeTensor(v.data_ptr(), None, v.numel(), 0, 0) for v in (w, x)))
    calls = [(lib.moe_cross_entropy_workspace_size(d), lambda **k: ops.cross_entropy(x, w, t, **k)),
             (lib.moe_cross_entropy_grad_workspace_size(d),
              lambda **k: ops.cross_entropy_grad(p["d_loss"], x, w, t, lse, **k).values()),
             (lib.moe_feed_forward_grad_workspace_size(f),
              lambda **k: ops.feed_forward_grad(p["dy"], x, p["gu"], p["down"], gu, p["off"], perm=p["perm"], top_k=2,
                                                **k).values()),
             (lib.moe_grad_norm_workspace_size(tensors, 2), lambda **k: [ops.grad_norm([w, x], **k)])]
    for need, call in calls:
        assert need > 0
        want = list(call())
        for fill in (0, 255, 127):
            wk = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            assert all(torch.equal(a, b) for a, b in zip(call(workspace=wk), want))
        with pytest.raises(ops.MoeError, match="WORKSPACE"):
            call(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ tiles that follow each other

@pytest.mark.parametrize("R", [2305, 2504])
@pytest.mark.parametrize("K", [72, 200])
def test_one_group_of_many_tiles(R, K):
    """More tiles of one group than the chip runs at a time, the last ones short, in every product."""
    N = 8200
    x, w, dy = randn(1, R, K).cuda(), randn(2, 1, N, K).cuda(), randn(3, R, N).cuda()
    off = offsets_of([R])
    d = lambda t: t.to(F8)
    for out in (BF16, F32):
        y, t = d(x) @ d(w[0]).t(), 2 * EPS32 * K * (d(x).abs() @ d(w[0]).abs().t())
        close(ops.grouped_matmul(x, w, None, out_dtype=out), y.cpu(), (t + eps_of(out) * y.abs()).cpu())
        wide = torch.full((R, N + 8), 3.0, dtype=out, device="cuda")
        ops.grouped_matmul(x, w, None, out=wide[:, :N])
        assert torch.equal(wide[:, :N], ops.grouped_matmul(x, w, None, out_dtype=out)) and (wide[:, N:] == 3).all()
        # rows' gradient with many columns: the roles of N and K change
        w2 = w.transpose(1, 2).contiguous()
        close(ops.grouped_matmul_grad_input(x, w2, None, out_dtype=out), y.cpu(), (t + eps_of(out) * y.abs()).cpu())
    wide = randn(4, R, 4104).cuda()
    for out in (BF16, F32):
        v, t = d(dy[:, :4360]).t() @ d(wide), 2 * EPS32 * R * (d(dy[:, :4360]).abs().t() @ d(wide).abs())
        got = ops.grouped_matmul_grad_weight(wide, dy[:, :4360], None, out_dtype=out)
        close(got[0], v.cpu(), (t + eps_of(out) * v.abs()).cpu())


@pytest.mark.parametrize("T", [2305, 2504])
def test_loss_of_many_tiles(T):
    V, H = 8199, 24
    x, w = randn(1, T, H).cuda(), randn(2, V, H, scale=0.4).cuda()
    t = torch.randint(-1, V, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    dl = torch.rand(T, generator=torch.Generator().manual_seed(4)).cuda()
    loss, lse = ops.cross_entropy(x, w, t)
    ref = U.loss_ref(x, w, t)
    close(loss, ref[0].cpu(), ref[1].cpu())
    close(lse, ref[2].cpu(), ref[3].cpu())
    (dx, tx), (dw, tw) = ((v.cpu() for v in p) for p in U.loss_grad_ref(dl, x, w, t))
    g = ops.cross_entropy_grad(dl, x, w, t, lse, dx_dtype=F32, dw_dtype=F32)
    close(g["x"], dx, tx + EPS32 * dx.abs())
    close(g["w"], dw, tw + EPS32 * dw.abs())
