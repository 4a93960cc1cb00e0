"""block_forward's handling of its arguments: which of its three parts each one reaches."""
import types

import pytest
import torch

from ops_util import randn
from sparse_moe_router_amd import moe, ops

BF16 = torch.bfloat16
EPS = 1e-6


def block(device, M=6, H=128, E=8, I=64):
    g = torch.Generator().manual_seed(1)
    w = lambda *s: (torch.randn(*s, generator=g) * 0.05).to(BF16).to(device)
    return dict(x=randn(2, M, H).to(device), router_w=w(E, H), expert_w=w(E, 3 * I * H), shared_w=None, top_k=2,
                norm_weight=1 + w(H), merge_weight=1 + w(H), eps=EPS)


@pytest.fixture
def parts(monkeypatch):
    """The three parts replaced by ones that record their keywords (no GPU)."""
    seen = {}

    def part(name):
        def f(x, *a, **kw):
            seen[name] = kw
            return x
        return f

    for mod, name in ((ops, "block_norm"), (moe, "forward"), (ops, "block_merge")):
        monkeypatch.setattr(mod, name, part(name))
    return seen


def test_out_is_the_blocks_result(parts):
    b = block("cpu")
    out = torch.empty_like(b["x"])
    ops.block_forward(**b, out=out)
    assert parts["block_merge"]["out"] is out and "out" not in parts["forward"]


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [BF16, torch.float32])
def test_out_holds_the_result(stream):
    b = block("cuda")
    b["x"] = b["x"].to(stream)
    want = ops.block_forward(**b)
    out = torch.full_like(b["x"], 7.0)
    got = ops.block_forward(**b, out=out)
    assert got is out and torch.equal(out, want)


@pytest.mark.parametrize("given", [{}, {"workspace": None}])
def test_workspace_is_the_calls_own(parts, given):
    """Not the layer's cached one, which captured graphs would share; a caller's is handed on."""
    b = block("cpu")
    seen = []
    for _ in range(2):
        ops.block_forward(**b, **given)
        seen.append(parts["forward"]["workspace"])
    need = moe.workspace_size(6, 128, 8, 64, 0, 2)
    assert all(w is not None and w.numel() >= need for w in seen) and seen[0] is not seen[1]
    mine = torch.empty(need, dtype=torch.uint8)
    ops.block_forward(**b, workspace=mine)
    assert parts["forward"]["workspace"] is mine


def test_no_rows_skip_the_layer(parts):
    ops.block_forward(**block("cpu", M=0))
    assert "forward" not in parts and "block_merge" in parts


@pytest.mark.gpu
def test_no_rows():
    b = block("cuda", M=0)
    out, h = ops.block_forward(**b, next_weight=b["norm_weight"])
    assert out.shape == h.shape == (0, 128)


@pytest.mark.gpu
def test_a_stream_of_another_device_is_refused():
    """(Its parts would otherwise run on the tensors' own device's current stream and on the other's.)"""
    b = block("cuda")
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ops.block_forward(**b, stream=other)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ops.block_norm(b["x"], b["norm_weight"], EPS, stream=other)
