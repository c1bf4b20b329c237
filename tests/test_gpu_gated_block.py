"""The block operators together with the 4-bit products and the training
operators: the example's gated block against the same block in binary32 by
automatic differentiation, and its steps."""
import math
import os
import sys

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_gated_block
    return train_gated_block


def _norm(x, w, b):
    m = x.mean(1, keepdim=True)
    return (x - m) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + 1e-5) * w + b


def _rope(x, w, at, freqs):
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    t = (at.double()[:, None] * freqs).float()[:, None, :]
    n = freqs.numel()
    a, b = x[..., :n], x[..., n:]
    return torch.cat([a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()], -1)


def _reference(block, x, params):
    qkv, out, both, down, w1, b1, w2, b2, wq, wk = params
    t = (_norm(x, w1, b1) @ qkv.t()).view(x.shape[0], -1, block.dim)
    h, g = block.heads, block.kv_heads
    ends = block.cu.tolist()
    at = torch.cat([torch.arange(b - a, device="cuda") for a, b in zip(ends, ends[1:])])
    q = _rope(t[:, :h], wq, at, block.freqs)
    k = _rope(t[:, h:h + g], wk, at, block.freqs).repeat_interleave(h // g, 1)
    v = t[:, h + g:].repeat_interleave(h // g, 1)
    rows = []
    for a, b in zip(ends, ends[1:]):
        s = torch.matmul(q[a:b].transpose(0, 1), k[a:b].transpose(0, 1).transpose(1, 2).contiguous()) / math.sqrt(block.dim)
        s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        rows.append(torch.matmul(torch.softmax(s, 2), v[a:b].transpose(0, 1)).transpose(0, 1))
    s = x + torch.cat(rows).reshape(x.shape) @ out.t()
    gate, up = (_norm(s, w2, b2) @ both.t()).chunk(2, 1)
    return s + (torch.nn.functional.silu(gate) * up) @ down.t()


def _cosine(a, b):
    a, b = a.double().flatten(), b.double().flatten()
    return (a @ b / (a.norm() * b.norm())).item()


def test_block_gradients(example):
    """Each gradient points where the binary32 one does.  An E2M1 element under its block's scale is off by about a
    tenth of its value (rms, RTN; more where rounded stochastically): two operands of a product and a chain of up to
    six products keep the angle's cosine above 0.9, those of the head norms' weights, at the end of the longest chain
    and sums of terms that cancel, above 0.8."""
    say("gated block gradients")
    block = example.GatedBlock()
    gen = torch.Generator(device="cuda").manual_seed(3)
    block.head_norms.copy_(1 + 0.2 * torch.randn(2, block.dim, generator=gen, device="cuda"))
    x = torch.randn(512, 256, generator=gen, device="cuda").to(torch.bfloat16)
    dy = (1e-3 * torch.randn(512, 256, generator=gen, device="cuda")).to(torch.bfloat16)
    y = block.forward(x)
    dx = block.backward(dy, 5)
    params = [l.weight.float().requires_grad_() for l in block.linears] + [
        n.clone().requires_grad_() for n in (*block.norms, *block.head_norms)]
    xf = x.float().requires_grad_()
    want = _reference(block, xf, params)
    grads = torch.autograd.grad(want, [xf] + params, dy.float())
    assert _cosine(y - x, want - xf) > 0.9
    got = [dx] + [l.grad for l in block.linears] + list(block.norm_grads) + list(block.head_grads)
    for name, a, b in zip(("x", "qkv", "out", "both", "down", "w1", "b1", "w2", "b2", "wq", "wk"), got, grads):
        c = _cosine(a, b)
        assert c > (0.8 if name in ("wq", "wk") else 0.9), "%s: cosine %.3f" % (name, c)


def test_block_steps(example):
    """It runs, moves every parameter by about what the learning rate says, and leaves the quantiser's maxima right."""
    say("gated block steps")
    block = example.GatedBlock()
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(512, 256, generator=gen, device="cuda").to(torch.bfloat16)
    old = [l.master.clone() for l in block.linears]
    for number in (1, 2):
        y = block.forward(x)
        assert block.amax[2].item() == block.h.abs().max().item()
        block.backward((1e-3 * (y - x)).to(torch.bfloat16), 10 * number)
        block.step(number, lr=1e-3)
    for l, o in zip(block.linears, old):
        assert torch.equal(l.weight, l.master.to(torch.bfloat16)) and l.amax.item() == l.weight.abs().max().item()
        moved = (l.master - o * (1 - 1e-5) ** 2).square().mean().sqrt().item()
        # two steps of 0.2 lr sqrt(max(n, k)) X, where X has min(n, k) singular values of 0.7 to 1.2 at most
        n, k = sorted(l.master.shape)
        one = 0.2 * 1e-3 * math.sqrt(k) * math.sqrt(n / (n * k))
        assert 0.2 * one < moved < 2.4 * one
    assert all(torch.isfinite(t).all() for t in (block.norms, block.head_norms))
    losses = example.train(3, report=None)
    assert all(math.isfinite(v) for v in losses)
