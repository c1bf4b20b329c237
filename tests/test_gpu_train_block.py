"""The training operators together with the 4-bit products: the example's
transformer block against the same block in binary32 by automatic
differentiation, and its training."""
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
    import train_block
    return train_block


def _norm(x, w, b):
    m = x.mean(1, keepdim=True)
    return (x - m) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + 1e-5) * w + b


def _reference(block, x, params):
    qkv, out, up, down, w1, b1, w2, b2 = params
    t = _norm(x, w1, b1) @ qkv.t()
    t = t.view(x.shape[0], -1, block.dim)
    h, g = block.heads, block.kv_heads
    q, k, v = t[:, :h], t[:, h:h + g].repeat_interleave(h // g, 1), t[:, h + g:].repeat_interleave(h // g, 1)
    o = torch.zeros_like(q)
    ends = block.packed["cu_q"].tolist()
    rows = []
    for a, b in zip(ends, ends[1:]):
        s = torch.matmul(q[a:b].transpose(0, 1), k[a:b].transpose(0, 1).transpose(1, 2).contiguous()) / math.sqrt(block.dim)
        s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        rows.append(torch.matmul(torch.softmax(s, 2), v[a:b].transpose(0, 1)).transpose(0, 1))
    o = torch.cat(rows).reshape(x.shape)
    s = x + o @ out.t()
    return s + torch.relu(_norm(s, w2, b2) @ up.t()) @ down.t()


def _cosine(a, b):
    a, b = a.double().flatten(), b.double().flatten()
    return (a @ b / (a.norm() * b.norm())).item()


def test_block_gradients(example):
    """Each gradient points where the binary32 one does.  An E2M1 element under its block's scale is off by about a
    tenth of its value (rms, RTN; more where rounded stochastically): two operands of a product and a chain of up to
    six products keep the angle's cosine above 0.9."""
    say("train block gradients")
    block = example.Block()
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(512, 256, generator=gen, device="cuda").to(torch.bfloat16)
    dy = (1e-3 * torch.randn(512, 256, generator=gen, device="cuda")).to(torch.bfloat16)
    y = block.forward(x)
    dx = block.backward(dy, 5)
    params = [l.weight.float().requires_grad_() for l in block.linears] + [n.clone().requires_grad_() for n in block.norms]
    xf = x.float().requires_grad_()
    want = _reference(block, xf, params)
    grads = torch.autograd.grad(want, [xf] + params, dy.float())
    assert _cosine(y - x, want - xf) > 0.9
    got = [dx] + [l.grad for l in block.linears] + list(block.norm_grads)
    for name, a, b in zip(("x", "qkv", "out", "up", "down", "w1", "b1", "w2", "b2"), got, grads):
        c = _cosine(a, b)
        assert c > 0.9, "%s: cosine %.3f" % (name, c)


def test_block_trains(example):
    say("train block")
    losses = example.train(20, report=None)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.6 * losses[0], losses
