"""One transformer block trained with the NVFP4 recipe and the training
operators, on synthetic data:

    python examples/train_block.py [steps]

Layer norm -> quantised QKV projection -> causal attention over packed
documents -> quantised output projection -> residual and layer norm ->
quantised FFN -> squared error; the whole gradient; one AdamW step with 8-bit
states.  The maxima that the layer norms and AdamW leave are the quantiser's
(NVFP4_AMAX_GIVEN), so that those tensors are not read for them again.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_bit_quantization_amd as nv  # noqa: E402

SPEC = nv.QuantSpec.of
RHT_SEED = 1234


class Linear:
    """y = x w^T with 4-bit products: activations in 1D blocks, weights in 2D blocks, gradients rounded
    stochastically, the random Hadamard transform on the weight gradient's operands."""

    def __init__(self, n, k, gen):
        self.master = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
        self.weight = self.master.to(torch.bfloat16)
        self.amax = self.weight.float().abs().max().reshape(1)
        self.grad = torch.zeros(n, k, device="cuda")
        self.workspace, self.batch_workspace = nv.new_workspace(), nv.new_workspace(jobs=2)

    def tensor(self):
        return nv.adamw_tensor(self.master, self.grad, state_bits=8, weight_decay=0.01, copy=self.weight, amax=self.amax)

    def quantise_weight(self):
        """The weight and its transpose, with the maximum that the optimiser's step left."""
        n, k = self.weight.shape
        outs = [nv.empty_qtensor(n, k, nv.SCALE_2D16), nv.empty_qtensor(k, n, nv.SCALE_2D16)]
        for o in outs:
            o.amax = self.amax
        specs = [SPEC("2d", amax_given=True), SPEC("2d_t", amax_given=True)]
        self.w, self.wt = nv.nvfp4_quantize(self.weight, specs, outs, self.workspace)

    def forward(self, x, amax=None):
        self.x = x
        out = nv.empty_qtensor(*x.shape, nv.SCALE_1D16)
        if amax is not None:
            out.amax = amax
        q = nv.nvfp4_quantize(x, [SPEC("row", amax_given=amax is not None)], [out], self.workspace)[0]
        return nv.gemm(q, self.w, "bf16")

    def backward(self, dy, seed):
        q = nv.quantize(dy, [SPEC("row", "sr", sr_seed=seed)], self.workspace)[0]
        dx = nv.gemm(q, self.wt, "bf16")
        t, n, k = dy.shape[0], dy.shape[1], self.x.shape[1]
        qa, qb = [nv.empty_qtensor(n, t, nv.SCALE_1D16, rht=1)], [nv.empty_qtensor(k, t, nv.SCALE_1D16, rht=1)]
        nv.nvfp4_quantize_batch([(dy, [SPEC("col", "sr", True, seed + 1, RHT_SEED)], qa),
                                 (self.x, [SPEC("col", "rtn", True, 0, RHT_SEED)], qb)], self.batch_workspace)
        nv.nvfp4_gemm(qa[0], qb[0], self.grad)
        return dx


class Block:
    def __init__(self, hidden=256, heads=4, kv_heads=2, ffn=1024, lengths=(200, 56, 128, 128), seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, hidden // heads
        self.qkv = Linear((heads + 2 * kv_heads) * self.dim, hidden, gen)
        self.out, self.up, self.down = Linear(hidden, hidden, gen), Linear(ffn, hidden, gen), Linear(hidden, ffn, gen)
        self.linears = (self.qkv, self.out, self.up, self.down)
        # the norms' weights and biases, and their gradients, as rows of common buffers
        self.norms = torch.tensor([1.0, 0.0, 1.0, 0.0], device="cuda")[:, None].repeat(1, hidden)
        self.norm_grads = torch.zeros(4, hidden, device="cuda")
        ends = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
        self.packed = dict(causal=True, cu_q=cu, cu_k=cu, max_q=max(lengths), max_k=max(lengths))
        self.optimiser = nv.AdamWList([l.tensor() for l in self.linears] +
                                      [nv.adamw_tensor(w, g) for w, g in zip(self.norms, self.norm_grads)])
        self.amax = torch.zeros(2, device="cuda")

    def forward(self, x):
        for l in self.linears:
            l.quantise_weight()
        self.amax.zero_()
        self.x = x
        y, self.mean1, self.rstd1, _ = nv.layernorm(x, self.norms[0], self.norms[1], amax=self.amax[:1])
        qkv = self.qkv.forward(y, self.amax[:1]).view(x.shape[0], -1, self.dim)
        h, g = self.heads, self.kv_heads
        self.q, self.k, self.v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        self.o, self.lse = nv.attention(self.q, self.k, self.v, **self.packed)
        a = self.out.forward(self.o.flatten(1))
        y, self.mean2, self.rstd2, self.sum = nv.layernorm(a, self.norms[2], self.norms[3], residual=x, amax=self.amax[1:])
        self.u = self.up.forward(y, self.amax[1:])
        return self.sum + self.down.forward(torch.relu(self.u))

    def backward(self, dy, seed):
        du = self.down.backward(dy, seed) * (self.u > 0)
        d = self.up.backward(du, seed + 2)
        ds, self.norm_grads[2], self.norm_grads[3] = nv.layernorm_backward(d, self.sum, self.norms[2], self.mean2, self.rstd2,
                                                                           dsum=dy)
        do = self.out.backward(ds, seed + 4).view_as(self.o)
        # the gradients of q, k and v side by side, as the projection made them
        dqkv = torch.empty(dy.shape[0], self.heads + 2 * self.kv_heads, self.dim, dtype=torch.bfloat16, device="cuda")
        parts = dqkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        workspace = nv.new_attention_workspace(self.q, self.k, self.v, **self.packed)
        nv.nvfp4_attention_backward(do, self.q, self.k, self.v, self.o, self.lse, *parts, workspace, **self.packed)
        d = self.qkv.backward(dqkv.flatten(1), seed + 6)
        dx, self.norm_grads[0], self.norm_grads[1] = nv.layernorm_backward(d, self.x, self.norms[0], self.mean1, self.rstd1,
                                                                           dsum=ds)
        return dx

    def step(self, number, lr=2e-3):
        for l in self.linears:
            l.amax.zero_()
        nv.adamw(self.optimiser, lr=lr, beta1=0.9, beta2=0.95, step=number, rounding="sr", seed=77)


def train(steps=30, report=print):
    """The losses of `steps` steps towards a fixed mixing of the tokens."""
    block = Block()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(512, 256, generator=gen, device="cuda").to(torch.bfloat16)
    target = x.float() + 0.5 * torch.tanh(x.float() @ torch.randn(256, 256, generator=gen, device="cuda") / 16)
    losses = []
    for number in range(1, steps + 1):
        y = block.forward(x)
        error = y.float() - target
        block.backward((2 / error.numel() * error).to(torch.bfloat16), 1000 * number)
        block.step(number)
        losses.append(error.square().mean().item())
        if report and (number == 1 or number % 5 == 0):
            report("step %3d  loss %.4f" % (number, losses[-1]), flush=True)
    return losses


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
