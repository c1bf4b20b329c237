"""One transformer block of the present kind trained with the NVFP4 recipe and the
block operators, on synthetic data:

    python examples/train_gated_block.py [steps]

Layer norm -> quantised QKV projection -> norm and rotation of the query and key
heads -> causal attention over packed documents -> quantised output projection ->
residual and layer norm -> gated feed-forward block on 4-bit operands -> squared
error; the whole gradient; one step of the matrices by their orthogonalised
momentum, of the vectors by AdamW.  The maxima that norms, gated products and
steps leave are the quantiser's (NVFP4_AMAX_GIVEN), so that those tensors are not
read for them again.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_bit_quantization_amd as nv  # noqa: E402
from train_block import RHT_SEED, SPEC, Linear  # noqa: E402


class MuonLinear(Linear):
    """A linear layer whose 32-bit weight is stepped by its orthogonalised momentum."""

    def tensor(self):
        return nv.muon_tensor(self.master, self.grad, weight_decay=0.01, copy=self.weight, amax=self.amax)


def quantised(x, amax, spec, kind=nv.SCALE_1D16, transposed=False, workspace=None):
    """x quantised with the maximum that its producer left."""
    rows, cols = (x.shape[1], x.shape[0]) if transposed else x.shape
    out = nv.empty_qtensor(rows, cols, kind, rht=int(spec.rht))
    out.amax = amax
    return nv.nvfp4_quantize(x, [spec], [out], workspace)[0]


class GatedBlock:
    def __init__(self, hidden=256, heads=4, kv_heads=2, ffn=512, lengths=(200, 56, 128, 128), seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.ffn = heads, kv_heads, hidden // heads, ffn
        self.qkv = MuonLinear((heads + 2 * kv_heads) * self.dim, hidden, gen)
        self.out, self.both, self.down = (MuonLinear(n, k, gen) for n, k in ((hidden, hidden), (2 * ffn, hidden), (hidden, ffn)))
        self.linears = (self.qkv, self.out, self.both, self.down)
        self.norms = torch.tensor([1.0, 0.0, 1.0, 0.0], device="cuda")[:, None].repeat(1, hidden)
        self.norm_grads = torch.zeros(4, hidden, device="cuda")
        self.head_norms, self.head_grads = torch.ones(2, self.dim, device="cuda"), torch.zeros(2, self.dim, device="cuda")
        ends = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        self.cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
        self.packed = dict(causal=True, cu_q=self.cu, cu_k=self.cu, max_q=max(lengths), max_k=max(lengths))
        self.freqs, magnitude = nv.rope_frequencies(self.dim)
        self.rope = dict(cu=self.cu, q_weight=self.head_norms[0], k_weight=self.head_norms[1], magnitude=magnitude)
        self.matrices = nv.MuonList([l.tensor() for l in self.linears])
        self.vectors = nv.AdamWList([nv.adamw_tensor(w, g) for a, b in ((self.norms, self.norm_grads), (self.head_norms, self.head_grads))
                                     for w, g in zip(a, b)])
        self.workspace, self.batch_workspace, self.muon_workspace = nv.new_workspace(), nv.new_workspace(jobs=2), self.matrices.new_workspace()
        self.amax = torch.zeros(7, device="cuda")  # of two norms, h, the gates' gradients: plain and with the RHT

    def halves(self, q):
        """The two weights of a quantised [2 ffn][hidden] one."""
        n = self.ffn
        return [nv.QTensor(q.codes[i * n:(i + 1) * n], q.scales[i * n // 16:(i + 1) * n // 16], q.global_scale, q.amax, n, q.cols,
                           q.scale_kind) for i in range(2)]

    def forward(self, x):
        for l in self.linears:
            l.quantise_weight()
        self.amax.zero_()
        self.x, h, g = x, self.heads, self.kv_heads
        y, self.mean1, self.rstd1, _ = nv.layernorm(x, self.norms[0], self.norms[1], amax=self.amax[:1])
        qkv = self.qkv.forward(y, self.amax[:1]).view(x.shape[0], -1, self.dim)
        self.q_in, self.k_in, self.v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        self.q, self.k = nv.qk_rope(self.q_in, self.k_in, self.freqs, **self.rope)
        self.o, self.lse = nv.attention(self.q, self.k, self.v, **self.packed)
        a = self.out.forward(self.o.flatten(1))
        self.y2, self.mean2, self.rstd2, self.sum = nv.layernorm(a, self.norms[2], self.norms[3], residual=x, amax=self.amax[1:2])
        q = quantised(self.y2, self.amax[1:2], SPEC("row", amax_given=True), workspace=self.workspace)
        self.h, self.gate, self.up = nv.gemm_gated(q, *self.halves(self.both.w), activation="silu", amax=self.amax[2:3])
        return self.sum + self.down.forward(self.h, self.amax[2:3])

    def backward(self, dy, seed):
        t, n = dy.shape[0], self.ffn
        # through the gated block: dgate and dup side by side, in the place of gate and up
        q = nv.quantize(dy, [SPEC("row", "sr", sr_seed=seed)], self.workspace)[0]
        plain, rht = self.amax[3:4], self.amax[4:5]
        nv.nvfp4_gemm_gated_backward(q, self.down.wt, self.gate, self.up, self.gate, self.up, activation="silu", amax_gate=plain,
                                     amax_up=plain, amax_rht_gate=rht, amax_rht_up=rht, rht_seed=RHT_SEED)
        both = torch.as_strided(self.gate, (t, 2 * n), (2 * n, 1))
        self.weight_gradient(dy, self.h, self.down.grad, seed + 1)
        q = quantised(both, plain, SPEC("row", "sr", sr_seed=seed + 2, amax_given=True), workspace=self.workspace)
        d = nv.gemm(q, self.both.wt, "bf16")
        self.weight_gradient(both, self.y2, self.both.grad, seed + 3, rht)
        ds, self.norm_grads[2], self.norm_grads[3] = nv.layernorm_backward(d, self.sum, self.norms[2], self.mean2, self.rstd2, dsum=dy)
        do = self.out.backward(ds, seed + 4).view_as(self.o)
        # the gradients of q, k and v side by side, as the projection made them
        dqkv = torch.empty(t, self.heads + 2 * self.kv_heads, self.dim, dtype=torch.bfloat16, device="cuda")
        dq, dk, dv = dqkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        workspace = nv.new_attention_workspace(self.q, self.k, self.v, **self.packed)
        nv.nvfp4_attention_backward(do, self.q, self.k, self.v, self.o, self.lse, dq, dk, dv, workspace, **self.packed)
        nv.nvfp4_qk_rope_backward(dq, dk, dq, dk, self.freqs, self.q_in, self.k_in, dq_weight=self.head_grads[0],
                                  dk_weight=self.head_grads[1], **self.rope)
        d = self.qkv.backward(dqkv.flatten(1), seed + 6)
        dx, self.norm_grads[0], self.norm_grads[1] = nv.layernorm_backward(d, self.x, self.norms[0], self.mean1, self.rstd1, dsum=ds)
        return dx

    def weight_gradient(self, dy, x, grad, seed, rht=None):
        """grad = dy^T x with both along the tokens under the Hadamard transform; rht: dy's maximum there, if it is known."""
        qa, qb = (nv.empty_qtensor(a.shape[1], a.shape[0], nv.SCALE_1D16, rht=1) for a in (dy, x))
        if rht is not None:
            qa.amax = rht
        nv.nvfp4_quantize_batch([(dy, [SPEC("col", "sr", True, seed, RHT_SEED, amax_given=rht is not None)], [qa]),
                                 (x, [SPEC("col", "rtn", True, 0, RHT_SEED)], [qb])], self.batch_workspace)
        nv.nvfp4_gemm(qa, qb, grad)

    def step(self, number, lr=2e-3):
        for l in self.linears:
            l.amax.zero_()
        nv.muon(self.matrices, lr, workspace=self.muon_workspace)
        nv.adamw(self.vectors, lr=lr, beta1=0.9, beta2=0.95, step=number)


def train(steps=30, report=print):
    """The losses of `steps` steps towards a fixed mixing of the tokens."""
    block = GatedBlock()
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
