"""The block operators' cases: norms of query and key heads with the position
rotation, their gradient, the gated feed-forward products on 4-bit operands,
their gradient, and the step of matrices by orthogonalised updates; each in a
plain form of elementary torch operations in 32 bits (``own`` false) and through
this package (``own`` true), with the 64-bit definition beside them (``exact``)."""
import math
import random

import torch

own = False

EPS_NORM = 1e-6
LR, MOMENTUM, DECAY, STEPS = 3e-4, 0.95, 0.1, 5
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one new token each of 16 sequences, far into their contexts: latency
        dict(name="rope 16 single tokens", op="rope", batch=16, tokens=1, heads=40, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, dtype="bf16", packed=0, far=1000000, factor=32.0),
        # 16384 tokens at hidden 5120 (40 heads of 128, 8 key heads), as the QKV projection leaves them
        dict(name="rope 2x8192", op="rope", batch=2, tokens=8192, heads=40, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, dtype="bf16", packed=0, far=0, factor=1.0),
        # the gradient of the same step, back to the projection's output
        dict(name="rope grad 2x8192", op="rope_grad", batch=2, tokens=8192, heads=40, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, dtype="bf16", packed=0, far=0, factor=1.0),
        # 4096 tokens of packed documents, a part of an odd head rotated, interleaved pairs, 32-bit projections
        dict(name="rope grad packed part", op="rope_grad", batch=23, tokens=4096, heads=10, kv_heads=5, dim=80, rot=36,
             interleaved=True, norm=True, dtype="f32", packed=7, far=0, factor=4.0),
        # the smallest batch of tokens that the 4-bit products take, for which the weights are read
        dict(name="gated 16 tokens", op="gated", rows=16, hidden=5120, ffn=20480, activation="silu", keep=False),
        # sizes that fill no tile
        dict(name="gated 1008 ragged", op="gated", rows=1008, hidden=1040, ffn=2736, activation="gelu_tanh", keep=True),
        # the linear-layer step's 16384 tokens, 5120 -> 20480
        dict(name="gated 16384x5120x20480", op="gated", rows=16384, hidden=5120, ffn=20480, activation="silu", keep=True),
        # sizes that fill no tile, backwards
        dict(name="gated grad 1008 ragged", op="gated_grad", rows=1008, hidden=1040, ffn=2736, activation="gelu"),
        # the linear-layer step's 16384 tokens, back through 20480 -> 5120
        dict(name="gated grad 16384x5120x20480", op="gated_grad", rows=16384, hidden=5120, ffn=20480, activation="silu"),
        # the matrices of a few small layers, up and down projections: latency
        dict(name="muon 20x 256x1024", op="muon", count=20, rows=256, cols=1024, turn=True, param="f32", grad="f32",
             copy=True, rounding="rtn", apply=True),
        # orthogonalised matrices alone, of odd sizes
        dict(name="orthogonalize 7x 1000x1111", op="muon", count=7, rows=1000, cols=1111, turn=False, param="f32", grad="bf16",
             copy=False, rounding="rtn", apply=False),
        # the two FFN weights of one layer, with the bf16 weights that the quantiser reads
        dict(name="muon 2x 5120x20480", op="muon", count=2, rows=5120, cols=20480, turn=True, param="f32", grad="bf16",
             copy=True, rounding="rtn", apply=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "gated", "gated_grad", "muon"])
    if op in ("rope", "rope_grad"):
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128, 128, 80, 96])
        total = _log(rng, 1, 16384)
        batch = rng.randrange(1, 1 + min(8, total))
        packed = rng.choice([0, 0, 1 + rng.randrange(1000)])
        return dict(op=op, batch=batch, tokens=total if packed else max(1, total // batch), heads=kv * rng.choice([1, 2, 5]),
                    kv_heads=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2, 4 * rng.randrange(1, dim // 4 + 1)]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    packed=packed, far=0 if packed else rng.choice([0, 0, _log(rng, 1000, 2000000)]),
                    factor=rng.choice([1.0, 4.0, 32.0]))
    if op in ("gated", "gated_grad"):
        c = dict(op=op, rows=16 * _log(rng, 1, 1024), hidden=16 * _log(rng, 4, 320), ffn=16 * _log(rng, 4, 1280),
                 activation=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]))
        if rng.random() < 0.4:  # whole tiles
            c.update(rows=-(-c["rows"] // 256) * 256, hidden=-(-c["hidden"] // 128) * 128, ffn=-(-c["ffn"] // 256) * 256)
        if op == "gated":
            c["keep"] = rng.random() < 0.7
        return c
    rows, cols = _log(rng, 16, 5120), _log(rng, 16, 5120)
    param = rng.choice(["f32", "f32", "bf16"])
    return dict(op=op, count=max(1, min(_log(rng, 1, 20), 100_000_000 // (rows * cols))), rows=rows, cols=cols,
                turn=rng.random() < 0.5, param=param, grad=rng.choice(["bf16", "f32"]),
                copy=param == "f32" and rng.random() < 0.5, rounding=rng.choice(["rtn", "sr"]), apply=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _laplace(g, *shape):
    u = torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32) - 0.5
    return -torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999))


def _lengths(case):
    """The lengths of a packed case's documents (one of them empty where there are three or more), from the case alone."""
    r, n, total = random.Random(case["packed"]), case["batch"], case["tokens"]
    cuts = sorted(r.randrange(total + 1) for _ in range(n - 1))
    if n >= 3:
        cuts[-1] = cuts[-2]
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _frequencies(rot, factor, base=500000.0, original=4096):
    """Radians for each position of the rot / 2 pairs, and the rotation's magnitude.  With a factor above 1 a context of
    `original` tokens is stretched by parts: pairs that turn less than once in it are slowed by the factor, those that
    turn more than 32 times are left, those between in proportion."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if factor == 1.0:
        return f, 1.0
    turns = original * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1


LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nvfp4(x, two_d):
    """x [rows][cols] as 4-bit codes, E4M3 scales of 1x16 or 16x16 blocks and a 32-bit scale for the tensor."""
    rows, cols = x.shape
    top = x.abs().max()
    S = 2688.0 / top
    blocks = x.abs().view(rows, cols // 16, 16).amax(2)
    if two_d:
        blocks = blocks.view(rows // 16, 16, cols // 16).amax(1)
    scale = (blocks / 6.0 * S).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    r = torch.where(s > 0, S / s, torch.zeros_like(s))
    r = (r.repeat_interleave(16, 0) if two_d else r).repeat_interleave(16, 1)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize((x * r).abs(), borders).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)
    return dict(codes=code[:, 0::2] | code[:, 1::2] << 4, scales=scale.view(torch.uint8), S=S.reshape(1), amax=top.reshape(1),
                rows=rows, cols=cols, two_d=two_d)


def _spectrum(g, m, n):
    """A gradient's kind of matrix: some strong directions over a bulk of weak ones."""
    rank = min(m, n, 32)
    strong = _normal(g, m, rank) / torch.arange(1, rank + 1, device="cuda").sqrt() @ _normal(g, rank, n)
    return 1e-4 * (0.3 * strong + _normal(g, m, n) * torch.exp(0.5 * _normal(g, m, 1)))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("rope", "rope_grad"):
        h, kv, dim, t = case["heads"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
        lead = (case["tokens"],) if case["packed"] else (case["batch"], case["tokens"])
        channel = torch.exp(0.3 * _normal(g, dim))
        qkv = (_normal(g, *lead, h + 2 * kv, dim) * channel).to(t)
        s["q"], s["k"] = qkv[..., :h, :], qkv[..., h:h + kv, :]
        s["freqs"], s["magnitude"] = _frequencies(case["rot"], case["factor"])
        s["positions"] = s["cu"] = None
        if case["packed"]:
            n = _lengths(case)
            s["cu"] = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")
        elif case["far"]:
            start = torch.randint(case["far"] // 2, case["far"], (case["batch"], 1), generator=g, device="cuda")
            s["positions"] = (start + torch.arange(case["tokens"], device="cuda")).reshape(-1)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = 1 + 0.1 * _normal(g, dim), 1 + 0.1 * _normal(g, dim)
        if case["op"] == "rope_grad":
            s["dq"], s["dk"] = ((1e-3 * _laplace(g, *s[n].shape)).to(torch.bfloat16) for n in ("q", "k"))
        return s
    if case["op"] in ("gated", "gated_grad"):
        m, k, n = case["rows"], case["hidden"], case["ffn"]
        if case["op"] == "gated":
            channel = torch.exp(0.5 * _normal(g, k))
            s["a"] = _nvfp4(_normal(g, m, k) * channel, False)
            s["gate_weight"] = _nvfp4(_normal(g, n, k) * (1.5 * k ** -0.5), True)
            s["up_weight"] = _nvfp4(_normal(g, n, k) * k ** -0.5, True)
        else:
            s["a"] = _nvfp4(1e-3 * _laplace(g, m, k), False)
            s["weight"] = _nvfp4(_normal(g, n, k) * n ** -0.5, True)
            # gate and up side by side, as one projection's output
            both = (_normal(g, m, 2 * n) * 1.5).to(torch.bfloat16)
            s["gate"], s["up"] = both[:, :n], both[:, n:]
        return s
    s["tensors"] = []
    s["grad_scale"], s["seed"], s["step"] = torch.tensor([0.75], device="cuda"), 99 + seed, 100
    for i in range(case["count"]):
        shape = (case["cols"], case["rows"]) if case["turn"] and i % 2 else (case["rows"], case["cols"])
        t = dict(grad=_spectrum(g, *shape).to(TYPES[case["grad"]]))
        if case["apply"]:
            t["m"] = 0.5 * t["grad"].float() + 0.3 * _spectrum(g, *shape)
            t["param"] = (0.02 * _normal(g, *shape)).to(TYPES[case["param"]])
            t["copy"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
        s["tensors"].append(t)
    return s


# ------------------------------------------------------------- plain forms --
def _positions(s):
    """The place of every token in its sequence, in 64 bits: of the shape of the leading dimensions."""
    n, lead = s["tokens"], s["q"].shape[:-2]
    if s["positions"] is not None:
        return s["positions"].double().reshape(lead)
    at = torch.arange(n, device="cuda")
    if s["cu"] is not None:
        at = at - s["cu"][torch.bucketize(at, s["cu"][1:].long(), right=True)]
    return at.double().expand(lead)


def _turns(s):
    """cos and sin of every token's pairs, in 32 bits, times the magnitude: [..., 1, rot / 2]."""
    angle = _positions(s)[..., None, None] * s["freqs"]
    return (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()


def _pairs(x, s):
    """The first and second elements of the rotated pairs, and what is not rotated."""
    r = s["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    return a, b, x[..., r:]


def _joined(a, b, rest, s):
    both = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _rope(s):
    cos, sin = _turns(s)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if s["norm"]:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS_NORM) * s[name + "_weight"]
        a, b, rest = _pairs(x, s)
        out[name] = _joined(a * cos - b * sin, b * cos + a * sin, rest, s).to(torch.bfloat16)
    return out


def _rope_grad(s):
    cos, sin = _turns(s)
    out = {}
    for name in ("q", "k"):
        a, b, rest = _pairs(s["d" + name].float(), s)
        g = _joined(a * cos + b * sin, b * cos - a * sin, rest, s)
        if s["norm"]:
            x = s[name].float()
            rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS_NORM)
            h = x * rstd
            out["d" + name + "_weight"] = (g * h).flatten(0, -2).sum(0)
            g = g * s[name + "_weight"]
            g = rstd * (g - h * (g * h).mean(-1, keepdim=True))
        out["d" + name] = g.to(s[name].dtype)
    return out


def _values(t):
    """The element times block scale values of a 4-bit tensor, in 32 bits (exact)."""
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], device="cuda")
    pair = torch.stack([t["codes"] & 15, t["codes"] >> 4], -1).flatten(1).int()
    scale = t["scales"].view(torch.float8_e4m3fn).float().repeat_interleave(16, 1)
    return levels[pair].mul_(scale.repeat_interleave(16, 0) if t["two_d"] else scale)


def _product(a, b):
    return torch.matmul(_values(a), _values(b).t()).mul_(1 / a["S"]).mul_(1 / b["S"])


def _activation(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    if kind == "relu":
        return x.clamp(min=0), (x > 0).float()
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _gated(s):
    gate, up = _product(s["a"], s["gate_weight"]), _product(s["a"], s["up_weight"])
    h = _activation(gate, s["activation"])[0].mul_(up).to(torch.bfloat16)
    out = dict(h=h, amax=h.abs().max().float().reshape(1))
    if s["keep"]:
        out.update(gate=gate.to(torch.bfloat16), up=up.to(torch.bfloat16))
    return out


def _gated_grad(s):
    dh = _product(s["a"], s["weight"])
    f, df = _activation(s["gate"].float(), s["activation"])
    return dict(dgate=(df.mul_(s["up"].float()).mul_(dh)).to(torch.bfloat16), dup=f.mul_(dh).to(torch.bfloat16))


LOW = 0xFFFFFFFF


def _uniforms(n, index, step, seed):
    """The 16-bit numbers of a tensor's n elements: element i takes half i & 1 of word (i & 7) / 2 of Philox4x32-10 with
    the counter (i / 8, index, step, tag), on 32-bit words held in int64 tensors."""
    group = torch.arange((n + 7) // 8, device="cuda")
    c0, c1, c2, c3 = (group & LOW, torch.full_like(group, index), torch.full_like(group, step & LOW),
                      torch.full_like(group, 0x4D550000 + (step >> 32)))
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & LOW) ^ c1 ^ k0, p1 & LOW, (p0 >> 32 & LOW) ^ c3 ^ k1, p0 & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack([x >> sh & 0xFFFF for x in (c0, c1, c2, c3) for sh in (0, 16)], 1).reshape(-1)[:n]


def _orthogonal(x):
    """Newton-Schulz products on a stack of matrices with no more rows than columns."""
    norm = torch.sqrt((x.double() ** 2).sum((1, 2), keepdim=True)).float()
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    for _ in range(STEPS):
        a = torch.matmul(x, x.transpose(1, 2))
        x = NS_A * x + torch.matmul(NS_B * a + NS_C * torch.matmul(a, a), x)
    return x


def _wide(x):
    """A matrix, turned if it has more rows than columns."""
    return x.t() if x.shape[0] > x.shape[1] else x


def _update(s, orthogonal, grads):
    """The updates of all tensors, each of its tensor's shape."""
    o = orthogonal(torch.stack([_wide(g) for g in grads]))
    return [x.t() if g.shape[0] > g.shape[1] else x for x, g in zip(o, grads)]


def _muon(s):
    if not s["apply"]:
        return dict(update=[o.to(torch.bfloat16) for o in _update(s, _orthogonal, [t["grad"].float() for t in s["tensors"]])])
    us = []
    for t in s["tensors"]:
        g = t["grad"].float() * s["grad_scale"]
        t["m"].mul_(MOMENTUM).add_(g, alpha=1 - MOMENTUM)
        us.append((1 - MOMENTUM) * g + MOMENTUM * t["m"])
    for i, (t, o) in enumerate(zip(s["tensors"], _update(s, _orthogonal, us))):
        p = t["param"].float() * (1 - LR * DECAY) - LR * 0.2 * math.sqrt(max(o.shape)) * o
        if t["param"].dtype == torch.bfloat16 and s["rounding"] == "sr":
            u = _uniforms(p.numel(), i, s["step"], s["seed"]).int().reshape(p.shape)
            p = ((p.contiguous().view(torch.int32) + u) & -65536).view(torch.float32)
        t["param"].copy_(p)
        if t["copy"] is not None:
            t["copy"].copy_(p)
    return _updated(s)


def _updated(s):
    out = dict(param=[t["param"] for t in s["tensors"]], m=[t["m"] for t in s["tensors"]])
    if s["copy"]:
        out["copy"] = [t["copy"] for t in s["tensors"]]
    return out


# ---------------------------------------------------------- the package's --
def _qtensor(nv, t):
    return nv.QTensor(t["codes"], t["scales"], t["S"], t["amax"], t["rows"], t["cols"],
                      nv.SCALE_2D16 if t["two_d"] else nv.SCALE_1D16)


def _run_own(s):
    import nvfp4_bit_quantization_amd as nv
    if s["op"] in ("rope", "rope_grad"):
        opts = dict(positions=s["positions"], cu=s["cu"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS_NORM,
                    interleaved=s["interleaved"], magnitude=s["magnitude"])
        if s["op"] == "rope":
            q, k = nv.qk_rope(s["q"], s["k"], s["freqs"], **opts)
            return dict(q=q, k=k)
        dq, dk, dqw, dkw = nv.qk_rope_backward(s["dq"], s["dk"], s["freqs"], s["q"], s["k"], **opts)
        return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw) if s["norm"] else dict(dq=dq, dk=dk)
    if s["op"] in ("gated", "gated_grad"):
        if "own" not in s:  # a program holds its quantised tensors
            s["own"] = {n: _qtensor(nv, s[n]) for n in ("a", "gate_weight", "up_weight", "weight") if n in s}
        q = s["own"]
        if s["op"] == "gated":
            amax = torch.zeros(1, device="cuda")
            h, gate, up = nv.gemm_gated(q["a"], q["gate_weight"], q["up_weight"], activation=s["activation"], keep=s["keep"],
                                        amax=amax)
            return dict(h=h, amax=amax, gate=gate, up=up) if s["keep"] else dict(h=h, amax=amax)
        dgate, dup = nv.gemm_gated_backward(q["a"], q["weight"], s["gate"], s["up"], activation=s["activation"])
        return dict(dgate=dgate, dup=dup)
    if not s["apply"]:
        return dict(update=nv.orthogonalize([t["grad"] for t in s["tensors"]], steps=STEPS, coefficients=(NS_A, NS_B, NS_C)))
    if "list" not in s:  # a training program lays its tensors' list out once
        s["list"] = nv.MuonList([nv.MuonTensor(t["param"], t["grad"], t["m"], weight_decay=DECAY,
                                               scale=0.2 * math.sqrt(max(t["param"].shape)), copy=t["copy"]) for t in s["tensors"]])
    nv.muon(s["list"], lr=LR, momentum=MOMENTUM, nesterov=True, steps=STEPS, coefficients=(NS_A, NS_B, NS_C),
            rounding=s["rounding"], seed=s["seed"], step=s["step"], grad_scale=s["grad_scale"])
    return _updated(s)


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope, "rope_grad": _rope_grad, "gated": _gated, "gated_grad": _gated_grad, "muon": _muon}[state["op"]](state)


# -------------------------------------------------------------------- work --
def work(case):
    if case["op"] in ("rope", "rope_grad"):
        tokens = case["tokens"] * (1 if case["packed"] else case["batch"])
        n = tokens * (case["heads"] + case["kv_heads"]) * case["dim"]
        x = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "rope":
            return dict(bytes=n * (x + 2), flops=n * (8 if case["norm"] else 3))
        return dict(bytes=n * (2 + x + (x if case["norm"] else 0)), flops=n * (14 if case["norm"] else 3))
    if case["op"] in ("gated", "gated_grad"):
        m, k, n = case["rows"], case["hidden"], case["ffn"]
        code = 9 / 16  # bytes of a 1D block's element
        weight = 0.5 + 1 / 256
        if case["op"] == "gated":
            return dict(bytes=code * m * k + 2 * weight * n * k + 2 * m * n * (3 if case["keep"] else 1), flops=4 * m * n * k)
        return dict(bytes=code * m * k + weight * n * k + 2 * m * n * 4, flops=2 * m * n * k)
    m, n = sorted((case["rows"], case["cols"]))
    size = {"bf16": 2, "f32": 4}
    held = size[case["grad"]] + (8 + 2 * size[case["param"]] + (2 if case["copy"] else 0) if case["apply"] else 2)
    # x x^T and its square are symmetric: half of each, then the product with x
    return dict(bytes=case["count"] * m * n * held, flops=case["count"] * STEPS * (m * m * n + m * m * m + 2 * m * m * n))


# ------------------------------------------------------------------- exact --
def _exact_rope(s, grad):
    lead = s["q"].shape[:-2]
    if s["positions"] is not None:
        at = s["positions"].reshape(lead)
    elif s["cu"] is not None:
        ends = s["cu"].tolist()
        at = torch.cat([torch.arange(b - a, device="cuda") for a, b in zip(ends, ends[1:])])
    else:
        at = torch.arange(s["tokens"], device="cuda")[None].repeat(lead[0], 1)
    r = s["rot"]
    turn = torch.polar(torch.full((*lead, 1, r // 2), s["magnitude"], dtype=torch.float64, device="cuda"),
                       at.double()[..., None, None] * s["freqs"])
    first = torch.arange(0, r, 2, device="cuda") if s["interleaved"] else torch.arange(r // 2, device="cuda")
    second = first + (1 if s["interleaved"] else r // 2)
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        w = s[name + "_weight"].double() if s["norm"] else None
        root = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS_NORM)
        if not grad:
            y = x / root * w if s["norm"] else x.clone()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
            continue
        y = s["d" + name].double()
        z = torch.complex(y[..., first], y[..., second]) * turn.conj()
        y[..., first], y[..., second] = z.real, z.imag
        if s["norm"]:
            out["d" + name + "_weight"] = (y * x / root).sum(tuple(range(x.dim() - 1)))
            y = y * w
            y = y / root - x * (x * y).mean(-1, keepdim=True) / root ** 3
        out["d" + name] = y
    return out


def _exact_values(t):
    lut = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    out = torch.empty(t["rows"], t["cols"], dtype=torch.float64, device="cuda")
    for half in (0, 1):
        c = (t["codes"] >> (4 * half)).long() & 15
        out[:, half::2] = lut[c & 7] * (1 - 2 * (c >> 3))
    b = t["scales"].long()
    e, m = b >> 3 & 15, b & 7
    scale = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m.double() / 8), m.double() / 512)
    view = out.view(-1, 16, t["cols"] // 16, 16) if t["two_d"] else out.view(t["rows"], 1, t["cols"] // 16, 16)
    view *= scale[:, None, :, None]
    return out / t["S"].double()


def _exact_act(x, kind):
    if kind == "silu":
        return x * torch.special.expit(x)
    if kind == "relu":
        return torch.relu(x)
    if kind == "gelu":
        return x * torch.special.ndtr(x)
    return x * torch.special.expit(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))


def _exact_gated(s):
    a = _exact_values(s["a"])
    gate, up = (a @ _exact_values(s[n]).t() for n in ("gate_weight", "up_weight"))
    h = _exact_act(gate, s["activation"]) * up
    out = dict(h=h, amax=h.to(torch.bfloat16).double().abs().max().reshape(1))
    if s["keep"]:
        out.update(gate=gate, up=up)
    return out


def _exact_gated_grad(s):
    dh = _exact_values(s["a"]) @ _exact_values(s["weight"]).t()
    dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
    step = max(1, 2 ** 26 // s["ffn"])
    for i in range(0, s["rows"], step):
        g = s["gate"][i:i + step].double().requires_grad_()
        f = _exact_act(g, s["activation"])
        dup[i:i + step] = f.detach() * dh[i:i + step]
        dgate[i:i + step] = torch.autograd.grad(f, g, s["up"][i:i + step].double() * dh[i:i + step])[0]
    return dict(dgate=dgate, dup=dup)


def _exact_orthogonal(x):
    if x.shape[0] > x.shape[1]:
        return _exact_orthogonal(x.t().contiguous()).t()
    x = x / torch.linalg.matrix_norm(x).clamp(min=1e-300)
    for _ in range(STEPS):
        a = x @ x.t()
        b = a @ a
        x = NS_A * x + NS_B * (a @ x) + NS_C * (b @ x)
    return x


def _exact_uniforms(n, index, step, seed):
    """The 16-bit numbers as fractions, by 16-bit limbs, so that no product passes 62 bits."""
    i = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)
    c = [i % 2 ** 32, torch.zeros_like(i) + index, torch.zeros_like(i) + step % 2 ** 32, torch.zeros_like(i) + (0x4D550000 + step // 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32]

    def product(x, by):
        low, high = x * (by % 65536), x * (by // 65536)
        low = low + high % 65536 * 65536
        return (low // 2 ** 32 + high // 65536) % 2 ** 32, low % 2 ** 32

    for _ in range(10):
        (h0, l0), (h1, l1) = product(c[0], 0xD2511F53), product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    half = torch.stack([torch.stack([w % 65536, w // 65536], 1) for w in c], 1)
    return half.reshape(-1)[:n].double() / 65536


def _exact_muon(s):
    if not s["apply"]:
        return dict(update=[_exact_orthogonal(t["grad"].double()) for t in s["tensors"]])
    out = dict(param=[], m=[], copy=[])
    for i, t in enumerate(s["tensors"]):
        g = t["grad"].double() * s["grad_scale"].double()
        m = MOMENTUM * t["m"].double() + (1 - MOMENTUM) * g
        o = _exact_orthogonal((1 - MOMENTUM) * g + MOMENTUM * m)
        p = t["param"].double()
        p = p - LR * DECAY * p - LR * 0.2 * math.sqrt(max(o.shape)) * o
        if t["param"].dtype == torch.bfloat16 and s["rounding"] == "sr":
            unit = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
            u = _exact_uniforms(p.numel(), i, s["step"], s["seed"]).reshape(p.shape)
            p = torch.copysign(torch.floor(p.abs() / unit + u) * unit, p)
        out["param"].append(p)
        out["m"].append(m)
        if s["copy"]:
            out["copy"].append(p)
    return {k: v for k, v in out.items() if v}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "rope_grad"):
        return _exact_rope(s, case["op"] == "rope_grad")
    return {"gated": _exact_gated, "gated_grad": _exact_gated_grad, "muon": _exact_muon}[case["op"]](s)
