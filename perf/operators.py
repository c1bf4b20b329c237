"""The training operators' cases: layer norm and its gradient, attention and its
gradient, and the AdamW step over many tensors, each in a plain form of
elementary torch operations in 32 bits (``own`` false) and through this
package (``own`` true), with the 64-bit definition beside them (``exact``)."""
import math
import random

import torch

own = False

EPS_NORM = 1e-5
LR, BETA1, BETA2, EPS_ADAM, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the 256x256 tensor of the smallest configuration: latency
        dict(name="norm 256x256", op="norm", rows=256, cols=256, dtype="bf16", residual=False, pad=0),
        # the residual add and norm before a quantised linear layer, hidden 5120
        dict(name="norm 8192x5120 residual", op="norm", rows=8192, cols=5120, dtype="bf16", residual=True, pad=0),
        # odd width, rows of a wider buffer, 32-bit activations
        dict(name="norm grad 1000x777 f32", op="norm_grad", rows=1000, cols=777, dtype="f32", residual=False, pad=3),
        # the full linear-layer step's 16384 tokens at hidden 5120
        dict(name="norm grad 16384x5120", op="norm_grad", rows=16384, cols=5120, dtype="bf16", residual=True, pad=0),
        # a few short sequences: latency
        dict(name="attention 4x100 dim 64", op="attention", batch=4, q_len=100, k_len=100, heads=4, kv_heads=2, dim=64,
             causal=True, window=0, packed=0),
        # 8192 tokens of one sequence at hidden 5120 (40 heads of 128), causal
        dict(name="attention 8192 causal", op="attention", batch=1, q_len=8192, k_len=8192, heads=40, kv_heads=8,
             dim=128, causal=True, window=0, packed=0),
        # 4096 tokens of packed documents of uneven lengths, sliding window
        dict(name="attention grad packed", op="attention_grad", batch=23, q_len=4096, k_len=4096, heads=16, kv_heads=16,
             dim=64, causal=True, window=500, packed=7),
        # 2 x 4096 tokens at hidden 5120, causal, shared key heads
        dict(name="attention grad 2x4096", op="attention_grad", batch=2, q_len=4096, k_len=4096, heads=40, kv_heads=8,
             dim=128, causal=True, window=0, packed=0),
        # every tensor of a small model: many short ones, 32-bit states
        dict(name="adamw 60 small f32", op="adamw", count=30, rows=256, cols=257, param="f32", grad="f32", state=32,
             copy=False, rounding="rtn"),
        # two FFN weights in 32-bit masters, with the bf16 weights that the quantiser reads
        dict(name="adamw 2x 5120x20480 f32", op="adamw", count=2, rows=5120, cols=20480, param="f32", grad="bf16",
             state=32, copy=True, rounding="rtn"),
        # the same weights as bf16 masters with 8-bit states, rounded stochastically
        dict(name="adamw 2x 5120x20480 8-bit", op="adamw", count=2, rows=5120, cols=20480, param="bf16", grad="bf16",
             state=8, copy=False, rounding="sr"),
        # an odd number of medium tensors with 8-bit states beside 32-bit masters
        dict(name="adamw 7x 1024x1000 8-bit", op="adamw", count=7, rows=1024, cols=1000, param="f32", grad="bf16",
             state=8, copy=True, rounding="sr"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "attention", "attention_grad", "adamw"])
    if op in ("norm", "norm_grad"):
        rows, cols = _log(rng, 1, 16384), _log(rng, 16, 5120)
        if rng.random() < 0.5:
            cols = max(16, cols // 16 * 16)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 8, 3]))
    if op == "adamw":
        n = _log(rng, 1000, 50_000_000)
        count = max(1, min(_log(rng, 1, 60), n // 500))
        cols = max(1, min(_log(rng, 16, 5120), n // count))
        state = rng.choice([8, 32])
        param = rng.choice(["bf16", "f32"])
        return dict(op=op, count=count, rows=max(1, n // count // cols), cols=cols, param=param,
                    grad=rng.choice(["bf16", "f32"]), state=state, copy=param == "f32" and rng.random() < 0.5,
                    rounding=rng.choice(["rtn", "sr"]))
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5])
    # a query with one key in sight has no gradient but through its value: lengths start where most have more
    k_len = _log(rng, 1 if op == "attention" else 16, 4096)
    packed = rng.choice([0, 0, 1 + rng.randrange(1000)])
    causal = rng.random() < 0.7
    q_len = k_len if packed or rng.random() < 0.7 else _log(rng, 1, 4096)
    batch = rng.randrange(1, max(2, min(30, k_len // 8))) if packed else max(1, min(_log(rng, 1, 8), 8192 // max(q_len, k_len)))
    return dict(op=op, batch=batch, q_len=q_len, k_len=k_len, heads=heads, kv_heads=kv, dim=rng.choice([64, 128, 128, 80]),
                causal=causal, window=rng.choice([0, _log(rng, 16, 1024)]) if causal else 0, packed=packed)


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _laplace(g, *shape):
    u = torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32) - 0.5
    return -torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999))


def _padded(t, pad):
    """t as the first columns of a buffer with rows longer by `pad`."""
    if not pad:
        return t
    b = t.new_zeros(t.shape[0], t.shape[1] + pad)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def _lengths(case):
    """The lengths of a packed case's documents (one of them empty where there are three or more), from the case alone."""
    r, n, total = random.Random(case["packed"]), case["batch"], case["k_len"]
    cuts = sorted(r.randrange(total + 1) for _ in range(n - 1))
    if n >= 3:
        cuts[-1] = cuts[-2]
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _pairs(q, k, causal, window):
    """The query-key pairs that a sequence of q queries and k keys has in sight."""
    if not causal:
        return q * k
    return sum(max(0, min(i + 1 + k - q, window or k)) for i in range(q))


def _case_pairs(case):
    if case["packed"]:
        return sum(_pairs(n, n, case["causal"], case["window"]) for n in _lengths(case))
    return case["batch"] * _pairs(case["q_len"], case["k_len"], case["causal"], case["window"])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("norm", "norm_grad"):
        t, rows, cols, pad = TYPES[case["dtype"]], case["rows"], case["cols"], case["pad"]
        channel = torch.exp(0.5 * _normal(g, cols))
        x = _normal(g, rows, cols) * channel + 0.1 * _normal(g, cols)
        s["weight"] = 1 + 0.1 * _normal(g, cols)
        s["bias"] = 0.1 * _normal(g, cols)
        if case["op"] == "norm":
            s["x"] = _padded(x.to(t), pad)
            s["residual"] = _padded(_normal(g, rows, cols).to(t), pad) if case["residual"] else None
        else:
            s["x"] = _padded(x.to(t), pad)
            xf = s["x"].double()
            s["mean"] = xf.mean(1).float()
            s["rstd"] = (1 / torch.sqrt(xf.var(1, unbiased=False) + EPS_NORM)).float()
            s["dy"] = _padded((1e-3 * _laplace(g, rows, cols)).to(t), pad)
            s["dsum"] = _padded((1e-3 * _laplace(g, rows, cols)).to(t), pad) if case["residual"] else None
        return s
    if case["op"] == "adamw":
        # the tensors' starts are spaced in common buffers, one row of a buffer each
        s["buffers"] = {}
        for kind, n, state in (("matrix", case["rows"] * case["cols"], case["state"]), ("vector", case["cols"], 32)):
            shape = (case["count"], -(-n // 64) * 64)
            live = torch.arange(shape[1], device="cuda") < n
            r = 1e-3 * torch.exp(0.5 * _normal(g, *shape)) * live
            m = 0.3 * r * _normal(g, *shape)
            b = dict(param=(0.02 * _normal(g, *shape) * live).to(TYPES[case["param"]] if kind == "matrix" else torch.float32))
            s[kind + "_grad"] = (r * _normal(g, *shape)).to(TYPES[case["grad"]])
            if state == 8:
                for key, x in (("m", m), ("v", r)):
                    code, scale = _encode(x.reshape(-1), None, key == "v")
                    b[key], b[key + "_scale"] = code.reshape(shape), scale.reshape(shape[0], -1)
            else:
                b["m"], b["v"] = m, r * r
            if case["copy"] and kind == "matrix":
                b["copy"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            s["buffers"][kind] = b
        s["tensors"] = []
        for i in range(case["count"]):
            for kind, shape, wd in (("matrix", (case["rows"], case["cols"]), DECAY), ("vector", (case["cols"],), 0.0)):
                n, b = math.prod(shape), s["buffers"][kind]
                t = {key: x[i, :n].view(shape) for key, x in b.items() if not key.endswith("_scale")}
                t.update({key: x[i, :-(-n // 32)] for key, x in b.items() if key.endswith("_scale")})
                t.update(grad=s[kind + "_grad"][i, :n].view(shape), decay=wd, state=8 if "m_scale" in t else 32)
                t.setdefault("copy", None)
                s["tensors"].append(t)
        s["seed"] = 1234 + seed
        s["step"] = 100
        s["grad_scale"] = torch.tensor([0.75], device="cuda")
        return s
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    nq, nk = (case["q_len"], case["k_len"])
    lead = () if case["packed"] else (case["batch"],)
    s["q"] = _normal(g, *lead, nq, heads, dim).to(torch.bfloat16)
    # keys and values side by side in one projection's output
    kvs = _normal(g, *lead, nk, 2, kv, dim).to(torch.bfloat16)
    s["k"], s["v"] = kvs[..., 0, :, :], kvs[..., 1, :, :]
    s["cu"] = None
    if case["packed"]:
        n = _lengths(case)
        at = [sum(n[:i]) for i in range(len(n) + 1)]
        s["cu"], s["longest"] = torch.tensor(at, dtype=torch.int32, device="cuda"), max(n)
    s["scale"] = 1 / math.sqrt(dim)
    if case["op"] == "attention_grad":
        o, lse = _attention(s)
        s["o"], s["lse"] = o, lse
        s["do"] = (1e-3 * _laplace(g, *s["q"].shape)).to(torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms --
def _norm(s):
    x = s["x"]
    total = None
    if s["residual"] is not None:
        total = (x.float() + s["residual"].float()).to(x.dtype)
        x = total
    xf = x.float()
    mean = xf.mean(1, keepdim=True)
    c = xf - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS_NORM)
    y = (c * rstd * s["weight"] + s["bias"]).to(x.dtype)
    out = dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0])
    if total is not None:
        out.update(sum=total, amax=y.abs().max().float().reshape(1))
    return out


def _norm_grad(s):
    dy, x = s["dy"].float(), s["x"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    a = dy * s["weight"]
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0), dbias=dy.sum(0))


def _hidden(s):
    """Which query-key pairs are out of sight: [q_len][k_len]."""
    nq, nk = s["q_len"], s["k_len"]
    i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")[None]
    if s["cu"] is not None:  # packed: equal lengths, so positions within the documents compare as those of the whole
        doc = torch.bucketize(torch.arange(nk, device="cuda"), s["cu"][1:].long(), right=True)
        out = doc[:, None] != doc[None]
    else:
        i = i + (nk - nq)
        out = torch.zeros(nq, nk, dtype=torch.bool, device="cuda")
    if s["causal"]:
        out = out | (j > i)
    if s["window"]:
        out = out | (j <= i - s["window"])
    return out


def _by_head(t, group=1):
    """[batch][len][heads][dim] in 32 bits by head, shared heads repeated."""
    t = t if t.dim() == 4 else t[None]
    return t.float().transpose(1, 2).repeat_interleave(group, 1).contiguous()


def _back(t, like):
    return t.transpose(1, 2).reshape(like.shape).to(like.dtype).contiguous()


def _by_token(x):
    """[batch][heads][len] as [heads][batch * len]."""
    return x.transpose(0, 1).reshape(x.shape[1], -1).contiguous()


def _attention(s):
    group = s["heads"] // s["kv_heads"]
    q, k, v = _by_head(s["q"]), _by_head(s["k"], group), _by_head(s["v"], group)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"]).masked_fill_(_hidden(s), -math.inf)
    top = p.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = p.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return _back(o, s["q"]), _by_token((top + torch.log(total))[..., 0])


def _attention_grad(s):
    group, kv = s["heads"] // s["kv_heads"], s["kv_heads"]
    q, k, v = _by_head(s["q"]), _by_head(s["k"], group), _by_head(s["v"], group)
    do, o = _by_head(s["do"]), _by_head(s["o"])
    b, h, n, d = q.shape
    lse = s["lse"].reshape(h, b, n).transpose(0, 1)[..., None]
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    p = p.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_().masked_fill_(_hidden(s), 0.0)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous()).sub_((do * o).sum(3, keepdim=True)).mul_(p).mul_(s["scale"])
    del p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    dk, dv = (t.reshape(b, kv, group, -1, d).sum(2) for t in (dk, dv))
    return dict(dq=_back(dq, s["q"]), dk=_back(dk, s["k"]), dv=_back(dv, s["v"]))


LOW = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on 32-bit words held in int64 tensors."""
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & LOW) ^ c1 ^ k0, p1 & LOW, (p0 >> 32 & LOW) ^ c3 ^ k1, p0 & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return c0, c1, c2, c3


def _uniforms(n, index, which, step, seed):
    """The 16-bit numbers of a tensor's n elements: element i takes half i & 1 of word (i & 7) / 2 of the draw with the
    counter (i / 8, index * 4 + which, step, tag)."""
    group = torch.arange((n + 7) // 8, device="cuda")
    full = torch.full_like
    w = _philox(group & LOW, full(group, index * 4 + which), full(group, step & LOW), full(group, 0x41440000 + (step >> 32)),
                seed & LOW, seed >> 32)
    return torch.stack([x >> sh & 0xFFFF for x in w for sh in (0, 16)], 1).reshape(-1)[:n]


def _blocks(x):
    n = x.numel()
    return torch.cat([x, x.new_zeros(-n % 32)]).reshape(-1, 32) if n % 32 else x.reshape(-1, 32)


def _encode(x, u, positive):
    """Blocks of 32 values as E4M3 elements (bytes) and one E8M0 scale (byte) each: the scale is the least power of two
    that keeps the block within 448; elements are rounded to nearest, or stochastically by the 16-bit numbers u.
    `positive`: what is not zero stays so."""
    b = _blocks(x)
    e = ((b.abs().amax(1).view(torch.int32) + 0x1FFFFF) >> 23) - 135
    e = e.clamp(min=-126)
    y = b.abs() * ((127 - e) << 23).view(torch.float32)[:, None]
    ey = (y.view(torch.int32) >> 23).sub_(127).clamp_(min=-6)
    t = y * ((130 - ey) << 23).view(torch.float32)
    c = torch.round(t) if u is None else torch.floor(t + _blocks(u.float()) * (1 / 65536))
    if positive:
        c = torch.where(b != 0, c.clamp(min=1), c)
    code = (ey + 6) * 8 + c.int()
    code = code + torch.signbit(b).int() * 128
    return code.to(torch.uint8).reshape(-1)[:x.numel()].clone(), (e + 127).to(torch.uint8)


def _decode(code, scale):
    x = _blocks(code.view(torch.float8_e4m3fn).float())
    return (x * torch.exp2(scale.float() - 127)[:, None]).reshape(-1)[:code.numel()]


def _adamw(s):
    t1, t2 = 1 / (1 - BETA1 ** s["step"]), 1 / math.sqrt(1 - BETA2 ** s["step"])
    for i, t in enumerate(s["tensors"]):
        sr, n = s["rounding"] == "sr", t["param"].numel()
        draws = (lambda which: _uniforms(n, i, which, s["step"], s["seed"]) if sr else None)
        g = t["grad"].float() * s["grad_scale"]
        if t["state"] == 8:
            m = _decode(t["m"].reshape(-1), t["m_scale"]).reshape(g.shape)
            r = _decode(t["v"].reshape(-1), t["v_scale"]).reshape(g.shape)
            v = r * r
        else:
            m, v = t["m"], t["v"]
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + g * g * (1 - BETA2)
        r = torch.sqrt(v)
        p = t["param"].float() * (1 - LR * t["decay"]) - LR * ((m * t1) / (r * t2 + EPS_ADAM))
        if t["param"].dtype == torch.bfloat16 and sr:
            p = ((p.view(torch.int32) + draws(2).int().reshape(p.shape)) & -65536).view(torch.float32)
        t["param"].copy_(p)
        if t["copy"] is not None:
            t["copy"].copy_(p)
        if t["state"] == 8:
            for key, x, which in (("m", m, 0), ("v", r, 1)):
                code, scale = _encode(x.reshape(-1), draws(which), which == 1)
                t[key].copy_(code.reshape(t[key].shape))
                t[key + "_scale"].copy_(scale)
        else:
            t["m"].copy_(m)
            t["v"].copy_(v)
    return _updated(s)


def _updated(s):
    """The buffers of all tensors' new values: 8-bit states as the numbers that their elements and block scales stand for."""
    return {kind: {key: x if x.dtype != torch.uint8 else
                   x.view(torch.float8_e8m0fnu if key.endswith("_scale") else torch.float8_e4m3fn) for key, x in b.items()}
            for kind, b in s["buffers"].items()}


# ---------------------------------------------------------- the package's --
def _run_own(s):
    import nvfp4_bit_quantization_amd as nv
    if s["op"] == "norm":
        amax = torch.zeros(1, device="cuda") if s["residual"] is not None else None
        y, mean, rstd, total = nv.layernorm(s["x"], s["weight"], s["bias"], EPS_NORM, residual=s["residual"], amax=amax)
        out = dict(y=y, mean=mean, rstd=rstd)
        if total is not None:
            out.update(sum=total, amax=amax)
        return out
    if s["op"] == "norm_grad":
        dx, dw, db = nv.layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dsum=s["dsum"])
        return dict(dx=dx, dweight=dw, dbias=db)
    if s["op"] == "adamw":
        if "list" not in s:  # a training program lays its tensors' list out once
            s["list"] = nv.AdamWList([nv.AdamWTensor(t["param"], t["grad"], t["m"], t["v"], t.get("m_scale"), t.get("v_scale"),
                                                     weight_decay=t["decay"], copy=t["copy"]) for t in s["tensors"]])
        nv.adamw(s["list"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS_ADAM, step=s["step"], rounding=s["rounding"],
                 seed=s["seed"], grad_scale=s["grad_scale"])
        return _updated(s)
    opts = dict(causal=s["causal"], window=s["window"], scale=s["scale"])
    if s["cu"] is not None:
        opts.update(cu_q=s["cu"], cu_k=s["cu"], max_q=s["longest"], max_k=s["longest"])
    if s["op"] == "attention":
        o, lse = nv.attention(s["q"], s["k"], s["v"], **opts)
        return dict(o=o, lse=lse)
    dq, dk, dv = nv.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **opts)
    return dict(dq=dq, dk=dk, dv=dv)


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "norm":
        return _norm(state)
    if state["op"] == "norm_grad":
        return _norm_grad(state)
    if state["op"] == "adamw":
        return _adamw(state)
    if state["op"] == "attention_grad":
        return _attention_grad(state)
    o, lse = _attention(state)
    return dict(o=o, lse=lse)


# -------------------------------------------------------------------- work --
def work(case):
    if case["op"] in ("norm", "norm_grad"):
        size = 2 if case["dtype"] == "bf16" else 4
        n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
        tensors = (4 if case["residual"] else 2) if case["op"] == "norm" else (4 if case["residual"] else 3)
        return dict(bytes=n * size * tensors + 8 * rows + (8 if case["op"] == "norm" else 12) * cols,
                    flops=n * (8 if case["op"] == "norm" else 14))
    if case["op"] == "adamw":
        size = {"bf16": 2, "f32": 4}
        n, c = case["rows"] * case["cols"], case["cols"]
        state = 2 * 2 * (4 if case["state"] == 32 else 1 + 1 / 32)
        per = 2 * size[case["param"]] + size[case["grad"]] + state + (2 if case["copy"] else 0)
        return dict(bytes=case["count"] * (n * per + c * (8 + size[case["grad"]] + 16)), flops=case["count"] * (n + c) * 16)
    q = case["q_len"] * (1 if case["packed"] else case["batch"])
    k = case["k_len"] * (1 if case["packed"] else case["batch"])
    d, h, kv = case["dim"], case["heads"], case["kv_heads"]
    pairs = max(1, _case_pairs(case))
    if case["op"] == "attention":
        return dict(bytes=2 * d * (2 * q * h + 2 * k * kv) + 4 * q * h, flops=4 * d * h * pairs)
    return dict(bytes=2 * d * (4 * q * h + 4 * k * kv) + 4 * q * h, flops=10 * d * h * pairs)


# ------------------------------------------------------------------- exact --
def _exact_norm(s):
    x = s["x"].double()
    if s["residual"] is not None:
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    var, mean = torch.var_mean(x, 1, correction=0)
    out = dict(y=(x - mean[:, None]) / torch.sqrt(var + EPS_NORM)[:, None] * s["weight"].double() + s["bias"].double(),
               mean=mean, rstd=1 / torch.sqrt(var + EPS_NORM))
    if s["residual"] is not None:
        out.update(sum=x, amax=out["y"].to(s["x"].dtype).double().abs().max().reshape(1))
    return out


def _exact_norm_grad(s):
    x = s["x"].double().requires_grad_()
    w, b = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    dy = s["dy"].double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    dx, dw, db = torch.autograd.grad((x - mean) / torch.sqrt(var + EPS_NORM) * w + b, (x, w, b), dy)
    return dict(dx=dx if s["dsum"] is None else dx + s["dsum"].double(), dweight=dw, dbias=db)


def _exact_sight(nq, nk, s):
    i = torch.arange(nq, device="cuda")[:, None] + (nk - nq)
    j = torch.arange(nk, device="cuda")[None]
    see = torch.ones(nq, nk, dtype=torch.bool, device="cuda")
    if s["causal"]:
        see &= j <= i
        if s["window"]:
            see &= i - j < s["window"]
    return see


def _exact_one(q, k, v, see, scale):
    """softmax(scale q k^T) v of the queries of one key head: q [group][nq][dim], k and v [nk][dim]; and the log-sum-exp."""
    some = see.any(1)
    a = (q @ k.t() * scale).masked_fill(~see, -math.inf)
    a = torch.where(some[:, None], a, torch.zeros_like(a))
    o = torch.softmax(a, 2) @ v * some[:, None]
    return o, torch.where(some, torch.logsumexp(a, 2), torch.full_like(a[..., 0], -math.inf))


def _exact_attention(s, grad):
    q, k, v = (s[n] if s["cu"] is not None else s[n].flatten(0, 1) for n in "qkv")
    outs = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in ((q, k, v) if grad else (q,))]
    lse = torch.full((s["heads"], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    if s["cu"] is not None:
        at = s["cu"].tolist()
        spans = [(a, b, a, b) for a, b in zip(at, at[1:])]
    else:
        spans = [(i * s["q_len"], (i + 1) * s["q_len"], i * s["k_len"], (i + 1) * s["k_len"]) for i in range(s["batch"])]
    group = s["heads"] // s["kv_heads"]
    for qa, qb, ka, kb in spans:
        if qa == qb or ka == kb:
            continue
        see = _exact_sight(qb - qa, kb - ka, s)
        for h in range(s["kv_heads"]):
            hs = slice(h * group, (h + 1) * group)
            one = [q[qa:qb, hs].double().transpose(0, 1).contiguous(), k[ka:kb, h].double().contiguous(),
                   v[ka:kb, h].double().contiguous()]
            if not grad:
                o, lse[hs, qa:qb] = _exact_one(*one, see, s["scale"])
                outs[0][qa:qb, hs] = o.transpose(0, 1)
                continue
            one = [t.requires_grad_() for t in one]
            do = s["do"].reshape(q.shape)[qa:qb, hs].double().transpose(0, 1)
            dq, dk, dv = torch.autograd.grad(_exact_one(*one, see, s["scale"])[0], one, do)
            outs[0][qa:qb, hs] = dq.transpose(0, 1)
            outs[1][ka:kb, h], outs[2][ka:kb, h] = dk, dv
    if grad:
        return dict(dq=outs[0].reshape(s["q"].shape), dk=outs[1].reshape(s["k"].shape), dv=outs[2].reshape(s["v"].shape))
    return dict(o=outs[0].reshape(s["q"].shape), lse=lse)


def _exact_draws(n, index, which, step, seed):
    """The 16-bit numbers by 16-bit limbs, so that no product passes 62 bits."""
    i = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)
    c = [i % 2 ** 32, torch.zeros_like(i) + (4 * index + which), torch.zeros_like(i) + step % 2 ** 32,
         torch.zeros_like(i) + (0x41440000 + step // 2 ** 32)]
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


def _exact_scaled(x, u, keep):
    """A 1-d tensor by blocks of 32: E4M3 elements as numbers, and the power-of-two scales."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % 32)).reshape(-1, 32)
    scale = torch.exp2(torch.ceil(torch.log2(b.abs().amax(1).clamp(min=1e-300) / 448)).clamp(min=-126.0))
    y = b.abs() / scale[:, None]
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    c = torch.round(y / step) if u is None else torch.floor(y / step + torch.nn.functional.pad(u, (0, -n % 32)).reshape(-1, 32))
    if keep:
        c = torch.where(y > 0, c.clamp(min=1.0), c)
    return torch.copysign(c * step, b).reshape(-1)[:n], scale


def _exact_adamw(s):
    out = {}
    for k, kind in enumerate(s["buffers"]):
        old = s["buffers"][kind]
        new = {key: [] for key in old}
        for i in range(s["count"]):
            t = s["tensors"][2 * i + k]
            n, width = t["param"].numel(), old["param"].shape[1]
            draws = (lambda which: _exact_draws(n, 2 * i + k, which, s["step"], s["seed"]) if s["rounding"] == "sr" else None)
            g = t["grad"].double().reshape(-1) * s["grad_scale"].double()
            m, v = t["m"].reshape(-1), t["v"].reshape(-1)
            if t["state"] == 8:
                m, r = (torch.repeat_interleave(torch.exp2(c.double() - 127), 32)[:n] * x.view(torch.float8_e4m3fn).double()
                        for x, c in ((m, t["m_scale"]), (v, t["v_scale"])))
                v = r ** 2
            m = BETA1 * m.double() + (1 - BETA1) * g
            v = BETA2 * v.double() + (1 - BETA2) * g ** 2
            p = t["param"].double().reshape(-1)
            p = p - LR * t["decay"] * p - LR * (m / (1 - BETA1 ** s["step"])) / (torch.sqrt(v / (1 - BETA2 ** s["step"])) + EPS_ADAM)
            if t["param"].dtype == torch.bfloat16 and s["rounding"] == "sr":
                step = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
                p = torch.copysign(torch.floor(p.abs() / step + draws(2)) * step, p)
            d = dict(param=p, m=m, v=v, copy=p)
            if t["state"] == 8:
                d["m"], d["m_scale"] = _exact_scaled(m, draws(0), False)
                d["v"], d["v_scale"] = _exact_scaled(torch.sqrt(v), draws(1), True)
            for key in new:
                small, fill = key.endswith("_scale"), 2.0 ** -126 if key.endswith("_scale") else 0.0
                full = (width // 32 if small else width) - d[key].numel()
                new[key].append(torch.nn.functional.pad(d[key], (0, full), value=fill))
        out[kind] = {key: torch.stack(x) for key, x in new.items()}
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(s)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    return _exact_attention(s, case["op"] == "attention_grad")
