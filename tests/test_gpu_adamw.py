"""The AdamW step on the GPU against the formulas in 64 bits, with the random
numbers of the stochastic rounding from a Philox written here and checked
against the published vectors.

Tolerances count roundings of binary32 (2^-24 of the value each): a state takes
at most 4, the update 12.  A rounding to 8 bits or bf16 is checked as a choice:
the stored neighbour has to be the one that the exact value and its random
number give, but for values within the binary32 error of the border."""
import os

import numpy as np
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ULP = 2.0 ** -24
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


def philox(c, k):
    """Philox4x32-10 on arrays of 32-bit words held in uint64."""
    c, (k0, k1), low = [np.asarray(x, np.uint64) for x in c], k, np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def test_philox_here_is_the_published_one():
    for line in open(os.path.join(HERE, "golden", "philox4x32_10_kat.txt")):
        if line.strip() and not line.startswith("#"):
            w = [int(x, 16) for x in line.split()]
            assert [int(x) for x in philox(w[:4], w[4:6])] == w[6:]


def uniforms(n, index, which, step, seed):
    group = np.arange((n + 7) // 8, dtype=np.uint64)
    one = np.ones_like(group)
    w = philox([group & np.uint64(0xFFFFFFFF), one * np.uint64(4 * index + which), one * np.uint64(step & 0xFFFFFFFF),
                one * np.uint64(0x41440000 + (step >> 32))], (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([x >> np.uint64(16 * s) & np.uint64(0xFFFF) for x in w for s in (0, 1)], 1)
    return halves.reshape(-1)[:n].astype(np.float64) / 65536


def e4m3_parts(codes):
    """(magnitude, step to the next) of E4M3 bytes."""
    c = codes.astype(np.int64) & 127
    e = np.maximum(c >> 3, 1)
    return np.where(c >> 3 > 0, 8 + (c & 7), c & 7) * 2.0 ** (e - 10), 2.0 ** (e - 10)


def decode(codes, scales):
    v, _ = e4m3_parts(codes)
    return np.where(codes & 128, -v, v) * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32)[:codes.size]


def check_blocks(codes, scales, x, tol, u, positive, what):
    """That an 8-bit state holds x (64-bit; binary32 values are within tol of it)."""
    n = x.size
    full, slack = np.zeros(-(-n // 32) * 32), np.zeros(-(-n // 32) * 32)
    full[:n], slack[:n] = np.abs(x), tol
    top, most = full.reshape(-1, 32).max(1), (full + slack).reshape(-1, 32).max(1)
    least = (full - slack).reshape(-1, 32).max(1)
    e = scales.astype(np.int64) - 127
    assert (e >= -126).all() and (least <= 448 * 2.0 ** e).all(), what + ": a block's scale is too small"
    assert ((e == -126) | (most > 448 * 2.0 ** (e - 1.0))).all(), what + ": a block's scale is too large"
    del top
    s = np.repeat(2.0 ** e, 32)[:n]
    y, ty = np.abs(x) / s, tol / s
    got, _ = e4m3_parts(codes)
    # the step of the value's binade (of the wider one next to a power of two)
    quantum = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y + ty, 2.0 ** -6))), -6) - 3)
    # binary32 keeps t + u (below 17) to 2^-20
    eps = ty / quantum + 2.0 ** -20
    if u is None:
        low, high = y / quantum - 0.5 - eps, y / quantum + 0.5 + eps
    else:
        low, high = y / quantum + u - 1 - eps, y / quantum + u + eps
    c = got / quantum
    ok = (c >= low) & (c <= high)
    if positive:
        ok |= (y > 0) & (c == 1) & (low <= 1)
        assert (got[y > ty] > 0).all(), what + ": a positive value is stored as zero"
    # one binade lower where the value is within its error of the border
    assert ok.all(), "%s: %d elements hold the wrong neighbour" % (what, np.count_nonzero(~ok))
    assert ((codes >= 128) == np.signbit(x))[np.abs(x) > tol].all(), what + ": sign"


def bf16(x):
    return x.to(torch.bfloat16)


def make(nv, g, n, tp, tg, bits, copy, amax, wd, offset):
    """A tensor of n elements starting `offset` elements into its buffers."""
    def buf(values, dtype):
        b = torch.full((n + offset + 40,), 3.0, device="cuda").to(dtype)
        b[offset:offset + n] = values.to(dtype)
        return b[offset:offset + n]
    r = 1e-3 * torch.exp(torch.randn(n, generator=g, device="cuda"))
    p = buf(0.02 * torch.randn(n, generator=g, device="cuda"), tp)
    gr = buf(r * torch.randn(n, generator=g, device="cuda"), tg)
    c = buf(torch.zeros(n, device="cuda"), torch.bfloat16) if copy else None
    a = torch.zeros(1, device="cuda") if amax else None
    if bits == 32:
        m, v = buf(0.3 * r * torch.randn(n, generator=g, device="cuda"), torch.float32), buf(r * r, torch.float32)
        return nv.AdamWTensor(p, gr, m, v, weight_decay=wd, copy=c, amax=a)
    m, v = (buf(torch.randint(0, 127, (n,), generator=g, device="cuda"), torch.uint8) for _ in range(2))
    m ^= (torch.randint(0, 2, (n,), generator=g, device="cuda") * 128).to(torch.uint8)
    ms, vs = (torch.randint(105, 110, (-(-n // 32),), generator=g, device="cuda").to(torch.uint8) for _ in range(2))
    return nv.AdamWTensor(p, gr, m, v, ms, vs, wd, c, a)


def host(t):
    return None if t is None else t.detach().cpu()


def snapshot(t):
    return {k: host(getattr(t, k)).clone() if getattr(t, k) is not None else None
            for k in ("param", "grad", "m", "v", "m_scale", "v_scale")}


HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, seed=0x123456789)


def check(old, t, index, step, rounding, gscale, what):
    n = old["param"].numel()
    if n == 0:
        return
    sr, bits8 = rounding == "sr", old["m_scale"] is not None
    f = np.float32
    b1, b2, lr, eps = HYPER["beta1"], HYPER["beta2"], float(f(HYPER["lr"])), float(f(HYPER["eps"]))
    p, g = old["param"].double().numpy(), old["grad"].double().numpy() * gscale
    if bits8:
        m = decode(old["m"].numpy(), old["m_scale"].numpy())
        v = decode(old["v"].numpy(), old["v_scale"].numpy()) ** 2
    else:
        m, v = old["m"].double().numpy(), old["v"].double().numpy()
    tm = 4 * ULP * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    tv = 6 * ULP * v
    draws = (lambda which: uniforms(n, index, which, step, HYPER["seed"]) if sr else None)
    if bits8:
        check_blocks(host(t.m).numpy(), host(t.m_scale).numpy(), m, tm + 1e-45, draws(0), False, what + " m")
        check_blocks(host(t.v).numpy(), host(t.v_scale).numpy(), np.sqrt(v), 4 * ULP * np.sqrt(v) + 1e-45, draws(1), True, what + " r")
    else:
        assert (np.abs(host(t.m).double().numpy() - m) <= tm).all(), what + " m"
        assert (np.abs(host(t.v).double().numpy() - v) <= tv).all(), what + " v"
    c1, c2 = 1 - b1 ** step, np.sqrt(1 - b2 ** step)
    den = np.sqrt(v) / c2 + eps
    upd = lr * (m / c1) / den
    tp = 4 * ULP * np.abs(p) + 12 * ULP * np.abs(upd) + lr * tm / c1 / den
    want = p - lr * t.weight_decay * p - upd
    got = host(t.param).double().numpy()
    if t.param.dtype == torch.float32:
        assert (np.abs(got - want) <= tp).all(), what + " param"
    else:
        q = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want) + tp, 2.0 ** -126))) - 7)
        lo, hi = ((np.abs(want) - tp) / q, (np.abs(want) + tp) / q)
        c, u = np.abs(got) / q, draws(2)
        ok = (c >= lo - 0.5) & (c <= hi + 0.5) if u is None else (c > lo + u - 1 - 2.0 ** -16) & (c <= hi + u + 2.0 ** -16)
        assert ok.all(), what + " param: %d elements hold the wrong neighbour" % np.count_nonzero(~ok)
    if t.copy is not None:
        src = host(t.param)
        assert torch.equal(host(t.copy), bf16(src) if src.dtype == torch.float32 else src), what + " copy"
    if t.amax is not None:
        src = host(t.copy) if t.copy is not None else host(t.param)
        assert host(t.amax).item() == src.float().abs().max().item(), what + " amax"


KINDS = [(tp, tg, bits) for tp in (torch.float32, torch.bfloat16) for tg in (torch.float32, torch.bfloat16)
         for bits in (32, 8)]
SIZES = [1, 7, 8, 31, 32, 33, 255, 4096, 4097, 12345]


@pytest.mark.parametrize("rounding", ["rtn", "sr"])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_every_type_and_size(nv, kind, rounding):
    """One call over tensors of many sizes, aligned and not, with and without copies and maxima."""
    tp, tg, bits = KINDS[kind]
    say("adamw", tp, tg, bits, rounding)
    g = torch.Generator(device="cuda").manual_seed(kind)
    ts = [make(nv, g, n, tp, tg, bits, i % 2 == 1, i % 3 == 1, 0.1 * (i % 4), (0, 1, 8)[i % 3]) for i, n in enumerate(SIZES * 2)]
    old = [snapshot(t) for t in ts]
    bufs = [(x._base, x.storage_offset(), x.numel(), x._base.clone()) for t in ts for x in (t.param, t.m, t.v, t.copy)
            if x is not None]
    scale = torch.tensor([0.75], device="cuda")
    nv.adamw(ts, step=7, rounding=rounding, grad_scale=scale, **HYPER)
    torch.cuda.synchronize()
    for i, (o, t) in enumerate(zip(old, ts)):
        check(o, t, i, 7, rounding, 0.75, "tensor %d (%d)" % (i, t.param.numel()))
    for b, at, n, before in bufs:  # nothing outside the tensors was written
        assert torch.equal(b[:at], before[:at]) and torch.equal(b[at + n:], before[at + n:])


def test_many_tensors_of_mixed_kinds(nv):
    """More tensors than one launch takes, empty ones among them."""
    g = torch.Generator(device="cuda").manual_seed(3)
    sizes = [(i * 977) % 5000 for i in range(95)]
    sizes[10] = sizes[40] = sizes[79] = sizes[94] = 0
    ts = [make(nv, g, n, *KINDS[i % 8], copy=False, amax=False, wd=0.1, offset=0) for i, n in enumerate(sizes)]
    old = [snapshot(t) for t in ts]
    plan = nv.AdamWList(ts)
    nv.adamw(plan, step=1, rounding="sr", **HYPER)
    torch.cuda.synchronize()
    for i, (o, t) in enumerate(zip(old, ts)):
        check(o, t, i, 1, "sr", 1.0, "tensor %d" % i)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_from_zero(nv, bits):
    """Twenty steps from zero states; each is checked from the state before it.  The step number is wide."""
    g = torch.Generator(device="cuda").manual_seed(4)
    p, gr = 0.02 * torch.randn(1000, generator=g, device="cuda"), torch.zeros(1000, device="cuda")
    t = nv.adamw_tensor(p, gr, state_bits=bits, weight_decay=0.1)
    plan = nv.AdamWList([t])
    for step in list(range(1, 20)) + [2 ** 40 + 5]:
        gr.copy_(1e-3 * torch.randn(1000, generator=g, device="cuda"))
        if step == 3:
            gr.zero_()
        if step == 5:
            gr[::2] = 0
        old = snapshot(t)
        nv.adamw(plan, step=step, rounding="sr", **HYPER)
        check(old, t, 0, step, "sr", 1.0, "step %d" % step)
    m, v = nv.adamw_state_values(t)
    assert torch.isfinite(m).all() and (v >= 0).all()


def test_extreme_values(nv):
    """Zero gradients on zero states leave the parameters but for the decay; huge and tiny gradients stay finite."""
    p = torch.ones(320, device="cuda")
    for scale in (0.0, 1e-30, 1e-12, 1e6, 1e15):
        for bits in (32, 8):
            q = p.clone()
            t = nv.adamw_tensor(q, torch.full((320,), scale, device="cuda"), state_bits=bits)
            for step in (1, 2, 3):
                nv.adamw([t], lr=1e-3, step=step, rounding="sr", seed=1)
            assert torch.isfinite(q).all()
            # each step moves by at most lr * (1 - beta1) / sqrt(1 - beta2) scaled by the corrections: below 4 lr here
            assert (q - p).abs().max().item() <= 3 * 4e-3, (scale, bits)
            if scale == 0.0:
                assert torch.equal(q, p)


def test_stochastic_rounding_is_unbiased(nv):
    """bf16 params moved by a hundredth of their step: the mean over many elements moves by that much."""
    n = 1 << 18
    p = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    t = nv.adamw_tensor(p, torch.ones(n, device="cuda"))
    nv.adamw([t], lr=2.0 ** -8 / 100, beta1=0.0, beta2=0.0, step=1, rounding="sr", seed=99)
    # below 1 the step is 2^-8: a hundredth of the elements moves by one; standard deviation sqrt(0.01 / n)
    moved = (p.float() < 1).float().mean().item()
    assert abs(moved - 0.01) <= 5 * (0.01 / n) ** 0.5 + 2.0 ** -16
    q = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    nv.adamw([nv.adamw_tensor(q, torch.ones(n, device="cuda"))], lr=2.0 ** -8 / 100, beta1=0.0, beta2=0.0, step=1)
    assert (q == 1).all()


def test_amax_serves_the_quantiser(nv):
    """The maximum of the bf16 copy is what a weight's quantisation takes as given."""
    g = torch.Generator(device="cuda").manual_seed(6)
    p = 0.02 * torch.randn(256, 512, generator=g, device="cuda")
    copy, amax = torch.empty(256, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    t = nv.adamw_tensor(p, torch.randn(256, 512, generator=g, device="cuda"), copy=copy, amax=amax)
    nv.adamw([t], lr=1e-3, step=1)
    want = nv.quantize(copy, [nv.QuantSpec.of("2d")])[0]
    out = nv.empty_qtensor(256, 512, nv.SCALE_2D16)
    out.amax.copy_(amax)
    nv.nvfp4_quantize(copy, [nv.QuantSpec.of("2d", amax_given=True)], [out], nv.new_workspace())
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)


def test_repeats_graph_and_stream(nv):
    """The same state and seed give the same bits, on any stream and from a graph."""
    g = torch.Generator(device="cuda").manual_seed(8)
    ts = [make(nv, g, n, *KINDS[i % 8], copy=False, amax=False, wd=0.1, offset=0) for i, n in enumerate([5000, 77, 4096, 33] * 2)]
    plan = nv.AdamWList(ts)
    keys = ("param", "m", "v", "m_scale", "v_scale")
    start = [{k: getattr(t, k).clone() for k in keys if getattr(t, k) is not None} for t in ts]

    def reset():
        for t, s in zip(ts, start):
            for k, x in s.items():
                getattr(t, k).copy_(x)

    def state():
        torch.cuda.synchronize()
        return [x.clone() for t in ts for k in keys for x in [getattr(t, k)] if x is not None]

    nv.adamw(plan, step=3, rounding="sr", **HYPER)
    want = state()
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nv.adamw(plan, step=3, rounding="sr", stream=side, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(want, state()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.adamw(plan, step=3, rounding="sr", **HYPER)
    for _ in range(3):
        reset()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, state()))


def test_replaced_gradients(nv):
    p = torch.zeros(64, device="cuda")
    plan = nv.AdamWList([nv.adamw_tensor(p, torch.zeros(64, device="cuda"))])
    plan.set_grad(0, torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    nv.adamw(plan, lr=0.5, step=1)
    # the first step moves by lr against the gradient's sign, eps aside
    assert (p + 0.5).abs().max().item() <= 0.5 * (1e-8 + 16 * ULP)
    with pytest.raises(ValueError):
        plan.set_grad(0, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        plan.set_grad(0, torch.ones(64, dtype=torch.float16, device="cuda"))
    assert plan.tensors[0].grad.dtype == torch.bfloat16
