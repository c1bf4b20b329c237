"""Norm and rotation of query and key heads, and their gradient, against the
definition in 64 bits.

Tolerances.  An output is rounded once to bf16 (2^-8 of its value) from binary32
values whose own error is at most some 20 roundings of 2^-24 of the head's
largest element: 2^-18 of that covers them.  A float32 gradient has the latter
alone.  The weights' gradients are sums of n products: binary32 partial sums of
at most a few hundred terms each, joined in a tree, so that 2^-24 * 512 of the sum
of magnitudes bounds them (2^-15)."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


EPS = 1e-6


def reference(x, w, at, freqs, interleaved, magnitude, eps=EPS):
    """y in 64 bits of x [tokens][heads][dim] (float64, may want a gradient)."""
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    if freqs is None:
        return x
    n = freqs.numel()
    t = (at.double()[:, None] * freqs)[:, None, :]
    c, s = torch.cos(t) * magnitude, torch.sin(t) * magnitude
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, v = a * c - b * s, b * c + a * s
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def close(got, want, rel, what):
    """|got - want| <= rel * |want| + 2^-18 of the head's largest."""
    got, want = got.double(), want.double()
    room = rel * want.abs() + 2.0 ** -18 * want.abs().amax(-1, keepdim=True) + 1e-30
    bad = ((got - want).abs() > room) | ~torch.isfinite(got)
    assert not bad.any(), "%s: %d of %d, worst %.3g" % (what, bad.sum(), bad.numel(), ((got - want).abs() / room).max())


def make(tokens, heads, kv, dim, dtype, seed, pad=0):
    """q and k as parts of one projection's output with `pad` more heads."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, heads + 2 * kv + pad, dim, generator=g, device="cuda") * torch.exp(
        torch.randn(dim, generator=g, device="cuda"))
    x = x.to(dtype)
    return x[:, :heads], x[:, heads:heads + kv], g


# (tokens, heads, kv_heads, dim, rot, interleaved, norm, dtype, weights' dtype)
B, F = torch.bfloat16, torch.float32
CASES = [(5, 8, 2, 128, 128, False, True, B, F), (5, 8, 2, 128, 128, True, True, B, B), (1, 1, 1, 8, 8, False, True, B, F),
         (3, 3, 1, 8, 2, True, False, B, F), (7, 5, 5, 40, 40, False, True, F, F), (33, 3, 3, 72, 36, False, True, B, F),
         (33, 3, 1, 72, 36, True, True, F, B), (130, 40, 8, 128, 64, False, True, B, F), (130, 40, 8, 128, 6, False, True, B, F),
         (17, 16, 2, 64, 64, False, False, B, F), (17, 16, 2, 64, 20, False, False, F, F), (9, 12, 4, 80, 80, False, True, B, F),
         (9, 12, 4, 80, 0, False, True, B, F), (2000, 10, 5, 96, 96, True, True, F, F), (5000, 2, 1, 64, 32, False, True, B, F),
         (700, 33, 7, 16, 12, False, True, B, F), (6000, 24, 24, 120, 120, False, True, B, B)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradient(nv, case):
    tokens, heads, kv, dim, rot, inter, norm, dtype, wt = case
    say("rope", *case)
    q, k, g = make(tokens, heads, kv, dim, dtype, 5)
    freqs = torch.rand(rot // 2, generator=g, device="cuda", dtype=torch.float64) if rot else None
    at = torch.randint(-1000, 1 << 22, (tokens,), generator=g, device="cuda")
    w = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(wt) for _ in range(2)] if norm else [None, None]
    mag = 1.0 if tokens % 2 else 1.34
    opts = dict(positions=at, q_weight=w[0], k_weight=w[1], eps=EPS, interleaved=inter, magnitude=mag)
    outs = nv.qk_rope(q, k, freqs, **opts)
    dys = [torch.randn(t.shape, generator=g, device="cuda").to(B) for t in (q, k)]
    dq, dk, dqw, dkw = nv.qk_rope_backward(*dys, freqs, q, k, **opts)
    again = nv.qk_rope_backward(*dys, freqs, q, k, **opts)
    for a, b in zip((dq, dk, dqw, dkw), again):
        assert a is None and b is None or torch.equal(a, b)  # a fixed order of sums
    for x, y, dy, dx, dw, wx, name in ((q, outs[0], dys[0], dq, dqw, w[0], "q"), (k, outs[1], dys[1], dk, dkw, w[1], "k")):
        xd = x.double().requires_grad_()
        wd = wx.double().requires_grad_() if norm else None
        want = reference(xd, wd, at, freqs, inter, mag)
        assert y.dtype == B and y.shape == x.shape
        close(y, want.detach(), 2.0 ** -8, "%s forward" % name)
        grads = torch.autograd.grad(want, [xd] + ([wd] if norm else []), dy.double())
        assert dx.dtype == dtype
        # cancellation: dx is what is left of a and h mean(a h), each of the size of |dy| |w| rstd
        rstd = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS) if norm else torch.ones_like(xd[..., :1])
        size = (dy.double().abs().amax(-1, keepdim=True) * mag * 2 ** 0.5 * rstd * (wd.detach().abs().max() if norm else 1.0) *
                (1 + (x.double() * rstd).abs().amax(-1, keepdim=True) if norm else 1.0))
        room = (2.0 ** -8 if dtype == B else 0.0) * grads[0].abs() + 2.0 ** -18 * size
        off = (dx.double() - grads[0]).abs()
        assert (off <= room).all(), "%s gradient: %.3g of what is allowed" % (name, (off / room).max())
        if norm:
            terms = (reference(dy.double(), None, -at, freqs, inter, mag) * x.double() * rstd).abs().sum((0, 1))
            off = (dw.double() - grads[1]).abs()
            assert dw.dtype == F and (off <= 2.0 ** -15 * terms).all(), "%s weight: %.3g" % (name, (off / terms).max())
        else:
            assert dw is None


# (dim, rot, interleaved): heads of up to 4, 8 and 16 lanes, with whole segments of 8 and with some cut short
LAYOUTS = [(64, 64, False), (56, 16, False), (32, 20, False), (64, 12, False), (48, 30, True), (128, 128, False), (88, 48, False),
           (80, 20, False), (128, 72, False), (128, 100, True), (72, 72, True), (128, 8, False), (128, 2, False)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [B, F], ids=str)
def test_layouts(nv, layout, norm, dtype):
    test_forward_and_gradient(nv, (21, 6, 3, *layout, norm, dtype, F))


def test_gradient_against_differences(nv):
    """The gradient's product with a direction is what the definition changes along it."""
    say("rope differences")
    q, k, g = make(12, 4, 2, 64, F, 3)
    freqs, _ = nv.rope_frequencies(32)
    w = [1 + 0.2 * torch.randn(64, generator=g, device="cuda") for _ in range(2)]
    at = torch.arange(12, device="cuda")
    dys = [torch.randn(t.shape, generator=g, device="cuda").to(B) for t in (q, k)]
    got = nv.qk_rope_backward(*dys, freqs, q, k, positions=at, q_weight=w[0], k_weight=w[1], eps=EPS)
    for x, dy, dx, dw, wx in ((q, dys[0], got[0], got[2], w[0]), (k, dys[1], got[1], got[3], w[1])):
        ex, ew = (torch.randn(t.shape, generator=g, device="cuda").double() for t in (x, wx))
        f = lambda e: (reference(x.double() + e * ex, wx.double() + e * ew, at, freqs, False, 1.0) * dy.double()).sum()  # noqa: E731
        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        have = (dx.double() * ex).sum() + (dw.double() * ew).sum()
        size = (dx.double() * ex).abs().sum() + (dw.double() * ew).abs().sum()
        assert (slope - have).abs() <= 1e-6 * size  # differences: 1e-10 of third derivatives; sums: 2^-24 each


def test_positions_are_the_places_in_sequences(nv):
    say("rope positions")
    q, k, g = make(24, 4, 2, 64, B, 4)
    freqs, mag = nv.rope_frequencies(64)
    assert mag == 1.0
    dense = nv.qk_rope(q.unflatten(0, (3, 8)), k.unflatten(0, (3, 8)), freqs)
    at = torch.arange(8, device="cuda").repeat(3)
    given = nv.qk_rope(q, k, freqs, positions=at)
    packed = nv.qk_rope(q, k, freqs, cu=torch.tensor([0, 8, 8, 16, 24], dtype=torch.int32, device="cuda"))
    for a, b, c in zip(dense, given, packed):
        assert torch.equal(a.flatten(0, 1), b) and torch.equal(b, c)


def test_far_positions(nv):
    """Angles keep their places at positions where a 32-bit product is off by radians."""
    say("rope far positions")
    q, k, g = make(64, 2, 1, 128, F, 6)
    freqs, _ = nv.rope_frequencies(128, base=10000.0)
    at = torch.randint(1 << 29, 1 << 40, (64,), generator=g, device="cuda")
    y = nv.qk_rope(q, k, freqs, positions=at)
    # the angle is at most 2^40 and is formed in 64 bits: within 2^-12 of a radian of the oracle's own
    for a, x in zip(y, (q, k)):
        want = reference(x.double(), None, at, freqs, False, 1.0)
        assert ((a.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * x.double().abs().amax(-1, keepdim=True)).all()


@pytest.mark.parametrize("cu,total", [([0, 3, 3, 10], 10), ([2, 5, 9], 12), ([4, 4], 6), ([0, 100], 7), ([0] * 90 + [5], 5)], ids=str)
def test_packed_tokens_of_no_sequence_are_left(nv, cu, total):
    say("rope packed", cu[:6], total)
    q, k, g = make(total, 4, 2, 64, B, 9)
    freqs, _ = nv.rope_frequencies(64)
    w = torch.ones(64, device="cuda")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    opts = dict(cu=cut, q_weight=w, k_weight=w, eps=EPS)
    outs = [torch.full_like(t, 7.0, memory_format=torch.contiguous_format) for t in (q, k)]
    nv.nvfp4_qk_rope(q, k, *outs, freqs, **opts)
    dys = [torch.randn(t.shape, generator=g, device="cuda").to(B) for t in (q, k)]
    dxs, dws = [torch.full_like(t, 7.0) for t in dys], [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    nv.nvfp4_qk_rope_backward(*dys, *dxs, freqs, q, k, dq_weight=dws[0], dk_weight=dws[1], **opts)
    at = torch.full((total,), -1)
    for a, b in zip(cu, cu[1:]):
        at[a:min(b, total)] = torch.arange(min(b, total) - a)
    inside = (at >= 0).cuda()
    at = at.cuda()
    for x, y, dy, dx, dw in zip((q, k), outs, dys, dxs, dws):
        assert (y[~inside] == 7.0).all() and (dx[~inside] == 7.0).all()
        xd, wd = x[inside].double().requires_grad_(), w.double().requires_grad_()
        want = reference(xd, wd, at[inside], freqs, False, 1.0)
        close(y[inside], want.detach(), 2.0 ** -8, "packed")
        ga, gw = torch.autograd.grad(want, (xd, wd), dy[inside].double())
        assert ((dw.double() - gw).abs() <= 2.0 ** -15 * (gw.abs() + inside.sum() * 16)).all()


def test_no_tokens(nv):
    say("rope of no tokens")
    freqs, _ = nv.rope_frequencies(64)
    w = torch.ones(64, device="cuda")
    q, k = torch.empty(0, 4, 64, dtype=B, device="cuda"), torch.empty(0, 2, 64, dtype=B, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    a, b = nv.qk_rope(q, k, freqs, cu=cu, q_weight=w, k_weight=w)
    assert a.shape == q.shape and b.shape == k.shape
    _, _, dw, _ = nv.qk_rope_backward(a, b, freqs, q, k, cu=cu, q_weight=w, k_weight=w)
    assert (dw == 0).all()


def test_in_place_strides_and_one_side(nv):
    say("rope in place")
    for dim, rot in ((128, 128), (72, 36)):
        q, k, g = make(50, 6, 3, dim, B, 11, pad=1)
        freqs, _ = nv.rope_frequencies(rot)
        w = torch.randn(dim, generator=g, device="cuda")
        at = torch.arange(50, device="cuda")
        opts = dict(positions=at, q_weight=w, k_weight=w)
        want = nv.qk_rope(q, k, freqs, **opts)
        alone = nv.qk_rope(q, None, freqs, positions=at, q_weight=w)
        assert torch.equal(alone[0], want[0]) and alone[1] is None
        dys = [torch.randn(t.shape, generator=g, device="cuda").to(B) for t in (q, k)]
        grads = nv.qk_rope_backward(*dys, freqs, q, k, **opts)
        dws = [torch.empty(dim, device="cuda") for _ in range(2)]
        nv.nvfp4_qk_rope_backward(*dys, *dys, freqs, q, k, dq_weight=dws[0], dk_weight=dws[1], **opts)  # in the gradients' place
        for a, b in zip(grads, [*dys, *dws]):
            assert torch.equal(a, b)
        nv.nvfp4_qk_rope(q, k, q, k, freqs, **opts)  # slices of one buffer, in their own place
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_broadcast_heads(nv):
    """An input that is one head, seen as many."""
    say("rope of expanded heads")
    x = torch.randn(5, 1, 64, device="cuda").to(B)
    freqs, _ = nv.rope_frequencies(64)
    at = torch.arange(5, device="cuda")
    y, _ = nv.qk_rope(x.expand(5, 12, 64), None, freqs, positions=at)
    z, _ = nv.qk_rope(x, None, freqs, positions=at)
    assert torch.equal(y, z.expand(5, 12, 64))


def test_far_offsets(nv):
    """Elements past 2^31 of a buffer are found: two tokens that far apart."""
    say("rope far offsets")
    step = (1 << 31) + 64
    big = torch.empty(step + 4096, dtype=B, device="cuda")
    q = big.as_strided((2, 2, 64), (step, 64, 1))
    q.copy_(torch.randn(2, 2, 64, device="cuda"))
    freqs, _ = nv.rope_frequencies(64)
    at = torch.tensor([3, 4], device="cuda")
    want, _ = nv.qk_rope(q.contiguous(), None, freqs, positions=at)
    got, _ = nv.qk_rope(q, None, freqs, positions=at)
    assert torch.equal(got, want)
    nv.nvfp4_qk_rope(q, None, q, None, freqs, positions=at)
    assert torch.equal(q, want)


def test_other_stream_and_graph(nv):
    say("rope on another stream, and captured")
    q, k, g = make(300, 8, 2, 128, B, 12)
    freqs, _ = nv.rope_frequencies(128)
    w = torch.randn(128, generator=g, device="cuda")
    opts = dict(q_weight=w, k_weight=w)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    want = nv.qk_rope(q, k, freqs, cu=cu, **opts)
    grads = nv.qk_rope_backward(*want, freqs, q, k, cu=cu, **opts)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = nv.qk_rope(q, k, freqs, cu=cu, stream=s, **opts)
    back = nv.qk_rope_backward(*got, freqs, q, k, cu=cu, stream=s, **opts)
    s.synchronize()
    for a, b in zip((*want, *grads), (*got, *back)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = nv.qk_rope(q, k, freqs, cu=cu, **opts)
        held_grads = nv.qk_rope_backward(*held, freqs, q, k, cu=cu, **opts)
    for turn in range(3):
        q.mul_(0.5 if turn else 1.0)
        graph.replay()
        want = nv.qk_rope(q, k, freqs, cu=cu, **opts)
        grads = nv.qk_rope_backward(*want, freqs, q, k, cu=cu, **opts)
        torch.cuda.synchronize()
        for a, b in zip((*want, *grads), (*held, *held_grads)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0)])
def test_frequencies(nv, scaling, factor):
    import math
    f, mag = nv.rope_frequencies(64, base=10000.0, scaling=scaling, factor=factor, original_length=2048)
    plain = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64, device="cuda")
    ratio = plain / f
    assert f.dtype == torch.float64 and f.shape == (32,)
    if scaling == "linear":
        assert torch.allclose(ratio, torch.full_like(ratio, factor))
    elif scaling == "ntk":
        assert abs(ratio[0] - 1) < 1e-12 and abs(ratio[-1] - factor) < 1e-9 * factor
    elif scaling == "yarn":
        turns = 2048 * plain / (2 * math.pi)
        assert torch.allclose(ratio[turns > 32], torch.ones_like(ratio[turns > 32]))
        assert torch.allclose(ratio[turns < 1], torch.full_like(ratio[turns < 1], factor))
        assert ((ratio > 1 - 1e-12) & (ratio < factor * (1 + 1e-12))).all() and abs(mag - (0.1 * math.log(32) + 1)) < 1e-12
    else:
        assert torch.allclose(ratio, torch.ones_like(ratio))
    if scaling != "yarn":
        assert mag == 1.0


def test_python_refusals(nv):
    say("rope refusals")
    q, k, g = make(8, 4, 2, 64, B, 1)
    freqs, _ = nv.rope_frequencies(64)
    w = torch.ones(64, device="cuda")
    at = torch.arange(8, device="cuda")
    bad = [dict(positions=at.int()), dict(positions=at[:7]), dict(positions=at, cu=torch.zeros(2, dtype=torch.int32, device="cuda")),
           dict(positions=at, q_weight=w), dict(positions=at, q_weight=w[:32], k_weight=w), dict(positions=at, q_weight=w, k_weight=w.to(B)),
           dict(cu=at), dict()]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            nv.qk_rope(q, k, freqs, **kw)
    for args in ((q, k.float(), freqs), (q, k[:7], freqs), (q, k[..., :32], freqs), (q, k, freqs.float()), (q.cpu(), k, freqs)):
        with pytest.raises((ValueError, TypeError)):
            nv.qk_rope(*args, positions=at)
    with pytest.raises(nv.Nvfp4Error):
        nv.qk_rope(q, k, None, positions=at)  # nothing to do
    with pytest.raises(ValueError):
        nv.qk_rope_backward(q, k, freqs, positions=at, q_weight=w, k_weight=w)  # without what was normalised
