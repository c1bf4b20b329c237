"""Attention and its gradient on the GPU against the formulas in 64 bits.

Bounds are derived per element from the magnitudes that go into it: a bf16
rounding (of a probability, of a score's gradient, of an output) is off by at
most 2^-8 of the value, a binary32 sum of n products by n 2^-24 of the sum of
their magnitudes, and an error d of a score moves its probability by the factor
exp(d)."""
import math

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


def _rand(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _see(nq, nk, causal, window):
    i = torch.arange(nq, device="cuda")[:, None] + (nk - nq)
    j = torch.arange(nk, device="cuda")[None]
    s = torch.ones(nq, nk, dtype=torch.bool, device="cuda")
    if causal:
        s &= j <= i
        if window:
            s &= j > i - window
    return s


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _over(got, want, bound):
    assert torch.isfinite(got).all()
    return ((got.double() - want).abs() - bound).max().item() if got.numel() else 0.0


def _check_sequence(q, k, v, do, o, lse, dq, dk, dv, see, scale, what):
    """One sequence: [len][heads][dim] tensors, lse [heads][len]; heads one key head at a time."""
    group = q.shape[1] // k.shape[1]
    nq, nk, dim = q.shape[0], k.shape[0], q.shape[2]
    some = see.any(1)
    for hk in range(k.shape[1]):
        hs = slice(hk * group, (hk + 1) * group)
        Q, K, V = q[:, hs].double().transpose(0, 1).contiguous(), k[:, hk].double(), v[:, hk].double()
        s = torch.matmul(Q, _t(K)) * scale
        # a score's own error: dim products, the scaling and the conversion to powers of two
        ds = (dim + 8) * F * scale * torch.matmul(Q.abs(), _t(K.abs())) + 4 * F * s.abs()
        s = s.masked_fill(~see, -math.inf)
        want = torch.logsumexp(s, 2) if nk else torch.full((group, nq), -math.inf, dtype=torch.float64, device="cuda")
        want = torch.where(some, want, torch.full_like(want, -math.inf))
        d = ds.masked_fill(~see, 0).amax(2) if nk else torch.zeros_like(want)
        got = lse[hs].double()
        assert torch.equal(got == -math.inf, (~some).expand_as(got)), what + ": rows that see nothing"
        fin = some.expand_as(got)
        # the sum's additions: 1/32 of the keys in a lane, and the exponentials' and logarithm's last bits
        bound = d + (nk / 32 + 64) * F + 8 * F * want.abs()
        assert _over(got[fin], want[fin], bound[fin]) <= 0, what + ": lse"
        p = torch.where(see, torch.exp(s - torch.where(some, want, torch.zeros_like(want))[..., None]), 0.0)
        rel = 2 * d + (nk / 32 + 80) * F
        O = torch.matmul(p, V)
        bound = (BF + rel)[..., None] * torch.matmul(p, V.abs()) + nk * F * torch.matmul(p, V.abs())
        go = o[:, hs].transpose(0, 1)
        over = _over(go, O, bound + BF * (O.abs() + bound))
        assert over <= 0, "%s: o is %g over its bound" % (what, over)
        assert (go[:, ~some] == 0).all()
        if do is None:
            continue
        # the gradient on the o and lse that it was given
        G, Og = do[:, hs].double().transpose(0, 1).contiguous(), o[:, hs].double().transpose(0, 1)
        L = torch.where(some.expand_as(got), got, torch.zeros_like(got))
        p = torch.where(see, torch.exp(s - L[..., None]), 0.0)
        rel = (ds + (8 * F * (s.masked_fill(~see, 0).abs() + L.abs()[..., None])) + 16 * F) * see
        delta = (G * Og).sum(2, keepdim=True)
        dp = torch.matmul(G, _t(V))
        e = (dim + 8) * F * (torch.matmul(G.abs(), _t(V.abs())) + (G * Og).abs().sum(2, keepdim=True))
        S = p * (dp - delta)
        es = S.abs() * (rel + BF + 4 * F) + p * (1 + rel) * e * (1 + BF)
        # the products' own binary32 sums: at most all queries of the group, or all keys
        n = (nq * group + nk) * F
        tests = [("dv", dv[:, hk], torch.matmul(_t(p), G).sum(0),
                  (torch.matmul(_t(p * (BF + rel)), G.abs()) + n * torch.matmul(_t(p), G.abs())).sum(0)),
                 ("dk", dk[:, hk], scale * torch.matmul(_t(S), Q).sum(0),
                  scale * (torch.matmul(_t(es), Q.abs()) + n * torch.matmul(_t(S.abs()), Q.abs())).sum(0)),
                 ("dq", dq[:, hs].transpose(0, 1), scale * torch.matmul(S, K),
                  scale * (torch.matmul(es, K.abs()) + n * torch.matmul(S.abs(), K.abs())))]
        for name, x, w, b in tests:
            over = _over(x, w, b + (BF + 4 * F) * (w.abs() + b) + 1e-38)
            assert over <= 0, "%s: %s is %g over its bound" % (what, name, over)


def _run(nv, q, k, v, do, **opts):
    o, lse = nv.attention(q, k, v, **opts)
    return (o, lse) + tuple(nv.attention_backward(do, q, k, v, o, lse, **opts))


CASES = [  # batch, queries, keys, heads, key heads, dim, causal, window
    (1, 1, 1, 1, 1, 64, True, 0), (2, 1, 77, 4, 2, 128, True, 0), (1, 1, 1000, 5, 1, 64, False, 0),
    (1, 31, 33, 2, 2, 8, True, 0), (2, 64, 64, 4, 4, 64, True, 0), (1, 65, 63, 3, 1, 72, True, 0),
    (1, 100, 40, 2, 1, 128, True, 0), (1, 128, 128, 1, 1, 128, False, 0), (3, 129, 257, 2, 1, 128, True, 0),
    (1, 300, 200, 2, 2, 40, True, 17), (1, 257, 513, 6, 2, 96, True, 64), (1, 500, 500, 2, 1, 128, True, 1),
    (1, 640, 640, 8, 2, 128, True, 100), (1, 1000, 777, 2, 1, 64, False, 0), (1, 1025, 2049, 4, 1, 128, True, 0),
    (1, 3, 5000, 2, 1, 128, True, 0), (2, 1, 4096, 8, 2, 64, True, 0), (1, 200, 3000, 4, 1, 80, False, 0),
    (1, 2100, 300, 8, 1, 64, False, 0), (1, 1, 3333, 3, 1, 128, True, 1500), (1, 900, 2600, 2, 1, 128, True, 1300),
    (1, 511, 1, 2, 1, 128, False, 0), (1, 130, 1, 2, 1, 64, True, 0), (2, 383, 385, 2, 1, 120, True, 1000)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_dense(nv, case):
    b, nq, nk, h, hk, dim, causal, window = case
    say("attention", case)
    g = torch.Generator(device="cuda").manual_seed(nq * 1000 + nk)
    q, k, v = _rand(g, b, nq, h, dim), _rand(g, b, nk, hk, dim), _rand(g, b, nk, hk, dim)
    do = _rand(g, b, nq, h, dim, scale=1e-3)
    o, lse, dq, dk, dv = _run(nv, q, k, v, do, causal=causal, window=window)
    see = _see(nq, nk, causal, window)
    for i in range(b):
        _check_sequence(q[i], k[i], v[i], do[i], o[i], lse[:, i * nq:(i + 1) * nq], dq[i], dk[i], dv[i], see, dim ** -0.5,
                        "sequence %d" % i)


PACKED = [  # query lengths, key lengths, heads, key heads, dim, causal, window
    ([5, 0, 130, 1, 64], None, 4, 2, 64, True, 0), ([200, 33, 7], [100, 70, 0], 2, 1, 128, True, 0),
    ([0, 300], [40, 500], 4, 1, 128, True, 50), ([64, 64, 64], [64, 1, 130], 2, 2, 80, False, 0), ([0, 0], [3, 0], 1, 1, 64, True, 0),
    ([1] * 40, None, 2, 1, 64, True, 0), ([3, 0, 60], [2500, 100, 1300], 2, 1, 128, True, 0),
    ([1500, 2, 0], [200, 3000, 5], 6, 1, 64, False, 0)]


@pytest.mark.parametrize("case", PACKED, ids=str)
def test_packed(nv, case):
    """Packed sequences, empty ones among them, in buffers whose other tokens hold NaN and stay as they are."""
    nq, nk, h, hk, dim, causal, window = case
    nk = nk or nq
    say("packed attention", case)
    g = torch.Generator(device="cuda").manual_seed(sum(nq) + 7 * sum(nk))
    nan = float("nan")

    def packed(lens, heads, scale=1.0):
        t = torch.full((sum(lens) + 9, heads, dim), nan, dtype=torch.bfloat16, device="cuda")
        t[4:4 + sum(lens)] = _rand(g, sum(lens), heads, dim, scale=scale)
        return t

    q, k, v, do = packed(nq, h), packed(nk, hk), packed(nk, hk), packed(nq, h, 1e-3)
    cq, ck = ([4 + sum(x[:i]) for i in range(len(x) + 1)] for x in (nq, nk))
    opts = dict(causal=causal, window=window, cu_q=torch.tensor(cq, dtype=torch.int32, device="cuda"),
                cu_k=torch.tensor(ck, dtype=torch.int32, device="cuda"), max_q=max(max(nq), 1), max_k=max(max(nk), 1))
    o, lse = torch.full_like(q, 7.0), torch.full((h, q.shape[0]), 7.0, device="cuda")
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ws = nv.new_attention_workspace(q, k, v, **opts)
    nv.nvfp4_attention(q, k, v, o, lse, workspace=ws, **opts)
    nv.nvfp4_attention_backward(do, q, k, v, o, lse, dq, dk, dv, ws, **opts)
    for i in range(len(nq)):
        a, b = slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1])
        _check_sequence(q[a], k[b], v[b], do[a], o[a], lse[:, a], dq[a], dk[b], dv[b], _see(nq[i], nk[i], causal, window),
                        dim ** -0.5, "sequence %d" % i)
    for t, c in ((o, cq), (dq, cq), (dk, ck), (dv, ck)):
        assert (t[:c[0]] == 7).all() and (t[c[-1]:] == 7).all(), "tokens of no sequence were written"
    assert (lse[:, :cq[0]] == 7).all() and (lse[:, cq[-1]:] == 7).all()


SHARED = [  # passes split into parts at short lengths: batch, queries, keys, heads, key heads, dim, causal, window
    (1, 260, 260, 8, 1, 128, True, 0), (2, 256, 256, 16, 4, 64, True, 0), (1, 700, 129, 10, 2, 72, False, 0),
    (3, 300, 310, 20, 4, 128, True, 90), (1, 2000, 140, 6, 1, 64, True, 0), (1, 96, 1100, 12, 1, 128, True, 33)]


@pytest.mark.parametrize("case", SHARED, ids=str)
def test_shared_key_heads(nv, case):
    test_dense(nv, case)


@pytest.mark.parametrize("dim,h,hk", [(64, 12, 12), (128, 10, 1), (64, 8, 2)])
def test_packed_order(nv, dim, h, hk):
    """Many documents of uneven lengths under a maximum above all of them, as long as the tokens or longer."""
    say("packed attention", dim, h, hk)
    lens = [307, 0, 88, 1, 523, 129, 64, 128, 343, 16, 256, 9]
    g = torch.Generator(device="cuda").manual_seed(dim + h)
    n = sum(lens)
    q, k, v, do = _rand(g, n, h, dim), _rand(g, n, hk, dim), _rand(g, n, hk, dim), _rand(g, n, h, dim, scale=1e-3)
    at = [sum(lens[:i]) for i in range(len(lens) + 1)]
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    for most, window in ((523, 0), (n, 200), (1 << 30, 0)):
        o, lse, dq, dk, dv = _run(nv, q, k, v, do, causal=True, window=window, cu_q=cu, cu_k=cu, max_q=most, max_k=most)
        for i, m in enumerate(lens):
            a = slice(at[i], at[i + 1])
            _check_sequence(q[a], k[a], v[a], do[a], o[a], lse[:, a], dq[a], dk[a], dv[a], _see(m, m, True, window),
                            dim ** -0.5, "maximum %d, sequence %d" % (most, i))


def test_bad_offsets_stay_inside(nv):
    """Offsets that descend or leave the tokens are clamped: nothing faults, and sequences that are sound are right."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (_rand(g, 100, 2, 64) for _ in range(3))
    cu = torch.tensor([0, 50, 40, 1000, -5], dtype=torch.int32, device="cuda")
    opts = dict(cu_q=cu, cu_k=cu, max_q=64, max_k=64)
    o, lse, dq, dk, dv = _run(nv, q, k, v, q, **opts)
    torch.cuda.synchronize()
    want = nv.attention(q[None, :50], k[None, :50], v[None, :50])[0][0]
    assert torch.equal(o[:40], want[:40])


def test_layouts(nv):
    """Fused projections, head-major tensors and broadcast key heads give the contiguous tensors' bits."""
    g = torch.Generator(device="cuda").manual_seed(2)
    b, n, h, dim = 2, 200, 4, 64
    qkv = _rand(g, b, n, 3, h, dim)
    q, k, v = qkv.unbind(2)
    do = _rand(g, b, h, n, dim, scale=1e-3).transpose(1, 2)
    want = _run(nv, q.contiguous(), k.contiguous(), v.contiguous(), do.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(_run(nv, q, k, v, do), want))
    major = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    assert all(torch.equal(x, y) for x, y in zip(_run(nv, *major, do), want))
    one = k[:, :, :1]
    wide = [t.expand(b, n, h, dim) for t in (one, v[:, :, :1])]
    assert all(torch.equal(x, y) for x, y in zip(_run(nv, q, *wide, do), _run(nv, q, *[t.contiguous() for t in wide], do)))
    same = k[:1].expand(b, n, h, dim)
    assert all(torch.equal(x, y) for x, y in zip(_run(nv, q, same, v, do), _run(nv, q, same.contiguous(), v, do)))


def test_strided_outputs(nv):
    """dq, dk and dv written side by side into the gradient of a fused projection."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, h, dim = 150, 4, 80
    qkv, do = _rand(g, 1, n, 3, h, dim), _rand(g, 1, n, h, dim, scale=1e-3)
    q, k, v = qkv.unbind(2)
    o, lse, dq, dk, dv = _run(nv, q, k, v, do)
    grad = torch.full((1, n, 3, h, dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")[..., :dim]
    nv.nvfp4_attention_backward(do, q, k, v, o, lse, *grad.unbind(2), nv.new_attention_workspace(q, k, v))
    assert torch.equal(grad, torch.stack([dq, dk, dv], 2))
    assert (grad._base[..., dim:] == 7).all()


def test_large_scores(nv):
    """Scores up to some thousands, where only differences to the maximum can be raised: one key takes all the weight."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = _rand(g, 1, 200, 2, 64, scale=30), _rand(g, 1, 200, 2, 64, scale=30), _rand(g, 1, 200, 2, 64)
    do = _rand(g, 1, 200, 2, 64, scale=1e-3)
    o, lse, dq, dk, dv = _run(nv, q, k, v, do)
    _check_sequence(q[0], k[0], v[0], do[0], o[0], lse, dq[0], dk[0], dv[0], _see(200, 200, True, 0), 0.125, "large scores")


def test_rising_scores(nv):
    """Keys whose scores rise along the sequence, so that the running maximum moves in every tile."""
    n, dim = 700, 64
    k = torch.zeros(1, n, 1, dim, device="cuda")
    k[0, :, 0, 0] = torch.arange(n, device="cuda") / 8
    q = torch.zeros(1, n, 1, dim, device="cuda")
    q[..., 0] = 8
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, do = q.to(torch.bfloat16), k.to(torch.bfloat16), _rand(g, 1, n, 1, dim), _rand(g, 1, n, 1, dim, scale=1e-3)
    o, lse, dq, dk, dv = _run(nv, q, k, v, do, causal=False)
    _check_sequence(q[0], k[0], v[0], do[0], o[0], lse, dq[0], dk[0], dv[0], _see(n, n, False, 0), 0.125, "rising scores")


def test_gradient_against_differences(nv):
    """d/dt of sum(do * attention(x + t z)) by central differences in 64 bits is sum(dx * z), to the bf16 roundings."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n, h, dim = 90, 2, 64
    q, k, v, do = (_rand(g, 1, n, h, dim) for _ in range(4))
    grads = _run(nv, q, k, v, do)[2:]
    see = _see(n, n, True, 0)

    def value(q, k, v):
        q, k, v = (t[0].transpose(0, 1) for t in (q, k, v))
        s = (torch.matmul(q, _t(k)) * dim ** -0.5).masked_fill(~see, -math.inf)
        return (torch.matmul(torch.softmax(s, 2), v).transpose(0, 1) * do[0].double()).sum().item()

    at = [t.double() for t in (q, k, v)]
    for i, grad in enumerate(grads):
        z = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        moved = [[t + (s * 1e-5 * z if j == i else 0) for j, t in enumerate(at)] for s in (1, -1)]
        want = (value(*moved[0]) - value(*moved[1])) / 2e-5
        # n h dim terms, each off by a few bf16 roundings of random sign
        slack = 6 * 4 * BF * (grad.double() * z).norm().item()
        assert abs((grad.double() * z).sum().item() - want) <= slack, "qkv"[i]


def test_repeats_graph_and_stream(nv):
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v, do = _rand(g, 1, 300, 4, 64), _rand(g, 1, 300, 2, 64), _rand(g, 1, 300, 2, 64), _rand(g, 1, 300, 4, 64)
    want = _run(nv, q, k, v, do)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = nv.attention(q, k, v, stream=side)
    got = (o, lse) + tuple(nv.attention_backward(do, q, k, v, o, lse, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(nv, q, k, v, do)
    for i in range(4):
        q.copy_(_rand(g, 1, 300, 4, 64))
        want = _run(nv, q, k, v, do)
        torch.cuda.synchronize()
        for t in out:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_far_tokens(nv):
    """A token stride that takes the tensors' ends past 2^31 elements."""
    g = torch.Generator(device="cuda").manual_seed(8)
    n, stride = 300, 8 * 1024 * 1024 - 8
    big = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")  # 5 GB
    views = [big.as_strided((1, n, 2, 64), (0, stride, 64, 1), i * 4096) for i in range(3)]
    src = [_rand(g, 1, n, 2, 64) for _ in range(3)]
    for a, b in zip(views, src):
        a.copy_(b)
    do = _rand(g, 1, n, 2, 64)
    assert all(torch.equal(a, b) for a, b in zip(_run(nv, *views, do), _run(nv, *src, do)))


@pytest.mark.parametrize("dim,h,hk,window", [(128, 5, 1, 0), (64, 4, 2, 300)])
def test_long(nv, dim, h, hk, window):
    """Several thousand tokens, against the same sequence's rows computed in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(9)
    n = 4100
    q, k, v = _rand(g, 1, n, h, dim), _rand(g, 1, n, hk, dim), _rand(g, 1, n, hk, dim)
    do = _rand(g, 1, n, h, dim, scale=1e-3)
    o, lse, dq, dk, dv = _run(nv, q, k, v, do, window=window)
    _check_sequence(q[0], k[0], v[0], do[0], o[0], lse, dq[0], dk[0], dv[0], _see(n, n, True, window), dim ** -0.5, "long")
