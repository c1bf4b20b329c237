"""The gated feed-forward products and their gradient against the definition in 64
bits on the operands' exact values.

Tolerances.  A product of K terms is summed in binary32, 16 at a time: its error is
at most E = (K / 16 + 8) 2^-24 sum |a b|.  An activation's slope is at most 1.13, its
own error 2^-20 of |x|; a result is rounded once to bf16 (2^-8 of its value).  So
h is within 2^-8 |h| + 1.13 E_gate |up| + E_up |act| + 2^-19 |gate up|, and the
gradients, whose activations come from given bf16 values, within 2^-8 of their
values + (E + 2^-19 |dh|) times what dh is multiplied by (at most 1.13 |up|, |gate|)."""
import math

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


def act(x, kind):
    if kind == "silu":
        return x * torch.special.expit(x)
    if kind == "relu":
        return torch.relu(x)
    if kind == "gelu":
        return x * torch.special.ndtr(x)
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def operand(nv, rows, cols, layout, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * std).to(torch.bfloat16)
    return nv.quantize(x, [nv.QuantSpec.of(layout)])[0]


def product(nv, a, b):
    """(a b^T, the bound of its binary32 sum's error) in 64 bits."""
    x, y = nv.dequantize(a).double(), nv.dequantize(b).double()
    return x @ y.t(), (a.cols / 16 + 8) * 2.0 ** -24 * (x.abs() @ y.abs().t())


# (M, N, K): the smallest, sizes that fill no tile of either path, whole tiles, several tiles of both
SHAPES = [(16, 16, 16), (16, 48, 64), (48, 80, 208), (64, 16, 5120), (80, 1040, 1040), (256, 128, 128), (272, 144, 128),
          (512, 384, 256), (16, 2736, 1024), (1008, 400, 2064), (1040, 656, 640), (2048, 1024, 512), (32, 4112, 384), (128, 512, 272)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_forward(nv, shape, kind):
    m, n, k = shape
    say("gated forward", shape, kind)
    a = operand(nv, m, k, "row", 1)
    wg, wu = operand(nv, n, k, "2d", 2, 1.5 * k ** -0.5), operand(nv, n, k, "row", 3, k ** -0.5)
    amax = torch.zeros(1, device="cuda")
    h, gate, up = nv.gemm_gated(a, wg, wu, activation=kind, amax=amax)
    (g, eg), (u, eu) = product(nv, a, wg), product(nv, a, wu)
    for got, want, e, what in ((gate, g, eg, "gate"), (up, u, eu, "up")):
        off = (got.double() - want).abs() - 2.0 ** -8 * want.abs() - e
        assert (off <= 0).all(), "%s: %.3g too far" % (what, off.max())
    want = act(g, kind) * u
    room = 2.0 ** -8 * want.abs() + 1.13 * eg * u.abs() + eu * act(g, kind).abs() + 2.0 ** -19 * (g * u).abs()
    off = (h.double() - want).abs() - room
    assert (off <= 0).all(), "h: %.3g too far" % off.max()
    assert amax.item() == h.abs().max().item()
    alone = nv.gemm_gated(a, wg, wu, activation=kind, keep=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[0], h)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient(nv, shape, kind):
    m, n, k = shape
    say("gated gradient", shape, kind)
    a, w = operand(nv, m, k, "row", 4, 1e-3), operand(nv, n, k, "2d", 5, n ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(6)
    gate, up = (torch.randn(m, n, generator=g, device="cuda").to(torch.bfloat16) * 2 for _ in range(2))
    tops = [torch.zeros(1, device="cuda") for _ in range(2)]
    dgate, dup = nv.gemm_gated_backward(a, w, gate, up, activation=kind, amax_gate=tops[0], amax_up=tops[1])
    dh, e = product(nv, a, w)
    x, y = gate.double().requires_grad_(), up.double()
    f = act(x, kind)
    df = torch.autograd.grad(f, x, torch.ones_like(f))[0]
    f = f.detach()
    room = e + 2.0 ** -19 * dh.abs()
    for got, want, by in ((dgate, dh * y * df, 1.13 * y.abs()), (dup, dh * f, x.detach().abs())):
        off = (got.double() - want).abs() - 2.0 ** -8 * want.abs() - room * by
        assert (off <= 0).all(), "%.3g too far" % off.max()
    assert tops[0].item() == dgate.abs().max().item() and tops[1].item() == dup.abs().max().item()


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gradient_against_differences(nv, kind):
    """With up = 1 a column's dgate is dh times the slope of what the forward pass computes."""
    say("gated differences", kind)
    m, n, k = 64, 128, 128
    a, w = operand(nv, m, k, "row", 7), operand(nv, n, k, "2d", 8)
    gate = torch.linspace(-6, 6, m * n, device="cuda").reshape(m, n).to(torch.bfloat16)
    gate[gate == 0] = 0.5
    up = torch.ones_like(gate)
    dgate, dup = nv.gemm_gated_backward(a, w, gate, up, activation=kind)
    dh, e = product(nv, a, w)
    x = gate.double()
    slope = (act(x + 1e-5, kind) - act(x - 1e-5, kind)) / 2e-5
    # the quotient is off by 1e-10 / 6 of the third derivative (below 3) and 2^-52 6 / 1e-5
    room = 2.0 ** -8 * (dh * slope).abs() + 1.13 * (e + 2.0 ** -19 * dh.abs()) + 1e-9 * dh.abs()
    assert ((dgate.double() - dh * slope).abs() <= room).all()
    assert ((dup.double() - dh * act(x, kind)).abs() <= 2.0 ** -8 * (dh * act(x, kind)).abs() + (e + 2.0 ** -19 * dh.abs()) * x.abs()).all()


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_extreme_gates(nv, kind):
    """Gates of any finite size have the derivative's limits, 0 and 1, and no NaN arises."""
    say("gated extremes", kind)
    a, w = operand(nv, 16, 16, "row", 7), operand(nv, 16, 16, "2d", 8)
    values = torch.tensor([3e38, -3e38, 1e20, -1e20, 1e10, -1e10, 200.0, -200.0, 0.0, -0.0, 1e-30, -1e-30, 1e-38, 20.0, -20.0, -100.0])
    gate = values.cuda().to(torch.bfloat16).repeat(16, 1)
    up = torch.ones_like(gate)
    dgate, dup = nv.gemm_gated_backward(a, w, gate, up, activation=kind)
    dh, e = product(nv, a, w)
    slope = torch.where(gate > 15, 1.0, torch.where(gate < -15, 0.0, 0.0 if kind == "relu" else 0.5)).double()
    if kind == "relu":
        slope = (gate > 0).double()
    assert torch.isfinite(dgate).all() and not torch.isnan(dup).any()
    # beyond 15 the slope is within 20 e^-15 of its limit
    assert ((dgate.double() - dh * slope).abs() <= 2.0 ** -8 * (dh * slope).abs() + 1.13 * e + 1e-5 * dh.abs()).all()
    assert (dup[gate < -15].abs() <= 1e-3 * dh.abs().max()).all()


def test_maxima_for_the_column_quantisation(nv):
    """amax_rht_col is what a quantisation of h along its rows with the RHT finds: its sums of 16 products are formed in
    another order, some 2^-20 apart."""
    say("gated RHT maxima")
    for m, n, k in ((272, 144, 128), (48, 80, 208), (16, 400, 256)):
        a, wg, wu = operand(nv, m, k, "row", 1), operand(nv, n, k, "2d", 2, k ** -0.5), operand(nv, n, k, "2d", 3, k ** -0.5)
        top = torch.zeros(1, device="cuda")
        h, gate, up = nv.gemm_gated(a, wg, wu, amax_rht_col=top, rht_seed=77)
        want = nv.quantize(h, [nv.QuantSpec.of("col", "rtn", True, 0, 77)])[0].amax
        assert abs(top.item() / want.item() - 1) < 2.0 ** -18
        d, wd = operand(nv, m, k, "row", 4, 1e-3), operand(nv, n, k, "2d", 5)
        tops = torch.zeros(4, 1, device="cuda").unbind()
        dgate, dup = nv.gemm_gated_backward(d, wd, gate, up, amax_gate=tops[0], amax_up=tops[1], amax_rht_gate=tops[2],
                                            amax_rht_up=tops[3], rht_seed=77)
        for t, plain, rht in ((dgate, tops[0], tops[2]), (dup, tops[1], tops[3])):
            assert plain.item() == t.abs().max().item()
            want = nv.quantize(t.contiguous(), [nv.QuantSpec.of("col", "rtn", True, 0, 77)])[0].amax
            assert abs(rht.item() / want.item() - 1) < 2.0 ** -18
        both = torch.zeros(1, device="cuda")
        nv.gemm_gated_backward(d, wd, gate, up, amax_gate=both, amax_up=both)
        assert both.item() == max(tops[0].item(), tops[1].item())


def test_in_place_and_strides(nv):
    say("gated in place")
    for m, n, k in ((272, 144, 128), (80, 48, 208), (16, 64, 512)):
        d, w = operand(nv, m, k, "row", 4, 1e-3), operand(nv, n, k, "2d", 5)
        both = torch.randn(m, 2 * n, device="cuda").to(torch.bfloat16)
        gate, up = both[:, :n], both[:, n:]
        want = nv.gemm_gated_backward(d, w, gate.contiguous(), up.contiguous())
        turned = both.clone()
        nv.nvfp4_gemm_gated_backward(d, w, turned[:, :n], turned[:, n:], turned[:, n:], turned[:, :n])  # each in the other's place
        assert torch.equal(turned[:, n:], want[0]) and torch.equal(turned[:, :n], want[1])
        nv.nvfp4_gemm_gated_backward(d, w, gate, up, gate, up)
        assert torch.equal(gate, want[0]) and torch.equal(up, want[1])
        # rows of wider buffers, the rest of which stays
        a, wg, wu = operand(nv, m, k, "row", 1), operand(nv, n, k, "2d", 2), operand(nv, n, k, "2d", 3)
        wide = torch.full((m + 16, n + 24), 5.0, dtype=torch.bfloat16, device="cuda")
        h, gate, up = nv.gemm_gated(a, wg, wu)
        nv.nvfp4_gemm_gated(a, wg, wu, wide[:m, 8:n + 8])
        assert torch.equal(wide[:m, 8:n + 8], h) and (wide[m:] == 5.0).all() and (wide[:, :8] == 5.0).all() and (wide[:, n + 8:] == 5.0).all()


# (M, N, K) of the tiles of 256 rows: whole ones, then rows and columns that end inside a tile; K of one K-tile and of several
LARGE = [(1024, 5120, 128), (1040, 5136, 128), (1040, 5136, 640)]
LARGE_BACK = [(1024, 10240, 128), (1040, 10256, 128), (1040, 10256, 640)]


@pytest.mark.parametrize("shape", LARGE, ids=str)
@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_forward_of_large_tiles(nv, shape, kind):
    test_forward(nv, shape, kind)


@pytest.mark.parametrize("shape", LARGE_BACK, ids=str)
@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gradient_of_large_tiles(nv, shape, kind):
    test_gradient(nv, shape, kind)


def test_large_tiles_maxima_places_and_graphs(nv):
    """As the tests of these for the other sizes."""
    say("gated large tiles")
    (m, n, k), wide = LARGE[1], LARGE_BACK[1][1]
    a, wg, wu = operand(nv, m, k, "row", 1), operand(nv, n, k, "2d", 2, k ** -0.5), operand(nv, n, k, "2d", 3, k ** -0.5)
    top = torch.zeros(1, device="cuda")
    h, gate, up = nv.gemm_gated(a, wg, wu, amax_rht_col=top, rht_seed=77)
    want = nv.quantize(h, [nv.QuantSpec.of("col", "rtn", True, 0, 77)])[0].amax
    assert abs(top.item() / want.item() - 1) < 2.0 ** -18
    buffer = torch.full((m + 16, n + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm_gated(a, wg, wu, buffer[:m, 8:n + 8])
    assert torch.equal(buffer[:m, 8:n + 8], h)
    assert (buffer[m:] == 5.0).all() and (buffer[:, :8] == 5.0).all() and (buffer[:, n + 8:] == 5.0).all()
    d, w = operand(nv, m, k, "row", 4, 1e-3), operand(nv, wide, k, "2d", 5)
    both = torch.randn(m, 2 * wide, device="cuda").to(torch.bfloat16)
    gate, up = both[:, :wide], both[:, wide:]
    tops = torch.zeros(4, 1, device="cuda").unbind()
    want = nv.gemm_gated_backward(d, w, gate, up, amax_gate=tops[0], amax_up=tops[1], amax_rht_gate=tops[2], amax_rht_up=tops[3],
                                  rht_seed=77)
    for t, plain, rht in ((want[0], tops[0], tops[2]), (want[1], tops[1], tops[3])):
        assert plain.item() == t.abs().max().item()
        assert abs(rht.item() / nv.quantize(t, [nv.QuantSpec.of("col", "rtn", True, 0, 77)])[0].amax.item() - 1) < 2.0 ** -18
    turned = both.clone()
    nv.nvfp4_gemm_gated_backward(d, w, turned[:, :wide], turned[:, wide:], turned[:, wide:], turned[:, :wide])
    assert torch.equal(turned[:, wide:], want[0]) and torch.equal(turned[:, :wide], want[1])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held, held_grads = nv.gemm_gated(a, wg, wu), nv.gemm_gated_backward(d, w, gate, up)
    for turn in range(3):
        a.codes.copy_(a.codes.roll(1, 0))
        d.codes.copy_(d.codes.roll(1, 0))
        graph.replay()
        now, grads = nv.gemm_gated(a, wg, wu), nv.gemm_gated_backward(d, w, gate, up)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*now, *grads), (*held, *held_grads)))


def test_one_quantised_tensor_of_both_weights(nv):
    """Gate and up as the two halves of one quantised weight."""
    say("gated halves of one weight")
    a, w = operand(nv, 64, 256, "row", 1), operand(nv, 512, 256, "2d", 2)
    half = lambda i: nv.QTensor(w.codes[256 * i:256 * i + 256], w.scales[16 * i:16 * i + 16], w.global_scale, w.amax, 256, 256,  # noqa: E731
                                w.scale_kind)
    h, gate, up = nv.gemm_gated(a, half(0), half(1))
    both = nv.gemm(a, w, "bf16")
    assert torch.equal(gate, both[:, :256]) and torch.equal(up, both[:, 256:])


def test_zeros(nv):
    say("gated zeros")
    z = nv.quantize(torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda"), [nv.QuantSpec.of("row")])[0]
    w = operand(nv, 48, 64, "2d", 2)
    h, gate, up = nv.gemm_gated(z, w, w, activation="gelu")
    assert not h.any() and not gate.any() and not up.any()


def test_repeats_streams_and_graphs(nv):
    say("gated on another stream, and captured")
    for m, n, k in ((272, 400, 256), (48, 80, 208), (16, 512, 1024)):
        a, wg, wu = operand(nv, m, k, "row", 1), operand(nv, n, k, "2d", 2), operand(nv, n, k, "2d", 3)
        d, wd = operand(nv, m, k, "row", 4, 1e-3), operand(nv, n, k, "2d", 5)
        want = nv.gemm_gated(a, wg, wu)
        grads = nv.gemm_gated_backward(d, wd, want[1], want[2])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = nv.gemm_gated(a, wg, wu, stream=s)
        back = nv.gemm_gated_backward(d, wd, got[1], got[2], stream=s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*want, *grads), (*got, *back)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = nv.gemm_gated(a, wg, wu)
            held_grads = nv.gemm_gated_backward(d, wd, held[1], held[2])
        for turn in range(3):
            a.codes.copy_(a.codes.roll(1, 0))
            graph.replay()
            want = nv.gemm_gated(a, wg, wu)
            grads = nv.gemm_gated_backward(d, wd, want[1], want[2])
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip((*want, *grads), (*held, *held_grads)))


def test_python_refusals(nv):
    a, w, v = operand(nv, 32, 64, "row", 1), operand(nv, 48, 64, "2d", 2), operand(nv, 48, 80, "2d", 2)
    x = torch.zeros(32, 48, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: nv.gemm_gated(a, w, v), lambda: nv.gemm_gated(a, w, operand(nv, 32, 64, "2d", 2)),
                 lambda: nv.nvfp4_gemm_gated(a, w, w, x[:16]), lambda: nv.nvfp4_gemm_gated(a, w, w, x.float()),
                 lambda: nv.nvfp4_gemm_gated(a, w, w, x, amax=torch.zeros(2, device="cuda")),
                 lambda: nv.gemm_gated_backward(a, w, x, x[:, :32]), lambda: nv.nvfp4_gemm_gated(a, w, w, x.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: nv.gemm_gated(a, w, w, activation=9), lambda: nv.nvfp4_gemm_gated(a, w, w, x, x),
                 lambda: nv.nvfp4_gemm_gated_backward(a, w, x, x, x, x)):
        with pytest.raises(nv.Nvfp4Error):
            call()


def test_gelu_over_all_gates(nv):
    """Every finite bfloat16 gate: x P(N < x) and its derivative, the tail's relative error below 2^-16 while it is normal."""
    say("gelu over all gates")
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32)
    x = (bits - (bits >> 15 << 16)).to(torch.int16).view(torch.bfloat16)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).reshape(1024, 64).contiguous()
    one = torch.zeros(1024, 16, device="cuda")
    one[:, 0] = 1
    a, w = (nv.quantize(t.to(torch.bfloat16), [nv.QuantSpec.of("row")])[0] for t in (one, one[:64]))
    dh, e = product(nv, a, w)
    unit = dh[0, 0].item()
    assert (dh == unit).all()
    dgate, dup = nv.gemm_gated_backward(a, w, x, torch.ones_like(x), activation="gelu")
    d = x.double()
    below = 0.5 * torch.special.erfc(-d / math.sqrt(2))  # (torch's ndtr is 1 + erf, which has no tail)
    f = d * below * unit
    tail = (d > -13) & (f.abs() > 1e-36)
    assert ((dup.double() - f).abs()[tail] <= ((2.0 ** -8 + 2.0 ** -16) * f.abs())[tail]).all()
    assert (dup.double()[d <= -13].abs() < 1e-35).all()
    df = (below + d * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)) * unit
    # the two terms cancel below 0: within 2^-16 of their sizes
    size = (below + d.abs() * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)) * unit
    assert ((dgate.double() - df).abs() <= 2.0 ** -8 * df.abs() + 2.0 ** -16 * size + 1e-36).all()
