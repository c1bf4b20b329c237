"""4-bit operands whose scales stand at any address: the same products as of aligned ones.

Tolerances.  The kernels sum the same exact terms in other orders: products of up to 512
terms, off by at most 512 2^-24 = 2^-15 of the sum of magnitudes, in float32.  Results are
rounded to bf16 once, 2^-8 of each of the two that are compared."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
B = torch.bfloat16


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


def rand(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(B)


def moved(nv, q, by):
    """The operand with its scales `by` bytes into another buffer."""
    flat = torch.empty(q.scales.numel() + 16, dtype=torch.uint8, device="cuda")
    scales = flat[by:by + q.scales.numel()].view(q.scales.shape)
    scales.copy_(q.scales)
    assert scales.data_ptr() % 4 == by % 4
    return nv.QTensor(q.codes, scales, q.global_scale, q.amax, q.rows, q.cols, q.scale_kind)


# few rows, tiles of 128, and what goes by tiles of 256 where scales are aligned
@pytest.mark.parametrize("rows,cols", [(48, 512), (1040, 720), (8192, 2048)], ids=str)
@pytest.mark.parametrize("by", [1, 2, 3, 6])
def test_products(nv, rows, cols, by):
    say("scales at", by, rows, cols)
    spec = nv.QuantSpec.of
    a = nv.quantize(rand(rows, 512, seed=1), [spec("row")])[0]
    g, u = (nv.quantize(rand(cols, 512, seed=s), [spec(kind)])[0] for s, kind in ((2, "row"), (3, "2d")))
    want = nv.gemm_gated(a, g, u, activation="relu")
    values = [nv.dequantize(q).double().abs() for q in (a, g, u)]
    eg, eu = (2 * 2.0 ** -15 * (values[0] @ v.t()) for v in values[1:])  # of the sums, in either order
    h, gate, up = (t.double().abs() * (1 + 2.0 ** -7) for t in want)  # before their rounding, at most
    for ops in ((moved(nv, a, by), g, u), (a, moved(nv, g, by), u), (a, g, moved(nv, u, by)), tuple(moved(nv, q, by) for q in (a, g, u))):
        got = nv.gemm_gated(*ops, activation="relu")
        product = eg * (up + eu) + gate * eu
        for x, y, size, room in zip(got, want, (h, gate, up), (product, eg, eu)):
            assert ((x.double() - y.double()).abs() <= 2 * 2.0 ** -8 * (size + room) + room).all()
    gate, up = want[1], want[2]
    dy = nv.quantize(rand(rows, 512, seed=5), [spec("row")])[0]
    want = nv.gemm_gated_backward(dy, g, gate, up, "relu")
    room = 2 * 2.0 ** -15 * (nv.dequantize(dy).double().abs() @ values[1].t())
    got = nv.gemm_gated_backward(moved(nv, dy, by), moved(nv, g, by), gate, up, "relu")
    for x, y, f in zip(got, want, (up.double().abs() * (gate > 0), gate.relu().double())):
        assert ((x.double() - y.double()).abs() <= 2 * 2.0 ** -8 * (y.double().abs() * (1 + 2.0 ** -7) + room * f) + room * f).all()
    if rows % 256 == 0:
        x, y = nv.gemm(a, g, "f32"), nv.gemm(moved(nv, a, by), moved(nv, g, by), "f32")
        assert ((x.double() - y.double()).abs() <= 1.01 * eg).all()
