"""The block operators on tensors of more than 2^31 elements: what stands far behind the first 2^32 bytes is as it is in a
small call."""
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
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("100 GB of free memory are wanted")
    yield nv
    torch.cuda.empty_cache()


def rows_of(nv, q, first, n):
    return nv.QTensor(q.codes[first:first + n], q.scales[first:first + n], q.global_scale, q.amax, n, q.cols, q.scale_kind)


@pytest.mark.parametrize("k", [16, 128])
def test_gated(nv, k):
    """Both kernels for many rows; single results are sums of the same products in the same order, at most 128 of them."""
    m, n = 69632, 32768
    say("gated beyond 2^31 elements", m, n, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    spec = nv.QuantSpec.of("row")
    a, wg, wu = (nv.quantize(torch.randn(r, k, generator=g, device="cuda").to(torch.bfloat16), [spec])[0] for r in (m, n, n))
    top = torch.zeros(1, device="cuda")
    h, gate, up = nv.gemm_gated(a, wg, wu, amax=top)
    dgate, dup = nv.gemm_gated_backward(a, wg, gate, up)
    for first in (0, 32768, 65536, m - 256):
        part = rows_of(nv, a, first, 256)
        want = nv.gemm_gated(part, wg, wu)
        at = slice(first, first + 256)
        for x, y in zip((h, gate, up), want):
            assert (x[at].float() - y.float()).norm() <= 2.0 ** -8 * y.float().norm()
        want = nv.gemm_gated_backward(part, wg, gate[at], up[at])
        for x, y in zip((dgate, dup), want):
            assert (x[at].float() - y.float()).norm() <= 2.0 ** -8 * y.float().norm()
    most = max(h[i:i + 4096].abs().max().item() for i in range(0, m, 4096))
    assert top.item() == most


def test_rope(nv):
    tokens, heads, dim = 440000, 40, 128
    say("rope beyond 2^31 elements", tokens, heads, dim)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.empty(1, tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    q.normal_(generator=g)
    w = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    freqs, _ = nv.rope_frequencies(dim)
    y, _ = nv.qk_rope(q, None, freqs, q_weight=w)
    dq, _, _, _ = nv.qk_rope_backward(y, None, freqs, q, None, q_weight=w)
    for first in (0, 419430 - 8, tokens - 64):
        at = torch.arange(first, first + 64, device="cuda")
        part = q[0, first:first + 64]
        want, _ = nv.qk_rope(part, None, freqs, positions=at, q_weight=w)
        assert torch.equal(y[0, first:first + 64], want)
        back, _, _, _ = nv.qk_rope_backward(want, None, freqs, part, None, positions=at, q_weight=w)
        assert torch.equal(dq[0, first:first + 64], back)


def test_orthogonalize(nv):
    """One element to each row, all of one size and in columns of their own: the result has them where they were, at
    what the iteration makes of 1 / sqrt(rows), and nothing else."""
    m, n = 16400, 131072
    say("orthogonalize beyond 2^31 elements", m, n)
    x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    row = torch.arange(m, device="cuda")
    col = n - 1 - 7 * row
    x[row, col] = 0.5
    y = nv.orthogonalize(x)
    s = m ** -0.5
    for _ in range(5):
        s = s * (3.4445 - 4.7750 * s * s + 2.0315 * s ** 4)
    # roundings to fp16 of X, A and the polynomial, each 2^-11 at most, carried by slopes below 4.1 (as of the small ones)
    assert ((y[row, col].float() - s).abs() <= 8.5e-3 * s + 2.0 ** -8 * s).all()
    assert sum(int(torch.count_nonzero(y[i:i + 1024])) for i in range(0, m, 1024)) == m
