"""Orthogonalised updates of matrices whose singular values lie far apart, as
gradients' do, against the definition in 64 bits: unrounded, as a float32
parameter receives them.

Tolerances.  An operand of the products is held as two fp16: 2^-22 of an element at
most, and the product of two second parts, left out, is as large at most: a product
is off by up to three times 2^-22 of its terms.  In a step X enters with a slope of
1, A with one below 3 and the polynomial with 1.2 (singular values up to 1.2): it
adds (1 + 3 + 1.2) 3 2^-22 of the iterate's norm at most where roundings do not all
point one way in a product's sum, which random signs keep them from.  Weak
directions, which the iteration brings to the size of the strong ones, carry that
on by up to a = 3.4445 a step, the largest slope: the sum over the steps k of
a^(steps - k) |X_k| / |X_last|, taken from the definition, bounds how far.  A chain of
steps rounds A, the polynomials' product and what lies between once more: twice that."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ABC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


def definition(u, steps=5, abc=ABC):
    """X in 64 bits, and how far a rounding of a step is carried on."""
    x = u / u.norm()
    norms = [1.0]
    for _ in range(steps):
        a = x @ x.t()
        x = abc[0] * x + (abc[1] * a + abc[2] * (a @ a)) @ x
        norms.append(x.norm().item())
    return x, sum(abc[0] ** (steps - k) * norms[k] for k in range(steps)) / norms[-1]


def spectrum(kind, m, n):
    """An m x n matrix, m <= n."""
    g = torch.Generator(device="cuda").manual_seed(m + n)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    if kind[0] == "strong":  # directions of one size over noise
        return rand(m, kind[1]) @ rand(kind[1], n) + kind[2] * rand(m, n)
    if kind[0] == "row":  # one row over weak ones
        x = rand(m, n)
        x[m // 3] *= kind[1]
        return x
    s = torch.arange(1, m + 1, device="cuda", dtype=torch.float64)
    s = s ** -kind[1] if kind[0] == "power" else torch.where(s <= m // 2, 1.0, kind[1])
    left, right = (torch.linalg.qr(rand(k, m).cpu())[0].cuda() for k in (m, n))
    return (left * s) @ right.t().contiguous()


def step(nv, x):
    """-X of float32 gradients (a list), as float32 parameters of zero get it."""
    p = [torch.zeros_like(t) for t in x]
    nv.muon([nv.MuonTensor(a, b, scale=1.0) for a, b in zip(p, x)], 1.0, nesterov=False)
    return p


KINDS = [("strong", 1, 1.0), ("strong", 1, 0.05), ("strong", 4, 0.05), ("strong", 1, 0.01), ("strong", 4, 0.003), ("strong", 1, 1e-4),
         ("power", 1.0), ("power", 1.5), ("power", 2.0), ("half", 1e-3), ("half", 1e-9), ("row", 1e4)]


# single steps in tiles of 64 and more, and steps in chains
@pytest.mark.parametrize("shape", [(64, 64), (250, 1000), (1000, 1111), (1040, 1600)], ids=str)
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_spectra(nv, shape, kind):
    say("muon spectrum", shape, kind)
    x = spectrum(kind, *shape).float()
    chained = shape == (1040, 1600)
    want, carried = definition(x.double())
    rel = (2 if chained else 1) * (1 + 3 + 1.2) * 3 * 2.0 ** -22 * carried
    upright, flat = step(nv, [x.t().contiguous(), x])
    for got in (flat, upright.t()):
        off = ((got.double() + want).norm() / want.norm()).item()
        print("off by %.2g, carried %.3g" % (off, carried), flush=True)
        assert torch.isfinite(got).all() and off <= rel, "off by %.3g of the norm, %.3g is allowed" % (off, rel)


def test_a_parameter_is_as_good_as_32_bits(nv):
    """A float32 step differs from the definition by its own roundings, three of at most 2^-24 of the parameter (the decay's
    factor, its product, the sum), and by lr scale times the update's error, which is a small part of that."""
    say("muon float32 parameter")
    lr, scale, wd = 3e-4, 0.2 * 1024 ** 0.5, 0.1
    for kind in (("strong", 1, 1.0), ("strong", 4, 0.05)):
        g = spectrum(kind, 256, 1024).float()
        p0 = 0.02 * spectrum(("strong", 1, 1.0), 256, 1024).float()
        p = p0.clone()
        nv.muon([nv.MuonTensor(p, g, weight_decay=wd, scale=scale)], lr, nesterov=False)
        want = p0.double() * (1 - lr * wd) - lr * scale * definition(g.double())[0]
        off = ((p.double() - want).norm() / want.norm()).item()
        print("off by %.2g" % off, flush=True)
        assert off <= 3 * 2.0 ** -24


@pytest.mark.parametrize("abc", [(3.5, 0.0, 0.0), (12.0, -24.0, 12.0), (-3.4, 0.0, 0.0)], ids=str)
def test_iterations_at_the_bound(nv, abc):
    """Singular values and polynomials as large as any that are taken: nothing leaves fp16's range.  One step: three
    products' errors of the polynomial's terms, whose sizes add up to (|a| + 2 |b| + 3 |c|) with A's own in them."""
    say("muon at the bound", abc)
    one = torch.zeros(70, 90, device="cuda")
    one[3, 5] = -2.0
    row = torch.zeros(300, 400, device="cuda")
    row[7] = torch.randn(400, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    for x in (one, one.t().contiguous(), row, spectrum(("strong", 1, 1.0), 64, 200).float(), spectrum(("half", 1e-3), 200, 300).float()):
        p = torch.zeros_like(x)
        nv.muon([nv.MuonTensor(p, x, scale=1.0)], 1.0, nesterov=False, steps=1, coefficients=abc)
        u = x.double() / x.double().norm()
        u = u.t() if u.shape[0] > u.shape[1] else u
        a = u @ u.t()
        want = abc[0] * u + (abc[1] * a + abc[2] * (a @ a)) @ u
        got = p.t() if p.shape[0] > p.shape[1] else p
        room = (abs(abc[0]) + 2 * abs(abc[1]) + 3 * abs(abc[2])) * 3 * 2.0 ** -22
        assert torch.isfinite(got).all() and (got.double() + want).norm() <= room  # (|u| = 1)
