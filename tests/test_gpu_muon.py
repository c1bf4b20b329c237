"""Steps by orthogonalised momentum against the definition in 64 bits.

Tolerances.  Every iteration rounds X, A and the polynomial to fp16 (2^-11 of an
element at most, evenly spread: 2^-11 / sqrt 3 of the Frobenius norm) after sums in
binary32.  With t singular values up to 1.2 a step's error is carried on by a slope
of at most about 1.2 in size once values are near 1, and grows like the values
themselves before; A and the polynomial enter with slopes of 2 |b + 2 c s| s < 3 and
s <= 1.2.  Five steps of sqrt(1 + 3 + 1.2) 2^-11 / sqrt 3 in squares give 1.4e-3, the
steps in a row up to 4.5e-3 if all point one way: 8.5e-3 with the rounding to bf16
(2^-8).  The momentum is up to three and a half roundings of 2^-24 of its terms (the
scaled gradient, the factor, the product, the sum); the parameter two of its own and lr
scale times the update's error."""
import math

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ABC = (3.4445, -4.7750, 2.0315)
UPDATE = 8.5e-3


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


def orthogonal(u, steps=5, abc=ABC):
    if u.shape[0] > u.shape[1]:
        return orthogonal(u.t().contiguous(), steps, abc).t()
    norm = u.norm()
    x = u / norm if norm > 0 else u
    for _ in range(steps):
        a = x @ x.t()
        x = abc[0] * x + (abc[1] * a + abc[2] * (a @ a)) @ x
    return x


def matrix(rows, cols, seed, dtype=torch.float32, size=1e-3):
    """Some strong directions over a bulk of weak ones."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = min(rows, cols, 8)
    x = torch.randn(rows, k, generator=g, device="cuda") @ torch.randn(k, cols, generator=g, device="cuda") * 0.3
    return (size * (x + torch.randn(rows, cols, generator=g, device="cuda"))).to(dtype)


def near(got, want, what, rel=UPDATE):
    off = (got.double() - want).norm() / want.norm()
    assert torch.isfinite(got).all() and off <= rel, "%s: off by %.3g of the norm" % (what, off)


SHAPES = [(1, 1), (1, 50), (50, 1), (2, 3), (16, 16), (31, 33), (64, 64), (65, 200), (200, 65), (130, 1000), (515, 513), (512, 640),
          (700, 512), (1000, 1111), (1600, 1540), (1537, 3001), (2560, 1536)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_orthogonalize(nv, shape, dtype):
    say("orthogonalize", shape, dtype)
    x = matrix(*shape, 7, dtype)
    got = nv.orthogonalize(x)
    assert got.shape == x.shape and got.dtype == torch.bfloat16
    near(got, orthogonal(x.double()), str(shape))
    assert torch.equal(got, nv.orthogonalize(x))


def test_singular_values(nv):
    """What the iteration is for: all singular values that are not tiny come near 1."""
    say("orthogonalize singular values")
    x = matrix(300, 700, 3)
    s = torch.linalg.svdvals(nv.orthogonalize(x).double())
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("size", [1e-38, 1e-20, 1e20, 1e36])
def test_sizes_of_gradients(nv, size):
    """The norm is taken in 64 bits: the size of the gradient does not matter."""
    say("orthogonalize sizes", size)
    x = matrix(96, 160, 5, size=1.0)
    y = x * size
    near(nv.orthogonalize(y), orthogonal(y.double()), "size %g" % size)


def test_zeros_and_zero_rows(nv):
    say("orthogonalize zeros")
    assert not nv.orthogonalize(torch.zeros(40, 70, device="cuda")).any()
    x = matrix(100, 170, 6)
    x[10:30] = 0
    x[:, 50:60] = 0
    y = nv.orthogonalize(x)
    assert not y[10:30].any() and not y[:, 50:60].any()
    near(y, orthogonal(x.double()), "zero rows")
    one = torch.zeros(70, 70, device="cuda")
    one[3, 5] = 2.0
    near(nv.orthogonalize(one), orthogonal(one.double()), "one element")


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, ABC), (3, (2.0, -1.5, 0.5)), (10, (1.5, -0.5, 0.0)), (6, (1.875, -1.25, 0.375))],
                         ids=str)
def test_other_iterations(nv, steps, abc):
    say("orthogonalize", steps, abc)
    for shape in ((60, 90), (180, 70)):
        x = matrix(*shape, 8)
        near(nv.orthogonalize(x, steps=steps, coefficients=abc), orthogonal(x.double(), steps, abc), str(abc), 2 * UPDATE)


def test_many_matrices_at_once(nv):
    """More than one group, of all tile sizes, in one call: each as by itself."""
    say("orthogonalize many")
    g = torch.Generator().manual_seed(1)
    shapes = [tuple(int(v) for v in torch.randint(1, 180, (2,), generator=g)) for _ in range(40)]
    shapes += [(520, 600), (1600, 1700), (600, 520), (0, 5), (1540, 1536)]
    xs = [matrix(*s, 100 + i, torch.bfloat16 if i % 2 else torch.float32) for i, s in enumerate(shapes)]
    for x, y in zip(xs, nv.orthogonalize(xs)):
        assert y.shape == x.shape
        if x.numel():
            assert torch.equal(y, nv.orthogonalize(x))
            near(y, orthogonal(x.double()), str(tuple(x.shape)))


# (matrices, rows, columns): lists whose products go in tiles of 256; of 128 and of 64, many to a compute unit, upright and flat
LISTS = [(5, 2040, 2290), (5, 2290, 2040), (7, 1000, 1111), (8, 1000, 1111), (20, 512, 500), (30, 300, 310), (20, 440, 445)]


@pytest.mark.parametrize("count,rows,cols", LISTS, ids=str)
def test_lists_of_one_size(nv, count, rows, cols):
    say("orthogonalize a list", count, rows, cols)
    xs = [matrix(rows, cols, 50 + i, torch.bfloat16 if i % 2 else torch.float32) for i in range(count)]
    out = nv.orthogonalize(xs)
    for i, (x, y) in enumerate(zip(xs, out)):
        near(y, orthogonal(x.double()), "matrix %d" % i)
    for x, y in zip(out, nv.orthogonalize(xs)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("steps,abc", [(5, ABC), (1, ABC), (2, ABC), (3, ABC), (4, ABC), (6, ABC), (10, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5)),
                                       (3, (4.03, -8.6, 4.25))], ids=str)
def test_long_matrices(nv, steps, abc):
    """Sides far apart: polynomials are multiplied before the iterate is, as far as their sizes let them be."""
    say("orthogonalize long", steps, abc)
    xs = [matrix(1040, 2200, 60), matrix(2110, 1030, 61, torch.bfloat16), matrix(1024, 5000, 62), torch.zeros(2100, 1025, device="cuda")]
    out = nv.orthogonalize(xs, steps=steps, coefficients=abc)
    for x, y in zip(xs[:3], out):
        near(y, orthogonal(x.double(), steps, abc), "%s" % (tuple(x.shape),), UPDATE if steps == 5 else 2 * UPDATE)
    assert not out[3].any()
    for x, y in zip(out, nv.orthogonalize(xs, steps=steps, coefficients=abc)):
        assert torch.equal(x, y)
    x = matrix(1030, 2110, 63)
    x[100:300] = 0
    y = nv.orthogonalize(x, steps=steps, coefficients=abc)
    assert not y[100:300].any()
    near(y, orthogonal(x.double(), steps, abc), "zero rows", UPDATE if steps == 5 else 2 * UPDATE)


def uniforms(n, index, step, seed):
    group = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    low = 0xFFFFFFFF
    c = [group & low, torch.full_like(group, index), torch.full_like(group, step & low), torch.full_like(group, 0x4D550000 + (step >> 32))]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32 & low) ^ c[1] ^ k0, p1 & low, (p0 >> 32 & low) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([x >> sh & 0xFFFF for x in c for sh in (0, 16)], 1).reshape(-1)[:n]


@pytest.mark.parametrize("shape", [(64, 200), (200, 64), (129, 77), (515, 520), (1, 9)], ids=str)
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("param,grad,rounding", [("f32", "bf16", "rtn"), ("bf16", "f32", "sr"), ("bf16", "bf16", "rtn")])
def test_step(nv, shape, nesterov, param, grad, rounding):
    say("muon step", shape, nesterov, param, grad, rounding)
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    lr, beta, wd, scale = 0.02, 0.9, 0.1, 0.7
    p0 = matrix(*shape, 1, types[param], 0.05)
    g, m0 = matrix(*shape, 2, types[grad]), matrix(*shape, 3)
    gs = torch.tensor([0.37], device="cuda")
    p, m = p0.clone(), m0.clone()
    copy = torch.zeros(shape, dtype=torch.bfloat16, device="cuda") if param == "f32" else None
    update, amax = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    other = nv.MuonTensor(None, matrix(20, 30, 9), update=torch.empty(20, 30, dtype=torch.bfloat16, device="cuda"))
    step, seed = (1 << 32) + 7, (5 << 32) + 11
    t = nv.MuonTensor(p, g, m, weight_decay=wd, scale=scale, copy=copy, update=update, amax=amax)
    nv.muon([other, t], lr, momentum=beta, nesterov=nesterov, rounding=rounding, seed=seed, step=step, grad_scale=gs)
    gd = g.double() * gs.double()
    md = beta * m0.double() + (1 - beta) * gd
    assert ((m.double() - md).abs() <= 4 * 2.0 ** -24 * (beta * m0.double().abs() + (1 - beta) * gd.abs()) + 1e-40).all()
    u = (1 - beta) * gd + beta * md if nesterov else md
    o = orthogonal(u)
    near(update, o, "update")
    want = p0.double() * (1 - lr * wd) - lr * scale * o
    # the parameter with the update as it was formed: elementwise, to its rounding (the update is off by bf16's own 2^-8)
    have = p0.double() * (1 - lr * wd) - lr * scale * update.double()
    room = lr * scale * 2.0 ** -8 * update.double().abs() + 2.0 ** -22 * p0.double().abs() + 2.0 ** -22 * lr * scale * update.double().abs() + 1e-7 * lr
    if param == "bf16":
        room = room + (2.0 ** -7 if rounding == "sr" else 2.0 ** -8) * have.abs()
    assert ((p.double() - have).abs() <= room).all()
    if param == "f32":
        assert (p.double() - want).norm() <= 2.0 ** -22 * p0.double().norm() + lr * scale * UPDATE * o.norm()
        assert torch.equal(copy, p.to(torch.bfloat16)) and amax.item() == copy.abs().max().item()
    else:
        assert amax.item() == p.abs().max().item()
    if rounding == "sr":
        # truncation after adding the uniforms: where the update's error cannot move the place
        unit = torch.exp2(torch.floor(torch.log2(have.abs().clamp(min=2.0 ** -126))) - 7)
        y = have.abs() / unit + uniforms(have.numel(), 1, step, seed).double().reshape(shape) / 65536
        sure = (y - torch.round(y)).abs() * unit > lr * scale * 2.0 ** -8 * update.double().abs() + 2.0 ** -20 * have.abs() + 1e-7 * lr
        exact = torch.copysign(torch.floor(y) * unit, have)
        assert torch.equal(p.double()[sure], exact[sure]) and sure.double().mean() > (0.3 if have.numel() > 100 else -1)


def test_steps_in_a_row(nv):
    """A list laid out once, its gradients replaced, a workspace of its own."""
    say("muon list")
    p, m = [matrix(70, 90, 1, size=0.05), matrix(90, 70, 2, size=0.05)], []
    want = [x.double() for x in p]
    mom = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in p]
    lst = nv.MuonList([nv.muon_tensor(x, matrix(*x.shape, 5)) for x in p])
    ws = lst.new_workspace()
    for k in range(4):
        grads = [matrix(*x.shape, 10 * k + i, torch.bfloat16 if k % 2 else torch.float32) for i, x in enumerate(p)]
        for i, g in enumerate(grads):
            lst.set_grad(i, g)
        nv.muon(lst, 0.01, workspace=ws)
        for i, g in enumerate(grads):
            mom[i] = 0.95 * mom[i] + 0.05 * g.double()
            o = orthogonal(0.05 * g.double() + 0.95 * mom[i])
            want[i] = want[i] - 0.01 * 0.2 * math.sqrt(90) * o
    for x, y in zip(p, want):
        assert (x.double() - y).norm() <= 4 * 0.01 * 0.2 * math.sqrt(90) * UPDATE * math.sqrt(70) + 1e-6 * y.norm()
    with pytest.raises(ValueError):
        lst.set_grad(0, p[1])


def test_unaligned_buffers(nv):
    """Matrices that begin at any element of a buffer."""
    say("muon unaligned")
    n = 33 * 45
    flat = lambda dtype, at: torch.zeros(n + 16, dtype=dtype, device="cuda")[at:at + n].view(33, 45)  # noqa: E731
    g, p, m = flat(torch.bfloat16, 3), flat(torch.float32, 1), flat(torch.float32, 5)
    c, u = flat(torch.bfloat16, 7), flat(torch.bfloat16, 9)
    g.copy_(matrix(33, 45, 2)), p.copy_(matrix(33, 45, 3))
    a = nv.MuonTensor(p, g, m, copy=c, update=u)
    b = nv.MuonTensor(p.clone(), g.clone(), m.clone(), copy=c.clone(), update=u.clone())
    nv.muon([a], 0.01)
    nv.muon([b], 0.01)
    assert all(torch.equal(x, y) for x, y in ((a.param, b.param), (a.m, b.m), (a.copy, b.copy), (a.update, b.update)))
    near(u, orthogonal(g.double() * 0.0975), "unaligned")


def test_other_stream_and_graph(nv):
    say("muon on another stream, and captured")
    grads = [matrix(100, 300, 1), matrix(520, 515, 2)]
    make = lambda: [nv.MuonTensor(matrix(*g.shape, 20, size=0.05), g, matrix(*g.shape, 30)) for g in grads]  # noqa: E731
    a, b, c = make(), make(), make()
    nv.muon(a, 0.01)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    nv.muon(b, 0.01, stream=s)
    s.synchronize()
    assert all(torch.equal(x.param, y.param) and torch.equal(x.m, y.m) for x, y in zip(a, b))
    lst = nv.MuonList(c)
    ws = lst.new_workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.muon(lst, 0.01, workspace=ws)
    for turn in range(3):
        graph.replay()
        if turn:
            nv.muon(a, 0.01)
        torch.cuda.synchronize()
        assert all(torch.equal(x.param, y.param) and torch.equal(x.m, y.m) for x, y in zip(a, c))
        for g in grads:
            g.mul_(1.5)


def test_python_refusals(nv):
    g = matrix(16, 24, 1)
    bad = [dict(param=g.t().contiguous()), dict(param=g, m=g.to(torch.bfloat16)), dict(param=g, copy=g), dict(param=g[:8]),
           dict(param=g, m=g.clone().t().contiguous().t()), dict(param=g, amax=torch.zeros(2, device="cuda")), dict(param=g.cpu())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            nv.MuonTensor(grad=g, **kw).c_struct()
    with pytest.raises(ValueError):
        nv.MuonTensor(None, g[0]).c_struct()
    for kw in (dict(steps=0), dict(steps=17), dict(momentum=1.0), dict(coefficients=(9.0, 0.0, 0.0)), dict(coefficients=(3.4445, -4.775, 9.0))):
        with pytest.raises(nv.Nvfp4Error):
            nv.muon([nv.MuonTensor(g.clone(), g, g.clone())], 0.01, **kw)
    with pytest.raises(nv.Nvfp4Error):
        nv.muon([nv.MuonTensor(None, g)], 0.01)  # nothing to write


def test_buffers_of_two_tensors_are_refused(nv):
    """What one tensor's step writes is no buffer of another's: their order within the call is not fixed."""
    p, m, u, g = (matrix(16, 24, i) for i in range(4))
    other, low = matrix(16, 24, 5), torch.zeros(16, 24, dtype=torch.bfloat16, device="cuda")
    for a, b in ((dict(param=p), dict(param=p)), (dict(param=p, m=m), dict(param=u, m=m)), (dict(param=p, copy=low), dict(param=u, update=low)),
                 (dict(param=g), dict(param=u))):
        with pytest.raises(ValueError):
            nv.muon([nv.MuonTensor(grad=other, **a), nv.MuonTensor(grad=g, **b)], 0.01)
    one = nv.MuonList([nv.MuonTensor(p, g, m), nv.MuonTensor(u, g), nv.MuonTensor(torch.empty(0, 3, device="cuda"), torch.empty(0, 3, device="cuda")),
                       nv.MuonTensor(torch.empty(0, 4, device="cuda"), torch.empty(0, 4, device="cuda"))])
    for at in (1, -3):
        with pytest.raises(ValueError):
            one.set_grad(at, m)
    one.set_grad(1, other)
    nv.muon(one, 0.01)
