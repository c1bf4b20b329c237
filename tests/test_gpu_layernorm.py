"""Layer norm and its gradient on the GPU against the formulas in 64 bits.

Tolerances count roundings.  A binary32 rounding is off by at most 2^-24 of the
value, a bf16 one by 2^-8.  A row's sum passes at most 32 additions in a thread,
6 across a wave and 16 across waves, and each value a dozen more operations: 80
roundings bound every binary32 result relative to the sum of the magnitudes
that went into it."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROUNDINGS = 80 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, rows, cols, dtype, pad=0, scale=1.0):
    """[rows][cols] as the first columns of a wider buffer whose rest is NaN."""
    b = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    b[:, :cols] = (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(dtype)
    return b[:, :cols]


def _within(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    over = ((got.double() - want).abs() - bound).max().item()
    assert over <= 0, "%s: %g over its bound" % (what, over)


SHAPES = [  # rows, cols, pad: one element, odd, each split's borders, strided, the workload's width, the widest
    (1, 1, 0), (3, 1, 0), (5, 7, 0), (1, 512, 0), (9, 520, 8), (130, 1024, 0), (4, 1032, 0), (77, 2048, 0),
    (6, 2056, 0), (33, 777, 3), (2, 5120, 0), (2100, 264, 0), (7, 8192, 0), (3, 8200, 0), (2, 20480, 16), (2, 32768, 0),
    (3, 32767, 1)]
TYPES = [(torch.bfloat16, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.float32),
         (torch.float32, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.bfloat16)]


def _forward64(x, r, w, b, eps):
    s = x.double()
    if r is not None:
        s = (x.float() + r.float()).to(x.dtype).double()
    mean = s.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((s - mean) ** 2).mean(1, keepdim=True) + eps)
    h = (s - mean) * rstd
    return s, mean, rstd, h, h * w.double() + (0 if b is None else b.double())


@pytest.mark.parametrize("rows,cols,pad", SHAPES)
@pytest.mark.parametrize("types", range(len(TYPES)))
def test_forward(nv, rows, cols, pad, types):
    tx, ty, tw = TYPES[types]
    say("layernorm", rows, cols, pad, TYPES[types])
    g = _gen(rows * 40000 + cols)
    x = _rand(g, rows, cols, tx, pad)
    r = _rand(g, rows, cols, tx, pad) if types % 2 == 0 else None
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(tw)
    b = None if types == 3 else torch.randn(cols, generator=g, device="cuda").to(tw)
    y = torch.full((rows, cols + pad), 7.0, dtype=ty, device="cuda")[:, :cols]
    total = torch.empty((rows, cols), dtype=tx, device="cuda") if r is not None else None
    mean, rstd, amax = (torch.zeros(n, device="cuda") for n in (rows, rows, 1))
    eps = 1e-5
    nv.nvfp4_layernorm(x, w, b, eps, y, mean, rstd, r, total, amax)
    s64, mean64, rstd64, h64, y64 = _forward64(x, r, w, b, eps)
    if r is not None:
        assert torch.equal(total.double(), s64)
    size = s64.abs().mean(1, keepdim=True)
    _within(mean, mean64[:, 0], ROUNDINGS * size[:, 0], "mean")
    # the mean's error moves every difference; rstd follows the differences' relative error
    dm = ROUNDINGS * size
    moved = dm * rstd64
    spread = (s64 - mean64).abs().mean(1, keepdim=True)
    _within(rstd, rstd64[:, 0], rstd64[:, 0] * (ROUNDINGS + 2 * (dm * spread * rstd64 ** 2)[:, 0] + (moved ** 2)[:, 0]), "rstd")
    bound = ((h64.abs() * (ROUNDINGS + 2 * dm * spread * rstd64 ** 2 + moved ** 2) + moved) * w.double().abs()
             + ROUNDINGS * y64.abs() + (0 if b is None else ROUNDINGS * b.double().abs()))
    _within(y, y64, bound + HALF[ty] * (y64.abs() + bound), "y")
    assert amax.item() == y.float().abs().max().item()
    if pad:
        assert (y._base[:, cols:] == 7.0).all(), "columns past the end were written"


@pytest.mark.parametrize("rows,cols,pad", SHAPES)
@pytest.mark.parametrize("types", range(len(TYPES)))
def test_backward(nv, rows, cols, pad, types):
    tx, ty, tw = TYPES[types]
    say("layernorm_backward", rows, cols, pad, TYPES[types])
    g = _gen(rows * 40000 + cols + 1)
    x, dy = _rand(g, rows, cols, tx, pad), _rand(g, rows, cols, ty, pad, 1e-3)
    ds = _rand(g, rows, cols, tx, pad, 1e-3) if types % 2 == 0 else None
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(tw)
    _, mean64, rstd64, _, _ = _forward64(x, None, w, None, 1e-5)
    mean, rstd = mean64[:, 0].float(), rstd64[:, 0].float()
    dx = torch.full((rows, cols + pad), 7.0, dtype=tx, device="cuda")[:, :cols]
    amax = torch.zeros(1, device="cuda")
    dw, db = (torch.full((cols,), 7.0, device="cuda") for _ in range(2))
    ws = torch.empty(nv.lib().nvfp4_layernorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    nv.nvfp4_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ds, amax, ws)
    # the formula on the given mean and rstd
    m, rs = mean.double()[:, None], rstd.double()[:, None]
    h = (x.double() - m) * rs
    q = dy.double() * w.double()
    c1, c2 = q.mean(1, keepdim=True), (q * h).mean(1, keepdim=True)
    want = rs * (q - c1 - h * c2)
    bound = ROUNDINGS * rs * (q.abs() + q.abs().mean(1, keepdim=True) + h.abs() * (q * h).abs().mean(1, keepdim=True))
    if ds is not None:
        want = want + ds.double()
        bound = bound + ROUNDINGS * want.abs()
    _within(dx, want, bound + HALF[tx] * (want.abs() + bound), "dx")
    assert amax.item() == dx.float().abs().max().item()
    # a column's sum: the rows of a thread, then at most 512 workgroups' sums
    steps = (rows / 512 + 600) * 2.0 ** -24
    _within(dw, (dy.double() * h).sum(0), steps * (dy.double() * h).abs().sum(0), "dweight")
    _within(db, dy.double().sum(0), steps * dy.double().abs().sum(0), "dbias")
    if pad:
        assert (dx._base[:, cols:] == 7.0).all(), "columns past the end were written"


@pytest.mark.parametrize("rows,cols,pad", [(37, 16393, 3), (131, 20487, 0), (600, 16392, 8), (2100, 18440, 0)])
@pytest.mark.parametrize("types", range(len(TYPES)))
def test_wide(nv, rows, cols, pad, types):
    """Rows whose sums over rows are a kernel of their own, and dx in the place of dy or of x."""
    test_forward(nv, rows, cols, pad, types)
    test_backward(nv, rows, cols, pad, types)
    if types != 1 or rows > 200:
        return
    g = _gen(cols)
    x, dy = _rand(g, rows, cols, torch.float32, 0), _rand(g, rows, cols, torch.float32, 0)
    w = torch.randn(cols, generator=g, device="cuda")
    _, mean, rstd, _ = nv.layernorm(x, w, w)
    want = nv.layernorm_backward(dy, x, w, mean, rstd)
    for place in (0, 1):
        t = [dy.clone(), x.clone()]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        ws = torch.empty(nv.lib().nvfp4_layernorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        nv.nvfp4_layernorm_backward(t[0], t[1], w, mean, rstd, t[place], dw, db, workspace=ws)
        assert torch.equal(t[place], want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])


def test_gradient_against_differences(nv):
    """d/dt of sum(dy * layernorm(x + t z)) by central differences in 64 bits is sum(dx * z); so for weight and bias."""
    rows, cols = 6, 200
    g = _gen(5)
    x, dy, z = (_rand(g, rows, cols, torch.float32) for _ in range(3))
    w, b = torch.randn(cols, generator=g, device="cuda"), torch.randn(cols, generator=g, device="cuda")
    y, mean, rstd, _ = nv.layernorm(x, w, b, 1e-5)
    dx, dw, db = nv.layernorm_backward(dy, x, w, mean, rstd)

    def value(x, w, b):
        mean = x.mean(1, keepdim=True)
        c = x - mean
        return (dy.double() * (c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w + b)).sum()

    t = 1e-5
    x, w, b, z = (v.double() for v in (x, w, b, z))
    for grad, up, down in ((dx * z, value(x + t * z, w, b), value(x - t * z, w, b)),
                           (dw * z[0], value(x, w + t * z[0], b), value(x, w - t * z[0], b)),
                           (db * z[0], value(x, w, b + t * z[0]), value(x, w, b - t * z[0]))):
        # the differences' own error is of order t^2, the gradient's 80 roundings of its terms
        got, want = grad.double().sum().item(), ((up - down) / (2 * t)).item()
        assert abs(got - want) <= 1e-4 * grad.double().abs().sum().item() / grad.numel() ** 0.5 + 1e-6


def test_constant_rows_and_in_place(nv):
    """A row of equal values has variance 0: y is the bias; y may be x, and the sum the residual."""
    x = torch.full((3, 640), 2.5, dtype=torch.bfloat16, device="cuda")
    r = torch.full((3, 640), -1.0, dtype=torch.bfloat16, device="cuda")
    w, b = torch.randn(640, device="cuda"), torch.randn(640, device="cuda")
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    nv.nvfp4_layernorm(x, w, b, 1e-5, x, mean, rstd, r, r)
    assert torch.equal(x, b.to(torch.bfloat16).expand(3, -1)) and (r == 1.5).all() and (mean == 1.5).all()
    g = _gen(9)
    x, q = _rand(g, 5, 5120, torch.bfloat16), _rand(g, 5, 5120, torch.bfloat16)
    w, b = torch.randn(5120, device="cuda"), torch.randn(5120, device="cuda")
    want = nv.layernorm(x, w, b, 1e-5, residual=q)
    xc, qc = x.clone(), q.clone()
    mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    nv.nvfp4_layernorm(xc, w, b, 1e-5, xc, mean, rstd, qc, qc)
    assert torch.equal(xc, want[0]) and torch.equal(qc, want[3])


def test_amax_serves_the_quantiser(nv):
    """The maxima that the norm and its gradient leave are the quantiser's own: the same codes with NVFP4_AMAX_GIVEN."""
    g = _gen(11)
    x, w, b = _rand(g, 256, 512, torch.bfloat16), torch.randn(512, device="cuda"), torch.randn(512, device="cuda")
    amax = torch.zeros(2, device="cuda")
    y, mean, rstd, _ = nv.layernorm(x, w, b, amax=amax[:1])
    dx, _, _ = nv.layernorm_backward(y, x, w, mean, rstd, amax=amax[1:])
    for t, top in ((y, amax[:1]), (dx, amax[1:])):
        want = nv.quantize(t, [nv.QuantSpec.of("row")])[0]
        out = nv.empty_qtensor(256, 512, nv.SCALE_1D16)
        out.amax.copy_(top)
        nv.nvfp4_quantize(t, [nv.QuantSpec.of("row", amax_given=True)], [out], nv.new_workspace())
        assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
        assert torch.equal(out.global_scale, want.global_scale)


def test_optional_outputs_and_repeats(nv):
    """Without dweight and dbias no workspace is needed; repeated calls give the same bits."""
    g = _gen(13)
    x, dy = _rand(g, 3000, 1000, torch.bfloat16), _rand(g, 3000, 1000, torch.bfloat16)
    w = torch.randn(1000, device="cuda")
    _, mean, rstd, _ = nv.layernorm(x, w)
    first = nv.layernorm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, nv.layernorm_backward(dy, x, w, mean, rstd)))
    dx = torch.empty_like(x)
    nv.nvfp4_layernorm_backward(dy, x, w, mean, rstd, dx, None, None)
    assert torch.equal(dx, first[0])
    db = torch.empty(1000, device="cuda")
    ws = torch.empty(nv.lib().nvfp4_layernorm_backward_workspace_bytes(3000, 1000), dtype=torch.uint8, device="cuda")
    nv.nvfp4_layernorm_backward(dy, x, w, mean, rstd, dx, None, db, workspace=ws)
    assert torch.equal(db, first[2])


def test_graph_and_stream(nv):
    """Forward and gradient captured in a graph and replayed, and run on another stream, give the eager bits."""
    g = _gen(17)
    x, dy = _rand(g, 300, 640, torch.bfloat16), _rand(g, 300, 640, torch.bfloat16)
    w, b = torch.randn(640, device="cuda"), torch.randn(640, device="cuda")

    def step(stream=None):
        y, mean, rstd, _ = nv.layernorm(x, w, b, stream=stream)
        return (y, mean, rstd) + tuple(nv.layernorm_backward(dy, x, w, mean, rstd, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(_rand(_gen(20 + k), 300, 640, torch.bfloat16))
        want = step()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, out)), k
