"""Layer norm and its gradient with outputs in the place of inputs, at widths that
end in a group of eight elements of which some are the neighbour's: the results
are those of buffers apart, bit for bit, and nothing past the rows is written."""
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


# below a group; a wave's border (the last group's neighbour is another wave's) and beside it, for each split; many rows
WIDTHS = [(5, 3), (40, 9), (9, 513), (70, 777), (6, 1025), (700, 1031), (5, 2049), (40, 5119), (300, 5121), (3, 8193), (9, 9223),
          (3, 16385), (40, 18433), (2, 32767)]


def _copy(t):
    """A copy with the rows' distance of t, as a view of a buffer whose other columns are NaN."""
    b = torch.full(t._base.shape, float("nan"), dtype=t.dtype, device="cuda")
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def _make(g, rows, cols, dtype, scale=1.0):
    b = torch.full((rows, cols + 3), float("nan"), dtype=dtype, device="cuda")
    b[:, :cols] = (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(dtype)
    return b[:, :cols]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_in_place(nv, rows, cols, dtype):
    say("layernorm in place", rows, cols, dtype)
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, r, dy, ds = (_make(g, rows, cols, dtype) for _ in range(4))
    w, b = torch.randn(cols, generator=g, device="cuda"), torch.randn(cols, generator=g, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    y, m, s, _ = nv.layernorm(x, w, b)
    t = _copy(x)
    nv.nvfp4_layernorm(t, w, b, 1e-5, t, mean, rstd)
    assert torch.equal(t, y) and torch.equal(mean, m) and torch.equal(rstd, s)
    assert t._base[:, cols:].isnan().all()

    y, m, s, total = nv.layernorm(x, w, b, residual=r)
    for swap in (False, True):  # y in x and the sum in the residual, and the other way round
        t, u = _copy(x), _copy(r)
        nv.nvfp4_layernorm(t, w, b, 1e-5, u if swap else t, mean, rstd, u, t if swap else u)
        got = (u, t) if swap else (t, u)
        assert torch.equal(got[0], y) and torch.equal(got[1], total) and torch.equal(mean, m) and torch.equal(rstd, s)
        assert t._base[:, cols:].isnan().all() and u._base[:, cols:].isnan().all()

    want = nv.layernorm_backward(dy, total, w, m, s, dsum=ds)
    ws = torch.empty(nv.lib().nvfp4_layernorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    for place in range(3):  # dx in dy, in x and in dsum
        t = [_copy(dy), _make(g, rows, cols, dtype).copy_(total), _copy(ds)]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        nv.nvfp4_layernorm_backward(t[0], t[1], w, m, s, t[place], dw, db, t[2], None, ws)
        assert torch.equal(t[place], want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2]), place
        assert t[place]._base[:, cols:].isnan().all()
