"""Block operators at the edges of what their contracts allow: values that are not
finite in the maxima, batches and lists of nothing."""
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


def rand(*shape, seed=1, dtype=B, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)


def quantised(nv, rows, cols, seed):
    return nv.quantize(rand(rows, cols, seed=seed), [nv.QuantSpec.of("row")])[0]


# few rows, tiles of 128, tiles of 256
@pytest.mark.parametrize("rows,cols", [(48, 80), (208, 144), (8192, 2048)], ids=str)
@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh", "relu"])
def test_maxima_of_gated_gradients_keep_a_nan(nv, rows, cols, activation):
    """As nvfp4_gemm_amax's do: a gradient that is not a number is not hidden by the ones beside it, nor hides an infinity."""
    say("gated gradient, NaN", rows, cols, activation)
    dy, w = quantised(nv, rows, 128, 1), quantised(nv, cols, 128, 2)
    gate, up = rand(rows, cols, seed=3), rand(rows, cols, seed=4)
    top = torch.zeros(2, device="cuda")
    gate[rows - 5, cols - 7] = float("nan")
    dgate, dup = nv.gemm_gated_backward(dy, w, gate, up, activation, amax_gate=top[:1], amax_up=top[1:])
    assert torch.isnan(dup[rows - 5, cols - 7]) and torch.isnan(top[1])
    assert torch.isnan(dgate).any() == torch.isnan(top[0])
    gate[rows - 5, cols - 7] = 1.0
    up[rows - 5, cols - 7] = float("inf")
    top.zero_()
    dgate, dup = nv.gemm_gated_backward(dy, w, gate, up, activation, amax_gate=top[:1], amax_up=top[1:])
    assert torch.isinf(dgate[rows - 5, cols - 7]) and torch.isinf(top[0]) and top[1] == dup.abs().max().float()


@pytest.mark.parametrize("rows,cols", [(48, 80), (208, 144), (4096, 2048)], ids=str)
def test_maxima_of_gated_products_keep_a_nan(nv, rows, cols):
    """An operand's scale that is not a number reaches h's maximum."""
    say("gated, NaN", rows, cols)
    a, g, u = quantised(nv, rows, 2048, 1), quantised(nv, cols, 2048, 2), quantised(nv, cols, 2048, 3)
    top = torch.zeros(1, device="cuda")
    a.scales.view(-1)[rows // 2 * 128 + 3] = 0x7F
    h, _, _ = nv.gemm_gated(a, g, u, keep=False, amax=top)
    assert torch.isnan(h[rows // 2]).all() and torch.isnan(h).sum() == cols and torch.isnan(top)


def test_maximum_of_a_step_keeps_a_nan(nv):
    say("muon, NaN")
    p, g = rand(70, 90, seed=5, dtype=torch.float32), rand(70, 90, seed=6, dtype=torch.float32)
    g[3, 4] = float("nan")
    top = torch.zeros(1, device="cuda")
    nv.muon([nv.MuonTensor(p, g, amax=top)], 0.1)
    assert torch.isnan(p).any() and torch.isnan(top)


@pytest.mark.parametrize("placed", [False, True], ids=["counted", "positions"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_rotation_of_an_empty_batch(nv, placed, norm):
    """No sequences, whether their tokens' positions are counted or given: empty results, zero gradients of the weights."""
    say("rope, no sequences", placed, norm)
    q, k = rand(0, 5, 8, 64), rand(0, 5, 2, 64)
    freqs, _ = nv.rope_frequencies(64)
    w = torch.ones(64, device="cuda") if norm else None
    opts = dict(positions=torch.empty(0, dtype=torch.int64, device="cuda") if placed else None, q_weight=w, k_weight=w)
    a, b = nv.qk_rope(q, k, freqs, **opts)
    assert a.shape == q.shape and b.shape == k.shape
    nv.nvfp4_qk_rope(q, k, a, b, freqs, **opts)
    dq, dk, dqw, dkw = nv.qk_rope_backward(a, b, freqs, q, k, **opts)
    assert dq.shape == q.shape and dk.shape == k.shape
    assert not norm or not (dqw.any() or dkw.any())
    with pytest.raises(ValueError):
        nv.qk_rope(q, k, freqs, positions=torch.zeros(5, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("heads,kv", [(0, 3), (3, 0)], ids=str)
@pytest.mark.parametrize("given", [False, True], ids=["allocated", "given"])
def test_weights_of_no_heads_have_a_gradient_of_zero(nv, heads, kv, given):
    say("rope, a side of no heads", heads, kv, given)
    both = rand(1, 9, 3, 64)
    freqs, _ = nv.rope_frequencies(64)
    w = torch.ones(64, device="cuda")
    sides = [both[:, :, :n] for n in (heads, kv)]
    opts = dict(q_weight=w, k_weight=w)
    outs = nv.qk_rope(*sides, freqs, **opts)
    want, _ = nv.qk_rope(both, None, freqs, q_weight=w)
    assert torch.equal(outs[1 if kv else 0], want) and outs[0 if kv else 1].numel() == 0
    _, _, dw, _ = nv.qk_rope_backward(want, None, freqs, both, None, q_weight=w)
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        torch.full((4096,), float("nan"), device="cuda")  # (what an uninitialised result may find)
        if given:
            got = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
            torch.cuda.synchronize()
            nv.nvfp4_qk_rope_backward(*outs, *(torch.empty_like(t) for t in sides), freqs, *sides, dq_weight=got[0], dk_weight=got[1],
                                      stream=stream, **opts)
        else:
            got = nv.qk_rope_backward(*outs, freqs, *sides, stream=stream, **opts)[2:]
        torch.cuda.synchronize()
        assert torch.equal(got[1 if kv else 0], dw) and not got[0 if kv else 1].any()


def test_gated_operands_that_are_not_what_they_say_are_refused(nv):
    """Before any launch: buffers that are too small, on other devices, with gaps."""
    say("gated operands refused")
    a, w, x = quantised(nv, 64, 128, 1), quantised(nv, 96, 128, 2), rand(64, 96)
    two = nv.quantize(rand(96, 128), [nv.QuantSpec.of("2d")])[0]

    def other(q, **kw):
        kw = {**dict(codes=q.codes, scales=q.scales, global_scale=q.global_scale, amax=q.amax, rows=q.rows, cols=q.cols, scale_kind=q.scale_kind), **kw}
        return nv.QTensor(**kw)

    assert nv.gemm_gated(a, w, other(two))[0].shape == x.shape
    more = other(w, codes=torch.cat([w.codes, w.codes]), scales=torch.cat([w.scales, w.scales]))  # (what lies behind is not read)
    assert torch.equal(nv.gemm_gated(a, more, w)[0], nv.gemm_gated(a, w, w)[0])
    for bad in (other(w, codes=w.codes[:95]), other(w, scales=w.scales[:95]), other(w, scales=w.scales.cpu()), other(w, global_scale=w.global_scale.cpu()),
                other(w, global_scale=w.global_scale.double()), other(w, codes=torch.cat([w.codes, w.codes], 1)[:, :64]),
                other(w, scales=torch.cat([w.scales, w.scales], 1)[:, :8]), other(w, global_scale=w.global_scale[:0]), other(two, scale_kind=nv.SCALE_1D16),
                other(two, scales=two.scales[:5])):
        for call in (lambda: nv.gemm_gated(a, bad, w), lambda: nv.gemm_gated(a, w, bad), lambda: nv.gemm_gated(bad, w, w),
                     lambda: nv.gemm_gated_backward(a, bad, x, x)):
            with pytest.raises(ValueError):
                call()
