"""Attention and its gradient at the borders of what the entry points take,
against the formulas in 64 bits (bounds: test_gpu_attention.py)."""
import pytest

from gpu_util import say
from test_gpu_attention import _check_sequence, _rand, _run, _see

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


@pytest.mark.parametrize("power,ones", [(-120, 58), (-120, 0), (120, -60)])
def test_scale_borders(nv, power, ones):
    """The least and the largest scale, with queries and keys of 2^ones: scores of some units, or next to zero."""
    say("attention scale", power, ones)
    g = torch.Generator(device="cuda").manual_seed(power + ones)
    q, k, v = _rand(g, 1, 200, 4, 64), _rand(g, 1, 200, 2, 64), _rand(g, 1, 200, 2, 64)
    q, k = q * 2.0 ** ones, k * 2.0 ** ones
    do = _rand(g, 1, 200, 4, 64, scale=1e-3)
    o, lse, dq, dk, dv = _run(nv, q, k, v, do, scale=2.0 ** power)
    _check_sequence(q[0], k[0], v[0], do[0], o[0], lse, dq[0], dk[0], dv[0], _see(200, 200, True, 0), 2.0 ** power, "scale")


@pytest.mark.parametrize("most", [0, 5])
@pytest.mark.parametrize("nq,nk", [(0, 300), (300, 0), (0, 0)])
def test_no_tokens(nv, nq, nk, most):
    """Packed tensors without any tokens, under a maximum of 0 or above: queries without keys give 0 and -inf and have
    no gradient, keys without queries neither."""
    say("attention without tokens", nq, nk, most)
    g = torch.Generator(device="cuda").manual_seed(nq + nk)
    q, k, v = _rand(g, nq, 4, 64), _rand(g, nk, 2, 64), _rand(g, nk, 2, 64)
    cu = [torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32, device="cuda") for n in (nq, nk)]
    o, lse, dq, dk, dv = _run(nv, q, k, v, torch.ones_like(q), cu_q=cu[0], cu_k=cu[1], max_q=nq or most, max_k=nk or most)
    assert o.shape == dq.shape == q.shape and dk.shape == dv.shape == k.shape and lse.shape == (4, nq)
    assert all((t == 0).all() for t in (o, dq, dk, dv)) and (lse == -float("inf")).all()


def test_maximum_of_zero_cuts_to_nothing(nv):
    """Sequences are cut to the stated maximum: with one of 0 nothing is read or written."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (_rand(g, 40, 2, 64) for _ in range(3))
    cu = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    for max_q, max_k in ((0, 40), (40, 0), (0, 0)):
        opts = dict(cu_q=cu, cu_k=cu, max_q=max_q, max_k=max_k)
        o, lse = torch.full_like(q, 7.0), torch.full((2, 40), 7.0, device="cuda")
        d = [torch.full_like(q, 7.0) for _ in range(3)]
        ws = nv.new_attention_workspace(q, k, v, **opts)
        nv.nvfp4_attention(q, k, v, o, lse, workspace=ws, **opts)
        nv.nvfp4_attention_backward(q, q, k, v, o, lse, *d, ws, **opts)
        assert (o == (0 if max_q else 7)).all() and (d[0] == (0 if max_q else 7)).all()
        assert (lse == (-float("inf") if max_q else 7)).all()
        assert all((t == (0 if max_k else 7)).all() for t in d[1:])


@pytest.mark.parametrize("nq,nk,causal", [(200, 200, True), (70, 1700, False), (1100, 90, False)])
def test_in_place(nv, nq, nk, causal):
    """o in the place of q, dq of o, dk and dv of k and v (and the other way round) give the bits that memory of their
    own gives; with few queries and with few keys the sums are split."""
    say("attention in place", nq, nk)
    g = torch.Generator(device="cuda").manual_seed(nq)
    q, k, v, do = (_rand(g, 1, n, 4, 64) for n in (nq, nk, nk, nq))
    o, lse, dq, dk, dv = _run(nv, q, k, v, do, causal=causal)
    ws = nv.new_attention_workspace(q, k, v, causal=causal)
    t = q.clone()
    nv.nvfp4_attention(t, k, v, t, torch.empty_like(lse), causal=causal, workspace=ws)
    assert torch.equal(t, o)
    for swap in (False, True):
        a, b, c = o.clone(), k.clone(), v.clone()
        nv.nvfp4_attention_backward(do, q, b, c, a, lse, a, *((c, b) if swap else (b, c)), ws, causal=causal)
        assert torch.equal(a, dq) and torch.equal(c if swap else b, dk) and torch.equal(b if swap else c, dv)


def test_outputs_in_place_of_inputs_still_read_are_refused(nv):
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v, do = (_rand(g, 1, 64, 2, 64) for _ in range(4))
    o, lse = nv.attention(q, k, v)
    ws = nv.new_attention_workspace(q, k, v)
    for dq in (q, do):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_attention_backward(do, q, k, v, o, lse, dq, torch.empty_like(k), torch.empty_like(v), ws)


def test_expanded_workspaces_are_refused(nv):
    """Their size is not the memory that they have."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (_rand(g, 1, 64, 2, 64) for _ in range(3))
    wide = torch.empty(1, device="cuda").expand(1 << 20)
    o, lse = nv.attention(q, k, v)
    x, w = q.view(64, 128), torch.ones(128, device="cuda")
    _, mean, rstd, _ = nv.layernorm(x, w)
    for call in (lambda: nv.attention(q, k, v, workspace=wide), lambda: nv.attention_backward(q, q, k, v, o, lse, workspace=wide),
                 lambda: nv.nvfp4_attention(q, k, v, o, lse, workspace=wide),
                 lambda: nv.nvfp4_attention_backward(q, q, k, v, o, lse, *(torch.empty_like(q) for _ in range(3)), wide),
                 lambda: nv.layernorm_backward(x, x, w, mean, rstd, workspace=wide),
                 lambda: nv.nvfp4_layernorm_backward(x, x, w, mean, rstd, torch.empty_like(x), w.clone(), w.clone(), workspace=wide)):
        with pytest.raises(ValueError):
            call()
