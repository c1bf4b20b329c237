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
