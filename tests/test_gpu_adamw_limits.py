"""AdamW where numbers leave the normal range, and where a step is smaller than
what 8 bits resolve, against the formulas in 64 bits."""
import numpy as np
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ULP, LEAST_NORMAL, HALF_LEAST = 2.0 ** -24, 2.0 ** -126, 2.0 ** -150


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_bit_quantization_amd as nv
    nv.lib()
    return nv


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 1e-20, LEAST_NORMAL])
def test_small_gradients(nv, bits, eps):
    """First steps on gradients of 1e-23 to 1e-12, whose squares are subnormal in binary32 up to some 1e-18, and on
    zeros.  A product or sum of subnormal result is off by half of 2^-149, any other by 2^-24 of itself; the update's
    other dozen operations by 16 * 2^-24."""
    say("adamw small gradients", bits, eps)
    n, lr, b1, b2 = 1024, float(np.float32(1e-3)), 0.9, 0.999
    g = np.float32(10.0 ** np.linspace(-23, -12, n)) * np.where(np.arange(n) % 3 == 1, -1, 1).astype(np.float32)
    g[::7] = 0
    p = torch.zeros(n, device="cuda")
    t = nv.adamw_tensor(p, torch.from_numpy(g).cuda(), state_bits=bits)
    nv.adamw([t], lr=1e-3, beta1=b1, beta2=b2, eps=eps, step=1, rounding="sr", seed=5)
    got, x, eps = p.double().cpu().numpy(), g.astype(np.float64), float(np.float32(eps))
    v = (1 - b2) * x * x
    tv = 4 * ULP * v + 2 * HALF_LEAST
    step = [lr * np.abs(x) / (np.sqrt(np.maximum(w, 0) / (1 - b2)) + eps) for w in (v + tv, v - tv)]
    assert np.isfinite(got).all()
    assert (got[x == 0] == 0).all()
    live = x != 0
    low, high = step[0] * (1 - 16 * ULP) - HALF_LEAST, step[1] * (1 + 16 * ULP) + HALF_LEAST
    assert ((got[live] < 0) == (x[live] > 0)).all()
    bad = live & ((np.abs(got) < low) | (np.abs(got) > high))
    assert not bad.any(), "%d updates; the first: gradient %g moved %g instead of %g" % (
        bad.sum(), x[bad][0], got[bad][0], step[0][bad][0])
    root = t.v.cpu().numpy()
    sure = v - tv > 0
    assert ((root & 127 if bits == 8 else root)[sure] > 0).all(), "a root is stored as zero"


def test_default_rounding_keeps_v_moving(nv):
    """300 default steps with 8-bit states on a constant gradient: a step moves the root by at most 0.05 % of it, where
    its format's steps are 6 to 12 %.  Stochastic rounding keeps the root's mean and adds to its square at most the
    root's way times a step of an eighth of it, which sums to 1/16 of v; 65536 elements leave the mean within 1 %.
    The root's spread, 1/16 of its square as well, raises the mean of its inverse by about as much."""
    n, g, lr = 65536, 1e-3, 1e-3
    p = torch.zeros(n, device="cuda")
    plan = nv.AdamWList([nv.adamw_tensor(p, torch.full((n,), g, device="cuda"), state_bits=8)])
    for step in range(1, 301):
        nv.adamw(plan, lr=lr, step=step, seed=3)
        if step in (1, 10, 100, 300):
            v = nv.adamw_state_values(plan.tensors[0])[1].double().mean().item()
            want = g * g * (1 - 0.999 ** step)
            assert 0.99 * want <= v <= 1.01 * (1 + 1 / 16) * want, (step, v / want)
            moved = -p.double().mean().item() / (lr * step)
            assert 0.95 <= moved <= 1.15, (step, moved)


def test_default_rounding_of_32_bit_states_is_to_nearest(nv):
    p = [torch.full((4096,), 1.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    grad = torch.ones(4096, device="cuda")
    for q, kw in zip(p, (dict(), dict(rounding="rtn"))):
        nv.adamw([nv.adamw_tensor(q, grad)], lr=2.0 ** -10, step=1, **kw)
    assert torch.equal(p[0], p[1])


@pytest.mark.parametrize("rounding", ["rtn", "sr"])
def test_conversion_is_the_rule(nv, rounding):
    """8-bit states hold exactly the neighbour that their value and uniform give: with beta1 = 0 and zero states m is the
    gradient, here values of every binade of E4M3 below a maximum that fixes the block's scale."""
    from test_gpu_adamw import e4m3_parts, uniforms
    n, seed = 1 << 20, 0x9876543210
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.exp2(torch.rand(n, generator=gen, device="cuda") * 21 - 12) * torch.sign(
        torch.rand(n, generator=gen, device="cuda") - 0.5)
    x[1::5] = torch.round(x[1::5] * 512) / 512          # ties and exact values
    x = x.clamp(-448, 448)
    x[::32] = 448
    t = nv.adamw_tensor(torch.zeros(n, device="cuda"), x, state_bits=8)
    nv.adamw([t], lr=0.0, beta1=0.0, step=3, rounding=rounding, seed=seed)
    assert (t.m_scale == 127).all()
    y = x.abs().double().cpu().numpy()
    quantum = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6) - 3)
    place = y / quantum
    want = np.floor(place + uniforms(n, 0, 0, 3, seed)) if rounding == "sr" else np.rint(place)
    codes = t.m.cpu().numpy()
    got, _ = e4m3_parts(codes)
    assert np.array_equal(got, want * quantum)
    assert ((codes >= 128) == (x.cpu().numpy() < 0)).all()
