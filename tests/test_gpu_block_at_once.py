"""Calls of the block operators that run at the same time, long matrices in captured graphs, and values that are not finite."""
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


def flat(x):
    return [t for y in x for t in (flat(y) if isinstance(y, (list, tuple)) else [y]) if t is not None]


def calls(nv, seed):
    """Calls of every operator on inputs of their own, each of which allocates what it needs."""
    freqs, _ = nv.rope_frequencies(64)
    q, k = rand(2, 700, 8, 128, seed=seed), rand(2, 700, 2, 128, seed=seed + 1)
    w = rand(128, seed=seed + 2, dtype=torch.float32)
    spec = nv.QuantSpec.of("row")
    few, a, wg, wu = (nv.quantize(rand(r, 384, seed=seed + i, size=0.1), [spec])[0] for i, r in enumerate((32, 1040, 5136, 5136)))
    gate, up = rand(1040, 5136, seed=seed + 6), rand(1040, 5136, seed=seed + 7)
    xs = [rand(1030, 2200, seed=seed + 8), rand(500, 300, seed=seed + 9, dtype=torch.float32), rand(64, 64, seed=seed + 10)]

    def step():
        p = [x.float().clone() for x in xs]  # (float() of a float32 matrix is itself)
        nv.muon([nv.MuonTensor(x, g, torch.zeros_like(x)) for x, g in zip(p, xs)], 0.1)
        return p
    return [lambda: nv.qk_rope(q, k, freqs, q_weight=w, k_weight=w), lambda: nv.qk_rope_backward(q, k, freqs, q, k, q_weight=w, k_weight=w),
            lambda: nv.gemm_gated(few, wg, wu), lambda: nv.gemm_gated(a, wg, wu), lambda: nv.gemm_gated_backward(a, wg, gate, up),
            lambda: nv.orthogonalize(xs), step]


def test_two_of_each_at_once(nv):
    say("block operators on two streams")
    both = calls(nv, 20), calls(nv, 60)
    want = [[flat(f()) for f in side] for side in both]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for turn in range(4):
        got = [[], []]
        for i in range(len(both[0])):
            for s in range(2):
                with torch.cuda.stream(streams[s]):
                    got[s].append(flat(both[s][(i + s * turn) % len(both[s])]()))
        torch.cuda.synchronize()
        for s in range(2):
            for i, now in enumerate(got[s]):
                for x, y in zip(now, want[s][(i + s * turn) % len(both[s])]):
                    assert torch.equal(x, y)


def test_long_steps_in_two_graphs(nv):
    """Two captured steps of long matrices with a workspace each, replayed at once with eager work between."""
    say("muon long, two graphs")
    sides = []
    for seed in (3, 4):
        p, m = rand(2100, 1040, seed=seed, dtype=torch.float32), torch.zeros(2100, 1040, device="cuda")
        g = rand(2100, 1040, seed=seed + 10)
        lst = nv.MuonList([nv.MuonTensor(p, g, m, copy=torch.empty(2100, 1040, dtype=B, device="cuda"))])
        ws = lst.new_workspace()
        p0 = p.clone()
        nv.muon(lst, 0.01, workspace=ws)  # the eager result of three steps
        nv.muon(lst, 0.01, workspace=ws)
        nv.muon(lst, 0.01, workspace=ws)
        want = p.clone(), m.clone()
        p.copy_(p0)
        m.zero_()
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            nv.muon(lst, 0.01, workspace=ws)
        sides.append((graph, stream, p, m, want, lst, ws))  # a graph does not hold its memory
    for turn in range(3):
        for graph, stream, *_ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
        nv.orthogonalize(rand(300, 200, seed=turn))
        torch.cuda.synchronize()
    for _, _, p, m, want, _, _ in sides:
        assert torch.equal(p, want[0]) and torch.equal(m, want[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_with_their_own(nv, bad):
    say("block operators, not finite", bad)
    xs = [rand(*s, seed=i, dtype=torch.float32) for i, s in enumerate([(1040, 1600), (1040, 1600), (70, 90), (70, 90)])]
    want = nv.orthogonalize(xs)
    xs[1][7, 9] = xs[3][60, 80] = bad
    got = nv.orthogonalize(xs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.isnan(got[1]).any() and torch.isnan(got[3]).any()  # a step of such a gradient does not pass for one
    q = rand(1, 50, 8, 128)
    freqs, _ = nv.rope_frequencies(64)
    w = torch.ones(128, device="cuda")
    want, _ = nv.qk_rope(q, None, freqs, q_weight=w)
    q[0, 20, 3, 100] = bad
    got, _ = nv.qk_rope(q, None, freqs, q_weight=w)
    assert not torch.isfinite(got[0, 20, 3]).all()
    got[0, 20, 3] = want[0, 20, 3]
    assert torch.equal(got, want)
    dq, _, dw, _ = nv.qk_rope_backward(want, None, freqs, q, None, q_weight=w)
    assert not torch.isfinite(dw).all() and not torch.isfinite(dq[0, 20, 3]).all()
    dq[0, 20, 3] = 0
    assert torch.isfinite(dq).all()
    # gates that are not finite reach their own elements
    a, b = (nv.quantize(rand(r, 128, seed=r), [nv.QuantSpec.of("row")])[0] for r in (64, 80))
    gate, up = rand(64, 80, seed=5), rand(64, 80, seed=6)
    want = nv.gemm_gated_backward(a, b, gate, up)
    gate[5, 6] = bad
    got = nv.gemm_gated_backward(a, b, gate, up)
    for x, y in zip(got, want):
        assert not torch.isfinite(x[5, 6]) or bad == float("inf")
        x[5, 6] = y[5, 6]
        assert torch.equal(x, y)
