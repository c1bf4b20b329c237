"""CPU-only checks of the block operators' entry points: every refusal comes from
the host before anything is enqueued (no GPU is touched)."""
import ctypes
import os

import pytest

import nvfp4_bit_quantization_amd as nv

FAKE = 0x10000  # aligned, not null, never dereferenced on the error paths
NULL, SHAPE, LD, ALIGN, UNSUPPORTED, WORKSPACE, VALUE = -1, -2, -3, -4, -5, -6, -8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_bit_quantization_amd import build
        build.build()
    return nv.lib()


def _heads(i, **kw):
    a = dict(data=FAKE * i, batch_stride=8 * 256, token_stride=256, head_stride=64)
    a.update(kw)
    return nv.nvfp4_heads(**a)


def _side(i, heads=4, **kw):
    a = dict(x=_heads(i), y=_heads(i + 1), dx=_heads(i + 2), weight=FAKE * 20, dweight=None, heads=heads)
    a.update(kw)
    return nv.nvfp4_rope_heads(**a)


def _rope(**kw):
    a = dict(q=_side(1), k=_side(4), batch=2, tokens=8, positions=None, cu=None, freqs=FAKE * 30, head_dim=64, rot_dim=64,
             interleaved=0, x_dtype=1, w_dtype=0, eps=1e-6, magnitude=1.0)
    a.update(kw)
    return nv.nvfp4_qk_rope_args(**a)


ROPE = [
    (dict(batch=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(batch=1 << 16, tokens=1 << 16), SHAPE), (dict(batch=1 << 31), SHAPE),
    (dict(q=_side(1, heads=-1)), SHAPE), (dict(q=_side(1, heads=65536)), SHAPE), (dict(q=_side(1, heads=0), k=_side(4, heads=0)), SHAPE),
    (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=60), UNSUPPORTED), (dict(head_dim=136), UNSUPPORTED),
    (dict(rot_dim=66), UNSUPPORTED), (dict(rot_dim=-2), UNSUPPORTED), (dict(rot_dim=33), UNSUPPORTED),
    (dict(interleaved=2), UNSUPPORTED), (dict(x_dtype=2), UNSUPPORTED), (dict(w_dtype=-1), UNSUPPORTED),
    (dict(positions=FAKE, cu=FAKE), UNSUPPORTED), (dict(k=_side(4, weight=None)), NULL), (dict(freqs=None), NULL),
    (dict(q=_side(1, weight=None), k=_side(4, weight=None), rot_dim=0), UNSUPPORTED),
    (dict(freqs=FAKE + 4), ALIGN), (dict(positions=FAKE + 4), ALIGN), (dict(cu=FAKE + 2), ALIGN),
    (dict(magnitude=float("inf")), VALUE), (dict(magnitude=float("nan")), VALUE), (dict(eps=0.0), VALUE), (dict(eps=-1.0), VALUE),
    (dict(eps=1e-45), VALUE), (dict(eps=float("nan")), VALUE),
    (dict(q=_side(1, weight=FAKE + 2)), ALIGN), (dict(q=_side(1, x=_heads(0))), NULL), (dict(q=_side(1, y=_heads(0))), NULL),
    (dict(q=_side(1, x=_heads(1, token_stride=-256))), LD), (dict(q=_side(1, x=_heads(1, head_stride=-64))), LD),
    (dict(q=_side(1, x=_heads(1, batch_stride=-8))), LD), (dict(q=_side(1, x=_heads(1, token_stride=252))), ALIGN),
    (dict(q=_side(1, x=nv.nvfp4_heads(FAKE + 8, 2048, 256, 64))), ALIGN), (dict(q=_side(1, x=_heads(1, batch_stride=2044))), ALIGN)]


@pytest.mark.parametrize("i", range(len(ROPE)))
def test_rope_refusals(L, i):
    change, status = ROPE[i]
    a = _rope(**change)
    assert L.nvfp4_qk_rope(ctypes.byref(a), None) == status
    assert L.nvfp4_qk_rope_backward(ctypes.byref(a), FAKE, 1 << 30, None) == status
    assert L.nvfp4_qk_rope_backward_workspace_bytes(ctypes.byref(a)) == 0


def test_rope_null(L):
    assert L.nvfp4_qk_rope(None, None) == NULL
    assert L.nvfp4_qk_rope_backward(None, None, 0, None) == NULL
    assert L.nvfp4_qk_rope_backward_workspace_bytes(None) == 0


FORWARD = [dict(q=_side(1, y=_heads(2, token_stride=0))), dict(q=_side(1, y=_heads(2, token_stride=56))),
           dict(q=_side(1, y=_heads(2, head_stride=56))), dict(q=_side(1, y=_heads(2, batch_stride=0)))]


@pytest.mark.parametrize("i", range(len(FORWARD)))
def test_rope_outputs_do_not_overlap_themselves(L, i):
    assert L.nvfp4_qk_rope(ctypes.byref(_rope(**FORWARD[i])), None) == LD


BACKWARD = [dict(q=_side(1, dx=_heads(3, token_stride=0))), dict(q=_side(1, dx=_heads(3, head_stride=56)))]


@pytest.mark.parametrize("i", range(len(BACKWARD)))
def test_rope_gradients_do_not_overlap_themselves(L, i):
    assert L.nvfp4_qk_rope_backward(ctypes.byref(_rope(**BACKWARD[i])), FAKE, 1 << 30, None) == LD


# outputs in the place of what others read, of each other, or of their own input with other strides or another type
CROSSED = [dict(q=_side(1, y=_heads(4))), dict(q=_side(1, y=_heads(5))), dict(k=_side(4, y=_heads(1))),
           dict(q=_side(1, y=_heads(1, token_stride=512))), dict(q=_side(1, y=_heads(1, head_stride=72, token_stride=512))),
           dict(q=_side(1, y=_heads(1, batch_stride=4096))), dict(q=_side(1, y=_heads(1)), x_dtype=0)]


@pytest.mark.parametrize("i", range(len(CROSSED)))
def test_rope_outputs_keep_off_what_is_read(L, i):
    assert L.nvfp4_qk_rope(ctypes.byref(_rope(**CROSSED[i])), None) == UNSUPPORTED


CROSSED_BACK = [dict(q=_side(1, dx=_heads(4))), dict(q=_side(1, dx=_heads(5))), dict(q=_side(1, dx=_heads(6))),
                dict(k=_side(4, dx=_heads(1))), dict(k=_side(4, dx=_heads(2))), dict(q=_side(1, dx=_heads(2)), x_dtype=0),
                dict(q=_side(1, dx=_heads(2, token_stride=512))), dict(q=_side(1, dx=_heads(1, batch_stride=4096))),
                dict(q=_side(1, dweight=FAKE * 40), k=_side(4, dweight=FAKE * 40)),
                dict(q=_side(1, weight=None, dweight=FAKE * 40), k=_side(4, weight=None))]


@pytest.mark.parametrize("i", range(len(CROSSED_BACK)))
def test_rope_gradients_keep_off_what_is_read(L, i):
    assert L.nvfp4_qk_rope_backward(ctypes.byref(_rope(**CROSSED_BACK[i])), FAKE, 1 << 30, None) == UNSUPPORTED


def test_rope_workspace(L):
    a = _rope(q=_side(1, dweight=FAKE * 40), k=_side(4, dweight=FAKE * 41))
    need = L.nvfp4_qk_rope_backward_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert L.nvfp4_qk_rope_backward(ctypes.byref(a), None, need, None) == WORKSPACE
    assert L.nvfp4_qk_rope_backward(ctypes.byref(a), FAKE, need - 1, None) == WORKSPACE
    assert L.nvfp4_qk_rope_backward(ctypes.byref(a), FAKE + 8, need, None) == ALIGN
    assert L.nvfp4_qk_rope_backward_workspace_bytes(ctypes.byref(_rope())) == 0  # no dweight
    assert L.nvfp4_qk_rope(ctypes.byref(_rope(q=_side(1, dweight=FAKE))), None) == UNSUPPORTED


def test_rope_of_nothing(L):
    none = dict(data=None)
    sides = dict(q=_side(1, x=_heads(1, **none), y=_heads(1, **none), dx=_heads(1, **none)),
                 k=_side(4, x=_heads(1, **none), y=_heads(1, **none), dx=_heads(1, **none)))
    a = _rope(tokens=0, cu=FAKE, **sides)
    assert L.nvfp4_qk_rope(ctypes.byref(a), None) == 0
    assert L.nvfp4_qk_rope_backward(ctypes.byref(a), None, 0, None) == 0


def _tensor(rows=32, cols=64, **kw):
    a = dict(codes=FAKE, scales=FAKE, global_scale=FAKE, amax=FAKE, rows=rows, cols=cols, scale_kind=0, rht=0)
    a.update(kw)
    return nv.nvfp4_tensor(**a)


def _matrix(i, **kw):
    a = dict(data=FAKE * i, ld=64, amax_plain=None, amax_rht_col=None)
    a.update(kw)
    return nv.nvfp4_gated_matrix(**a)


def _gated(L, activation=0, **kw):
    t = dict(a=_tensor(32), g=_tensor(48), u=_tensor(48), h=_matrix(2), gate=_matrix(3), up=_matrix(4))
    t.update(kw)
    p = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return L.nvfp4_gemm_gated(p(t["a"]), p(t["g"]), p(t["u"]), activation, p(t["h"]), p(t["gate"]), p(t["up"]), 0, None)


def _gated_back(L, activation=0, **kw):
    t = dict(a=_tensor(32), b=_tensor(48), gate=_matrix(3), up=_matrix(4), dgate=_matrix(5), dup=_matrix(6))
    t.update(kw)
    p = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return L.nvfp4_gemm_gated_backward(p(t["a"]), p(t["b"]), activation, p(t["gate"]), p(t["up"]), p(t["dgate"]), p(t["dup"]), 0, None)


OPERANDS = [(None, NULL), (_tensor(codes=None), NULL), (_tensor(scales=None), NULL), (_tensor(global_scale=None), NULL),
            (_tensor(rows=0), SHAPE), (_tensor(rows=40), SHAPE), (_tensor(cols=72), SHAPE), (_tensor(cols=0), SHAPE),
            (_tensor(scale_kind=2), UNSUPPORTED), (_tensor(codes=FAKE + 8), ALIGN)]


@pytest.mark.parametrize("i", range(len(OPERANDS)))
def test_gated_operands(L, i):
    t, status = OPERANDS[i]
    for name in "agu":
        assert _gated(L, **{name: t}) == status
    for name in "ab":
        assert _gated_back(L, **{name: t}) == status


def test_gated_shapes_and_activations(L):
    assert _gated(L, a=_tensor(32, 80)) == UNSUPPORTED
    assert _gated(L, u=_tensor(64, 64)) == UNSUPPORTED
    assert _gated(L, g=_tensor(48, 80), u=_tensor(48, 80)) == UNSUPPORTED
    assert _gated_back(L, a=_tensor(32, 80)) == UNSUPPORTED
    for bad in (-1, 4):
        assert _gated(L, activation=bad) == UNSUPPORTED
        assert _gated_back(L, activation=bad) == UNSUPPORTED
    big = _tensor(1 << 24)
    assert _gated(L, a=big, g=big, u=big, h=_matrix(2, ld=1 << 24)) == SHAPE
    assert _gated_back(L, a=big, b=big) == SHAPE
    wide = _tensor(1 << 28)
    for rows in (16, 64):
        assert _gated(L, a=_tensor(rows), g=wide, u=wide, h=_matrix(2, ld=1 << 28)) == SHAPE
        assert _gated_back(L, a=_tensor(rows), b=wide) == SHAPE


MATRICES = [(_matrix(0), NULL), (_matrix(9, ld=40), LD), (_matrix(9, ld=52), ALIGN), (nv.nvfp4_gated_matrix(FAKE + 8, 64, None, None), ALIGN),
            (_matrix(9, amax_plain=FAKE + 2), ALIGN), (_matrix(9, amax_rht_col=FAKE + 1), ALIGN)]


@pytest.mark.parametrize("i", range(len(MATRICES)))
def test_gated_matrices(L, i):
    t, status = MATRICES[i]
    for name in ("h", "gate", "up"):
        assert _gated(L, **{name: t}) == status
    for name in ("gate", "up", "dgate", "dup"):
        assert _gated_back(L, **{name: t}) == status


def test_gated_outputs_stand_apart(L):
    assert _gated(L, h=None) == NULL
    assert _gated(L, gate=_matrix(2)) == UNSUPPORTED
    assert _gated(L, up=_matrix(2)) == UNSUPPORTED
    assert _gated(L, up=_matrix(3)) == UNSUPPORTED
    assert _gated(L, gate=_matrix(3, amax_plain=FAKE)) == UNSUPPORTED
    assert _gated(L, up=_matrix(4, amax_rht_col=FAKE)) == UNSUPPORTED
    for name in ("gate", "up", "dgate", "dup"):
        assert _gated_back(L, **{name: None}) == NULL
    assert _gated_back(L, dup=_matrix(5)) == UNSUPPORTED
    for out in ("dgate", "dup"):
        for place in (3, 4):
            assert _gated_back(L, **{out: _matrix(place, ld=128)}) == UNSUPPORTED


def _muon_tensor(**kw):
    a = dict(param=FAKE * 2, grad=FAKE * 3, m=FAKE * 4, copy=FAKE * 5, update=FAKE * 6, amax=FAKE * 7, rows=40, cols=64,
             param_dtype=0, grad_dtype=1, weight_decay=0.1, scale=1.0)
    a.update(kw)
    return nv.nvfp4_muon_tensor(**a)


def _muon_config(**kw):
    a = dict(lr=0.01, momentum=0.95, nesterov=1, steps=5, a=3.4445, b=-4.775, c=2.0315, rounding=0, step=1, seed=0, grad_scale=None)
    a.update(kw)
    return nv.nvfp4_muon_config(**a)


def _muon(L, tensors, config, ws=FAKE, nbytes=1 << 40):
    arr = (nv.nvfp4_muon_tensor * len(tensors))(*tensors)
    return L.nvfp4_muon(arr, len(tensors), ctypes.byref(config), ws, nbytes, None)


NAN, INF = float("nan"), float("inf")
MUON = [(dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(rows=(1 << 17) + 1), SHAPE), (dict(rows=1 << 17, cols=(1 << 16) + 1), SHAPE),
        (dict(param_dtype=2), UNSUPPORTED), (dict(grad_dtype=-1), UNSUPPORTED), (dict(weight_decay=-0.1), VALUE),
        (dict(weight_decay=NAN), VALUE), (dict(scale=INF), VALUE), (dict(grad=None), NULL), (dict(param=None), UNSUPPORTED),
        (dict(param=None, copy=None, amax=None, update=None), NULL), (dict(grad=FAKE + 1), ALIGN), (dict(param=FAKE + 2), ALIGN),
        (dict(m=FAKE + 2), ALIGN), (dict(copy=FAKE + 1), ALIGN), (dict(update=FAKE + 1), ALIGN), (dict(amax=FAKE + 2), ALIGN),
        (dict(m=FAKE * 3), UNSUPPORTED), (dict(m=FAKE * 2), UNSUPPORTED), (dict(copy=FAKE * 2), UNSUPPORTED),
        (dict(update=FAKE * 5), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", MUON, ids=str)
def test_muon_tensors(L, change, status):
    assert _muon(L, [_muon_tensor(rows=0), _muon_tensor(**change)], _muon_config()) == status


CONFIGS = [(dict(lr=-1.0), VALUE), (dict(lr=NAN), VALUE), (dict(momentum=1.0), VALUE), (dict(momentum=-0.1), VALUE),
           (dict(nesterov=2), UNSUPPORTED), (dict(rounding=2), UNSUPPORTED), (dict(steps=0), VALUE), (dict(steps=17), VALUE),
           (dict(step=-1), VALUE), (dict(step=1 << 47), VALUE), (dict(a=NAN), VALUE), (dict(a=4.0, b=0.0, c=0.0), VALUE),
           (dict(a=-4.0, b=0.0, c=0.0), VALUE), (dict(c=9.0), VALUE), (dict(b=-40.0), VALUE), (dict(c=INF), VALUE),
           (dict(a=15.0, b=-12.0, c=0.0), VALUE), (dict(grad_scale=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("change,status", CONFIGS, ids=str)
def test_muon_configs(L, change, status):
    assert _muon(L, [_muon_tensor()], _muon_config(**change)) == status


@pytest.mark.parametrize("abc", [(3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (1.0, 0.0, 0.0), (0.0, 0.0, 0.0)])
def test_muon_iterations_that_stay_bounded(L, abc):
    a, b, c = abc
    for steps in (1, 5, 16):
        assert _muon(L, [_muon_tensor(rows=0)], _muon_config(a=a, b=b, c=c, steps=steps)) == 0  # nothing to do


def test_muon_bound_is_the_iterations_own(L):
    """The refusal goes by the largest singular value that the iteration can reach, here found on a grid."""
    import random
    r = random.Random(4)
    for _ in range(300):
        a, b, c = r.uniform(-4, 4), r.uniform(-8, 8), r.uniform(-4, 4)
        steps, top, high = r.randrange(1, 5), 1.0, 0.0
        worst = 0.0
        for _ in range(steps):
            grid = [top * i / 2000 for i in range(2001)]
            high = max(high, max(abs(a + b * s * s + c * s ** 4) for s in grid))
            top = max(s * abs(a + b * s * s + c * s ** 4) for s in grid)
            worst = max(worst, top)
            if worst > 3.5 or high > 14:
                break
        if abs(worst - 3.5) < 0.01 or abs(high - 14) < 0.05:
            continue  # the grid cannot say
        want = VALUE if worst > 3.5 or high > 14 else 0
        assert _muon(L, [_muon_tensor(rows=0)], _muon_config(a=a, b=b, c=c, steps=steps)) == want, (a, b, c, steps, worst, high)


def test_muon_workspace(L):
    t = [_muon_tensor(), _muon_tensor(rows=0), _muon_tensor(rows=2000, cols=1600, grad=FAKE * 9)]
    arr = (nv.nvfp4_muon_tensor * 3)(*t)
    need = L.nvfp4_muon_workspace_bytes(arr, 3)
    assert need >= 2 * (3 * 2000 * 1600 + 2 * 1600 * 1600)  # three of the iterate, two of its square
    c = _muon_config()
    assert _muon(L, t, c, None, need) == WORKSPACE
    assert _muon(L, t, c, FAKE, need - 1) == WORKSPACE
    assert _muon(L, t, c, FAKE + 8, need) == ALIGN
    assert L.nvfp4_muon_workspace_bytes(None, 1) == 0 and L.nvfp4_muon_workspace_bytes(arr, 0) == 0
    assert L.nvfp4_muon_workspace_bytes((nv.nvfp4_muon_tensor * 1)(_muon_tensor(rows=0)), 1) == 0
    assert L.nvfp4_muon(None, 1, ctypes.byref(c), FAKE, need, None) == NULL
    assert L.nvfp4_muon(arr, 3, None, FAKE, need, None) == NULL
    assert L.nvfp4_muon(arr, 0, ctypes.byref(c), FAKE, need, None) == SHAPE
