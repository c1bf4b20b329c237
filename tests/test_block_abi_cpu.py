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
