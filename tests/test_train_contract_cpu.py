"""CPU-only checks of what the training operators' entry points accept and
refuse at the borders of their contracts."""
import ctypes
import os

import pytest

import nvfp4_bit_quantization_amd as nv
from test_train_abi_cpu import ALIGN, FAKE, LD, NULL, SHAPE, UNSUPPORTED, VALUE, WORKSPACE, _adam, _config, _heads, _shape


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_bit_quantization_amd import build
        build.build()
    return nv.lib()


@pytest.mark.parametrize("eps,status", [(1e-45, VALUE), (1.17e-38, VALUE), (2.0 ** -126, 0), (1e-20, 0)])
def test_adamw_eps_is_normal(L, eps, status):
    """The reciprocal instruction takes subnormal numbers for zero."""
    arr = (nv.nvfp4_adamw_tensor * 1)(_adam(n=0))  # nothing to launch
    assert L.nvfp4_adamw(arr, 1, ctypes.byref(_config(eps=eps)), None) == status
