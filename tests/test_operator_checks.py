"""CPU checks of the argument validation of nsn_dequantize_kv: refused before any launch."""
import ctypes

import pytest

from calibration_free_vector_b200 import nsn
from calibration_free_vector_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return nsn.load()


def cache(batch=2, heads=2, capacity=256, window=128, mode=2, dq=0):
    return nsn.nsn_cache(batch, heads, capacity, window, mode, 1, 16, 16, 16, 16, 16, 16, 16, None, dq, 16 if dq else None,
                         16 if dq else None)


@pytest.mark.parametrize("change,status", [
    (dict(codebook=None), 1), (dict(codebook=20), 1), (dict(out=None), 1), (dict(out=24), 1), (dict(dtype=3), 1),
    (dict(start=-1), 1), (dict(n=-1), 1), (dict(st=260), 1), (dict(sb=-65536), 1),
    (dict(sh=0), 1), (dict(st=0), 1),                          # rows on top of each other
    (dict(sh=64), 1), (dict(st=128, sh=128), 1), (dict(sb=256 * 99), 1), (dict(sb=2 ** 62), 1),
    (dict(n=0, out=None), 0), (dict(start=10 ** 6), 0),         # nothing to do
])
def test_readback_arguments(lib, change, status):
    a = dict(start=0, n=100, codebook=16, out=16, dtype=1, sb=256 * 100, st=256, sh=128) | change
    c = cache()
    assert lib.nsn_dequantize_kv(ctypes.byref(c), a["start"], a["n"], a["codebook"], a["out"], a["dtype"], a["sb"], a["st"],
                                 a["sh"], None) == status


def test_readback_refuses_a_bad_cache(lib):
    args = (0, 100, 16, 16, 1, 256 * 100, 256, 128, None)
    assert lib.nsn_dequantize_kv(None, *args) == 1
    assert lib.nsn_dequantize_kv(ctypes.byref(cache(capacity=100)), *args) == 1
    assert lib.nsn_dequantize_kv(ctypes.byref(cache(window=64)), *args) == 2
