"""CPU checks of the argument validation of nsn_dequantize_kv and the shared-prefix attention: refused before any launch."""
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


def prefix_call(lib, pk=None, pv=None, k=None, v=None, chunk=None, **change):
    pk, pv = pk or cache(batch=1), pv or cache(batch=1, mode=1)
    k, v = k or cache(), v or cache(mode=1)
    a = dict(q=16, dtype=1, heads=8, sb=1024, st=1024, sh=128, scale=0.1, cbk=16, cbv=16, out=16, odt=1, ws=256,
             bytes=1 << 40) | change
    refs = [ctypes.byref(c) for c in (pk, pv, k, v)]
    if chunk is None:
        return lib.nsn_decode_attention_prefix(*refs, a["q"], a["dtype"], a["heads"], a["sb"], a["sh"], a["scale"], a["cbk"],
                                               a["cbv"], a["out"], a["odt"], a["ws"], a["bytes"], None)
    return lib.nsn_extend_attention_prefix(*refs, a["q"], a["dtype"], a["heads"], chunk, a["sb"], a["st"], a["sh"], a["scale"],
                                           a["cbk"], a["cbv"], a["out"], a["odt"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("chunk", [None, 4])
@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(q=18), 1), (dict(dtype=5), 1), (dict(odt=-1), 1), (dict(heads=7), 1), (dict(heads=0), 1),
    (dict(heads=6), 2), (dict(heads=32), 2), (dict(sb=-1024), 1), (dict(sh=129), 1), (dict(cbk=None), 1), (dict(cbv=24), 1),
    (dict(out=None), 1), (dict(out=40), 1), (dict(ws=None), 1), (dict(ws=128), 1), (dict(bytes=1000), 3),
    (dict(scale=float("nan")), 1),
    (dict(pk=cache(batch=2)), 1), (dict(pk=cache(batch=1, heads=4)), 1), (dict(pk=cache(batch=1, mode=1)), 1),
    (dict(pk=cache(batch=1, dq=1)), 1), (dict(pv=cache(batch=1, mode=1, capacity=384)), 1), (dict(v=cache(mode=1, window=0)), 1),
    (dict(v=cache(mode=2)), 1), (dict(k=cache(capacity=100)), 1), (dict(k=cache(window=64)), 2),
])
def test_prefix_arguments(lib, chunk, change, status):
    assert prefix_call(lib, chunk=chunk, **change) == status


def test_extend_prefix_chunk_and_window(lib):
    assert prefix_call(lib, chunk=0) == 1
    assert prefix_call(lib, chunk=129) == 1
    assert prefix_call(lib, chunk=4, k=cache(window=0), v=cache(mode=1, window=0)) == 2


def test_prefix_workspace_size(lib):
    size = lambda k, heads, n, pk=None: lib.nsn_prefix_workspace_bytes(  # noqa: E731
        ctypes.byref(pk or cache(batch=1)), ctypes.byref(k), heads, n)
    assert size(cache(), 8, 1) > 0
    assert size(cache(), 8, 128) > size(cache(), 8, 1)
    assert size(cache(batch=64), 8, 1) > size(cache(), 8, 1)
    assert size(cache(), 7, 1) == 0 and size(cache(), 8, 0) == 0 and size(cache(), 8, 129) == 0
    assert size(cache(), 8, 1, cache(batch=2)) == 0
    assert size(cache(batch=1 << 24), 16, 128) == 0     # rows past what 32-bit counts allow
