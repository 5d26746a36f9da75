"""Refusals of the chunk-attention and 8-bit-cache entry points that the host
can see, without touching a GPU.  As in test_abi.py, the checks that need
non-null device pointers pass an address that is never dereferenced and run
only where no GPU is present."""
import ctypes

import pytest

from paged_kv_cache_150_gb300 import _lib

BAD, UNSUP = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
P = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return _lib.load()


def _no_gpu():
    try:
        import torch
        return not torch.cuda.is_available()
    except Exception:  # noqa: BLE001
        return True


def desc(nb=8, bs=16, hk=8, d=128, dt=_lib.PA_BF16, layout=0):
    return _lib.CacheDesc(nb, bs, hk, d, dt, layout)


def prefill(lib, c, n=2, t=10, h=32, splits=4, kernel=0, ptr=None, ws=1 << 30, mb=4, scale=1.0, wsp=None, q=None):
    o = _lib.PrefillOpts(splits, kernel)
    return lib.pa_prefill(ptr, q or ptr, ptr, ptr, ctypes.byref(c), ptr, mb, ptr, ptr, n, t, h, scale, wsp or ptr, ws,
                          ctypes.byref(o), None)


def decode8(lib, c, n=2, h=32, splits=4, kernel=0, ptr=None, ws=1 << 30, mb=4, scale=1.0, wsp=None, q=None):
    o = _lib.PrefillOpts(splits, kernel)
    return lib.pa_decode_fp8(ptr, q or ptr, ptr, ptr, ptr, ptr, ctypes.byref(c), ptr, mb, ptr, n, h, scale, wsp or ptr, ws,
                             ctypes.byref(o), None)


def test_prefill_refusals(lib):
    assert prefill(lib, desc()) == BAD  # null pointers
    assert prefill(lib, desc(), n=0) == _lib.PA_OK
    assert prefill(lib, desc(), t=0) == _lib.PA_OK
    for kw in (dict(n=-1), dict(t=-1), dict(h=0), dict(h=12), dict(splits=-1), dict(kernel=3)):
        assert prefill(lib, desc(), **kw) == BAD, kw
    for c in (desc(nb=0), desc(bs=0), desc(hk=0), desc(d=0), desc(dt=7), desc(dt=_lib.PA_FP8_E4M3), desc(layout=2),
              desc(nb=1 << 28)):
        assert prefill(lib, c) == BAD
    assert prefill(lib, desc(d=96)) == UNSUP
    assert prefill(lib, desc(hk=1), h=65) == UNSUP
    for c in (desc(dt=_lib.PA_F32), desc(d=256), desc(bs=4), desc(layout=_lib.PA_LAYOUT_SPLIT)):
        assert prefill(lib, c, kernel=_lib.PA_KERNEL_MMA) == UNSUP
    if not _no_gpu():
        return
    assert prefill(lib, desc(), ptr=P, ws=16) == _lib.PA_ERR_WORKSPACE
    assert prefill(lib, desc(), ptr=P, wsp=ctypes.c_void_p(0x1010)) == BAD
    assert prefill(lib, desc(), ptr=P, mb=0) == BAD
    assert prefill(lib, desc(), ptr=P, mb=1 << 30) == BAD
    assert prefill(lib, desc(), ptr=P, scale=float("nan")) == BAD
    assert prefill(lib, desc(), ptr=P, q=ctypes.c_void_p(0x1002)) == BAD
    assert prefill(lib, desc(), ptr=ctypes.c_void_p(0x1008), wsp=P) == BAD  # the caches' alignment


def test_prefill_workspace_grows_with_the_batch(lib):
    def need(n, t, splits=152):
        o = _lib.PrefillOpts(splits, 0)
        return lib.pa_prefill_workspace_bytes(ctypes.byref(desc()), n, t, 32, ctypes.byref(o))

    assert 0 < need(1, 1) <= need(64, 1) <= need(64, 100000) and need(1, 1, 8) < need(1, 1)
    assert lib.pa_prefill_workspace_bytes(ctypes.byref(desc(d=96)), 1, 1, 32, None) == 0


def test_decode_fp8_refusals(lib):
    f8 = dict(dt=_lib.PA_FP8_E4M3)
    assert decode8(lib, desc(**f8)) == BAD
    assert decode8(lib, desc(**f8), n=0) == _lib.PA_OK
    for c in (desc(), desc(dt=_lib.PA_F32), desc(nb=0, **f8), desc(layout=5, **f8), desc(nb=1 << 28, **f8)):
        assert decode8(lib, c) == BAD
    assert decode8(lib, desc(layout=_lib.PA_LAYOUT_SPLIT, **f8)) == UNSUP
    assert decode8(lib, desc(d=96, **f8)) == UNSUP
    assert decode8(lib, desc(**f8), h=128) == UNSUP
    for kw in (dict(n=-1), dict(h=12), dict(splits=-2), dict(kernel=-1)):
        assert decode8(lib, desc(**f8), **kw) == BAD
    assert decode8(lib, desc(d=256, **f8), kernel=_lib.PA_KERNEL_MMA) == UNSUP
    assert decode8(lib, desc(bs=4, **f8), kernel=_lib.PA_KERNEL_MMA) == UNSUP
    if not _no_gpu():
        return
    assert decode8(lib, desc(**f8), ptr=P, ws=16) == _lib.PA_ERR_WORKSPACE
    assert decode8(lib, desc(**f8), ptr=P, wsp=ctypes.c_void_p(0x1010)) == BAD
    assert decode8(lib, desc(**f8), ptr=P, q=ctypes.c_void_p(0x1002)) == BAD
    assert decode8(lib, desc(**f8), ptr=P, scale=float("nan")) == BAD


def test_rows_and_copies_refusals(lib):
    f8 = desc(dt=_lib.PA_FP8_E4M3)

    def write(c, t=4, dt=_lib.PA_BF16, p=None):
        return lib.pa_reshape_and_cache_fp8(p, p, dt, p, t, p, p, p, p, ctypes.byref(c), None)

    def read(c, t=4, dt=_lib.PA_BF16, p=None):
        return lib.pa_gather_cache_fp8(p, p, dt, p, t, p, p, p, p, ctypes.byref(c), None)

    for call in (write, read):
        assert call(f8) == BAD and call(f8, t=-1) == BAD and call(f8, t=0) == _lib.PA_OK
        assert call(f8, dt=_lib.PA_FP8_E4M3) == BAD and call(f8, dt=9) == BAD
        assert call(desc()) == BAD and call(desc(d=0, dt=2)) == BAD
        if _no_gpu():
            assert call(f8, p=ctypes.c_void_p(0x1001)) == BAD
    assert lib.pa_copy_blocks_fp8(None, None, None, None, ctypes.byref(f8), None, 0, None) == _lib.PA_OK
    assert lib.pa_copy_blocks_fp8(None, None, None, None, ctypes.byref(f8), None, 2, None) == BAD
    assert lib.pa_copy_blocks_fp8(None, None, None, None, ctypes.byref(f8), None, -2, None) == BAD
    assert lib.pa_copy_blocks_fp8(None, None, None, None, ctypes.byref(desc()), None, 2, None) == BAD
    # the plain cache's calls do not take an 8-bit descriptor
    assert lib.pa_copy_blocks(None, None, ctypes.byref(f8), None, 1, None) == BAD
    assert lib.pa_reshape_and_cache(None, None, None, 4, None, None, ctypes.byref(f8), None) == BAD
