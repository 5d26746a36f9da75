"""Refusals of the tables', block-scaled cache's and cross attention's entry
points that the host can see, without touching a GPU.  As in test_abi.py, the
checks that need non-null device pointers pass an address that is never
dereferenced and run only where no GPU is present."""
import ctypes

import pytest

from paged_kv_cache_150_gb300 import _lib

OK, BAD, UNSUP = _lib.PA_OK, _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED
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


def desc(nb=8, bs=16, hk=8, d=128, dt=_lib.PA_FP8_E4M3_BLOCK, layout=0):
    return _lib.CacheDesc(nb, bs, hk, d, dt, layout)


def chunk(lib, name, c, n=2, t=10, h=32, splits=4, kernel=0, ptr=None, ws=1 << 30, mb=4, scale=1.0, wsp=None, q=None, sc=None):
    o = _lib.PrefillOpts(splits, kernel)
    scales = (sc or ptr, sc or ptr) if name == "pa_prefill_fp8" else ()
    return getattr(lib, name)(ptr, q or ptr, ptr, ptr, *scales, ctypes.byref(c), ptr, mb, ptr, ptr, n, t, h, scale,
                              wsp or ptr, ws, ctypes.byref(o), None)


@pytest.mark.parametrize("name,good", [("pa_cross", dict(dt=_lib.PA_BF16)), ("pa_prefill_fp8", {})])
def test_chunk_refusals(lib, name, good):
    def call(c, **kw):
        return chunk(lib, name, c, **kw)

    assert call(desc(**good)) == BAD  # null pointers
    assert call(desc(**good), n=0) == OK and call(desc(**good), t=0) == OK
    for kw in (dict(n=-1), dict(t=-1), dict(h=0), dict(h=12), dict(splits=-1), dict(kernel=3)):
        assert call(desc(**good), **kw) == BAD, kw
    for kw in (dict(nb=0), dict(bs=0), dict(hk=0), dict(d=0), dict(dt=7), dict(layout=2), dict(nb=1 << 28)):
        assert call(desc(**dict(good, **kw))) == BAD, kw
    assert call(desc(**dict(good, d=96))) == UNSUP
    assert call(desc(**dict(good, hk=1)), h=65) == UNSUP
    for kw in (dict(d=256), dict(bs=4)):
        assert call(desc(**dict(good, **kw)), kernel=_lib.PA_KERNEL_MMA) == UNSUP
    if name == "pa_prefill_fp8":
        assert call(desc(dt=_lib.PA_BF16)) == BAD and call(desc(dt=_lib.PA_F32)) == BAD
        assert call(desc(dt=_lib.PA_FP8_E4M3)) == UNSUP and call(desc(layout=1)) == UNSUP
    else:
        assert call(desc()) == BAD and call(desc(dt=_lib.PA_FP8_E4M3)) == BAD
    if not _no_gpu():
        return
    c = desc(**good)
    assert call(c, ptr=P, ws=16) == _lib.PA_ERR_WORKSPACE
    assert call(c, ptr=P, wsp=ctypes.c_void_p(0x1010)) == BAD
    assert call(c, ptr=P, mb=0) == BAD and call(c, ptr=P, mb=1 << 30) == BAD
    assert call(c, ptr=P, scale=float("nan")) == BAD
    assert call(c, ptr=P, q=ctypes.c_void_p(0x1002)) == BAD
    assert call(c, ptr=ctypes.c_void_p(0x1008), wsp=P) == BAD  # the caches' alignment


def test_workspaces(lib):
    o = _lib.PrefillOpts(152, 0)

    def need(c, n=64, t=1000):
        return lib.pa_prefill_fp8_workspace_bytes(ctypes.byref(c), n, t, 32, ctypes.byref(o))

    assert 0 < need(desc(), 1, 1) <= need(desc()) <= need(desc(), 64, 100000)
    assert need(desc(d=96)) == 0 and need(desc(dt=_lib.PA_FP8_E4M3)) == 0 and need(desc(dt=_lib.PA_BF16)) == 0
    assert lib.pa_decode_fp8_workspace_bytes(ctypes.byref(desc()), 64, 32, ctypes.byref(o)) > 0
    assert 0 < lib.pa_tables_workspace_bytes(0, 1) <= lib.pa_tables_workspace_bytes(100, 1) < lib.pa_tables_workspace_bytes(100, 5000)
    assert lib.pa_tables_workspace_bytes(-1, 4) == 0 and lib.pa_tables_workspace_bytes(1, 0) == 0


def test_write_and_other_calls_of_the_block_cache(lib):
    def write(c, n=2, t=4, dt=_lib.PA_BF16, p=None, mb=4, k=None):
        return lib.pa_write_blocks_fp8(k or p, p, dt, p, mb, p, p, n, t, p, p, p, p, ctypes.byref(c), None)

    assert write(desc()) == BAD and write(desc(), n=0) == OK and write(desc(), t=0) == OK
    assert write(desc(), n=-1) == BAD and write(desc(), t=-1) == BAD and write(desc(), dt=_lib.PA_FP8_E4M3) == BAD
    assert write(desc(dt=_lib.PA_FP8_E4M3)) == BAD and write(desc(dt=_lib.PA_BF16)) == BAD and write(desc(layout=1)) == UNSUP
    c = desc()
    assert lib.pa_reshape_and_cache_fp8(None, None, _lib.PA_BF16, None, 4, None, None, None, None, ctypes.byref(c), None) == UNSUP
    assert lib.pa_gather_cache_fp8(None, None, _lib.PA_BF16, None, 4, None, None, None, None, ctypes.byref(c), None) == BAD
    assert lib.pa_copy_blocks_fp8(None, None, None, None, ctypes.byref(c), None, 0, None) == OK
    assert lib.pa_copy_blocks_fp8(None, None, None, None, ctypes.byref(c), None, 2, None) == BAD
    assert lib.pa_copy_blocks(None, None, ctypes.byref(c), None, 1, None) == BAD
    o = _lib.PrefillOpts(4, 0)

    def decode(c, n=2, h=32, p=None, q=None, sc=None):
        return lib.pa_decode_fp8(p, q or p, p, p, sc or p, sc or p, ctypes.byref(c), p, 4, p, n, h, 1.0, p, 16,
                                 ctypes.byref(o), None)

    assert decode(c) == BAD and decode(c, n=0) == OK and decode(c, h=128) == UNSUP
    assert lib.pa_decode_fp8(None, None, None, None, None, None, None, None, 4, None, 2, 32, 1.0, None, 16, None, None) == BAD
    if not _no_gpu():
        return
    assert write(c, p=P, mb=0) == BAD and write(c, p=P, mb=1 << 30) == BAD
    assert write(c, p=P, k=ctypes.c_void_p(0x1001)) == BAD
    assert decode(c, p=P, sc=ctypes.c_void_p(0x1001)) == _lib.PA_ERR_WORKSPACE  # scales at any alignment


def test_tables_refusals(lib):
    def state(p=P, **kw):
        s = _lib.Tables(p, p, None, p, p, None, 8, 16, 100, 16)
        for k, v in kw.items():
            setattr(s, k, v)
        return s

    def extend(s, n=4, t=4, p=None, bt=None, bw=16, ws=1 << 20, wsp=None):
        return lib.pa_extend_tables(ctypes.byref(s), None, p, n, bt, bw, p, p, p, t, wsp or p, ws, None)

    def release(s, n=4, p=None, ws=1 << 20):
        return lib.pa_release_tables(ctypes.byref(s), p, n, p, ws, None)

    assert lib.pa_extend_tables(None, None, None, 0, None, 0, None, None, None, 0, None, 0, None) == BAD
    for call in (extend, release):
        assert call(state()) == BAD  # no workspace
        assert call(state(), n=-1) == BAD
        for kw in (dict(num_rows=0), dict(max_blocks_per_row=0), dict(num_blocks=0), dict(block_size=0),
                   dict(max_blocks_per_row=1 << 28), dict(num_blocks=1 << 28), dict(block_size=1 << 28)):
            assert call(state(**kw)) == BAD, kw
        if _no_gpu():
            assert call(state(), p=P, n=9) == BAD  # more requests than rows
            assert call(state(p=None), p=P) == BAD
            assert call(state(), p=P, ws=16) == _lib.PA_ERR_WORKSPACE
    if _no_gpu():
        for call in (extend, release):
            for kw in (dict(num_rows=(1 << 30) + 1, max_blocks_per_row=1), dict(num_rows=1, max_blocks_per_row=(1 << 30) + 1)):
                assert call(state(block_size=1, **kw), n=1, p=P, ws=1 << 40) == UNSUP, kw
        assert extend(state(), p=P, t=(1 << 30) + 1) == UNSUP
        assert extend(state(), n=1, p=P, bt=P, bw=(1 << 30) + 1) == UNSUP
        assert extend(state(), p=P, wsp=ctypes.c_void_p(0x1010)) == BAD
        assert lib.pa_extend_tables(ctypes.byref(state()), None, P, 4, P, 0, P, P, P, 4, P, 1 << 20, None) in (BAD, _lib.PA_ERR_CUDA)
