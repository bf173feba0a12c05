"""dkv_kv_meta_append_tokens rejects bad arguments on the host, before any CUDA
call, so this runs without a GPU."""

import ctypes

import pytest

from test_fp8_abi import ALIGN, NULL, OK, SHAPE, _kv, _params, dkv  # noqa: F401


@pytest.mark.parametrize("fmt", ["DENSE", "PAGED", "FP8", "FP8_PAGED"])
def test_validation(dkv, fmt):  # noqa: F811
    L = dkv.lib()
    kv = _kv(dkv, getattr(dkv, "DKV_KV_" + fmt))
    m = ctypes.c_void_p(1 << 16)

    def call(T, news=None, p=None, K=kv, mn=m):
        return L.dkv_kv_meta_append_tokens(ctypes.byref(p or _params(dkv)),
                                           ctypes.byref(K) if K else None, T, news, mn, m, None)

    assert call(0) == OK  # nothing was appended: nothing is launched
    assert call(-1) == SHAPE and call(1001) == SHAPE
    assert call(0, ctypes.c_void_p(4098)) == ALIGN
    assert call(0, ctypes.c_void_p(4100)) == OK
    assert call(0, mn=None) == NULL and call(0, K=None) == NULL
    assert call(0, mn=ctypes.c_void_p(8)) == ALIGN
    assert call(0, p=_params(dkv, seq_len=0)) == SHAPE


def test_more_rows_than_tokens(dkv):  # noqa: F811
    # as dkv_kv_append: what fits is known on the device, so only an address is wrong here
    L, kv = dkv.lib(), _kv(dkv, dkv.DKV_KV_DENSE)
    lens, bad = ctypes.c_void_p(4096), ctypes.c_void_p(8)
    for p, news in ((_params(dkv), lens), (_params(dkv, seq_lens=4096), None)):
        assert L.dkv_kv_meta_append_tokens(ctypes.byref(p), ctypes.byref(kv), 5000, news, bad, bad,
                                           None) == ALIGN
