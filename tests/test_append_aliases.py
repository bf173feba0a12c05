"""kv_append writes keys and values: caches that are one memory, or 8-bit caches
that share their scales, are refused on the host.  (Reading them is fine.)"""

import ctypes

import pytest
import torch

from test_fp8_abi import SHAPE, _append, _kv, dkv  # noqa: F401

CUDA = 7  # what a host without a GPU gets to with valid arguments


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("fmt", ["DENSE", "PAGED", "FP8", "FP8_PAGED"])
def test_same_memory(dkv, fmt):  # noqa: F811
    f = getattr(dkv, "DKV_KV_" + fmt)
    eight = "FP8" in fmt

    def call(**v):
        K, V = _kv(dkv, f), _kv(dkv, f, **v)
        return dkv.lib().dkv_kv_append(ctypes.byref(_append(dkv)), ctypes.byref(K),
                                       ctypes.byref(V), None, None)

    other = dict(data=1 << 24) | (dict(scale=1 << 25) if eight else {})
    assert call(**other) == CUDA
    assert call(**(other | dict(data=4096))) == SHAPE
    if eight:
        assert call(**(other | dict(scale=8192))) == SHAPE
