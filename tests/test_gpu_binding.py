"""What the Python calls take and refuse that only shows with CUDA tensors."""

import pytest
import torch

from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_cuda()


@pytest.fixture(scope="module")
def dkv():
    import decode_attention_paged_kv_gb300 as m
    return m


def problem(dev, B=2, Hq=4, H=2, N=100, d=64, dt=torch.bfloat16):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(*s, generator=g).to(dt).to(dev)
            for s in ((B, Hq, d), (B, H, N, d), (B, H, N, d))]


def test_tensors_without_memory(dev, dkv):
    # a batched query of torch.func has no address: a Python exception, and the
    # interpreter goes on
    q, K, V = problem(dev)
    meta = dkv.kv_meta_build(K)
    for f in (lambda x: dkv.decode_attn_full(x, K, V),
              lambda x: dkv.decode_attn_select(x, K, V, meta, 2)):
        with pytest.raises(RuntimeError):
            torch.func.vmap(f)(torch.stack((q, q)))
        assert torch.equal(f(q), f(q))
