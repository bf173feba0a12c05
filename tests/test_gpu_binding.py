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


def test_rows_of_more_dimensions(dev, dkv):
    # out [B, Hq, 1, d], [B, Hq, 2, d / 2], ... and q [B, Hq, d, 1]
    q, K, V = problem(dev)
    q16, K16, V16 = problem(dev, N=104, dt=torch.float16)
    meta, q4 = dkv.kv_meta_build(K), dkv.kv_quant4(K16.contiguous())
    q4v = dkv.kv_quant4(V16.contiguous())
    for f, x in ((lambda x, **o: dkv.decode_attn_full(x, K, V, **o), q),
                 (lambda x, **o: dkv.decode_attn_full(x, q4, q4v, **o), q16),
                 (lambda x, **o: dkv.decode_attn_select(x, K, V, meta, 3, **o), q),
                 (lambda x, **o: dkv.decode_attn_topk_tokens(x, K, V, 9, **o), q)):
        want = f(x)
        assert want.shape == (2, 4, 64)
        for shape in ((2, 4, 1, 64), (2, 4, 2, 32), (2, 4, 64, 1), (3, 5, 2, 1, 64), (2, 4, 3, 32), (2, 4, 64, 2)):
            out = torch.full(shape, 7.0, device=dev)
            assert f(x, out=out) is out
            rows = out[:2, :4].reshape(2, 4, -1)
            assert torch.equal(rows[..., :64], want) and (rows[..., 64:] == 7.0).all()
        assert torch.equal(f(x[..., None]), want)
        for bad in (torch.zeros(2, 4, 1, 32, device=dev), torch.zeros(2, 4, 2, 64, device=dev)[..., :32],
                    torch.zeros(2, 4, 64, 2, device=dev)[..., :1], torch.zeros(2, 64, device=dev)):
            with pytest.raises(ValueError, match="out must hold"):
                f(x, out=bad)


def test_counts_out_of_range(dev, dkv):
    # refused with the library's status, as callers that catch DkvError expect; more
    # pages than there are: all of them
    q, K, V = problem(dev)
    meta = dkv.kv_meta_build(K)
    state = dkv.hot_state(2, 2, 100, dev)
    for k in (0, -1, -5, -(1 << 40)):
        for wanted in (False, True):
            with pytest.raises(dkv.DkvError):
                dkv.decode_attn_select(q, K, V, meta, k, return_selected=wanted)
        with pytest.raises(dkv.DkvError):
            dkv.decode_attn_select(q, K, V, meta, 2, hot=state, step=k)
    want = dkv.decode_attn_select(q, K, V, meta, 7, return_selected=True)
    got = dkv.decode_attn_select(q, K, V, meta, (1 << 31) - 1, return_selected=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
