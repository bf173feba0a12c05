"""kv_append at the ends of its domain."""

import pytest
import torch

import fp8_helpers as ref
from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_cuda()


@pytest.fixture(scope="module")
def dkv():
    import decode_attention_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("eight", [False, True])
def test_few_tokens_at_the_longest_length(eight, dev, dkv):
    # sequences of 2^31 - 1 tokens that get one token each in a call of 4096 rows: the
    # pages that the other rows could have touched start past 2^31
    B, d, N, T, dt = 129, 64, (1 << 31) - 1, 4096, torch.bfloat16
    if torch.cuda.mem_get_info(dev)[0] < 100 << 30:
        pytest.skip("a block table of 69 GB")
    P = 1 << 27
    bt = torch.zeros(B, P, dtype=torch.int32, device=dev)
    bt[:, -1] = torch.arange(1, B + 1)
    nb = B + 2
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, 1, 1, d, generator=g).to(dt)
    k = torch.zeros(B, T, 1, d, dtype=dt)
    k[:, :1] = x
    lens = torch.full((B,), N, dtype=torch.int32, device=dev)
    news = torch.ones(B, dtype=torch.int32, device=dev)
    old = torch.randn(nb, 1, 16, d, generator=g)
    caches, want = [], []
    for _ in range(2):
        if eight:
            c, s = ref.quantise(old.transpose(0, 1).reshape(1, 1, nb * 16, d), dt)
            pool, scale = c.view(nb, 1, 16, d), s.view(nb, 1)
            lc, ls = pool.view(torch.uint8)[1:B + 1].clone(), scale[1:B + 1, :, None].clone()
            ref.append(x, x, (lc, ls, dt), (lc.clone(), ls.clone(), dt), [15] * B, [1] * B)
            full = pool.view(torch.uint8).clone(), scale.clone()
            full[0][1:B + 1], full[1][1:B + 1] = lc, ls[:, :, 0]
            caches.append(dkv.Fp8PagedCache(pool.to(dev), scale.to(dev), bt, N, dt))
        else:
            pool = old.to(dt)
            full = pool.clone()
            full[1:B + 1, :, 14] = x[:, 0]
            caches.append(dkv.PagedCache(pool.to(dev), bt, N))
        want.append(full)
    kd = k.to(dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    dkv.kv_append(kd, kd, *caches, seq_lens=lens, new_lens=news, workspace=ws)
    assert dkv.read_device_status(ws) == 0
    for c, w in zip(caches, want):
        if eight:
            assert torch.equal(c.pool.view(torch.uint8).cpu(), w[0])
            assert torch.equal(c.scale.cpu(), w[1])
        else:
            assert torch.equal(c.pool.cpu(), w)
