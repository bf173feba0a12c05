"""Tensors that the kernels would read as what they are not are refused for every
cache format.  The checks run on CPU tensors (before any CUDA call), so this needs
no GPU."""

import pytest
import torch

B, HQ, H, N, D, P = 2, 4, 2, 40, 64, 3


@pytest.fixture(scope="module")
def dkv():
    from decode_attention_paged_kv_gb300 import build as b
    b.build()
    import decode_attention_paged_kv_gb300 as m
    m.lib()
    return m


def cache(dkv, kind, dt):
    if kind == "dense":
        return torch.zeros(B, H, N, D, dtype=dt)
    bt = torch.zeros(B, P, dtype=torch.int32)
    if kind == "paged":
        return dkv.PagedCache(torch.zeros(7, H, 16, D, dtype=dt), bt, N)
    if kind == "fp8":
        return dkv.Fp8Cache(torch.zeros(B, H, N, D, dtype=torch.float8_e4m3fn),
                            torch.ones(B, H, P), dt)
    if kind == "fp8_paged":
        return dkv.Fp8PagedCache(torch.zeros(7, H, 16, D, dtype=torch.float8_e4m3fn),
                                 torch.ones(7, H), bt, N, dt)
    g = torch.zeros(B, H, N, D // 64, dtype=torch.float16)
    return dkv.Q4Cache(torch.zeros(B, H, N, D // 2, dtype=torch.uint8), g, g)


KINDS = [("dense", torch.bfloat16), ("dense", torch.float16), ("paged", torch.bfloat16),
         ("q4", torch.float16), ("fp8", torch.bfloat16), ("fp8_paged", torch.float16)]
OTHERS = [torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int16]


@pytest.mark.parametrize("kind,dt", KINDS, ids=str)
def test_dtypes(kind, dt, dkv):
    K = cache(dkv, kind, dt)
    V = K if kind not in ("paged", "fp8_paged") else cache(dkv, kind, dt)._replace(
        block_table=K.block_table)
    q = torch.zeros(B, HQ, D, dtype=dt)
    mn = torch.zeros(B, H, P, D, dtype=dt)
    m8 = dkv.Meta8(torch.zeros(B, H, P, D, dtype=torch.uint8),
                   torch.zeros(B, H, P, D, dtype=torch.uint8), torch.zeros(B, H, P),
                   torch.zeros(B, H, P))
    # what is right gets as far as the tensors' device
    for call in (lambda: dkv.decode_attn_full(q, K, V),
                 lambda: dkv.decode_attn_select(q, K, V, (mn, mn), 2),
                 lambda: dkv.decode_attn_select(q, K, V, m8, 2)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for t in OTHERS:
        if t == dt:
            continue
        for meta in ((mn, mn), m8):
            with pytest.raises(ValueError, match="dtype"):
                dkv.decode_attn_select(q.to(t), K, V, meta, 2)
        with pytest.raises(ValueError, match="dtype"):
            dkv.decode_attn_full(q.to(t), K, V)
        if kind == "dense":
            with pytest.raises(ValueError, match="dtype"):
                dkv.decode_attn_topk_tokens(q.to(t), K, V, 2)
        for meta in ((mn.to(t), mn), (mn, mn.to(t))):
            with pytest.raises(ValueError, match="dtype"):
                dkv.decode_attn_select(q, K, V, meta, 2)
            with pytest.raises(ValueError, match="dtype"):
                dkv.kv_meta_append(K, meta)
    for i in range(4):
        for t in (torch.int8, torch.float16, torch.float64):
            with pytest.raises(ValueError, match="dtype"):
                dkv.decode_attn_select(q, K, V, dkv.Meta8(*(x.to(t) if j == i else x
                                                            for j, x in enumerate(m8))), 2)


@pytest.mark.parametrize("kind,dt", KINDS, ids=str)
def test_scratch_with_gaps(kind, dt, dkv):
    # a workspace or reuse state is used as one piece: a view with gaps would have
    # the kernels write between its elements
    K = cache(dkv, kind, dt)
    q, mn = torch.zeros(B, HQ, D, dtype=dt), torch.zeros(B, H, P, D, dtype=dt)
    gaps = torch.zeros(1 << 20, 2, dtype=torch.uint8)[:, 0]
    for call in (lambda: dkv.decode_attn_full(q, K, K, workspace=gaps),
                 lambda: dkv.decode_attn_select(q, K, K, (mn, mn), 2, workspace=gaps),
                 lambda: dkv.decode_attn_select(q, K, K, (mn, mn), 2, hot=gaps, step=1)):
        with pytest.raises(ValueError, match="contiguous"):
            call()
    if kind == "dense":
        with pytest.raises(ValueError, match="contiguous"):
            dkv.decode_attn_topk_tokens(q, K, K, 2, workspace=gaps)


def test_4_bit_bounds(dkv):
    # gmin / gmax that are smaller than the codes, or elsewhere, would be read past
    # their end
    K = cache(dkv, "q4", torch.float16)
    q = torch.zeros(B, HQ, D, dtype=torch.float16)
    g = lambda b, h, n: torch.zeros(b, h, n, D // 64, dtype=torch.float16)
    meta_dev = K.gmin.to("meta")
    for lo, hi in ((g(B, H, N - 1), g(B, H, N - 1)), (g(B, 1, N), g(B, 1, N)),
                   (g(1, H, N), g(1, H, N)), (K.gmin, g(1, H, N)), (meta_dev, meta_dev),
                   (K.gmin, meta_dev)):
        bad = dkv.Q4Cache(K.codes, lo, hi)
        for call in (lambda: dkv.decode_attn_full(q, bad, K), lambda: dkv.kv_meta_build(bad)):
            with pytest.raises(ValueError, match="gmin / gmax must hold"):
                call()
    with pytest.raises(ValueError, match="CUDA"):  # room to spare is fine
        room = g(B + 1, H, N)
        dkv.kv_meta_build(dkv.Q4Cache(K.codes, room, room))
