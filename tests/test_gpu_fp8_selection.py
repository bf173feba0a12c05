"""Page-sparse attention over 8-bit caches: that the pages chosen are the right ones
-- over 8-bit metadata, beside empty sequences, and in a captured decode loop whose
metadata is kept up by kv_meta_append."""

import math

import numpy as np
import pytest
import torch

import fp8_helpers as ref
import oracle
from gpu_helpers import check_selection, require_cuda
from test_gpu_fp8 import caches, make
from workloads import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_cuda()


@pytest.fixture(scope="module")
def dkv():
    import decode_attention_paged_kv_gb300 as m
    return m


def check_pages(sel, r, top_k, group=1):
    """sel [Hq, kk] of one sequence against its scores r [Hq, pages]: the best
    pages, ascending, and -1 behind them."""
    Hq, Pb = r.shape
    kk = min(top_k, Pb)
    if group > 1:
        r = np.repeat(r.reshape(Hq // group, group, Pb).sum(1), group, axis=0)
    check_selection(sel[:, :kk].numpy(), r, top_k)
    assert torch.all(sel[:, kk:] == -1)


@pytest.mark.parametrize("case", [  # B, Hq, Hkv, d, N, dtype, S, top_k, lens, group
    (2, 8, 2, 128, 900, torch.bfloat16, 16, 9, [900, 77], False),
    (1, 4, 4, 64, 1500, torch.float16, 16, 11, None, False),
    (2, 8, 2, 128, 6000, torch.bfloat16, 16, 30, [6000, 4700], False),
    (1, 8, 1, 64, 5000, torch.float16, 16, 25, None, True),
    (1, 8, 2, 128, 2000, torch.bfloat16, 4, 40, None, False),
    (1, 4, 2, 64, 9000, torch.float16, 32, 12, None, False),
], ids=str)
@pytest.mark.parametrize("paged", [False, True])
def test_8_bit_metadata(case, paged, dev, dkv):
    B, Hq, Hkv, d, N, dt, S, top_k, lens, group = case
    q, K, V = make(B, Hq, Hkv, d, N, dt, seed=N + S)
    Kd, Vd = caches(dkv, dev, K, V, dt, paged, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    meta = dkv.kv_meta_build(Kd, page_size=S, seq_lens=lt)
    m8 = dkv.kv_meta8_build(meta, page_size=S, seq_lens=lt)
    out, sel = dkv.decode_attn_select(q.to(dev), Kd, Vd, m8, top_k, return_selected=True,
                                      group_select=group, seq_lens=lt, page_size=S)
    sel, code = sel.cpu(), 0 if dt == torch.bfloat16 else 1
    kv, vv = ref.values(*K), ref.values(*V)
    for b in range(B):
        n = N if lens is None else lens[b]
        Pb = -(-n // S)
        mn, mx = (torch.stack([getattr(kv[b, :, S * j:min(n, S * j + S)], f)(1)
                               for j in range(Pb)], 1).to(dt)[None] for f in ("amin", "amax"))
        cmin, cmax, lo, step = oracle.meta8(bits(mn), bits(mx), code)
        for a, w in zip(m8, (cmin, cmax, lo, step)):
            assert np.array_equal(a[b:b + 1, :, :Pb].cpu().numpy(), w)
        r = oracle.scores8(bits(q[b:b + 1]), cmin, cmax, lo, step, code)[0]
        check_pages(sel[b], r, top_k, Hq // Hkv if group else 1)
    want = ref.attention(q, kv, vv, 1 / math.sqrt(d), lens, pages=sel.tolist(), S=S)
    assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, 1 / math.sqrt(d))


@pytest.mark.parametrize("N,top_k", [(48, 2), (5000, 12)])
def test_beside_an_empty_sequence(N, top_k, dev, dkv):
    q, K, V = make(4, 4, 2, 64, N, torch.bfloat16, seed=N)
    lens = [N, 0, 20, -1]
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, True, lens)
    lt = torch.tensor(lens, dtype=torch.int32, device=dev)
    meta = [m.nan_to_num(3.0) for m in dkv.kv_meta_build(Kd, seq_lens=lt)]
    out, sel = dkv.decode_attn_select(q.to(dev), Kd, Vd, meta, top_k, return_selected=True,
                                      seq_lens=lt)
    sel = sel.cpu()
    for b, n in enumerate(lens):
        if n <= 0:  # the rows of length 1
            assert torch.all(sel[b, :, 0] == 0) and torch.all(sel[b, :, 1:] == -1)
            assert not out[b].any()
            continue
        Pb = -(-n // 16)
        mn, mx = (bits(m[b:b + 1, :, :Pb].contiguous().cpu()) for m in meta)
        check_pages(sel[b], oracle.scores(bits(q[b:b + 1]), mn, mx, 0)[0], top_k)


@pytest.mark.parametrize("T,S,N", [(1, 16, 4608), (1, 4, 200), (5, 16, 300), (5, 8, 4608)])
def test_captured_loop(T, S, N, dev, dkv):
    # append, metadata and selection in one graph, replayed: the metadata after each
    # step is that of the tokens that the plain form appended, and so are the pages
    B, Hq, H, d, dt, top_k = 2, 8, 2, 64, torch.float16, 7
    P16 = -(-N // 16)
    g = torch.Generator().manual_seed(T + S)
    rope = dkv.rope_table(N, d)
    grope = tuple(t.to(dev) for t in rope)
    refs = [(torch.zeros(B, H, P16 * 16, d, dtype=torch.uint8), torch.zeros(B, H, P16), dt)
            for _ in range(2)]
    bt = torch.randperm(B * P16, generator=g).view(B, P16).to(torch.int32).to(dev)
    K, V = (dkv.Fp8PagedCache(
        torch.zeros(B * P16, H, 16, d, dtype=torch.float8_e4m3fn, device=dev),
        torch.zeros(B * P16, H, device=dev), bt, N, dt) for _ in range(2))
    cut = lambda t: (t[:, :, Hq:Hq + H], t[:, :, Hq + H:])
    now = torch.tensor([N - 60, N - 110], dtype=torch.int32)
    x = torch.randn(B, N - 60, Hq + 2 * H, d, generator=g).to(dt)
    lens, new, xd = now.to(dev), torch.zeros(B, dtype=torch.int32, device=dev), x.to(dev)
    dkv.kv_append(*cut(xd), K, V, seq_lens=lens, new_lens=lens.clone(), rope=grope)
    ref.append(*cut(x), *refs, now, now, rope=rope)
    meta = dkv.kv_meta_build(K, page_size=S, seq_lens=lens)
    ws = torch.zeros(dkv.workspace_bytes(B, Hq, H, d, N, top_k, page_size=S, fp8=True),
                     dtype=torch.uint8, device=dev)
    rows = torch.zeros(B, T, Hq + 2 * H, d, dtype=dt, device=dev)
    q_out = torch.zeros(B, T, Hq, d, dtype=dt, device=dev)
    out = torch.zeros(B, Hq, d, device=dev)
    sel = torch.zeros(B, Hq, top_k, dtype=torch.int32, device=dev)

    def step():
        lens.add_(new)
        dkv.kv_append(*cut(rows), K, V, seq_lens=lens, new_lens=new, q=rows[:, :, :Hq],
                      q_out=q_out, rope=grope, workspace=ws)
        dkv.kv_meta_append(K, meta, page_size=S, seq_lens=lens, new_tokens=T, new_lens=new)
        # (the first drafted token's query, which every sequence has)
        dkv.decode_attn_select(q_out[:, 0], K, V, meta, top_k, out=out, return_selected=True,
                               selected=sel, seq_lens=lens, page_size=S, workspace=ws)

    graph = None
    for i in range(10):
        n_new = torch.randint(1, T + 1, (B,), generator=g, dtype=torch.int32)
        x = torch.randn(B, T, Hq + 2 * H, d, generator=g)
        x = (x * 1.7 ** i).clamp(-60000, 60000).to(dt)  # scales rise
        rows.copy_(x)
        new.copy_(n_new)
        if i == 0:
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        now += n_new
        q_ref = torch.zeros(B, T, Hq, d, dtype=dt)
        ref.append(*cut(x), *refs, now, n_new, x[:, :, :Hq], q_ref, rope)
        q = q_ref[:, 0]
        assert torch.equal(q_out[:, 0].cpu(), q)
        kv, vv = (ref.values(c.view(torch.float8_e4m3fn), s) for c, s, _ in refs)
        for b, n in enumerate(now.tolist()):
            Pb = -(-n // S)
            mn, mx = (torch.stack([getattr(kv[b, :, S * j:min(n, S * j + S)], f)(1)
                                   for j in range(Pb)], 1).to(dt)[None] for f in ("amin", "amax"))
            for a, w in zip(meta, (mn, mx)):
                assert torch.equal(a[b:b + 1, :, :Pb].cpu(), w)
            r = oracle.scores(bits(q[b:b + 1]), bits(mn), bits(mx), 1)[0]
            check_pages(sel[b].cpu(), r, top_k)
        want = ref.attention(q, kv, vv, 1 / 8, now.tolist(), pages=sel.tolist(), S=S)
        assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, 1 / 8)
    assert dkv.read_device_status(ws) == 0
