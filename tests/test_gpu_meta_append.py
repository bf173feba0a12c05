"""Page metadata kept up append by append: after tokens were appended,
kv_meta_append leaves what kv_meta_build of the whole cache gives, bit for bit,
and touches no page past a sequence's end; a draft step's selection over it."""

import math

import pytest
import torch

import fp8_helpers as ref
import oracle
from gpu_helpers import check_selection, require_cuda
from workloads import bits

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(scope="module")
def dev():
    return require_cuda()


@pytest.fixture(scope="module")
def dkv():
    import decode_attention_paged_kv_gb300 as m
    return m


def empty_caches(dkv, kind, B, H, N, d, dt, dev, seed):
    """A K and a V cache of the kind that hold nothing yet."""
    P = -(-N // PAGE)
    nb = B * P + 3
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(seed))[:B * P]
    bt = bt.view(B, P).to(torch.int32).to(dev)
    out = []
    for _ in range(2):
        if kind == "dense":
            out.append(torch.zeros(B, H, N, d, dtype=dt, device=dev))
        elif kind == "paged":
            out.append(dkv.PagedCache(torch.zeros(nb, H, PAGE, d, dtype=dt, device=dev), bt, N))
        elif kind == "fp8":
            out.append(dkv.Fp8Cache(torch.zeros(B, H, N, d, dtype=torch.float8_e4m3fn, device=dev),
                                    torch.zeros(B, H, P, device=dev), dt))
        else:
            out.append(dkv.Fp8PagedCache(
                torch.zeros(nb, H, PAGE, d, dtype=torch.float8_e4m3fn, device=dev),
                torch.zeros(nb, H, device=dev), bt, N, dt))
    return out


def check_against_build(dkv, K, meta, lens, S):
    """meta equals a fresh build on every page that holds tokens, and keeps the
    sentinel 9 on the others."""
    full = dkv.kv_meta_build(K, page_size=S, seq_lens=lens)
    for b, n in enumerate(lens.tolist()):
        pages = -(-n // S)
        for a, w in zip(meta, full):
            assert torch.equal(a[b, :, :pages].view(torch.int16), w[b, :, :pages].view(torch.int16))
            assert (a[b, :, pages:] == 9.0).all()


@pytest.mark.parametrize("S", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("kind", ["dense", "paged", "fp8", "fp8_paged"])
def test_one_token_at_a_time(kind, S, dev, dkv):
    # each token 100 times as large as the one before: an 8-bit block's scale rises
    # with it and its older codes are rounded again, in all the block's pages
    B, H, d, N, dt = 3, 2, 64, 300, torch.bfloat16
    g = torch.Generator().manual_seed(S)
    K, V = empty_caches(dkv, kind, B, H, N, d, dt, dev, S)
    lens = torch.tensor([37, 100, 259], dtype=torch.int32, device=dev)
    x = torch.randn(B, 259, H, d, generator=g).to(dt).to(dev)
    dkv.kv_append(x, x, K, V, seq_lens=lens, new_lens=lens.clone())
    meta = [torch.full((B, H, -(-N // S), d), 9.0, dtype=dt, device=dev) for _ in range(2)]
    for m, w in zip(meta, dkv.kv_meta_build(K, page_size=S, seq_lens=lens)):
        for b, n in enumerate(lens.tolist()):
            m[b, :, :-(-n // S)] = w[b, :, :-(-n // S)]
    for i in range(20):
        lens += 1
        y = (torch.randn(B, 1, H, d, generator=g) * 100.0 ** (i % 6)).to(dt).to(dev)
        dkv.kv_append(y, y, K, V, seq_lens=lens)
        dkv.kv_meta_append(K, meta, page_size=S, seq_lens=lens)
        check_against_build(dkv, K, meta, lens, S)


@pytest.mark.parametrize("S", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("kind", ["dense", "paged", "fp8", "fp8_paged"])
def test_several_tokens(kind, S, dev, dkv):
    # a prompt, drafts and a chunk, some sequences with fewer tokens or none; the
    # prompt's metadata too comes from kv_meta_append
    B, H, d, N, dt = 4, 2, 128, 300, torch.float16
    g = torch.Generator().manual_seed(S + 1)
    K, V = empty_caches(dkv, kind, B, H, N, d, dt, dev, S)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    meta = [torch.full((B, H, -(-N // S), d), 9.0, dtype=dt, device=dev) for _ in range(2)]
    for i, (T, news) in enumerate([(101, [101, 16, 1, 50]), (5, [5, 0, 3, 1]), (5, None),
                                   (40, [40, 17, 0, 33]), (1, [1, 0, 1, 1]), (140, [2, 140, 3, 139])]):
        new = torch.tensor(news or [T] * B, dtype=torch.int32, device=dev)
        lens += new
        given = None if news is None else new
        y = (torch.randn(B, T, H, d, generator=g) * 4.0 ** i).to(dt).to(dev)
        dkv.kv_append(y, y, K, V, seq_lens=lens, new_lens=given)
        dkv.kv_meta_append(K, meta, page_size=S, seq_lens=lens, new_tokens=T, new_lens=given)
        check_against_build(dkv, K, meta, lens, S)


@pytest.mark.parametrize("S", [4, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_4_bit(d, S, dev, dkv):
    # no call appends to a 4-bit cache; its newest tokens are quantised in place
    B, H, N = 2, 2, 400
    g = torch.Generator().manual_seed(d + S)
    x = torch.randn(B, H, N, d, generator=g).half().to(dev)
    q4 = dkv.kv_quant4(x)
    lens = torch.tensor([150, 311], dtype=torch.int32, device=dev)
    meta = [torch.full((B, H, -(-N // S), d), 9.0, dtype=torch.float16, device=dev)
            for _ in range(2)]
    dkv.kv_meta_append(q4, meta, page_size=S, seq_lens=lens, new_tokens=311, new_lens=lens.clone())
    check_against_build(dkv, q4, meta, lens, S)
    for T, news in ((1, None), (5, [0, 5]), (70, [70, 44])):
        new = torch.tensor(news or [T] * B, dtype=torch.int32, device=dev)
        lens += new
        for b, (n, k) in enumerate(zip(lens.tolist(), new.tolist())):
            x[b, :, n - k:n] *= 10.0
        for old, now in zip(q4, dkv.kv_quant4(x)):
            old.copy_(now)
        dkv.kv_meta_append(q4, meta, page_size=S, seq_lens=lens, new_tokens=T,
                           new_lens=None if news is None else new)
        check_against_build(dkv, q4, meta, lens, S)


@pytest.mark.parametrize("kind", ["dense", "fp8", "fp8_paged"])
def test_odd_counts(kind, dev, dkv):
    # counts past T, below 0 or past the length; lengths past the cache and empty
    # ones: what is rebuilt is what a build gives, the rest is left alone
    B, H, d, N, S, dt = 6, 2, 64, 100, 16, torch.bfloat16
    K, V = empty_caches(dkv, kind, B, H, N, d, dt, dev, 5)
    x = torch.randn(B, N, H, d, generator=torch.Generator().manual_seed(5)).to(dt).to(dev)
    dkv.kv_append(x, x, K, V)
    lens = torch.tensor([90, 90, 7, 200, 0, 90], dtype=torch.int32, device=dev)
    news = torch.tensor([40, -3, 20, 1, 2, 0], dtype=torch.int32, device=dev)
    meta = [torch.full((B, H, 7, d), 9.0, dtype=dt, device=dev) for _ in range(2)]
    dkv.kv_meta_append(K, meta, seq_lens=lens, new_tokens=20, new_lens=news)
    # sequence 0: its last 20 tokens, 70 .. 89; 2: all 7; 3: the last page of 100
    full = dkv.kv_meta_build(K, seq_lens=lens.clamp(1, N))
    want = [torch.full_like(m, 9.0) for m in meta]
    for w, f in zip(want, full):
        w[0, :, 4:6], w[2, :, :1], w[3, :, 6:] = f[0, :, 4:6], f[2, :, :1], f[3, :, 6:]
        if kind == "dense":  # (an empty 16-bit sequence counts as one token)
            w[4, :, :1] = f[4, :, :1]
    for a, w in zip(meta, want):
        assert torch.equal(a, w)


def test_refusals(dev, dkv):
    K = torch.zeros(2, 1, 40, 64, dtype=torch.bfloat16, device=dev)
    meta = dkv.kv_meta_build(K)
    one = torch.ones(2, dtype=torch.int32, device=dev)
    for bad in (dict(new_lens=one), dict(new_tokens=2, new_lens=one.cpu()),
                dict(new_tokens=2, new_lens=one.long()), dict(new_tokens=2, new_lens=one[:1])):
        with pytest.raises(ValueError):
            dkv.kv_meta_append(K, meta, **bad)
    with pytest.raises(dkv.DkvError):
        dkv.kv_meta_append(K, meta, new_tokens=-1)
    keep = [m.clone() for m in meta]
    dkv.kv_meta_append(K + 1, meta, new_tokens=0)
    assert all(torch.equal(a, b) for a, b in zip(keep, meta))
    with pytest.raises(dkv.DkvError):  # more new tokens than the cache holds
        dkv.kv_meta_append(K, meta, new_tokens=41)


@pytest.mark.parametrize("S", [4, 16])
def test_draft_steps(S, dev, dkv):
    """Steps of five drafted tokens: append, metadata, selection of the newest
    token's query: metadata, pages and outputs against 64-bit forms."""
    B, Hq, H, d, N, dt, T, top_k = 3, 8, 2, 128, 700, torch.bfloat16, 5, 6
    g = torch.Generator().manual_seed(S)
    K, V = empty_caches(dkv, "fp8_paged", B, H, N, d, dt, dev, S)
    P16, code = -(-N // PAGE), 0
    refs = [(torch.zeros(B, H, P16 * PAGE, d, dtype=torch.uint8), torch.zeros(B, H, P16), dt)
            for _ in range(2)]
    rope = dkv.rope_table(N, d)
    grope = tuple(t.to(dev) for t in rope)
    lens = torch.zeros(B, dtype=torch.int32)
    meta = [torch.full((B, H, -(-N // S), d), 9.0, dtype=dt, device=dev) for _ in range(2)]
    for i in range(8):
        rows = T if i else 600
        new = (torch.tensor([600, 333, 590], dtype=torch.int32) if i == 0 else
               torch.randint(1, T + 1, (B,), generator=g, dtype=torch.int32))
        lens += new
        x = torch.randn(B, rows, Hq + 2 * H, d, generator=g).to(dt)
        cut = lambda t: (t[:, :, Hq:Hq + H], t[:, :, Hq + H:])
        xd, ld, nd = x.to(dev), lens.to(dev), new.to(dev)
        q_ref = torch.zeros(B, rows, Hq, d, dtype=dt)
        q_out = dkv.kv_append(*cut(xd), K, V, seq_lens=ld, new_lens=nd, q=xd[:, :, :Hq], rope=grope)
        dkv.kv_meta_append(K, meta, page_size=S, seq_lens=ld, new_tokens=rows, new_lens=nd)
        ref.append(*cut(x), *refs, lens, new, x[:, :, :Hq], q_ref, rope)
        at = new.long() - 1
        q = q_out[torch.arange(B), at]
        assert torch.equal(q.cpu(), q_ref[torch.arange(B), at])
        out, sel = dkv.decode_attn_select(q, K, V, meta, top_k, return_selected=True, seq_lens=ld,
                                          page_size=S)
        kv, vv = (ref.values(c.view(torch.float8_e4m3fn), s)[:, :, :N] for c, s, _ in refs)
        for b, n in enumerate(lens.tolist()):
            Pb = -(-n // S)
            want = [torch.stack([getattr(kv[b, :, S * j:min(n, S * j + S)], f)(1)
                                 for j in range(Pb)], 1).to(dt) for f in ("amin", "amax")]
            for a, w in zip(meta, want):
                assert torch.equal(a[b, :, :Pb].cpu(), w)
            mn, mx = (bits(w[None].contiguous()) for w in want)
            r = oracle.scores(bits(q[b:b + 1].cpu()), mn, mx, code)[0]
            check_selection(sel[b].cpu().numpy(), r, top_k)
        want = ref.attention(q.cpu(), kv, vv, 1 / math.sqrt(d), lens, pages=sel.tolist(), S=S)
        err = (out.cpu().double() - want).abs().max()
        assert err <= ref.tolerance(q.cpu(), kv, vv, 1 / math.sqrt(d))


@pytest.mark.parametrize("kind", ["dense", "fp8"])
def test_more_rows_than_tokens(kind, dev, dkv):
    # a draft buffer of more rows than the cache holds tokens, a few of them in use
    B, H, d, N, S, T, dt = 2, 2, 64, 40, 8, 64, torch.bfloat16
    K, V = empty_caches(dkv, kind, B, H, N, d, dt, dev, 1)
    meta = [torch.full((B, H, 5, d), 9.0, dtype=dt, device=dev) for _ in range(2)]
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    g = torch.Generator().manual_seed(1)
    for news in ([3, 20], [37, 1]):
        new = torch.tensor(news, dtype=torch.int32, device=dev)
        lens += new
        y = torch.randn(B, T, H, d, generator=g).to(dt).to(dev)
        dkv.kv_append(y, y, K, V, seq_lens=lens, new_lens=new)
        dkv.kv_meta_append(K, meta, page_size=S, seq_lens=lens, new_tokens=T, new_lens=new)
        check_against_build(dkv, K, meta, lens, S)
