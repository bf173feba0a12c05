"""Latent caches on the GPU: appending, attention of new tokens (absorbed form) and of
prompts (expanded form), against 64-bit forms of the same inputs."""

import itertools
import math
import zlib

import pytest
import torch

from gpu_helpers import require_cuda
from latent_helpers import (DT, attn64, check, eps, hide_tail, make_cache, rotate64, rows_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dkv():
    require_cuda()
    import decode_attention_paged_kv_gb300 as m
    return m


def gen_of(*key):
    return torch.Generator("cuda").manual_seed(zlib.crc32(repr(key).encode()))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ append
def append_inputs(B, T, H, dc, dt, gen, strided=False):
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    if not strided:
        return (3 * r(B, T, dc)).to(dt), r(B, T, 64).to(dt), r(B, T, H, 64).to(dt)
    x = (3 * r(T, B, dc + 64 + 8)).to(dt).transpose(0, 1)  # as one projection gives both
    return x[..., :dc], x[..., dc:dc + 64], r(B, H, T, 192).to(dt).transpose(1, 2)[..., 128:]


@pytest.mark.parametrize("block", [0, 16, 32, 64])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("B,T,H,dc,N,il,norm,strided", [
    (3, 1, 16, 512, 100, False, True, False),
    (2, 70, 5, 256, 131, True, True, True),
    (5, 17, 0, 512, 33, False, True, False),
    (2, 9, 40, 256, 64, False, False, True),
    (1, 1, 1, 512, 1, True, True, False),
])
def test_append(dkv, block, dt, B, T, H, dc, N, il, norm, strided):
    dt = DT[dt]
    gen = gen_of("append", block, B, T, H, dc, N)
    cache, _ = make_cache(B, N, dc, block, dt, gen, pad=8 if strided else 0)
    c, k, q = append_inputs(B, T, H, dc, dt, gen, strided)
    lens = [max(1, N - 3 * b) for b in range(B)]
    new = [min(T - b % 2 if T > 1 else 1, lens[b]) for b in range(B)]
    w = (1 + 0.2 * torch.randn(dc, generator=gen, device="cuda")).to(dt) if norm else None
    rope = dkv.rope_table(N, 64, device="cuda")
    before = [rows_of(cache, b).clone() for b in range(B)]
    q_out = torch.full((B, T, H, 64), 7.0, dtype=dt, device="cuda") if H else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = dkv.latent_append(c, k, cache, seq_lens=ints(lens), new_lens=ints(new),
                            q_rope=q if H else None, q_out=q_out, rope=rope, norm=w, eps=1e-5,
                            interleaved=il, workspace=ws)
    assert got is q_out
    assert dkv.read_device_status(ws) == 0
    half = eps(dt) / 2
    for b in range(B):
        m, n = lens[b], new[b]
        want = before[b].double()
        x = c[b, :n].double()
        if norm:
            x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-5) * w.double()
        cos, sin = rope[0][m - n:m], rope[1][m - n:m]
        want[m - n:m] = torch.cat((x, rotate64(k[b, :n], cos, sin, il)), dim=-1)
        now = rows_of(cache, b)
        # one rounding of the result; the norm's fp32 steps (a sum of dc squares in blocks, a
        # root, a quotient, two products) and the rotation's three add 2^-20 of their size
        size = want.abs()
        size[m - n:m, dc:] = rotate64(k[b, :n].abs(), cos.abs(), -sin.abs(), il).abs() + \
            k[b, :n].double().abs()
        tol = half * want.abs() + 2.0 ** -20 * size + (2.0 ** -25 if dt == torch.float16 else 1e-38)
        assert bool(((now.double() - want).abs() <= tol)[m - n:m].all()), b
        keep = torch.ones(len(now), dtype=torch.bool, device="cuda")
        keep[m - n:m] = False
        assert torch.equal(now[keep].view(torch.int16), before[b][keep].view(torch.int16)), b
        if H:
            want = rotate64(q[b, :n], cos[:, None], sin[:, None], il)
            tol = half * want.abs() + 2.0 ** -20 * 2 * q[b, :n].double().abs().amax() + 2.0 ** -25
            assert bool(((q_out[b, :n].double() - want).abs() <= tol).all())
            assert bool((q_out[b, n:] == 7).all())


def test_append_leaves_what_does_not_fit(dkv):
    # lengths past the cache, the table of angles or the rows; bad blocks
    gen = gen_of("misfit")
    cache, table = make_cache(4, 40, 256, 16, torch.bfloat16, gen)
    before = cache.pool.clone()
    c, k, q = append_inputs(4, 2, 3, 256, torch.bfloat16, gen)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rope = dkv.rope_table(38, 64, device="cuda")
    q_out = torch.zeros_like(q)
    dkv.latent_append(c, k, cache, seq_lens=ints([41, 39, 0, 1]), new_lens=ints([2, 2, 2, 2]),
                      q_rope=q, q_out=q_out, rope=rope, workspace=ws)
    assert dkv.read_device_status(ws) == 9
    assert torch.equal(cache.pool.view(torch.int16), before.view(torch.int16))
    assert not bool(q_out.any())
    table[1, 0] = -1
    table[2, 0] = cache.pool.shape[0]
    dkv.latent_append(c, k, cache, seq_lens=ints([0, 2, 2, 2]), q_rope=q, q_out=q_out, rope=rope,
                      workspace=ws)
    assert dkv.read_device_status(ws) == 9
    blk = int(table[3, 0])
    same = torch.ones(len(before), dtype=torch.bool)
    same[blk] = False
    assert torch.equal(cache.pool[same].view(torch.int16), before[same].view(torch.int16))
    assert torch.equal(cache.pool[blk, :2, :256], c[3])
    assert not bool(q_out[0].any()) and bool(q_out[1].any())  # (queries need no block)


def test_append_rotates_in_place(dkv):
    gen = gen_of("in place")
    cache, _ = make_cache(2, 50, 512, 16, torch.bfloat16, gen)
    c, k, q = append_inputs(2, 3, 4, 512, torch.bfloat16, gen)
    rope = dkv.rope_table(50, 64, device="cuda")
    a = dkv.latent_append(c, k, cache, seq_lens=ints([50, 9]), q_rope=q, rope=rope)
    dkv.latent_append(c, k, cache, seq_lens=ints([50, 9]), q_rope=q, q_out=q, rope=rope)
    assert torch.equal(a, q)


# ---------------------------------------------------------------- absorbed form
def decode_case(B, T, H, dc, N, block, dt, gen, lens, new, pad=0, out_dtype=torch.float32):
    cache, _ = make_cache(B, N, dc, block, dt, gen, pad=pad)
    hide_tail(cache, lens)
    ql = torch.randn(H, B, T, dc, generator=gen, device="cuda").to(dt).permute(1, 2, 0, 3)
    qr = torch.randn(B, T, H, 192, generator=gen, device="cuda").to(dt)[..., 128:]
    out = torch.full((B, T, H, dc), 5.0, dtype=out_dtype, device="cuda")
    return cache, ql, qr, out


def check_decode(cache, ql, qr, out, lens, new, scale):
    B, T, H, dc = ql.shape
    for b in range(B):
        x = rows_of(cache, b)
        for t in range(T):
            if t >= new[b]:
                assert bool((out[b, t] == 5.0).all()), (b, t)
                continue
            n = lens[b] - new[b] + t + 1
            if n <= 0:
                assert not bool(out[b, t].any()), (b, t)
                continue
            q = torch.cat((ql[b, t], qr[b, t]), dim=-1)
            ref, mag, rel = attn64(q, x[:n], x[:n, :dc], scale)
            check(out[b, t], ref, mag, rel, ql.dtype, (b, t))


DECODE = [
    # B, T, H, dc, N, lens, new
    (1, 1, 1, 512, 1, [1], [1]),
    (1, 1, 16, 256, 64, [64], [1]),
    (3, 1, 16, 512, 200, [200, 63, 65], [1, 1, 1]),
    (2, 1, 128, 512, 777, [777, 1], [1, 1]),
    (4, 1, 20, 512, 500, [0, 500, -3, 129], [1, 1, 1, 1]),
    (3, 4, 40, 512, 333, [333, 4, 2], [4, 3, 2]),
    (2, 5, 8, 256, 130, [130, 3], [0, 5]),
    (2, 3, 64, 256, 1000, [1000, 512], [3, 2]),
    (5, 1, 33, 512, 4099, [4099, 128, 4000, 17, 2500], [1, 1, 1, 0, 1]),
    (1, 1, 128, 512, 20011, [20011], [1]),
    (40, 1, 7, 256, 260, [7 * i - 8 for i in range(38)] + [260, 256], [1] * 40),
    (2, 1, 300, 512, 150, [150, 77], [1, 1]),
    # row tiles with few sequences, with one, with none
    (9, 5, 40, 512, 900, [900, 700, 5, 0, 64, 129, 333, 900, 1], [1, 5, 5, 5, 1, 2, 1, 0, 1]),
    (3, 6, 70, 256, 400, [400, 399, 64], [2, 1, 2]),
    (3, 2, 64, 512, 5000, [5000, 4999, 4000], [1, 1, 2]),
]


@pytest.mark.parametrize("block", [0, 16, 32, 64])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c[:5])))
def test_decode(dkv, case, dt, block):
    B, T, H, dc, N, lens, new = case
    dt = DT[dt]
    gen = gen_of("decode", B, T, H, dc, N, block)
    out_dtype = dt if block in (16, 64) else torch.float32
    cache, ql, qr, out = decode_case(B, T, H, dc, N, block, dt, gen, lens, new,
                                     pad=16 if block == 32 else 0, out_dtype=out_dtype)
    ws = torch.zeros(dkv.latent_workspace_bytes(B, T, H, dc, N), dtype=torch.uint8, device="cuda")
    got = dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), new_lens=ints(new),
                                 out=out, workspace=ws)
    assert got is out
    assert dkv.read_device_status(ws) == 0
    check_decode(cache, ql, qr, out, lens, new, 0.07)
    # the same call gives the same bits
    again = torch.full_like(out, 5.0)
    dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), new_lens=ints(new),
                           out=again, workspace=ws)
    assert torch.equal(out, again)


def test_decode_defaults(dkv):
    # no lengths: every sequence whole, every row new; out made by the call
    gen = gen_of("defaults")
    cache, ql, qr, _ = decode_case(3, 2, 12, 256, 90, 16, torch.bfloat16, gen, [90] * 3, [2] * 3)
    out = dkv.latent_decode_attn(ql, qr, cache, 0.1)
    assert out.dtype == torch.float32
    check_decode(cache, ql, qr, out, [90] * 3, [2] * 3, 0.1)
    half = dkv.latent_decode_attn(ql, qr, cache, 0.1, out_dtype=torch.bfloat16)
    check_decode(cache, ql, qr, half, [90] * 3, [2] * 3, 0.1)
    # lengths past the cache count as its whole, counts past T as T
    more = dkv.latent_decode_attn(ql, qr, cache, 0.1, seq_lens=ints([1 << 30] * 3),
                                  new_lens=ints([9] * 3))
    assert torch.equal(more, out)


@pytest.mark.parametrize("big", [20.0, -20.0, 0.0])
def test_decode_score_ranges(dkv, big):
    # scores of thousands, of both signs; all scores equal (scale 0): the mean
    gen = gen_of("ranges", big)
    cache, ql, qr, out = decode_case(2, 1, 16, 256, 400, 16, torch.bfloat16, gen, [400, 390], [1, 1])
    dkv.latent_decode_attn(ql, qr, cache, big, seq_lens=ints([400, 390]), out=out)
    check_decode(cache, ql, qr, out, [400, 390], [1, 1], big)


def test_decode_rising_scores(dkv):
    # every tile raises the maximum; then every tile lies far below it
    for order in (1, -1):
        x = torch.zeros(1, 1024, 320, dtype=torch.bfloat16, device="cuda")
        x[0, :, :256] = torch.randn(1024, 256, generator=gen_of("rise"), device="cuda")
        up = torch.arange(1024, device="cuda")
        x[0, :, 256] = (up if order > 0 else 1023 - up) / 8
        ql = torch.zeros(1, 1, 9, 256, dtype=torch.bfloat16, device="cuda")
        qr = torch.zeros(1, 1, 9, 64, dtype=torch.bfloat16, device="cuda")
        qr[..., 0] = torch.arange(9, device="cuda") / 4
        out = torch.zeros(1, 1, 9, 256, device="cuda")
        dkv.latent_decode_attn(ql, qr, x, 1.0, out=out)
        check_decode(x, ql, qr, out, [1024], [1], 1.0)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_decode_nan_scores(dkv, dt):
    # NaN queries, and a NaN row among those that are seen, give rows of NaN, whether one CTA
    # holds the sequence, some share it or all do; other heads and sequences are as ever
    dt = DT[dt]
    for lens in ([1000], [20000], [64] * 160, [30000, 5, 64, 700, 130], [9, 9]):
        B, N, H, dc = len(lens), max(lens), 20, 256
        gen = gen_of("nan", B, N)
        cache, ql, qr, out = decode_case(B, 1, H, dc, N, 16, dt, gen, lens, [1] * B)
        ql[0, 0, 3], qr[0, 0, 17, 5] = math.nan, math.nan
        bad = torch.zeros(B, H, dtype=torch.bool, device="cuda")
        bad[0, 3] = bad[0, 17] = True
        if B > 2:
            cache.pool[int(cache.block_table[2, 0]), 1, 7] = math.nan
            bad[2] = True
        dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), out=out)
        assert torch.equal(out[:, 0].isnan().all(-1), bad), lens
        for b in range(min(B, 8)):
            x, on = rows_of(cache, b)[:lens[b]], ~bad[b]
            if not bool(on.any()):
                continue
            q = torch.cat((ql[b, 0], qr[b, 0]), -1)[on]
            check(out[b, 0][on], *attn64(q, x, x[:, :dc], 0.07), dt, (lens, b))


@pytest.mark.parametrize("gap", [19.7, 23.4, 25.05])
def test_decode_fp16_long_tail(dkv, gap):
    # one token 2^gap ahead of 32K others, every sequence whole in a CTA: the tail's weights
    # lie far below what fp16 holds beside 1, their sum does not.  A weight is 2^7 at its row's
    # reference and rounded by 2^-25 at most where it is an fp16 subnormal: N 2^-25 of a sum of
    # 2^7 or more, 2^-17 of the values, beside the half step that `check` allows.
    N, B, dc, H = 1 << 15, 152, 256, 5
    gen = gen_of("tail", gap)
    x = torch.zeros(1, N, dc + 64, dtype=torch.float16, device="cuda")
    x[..., :dc] = 0.5 + torch.rand(dc, generator=gen, device="cuda")
    x[0, 0, dc] = gap * math.log(2)
    ql = torch.zeros(1, 1, H, dc, dtype=torch.float16, device="cuda")
    qr = torch.zeros(1, 1, H, 64, dtype=torch.float16, device="cuda")
    qr[..., 0] = 1.0
    ql, qr = ql.expand(B, 1, H, dc), qr.expand(B, 1, H, 64)
    out = dkv.latent_decode_attn(ql, qr, x.expand(B, N, dc + 64), 1.0)
    q = torch.cat((ql[0, 0, :1], qr[0, 0, :1]), -1)
    ref, mag, rel = attn64(q, x[0], x[0, :, :dc], 1.0)
    check(out.flatten(0, 2), ref, mag, rel, torch.float16, gap)


@pytest.mark.parametrize("dt,power", [("bf16", 12), ("bf16", 30), ("bf16", 60), ("bf16", 100),
                                      ("fp16", 12), ("fp16", 21), ("fp16", 26), ("fp16", 30)])
def test_decode_large_scores(dkv, dt, power):
    # Scores up to 2^107: a row's largest are equal, the next ones half as large, so that the
    # output is the mean of the largest ones' values, wherever the scores lie.  (Scores are
    # whole numbers below 2^7 times a power of two, exact in fp32.)  Equal weights are
    # rounded alike, by half a step of the type; the sums add 2^-12.
    dt, H, dc, N = DT[dt], 9, 256, 700
    gen = gen_of("large", power)
    for scale in (0.08, -0.0721):
        cache, ql, qr, _ = decode_case(2, 1, H, dc, N, 0, dt, gen, [N, N], [1, 1])
        hot = torch.zeros(N, dtype=torch.bool, device="cuda")
        hot[torch.randperm(N, generator=gen, device="cuda")[:9]] = True
        ql.zero_()
        qr.fill_(2.0 ** (power // 2))
        for h in range(H):  # channels that count
            qr[:, :, h, 61 - 5 * h:] = 0.0
        top, low = 2.0 ** (power - power // 2), 2.0 ** (power - power // 2 - 1)
        cache[..., dc:] = torch.where(hot, *((top, low) if scale > 0 else (low, top)))[:, None]
        # shared by several CTAs; whole in each
        for B in (2, 160):
            c, q, r = (x if B == 2 else x[:1].expand(B, *x.shape[1:]) for x in (cache, ql, qr))
            out = dkv.latent_decode_attn(q, r, c, scale)
            x = c[:, hot, :dc].double()
            tol = (eps(dt) / 2 * 1.01 + 2.0 ** -12) * x.abs().mean(1)
            assert bool(((out[:, 0] - x.mean(1)[:, None]).abs() <= tol[:, None]).all()), scale


@pytest.mark.parametrize("H,dt,gap", [(5, "fp16", 20.3), (5, "fp16", 25.2), (40, "fp16", -3.0),
                                      (16, "bf16", -3.0), (24, "bf16", 12.0)])
def test_decode_long_sums(dkv, H, dt, gap):
    # a million tokens with values of one sign, every sequence whole in a CTA, one token 2^gap
    # ahead of the others: what a product's adders cut off (of a term 2^-26 of the sum so far)
    # must not add up over the sequence.  (fp16 weights: test_decode_fp16_long_tail.)
    N, B, dc, dt = 1 << 20, 152, 256, DT[dt]
    gen = gen_of("sums", gap)
    x = torch.zeros(1, N, dc + 64, dtype=dt, device="cuda")
    x[..., :dc] = 0.5 + torch.rand(N, dc, generator=gen, device="cuda")
    x[0, 0, dc] = gap * math.log(2)
    ql = torch.zeros(1, 1, H, dc, dtype=dt, device="cuda")
    qr = torch.zeros(1, 1, H, 64, dtype=dt, device="cuda")
    qr[..., 0] = 1.0
    ql, qr = ql.expand(B, 1, H, dc), qr.expand(B, 1, H, 64)
    out = dkv.latent_decode_attn(ql, qr, x.expand(B, N, dc + 64), 1.0)
    q = torch.cat((ql[0, 0, :1], qr[0, 0, :1]), -1)
    ref, mag, rel = attn64(q, x[0], x[0, :, :dc], 1.0)
    check(out.flatten(0, 2), ref, mag, rel, dt, gap)
    # the weights' rounding is the same for all of the tail, or beside nothing: the sums alone
    if gap < 0:
        assert float(((out - ref) / ref).abs().max()) < 2.0 ** -12


@pytest.mark.parametrize("T,H,dc", [(1, 16, 512), (3, 64, 256)])
def test_decode_long_ragged(dkv, T, H, dc):
    # sequences of many times the tokens that are summed up at a time, whole in a CTA and cut
    # between CTAs, among short and empty ones; the same bits each time
    gen, B, N = gen_of("runs", T), 40, 70000
    lens = [(0, 7, 70000, 16385, 8193, 16384, 33000, 50)[b % 8] for b in range(B)]
    new = [1 if T == 1 else (3, 1, 2, 0)[b % 4] for b in range(B)]
    x = torch.randn(1, N, dc + 64, generator=gen, device="cuda").bfloat16()
    cache = x.expand(B, N, dc + 64)
    ql = torch.randn(B, T, H, dc, generator=gen, device="cuda").bfloat16()
    qr = torch.randn(B, T, H, 64, generator=gen, device="cuda").bfloat16()
    out = torch.full((B, T, H, dc), 5.0, device="cuda")
    ws = torch.zeros(dkv.latent_workspace_bytes(B, T, H, dc, N), dtype=torch.uint8, device="cuda")
    again = out.clone()
    for o in (out, again):
        dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), new_lens=ints(new), out=o,
                               workspace=ws)
    assert dkv.read_device_status(ws) == 0
    assert torch.equal(out, again)
    check_decode(cache, ql, qr, out, lens, new, 0.07)


def test_decode_long_sequence_of_many_row_tiles(dkv):
    # more row tiles (160) than CTAs share a sequence, and more tokens than are summed at a time
    lens, new = [20000], [40]
    cache, ql, qr, out = decode_case(1, 40, 256, 256, 20000, 64, torch.bfloat16, gen_of("rows+"),
                                     lens, new)
    dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), out=out)
    check_decode(cache, ql, qr, out, lens, new, 0.07)


def test_decode_long_nan_scores(dkv):
    # NaN queries and a NaN row in sequences that are summed up in segments, whole and cut
    B, N, H, dc = 40, 33000, 20, 256
    gen = gen_of("long nan")
    x = torch.randn(1, N, dc + 64, generator=gen, device="cuda").bfloat16()
    ql = torch.randn(B, 1, H, dc, generator=gen, device="cuda").bfloat16()
    qr = torch.randn(B, 1, H, 64, generator=gen, device="cuda").bfloat16()
    ql[::3, 0, 3], qr[1, 0, 17, 5] = math.nan, math.nan
    x[0, 30000, 2] = math.nan
    lens = [33000 if b % 4 == 0 else 30000 for b in range(B)]
    out = dkv.latent_decode_attn(ql, qr, x.expand(B, N, dc + 64), 0.07, seq_lens=ints(lens))
    bad = torch.zeros(B, H, dtype=torch.bool, device="cuda")
    bad[::3, 3] = bad[1, 17] = True
    bad[::4] = True
    assert torch.equal(out[:, 0].isnan().all(-1), bad)
    x = x[0, :30000]
    for b in (1, 2, 3, 39):
        q = torch.cat((ql[b, 0], qr[b, 0]), -1)[~bad[b]]
        check(out[b, 0][~bad[b]], *attn64(q, x, x[:, :dc], 0.07), torch.bfloat16, b)


def test_decode_shared_operands(dkv):
    # one cache for all sequences, one query for all heads: dimensions of stride 0
    gen = gen_of("expanded")
    x = torch.randn(1, 200, 576, generator=gen, device="cuda").bfloat16().expand(3, 200, 576)
    ql = torch.randn(3, 1, 1, 512, generator=gen, device="cuda").bfloat16().expand(3, 1, 20, 512)
    qr = torch.randn(1, 1, 20, 64, generator=gen, device="cuda").bfloat16().expand(3, 1, 20, 64)
    lens = [200, 7, 130]
    out = torch.zeros(3, 1, 20, 512, device="cuda")
    dkv.latent_decode_attn(ql, qr, x, 0.07, seq_lens=ints(lens), out=out)
    check_decode(x, ql, qr, out, lens, [1] * 3, 0.07)


@pytest.mark.parametrize("B,T,H,dc", [(257, 1, 16, 256), (1000, 1, 20, 512), (300, 3, 64, 512),
                                      (1000, 4, 40, 256)])
def test_decode_many_sequences(dkv, B, T, H, dc):
    # more sequences than a warp counts for itself, with one row tile and several; some empty,
    # some without new tokens
    gen, N = gen_of("many", B, T), 150
    lens = [(37 * b) % 160 - 9 for b in range(B)]  # (past N: all N)
    new = [1 if T == 1 else b % (T + 1) for b in range(B)]
    cache, ql, qr, out = decode_case(B, T, H, dc, N, 16, torch.bfloat16, gen, lens, new)
    ws = torch.zeros(dkv.latent_workspace_bytes(B, T, H, dc, N), dtype=torch.uint8, device="cuda")
    again = out.clone()
    for o in (out, again):
        dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), new_lens=ints(new), out=o,
                               workspace=ws)
    assert dkv.read_device_status(ws) == 0
    assert torch.equal(out, again)
    check_decode(cache, ql, qr, out, [min(n, N) for n in lens], new, 0.07)


def test_decode_many_row_tiles(dkv):
    # more row tiles (160, of 64) than there are CTAs to share a sequence's tokens
    lens, new = [130, 41, 7, 0], [40, 38, 9, 0]
    cache, ql, qr, out = decode_case(4, 40, 256, 256, 130, 16, torch.bfloat16, gen_of("rows"), lens,
                                     new)
    ws = torch.zeros(dkv.latent_workspace_bytes(4, 40, 256, 256, 130), dtype=torch.uint8,
                     device="cuda")
    again = out.clone()
    for o in (out, again):
        dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), new_lens=ints(new), out=o,
                               workspace=ws)
    assert dkv.read_device_status(ws) == 0
    assert torch.equal(out, again)
    check_decode(cache, ql, qr, out, lens, new, 0.07)


def test_decode_workspace_of_larger_sizes(dkv):
    # one workspace for the largest call serves those of fewer new tokens and heads, in turn
    gen = gen_of("one workspace")
    ws = torch.zeros(dkv.latent_workspace_bytes(4, 4, 200, 512, 700), dtype=torch.uint8,
                     device="cuda")
    for T, H, new in ((4, 200, [4, 1, 3, 2]), (1, 16, [1] * 4), (3, 40, [3, 3, 1, 0])):
        lens = [700, 333, 64, 65]
        cache, ql, qr, out = decode_case(4, T, H, 512, 700, 16, torch.bfloat16, gen, lens, new)
        dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints(lens), new_lens=ints(new),
                               out=out, workspace=ws)
        check_decode(cache, ql, qr, out, lens, new, 0.07)


def test_decode_bad_blocks_are_reported(dkv):
    gen = gen_of("bad blocks")
    cache, ql, qr, out = decode_case(2, 1, 8, 256, 100, 16, torch.bfloat16, gen, [100, 100], [1, 1])
    ws = torch.zeros(dkv.latent_workspace_bytes(2, 1, 8, 256, 100), dtype=torch.uint8,
                     device="cuda")
    cache.block_table[0, 3] = -1
    cache.block_table[0, 4] = cache.pool.shape[0]
    want = out.clone()
    dkv.latent_decode_attn(ql, qr, cache, 0.1, seq_lens=ints([100, 100]), out=out, workspace=ws)
    assert dkv.read_device_status(ws) == 9
    x = rows_of(cache, 1)
    ref, mag, rel = attn64(torch.cat((ql[1, 0], qr[1, 0]), -1), x[:100], x[:100, :256], 0.1)
    check(out[1, 0], ref, mag, rel, torch.bfloat16)
    # entries past the length are not read
    dkv.latent_decode_attn(ql, qr, cache, 0.1, seq_lens=ints([48, 100]), out=out, workspace=ws)
    assert dkv.read_device_status(ws) == 0


def test_decode_captured_with_new_lengths(dkv):
    # a graph replayed after the lengths and the cache have changed; two graphs that share
    # one workspace, one after the other
    gen = gen_of("graph")
    B, T, H, dc, N = 3, 2, 24, 512, 700
    cache, ql, qr, out = decode_case(B, T, H, dc, N, 16, torch.bfloat16, gen, [N] * B, [T] * B)
    lens, new = ints([N] * B), ints([T] * B)
    out2 = torch.full_like(out, 5.0)
    ws = torch.zeros(dkv.latent_workspace_bytes(B, T, H, dc, N), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for scale, o in ((0.07, out), (0.02, out2)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                dkv.latent_decode_attn(ql, qr, cache, scale, seq_lens=lens, new_lens=new, out=o,
                                       workspace=ws)
            graphs.append(g)
    for case in ([N, 1, 300], [2, 2, 2]), ([64, 700, 0], [1, 0, 2]):
        lens.copy_(ints(case[0])), new.copy_(ints(case[1]))
        for o in (out, out2):
            o.fill_(5.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        check_decode(cache, ql, qr, out, *case, 0.07)
        check_decode(cache, ql, qr, out2, *case, 0.02)
    assert dkv.read_device_status(ws) == 0


def test_decode_timeout(dkv):
    # every bounded wait gives up at once: the status says so, and the next call is right
    gen = gen_of("timeout")
    cache, ql, qr, out = decode_case(2, 1, 16, 512, 900, 16, torch.bfloat16, gen, [900, 300], [1, 1])
    ws = torch.zeros(dkv.latent_workspace_bytes(2, 1, 16, 512, 900), dtype=torch.uint8,
                     device="cuda")
    dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints([900, 300]), out=out, workspace=ws,
                           flags=dkv.DKV_FLAG_FORCE_TIMEOUT)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_TIMEOUT
    dkv.latent_decode_attn(ql, qr, cache, 0.07, seq_lens=ints([900, 300]), out=out, workspace=ws)
    assert dkv.read_device_status(ws) == 0
    check_decode(cache, ql, qr, out, [900, 300], [1, 1], 0.07)


def test_decode_two_streams(dkv):
    gen = gen_of("streams")
    cases = []
    for i in range(2):
        lens = [3000 - 700 * i, 41]
        cache, ql, qr, out = decode_case(2, 1, 32, 512, 3001, 32, torch.bfloat16, gen, lens, [1, 1])
        ws = torch.zeros(dkv.latent_workspace_bytes(2, 1, 32, 512, 3001), dtype=torch.uint8,
                         device="cuda")
        cases.append((cache, ql, qr, out, lens, ints(lens), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for cache, ql, qr, out, _, n, ws, s in cases:
            with torch.cuda.stream(s):
                dkv.latent_decode_attn(ql, qr, cache, 0.05, seq_lens=n, out=out, workspace=ws)
    torch.cuda.synchronize()
    for cache, ql, qr, out, lens, _, _, _ in cases:
        check_decode(cache, ql, qr, out, lens, [1, 1], 0.05)


def test_decode_long(dkv):
    # offsets past 2^31 elements: a dense cache of 4 x 1M tokens, one of them whole
    gen = gen_of("long")
    N = (1 << 20) + 13
    x = torch.empty(4, N, 576, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    ql = torch.randn(4, 1, 16, 512, generator=gen, device="cuda").bfloat16()
    qr = torch.randn(4, 1, 16, 64, generator=gen, device="cuda").bfloat16()
    out = torch.empty(4, 1, 16, 512, device="cuda")
    lens = [5, 1000, 70001, N]
    dkv.latent_decode_attn(ql, qr, x, 0.07, seq_lens=ints(lens), out=out)
    check_decode(x, ql, qr, out, lens, [1] * 4, 0.07)


# ---------------------------------------------------------------- expanded form
def prompt_case(H, dn, nq, nk, dt, gen, extra=5, out_dtype=torch.float32):
    Tq, Tk = sum(nq) + extra, sum(nk) + extra
    q = torch.randn(Tq, H, dn + 64, generator=gen, device="cuda").to(dt)
    kv = torch.randn(Tk, H, 2 * dn, generator=gen, device="cuda").to(dt)
    kr = torch.randn(Tk, 72, generator=gen, device="cuda").to(dt)[:, :64]
    q[sum(nq):], kv[sum(nk):], kr[sum(nk):] = math.nan, math.nan, math.nan
    cu = [ints([0] + list(itertools.accumulate(n))) for n in (nq, nk)]
    out = torch.full((Tq, H, dn), 5.0, dtype=out_dtype, device="cuda")
    return (q[..., :dn], q[..., dn:], kv[..., :dn], kr, kv[..., dn:], *cu), out


def check_prompt(args, out, nq, nk, scale, causal):
    qn, qr, kn, kr, v = args[:5]
    i = j = 0
    for n, m in zip(nq, nk):
        for h in range(qn.shape[1]):
            q = torch.cat((qn[i:i + n, h], qr[i:i + n, h]), -1).double()
            k = torch.cat((kn[j:j + m, h], kr[j:j + m]), -1).double()
            x = v[j:j + m, h].double()
            if n == 0:
                continue
            if m == 0:
                assert not bool(out[i:i + n, h].any())
                continue
            seen = torch.full((n,), m, device="cuda")
            if causal:
                seen = torch.arange(m - n + 1, m + 1, device="cuda")
            off = torch.arange(m, device="cuda") >= seen[:, None]
            s = (scale * (q @ k.t())).masked_fill(off, -math.inf)
            w = torch.softmax(s, -1).masked_fill(seen[:, None] <= 0, 0.0)
            size = abs(scale) * (q.abs() @ k.abs().t()).amax(1, keepdim=True)
            top = (scale * (q @ k.t())).abs().amax(1, keepdim=True)
            rel = 2 * (q.shape[1] * 2.0 ** -23 * size + 2.0 ** -21 * (1 + top)) + \
                min(m * 2.0 ** -23, 2.0 ** -12)
            check(out[i:i + n, h], w @ x, w @ x.abs(), rel, qn.dtype, (i, h))
        i, j = i + n, j + m
    assert bool((out[i:] == 5.0).all())


PROMPT = [
    # H, dn, nq, nk
    (1, 64, [1], [1]),
    (2, 128, [128], [128]),
    (3, 128, [129, 1, 255], [129, 1, 255]),
    (2, 64, [7, 300, 0, 64], [500, 300, 20, 65]),
    (4, 128, [1, 257, 130], [1, 1000, 131]),
    (1, 128, [5, 300], [3, 200]),          # more queries than keys: the first see none
    (2, 64, [40, 3], [0, 3]),              # no keys at all
    (1, 64, [600], [1111]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", PROMPT, ids=str)
def test_prompt(dkv, case, dt, causal):
    H, dn, nq, nk = case
    dt = DT[dt]
    args, out = prompt_case(H, dn, nq, nk, dt, gen_of("prompt", H, dn, len(nq), nq[0]),
                            out_dtype=dt if causal else torch.float32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = dkv.latent_prompt_attn(*args, 0.08, causal=causal, out=out, workspace=ws)
    assert got is out and dkv.read_device_status(ws) == 0
    check_prompt(args, out, nq, nk, 0.08, causal)
    again = torch.full_like(out, 5.0)
    dkv.latent_prompt_attn(*args, 0.08, causal=causal, out=again)
    assert torch.equal(out, again)


def test_prompt_defaults_and_ranges(dkv):
    # cu_k None: keys as queries; out made by the call; large scores of both signs
    for scale in (10.0, -10.0, 0.0):
        args, _ = prompt_case(2, 64, [200, 77], [200, 77], torch.bfloat16, gen_of("p", scale),
                              extra=0)
        out = dkv.latent_prompt_attn(*args[:6], None, scale)
        assert out.dtype == torch.float32
        check_prompt(args, out, [200, 77], [200, 77], scale, True)


def test_prompt_shared_operands(dkv):
    # keys and values that the heads share: dimensions of stride 0
    gen = gen_of("pexpanded")
    args, out = prompt_case(5, 64, [150, 20], [160, 20], torch.bfloat16, gen)
    args = list(args)
    args[2], args[4] = (args[i][:, :1].expand(-1, 5, -1) for i in (2, 4))
    dkv.latent_prompt_attn(*args, 0.1, out=out)
    check_prompt(args, out, [150, 20], [160, 20], 0.1, True)


def test_prompt_many_sequences(dkv):
    # more sequences than a warp looks at at once, most of one query
    nq = [1 + (i % 7 == 0) * 300 for i in range(100)]
    nk = [n + i % 5 for i, n in enumerate(nq)]
    args, out = prompt_case(2, 64, nq, nk, torch.bfloat16, gen_of("many seqs"))
    dkv.latent_prompt_attn(*args, 0.1, out=out)
    check_prompt(args, out, nq, nk, 0.1, True)


def test_prompt_bad_bounds_are_left_alone(dkv):
    args, out = prompt_case(2, 64, [50, 60, 30], [50, 60, 30], torch.bfloat16, gen_of("bounds"),
                            extra=0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for cu_q, cu_k in (([0, 50, 110, 141], [0, 50, 110, 140]), ([0, 50, 110, 140], [0, 50, 110, 999]),
                       ([0, 50, 110, 100], [0, 50, 110, 140])):
        out.fill_(5.0)
        dkv.latent_prompt_attn(*args[:5], ints(cu_q), ints(cu_k), 0.1, out=out, workspace=ws)
        assert dkv.read_device_status(ws) == 9
        check_prompt(args[:5], out[:110], [50, 60], [50, 60], 0.1, True)
        assert bool((out[110:] == 5.0).all())


def test_prompt_timeout(dkv):
    # every bounded wait gives up at once: the status says so, and the next call is right
    args, out = prompt_case(2, 128, [300, 5], [700, 5], torch.bfloat16, gen_of("ptime"))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dkv.latent_prompt_attn(*args, 0.1, out=out, workspace=ws, flags=dkv.DKV_FLAG_FORCE_TIMEOUT)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_TIMEOUT
    out.fill_(5.0)
    dkv.latent_prompt_attn(*args, 0.1, out=out, workspace=ws)
    assert dkv.read_device_status(ws) == 0
    check_prompt(args, out, [300, 5], [700, 5], 0.1, True)


def test_prompt_many_blocks(dkv):
    # more blocks of queries than multiprocessors, so that they follow one another
    nq, nk = [700, 1, 2049, 513], [700, 900, 2049, 1500]
    args, out = prompt_case(40, 128, nq, nk, torch.bfloat16, gen_of("many"))
    dkv.latent_prompt_attn(*args, 0.08, out=out)
    check_prompt(args, out, nq, nk, 0.08, True)
    again = torch.full_like(out, 5.0)
    for _ in range(3):
        dkv.latent_prompt_attn(*args, 0.08, out=again)
        assert torch.equal(out, again)


@pytest.mark.parametrize("dn", [64, 128])
@pytest.mark.parametrize("kind", ["one tile", "no keys", "mixed"])
def test_prompt_blocks_that_use_one_query_tile_or_none(dkv, dn, kind):
    # many blocks, one after another on a multiprocessor, of which only the first query tile has
    # keys, or neither: what a block does not use must not let a warp run ahead
    B, H = 48, 16
    nq = [{"one tile": 100, "no keys": 300, "mixed": (100, 300, 280, 513)[b % 4]}[kind]
          for b in range(B)]
    nk = [{"one tile": 100, "no keys": 0, "mixed": (100, 0, 150, (1, 600)[b % 8 < 4])[b % 4]}[kind]
          for b in range(B)]
    args, out = prompt_case(H, dn, nq, nk, torch.bfloat16, gen_of("unused", kind, dn))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dkv.latent_prompt_attn(*args, 0.08, out=out, workspace=ws)
    assert dkv.read_device_status(ws) == 0
    check_prompt(args, out, nq, nk, 0.08, True)
    again = torch.full_like(out, 5.0)
    for _ in range(20):
        dkv.latent_prompt_attn(*args, 0.08, out=again, workspace=ws)
    assert dkv.read_device_status(ws) == 0
    assert torch.equal(out, again)


def test_prompt_heads_in_groups(dkv):
    # so many keys that heads are taken some at a time, the last group smaller; not by one
    for H, nq, nk in (64, [300, 520], [2100, 5000]), (5, [260], [30000]):
        args, out = prompt_case(H, 128, nq, nk, torch.bfloat16, gen_of("groups", H))
        dkv.latent_prompt_attn(*args, 0.08, out=out)
        check_prompt(args, out, nq, nk, 0.08, True)


def test_prompt_rising_scores(dkv):
    # every key tile raises the maximum, or lies far below it
    n = 1000
    for order in (1, -1):
        args, out = prompt_case(1, 64, [300], [n], torch.bfloat16, gen_of("prise"), extra=0)
        q, k = args[1], args[3]
        q.zero_(), k.zero_()
        q[..., 0] = 1.0
        up = torch.arange(n, device="cuda")
        k[:, 0] = (up if order > 0 else n - 1 - up) / 4
        dkv.latent_prompt_attn(*args, 1.0, causal=False, out=out)
        check_prompt(args, out, [300], [n], 1.0, False)


@pytest.mark.parametrize("dn", [64, 128])
@pytest.mark.parametrize("gap", [19.7, 23.4, 25.05])
def test_prompt_fp16_long_tail(dkv, gap, dn):
    # one key 2^gap ahead of 32K others (see test_decode_fp16_long_tail)
    N, H, n = 1 << 15, 2, 3
    gen = gen_of("ptail", gap, dn)
    z = torch.zeros(1, 1, dn, dtype=torch.float16, device="cuda")
    qn, kn = z.expand(n, H, dn), z.expand(N, H, dn)
    qr = torch.zeros(n, H, 64, dtype=torch.float16, device="cuda")
    kr = torch.zeros(N, 64, dtype=torch.float16, device="cuda")
    qr[..., 0] = 1.0
    kr[0, 0] = gap * math.log(2)
    v = (0.5 + torch.rand(1, H, dn, generator=gen, device="cuda")).half().expand(N, H, dn)
    args = (qn, qr, kn, kr, v, ints([0, n]), ints([0, N]))
    out = dkv.latent_prompt_attn(*args, 1.0)
    check_prompt(args, out, [n], [N], 1.0, True)


@pytest.mark.parametrize("dn", [64, 128])
@pytest.mark.parametrize("dt,power", [("bf16", 12), ("bf16", 30), ("bf16", 60), ("bf16", 100),
                                      ("fp16", 12), ("fp16", 21), ("fp16", 26), ("fp16", 30)])
def test_prompt_large_scores(dkv, dt, power, dn):
    # Scores up to 2^107: a row's largest are equal, the next ones half as large, so that the
    # output is the mean of the largest ones' values, wherever the scores lie and however the
    # scale rounds.  (Scores are whole numbers below 2^7 times a power of two, exact in fp32.)
    # Equal weights are rounded alike, by half a step of the type; the sums add 2^-12.
    dt, H, n, m = DT[dt], 4, 140, 700
    gen = gen_of("large", power, dn)
    for scale in (0.08, -0.0721):
        args, _ = prompt_case(H, dn, [n], [m], dt, gen, extra=0)
        qn, qr, kn, kr, v = args[:5]
        hot = torch.zeros(m, dtype=torch.bool, device="cuda")
        hot[torch.randperm(m, generator=gen, device="cuda")[:9]] = True
        qr.zero_(), kr.zero_()
        qn.fill_(2.0 ** (power // 2))
        for h, count in enumerate((61, 53, 47, 31)):  # channels that count
            qn[:, h, count:] = 0.0
        top, low = 2.0 ** (power - power // 2), 2.0 ** (power - power // 2 - 1)
        kn[:] = torch.where(hot, *((top, low) if scale > 0 else (low, top)))[:, None, None]
        out = dkv.latent_prompt_attn(*args, scale, causal=False)
        x = v[hot].double()
        tol = (eps(dt) / 2 * 1.01 + 2.0 ** -12) * x.abs().mean(0)
        assert bool(((out - x.mean(0)).abs() <= tol).all()), scale


@pytest.mark.parametrize("dn", [64, 128])
@pytest.mark.parametrize("dt,gap,out_dtype", [
    ("fp16", 20.3, "fp16"), ("fp16", 25.2, "fp32"), ("fp16", -3.0, "fp16"), ("bf16", -3.0, "fp32"),
    ("bf16", 12.0, "bf16"), ("fp16", 20.3, "bf16"), ("bf16", -3.0, "fp16")])
def test_prompt_long_sums(dkv, dt, gap, out_dtype, dn):
    # a million keys with values of one sign, one key 2^gap ahead of the others: what a
    # product's adders cut off (of a term 2^-26 of the sum so far) must not add up over the
    # keys.  (fp16 weights: N 2^-25 of a sum of 2^7 or more, 2^-12 of the values at the most.)
    N, H, dt = 1 << 20, 2, DT[dt]
    nq = [1, 2, 255]
    gen = gen_of("psums", gap, dn)
    z = torch.zeros(1, 1, dn, dtype=dt, device="cuda")
    n = sum(nq)
    qn, kn = z.expand(n, H, dn), z.expand(3 * N, H, dn)
    qr = torch.zeros(n, H, 64, dtype=dt, device="cuda")
    kr = torch.zeros(3 * N, 64, dtype=dt, device="cuda")
    qr[..., 0] = 1.0
    kr[::N, 0] = gap * math.log(2)
    v = (0.5 + torch.rand(3 * N, H, dn, generator=gen, device="cuda")).to(dt)
    out_dtype = DT.get(out_dtype, torch.float32)
    out = torch.full((n + 1, H, dn), 5.0, dtype=out_dtype, device="cuda")
    dkv.latent_prompt_attn(qn, qr, kn, kr, v, ints([0, 1, 3, n]), ints([0, N, 2 * N, 3 * N]), 1.0,
                           causal=False, out=out[:n])
    assert bool((out[n] == 5.0).all())
    for h in range(H):
        i = 0
        for b, m in enumerate(nq):
            keys, x = kr[b * N:(b + 1) * N], v[b * N:(b + 1) * N, h]
            ref, mag, rel = attn64(qr[:1, h], keys, x, 1.0)
            check(out[i:i + m, h], ref, mag, rel, dt, (h, b))
            # (the weights' rounding is the same for all of the tail: the sums alone)
            if gap < 0 and out_dtype == torch.float32:
                assert float(((out[i:i + m, h] - ref) / ref).abs().max()) < 2.0 ** -12
            i += m


@pytest.mark.parametrize("dt,out_dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
def test_prompt_long_rising(dkv, dt, out_dtype):
    # sums kept aside while the running maximum rises, near 0 and far from it, among rows of a
    # short sequence; a row of NaN queries leaves the others alone
    dt, (nq, nk) = DT[dt], ([700, 40], [40000, 20])
    args, out = prompt_case(2, 64, nq, nk, dt, gen_of("prise+"), out_dtype=DT.get(out_dtype,
                                                                                 torch.float32))
    q, k = args[1], args[3]
    q[:740].zero_(), k[:40020].zero_()
    q[:740, :, 0] = 1.0
    k[:40000, 0] = torch.arange(40000, device="cuda") / 1024
    for scale in (1.0, -1.0, 100.0):
        out.fill_(5.0)
        dkv.latent_prompt_attn(*args, scale, out=out)
        check_prompt(args, out, nq, nk, scale, True)
        q[50, 1, 3] = math.nan
        other = torch.full_like(out, 5.0)
        dkv.latent_prompt_attn(*args, scale, out=other)
        q[50, 1, 3] = 0.0
        assert bool(other[50, 1].isnan().all())
        other[50, 1] = out[50, 1]
        assert torch.equal(out, other)


@pytest.mark.parametrize("n", [200, 100])
def test_prompt_longer_than_a_waits_limit(dkv, n):
    # 2^25 keys: a block of queries takes longer than the 200 ms that a wait may, with both
    # query tiles at work and with one whose warps wait for the other's block to end.
    # (Equal keys and values, one row in memory: every sum is a whole number that fp32 holds.)
    N = 1 << 25
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    q, k = z(n, 1, 128), z(1, 1, 128).expand(N, 1, 128)
    v = z(1, 1, 64)
    v[0, 0] = torch.arange(64, device="cuda") % 8 + 1
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = dkv.latent_prompt_attn(q[..., :64], q[..., 64:], k[..., :64], k[:, 0, 64:],
                                 v.expand(N, 1, 64), ints([0, n]), ints([0, N]), 0.1, causal=False,
                                 workspace=ws)
    assert dkv.read_device_status(ws) == 0
    assert bool(((out - v.float()).abs() <= eps(torch.bfloat16) / 2 * v.float()).all())


def test_prompt_captured(dkv):
    args, out = prompt_case(3, 128, [300, 100], [400, 100], torch.bfloat16, gen_of("pg"), extra=300)
    cu_q, cu_k = args[5], args[6]
    kept = [a.clone() for a in args[:5]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dkv.latent_prompt_attn(*args, 0.1, out=out)
    for nq, nk in ([300, 100], [400, 100]), ([20, 350], [20, 450]), ([0, 1], [0, 1]):
        for a in (args[0], args[1], args[2], args[3], args[4]):
            a.nan_to_num_(0.5)
        cu_q.copy_(ints([0, nq[0], sum(nq)])), cu_k.copy_(ints([0, nk[0], sum(nk)]))
        out.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        check_prompt(args, out, nq, nk, 0.1, True)


# ------------------------------------------------------------------ run together
@pytest.mark.parametrize("block", [16, 64])
def test_serving_loop(dkv, block):
    """A prompt through the expanded form, its cache appended; then beams forked, drafts
    appended and attended in the absorbed form, the pool compacted on the way: every step
    against 64 bits of what the steps before stored."""
    gen = gen_of("serving", block)
    B, H, dn, dc, N = 4, 6, 64, 256, 400
    dt = torch.bfloat16
    P = -(-N // block)
    nb = B * P + 7
    pool = torch.full((nb, block, dc + 64), math.nan, dtype=dt, device="cuda")
    table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    refs[3] = 1  # a block that something else holds
    cache = dkv.LatentCache(pool, table, N)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(dkv.pages_workspace_bytes(B, P, nb),
                         dkv.latent_workspace_bytes(B, 40, H, dc, N)), dtype=torch.uint8,
                     device="cuda")
    rope = dkv.rope_table(N, 64, device="cuda")
    norm = torch.ones(dc, dtype=dt, device="cuda")
    up_k = (torch.randn(H, dc, dn, generator=gen, device="cuda") / 16).to(dt)
    up_v = (torch.randn(H, dc, dn, generator=gen, device="cuda") / 16).to(dt)
    scale = 1 / math.sqrt(dn + 64)
    model = [torch.zeros(0, dc + 64, dtype=dt, device="cuda") for _ in range(B)]

    def step(new, parents=None, T=None):
        nonlocal lens, model
        T = T or max(new)
        n = ints(new)
        par = None if parents is None else ints(parents)
        dkv.kv_pages_fork([cache], refs, lens, parents=par, new_lens=n, workspace=ws)
        assert dkv.read_device_status(ws) == 0
        if parents is not None:
            model = [model[p] if p >= 0 else model[0][:0] for p in parents]
            lens = torch.where(par >= 0, lens[par.clamp(min=0).long()], 0).to(torch.int32)
        lens = lens + n
        c = torch.randn(B, T, dc, generator=gen, device="cuda").to(dt)
        k = torch.randn(B, T, 64, generator=gen, device="cuda").to(dt)
        qn = torch.randn(B, T, H, dn, generator=gen, device="cuda").to(dt)
        qr = torch.randn(B, T, H, 64, generator=gen, device="cuda").to(dt)
        qr = dkv.latent_append(c, k, cache, seq_lens=lens, new_lens=n, q_rope=qr, rope=rope,
                               norm=norm, workspace=ws)
        for b in range(B):
            m, j = int(lens[b]), new[b]
            got = rows_of(cache, b)[:m]
            assert torch.equal(got[:m - j], model[b]), b  # what was stored is kept
            model[b] = got.clone()
        return n, qn, qr

    # prompts: the expanded form over what the cache stored
    new = [130, 0, 77, 16]
    n, qn, qr = step(new)
    flat = lambda t: torch.cat([t[b, :new[b]] for b in range(B)])
    lat = torch.cat([model[b] for b in range(B)])
    kn = torch.einsum("tc,hcd->thd", lat[:, :dc], up_k)
    v = torch.einsum("tc,hcd->thd", lat[:, :dc], up_v)
    cu = ints([0, *itertools.accumulate(new)])
    args = (flat(qn), flat(qr), kn, lat[:, dc:], v, cu, cu)
    out = torch.zeros(len(lat), H, dn, device="cuda")
    dkv.latent_prompt_attn(*args, scale, out=out)
    check_prompt(args, out, new, new, scale, True)
    # the absorbed form of the same tokens agrees with it, but for the rounding of what
    # each multiplies in 16 bits: values up to 6 rounded by 2^-9, and scores that the two
    # forms' operands, rounded by 2^-9 in some 300 channels, move by about 0.002
    ql = torch.einsum("bthd,hcd->bthc", qn, up_k)
    T = max(new)
    absorbed = dkv.latent_decode_attn(ql[:, :T], qr, cache, scale, seq_lens=lens, new_lens=n)
    both = torch.einsum("bthc,hcd->bthd", absorbed, up_v.float())
    assert float((flat(both) - out).abs().max()) < 0.05

    def decode(new, parents=None):
        n, qn, qr = step(new, parents)
        ql = torch.einsum("bthd,hcd->bthc", qn, up_k)
        out = torch.full((B, qn.shape[1], H, dc), 5.0, device="cuda")
        dkv.latent_decode_attn(ql, qr, cache, scale, seq_lens=lens, new_lens=n, out=out,
                               workspace=ws)
        assert dkv.read_device_status(ws) == 0
        check_decode(cache, ql, qr, out, lens.tolist(), new, scale)
        held = table[table >= 0].long()
        count = torch.bincount(held, minlength=nb)
        count[hold] += 1
        assert torch.equal(refs.long(), count)

    hold = 3
    decode([1, 1, 1, 1])
    decode([3, 1, 2, 3], [0, 0, 0, 2])   # beams of row 0; row 1 was nearly empty
    decode([1, 1, 1, 1], [3, 1, 1, -1])  # a row ends and starts anew
    moved = dkv.kv_pages_compact([cache], refs, workspace=ws)
    hold = int(moved[3])
    used = int((refs > 0).sum())
    assert bool((refs[:used] > 0).all()) and not bool(refs[used:].any())
    decode([2, 2, 1, 2], [0, 0, 1, 2])
    decode([1, 0, 1, 1], [2, -1, 2, 3])


@pytest.mark.parametrize("H,interleaved", [(39, False), (40, True), (128, False), (300, True)])
def test_append_many_heads(dkv, H, interleaved):
    # heads past a warp's: further warps of the same token, with and without room to spare
    gen = gen_of("heads", H)
    cache, _ = make_cache(2, 30, 512, 16, torch.bfloat16, gen)
    c, k, q = append_inputs(2, 3, H, 512, torch.bfloat16, gen)
    rope = dkv.rope_table(30, 64, device="cuda")
    out = torch.full((2, 3, H + 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dkv.latent_append(c, k, cache, seq_lens=ints([30, 9]), new_lens=ints([3, 2]), q_rope=q,
                      q_out=out[:, :, :H], rope=rope, interleaved=interleaved)
    for b, (m, n) in enumerate(((30, 3), (9, 2))):
        cos, sin = rope[0][m - n:m, None], rope[1][m - n:m, None]
        want = rotate64(q[b, :n], cos, sin, interleaved)
        # one rounding to bf16, and three of fp32 (2^-24 each) of terms up to |x|
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * q[b, :n].double().abs().amax()
        assert bool(((out[b, :n, :H].double() - want).abs() <= tol).all())
        assert bool((out[b, n:, :H] == 7).all())
        assert torch.equal(rows_of(cache, b)[m - n:m, :512], c[b, :n])
    assert bool((out[:, :, H] == 7).all())


def test_step_captured_on_another_stream(dkv):
    """A whole step -- pages, append, attention, compaction -- in one graph on a stream of its
    own, replayed with other lengths, parents and inputs; the same calls made eagerly beside
    it give the same bits."""
    gen = gen_of("step graph")
    B, T, H, dc, N, block, nb = 3, 2, 20, 256, 200, 16, 60
    P = -(-N // block)
    scale = 0.06
    dt = torch.bfloat16

    def state():
        return dict(pool=torch.zeros(nb, block, dc + 64, dtype=dt, device="cuda"),
                    table=torch.full((B, P), -1, dtype=torch.int32, device="cuda"),
                    refs=torch.zeros(nb, dtype=torch.int32, device="cuda"),
                    old=ints([0] * B), lens=ints([0] * B), parents=ints([-1] * B),
                    new=ints([0] * B),
                    c=torch.zeros(B, T, dc, dtype=dt, device="cuda"),
                    k=torch.zeros(B, T, 64, dtype=dt, device="cuda"),
                    q=torch.zeros(B, T, H, 64, dtype=dt, device="cuda"),
                    ql=torch.zeros(B, T, H, dc, dtype=dt, device="cuda"),
                    qr=torch.zeros(B, T, H, 64, dtype=dt, device="cuda"),
                    out=torch.zeros(B, T, H, dc, device="cuda"),
                    to=torch.zeros(nb, dtype=torch.int32, device="cuda"),
                    ws=torch.zeros(max(dkv.pages_workspace_bytes(B, P, nb),
                                       dkv.latent_workspace_bytes(B, T, H, dc, N)),
                                   dtype=torch.uint8, device="cuda"))

    rope = dkv.rope_table(N, 64, device="cuda")

    def step(s):
        cache = dkv.LatentCache(s["pool"], s["table"], N)
        dkv.kv_pages_fork([cache], s["refs"], s["old"], parents=s["parents"], new_lens=s["new"],
                          workspace=s["ws"])
        dkv.latent_append(s["c"], s["k"], cache, seq_lens=s["lens"], new_lens=s["new"],
                          q_rope=s["q"], q_out=s["qr"], rope=rope, workspace=s["ws"])
        dkv.latent_decode_attn(s["ql"], s["qr"], cache, scale, seq_lens=s["lens"],
                               new_lens=s["new"], out=s["out"], workspace=s["ws"])
        s["to"].copy_(dkv.kv_pages_compact([cache], s["refs"], workspace=s["ws"]))

    graphed, eager = state(), state()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step(graphed)
    lens = [0] * B
    for i, (parents, new) in enumerate([([-1] * 3, [2, 1, 2])] + [([0, 1, 2], [2, 2, 1])] * 12 +
                                       [([1, 1, 2], [1, 2, 0]), ([0, -1, 0], [2, 0, 1])]):
        old, lens = lens, [(lens[p] if p >= 0 else 0) + n for p, n in zip(parents, new)]
        fresh = {x: torch.randn(eager[x].shape, generator=gen, device="cuda").to(dt)
                 for x in ("c", "k", "q", "ql")}
        for s in graphed, eager:
            for name, x in (("old", old), ("lens", lens), ("parents", parents), ("new", new)):
                s[name].copy_(ints(x))
            for name, x in fresh.items():
                s[name].copy_(x)
            s["out"].fill_(5.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            g.replay()
        step(eager)  # at the same time
        torch.cuda.synchronize()
        for s in graphed, eager:
            assert dkv.read_device_status(s["ws"]) == 0
        for name in ("table", "refs", "out", "to"):
            assert torch.equal(graphed[name], eager[name]), (i, name)
        assert torch.equal(graphed["pool"], eager["pool"]), i
        cache = dkv.LatentCache(eager["pool"], eager["table"], N)
        check_decode(cache, eager["ql"], eager["qr"], eager["out"], lens, new, scale)
