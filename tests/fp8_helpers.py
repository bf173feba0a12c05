"""Plain 64-bit forms of the 8-bit cache, of appending with the position
rotation and of attention, for the tests (no code shared with the kernels)."""

import math

import numpy as np
import torch

PAGE = 16
EXP = {torch.bfloat16: (-117, 119), torch.float16: (-15, 7)}


def e4m3_values() -> np.ndarray:
    """The 256 values of the e4m3 format, by its fields (0x7f and 0xff: NaN)."""
    out = np.empty(256)
    for w in range(256):
        e, m = (w >> 3) & 15, w & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = math.nan
        out[w] = -v if w & 128 else v
    return out


TABLE = torch.from_numpy(e4m3_values())


def decode(codes: torch.Tensor) -> torch.Tensor:
    """float8 codes as 64-bit values, on the CPU."""
    return TABLE[codes.cpu().view(torch.uint8).long()]


def encode(x: torch.Tensor) -> torch.Tensor:
    """64-bit values to the nearest e4m3 value, ties to even, saturated."""
    step = torch.exp2(torch.frexp(x)[1].double().sub(1).clamp(min=-6) - 3)
    y = (torch.round(x / step) * step).clamp(-448.0, 448.0)
    c = y.to(torch.float8_e4m3fn)  # exact: y is an e4m3 value
    assert torch.equal(TABLE[c.view(torch.uint8).long()], y)
    return c


def block_scale(amax: torch.Tensor, dtype) -> torch.Tensor:
    """2^e, e the smallest with amax <= 448 * 2^e, clamped (64-bit)."""
    lo, hi = EXP[dtype]
    a = amax.double()
    e = torch.full_like(a, lo)
    for k in range(lo, hi):  # by the definition
        e = torch.where(a > 448.0 * 2.0 ** k, float(k + 1), e)
    return torch.exp2(e)


def quantise(x: torch.Tensor, dtype):
    """x [B, Hkv, N, d] -> codes [B, Hkv, N, d], scale [B, Hkv, P] (float32)."""
    B, H, N, d = x.shape
    P = -(-N // PAGE)
    y = torch.zeros(B, H, P * PAGE, d, dtype=torch.float64)
    y[:, :, :N] = x.double()
    y = y.view(B, H, P, PAGE, d)
    s = block_scale(y.abs().amax(dim=(3, 4)), dtype)
    c = encode(y / s[..., None, None]).view(B, H, P * PAGE, d)[:, :, :N].contiguous()
    return c, s.float()


def values(codes, scale, N=None):
    """codes [B, Hkv, N, d], scale [B, Hkv, P] -> 64-bit values."""
    n = codes.shape[2]
    return decode(codes) * scale.cpu().double().repeat_interleave(PAGE, dim=2)[:, :, :n, None]


def to_pool(codes, scale, spare=5, spare_cols=3, seed=0, lens=None):
    """A shuffled pool of the same blocks.  What no sequence owns -- slots past
    a sequence's end, spare blocks and their scales -- is NaN."""
    B, H, N, d = codes.shape
    P = scale.shape[2]
    nb = B * P + spare
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(seed))[:B * P]
    bt = torch.full((B, P + spare_cols), -7, dtype=torch.int32)
    bt[:, :P] = order.view(B, P).to(torch.int32)
    full = torch.full((B, H, P * PAGE, d), 0x7F, dtype=torch.uint8)
    full[:, :, :N] = codes.view(torch.uint8)
    sc = scale.clone()
    if lens is not None:
        for b, n in enumerate(lens):
            n = max(0, int(n))
            full[b, :, n:] = 0x7F
            sc[b, :, -(-n // PAGE):] = math.nan
    pool = torch.full((nb, H, PAGE, d), 0x7F, dtype=torch.uint8)
    pool[order] = full.view(B, H, P, PAGE, d).permute(0, 2, 1, 3, 4).reshape(B * P, H, PAGE, d)
    ps = torch.full((nb, H), math.nan)
    ps[order] = sc.permute(0, 2, 1).reshape(B * P, H)
    return pool.view(torch.float8_e4m3fn), ps, bt


def attention(q, k, v, scale, lens=None, pages=None, S=PAGE):
    """64-bit attention; q [B, Hq, d], k / v [B, Hkv, N, d] values; pages: for
    each (b, h) the page indices attended (a list of lists of lists), else all."""
    B, Hq, d = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(B, Hq, d, dtype=torch.float64)
    for b in range(B):
        n = k.shape[2] if lens is None else int(lens[b])
        if n <= 0:
            continue
        for h in range(Hq):
            s = (k[b, h // G, :n] @ q[b, h].double()) * scale
            if pages is not None:
                on = torch.zeros(-(-n // S), dtype=torch.bool)
                on[[int(j) for j in pages[b][h] if j >= 0]] = True
                s = s.masked_fill(~on.repeat_interleave(S)[:n], -math.inf)
            out[b, h] = torch.softmax(s, dim=0) @ v[b, h // G, :n]
    return out


def tolerance(q, k, v, scale) -> float:
    """Bound on |out - exact| of the kernels with an fp32 output.

    Queries, codes and scales enter exactly.  A score is a sum of d products
    accumulated in fp32 over at most 8 steps plus two scalings: off by at most
    d_s = 12 * 2^-23 * sum |q_i k_i| * scale (2^-23 covers a truncating
    accumulator), so numerator and denominator weights are off by 2 d_s
    relative together.  2^x is off by 2^-21, the weights' two fp16 halves by
    2^-21, and summing them by 2^-23 of sum p |v| a step, at most 256 steps:
    2^-15.  All relative to sum p |v| <= max |v|."""
    G = q.shape[1] // k.shape[1]
    top = 0.0
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            kk = k[b, h // G].nan_to_num().abs()
            top = max(top, float((kk @ q[b, h].double().abs()).max()) * scale)
    d_s = 12 * 2.0 ** -23 * top
    return float(v.nan_to_num().abs().max()) * (2 * d_s + 2 * 2.0 ** -21 + 2.0 ** -15)


def rotated(x, pos, rope, interleaved):
    """x [n, H, d] (16-bit) rotated at positions [n]; fp32, step by step."""
    y = x.float().clone()
    if rope is None:
        return y
    c, s = rope[0][pos][:, None], rope[1][pos][:, None]
    h = c.shape[-1]
    a, b = ((slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved
            else (slice(0, h), slice(h, 2 * h)))
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


def quotient(y, s):
    """fp32 y [Hkv, ...] over the scales s [Hkv], rounded to fp32 (exact for
    powers of two), as 64-bit values."""
    return (y.float() / s.float()[:, None, None]).double()


def append(k, v, K, V, lens, news, q=None, q_out=None, rope=None, interleaved=False):
    """The reference of kv_append on CPU tensors, in place.  K, V: logical
    caches: values [B, Hkv, L, d], or (codes uint8 [B, Hkv, L, d], scale
    [B, Hkv, L / 16], dtype) with L a multiple of 16."""
    B = k.shape[0]
    for b in range(B):
        n, end = int(news[b]), int(lens[b])
        if n == 0 or end <= 0:
            continue
        start = end - n
        pos = torch.arange(start, end)
        if q is not None:
            q_out[b, :n] = rotated(q[b, :n], pos, rope, interleaved).to(q.dtype)
        for x, cache in ((rotated(k[b, :n], pos, rope, interleaved), K), (v[b, :n].float(), V)):
            if not isinstance(cache, tuple):
                cache[b, :, start:end] = x.transpose(0, 1).to(cache.dtype)
                continue
            codes, scale, dt = cache
            for p in range(start // PAGE, -(-end // PAGE)):
                lo, hi = max(start, p * PAGE), min(end, (p + 1) * PAGE)
                new = x[lo - start:hi - start].transpose(0, 1)  # [Hkv, tokens, d]
                s = block_scale(new.abs().amax(dim=(1, 2)), dt)
                if lo > p * PAGE:
                    old = scale[b, :, p].double()
                    s = torch.maximum(s, old)
                    at = codes[b, :, p * PAGE:lo]
                    again = encode(quotient(TABLE[at.long()].float()
                                            * old.float()[:, None, None], s))
                    rise = (s > old)[:, None, None]
                    codes[b, :, p * PAGE:lo] = torch.where(rise, again.view(torch.uint8), at)
                scale[b, :, p] = s.float()
                codes[b, :, lo:hi] = encode(quotient(new, s)).view(torch.uint8)
