"""64-bit forms of the calls on latent caches, inputs, and the errors that the formats
allow, for their GPU tests."""

import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def eps(dt):
    return torch.finfo(dt).eps


def make_cache(B, N, dc, block, dt, gen, pad=0, spare=2):
    """(cache, the sequences' rows [B, N', dc + 64] as views to read or write through).
    Paged: shuffled blocks with some that no sequence holds, NaN in those.  pad: extra
    elements between rows."""
    import decode_attention_paged_kv_gb300 as dkv
    w = dc + 64
    if block == 0:
        t = torch.randn(B, N, w + pad, generator=gen, device="cuda").to(dt)[..., :w]
        return t, None
    P = -(-N // block)
    nb = B * P + spare
    pool = torch.randn(nb, block, w + pad, generator=gen, device="cuda").to(dt)[..., :w]
    order = torch.randperm(nb, generator=gen, device="cuda")
    pool[order[B * P:]] = math.nan
    table = order[:B * P].view(B, P).to(torch.int32)
    return dkv.LatentCache(pool, table, N), table


def rows_of(cache, b):
    """Sequence b's rows [N', w] in order."""
    if isinstance(cache, torch.Tensor):
        return cache[b]
    return cache.pool[cache.block_table[b].long()].flatten(0, 1)


def hide_tail(cache, lens):
    """NaN in every row that lies past its sequence."""
    for b, n in enumerate(lens):
        n = max(n, 0)
        if isinstance(cache, torch.Tensor):
            cache[b, n:] = math.nan
            continue
        S = cache.pool.shape[1]
        for j, blk in enumerate(cache.block_table[b].tolist()):
            cache.pool[blk, min(max(n - j * S, 0), S):] = math.nan


def attn64(q, keys, values, scale):
    """(out, bound): softmax(scale q . keys) values in 64 bits for q [R, w], keys [n, w],
    values [n, c]; and what the scores' fp32 sums and the weights' rounding to 16 bits may
    change of it.

    A score is a sum of w products of 16-bit values (exact in fp32): any order of fp32
    additions, also truncating ones, is off by at most w 2^-23 sum |q k|; scaling and the
    exponential add 2^-21 relative to the exponent's size.  An error e of all scores
    changes a weight by 2 e at most.  A weight rounded to the type is off by eps / 2; the
    fp32 sums of the weights and of the product by 2^-23 a step, counted for n steps up to
    2^-12 (the sums run in blocks)."""
    q, keys, values = q.double(), keys.double(), values.double()
    s = scale * (q @ keys.t())
    size = abs(scale) * (q.abs() @ keys.abs().t()).amax(dim=1, keepdim=True)
    w = torch.softmax(s, dim=-1)
    mag = w @ values.abs()
    rel = 2 * (q.shape[1] * 2.0 ** -23 * size + 2.0 ** -21 * (1 + s.abs().amax(dim=1, keepdim=True)))
    steps = min(keys.shape[0] * 2.0 ** -23, 2.0 ** -12)
    return w @ values, mag, rel + steps


def check(out, ref, mag, rel, dt, what=""):
    """out within the weights' rounding (type dt), the scores' error and its own rounding."""
    o = eps(out.dtype) / 2 if out.dtype != torch.float32 else 2.0 ** -23
    tol = (eps(dt) / 2 * 1.01 + rel) * mag * (1 + o) + o * ref.abs() + 1e-30
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormals
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((out.double() - ref).abs().max()),
                                 float(tol.min()))


def rotate64(x, cos, sin, interleaved):
    x, cos, sin = x.double(), cos.double(), sin.double()
    h = x.shape[-1] // 2
    a, b = ((slice(0, None, 2), slice(1, None, 2)) if interleaved
            else (slice(0, h), slice(h, None)))
    y = torch.empty_like(x)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y
