"""Timed cases of the 8-bit KV cache and of appending to a cache.

Four operators that a decode loop runs on one cache:

  append  rotate the new tokens' keys (and queries) by their positions and write
          keys and values into the cache's pages, 16-bit or 8-bit with a scale
          per block of 16 tokens and kv head
  full    exact decode attention over an 8-bit cache
  select  page-sparse decode attention over an 8-bit cache (bound scores from
          the page metadata, top-K pages, attention over them)
  meta    the page metadata (channel-wise min / max) of an 8-bit cache: of every
          page, or of the page that each sequence's newest token lands in

``run`` computes them in plain torch operations, or with ``own`` through this
package's entry points; ``exact`` computes them in 64 bits.
"""

import math

import torch

own = False

PAGE = 16
# Largest finite e4m3 value, and the exponents a block's scale may take: the
# values code * 2^e are then all exact in the cache's 16-bit type.
E4M3_MAX = 448.0
SCALE_EXP = {"bf16": (-117, 119), "fp16": (-15, 7)}
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def _append(name, B, Hq, Hkv, d, N, T, cache, dtype="bf16", ragged=True, rotary=None,
            interleaved=False):
    return dict(name=name, op="append", B=B, Hq=Hq, Hkv=Hkv, d=d, N=N, T=T, cache=cache,
                dtype=dtype, ragged=ragged, rotary=d if rotary is None else rotary,
                interleaved=interleaved)


def _attend(name, op, B, Hq, Hkv, d, N, paged, dtype="bf16", ragged=False, top_k=0, last=False):
    return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, N=N, paged=paged, dtype=dtype,
                ragged=ragged, top_k=top_k, last=last)


def listed():
    return [
        # One decode step of a served batch of 64, 16-bit pages: the smallest call.
        _append("append-decode-bf16-paged", 64, 32, 8, 128, 4096, 1, "paged"),
        # The same step on the 32K GQA batch's 8-bit pages.
        _append("append-decode-fp8-paged", 16, 32, 8, 128, 32768, 1, "fp8_paged"),
        # Five drafted tokens a sequence, not all of them used, 1.3B-style heads.
        _append("append-draft5-fp8-mha", 37, 32, 32, 64, 2005, 5, "fp8_paged", "fp16"),
        # Prompts of up to 8K tokens entering an 8-bit cache, odd lengths.
        _append("append-prompt-fp8-paged", 8, 32, 8, 128, 8192, 8192, "fp8_paged"),
        # A tiny context: latency counts.
        _attend("full-fp8-tiny-n1k", "full", 1, 16, 16, 64, 1024, False),
        # 1.3B-style MHA batch at 8K.
        _attend("full-fp8-mha-n8k", "full", 8, 32, 32, 64, 8192, False, "fp16"),
        # The GQA batch at up to 32K tokens, every sequence its own length.
        _attend("full-fp8-gqa-n32k", "full", 16, 32, 8, 128, 32768, True, ragged=True),
        # One sequence of a million tokens.
        _attend("full-fp8-gqa-n1m", "full", 1, 32, 8, 128, 1048576, False),
        # The GQA batch at 32K with a budget of 2048 tokens.
        _attend("select-fp8-gqa-n32k", "select", 16, 32, 8, 128, 32768, True, top_k=128),
        # OPT-30B heads, a quarter of a 2K context, ragged.
        _attend("select-fp8-opt30b-n2k", "select", 64, 56, 56, 128, 2039, True, "fp16",
                ragged=True, top_k=32),
        # Metadata of the whole 32K batch, as after its prompt.
        _attend("meta-fp8-gqa-n32k", "meta", 16, 32, 8, 128, 32768, True),
        # Metadata of the newest page, as in each decode step.
        _attend("meta-fp8-last-page", "meta", 16, 32, 8, 128, 32768, True, ragged=True,
                last=True),
    ]


HEADS = [(16, 16), (32, 32), (32, 8), (56, 56), (8, 1), (12, 4), (6, 2), (28, 4), (40, 8)]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "append", "full", "full", "select", "meta"])
    Hq, Hkv = rng.choice(HEADS)
    d = rng.choice([64, 128])
    B = _spread(rng, 1, 64)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    N = _spread(rng, 1, 32768)
    N = max(1, min(N, (1 << 28) // (B * Hq * d)))
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, N=N, dtype=dtype, ragged=rng.random() < 0.7)
    if op == "append":
        T = 1 if rng.random() < 0.4 else _spread(rng, 1, min(N, 4096))
        c |= dict(T=T, cache=rng.choice(["dense", "paged", "fp8", "fp8_paged", "fp8_paged"]),
                  rotary=rng.choice([0, d // 2, d, d]), interleaved=rng.random() < 0.3)
        return c
    c |= dict(paged=rng.random() < 0.6, top_k=0, last=False)
    if op == "select":
        P = -(-N // PAGE)
        c["top_k"] = min(_spread(rng, 1, P), max(1, (1 << 27) // (B * Hq * PAGE * d)))
    if op == "meta":
        c["last"] = c["ragged"]
    return c


# --------------------------------------------------------------------- inputs
def _lens(case, gen):
    """Lengths [B] with the new tokens: up to N, one of them whole, one short."""
    B, N, T = case["B"], case["N"], case.get("T", 1)
    if not case["ragged"]:
        return torch.full((B,), N, dtype=torch.int32)
    lo = max(1, min(T, N), N // 4)
    lens = torch.randint(lo, N + 1, (B,), generator=gen, dtype=torch.int32)
    lens[-1] = lo
    lens[0] = N
    return lens


def _scale_exp(amax, dtype):
    """The smallest e with amax <= 448 * 2^e, within the type's range."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1)
    lo, hi = SCALE_EXP[dtype]
    e = e - 9 + (m > 0.875)
    return torch.where(amax == 0, lo, e).clamp(lo, hi)


def _blocks(case, gen, hot=None):
    """An 8-bit cache as blocks: codes [B, P, Hkv, 16, d] and scales [B, P, Hkv].

    Values ~ N(0, 1); the pages of `hot` = (mask [B, P, Hkv], direction
    [B, Hkv, d]) lie 10 along the direction, the pages that the queries look for."""
    B, N, Hkv, d = case["B"], case["N"], case["Hkv"], case["d"]
    P = -(-N // PAGE)
    x = torch.randn(B, P, Hkv, PAGE, d, generator=gen, device="cuda")
    if hot is not None:
        x += 10.0 * hot[0][..., None, None] * hot[1][:, None, :, None, :]
    e = _scale_exp(x.abs().amax(dim=(3, 4)), case["dtype"])
    s = torch.ldexp(torch.ones_like(x[..., 0, 0]), e)
    x /= s[..., None, None]
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), s


def _table(B, P, gen):
    """A block table of shuffled blocks, with a few blocks that no sequence holds."""
    nb = B * P + 3
    return torch.randperm(nb, generator=gen)[:B * P].view(B, P), nb


def _store(case, codes, scale, table, nb):
    """codes [B, P, Hkv, 16, d] and scales [B, P, Hkv] as the cache keeps them."""
    B, P, Hkv, _, d = codes.shape
    if table is None:
        c = codes.permute(0, 2, 1, 3, 4).reshape(B, Hkv, P * PAGE, d).contiguous()
        return c, scale.permute(0, 2, 1).contiguous()
    pool = torch.zeros(nb, Hkv, PAGE, d, dtype=codes.dtype, device="cuda")
    sc = torch.ones(nb, Hkv, device="cuda")
    pool[table.cuda().view(-1)] = codes.view(B * P, Hkv, PAGE, d)
    sc[table.cuda().view(-1)] = scale.view(B * P, Hkv)
    return pool, sc


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    B, Hq, Hkv, d, N = (case[k] for k in ("B", "Hq", "Hkv", "d", "N"))
    dt = TORCH[case["dtype"]]
    P = -(-N // PAGE)
    lens = _lens(case, host)
    s = dict(case=case, lens=lens.cuda(), lens_or_none=lens.cuda() if case["ragged"] else None)
    paged = case["paged"] if "paged" in case else case["cache"].endswith("paged")
    table, nb = _table(B, P, host) if paged else (None, 0)
    s["table"] = table.to(torch.int32).cuda() if paged else None

    if case["op"] == "append":
        T = case["T"]
        eight = case["cache"].startswith("fp8")
        qkv = torch.randn(B, T, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["q_out"] = torch.zeros(B, T, Hq, d, dtype=dt, device="cuda")
        # drafts and prompts of different lengths: not every row holds a token
        new = torch.full((B,), T, dtype=torch.int32)
        if case["ragged"] and T > 1:
            new = torch.randint(0, T + 1, (B,), generator=host, dtype=torch.int32)
            new[0] = T
        new = torch.minimum(new, lens)
        s["new"] = new.cuda()
        s["new_or_none"] = s["new"] if bool((new != T).any()) else None
        r = case["rotary"]
        pos = torch.arange(N, dtype=torch.float64)[:, None]
        inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / max(r, 1))
        s["cos"], s["sin"] = (f(pos * inv).float().cuda() for f in (torch.cos, torch.sin))
        if eight:
            for t in "KV":
                s[t], s[t + "s"] = _store(case, *_blocks(case, gen), table, nb)
        else:
            shape = (nb, Hkv, PAGE, d) if paged else (B, Hkv, P * PAGE, d)
            for t in "KV":
                s[t] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    else:
        u = torch.randn(B, Hkv, d, generator=gen, device="cuda")
        u /= u.norm(dim=-1, keepdim=True)
        hot = None
        q = torch.randn(B, Hkv, Hq // Hkv, d, generator=gen, device="cuda")
        if case["op"] == "select":
            # as many pages as the budget lie along the queries' direction; a
            # short last page's bound is over fewer keys, so it is not one of them
            q += 12.0 * u[:, :, None]
            whole = (s["lens"] // PAGE)[:, None, None]
            key = torch.rand(B, Hkv, P, generator=gen, device="cuda")
            key = torch.where(torch.arange(P, device="cuda") < whole, key, -1.0)
            at = key.argsort(dim=-1, descending=True).argsort(dim=-1)
            hot = (((at < case["top_k"]) & (key >= 0)).permute(0, 2, 1).float(), u)
        s["q"] = q.view(B, Hq, d).to(dt)
        kc, ks = _blocks(case, gen, hot)
        if case["op"] in ("select", "meta"):
            s["mn"], s["mx"] = _page_bounds(case, kc, ks, s["lens"])
        s["K"], s["Ks"] = _store(case, kc, ks, table, nb)
        del kc, ks
        if case["op"] != "meta":
            s["V"], s["Vs"] = _store(case, *_blocks(case, gen), table, nb)
            s["out"] = torch.empty(B, Hq, d, dtype=dt, device="cuda")
        if case["op"] == "select":
            s["selected"] = torch.empty(B, Hq, min(case["top_k"], P), dtype=torch.int32,
                                        device="cuda")
    if own:
        import decode_attention_paged_kv_gb300 as dkv

        for t in "KV":
            if t in s:
                s["cache" + t] = _handle(dkv, s, t)
        if case["op"] in ("full", "select"):
            n = dkv.workspace_bytes(B, Hq, Hkv, d, N, case["top_k"], fp8=True)
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        s["dkv"] = dkv
    return s


def _handle(dkv, s, t):
    """The cache object that a user's program keeps."""
    case, N, dt = s["case"], s["case"]["N"], TORCH[s["case"]["dtype"]]
    if t + "s" not in s:
        return (s[t][:, :, :N] if s["table"] is None
                else dkv.PagedCache(s[t], s["table"], N))
    codes = s[t].view(torch.float8_e4m3fn)
    if s["table"] is None:
        return dkv.Fp8Cache(codes[:, :, :N], s[t + "s"], dt)
    return dkv.Fp8PagedCache(codes, s[t + "s"], s["table"], N, dt)


# ----------------------------------------------------------------- plain forms
def _values(codes, scale):
    """The fp32 values of codes [..., 16, d] with scales [...]."""
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None, None]


def _pages(s, t):
    """(codes [B, P, Hkv, 16, d], scales [B, P, Hkv]) of a stored cache."""
    c, sc = s[t], s[t + "s"]
    if s["table"] is None:
        B, Hkv, L, d = c.shape
        return (c.view(B, Hkv, L // PAGE, PAGE, d).permute(0, 2, 1, 3, 4), sc.permute(0, 2, 1))
    bt = s["table"].long()
    return c[bt], sc[bt]


def _page_bounds(case, codes, scale, lens):
    """Channel-wise min and max of every page's keys [B, Hkv, P, d], 16-bit (exact)."""
    B, P, Hkv, _, d = codes.shape
    x = _values(codes, scale)
    tok = torch.arange(P * PAGE, device="cuda").view(P, PAGE)
    off = (tok >= lens[:, None, None])[:, :, None, :, None]
    mn = x.masked_fill(off, math.inf).amin(dim=3).permute(0, 2, 1, 3)
    mx = x.masked_fill(off, -math.inf).amax(dim=3).permute(0, 2, 1, 3)
    none = (tok[:, 0] >= lens[:, None])[:, None, :, None]
    dt = TORCH[case["dtype"]]
    return (mn.masked_fill(none, 0.0).to(dt).contiguous(),
            mx.masked_fill(none, 0.0).to(dt).contiguous())


def _softmax_v(scores, mask, v):
    """Softmax of scores [..., G, N] where the mask holds, times v [..., N, d]."""
    scores = scores.masked_fill(~mask, -math.inf)
    w = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    return torch.matmul(w, v) / w.sum(dim=-1, keepdim=True)


def _plain_full(s):
    case = s["case"]
    B, Hq, Hkv, d, N = (case[k] for k in ("B", "Hq", "Hkv", "d", "N"))
    K, V = (_values(*_pages(s, t)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d) for t in "KV")
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    sc = torch.matmul(q, K.transpose(2, 3)) / math.sqrt(d)
    mask = torch.arange(K.shape[2], device="cuda") < s["lens"][:, None, None, None]
    s["out"].copy_(_softmax_v(sc, mask, V).reshape(B, Hq, d))
    return s["out"]


def _top_pages(r, lens, kk):
    """The kk best pages of each row of r [B, Hq, P], ties to the lower page,
    ascending, padded with -1."""
    B, Hq, P = r.shape
    mine = torch.arange(P, device=r.device) < ((lens + PAGE - 1) // PAGE)[:, None, None]
    order = r.masked_fill(~mine, -math.inf).sort(dim=-1, descending=True, stable=True)[1]
    at = order[..., :kk]
    at = at.masked_fill(~mine.expand(B, Hq, P).gather(-1, at), P).sort(dim=-1)[0]
    return at.masked_fill(at == P, -1).to(torch.int32)


def _plain_select(s):
    case = s["case"]
    B, Hq, Hkv, d, N = (case[k] for k in ("B", "Hq", "Hkv", "d", "N"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Hkv, G, d)
    r = (torch.matmul(q.clamp(min=0), s["mx"].float().transpose(2, 3))
         + torch.matmul(q.clamp(max=0), s["mn"].float().transpose(2, 3)))
    kk = s["selected"].shape[-1]
    s["selected"].copy_(_top_pages(r.view(B, Hq, -1), s["lens"], kk))
    sel = s["selected"].long()
    (kc, ks), (vc, vs) = _pages(s, "K"), _pages(s, "V")
    b = torch.arange(B, device="cuda")[:, None, None]
    h = (torch.arange(Hq, device="cuda") // G)[None, :, None]
    j = sel.clamp(min=0)
    K, V = _values(kc[b, j, h], ks[b, j, h]), _values(vc[b, j, h], vs[b, j, h])
    tok = j[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    mask = ((sel >= 0)[..., None] & (tok < s["lens"][:, None, None, None])).view(B, Hq, 1, -1)
    sc = torch.matmul(s["q"].float()[:, :, None], K.view(B, Hq, -1, d).transpose(2, 3))
    s["out"].copy_(_softmax_v(sc / math.sqrt(d), mask, V.view(B, Hq, -1, d))[:, :, 0])
    return s["out"], s["selected"]


def _plain_meta(s):
    case = s["case"]
    if not case["last"]:
        return _page_bounds(case, *_pages(s, "K"), s["lens"])
    c, sc = _pages(s, "K")
    b = torch.arange(case["B"], device="cuda")
    j = (s["lens"].long() - 1) // PAGE
    x = _values(c[b, j], sc[b, j])  # [B, Hkv, 16, d]
    off = (j[:, None] * PAGE + torch.arange(PAGE, device="cuda") >= s["lens"][:, None])
    off = off[:, None, :, None]
    s["mn"][b, :, j] = x.masked_fill(off, math.inf).amin(dim=2).to(s["mn"].dtype)
    s["mx"][b, :, j] = x.masked_fill(off, -math.inf).amax(dim=2).to(s["mx"].dtype)
    return s["mn"], s["mx"]


def _rotate(x, cos, sin, interleaved):
    """x [n, H, d] rotated by cos / sin [n, r / 2]: pairs (i, i + r/2), or (2i, 2i + 1)."""
    r = 2 * cos.shape[-1]
    if r == 0:
        return x
    c, s_ = cos[:, None], sin[:, None]
    a, b = (x[..., :r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * c - b * s_, b * c + a * s_
    y = torch.stack((u, w), dim=-1).flatten(-2) if interleaved else torch.cat((u, w), dim=-1)
    return torch.cat((y, x[..., r:]), dim=-1)


def _quantised(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _new_tokens(s):
    """(sequence, row, position) of every new token."""
    T = s["case"]["T"]
    b, t = (torch.arange(T, device="cuda") < s["new"][:, None]).nonzero(as_tuple=True)
    return b, t, s["lens"].long()[b] - s["new"].long()[b] + t


def _slots(s, b, page):
    """Where page `page` of sequence b lies: indices of a stored cache's first dimensions."""
    return (s["table"].long()[b, page],) if s["table"] is not None else (b, page)


def _plain_append(s, wide=torch.float32):
    case = s["case"]
    B, Hkv, d, P = case["B"], case["Hkv"], case["d"], -(-case["N"] // PAGE)
    b, t, pos = _new_tokens(s)
    cos, sin = s["cos"].to(wide)[pos], s["sin"].to(wide)[pos]
    s["q_out"][b, t] = _rotate(s["q"][b, t].to(wide), cos, sin,
                               case["interleaved"]).to(s["q_out"].dtype)
    page, slot = pos // PAGE, pos % PAGE
    paged = s["table"] is not None
    for name, src in (("K", s["k"]), ("V", s["v"])):
        x = src[b, t].to(wide)
        if name == "K":
            x = _rotate(x, cos, sin, case["interleaved"])
        c = s[name]
        # a view [blocks, Hkv, 16, d] (paged) or [B, P, Hkv, 16, d]
        c = c if paged else c.view(B, Hkv, P, PAGE, d).permute(0, 2, 1, 3, 4)
        blk = _slots(s, b, page)
        if name + "s" not in s:
            c[(*blk, slice(None), slot)] = x.to(c.dtype)
            continue
        sc = s[name + "s"] if paged else s[name + "s"].permute(0, 2, 1)
        # the scale that the new tokens of each touched page need
        need = torch.full((B * P, Hkv), -1.0, device="cuda")
        at = (b * P + page)[:, None].expand(-1, Hkv)
        need.scatter_reduce_(0, at, x.abs().amax(dim=-1).float(), "amax")
        rows = torch.zeros(B * P, dtype=torch.bool, device="cuda")
        rows[b * P + page] = True
        rows = rows.nonzero()[:, 0]
        rb, rp = rows // P, rows % P
        e = _scale_exp(need[rows], case["dtype"])
        fresh = torch.ldexp(torch.ones_like(need[rows]), e)
        rblk = _slots(s, rb, rp)
        start = (s["lens"] - s["new"]).long()[rb]
        kept = (start - rp * PAGE).clamp(min=0)  # tokens that the page held before
        old = torch.where(kept[:, None] > 0, sc[rblk], 0.0)
        now = torch.maximum(fresh, old)
        # older tokens of a page whose scale rises are stored again
        codes = c[rblk]
        again = _quantised(codes.view(torch.float8_e4m3fn).float() * old[..., None, None],
                           now[..., None, None])
        mine = torch.arange(PAGE, device="cuda") < kept[:, None]
        c[rblk] = torch.where(mine[:, None, :, None], again, codes)
        sc[rblk] = now
        c[(*blk, slice(None), slot)] = _quantised(x, sc[blk][..., None])
    return _append_outputs(s)


def _append_outputs(s):
    r = {"q": s["q_out"], "K": s["K"], "V": s["V"]}
    if "Ks" in s:
        r = {"q": s["q_out"], "K": s["K"].view(torch.float8_e4m3fn),
             "V": s["V"].view(torch.float8_e4m3fn), "Ks": s["Ks"], "Vs": s["Vs"]}
    return r


def _own(s):
    case, dkv = s["case"], s["dkv"]
    if case["op"] == "append":
        dkv.kv_append(s["k"], s["v"], s["cacheK"], s["cacheV"], seq_lens=s["lens"],
                      new_lens=s["new_or_none"], q=s["q"], q_out=s["q_out"],
                      rope=(s["cos"], s["sin"]) if case["rotary"] else None,
                      interleaved=case["interleaved"])
        return _append_outputs(s)
    if case["op"] == "full":
        return dkv.decode_attn_full(s["q"], s["cacheK"], s["cacheV"], out=s["out"],
                                    workspace=s["workspace"], seq_lens=s["lens_or_none"])
    if case["op"] == "select":
        return dkv.decode_attn_select(s["q"], s["cacheK"], s["cacheV"], (s["mn"], s["mx"]),
                                      case["top_k"], out=s["out"], return_selected=True,
                                      selected=s["selected"], workspace=s["workspace"],
                                      seq_lens=s["lens_or_none"])
    if case["last"]:
        return dkv.kv_meta_append(s["cacheK"], (s["mn"], s["mx"]), seq_lens=s["lens_or_none"])
    return dkv.kv_meta_build(s["cacheK"], seq_lens=s["lens_or_none"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "full": _plain_full, "select": _plain_select,
            "meta": _plain_meta}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work, exact
def work(case):
    B, Hq, Hkv, d, N = (case[k] for k in ("B", "Hq", "Hkv", "d", "N"))
    # ragged lengths are spread over [N / 4, N]
    mean = N * (0.625 if case["ragged"] else 1.0)
    P = -(-N // PAGE)
    if case["op"] == "append":
        tokens = B * case["T"] * (0.5 if case["ragged"] and case["T"] > 1 else 1.0)
        eight = case["cache"].startswith("fp8")
        moved = tokens * d * (4 * Hq + 2 * Hkv * (2 + (1 if eight else 2)))
        if eight:  # one scale a touched page
            moved += 8 * Hkv * max(B, tokens / PAGE)
        return {"bytes": moved + 4 * tokens * case["rotary"],
                "flops": 3 * tokens * case["rotary"] * (Hq + Hkv)}
    head = B * Hq * d * 4  # q and out
    if case["op"] == "full":
        return {"bytes": head + 2 * B * Hkv * (mean * d + 4 * mean / PAGE),
                "flops": 4 * B * Hq * mean * d}
    if case["op"] == "select":
        pages = mean / PAGE
        kk = min(case["top_k"], pages)
        # the same pages serve the query heads of a kv head
        return {"bytes": head + 4 * B * Hq * kk
                + B * Hkv * (pages * d * 4 + 2 * kk * (PAGE * d + 4)),
                "flops": 2 * B * Hq * pages * d * 2 + 4 * B * Hq * kk * PAGE * d}
    pages = B * Hkv * (1 if case["last"] else P)
    return {"bytes": pages * (PAGE * d + 4 + 4 * d), "flops": 2 * pages * PAGE * d}


def _e4m3_64(x):
    """x (64-bit) rounded to the nearest e4m3 value, ties to even, saturated."""
    step = torch.exp2(torch.frexp(x)[1].double().sub(1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _decoded64(codes):
    """e4m3 bit patterns (uint8) as 64-bit values, from the format's fields."""
    w = codes.to(torch.int64)
    e, m = (w >> 3) & 15, (w & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    return torch.where(w >= 128, -v, v)


def _exact_attend(s, pages=None):
    """64-bit attention of every head, one sequence at a time; pages [B, Hq, P] or all."""
    case = s["case"]
    B, Hq, Hkv, d = (case[k] for k in ("B", "Hq", "Hkv", "d"))
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    for i in range(B):
        n = int(s["lens"][i])
        kv = []
        for t in "KV":
            if s["table"] is None:
                c, sc = s[t][i], s[t + "s"][i]
            else:
                at = s["table"][i].long()
                c = s[t][at].transpose(0, 1).reshape(Hkv, -1, d)
                sc = s[t + "s"][at].transpose(0, 1)
            kv.append(_decoded64(c[:, :n])
                      * sc.double().repeat_interleave(PAGE, dim=1)[:, :n, None])
        q = s["q"][i].double().view(Hkv, Hq // Hkv, d)
        sc = torch.einsum("hgd,hnd->hgn", q, kv[0]) * d ** -0.5
        if pages is not None:
            on = pages[i].repeat_interleave(PAGE, dim=-1)[:, :n]
            sc = sc.masked_fill(~on.view(Hkv, Hq // Hkv, n), -math.inf)
        out[i] = torch.einsum("hgn,hnd->hgd", torch.softmax(sc, dim=-1), kv[1]).view(Hq, d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, d, N = (case[k] for k in ("B", "Hq", "Hkv", "d", "N"))
    P = -(-N // PAGE)
    if case["op"] == "full":
        return _exact_attend(s)
    if case["op"] == "select":
        q = s["q"].double()
        kv = torch.arange(Hq, device="cuda") // (Hq // Hkv)
        pages = torch.zeros(B, Hq, P, dtype=torch.bool, device="cuda")
        for i in range(B):
            mn, mx = s["mn"][i].double()[kv], s["mx"][i].double()[kv]
            qi = q[i][:, None]
            r = torch.where(qi >= 0, qi * mx, qi * mn).sum(dim=-1)
            n = -(-int(s["lens"][i]) // PAGE)
            best = r[:, :n].sort(dim=-1, descending=True, stable=True)[1][:, :case["top_k"]]
            pages[i].scatter_(1, best, True)
        return _exact_attend(s, pages), None
    if case["op"] == "meta":
        mn, mx = s["mn"].double(), s["mx"].double()
        for i in range(B):
            n = int(s["lens"][i])
            for j in range(-(-n // PAGE) - 1 if case["last"] else 0, -(-n // PAGE)):
                at = (s["table"][i, j].long(),) if s["table"] is not None else (i,)
                sl = slice(0, PAGE) if s["table"] is not None else slice(PAGE * j, PAGE * j + PAGE)
                sc = s["Ks"][at] if s["table"] is not None else s["Ks"][i, :, j]
                x = _decoded64(s["K"][at][:, sl][:, :n - PAGE * j]) * sc.double()[:, None, None]
                mn[i, :, j], mx[i, :, j] = x.amin(dim=1), x.amax(dim=1)
        return mn, mx
    # append: the new tokens, one sequence at a time
    r = {k: v.double() if not k[0] in "KV" or len(k) == 2 else
         (_decoded64(s[k]) if k + "s" in s else v.double())
         for k, v in _append_outputs(s).items()}
    lo, hi = SCALE_EXP[case["dtype"]]
    for i in range(B):
        n, m = int(s["new"][i]), int(s["lens"][i])
        if n == 0:
            continue
        first = m - n
        cos, sin = s["cos"][first:m].double()[:, None], s["sin"][first:m].double()[:, None]
        h = case["rotary"] // 2

        def turned(x):
            y = x.double().clone()
            a, b = ((slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["interleaved"]
                    else (slice(0, h), slice(h, 2 * h)))
            y[..., a] = x.double()[..., a] * cos - x.double()[..., b] * sin
            y[..., b] = x.double()[..., b] * cos + x.double()[..., a] * sin
            return y

        r["q"][i, :n] = turned(s["q"][i, :n])
        p0, p1 = first // PAGE, (m - 1) // PAGE + 1
        for t, x in (("K", turned(s["k"][i, :n])), ("V", s["v"][i, :n].double())):
            # the touched pages [pages, Hkv, 16, d], with the new tokens in place
            at = s["table"][i, p0:p1].long() if s["table"] is not None else None
            old = (r[t][at] if at is not None else
                   r[t].view(B, Hkv, P, PAGE, d)[i, :, p0:p1].transpose(0, 1))
            tok = torch.arange(p0 * PAGE, p1 * PAGE, device="cuda").view(-1, 1, PAGE, 1)
            is_new, is_old = (tok >= first) & (tok < m), tok < first
            put = torch.zeros((p1 - p0) * PAGE, Hkv, d, dtype=torch.float64, device="cuda")
            put[first - p0 * PAGE:m - p0 * PAGE] = x
            put = put.view(p1 - p0, PAGE, Hkv, d).transpose(1, 2)
            if t + "s" in r:
                sc = r[t + "s"][at] if at is not None else r[t + "s"][i, :, p0:p1].t()
                had = torch.where(is_old.any(dim=2)[..., 0], sc, 0.0)
                amax = put.abs().amax(dim=(2, 3))
                e = torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(lo, hi)
                now = torch.maximum(torch.exp2(e), had)[..., None, None]
                put = _e4m3_64(put / now)
                old = torch.where(is_old, _e4m3_64(old * had[..., None, None] / now), old)
                if at is not None:
                    r[t + "s"][at] = now[..., 0, 0]
                else:
                    r[t + "s"][i, :, p0:p1] = now[..., 0, 0].t()
            new = torch.where(is_new, put, old)
            if at is not None:
                r[t][at] = new
            else:
                r[t].view(B, Hkv, P, PAGE, d)[i, :, p0:p1] = new.transpose(0, 1)
    return r
