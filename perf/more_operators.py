"""Timed cases of latent caches and of the life of a cache's pages.

Five operators around a cache that holds one latent vector and one rotated key a
token, shared by all heads, and around the pages that caches are made of:

  append   normalise the new tokens' latent vectors, rotate their shared keys (and
           the queries' rotary parts) by their positions, write both into the cache
  decode   attention of one or a few new tokens a sequence over the latent cache:
           the latent vectors are keys and values at once (the absorbed form)
  prompt   causal attention of prompts, or of their last chunks, with keys and
           values expanded a head (the expanded form); the rotated key stays shared
  fork     one step of a cache's block table: rows continue a parent row, share its
           whole pages, copy its last one, take pages for new tokens, free the rest
  compact  move a pool's pages in use to its front and rename them in the table

``run`` computes them in plain torch operations, or with ``own`` through this
package's entry points; ``exact`` computes them in 64 bits.
"""

import math

import torch

own = False

PAGE = 16
EPS = 1e-6
ROPE = 64  # channels of the rotated part
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def _append(name, B, T, H, dc, N, page, dtype="bf16", ragged=True, interleaved=False):
    return dict(name=name, op="append", B=B, T=T, H=H, dc=dc, N=N, page=page, dtype=dtype,
                ragged=ragged, interleaved=interleaved)


def _decode(name, B, T, H, dc, N, page, dtype="bf16", ragged=True):
    return dict(name=name, op="decode", B=B, T=T, H=H, dc=dc, N=N, page=page, dtype=dtype,
                ragged=ragged)


def _prompt(name, B, H, dn, nq, nk, dtype="bf16", ragged=True):
    return dict(name=name, op="prompt", B=B, H=H, dn=dn, nq=nq, nk=nk, dtype=dtype, ragged=ragged)


def _fork(name, B, N, blocks, beams, cache, Hkv=8, d=128):
    return dict(name=name, op="fork", B=B, N=N, blocks=blocks, beams=beams, cache=cache, Hkv=Hkv,
                d=d)


def _compact(name, B, N, blocks, live, cache, Hkv=8, d=128):
    return dict(name=name, op="compact", B=B, N=N, blocks=blocks, live=live, cache=cache, Hkv=Hkv,
                d=d)


def listed():
    return [
        # One decode step of a served batch of 64.
        _append("append-latent-decode", 64, 1, 32, 512, 4096, 16),
        # Prompts of up to 8K tokens entering the cache, odd lengths.
        _append("append-latent-prompt", 8, 8192, 32, 512, 8192, 64),
        # A tiny context: latency counts.
        _decode("decode-latent-tiny-n1k", 1, 1, 16, 256, 1024, 0, "fp16", False),
        # The long batch, few heads a GPU: every sequence its own length.
        _decode("decode-latent-h16-n32k", 16, 1, 16, 512, 32768, 16),
        # All 128 heads of a model on one GPU.
        _decode("decode-latent-h128-n8k", 32, 1, 128, 512, 8192, 64, ragged=False),
        # Four drafted tokens a sequence, not all of them used.
        _decode("decode-latent-draft4", 7, 4, 40, 512, 16001, 32, "fp16"),
        # The last 2K-token chunk of prompts of up to 8K tokens.
        _prompt("prompt-latent-chunk", 4, 16, 128, 2048, 8192),
        # A batch of short prompts, odd lengths.
        _prompt("prompt-latent-short", 16, 32, 64, 777, 777, "fp16"),
        # One step of 64 beams in groups of four over 32K-token contexts.
        _fork("fork-beams-n32k", 64, 32768, 34000, 4, "kv16", 2),
        # Four beams over a short context, 8-bit pages: latency counts.
        _fork("fork-beams-small", 4, 1021, 301, 4, "fp8", 3, 64),
        # A pool of a gigabyte, half of it in use after sequences ended.
        _compact("compact-half", 48, 8192, 16384, 0.5, "kv16"),
        # A latent pool of odd size, most of it in use.
        _compact("compact-latent", 9, 5000, 1201, 0.8, "latent"),
    ]


HEADS = [8, 16, 20, 32, 40, 64, 128]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("append", "decode"):
        B, H = _spread(rng, 1, 64), rng.choice(HEADS)
        dc, page = rng.choice([256, 512, 512]), rng.choice([0, 16, 16, 32, 64])
        N = _spread(rng, 1, 32768)
        ragged = rng.random() < 0.7
        if op == "append":
            N = max(1, min(N, 65536 // B))
            T = 1 if rng.random() < 0.4 else _spread(rng, 1, min(N, 8192))
            return dict(op=op, B=B, T=T, H=min(H, 32), dc=dc, N=N, page=page, dtype=dtype,
                        ragged=ragged, interleaved=rng.random() < 0.3)
        T = 1 if rng.random() < 0.6 else rng.randint(1, 5)
        N = max(T, min(N, (32 * 8192 * 128) // (B * T * max(H, 64))))
        return dict(op=op, B=B, T=T, H=H, dc=dc, N=N, page=page, dtype=dtype, ragged=ragged)
    if op == "prompt":
        H, dn = rng.choice([4, 5, 8, 16, 32]), rng.choice([64, 128, 128])
        B = _spread(rng, 1, 16)
        nk = _spread(rng, 1, 8192)
        nq = nk if rng.random() < 0.5 else _spread(rng, 1, nk)
        nq = max(1, min(nq, (1 << 30) // (B * H * nk)))
        return dict(op=op, B=B, H=H, dn=dn, nq=nq, nk=nk, dtype=dtype, ragged=rng.random() < 0.7)
    cache = rng.choice(["kv16", "fp8", "latent"])
    Hkv, d = rng.choice([1, 2, 3, 8]), rng.choice([64, 128])
    B = _spread(rng, 1, 64)
    if op == "fork":
        beams = rng.choice([1, 2, 4, 8])
        N = max(1, min(_spread(rng, 1, 32768), 16 * 30000 // -(-B // beams)))
        need = (-(-B // beams) + 1) * (-(-N // PAGE) + 2) + 4 * B
        return dict(op=op, B=B, N=N, blocks=need + _spread(rng, 1, 2000), beams=beams,
                    cache=cache, Hkv=min(Hkv, 3), d=d)
    return dict(op=op, B=B, N=_spread(rng, 1, 8192), blocks=_spread(rng, 16, 16384),
                live=rng.choice([0.1, 0.3, 0.5, 0.8, 1.0]), cache=cache, Hkv=Hkv, d=d)


# --------------------------------------------------------------------- inputs
def _lens(case, gen):
    """Lengths [B] with the new tokens: up to N, one of them whole, one short."""
    B, N, T = case["B"], case["N"], case["T"]
    if not case["ragged"]:
        return torch.full((B,), N, dtype=torch.int32)
    lo = max(1, min(T, N), N // 4)
    lens = torch.randint(lo, N + 1, (B,), generator=gen, dtype=torch.int32)
    lens[-1] = lo
    lens[0] = N
    return lens


def _latent_inputs(case, s, host, gen):
    B, T, H, dc, N, page = (case[k] for k in ("B", "T", "H", "dc", "N", "page"))
    dt = TORCH[case["dtype"]]
    lens = _lens(case, host)
    # drafts and prompts of different lengths: not every row holds a token
    new = torch.full((B,), T, dtype=torch.int32)
    if case["ragged"] and T > 1:
        new = torch.randint(0, T + 1, (B,), generator=host, dtype=torch.int32)
        new[0] = T
    new = torch.minimum(new, lens)
    s["lens"], s["new"] = lens.cuda(), new.cuda()
    s["lens_or_none"] = s["lens"] if case["ragged"] else None
    s["new_or_none"] = s["new"] if bool((new != T).any()) else None
    if page:
        P = -(-N // page)
        nb = B * P + 3
        s["table"] = torch.randperm(nb, generator=host)[:B * P].view(B, P).to(torch.int32).cuda()
        shape = (nb, page, dc + ROPE)
    else:
        s["table"] = None
        shape = (B, N, dc + ROPE)
    s["cache"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen)
    if case["op"] == "append":
        s["c"] = (3.0 * torch.randn(B, T, dc, generator=gen, device="cuda")).to(dt)
        s["k"] = torch.randn(B, T, ROPE, generator=gen, device="cuda").to(dt)
        s["q"] = torch.randn(B, T, H, ROPE, generator=gen, device="cuda").to(dt)
        s["norm"] = (1.0 + 0.1 * torch.randn(dc, generator=gen, device="cuda")).to(dt)
        s["q_out"] = torch.zeros(B, T, H, ROPE, dtype=dt, device="cuda")
        pos = torch.arange(N, dtype=torch.float64)[:, None]
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)
        s["cos"], s["sin"] = (f(pos * inv).float().cuda() for f in (torch.cos, torch.sin))
        return
    # the absorbed queries come out of a product over the heads, [H, B * T, dc]
    s["ql"] = torch.randn(H, B, T, dc, generator=gen, device="cuda").to(dt).permute(1, 2, 0, 3)
    s["qr"] = torch.randn(B, T, H, ROPE, generator=gen, device="cuda").to(dt)
    s["out"] = torch.zeros(B, T, H, dc, dtype=dt, device="cuda")
    s["scale"] = 1.0 / math.sqrt(128 + ROPE)


def _prompt_inputs(case, s, host, gen):
    B, H, dn, nq, nk = (case[k] for k in ("B", "H", "dn", "nq", "nk"))
    dt = TORCH[case["dtype"]]
    q, k = torch.full((B,), nq), torch.full((B,), nk)
    if case["ragged"]:
        k = torch.randint(max(1, nk // 4), nk + 1, (B,), generator=host)
        k[0] = nk
        if nq == nk:
            q = k.clone()
        else:
            q = torch.randint(max(1, nq // 4), nq + 1, (B,), generator=host)
            q[0] = nq
            q = torch.minimum(q, k)
    s["nq"], s["nk"] = q.tolist(), k.tolist()
    cum = lambda n: torch.cat((torch.zeros(1, dtype=torch.int64), n.cumsum(0))).to(torch.int32).cuda()
    s["cu_q"], s["cu_k"] = cum(q), cum(k)
    # buffers of a captured step: the sequences lie one after another at their front
    Tq, Tk = B * nq, B * nk
    qs = torch.randn(Tq, H, dn + ROPE, generator=gen, device="cuda").to(dt)
    kv = torch.randn(Tk, H, 2 * dn, generator=gen, device="cuda").to(dt)
    s["qn"], s["qr"], s["kn"], s["v"] = qs[..., :dn], qs[..., dn:], kv[..., :dn], kv[..., dn:]
    s["kr"] = torch.randn(Tk, ROPE, generator=gen, device="cuda").to(dt)
    s["out"] = torch.zeros(Tq, H, dn, dtype=dt, device="cuda")
    s["scale"] = 1.0 / math.sqrt(dn + ROPE)


def _pools(case, gen):
    """The tensors of a cache whose first dimension counts its blocks."""
    nb, H, d = case["blocks"], case["Hkv"], case["d"]
    rnd = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(
        generator=gen)
    if case["cache"] == "latent":
        return [rnd(nb, PAGE, 512 + ROPE)]
    if case["cache"] == "kv16":
        return [rnd(nb, H, PAGE, d) for _ in "KV"]
    codes = [rnd(nb, H, PAGE, d).to(torch.float8_e4m3fn).view(torch.uint8) for _ in "KV"]
    scales = [torch.exp2(torch.randint(-8, 9, (nb, H), generator=gen, device="cuda").float())
              for _ in "KV"]
    return [codes[0], scales[0], codes[1], scales[1]]


def _fork_inputs(case, s, host, gen):
    B, N, nb, beams = (case[k] for k in ("B", "N", "blocks", "beams"))
    P = -(-N // PAGE) + 1
    groups = -(-B // beams)
    # the beams of a group have one length and share their whole pages
    glen = torch.randint(max(1, N // 4), N + 1, (groups,), generator=host)
    glen[0] = N
    group = torch.arange(B) // beams
    lens = glen[group]
    whole, some = lens // PAGE, lens % PAGE != 0
    perm = torch.randperm(nb, generator=host)
    start = torch.cat((torch.zeros(1, dtype=torch.int64), (glen // PAGE).cumsum(0)))
    j = torch.arange(P)
    table = torch.full((B, P), -1, dtype=torch.int64)
    at = (start[group][:, None] + j).clamp(max=nb - 1)
    table = torch.where(j < whole[:, None], perm[at], table)
    own_page = perm[start[-1] + torch.arange(B)]  # a last page of each beam's own
    table = torch.where((j == whole[:, None]) & some[:, None], own_page[:, None], table)
    refs = torch.bincount(table[table >= 0], minlength=nb)
    # a beam continues some beam of its group
    size = torch.where(group == groups - 1, B - (groups - 1) * beams, beams)
    parents = group * beams + (torch.rand(B, generator=host) * size).long()
    s["table"], s["refs"] = table.to(torch.int32).cuda(), refs.to(torch.int32).cuda()
    s["lens"], s["parents"] = lens.to(torch.int32).cuda(), parents.to(torch.int32).cuda()
    s["new"] = torch.ones(B, dtype=torch.int32, device="cuda")


def _compact_inputs(case, s, host):
    B, N, nb = case["B"], case["N"], case["blocks"]
    P = -(-N // PAGE)
    live = torch.randperm(nb, generator=host)[:max(1, int(nb * case["live"]))]
    # rows hold the live pages between them, the first few pages are shared
    table = torch.full((B * P,), -1, dtype=torch.int64)
    n = min(B * P, len(live))
    table[torch.randperm(B * P, generator=host)[:n]] = live[:n]
    table = table.view(B, P)
    table[:, 0] = live[0]
    refs = torch.bincount(table[table >= 0], minlength=nb)
    refs[live] += refs[live] == 0  # pages that a prefix index holds
    s["table"], s["refs"] = table.to(torch.int32).cuda(), refs.to(torch.int32).cuda()
    s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("append", "decode"):
        _latent_inputs(case, s, host, gen)
    elif op == "prompt":
        _prompt_inputs(case, s, host, gen)
    else:
        s["pools"] = _pools(case, gen)
        if op == "fork":
            _fork_inputs(case, s, host, gen)
        else:
            _compact_inputs(case, s, host)
    if own:
        import decode_attention_paged_kv_gb300 as dkv

        s["dkv"] = dkv
        if op in ("append", "decode"):
            s["handle"] = (s["cache"] if s["table"] is None
                           else dkv.LatentCache(s["cache"], s["table"], case["N"]))
            if op == "decode":
                n = dkv.latent_workspace_bytes(case["B"], case["T"], case["H"], case["dc"],
                                               case["N"])
                s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        elif op in ("fork", "compact"):
            s["handles"] = _handles(dkv, s)
            n = dkv.pages_workspace_bytes(case["B"], s["table"].shape[1], case["blocks"])
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s


def _handles(dkv, s):
    """The cache objects that a user's program keeps."""
    p, table, N = s["pools"], s["table"], s["case"]["N"]
    if s["case"]["cache"] == "latent":
        return [dkv.LatentCache(p[0], table, N)]
    if s["case"]["cache"] == "kv16":
        return [dkv.PagedCache(x, table, N) for x in p]
    return [dkv.Fp8PagedCache(p[i].view(torch.float8_e4m3fn), p[i + 1], table, N) for i in (0, 2)]


# ----------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, interleaved):
    """x [n, H, r] rotated by cos / sin [n, r / 2]: pairs (i, i + r/2), or (2i, 2i + 1)."""
    h = cos.shape[-1]
    c, s_ = cos[:, None], sin[:, None]
    a, b = (x[..., ::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    u, w = a * c - b * s_, b * c + a * s_
    return torch.stack((u, w), dim=-1).flatten(-2) if interleaved else torch.cat((u, w), dim=-1)


def _plain_append(s):
    case, dt = s["case"], s["cache"].dtype
    T, page = case["T"], case["page"]
    b, t = (torch.arange(T, device="cuda") < s["new"][:, None]).nonzero(as_tuple=True)
    pos = s["lens"].long()[b] - s["new"].long()[b] + t
    cos, sin = s["cos"][pos], s["sin"][pos]
    c = s["c"][b, t].float()
    c = c * torch.rsqrt((c * c).mean(dim=-1, keepdim=True) + EPS) * s["norm"].float()
    k = _rotate(s["k"][b, t].float()[:, None], cos, sin, case["interleaved"])[:, 0]
    at = (s["table"].long()[b, pos // page], pos % page) if page else (b, pos)
    s["cache"][at] = torch.cat((c, k), dim=-1).to(dt)
    s["q_out"][b, t] = _rotate(s["q"][b, t].float(), cos, sin, case["interleaved"]).to(dt)
    return s["cache"], s["q_out"]


def _tokens(s):
    """The latent cache as [B, N', dc + r], a sequence's tokens in order."""
    if s["table"] is None:
        return s["cache"]
    return s["cache"][s["table"].long()].flatten(1, 2)


def _plain_decode(s):
    case = s["case"]
    B, T, H, dc = (case[k] for k in ("B", "T", "H", "dc"))
    x = _tokens(s).float()
    n = x.shape[1]
    q = torch.cat((s["ql"], s["qr"]), dim=-1).float().view(B, T * H, -1)
    sc = (torch.matmul(q, x.transpose(1, 2)) * s["scale"]).view(B, T, H, n)
    # new token t is the sequence's token len - new + t, and sees those up to itself
    t = torch.arange(T, device="cuda")
    seen = (s["lens"] - s["new"])[:, None] + t + 1
    sc = sc.masked_fill((torch.arange(n, device="cuda") >= seen[..., None])[:, :, None], -math.inf)
    w = torch.exp(sc - sc.amax(dim=-1, keepdim=True))
    x = x[..., :dc].masked_fill(
        (torch.arange(n, device="cuda") >= s["lens"][:, None])[..., None], 0.0)
    o = torch.matmul(w.view(B, T * H, n), x).view(B, T, H, dc) / w.sum(dim=-1, keepdim=True)
    rows = (t < s["new"][:, None])[..., None, None]
    s["out"].copy_(torch.where(rows, o, s["out"].float()))
    return s["out"]


def _plain_prompt(s):
    i = j = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        qn, qr = (s[k][i:i + nq].float().transpose(0, 1) for k in ("qn", "qr"))
        kn, v = (s[k][j:j + nk].float().transpose(0, 1) for k in ("kn", "v"))
        sc = torch.matmul(qn, kn.transpose(1, 2)) + torch.matmul(qr, s["kr"][j:j + nk].float().t())
        # the queries are the last tokens of their sequence
        last = torch.arange(nk - nq, nk, device="cuda")[:, None]
        sc = (sc * s["scale"]).masked_fill(torch.arange(nk, device="cuda") > last, -math.inf)
        w = torch.exp(sc - sc.amax(dim=-1, keepdim=True))
        o = torch.matmul(w, v) / w.sum(dim=-1, keepdim=True)
        s["out"][i:i + nq] = o.transpose(0, 1).to(s["out"].dtype)
        i, j = i + nq, j + nk
    return s["out"]


def _plain_fork(s):
    table, refs, par = s["table"], s["refs"], s["parents"].long()
    B, P = table.shape
    row, j = torch.arange(B, device="cuda"), torch.arange(P, device="cuda")
    kept = torch.where(par >= 0, s["lens"][par.clamp(min=0)].long(), 0)
    whole, pages = kept // PAGE, (kept + PAGE - 1) // PAGE
    end = (kept + s["new"].long() + PAGE - 1) // PAGE
    old = torch.where(par[:, None] >= 0, table[par.clamp(min=0)].long(), -1)
    # the last page, where it is not whole, stays with the first child that continues
    # it, unless another row holds it too; other children copy it
    first = torch.full((B + 1,), B, device="cuda").scatter_reduce(0, par.clamp(min=-1) % (B + 1),
                                                                 row, "amin")
    last = old.gather(1, whole.clamp(max=P - 1)[:, None])[:, 0]
    copied = (pages > whole) & ((first[par % (B + 1)] != row) | (refs[last.clamp(min=0)] > 1))
    fresh = ((j >= pages[:, None]) & (j < end[:, None])) | (copied[:, None] & (j == whole[:, None]))
    free = (refs == 0).nonzero()[:, 0]
    rank = fresh.view(-1).cumsum(0).view(B, P) - 1
    now = torch.where(j < pages[:, None], old, -1)
    now = torch.where(fresh, free[rank.clamp(0, len(free) - 1)], now)
    src, dst = last[copied], now.gather(1, whole.clamp(max=P - 1)[:, None])[:, 0][copied]
    for p in s["pools"]:
        p[dst] = p[src]
    count = lambda t: torch.bincount(t[t >= 0].long(), minlength=len(refs)).to(torch.int32)
    refs += count(now) - count(table)
    table.copy_(now)
    return table, refs, *_values(s)


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    live = refs > 0
    n = int(live.sum())
    src, dst = live[n:].nonzero()[:, 0] + n, (~live[:n]).nonzero()[:, 0]
    for p in s["pools"]:
        p[dst] = p[src]
    to = torch.arange(len(refs), device="cuda", dtype=torch.int32)
    to[src] = dst.to(torch.int32)
    to[~live] = -1
    s["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][n:] = 0
    return s["table_out"], s["refs_out"], to, *_values(s)


def _values(s):
    return [p.view(torch.float8_e4m3fn) if p.dtype == torch.uint8 else p for p in s["pools"]]


def _own(s):
    case, dkv = s["case"], s["dkv"]
    if case["op"] == "append":
        dkv.latent_append(s["c"], s["k"], s["handle"], seq_lens=s["lens"],
                          new_lens=s["new_or_none"], q_rope=s["q"], q_out=s["q_out"],
                          rope=(s["cos"], s["sin"]), norm=s["norm"], eps=EPS,
                          interleaved=case["interleaved"])
        return s["cache"], s["q_out"]
    if case["op"] == "decode":
        return dkv.latent_decode_attn(s["ql"], s["qr"], s["handle"], s["scale"],
                                      seq_lens=s["lens_or_none"], new_lens=s["new_or_none"],
                                      out=s["out"], workspace=s["workspace"])
    if case["op"] == "prompt":
        return dkv.latent_prompt_attn(s["qn"], s["qr"], s["kn"], s["kr"], s["v"], s["cu_q"],
                                      s["cu_k"], s["scale"], out=s["out"])
    if case["op"] == "fork":
        dkv.kv_pages_fork(s["handles"], s["refs"], s["lens"], parents=s["parents"],
                          new_lens=s["new"], workspace=s["workspace"])
        return s["table"], s["refs"], *_values(s)
    to = dkv.kv_pages_compact(s["handles"], s["refs"], refs_out=s["refs_out"],
                              block_table_out=s["table_out"], workspace=s["workspace"])
    return s["table_out"], s["refs_out"], to, *_values(s)


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt,
            "fork": _plain_fork, "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work, exact
def _block_bytes(case):
    if case["cache"] == "latent":
        return PAGE * (512 + ROPE) * 2
    return 2 * case["Hkv"] * (PAGE * case["d"] * 2 if case["cache"] == "kv16"
                              else PAGE * case["d"] + 4)


def work(case):
    op, B = case["op"], case["B"]
    # ragged lengths are spread over [N / 4, N], ragged new tokens over [0, T]
    part = 0.625 if case.get("ragged") else 1.0
    if op in ("append", "decode"):
        T, H, dc = case["T"], case["H"], case["dc"]
        tokens = B * T * (0.5 if case["ragged"] and T > 1 else 1.0)
        if op == "append":
            return {"bytes": tokens * (4 * (dc + ROPE) + 4 * H * ROPE + 4 * ROPE),
                    "flops": tokens * (4 * dc + 3 * ROPE * (H + 1))}
        n = case["N"] * part
        return {"bytes": B * n * (dc + ROPE) * 2 + tokens * H * (2 * dc + ROPE) * 2,
                "flops": 2 * tokens * H * n * (2 * dc + ROPE)}
    if op == "prompt":
        H, dn, nq, nk = (case[k] for k in ("H", "dn", "nq", "nk"))
        q, k = B * nq * part, B * nk * part
        seen = B * (nq * nk - nq * nq / 2) * (0.42 if case["ragged"] else 1.0)
        return {"bytes": 2 * (q * H * (2 * dn + ROPE) + k * (2 * H * dn + ROPE)),
                "flops": 2 * H * seen * (2 * dn + ROPE)}
    P = -(-case["N"] // PAGE)
    if op == "fork":
        # the table read and written, and about a page copied every other row
        return {"bytes": 8 * B * (P + 1) + 4 * case["blocks"] + B * _block_bytes(case),
                "flops": 4 * B * P}
    moves = case["blocks"] * case["live"] * (1 - case["live"])
    return {"bytes": 2 * moves * _block_bytes(case) + 8 * B * P + 12 * case["blocks"],
            "flops": 4 * case["blocks"]}


def _exact_append(s):
    case = s["case"]
    page, dc = case["page"], case["dc"]
    cache, q_out = s["cache"].double(), s["q_out"].double()
    a, b = ((slice(0, ROPE, 2), slice(1, ROPE, 2)) if case["interleaved"]
            else (slice(0, ROPE // 2), slice(ROPE // 2, ROPE)))
    for i, (m, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        if n == 0:
            continue
        cos, sin = s["cos"][m - n:m].double(), s["sin"][m - n:m].double()

        def turned(x, cos, sin):
            x = x.double()
            y = torch.empty_like(x)
            y[..., a] = x[..., a] * cos - x[..., b] * sin
            y[..., b] = x[..., a] * sin + x[..., b] * cos
            return y

        c = s["c"][i, :n].double()
        c = s["norm"].double() * c / (c.square().sum(dim=-1, keepdim=True) / dc + EPS).sqrt()
        y = torch.cat((c, turned(s["k"][i, :n], cos, sin)), dim=-1)
        if page:
            blocks = s["table"][i].long().repeat_interleave(page)[m - n:m]
            cache[blocks, torch.arange(m - n, m, device="cuda") % page] = y
        else:
            cache[i, m - n:m] = y
        q_out[i, :n] = turned(s["q"][i, :n], cos[:, None], sin[:, None])
    return cache, q_out


def _exact_decode(s):
    case = s["case"]
    out = s["out"].double()
    for i, (m, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        x = (s["cache"][i] if s["table"] is None
             else s["cache"][s["table"][i].long()].flatten(0, 1))[:m].double()
        for t in range(n):
            y = x[:m - n + t + 1]
            lat, rot = y[:, :case["dc"]], y[:, case["dc"]:]
            sc = s["ql"][i, t].double() @ lat.t() + s["qr"][i, t].double() @ rot.t()
            out[i, t] = torch.softmax(sc * s["scale"], dim=-1) @ lat
    return out


def _exact_prompt(s):
    out = s["out"].double()
    i = j = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        rot = s["kr"][j:j + nk].double()
        hide = torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for h in range(s["case"]["H"]):
            sc = torch.einsum("qc,kc->qk", s["qn"][i:i + nq, h].double(),
                              s["kn"][j:j + nk, h].double())
            sc += torch.einsum("qc,kc->qk", s["qr"][i:i + nq, h].double(), rot)
            sc = (sc * s["scale"]).masked_fill(hide, -math.inf)
            out[i:i + nq, h] = torch.softmax(sc, dim=-1) @ s["v"][j:j + nk, h].double()
        i, j = i + nq, j + nk
    return out


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode,
            "prompt": _exact_prompt}[case["op"]](s)
