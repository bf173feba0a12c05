"""Decode attention, page selection and page metadata over 8-bit caches, against
64-bit forms on the same codes and scales."""

import math

import numpy as np
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


def make(B, Hq, Hkv, d, N, dt, seed, scales="pow2", spread=False):
    """q, (codes, scale) of K and V on the CPU."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, d, generator=g).to(dt)
    kv = []
    for i in range(2):
        x = torch.randn(B, Hkv, N, d, generator=g)
        if spread and i == 1:  # V blocks of very different sizes
            P = -(-N // PAGE)
            e = torch.randint(-12, 8, (B, Hkv, P, 1), generator=g).float()
            x *= torch.exp2(e).repeat_interleave(PAGE, dim=2)[:, :, :N]
        c, s = ref.quantise(x, dt)
        if scales == "any":
            s = s * (0.6 + torch.rand(s.shape, generator=g))
        if scales == "some zero":
            s[torch.rand(s.shape, generator=g) < 0.4] = 0.0
        kv.append((c, s))
    return q, kv[0], kv[1]


def caches(dkv, dev, K, V, dt, paged, lens=None):
    if not paged:
        return [dkv.Fp8Cache(c.to(dev), s.to(dev), dt) for c, s in (K, V)]
    out, bt = [], None
    for c, s in (K, V):
        pool, ps, table = ref.to_pool(c, s, lens=lens)
        bt = table.to(dev) if bt is None else bt
        out.append(dkv.Fp8PagedCache(pool.to(dev), ps.to(dev), bt, c.shape[2], dt))
    return out


SHAPES = [  # B, Hq, Hkv, d, N, dtype, lens
    (1, 1, 1, 64, 1, torch.bfloat16, None),
    (2, 8, 1, 128, 16, torch.bfloat16, None),
    (2, 6, 2, 128, 17, torch.float16, [17, 1]),
    (3, 10, 2, 64, 33, torch.bfloat16, [33, 16, 5]),
    (1, 7, 1, 64, 259, torch.float16, None),
    (2, 8, 8, 64, 1000, torch.bfloat16, [1000, 77]),
    (3, 8, 2, 128, 1043, torch.bfloat16, [1043, 1024, 1]),
    (1, 4, 2, 128, 4099, torch.float16, None),
    (40, 4, 2, 64, 4000, torch.bfloat16, None),  # 125-page chunks, several a sequence
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("paged", [False, True])
def test_full(shape, paged, dev, dkv):
    B, Hq, Hkv, d, N, dt, lens = shape
    q, K, V = make(B, Hq, Hkv, d, N, dt, seed=N + d)
    if lens is not None and not paged:  # slots past a sequence's end: NaN codes and scales
        for c, s in (K, V):
            for b, n in enumerate(lens):
                c.view(torch.uint8)[b, :, n:] = 0xFF
                s[b, :, -(-n // PAGE):] = math.nan
    Kd, Vd = caches(dkv, dev, K, V, dt, paged, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    scale = 1.0 / math.sqrt(d)
    out = dkv.decode_attn_full(q.to(dev), Kd, Vd, seq_lens=lt)
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, scale, lens)
    err = (out.cpu().double() - want).abs().max()
    assert err <= ref.tolerance(q, kv, vv, scale)


@pytest.mark.parametrize("scales", ["any", "some zero", "spread"])
@pytest.mark.parametrize("d,dt", [(64, torch.float16), (128, torch.bfloat16)])
def test_scales(scales, d, dt, dev, dkv):
    # scales that are no powers of two, zero, or 2^20 apart from block to block
    q, K, V = make(2, 8, 2, d, 700, dt, seed=9, scales=scales, spread=scales == "spread")
    Kd, Vd = caches(dkv, dev, K, V, dt, True)
    out = dkv.decode_attn_full(q.to(dev), Kd, Vd)
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, 1 / math.sqrt(d))
    assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, 1 / math.sqrt(d))


def test_large_values_of_little_weight(dev, dkv):
    # one block's values are 2^40 times the others' but its weight is e^-60: the
    # others keep their precision
    d, N = 64, 64
    q = torch.zeros(1, 1, d)
    q[..., 0] = 60.0 * 8
    k = torch.zeros(1, 1, N, d)
    k[:, :, 16:, 0] = 1.0
    v = torch.randn(1, 1, N, d, generator=torch.Generator().manual_seed(1))
    v[:, :, :16] *= 2.0 ** 40
    K, V = ref.quantise(k, torch.bfloat16), ref.quantise(v, torch.bfloat16)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, False)
    out = dkv.decode_attn_full(q.to(torch.bfloat16).to(dev), Kd, Vd, scale=1 / 8)
    want = ref.attention(q, ref.values(*K), ref.values(*V), 1 / 8)
    rest = ref.values(*V)[:, :, 16:].abs().max()
    # scores are 60 and 0, exact; weights as in tolerance(), on values of 48 tokens
    assert (out.cpu().double() - want).abs().max() <= float(rest) * (2.0 ** -15 + 2.0 ** -20)


@pytest.mark.parametrize("scale_q", [2.0 ** -130, 2.0 ** 60, 0.0])
def test_query_range(scale_q, dev, dkv):
    # bf16 queries far from 1, with a component 2^-20 of the largest
    q, K, V = make(1, 4, 1, 128, 200, torch.bfloat16, seed=4)
    q[..., 3] = 2.0 ** -18
    q = (q.double() * scale_q).to(torch.bfloat16)
    if scale_q == 2.0 ** -130:
        assert (q != 0).any()  # subnormal
    s = (1 / math.sqrt(128)) / (scale_q if scale_q else 1.0)
    s = float(min(max(s, 2.0 ** -100), 2.0 ** 100))
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, False)
    out = dkv.decode_attn_full(q.to(dev), Kd, Vd, scale=s)
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, s)
    assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, s)


@pytest.mark.parametrize("od", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N", [40, 5000])
def test_empty_sequences_and_out_types(od, N, dev, dkv):
    # length 0 (and below): a zero row, nothing of it read (its table is rubbish);
    # one work item a unit (N = 40) and several
    q, K, V = make(4, 4, 2, 64, N, torch.bfloat16, seed=2)
    lens = [0, N, -3, 7]
    for paged in (False, True):
        Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, paged, lens)
        if paged:
            Kd.block_table[0], Kd.block_table[2] = -1, 1 << 30
        lt = torch.tensor(lens, dtype=torch.int32, device=dev)
        ws = torch.zeros(dkv.workspace_bytes(4, 4, 2, 64, N, fp8=True), dtype=torch.uint8,
                         device=dev)
        out = torch.full((4, 4, 64), float("nan"), dtype=od, device=dev)
        dkv.decode_attn_full(q.to(dev), Kd, Vd, out=out, seq_lens=lt, workspace=ws)
        assert dkv.read_device_status(ws) == 0
        kv, vv = ref.values(*K), ref.values(*V)
        want = ref.attention(q, kv, vv, 1 / 8, lens)
        tol = ref.tolerance(q, kv, vv, 1 / 8)
        half = 0.0 if od == torch.float32 else torch.finfo(od).eps / 2
        assert not out[0].any() and not out[2].any()
        err = (out.cpu().double() - want).abs()
        assert torch.all(err <= tol + half * (want.abs() + tol))


def test_paged_head_wise_and_strided_bitwise(dev, dkv):
    B, Hq, H, d, N = 3, 8, 4, 128, 2300
    q, K, V = make(B, Hq, H, d, N, torch.bfloat16, seed=6)
    lens = [2300, 16, 1500]
    lt = torch.tensor(lens, dtype=torch.int32, device=dev)
    qd = q.to(dev)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, False)
    out = dkv.decode_attn_full(qd, Kd, Vd, seq_lens=lt)
    Kp, Vp = caches(dkv, dev, K, V, torch.bfloat16, True, lens)
    assert torch.equal(out, dkv.decode_attn_full(qd, Kp, Vp, seq_lens=lt))
    assert torch.equal(out, dkv.decode_attn_full(qd, Kd, Vd, seq_lens=lt))
    # one kv head at a time
    cut = lambda c, h: dkv.Fp8Cache(c.codes[:, h:h + 1], c.scale[:, h:h + 1], c.dtype)
    for h in range(H):
        o = dkv.decode_attn_full(qd[:, 2 * h:2 * h + 2], cut(Kd, h), cut(Vd, h), seq_lens=lt)
        assert torch.equal(o, out[:, 2 * h:2 * h + 2])
    # heads before batch, a longer buffer, q out of a fused row, out with gaps
    def wide(c):
        codes = torch.zeros(H, B, N + 50, d, dtype=torch.uint8, device=dev)
        codes[:, :, :N] = c.codes.view(torch.uint8).transpose(0, 1)
        sc = torch.full((H, B, c.scale.shape[2] + 3), float("nan"), device=dev)
        sc[:, :, :-3] = c.scale.transpose(0, 1)
        return dkv.Fp8Cache(codes.view(torch.float8_e4m3fn).transpose(0, 1)[:, :, :N],
                            sc.transpose(0, 1)[:, :, :-3], c.dtype)
    fused = torch.zeros(B, Hq + 5, d + 8, dtype=torch.bfloat16, device=dev)
    fused[:, 3:3 + Hq, :d] = qd
    o = torch.full((B, Hq + 1, 2 * d), 5.0, device=dev)
    dkv.decode_attn_full(fused[:, 3:3 + Hq, :d], wide(Kd), wide(Vd), out=o[:, :Hq, :d],
                         seq_lens=lt)
    assert torch.equal(o[:, :Hq, :d], out)
    assert torch.all(o[:, Hq] == 5.0) and torch.all(o[:, :, d:] == 5.0)


@pytest.mark.parametrize("Hq", [3, 9, 18])
@pytest.mark.parametrize("ragged", [False, True])
def test_many_items_a_cta(Hq, ragged, dev, dkv):
    # more work items than resident CTAs, every second one of five pages or fewer
    # (warps without a page run ahead of the others), run twice on one workspace
    B, H, d, N = 120, 3, 128, 1104
    q, K, V = make(B, Hq, H, d, N, torch.bfloat16, seed=Hq)
    lens = None
    if ragged:
        lens = torch.randint(1025, N + 1, (B,), generator=torch.Generator().manual_seed(1)).tolist()
        lens[::9] = [17] * len(lens[::9])
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    kv, vv = ref.values(*K), ref.values(*V)
    scale = 1 / math.sqrt(d)
    want = ref.attention(q, kv, vv, scale, lens)
    ws = torch.zeros(dkv.workspace_bytes(B, Hq, H, d, N, fp8=True), dtype=torch.uint8, device=dev)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, True)
    for _ in range(2):
        out = dkv.decode_attn_full(q.to(dev), Kd, Vd, seq_lens=lt, workspace=ws)
        assert dkv.read_device_status(ws) == 0
        assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, scale)


def test_more_sequences_than_are_counted(dev, dkv):
    # past 128 sequences items are not counted by length; some of them empty
    B, Hq, H, d, N = 131, 4, 2, 64, 600
    q, K, V = make(B, Hq, H, d, N, torch.bfloat16, seed=5)
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, N + 1, (B,), generator=g)
    lens[7], lens[130] = 0, N
    lt = lens.to(torch.int32).to(dev)
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, 1 / 8, lens.tolist())
    for paged in (False, True):
        Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, paged)
        out = dkv.decode_attn_full(q.to(dev), Kd, Vd, seq_lens=lt)
        assert not out[7].any()
        assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, 1 / 8)


def test_blocks_past_two_gib(dev, dkv):
    # the tokens lie in the last blocks of pools whose offsets pass 2^31
    H, d, N = 8, 128, 70
    nb = (1 << 31) // (H * 16 * d) + 9
    q, K, V = make(1, 16, H, d, N, torch.bfloat16, seed=3)
    bt = torch.arange(nb - 5, nb, dtype=torch.int32).view(1, 5)
    out = []
    for c, s in (K, V):
        pool = torch.zeros(nb, H, 16, d, dtype=torch.uint8, device=dev)
        scale = torch.zeros(nb, H, device=dev)
        full = torch.zeros(H, 80, d, dtype=torch.uint8)
        full[:, :N] = c[0].view(torch.uint8)
        pool[nb - 5:] = full.view(H, 5, 16, d).transpose(0, 1).to(dev)
        scale[nb - 5:] = s[0].t().to(dev)
        out.append((pool, scale))
    table = bt.to(dev)
    Kd, Vd = (dkv.Fp8PagedCache(p.view(torch.float8_e4m3fn), s, table, N) for p, s in out)
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, 1 / math.sqrt(d))
    tol = ref.tolerance(q, kv, vv, 1 / math.sqrt(d))
    assert (dkv.decode_attn_full(q.to(dev), Kd, Vd).cpu().double() - want).abs().max() <= tol
    meta = dkv.kv_meta_build(Kd)
    o = dkv.decode_attn_select(q.to(dev), Kd, Vd, meta, 5)
    assert (o.cpu().double() - want).abs().max() <= tol


def deq16(c, s, dt):
    """An 8-bit cache's values in its 16-bit type (exact for powers of two)."""
    x = ref.values(c, s)
    y = x.to(dt)
    assert torch.equal(y.double(), x)
    return y


@pytest.mark.parametrize("S", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("d,dt", [(64, torch.float16), (128, torch.bfloat16)])
def test_meta(S, d, dt, dev, dkv):
    B, H, N = 2, 3, 301
    _, K, V = make(B, H, H, d, N, dt, seed=S)
    for lens in (None, [301, 90]):
        want = oracle.meta(bits(deq16(*K, dt)), S, 0 if dt == torch.bfloat16 else 1)
        want = [torch.from_numpy(w.view(np.int16)).view(dt) for w in want]
        lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
        for paged in (False, True):
            Kd, _ = caches(dkv, dev, K, V, dt, paged, lens)
            mn, mx = dkv.kv_meta_build(Kd, page_size=S, seq_lens=lt)
            assert mn.dtype == dt
            # the newest page alone, of metadata that is stale there
            again = [m.clone() for m in (mn, mx)]
            for b in range(B):
                n = N if lens is None else lens[b]
                for m in again:
                    m[b, :, (n - 1) // S] = 9.0
            dkv.kv_meta_append(Kd, again, page_size=S, seq_lens=lt)
            for b in range(B):
                n = N if lens is None else lens[b]
                whole, last = n // S, (n - 1) // S
                x = deq16(*K, dt)[b, :, last * S:n]
                for m, w, e, a in ((mn, want[0], x.amin(1), again[0]),
                                   (mx, want[1], x.amax(1), again[1])):
                    assert torch.equal(m[b, :, :whole].cpu(), w[b, :, :whole])
                    assert torch.equal(m[b, :, last].cpu(), e)
                    assert torch.equal(a[b, :, :last + 1], m[b, :, :last + 1])


def test_meta_outward_and_empty(dev, dkv):
    # scales that are no powers of two: never inside the values, one step off at most
    for dt in (torch.bfloat16, torch.float16):
        _, K, V = make(2, 2, 2, 64, 200, dt, seed=8, scales="any")
        Kd, _ = caches(dkv, dev, K, V, dt, True)
        mn, mx = (m.cpu().double() for m in dkv.kv_meta_build(Kd))
        x = ref.values(*K)
        for j in range(13):
            y = x[:, :, 16 * j:16 * j + 16]
            lo, hi = y.amin(2), y.amax(2)
            step = torch.finfo(dt).eps
            assert torch.all(mn[:, :, j] <= lo) and torch.all(mx[:, :, j] >= hi)
            assert torch.all(lo - mn[:, :, j] <= step * lo.abs() + 2.0 ** -24)
            assert torch.all(mx[:, :, j] - hi <= step * hi.abs() + 2.0 ** -24)
    # an empty sequence's metadata is not written
    lt = torch.tensor([0, 200], dtype=torch.int32, device=dev)
    mn = torch.full((2, 2, 13, 64), 7.0, dtype=torch.float16, device=dev)
    mx = mn.clone()
    dkv.kv_meta_append(Kd, (mn, mx), seq_lens=lt)
    assert torch.all(mn[0] == 7.0) and torch.all(mx[0] == 7.0)
    assert torch.all(mn[1, :, :12] == 7.0) and not torch.any(mn[1, :, 12] == 7.0)


SELECT = [  # B, Hq, Hkv, d, N, dtype, S, top_k, lens, group
    (2, 8, 2, 128, 333, torch.bfloat16, 16, 5, [333, 40], False),
    (1, 4, 4, 64, 1000, torch.float16, 16, 9, None, False),
    (2, 16, 4, 128, 5000, torch.bfloat16, 16, 20, None, True),     # per-unit selection
    (2, 8, 8, 64, 5001, torch.float16, 16, 300, [5001, 4200], False),
    (1, 8, 1, 64, 2000, torch.bfloat16, 4, 60, None, False),
    (1, 8, 2, 128, 2000, torch.float16, 8, 33, None, False),
    (1, 6, 2, 64, 20000, torch.bfloat16, 32, 17, None, False),
    (1, 8, 2, 128, 3000, torch.bfloat16, 64, 6, [2911], False),
    (1, 8, 4, 128, 40000, torch.bfloat16, 16, 64, None, False),    # past 2048 pages
    (3, 4, 2, 64, 50, torch.bfloat16, 16, 9, [50, 1, 17], False),  # every page kept
]


@pytest.mark.parametrize("case", SELECT, ids=str)
@pytest.mark.parametrize("paged", [False, True])
def test_select(case, paged, dev, dkv):
    B, Hq, Hkv, d, N, dt, S, top_k, lens, group = case
    q, K, V = make(B, Hq, Hkv, d, N, dt, seed=N)
    Kd, Vd = caches(dkv, dev, K, V, dt, paged, lens)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    meta = dkv.kv_meta_build(Kd, page_size=S, seq_lens=lt)
    out, sel = dkv.decode_attn_select(q.to(dev), Kd, Vd, meta, top_k, return_selected=True,
                                      group_select=group, seq_lens=lt, page_size=S)
    sel = sel.cpu()
    kv, vv = ref.values(*K), ref.values(*V)
    code = 0 if dt == torch.bfloat16 else 1
    for b in range(B):
        n = N if lens is None else lens[b]
        Pb = -(-n // S)
        mn, mx = (m[b:b + 1, :, :Pb].contiguous().cpu() for m in meta)
        r = oracle.scores(bits(q[b:b + 1]), bits(mn), bits(mx), code)[0]
        if group:
            r = np.repeat(r.reshape(Hkv, Hq // Hkv, Pb).sum(1), Hq // Hkv, axis=0)
        kk = min(top_k, Pb)
        check_selection(sel[b, :, :kk].numpy(), r, top_k)
        assert torch.all(sel[b, :, kk:] == -1)
    want = ref.attention(q, kv, vv, 1 / math.sqrt(d), lens, pages=sel.tolist(), S=S)
    err = (out.cpu().double() - want).abs().max()
    assert err <= ref.tolerance(q, kv, vv, 1 / math.sqrt(d))


def test_select_empty_sequence(dev, dkv):
    for N, top_k in ((48, 2), (5000, 12)):
        q, K, V = make(3, 4, 2, 64, N, torch.bfloat16, seed=1)
        lens = [N, 0, 20]
        Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, True, lens)
        lt = torch.tensor(lens, dtype=torch.int32, device=dev)
        meta = [torch.zeros(3, 2, -(-N // 16), 64, dtype=torch.bfloat16, device=dev)
                for _ in range(2)]
        for m, w in zip(meta, dkv.kv_meta_build(Kd, seq_lens=lt)):
            m.copy_(w)
            m[1] = float("nan")
        Kd.block_table[1] = -1
        ws = torch.zeros(dkv.workspace_bytes(3, 4, 2, 64, N, top_k, fp8=True), dtype=torch.uint8,
                         device=dev)
        out, sel = dkv.decode_attn_select(q.to(dev), Kd, Vd, meta, top_k, return_selected=True,
                                          seq_lens=lt, workspace=ws)
        assert dkv.read_device_status(ws) == 0
        assert not out[1].any()
        kv, vv = ref.values(*K), ref.values(*V)
        want = ref.attention(q, kv, vv, 1 / 8, lens, pages=sel.tolist())
        assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, 1 / 8)


def test_select_meta8(dev, dkv):
    q, K, V = make(2, 8, 2, 128, 6000, torch.bfloat16, seed=3)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, True)
    meta = dkv.kv_meta8_build(dkv.kv_meta_build(Kd))
    out, sel = dkv.decode_attn_select(q.to(dev), Kd, Vd, meta, 30, return_selected=True)
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, 1 / math.sqrt(128), pages=sel.tolist())
    assert (out.cpu().double() - want).abs().max() <= ref.tolerance(q, kv, vv, 1 / math.sqrt(128))


def test_bad_block_is_clamped_and_reported(dev, dkv):
    q, K, V = make(2, 4, 2, 64, 100, torch.bfloat16, seed=1)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, True)
    Kd.scale.nan_to_num_(0.0), Vd.scale.nan_to_num_(0.0)
    Kd.block_table[1, 3] = 1 << 20
    ws = torch.zeros(dkv.workspace_bytes(2, 4, 2, 64, 100, fp8=True), dtype=torch.uint8, device=dev)
    out = dkv.decode_attn_full(q.to(dev), Kd, Vd, workspace=ws)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_CHECK
    want = ref.attention(q, ref.values(*K), ref.values(*V), 1 / 8)
    assert (out[0].cpu().double() - want[0]).abs().max() <= ref.tolerance(
        q, ref.values(*K), ref.values(*V), 1 / 8)


def test_forced_timeout_returns(dev, dkv):
    q, K, V = make(2, 4, 2, 128, 3000, torch.bfloat16, seed=1)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, False)
    ws = torch.zeros(dkv.workspace_bytes(2, 4, 2, 128, 3000, fp8=True), dtype=torch.uint8,
                     device=dev)
    dkv.decode_attn_full(q.to(dev), Kd, Vd, workspace=ws, flags=dkv.DKV_FLAG_FORCE_TIMEOUT)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_TIMEOUT
    out = dkv.decode_attn_full(q.to(dev), Kd, Vd, workspace=ws)
    assert dkv.read_device_status(ws) == 0
    want = ref.attention(q, ref.values(*K), ref.values(*V), 1 / math.sqrt(128))
    assert (out.cpu().double() - want).abs().max() <= ref.tolerance(
        q, ref.values(*K), ref.values(*V), 1 / math.sqrt(128))


@pytest.mark.parametrize("sparse", [0, 1])
def test_resident_ctas(sparse, dev, dkv):
    import ctypes
    n = ctypes.c_int32(0)
    for d in (64, 128):
        for dt in (dkv.DKV_BF16, dkv.DKV_FP16):
            assert dkv.lib().dkv_attn_ctas_per_sm(d, dt, dkv.DKV_KV_FP8, sparse,
                                                  ctypes.byref(n)) == 0
            assert n.value == (4 if d == 64 else 3)


def test_python_refusals(dev, dkv):
    q, K, V = make(1, 2, 1, 64, 40, torch.bfloat16, seed=1)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, False)
    qd = q.to(dev)
    with pytest.raises(ValueError):
        dkv.decode_attn_full(qd.half(), Kd, Vd)
    with pytest.raises(dkv.DkvError):
        dkv.decode_attn_full(qd, Kd, dkv.Fp8Cache(Vd.codes, Vd.scale, torch.float16))
    with pytest.raises(ValueError):
        dkv.decode_attn_full(qd, Kd, dkv.Fp8Cache(Vd.codes[:, :, :39], Vd.scale))
    with pytest.raises(ValueError):  # a 16-bit cache's workspace size may be too small
        dkv.decode_attn_full(qd, Kd, Vd, workspace=torch.zeros(64, dtype=torch.uint8, device=dev))
    meta = [m.half() for m in dkv.kv_meta_build(Kd)]
    with pytest.raises(ValueError):
        dkv.decode_attn_select(qd, Kd, Vd, meta, 1)
    with pytest.raises(ValueError):
        dkv.kv_meta_append(Kd, meta)
    with pytest.raises(dkv.DkvError):
        dkv.decode_attn_topk_tokens(qd, Kd, Vd, 4)
    # tensors of another device, of another shape or stride
    cpu = dkv.Fp8Cache(K[0], K[1])
    k16, v16 = (deq16(*c, torch.bfloat16).to(dev) for c in (K, V))
    for call in (lambda: dkv.decode_attn_full(qd, cpu, Vd), lambda: dkv.decode_attn_full(q, Kd, Vd),
                 lambda: dkv.decode_attn_full(qd, k16, v16.cpu()),
                 lambda: dkv.decode_attn_full(qd, k16, v16, out=torch.zeros(1, 2, 64)),
                 lambda: dkv.decode_attn_full(qd, k16, v16, workspace=torch.zeros(1 << 20)),
                 lambda: dkv.decode_attn_full(qd, Kd, Vd, out=torch.zeros(1, 1, 64, device=dev)),
                 lambda: dkv.decode_attn_full(
                     qd, Kd, Vd, out=torch.zeros(1, 64, 2, device=dev).transpose(1, 2)),
                 lambda: dkv.decode_attn_full(qd, Kd, Vd, seq_lens=torch.ones(1, dtype=torch.int32)),
                 lambda: dkv.decode_attn_select(
                     qd, Kd, Vd, dkv.kv_meta_build(Kd), 2,
                     selected=torch.zeros(1, 2, 1, dtype=torch.int32, device=dev))):
        with pytest.raises(ValueError):
            call()


def test_two_calls_at_once(dev, dkv):
    # two streams, a workspace each, caches and metadata shared
    q, K, V = make(4, 8, 2, 128, 9000, torch.bfloat16, seed=4)
    Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, True)
    meta = dkv.kv_meta_build(Kd)
    qs = [q.to(dev), q.flip(1).contiguous().to(dev)]
    want = [(dkv.decode_attn_full(x, Kd, Vd), dkv.decode_attn_select(x, Kd, Vd, meta, 20))
            for x in qs]
    n = max(dkv.workspace_bytes(4, 8, 2, 128, 9000, k, fp8=True) for k in (0, 20))
    ws = [torch.zeros(n, dtype=torch.uint8, device=dev) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((dkv.decode_attn_full(qs[i], Kd, Vd, workspace=ws[i]),
                               dkv.decode_attn_select(qs[i], Kd, Vd, meta, 20, workspace=ws[i])))
    torch.cuda.synchronize()
    for i in range(2):
        assert dkv.read_device_status(ws[i]) == 0
        for full, sparse in got[i]:
            assert torch.equal(full, want[i][0]) and torch.equal(sparse, want[i][1])


def test_arguments_that_16_bit_calls_take(dev, dkv):
    # outputs and selections with room to spare, metadata as one tensor, counts
    # that int() takes
    g = torch.Generator().manual_seed(6)
    q = torch.randn(2, 4, 64, generator=g).to(torch.bfloat16).to(dev)
    K, V = (torch.randn(2, 2, 100, 64, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    mn, mx = dkv.kv_meta_build(K)
    want = dkv.decode_attn_select(q, K, V, (mn, mx), 3, return_selected=True)
    got = dkv.decode_attn_select(q, K, V, torch.stack((mn, mx)), np.float64(3.0),
                                 return_selected=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for f in (lambda **o: dkv.decode_attn_topk_tokens(q, K, V, 5, **o),
              lambda **o: dkv.decode_attn_full(q, K, V, **o)):
        out = torch.full((3, 5, 80), 9.0, device=dev)
        assert f(out=out) is out
        assert torch.equal(out[:2, :4, :64], f())
        out[:2, :4, :64] = 9.0
        assert (out == 9.0).all()
        for bad in (out[:1], out[:, :3], out[:, :, :32], out[0]):
            with pytest.raises(ValueError, match="out must hold"):
                f(out=bad)


def test_decode_loop(dev, dkv):
    """A prompt, then steps of append, newest-page metadata, exact and sparse
    attention, captured in two graphs that share a workspace: against 64-bit
    attention over the tokens that the plain form appended."""
    B, Hq, H, d, N, dt = 2, 8, 2, 128, 96, torch.bfloat16
    P = N // 16
    g = torch.Generator().manual_seed(3)
    prompt = torch.tensor([37, 16], dtype=torch.int32)
    rope = dkv.rope_table(N, d)
    grope = tuple(t.to(dev) for t in rope)
    refs = [(torch.zeros(B, H, N, d, dtype=torch.uint8), torch.zeros(B, H, P), dt)
            for _ in range(2)]
    bt = torch.randperm(B * P, generator=g).view(B, P).to(torch.int32).to(dev)
    Kd, Vd = (dkv.Fp8PagedCache(
        torch.full((B * P, H, 16, d), 0x7F, dtype=torch.uint8, device=dev)
        .view(torch.float8_e4m3fn), torch.full((B * P, H), float("nan"), device=dev), bt, N, dt)
        for _ in range(2))
    x = torch.randn(B, 37, Hq + 2 * H, d, generator=g).to(dt)
    lens = prompt.to(dev)
    xd = x.to(dev)
    cut = lambda t: (t[:, :, Hq:Hq + H], t[:, :, Hq + H:])
    dkv.kv_append(*cut(xd), Kd, Vd, seq_lens=lens, new_lens=lens.clone(), rope=grope)
    ref.append(*cut(x), *refs, prompt, prompt, rope=rope)
    meta = dkv.kv_meta_build(Kd, seq_lens=lens)

    need = max(dkv.workspace_bytes(B, Hq, H, d, N, k, fp8=True) for k in (0, 3))
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    row = torch.zeros(B, 1, Hq + 2 * H, d, dtype=dt, device=dev)
    full, sparse = (torch.zeros(B, Hq, d, device=dev) for _ in range(2))
    sel = torch.zeros(B, Hq, 3, dtype=torch.int32, device=dev)
    q_out = torch.zeros(B, 1, Hq, d, dtype=dt, device=dev)

    def first():
        lens.add_(1)
        dkv.kv_append(*cut(row), Kd, Vd, seq_lens=lens, q=row[:, :, :Hq], q_out=q_out, rope=grope,
                      workspace=ws)
        dkv.kv_meta_append(Kd, meta, seq_lens=lens)
        dkv.decode_attn_full(q_out[:, 0], Kd, Vd, out=full, seq_lens=lens, workspace=ws)

    def second():
        dkv.decode_attn_select(q_out[:, 0], Kd, Vd, meta, 3, out=sparse, return_selected=True,
                               selected=sel, seq_lens=lens, workspace=ws)

    steps = torch.randn(24, B, 1, Hq + 2 * H, d, generator=g).to(dt)
    graphs = []
    side = torch.cuda.Stream()
    for i in range(24):
        row.copy_(steps[i])
        if i == 0:
            first()
            second()
            torch.cuda.synchronize()
            for f in (first, second):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    f()
                graphs.append(graph)
        else:
            for graph in graphs:
                graph.replay()
        now = prompt + i + 1
        q_ref = torch.zeros(B, 1, Hq, d, dtype=dt)
        ref.append(*cut(steps[i]), *refs, now, [1, 1], steps[i][:, :, :Hq], q_ref, rope)
        kv, vv = (ref.values(c.view(torch.float8_e4m3fn), s) for c, s, _ in refs)
        q = q_ref[:, 0]
        assert torch.equal(q_out.cpu(), q_ref)
        n = now.tolist()
        tol = ref.tolerance(q, kv, vv, 1 / math.sqrt(d))
        want = ref.attention(q, kv, vv, 1 / math.sqrt(d), n)
        assert (full.cpu().double() - want).abs().max() <= tol
        want = ref.attention(q, kv, vv, 1 / math.sqrt(d), n, pages=sel.tolist())
        assert (sparse.cpu().double() - want).abs().max() <= tol
    assert dkv.read_device_status(ws) == 0
