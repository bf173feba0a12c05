"""Decode attention over 8-bit caches at the edges of its domain, against 64-bit
forms."""

import ctypes
import math

import pytest
import torch

import fp8_helpers as ref
from gpu_helpers import require_cuda
from test_gpu_fp8 import caches, make

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(scope="module")
def dev():
    return require_cuda()


@pytest.fixture(scope="module")
def dkv():
    import decode_attention_paged_kv_gb300 as m
    return m


def one_hot_case(N, d, log_score, v_exp, seed, negative):
    """bf16 q, K, V whose scores are +- 2^log_score * (1 + j / 8), one token
    a kv head ahead of the others by 2^log_score / 8: the softmax is one-hot.  V
    blocks are 2^v_exp apart in size, the winners' block the smallest."""
    B, Hkv = 2, 2
    g = torch.Generator().manual_seed(seed)
    half = log_score // 2
    q = torch.zeros(B, Hkv * 8, d)
    q[..., 0] = 2.0 ** (log_score - half) * (-1.0 if negative else 1.0)
    j = torch.randint(1, 7, (B, Hkv, N), generator=g).float()
    win = torch.randint(0, N, (B, Hkv, 1), generator=g)
    j.scatter_(2, win, 0.0 if negative else 7.0)
    k = torch.zeros(B, Hkv, N, d)
    k[..., 0] = (1 + j / 8) * 2.0 ** half
    v = torch.randn(B, Hkv, N, d, generator=g)
    P = -(-N // PAGE)
    e = torch.randint(-v_exp, v_exp + 1, (B, Hkv, P), generator=g).float()
    e.scatter_(2, win // PAGE, -float(v_exp))
    v *= torch.exp2(e).repeat_interleave(PAGE, dim=2)[:, :, :N, None]
    return q.to(torch.bfloat16), ref.quantise(k, torch.bfloat16), ref.quantise(v, torch.bfloat16), win


def check_one_hot(case, N, heads, dev, dkv):
    q, K, V, win = case
    q = q.view(2, 2, 8, 64)[:, :, :heads].reshape(2, 2 * heads, 64).contiguous()
    kv, vv = ref.values(*K), ref.values(*V)
    want = ref.attention(q, kv, vv, 1.0)
    pick = vv.gather(2, win[..., None].expand(-1, -1, -1, 64))  # [B, Hkv, 1, d]
    assert torch.equal(want.view(2, 2, heads, 64), pick.expand(-1, -1, heads, -1))
    for paged in (False, True):
        Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, paged)
        meta = dkv.kv_meta_build(Kd)
        for out in (dkv.decode_attn_full(q.to(dev), Kd, Vd, scale=1.0),
                    dkv.decode_attn_select(q.to(dev), Kd, Vd, meta, 3, scale=1.0)):
            # the winner's weight is 1 and the others' 0: what is left is the
            # weight's two halves (22 bits) and the fp32 steps of the joins
            assert torch.all((out.cpu().double() - want).abs() <= want.abs() * 2.0 ** -18)


@pytest.mark.parametrize("heads", [1, 4, 8])
@pytest.mark.parametrize("N", [40, 9000])  # one work item a unit, and several
def test_scores_all_below(N, heads, dev, dkv):
    # every score lies below -1e30
    check_one_hot(one_hot_case(N, 64, 105, 0, heads, True), N, heads, dev, dkv)


@pytest.mark.parametrize("heads", [1, 4, 8])
@pytest.mark.parametrize("N", [40, 9000])
@pytest.mark.parametrize("log_score,v_exp,negative", [(105, 20, True), (40, 40, False),
                                                      (40, 40, True), (100, 40, False)])
def test_scales_beside_large_scores(log_score, v_exp, negative, N, heads, dev, dkv):
    # scores so large that a V scale's exponent, added to one, has no digits left
    check_one_hot(one_hot_case(N, 64, log_score, v_exp, heads, negative), N, heads, dev, dkv)


@pytest.mark.parametrize("Hq", [2, 6, 16])
@pytest.mark.parametrize("N", [40, 9000])
def test_not_a_number(N, Hq, dev, dkv):
    # a NaN query gives NaN rows, a NaN key NaN rows of its kv head's queries, a
    # NaN value its channel; other rows keep their results
    B, H, d = 2, 2, 64
    G = Hq // H
    q, K, V = make(B, Hq, H, d, N, torch.bfloat16, seed=N + Hq)
    scale = 1 / math.sqrt(d)
    for paged in (False, True):
        Kd, Vd = caches(dkv, dev, K, V, torch.bfloat16, paged)
        clean = dkv.decode_attn_full(q.to(dev), Kd, Vd)
        bad = q.clone()
        bad[1, G - 1, 5] = math.nan
        out = dkv.decode_attn_full(bad.to(dev), Kd, Vd)
        assert out[1, G - 1].isnan().all()
        keep = torch.ones(B, Hq, dtype=torch.bool)
        keep[1, G - 1] = False
        assert torch.equal(out[keep], clean[keep])
        meta = dkv.kv_meta_build(Kd)
        top_k = -(-N // PAGE)  # every page
        for t, channels in ((0, slice(None)), (1, slice(9, 10))):
            c = [x[0].clone() for x in (K, V)]
            c[t].view(torch.uint8)[0, 1, N // 2, 9] = 0x7F
            Kb, Vb = caches(dkv, dev, (c[0], K[1]), (c[1], V[1]), torch.bfloat16, paged)
            for f in (lambda a, b: dkv.decode_attn_full(q.to(dev), a, b),
                      lambda a, b: dkv.decode_attn_select(q.to(dev), a, b, meta, top_k)):
                clean, out = f(Kd, Vd), f(Kb, Vb)
                hit = torch.zeros(B, Hq, d, dtype=torch.bool, device=dev)
                hit[0, G:, channels] = True
                assert torch.equal(out.isnan(), hit)
                assert torch.equal(out[~hit], clean[~hit])


def noalloc(dkv, q, K, V, out):
    ks, B, H, N, d = dkv._kv_struct(K)
    vs = dkv._kv_struct(V)[0]
    p = dkv._params(q, B, H, N, d, out, None)
    fn = dkv.lib().dkv_decode_attn_full_noalloc
    fn.argtypes = [ctypes.POINTER(dkv._Params), ctypes.c_void_p, ctypes.POINTER(dkv._KV),
                   ctypes.POINTER(dkv._KV), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    return fn(ctypes.byref(p), q.data_ptr(), ctypes.byref(ks), ctypes.byref(vs), out.data_ptr(),
              dkv.DKV_FP32, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


def test_fixed_scratch(dev, dkv):
    # the size that counts is the 8-bit layout's: it fits where the 16-bit one's
    # does not, and the other way round
    limit = 16 << 20
    for B, Hq, H, N, fits in ((2, 8, 2, 3000, True), (4, 256, 32, 32768, True),
                              (1, 640, 80, 32768, False)):
        d = 128
        need = [dkv.workspace_bytes(B, Hq, H, d, N, fp8=f) for f in (False, True)]
        assert (need[1] <= limit) == fits and (N == 3000 or (need[0] <= limit) != fits)
        g = torch.Generator(dev).manual_seed(N)
        q = torch.randn(B, Hq, d, generator=g, device=dev).to(torch.bfloat16)
        K, V = (dkv.Fp8Cache(torch.randint(0, 0x7F, (B, H, N, d), generator=g, device=dev,
                                           dtype=torch.uint8).view(torch.float8_e4m3fn),
                             torch.full((B, H, -(-N // 16)), 2.0 ** -8, device=dev))
                for _ in range(2))
        out = torch.full((B, Hq, d), 5.0, device=dev)
        status = noalloc(dkv, q, K, V, out)
        if fits:
            assert status == dkv.DKV_OK
            assert torch.equal(out, dkv.decode_attn_full(q, K, V))
        else:
            assert status == 6  # DKV_ERR_WORKSPACE
            assert (out == 5.0).all()


def test_longest_sequence(dev, dkv):
    # N = 2^31 - 1: the last page holds 15 tokens, and its sixteenth slot is not
    # attended (NaN there).  Every other page is the same block
    N, d = (1 << 31) - 1, 64
    q, K, V = make(1, 1, 1, d, 32, torch.bfloat16, seed=1)
    for c, _ in (K, V):
        c.view(torch.uint8)[0, 0, 31] = 0x7F
    bt = torch.zeros(1, 1 << 27, dtype=torch.int32, device=dev)
    bt[0, -1] = 1
    Kd, Vd = (dkv.Fp8PagedCache(c.view(2, 1, 16, d).to(dev), s.view(2, 1).to(dev), bt, N)
              for c, s in (K, V))
    out = dkv.decode_attn_full(q.to(dev), Kd, Vd).cpu().double()[0, 0]
    kv, vv = ref.values(*K)[0, 0], ref.values(*V)[0, 0]
    p = torch.exp(kv[:31] @ q[0, 0].double() / 8)
    p[:16] *= (1 << 27) - 1  # times that the first block is attended
    want = (p @ vv[:31]) / p.sum()
    # A page of the first block gives the same terms each time, so l and o grow by
    # equal steps, and from 2^24 steps on a step is below half an ulp of the sum: a
    # warp takes 2^27 / (256 items * 4) = 2^17 pages of 16 tokens, an item joins four
    # warps' sums and the merge 256 items': 2^17 sums of at most 2^-24 each, relative
    # to max |v|, beside tolerance()'s terms
    tol = ref.tolerance(q, ref.values(*K)[:, :, :31], ref.values(*V)[:, :, :31], 1 / 8)
    assert (out - want).abs().max() <= tol + 2.0 ** 17 * 2.0 ** -24 * float(vv[:31].abs().max())
