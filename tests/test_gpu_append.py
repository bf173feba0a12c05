"""kv_append against the plain form, bit for bit: the rotation's fp32 steps are
defined one by one, codes and scales follow from its results, so nothing is
left to a tolerance.  Every cache slot, scale and query row that is no new
token's must keep its bytes."""

import pytest
import torch

import fp8_helpers as ref
from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(scope="module")
def dev():
    return require_cuda()


@pytest.fixture(scope="module")
def dkv():
    import decode_attention_paged_kv_gb300 as m
    return m


class Cache:
    """One cache on both sides: the logical tensors on the CPU and the device's
    object, dense or a shuffled pool with spare blocks."""

    def __init__(self, dkv, kind, B, H, N, d, dt, gen, dev, table):
        P = -(-N // PAGE)
        self.eight, self.paged, self.N, self.table = "fp8" in kind, "paged" in kind, N, table
        # (older tokens lie where appending left them: values under a block's scale)
        x = torch.randn(B, H, P * PAGE, d, generator=gen)
        if self.eight:
            c, s = ref.quantise(x, dt)
            self.ref = (c.view(torch.uint8), s, dt)
            data = self.ref[0]
        else:
            self.ref = data = x.to(dt)
        blocks = lambda t: t.view(B, H, P, PAGE, d).permute(0, 2, 1, 3, 4).reshape(-1, H, PAGE, d)
        if self.paged:
            nb = B * P + 4
            pool = torch.zeros(nb, H, PAGE, d, dtype=data.dtype)
            pool[table.view(-1).long()] = blocks(data)
            self.dev = pool.to(dev)
            self.spare = sorted(set(range(nb)) - set(table.view(-1).tolist()))
            if self.eight:
                sc = torch.full((nb, H), 3.0)
                sc[table.view(-1).long()] = self.ref[1].permute(0, 2, 1).reshape(-1, H)
                self.scale = sc.to(dev)
                self.obj = dkv.Fp8PagedCache(self.dev.view(torch.float8_e4m3fn), self.scale,
                                             table.to(dev), N, dt)
            else:
                self.obj = dkv.PagedCache(self.dev, table.to(dev), N)
        else:
            self.dev = data.to(dev)
            if self.eight:
                self.scale = self.ref[1].to(dev)
                self.obj = dkv.Fp8Cache(self.dev.view(torch.float8_e4m3fn)[:, :, :N], self.scale, dt)
            else:
                self.obj = self.dev[:, :, :N]

    def logical(self):
        """The device's cache as the CPU side lays it out."""
        x = self.dev.cpu()
        B, P = self.table.shape
        if self.paged:
            assert not x[self.spare].any()
            H, d = x.shape[1], x.shape[3]
            at = self.table.view(-1).long()
            x = x[at].view(B, P, H, PAGE, d).permute(0, 2, 1, 3, 4).reshape(B, H, P * PAGE, d)
        if not self.eight:
            return x
        s = self.scale.cpu()
        if self.paged:
            s = s[self.table.view(-1).long()].view(B, P, -1).permute(0, 2, 1)
        return x, s

    def check(self):
        got = self.logical()
        if not self.eight:
            assert torch.equal(got.view(torch.int16), self.ref.view(torch.int16))
            return
        assert torch.equal(got[1], self.ref[1])
        assert torch.equal(got[0], self.ref[0])


def table_for(B, N, gen):
    P = -(-N // PAGE)
    return torch.randperm(B * P + 4, generator=gen)[:B * P].view(B, P).to(torch.int32)


def run(dkv, dev, kind, B, Hq, Hkv, d, N, T, lens, news, dt, r, il, seed=0, scale=1.0,
        in_place=False, workspace=None):
    gen = torch.Generator().manual_seed(seed)
    table = table_for(B, N, gen)
    K = Cache(dkv, kind, B, Hkv, N, d, dt, gen, dev, table)
    V = Cache(dkv, kind, B, Hkv, N, d, dt, gen, dev, table)
    if V.paged:  # one table object for both
        V.obj = V.obj._replace(block_table=K.obj.block_table)
    qkv = (torch.randn(B, T, Hq + 2 * Hkv, d, generator=gen) * scale).to(dt)
    g = qkv.to(dev)
    cut = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:])
    (q, k, v), (gq, gk, gv) = cut(qkv), cut(g)
    rope = dkv.rope_table(N, r) if r else None
    grope = tuple(t.to(dev) for t in rope) if r else None
    lens_t = torch.tensor(lens, dtype=torch.int32) if lens is not None else None
    news_t = torch.tensor(news, dtype=torch.int32) if news is not None else None
    q_ref = q.clone() if in_place else torch.full((B, T, Hq, d), 7.0, dtype=dt)
    q_out = gq if in_place else q_ref.to(dev)
    back = dkv.kv_append(gk, gv, K.obj, V.obj, seq_lens=None if lens is None else lens_t.to(dev),
                         new_lens=None if news is None else news_t.to(dev),
                         q=gq if Hq else None, q_out=q_out if Hq else None, rope=grope,
                         interleaved=il, workspace=workspace)
    torch.cuda.synchronize()
    full = torch.full((B,), N, dtype=torch.int32)
    end = full if lens_t is None else lens_t
    new = torch.full((B,), T, dtype=torch.int32) if news_t is None else news_t
    bad = (new < 0) | (new > T) | (new > end) | (end > N)
    new = torch.where(bad | (end <= 0), 0, new)
    ref.append(k, v, K.ref, V.ref, end, new, q if Hq else None, q_ref, rope, il)
    K.check()
    V.check()
    if Hq:
        assert back is q_out
        assert torch.equal(q_out.cpu().view(torch.int16), q_ref.view(torch.int16))
    if in_place:  # the rest of the fused rows is only read
        assert torch.equal(g[:, :, Hq:].cpu().view(torch.int16), qkv[:, :, Hq:].view(torch.int16))
    return int(bad.sum())


KINDS = ["dense", "paged", "fp8", "fp8_paged"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,dt,r,il", [(128, torch.bfloat16, 128, False),
                                       (64, torch.float16, 64, True),
                                       (128, torch.float16, 48, False),
                                       (64, torch.bfloat16, 16, True),
                                       (64, torch.bfloat16, 0, False)])
@pytest.mark.parametrize("T,lens,news", [
    (1, [1, 16, 17, 40, 45], None),                 # one token each: first, last, next block
    (1, [1, 0, 17, 40, 45], [1, 1, 0, 1, 0]),       # unused entries
    (3, [3, 17, 16, 45, 33], [3, 3, 2, 1, 0]),
    (45, [45, 20, 45, 16, 0], [45, 20, 1, 15, 9]),  # prompts
])
def test_append(kind, d, dt, r, il, T, lens, news, dev, dkv):
    run(dkv, dev, kind, 5, 6, 3, d, 45, T, lens, news, dt, r, il, seed=d + T + r)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,Hq,Hkv,N,T", [(1, 0, 1, 1, 1), (2, 0, 2, 16, 16), (3, 8, 8, 300, 300),
                                          (1, 7, 1, 2000, 1999), (2, 3, 1, 31, 2)])
def test_append_without_lengths(kind, B, Hq, Hkv, N, T, dev, dkv):
    # the last T of N tokens of every sequence; no queries where Hq = 0
    run(dkv, dev, kind, B, Hq, Hkv, 128, N, T, None, None, torch.bfloat16, 128 if N > 1 else 0,
        False, seed=N)


# More rows than a device holds threads for: 16-bit caches change kernels there.
@pytest.mark.parametrize("kind", ["dense", "paged"])
@pytest.mark.parametrize("d,dt,r,il", [(128, torch.bfloat16, 128, False),
                                       (64, torch.float16, 48, True)])
@pytest.mark.parametrize("lens,news", [
    (None, None), ([650, 41, 700, 17, 0], [601, 30, 650, 1, 0]),
    ([701, 600, 600, 699, 33], [5, 651, 600, -1, 33])])
def test_many_tokens(kind, d, dt, r, il, lens, news, dev, dkv):
    ws = torch.zeros(dkv.DKV_WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=dev)
    bad = run(dkv, dev, kind, 5, 9, 5 if d == 128 else 15, d, 700, 650, lens, news, dt, r, il,
              seed=d, workspace=ws)
    assert dkv.read_device_status(ws) == (dkv.DKV_ERR_DEVICE_CHECK if bad else 0)


def test_many_tokens_with_a_bad_block(dev, dkv):
    gen = torch.Generator().manual_seed(3)
    B, H, N = 4, 11, 700
    table = table_for(B, N, gen)
    K = Cache(dkv, "paged", B, H, N, 128, torch.bfloat16, gen, dev, table)
    V = Cache(dkv, "paged", B, H, N, 128, torch.bfloat16, gen, dev, table)
    bt = table.clone()
    bt[1, 2], bt[3, 43] = -1, 1 << 30  # tokens 32 .. 47 of one, the last 12 of another
    K.obj = K.obj._replace(block_table=bt.to(dev))
    V.obj = V.obj._replace(block_table=K.obj.block_table)
    x = torch.randn(B, N, H, 128, generator=gen).to(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    q = dkv.kv_append(x.to(dev), x.to(dev), K.obj, V.obj, q=x.to(dev), workspace=ws)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_CHECK
    assert torch.equal(q.cpu(), x)
    for c in (K, V):
        keep = c.ref[1, :, 32:48].clone(), c.ref[3, :, 688:].clone()
        c.ref[:, :, :N] = x.permute(0, 2, 1, 3)
        c.ref[1, :, 32:48], c.ref[3, :, 688:] = keep
        c.check()


@pytest.mark.parametrize("kind", ["paged", "fp8"])
@pytest.mark.parametrize("T", [1, 18])
def test_more_sequences_than_are_counted(kind, T, dev, dkv):
    g = torch.Generator().manual_seed(T)
    lens = torch.randint(T, 41, (131,), generator=g)
    news = torch.randint(0, T + 1, (131,), generator=g)
    lens[3], news[3], news[130] = 0, T, T
    run(dkv, dev, kind, 131, 1, 1, 64, 40, T, lens.tolist(), news.tolist(), torch.bfloat16, 64, False)


@pytest.mark.parametrize("kind", ["dense", "fp8_paged"])
def test_queries_in_place(kind, dev, dkv):
    run(dkv, dev, kind, 2, 4, 2, 128, 64, 6, [50, 6], None, torch.bfloat16, 128, False,
        in_place=True)
    run(dkv, dev, kind, 2, 4, 2, 64, 64, 1, [50, 6], None, torch.float16, 64, True, in_place=True)


@pytest.mark.parametrize("dt,scale", [(torch.bfloat16, 2.0 ** 100), (torch.bfloat16, 2.0 ** -122),
                                      (torch.float16, 15000.0), (torch.float16, 2.0 ** -20),
                                      (torch.bfloat16, 0.0), (torch.bfloat16, 300.0)])
@pytest.mark.parametrize("T", [1, 5])
def test_scales_at_their_ends(dt, scale, T, dev, dkv):
    # scales that rise over older tokens by far, clamp, or are asked for by zeros
    run(dkv, dev, "fp8_paged", 4, 2, 2, 64, 40, T, [40, 22, 5, 17], None, dt, 0, False,
        scale=scale, seed=3)
    run(dkv, dev, "fp8", 4, 2, 2, 128, 40, T, [40, 22, 5, 17], None, dt, 0, False, scale=scale,
        seed=4)


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("factor", [3.0, 0.37])
def test_scales_of_another_maker(T, factor, dev, dkv):
    # blocks whose scale is no power of two keep it while it is large enough
    gen = torch.Generator().manual_seed(T)
    table = table_for(3, 64, gen)
    K = Cache(dkv, "fp8_paged", 3, 2, 64, 64, torch.bfloat16, gen, dev, table)
    V = Cache(dkv, "fp8_paged", 3, 2, 64, 64, torch.bfloat16, gen, dev, table)
    V.obj = V.obj._replace(block_table=K.obj.block_table)
    for c in (K, V):
        c.scale[table.view(-1).long().to(dev)] *= factor
        c.ref[1].mul_(factor)
    x = torch.randn(3, T, 2, 64, generator=gen).to(torch.bfloat16)
    lens = torch.tensor([30, 64, 17], dtype=torch.int32)
    dkv.kv_append(x.to(dev), x.to(dev), K.obj, V.obj, seq_lens=lens.to(dev))
    ref.append(x, x, K.ref, V.ref, lens, [T] * 3)
    K.check()
    V.check()


def test_largest_value_at_a_scale_border(dev, dkv):
    # amax = 448 * 2^e exactly, one step above it, and the largest fp16
    for top in (448.0, 450.0, 3.5, 3.515625, 65504.0):
        x = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
        x[..., 5], x[..., 6] = top, -top / 2
        c = torch.zeros(1, 1, 16, 64, dtype=torch.float8_e4m3fn, device=dev)
        s = torch.full((1, 1, 1), float("nan"), device=dev)
        K = dkv.Fp8Cache(c, s, torch.float16)
        V = dkv.Fp8Cache(c.clone(), s.clone(), torch.float16)
        one = torch.ones(1, dtype=torch.int32, device=dev)
        dkv.kv_append(x.to(dev), x.to(dev), K, V, seq_lens=one)
        want = ref.block_scale(x.abs().amax().view(1), torch.float16)
        assert s.cpu().double().view(-1) == want
        got = ref.decode(c[0, 0, 0]) * want
        assert torch.equal(got, ref.TABLE[ref.encode(x[0, 0, 0].double() / want)
                                          .view(torch.uint8).long()] * want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 4])
def test_what_does_not_fit_is_left_alone(kind, T, dev, dkv):
    # too long for the cache, more new tokens than rows or than the length, a
    # negative count; a valid sequence beside them is appended
    ws = torch.zeros(dkv.DKV_WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=dev)
    n = run(dkv, dev, kind, 5, 2, 2, 64, 40, T, [41, 30, 2, 30, 30], [1, T + 1, 3 if T > 2 else 1,
            -1, 1], torch.bfloat16, 64, False, workspace=ws)
    assert n >= 3
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_CHECK
    assert dkv.read_device_status(ws) == 0
    run(dkv, dev, kind, 2, 2, 2, 64, 40, T, [40, 30], None, torch.bfloat16, 64, False,
        workspace=ws)
    assert dkv.read_device_status(ws) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 4])
def test_short_table_of_angles(kind, T, dev, dkv):
    gen = torch.Generator().manual_seed(1)
    table = table_for(2, 48, gen)
    K = Cache(dkv, kind, 2, 2, 48, 64, torch.bfloat16, gen, dev, table)
    V = Cache(dkv, kind, 2, 2, 48, 64, torch.bfloat16, gen, dev, table)
    if V.paged:
        V.obj = V.obj._replace(block_table=K.obj.block_table)
    x = torch.randn(2, T, 2, 64, generator=gen).to(torch.bfloat16)
    rope = tuple(t.to(dev) for t in dkv.rope_table(32, 64))
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    lens = torch.tensor([33, 32], dtype=torch.int32)
    dkv.kv_append(x.to(dev), x.to(dev), K.obj, V.obj, seq_lens=lens.to(dev), rope=rope,
                  workspace=ws)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_CHECK
    ref.append(x, x, K.ref, V.ref, lens, [0, T], rope=dkv.rope_table(32, 64))
    K.check()
    V.check()


@pytest.mark.parametrize("kind", ["paged", "fp8_paged"])
@pytest.mark.parametrize("T,bad", [(1, -1), (1, 1 << 30), (20, -1), (20, 10 ** 6)])
def test_bad_block_is_not_written(kind, T, bad, dev, dkv):
    gen = torch.Generator().manual_seed(2)
    table = table_for(2, 64, gen)
    K = Cache(dkv, kind, 2, 2, 64, 64, torch.bfloat16, gen, dev, table)
    V = Cache(dkv, kind, 2, 2, 64, 64, torch.bfloat16, gen, dev, table)
    bt = table.clone()
    bt[1, 2] = bad  # tokens 32 .. 47 of sequence 1
    K.obj = K.obj._replace(block_table=bt.to(dev))
    V.obj = V.obj._replace(block_table=K.obj.block_table)
    x = torch.randn(2, T, 2, 64, generator=gen).to(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    lens = torch.tensor([40, 40], dtype=torch.int32)
    q = dkv.kv_append(x.to(dev), x.to(dev), K.obj, V.obj, seq_lens=lens.to(dev), q=x.to(dev),
                      workspace=ws)
    assert dkv.read_device_status(ws) == dkv.DKV_ERR_DEVICE_CHECK
    assert torch.equal(q.cpu(), x)
    ref.append(x[:1], x[:1], *(tuple(t[:1] for t in c.ref[:2]) + (c.ref[2],) if c.eight
                               else c.ref[:1] for c in (K, V)), lens[:1], [T])
    n = max(0, T - 8)  # sequence 1's tokens before the bad page
    cut = lambda c: (tuple(t[1:] for t in c.ref[:2]) + (c.ref[2],) if c.eight else c.ref[1:])
    ref.append(x[1:, :n], x[1:, :n], cut(K), cut(V), [32], [n])
    K.check()
    V.check()


@pytest.mark.parametrize("kind", ["paged", "fp8_paged"])
def test_captured_step_and_stream(kind, dev, dkv):
    # a captured append replayed as the lengths advance on the device equals the
    # plain form run token by token
    B, Hq, H, d, N = 2, 4, 2, 128, 64
    gen = torch.Generator().manual_seed(5)
    table = table_for(B, N, gen)
    K = Cache(dkv, kind, B, H, N, d, torch.bfloat16, gen, dev, table)
    V = Cache(dkv, kind, B, H, N, d, torch.bfloat16, gen, dev, table)
    V.obj = V.obj._replace(block_table=K.obj.block_table)
    rope = dkv.rope_table(N, d)
    grope = tuple(t.to(dev) for t in rope)
    xs = torch.randn(20, B, 1, Hq + 2 * H, d, generator=gen).to(torch.bfloat16)
    row = torch.zeros(B, 1, Hq + 2 * H, d, dtype=torch.bfloat16, device=dev)
    q_out = torch.zeros(B, 1, Hq, d, dtype=torch.bfloat16, device=dev)
    lens = torch.tensor([13, 30], dtype=torch.int32, device=dev)

    def step():
        lens.add_(1)
        dkv.kv_append(row[:, :, Hq:Hq + H], row[:, :, Hq + H:], K.obj, V.obj, seq_lens=lens,
                      q=row[:, :, :Hq], q_out=q_out, rope=grope)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        row.copy_(xs[0])
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for i in range(1, 20):
            row.copy_(xs[i])
            graph.replay()
    torch.cuda.synchronize()
    at = torch.tensor([13, 30])
    for i in range(20):
        at = at + 1
        q_ref = torch.zeros(B, 1, Hq, d, dtype=torch.bfloat16)
        ref.append(xs[i][:, :, Hq:Hq + H], xs[i][:, :, Hq + H:], K.ref, V.ref, at, [1, 1],
                   xs[i][:, :, :Hq], q_ref, rope)
    K.check()
    V.check()
    assert torch.equal(q_out.cpu(), q_ref)


def test_blocks_past_two_gib(dev, dkv):
    # the last block of a pool whose offsets pass 2^31 elements (and bytes)
    nb, H, d = (1 << 31) // (8 * 16 * 128) + 3, 8, 128
    x = torch.randn(1, 2, H, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    bt = torch.tensor([[nb - 1]], dtype=torch.int32, device=dev)
    lens = torch.tensor([2], dtype=torch.int32, device=dev)
    for eight in (True, False):
        pool = torch.zeros(nb, H, 16, d, dtype=torch.uint8 if eight else torch.bfloat16, device=dev)
        if eight:
            sc = torch.zeros(nb, H, device=dev)
            c = dkv.Fp8PagedCache(pool.view(torch.float8_e4m3fn), sc, bt, 16)
            # one pool for both: K and V blocks of a table may not share one, so
            # V goes to a small pool of its own with the same strides and table
            small = torch.empty_strided((nb, H, 16, d), pool.stride(), dtype=torch.uint8, device=dev)
            cv = dkv.Fp8PagedCache(small.view(torch.float8_e4m3fn), sc.clone(), bt, 16)
        else:
            c, cv = dkv.PagedCache(pool, bt, 16), dkv.PagedCache(torch.empty_like(pool), bt, 16)
        dkv.kv_append(x.to(dev), x.to(dev), c, cv, seq_lens=lens)
        got = pool[nb - 1, :, :2].cpu()
        if eight:
            want, s = ref.quantise(x.transpose(1, 2).float(), torch.bfloat16)
            assert torch.equal(got, want[0].view(torch.uint8))
            assert torch.equal(sc[nb - 1].cpu(), s[0, :, 0])
        else:
            assert torch.equal(got, x[0].transpose(0, 1))
        assert not pool[:nb - 1].any()
        del pool, c, cv


def test_python_refusals(dev, dkv):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=dev)
    K, V, x = z(2, 2, 40, 64), z(2, 2, 40, 64), z(2, 3, 2, 64)
    ok = dict(seq_lens=torch.tensor([3, 9], dtype=torch.int32, device=dev))
    dkv.kv_append(x, x, K, V, **ok)
    assert dkv.kv_append(x[:, :0], x[:, :0], K, V, **ok) is None  # no rows: nothing to do
    for bad in (dict(seq_lens=torch.tensor([3, 9], device=dev)), dict(seq_lens=torch.zeros(
            2, dtype=torch.int32)), dict(new_lens=torch.zeros(3, dtype=torch.int32, device=dev)),
            dict(q=z(2, 3, 4, 64, dt=torch.float16)), dict(q=z(2, 2, 4, 64)),
            dict(q_out=z(2, 3, 4, 64)), dict(q=z(2, 3, 4, 64), q_out=z(2, 3, 4, 32)),
            dict(rope=(z(40, 32), z(40, 32))), dict(rope=dkv.rope_table(40, 64)),
            dict(workspace=z(8))):
        with pytest.raises((ValueError, TypeError)):
            dkv.kv_append(x, x, K, V, **(ok | bad))
    for k, v, kk, vv in ((x.half(), x, K, V), (x, x[:, :2], K, V), (x, x, K, V[:, :, :39]),
                         (x[..., :32], x[..., :32], K, V), (x[0], x[0], K, V)):
        with pytest.raises(ValueError):
            dkv.kv_append(k, v, kk, vv, **ok)
    with pytest.raises(dkv.DkvError):  # a rotary width of 24
        dkv.kv_append(x, x, K, V, rope=(z(40, 12, dt=torch.float32),) * 2, **ok)
    with pytest.raises(dkv.DkvError):  # a cache whose heads are one tensor
        dkv.kv_append(x, x, K[:, :1].expand(2, 2, 40, 64), V, **ok)
