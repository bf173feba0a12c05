"""Calls on latent caches and on pages that do not fit together are refused before any CUDA
call: by the binding on CPU tensors, and by the C ABI on made-up addresses.  No GPU."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def dkv():
    from decode_attention_paged_kv_gb300 import build as b
    b.build()
    import decode_attention_paged_kv_gb300 as m
    m.lib()
    return m


def test_the_device_is_needed(dkv):
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    dense = t(2, 40, 320)
    paged = dkv.LatentCache(t(9, 16, 320), i(2, 3), 40)
    for cache in (dense, paged):
        with pytest.raises(ValueError, match="CUDA"):
            dkv.latent_append(t(2, 1, 256), t(2, 1, 64), cache)
        with pytest.raises(ValueError, match="CUDA"):
            dkv.latent_decode_attn(t(2, 1, 4, 256), t(2, 1, 4, 64), cache, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        dkv.latent_prompt_attn(t(5, 2, 64), t(5, 2, 64), t(5, 2, 64), t(5, 64), t(5, 2, 64), i(2),
                               None, 0.1)
    for f in (lambda: dkv.kv_pages_fork([paged], i(9), i(2)),
              lambda: dkv.kv_pages_compact([paged], i(9))):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_caches_that_are_not(dkv):
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bad = [
        (t(2, 40, 320).transpose(1, 2), "channel stride"),
        (t(40, 320), "must be"),
        (dkv.LatentCache(t(9, 24, 320), i(2, 3), 40), "16, 32 or 64"),
        (dkv.LatentCache(t(9, 16, 320), i(2, 2), 40), "fewer"),
        (dkv.LatentCache(t(9, 16, 320), i(2, 3).long(), 40), "int32"),
        (dkv.LatentCache(t(9, 16, 320), i(2, 3), 0), "fewer"),
        (dkv.LatentCache(t(9, 16, 320), i(2, 6)[:, ::2], 40), "unit column stride"),
    ]
    for cache, text in bad:
        with pytest.raises(ValueError, match=text):
            dkv.latent_append(t(2, 1, 256), t(2, 1, 64), cache)
        with pytest.raises(ValueError, match=text):
            dkv.latent_decode_attn(t(2, 1, 4, 256), t(2, 1, 4, 64), cache, 0.1)
    with pytest.raises(TypeError):
        dkv.latent_append(t(2, 1, 256), t(2, 1, 64), [t(2, 40, 320)])
    with pytest.raises(TypeError):
        dkv.latent_append(t(2, 1, 256), t(2, 1, 64), t(2, 40, 320).long())


def test_lists_of_caches(dkv):
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    table = torch.zeros(2, 3, dtype=torch.int32)
    one = dkv.PagedCache(t(9, 2, 16, 64), table, 40)
    for bad in (one, [], (), t(2)):
        with pytest.raises(ValueError, match="list"):
            dkv.kv_pages_fork(bad, table, table)
    for bad in ([t(2, 2, 40, 64)], [None]):
        with pytest.raises(TypeError, match="PagedCache"):
            dkv.kv_pages_compact(bad, table)


def test_workspace_sizes(dkv):
    assert dkv.latent_workspace_bytes(1, 1, 1, 256, 1) >= 256
    assert dkv.latent_workspace_bytes(64, 4, 128, 512, 1 << 20) < 1 << 28
    assert dkv.pages_workspace_bytes(1, 1, 1) >= 256
    for bad in ((0, 1, 1, 256, 1), (1, 0, 1, 256, 1), (1, 1, 0, 256, 1), (1, 1, 1, 128, 1),
                (1, 1, 1, 256, 0), (16385, 1, 1, 256, 1), (1, 1 << 10, 1 << 10, 256, 1)):
        with pytest.raises(dkv.DkvError):
            dkv.latent_workspace_bytes(*bad)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (16385, 1, 1), (16384, 1 << 17, 1)):
        with pytest.raises(dkv.DkvError):
            dkv.pages_workspace_bytes(*bad)


def test_workspaces_rise_with_every_size(dkv):
    # (a workspace for the largest call serves the smaller ones)
    import itertools
    sizes = ([1, 3, 64], [1, 2, 5, 9], [1, 8, 16, 17, 40, 128, 200], [256, 512],
             [1, 64, 65, 1000, 100000])
    need = {k: dkv.latent_workspace_bytes(*k) for k in itertools.product(*sizes)}
    for k, n in need.items():
        for i, options in enumerate(sizes):
            at = options.index(k[i])
            if at:
                assert need[k[:i] + (options[at - 1],) + k[i + 1:]] <= n, (k, i)
    for a, b in itertools.pairwise([1, 2, 100, 10000]):
        assert dkv.pages_workspace_bytes(a, 7, 7) <= dkv.pages_workspace_bytes(b, 7, 7)
        assert dkv.pages_workspace_bytes(7, a, 7) <= dkv.pages_workspace_bytes(7, b, 7)
        assert dkv.pages_workspace_bytes(7, 7, a) <= dkv.pages_workspace_bytes(7, 7, b)


# ---------------------------------------------------------------- the C ABI's own checks
OK, NULL, SHAPE, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = range(7)
ADDR = 1 << 20  # an address that nothing reads before it is refused


class Prompt(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_heads", "nope_dim", "rope_dim", "dtype",
                                               "out_dtype", "causal")]
                + [("flags", ctypes.c_uint32), ("scale", ctypes.c_float),
                   ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32)]
                + [(n, ctypes.c_void_p) for n in ("q_nope", "q_rope", "k_nope", "v", "k_rope", "out")]
                + [(n, ctypes.c_int64) for n in ("qn_t", "qn_h", "qr_t", "qr_h", "kn_t", "kn_h",
                                                 "v_t", "v_h", "kr_t", "o_t", "o_h")]
                + [("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p)])


class AppendArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_q_heads", "new_tokens", "rope_len",
                                               "interleaved")]
                + [("eps", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("c", "k", "q", "q_out", "norm")]
                + [(n, ctypes.c_int64) for n in ("c_b", "c_t", "k_b", "k_t", "q_b", "q_t", "q_h",
                                                 "o_b", "o_t", "o_h")]
                + [(n, ctypes.c_void_p) for n in ("cos", "sin", "seq_lens", "new_lens")])


class Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("bytes", ctypes.c_int64)]


class Pages(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("rows", "cols", "block_size", "num_blocks",
                                               "num_pools")]
                + [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                   ("refs", ctypes.c_void_p), ("pools", Pool * 16)])


def refusals(make, call, cases):
    for changes, want in cases:
        objs = make()
        for key, value in changes.items():
            name, field = key.split(".")
            setattr(objs[name], field, value)
        assert call(**objs) == want, changes


def latent(dkv, block=16):
    return dkv._LatentCache(dtype=0, latent_dim=512, rope_dim=64, seq_len=100, block_size=block,
                            num_blocks=20, data=ADDR, stride_b=16 * 576, stride_t=576,
                            block_table=ADDR, block_table_stride=7)


CACHE = [({"c.dtype": 2}, DTYPE), ({"c.latent_dim": 128}, UNSUPPORTED),
         ({"c.rope_dim": 32}, UNSUPPORTED), ({"c.seq_len": 0}, SHAPE),
         ({"c.block_size": 8}, UNSUPPORTED), ({"c.block_size": -1}, SHAPE),
         ({"c.num_blocks": 0}, SHAPE), ({"c.data": None}, NULL), ({"c.data": ADDR + 8}, ALIGN),
         ({"c.stride_t": 575}, SHAPE), ({"c.stride_t": 580}, ALIGN), ({"c.stride_b": 4}, ALIGN),
         ({"c.stride_b": -8}, SHAPE), ({"c.block_table": None}, NULL),
         ({"c.block_table": ADDR + 2}, ALIGN), ({"c.block_table_stride": 6}, SHAPE)]


def test_c_latent_append(dkv):
    f = dkv.lib().dkv_latent_append
    f.argtypes = [ctypes.c_void_p] * 4

    def make():
        p = AppendArgs(2, 4, 3, 100, 0, 1e-6, ADDR, ADDR, ADDR, ADDR, ADDR, 1536, 512, 192, 64,
                       768, 256, 64, 768, 256, 64, ADDR, ADDR, None, None)
        return {"p": p, "c": latent(dkv)}

    refusals(make, lambda p, c: f(ctypes.byref(p), ctypes.byref(c), None, None), CACHE + [
        ({"p.batch": 0}, SHAPE), ({"p.batch": 65536}, SHAPE), ({"p.new_tokens": -1}, SHAPE),
        ({"p.new_tokens": 101}, SHAPE), ({"p.rope_len": 99}, SHAPE), ({"p.interleaved": 2}, SHAPE),
        ({"p.eps": -1.0}, SHAPE), ({"p.eps": float("nan")}, SHAPE), ({"p.c": None}, NULL),
        ({"p.k": None}, NULL), ({"p.q": None}, NULL), ({"p.q_out": None}, NULL),
        ({"p.cos": None}, NULL), ({"p.norm": ADDR + 2}, ALIGN), ({"p.c": ADDR + 8}, ALIGN),
        ({"p.sin": ADDR + 4}, ALIGN), ({"p.c_t": 516}, ALIGN), ({"p.q_h": -64}, SHAPE),
        ({"p.o_h": 56}, SHAPE),             # queries that would be written over one another
        ({"c.stride_b": 576}, SHAPE),       # blocks that overlap
        ({"p.new_tokens": 0}, OK),          # nothing to do
    ])
    assert f(None, None, None, None) == NULL


def test_c_latent_decode(dkv):
    f = dkv.lib().dkv_latent_decode_attn
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                  ctypes.c_void_p]

    def make():
        p = dkv._LatentAttn(2, 8, 2, 0, 0.1, 2, ADDR, ADDR, ADDR, 8192, 4096, 512, 1024, 512, 64,
                            8192, 4096, 512, None, None)
        return {"p": p, "c": latent(dkv)}

    big = 1 << 40
    refusals(make, lambda p, c: f(ctypes.byref(p), ctypes.byref(c), ADDR, big, None), CACHE + [
        ({"p.batch": 0}, SHAPE), ({"p.batch": 16385}, UNSUPPORTED), ({"p.num_heads": 0}, SHAPE),
        ({"p.new_tokens": 0}, SHAPE), ({"p.num_heads": 1 << 19}, UNSUPPORTED),
        ({"p.scale": float("inf")}, SHAPE), ({"p.scale": float("nan")}, SHAPE),
        ({"p.out_dtype": 3}, DTYPE), ({"p.q_latent": None}, NULL), ({"p.q_rope": None}, NULL),
        ({"p.out": None}, NULL), ({"p.out": ADDR + 8}, ALIGN), ({"p.seq_lens": ADDR + 1}, ALIGN),
        ({"p.ql_stride_h": 500}, ALIGN), ({"p.qr_stride_b": -8}, SHAPE),
        ({"p.o_stride_h": 511}, ALIGN), ({"p.o_stride_h": 508}, SHAPE)])
    o = make()
    need = dkv.latent_workspace_bytes(2, 2, 8, 512, 100)
    for ws, n in ((None, need), (ADDR, need - 1)):
        assert f(ctypes.byref(o["p"]), ctypes.byref(o["c"]), ws, n, None) == WORKSPACE
    assert f(ctypes.byref(o["p"]), ctypes.byref(o["c"]), ADDR + 8, need, None) == ALIGN


def test_c_latent_prompt(dkv):
    f = dkv.lib().dkv_latent_prompt_attn
    f.argtypes = [ctypes.c_void_p] * 3

    def make():
        return {"p": Prompt(2, 4, 128, 64, 0, 2, 1, 0, 0.1, 50, 60, ADDR, ADDR, ADDR, ADDR, ADDR,
                            ADDR, 512, 128, 256, 64, 512, 128, 512, 128, 64, 512, 128, ADDR, ADDR)}

    refusals(make, lambda p: f(ctypes.byref(p), None, None), [
        ({"p.batch": 0}, SHAPE), ({"p.batch": 16385}, UNSUPPORTED), ({"p.num_heads": 0}, SHAPE),
        ({"p.num_heads": 65536}, SHAPE), ({"p.nope_dim": 96}, UNSUPPORTED),
        ({"p.rope_dim": 0}, UNSUPPORTED), ({"p.dtype": 2}, DTYPE), ({"p.out_dtype": 5}, DTYPE),
        ({"p.causal": 2}, SHAPE), ({"p.scale": float("nan")}, SHAPE), ({"p.total_q": -1}, SHAPE),
        ({"p.q_nope": None}, NULL), ({"p.k_rope": None}, NULL), ({"p.v": None}, NULL),
        ({"p.cu_q": None}, NULL), ({"p.cu_k": ADDR + 2}, ALIGN), ({"p.v": ADDR + 8}, ALIGN),
        ({"p.kn_t": 516}, ALIGN), ({"p.kr_t": -64}, SHAPE), ({"p.o_h": 120}, SHAPE),
        ({"p.o_t": 510}, ALIGN), ({"p.v_t": 1 << 40}, SHAPE), ({"p.total_q": 0}, OK)])


def test_c_pages(dkv):
    fork, compact = dkv.lib().dkv_kv_pages_fork, dkv.lib().dkv_kv_pages_compact
    fork.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]
    compact.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    other = ADDR << 4

    def make():
        p = Pages(4, 10, 16, 100, 2, ADDR, 10, ADDR)
        p.pools[0] = Pool(ADDR, 4096, 4096)
        p.pools[1] = Pool(other, 12, 12)
        return {"p": p, "a": p.pools[0], "b": p.pools[1]}

    cases = [({"p.rows": 0}, SHAPE), ({"p.cols": 0}, SHAPE), ({"p.block_size": 0}, SHAPE),
             ({"p.num_blocks": 0}, SHAPE), ({"p.num_pools": 17}, SHAPE),
             ({"p.num_pools": -1}, SHAPE), ({"p.rows": 16385}, UNSUPPORTED), ({"p.table": None}, NULL),
             ({"p.refs": None}, NULL), ({"p.refs": ADDR + 4}, ALIGN), ({"p.table": ADDR + 2}, ALIGN),
             ({"p.table_stride": 9}, SHAPE), ({"a.data": None}, NULL), ({"a.data": ADDR + 2}, ALIGN),
             ({"a.stride": 4092}, SHAPE), ({"a.bytes": 0}, SHAPE), ({"b.bytes": 10}, ALIGN),
             ({"b.data": ADDR}, SHAPE)]
    big = 1 << 40
    refusals(make, lambda p, a, b: fork(ctypes.byref(p), ADDR, None, None, ADDR, big, None), cases)
    refusals(make, lambda p, a, b: compact(ctypes.byref(p), ADDR, 10, ADDR, other, ADDR, big, None),
             cases)
    p = make()["p"]
    need = dkv.pages_workspace_bytes(4, 10, 100)
    r = ctypes.byref(p)
    assert fork(r, None, None, None, ADDR, need, None) == NULL
    assert fork(r, ADDR, ADDR + 1, None, ADDR, need, None) == ALIGN
    assert fork(r, ADDR, None, None, ADDR, need - 1, None) == WORKSPACE
    assert fork(r, ADDR, None, None, None, need, None) == WORKSPACE
    assert compact(r, None, 10, ADDR, other, ADDR, need, None) == NULL
    assert compact(r, ADDR, 11, ADDR, other, ADDR, need, None) == SHAPE  # the table, other rows
    assert compact(r, other, 9, ADDR, other, ADDR, need, None) == SHAPE
    assert compact(r, ADDR, 10, other, other, ADDR, need, None) == SHAPE  # counts and names in one


def test_c_pools_that_share_bytes(dkv):
    # blocks of two pools may alternate in memory, at one stride; no byte may be in two
    fork = dkv.lib().dkv_kv_pages_fork
    fork.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]

    def call(a, b, blocks=100):
        p = Pages(4, 10, 16, blocks, 2, ADDR, 10, ADDR)
        p.pools[0], p.pools[1] = Pool(*a), Pool(*b)
        # (no lengths: sound pools are refused for that, after their check)
        return fork(ctypes.byref(p), None, None, None, ADDR, 1 << 40, None)

    for a, b, want in [
            ((ADDR, 8192, 4096), (ADDR + 4096, 8192, 4096), NULL),   # keys, values of one tensor
            ((ADDR + 4096, 8192, 4096), (ADDR, 8192, 4096), NULL),
            ((ADDR, 8192, 4096), (ADDR + 3 * 8192 + 4096, 8192, 4096), NULL),
            ((ADDR, 8192, 4096), (ADDR + 4080, 8192, 4096), SHAPE),  # ends inside, begins inside
            ((ADDR, 8192, 4096), (ADDR + 4112, 8192, 4096), SHAPE),
            ((ADDR, 4096, 4096), (ADDR + 5 * 4096, 4096, 4096), SHAPE),
            ((ADDR, 4096, 4096), (ADDR + 100 * 4096, 4096, 4096), NULL),
            ((ADDR + 100 * 4096, 4096, 4096), (ADDR, 4096, 4096), NULL),
            ((ADDR, 4096, 4096), (ADDR + 99 * 4096, 4096, 64), SHAPE),
            ((ADDR, 8192, 64), (ADDR + 64, 4096, 64), SHAPE),         # two strides in one range
            ((ADDR, (1 << 62), 64), (ADDR + 64, 4096, 64), SHAPE)]:
        assert call(a, b) == want, (a, b)
    assert call((ADDR, 0, 64), (ADDR + 64, 0, 64), blocks=1) == NULL
    assert call((ADDR, 0, 64), (ADDR + 60, 0, 64), blocks=1) == SHAPE
