"""The 8-bit cache formats and dkv_kv_append reject bad arguments on the host,
before any CUDA call, so this runs without a GPU; and the plain forms that the
GPU tests compare with hold what defines them."""

import ctypes
import os
import subprocess

import pytest
import torch

import fp8_helpers as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def dkv():
    from decode_attention_paged_kv_gb300 import build as b
    b.build()
    import decode_attention_paged_kv_gb300 as m
    m.lib()
    return m


def _params(dkv, **kw):
    p = dkv._Params()
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim, p.seq_len, p.page_size = 2, 8, 2, 128, 1000, 16
    p.q_stride_b, p.q_stride_h, p.o_stride_b, p.o_stride_h = 8 * 128, 128, 8 * 128, 128
    p.scale = 0.088
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _kv(dkv, fmt, **kw):
    kv = dkv._KV()
    kv.format, kv.dtype, kv.data = fmt, 0, 4096
    eight = fmt in (dkv.DKV_KV_FP8, dkv.DKV_KV_FP8_PAGED)
    paged = fmt in (dkv.DKV_KV_PAGED, dkv.DKV_KV_FP8_PAGED)
    kv.stride_h = (16 if paged else 1000) * 128
    kv.stride_b = 2 * kv.stride_h
    if eight:
        kv.scale, kv.sstride_h, kv.sstride_b = 8192, 1 if paged else 63, 2 if paged else 126
    if paged:
        kv.block_table, kv.block_table_stride, kv.num_blocks = 1 << 14, 63, 200
    for k, v in kw.items():
        setattr(kv, k, v)
    return kv


@pytest.mark.parametrize("paged", [False, True])
def test_fp8_cache_validation(dkv, paged):
    L = dkv.lib()
    fmt = dkv.DKV_KV_FP8_PAGED if paged else dkv.DKV_KV_FP8
    p = _params(dkv)
    need = L.dkv_workspace_bytes_fp8(ctypes.byref(p), 0)
    need_sel = L.dkv_workspace_bytes_fp8(ctypes.byref(p), 8)
    assert need > 256 and need_sel > 256
    assert L.dkv_workspace_bytes_fp8(None, 0) == 0
    assert L.dkv_workspace_bytes_fp8(ctypes.byref(_params(dkv, head_dim=96)), 0) == 0
    ws, q, out = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 16), ctypes.c_void_p(1 << 17)

    def full(K, V, size=need, pp=p):
        return L.dkv_decode_attn_full(ctypes.byref(pp), q, ctypes.byref(K), ctypes.byref(V), out,
                                      2, ws, size, None)

    good = _kv(dkv, fmt)
    assert full(good, _kv(dkv, fmt), size=need - 1) == WORKSPACE
    assert full(_kv(dkv, fmt, scale=None), good) == NULL
    assert full(_kv(dkv, fmt, scale=8194), good) == ALIGN
    assert full(_kv(dkv, fmt, sstride_h=-1), good) == SHAPE
    assert full(_kv(dkv, fmt, stride_h=good.stride_h + 8), good) == ALIGN
    assert full(_kv(dkv, fmt, dtype=2), good) == DTYPE
    assert full(good, _kv(dkv, fmt, dtype=1)) == DTYPE          # K and V differ
    assert full(good, _kv(dkv, dkv.DKV_KV_DENSE)) == DTYPE
    if paged:
        assert full(_kv(dkv, fmt, block_table=None), good) == NULL
        assert full(good, _kv(dkv, fmt, num_blocks=199)) == SHAPE
        assert full(_kv(dkv, fmt, block_table_stride=62), good) == SHAPE
    # cross-step reuse and the token-level call take 16-bit caches only
    hb = L.dkv_hot_state_bytes(ctypes.byref(p))
    assert L.dkv_decode_attn_select_hot(
        ctypes.byref(p), q, ctypes.byref(good), ctypes.byref(good), q, q, 4, out, 2, None, ws, hb,
        1, ws, need_sel, None) == UNSUPPORTED
    assert L.dkv_decode_attn_topk_tokens(ctypes.byref(p), q, ctypes.byref(good),
                                         ctypes.byref(good), 4, out, 2, None, ws, 1 << 30,
                                         None) == DTYPE
    n = ctypes.c_int32(0)
    assert L.dkv_attn_ctas_per_sm(128, 2, fmt, 0, ctypes.byref(n)) == UNSUPPORTED


def _append(dkv, **kw):
    a = dkv._Append(2, 8, 2, 128, 1000, 4)
    a.k, a.v, a.q, a.q_out = 1 << 16, 1 << 17, 1 << 18, 1 << 19
    for t, h in (("k", 2), ("v", 2), ("q", 8), ("o", 8)):
        setattr(a, f"{t}_stride_h", 128)
        setattr(a, f"{t}_stride_t", 128 * h)
        setattr(a, f"{t}_stride_b", 128 * h * 4)
    a.rotary_dim, a.rope_len, a.cos, a.sin = 128, 1000, 1 << 20, 1 << 21
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("fmt", ["DENSE", "PAGED", "FP8", "FP8_PAGED"])
def test_append_validation(dkv, fmt):
    L = dkv.lib()
    f = getattr(dkv, "DKV_KV_" + fmt)
    kv = _kv(dkv, f)

    def call(K=None, V=None, ws=None, **kw):
        K, V = K or kv, V or kv
        # new_tokens = 0: a valid call launches nothing and returns OK
        return L.dkv_kv_append(ctypes.byref(_append(dkv, **({"new_tokens": 0} | kw))),
                               ctypes.byref(K), ctypes.byref(V), ws, None)

    assert call() == OK
    assert L.dkv_kv_append(None, ctypes.byref(kv), ctypes.byref(kv), None, None) == NULL
    assert call(num_q_heads=0, q=None, q_out=None) == OK
    assert call(rotary_dim=0, cos=None, sin=None, rope_len=0) == OK
    for bad in (dict(batch=0), dict(batch=65536), dict(num_kv_heads=0), dict(seq_len=0),
                dict(new_tokens=-1), dict(new_tokens=1001), dict(num_q_heads=-1),
                dict(rotary_dim=-16), dict(rotary_dim=144), dict(rotary_dim=24),
                dict(interleaved=2), dict(rope_len=0), dict(rope_len=999), dict(k_stride_t=-8),
                dict(o_stride_h=-8)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(cos=None),
                dict(sin=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(k=8), dict(v=24), dict(q=2), dict(q_out=4), dict(cos=4), dict(sin=8),
                dict(k_stride_t=132), dict(o_stride_b=4), dict(new_lens=2), dict(seq_lens=1),
                dict(ws=ctypes.c_void_p(8))):
        assert call(**bad) == ALIGN, bad
    assert call(head_dim=96) == UNSUPPORTED
    # written elements have places of their own
    assert call(new_tokens=2, o_stride_t=0) == SHAPE
    assert call(new_tokens=2, o_stride_h=64) == SHAPE
    assert call(K=_kv(dkv, f, stride_b=0)) == SHAPE
    assert call(V=_kv(dkv, f, stride_h=kv.stride_h // 2)) == SHAPE
    if "FP8" in fmt:
        assert call(K=_kv(dkv, f, sstride_h=0)) == SHAPE
        assert call(V=_kv(dkv, f, sstride_b=kv.sstride_b - 1)) == SHAPE
        assert call(K=_kv(dkv, f, scale=None)) == NULL
    assert call(V=_kv(dkv, f, dtype=1)) == DTYPE
    other = dkv.DKV_KV_DENSE if f != dkv.DKV_KV_DENSE else dkv.DKV_KV_PAGED
    assert call(V=_kv(dkv, other)) == DTYPE
    if "PAGED" in fmt:
        assert call(V=_kv(dkv, f, block_table=1 << 15)) == SHAPE
    q4 = _kv(dkv, dkv.DKV_KV_DENSE, format=dkv.DKV_KV_Q4G64, dtype=1, gmin=4096, gmax=4096)
    assert call(K=q4, V=q4) == UNSUPPORTED
    # more rows than one launch covers
    big = dict(new_tokens=1 << 30, seq_lens=4096, seq_len=1 << 30, k_stride_b=1 << 40,
               o_stride_b=1 << 40)
    wide = dict(stride_h=1 << 40, stride_b=1 << 41, block_table_stride=1 << 27,
                sstride_h=1 << 30, sstride_b=1 << 31)
    assert call(K=_kv(dkv, f, **wide), V=_kv(dkv, f, **wide), **big) == UNSUPPORTED


def test_append_struct_matches_header(dkv, tmp_path):
    fields = [n for n, _ in dkv._Append._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dkv.h"\nint main(void) {\n'
                   + '  printf("%zu\\n", sizeof(dkv_append));\n'
                   + "".join(f'  printf("%zu\\n", offsetof(dkv_append, {n}));\n' for n in fields)
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got[0] == ctypes.sizeof(dkv._Append)
    assert got[1:] == [getattr(dkv._Append, n).offset for n in fields]


def test_python_checks(dkv):
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    c = torch.zeros(2, 2, 40, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="scale must be"):
        dkv.kv_meta_build(dkv.Fp8Cache(c, torch.ones(2, 2, 2)))
    with pytest.raises(TypeError):
        dkv.kv_meta_build(dkv.Fp8Cache(c.view(torch.uint8), torch.ones(2, 2, 3)))
    with pytest.raises(ValueError, match="CUDA"):  # no CPU form
        dkv.kv_append(t(2, 1, 2, 64), t(2, 1, 2, 64), t(2, 2, 40, 64), t(2, 2, 40, 64))


def test_plain_forms():
    v = ref.e4m3_values()
    assert v[0x7E] == 448.0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6
    # the values are those of torch's type, and encode() rounds as it does
    c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert torch.equal(torch.nan_to_num(c.float(), 1e9).double(),
                       torch.nan_to_num(ref.TABLE, 1e9))
    x = torch.randn(20000, dtype=torch.float64) * torch.exp2(
        torch.randint(-12, 9, (20000,)).double())
    x = x.clamp(-448, 448)
    assert torch.equal(ref.encode(x).view(torch.uint8),
                       x.to(torch.float8_e4m3fn).view(torch.uint8))
    for dt in (torch.bfloat16, torch.float16):
        lo, hi = ref.EXP[dt]
        a = torch.tensor([0.0, 448.0, 448.0000001, 3.5, 3.6, 1e-30])
        s = ref.block_scale(a, dt)
        assert torch.all((s == 2.0 ** lo) | (a.double() > 448 * s / 2))
        assert torch.all((a.double() <= 448 * s) | (s == 2.0 ** hi))
        # every value of a block is exact in the 16-bit type
        for e in (lo, hi):
            w = ref.TABLE[~ref.TABLE.isnan()] * 2.0 ** e
            assert torch.equal(w.to(dt).double(), w)
    # the position rotation keeps lengths and turns relative angles
    import decode_attention_paged_kv_gb300 as m
    rope = m.rope_table(64, 32)
    x = torch.randn(64, 1, 64)
    for il in (False, True):
        y = ref.rotated(x, torch.arange(64), rope, il)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-5)
        assert torch.equal(y[..., 32:], x[..., 32:])
        assert torch.equal(y[0], x[0])
