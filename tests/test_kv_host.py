"""Host-side checks of the cache's and the attention's entry points (no GPU needed): sizes, structs, refusals."""
import ctypes

import pytest
import torch

import gemm_dequant_gemv_q8_b200 as q
import kv_reference as ref
from gemm_dequant_gemv_q8_b200 import build as qbuild

# as in test_abi.py: made-up device addresses only where no kernel can launch
made_up_addresses = pytest.mark.skipif(torch.cuda.is_available(),
                                       reason="made-up device addresses: run only where no kernel can launch")
P = ctypes.c_void_p
ARG, UNSUP, ALIGN, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.lib()


def test_sizes(lib):
    assert q.qlin_kv_cache_bytes(10, 16, 8, 128) == 10 * 8 * 16 * 144
    assert q.qlin_kv_cache_bytes(3, 256, 1, 64) == 3 * 256 * 72
    for bad in ((0, 16, 8, 128), (10, 8, 8, 128), (10, 48, 8, 128), (10, 512, 8, 128), (10, 16, 0, 128), (10, 16, 1025, 128),
                (10, 16, 8, 96), (10, 16, 8, 256), (1 << 27, 16, 8, 128)):
        assert q.qlin_kv_cache_bytes(*bad) == 0, bad
    assert ctypes.sizeof(q.KVCacheDesc) == 40 and ctypes.sizeof(q.QKParams) == 48


def cache(data=0x100000, n_pages=10, page=16, Hkv=2, D=64, ks=1.0, vs=1.0):
    return q.KVCacheDesc(data, n_pages, page, Hkv, D, ks, vs)


def params(qw=0x200000, kw=0x200100, cs=0x300000, n_pos=100, rot=64, flags=0, eps=1e-6):
    return q.QKParams(qw, kw, cs, n_pos, rot, flags, eps)


def rope(lib, x=0x400000, xdt=0, T=4, ldx=384, Hq=4, Hkv=2, D=64, p=None, pos=0x500000, qo=0x600000, ldq=256, k=0x700000,
         ldk=128, ydt=0, flags=0, ws=0x800000, n=256):
    p = params() if p is None else p
    return lib.qlin_qk_norm_rope(P(x), xdt, T, ldx, Hq, Hkv, D, ctypes.addressof(p), P(pos), P(qo), ldq, P(k), ldk, ydt, flags,
                                 P(ws), n, None)


def append(lib, c=None, x=0x400000, xdt=0, T=4, ldx=512, Hq=4, p=None, pos=0x500000, slots=0x510000, qo=0x600000, ldq=256,
           flags=0, ws=0x800000, n=256):
    c, p = cache() if c is None else c, params() if p is None else p
    return lib.qlin_kv_append(ctypes.addressof(c), P(x), xdt, T, ldx, Hq, ctypes.addressof(p), P(pos), P(slots), P(qo), ldq, flags,
                              P(ws), n, None)


def gather(lib, c=None, T=4, slots=0x500000, k=0x600000, v=0x700000, ydt=0, ws=0x800000, n=256):
    c = cache() if c is None else c
    return lib.qlin_kv_gather(ctypes.addressof(c), T, P(slots), P(k), P(v), ydt, P(ws), n, None)


def attn(lib, c=None, qq=0x400000, ldq=256, table=0x500000, ldb=8, pages=8, lens=0x510000, cu=0x520000, B=2, max_q=1, total=2,
         Hq=4, scale=0.1, window=0, out=0x600000, ldo=256, flags=0, ws=0x800000, n=1 << 40):
    c = cache() if c is None else c
    return lib.qlin_attn_kv4(ctypes.addressof(c), P(qq), ldq, P(table), ldb, pages, P(lens), P(cu), B, max_q, total, Hq, scale,
                             window, P(out), ldo, flags, P(ws), n, None)


BAD_CACHES = [(dict(data=0), ARG), (dict(data=0x100010), ALIGN), (dict(n_pages=0), ARG), (dict(page=24), ARG),
              (dict(Hkv=0), ARG), (dict(D=80), UNSUP), (dict(ks=0.0), ARG), (dict(vs=-1.0), ARG),
              (dict(ks=float("nan")), ARG), (dict(vs=float("inf")), ARG)]


@made_up_addresses
def test_norm_rope_refusals(lib):
    for kw, want in [(dict(x=0), ARG), (dict(xdt=2), ARG), (dict(ydt=5), ARG), (dict(T=-1), ARG), (dict(T=1 << 21), ARG),
                     (dict(ldx=383), ARG), (dict(ldx=386), ALIGN), (dict(xdt=1, ldx=388), ALIGN), (dict(x=0x400008), ALIGN),
                     (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(D=96), UNSUP), (dict(D=0), ARG), (dict(qo=0), ARG),
                     (dict(ldq=252), ARG), (dict(ldq=258), ALIGN), (dict(qo=0x600004), ALIGN), (dict(k=0), ARG),
                     (dict(ldk=64), ARG), (dict(flags=1), ARG), (dict(ws=0), WS), (dict(n=255), WS), (dict(ws=0x800010), ALIGN),
                     (dict(pos=0), ARG), (dict(pos=0x500002), ALIGN), (dict(p=params(rot=8)), ARG),
                     (dict(p=params(rot=80)), ARG), (dict(p=params(rot=-16)), ARG), (dict(p=params(flags=2)), ARG),
                     (dict(p=params(cs=0)), ARG), (dict(p=params(n_pos=0)), ARG), (dict(p=params(eps=-1.0)), ARG),
                     (dict(p=params(eps=float("nan"))), ARG), (dict(p=params(qw=0x200004)), ALIGN),
                     (dict(p=params(cs=0x300008)), ALIGN)]:
        assert rope(lib, **kw) == want, kw
    assert rope(lib, T=0) == 0  # nothing to do


@made_up_addresses
def test_append_and_gather_refusals(lib):
    for kw, want in BAD_CACHES:
        assert append(lib, c=cache(**kw)) == want, kw
        assert gather(lib, c=cache(**kw)) == want, kw
    for kw, want in [(dict(x=0), ARG), (dict(xdt=3), ARG), (dict(T=-1), ARG), (dict(ldx=511), ARG), (dict(ldx=514), ALIGN),
                     (dict(Hq=-1), ARG), (dict(slots=0), ARG), (dict(slots=0x510001), ALIGN), (dict(ldq=250), ARG),
                     (dict(qo=0x600008), ALIGN), (dict(ldq=260), ALIGN), (dict(flags=1), ARG), (dict(ws=0), WS),
                     (dict(n=0), WS), (dict(p=params(rot=24)), ARG)]:
        assert append(lib, **kw) == want, kw
    for kw, want in [(dict(T=-1), ARG), (dict(slots=0), ARG), (dict(k=0), ARG), (dict(v=0), ARG), (dict(ydt=2), ARG),
                     (dict(k=0x600004), ALIGN), (dict(ws=0), WS), (dict(n=100), WS)]:
        assert gather(lib, **kw) == want, kw
    assert append(lib, T=0) == 0 and gather(lib, T=0) == 0


@made_up_addresses
def test_attention_refusals(lib):
    for kw, want in BAD_CACHES:
        assert attn(lib, c=cache(**kw)) == want, kw
    for kw, want in [(dict(qq=0), ARG), (dict(out=0), ARG), (dict(table=0), ARG), (dict(lens=0), ARG), (dict(cu=0), ARG),
                     (dict(ldq=255), ARG), (dict(ldq=260), ALIGN), (dict(qq=0x400008), ALIGN), (dict(ldo=128), ARG),
                     (dict(out=0x600002), ALIGN), (dict(ldb=7), ARG), (dict(pages=0), ARG), (dict(pages=1 << 27, ldb=1 << 27), ARG),
                     (dict(B=0), ARG), (dict(B=1025), ARG), (dict(max_q=0), ARG), (dict(total=-1), ARG), (dict(Hq=3), ARG),
                     (dict(Hq=0), ARG), (dict(Hq=130, ldq=8320, ldo=8320), UNSUP), (dict(window=-1), ARG),
                     (dict(scale=float("inf")), ARG), (dict(scale=2e38), ARG), (dict(scale=1e30, c=cache(ks=1e10)), ARG),
                     (dict(pages=(1 << 22) + 1, ldb=1 << 23), ARG), (dict(flags=1), ARG), (dict(ws=0), WS), (dict(n=8), WS),
                     (dict(ws=0x800080), ALIGN), (dict(table=0x500002), ALIGN)]:
        assert attn(lib, **kw) == want, kw
    assert attn(lib, total=0) == 0


def test_binding_refuses_host_tensors():
    with pytest.raises(TypeError):
        q.KVCache(torch.zeros(2304, dtype=torch.uint8), 16, 1, 128)
    with pytest.raises(q.QlinError):
        q.kv_cache(1, 17, 1, 128)
    with pytest.raises(TypeError):
        q.qlin_qk_norm_rope(torch.zeros(1, 192), 2, 1, 64)


# ----------------------------------------------------------------------------- the plain forms themselves
def test_reference_layout_is_one_layout():
    # the whole-cache writer and the slot writer of the plain forms lay the same tokens alike
    g = torch.Generator()
    g.manual_seed(1)
    page, Hkv, D = 32, 2, 64
    c, k, v = ref.random_cache(2, page, Hkv, D, g)
    d = torch.zeros_like(c)
    kc, kb = ref.quantize(k.float(), 1.0)
    vc, vb = ref.quantize(v.float(), 1.0)
    ref.put(d, page, Hkv, D, torch.arange(2 * page), kc, kb, vc, vb)
    kk, vv = ref.values(kc, kb), ref.values(vc, vb)
    assert torch.equal(kk, k) and torch.equal(vv, v)  # values quantize to themselves
    groups = d.view(2, Hkv, page // 16, 18 * D)
    for slot, h, e in ((0, 0, 0), (17, 1, 33), (63, 0, 63), (40, 1, 16)):
        gr, r = groups[slot // page, h, slot % page // 16], slot % 16
        code = int(gr[r * (D // 2) + e // 2]) >> (4 * (e % 2)) & 15
        s = gr[8 * D + r * (D // 16) + e // 16].view(torch.float8_e4m3fn).double()
        assert float(ref.E2M1[code] * s) == float(k[slot, h, e])
        code = int(gr[9 * D + e // 16 * 128 + r * 8 + e % 16 // 2]) >> (4 * (e % 2)) & 15
        s = gr[17 * D + e // 16 * 16 + r].view(torch.float8_e4m3fn).double()
        assert float(ref.E2M1[code] * s) == float(v[slot, h, e])


def test_reference_code_rounding_ties_to_even():
    x = torch.zeros(1, 16)
    x[0, :10] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.75, -0.25])
    codes, s = ref.quantize(x, 1.0)
    assert s.view(torch.float8_e4m3fn).float().item() == 1.0
    assert codes[0, :10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 10, 8]
