"""Edges of the cache's and the attention's calls: far tails of a softmax, scores near the limits of 32 bits, NaN and
junk in the cache, the range of the norms, pages that are missing, every token counted once, mixed batches, the largest sizes."""
import math

import pytest
import torch

import gemm_dequant_gemv_q8_b200 as q
import kv_reference as ref
from test_kv_attn_gpu import BF16, F32, attn_case, check_attn, gen, rope_tol, run_attn

pytestmark = pytest.mark.gpu


def exact_cache(k, v, page):
    """A cache of one sequence whose token t has the key k[t] and the value v[t], (L, Hkv, D) each of exact NVFP4 values
    (0 and 6, or 4 beside a 6), at slots 0 .. L - 1."""
    L, Hkv, D = k.shape
    cache = q.kv_cache(-(-L // page), page, Hkv, D)
    for t0 in range(0, L, 1 << 18):
        x = torch.cat([k[t0:t0 + (1 << 18)].flatten(1), v[t0:t0 + (1 << 18)].flatten(1)], 1)
        q.qlin_kv_append(cache, x, 0, None, torch.arange(t0, t0 + len(x), dtype=torch.int32, device="cuda"))
    return cache


def call(cache, L, nq, Hq, B=1, scale=None, query=None, window=0):
    """B sequences over the same pages, nq queries each, all alike: `query` gives a query's values, 0 elsewhere."""
    D, n = cache.D, -(-L // cache.page)
    qs = torch.zeros(B * nq, Hq, D, dtype=BF16, device="cuda")
    for d, x in (query or {}).items():
        qs[..., d] = x
    table = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, n).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * nq
    ws = q.workspace(q.qlin_attn_kv4_workspace_bytes(cache, B, nq, Hq))
    o = q.qlin_attn_kv4(cache, qs, table, lens, cu, nq, scale, window=window, ws=ws)
    assert q.qlin_ws_status(ws) == 0
    return o


@pytest.mark.parametrize("octaves", [18.0, 22.5, 25.5, 27.0])
@pytest.mark.parametrize("L,B,nq,Hkv", [(65536, 256, 1, 8), (65536, 1, 8192, 8), (131072, 1, 1, 1)])
def test_a_tail_far_below_the_largest_score_keeps_its_mass(L, B, nq, Hkv, octaves):
    # The first token takes nearly all and has the value 0; the others, 6 each, lie `octaves` below it.  Query at place p:
    # 6 p 2^-octaves / (1 + p 2^-octaves).
    D, page = 64, 64
    k, v = torch.zeros(L, Hkv, D, device="cuda"), torch.full((L, Hkv, D), 6.0, device="cuda")
    k[0, :, 0], v[0] = 6, 0
    scale = octaves * math.log(2) / 6
    o = call(exact_cache(k, v, page), L, nq, Hkv, B, scale, {0: 1.0}).double().cpu()
    p = torch.arange(L - nq, L, dtype=torch.float64).repeat(B)[:, None, None]
    r = p * 2.0 ** -octaves
    want = (6 * r / (1 + r)).expand_as(o)
    A = octaves * math.log(2)
    e = 2 * (2 * D + 4) * 2.0 ** -24 * A
    rel = 2 * (math.expm1(e) + 2.0 ** -21) + 2.0 ** -11 + (4 * L + 32) * 2.0 ** -24
    tol = want * rel + 6 * p * 2.0 ** -32
    tol = tol + 2.0 ** -8 * (want + tol)
    err = (o - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("nq", [1, 70])
def test_scores_of_a_hundred_million(nq):
    # Between 2^27 and 2^28 a score rises by one step of its last bit, 16, whose half is 8.  All values are 6, and so is the
    # output, whatever the weights.
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    for i in range(100):  # a scale that puts the two scores at odd and even last bits, with the kernels' roundings
        scale = f(1.5 * 2.0 ** 27 / 1.4426950408889634 / 6 * (1 + i * 2.0 ** -22))
        rs = scale * f(1.4426950408889634) * f(2.0 ** -14)
        lo, hi = f(6 * 2.0 ** 14) * rs, f(6 * 2.0 ** 14 + 2.0 ** -7) * rs
        if hi - lo == 16 and lo + 8 == hi:
            break
    assert hi - lo == 16 and lo + 8 == hi
    D, page, L, B = 64, 64, 4096, 64
    k, v = torch.zeros(L, 1, D, device="cuda"), torch.full((L, 1, D), 6.0, device="cuda")
    k[..., 0] = k[..., 17] = 6
    k[..., 16] = torch.where(torch.arange(L, device="cuda") // 512 % 2 == 1, 4.0, 0.0)[:, None]
    cache = exact_cache(k, v, page)
    o = call(cache, L, nq, 1, B, scale.item(), {0: 1.0, 16: 2.0 ** -23})
    assert (o == 6).all()


@pytest.mark.parametrize("nq", [1, 70])
@pytest.mark.parametrize("vs", [2.0 ** -120, 2.0 ** -126, 2.0 ** -136])
def test_the_smallest_value_scales(nq, vs):
    # V is 6 * 448 everywhere, the largest value of the cache, so the output is that times the scale: a normal number in bf16
    # although the scale over the softmax sum is none in fp32.
    D, page, L = 64, 64, 30000
    v = torch.full((L, 2, D), 6.0 * 448, device="cuda")
    cache = exact_cache(torch.zeros_like(v), v, page)
    small = q.KVCache(cache.data, page, 2, D, 1.0, vs)
    o = call(small, L, nq, 4).double()
    want = 6 * 448 * vs
    assert ((o - want).abs() <= (2.0 ** -8 + 8 * 2.0 ** -24) * want).all()


def test_rotation_without_a_table_is_refused():
    D, page = 64, 16
    x = torch.randn(3, 4 * D, generator=gen(1)).cuda()
    pos = torch.arange(3, dtype=torch.int32).cuda()
    cache = q.kv_cache(1, page, 1, D)
    for f in (lambda r: q.qlin_qk_norm_rope(x, 2, 1, D, pos, None, rot=r), lambda r: q.qlin_kv_append(cache, x, 2, pos, pos, None, rot=r)):
        f(0)
        for r in (16, D, -16):
            with pytest.raises(q.QlinError) as e:
                f(r)
            assert e.value.status == 1


@pytest.mark.parametrize("xdt", [F32, BF16])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rot,inter", [(0, False), (128, False), (48, False), (64, True)])
def test_append_of_nan_leaves_finite_values(xdt, norm, rot, inter):
    T, Hq, Hkv, D, page = 9, 1, 2, 128, 16
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen(2))
    x[0] = float("nan")
    x[2, Hq * D:(Hq + Hkv) * D] = float("nan")
    x[4, -D:] = float("nan")
    x[5, -5] = float("nan")
    x[6, Hq * D + 7] = float("nan")
    x[7, Hq * D + 40] = float("inf")
    x[8, Hq * D + 32:Hq * D + 48] = -float("inf")
    cache = q.kv_cache(1, page, Hkv, D)
    cs = ref.table(T, rot).cuda() if rot else None
    w = torch.ones(D).cuda() if norm else None
    slots = torch.arange(T, dtype=torch.int32).cuda()
    q.qlin_kv_append(cache, x.to(xdt).cuda(), Hq, slots, slots, cs, w, w, flags=int(inter))
    k, v = q.qlin_kv_gather(cache, slots, ydt=q.QLIN_F32)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    assert (v[0] == 0).all() and (k[2] == 0).all() and (v[4, 1] == 0).all()  # blocks of nothing but NaN
    kc, kb = ref.quantize(x[[1, 3, 4, 5, 6, 7, 8]].to(xdt)[:, -2 * D:].double().view(-1, Hkv, D)[:, :1].float(), 1.0)
    assert torch.equal(v[[1, 3, 4, 5, 6, 7, 8]][:, :1].cpu(), ref.values(kc, kb).float())


def test_a_nan_token_of_a_prompt_leaves_the_queries_before_it():
    Hq, Hkv, D, page, T = 4, 2, 64, 16, 90
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen(3)).cuda()
    bad = x.clone()
    bad[70:] = float("nan")
    slots = torch.arange(96, dtype=torch.int32).cuda()
    w = torch.ones(D).cuda()
    outs = []
    for xi in (x, bad):
        cache = q.kv_cache(6, page, Hkv, D)
        qo = q.qlin_kv_append(cache, xi, Hq, None, slots[:T], None, w, w)
        for nq in (T, 24):
            outs.append(q.qlin_attn_kv4(cache, qo[T - nq:], torch.arange(6, dtype=torch.int32)[None].cuda(),
                                        torch.tensor([T], dtype=torch.int32).cuda(), torch.tensor([0, nq], dtype=torch.int32).cuda(), nq))
    assert torch.equal(outs[0][:70], outs[2][:70]) and torch.equal(outs[1][:4], outs[3][:4])


@pytest.mark.parametrize("nq", [1, 5, 70])
@pytest.mark.parametrize("window", [1, 40, 300])
def test_attention_uses_nothing_before_the_window(nq, window):
    # places that no query sees hold anything, in groups and pages with others that are seen too
    lens, Hq, Hkv, D, page = [700, 333, 128], 8, 2, 128, 64
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq] * 3, Hq, Hkv, D, page, 86)
    want, _ = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    pages = c.view(-1, Hkv, page // 16, 18 * D)
    for b, L in enumerate(lens):
        for t in range(max(0, L - nq - window + 1)):
            gr, r = pages[table[b, t // page], :, t % page // 16], t % 16
            gr[:, 8 * D + r * (D // 16):8 * D + (r + 1) * (D // 16)] = 0x7F
            gr[:, r * (D // 2):(r + 1) * (D // 2)] = 0xA5
            gr[:, 17 * D + r::16] = 0xFF
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 0 and torch.equal(o, want)


RANGE = [(F32, 0.0, 2.0 ** 62), (F32, 1e-6, 2.0 ** 100), (F32, 1e-6, 2.0 ** 126), (F32, 0.0, 2.0 ** -70), (F32, 0.0, 2.0 ** -130),
         (BF16, 0.0, 2.0 ** 64), (BF16, 0.0, 2.0 ** -80), (F32, 1e-38, 2.0 ** -64), (F32, 1e38, 2.0 ** 63), (F32, 3e38, 1.0)]


@pytest.mark.parametrize("xdt,eps,size", RANGE)
@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, True), (128, 16, False)])
def test_norms_over_the_whole_range(xdt, eps, size, D, rot, inter):
    T, Hq, Hkv = 7, 5, 2
    g = gen(4)
    x = torch.randn(T, (Hq + Hkv) * D, generator=g)
    x[:, :3 * D] *= size / 4
    x[:, (Hq + 1) * D:] *= size / 4
    x = x.to(xdt)
    assert torch.isfinite(x).all()
    w = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)]
    pos, cs = torch.arange(T, dtype=torch.int32), ref.table(T, rot)
    qo, ko = q.qlin_qk_norm_rope(x.cuda(), Hq, Hkv, D, pos.cuda(), cs.cuda(), w[0].cuda(), w[1].cuda(), eps, flags=int(inter), ydt=q.QLIN_F32)
    xd = x.double().view(T, Hq + Hkv, D)
    for got, part, wt in ((qo, xd[:, :Hq], w[0]), (ko, xd[:, Hq:], w[1])):
        y, A = ref.norm_rope(part, wt, eps, cs, pos, rot, inter)
        assert ((got.cpu().double() - y).abs() <= rope_tol(y, A, F32)).all()
    # in place: heads that are written late are read first
    xc, dt = x.cuda(), q.QLIN_F32 if xdt == F32 else q.QLIN_BF16
    args = (Hq, Hkv, D, pos.cuda(), cs.cuda(), w[0].cuda(), w[1].cuda(), eps)
    want = torch.cat([t.flatten(1) for t in q.qlin_qk_norm_rope(xc, *args, flags=int(inter), ydt=dt)], 1)
    q.qlin_qk_norm_rope(xc, *args, flags=int(inter), ydt=dt, q=xc[:, :Hq * D], k=xc[:, Hq * D:])
    assert torch.equal(xc, want)


def masked_attention(qs, k, v, L, scale, valid, window=0):
    """ref.attention with a mask of a sequence's places beside the causal one, a row at a time: (out, tol)."""
    n, Hq, D = qs.shape
    G = Hq // k.shape[1]
    out, tol = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    for i in range(n):
        p = L - n + i
        idx = torch.arange(max(0, p - window + 1) if window else 0, p + 1)
        idx = idx[valid[idx]]
        if len(idx) == 0:
            continue
        o, tp, ts, tv = ref.attention(qs[i:i + 1].double(), k[idx], v[idx], len(idx), scale)
        out[i], tol[i] = o[0], ref.attention_tol(o, tp, ts, tv, D, len(idx))[0]
    return out, tol


@pytest.mark.parametrize("nq,window", [(1, 0), (5, 0), (40, 0), (300, 0), (40, 200), (5, 90)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_attention_missing_pages_are_masked_places(nq, window, D, page):
    # Pages outside the cache in many tiles of a long context, in the first ones of another, and all of a third's: rows that
    # see nothing are zeros.
    lens, Hq, Hkv = [1900, 700, 310], 8, 2
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq] * 3, Hq, Hkv, D, page, 110)
    valid = [torch.ones(L, dtype=torch.bool) for L in lens]

    def drop(b, j, number):
        table[b, j] = number
        valid[b][j * page:(j + 1) * page] = False

    for j in range(0, -(-lens[0] // page), 3):
        drop(0, j, 10 ** 6 if j % 2 else -1 - j)
    for j in range(max(1, -(-(lens[1] - nq // 2) // page))):
        drop(1, j, len(c) // q.qlin_kv_cache_bytes(1, page, Hkv, D))  # the first number behind the cache
    for j in range(-(-lens[2] // page)):
        drop(2, j, -2 ** 31)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 1
    o = o.cpu().double()
    for b, L in enumerate(lens):
        want, tol = masked_attention(qs[b], ks[b], vs[b], L, D ** -0.5, valid[b], window)
        got = o[cu[b]:cu[b + 1]]
        assert ((got - want).abs() <= tol).all(), (b, float(((got - want).abs() - tol).max()))


@pytest.mark.parametrize("nq", [1, 3, 16, 64, 300])
@pytest.mark.parametrize("L,Hq,Hkv,D,page,window", [(30000, 8, 4, 64, 64, 0), (100001, 4, 4, 128, 16, 0), (5001, 32, 2, 64, 128, 0),
                                                    (40000, 8, 1, 128, 256, 17777), (1000, 24, 8, 64, 32, 0)])
def test_every_token_counts_once(nq, L, Hq, Hkv, D, page, window):
    # All scores are 0, so every seen token has the same weight, and the tokens of group i (16 tokens) have the value 6 at
    # place i % D: an output value is 6 times the share of the tokens whose value it is.  The sums are exact (whole multiples of
    # one power of two, below 2^24 of them); the quotient, the product with it and the output are rounded (2^-24 each for the
    # first two, at most 2^-8).
    t = torch.arange(L, device="cuda")
    v = torch.zeros(L, Hkv, D, device="cuda")
    v[t, :, t // 16 % D] = 6
    cache = exact_cache(torch.zeros(L, Hkv, D, device="cuda"), v, page)
    o = call(cache, L, nq, Hq, window=window).double()
    counts = torch.zeros(L + 1, D, dtype=torch.float64, device="cuda")
    counts[1:] = (v[:, 0] / 6).double().cumsum(0)
    p = torch.arange(L - nq, L, device="cuda")
    first = (p - window + 1).clamp(min=0) if window else torch.zeros_like(p)
    want = 6 * (counts[p + 1] - counts[first]) / (p + 1 - first)[:, None]
    err = (o - want[:, None]).abs()
    assert (err <= (2.0 ** -8 + 4 * 2.0 ** -24) * want[:, None]).all(), float((err / want[:, None]).max())


MIXED = [  # queries, contexts, Hq, Hkv, D, page, window
    ([1] * 12 + [300, 1, 0, 1], [77 * (b + 1) for b in range(12)] + [900, 64, 5, 4000], 8, 2, 128, 64, 0),
    ([1, 1, 8, 1, 0, 2], [500, 3, 2000, 128, 40, 33], 8, 1, 64, 16, 0),       # few rows: one and eight row blocks' worth
    ([130, 1, 1, 130], [130, 2500, 1, 131], 4, 4, 64, 32, 100),
    ([1, 32, 1], [6000, 32, 700], 32, 8, 128, 16, 0),
]


@pytest.mark.parametrize("nqs,lens,Hq,Hkv,D,page,window", MIXED)
def test_single_tokens_beside_chunks(nqs, lens, Hq, Hkv, D, page, window):
    # every sequence of a call as it is alone
    c, table, ln, cu, qs, ks, vs = attn_case(lens, nqs, Hq, Hkv, D, page, 120)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5, window)


@pytest.mark.parametrize("nq,Hq,Hkv", [(1, 4, 1), (5, 8, 2), (200, 2, 1)])
@pytest.mark.parametrize("L", [2 ** 26, 2 ** 26 - 37])
def test_the_longest_context(nq, Hq, Hkv, L):
    # 2^26 tokens through a table that names eight pages again and again.  As above, but the sums of so many tokens are rounded:
    # each warp or part sums up to some 2^20 equal terms (below 2^24 of them: exact), then 2^12 at most are joined (2^-24 each).
    D, page, P = 64, 256, 8
    v = torch.zeros(P * page, Hkv, D, device="cuda")
    t = torch.arange(P * page, device="cuda")
    v[t, :, t // 16 % D] = 6
    cache = exact_cache(torch.zeros_like(v), v, page)
    n = -(-L // page)
    table = torch.randint(0, P, (n,), generator=gen(5), dtype=torch.int32)
    ws = q.workspace(q.qlin_attn_kv4_workspace_bytes(cache, 1, nq, Hq))
    o = q.qlin_attn_kv4(cache, torch.zeros(nq, Hq, D, dtype=BF16, device="cuda"), table[None].cuda(),
                        torch.tensor([L], dtype=torch.int32).cuda(), torch.tensor([0, nq], dtype=torch.int32).cuda(), nq, ws=ws)
    assert q.qlin_ws_status(ws) == 0
    o = o.double().cpu()
    ones = (v[:, 0].view(P, page, D) / 6).double().cpu()
    counts = torch.bincount(table[:n - 1].long(), minlength=P).double() @ ones.sum(1)
    for i in range(nq):
        seen = L - nq + i + 1
        want = 6 * (counts + ones[int(table[-1])][:seen - (n - 1) * page].sum(0)) / seen
        assert seen > (n - 1) * page and ((o[i] - want).abs() <= (2.0 ** -8 + 2.0 ** -12) * want).all()


def test_the_longest_chunk():
    # 2^20 queries over their own tokens: query i averages the first i + 1
    n, D, page = 1 << 20, 64, 256
    v = torch.zeros(n, 1, D, device="cuda")
    t = torch.arange(n, device="cuda")
    v[t, :, t // 16 % D] = 6
    cache = exact_cache(torch.zeros_like(v), v, page)
    o = call(cache, n, n, 1)[:, 0].double()
    want = 6 * (v[:, 0] / 6).double().cumsum(0) / (t + 1)[:, None]
    assert ((o - want).abs() <= (2.0 ** -8 + 2.0 ** -12) * want).all()


@pytest.mark.parametrize("nq", [1, 3, 40])
@pytest.mark.parametrize("G", [1, 2])
def test_the_most_heads(nq, G):
    Hq, Hkv, D, page = 1024, 1024 // G, 64, 16
    c, table, ln, cu, qs, ks, vs = attn_case([100, 37], [nq] * 2, Hq, Hkv, D, page, 130)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5)
