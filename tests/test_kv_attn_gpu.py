"""The query / key norm and rotation, the append to the paged NVFP4 cache, its read-back and the attention over it,
against plain 64-bit forms (kv_reference.py), at the sizes, masks and layouts where they can go wrong."""
import pytest
import torch

import gemm_dequant_gemv_q8_b200 as q
import kv_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ----------------------------------------------------------------------------- norm and rotation
# 32-bit arithmetic: the sum of squares (13 roundings, halved by the root), root, quotient, two products, the
# rotation's two: 14 of them at most; 16 are allowed, of the magnitudes behind the value, and the output's own half step.
def rope_tol(y, A, dtype):
    t = 16 * 2.0 ** -24 * A
    return t + (torch.finfo(dtype).eps / 2) * (y.abs() + t) + 1e-38


ROPE = [  # T, Hq, Hkv, D, rot, interleaved, norm, x, y
    (1, 32, 8, 128, 128, False, True, F32, BF16),
    (3, 5, 1, 64, 64, True, True, F32, F32),
    (17, 3, 3, 128, 64, True, True, BF16, F32),
    (33, 6, 2, 64, 32, False, True, BF16, BF16),
    (129, 16, 4, 128, 16, False, False, F32, F32),
    (7, 1, 1, 64, 0, False, True, BF16, F32),
    (300, 9, 3, 128, 128, False, True, BF16, BF16),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm,xdt,ydt", ROPE)
def test_norm_rope(T, Hq, Hkv, D, rot, inter, norm, xdt, ydt):
    g = gen(T + D)
    extra = 8  # rows wider than the heads: a stride of their own
    x = (torch.randn(T, (Hq + Hkv) * D + extra, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(xdt)
    x[0] = 0  # a head of zeros: eps alone keeps it finite
    w = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    cs = ref.table(5000, rot) if rot else None
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ws = q.workspace(256)
    qo, ko = q.qlin_qk_norm_rope(x.cuda(), Hq, Hkv, D, pos.cuda(), cu(cs), cu(w[0]), cu(w[1]), 1e-6,
                                 flags=q.QLIN_ROPE_INTERLEAVED if inter else 0,
                                 ydt=q.QLIN_F32 if ydt == F32 else q.QLIN_BF16, ws=ws)
    assert q.qlin_ws_status(ws) == 0
    xd = x[:, :(Hq + Hkv) * D].double().view(T, Hq + Hkv, D)
    for got, part, wt in ((qo, xd[:, :Hq], w[0]), (ko, xd[:, Hq:], w[1])):
        y, A = ref.norm_rope(part, wt, 1e-6, cs, pos, rot, inter)
        assert ((got.cpu().double() - y).abs() <= rope_tol(y, A, ydt)).all()


def test_norm_rope_in_place_and_strided_outputs():
    T, Hq, Hkv, D = 37, 6, 2, 64
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen(5)).cuda()
    pos, cs = torch.arange(T, dtype=torch.int32).cuda(), ref.table(64, D).cuda()
    w = torch.ones(D).cuda()
    a, b = q.qlin_qk_norm_rope(x, Hq, Hkv, D, pos, cs, w, w, ydt=q.QLIN_F32)
    buf = torch.full((T, (Hq + Hkv) * D + 12), 7.0, device="cuda")
    q.qlin_qk_norm_rope(x, Hq, Hkv, D, pos, cs, w, w, ydt=q.QLIN_F32, q=buf[:, :Hq * D],
                        k=buf[:, Hq * D:(Hq + Hkv) * D])
    assert torch.equal(buf[:, :Hq * D], a.flatten(1)) and torch.equal(buf[:, Hq * D:(Hq + Hkv) * D], b.flatten(1))
    assert (buf[:, (Hq + Hkv) * D:] == 7).all()
    v = x[:, (Hq + Hkv) * D:].clone()
    q.qlin_qk_norm_rope(x, Hq, Hkv, D, pos, cs, w, w, ydt=q.QLIN_F32, q=x[:, :Hq * D], k=x[:, Hq * D:(Hq + Hkv) * D])
    assert torch.equal(x[:, :Hq * D], a.flatten(1)) and torch.equal(x[:, Hq * D:(Hq + Hkv) * D], b.flatten(1))
    assert torch.equal(x[:, (Hq + Hkv) * D:], v)


def test_norm_rope_bad_positions_leave_their_rows():
    T, Hq, Hkv, D = 5, 2, 1, 64
    x = torch.randn(T, (Hq + Hkv) * D, generator=gen(6)).cuda()
    cs = ref.table(10, D).cuda()
    pos = torch.tensor([0, -1, 9, 10, 3], dtype=torch.int32).cuda()
    qo = torch.full((T, Hq, D), 7.0, device="cuda")
    ko = torch.full((T, Hkv, D), 7.0, device="cuda")
    ws = q.workspace(256)
    q.qlin_qk_norm_rope(x, Hq, Hkv, D, pos, cs, ydt=q.QLIN_F32, q=qo, k=ko, ws=ws)
    assert q.qlin_ws_status(ws) == 1 and q.qlin_ws_status(ws) == 0
    assert (qo[[1, 3]] == 7).all() and (ko[[1, 3]] == 7).all()
    good = [0, 2, 4]
    a, b = q.qlin_qk_norm_rope(x[good].contiguous(), Hq, Hkv, D, pos[good].contiguous(), cs, ydt=q.QLIN_F32)
    assert torch.equal(qo[good], a) and torch.equal(ko[good], b)


# ----------------------------------------------------------------------------- append and read-back
APPEND = [  # T, Hq, Hkv, D, rot, interleaved, norm, x, page, ks, vs
    (1, 32, 8, 128, 128, False, True, F32, 16, 1.0, 1.0),
    (5, 0, 2, 64, 32, True, True, F32, 32, 0.37, 2.5),
    (45, 4, 4, 128, 64, True, False, BF16, 64, 0.01, 0.3),
    (130, 3, 1, 64, 64, False, True, BF16, 128, 3.0, 1.0),
    (77, 16, 8, 128, 0, False, True, F32, 256, 1.0, 0.125),
    (33, 4, 2, 64, 48, False, True, F32, 16, 1.0, 1.0),    # an odd number of blocks rotated, by halves
    (21, 2, 3, 128, 16, False, True, BF16, 32, 0.7, 1.0),
    (9, 1, 5, 128, 112, False, False, F32, 16, 1.0, 1.0),
    (12, 2, 2, 128, 48, True, True, F32, 16, 1.0, 1.0),
]


def append_inputs(T, Hq, Hkv, D, rot, xdt, norm, page, seed):
    g = gen(seed)
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g) * torch.exp(torch.randn((Hq + 2 * Hkv) * D, generator=g))
    x[T // 2, -D:-D + 16] = 0      # a block of zeros: scale 0, codes 0
    x[0, -16:] *= 1e4              # a block that saturates its scale
    x[T // 3, -32:-16] *= 1e-4     # a block below the smallest scale's reach
    x = x.to(xdt)
    w = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    pos = torch.randint(0, 3000, (T,), generator=g, dtype=torch.int32)
    n_pages = T // page + 3
    slots = torch.randperm(n_pages * page, generator=g)[:T].int()
    return x, w, pos, ref.table(3000, rot) if rot else None, n_pages, slots


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm,xdt,page,ks,vs", APPEND)
def test_append_and_gather(T, Hq, Hkv, D, rot, inter, norm, xdt, page, ks, vs):
    x, w, pos, cs, n_pages, slots = append_inputs(T, Hq, Hkv, D, rot, xdt, norm, page, T + page)
    if T > 4:
        slots[3] = -1
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    before = torch.randint(0, 256, (q.qlin_kv_cache_bytes(n_pages, page, Hkv, D),), generator=gen(9), dtype=torch.uint8)
    cache = q.kv_cache(n_pages, page, Hkv, D, ks, vs)
    cache.data.copy_(before)
    ws = q.workspace(256)
    qo = torch.full((T, max(Hq, 1), D), 7.0, dtype=BF16, device="cuda")[:, :Hq]
    q.qlin_kv_append(cache, x.cuda(), Hq, pos.cuda(), slots.cuda(), cu(cs), cu(w[0]), cu(w[1]), 1e-6,
                     flags=q.QLIN_ROPE_INTERLEAVED if inter else 0, q=qo if Hq else None, ws=ws)
    assert q.qlin_ws_status(ws) == 0
    xd = x.double().view(T, Hq + 2 * Hkv, D)
    live = slots >= 0
    if Hq:
        y, A = ref.norm_rope(xd[:, :Hq], w[0], 1e-6, cs, pos, rot, inter)
        got = qo.cpu().double()
        assert ((got - y).abs() <= rope_tol(y, A, BF16))[live].all()
        assert (got[~live] == 7).all()
    k, _ = ref.norm_rope(xd[:, Hq:Hq + Hkv], w[1], 1e-6, cs, pos, rot, inter)
    kc, kb = ref.quantize(k.float(), ks)
    vc, vb = ref.quantize(xd[:, Hq + Hkv:].float(), vs)
    want = before.clone()
    ref.put(want, page, Hkv, D, slots, kc, kb, vc, vb)
    assert torch.equal(cache.data.cpu(), want)  # every other byte as it was
    for dt, ydt in ((q.QLIN_F32, F32), (q.QLIN_BF16, BF16)):
        gk, gv = q.qlin_kv_gather(cache, slots.cuda(), ydt=dt, ws=ws)
        assert torch.equal(gk.cpu()[live], ref.values(kc, kb, ks).float().to(ydt)[live])
        assert torch.equal(gv.cpu()[live], ref.values(vc, vb, vs).float().to(ydt)[live])
    assert q.qlin_ws_status(ws) == 0


def test_append_alone_gives_the_chunks_bytes():
    T, Hq, Hkv, D, page = 40, 4, 2, 128, 16
    x, w, pos, cs, n_pages, slots = append_inputs(T, Hq, Hkv, D, D, F32, True, page, 3)
    xc, pc, sc, w, cs = x.cuda(), pos.cuda(), slots.cuda(), [t.cuda() for t in w], cs.cuda()
    a, b = q.kv_cache(n_pages, page, Hkv, D), q.kv_cache(n_pages, page, Hkv, D)
    qa = q.qlin_kv_append(a, xc, Hq, pc, sc, cs, *w)
    qb = torch.cat([q.qlin_kv_append(b, xc[t:t + 1], Hq, pc[t:t + 1], sc[t:t + 1], cs, *w) for t in range(T)])
    assert torch.equal(a.data, b.data) and torch.equal(qa, qb)


def test_append_edge_values():
    # exact ties of the code's and the scale's rounding, infinities, the largest finite value, both zeros
    D, page = 64, 16
    x = torch.zeros(8, 2 * D)
    x[0, D:D + 16] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25])
    x[1, D:D + 16] = x[0, D:D + 16] * 17 / 16    # the scale is a tie of E4M3
    x[2, D:D + 16] = x[0, D:D + 16] * 2.0 ** -10  # the scale is half the smallest
    x[3, D:D + 16] = x[0, D:D + 16] * 3e38 / 6
    x[4, D] = float("inf")
    x[4, D + 1] = -1.0
    x[5, D] = -0.0
    x[6, D:] = 1e-40
    x[7, :D] = torch.arange(D) - 31.0
    cache = q.kv_cache(1, page, 1, D)
    slots = torch.arange(8, dtype=torch.int32)
    q.qlin_kv_append(cache, x.cuda(), 0, None, slots.cuda(), None, q=None)
    kc, kb = ref.quantize(x[:, :D].view(8, 1, D), 1.0)
    vc, vb = ref.quantize(x[:, D:].view(8, 1, D), 1.0)
    k, v = q.qlin_kv_gather(cache, slots.cuda(), ydt=q.QLIN_F32)
    assert torch.equal(k.cpu(), ref.values(kc, kb).float())
    assert torch.equal(v.cpu()[[0, 1, 2, 3, 5, 6, 7]], ref.values(vc, vb).float()[[0, 1, 2, 3, 5, 6, 7]])
    assert v[4, 0, 0].item() == 6 * 448 and v[4, 0, 1].item() == 0


def test_append_bad_slots_and_positions():
    T, Hq, Hkv, D, page = 6, 1, 1, 64, 16
    x = torch.randn(T, 3 * D, generator=gen(8)).cuda()
    cs = ref.table(10, D).cuda()
    cache = q.kv_cache(2, page, Hkv, D)
    pos = torch.tensor([0, 1, 2, 10, 4, -3], dtype=torch.int32).cuda()
    slots = torch.tensor([0, 32, -2, 3, 31, 5], dtype=torch.int32).cuda()
    ws = q.workspace(256)
    qo = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda")
    q.qlin_kv_append(cache, x, Hq, pos, slots, cs, q=qo, ws=ws)
    assert q.qlin_ws_status(ws) == 1
    assert (qo[[1, 2, 3, 5]] == 7).all() and (qo[[0, 4]] != 7).any()
    want = q.kv_cache(2, page, Hkv, D)
    q.qlin_kv_append(want, x[[0, 4]].contiguous(), Hq, pos[[0, 4]].contiguous(), slots[[0, 4]].contiguous(), cs)
    assert torch.equal(cache.data, want.data)
    k, v = torch.full((T, Hkv, D), 7.0, device="cuda"), torch.full((T, Hkv, D), 7.0, device="cuda")
    q.qlin_kv_gather(cache, slots, k=k, v=v, ydt=q.QLIN_F32, ws=ws)
    assert q.qlin_ws_status(ws) == 1
    assert (k[[1, 2]] == 7).all() and (v[[1, 2]] == 7).all() and (k[[0, 4]] != 7).any()


# ----------------------------------------------------------------------------- attention
def attn_case(lens, nqs, Hq, Hkv, D, page, seed, spare=2, junk=True, k_size=1.0):
    """Sequences on random pages.  What lies behind each sequence's end is junk: NaN scales, any codes."""
    g = gen(seed)
    need = [-(-L // page) for L in lens]
    n_pages = sum(need) + spare
    cache, k, v = ref.random_cache(n_pages, page, Hkv, D, g, k_size=k_size)
    order = torch.randperm(n_pages, generator=g)
    width = max(max(need), 1) + 1
    table = torch.full((len(lens), width), n_pages - 1, dtype=torch.int32)
    at, ks, vs = 0, [], []
    c = cache.view(n_pages, Hkv, page // 16, 18 * D)
    used = set()
    for b, n in enumerate(need):
        ids = order[at:at + n]
        at += n
        table[b, :n] = ids.int()
        used |= set(ids.tolist())
        idx = (ids[:, None] * page + torch.arange(page)).flatten()[:lens[b]]
        ks.append(k[idx])
        vs.append(v[idx])
        if junk and lens[b] % page:
            last = c[ids[-1]]
            for t in range(lens[b] % page, page):
                gr, r = last[:, t // 16], t % 16
                gr[:, 8 * D + r * (D // 16):8 * D + (r + 1) * (D // 16)] = 0x7F
                gr[:, r * (D // 2):(r + 1) * (D // 2)] = 0xA5
                gr[:, 17 * D + r::16] = 0xFF
    if junk:
        for p in set(range(n_pages)) - used:
            c[p] = 0x7F
    qs = [(1.5 * torch.randn(n, Hq, D, generator=g)).bfloat16() for n in nqs]
    cu = torch.tensor([0] + torch.tensor(nqs).cumsum(0).tolist(), dtype=torch.int32)
    return cache, table, torch.tensor(lens, dtype=torch.int32), cu, qs, ks, vs


def run_attn(cache, page, Hkv, D, table, lens, cu, qs, max_q=None, scale=None, window=0, ks=1.0, vs=1.0, ws=None, out=None):
    kv = q.KVCache(dev_cache(cache), page, Hkv, D, ks, vs)
    qq = torch.cat(qs).cuda()
    mq = max(len(t) for t in qs) if max_q is None else max_q
    if ws is None:
        ws = q.workspace(q.qlin_attn_kv4_workspace_bytes(kv, len(lens), mq, qq.shape[1]))
    o = q.qlin_attn_kv4(kv, qq, table.cuda(), lens.cuda(), cu.cuda(), mq, scale, window=window, ws=ws, out=out)
    return o, q.qlin_ws_status(ws)


def dev_cache(cache):
    d = q._alloc_aligned(cache.numel(), "cuda")
    return d.copy_(cache)


def check_attn(o, lens, cu, qs, ks, vs, D, scale, window=0, kscale=1.0, vscale=1.0):
    o = o.cpu().double()
    for b, L in enumerate(lens.tolist()):
        out, tp, ts, tv = ref.attention(qs[b].double(), ks[b] * kscale, vs[b] * vscale, L, scale, window)
        got = o[cu[b]:cu[b + 1]]
        tol = ref.attention_tol(out, tp, ts, tv, D, L)
        err = (got - out).abs()
        assert (err <= tol + 1e-30).all(), (b, L, float((err / (tol + 1e-30)).max()))


DECODE = [  # lens, Hq, Hkv, D, page, window
    ([1], 1, 1, 64, 16, 0),
    ([1, 2, 15, 16, 17, 31, 32, 33], 8, 2, 128, 16, 0),
    ([63, 64, 65, 127, 128, 129, 0, 300], 6, 2, 64, 64, 0),
    ([1000, 3, 517], 32, 8, 128, 32, 0),
    ([2500], 5, 1, 128, 128, 0),
    ([700, 44], 16, 2, 64, 256, 0),
    ([900, 77, 1], 4, 4, 128, 16, 100),
    ([640, 641], 16, 1, 128, 64, 1),
    ([333, 12], 40, 2, 128, 16, 0),
    ([257], 64, 1, 64, 16, 33),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,window", DECODE)
def test_decode(lens, Hq, Hkv, D, page, window):
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [1] * len(lens), Hq, Hkv, D, page, Hq + D + page)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5, window)


LONG = [  # lens, queries, Hq, Hkv, D, page, window
    ([30000, 9000, 5, 0], 1, 32, 4, 128, 64, 0),    # whole CTAs for each segment
    ([20000, 31, 7000], 4, 8, 2, 64, 16, 0),
    ([30000, 9000], 1, 8, 8, 64, 256, 25000),
    ([2080] * 18, 1, 8, 4, 64, 32, 0),              # equal parts: the shares would need more CTAs
    ([6000 - 300 * b for b in range(9)], 1, 16, 8, 128, 16, 0),
]


@pytest.mark.parametrize("lens,nq,Hq,Hkv,D,page,window", LONG)
def test_decode_long(lens, nq, Hq, Hkv, D, page, window):
    nqs = [min(nq, L) if L else 1 for L in lens]
    c, table, ln, cu, qs, ks, vs = attn_case(lens, nqs, Hq, Hkv, D, page, 60 + len(lens))
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5, window)
    o2, _ = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert torch.equal(o, o2)


CHUNK = [  # lens, queries, Hq, Hkv, D, page, window
    ([2], [2], 2, 1, 64, 16, 0),
    ([40, 9, 200], [4, 3, 1], 8, 2, 128, 16, 0),
    ([100, 7], [5, 7], 6, 2, 64, 32, 0),
    ([128], [128], 4, 1, 128, 64, 0),
    ([129], [127], 4, 2, 128, 16, 0),
    ([513, 300, 64], [200, 300, 1], 8, 2, 128, 64, 0),
    ([700, 260], [257, 31], 6, 2, 64, 16, 0),
    ([600], [320], 5, 1, 128, 128, 0),
    ([640, 385], [300, 129], 8, 1, 64, 32, 70),
    ([900], [150], 3, 3, 128, 16, 333),
    ([400], [90], 64, 1, 64, 16, 0),
    ([50, 0, 3], [60, 4, 9], 4, 2, 128, 16, 0),   # more queries than tokens: the first see nothing
    ([333, 20], [0, 20], 8, 4, 128, 32, 0),       # a sequence without queries
]


@pytest.mark.parametrize("lens,nqs,Hq,Hkv,D,page,window", CHUNK)
def test_chunk(lens, nqs, Hq, Hkv, D, page, window):
    c, table, ln, cu, qs, ks, vs = attn_case(lens, nqs, Hq, Hkv, D, page, Hq + D + page + sum(nqs))
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5, window)


@pytest.mark.parametrize("nq", [1, 70])
def test_attention_scales_and_sharp_scores(nq):
    # scores up to some hundreds: one token takes nearly all; scales other than 1; a scale argument
    lens, Hq, Hkv, D, page = [700, 333], 8, 2, 128, 32
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq, nq], Hq, Hkv, D, page, 77, k_size=8.0)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, scale=0.25, ks=0.5, vs=3.0)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, 0.25, kscale=0.5, vscale=3.0)


@pytest.mark.parametrize("nq", [1, 70])
def test_attention_rising_and_falling_scores(nq):
    # the running maximum moves at every tile, or never: keys along one query, growing or shrinking with the place
    Hq, Hkv, D, page, L = 2, 1, 64, 16, 600
    g = gen(4)
    d = torch.randn(D, generator=g)
    for up in (True, False):
        f = torch.arange(L).float() / L * 6
        f = f if up else f.flip(0)
        kc, kb = ref.quantize((f[:, None] * d)[:, None], 1.0)
        vc, vb = ref.quantize(torch.randn(L, 1, D, generator=g), 1.0)
        n_pages = -(-L // page)
        c = torch.zeros(q.qlin_kv_cache_bytes(n_pages, page, 1, D), dtype=torch.uint8)
        ref.put(c, page, 1, D, torch.arange(L), kc, kb, vc, vb)
        qs = [(d * torch.ones(nq, Hq, 1)).bfloat16()]
        table = torch.arange(n_pages, dtype=torch.int32)[None]
        cu = torch.tensor([0, nq], dtype=torch.int32)
        ln = torch.tensor([L], dtype=torch.int32)
        o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs)
        assert st == 0
        check_attn(o, ln, cu, qs, [ref.values(kc, kb)], [ref.values(vc, vb)], D, D ** -0.5)


@pytest.mark.parametrize("nq", [1, 70])
def test_attention_query_sizes(nq):
    # queries far outside fp16's range, rows of zeros beside them; q and out as strided views
    lens, Hq, Hkv, D, page = [200], 4, 2, 64, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq], Hq, Hkv, D, page, 78)
    big = qs[0].clone()
    big[:, 0] *= 1e30
    big[:, 1] *= 1e-30
    big[:, 2] = 0
    kv = q.KVCache(dev_cache(c), page, Hkv, D)
    wide = torch.zeros(nq, Hq * D + 64, dtype=BF16, device="cuda")
    qv = wide[:, :Hq * D].unflatten(1, (Hq, D))
    qv.copy_(big.cuda())
    ob = torch.full((nq + 3, Hq * D + 8), 7.0, dtype=BF16, device="cuda")
    q.qlin_attn_kv4(kv, qv, table.cuda(), ln.cuda(), cu.cuda(), nq, 1e-2, out=ob[:nq, :Hq * D].unflatten(1, (Hq, D)))
    assert (ob[nq:] == 7).all() and (ob[:, Hq * D:] == 7).all()
    o = ob[:nq, :Hq * D].unflatten(1, (Hq, D))
    # scores of 1e28: the largest one takes all, so the row is that token's V
    out, tp, ts, tv = ref.attention(big.double(), ks[0], vs[0], 200, 1e-2)
    got = o.cpu().double()
    for h in (1, 2, 3):
        tol = ref.attention_tol(out, tp, ts, tv, D, 200)[:, h]
        assert ((got[:, h] - out[:, h]).abs() <= tol).all()
    assert ((got[:, 0] - out[:, 0]).abs() <= 2.0 ** -8 * out[:, 0].abs() + 2.0 ** -10).all()


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_rows_behind_the_last_sequence_stay(nq):
    lens, Hq, Hkv, D, page = [90, 33], 8, 2, 64, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq, nq], Hq, Hkv, D, page, 79)
    pad = torch.full((5, Hq, D), float("nan"), dtype=BF16)
    out = torch.full((2 * nq + 5, Hq, D), 7.0, dtype=BF16, device="cuda")
    run_attn(c, page, Hkv, D, table, ln, cu, [*qs, pad], max_q=nq, out=out)
    assert (out[2 * nq:] == 7).all()
    check_attn(out, ln, cu, qs, ks, vs, D, D ** -0.5)


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_bad_sequences_are_skipped(nq):
    lens, Hq, Hkv, D, page = [90, 60, 33, 50], 8, 2, 64, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq] * 4, Hq, Hkv, D, page, 80)
    bad = ln.clone()
    bad[1] = -5
    bad[3] = 10 ** 9
    out = torch.full((4 * nq, Hq, D), 7.0, dtype=BF16, device="cuda")
    o, st = run_attn(c, page, Hkv, D, table, bad, cu, qs, out=out)
    assert st == 1
    assert (o[nq:2 * nq] == 7).all() and (o[3 * nq:] == 7).all()
    keep = [0, 2]
    for b in keep:
        got = o[b * nq:(b + 1) * nq].cpu().double()
        ref_out, tp, ts, tv = ref.attention(qs[b].double(), ks[b], vs[b], lens[b], D ** -0.5)
        assert ((got - ref_out).abs() <= ref.attention_tol(ref_out, tp, ts, tv, D, lens[b])).all()
    # a page number outside the cache: its tokens count as masked
    t2 = table.clone()
    t2[0, 1] = 10 ** 6
    t2[2, 0] = -1
    o, st = run_attn(c, page, Hkv, D, t2, ln, cu, qs)
    assert st == 1
    i = torch.cat([torch.arange(16), torch.arange(32, 90)])
    if nq == 1:
        ref_out, tp, ts, tv = ref.attention(qs[0].double(), ks[0][i], vs[0][i], 74, D ** -0.5)
        assert ((o[:1].cpu().double() - ref_out).abs() <= ref.attention_tol(ref_out, tp, ts, tv, D, 90)).all()


@pytest.mark.parametrize("nq", [1, 64])
def test_attention_repeats_replays_and_streams(nq):
    # the same bits again, on a dirty workspace, from a captured graph with new lengths, and on another stream
    Hq, Hkv, D, page = 8, 2, 128, 16
    lens = [800, 90, 371]
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq] * 3, Hq, Hkv, D, page, 81)
    kv = q.KVCache(dev_cache(c), page, Hkv, D)
    qq, tb, l2, cc = torch.cat(qs).cuda(), table.cuda(), ln.cuda(), cu.cuda()
    ws = q.workspace(q.qlin_attn_kv4_workspace_bytes(kv, 3, nq, Hq))
    a = q.qlin_attn_kv4(kv, qq, tb, l2, cc, nq, ws=ws)
    out = torch.empty_like(a)
    for _ in range(3):
        q.qlin_attn_kv4(kv, qq, tb, l2, cc, nq, ws=ws, out=out)
        assert torch.equal(out, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        q.qlin_attn_kv4(kv, qq, tb, l2, cc, nq, ws=ws, out=out)
        assert torch.equal(out, a)
        with torch.cuda.graph(graph, stream=side):
            q.qlin_attn_kv4(kv, qq, tb, l2, cc, nq, ws=ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for new in ([800, 90, 371], [nq, 700, 1 + nq], [12, 0, 371]):
        fit = [min(n, len(tb[0]) * page, -(-len(k) // page) * page) for n, k in zip(new, ks)]
        fit = [min(n, len(k)) for n, k in zip(fit, ks)]
        l2.copy_(torch.tensor(fit, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_attn(out, torch.tensor(fit), cu, qs, [k[:n] for k, n in zip(ks, fit)], [v[:n] for v, n in zip(vs, fit)], D,
                   D ** -0.5)
    assert q.qlin_ws_status(ws) == 0


@pytest.mark.parametrize("nq", [1, 20])
def test_attention_cache_beyond_32_bits(nq):
    # byte offsets past 2^32: the sequence's pages lie at the end of a 4.4 GB cache
    Hq, Hkv, D, page, L = 8, 8, 128, 256, 500
    per = q.qlin_kv_cache_bytes(1, page, Hkv, D)
    n_pages = (1 << 32) // per + 40
    small, k, v = ref.random_cache(2, page, Hkv, D, gen(82))
    data = q._alloc_aligned(n_pages * per, "cuda")
    data[-2 * per:].copy_(small)
    kv = q.KVCache(data, page, Hkv, D)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32)
    k, v = torch.cat([k[page:], k[:page]])[:L], torch.cat([v[page:], v[:page]])[:L]
    qs = torch.randn(nq, Hq, D, generator=gen(83)).bfloat16()
    ln, cu = torch.tensor([L], dtype=torch.int32), torch.tensor([0, nq], dtype=torch.int32)
    o = q.qlin_attn_kv4(kv, qs.cuda(), table.cuda(), ln.cuda(), cu.cuda(), nq)
    check_attn(o, ln, cu, [qs], [k], [v], D, D ** -0.5)
    # and the append and read-back at the last slot
    x = torch.randn(1, 2 * Hkv * D, generator=gen(84))
    last = torch.tensor([n_pages * page - 1], dtype=torch.int32).cuda()
    q.qlin_kv_append(kv, x.cuda(), 0, None, last, None)
    gk, _ = q.qlin_kv_gather(kv, last, ydt=q.QLIN_F32)
    kc, kb = ref.quantize(x[:, :Hkv * D].view(1, Hkv, D), 1.0)
    assert torch.equal(gk.cpu(), ref.values(kc, kb).float())


@pytest.mark.parametrize("B,nq,Hq,Hkv", [(300, 1, 4, 2), (1024, 1, 2, 2), (1024, 3, 16, 1)])
def test_attention_many_sequences(B, nq, Hq, Hkv):
    # more sequences than one launch takes; empty ones among them
    D, page = 64, 16
    lens = [(37 * b) % 71 for b in range(B)]
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq] * B, Hq, Hkv, D, page, 85)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5)


@pytest.mark.parametrize("nq", [1, 5, 70])
@pytest.mark.parametrize("window", [1, 40, 300])
def test_attention_pages_before_the_window_are_free(nq, window):
    # a user may give the pages before the window away: numbers outside the cache, or any bits in them
    lens, Hq, Hkv, D, page = [700, 333, 128], 8, 2, 128, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq] * 3, Hq, Hkv, D, page, 86)
    pages = c.view(-1, q.qlin_kv_cache_bytes(1, page, Hkv, D))
    for b, L in enumerate(lens):
        gone = max(0, L - nq - window + 1) // page  # whole pages that no query sees
        for j in range(gone):
            pages[table[b, j]] = 0x7F
            if b != 1:
                table[b, j] = -1
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, window=window)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5, window)


@pytest.mark.parametrize("nq", [1, 33])
def test_attention_shared_pages(nq):
    # sequences with a common beginning, one of them twice, and one whose page table repeats a page
    Hq, Hkv, D, page = 8, 2, 64, 32
    c, k, v = ref.random_cache(12, page, Hkv, D, gen(87))
    rows = [[0, 1, 2, 3, 4], [0, 1, 2, 5, 6], [0, 1, 2, 3, 4], [7, 7, 7, 0, 7]]
    lens = [150, 139, 150, 160]
    table, ln = torch.tensor(rows, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    cu = torch.arange(5, dtype=torch.int32) * nq
    qs = [torch.randn(nq, Hq, D, generator=gen(88 + b % 2)).bfloat16() for b in range(4)]
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs)
    assert st == 0
    idx = [(torch.tensor(r)[:, None] * page + torch.arange(page)).flatten()[:L] for r, L in zip(rows, lens)]
    check_attn(o, ln, cu, qs, [k[i] for i in idx], [v[i] for i in idx], D, D ** -0.5)
    assert torch.equal(o[:nq], o[2 * nq:3 * nq])


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30])
@pytest.mark.parametrize("nq", [1, 70])
def test_attention_any_scale(nq, scale):
    lens, Hq, Hkv, D, page = [200, 31], 4, 2, 64, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq, min(nq, 31)], Hq, Hkv, D, page, 90)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, scale=scale)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, scale)


@pytest.mark.parametrize("nq", [1, 5, 70])
def test_attention_rows_of_nan_and_infinity_stay_alone(nq):
    lens, Hq, Hkv, D, page = [300], 8, 1, 128, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [nq], Hq, Hkv, D, page, 91)
    bad = [t.clone() for t in qs]
    bad[0][:, 1, 3] = float("nan")
    bad[0][:, 4, 7] = float("inf")
    bad[0][:, 6] = -float("inf")
    o, _ = run_attn(c, page, Hkv, D, table, ln, cu, bad)
    clean, _ = run_attn(c, page, Hkv, D, table, ln, cu, qs)
    keep = [0, 2, 3, 5, 7]
    check_attn(clean, ln, cu, qs, ks, vs, D, D ** -0.5)
    assert torch.isnan(o[:, 1]).all()
    out, tp, ts, tv = ref.attention(qs[0].double(), ks[0], vs[0], 300, D ** -0.5)
    err = (o.cpu().double() - out).abs() <= ref.attention_tol(out, tp, ts, tv, D, 300)
    assert err[:, keep].all()


def test_attention_falling_rows_are_refused_by_the_status():
    lens, Hq, Hkv, D, page = [90, 60, 33], 4, 2, 64, 16
    c, table, ln, _, qs, ks, vs = attn_case(lens, [4, 3, 2], Hq, Hkv, D, page, 92)
    for nq_max in (4, 200):  # few rows, and the other kernel
        cu = torch.tensor([4, 8, 2, 4], dtype=torch.int32)
        rows = torch.cat([torch.zeros(2, Hq, D).bfloat16(), qs[2], qs[0]])
        out = torch.full((8, Hq, D), 7.0, dtype=BF16, device="cuda")
        o, st = run_attn(c, page, Hkv, D, table, ln, cu, [rows], max_q=nq_max, out=out)
        assert st == 1 and (o[:2] == 7).all()
        check_attn(o[4:], ln[:1], torch.tensor([0, 4]), qs[:1], ks[:1], vs[:1], D, D ** -0.5)
        check_attn(o[2:4], ln[2:], torch.tensor([0, 2]), qs[2:], ks[2:], vs[2:], D, D ** -0.5)


def test_attention_max_q_above_the_queries():
    # the bound on the queries chooses the kernel: single tokens through each
    lens, Hq, Hkv, D, page = [500, 64, 1, 0], 8, 2, 128, 16
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [1] * 4, Hq, Hkv, D, page, 93)
    for mq in (1, 2, 3, 8, 9, 32, 33, 4000):
        o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs, max_q=mq)
        assert st == 0
        check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5)


@pytest.mark.parametrize("rows", [32, 36, 128, 132])
@pytest.mark.parametrize("B", [1, 9])
def test_attention_on_both_sides_of_the_choice(rows, B):
    Hq, Hkv, D, page = 8, 2, 64, 16
    lens = [200 + 13 * b for b in range(B)]
    c, table, ln, cu, qs, ks, vs = attn_case(lens, [rows // 4] * B, Hq, Hkv, D, page, 94 + rows)
    o, st = run_attn(c, page, Hkv, D, table, ln, cu, qs)
    assert st == 0
    check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5)


def test_attention_one_workspace_for_many_shapes_and_two_graphs():
    # every call leaves the workspace fit for any other that it is large enough for; graphs that share it run in turn
    Hq, Hkv, D, page = 8, 2, 128, 16
    shapes = [([3000], 1), ([900, 30, 5], 70), ([2000, 700], 6), ([60, 1200], 1), ([1500], 257)]
    cases = [attn_case(lens, [min(nq, L) for L in lens], Hq, Hkv, D, page, 95 + i) for i, (lens, nq) in enumerate(shapes)]
    calls, need = [], 0
    for (lens, nq), (c, table, ln, cu, qs, ks, vs) in zip(shapes, cases):
        kv = q.KVCache(dev_cache(c), page, Hkv, D)
        need = max(need, q.qlin_attn_kv4_workspace_bytes(kv, len(lens), nq, Hq))
        calls.append((kv, torch.cat(qs).cuda(), table.cuda(), ln.cuda(), cu.cuda(), nq))
    ws = q.workspace(need)
    alone = [q.qlin_attn_kv4(*call) for call in calls]
    for o, (c, table, ln, cu, qs, ks, vs) in zip(alone, cases):
        check_attn(o, ln, cu, qs, ks, vs, D, D ** -0.5)
    for i in (0, 1, 2, 3, 4, 3, 1, 4, 0, 2):
        assert torch.equal(q.qlin_attn_kv4(*calls[i], ws=ws), alone[i]), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for call in calls[:2]:
        out = torch.empty_like(call[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            q.qlin_attn_kv4(*call, ws=ws, out=out)
        graphs.append((graph, out))
    for _ in range(3):
        for (graph, out), want in zip(graphs, alone):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
    assert q.qlin_ws_status(ws) == 0


def test_calls_on_two_streams_at_once():
    # append, read-back and attention of two caches side by side, each with a workspace of its own; the stream argument
    Hq, Hkv, D, page, T = 8, 2, 128, 16, 700
    x = [torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen(i)).cuda() for i in (1, 2)]
    pos, cs = torch.arange(T, dtype=torch.int32).cuda(), ref.table(T, D).cuda()
    table = torch.arange(44, dtype=torch.int32)[None].cuda()
    lens, cu = torch.tensor([T], dtype=torch.int32).cuda(), torch.tensor([0, T], dtype=torch.int32).cuda()
    one = torch.tensor([0, 1], dtype=torch.int32).cuda()

    def run(cache, x, ws, **kw):
        qo = q.qlin_kv_append(cache, x, Hq, pos, pos, cs, ws=ws, **kw)
        a = q.qlin_attn_kv4(cache, qo, table, lens, cu, T, ws=ws, **kw)
        b = q.qlin_attn_kv4(cache, qo[-1:], table, lens, one, 1, ws=ws, **kw)
        return [qo, a, b, *q.qlin_kv_gather(cache, pos, ws=ws, **kw)]

    caches = [q.kv_cache(44, page, Hkv, D) for _ in x]
    n = max(q.qlin_attn_kv4_workspace_bytes(caches[0], 1, m, Hq) for m in (1, T))
    want = [run(c, xi, q.workspace(n)) for c, xi in zip(caches, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    fresh = [q.kv_cache(44, page, Hkv, D) for _ in x]
    ws = [q.workspace(n) for _ in x]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = [run(c, xi, w, stream=s) for c, xi, w, s in zip(fresh, x, ws, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    qk = q.qlin_qk_norm_rope(x[0], Hq, Hkv, D, pos, cs, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(qk[0], want[0][0])


def test_strided_rows_and_tables():
    # rows of x, of the block table and of the outputs as parts of wider ones, for one sequence and for several
    Hq, Hkv, D, page = 4, 2, 64, 16
    W = (Hq + 2 * Hkv) * D
    for B in (1, 3):
        T = 5 * B
        wide = torch.randn(T, W + 16, generator=gen(30 + B)).cuda()
        x = wide[:, 8:8 + W]
        slots = torch.randperm(B * 16, generator=gen(31))[:T].int().cuda()
        a, b = q.kv_cache(B, page, Hkv, D), q.kv_cache(B, page, Hkv, D)
        qa = q.qlin_kv_append(a, x, Hq, None, slots)
        qw = torch.full((T, Hq * D + 8), 7.0, dtype=BF16, device="cuda")
        q.qlin_kv_append(b, x.contiguous(), Hq, None, slots, q=qw[:, :Hq * D])
        assert torch.equal(a.data, b.data) and torch.equal(qa.flatten(1), qw[:, :Hq * D]) and (qw[:, Hq * D:] == 7).all()
        tab = torch.full((B, 9), -1, dtype=torch.int32, device="cuda")
        tab[:, 3] = torch.arange(B, device="cuda")
        lens = torch.full((B,), 16, dtype=torch.int32, device="cuda")
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 5
        # slots that no token was appended to hold zeros: places like any other
        o1 = q.qlin_attn_kv4(a, qw[:, :Hq * D].unflatten(1, (Hq, D)), tab[:, 3:4], lens, cu, 5)
        o2 = q.qlin_attn_kv4(a, qa, tab[:, 3:4].contiguous(), lens, cu, 5)
        assert torch.equal(o1, o2) and torch.isfinite(o1.float()).all()


def test_decode_loop_in_one_graph():
    """The append, the attention and the read-back of a decode step captured once and replayed for many steps, positions,
    slots and lengths renewed in place, against the same calls made one by one on another cache."""
    Hq, Hkv, D, page, B, steps = 8, 2, 128, 16, 3, 40
    W = (Hq + 2 * Hkv) * D
    xs = torch.randn(steps, B, W, generator=gen(40)).cuda()
    cs, w = ref.table(200, D).cuda(), [(1 + 0.2 * torch.randn(D, generator=gen(i))).cuda() for i in (41, 42)]
    start = [0, 100, 31]
    table = torch.randperm(27, generator=gen(43)).view(3, 9).int().cuda()
    past = torch.randn(B, 144, W, generator=gen(44)).cuda()
    caches = [q.kv_cache(27, page, Hkv, D, 0.5, 2.0) for _ in range(2)]
    place = lambda b, p: table[b, p // page] * page + p % page  # noqa: E731
    for c in caches:
        for b in range(B):
            if start[b]:
                p = torch.arange(start[b], device="cuda")
                q.qlin_kv_append(c, past[b, :start[b]], Hq, p.int(), place(b, p).int(), cs, *w)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ws = q.workspace(q.qlin_attn_kv4_workspace_bytes(caches[0], B, 1, Hq))
    x, pos, slots, lens = torch.zeros(B, W, device="cuda"), cu[:B].clone(), cu[:B].clone(), cu[:B].clone()

    def renew(s):
        x.copy_(xs[s])
        pos.copy_(torch.tensor([n + s for n in start], dtype=torch.int32))
        slots.copy_(torch.stack([place(b, start[b] + s) for b in range(B)]))
        lens.copy_(torch.tensor([n + s + 1 for n in start], dtype=torch.int32))

    def step(c):
        qo = q.qlin_kv_append(c, x, Hq, pos, slots, cs, *w, ws=ws)
        o = q.qlin_attn_kv4(c, qo, table, lens, cu, 1, ws=ws)
        return [o, *q.qlin_kv_gather(c, slots, ws=ws)]

    renew(0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step(caches[0])
    for s in range(steps):
        renew(s)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, step(caches[1]))), s
    assert q.qlin_ws_status(ws) == 0 and torch.equal(caches[0].data, caches[1].data)


def test_calls_without_rows():
    D, page = 64, 16
    cache = q.kv_cache(2, page, 1, D)
    before = cache.data.clone()
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 4 * D, device="cuda")
    cs = ref.table(4, D).cuda()
    qo, ko = q.qlin_qk_norm_rope(x, 2, 1, D, e, cs)
    assert qo.shape == (0, 2, D) and ko.shape == (0, 1, D)
    assert q.qlin_kv_append(cache, x, 2, e, e, cs).shape == (0, 2, D)
    assert q.qlin_kv_gather(cache, e)[0].shape == (0, 1, D)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    o = q.qlin_attn_kv4(cache, torch.zeros(0, 2, D, dtype=BF16, device="cuda"), z[None], z[:1], z, 1)
    assert o.shape == (0, 2, D) and torch.equal(cache.data, before)


def test_append_needs_no_positions_without_rotation_and_no_queries():
    T, Hq, Hkv, D, page = 5, 3, 2, 64, 16
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen(12)).cuda()
    slots = torch.arange(T, dtype=torch.int32).cuda()
    w = torch.full((D,), 1.5).cuda()
    a, b = q.kv_cache(1, page, Hkv, D), q.kv_cache(1, page, Hkv, D)
    q.qlin_kv_append(a, x, Hq, None, slots, None, w, w)
    q.qlin_kv_append(b, x[:, Hq * D:].contiguous(), 0, None, slots, None, None, w)
    assert torch.equal(a.data, b.data)


# ----------------------------------------------------------------------------- as they are used
def test_decode_step_from_qkv_projection_to_o_projection():
    """Prompt and decode steps of one attention layer: the Q4_0 qkv projection, the append, the attention, the o
    projection; every step's attention output against the 64-bit form of the same projections' outputs."""
    import synth
    H, Hq, Hkv, D, page, B = 512, 8, 2, 64, 16, 2
    W = (Hq + 2 * Hkv) * D
    qkv_w = q.qlin_pack_weights(q.QLIN_Q4_0, W, H, synth.weights(q.QLIN_Q4_0, W, H, synth.gen(1))[0].cuda())
    o_w = q.qlin_pack_weights(q.QLIN_Q4_0, H, Hq * D, synth.weights(q.QLIN_Q4_0, H, Hq * D, synth.gen(2))[0].cuda())
    cs = ref.table(200, D)
    w = [1 + 0.2 * torch.randn(D, generator=gen(i)) for i in (3, 4)]
    cache = q.kv_cache(20, page, Hkv, D, 0.5, 0.25)
    table = torch.stack([torch.randperm(10, generator=gen(5)), torch.randperm(10, generator=gen(6)) + 10]).int()
    ws = q.workspace(q.qlin_attn_kv4_workspace_bytes(cache, B, 40, Hq))
    past = [(torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)) for _ in range(B)]
    lens = [0, 0]
    for step, nqs in enumerate(([40, 7], [1, 1], [1, 1], [1, 3], [1, 1])):
        n = sum(nqs)
        if n <= 8:
            hid = synth.activations(n, H, synth.gen(10 + step)).cuda()
            x = q.qlin_gemv(q.QLIN_Q4_0, qkv_w, W, H, hid)
        else:
            x = torch.randn(n, W, generator=gen(20 + step)).cuda()
        pos = torch.cat([torch.arange(c) + L for c, L in zip(nqs, lens)]).int()
        seq = torch.tensor([b for b in range(B) for _ in range(nqs[b])])
        slots = table[seq, (pos // page).long()] * page + pos % page
        lens = [L + c for L, c in zip(lens, nqs)]
        cu = torch.tensor([0, nqs[0], n], dtype=torch.int32)
        qo = q.qlin_kv_append(cache, x, Hq, pos.cuda(), slots.int().cuda(), cs.cuda(), w[0].cuda(), w[1].cuda())
        o = q.qlin_attn_kv4(cache, qo, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu.cuda(), max(nqs), ws=ws)
        xd = x.cpu().double().view(n, -1, D)
        k, _ = ref.norm_rope(xd[:, Hq:Hq + Hkv], w[1], 1e-6, cs, pos, D, False)
        kx = ref.values(*ref.quantize(k.float(), 0.5), 0.5)
        vx = ref.values(*ref.quantize(xd[:, Hq + Hkv:].float(), 0.25), 0.25)
        past = [(torch.cat([pk, kx[seq == b]]), torch.cat([pv, vx[seq == b]])) for b, (pk, pv) in enumerate(past)]
        qh = qo.cpu()
        check_attn(o, torch.tensor(lens), cu, [qh[seq == b] for b in range(B)], [p[0].double() for p in past],
                   [p[1].double() for p in past], D, D ** -0.5)
        if n <= 8:
            y = q.qlin_gemv(q.QLIN_Q4_0, o_w, H, Hq * D, o.flatten(1))
            assert y.shape == (n, H) and torch.isfinite(y).all()
    assert q.qlin_ws_status(ws) == 0
