"""What stands between a decode step's fused qkv projection and its o projection, case by case: the
norm and rotation of queries and keys, the append to a paged NVFP4 cache of keys and values, and the
attention that reads that cache, for single tokens and for prompt chunks.

`run` computes them in plain torch operations where `own` is false, and with the library's calls
where it is true.  The cache is one uint8 buffer [pages][kv heads][page / 16 groups][18 * D bytes];
a group holds 16 tokens of one head: K codes (token-major, two E2M1 codes a byte, the even element
in the low nibble), K scales (E4M3, one per 16 values, token-major), V codes (16-value block-major:
block, token, 8 bytes), V scales (block-major: block, token).
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------------------ the cases
def _rope(name, T, Hq, Hkv, D, rot, interleaved, x, y, n_pos=40960):
    return dict(name=name, op="rope", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved, norm=True, x=x, y=y,
                n_pos=n_pos)


def _append(name, T, Hq, Hkv, D, rot, interleaved, norm, x, page, decode, n_pos=40960):
    return dict(name=name, op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved, norm=norm, x=x,
                page=page, decode=decode, n_pos=n_pos)


def _attn(name, B, nq, L, ragged, Hq, Hkv, D, page, window=0):
    return dict(name=name, op="attn", B=B, nq=nq, L=L, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, page=page, window=window)


def listed():
    return [
        # one token of a decode step: the 4B stack's 6144 fused outputs (32 query and 8 key heads of 128), fp32 as
        # the decode projections write them
        _rope("rope 1 token", 1, 32, 8, 128, 128, False, "f32", "bf16"),
        # a prompt chunk of the same layer, bf16 in and out
        _rope("rope 2048 tokens", 2048, 32, 8, 128, 128, False, "bf16", "bf16"),
        # an odd number of tokens, heads of 64 in groups of three, half of each head rotated, neighbouring pairs
        _rope("rope 1237 tokens partial", 1237, 24, 8, 64, 32, True, "f32", "f32"),
        # a decode step of eight sequences: each appends one token to a page of its own
        _append("append 8 sequences", 8, 32, 8, 128, 128, False, True, "f32", 16, True),
        # the largest prompt chunk
        _append("append 8192 tokens", 8192, 32, 8, 128, 128, False, True, "bf16", 64, False),
        # an odd chunk without head norms, heads of 64
        _append("append 777 tokens", 777, 16, 4, 64, 64, True, False, "bf16", 32, False),
        # one sequence, a short context: the smallest call of a decode step
        _attn("decode 1 x 1000", 1, 1, 1000, False, 32, 8, 128, 16),
        # a small ragged batch, heads of 64 in groups of three
        _attn("decode 16 x 4096 ragged", 16, 1, 4096, True, 24, 8, 64, 32),
        # a full serving batch
        _attn("decode 64 x 8192", 64, 1, 8192, True, 32, 8, 128, 64),
        # one long document: few rows, a long axis
        _attn("decode 1 x 131071", 1, 1, 131071, False, 32, 8, 128, 64),
        # the first chunk of a prompt
        _attn("chunk 512 fresh", 1, 512, 512, False, 32, 8, 128, 16),
        # later chunks of two prompts of odd lengths
        _attn("chunk 2 x 2047 of 8189", 2, 2047, 8189, True, 32, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    Hkv = rng.choice([1, 2, 4, 8]) if G * 8 > 32 else rng.choice([2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["rope", "append", "decode", "decode", "chunk", "chunk"])
    if kind in ("rope", "append"):
        case = dict(op=kind, T=_log(rng, 1, 8000), Hq=G * Hkv, Hkv=Hkv, D=D, rot=rng.choice([D, D // 2]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, x=rng.choice(["f32", "bf16"]),
                    n_pos=40960)
        if kind == "rope":
            case["y"] = rng.choice(["f32", "bf16"])
        else:
            case["page"], case["decode"] = page, rng.random() < 0.3
        return case
    window = rng.choice([0, 0, 0, _log(rng, 32, 4096)])
    if kind == "decode":
        B = _log(rng, 1, 64)
        L = min(_log(rng, 1, 131072), 64 * 8192 // B)
        return dict(op="attn", B=B, nq=rng.choice([1, 1, 1, 2, 4]), L=L, ragged=rng.random() < 0.6, Hq=G * Hkv,
                    Hkv=Hkv, D=D, page=page, window=window)
    B = rng.choice([1, 1, 2, 3])
    nq = _log(rng, 24, 2048 // B)
    return dict(op="attn", B=B, nq=nq, L=nq + rng.choice([0, _log(rng, 1, 6000)]), ragged=rng.random() < 0.6,
                Hq=G * Hkv, Hkv=Hkv, D=D, page=page, window=window)


# ----------------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _table(n_pos, rot):
    # cos and sin of pos * theta^(-2i / rot), the angles in 64 bits: at far positions they are thousands of radians
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * THETA ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _lut():
    m = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(m + [-v for v in m], device="cuda")


def _codes(v):
    """E2M1 codes of v, round to nearest, ties to the even code, saturating at 6."""
    a = v.abs()
    up = torch.zeros_like(a, dtype=torch.uint8)
    for bound, closed in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        up += (a >= bound) if closed else (a > bound)
    return up | (torch.signbit(v).to(torch.uint8) << 3)


def _quantize(x, g):
    """NVFP4 of fp32 rows of D values under the per-tensor scale g: codes and E4M3 scales of 16 values."""
    b = x.unflatten(-1, (-1, 16))
    g = torch.tensor(g, device=x.device, dtype=torch.float32)
    s = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    div = (s.float() * g)[..., None]
    v = torch.where(div > 0, b / torch.where(div > 0, div, torch.ones_like(div)), torch.zeros_like(b))
    return _codes(v).flatten(-2), s


def _values(codes, s, g):
    """The values that codes and scales stand for: fp32(code * scale * g), one rounding."""
    v = _lut()[codes.int()].unflatten(-1, (-1, 16)) * s.float()[..., None]
    return (v * torch.tensor(g, device=codes.device, dtype=torch.float32)).flatten(-2)


def _bytes(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _fill(cache, pages, kx, vx, ks, vs):
    """Lays K and V (pages, page, kv heads, D) into the cache's pages."""
    n, page, Hkv, D = kx.shape
    view = cache.view(-1, Hkv, page // 16, 18 * D)
    kc, ksc = _quantize(kx, ks)
    kc, ksc = _bytes(kc), ksc.view(torch.uint8)
    k = kc.view(n, page // 16, 16, Hkv, D // 2).permute(0, 3, 1, 2, 4).reshape(n, Hkv, page // 16, 8 * D)
    a = ksc.view(n, page // 16, 16, Hkv, D // 16).permute(0, 3, 1, 2, 4).reshape(n, Hkv, page // 16, D)
    vc, vsc = _quantize(vx, vs)
    vc, vsc = _bytes(vc), vsc.view(torch.uint8)
    v = vc.view(n, page // 16, 16, Hkv, D // 16, 8).permute(0, 3, 1, 4, 2, 5).reshape(n, Hkv, page // 16, 8 * D)
    b = vsc.view(n, page // 16, 16, Hkv, D // 16).permute(0, 3, 1, 4, 2).reshape(n, Hkv, page // 16, D)
    view[pages] = torch.cat([k, a, v, b], -1)


def _lengths(case):
    """(queries, context) of each sequence, by the case alone; the context counts the call's own tokens."""
    g = torch.Generator()
    g.manual_seed(case["L"] + case["B"])
    n, L = [case["nq"]] * case["B"], [case["L"]] * case["B"]
    if case["ragged"] and case["B"] > 1:
        f = torch.rand(case["B"], generator=g, dtype=torch.float64).tolist()
        n = [case["nq"]] + [max(1, int(case["nq"] * (0.25 + 0.75 * f[i]))) for i in range(1, case["B"])]
        L = [case["L"]] + [max(n[i], int(case["L"] * (0.25 + 0.75 * f[-i]))) for i in range(1, case["B"])]
    return n, [max(a, b) for a, b in zip(n, L)]


def prepare(case, seed):
    g, dev = _gen(seed), "cuda"
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    st = dict(case=case, ks=0.75, vs=1.5)
    if case["op"] in ("rope", "append"):
        T, W = case["T"], (Hq + 2 * Hkv) * D
        # channels of uneven size, as projections have them
        x = randn(T, W) * torch.exp(0.5 * randn(W))
        st["x"] = x if case["x"] == "f32" else x.bfloat16()
        st["qw"] = 1 + 0.2 * randn(D) if case["norm"] else None
        st["kw"] = 1 + 0.2 * randn(D) if case["norm"] else None
        st["table"] = _table(case["n_pos"], case["rot"])
        if case["op"] == "append" and not case["decode"]:
            first = int(torch.randint(0, case["n_pos"] - T, (1,), generator=g, device=dev))
            st["pos"] = torch.arange(first, first + T, device=dev, dtype=torch.int32)
        else:
            st["pos"] = torch.randint(0, case["n_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
        if case["op"] == "append":
            page = case["page"]
            # a chunk fills consecutive places of pages in any order; decode tokens go to pages of their own
            per = 1 if case["decode"] else page
            used = -(-T // per)
            pages = torch.randperm(used + 5, generator=g, device=dev)[:used]
            t = torch.arange(T, device=dev)
            off = torch.randint(0, page, (T,), generator=g, device=dev) if case["decode"] else t % page
            st["slots"] = (pages[t // per] * page + off).int()
            st["cache"] = torch.randint(0, 256, ((used + 5) * Hkv * page // 16 * 18 * D,), generator=g, device=dev,
                                        dtype=torch.uint8)
        return st
    B, page = case["B"], case["page"]
    n, L = _lengths(case)
    per_seq = max(-(-v // page) for v in L)
    total = sum(-(-v // page) for v in L)
    order = torch.randperm(total + 3, generator=g, device=dev)
    table = torch.zeros(B, per_seq, dtype=torch.int32)
    at = 0
    order_host = order.tolist()
    for b in range(B):
        c = -(-L[b] // page)
        table[b, :c] = torch.tensor(order_host[at:at + c], dtype=torch.int32)
        at += c
    # normed keys with channels of uneven size; places behind a sequence's end hold what an earlier user left
    st["cache"] = torch.empty((total + 3) * Hkv * page // 16 * 18 * D, device=dev, dtype=torch.uint8)
    shape = torch.exp(0.3 * randn(Hkv, D))
    step = max(1, (1 << 27) // (page * Hkv * D))
    for p in range(0, total + 3, step):
        ids = order[p:p + step]
        _fill(st["cache"], ids, randn(len(ids), page, Hkv, D) * shape, randn(len(ids), page, Hkv, D), st["ks"], st["vs"])
    st["table"] = table.to(dev)
    st["lens"] = torch.tensor(L, device=dev, dtype=torch.int32)
    st["cu"] = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), device=dev, dtype=torch.int32)
    st["q"] = (1.5 * randn(sum(n), Hq, D)).bfloat16()
    st["max_q"] = max(n)
    st["scale"] = D ** -0.5
    return st


# ------------------------------------------------------------------------------- the plain forms
def _norm_rope(h, w, table, pos, rot, interleaved):
    """Rows (T, heads, D) of fp64: each head normed (where w is given), its first rot values rotated."""
    if w is not None:
        # eps reaches the library as a 32-bit number
        eps = torch.tensor(EPS, dtype=torch.float32).double().item()
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * w.double()
    cs = table[pos.long()].double()[:, None, :]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    r, rest = h[..., :rot], h[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        out = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([out, rest], -1)


def _heads(st):
    c = st["case"]
    x = st["x"].double().view(c["T"], -1, c["D"])
    return x[:, :c["Hq"]], x[:, c["Hq"]:c["Hq"] + c["Hkv"]], x[:, c["Hq"] + c["Hkv"]:]


def _plain_rope(st):
    c = st["case"]
    q, k, _ = _heads(st)
    y = torch.float32 if c["y"] == "f32" else torch.bfloat16
    args = (st["table"], st["pos"], c["rot"], c["interleaved"])
    return {"q": _norm_rope(q, st["qw"], *args).to(y), "k": _norm_rope(k, st["kw"], *args).to(y)}


def _plain_append(st):
    # in 64 bits up to the fp32 values that are quantized: a code next to a border must not depend on the
    # order of a sum
    c = st["case"]
    q, k, v = _heads(st)
    args = (st["table"], st["pos"], c["rot"], c["interleaved"])
    k = _values(*_quantize(_norm_rope(k, st["kw"], *args).float(), st["ks"]), st["ks"])
    v = _values(*_quantize(v.float(), st["vs"]), st["vs"])
    return {"q": _norm_rope(q, st["qw"], *args).bfloat16(), "k": k.bfloat16(), "v": v.bfloat16()}


def _read(st):
    """K and V of every sequence, (B, kv heads, tokens, D) fp32, from the cache's pages."""
    c = st["case"]
    D, Hkv, page, B = c["D"], c["Hkv"], c["page"], c["B"]
    per = st["table"].shape[1]
    grp = st["cache"].view(-1, Hkv, page // 16, 18 * D)[st["table"].long()].transpose(1, 2)
    lut = _lut()

    def codes(b):
        return torch.stack([lut[(b & 15).int()], lut[(b >> 4).int()]], -1).flatten(-2)

    def scales(b):
        return b.contiguous().view(torch.float8_e4m3fn).float()[..., None]

    k = codes(grp[..., :8 * D].unflatten(-1, (16, D // 16, 8))) * scales(grp[..., 8 * D:9 * D].unflatten(-1, (16, D // 16)))
    v = codes(grp[..., 9 * D:17 * D].unflatten(-1, (D // 16, 16, 8))) * scales(grp[..., 17 * D:].unflatten(-1, (D // 16, 16)))
    v = v.transpose(-2, -3)
    return k.reshape(B, Hkv, per * page, D) * st["ks"], v.reshape(B, Hkv, per * page, D) * st["vs"]


def _plain_attn(st):
    c = st["case"]
    D, Hq, Hkv, B = c["D"], c["Hq"], c["Hkv"], c["B"]
    G, nq = Hq // Hkv, st["max_q"]
    k, v = _read(st)
    n = k.shape[2]
    lens, cu = st["lens"].long(), st["cu"].long()
    cnt = cu[1:] - cu[:-1]
    i, t = torch.arange(nq, device=k.device), torch.arange(n, device=k.device)
    row = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[row].view(B, nq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nq * G, D)
    last = lens[:, None] - cnt[:, None] + i                      # the context place of query i
    seen = (t <= last[..., None]) & (t < lens[:, None, None])
    if c["window"]:
        seen &= t > last[..., None] - c["window"]
    seen = seen[:, None, :, None].expand(B, 1, nq, G, n).reshape(B, 1, nq * G, n)
    s = torch.where(seen, q @ k.transpose(-1, -2) * st["scale"], -torch.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    held = t < lens[:, None]
    o = (p @ torch.where(held[:, None, :, None], v, 0.0)) / p.sum(-1, keepdim=True)
    o = o.view(B, Hkv, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, Hq, D)
    return o[i < cnt[:, None]].bfloat16()


# ---------------------------------------------------------------------------- the library's calls
def _own_rope(st):
    import gemm_dequant_gemv_q8_b200 as q
    c = st["case"]
    if "ws" not in st:
        st["ws"] = q.workspace(256)
    qo, ko = q.qlin_qk_norm_rope(st["x"], c["Hq"], c["Hkv"], c["D"], st["pos"], st["table"], st["qw"], st["kw"], EPS,
                                 rot=c["rot"], flags=q.QLIN_ROPE_INTERLEAVED if c["interleaved"] else 0,
                                 ydt=q.QLIN_F32 if c["y"] == "f32" else q.QLIN_BF16, ws=st["ws"])
    return {"q": qo, "k": ko}


def _own_append(st):
    import gemm_dequant_gemv_q8_b200 as q
    c = st["case"]
    if "ws" not in st:
        st["ws"] = q.workspace(256)
        st["kv"] = q.KVCache(st["cache"], c["page"], c["Hkv"], c["D"], st["ks"], st["vs"])
    qo = q.qlin_kv_append(st["kv"], st["x"], c["Hq"], st["pos"], st["slots"], st["table"], st["qw"], st["kw"], EPS,
                          rot=c["rot"], flags=q.QLIN_ROPE_INTERLEAVED if c["interleaved"] else 0, ws=st["ws"])
    k, v = q.qlin_kv_gather(st["kv"], st["slots"], ydt=q.QLIN_BF16, ws=st["ws"])
    return {"q": qo, "k": k, "v": v}


def _own_attn(st):
    import gemm_dequant_gemv_q8_b200 as q
    c = st["case"]
    if "ws" not in st:
        st["kv"] = q.KVCache(st["cache"], c["page"], c["Hkv"], c["D"], st["ks"], st["vs"])
        st["ws"] = q.workspace(q.qlin_attn_kv4_workspace_bytes(st["kv"], c["B"], st["max_q"], c["Hq"]))
    return q.qlin_attn_kv4(st["kv"], st["q"], st["table"], st["lens"], st["cu"], st["max_q"], st["scale"],
                           window=c["window"], ws=st["ws"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn": _own_attn}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------------------------------- the floor
def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] in ("rope", "append"):
        T, xb = case["T"], 4 if case["x"] == "f32" else 2
        rows = 4 * case["rot"] * min(T, case["n_pos"])
        if case["op"] == "rope":
            n = T * (Hq + Hkv) * D
            return {"bytes": n * (xb + (4 if case["y"] == "f32" else 2)) + rows, "flops": 8 * n}
        n = T * (Hq + 2 * Hkv) * D
        # read the projections, write the rotated queries, the cache's 4.5 bits a value and the values returned
        return {"bytes": n * xb + T * Hq * D * 2 + 2 * T * Hkv * D * (9 / 16 + 2) + rows, "flops": 8 * n}
    n, L = _lengths(case)
    pairs = read = 0
    for a, b in zip(n, L):
        w = case["window"] or b + 1
        first = max(0, b - a + 1 - w)
        read += b - first
        # query i sees min(b - a + i + 1, w) tokens
        full = max(0, min(a, w - (b - a) - 1)) if b - a + 1 <= w else 0
        pairs += full * (b - a) + full * (full + 1) // 2 + (a - full) * w
    return {"bytes": read * Hkv * D * 9 / 8 + sum(n) * Hq * D * 4, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------- from the definition
def _exact_rotated(st, heads, w):
    """One complex product a pair: the head as complex numbers, turned by the table's angle."""
    c = st["case"]
    h, rot = heads.double(), c["rot"]
    if w is not None:
        norm = torch.linalg.vector_norm(h, dim=-1, keepdim=True)
        h = h / torch.sqrt(norm * norm / c["D"] + float(torch.tensor(EPS, dtype=torch.float32))) * w.double()
    t = st["table"].double()[st["pos"].long()]
    turn = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
    r = h[..., :rot]
    pairs = r.reshape(*r.shape[:-1], rot // 2, 2) if c["interleaved"] else r.reshape(*r.shape[:-1], 2, rot // 2).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z if c["interleaved"] else z.transpose(-1, -2)
    return torch.cat([z.reshape(r.shape), h[..., rot:]], -1)


def _exact_nvfp4(x, g):
    """The values NVFP4 holds for x: the nearest of the 15 values of a code, the even code on a tie."""
    x = x.float().double()
    g = float(torch.tensor(g, dtype=torch.float32))
    b = x.reshape(*x.shape[:-1], -1, 16)
    s = torch.clamp(b.abs().max(-1, keepdim=True).values / (6 * g), max=448).float().to(torch.float8_e4m3fn).double()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device, dtype=torch.float64)
    v = b.abs() / torch.where(s == 0, 1.0, s * g)
    lo = (torch.searchsorted(grid, v.contiguous(), right=True) - 1).clamp(0, 6)
    down, up = v - grid[lo], grid[lo + 1] - v
    code = torch.where((up < down) | ((up == down) & (lo % 2 == 1)), lo + 1, lo)
    return (torch.where(s == 0, 0.0, torch.sign(b) * grid[code] * s * g)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("rope", "append"):
        T, D, Hq, Hkv = case["T"], case["D"], case["Hq"], case["Hkv"]
        x = st["x"].reshape(T, Hq + 2 * Hkv, D)
        out = {"q": _exact_rotated(st, x[:, :Hq], st["qw"])}
        k = _exact_rotated(st, x[:, Hq:Hq + Hkv], st["kw"])
        if case["op"] == "rope":
            return {**out, "k": k}
        return {**out, "k": _exact_nvfp4(k, st["ks"]), "v": _exact_nvfp4(x[:, Hq + Hkv:], st["vs"])}
    # one sequence and one kv head at a time: the tokens by their page and place, a softmax in 64 bits
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    G = Hq // Hkv
    lut = _lut().double()
    lens, cu, table = st["lens"].tolist(), st["cu"].tolist(), st["table"].long()
    mem = st["cache"].view(-1, Hkv, page // 16, 18 * D)
    out = torch.empty(cu[-1], Hq, D, device="cuda", dtype=torch.float64)
    e = torch.arange(D, device="cuda")
    for b in range(case["B"]):
        t = torch.arange(lens[b], device="cuda")
        pg, gr, r = table[b][t // page], t % page // 16, (t % 16)[:, None]
        i = torch.arange(cu[b + 1] - cu[b], device="cuda") + lens[b] - (cu[b + 1] - cu[b])
        seen = t[None] <= i[:, None]
        if case["window"]:
            seen &= i[:, None] - t[None] < case["window"]
        for h in range(Hkv):
            rows = mem[pg, h, gr]
            take = lambda at: torch.gather(rows, 1, at)  # noqa: E731
            shift = (4 * (e % 2)).to(torch.uint8)
            kc = lut[((take(r * (D // 2) + e // 2) >> shift) & 15).long()]
            ks = take(8 * D + r * (D // 16) + e // 16).view(torch.float8_e4m3fn).double()
            vc = lut[((take(9 * D + (e // 16) * 128 + r * 8 + e % 16 // 2) >> shift) & 15).long()]
            vs = take(17 * D + (e // 16) * 16 + r).view(torch.float8_e4m3fn).double()
            q = st["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            s = torch.einsum("igd,td->igt", q, kc * ks) * (st["ks"] * st["scale"])
            s = s.masked_fill(~seen[:, None], -torch.inf)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("igt,td->igd", torch.softmax(s, -1), vc * vs) * st["vs"]
    return out
