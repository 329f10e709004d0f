"""Plain 64-bit forms of the query / key norm and rotation, the NVFP4 cache append and the attention over the cache,
from the formulas (CPU, torch double), for the tests.  Nothing here uses the package.
"""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def table(n_pos, rot, theta=1e4):
    i = torch.arange(rot // 2, dtype=torch.float64)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * theta ** (-2 * i / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def norm_rope(x, w, eps, cs, pos, rot, interleaved):
    """x: (T, heads, D) double.  Returns (y, A): A the sum of magnitudes behind each output value."""
    T, H, D = x.shape
    n = x
    if w is not None:
        eps = float(torch.tensor(eps, dtype=torch.float32))
        n = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, A = n.clone(), n.abs()
    if rot:
        c, s = cs[pos.long(), :rot // 2].double()[:, None], cs[pos.long(), rot // 2:rot].double()[:, None]
        ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        a, b = n[..., ia], n[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        A[..., ia], A[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, A


def quantize(x32, g):
    """NVFP4 of fp32 rows by the rule's fp32 steps: (codes 0..15, E4M3 scale bytes)."""
    g = torch.tensor(g, dtype=torch.float32)
    b = x32.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / (torch.tensor(6.0) * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    div = (s.float() * g)[..., None].expand_as(b)
    v = torch.where(div > 0, b / div, torch.zeros(()))
    a = v.abs().double()
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    lo = (a[..., None] > mid).sum(-1)
    tie = (a[..., None] == mid).any(-1)
    code = lo + (tie & (lo % 2 == 1))
    code = code + 8 * ((v < 0) | ((v == 0) & torch.signbit(v))).long()
    return code.flatten(-2), s.view(torch.uint8)


def values(codes, scales, g=1.0):
    v = E2M1[codes].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).double()[..., None]
    return (v * float(torch.tensor(g, dtype=torch.float32))).flatten(-2)


def put(cache, page, Hkv, D, slots, kc, ks, vc, vs):
    """Write codes (T, Hkv, D) and scale bytes (T, Hkv, D / 16) of K and V into the cache's bytes, in place."""
    c = cache.view(-1, Hkv, page // 16, 18 * D)
    byte = lambda t: (t[..., 0::2] | (t[..., 1::2] << 4)).to(torch.uint8)  # noqa: E731
    kb, vb = byte(kc), byte(vc)
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        g, r = c[s // page, :, s % page // 16], s % 16
        g[:, r * (D // 2):(r + 1) * (D // 2)] = kb[t]
        g[:, 8 * D + r * (D // 16):8 * D + (r + 1) * (D // 16)] = ks[t]
        for blk in range(D // 16):
            g[:, 9 * D + blk * 128 + r * 8:9 * D + blk * 128 + r * 8 + 8] = vb[t, :, blk * 8:blk * 8 + 8]
            g[:, 17 * D + blk * 16 + r] = vs[t, :, blk]


def random_cache(n_pages, page, Hkv, D, gen, k_size=1.0, v_size=1.0):
    """(cache bytes, K values, V values) of random tokens; values (slots, Hkv, D) double under scale 1."""
    n = n_pages * page
    kx, vx = k_size * torch.randn(n, Hkv, D, generator=gen), v_size * torch.randn(n, Hkv, D, generator=gen)
    kc, ks = quantize(kx, 1.0)
    vc, vs = quantize(vx, 1.0)
    cache = torch.zeros(n_pages * Hkv * page // 16 * 18 * D, dtype=torch.uint8)
    # the bytes of every slot at once, by the layout
    c = cache.view(n_pages, Hkv, page // 16, 18 * D)
    byte = lambda t: (t[..., 0::2] | (t[..., 1::2] << 4)).to(torch.uint8)  # noqa: E731
    tok = lambda t: t.view(n_pages, page // 16, 16, Hkv, -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    c[..., :8 * D] = tok(byte(kc)).reshape(n_pages, Hkv, page // 16, 8 * D)
    c[..., 8 * D:9 * D] = tok(ks).reshape(n_pages, Hkv, page // 16, D)
    c[..., 9 * D:17 * D] = tok(byte(vc)).unflatten(-1, (D // 16, 8)).transpose(3, 4).reshape(n_pages, Hkv, page // 16, 8 * D)
    c[..., 17 * D:] = tok(vs).transpose(3, 4).reshape(n_pages, Hkv, page // 16, D)
    return cache, values(kc, ks), values(vc, vs)


def attention(q, k, v, L, scale, window=0):
    """One sequence: q (n, Hq, D), k and v (L, Hkv, D), all double.  Returns (out, tol_p, tol_s): out (n, Hq, D);
    tol_p = sum of p |v| per value; tol_s = the largest scale * sum |q k| of a row's visible tokens; and
    tol_v = sum |v| / l over visible tokens, l the softmax sum relative to its largest term."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("ihd,thd->iht", q, kk) * scale
    A = torch.einsum("ihd,thd->iht", q.abs(), kk.abs()) * abs(scale)
    t, p = torch.arange(L), torch.arange(n) + L - n
    seen = t[None] <= p[:, None]
    if window:
        seen &= t[None] > p[:, None] - window
    seen = seen[:, None].expand(n, Hq, L)
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    tp, tv = torch.zeros_like(out), torch.zeros_like(out)
    if L == 0:
        return out, tp, torch.zeros(n, Hq, dtype=torch.float64), tv
    m = s.masked_fill(~seen, -torch.inf).amax(-1, keepdim=True)
    e = torch.where(seen, (s - torch.where(m.isinf(), 0.0, m)).exp(), 0.0)
    l = e.sum(-1, keepdim=True)
    l1 = torch.where(l > 0, l, 1.0)
    out = torch.einsum("iht,thd->ihd", e / l1, vv)
    tp = torch.einsum("iht,thd->ihd", e / l1, vv.abs())
    tv = torch.einsum("iht,thd->ihd", seen.double(), vv.abs()) / l1
    ts = torch.where(seen, A, 0.0).amax(-1)
    return out, tp, ts, tv


def attention_tol(out, tp, ts, tv, D, L):
    """How far the kernel's bf16 output may be from `out`.
    A score is a sum of D exact products in fp32: within (2 D + 4) 2^-24 A of its value (any order, one truncation
    an add, the scale's two roundings), and the running maximum that is taken off it is such a score: a
    probability is off by twice that, by the exponential (2^-21) and by its rounding to fp16 (half a step, 2^-11,
    or 2^-25 of the largest probability where fp16 has no normal numbers).  The sum below it has the same without
    the fp16 part.  P V and the sum are fp32 sums of L terms (2 L 2^-24), joined in a few more roundings (32 2^-24).
    The output is rounded to bf16 (2^-8)."""
    e = 2 * (2 * D + 4) * 2.0 ** -24 * ts[..., None]
    rel = 2 * (torch.expm1(e) + 2.0 ** -21) + 2.0 ** -11 + (4 * L + 32) * 2.0 ** -24
    t = tp * rel + tv * 2.0 ** -25
    return t + 2.0 ** -8 * (out.abs() + t)
