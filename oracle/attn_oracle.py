"""Plain definitions of the attention layers' operators: rotation, the 4-bit key/value format
and attention, in numpy.  Shares no code with the GPU path.

Integers and bf16 results that the format fixes (codes, scales, biases, rotated values) are
computed with the format's own fp32 roundings and are exact; attention is fp64, and comes with
a bound on what the kernels' arithmetic may differ by."""
from __future__ import annotations

import numpy as np

TILE = 16


def bf16_round(x):
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    x = np.asarray(x, np.float32)
    u = x.view(np.uint32)
    r = ((u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def rotate(x, table, positions):
    """x fp32 (bf16 values) [T][heads][D], table fp32 [positions][2][R/2] -> bf16 values."""
    x = np.asarray(x, np.float32)
    half = table.shape[2]
    c, s = (table[positions][:, i][:, None].astype(np.float32) for i in range(2))
    a, b = x[..., :half], x[..., half:2 * half]
    y = x.copy()
    y[..., :half] = bf16_round(a * c - b * s)
    y[..., half:2 * half] = bf16_round(b * c + a * s)
    return y


def quantise(x):
    """x fp32 (bf16 values) [..., 64] -> codes uint8 [..., 64], scale and bias fp32 [...]."""
    x = np.asarray(x, np.float32)
    h = np.float32(0.5)
    lo, hi = x.min(-1), x.max(-1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        s = bf16_round((hi * h - lo * h) / np.float32(7.5))
        c = np.rint((x * h - (lo * h)[..., None]) / (s * h)[..., None])
        c = np.where(s[..., None] > 0, np.clip(c, 0, 15), 0)
    odd = ~np.isfinite(x).all(-1)
    codes = np.where(odd[..., None], 0, np.nan_to_num(c)).astype(np.uint8)
    return codes, np.where(odd, np.float32(0), s).astype(np.float32), np.where(odd, np.float32(np.nan), lo).astype(np.float32)


def cache_bytes(kv_heads, D, P):
    return kv_heads * (P // TILE) * TILE * (D + D // 8)


def _regions(D):
    n = D // 64
    v, ks = TILE * D // 2, TILE * D
    vs = ks + TILE * n * 4
    return (0, ks), (v, vs)


def store(cache, P, slot, head, which, x):
    """One row x (fp32, bf16 values [D]) into slot `slot` of cache uint8 [pages][bytes]."""
    D = x.shape[0]
    n = D // 64
    codes, s, b = quantise(x.reshape(n, 64))
    page, place = divmod(int(slot), P)
    tile = (head * (P // TILE) + place // TILE) * TILE * (D + D // 8)
    q_at, sb_at = _regions(D)[which]
    row = place % TILE
    words = np.zeros(D // 8, np.uint32)
    for j in range(8):
        for g in range(n):
            for i in range(8):
                words[j * n + g] |= np.uint32(codes[g, 8 * j + i]) << np.uint32(4 * i)
    at = tile + q_at + row * D // 2
    cache[page, at:at + D // 2] = words.view(np.uint8)
    sb = (s.view(np.uint32) >> np.uint32(16)) | (b.view(np.uint32) & np.uint32(0xFFFF0000))
    sb = np.where(np.isnan(b), np.uint32(0x7FC00000), sb).astype(np.uint32)
    at = tile + sb_at + row * n * 4
    cache[page, at:at + 4 * n] = sb.view(np.uint8)


def load(cache, D, P, page_table, count):
    """Codes, scales and biases (fp64) of tokens 0 .. count - 1: [2 (k, v)][heads][count][D], the
    last two spread over their groups."""
    n, tpp = D // 64, P // TILE
    tb = TILE * (D + D // 8)
    heads = cache.shape[1] // (tpp * tb)
    pages = cache[np.asarray(page_table[:-(-count // P)], np.int64)].reshape(-1, heads, tpp, tb)
    tiles = pages.transpose(1, 0, 2, 3).reshape(heads, -1, tb)
    out = []
    for q_at, sb_at in _regions(D):
        w = np.ascontiguousarray(tiles[..., q_at:q_at + TILE * D // 2]).view("<u4").reshape(heads, -1, TILE, 8, n)
        codes = (w[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15  # [.., j, g, i]
        codes = codes.transpose(0, 1, 2, 4, 3, 5).reshape(heads, -1, D)[:, :count].astype(np.float64)
        sb = np.ascontiguousarray(tiles[..., sb_at:sb_at + TILE * n * 4]).view("<u4").reshape(heads, -1, n)[:, :count]
        s = (sb << np.uint32(16)).view(np.float32).astype(np.float64)
        b = (sb & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
        out.append((codes, np.repeat(s, 64, -1), np.repeat(b, 64, -1)))
    return out


def weights(scores, seen):
    """Softmax over the last axis where `seen`; rows that see nothing are zeros."""
    x = np.where(seen, scores, -np.inf)
    m = x.max(-1, keepdims=True) if x.shape[-1] else np.zeros(x.shape[:-1] + (1,))
    p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    p = np.where(seen, p, 0.0)
    t = p.sum(-1, keepdims=True)
    return p / np.where(t == 0, 1.0, t)


# Half a step of bf16 and of fp32, relative to the value.
U16, U32 = 2.0 ** -8, 2.0 ** -24


def decode(q, cache, D, P, page_table, count, scale):
    """One query row q (fp64 [q_heads][D]) over the cached tokens -> (o, bound), fp64.

    The bound counts the kernel's roundings:
      o rounded to bf16                                       U16 |o|
      the weights p a rounded to bf16 with centred codes      U16 sum p a |c - 8|
      a score: at most D/16 + 24 fp32 roundings of terms whose magnitudes sum to
        t = scale sum_c |q_c| (33 a + |b|), an exponential error of 2^-22 and the rescalings;
        an error d of a score changes o by at most 2 d sum p |v|
      sums of the value side: at most count/16 + 64 fp32 roundings of terms that sum to
        sum p (64 a + |b|)"""
    H = q.shape[0]
    out, bound = np.zeros((H, D)), np.zeros((H, D))
    if count <= 0:
        return out, bound
    (kc, ka, kb), (vc, va, vb) = load(cache, D, P, page_table, count)
    G = H // kc.shape[0]
    for h in range(H):
        g = h // G
        k, v = kc[g] * ka[g] + kb[g], vc[g] * va[g] + vb[g]
        p = weights(scale * (k @ q[h]), np.ones(count, bool))
        o = p @ v
        t = abs(scale) * (np.abs(q[h]) * (33 * np.abs(ka[g]) + np.abs(kb[g]))).sum(-1)
        d = (D / 16 + 24) * U32 * t.max() + 2.0 ** -21
        out[h] = o
        bound[h] = (U16 * np.abs(o) + U16 * (p @ (np.abs(va[g]) * np.abs(vc[g] - 8))) + 2 * d * (p @ np.abs(v))
                    + (count / 16 + 64) * U32 * (p @ (64 * np.abs(va[g]) + np.abs(vb[g])))) * 1.01
    return out, bound


def prompt(q, k, v, scale):
    """One sequence: q [Lq][H][D], k, v [Lk][KV][D] (fp64) -> (o, bound).

    The bound: o rounded to bf16, p rounded to bf16 (U16 sum p |v|), scores with D + 8 fp32
    roundings of terms that sum to scale sum |q k| and the exponential's error, sums of at most
    Lk fp32 roundings of p |v|."""
    Lq, H, D = q.shape
    Lk, KV = k.shape[:2]
    G = H // KV
    out, bound = np.zeros((Lq, H, D)), np.zeros((Lq, H, D))
    if Lk == 0:
        return out, bound
    seen = np.arange(Lk)[None] <= np.arange(Lq)[:, None] + Lk - Lq
    for h in range(H):
        kh, vh = k[:, h // G], v[:, h // G]
        p = weights(scale * (q[:, h] @ kh.T), seen)
        o = p @ vh
        t = abs(scale) * np.where(seen, np.abs(q[:, h]) @ np.abs(kh).T, 0.0).max(-1, keepdims=True)
        d = (D + 8) * U32 * t + 2.0 ** -21
        w = p @ np.abs(vh)
        out[:, h] = o
        bound[:, h] = (U16 * np.abs(o) + U16 * w + 2 * d * w + Lk * U32 * w) * 1.01
    return out, bound
