"""Independent NumPy oracle of the rotary positions and of the paged 4-bit
cache: the rotation, the quantisation (its codes are whole numbers that
float32 steps decide, so those are taken in float32 one by one), the byte
layout of a page, written here from its description bit by bit, and decode
attention in float64 over what the bytes stand for.

Shares no code with the CUDA library; bf16 tensors come and go as uint16 bits.
"""
from __future__ import annotations

import numpy as np

from oracle.kvz_oracle import bf16_bits_to_f64, decode_attention

__all__ = ["round_bf16", "rotary_table", "rotary", "quantize_groups", "group_values", "block_bytes", "unpack_block",
           "pack_block", "read_head", "decode_int4", "decode_bound", "decode_bound_by_group"]

GROUP = 64
ROWS = 16


def round_bf16(x) -> np.ndarray:
    """bf16 bits (uint16) of float32 values, round to nearest even; NaN stays NaN."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(np.asarray(x, dtype=np.float32)), np.uint16(0x7FC0), r)


def _f32(bits):
    return bf16_bits_to_f64(bits).astype(np.float32)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------
def rotary_table(freqs, n_pos, factor=1.0):
    a = np.arange(n_pos, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)
    return np.concatenate([np.cos(a) * factor, np.sin(a) * factor], 1).astype(np.float32)


def rotary(x_bits, positions, table, interleaved=False, inverse=False):
    """x_bits [..., n, d]; positions broadcast to [..., n]; returns bits."""
    x = _f32(x_bits)
    rot = table.shape[1]
    pos = np.broadcast_to(positions, x.shape[:-1])
    c, s = table[pos][..., : rot // 2], table[pos][..., rot // 2:]
    if inverse:
        s = -s
    y = x.copy()
    for i in range(rot // 2):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = a * c[..., i] - b * s[..., i]
        y[..., ib] = b * c[..., i] + a * s[..., i]
    out = np.array(x_bits, dtype=np.uint16, copy=True)
    out[..., :rot] = round_bf16(y[..., :rot])
    return out


# ---------------------------------------------------------------------------
# Quantisation
# ---------------------------------------------------------------------------
def quantize_groups(bits):
    """bf16 rows [R, d] -> (codes uint8 [R, d], step bits, minimum bits [R, NG] uint16)."""
    x = _f32(bits).reshape(bits.shape[0], -1, GROUP)
    with np.errstate(all="ignore"):
        m = x.min(-1)
        r = (x.max(-1) - m).astype(np.float32)
        s = _f32(round_bf16(r * np.float32(1.0 / 15.0)))
        s = np.where(s < np.float32(2.0 ** -126), np.float32(0), s)
        inv = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0)).astype(np.float32)
        y = ((x - m[..., None]).astype(np.float32) * inv[..., None]).astype(np.float32)
        fine = r < np.inf
        codes = np.where(fine[..., None], np.rint(np.where(fine[..., None], y, 0)), 0).astype(np.uint8)
    sb = np.where(fine, round_bf16(s), np.uint16(0x7FC0))
    mb = np.where(fine, round_bf16(m), np.uint16(0))
    return codes.reshape(bits.shape), sb, mb


def group_values(codes, sb, mb):
    """float32 values s * code + m of rows [R, d]."""
    R, d = codes.shape
    s, m = _f32(sb)[..., None], _f32(mb)[..., None]
    c = codes.reshape(R, d // GROUP, GROUP).astype(np.float32)
    with np.errstate(all="ignore"):
        return ((s * c).astype(np.float32) + m).astype(np.float32).reshape(R, d)


# ---------------------------------------------------------------------------
# Layout
# ---------------------------------------------------------------------------
def block_bytes(d):
    return 18 * d


def _places(d):
    """Bit position within a block of the lowest bit of every K nibble (a list
    of four bit positions each: a rotated word's nibble may wrap) and of every
    V nibble; [16][d]."""
    NG = d // GROUP
    k = np.zeros((ROWS, d, 4), dtype=np.int64)
    v = np.zeros((ROWS, d, 4), dtype=np.int64)
    order = [0, 2, 4, 6, 1, 3, 5, 7]              # the dim that each nibble holds
    for row in range(ROWS):
        for dim in range(d):
            g, o = divmod(dim, GROUP)
            c, u, e = o // 16, (o % 16) // 8, o % 8
            word = row * (d // 8) + (c * NG + g) * 2 + u
            nib = order.index(e)
            for bit in range(4):
                k[row, dim, bit] = 32 * word + (4 * nib + bit + 3) % 32
            r, w, e = o // 8, (o % 8) // 4, o % 4
            half = ((row // 2) * 8 + r) * NG + g
            half = (half * 2 + w) * 2 + row % 2
            for bit in range(4):
                v[row, dim, bit] = 8 * (8 * d) + 16 * half + 4 * e + bit
    return k, v


_PLACES = {}


def _bits_of(d):
    if d not in _PLACES:
        _PLACES[d] = _places(d)
    return _PLACES[d]


def pack_block(kc, ks, km, vc, vs, vm):
    """16 rows of codes [16, d], step and minimum bits [16, NG] -> bytes."""
    d = kc.shape[1]
    kp, vp = _bits_of(d)
    bits = np.zeros(8 * block_bytes(d), dtype=np.uint8)
    for bit in range(4):
        bits[kp[..., bit]] = (kc >> bit) & 1
        bits[vp[..., bit]] = (vc >> bit) & 1
    out = np.packbits(bits, bitorder="little")
    sm = np.stack([np.stack([ks, km], -1), np.stack([vs, vm], -1)])      # [2, 16, NG, 2]
    out[16 * d:] = np.ascontiguousarray(sm.astype(np.uint16)).view(np.uint8).reshape(-1)
    return out


def unpack_block(raw, d):
    """bytes of a block -> (kc, ks, km, vc, vs, vm)."""
    kp, vp = _bits_of(d)
    bits = np.unpackbits(np.asarray(raw, dtype=np.uint8), bitorder="little")
    kc = sum((bits[kp[..., b]] << b) for b in range(4)).astype(np.uint8)
    vc = sum((bits[vp[..., b]] << b) for b in range(4)).astype(np.uint8)
    sm = np.ascontiguousarray(raw[16 * d:]).view(np.uint16).reshape(2, ROWS, d // GROUP, 2)
    return kc, sm[0, ..., 0], sm[0, ..., 1], vc, sm[1, ..., 0], sm[1, ..., 1]


def read_head(cache, page_ids, page_size, d, n):
    """(K, V) float32 [n, d], the first n rows of a head whose pages are page_ids."""
    K, V = np.zeros((n, d), np.float32), np.zeros((n, d), np.float32)
    per = page_size // ROWS
    for blk in range(-(-n // ROWS)):
        raw = cache[page_ids[blk // per]].reshape(per, block_bytes(d))[blk % per]
        kc, ks, km, vc, vs, vm = unpack_block(raw, d)
        m = min(ROWS, n - blk * ROWS)
        K[blk * ROWS: blk * ROWS + m] = group_values(kc, ks, km)[:m]
        V[blk * ROWS: blk * ROWS + m] = group_values(vc, vs, vm)[:m]
    return K, V


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------
def decode_int4(q, cache, pages, counts, page_size, scale):
    """q float64 [B, G, d]; returns (out, lse2) float64."""
    outs, lses = [], []
    for b in range(q.shape[0]):
        K, V = read_head(cache, pages[b], page_size, q.shape[2], int(counts[b]))
        o, lse = decode_attention(q[b:b + 1], K.astype(np.float64), V.astype(np.float64),
                                  np.array([counts[b]]), np.array([0, counts[b]]), scale)
        outs.append(o[0])
        lses.append(lse[0])
    return np.stack(outs), np.stack(lses)


def decode_bound(q, K, V, scale):
    """What float32 can cost the attention of one head's queries q [G, d] over
    float rows K, V [n, d]: (bound on |d out| per query, on |d lse2|).

    A row's logit is a sum over d products q_i * (16 + code), at most 31 q_i
    steps, less 16 sum(q) steps, plus sum(q) times the minimum.  With r the
    largest step (range / 15) and u = 2^-24, each of the at most d / 16 + 8
    float32 additions on its way rounds by u times what has gathered, so a
    logit is off by at most (d / 16 + 8) u (47 r + |m|) sum|q| scale; exp2
    adds 2^-21.  A weight off by a factor 1 + e moves the normalised output by
    at most 2 e max|v|, and the output's own sums round by u times 47 r + |m|
    for each of the blocks a warp adds up, which is at most n / 16 + 32."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    n, d = K.shape
    u = 2.0 ** -24

    def reach(x):
        g = x.reshape(n, -1, GROUP)
        return float((47.0 / 15.0 * (g.max(-1) - g.min(-1)) + np.abs(g).max(-1)).max())

    e = (d / 16 + 8) * u * reach(K) * np.abs(q).sum(-1) * scale + 2.0 ** -21
    return 2 * e * np.abs(V).max() + (n / 16 + 32) * u * reach(V), 2 * e / np.log(2.0) + 2.0 ** -20


def decode_bound_by_group(q, K, V, scale):
    """The same per group of 64 dims and weighted by what each row counts for:
    float64 (out [G, d], bound on |d out| [G, d]) of one head.

    Every float32 step rounds by u = 2^-24 of what it holds, a matrix
    instruction's sum, which truncates, by 2 u.  With R = range + |min| of a
    row's group, a logit passes at most d / 16 + 8 such steps over at most
    sum_groups R sum|q|, a q below 2^-27 of the query's largest entry is held
    to 2^-35 of it, and the product with the scale and the reference's
    subtraction add 4 u (max |logit| + 20); exp2 adds 2^-21.  That makes e_j,
    the relative error of row j's weight.  Weights P_j (1 + e_j), normalised,
    move the output by at most sum_j P_j e_j (|v_j| + |out|).  A weight times a
    step is held to u of itself and to 2^-35 of the largest in its group (8
    codes of it at most are 2^-35 of that row's R), and the sums of what it
    multiplies round by 2 u of sum_j P_j R_j at most n / 32 + 32 times, the
    denominator's by as much of the output."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    n, d = K.shape
    u = 2.0 ** -24

    def reach(x):
        g = x.reshape(n, -1, GROUP)
        return (g.max(-1) - g.min(-1)) + np.abs(g.min(-1))                   # [n, NG]

    z = q @ K.T * scale                                                      # [G, n]
    P = np.exp(z - z.max(-1, keepdims=True))
    P /= P.sum(-1, keepdims=True)
    out = P @ V
    qa = np.abs(q).reshape(q.shape[0], -1, GROUP).sum(-1)                    # [G, NG]
    e = (d / 16 + 8) * 2 * u * (qa @ reach(K).T) * scale
    e += 2.0 ** -35 * np.abs(q).max(-1, keepdims=True) * GROUP * reach(K).sum(-1)[None] * scale
    e += 4 * u * (np.abs(z).max(-1, keepdims=True) + 20) + 2.0 ** -21
    steps = (n / 32 + 32) * 2 * u
    sums = np.repeat(P @ reach(V), GROUP, axis=-1)
    rest = np.repeat((P[..., None] * reach(V)[None]).max(1), GROUP, axis=-1) * n * 2.0 ** -35
    return out, rest + (P * e) @ np.abs(V) + (P * e).sum(-1, keepdims=True) * np.abs(out) + steps * (sums + np.abs(out))
