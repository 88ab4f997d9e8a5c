"""Measured cases of the 4-bit paged cache and of the rotary positions.

The pruned cache in four bits: a pool of pages, ``cache`` uint8
[n_pages, page_bytes], and a page table, ``pages`` int32 [B, max_pages]; head
b's row j lies in page pages[b, j // page_size].  A page is page_size / 16
blocks of 16 rows, one after another; a block holds, for head dimension d
with NG = d / 64 groups,

  K codes   16 rows of d/2 bytes: 32-bit words [4 c][NG g][2 u], the word of
            (c, g, u) holding dims 64g + 16c + 8u + 0..7 as nibbles
            0, 2, 4, 6, 1, 3, 5, 7 from bit 0 up, the word rotated left by 3
  V codes   8 row pairs of d bytes: 16-bit units [8 r][NG g][2 w][2 row], the
            unit of (r, g, w, row) holding dims 64g + 8r + 4w + 0..3 of that
            row as nibbles from bit 0 up
  K scales  [16 rows][NG] pairs of bf16 (step s, minimum m)
  V scales  the same

A value is s * code + m.  A row and group of 64 values is quantised as
m = min, s = bf16((max - min) * (1/15)), code = round((x - m) * (1/s)), each
step one float32 operation.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 64
ROWS = 16                                            # rows of a block
NIBBLE = [0, 16, 4, 20, 8, 24, 12, 28]               # shift of dim 0..7 in an (unrotated) K word


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the grouped queries of a whole 8K-token layer, taken as a projection leaves them (token-major) and laid
        # out per head for scoring while they are rotated
        dict(name="rotary_layer", op="rotary", B=8, G=4, n=8224, d=128, rot=128, interleaved=False, inverse=False,
             token_major=True, start=0, mix=1),
        # half of each head, pairs interleaved, turned back (the gradient): a short ragged prompt far into a context
        dict(name="rotary_back_part", op="rotary", B=8, G=1, n=1003, d=128, rot=64, interleaved=True, inverse=True,
             token_major=False, start=131072, mix=2),
        # one new token of a decoding batch: 16 sequences x 8 heads, each at its own length
        dict(name="append_token", op="append", B=128, G=4, T=1, d=128, fill=900, page=64, rot=128, interleaved=False,
             ragged=False, mix=3),
        # a question appended behind a compressed context in one call, a padded batch of 4 sequences x 8 heads
        dict(name="append_prompt", op="append", B=32, G=4, T=515, d=128, fill=2457, page=64, rot=128,
             interleaved=False, ragged=True, mix=4),
        # a whole decoding step of one layer: rotate, append, attend
        dict(name="step_layer", op="step", B=64, G=4, T=1, d=128, fill=2457, page=64, rot=128, interleaved=False,
             ragged=False, mix=5),
        # attention of one new token over one pruned layer (8 heads, 30% of 8192 keys)
        dict(name="decode_layer", op="decode", B=8, G=4, d=128, mean=2457, uneven=False, page=64, mix=6),
        # 8 layers of a 128K context at a quarter of the keys
        dict(name="decode_128k", op="decode", B=64, G=5, d=128, mean=32768, uneven=False, page=128, mix=7),
        # heads of very different lengths, as a selection across all heads leaves them; short pages, narrow heads
        dict(name="decode_uneven", op="decode", B=96, G=8, d=64, mean=5001, uneven=True, page=16, mix=8),
        # a pruned 8K layer written to four bits
        dict(name="compact_layer", op="compact", B=8, n_c=8192, d=128, ratio=0.3, uneven=False, page=64, mix=9),
        # 4 layers of 32K context, the budget shared by all heads
        dict(name="compact_stack", op="compact", B=32, n_c=32768, d=128, ratio=0.3, uneven=True, page=64, mix=10),
        # a short pruned cache read back as bf16 rows
        dict(name="expand_layer", op="expand", B=8, d=128, mean=2457, uneven=False, page=64, mix=11),
        # a large uneven one with narrow heads
        dict(name="expand_uneven", op="expand", B=64, d=64, mean=9001, uneven=True, page=48, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "step", "decode", "decode", "compact", "expand"])
    d = rng.choice([64, 128])
    mix = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 48, 64, 128])
    rot = 16 * rng.randint(1, d // 16)
    if op == "rotary":
        B, G = rng.randint(1, 16), rng.randint(1, 8)
        return dict(op=op, B=B, G=G, n=_log(rng, 1, 262144 // (B * G)), d=d, rot=rot,
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, token_major=rng.random() < 0.5,
                    start=rng.choice([0, rng.randrange(131072)]), mix=mix)
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, G=rng.randint(1, 8), T=_log(rng, 1, max(1, 16384 // B)), d=d,
                    fill=_log(rng, 1, 3000), page=page, rot=rot, interleaved=rng.random() < 0.5,
                    ragged=rng.random() < 0.5, mix=mix)
    if op == "step":
        B = _log(rng, 1, 128)
        return dict(op=op, B=B, G=rng.randint(1, 8), T=1, d=d, fill=_log(rng, 1, 262144 // B), page=page, rot=rot,
                    interleaved=rng.random() < 0.5, ragged=False, mix=mix)
    if op == "compact":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, n_c=_log(rng, 16, 1048576 // B), d=d, ratio=rng.choice([0.1, 0.25, 0.3, 0.5]),
                    uneven=rng.random() < 0.5, page=page, mix=mix)
    B = _log(rng, 1, 128)
    case = dict(op=op, B=B, d=d, mean=_log(rng, 1, (2097152 if op == "decode" else 524288) // B),
                uneven=rng.random() < 0.5, page=page, mix=mix)
    if op == "decode":
        case["G"] = rng.randint(1, 8)
    return case


def _lengths(case, mean):
    """Rows of each head: all `mean`, or spread as a budget across heads spreads them (some heads empty)."""
    B = case["B"]
    if not case.get("uneven"):
        return [mean] * B
    r = random.Random(case["mix"])
    w = [0.0 if r.random() < 0.05 else math.exp(r.gauss(0.0, 0.8)) for _ in range(B)]
    total = sum(w) or 1.0
    got = [min(int(mean * B * x / total), 8 * mean) for x in w]
    return [max(1, got[0])] + got[1:]


def _fills(case):
    """Rows each head holds before an append, and how many it gets."""
    r = random.Random(case["mix"])
    fill = [r.randint(max(1, case["fill"] // 2), case["fill"]) for _ in range(case["B"])]
    new = [r.randint(0, case["T"]) if case["ragged"] else case["T"] for _ in range(case["B"])]
    return fill, new


def _kept(case):
    if case["uneven"]:
        mean = max(1, int(case["ratio"] * case["n_c"]))
        return [min(x, case["n_c"]) for x in _lengths(case, mean)]
    return [int(math.floor(case["ratio"] * case["n_c"]))] * case["B"]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _channels(g, d):
    """A few large channels, as key caches have."""
    return torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))


def _table(n_pos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _to_blocks(codes_k, sm_k, codes_v, sm_v):
    """Rows of codes (uint8 [R, d]) and scales (bf16 [R, NG, 2]) as the bytes of R / 16 blocks."""
    R, d = codes_k.shape
    NG = d // GROUP
    sh = torch.tensor(NIBBLE, dtype=torch.int32, device=DEV)
    w = codes_k.view(R, NG, 4, 2, 8).int() << sh
    w = w[..., :4].sum(-1, dtype=torch.int32) | (w[..., 4:6].sum(-1, dtype=torch.int32) |
                                                 (w[..., 6] | w[..., 7]))
    w = (w << 3) | ((w >> 29) & 7)
    kb = w.permute(0, 2, 1, 3).contiguous().view(torch.uint8).view(R // ROWS, -1)
    v = codes_v.view(R // 2, 2, NG, 8, 2, 4).int()
    h = (v[..., 0] | (v[..., 1] << 4) | (v[..., 2] << 8) | (v[..., 3] << 12))
    h = torch.where(h > 32767, h - 65536, h).to(torch.int16)                     # [pair, row, g, r, w]
    vb = h.permute(0, 3, 2, 4, 1).contiguous().view(torch.uint8).view(R // ROWS, -1)
    ks = sm_k.contiguous().view(torch.uint8).view(R // ROWS, -1)
    vs = sm_v.contiguous().view(torch.uint8).view(R // ROWS, -1)
    return torch.cat([kb, vb, ks, vs], 1)


def _quantise(x):
    """Codes (float), steps and minima (bf16-valued float) of float32 rows [R, d]."""
    R, d = x.shape
    x = x.view(R, d // GROUP, GROUP)
    m = x.amin(-1, keepdim=True)
    r = x.amax(-1, keepdim=True) - m
    s = (r * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).to(torch.bfloat16).float()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    inv = torch.where(s > 0, torch.reciprocal(torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(s))
    return torch.round((x - m) * inv), s, m


def _value(x):
    """The values that float32 rows [R, d] stand for once they are held in four bits, in bf16."""
    c, s, m = _quantise(x)
    return (s * c + m).to(torch.bfloat16).view(x.shape)


def _pool(case, g, lengths, spare):
    """A pool of shuffled pages with keys and values of `lengths` rows a head (and room for `spare` more)."""
    d, page = case["d"], case["page"]
    per = [max(1, -(-(n + e) // page)) for n, e in zip(lengths, spare)]
    total = sum(per)
    width = max(per)
    perm = torch.randperm(total + 2, generator=g, device=DEV)
    table = torch.full((case["B"], width), -1, dtype=torch.int32)
    at = [0]
    for n in per:
        at.append(at[-1] + n)
    cols = torch.arange(width)
    n_of, first = torch.tensor(per), torch.tensor(at[:-1])
    index = (first[:, None] + cols).to(DEV)
    inside = (cols < n_of[:, None]).to(DEV)
    table = torch.where(inside, perm[index.clamp(max=total - 1)].int(), table.to(DEV))
    bytes_ = page * d * 9 // 8
    cache = torch.full((total + 2, bytes_), 255, dtype=torch.uint8, device=DEV)   # unused pages hold NaN scales
    chan = _channels(g, d)
    step = max(1, (1 << 20) // page)                                              # pages filled at a time
    for p0 in range(0, total, step):
        p1 = min(total, p0 + step)
        R = (p1 - p0) * page
        parts = []
        for mul in (chan, 1.0):
            x = (torch.randn((R, d), generator=g, device=DEV) * mul).to(torch.bfloat16).float()
            c, s, m = _quantise(x)
            parts += [c.to(torch.uint8).view(R, d), torch.cat([s, m], -1).to(torch.bfloat16)]
        cache[perm[p0:p1]] = _to_blocks(*parts).view(p1 - p0, bytes_)
    return cache, table


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)
    op, B, d = case["op"], case["B"], case["d"]
    st = dict(case)
    if op == "rotary":
        n, G = case["n"], case["G"]
        st["x"] = _normal(g, (n, B, G, d)).permute(1, 2, 0, 3) if case["token_major"] else _normal(g, (B, G, n, d))
        st["positions"] = torch.arange(case["start"], case["start"] + n, dtype=torch.int32, device=DEV)
        st["table"] = _table(case["start"] + n, case["rot"])
        return st
    if op in ("append", "step"):
        T, G = case["T"], case["G"]
        fill, new = _fills(case)
        st["cache"], st["pages"] = _pool(case, g, fill, new)
        st["counts"] = torch.tensor(fill, dtype=torch.int32, device=DEV)
        st["n_new"] = torch.tensor(new, dtype=torch.int32, device=DEV) if case["ragged"] else None
        st["offsets"] = torch.tensor([0] + new, dtype=torch.int64, device=DEV).cumsum(0)
        st["rows"] = sum(new)
        st["k"] = (torch.randn((T, B, d), generator=g, device=DEV) * _channels(g, d)).to(torch.bfloat16).permute(1, 0, 2)
        st["v"] = _normal(g, (T, B, d)).permute(1, 0, 2)
        st["q"] = _normal(g, (T, B, G, d)).permute(1, 2, 0, 3)
        st["q_out"] = torch.zeros((B, G, T, d), dtype=torch.bfloat16, device=DEV)
        far = random.Random(case["mix"] + 1)
        starts = torch.tensor([n + far.randrange(4096) for n in fill], dtype=torch.int32)
        st["positions"] = (starts[:, None] + torch.arange(T, dtype=torch.int32)).to(DEV)
        st["table"] = _table(int(starts.max()) + T, case["rot"])
        live = torch.arange(T) < torch.tensor(new)[:, None]
        st["live"] = live.to(DEV)
        st["index"] = live.reshape(-1).nonzero().view(-1).to(DEV)                  # the new rows that count
        return st
    if op == "compact":
        n_c = case["n_c"]
        kept = _kept(case)
        chan = _channels(g, d)
        st["K"] = torch.empty((B, n_c, d), dtype=torch.bfloat16, device=DEV)
        st["V"] = torch.empty((B, n_c, d), dtype=torch.bfloat16, device=DEV)
        for b in range(0, B, 8):
            shape = st["K"][b:b + 8].shape
            st["K"][b:b + 8] = (torch.randn(shape, generator=g, device=DEV) * chan).to(torch.bfloat16)
            st["V"][b:b + 8] = _normal(g, shape)
        counts = torch.tensor(kept, dtype=torch.int32, device=DEV)
        rank = torch.rand((B, n_c), generator=g, device=DEV).argsort(1).argsort(1)
        st["idx"] = (rank < counts[:, None]).nonzero()[:, 1].int().contiguous()
        if not st["idx"].numel():
            st["idx"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        st["counts"] = counts
        st["offsets"] = torch.tensor([0] + kept, dtype=torch.int64, device=DEV).cumsum(0)
        st["rows"] = sum(kept)
        page = case["page"]
        per = [-(-n // page) for n in kept]
        width = max(1, max(per))
        perm = torch.randperm(B * width, generator=g, device=DEV).int().view(B, width)
        st["pages"] = perm
        st["cache"] = torch.full((B * width, page * d * 9 // 8), 255, dtype=torch.uint8, device=DEV)
        st["head"] = torch.repeat_interleave(torch.arange(B, device=DEV), counts.long())
        return st
    lengths = _lengths(case, case["mean"])
    st["cache"], st["pages"] = _pool(case, g, lengths, [0] * B)
    st["counts"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    if op == "decode":
        st["q"] = _normal(g, (B, case["G"], d))
    else:
        st["offsets"] = torch.tensor([0] + lengths, dtype=torch.int64, device=DEV).cumsum(0)
        st["rows"] = sum(lengths)
        st["slots"] = (torch.arange(st["pages"].shape[1] * case["page"], device=DEV) <
                       st["counts"][:, None]).view(-1).nonzero().view(-1)         # the rows that count
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rotate(x, positions, table, rot, interleaved, inverse):
    """Rotary positions of x [..., n, d] (positions [..., n]); float32, rounded once."""
    t = table[positions.long()]
    c, s = t[..., : rot // 2], t[..., rot // 2:]
    s = -s if inverse else s
    f = x[..., :rot].float()
    if interleaved:
        a, b = f[..., 0::2], f[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = f[..., : rot // 2], f[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y.to(torch.bfloat16), x[..., rot:]], -1)


def _rows(st):
    """Every row of the cache as float32 (K, V) [B, max_pages * page, d]; rows past a head's count mean nothing."""
    d, B = st["d"], st["B"]
    NG = d // GROUP
    rec = st["cache"][st["pages"].clamp(min=0).long()].view(-1, ROWS * d * 9 // 8)
    n = rec.shape[0]
    half = ROWS * d // 2
    w = rec[:, :half].contiguous().view(torch.int32)
    w = ((w >> 3) & 0x1FFFFFFF) | (w << 29)
    w = w.view(n, ROWS, 4, NG, 2).permute(0, 1, 3, 2, 4)
    sh = torch.tensor(NIBBLE, dtype=torch.int32, device=DEV)
    ck = ((w.unsqueeze(-1) >> sh) & 15).float().reshape(n, ROWS, NG, GROUP)
    h = rec[:, half:2 * half].contiguous().view(torch.int16).view(n, 8, 8, NG, 2, 2).permute(0, 1, 5, 3, 2, 4)
    cv = ((h.unsqueeze(-1).int() >> torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=DEV)) & 15).float()
    cv = cv.reshape(n, ROWS, NG, GROUP)
    sm = rec[:, 2 * half:].contiguous().view(torch.bfloat16).view(n, 2, ROWS, NG, 2).float()
    k = ck * sm[:, 0, ..., :1] + sm[:, 0, ..., 1:]
    v = cv * sm[:, 1, ..., :1] + sm[:, 1, ..., 1:]
    return k.view(B, -1, d), v.view(B, -1, d)


def _attend(q, k, v, counts, scale):
    """Attention of q [B, G, d] over the first counts[b] rows of k, v [B, N, d]: (out, log2 of the denominator)."""
    x = torch.matmul(q.float(), k.transpose(1, 2)) * (scale * math.log2(math.e))
    out_of = (torch.arange(k.shape[1], device=k.device) >= counts[:, None])[:, None]
    x = x.masked_fill(out_of, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp2(x - m)
    den = p.sum(-1, keepdim=True)
    v = v.masked_fill(out_of.transpose(1, 2), 0.0)
    out = torch.matmul(p, v) / torch.where(den > 0, den, torch.ones_like(den))
    return out, (m + torch.log2(den))[..., 0]


def _plain(st):
    op, B, d = st["op"], st["B"], st["d"]
    if op == "rotary":
        return _rotate(st["x"], st["positions"], st["table"], st["rot"], st["interleaved"], st["inverse"])
    if op in ("append", "step"):
        k = _rotate(st["k"], st["positions"], st["table"], st["rot"], st["interleaved"], False)
        q = _rotate(st["q"], st["positions"][:, None], st["table"], st["rot"], st["interleaved"], False)
        q = q.masked_fill(~st["live"][:, None, :, None], 0.0)
        lengths = st["counts"] + (st["T"] if st["n_new"] is None else st["n_new"])
        if op == "append":
            kr = k.reshape(-1, d)[st["index"]].float()
            vr = st["v"].reshape(-1, d)[st["index"]].float()
            return dict(q=q, counts=lengths, K=_value(kr), V=_value(vr))
        kc, vc = _rows(st)
        at = st["counts"].long()
        rows = torch.arange(B, device=DEV)
        (ck, sk, mk), (cv, sv, mv) = (_quantise(t.reshape(-1, d).float()) for t in (k, st["v"]))
        kc[rows, at] = (sk * ck + mk).view(B, d)
        vc[rows, at] = (sv * cv + mv).view(B, d)
        out, lse2 = _attend(q.view(B, st["G"], d), kc, vc, lengths, d ** -0.5)
        return dict(out=out, lse2=lse2, counts=lengths)
    if op == "compact":
        j = st["idx"].long()[: st["rows"]]
        return dict(K=_value(st["K"][st["head"], j].float()), V=_value(st["V"][st["head"], j].float()))
    k, v = _rows(st)
    if op == "decode":
        out, lse2 = _attend(st["q"], k, v, st["counts"], d ** -0.5)
        return dict(out=out, lse2=lse2)
    return dict(K=k.view(-1, d)[st["slots"]].to(torch.bfloat16), V=v.view(-1, d)[st["slots"]].to(torch.bfloat16))


def _own(st):
    import query_agnostic_kv_kvz_b200 as kvz
    op, d = st["op"], st["d"]
    if op == "rotary":
        return kvz.kvz_rotary(st["x"], st["positions"], st["table"], interleaved=st["interleaved"],
                              inverse=st["inverse"])
    cache, pages, page = st["cache"], st["pages"], st["page"]
    if op in ("append", "step"):
        counts, q = kvz.kvz_append_int4(st["k"], st["v"], cache, pages, st["counts"], page,
                                        positions=st["positions"], table=st["table"],
                                        interleaved=st["interleaved"], q=st["q"], q_out=st["q_out"],
                                        n_new=st["n_new"])
        if op == "append":
            K, V = kvz.kvz_expand_int4(cache, pages, counts, st["offsets"], page, first=st["counts"],
                                       out_rows=st["rows"])
            return dict(q=q, counts=counts, K=K, V=V)
        out, lse2 = kvz.kvz_decode_int4(q.view(st["B"], st["G"], d), cache, pages, counts, page)
        return dict(out=out, lse2=lse2, counts=counts)
    if op == "decode":
        out, lse2 = kvz.kvz_decode_int4(st["q"], cache, pages, st["counts"], page)
        return dict(out=out, lse2=lse2)
    if op == "compact":
        kvz.kvz_compact_int4(st["K"], st["V"], st["idx"], st["counts"], st["offsets"], cache, pages, page)
    K, V = kvz.kvz_expand_int4(cache, pages, st["counts"], st["offsets"], page, out_rows=st["rows"])
    return dict(K=K, V=V)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, B, d = case["op"], case["B"], case["d"]
    row4, row16 = d * 9 // 8, 4 * d                       # a row of K and V in four bits, in bf16
    if op == "rotary":
        values = B * case["G"] * case["n"] * d
        return dict(bytes=4 * values + case["n"] * (4 * case["rot"] + 4),
                    flops=3 * B * case["G"] * case["n"] * case["rot"])
    if op in ("append", "step"):
        fill, new = _fills(case)
        n = sum(new)
        moved = n * (row16 + row4) + n * case["G"] * 4 * d + 12 * B + n * (4 * case["rot"] + 4)
        flops = n * (3 * case["rot"] * (1 + case["G"]) + 10 * d)
        if op == "append":
            return dict(bytes=moved + n * row16, flops=flops + 4 * n * d)
        rows = sum(fill)
        return dict(bytes=moved + rows * row4 + B * case["G"] * (4 * d + 4), flops=flops + 4 * (rows + n) * case["G"] * d)
    if op == "compact":
        n = sum(_kept(case))
        return dict(bytes=n * (2 * row16 + row4 + 4), flops=n * 14 * d)
    n = sum(_lengths(case, case["mean"]))
    if op == "decode":
        return dict(bytes=n * row4 + B * case["G"] * (6 * d + 4), flops=4 * n * case["G"] * d)
    return dict(bytes=n * (row4 + row16), flops=4 * n * d)


# ---------------------------------------------------------------------------
# The same from the definition, in 64 bits
# ---------------------------------------------------------------------------
def _f32(x):
    """A float64 step result as the float32 step of the definition leaves it."""
    return x.float().double()


def _same(x):
    return x


def _exact_turn(x, positions, table, rot, interleaved, sign, step=_same):
    z = x.double().clone()
    ang = table[positions.long()].double()
    co, si = ang[..., : rot // 2], sign * ang[..., rot // 2:]
    i = torch.arange(rot // 2, device=DEV)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    re, im = z[..., ia], z[..., ib]
    z[..., ia] = step(step(re * co) - step(im * si))
    z[..., ib] = step(step(im * co) + step(re * si))
    return z


def _exact_value(x):
    """Values of bf16 rows [R, d] held in four bits.  A code is a whole number that float32 steps decide (a value
    next to a border falls to one side by them), so these are taken one by one; what they are applied to is 64 bits."""
    x = x.double().view(x.shape[0], -1, GROUP)
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    fifteenth = _f32(torch.tensor(1.0 / 15.0, dtype=torch.float64, device=DEV))
    s = _f32(_f32(hi - lo) * fifteenth).to(torch.bfloat16).double()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    inv = _f32(1.0 / torch.where(s > 0, s, torch.ones_like(s)))
    q = torch.where(s > 0, torch.round(_f32(_f32(x - lo) * inv)), torch.zeros_like(x))
    return (q * s + lo).view(x.shape[0], -1)


def _exact_head(st, b, n):
    """The first n rows of head b, byte by byte: (K, V) float64 [n, d]."""
    d, page = st["d"], st["page"]
    NG = d // GROUP
    rec = st["cache"].view(-1, page // ROWS, ROWS * d * 9 // 8)[st["pages"][b, : -(-n // page)].long()]
    rec = rec.flatten(0, 1)[: -(-n // ROWS)].long()
    dim = torch.arange(d, device=DEV)
    row = torch.arange(ROWS, device=DEV)[:, None]
    g, o = dim // 64, dim % 64
    # K: bit position of each dim's nibble within its row of d / 2 bytes (words rotated left by 3)
    word = (o // 16) * NG * 2 + g * 2 + (o % 16) // 8
    e = o % 8
    k = torch.zeros((rec.shape[0], ROWS, d), dtype=torch.float64, device=DEV)
    for bit in range(4):
        p = ((e % 2) * 16 + (e // 2) * 4 + bit + 3) % 32
        k += ((rec[:, row * (d // 2) + word * 4 + p // 8] >> (p % 8)) & 1).double() * (1 << bit)
    unit = (row // 2) * (d // 2) + (((o // 8) * NG + g) * 2 + (o % 8) // 4) * 2 + row % 2
    at = ROWS * d // 2 + unit * 2 + (o % 4) // 2
    v = ((rec[:, at] >> (4 * (o % 2))) & 15).double()
    sm = rec[:, ROWS * d:].to(torch.uint8).contiguous().view(torch.bfloat16).double().view(-1, 2, ROWS, NG, 2)
    sm = sm.repeat_interleave(GROUP, dim=3)
    k = k * sm[:, 0, ..., 0] + sm[:, 0, ..., 1]
    v = v * sm[:, 1, ..., 0] + sm[:, 1, ..., 1]
    return k.view(-1, d)[:n], v.view(-1, d)[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op, B, d = case["op"], case["B"], case["d"]
    if op == "rotary":
        return _exact_turn(st["x"], st["positions"], st["table"], case["rot"], case["interleaved"],
                           -1.0 if case["inverse"] else 1.0)
    if op == "compact":
        pick = st["idx"][: st["rows"]].long()
        return dict(K=_exact_value(st["K"][st["head"], pick]), V=_exact_value(st["V"][st["head"], pick]))
    if op in ("append", "step"):
        rot, il = case["rot"], case["interleaved"]
        k = _exact_turn(st["k"], st["positions"], st["table"], rot, il, 1.0, _f32).to(torch.bfloat16)
        q = _exact_turn(st["q"], st["positions"][:, None], st["table"], rot, il, 1.0, _f32)
        q = q * st["live"][:, None, :, None]
        kn = _exact_value(k.reshape(-1, d)[st["index"]])
        vn = _exact_value(st["v"].reshape(-1, d)[st["index"]])
        if op == "append":
            return dict(q=q, counts=None, K=kn, V=vn)
        q = q.to(torch.bfloat16).double()
    if op == "expand":
        heads = [_exact_head(st, b, n) for b, n in enumerate(st["counts"].tolist()) if n]
        return dict(K=torch.cat([h[0] for h in heads]), V=torch.cat([h[1] for h in heads])) if heads else None
    outs, lses = [], []
    for b, n in enumerate(st["counts"].tolist()):
        k, v = _exact_head(st, b, n)
        qb = q[b, :, 0] if op == "step" else st["q"][b].double()
        if op == "step":
            k, v = torch.cat([k, kn[b:b + 1]]), torch.cat([v, vn[b:b + 1]])
        z = qb @ k.T * d ** -0.5
        lse = torch.logsumexp(z, -1)
        outs.append(torch.exp(z - lse[:, None].clamp(min=-1e300)) @ v)
        lses.append(lse / math.log(2.0))
    return dict(out=torch.stack(outs), lse2=torch.stack(lses), counts=None)
