"""GPU parity of the paged 4-bit cache.  What is written (codes, scales and
their places) is bit for bit the oracle's, which takes the same float32 steps;
reading back is one float32 sum rounded to bf16, also bit for bit; attention
is held to the bound that its float32 steps allow (decode_bound), against
float64 over the values that the bytes stand for."""
import numpy as np
import pytest
import torch

from kvz_testutil import bits, f64
from oracle import kvz_oracle as orc
from oracle import kvz_oracle_int4 as o4
from query_agnostic_kv_kvz_b200 import synth

pytestmark = pytest.mark.gpu

kvz = pytest.importorskip("query_agnostic_kv_kvz_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kvz.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).bfloat16()


def table(rot, n_pos):
    f, a = kvz.kvz_rotary_freqs(rot)
    return kvz.kvz_rotary_table(f.cuda(), n_pos, a)


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def pool(caps, d, page, seed, spare=3):
    """Shuffled pages for heads of `caps` rows; unused bytes are 0xFF (NaN scales), unused entries -1."""
    per = [max(1, -(-n // page)) for n in caps]
    ids = torch.randperm(sum(per) + spare, generator=torch.Generator().manual_seed(seed))
    pages = torch.full((len(caps), max(per)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        pages[b, :n] = ids[at:at + n].int()
        at += n
    cache = torch.full((sum(per) + spare, page * d * 9 // 8), 255, dtype=torch.uint8, device="cuda")
    return cache, pages.cuda()


def filled(counts, d, page, seed, scale=1.0):
    """A cache that holds random rows, written by append: (cache, pages, counts, K bits, V bits per head)."""
    B, T = len(counts), max(1, max(counts))
    cache, pages = pool([n + 1 for n in counts], d, page, seed)
    k, v = rand((B, T, d), seed, scale), rand((B, T, d), seed + 1)
    n = torch.tensor(counts, dtype=torch.int32, device="cuda")
    st = new_status()
    out, _ = kvz.kvz_append_int4(k, v, cache, pages, torch.zeros(B, dtype=torch.int32, device="cuda"), page, n_new=n,
                                 status=st)
    assert st.item() == 0 and torch.equal(out, n)
    return cache, pages, n, k, v


def wide(pages, page, rows=40000):
    """The page table with unused entries up to `rows` rows: attention then takes shares of equal work."""
    more = torch.full((pages.shape[0], max(0, rows // page - pages.shape[1])), -1, dtype=torch.int32, device="cuda")
    return torch.cat([pages, more], 1)


def offsets_of(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int64, device="cuda")


def expected_bytes(cache0, pages, page, d, rows):
    """cache0 with rows {(b, slot): (k bits, v bits)} written, by the oracle."""
    ref = cache0.copy()
    blocks = {}
    for (b, slot), kv in rows.items():
        blocks.setdefault((int(pages[b, slot // page]), slot % page // 16), []).append((slot % 16, *kv))
    for (pid, blk), put in blocks.items():
        view = ref[pid].reshape(page // 16, 18 * d)[blk]
        parts = [x.copy() for x in o4.unpack_block(view, d)]
        at = [r for r, _, _ in put]
        for o, i in ((0, 1), (3, 2)):
            c, s, m = o4.quantize_groups(np.stack([p[i] for p in put]))
            parts[o][at], parts[o + 1][at], parts[o + 2][at] = c, s, m
        view[:] = o4.pack_block(*parts)
    return ref


# ---------------------------------------------------------------------------
# Writing
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,n_c,ratio,mode", [(16, 40, 0.5, "per_head"), (48, 500, 0.33, "global"),
                                                 (64, 1000, 0.1, "global"), (1024, 3000, 0.9, "per_head"),
                                                 (32, 1, 1.0, "per_head")])
def test_compact_bytes(d, page, n_c, ratio, mode):
    B = 5
    K = rand((B, n_c, d), n_c) * torch.exp(torch.randn((B, n_c, 1), generator=gen(1), device="cuda")).bfloat16()
    V = rand((B, n_c, d), n_c + 1)
    K[0, 0], V[0, 0] = 0.0, 1.5                       # constant rows
    S = synth.synthetic_scores(B, n_c, seed=n_c, device="cuda")
    S[0, 0] = float("inf")
    if mode == "global":
        S[2] = 0.0                                    # a head that keeps nothing
    idx, counts, offsets = kvz.kvz_select(S, ratio, mode)
    cnt = counts.cpu().numpy()
    cache, pages = pool(cnt, d, page, n_c)
    before, st = cache.cpu().numpy(), new_status()
    assert kvz.kvz_compact_int4(K, V, idx, counts, offsets, cache, pages, page, status=st) is cache
    assert st.item() == 0
    ih, oh, Kb, Vb = idx.cpu().numpy(), offsets.cpu().numpy(), bits(K), bits(V)
    rows = {(b, p): (Kb[b, ih[oh[b] + p]], Vb[b, ih[oh[b] + p]]) for b in range(B) for p in range(cnt[b])}
    np.testing.assert_array_equal(cache.cpu().numpy(), expected_bytes(before, pages.cpu().numpy(), page, d, rows))


def test_compact_corner_values():
    # NaN, infinities, a range past float32, steps under the smallest normal number, exact ties, constant groups
    d, page = 64, 16
    x = torch.zeros((1, 16, d))
    x[0, 0, 3] = float("nan")
    x[0, 1, 5], x[0, 2, 5] = float("inf"), float("-inf")
    x[0, 3, 0], x[0, 3, 1] = 3e38, -3e38
    x[0, 4, 7], x[0, 5, 7] = 2.0 ** -130, 2.0 ** -121
    x[0, 6] = torch.arange(64) % 31 * 0.5             # step 1: halves are ties
    x[0, 7] = -2.0
    x[0, 8, :2] = torch.tensor([-0.0, 0.0])
    x[0, 9] = torch.linspace(-1e38, 1e38, 64)
    K = x.bfloat16().cuda()
    V = K.flip(1).contiguous()
    idx = torch.arange(16, dtype=torch.int32, device="cuda")
    counts, offsets = torch.tensor([16], dtype=torch.int32, device="cuda"), offsets_of([16])
    cache, pages = pool([16], d, page, 0)
    before = cache.cpu().numpy()
    kvz.kvz_compact_int4(K, V, idx, counts, offsets, cache, pages, page)
    Kb, Vb = bits(K)[0], bits(V)[0]
    ref = expected_bytes(before, pages.cpu().numpy(), page, d, {(0, p): (Kb[p], Vb[p]) for p in range(16)})
    got, want = (o4.unpack_block(c[int(pages[0, 0])], d) for c in (cache.cpu().numpy(), ref))
    for i in (0, 1, 3, 4):
        np.testing.assert_array_equal(got[i], want[i])
    # minima may differ in the sign of a zero: they stand for the same value
    for i in (2, 5):
        np.testing.assert_array_equal(orc.bf16_bits_to_f64(got[i]), orc.bf16_bits_to_f64(want[i]))


@pytest.mark.parametrize("d,rot,il", [(128, 128, False), (128, 64, True), (64, 48, False), (64, 64, True), (64, 0, False),
                                      (128, 96, False)])
@pytest.mark.parametrize("T", [1, 2, 3, 37])
def test_append_bytes(d, rot, il, T):
    counts = [0, 1, 15, 16, 17, 30, 47, 5]
    B, G, page = len(counts), 3, 16
    cache, pages = pool([c + T for c in counts], d, page, T)
    cache.copy_(torch.randint(0, 256, cache.shape, generator=gen(T), device="cuda", dtype=torch.uint8))
    before = cache.cpu().numpy()
    k = rand((T, B, d), T).permute(1, 0, 2)
    v = rand((T, B, 2 * d), T + 1)[..., d:].permute(1, 0, 2)
    q = rand((T, B, G, d), T + 2).permute(1, 2, 0, 3)
    n_new = torch.tensor([T, T, 0, T, max(T - 1, 0), T, T // 2, T], dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    pos = torch.randint(0, 900, (B, T), dtype=torch.int32, device="cuda")
    kw = dict(positions=pos, table=table(rot, 900), interleaved=il) if rot else {}
    q_out = torch.full((B, G, T, d), 9.0, dtype=torch.bfloat16, device="cuda")
    st = new_status()
    out, qo = kvz.kvz_append_int4(k, v, cache, pages, cnt, page, q=q, q_out=q_out, n_new=n_new, status=st, **kw)
    assert st.item() == 0 and qo is q_out
    assert torch.equal(out, cnt + n_new)
    kb, vb, qb = bits(k), bits(v), bits(q)
    if rot:
        t = kw["table"].cpu().numpy()
        kb = o4.rotary(kb, pos.cpu().numpy(), t, il)
        qb = o4.rotary(qb, pos.cpu().numpy()[:, None], t, il)
    nn = n_new.cpu().numpy()
    rows = {(b, counts[b] + i): (kb[b, i], vb[b, i]) for b in range(B) for i in range(nn[b])}
    np.testing.assert_array_equal(cache.cpu().numpy(), expected_bytes(before, pages.cpu().numpy(), page, d, rows))
    got = bits(q_out)
    for b in range(B):
        np.testing.assert_array_equal(got[b, :, :nn[b]], qb[b, :, :nn[b]])
        assert bool((q_out[b, :, nn[b]:] == 9).all())


def test_append_shared_positions_match_rotary():
    # positions [T] for all heads; the appended keys are kvz_rotary's rows
    B, T, d, page = 6, 130, 128, 32
    t = table(d, 700)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 500
    k, v = rand((B, T, d), 1), rand((B, T, d), 2)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    a, pages = pool([T] * B, d, page, 1)
    b = a.clone()
    kvz.kvz_append_int4(k, v, a, pages, zero, page, positions=pos, table=t)
    kvz.kvz_append_int4(kvz.kvz_rotary(k, pos, t), v, b, pages, zero, page)
    assert torch.equal(a, b)


def test_append_one_by_one_equals_at_once_and_compact():
    B, T, d, page = 3, 50, 64, 16
    k, v = rand((B, T, d), 3), rand((B, T, d), 4)
    one, pages = pool([T] * B, d, page, 2)
    many, whole = one.clone(), one.clone()
    cnt = torch.zeros(B, dtype=torch.int32, device="cuda")
    kvz.kvz_append_int4(k, v, many, pages, cnt, page)
    nxt = torch.empty_like(cnt)
    for i in range(T):
        kvz.kvz_append_int4(k[:, i:i + 1], v[:, i:i + 1], one, pages, cnt, page, counts_out=nxt)
        cnt, nxt = nxt, cnt
    assert cnt.tolist() == [T] * B
    idx = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B)
    kvz.kvz_compact_int4(k, v, idx, cnt, offsets_of([T] * B), whole, pages, page)
    assert torch.equal(one, many) and torch.equal(one, whole)


# ---------------------------------------------------------------------------
# Reading back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts,page", [([1], 16), ([0, 0, 3], 16), ([100, 0, 33, 16, 15, 1, 0], 48),
                                         ([700, 1, 2], 256)])
def test_expand(d, counts, page):
    cache, pages, n, k, v = filled(counts, d, page, 7)
    gap = [c + 2 for c in counts]                     # two spare rows behind every head
    off = offsets_of(gap)
    K = torch.full((sum(gap), d), 3.0, dtype=torch.bfloat16, device="cuda")
    V = K.clone()
    st = new_status()
    kvz.kvz_expand_int4(cache, pages, n, off, page, K_out=K, V_out=V, status=st)
    assert st.item() == 0
    kb, vb = bits(k), bits(v)
    for b, c in enumerate(counts):
        o = int(off[b])
        for src, out in ((kb, K), (vb, V)):
            if c:
                ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(src[b, :c])))
                np.testing.assert_array_equal(bits(out[o:o + c]), ref)
            assert bool((out[o + c:o + c + 2] == 3).all())


def test_expand_part():
    counts = [40, 5, 17, 64, 9]
    cache, pages, n, _, _ = filled(counts, 128, 32, 8)
    full = kvz.kvz_expand_int4(cache, pages, n, offsets_of(counts), 32, out_rows=sum(counts))
    first = torch.tensor([3, 5, 16, 0, 8], dtype=torch.int32, device="cuda")
    part = [c - f for c, f in zip(counts, first.tolist())]
    got = kvz.kvz_expand_int4(cache, pages, n, offsets_of(part), 32, first=first, out_rows=sum(part))
    at, o = 0, 0
    for c, f, m in zip(counts, first.tolist(), part):
        for x, y in zip(full, got):
            assert torch.equal(x[at + f:at + c], y[o:o + m])
        at, o = at + c, o + m
    none = kvz.kvz_expand_int4(cache, pages, torch.zeros_like(n), offsets_of([0] * 5), 32, out_rows=0)
    assert none[0].shape == (0, 128)


@pytest.mark.parametrize("d", [64, 128])
def test_expand_of_many_rows(d):
    # so many blocks that a warp takes K and V of several, in heads of very different lengths
    counts = [17, 0, 30011, 1, 9000, 64]
    cache, pages, n, k, v = filled(counts, d, 48, 9)
    st = new_status()
    got = kvz.kvz_expand_int4(cache, pages, n, offsets_of(counts), 48, out_rows=sum(counts), status=st)
    assert st.item() == 0
    for src, out in ((k, got[0]), (v, got[1])):
        rows = torch.cat([src[b, :c] for b, c in enumerate(counts)])
        ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(bits(rows))))
        np.testing.assert_array_equal(bits(out), ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("start", [5, 16, 256, 1000])
@pytest.mark.parametrize("counts,page", [([100, 0, 37], 16), ([0, 100, 17, 1], 64), ([5000, 3, 40000], 48)])
def test_offsets_that_start_behind_other_rows(counts, page, start, d):
    # one layer's heads in the outputs of a stack: compaction takes its run of idx, expansion leaves the rows in front
    cache, pages, n, k, v = filled(counts, d, page, start)
    off = offsets_of(counts) + start
    rows = start + sum(counts) + 3
    K = torch.full((rows, d), 3.0, dtype=torch.bfloat16, device="cuda")
    V, st = K.clone(), new_status()
    kvz.kvz_expand_int4(cache, pages, n, off, page, K_out=K, V_out=V, status=st)
    assert st.item() == 0
    want = kvz.kvz_expand_int4(cache, pages, n, offsets_of(counts), page, out_rows=sum(counts))
    for out, ref in ((K, want[0]), (V, want[1])):
        assert torch.equal(out[start:-3], ref)
        assert bool((out[:start] == 3).all()) and bool((out[-3:] == 3).all())
    first = n // 2
    part = n - first
    off_part = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), part.long().cumsum(0)]) + start
    got = kvz.kvz_expand_int4(cache, pages, n, off_part, page, first=first, out_rows=rows, status=st)
    at, o = 0, start
    for c, m in zip(counts, part.tolist()):
        for x, y in zip(want, got):
            assert torch.equal(x[at + c - m:at + c], y[o:o + m])
        at, o = at + c, o + m
    other = torch.full_like(cache, 255)
    idx = torch.full((rows,), -7, dtype=torch.int32, device="cuda")         # what lies in front is another head's
    idx[start:start + sum(counts)] = torch.cat([torch.arange(c, dtype=torch.int32, device="cuda") for c in counts])
    kvz.kvz_compact_int4(k, v, idx, n, off, other, pages, page, status=st)
    assert st.item() == 0 and torch.equal(other, cache)


@pytest.mark.parametrize("d", [64, 128])
def test_offsets_with_much_room(d):
    # the last head's room ends at 2^50: what no row fills is passed over, not walked through
    counts, page = [100, 0, 37, 500], 32
    cache, pages, n, k, v = filled(counts, d, page, 4)
    off, st = offsets_of(counts), new_status()
    off[-1] = 1 << 50
    got = kvz.kvz_expand_int4(cache, pages, n, off, page, out_rows=sum(counts), status=st)
    for x, y in zip(got, kvz.kvz_expand_int4(cache, pages, n, offsets_of(counts), page, out_rows=sum(counts))):
        assert torch.equal(x, y)
    other = torch.full_like(cache, 255)
    idx = torch.cat([torch.arange(c, dtype=torch.int32, device="cuda") for c in counts])
    kvz.kvz_compact_int4(k, v, idx, n, off, other, pages, page, status=st)
    assert st.item() == 0 and torch.equal(other, cache)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def check_decode(q, cache, pages, counts, page, scale, **kw):
    st = new_status()
    out, lse2 = kvz.kvz_decode_int4(q, cache, pages, counts, page, scale=scale, status=st, **kw)
    assert st.item() == 0
    ch, ph, cn, qd = cache.cpu().numpy(), pages.cpu().numpy(), counts.cpu().numpy(), f64(q)
    o, ls = out.cpu().double().numpy(), lse2.cpu().double().numpy()
    for b in range(len(cn)):
        if cn[b] == 0:
            assert np.all(o[b] == 0) and np.all(np.isneginf(ls[b]))
            continue
        K, V = o4.read_head(ch, ph[b], page, q.shape[2], int(cn[b]))
        ro, rl = orc.decode_attention(qd[b:b + 1], K.astype(np.float64), V.astype(np.float64), np.array([cn[b]]),
                                      np.array([0, cn[b]]), scale)
        tol, ltol = o4.decode_bound(qd[b], K, V, scale)
        assert np.all(np.abs(o[b] - ro[0]) <= tol[:, None]), (b, np.abs(o[b] - ro[0]).max(), tol)
        assert np.all(np.abs(ls[b] - rl[0]) <= ltol)
    return out, lse2


@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("counts,page,d", [
    ([1], 16, 128),                                   # one row
    ([15, 16, 17, 0, 31, 33, 1, 128], 16, 64),        # a block's edges, an empty head
    ([300, 2457, 64, 5], 48, 128),                    # pages of three blocks
    ([2457] * 8, 64, 128),                            # the pruned 8K layer
    ([20000, 3, 0, 777], 1024, 64),
])
def test_decode(G, counts, page, d):
    cache, pages, n, _, _ = filled(counts, d, page, len(counts) + G)
    q, B = rand((len(counts), G, d), G), len(counts)
    out, lse2 = check_decode(q, cache, pages, n, page, d ** -0.5)
    more = wide(pages, page)
    assert kvz.kvz_decode_int4_workspace_size(B, G, more.shape[1] * page, d) > 0
    out2, lse22 = check_decode(q, cache, more, n, page, d ** -0.5)
    assert torch.equal(torch.isneginf(lse2), torch.isneginf(lse22))


@pytest.mark.parametrize("d,G", [(128, 4), (64, 7), (128, 8), (64, 1)])
@pytest.mark.parametrize("B", [1, 7, 12, 13, 24, 25, 33, 64, 65, 129])
def test_decode_by_clusters_of_every_size(B, d, G):
    counts = [0 if b % 5 == 3 else (b * 97 + 350) % 701 for b in range(B)]
    cache, pages, n, _, _ = filled(counts, d, 32, B)
    assert kvz.kvz_decode_int4_workspace_size(B, G, pages.shape[1] * 32, d) == 0
    check_decode(rand((B, G, d), B), cache, pages, n, 32, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("widest", [1, 2, 4, 8, 16])
def test_decode_by_narrower_clusters_than_chosen(widest, d):
    # a part of a GPU that has no room for clusters of 16: the heads that would have them, up to their longest, by fewer
    # CTAs, whose warps then look up their pages several times
    counts, page, G = [20480, 1, 0, 12345, 700], 32, 4
    cache, pages, n, _, _ = filled([c - 1 if c == 20480 else c for c in counts], d, page, 12)
    assert kvz.kvz_decode_int4_workspace_size(5, G, pages.shape[1] * page, d) == 0
    q, st = rand((5, G, d), 13), new_status()
    ref, rl = check_decode(q, cache, pages, n, page, d ** -0.5)
    out, lse2 = kvz.kvz_testing_decode_int4_withhold(q, cache, pages, n, page, 1_000_000_000, -1, max_cluster=widest,
                                                     status=st)
    assert st.item() == 0
    if widest == 16:
        assert torch.equal(out, ref) and torch.equal(lse2, rl)
    ch, ph, cn, qd = cache.cpu().numpy(), pages.cpu().numpy(), n.cpu().numpy(), f64(q)
    for b in range(5):
        if cn[b] == 0:
            assert bool((out[b] == 0).all()) and bool(torch.isneginf(lse2[b]).all())
            continue
        K, V = o4.read_head(ch, ph[b], page, d, int(cn[b]))
        want, tol = o4.decode_bound_by_group(qd[b], K, V, d ** -0.5)
        assert np.all(np.abs(out[b].cpu().double().numpy() - want) <= tol)


def test_decode_one_long_head():
    cache, pages, n, _, _ = filled([100003], 128, 128, 11)    # every CTA reads a part of it
    check_decode(rand((1, 5, 128), 1), cache, pages, n, 128, 0.088)


def test_decode_many_heads():
    # more heads than counts kept on chip and than CTAs, many empty: every CTA's share spans several
    counts = [(n * 7) % 40 if n % 3 else 0 for n in range(1500)]
    cache, pages, n, _, _ = filled(counts, 64, 16, 12)
    check_decode(rand((1500, 2, 64), 2), cache, pages, n, 16, 0.125)


def test_decode_many_heads_in_shares():
    # a table wide enough for shares of equal work: more heads than counts kept on chip, many empty, every CTA's share
    # spans several
    counts = [(n * 7) % 40 if n % 3 else 0 for n in range(1500)]
    cache, pages, n, _, _ = filled(counts, 64, 16, 12)
    pages = wide(pages, 16)
    assert kvz.kvz_decode_int4_workspace_size(1500, 2, pages.shape[1] * 16, 64) > 0
    check_decode(rand((1500, 2, 64), 2), cache, pages, n, 16, 0.125)


def test_decode_many_heads_and_a_long_one():
    # the same with a head long enough for shares of equal work: most CTAs begin, hold and end several heads
    counts = [(n * 7) % 40 if n % 3 else 0 for n in range(1500)]
    counts[700] = 9000
    cache, pages, n, _, _ = filled(counts, 64, 16, 12)
    assert kvz.kvz_decode_int4_workspace_size(1500, 2, pages.shape[1] * 16, 64) > 0
    check_decode(rand((1500, 2, 64), 2), cache, pages, n, 16, 0.125)


def test_the_most_heads():
    # 65,535 heads of 0 to 16 rows: every call numbers them, and both forms of attention read them
    B, d, page = 65535, 64, 16
    n = (torch.arange(B, device="cuda", dtype=torch.int32) * 5) % 17
    cache = torch.full((B, page * 72), 255, dtype=torch.uint8, device="cuda")
    pages = torch.randperm(B, generator=torch.Generator().manual_seed(1))[:, None].int().cuda()
    k, v, q = rand((B, 16, d), 91), rand((B, 16, d), 92), rand((B, 1, d), 93)
    st = new_status()
    got, _ = kvz.kvz_append_int4(k, v, cache, pages, torch.zeros_like(n), page, n_new=n, status=st)
    assert torch.equal(got, n)
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.long().cumsum(0)])
    rows = int(off[-1])
    K, V = kvz.kvz_expand_int4(cache, pages, n, off, page, out_rows=rows, status=st)
    live = torch.arange(16, device="cuda")[None] < n[:, None]
    for src, out in ((k[live], K), (v[live], V)):
        pick = torch.cat([torch.arange(500), torch.arange(rows - 500, rows)]).cuda()
        ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(bits(src[pick]))))
        np.testing.assert_array_equal(bits(out[pick]), ref)
    again = torch.full_like(cache, 255)
    idx = torch.arange(16, device="cuda", dtype=torch.int32)[None].expand(B, 16)[live]
    kvz.kvz_compact_int4(k, v, idx, n, off, again, pages, page, status=st)
    assert torch.equal(again, cache)
    a = kvz.kvz_decode_int4(q, cache, pages, n, page, status=st)
    b = kvz.kvz_decode_int4(q, cache, wide(pages, page, 2080), n, page, status=st)
    assert kvz.kvz_decode_int4_workspace_size(B, 1, 2080, d) > 0 and st.item() == 0
    for x, y in zip(a, b):
        assert torch.allclose(x, y, atol=1e-5)
    pick = torch.tensor([0, 1, 2, 3, 30000, B - 2, B - 1], device="cuda")
    ref, _ = check_decode(q[pick], cache, pages[pick], n[pick], page, d ** -0.5)
    assert torch.allclose(a[0][pick], ref, atol=1e-5)


def test_decode_all_empty():
    cache, pages, n, _, _ = filled([0, 0, 0], 128, 16, 13)
    check_decode(rand((3, 4, 128), 3), cache, pages, n, 16, 0.1)


@pytest.mark.parametrize("scale", [1e-6, 0.088, 3.0])
def test_decode_peaked_and_flat(scale):
    # logits of hundreds in both orders: the running reference moves often, or never again
    d, page, N = 128, 32, 600
    k = rand((2, N, d), 14)
    ramp = torch.linspace(0, 3, N, device="cuda").bfloat16()
    k[0] = k[0] * ramp[:, None]
    k[1] = k[1] * ramp.flip(0)[:, None]
    v = rand((2, N, d), 15)
    cache, pages = pool([N, N], d, page, 3)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    n, _ = kvz.kvz_append_int4(k, v, cache, pages, zero, page)
    check_decode(rand((2, 8, d), 16), cache, pages, n, page, scale)


@pytest.mark.parametrize("n", [1, 40, 3000])
def test_decode_of_the_largest_values(n):
    # V near the end of float32: what is finite in the cache and on average stays finite on the way
    d, page, B = 128, 32, 3
    k, v = rand((B, n, d), 81), (torch.rand((B, n, d), generator=gen(82), device="cuda") * 2 - 1) * 1.62e38
    v[..., ::64], v[..., 1::64] = 1.62e38, -1.62e38   # steps of 2^124 and more in every group
    v[1] = 3.3e38                                     # constant rows: the mean is the largest number there is
    k[0] = k[0] * torch.linspace(0, 3, n, device="cuda").bfloat16()[:, None]   # logits that climb past the reference
    cache, pages = pool([n] * B, d, page, 5)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    cnt, _ = kvz.kvz_append_int4(k, v.bfloat16(), cache, pages, zero, page)
    for p in (pages, wide(pages, page)):
        for scale in (1e-6, 0.088, 1.0):
            out, _ = check_decode(rand((B, 4, d), 83), cache, p, cnt, page, scale)
            assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("size", [1.0, 2.0 ** 20, 2.0 ** 100])
@pytest.mark.parametrize("d,n,at", [(64, 1, 0), (128, 40, 5), (128, 40, 39), (64, 3000, 2900)])
def test_decode_of_zeros_beside_values_of_no_weight(n, d, at, size):
    # V is 0 but for one row, whose logit is so far below that its weight is 0 in any precision: the output is 0
    page, G = 32, 4
    q = (4.0 + rand((1, G, d), 88).clamp(-1, 1)).bfloat16()
    k, v = rand((1, n, d), 89), torch.zeros((1, n, d), dtype=torch.bfloat16, device="cuda")
    if n > 1:
        k[:, at], v[:, at] = -200.0, rand((d,), 90) * size
    cache, pages = pool([n], d, page, 5)
    cnt, _ = kvz.kvz_append_int4(k, v, cache, pages, torch.zeros(1, dtype=torch.int32, device="cuda"), page)
    for p in (pages, wide(pages, page)):
        out, _ = kvz.kvz_decode_int4(q, cache, p, cnt, page)
        assert bool((out == 0).all())


SPREADS = {
    # what row j and group g of V are multiplied by
    "second group 2^-10": lambda n, NG: torch.tensor([1.0, 2.0 ** -10])[:NG].expand(n, NG),
    "second group 2^-14": lambda n, NG: torch.tensor([1.0, 2.0 ** -14])[:NG].expand(n, NG),
    "second group 2^-40": lambda n, NG: torch.tensor([2.0 ** 20, 2.0 ** -20])[:NG].expand(n, NG),
    "last rows 2^-12": lambda n, NG: torch.where(torch.arange(n)[:, None] < n // 4, 1.0, 2.0 ** -12).expand(n, NG),
    "one row 2^20": lambda n, NG: torch.where(torch.arange(n)[:, None] == 5 % n, 2.0 ** 20, 1.0).expand(n, NG),
    "one row 2^30": lambda n, NG: torch.where(torch.arange(n)[:, None] == 5 % n, 2.0 ** 30, 1.0).expand(n, NG),
    "one row 2^90": lambda n, NG: torch.where(torch.arange(n)[:, None] == 5 % n, 2.0 ** 90, 1.0).expand(n, NG),
    "rows and groups 2^-60 to 2^60": lambda n, NG: 2.0 ** torch.randint(
        -60, 61, (n, NG), generator=torch.Generator().manual_seed(n)).double(),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", SPREADS)
@pytest.mark.parametrize("n", [40, 2500])
def test_decode_of_values_of_very_different_size(n, name, d):
    # every group's output is held to its own size, whatever the other group's steps and those of rows that hardly
    # count: with "one row", that row's logit is far below the others'
    page, G = 32, 4
    mul = SPREADS[name](n, d // 64).double().repeat_interleave(64, 1).cuda()
    v = (torch.randn((1, n, d), generator=gen(84), device="cuda").double() * mul).bfloat16()
    base = rand((1, 1, d), 85)
    q = (base + 0.1 * rand((1, G, d), 86)).bfloat16()
    k = rand((1, n, d), 87)
    if name.startswith("one row"):
        k[:, 5 % n] = -8.0 * base[:, 0]               # at d = 64 a logit of about -60 against +-8
    cache, pages = pool([n], d, page, 5)
    cnt, _ = kvz.kvz_append_int4(k, v, cache, pages, torch.zeros(1, dtype=torch.int32, device="cuda"), page)
    K, V = o4.read_head(cache.cpu().numpy(), pages[0].cpu().numpy(), page, d, n)
    want, tol = o4.decode_bound_by_group(f64(q)[0], K, V, d ** -0.5)
    for p in (pages, wide(pages, page)):
        got = kvz.kvz_decode_int4(q, cache, p, cnt, page)[0][0].cpu().double().numpy()
        off = np.abs(got - want) / tol
        assert np.all(off <= 1), (off.max(), np.abs(got - want).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("v_exp,q_exp", [(-95, 0), (-60, 0), (100, 0), (0, -24), (0, 40), (0, -90)])
def test_decode_of_small_and_large_values_and_queries(v_exp, q_exp, d):
    # all of V at one size; queries at another with keys at the inverse, so that the logits stay as they are, and half
    # of the dims (a group, or every other 16) 2^-20 of the rest with keys 2^20 times as large
    n, page, G = 700, 32, 3
    half = (torch.arange(d, device="cuda") // (64 if d == 128 else 16)) % 2 == 1
    skew = torch.where(half, 2.0 ** -20, 1.0).double()
    q = (rand((1, G, d), 91).double() * skew * 2.0 ** q_exp).bfloat16()
    k = (rand((1, n, d), 92).double() / skew * 2.0 ** -q_exp).bfloat16()
    v = (rand((1, n, d), 93).double() * 2.0 ** v_exp).bfloat16()
    cache, pages = pool([n], d, page, 5)
    cnt, _ = kvz.kvz_append_int4(k, v, cache, pages, torch.zeros(1, dtype=torch.int32, device="cuda"), page)
    K, V = o4.read_head(cache.cpu().numpy(), pages[0].cpu().numpy(), page, d, n)
    want, tol = o4.decode_bound_by_group(f64(q)[0], K, V, d ** -0.5)
    for p in (pages, wide(pages, page)):
        got = kvz.kvz_decode_int4(q, cache, p, cnt, page)[0][0].cpu().double().numpy()
        assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()


def test_decode_ignores_rows_past_the_end():
    # NaN scales behind the last row, in its block and on unused pages
    counts, d, page = [1, 18, 47], 128, 16
    cache, pages, n, k, v = filled(counts, d, page, 17)
    bad = torch.full((3, 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    room = [int((pages[b] >= 0).sum()) * page - c for b, c in enumerate(counts)]
    n_bad = torch.tensor([min(3, r) for r in room], dtype=torch.int32, device="cuda")
    kvz.kvz_append_int4(bad, bad, cache, pages, n, page, n_new=n_bad)
    out, _ = check_decode(rand((3, 4, d), 18), cache, pages, n, page, 0.1)
    assert bool(torch.isfinite(out).all())
    # a NaN row that does count reaches its head's output and no other's
    n2 = n.clone()
    n2[1] += 1
    out2, _ = kvz.kvz_decode_int4(rand((3, 4, d), 18), cache, pages, n2, page, scale=0.1)
    assert bool(torch.isnan(out2[1]).all()) and torch.equal(out2[0], out[0]) and torch.equal(out2[2], out[2])


def test_decode_matches_decode_over_expanded_rows():
    counts, d, page = [500, 33, 2000, 0], 128, 64
    cache, pages, n, _, _ = filled(counts, d, page, 19)
    q = rand((4, 4, d), 20)
    out, lse2 = kvz.kvz_decode_int4(q, cache, pages, n, page)
    K, V = kvz.kvz_expand_int4(cache, pages, n, offsets_of(counts), page, out_rows=sum(counts))
    o2, l2 = kvz.kvz_decode(q, K, V, n, offsets_of(counts), 2000)
    # the expanded rows carry a bf16 rounding, 2^-8 of a value: a logit moves by 2^-8 sum |q k| scale at most
    dl = 2.0 ** -8 * (q.float().abs().sum(-1).max().item() * K.float().abs().max().item()) * d ** -0.5
    tol = (2 * dl + 2.0 ** -8) * V.float().abs().max().item() + 1e-4
    assert (out - o2).abs().max().item() <= tol
    assert torch.equal(torch.isneginf(lse2), torch.isneginf(l2))


def test_decode_shared_pages():
    # two heads that name the same pages read the same rows
    cache, pages, n, _, _ = filled([200, 200], 64, 16, 21)
    pages[1] = pages[0]
    q = rand((1, 4, 64), 22).expand(2, 4, 64).contiguous()
    out, lse2 = check_decode(q, cache, pages, n, 16, 0.125)
    assert torch.allclose(out[0], out[1], atol=1e-5)


def test_decode_is_deterministic_and_leaves_inputs():
    cache, pages, n, _, _ = filled([5000, 40, 9000, 123], 128, 64, 23)
    pages = wide(pages, 64)
    q, c0 = rand((4, 8, 128), 24), cache.clone()
    need = kvz.kvz_decode_int4_workspace_size(4, 8, pages.shape[1] * 64, 128)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    a = kvz.kvz_decode_int4(q, cache, pages, n, 64, workspace=ws)
    for _ in range(3):
        b = kvz.kvz_decode_int4(q, cache, pages, n, 64, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(cache, c0)


def test_offsets_past_32_bits():
    # pages that lie 2^32 bytes and more into the pool
    d, page = 128, 64
    cache = torch.empty((600000, page * 144), dtype=torch.uint8, device="cuda")
    pages = torch.tensor([[599999, 470000], [3, 466034]], dtype=torch.int32, device="cuda")
    k, v = rand((2, 100, d), 25), rand((2, 100, d), 26)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    n, _ = kvz.kvz_append_int4(k, v, cache, pages, zero, page)
    K, V = kvz.kvz_expand_int4(cache, pages, n, offsets_of([100, 100]), page, out_rows=200)
    for src, got in ((k, K), (v, V)):
        ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(bits(src).reshape(200, d))))
        np.testing.assert_array_equal(bits(got), ref)
    small = cache[pages.flatten().long()].clone()
    q = rand((2, 4, d), 27)
    a = kvz.kvz_decode_int4(q, cache, pages, n, page)
    b = kvz.kvz_decode_int4(q, small, torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda"), n, page)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# Device-detected errors
# ---------------------------------------------------------------------------
def test_bad_counts_are_left_out():
    counts, d, page = [100, 50, 60], 128, 16
    cache, pages, n, _, _ = filled(counts, d, page, 28)
    q = rand((3, 2, d), 29)
    good = kvz.kvz_decode_int4(q, cache, pages, n, page)
    for bad in (-1, pages.shape[1] * page + 1):
        m = n.clone()
        m[1] = bad
        st = new_status()
        out = torch.full((3, 2, d), 5.0, device="cuda")
        kvz.kvz_decode_int4(q, cache, pages, m, page, out=out, status=st)
        assert st.item() == 1 and bool((out[1] == 5).all())
        assert torch.allclose(out[0], good[0][0], atol=1e-5) and torch.allclose(out[2], good[0][2], atol=1e-5)
        K = torch.full((210, d), 5.0, dtype=torch.bfloat16, device="cuda")
        st = new_status()
        kvz.kvz_expand_int4(cache, pages, m, offsets_of(counts), page, K_out=K, V_out=K.clone(), status=st)
        assert st.item() == 1 and bool((K[100:150] == 5).all()) and not bool((K[:100] == 5).all())
        st, c0 = new_status(), cache.clone()
        k = rand((3, 1, d), 30)
        out_n, _ = kvz.kvz_append_int4(k, k, cache, pages, m, page, status=st)
        assert st.item() == 1 and out_n[1].item() == bad
        p1 = pages[1][pages[1] >= 0].long()
        assert torch.equal(cache[p1], c0[p1])
        cache.copy_(c0)


def test_bad_pages_are_reported():
    counts, d, page = [40, 40], 64, 16
    cache, pages, n, _, _ = filled(counts, d, page, 31)
    k = rand((2, 1, d), 32)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        p = pages.clone()
        p[1, 2] = bad
        st, c0 = new_status(), cache.clone()
        out_n, _ = kvz.kvz_append_int4(k, k, cache, p, n, page, status=st)
        assert st.item() == 1 and out_n.tolist() == [41, 40]
        p0 = pages[0][pages[0] >= 0].long()
        c0[p0] = cache[p0]
        assert torch.equal(cache, c0)
        st = new_status()
        out, _ = kvz.kvz_decode_int4(rand((2, 2, d), 33), cache, p, n, page, status=st)
        assert st.item() == 1 and bool(torch.isfinite(out[0]).all())
        st = new_status()
        K = torch.full((80, d), 5.0, dtype=torch.bfloat16, device="cuda")
        kvz.kvz_expand_int4(cache, p, n, offsets_of(counts), page, K_out=K, V_out=K.clone(), status=st)
        assert st.item() == 1 and bool((K[72:] == 5).all()) and not bool((K[40:72] == 5).any())


def test_bad_counts_and_pages_in_shares_of_equal_work():
    # heads that several CTAs read, with one left out before them, and a bad page in the middle of one
    counts, d, page = [9000, 50, 12000, 0, 700], 64, 32
    cache, pages, n, _, _ = filled(counts, d, page, 34)
    pages = wide(pages, page)
    q = rand((5, 3, d), 35)
    good = kvz.kvz_decode_int4(q, cache, pages, n, page)
    for bad in (-1, pages.shape[1] * page + 1, -2 ** 31):
        m, st = n.clone(), new_status()
        m[0] = bad
        out = torch.full((5, 3, d), 5.0, device="cuda")
        kvz.kvz_decode_int4(q, cache, pages, m, page, out=out, status=st)
        assert st.item() == 1 and bool((out[0] == 5).all())
        assert torch.allclose(out[1:], good[0][1:], atol=1e-5)
    for bad in (-1, cache.shape[0], -2 ** 31):
        p, st = pages.clone(), new_status()
        p[2, 200] = bad
        out, _ = kvz.kvz_decode_int4(q, cache, p, n, page, status=st)
        assert st.item() == 1
        keep = torch.tensor([0, 1, 3, 4], device="cuda")
        assert torch.equal(out[keep], good[0][keep])


def test_tensors_on_the_host_are_refused():
    counts, d, page = [40, 3], 64, 16
    cache, pages, n, k, v = filled(counts, d, page, 36)
    q, c0 = rand((2, 2, d), 37), cache.clone()
    pos = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    calls = {
        kvz.kvz_decode_int4: dict(q=q, cache=cache, pages=pages, counts=n, page_size=page, status=new_status()),
        kvz.kvz_append_int4: dict(k=k[:, :1], v=v[:, :1], cache=cache, pages=pages, counts=n, page_size=page,
                                  positions=pos, table=table(64, 8), n_new=torch.ones_like(n), status=new_status()),
        kvz.kvz_expand_int4: dict(cache=cache, pages=pages, counts=n, offsets=offsets_of(counts), page_size=page,
                                  out_rows=43, status=new_status()),
        kvz.kvz_compact_int4: dict(K=k, V=v, idx=torch.zeros(43, dtype=torch.int32, device="cuda"), counts=n,
                                   offsets=offsets_of(counts), cache=cache, pages=pages, page_size=page),
        kvz.kvz_rotary: dict(x=k[:, :1], positions=pos, table=table(64, 8), status=new_status()),
    }
    for f, kw in calls.items():
        for name, t in kw.items():
            if isinstance(t, torch.Tensor):
                with pytest.raises(ValueError):
                    f(**{**kw, name: t.cpu()})
    assert torch.equal(cache, c0)


def test_append_refusals_on_the_device():
    d, page = 64, 16
    cache, pages, n, _, _ = filled([30, 30, 30, 30], d, page, 34)
    cap = pages.shape[1] * page
    c0 = cache.clone()
    k = rand((4, 3, d), 35)
    t = table(64, 20)
    pos = torch.tensor([[1, 2, 3], [4, 25, 5], [0, 1, 2], [3, 3, 3]], dtype=torch.int32, device="cuda")
    n_new = torch.tensor([4, 2, -1, 1], dtype=torch.int32, device="cuda")
    st = new_status()
    out_n, _ = kvz.kvz_append_int4(k, k, cache, pages, n, page, positions=pos, table=t, n_new=n_new, status=st)
    assert st.item() == 1 and out_n.tolist() == [30, 30, 30, 31] and cap == 32
    for b in (0, 2):
        ids = pages[b].long()
        assert torch.equal(cache[ids], c0[ids])
    # a run that would pass the table's last page
    st, c1 = new_status(), cache.clone()
    out_n, _ = kvz.kvz_append_int4(k, k, cache, pages, n, page, status=st)
    assert st.item() == 1 and out_n.tolist() == [30] * 4 and torch.equal(cache, c1)


def test_append_refuses_outputs_over_what_it_reads(monkeypatch):
    cache, pages, n, k, v = filled([30, 30], 64, 16, 35)
    k, v, q = k[:, :2], v[:, :2], rand((2, 3, 2, 64), 36)
    pos, t, c0 = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), table(64, 8), cache.clone()
    new = torch.ones_like(n)
    for short in (kvz._fast, None):
        monkeypatch.setattr(kvz, "_fast", short)
        for kw in (dict(n_new=new, counts_out=new), dict(positions=pos, table=t, counts_out=pos.view(-1)),
                   dict(k=q[:, 0], q_out=q), dict(v=q[:, 0], q_out=q)):
            with pytest.raises(ValueError):
                kvz.kvz_append_int4(**{**dict(k=k, v=v, cache=cache, pages=pages, counts=n, page_size=16,
                                              q=rand((2, 3, 2, 64), 37)), **kw})
    assert torch.equal(cache, c0)


def test_compact_reports_bad_idx_and_counts():
    B, n_c, d, page = 2, 100, 64, 16
    K, V = rand((B, n_c, d), 36), rand((B, n_c, d), 37)
    idx = torch.arange(20, dtype=torch.int32, device="cuda").repeat(2)
    idx[3], idx[25] = n_c, -1
    counts = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    cache, pages = pool([20, 20], d, page, 4)
    st = new_status()
    kvz.kvz_compact_int4(K, V, idx, counts, offsets_of([20, 20]), cache, pages, page, status=st)
    assert st.item() == 1
    Kx, _ = kvz.kvz_expand_int4(cache, pages, counts, offsets_of([20, 20]), page, out_rows=40)
    assert bool((Kx[3] == 0).all()) and bool((Kx[25] == 0).all()) and not bool((Kx[4] == 0).all())
    st, c0 = new_status(), cache.clone()
    idx[3], idx[25] = 3, 5
    counts[1] = 21                                    # more than its run of idx
    kvz.kvz_compact_int4(V, K, idx, counts, offsets_of([20, 20]), cache, pages, page, status=st)
    assert st.item() == 1
    p1 = pages[1].long()
    assert torch.equal(cache[p1], c0[p1]) and not torch.equal(cache[pages[0].long()], c0[pages[0].long()])


def test_short_and_long_way_on_the_host_agree(monkeypatch):
    # the same calls with and without the host module: results, given outputs, refusals and their codes
    assert kvz._fast is not None, "csrc/fast_calls.cpp is not built"
    B, T, G, d, page = 3, 5, 2, 64, 16
    t = table(d, 300)
    pos = torch.randint(0, 300, (B, T), dtype=torch.int32, device="cuda")
    k, v, q = rand((B, T, d), 1), rand((T, B, d), 2).permute(1, 0, 2), rand((B, G, T, d), 3)
    one = torch.arange(T, dtype=torch.int32, device="cuda")
    n_new = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    K = rand((B, 40, d), 4)
    idx = torch.arange(10, dtype=torch.int32, device="cuda").repeat(B)

    def run():
        st = new_status()
        cache, pages = pool([20] * B, d, page, 9)
        ten = torch.full((B,), 10, dtype=torch.int32, device="cuda")
        res = [kvz.kvz_compact_int4(K, K, idx, ten, offsets_of([10] * B), cache, pages, page, status=st)]
        n_out, q_out = torch.zeros_like(ten), torch.zeros((B, G, T, d), dtype=torch.bfloat16, device="cuda")
        got = kvz.kvz_append_int4(k, v, cache, pages, ten, page, positions=pos, table=t, interleaved=True, q=q,
                                  q_out=q_out, n_new=n_new, counts_out=n_out, status=st)
        assert got[0] is n_out and got[1] is q_out
        res += [*got, *kvz.kvz_append_int4(k[:, :1], v[:, :1], cache, pages, n_out, page)[:1]]
        res += kvz.kvz_expand_int4(cache, pages, n_out, offsets_of(n_out.tolist()), page, first=None,
                                   out_rows=int(n_out.sum()), status=st)
        out = torch.empty((B, G, d), device="cuda")
        got = kvz.kvz_decode_int4(q_out[:, :, 0].contiguous(), cache, pages, n_out, page, out=out, status=st)
        assert got[0] is out
        res += [*got, *kvz.kvz_decode_int4(q_out[:, :, 0].contiguous(), cache, pages, n_out, page, scale=0.25)]
        res += [kvz.kvz_rotary(q, one, t, inverse=True), kvz.kvz_rotary(v, pos, t, interleaved=True, status=st)]
        assert st.item() == 0
        bad = []
        for call in (lambda: kvz.kvz_append_int4(k, v, cache, pages, ten, page, positions=one, table=t[:, :24]),
                     lambda: kvz.kvz_append_int4(k, v, cache, pages, ten, page, counts_out=ten),
                     lambda: kvz.kvz_append_int4(k, v, cache, pages, ten, page, q=q, q_out=q),
                     lambda: kvz.kvz_append_int4(k, v.cpu(), cache, pages, ten, page),
                     lambda: kvz.kvz_rotary(q, one, t[:, :40].contiguous()),
                     lambda: kvz.kvz_rotary(q, one[:4], t),
                     lambda: kvz.kvz_decode_int4(rand((B, 9, d), 1), cache, pages, ten, page),
                     lambda: kvz.kvz_decode_int4(rand((B, 2, d), 1), cache, pages, ten, page, scale=-1.0),
                     lambda: kvz.kvz_decode_int4(rand((B, 2, d), 1), cache, pages, ten, 24),
                     lambda: kvz.kvz_expand_int4(cache, pages, ten, offsets_of([10] * B), page),
                     lambda: kvz.kvz_compact_int4(K, K, idx, ten, offsets_of([10] * B), cache, pages[:2], page)):
            with pytest.raises((ValueError, kvz.KvzError)) as e:
                call()
            bad.append((type(e.value), getattr(e.value, "code", None)))
        return res, bad

    quick, bad = run()
    monkeypatch.setattr(kvz, "_fast", None)
    slow, bad2 = run()
    assert bad == bad2
    for a, b in zip(quick, slow):
        assert a.dtype == b.dtype and a.shape == b.shape
        assert torch.equal(a.view(torch.uint8) if a.is_contiguous() else a, b.view(torch.uint8) if b.is_contiguous() else b)


def _spaced(t):
    w = torch.zeros((*t.shape[:-1], t.shape[-1] + 8), dtype=t.dtype, device=t.device)
    w[..., : t.shape[-1]] = t
    return w[..., : t.shape[-1]]


def _shifted(t):
    w = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    w[1:] = t.reshape(-1)
    return w[1:].view(t.shape)


OTHER_TYPE = {torch.bfloat16: torch.float32, torch.float32: torch.bfloat16, torch.int32: torch.int64,
              torch.int64: torch.int32, torch.uint8: torch.int32}
OTHER_TENSORS = {
    "None": lambda t: None, "on the host": lambda t: t.cpu(), "type": lambda t: t.to(OTHER_TYPE[t.dtype]),
    "list": lambda t: t.tolist(), "number": lambda t: 3, "one less": lambda t: t[:-1].contiguous(),
    "narrower": lambda t: t[..., :-1].contiguous(), "twice": lambda t: torch.cat([t, t]), "one more dim": lambda t: t[None],
    "flat": lambda t: t.reshape(-1), "empty": lambda t: t[:0], "rows apart": _spaced, "odd address": _shifted,
    "transposed": lambda t: t.transpose(0, -1), "expanded": lambda t: t[:1].expand(t.shape),
    "no dim": lambda t: t.reshape(-1)[0], "parameter": lambda t: torch.nn.Parameter(t) if t.is_floating_point() else t,
}
OTHER_VALUES = {"page_size": [0, 8, 24, 32, 48, 2048, -16, 16.0, "16", True, 1 << 40],
                "scale": [None, 1, 0.0, -1.0, float("nan"), float("inf"), 1e-50, 1e50, True],
                "interleaved": [True, 1, 0, None, "x", 2], "inverse": [True, 1, 0, None, 2],
                "out_rows": [None, 0, -1, 39, 100, 40.0, True]}


@pytest.mark.parametrize("name", ["append", "decode", "expand", "compact", "rotary"])
def test_every_argument_changed_both_ways_on_the_host(name, monkeypatch):
    # each tensor and value of a call changed in the usual ways: with and without the host module it is accepted with
    # outputs of the same form, or refused by the same error
    short = kvz._fast
    assert short is not None, "csrc/fast_calls.cpp is not built"
    B, T, G, d, page = 3, 2, 2, 64, 16
    cache, pages, n, k, v = filled([20, 3, 17], d, page, 3)
    pages = torch.cat([pages, torch.full_like(pages[:, :1], -1)], 1)
    k, v, q, t = k[:, :T].contiguous(), v[:, :T].contiguous(), rand((B, G, T, d), 5), table(d, 90)
    pos = torch.randint(0, 90, (B, T), dtype=torch.int32, device="cuda")
    K, idx, off = rand((B, 40, d), 6), torch.arange(40, dtype=torch.int32, device="cuda"), offsets_of([20, 3, 17])
    at = dict(cache=cache, pages=pages, counts=n, page_size=page)
    f, base = {
        "append": (kvz.kvz_append_int4, dict(k=k, v=v, positions=pos, table=t, interleaved=False, q=q, n_new=n // n,
                                             q_out=torch.zeros_like(q), counts_out=torch.zeros_like(n), **at)),
        "decode": (kvz.kvz_decode_int4, dict(q=q[:, :, 0].contiguous(), scale=0.125, out=torch.zeros((B, G, d), device="cuda"),
                                             lse2=torch.zeros((B, G), device="cuda"),
                                             workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"), **at)),
        "expand": (kvz.kvz_expand_int4, dict(offsets=off, first=n - n, out_rows=40, **at)),
        "compact": (kvz.kvz_compact_int4, dict(K=K, V=K, idx=idx, offsets=off, **at)),
        "rotary": (kvz.kvz_rotary, dict(x=q, positions=pos, table=t, interleaved=False, inverse=False)),
    }[name]
    base["status"] = new_status()
    c0 = cache.clone()

    def outcome(kw):
        try:
            r = f(**kw)
        except (ValueError, kvz.KvzError) as e:
            return type(e), getattr(e, "code", None)
        finally:
            cache.copy_(c0)
        return [x if x is None else (x.dtype, x.shape, x.stride()) for x in (r if isinstance(r, tuple) else (r,))]

    assert isinstance(outcome(base), list)
    for arg, val in base.items():
        others = OTHER_VALUES[arg] if arg in OTHER_VALUES else [
            change(val) for kind, change in OTHER_TENSORS.items()]
        for i, x in enumerate(others):
            kw = {**base, arg: x}
            monkeypatch.setattr(kvz, "_fast", short)
            a = outcome(kw)
            monkeypatch.setattr(kvz, "_fast", None)
            assert a == outcome(kw), (arg, i)


@pytest.mark.parametrize("short", [True, False])
def test_new_outputs_are_filled_where_torch_fills_them(short, monkeypatch):
    # torch.empty fills with NaN under deterministic algorithms; rows that no call writes show it
    if not short:
        monkeypatch.setattr(kvz, "_fast", None)
    cache, pages, n, k, v = filled([3, 3], 64, 16, 7)
    q = rand((2, 2, 3, 64), 8)
    torch.use_deterministic_algorithms(True)
    try:
        got, q_out = kvz.kvz_append_int4(k, v, cache, pages, torch.zeros_like(n), 16, q=q,
                                         n_new=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
        K, V = kvz.kvz_expand_int4(cache, pages, got, offsets_of([1, 2]), 16, out_rows=5)
    finally:
        torch.use_deterministic_algorithms(False)
    assert torch.equal(q_out[0, :, 0], q[0, :, 0]) and torch.equal(q_out[1, :, :2], q[1, :, :2])
    assert bool(torch.isnan(q_out[0, :, 1:]).all()) and bool(torch.isnan(q_out[1, :, 2:]).all())
    assert bool(torch.isnan(K[3:]).all()) and bool(torch.isnan(V[3:]).all()) and bool(torch.isfinite(K[:3]).all())


# ---------------------------------------------------------------------------
# Streams, graphs, and the whole path
# ---------------------------------------------------------------------------
def test_streams():
    cache, pages, n, _, _ = filled([900, 4000], 128, 64, 38)
    q = rand((2, 4, 128), 39)
    ref = kvz.kvz_decode_int4(q, cache, pages, n, 64)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):                                # two streams at once, scratch allocated by each call
        s = sides[i % 2]
        s.wait_stream(torch.cuda.current_stream())
        outs.append(kvz.kvz_decode_int4(q, cache, pages, n, 64, stream=s if i < 4 else s.cuda_stream))
    for s in sides:
        s.synchronize()
    for o, l2 in outs:
        assert torch.equal(o, ref[0]) and torch.equal(l2, ref[1])


def test_streams_with_scratch():
    # the same with shares of equal work, whose scratch every call allocates: each stream asks other questions of
    # another cache, so scratch that two calls shared would show
    page, d, G = 64, 128, 4
    sides = [torch.cuda.Stream() for _ in range(3)]
    sets = []
    for i in range(len(sides)):
        cache, pages, n, _, _ = filled([9000, 40 + i, 15000 - 999 * i], d, page, 38 + i)
        pages = wide(pages, page)
        assert kvz.kvz_decode_int4_workspace_size(3, G, pages.shape[1] * page, d) > 0
        q = [rand((3, G, d), 500 + 10 * i + j) for j in range(8)]
        sets.append((cache, pages, n, q, [kvz.kvz_decode_int4(x, cache, pages, n, page) for x in q]))
    torch.cuda.synchronize()
    outs = [[] for _ in sides]
    for j in range(8):
        for i, s in enumerate(sides):
            cache, pages, n, q, _ = sets[i]
            if j % 2:
                outs[i].append(kvz.kvz_decode_int4(q[j], cache, pages, n, page, stream=s))
            else:
                with torch.cuda.stream(s):
                    outs[i].append(kvz.kvz_decode_int4(q[j], cache, pages, n, page))
    for s in sides:
        s.synchronize()
    for i in range(len(sides)):
        for got, ref in zip(outs[i], sets[i][4]):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_decoding_in_graphs_that_share_a_workspace():
    # one graph appends, another attends, a third attends over another cache with the same workspace; replayed in turn
    d, page, B, G = 128, 16, 3, 4
    counts = [100, 7, 9250]
    cache, pages = pool([c + 8 for c in counts], d, page, 5)
    k0, v0 = rand((B, 9250, d), 40), rand((B, 9250, d), 41)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    n0 = torch.tensor(counts, dtype=torch.int32, device="cuda")
    kvz.kvz_append_int4(k0, v0, cache, pages, zero, page, n_new=n0)
    other = filled([33, 12000, 1], d, page, 42)
    pages, other = wide(pages, page), (other[0], wide(other[1], page), other[2])
    need = kvz.kvz_decode_int4_workspace_size(B, G, pages.shape[1] * page, d)
    assert need == kvz.kvz_decode_int4_workspace_size(B, G, other[1].shape[1] * page, d) > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    cnt, nxt = n0.clone(), n0.clone()
    k, v, q = rand((B, 1, d), 43), rand((B, 1, d), 44), rand((B, G, 1, d), 45)
    t = table(d, 9400)
    pos = n0[:, None].clone()
    q_out = torch.empty_like(q)
    out, lse2 = torch.empty((B, G, d), device="cuda"), torch.empty((B, G), device="cuda")
    out2 = torch.empty((B, G, d), device="cuda")
    g1, g2, g3 = (torch.cuda.CUDAGraph() for _ in range(3))
    with torch.cuda.graph(g1):
        kvz.kvz_append_int4(k, v, cache, pages, cnt, page, positions=pos, table=t, q=q, q_out=q_out, counts_out=nxt)
        cnt.copy_(nxt)
        pos.add_(1)
    with torch.cuda.graph(g2):
        kvz.kvz_decode_int4(q_out.view(B, G, d), cache, pages, cnt, page, out=out, lse2=lse2, workspace=ws)
    with torch.cuda.graph(g3):
        kvz.kvz_decode_int4(q_out.view(B, G, d), other[0], other[1], other[2], page, out=out2, lse2=lse2, workspace=ws)
    for step in range(5):
        for x, s in ((k, 50), (v, 60), (q, 70)):
            x.copy_(rand(tuple(x.shape), s + step))
        g1.replay()
        g2.replay()
        got = out.clone()
        g3.replay()
        torch.cuda.synchronize()
        assert cnt.tolist() == [c + step + 1 for c in counts]
        ref, _ = check_decode(q_out.view(B, G, d), cache, pages, cnt, page, d ** -0.5)
        assert torch.equal(got, ref)
        assert torch.equal(out2, kvz.kvz_decode_int4(q_out.view(B, G, d), other[0], other[1], other[2], page)[0])


def test_calls_that_follow_each_other_at_once():
    # a kernel may start while the one before it ends: the same steps with and without a wait after each call
    d, page, B, G, T = 128, 32, 5, 4, 40
    t = table(d, 200)
    k, v, q = rand((T, B, 1, d), 50), rand((T, B, 1, d), 51), rand((T, B, G, 1, d), 52)
    runs = []
    for wait in (True, False):
        cache, pages = pool([T + 60] * B, d, page, 4)
        pages = torch.stack([pages, pages])               # copies, so that the two forms alternate
        n = torch.tensor([0, 1, 17, 31, 60], dtype=torch.int32, device="cuda")
        kvz.kvz_append_int4(rand((B, 60, d), 53), rand((B, 60, d), 54), cache, pages[0],
                            torch.zeros_like(n), page, n_new=n)
        tabs = (pages[0], wide(pages[1], page))
        torch.cuda.synchronize()
        outs = []
        for i in range(T):
            n, qr = kvz.kvz_append_int4(k[i], v[i], cache, tabs[0], n, page, positions=n[:, None], table=t, q=q[i])
            if wait:
                torch.cuda.synchronize()
            qi = kvz.kvz_rotary(qr, n[:, None], t, inverse=True)
            if wait:
                torch.cuda.synchronize()
            o, l2 = kvz.kvz_decode_int4(qr.view(B, G, d), cache, tabs[i % 2], n, page)
            if wait:
                torch.cuda.synchronize()
            outs += [qr, qi, o, l2]
        K, V = kvz.kvz_expand_int4(cache, tabs[0], n, offsets_of([T + c for c in (0, 1, 17, 31, 60)]), page,
                                   out_rows=5 * T + 109)
        torch.cuda.synchronize()
        runs.append(outs + [n, K, V, cache])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
def test_pages_read_again_after_a_write_between(d):
    # expand, append, expand, ... with no wait: each reading finds what the writing just before it left, in the same
    # lines of the same pages; and rows turned in place, compacted, turned on and compacted again
    page, B, rounds = 16, 40, 12
    cnt = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache, pages = pool([16 * 3] * B, d, page, 6)
    off = offsets_of([1] * B)
    k = [rand((B, 1, d), 300 + i) for i in range(rounds)]
    torch.cuda.synchronize()
    got = []
    for i in range(rounds):                           # the same slot of every head, over and over
        n, _ = kvz.kvz_append_int4(k[i], k[i], cache, pages, cnt, page)
        got.append(kvz.kvz_expand_int4(cache, pages, n, off, page, out_rows=B))
    for i in range(rounds):
        ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(bits(k[i])[:, 0])))
        for x in got[i]:
            np.testing.assert_array_equal(bits(x), ref)
    t = table(d, 100)
    n_c = 64
    pos = torch.full((n_c,), 7, dtype=torch.int32, device="cuda")
    idx = torch.arange(n_c, dtype=torch.int32, device="cuda").repeat(B)
    full = torch.full((B,), n_c, dtype=torch.int32, device="cuda")
    off = offsets_of([n_c] * B)
    caches = [pool([n_c] * B, d, page, 6) for _ in range(rounds)]
    x = rand((B, n_c, d), 400)
    y, want = x.clone(), []
    for i in range(rounds):
        y = kvz.kvz_rotary(y, pos, t)
        torch.cuda.synchronize()
        want.append(y)
    for c, p in caches:
        kvz.kvz_rotary(x, pos, t, out=x)
        kvz.kvz_compact_int4(x, x, idx, full, off, c, p, page)
    for (c, p), w in zip(caches, want):
        other = torch.full_like(c, 255)
        kvz.kvz_compact_int4(w, w, idx, full, off, other, p, page)
        assert torch.equal(c, other)


def test_two_streams_at_once():
    # the same cache read by two streams, each with its own workspace, and a third call over another cache
    cache, pages, n, _, _ = filled([3000, 12, 9000], 128, 64, 60)
    pages = wide(pages, 64)
    q = [rand((3, 4, 128), 61 + i) for i in range(2)]
    ref = [kvz.kvz_decode_int4(x, cache, pages, n, 64) for x in q]
    need = kvz.kvz_decode_int4_workspace_size(3, 4, pages.shape[1] * 64, 128)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in q]
    out = [[torch.empty_like(r) for r in rs] for rs in ref]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                kvz.kvz_decode_int4(q[i], cache, pages, n, 64, out=out[i][0], lse2=out[i][1], workspace=ws[i])
    torch.cuda.synchronize()
    for a, b in zip(ref, out):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_compact_uses_the_counted_indexes_only():
    # offsets may leave a head more room than its rows; what lies there is no index
    B, n_c, d, page, room = 3, 300, 64, 32, 200
    K, V = rand((B, n_c, d), 71), rand((B, n_c, d), 72)
    counts = [17, 0, 160]
    idx = torch.full((B * room,), -5, dtype=torch.int32, device="cuda")
    for b, c in enumerate(counts):
        idx[b * room:b * room + c] = torch.arange(c, dtype=torch.int32, device="cuda") + b
    n = torch.tensor(counts, dtype=torch.int32, device="cuda")
    cache, pages = pool(counts, d, page, 8)
    st = new_status()
    kvz.kvz_compact_int4(K, V, idx, n, offsets_of([room] * B), cache, pages, page, status=st)
    got = kvz.kvz_expand_int4(cache, pages, n, offsets_of(counts), page, out_rows=sum(counts))
    assert st.item() == 0
    for src, out in ((K, got[0]), (V, got[1])):
        rows = torch.cat([src[b, b:b + c] for b, c in enumerate(counts)])
        ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(bits(rows))))
        np.testing.assert_array_equal(bits(out), ref)


def test_every_step():
    # a group for every normal bf16 as its range: the step's reciprocal is division's for each
    top = (torch.arange(128, 255 * 128, dtype=torch.int32) << 16).view(torch.float32)
    g = torch.Generator().manual_seed(70)
    x = torch.rand((top.numel(), 64), generator=g)
    x[:, 0], x[:, 1] = 0.0, 1.0
    x = (x.double() * top[:, None].double()).to(torch.bfloat16)
    rows = x.view(-1, 128).cuda()
    n = rows.shape[0]
    cache, pages = pool([n], 128, 64, 7)
    counts = torch.tensor([n], dtype=torch.int32, device="cuda")
    idx = torch.arange(n, dtype=torch.int32, device="cuda")
    other = rows.flip(0).contiguous()
    kvz.kvz_compact_int4(rows[None], other[None], idx, counts, offsets_of([n]), cache, pages, 64)
    K, V = kvz.kvz_expand_int4(cache, pages, counts, offsets_of([n]), 64, out_rows=n)
    for src, got in ((rows, K), (other, V)):
        ref = o4.round_bf16(o4.group_values(*o4.quantize_groups(bits(src))))
        np.testing.assert_array_equal(bits(got), ref)


def test_whole_path_from_scores_to_answers():
    # score, select, compact into four bits, then tokens one by one: the cache equals the oracle's, byte for byte,
    # and so does what every step attends to
    w = synth.WORKLOADS["tiny"]
    x = synth.layer_inputs(w, device="cuda:0")
    B, G, d, page, steps = w.B, w.G, w.d, 16, 6
    t = table(d, 400)
    pos_ctx = torch.arange(w.n_c[0], dtype=torch.int32, device="cuda")
    pos_in = torch.arange(w.n_in(), dtype=torch.int32, device="cuda") + w.n_c[0]
    t_in = table(d, int(pos_in[-1]) + 1)
    K_ctx = kvz.kvz_rotary(x["K_ctx"], pos_ctx, t_in)
    S = kvz.kvz_score(kvz.kvz_rotary(x["Q"], pos_in, t_in), K_ctx, kvz.kvz_rotary(x["K_in"], pos_in, t_in))
    idx, counts, offsets = kvz.kvz_select(S, w.ratio, w.mode)
    kept = int(offsets[-1])
    cache, pages = pool([kept + steps], d, page, 6)
    before, st = cache.cpu().numpy(), new_status()
    kvz.kvz_compact_int4(K_ctx, x["V"], idx, counts, offsets, cache, pages, page, status=st)
    ih, Kb, Vb = idx.cpu().numpy(), bits(K_ctx)[0], bits(x["V"])[0]
    rows = {(0, p): (Kb[ih[p]], Vb[ih[p]]) for p in range(kept)}
    n = counts
    for i in range(steps):
        k, v, q = rand((1, 1, d), 80 + i), rand((1, 1, d), 90 + i), rand((1, G, 1, d), 100 + i)
        pos = torch.tensor([w.n_c[0] + i], dtype=torch.int32, device="cuda")   # positions go on from the whole context
        n, qr = kvz.kvz_append_int4(k, v, cache, pages, n, page, positions=pos, table=t, q=q, status=st)
        rows[(0, kept + i)] = (o4.rotary(bits(k), pos.cpu().numpy(), t.cpu().numpy())[0, 0], bits(v)[0, 0])
        check_decode(qr.view(1, G, d), cache, pages, n, page, d ** -0.5)
    assert st.item() == 0 and n.tolist() == [kept + steps]
    np.testing.assert_array_equal(cache.cpu().numpy(), expected_bytes(before, pages.cpu().numpy(), page, d, rows))
