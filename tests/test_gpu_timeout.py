"""The bounded ordering wait of in-place compaction, made to expire on
purpose through the test entry point (include/kvz_testing.h): one chunk
never reports its source rows as read, so the chunk whose rows they are
gives up after 1 ms.  The launch must return, report KVZ_ERR_TIMEOUT (7)
in the device status word, leave every other head exactly compacted, and
leave the context usable.  Nothing here faults, traps or spins unbounded."""
import time

import numpy as np
import pytest
import torch

from kvz_testutil import bits
from oracle import kvz_oracle as orc
from query_agnostic_kv_kvz_b200 import synth

pytestmark = pytest.mark.gpu

kvz = pytest.importorskip("query_agnostic_kv_kvz_b200")

CHUNK = 16          # slots per in-place chunk (the kernel's unit of ordering)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kvz.lib()


def _held_chunk(sel):
    """A chunk k that reads a row some later chunk c > k overwrites (so
    chunk c waits for k), and that c."""
    for k in range(len(sel) // CHUNK):
        later = [int(j) // CHUNK for j in sel[k * CHUNK:(k + 1) * CHUNK] if int(j) // CHUNK > k]
        if later:
            return k, later[0]
    raise AssertionError("no chunk has a later reader")


@pytest.mark.parametrize("d,ratio,hold_head", [(128, 0.3, 2), (64, 0.25, 0)])
def test_in_place_wait_expires_with_timeout_status(d, ratio, hold_head):
    B, n_c = 6, 4096
    g = torch.Generator(device="cuda").manual_seed(d)
    K = torch.randn((B, n_c, d), generator=g, device="cuda").to(torch.bfloat16)
    V = torch.randn((B, n_c, d), generator=g, device="cuda").to(torch.bfloat16)
    S = synth.synthetic_scores(B, n_c, seed=d, device="cuda")
    idx, counts, offsets = kvz.kvz_select(S, ratio, "per_head")
    torch.cuda.synchronize()
    ri, rc, ro = orc.select(S.cpu().numpy(), ratio, "per_head")
    np.testing.assert_array_equal(idx.cpu().numpy()[: len(ri)], ri)
    k, c = _held_chunk(ri[ro[hold_head]:ro[hold_head + 1]])
    assert c > k
    Kh, Vh = bits(K), bits(V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t0 = time.perf_counter()
    kvz.kvz_testing_compact_in_place_withhold(K, V, idx, counts, offsets, wait_ns=1_000_000, hold_head=hold_head,
                                              hold_chunk=k, status=status)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert elapsed < 10.0, "the launch did not return promptly (%.1f s)" % elapsed
    assert int(status.item()) == 7, kvz.STATUS.get(int(status.item()))
    Ko, Vo = bits(K), bits(V)
    for b in range(B):
        if b == hold_head:
            continue
        sel = ri[ro[b]:ro[b + 1]]
        np.testing.assert_array_equal(Ko[b, : len(sel)], Kh[b][sel], err_msg="head %d" % b)
        np.testing.assert_array_equal(Vo[b, : len(sel)], Vh[b][sel], err_msg="head %d" % b)
    # the chunks of the held head below the waiting chunk's readers are done
    sel = ri[ro[hold_head]:ro[hold_head + 1]]
    np.testing.assert_array_equal(Ko[hold_head, : k * CHUNK], Kh[hold_head][sel[: k * CHUNK]])

    # the context is still usable: a normal in-place compaction is exact
    K2 = torch.from_numpy(Kh.view(np.int16)).cuda().view(torch.bfloat16)
    V2 = torch.from_numpy(Vh.view(np.int16)).cuda().view(torch.bfloat16)
    status.zero_()
    kvz.kvz_compact(K2, V2, idx, counts, offsets, in_place=True, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    Ko2, Vo2 = bits(K2), bits(V2)
    for b in range(B):
        sel = ri[ro[b]:ro[b + 1]]
        np.testing.assert_array_equal(Ko2[b, : len(sel)], Kh[b][sel])
        np.testing.assert_array_equal(Vo2[b, : len(sel)], Vh[b][sel])


def test_withhold_arguments_are_checked():
    K = torch.zeros((2, 64, 128), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    idx = torch.zeros(2, dtype=torch.int32, device="cuda")
    counts = torch.ones(2, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 1, 2], dtype=torch.int64, device="cuda")
    for wait_ns, hb, hc in [(10, 0, 0), (2_000_000_000, 0, 0), (1_000_000, 2, 0), (1_000_000, 0, -1)]:
        with pytest.raises(kvz.KvzError) as e:
            kvz.kvz_testing_compact_in_place_withhold(K, V, idx, counts, offsets, wait_ns, hb, hc)
        assert e.value.code == 1


def _four_bit(counts, d, page, seed, rows=0):
    """A 4-bit cache of `counts` rows a head on consecutive pages, its table at least `rows` rows wide."""
    B, width = len(counts), max(-(-max(counts) // page), 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((B, max(counts), d), generator=g, device="cuda").bfloat16() for _ in range(2))
    pages = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    cache = torch.zeros((B * width, page * d * 9 // 8), dtype=torch.uint8, device="cuda")
    n = torch.tensor(counts, dtype=torch.int32, device="cuda")
    kvz.kvz_append_int4(k, v, cache, pages, torch.zeros_like(n), page, n_new=n)
    more = torch.full((B, max(0, rows // page - width)), -1, dtype=torch.int32, device="cuda")
    return cache, torch.cat([pages, more], 1), n, torch.randn((B, 4, d), generator=g, device="cuda").bfloat16()


def _withheld(cache, pages, n, q, page, head, cta, workspace=None):
    """The outputs with the wait expired, and those of the same call without it."""
    good = kvz.kvz_decode_int4(q, cache, pages, n, page)
    if workspace is not None:                         # partials that look right: another question's
        kvz.kvz_decode_int4(q.flip(0).contiguous(), cache, pages, n, page, workspace=workspace)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse2 = torch.full_like(good[0], 5.0), torch.full_like(good[1], 5.0)
    t0 = time.perf_counter()
    kvz.kvz_testing_decode_int4_withhold(q, cache, pages, n, page, 5_000_000, head, cta, out=out, lse2=lse2,
                                         workspace=workspace, status=status)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 10.0
    assert int(status.item()) == 7, kvz.STATUS.get(int(status.item()))
    bad = torch.isnan(out).all(-1).all(-1)
    assert torch.equal(bad, torch.isnan(lse2).all(-1))
    for x, ref in ((out, good[0]), (lse2, good[1])):
        assert torch.equal(x[~bad], ref[~bad])        # every head is NaN or as it should be
    status.zero_()                                    # and the next call is right
    again = kvz.kvz_decode_int4(q, cache, pages, n, page, workspace=workspace, status=status)
    assert int(status.item()) == 0 and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    return bad.nonzero().view(-1).tolist()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cta", [-1, 43, 60, 89])
def test_attention_in_shares_whose_wait_expires(d, cta):
    # shares of 16 blocks: head 2 is read by CTAs 43 (after its beginning) to 89; one of them fails, or all
    page = 32
    cache, pages, n, q = _four_bit([9000, 50, 12000, 0, 700], d, page, d, 40000)
    ws = torch.empty(kvz.kvz_decode_int4_workspace_size(5, 4, pages.shape[1] * page, d), dtype=torch.uint8, device="cuda")
    assert _withheld(cache, pages, n, q, page, 2, cta, ws) == [2]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("head", [0, 5, 300, 599])
def test_attention_in_shares_of_many_heads_whose_wait_expires(d, head):
    # a share holds several heads: the failing one and those after it in the share are NaN, and one that the share
    # begins and the next goes on with
    page = 32
    counts = [(b * 37) % 90 + 1 for b in range(600)]
    counts[301] = 3000
    cache, pages, n, q = _four_bit(counts, d, page, d, 40000)
    ws = torch.empty(kvz.kvz_decode_int4_workspace_size(600, 4, pages.shape[1] * page, d), dtype=torch.uint8,
                     device="cuda")
    bad = _withheld(cache, pages, n, q, page, head, -1, ws)
    assert bad[0] == head and bad == list(range(head, head + len(bad))) and len(bad) <= 6


@pytest.mark.parametrize("B,head", [(3, 1), (64, 63), (200, 7)])
def test_attention_by_clusters_whose_wait_expires(B, head):
    page = 32
    cache, pages, n, q = _four_bit([(b * 37) % 900 + 1 for b in range(B)], 128, page, B)
    assert kvz.kvz_decode_int4_workspace_size(B, 4, pages.shape[1] * page, 128) == 0
    assert _withheld(cache, pages, n, q, page, head, -1) == [head]


def test_attention_withhold_arguments_are_checked():
    cache, pages, n, q = _four_bit([40, 40], 64, 32, 1)
    for wait_ns, hb, hc in [(10, 0, 0), (2_000_000_000, 0, 0), (1_000_000, 2, 0), (1_000_000, -2, 0), (1_000_000, 0, -2)]:
        with pytest.raises(kvz.KvzError) as e:
            kvz.kvz_testing_decode_int4_withhold(q, cache, pages, n, 32, wait_ns, hb, hc)
        assert e.value.code == 1
