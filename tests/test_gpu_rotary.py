"""GPU parity of the rotary positions: bit for bit against the oracle's
float32 steps (the table's entries are rounded once from float64), over
layouts, widths, strides, in place, and the inverse as the gradient."""
import numpy as np
import pytest
import torch

from kvz_testutil import bits
from oracle import kvz_oracle_int4 as o4

pytestmark = pytest.mark.gpu

kvz = pytest.importorskip("query_agnostic_kv_kvz_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kvz.lib()


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def table(rot, n_pos, **kw):
    f, a = kvz.kvz_rotary_freqs(rot, **kw)
    return kvz.kvz_rotary_table(f.cuda(), n_pos, a)


@pytest.mark.parametrize("rot,n_pos,kw", [(128, 5000, {}), (16, 1, {}), (64, 131072, {}),
                                          (96, 3000, dict(base=1e6, scaling={"type": "yarn", "factor": 8,
                                                                             "original": 1024}))])
def test_table(rot, n_pos, kw):
    f, a = kvz.kvz_rotary_freqs(rot, **kw)
    t = table(rot, n_pos, **kw).cpu().double().numpy()
    ang = np.arange(n_pos)[:, None] * f.numpy()
    ref = np.concatenate([np.cos(ang), np.sin(ang)], 1) * a
    # one float32 rounding of a float64 value that is itself good to a few 2^-53
    assert np.all(np.abs(t - ref) <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -50)


def check(x, pos, t, il, inv, y):
    p = pos.cpu().numpy()
    if x.dim() == 4 and p.ndim == 2:
        p = p[:, None]
    ref = o4.rotary(bits(x), p, t.cpu().numpy(), il, inv)
    np.testing.assert_array_equal(bits(y), ref)


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("shape,rot", [((1, 1, 1, 128), 128), ((3, 5, 17, 128), 96), ((2, 4, 333, 64), 64),
                                       ((9, 1, 40, 64), 16), ((64, 8, 1, 128), 64), ((2, 3, 1000, 128), 128),
                                       ((1, 13, 3, 64), 48)])
def test_rotary_matches_oracle(shape, rot, il):
    B, G, n, d = shape
    x = rand(shape, n)
    t = table(rot, 4000)
    pos = torch.randint(0, 4000, (n,), dtype=torch.int32, device="cuda")
    own = torch.randint(0, 4000, (B, n), dtype=torch.int32, device="cuda")
    for inv in (False, True):
        for p in (pos, own):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            check(x, p, t, il, inv, kvz.kvz_rotary(x, p, t, interleaved=il, inverse=inv, status=status))
            assert status.item() == 0
    k = x[:, 0]                                       # [B, n, d], a strided view where G > 1
    check(k, pos, t, il, False, kvz.kvz_rotary(k, pos, t, interleaved=il))


def test_rotary_views_in_place_and_out():
    B, G, n, d, rot = 3, 4, 70, 128, 64
    t = table(rot, 500)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + 300
    fused = rand((n, B, G + 2, d), 1)                 # a projection's rows: G query heads and two others
    x = fused[:, :, :G].permute(1, 2, 0, 3)
    ref = kvz.kvz_rotary(x, pos, t)
    check(x, pos, t, False, False, ref)
    keep = fused.clone()
    out = torch.full((B, G, n, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kvz.kvz_rotary(x, pos, t, out=out[..., d:]).data_ptr() == out[..., d:].data_ptr()
    assert torch.equal(out[..., d:], ref) and bool((out[..., :d] == 7).all())
    y = kvz.kvz_rotary(x, pos, t, out=x)              # in place through the view
    assert y.data_ptr() == fused.data_ptr() and torch.equal(x, ref)
    assert torch.equal(fused[:, :, G:], keep[:, :, G:])
    wide = rand((B, 1, n, d), 2).expand(B, G, n, d)   # one row read by every query head
    check(wide, pos, t, True, False, kvz.kvz_rotary(wide, pos, t, interleaved=True))


def test_inverse_turns_back_and_is_the_gradient():
    B, n, d = 2, 50, 128
    t = table(d, 1000)
    pos = torch.randint(0, 1000, (n,), dtype=torch.int32, device="cuda")
    x, w = rand((B, n, d), 3), rand((B, n, d), 4)
    y = kvz.kvz_rotary(x, pos, t)
    back = kvz.kvz_rotary(y, pos, t, inverse=True)
    # each entry of y carries a rounding of 2^-8 of the pair's length at most, and back one of its own
    pair = (x.float()[..., :64] ** 2 + x.float()[..., 64:] ** 2).sqrt().repeat(1, 1, 2)
    assert bool(((back.float() - x.float()).abs() <= 3 * 2.0 ** -8 * pair + 1e-6).all())
    # <rotary(x), w> differentiated by float64 autograd through the plain formula
    xd = x.double().requires_grad_()
    c, s = t.double()[pos.long()][:, :64], t.double()[pos.long()][:, 64:]
    a, b = xd[..., :64], xd[..., 64:]
    (torch.cat([a * c - b * s, b * c + a * s], -1) * w.double()).sum().backward()
    g = kvz.kvz_rotary(w, pos, t, inverse=True)
    # one bf16 rounding; the float32 steps before it lose 2^-22 of the pair's length
    wp = (w.double()[..., :64] ** 2 + w.double()[..., 64:] ** 2).sqrt().repeat(1, 1, 2)
    assert bool(((g.double() - xd.grad).abs() <= 2.0 ** -8 * xd.grad.abs() * 1.001 + 2.0 ** -22 * wp).all())


def test_rotary_reports_positions_outside_the_table():
    t = table(64, 10)
    x = rand((2, 5, 64), 5)
    pos = torch.tensor([0, 9, 10, -1, 3], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvz.kvz_rotary(x, pos, t, out=out, status=status)
    assert status.item() == 1
    assert bool((out[:, 2:4] == 5).all())
    good = torch.tensor([0, 1, 4], device="cuda")
    check(x[:, good], pos[good], t, False, False, out[:, good])


def test_rotary_stream_and_graph():
    t = table(128, 3000)
    x = rand((8, 4, 300, 128), 6)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    ref = kvz.kvz_rotary(x, pos, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = kvz.kvz_rotary(x, pos, t, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvz.kvz_rotary(x, pos, t, out=out)
    for k in range(3):
        x.copy_(rand(tuple(x.shape), 7 + k))
        out.zero_()
        g.replay()
        assert torch.equal(out, kvz.kvz_rotary(x, pos, t))


def test_rotary_offsets_past_32_bits():
    # a view whose rows lie 2^32 bytes and more apart
    base = torch.empty(5 << 30, dtype=torch.uint8, device="cuda").view(torch.bfloat16)
    x = torch.as_strided(base, (2, 3, 64), (base.numel() - 3 * 64, 64, 1))
    x.copy_(rand((2, 3, 64), 9))
    t = table(64, 10)
    pos = torch.tensor([1, 5, 9], dtype=torch.int32, device="cuda")
    check(x, pos, t, False, False, kvz.kvz_rotary(x, pos, t))
