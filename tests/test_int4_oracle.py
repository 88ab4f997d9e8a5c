"""Pins of the 4-bit oracle, on the CPU: the layout against hand-placed
nibbles, the quantisation against its bounds and corner groups, the rotation
against complex numbers, its inverse and its gradient."""
import numpy as np
import pytest

from oracle import kvz_oracle as orc
from oracle import kvz_oracle_int4 as o4


def bits_of(x):
    return o4.round_bf16(np.asarray(x, dtype=np.float32))


def test_round_bf16_ties_to_even():
    x = np.array([1.0, 1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, -1.0 - 2.0 ** -8, 0.0, np.inf], np.float32)
    assert [hex(v) for v in o4.round_bf16(x)] == ["0x3f80", "0x3f80", "0x3f82", "0xbf80", "0x0", "0x7f80"]
    assert np.isnan(orc.bf16_bits_to_f64(o4.round_bf16(np.array([np.nan], np.float32))))[0]


@pytest.mark.parametrize("d", [64, 128])
def test_layout_places_every_bit_once(d):
    k, v = o4._places(d)
    flat = np.concatenate([k.reshape(-1), v.reshape(-1)])
    assert len(np.unique(flat)) == flat.size == 8 * 16 * d
    assert flat.max() < 8 * 16 * d


def test_layout_by_hand():
    d = 128
    z = np.zeros((16, d), np.uint8)
    s = np.zeros((16, 2), np.uint16)
    kc, vc = z.copy(), z.copy()
    kc[3, 64 + 16 + 8 + 1] = 0xF       # row 3, g = 1, c = 1, u = 1, dim 1 of 8: nibble 4, rotated by 3
    vc[5, 64 + 8 * 2 + 4 + 3] = 0xF    # row 5 (pair 2, odd), g = 1, r = 2, w = 1, nibble 3
    ks, km = s.copy(), s.copy()
    ks[7, 1], km[7, 1] = 0x1234, 0x5678
    raw = o4.pack_block(kc, ks, km, vc, s, s)
    word = (3 * 16 + (1 * 2 + 1) * 2 + 1)
    assert raw[4 * word: 4 * word + 4].view(np.uint32)[0] == 0xF << 19
    half = ((2 * 8 + 2) * 2 + 1) * 4 + 1 * 2 + 1
    assert raw[8 * d:].view(np.uint16)[half] == 0xF000
    assert raw[16 * d:].view(np.uint16)[2 * (7 * 2 + 1): 2 * (7 * 2 + 1) + 2].tolist() == [0x1234, 0x5678]
    assert np.count_nonzero(raw) == 1 + 1 + 4          # (0xF << 19 is the byte 0x78)
    back = o4.unpack_block(raw, d)
    for a, b in zip(back, (kc, ks, km, vc, s, s)):
        np.testing.assert_array_equal(a, b)


def test_quantisation_bounds_and_corners():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)) * np.exp(rng.standard_normal((50, 1)) * 3)
    b = bits_of(x)
    codes, s, m = o4.quantize_groups(b)
    assert codes.max() == 15 and codes.min() == 0
    y, xb = o4.group_values(codes, s, m), orc.bf16_bits_to_f64(b)
    step = orc.bf16_bits_to_f64(s).repeat(64, 1)
    # half a step, and up to 15 roundings of the bf16 step (2^-8 each) where it was rounded down
    assert np.all(np.abs(y - xb) <= step * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -22 * np.abs(xb))
    c = np.zeros((6, 64), np.float32)
    c[0] = 3.25                         # a constant group is exact
    c[1, 5] = np.nan
    c[2, 5] = np.inf
    c[3, 0], c[3, 1] = 3e38, -3e38      # finite, but the range is not
    c[4, 7] = 2.0 ** -130               # a step under the smallest normal number
    c[5, 1] = 15.0
    codes, s, m = o4.quantize_groups(bits_of(c))
    y = o4.group_values(codes, s, m)
    assert np.all(y[0] == 3.25) and np.all(np.isnan(y[1:4])) and np.all(y[4] == 0.0)
    assert y[5, 1] == 15.0 and codes[5, 1] == 15


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    rot, d, n = 32, 64, 7
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    t = o4.rotary_table(f, 200)
    pos = rng.integers(0, 200, n)
    b = bits_of(rng.standard_normal((n, d)))
    y = orc.bf16_bits_to_f64(o4.rotary(b, pos, t, interleaved))
    x = orc.bf16_bits_to_f64(b)
    ia = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    z = (x[:, ia] + 1j * x[:, ib]) * np.exp(1j * pos[:, None] * f)
    tol = 2.0 ** -8 * np.abs(z) + 1e-6                      # one bf16 rounding, float32 before it
    assert np.all(np.abs(y[:, ia] - z.real) <= tol) and np.all(np.abs(y[:, ib] - z.imag) <= tol)
    np.testing.assert_array_equal(y[:, rot:], x[:, rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    # <rotary(x), w> has the gradient inverse(w) in x, and its differences say the same
    rng = np.random.default_rng(2)
    rot = d = 64
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    t = o4.rotary_table(f, 100, factor=1.25)
    pos = np.array([77])
    w = bits_of(rng.standard_normal((1, d)))
    g = orc.bf16_bits_to_f64(o4.rotary(w, pos, t, interleaved, inverse=True))[0]
    wv = orc.bf16_bits_to_f64(w)[0]
    for j in range(d):
        e = np.zeros((1, d), np.float32)
        e[0, j] = 1.0
        # linear, so one unit step is the difference; two entries of the column, a bf16 rounding each
        col = orc.bf16_bits_to_f64(o4.rotary(bits_of(e), pos, t, interleaved))[0]
        assert abs(col @ wv - g[j]) <= 2.0 ** -8 * (np.abs(col) @ np.abs(wv) + abs(g[j])) + 1e-6
