"""The rotary and 4-bit cache calls refuse malformed arguments before
anything is launched: the Python binding (with a stand-in for the library
whose compute entry points fail the test), and the C ABI's own checks (the
real library, which refuses before it touches the GPU).  Runs on the CPU."""
import ctypes
import glob
import os
import re

import numpy as np
import pytest
import torch

import query_agnostic_kv_kvz_b200 as kvz

bf16, f32, f64, i32, i64, u8 = (torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64, torch.uint8)


class _NoLaunchLib:
    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 1 << 16

        def launched(*a):
            raise AssertionError("%s reached the C ABI with a malformed argument" % name)
        return launched


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setattr(kvz, "lib", lambda: _NoLaunchLib())


def z(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


B, G, T, n_c, d, page = 2, 3, 4, 50, 64, 32
pb = page * d * 9 // 8
x3, x4 = z((B, T, d), bf16), z((B, G, T, d), bf16)
pos, tab = z(T, i32), z((100, d), f32)
cache, pages, cnt, off = z((6, pb), u8), z((B, 3), i32), z(B, i32), z(B + 1, i64)
idx, KV = z(B * 15, i32), z((B, n_c, d), bf16)
q3 = z((B, G, d), bf16)


def append(k=x3, v=x3, cache=cache, pages=pages, counts=cnt, ps=page, **kw):
    return lambda: kvz.kvz_append_int4(k, v, cache, pages, counts, ps, **kw)


CASES = {
    "table: freqs dtype": lambda: kvz.kvz_rotary_table(z(32, f32), 10),
    "table: freqs rank": lambda: kvz.kvz_rotary_table(z((4, 8), f64), 10),
    "table: n_pos": lambda: kvz.kvz_rotary_table(z(32, f64), 0),
    "table: shape": lambda: kvz.kvz_rotary_table(z(32, f64), 10, table=z((10, 32), f32)),
    "table: CPU": lambda: kvz.kvz_rotary_table(z(32, f64), 10),
    "rotary: dtype": lambda: kvz.kvz_rotary(x3.float(), pos, tab),
    "rotary: rank": lambda: kvz.kvz_rotary(z((T, d), bf16), pos, tab),
    "rotary: last dimension": lambda: kvz.kvz_rotary(z((B, d, T), bf16).transpose(1, 2), pos, tab),
    "rotary: stride": lambda: kvz.kvz_rotary(z((B, T, d + 4), bf16)[..., :d], pos, tab),
    "rotary: base": lambda: kvz.kvz_rotary(z(B * T * d + 8, bf16)[4:-4].view(B, T, d), pos, tab),
    "rotary: positions dtype": lambda: kvz.kvz_rotary(x3, pos.long(), tab),
    "rotary: positions shape": lambda: kvz.kvz_rotary(x3, z(T + 1, i32), tab),
    "rotary: positions per head": lambda: kvz.kvz_rotary(x4, z((B * G, T), i32), tab),
    "rotary: table dtype": lambda: kvz.kvz_rotary(x3, pos, tab.double()),
    "rotary: no table": lambda: kvz.kvz_rotary(x3, pos, None),
    "rotary: out shape": lambda: kvz.kvz_rotary(x3, pos, tab, out=z((B, T, 2 * d), bf16)),
    "rotary: out overlaps itself": lambda: kvz.kvz_rotary(x3, pos, tab, out=z((1, T, d), bf16).expand(B, T, d)),
    "rotary: out overlaps x": lambda: kvz.kvz_rotary(*(lambda m: (m[:B], pos, tab, False, False, m[1:]))(
        z((B + 1, T, d), bf16))),
    "rotary: CPU": lambda: kvz.kvz_rotary(x3, pos, tab),
    "compact: cache width": lambda: kvz.kvz_compact_int4(KV, KV, idx, cnt, off, z((6, pb + 16), u8), pages, page),
    "compact: page size": lambda: kvz.kvz_compact_int4(KV, KV, idx, cnt, off, cache, pages, 24),
    "compact: pages rows": lambda: kvz.kvz_compact_int4(KV, KV, idx, cnt, off, cache, z((B + 1, 3), i32), page),
    "compact: pages dtype": lambda: kvz.kvz_compact_int4(KV, KV, idx, cnt, off, cache, pages.long(), page),
    "compact: V shape": lambda: kvz.kvz_compact_int4(KV, z((B, n_c - 1, d), bf16), idx, cnt, off, cache, pages, page),
    "compact: counts short": lambda: kvz.kvz_compact_int4(KV, KV, idx, z(B - 1, i32), off, cache, pages, page),
    "compact: offsets short": lambda: kvz.kvz_compact_int4(KV, KV, idx, cnt, z(B, i64), cache, pages, page),
    "compact: no idx": lambda: kvz.kvz_compact_int4(KV, KV, None, cnt, off, cache, pages, page),
    "compact: CPU": lambda: kvz.kvz_compact_int4(KV, KV, idx, cnt, off, cache, pages, page),
    "append: k rank": append(k=z((T, d), bf16)),
    "append: v shape": append(v=z((B, T + 1, d), bf16)),
    "append: k stride": append(k=z((B, T, d + 2), bf16)[..., :d]),
    "append: counts dtype": append(counts=z(B, i64)),
    "append: no counts": append(counts=None),
    "append: counts in place": append(counts_out=cnt),
    "append: counts over n_new": (lambda m: append(n_new=m, counts_out=m))(z(B, i32)),
    "append: counts over positions": (lambda m: append(positions=m, table=tab, counts_out=m.view(-1)))(z((B, T), i32)),
    "append: q_out over k": (lambda m: append(k=m[:, 0], q=x4, q_out=m))(z((B, G, T, d), bf16)),
    "append: q_out over v": (lambda m: append(v=m[:, 1], q=x4, q_out=m))(z((B, G, T, d), bf16)),
    "append: positions without table": append(positions=pos),
    "append: table without positions": append(table=tab),
    "append: q heads": append(q=z((B + 1, G, T, d), bf16)),
    "append: q rank": append(q=x3),
    "append: q_out without q": append(q_out=x4),
    "append: q_out shape": append(q=x4, q_out=z((B, G, T + 1, d), bf16)),
    "append: q_out is q": append(q=x4, q_out=x4),
    "append: n_new short": append(n_new=z(B - 1, i32)),
    "append: n_new dtype": append(n_new=z(B, i64)),
    "append: no cache": append(cache=None),
    "append: pages rank": append(pages=z(6, i32)),
    "append: cache of d = 128": append(cache=z((6, page * 144), u8)),
    "append: page size 0": append(ps=0),
    "append: cache of no dimension": append(cache=z((), u8)),
    "append: cache flat": append(cache=z(6 * pb, u8)),
    "append: too many rows": append(pages=z((B, (1 << 30) // page + 1), i32).expand(B, -1)),
    "append: CPU": append(),
    "expand: no rows given": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page),
    "expand: negative rows": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page, out_rows=-1),
    "expand: K_out width": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page, K_out=z((5, 128), bf16),
                                                       V_out=z((5, 64), bf16)),
    "expand: K_out rows": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page, out_rows=9,
                                                      K_out=z((5, d), bf16)),
    "expand: one output twice": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page, K_out=z((5, d), bf16),
                                                            V_out=None, out_rows=None),
    "expand: outputs overlap": lambda: kvz.kvz_expand_int4(*(lambda m: (cache, pages, cnt, off, page, None, None,
                                                                       m[:5], m[2:7]))(z((7, d), bf16))),
    "expand: first dtype": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page, first=off, out_rows=3),
    "expand: cache width": lambda: kvz.kvz_expand_int4(z((6, pb - 1), u8), pages, cnt, off, page, out_rows=3),
    "expand: CPU": lambda: kvz.kvz_expand_int4(cache, pages, cnt, off, page, out_rows=3),
    "decode: q dtype": lambda: kvz.kvz_decode_int4(q3.float(), cache, pages, cnt, page),
    "decode: no q": lambda: kvz.kvz_decode_int4(None, cache, pages, cnt, page),
    "decode: q heads": lambda: kvz.kvz_decode_int4(z((B + 1, G, d), bf16), cache, pages, cnt, page),
    "decode: q width": lambda: kvz.kvz_decode_int4(z((B, G, 96), bf16), cache, pages, cnt, page),
    "decode: out dtype": lambda: kvz.kvz_decode_int4(q3, cache, pages, cnt, page, out=q3),
    "decode: lse2 shape": lambda: kvz.kvz_decode_int4(q3, cache, pages, cnt, page, lse2=z(B * G, f32)),
    "decode: workspace dtype": lambda: kvz.kvz_decode_int4(q3, cache, pages, cnt, page, workspace=z(9, f32)),
    "decode: status dtype": lambda: kvz.kvz_decode_int4(q3, cache, pages, cnt, page, status=z(1, i64)),
    "decode: CPU": lambda: kvz.kvz_decode_int4(q3, cache, pages, cnt, page),
    "freqs: rot": lambda: kvz.kvz_rotary_freqs(24),
    "freqs: base": lambda: kvz.kvz_rotary_freqs(64, base=0.5),
    "freqs: factor": lambda: kvz.kvz_rotary_freqs(64, scaling={"type": "linear", "factor": 0.5}),
    "freqs: type": lambda: kvz.kvz_rotary_freqs(64, scaling={"type": "other", "factor": 2}),
    "freqs: original": lambda: kvz.kvz_rotary_freqs(64, scaling={"type": "yarn", "factor": 2}),
}


@pytest.mark.parametrize("name", CASES)
def test_binding_refuses(no_launch, name):
    with pytest.raises(ValueError):
        CASES[name]()


# ---------------------------------------------------------------------------
# The C ABI
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from query_agnostic_kv_kvz_b200 import build
    build.build()
    return kvz.lib()


P = 4096                                     # an aligned address that no refused call reads
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


def _rotary(lib, **kw):
    a = dict(x=P, x_sb=64, x_sg=64, x_st=64, B=1, G=1, n=4, d=64, pos=P, pos_sb=0, table=P, n_pos=9, rot=64, il=0,
             inv=0, y=2 * P, y_sb=64, y_sg=64, y_st=64, st=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kvz_rotary(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=80), UNSUPPORTED), (dict(rot=0), UNSUPPORTED),
    (dict(B=0), INVALID), (dict(B=65536), INVALID), (dict(G=0), INVALID), (dict(n=0), INVALID),
    (dict(n=1 << 31), INVALID), (dict(n_pos=0), INVALID), (dict(il=2), INVALID), (dict(inv=-1), INVALID),
    (dict(pos_sb=-1), INVALID), (dict(x_st=4), ALIGNMENT), (dict(x_sb=-64), ALIGNMENT), (dict(y_sg=(1 << 41)), ALIGNMENT),
    (dict(x=P + 8), ALIGNMENT), (dict(y=P + 2), ALIGNMENT), (dict(table=P + 4), ALIGNMENT), (dict(pos=P + 1), ALIGNMENT),
    (dict(y=P, y_st=128), INVALID),
])
def test_c_rotary_refuses(lib, kw, code):
    assert _rotary(lib, **kw) == code


def test_c_table_refuses(lib):
    ok = (P, 10, 64, 1.0, P, None)
    for at, v, code in ((0, None, INVALID), (1, 0, INVALID), (2, 24, UNSUPPORTED), (2, 256, UNSUPPORTED),
                        (3, float("inf"), INVALID), (4, None, INVALID), (4, P + 4, ALIGNMENT), (0, P + 4, ALIGNMENT)):
        a = list(ok)
        a[at] = v
        assert lib.kvz_rotary_table(*a) == code


PAGES = dict(cache=P, n_pages=4, page=32, pages=P, max_pages=2)
BAD_PAGES = [(dict(cache=None), INVALID), (dict(pages=None), INVALID), (dict(n_pages=0), INVALID),
             (dict(n_pages=1 << 31), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=0), UNSUPPORTED),
             (dict(page=2048), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(max_pages=(1 << 25) + 1), INVALID),
             (dict(cache=P + 8), ALIGNMENT), (dict(pages=P + 2), ALIGNMENT), (dict(d=32), UNSUPPORTED),
             (dict(B=0), INVALID), (dict(B=65536), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_PAGES + [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(idx=None), INVALID), (dict(counts=None), INVALID),
    (dict(offsets=None), INVALID), (dict(n_c=0), INVALID), (dict(K=P + 8), ALIGNMENT), (dict(offsets=P + 4), ALIGNMENT)])
def test_c_compact_refuses(lib, kw, code):
    a = dict(K=P, V=P, B=1, n_c=50, d=64, idx=P, counts=P, offsets=P, **PAGES, st=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.kvz_compact_int4(*a.values()) == code


@pytest.mark.parametrize("kw,code", BAD_PAGES + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(counts=None), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(T=0), INVALID), (dict(T=1 << 31), INVALID), (dict(G=0), INVALID),
    (dict(T=1 << 20, B=60000), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID),
    (dict(rot=8), UNSUPPORTED), (dict(il=3), INVALID), (dict(k_st=12), ALIGNMENT), (dict(v_sb=-8), ALIGNMENT),
    (dict(q_sg=1), ALIGNMENT), (dict(k=P + 4), ALIGNMENT), (dict(q_out=P + 8), ALIGNMENT), (dict(n_new=P + 1), ALIGNMENT),
    (dict(counts_out=P), INVALID), (dict(n_new=2 * P), INVALID), (dict(pos=2 * P), INVALID)])
def test_c_append_refuses(lib, kw, code):
    a = dict(k=P, k_sb=64, k_st=64, v=P, v_sb=64, v_st=64, q=P, q_sb=64, q_sg=64, q_st=64, q_out=2 * P, B=1, G=2, T=3,
             d=64, pos=P, pos_sb=0, table=P, n_pos=9, rot=64, il=0, **PAGES, counts=P, n_new=None, counts_out=2 * P,
             st=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.kvz_append_int4(*a.values()) == code


@pytest.mark.parametrize("kw,code", BAD_PAGES + [
    (dict(counts=None), INVALID), (dict(offsets=None), INVALID), (dict(K_out=None), INVALID),
    (dict(V_out=P), INVALID), (dict(n_rows=-1), INVALID), (dict(K_out=P + 8), ALIGNMENT), (dict(first=P + 2), ALIGNMENT)])
def test_c_expand_refuses(lib, kw, code):
    a = dict(**PAGES, counts=P, first=None, offsets=P, B=1, d=64, K_out=P, V_out=2 * P, n_rows=8, st=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.kvz_expand_int4(*a.values()) == code


@pytest.mark.parametrize("kw,code", BAD_PAGES + [
    (dict(q=None), INVALID), (dict(counts=None), INVALID), (dict(out=None), INVALID), (dict(G=0), UNSUPPORTED),
    (dict(G=9), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(q=P + 8), ALIGNMENT),
    (dict(out=P + 4), ALIGNMENT), (dict(lse2=P + 1), ALIGNMENT), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(ws=P + 16), ALIGNMENT), (dict(n_pages=0x7FFFFFFF), INVALID)])
def test_c_decode_refuses(lib, kw, code):
    a = dict(q=P, **{**PAGES, "max_pages": 5000}, counts=P, B=1, G=2, d=64, scale=0.125, out=P, lse2=P, ws=P,
             ws_bytes=1 << 24, st=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.kvz_decode_int4(*a.values()) == code


def test_sizes(lib):
    assert lib.kvz_cache4_page_bytes(64, 128) == 64 * 144 and lib.kvz_cache4_page_bytes(16, 64) == 16 * 72
    for bad in ((0, 128), (24, 128), (2048, 64), (64, 96)):
        assert lib.kvz_cache4_page_bytes(*bad) == 0
    size = lib.kvz_decode_int4_workspace_size
    assert size(0, 4, 1 << 20, 128) == 0 and size(4, 9, 1 << 20, 64) == 0 and size(4, 4, 1 << 20, 96) == 0
    assert size(64, 8, 1 << 20, 128) > 2 * 296 * 8 * 128 * 4
    assert size(8, 4, 100, 128) == 0                  # short heads need no scratch


def test_page_division_is_exact():
    # the host's reciprocal, as the device applies it, over block numbers around every multiple that a table can reach
    for blocks in range(2, 65):
        inv = (1 << 32) // blocks + 1
        top = (1 << 26) - 1
        q = np.unique(np.concatenate([np.arange(0, 2000), np.linspace(0, top // blocks, 5000).astype(np.int64)]))
        n = (q[:, None] * blocks + np.arange(-1, 2)).reshape(-1)
        n = n[(n >= 0) & (n <= top)]
        assert np.array_equal((n.astype(object) * inv >> 32).astype(np.int64), n // blocks)


def test_rotary_freqs():
    f, a = kvz.kvz_rotary_freqs(64, 10000.0)
    ref = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert a == 1.0 and np.allclose(f.numpy(), ref, rtol=1e-14)
    f2, _ = kvz.kvz_rotary_freqs(64, scaling={"type": "linear", "factor": 4})
    assert np.allclose(f2.numpy(), ref / 4, rtol=1e-14)
    f3, _ = kvz.kvz_rotary_freqs(64, scaling={"type": "ntk", "factor": 4})
    assert f3[0] == 1.0 and np.isclose(f3[-1].item(), ref[-1] / 4, rtol=1e-12)
    f4, a4 = kvz.kvz_rotary_freqs(64, scaling={"type": "yarn", "factor": 4, "original": 4096})
    turns = 4096 * ref / (2 * np.pi)
    r = f4.numpy() / ref
    assert np.allclose(r[turns > 40], 1.0) and np.allclose(r[turns < 0.8], 0.25) and np.all(np.diff(r) <= 1e-12)
    assert np.isclose(a4, 0.1 * np.log(4) + 1)


def test_kernels_that_start_early_read_by_ordinary_loads():
    # they are resident while their inputs are still written, which rules out read-only loads (restrict pointers to
    # const become such)
    csrc = os.path.join(os.path.dirname(kvz.__file__), "csrc")
    text = {p: open(p).read() for p in glob.glob(os.path.join(csrc, "*.cu*"))}
    early = [p for p, s in text.items() if "after_prior(" in s or p.endswith(("kvz_cache4.cuh", "kvz_rotary.cuh"))]
    assert len(early) >= 6
    for p in early:
        assert not re.search(r"__ldg|\.nc\b|__restrict__", re.sub(r"//[^\n]*", "", text[p])), p


# ---------------------------------------------------------------------------
# The host module
# ---------------------------------------------------------------------------
def test_a_host_module_that_cannot_be_compiled_leaves_none_behind(tmp_path, monkeypatch):
    # the module of an earlier build, of an earlier header, must not be imported in its place
    from query_agnostic_kv_kvz_b200 import build
    old = [tmp_path / os.path.basename(build.FAST), tmp_path / "_kvz_fast.so"]
    for p in old:
        p.write_bytes(b"an earlier build")
    stamp = tmp_path / "stamp"
    stamp.write_text("x")
    monkeypatch.setattr(build, "FAST", str(old[0]))
    monkeypatch.setattr(build, "FAST_STAMP", str(stamp))
    monkeypatch.setenv("CXX", "false")
    assert build.build_fast() is False
    assert not any(p.exists() for p in old) and not stamp.exists()


@pytest.mark.parametrize("wrong", ["torch_version", "header_id"])
def test_a_host_module_of_another_build_is_not_bound(monkeypatch, wrong):
    from types import SimpleNamespace

    from query_agnostic_kv_kvz_b200 import build

    def bind(*a):
        raise AssertionError("bound")
    fake = dict(torch_version=torch.__version__, header_id=build.header_id(), bind=bind)
    fake[wrong] = "another"
    kvz.lib()
    monkeypatch.setattr(kvz, "_kvz_fast", SimpleNamespace(**fake), raising=False)
    monkeypatch.setattr(kvz, "_fast", None)
    kvz._load_fast()
    assert kvz._fast is None
    del fake[wrong]                                   # a module of before it said so
    monkeypatch.setattr(kvz, "_kvz_fast", SimpleNamespace(**{"torch_version": torch.__version__, **fake}))
    if wrong == "header_id":
        kvz._load_fast()
        assert kvz._fast is None
