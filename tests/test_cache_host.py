"""CPU checks of the cache operators: every declared symbol is exported, refusals come before any
device call, and the index arithmetic that the kernels use (compiled for the host) stays inside the
cache for slots, lengths, counts and pages that are out of range."""
import ctypes
import os
import re
import subprocess
import tempfile

import numpy as np
import pytest

import quantized_base_linear_amd as q
from quantized_base_linear_amd import cache
from tests import cache_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned address that is never dereferenced: every case fails validation first
LIB = cache._lib


def _kv(**over):
    d = dict(n_layers=2, n_pages=10, page_tokens=64, n_kv_heads=2, head_dim=128, n_slots=4, max_pages=8, reserved=0,
             store=FAKE, refs=FAKE, lens=FAKE, table=FAKE, status=FAKE)
    d.update(over)
    return cache.qbl_kv(*[d[f] for f, _ in cache.qbl_kv._fields_])


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "qbl_cache.h")).read()
    names = set(re.findall(r"\b(qbl_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert len(names) == 13
    out = subprocess.run(["nm", "-D", "--defined-only", q.library_path()], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\bT (qbl_\w+)", out))
    assert names <= set(cache.EXPORTS)


def test_page_bytes():
    assert cache.qbl_kv_page_bytes(64, 8, 128) == 2 * 8 * (32 * 128 + 256 * 4)
    assert cache.qbl_kv_page_bytes(32, 1, 64) == 32 * 64 + 256 * 2
    for bad in ((16, 8, 128), (96, 8, 128), (512, 8, 128), (64, 0, 128), (64, 8, 96), (64, 8, 0), (64, 2000, 64)):
        assert cache.qbl_kv_page_bytes(*bad) == 0


BAD_CACHES = [
    (dict(page_tokens=48), "QBL_E_SHAPE"), (dict(head_dim=96), "QBL_E_SHAPE"), (dict(n_kv_heads=0), "QBL_E_SHAPE"),
    (dict(n_layers=0), "QBL_E_SHAPE"), (dict(n_pages=0), "QBL_E_SHAPE"), (dict(n_slots=-1), "QBL_E_SHAPE"),
    (dict(max_pages=0), "QBL_E_SHAPE"), (dict(max_pages=1 << 20), "QBL_E_LIMIT"), (dict(reserved=1), "QBL_E_ARG"),
    (dict(store=None), "QBL_E_ARG"), (dict(refs=None), "QBL_E_ARG"), (dict(lens=None), "QBL_E_ARG"),
    (dict(table=None), "QBL_E_ARG"), (dict(status=None), "QBL_E_ARG"), (dict(store=FAKE + 8), "QBL_E_ARG"),
    (dict(lens=FAKE + 2), "QBL_E_ARG"), (dict(n_pages=1 << 27), "QBL_E_LIMIT"),
]


@pytest.mark.parametrize("over,name", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(over, name):
    kv = _kv(**over)
    p, s = ctypes.addressof(kv), ctypes.addressof(_strides(256, 256, 128))
    big = 1 << 40
    calls = [
        LIB.qbl_kv_extend(p, None, FAKE, 1, FAKE, big, None),
        LIB.qbl_kv_fork(p, FAKE, FAKE, None, 1, None),
        LIB.qbl_kv_truncate(p, None, FAKE, 1, None),
        LIB.qbl_kv_compact(p, FAKE, big, None),
        LIB.qbl_kv_copy(p, FAKE, FAKE, 1, None),
        LIB.qbl_kv_append(p, 0, None, None, 1, 1, FAKE, s, FAKE, s, 0, None),
        LIB.qbl_kv_read(p, 0, None, None, 1, 1, FAKE, FAKE, None),
        LIB.qbl_kv_attend(p, 0, None, None, 1, 1, 2, FAKE, s, FAKE + 4096, s, 0, 64, 0, 0, 0.0, FAKE, big, None),
    ]
    assert calls == [q.CODE[name]] * len(calls)
    assert q.qbl_last_error()


def test_page_call_refusals():
    kv = _kv()
    p = ctypes.addressof(kv)
    need = ctypes.c_int64(-7)
    assert LIB.qbl_kv_pages_ws_bytes(p, 4, ctypes.addressof(need)) == 0 and need.value > 0
    E = q.CODE
    assert LIB.qbl_kv_pages_ws_bytes(p, 4, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_pages_ws_bytes(p, 1025, ctypes.addressof(need)) == E["QBL_E_LIMIT"]
    assert LIB.qbl_kv_extend(p, None, None, 4, FAKE, need.value, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_extend(p, None, FAKE, 0, FAKE, need.value, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_extend(p, None, FAKE, 1025, FAKE, 1 << 40, None) == E["QBL_E_LIMIT"]
    assert LIB.qbl_kv_extend(p, None, FAKE, 4, None, need.value, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_extend(p, None, FAKE, 4, FAKE + 4, need.value, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_extend(p, None, FAKE, 4, FAKE, need.value - 1, None) == E["QBL_E_BUDGET"]
    assert LIB.qbl_kv_fork(p, None, FAKE, None, 1, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_fork(p, FAKE, None, None, 1, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_truncate(p, FAKE, None, 1, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_truncate(p, FAKE, FAKE, 2000, None) == E["QBL_E_LIMIT"]
    assert LIB.qbl_kv_compact(p, FAKE, 16, None) == E["QBL_E_BUDGET"]
    assert LIB.qbl_kv_copy(p, FAKE, FAKE, 0, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_copy(p, FAKE, None, 1, None) == E["QBL_E_ARG"]


def test_append_read_attend_refusals():
    kv = _kv()
    p, E = ctypes.addressof(kv), q.CODE
    good = _strides(256, 256, 128)
    s = ctypes.addressof(good)
    neg = _strides(256, -1, 128)
    big = 1 << 40
    app = lambda layer=0, slots=None, n=1, ql=1, k=FAKE, ks=s, v=FAKE, vs=s, dt=0: LIB.qbl_kv_append(
        p, layer, slots, None, n, ql, k, ks, v, vs, dt, None)
    assert app(layer=2) == app(layer=-1) == app(n=0) == app(ql=0) == app(n=5) == E["QBL_E_ARG"]
    assert app(k=None) == app(v=None) == app(ks=None) == app(k=FAKE + 2) == E["QBL_E_ARG"]
    assert app(dt=3) == E["QBL_E_FORMAT"] and app(vs=ctypes.addressof(neg)) == E["QBL_E_SHAPE"]
    assert app(n=70000, slots=FAKE) == app(ql=1 << 21) == E["QBL_E_LIMIT"]
    assert LIB.qbl_kv_read(p, 0, None, None, 1, 1, FAKE, None, None) == E["QBL_E_ARG"]
    assert LIB.qbl_kv_read(p, 0, None, None, 1, 1, FAKE + 4, FAKE, None) == E["QBL_E_ARG"]
    o = FAKE + 65536
    att = lambda heads=4, x=FAKE, xs=s, out=o, os=s, dt=0, ml=64, win=0, snk=0, sc=0.0, ws=FAKE, wb=big, n=1, ql=1: \
        LIB.qbl_kv_attend(p, 0, None, None, n, ql, heads, x, xs, out, os, dt, ml, win, snk, sc, ws, wb, None)
    assert att(heads=3) == att(heads=0) == E["QBL_E_SHAPE"]
    assert att(x=None) == att(out=None) == att(out=FAKE) == att(ml=0) == att(ml=1 << 25) == E["QBL_E_ARG"]
    assert att(win=-1) == att(snk=-1) == E["QBL_E_ARG"]
    assert att(sc=float("nan")) == att(sc=float("inf")) == E["QBL_E_NONFINITE"]
    assert att(dt=9) == E["QBL_E_FORMAT"]
    need = ctypes.c_int64()
    assert LIB.qbl_kv_attend_ws_bytes(p, 1, 1, 4, 0, 512, 0, 0, ctypes.addressof(need)) == 0 and need.value > 0
    assert att(ml=512, ws=None) == E["QBL_E_ARG"] and att(ml=512, wb=need.value - 1) == E["QBL_E_BUDGET"]
    assert att(ql=1 << 20, heads=1 << 16) == E["QBL_E_LIMIT"]


def test_verify_refusals():
    E = q.CODE
    s2 = (ctypes.c_int64 * 2)(300, 100)
    s = ctypes.addressof(s2)
    call = lambda t=FAKE, ts=s, d=FAKE, ds=s, dt=0, tok=FAKE, u=FAKE, n=2, ql=2, vocab=100, acc=FAKE, nxt=FAKE, ws=FAKE, \
        wb=1 << 30: LIB.qbl_verify(t, ts, d, ds, dt, tok, None, u, n, ql, vocab, acc, nxt, ws, wb, None)
    assert call(t=None) == call(ts=None) == call(ds=None) == call(tok=None) == call(u=None) == E["QBL_E_ARG"]
    assert call(acc=None) == call(nxt=None) == call(n=0) == call(ql=-1) == call(vocab=0) == call(ws=None) == E["QBL_E_ARG"]
    assert call(dt=5) == E["QBL_E_FORMAT"] and call(ql=257) == call(n=70000) == call(vocab=1 << 29) == E["QBL_E_LIMIT"]
    assert call(wb=16) == E["QBL_E_BUDGET"] and call(t=FAKE + 2) == E["QBL_E_ARG"]


# ------------------------------------------------------------ index arithmetic, on the host ----

HARNESS = r"""
#include "qbl_cache_index.h"
using namespace qbl;
extern "C" void entry(const qbl_kv* kv, const int32_t* slots, const int32_t* counts, int n, int q_len, int i, int* out) {
  const Entry e = load_entry(*kv, KvRows{slots, counts, n, q_len}, i);
  out[0] = e.slot, out[1] = e.len, out[2] = e.c;
}
extern "C" int page(const qbl_kv* kv, int slot, int pos, int sh) { return page_of(*kv, slot, pos, sh); }
extern "C" int64_t tile(const qbl_kv* kv, int layer, int p, int h, int pos, int sh) {
  return tile_offset(*kv, layer, p, h, pos, sh, kv->head_dim);
}
extern "C" void span(int slot, int len, int c, int r0, int cols, int group, int max_len, int window, int sinks, int* out) {
  const Span s = row_span(Entry{slot, len, c}, r0, cols, group, max_len, window, sinks);
  out[0] = s.first, out[1] = s.last, out[2] = s.lo, out[3] = s.end, out[4] = s.sink, out[5] = s.tiles;
  for (int v = 0; v < s.tiles && v < 64; ++v) out[6 + v] = span_pos(s, v);
}
"""


@pytest.fixture(scope="module")
def index():
    d = tempfile.mkdtemp(prefix="qbl_index_")
    src, so = os.path.join(d, "h.cpp"), os.path.join(d, "h.so")
    open(src, "w").write(HARNESS)
    csrc = os.path.join(ROOT, "quantized_base_linear_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", csrc, src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.tile.restype = ctypes.c_int64
    return lib


def _host_kv(lens, table, n_pages=10, page_tokens=32, layers=2, heads=3, dim=64):
    lens, table = np.array(lens, np.int32), np.array(table, np.int32)
    kv = cache.qbl_kv(layers, n_pages, page_tokens, heads, dim, len(lens), table.shape[1], 0, FAKE, FAKE,
                      lens.ctypes.data, table.ctypes.data, FAKE)
    return kv, (lens, table)


def test_entries_and_pages_out_of_range(index):
    kv, keep = _host_kv([5, -3, 1 << 30, 64], [[0, 1], [-1, 10], [1 << 30, -(1 << 31)], [9, 2]])
    out = (ctypes.c_int * 3)()
    p = ctypes.byref(kv)
    for slot, count, want in ((0, 1, (0, 5, 1)), (0, -4, (0, 5, 0)), (0, 99, (0, 5, 7)), (1, 1, (1, 0, 1)),
                              (2, 7, (2, 64, 7)), (4, 1, (-1, 0, 0)), (-1, 1, (-1, 0, 0)), (1 << 30, 1, (-1, 0, 0))):
        s, c = (ctypes.c_int32 * 1)(slot), (ctypes.c_int32 * 1)(count)
        index.entry(p, s, c, 1, 7, 0, out)
        assert tuple(out) == want, (slot, count)
    assert [index.page(p, s, pos, 5) for s, pos in ((0, 0), (0, 63), (1, 0), (1, 32), (2, 0), (2, 63), (3, 31))] == \
        [0, 1, -1, -1, -1, -1, 9]


@pytest.mark.parametrize("page_tokens,heads,dim", [(32, 3, 64), (64, 1, 128), (256, 2, 256)])
def test_tiles_are_disjoint_and_inside_the_store(index, page_tokens, heads, dim):
    kv, keep = _host_kv([0], [[0]], 5, page_tokens, 2, heads, dim)
    page = cache.qbl_kv_page_bytes(page_tokens, heads, dim)
    sh = page_tokens.bit_length() - 1
    seen = sorted(index.tile(ctypes.byref(kv), layer, p, h, pos, sh) for layer in range(2) for p in range(5)
                  for h in range(heads) for pos in range(0, page_tokens, 32))
    assert seen == list(range(0, 2 * 5 * page, 40 * dim))


def test_offsets_pass_32_bits(index):
    kv, keep = _host_kv([0], [[0]], 1 << 20, 256, 4, 64, 256)
    page = cache.qbl_kv_page_bytes(256, 64, 256)
    assert index.tile(ctypes.byref(kv), 3, (1 << 20) - 1, 63, 255, 8) == 4 * (1 << 20) * page - 40 * 256


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 1), (40, 4), (100, 33), (7, 1 << 24), (1 << 23, 2)])
def test_spans_hold_exactly_the_visible_tiles(index, window, sinks):
    rng = np.random.default_rng(window + sinks)
    out = (ctypes.c_int * 80)()
    for _ in range(300):
        n = int(rng.integers(0, 400))
        c = int(rng.integers(0, 40))
        group, cols = int(rng.integers(1, 9)), int(rng.choice([16, 32, 64]))
        max_len = int(rng.choice([n, max(1, n // 2), n + 50])) or 1
        r0 = cols * int(rng.integers(0, 4))
        index.span(0, n, c, r0, cols, group, max_len, window, sinks, out)
        first, last, lo, end, sink, tiles = out[:6]
        got = [out[6 + v] for v in range(tiles)]
        valid = sorted({n - c + r // group for r in range(r0, min(r0 + cols, c * group))
                        if 0 <= n - c + r // group < min(n, max_len)})
        if not valid:
            assert tiles == 0 and last < first
            continue
        assert (first, last) == (valid[0], valid[-1])
        want = {t // 32 * 32 for i in valid for t in range(i + 1) if not window or i - t < window or t < sinks}
        assert len(set(got)) == len(got) and set(got) >= want
        assert all(0 <= t <= last for t in got)


# ------------------------------------------------------------------- the reference itself ----

def test_reference_quantiser_is_the_librarys():
    rng = np.random.default_rng(3)
    w = (rng.standard_normal((64, 256)) * 3).astype(np.float32)
    w[0, :32], w[1, :32], w[2, :32] = 0.0, 0.125, np.arange(32) - 16
    code, d, m = ref.quantise(w)
    blocks = q.qbl_quantize(q.QBL_Q4_SM, w).reshape(64, 8, 20)
    assert np.array_equal(blocks[..., :2].copy().view(np.float16), d[..., 0][..., None])
    assert np.array_equal(blocks[..., 2:4].copy().view(np.float16), m[..., 0][..., None])
    assert np.array_equal(blocks[..., 4:] & 15, code[..., 0::2]) and np.array_equal(blocks[..., 4:] >> 4, code[..., 1::2])


def test_reference_attention_closed_forms():
    v = np.random.default_rng(0).standard_normal((9, 1, 64))
    out, _, _ = ref.attend(np.zeros((2, 1, 64)), np.ones((9, 1, 64)), v, 7)
    assert np.allclose(out[0, 0], v[:8, 0].mean(0)) and np.allclose(out[1, 0], v[:, 0].mean(0))
    out, _, _ = ref.attend(np.zeros((1, 1, 64)), np.ones((9, 1, 64)), v, 8, window=2, sinks=1)
    assert np.allclose(out[0, 0], v[[0, 7, 8], 0].mean(0))
    out, _, _ = ref.attend(np.zeros((1, 1, 64)), np.ones((9, 1, 64)), v, 8, hidden=np.ones(9, bool))
    assert np.array_equal(out, np.zeros_like(out))


def test_reference_verification_keeps_the_targets_distribution():
    """Accepting a token of q with min(1, p/q), else drawing from max(p - q, 0), draws from p: the
    probability of each token, summed over drafts exactly and over the draw's intervals, is p."""
    p, d = np.array([0.5, 0.3, 0.2, 0.0]), np.array([0.2, 0.2, 0.1, 0.5])
    grid = (np.arange(2000) + 0.5) / 2000
    got = np.zeros(4)
    for x in range(4):
        for ua in grid[::40]:
            a, t = ref.verify(np.repeat(np.stack([p, [1, 0, 0, 0]])[None], 50, 0), np.repeat(d[None, None], 50, 0),
                              np.full((50, 1), x), np.ones(50), np.stack([np.full(50, ua), grid[::40]], 1), 1)
            tok = np.where(a == 1, x, t)
            np.add.at(got, tok, d[x] / 2500)
    assert np.abs(got - p).max() < 0.02  # intervals of 1/50 in each of the two numbers


def test_reference_pages_share_and_copy():
    c = ref.Pages(6, 32, 3, 4)
    assert c.extend([0], [40])
    c.fork([0], [1])
    assert c.refs == [2, 2, 0, 0, 0, 0] and c.table[1] == [0, 1]
    assert c.extend([0, 1], [1, 1]) and c.copies == [(1, 2)] and c.table[:2] == [[0, 2], [0, 1]]
    c.truncate([0], [0])
    assert c.refs == [1, 1, 0, 0, 0, 0]
    assert not c.extend([2], [32 * 4 + 1]) and c.lens == [0, 41, 0]
