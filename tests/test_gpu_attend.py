"""GPU tests of attention over the 4-bit cache against a 64-bit implementation on the dequantised
values, by element.

Tolerances, before any run: with A = sum p |v| of the output element, S = the largest scale*sum |q k|
over the row's visible keys and N visible keys, and u a relative rounding,
  - the output's own rounding: half a step of its type, eps/2 * |out|;
  - float32 operands: products and sums of D channels and N weights in float32, u = 2^-24 each, at most
    (D + 64) roundings in a score (an error of (D + 64) u S in the exponent, twice: numerator and
    denominator) and N + 64 in a sum: A * u * (2 (D + 64) S + 2 (N + 64));
  - f16 and bf16 outputs may have keys, queries, values and weights rounded to f16 (2^-11 each): the
    exponent is off by at most 2 * 2^-11 S, twice, and the products by 2 * 2^-11, the weights' sum by
    2^-11: A * 2^-11 * (4 S + 3) on top."""
import numpy as np
import pytest

import quantized_base_linear_amd as q
from quantized_base_linear_amd import cache
from tests import cache_reference as ref
from tests.test_gpu_cache import TYPES, dev, fill, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def close(got, want, spread, logit, n, dim, dtype, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    u = 2.0 ** -24
    tol = EPS[dtype] * np.abs(want) + spread * u * (2 * (dim + 64) * logit + 2 * (n + 64))
    if dtype != "f32":
        tol = tol + spread * 2.0 ** -11 * (4 * logit + 3)
    bad = np.abs(got - want) > tol + 1e-30
    assert not bad.any(), (what, np.abs(got - want)[bad].max(), int(bad.sum()))


def build(dim, page, kv_heads, lens, seed, slots=None, layers=1, layer=0):
    """A cache with random contents for the given lengths; returns it and the float64 keys and values."""
    rng = np.random.default_rng(seed)
    slots = list(range(len(lens))) if slots is None else slots
    need = sum(-(-n // page) for n in lens)
    kv, _ = make(need + 2, page, kv_heads, dim, max(slots) + 1, max(1, max(-(-n // page) for n in lens)), layers, seed)
    fill(kv, slots, lens, None, seed)
    top = max(max(lens), 1)
    k = rng.standard_normal((len(lens), top, kv_heads, dim)).astype(np.float32)
    k[..., ::17] += 2.0
    v = rng.standard_normal(k.shape).astype(np.float32) + 0.25
    cache.qbl_kv_append(kv, layer, dev(slots), dev(lens), torch.tensor(k).cuda(), torch.tensor(v).cuda())
    return kv, ref.values(*ref.quantise(k)), ref.values(*ref.quantise(v))


def run(kv, qt, counts, max_len, slots=None, layer=0, window=0, sinks=0, scale=0.0, out=None):
    n, q_len, heads, dim = qt.shape
    ws = cache.attend_workspace(kv, n, q_len, heads, max_len, window, sinks, qt.dtype)
    if out is None:
        out = torch.full(qt.shape, float("nan"), dtype=qt.dtype, device="cuda")
    cache.qbl_kv_attend(kv, layer, None if slots is None else dev(slots), None if counts is None else dev(counts), qt,
                        out, max_len, window=window, sinks=sinks, scale=scale, ws=ws)
    torch.cuda.synchronize()
    return out


def compare(kv, k, v, qt, counts, lens, out, dtype, window=0, sinks=0, scale=0.0, hidden=None, what=""):
    x = qt.double().cpu().numpy()
    for i, (n, c) in enumerate(zip(lens, counts)):
        start = max(0, c - n)  # rows before the cache begins are padding
        want, spread, logit = ref.attend(x[i, start:c], k[i, :n], v[i, :n], n - c + start, window, sinks, scale,
                                         None if hidden is None else hidden[i][:n])
        close(out[i, start:c], want, spread, logit, n, x.shape[-1], dtype, f"{what} entry {i}")
        rest = torch.cat([out[i, :start], out[i, c:]]).float()
        assert torch.equal(rest, torch.zeros_like(rest)), f"{what} entry {i}: padding"


CASES = [  # dim, page, kv heads, group, q_len, lens, counts
    (128, 64, 2, 4, 1, [1, 31, 32, 33, 64, 65, 700], [1] * 7),
    (64, 32, 1, 1, 1, [5, 32, 200], [1, 1, 1]),
    (256, 128, 2, 3, 1, [129, 400], [1, 1]),
    (128, 256, 1, 16, 2, [2, 257, 300], [2, 1, 2]),
    (64, 64, 3, 5, 7, [7, 9, 128, 333], [7, 2, 7, 5]),
    (128, 32, 2, 7, 5, [5, 40, 100], [5, 5, 3]),
    (256, 32, 1, 8, 4, [4, 90], [4, 4]),
    (128, 64, 2, 4, 100, [100, 230, 64], [100, 70, 1]),
    (64, 128, 1, 2, 150, [150, 513], [150, 149]),
    (256, 64, 1, 2, 70, [70, 200], [70, 33]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"d{c[0]}p{c[1]}h{c[2]}g{c[3]}q{c[4]}")
def test_attention_matches_the_formula(case, dtype):
    dim, page, kvh, group, q_len, lens, counts = case
    kv, k, v = build(dim, page, kvh, lens, seed=dim + q_len)
    qt = torch.randn((len(lens), q_len, kvh * group, dim), device="cuda",
                     generator=torch.Generator(device="cuda").manual_seed(2)).to(TYPES[dtype])
    out = run(kv, qt, counts, max(lens))
    compare(kv, k, v, qt, counts, lens, out, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (31, 0), (32, 32), (33, 5), (100, 40), (500, 3), (40, 1 << 30)])
@pytest.mark.parametrize("q_len,group", [(1, 4), (6, 3), (90, 2)])
def test_window_and_sinks(window, sinks, q_len, group, dtype):
    lens = [q_len, 64 + q_len, 401]
    counts = [q_len, q_len, max(1, q_len - 1)]
    kv, k, v = build(128, 32, 2, lens, seed=window)
    qt = torch.randn((3, q_len, 2 * group, 128), device="cuda",
                     generator=torch.Generator(device="cuda").manual_seed(3)).to(TYPES[dtype])
    out = run(kv, qt, counts, 401, window=window, sinks=sinks)
    compare(kv, k, v, qt, counts, lens, out, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len", [1, 3, 80])
def test_rows_that_see_nothing_are_zero(q_len, dtype):
    """Empty slots, no new tokens, slots out of range, more new tokens than held, no pages at all."""
    lens = [0, 50, 2, 40]
    kv, k, v = build(128, 32, 1, lens, seed=4)
    kv.table[3] = torch.tensor([kv.n_pages, -5], dtype=torch.int32)
    qt = torch.randn((5, q_len, 2, 128), device="cuda").to(TYPES[dtype])
    out = run(kv, qt, [1, 0, q_len, q_len, 1], 50, slots=[0, 1, 2, 3, 99])
    for i in (0, 1, 3, 4):
        assert torch.equal(out[i].float(), torch.zeros_like(out[i].float())), i
    compare(kv, k[2:3], v[2:3], qt[2:3], [q_len], [2], out[2:3], dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("q_len", [1, 70])
def test_missing_pages_hide_their_tokens(q_len, dtype):
    lens = [200, 300]
    kv, k, v = build(64, 32, 2, lens, seed=5)
    table = kv.table.clone()
    hidden = [np.zeros(n, bool) for n in lens]
    for i, p, bad in ((0, 0, -1), (0, 3, 1 << 30), (1, 8, kv.n_pages), (1, 2, -(1 << 31))):
        table[i, p] = bad
        hidden[i][p * 32:(p + 1) * 32] = True
    kv.table.copy_(table)
    qt = torch.randn((2, q_len, 4, 64), device="cuda").to(TYPES[dtype])
    out = run(kv, qt, [q_len] * 2, 300)
    compare(kv, k, v, qt, [q_len] * 2, lens, out, dtype, hidden=hidden)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_len,window,sinks", [(1, 0, 0), (1, 37, 2), (5, 37, 2), (66, 0, 0), (66, 37, 2)])
def test_hidden_places_may_hold_anything(dim, q_len, window, sinks, dtype):
    """Every byte of the store outside the visible tokens is 0xFF: scales there are NaN."""
    lens = [q_len + 1, 170]
    kv, k, v = build(dim, 64, 1, lens, seed=6)
    qt = torch.randn((2, q_len, 2, dim), device="cuda").to(TYPES[dtype])
    counts = [q_len, q_len]
    tiles = kv.store.view(kv.n_pages, 2, 40 * dim)
    from tests.test_gpu_cache import tile_mask
    keep = torch.zeros_like(tiles)
    for i, n in enumerate(lens):
        first = n - q_len
        seen = [t for t in range(n) if not window or t < sinks or t > first - window]
        for t0 in range(0, n, 32):
            m = tile_mask([t - t0 for t in seen if t0 <= t < t0 + 32], dim)
            keep[int(kv.table[i, t0 // 64]), t0 % 64 // 32] = torch.tensor(m).cuda()
    tiles.copy_((tiles & keep) | ~keep)
    out = run(kv, qt, counts, 170, window=window, sinks=sinks)
    compare(kv, k, v, qt, counts, lens, out, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strides_alignments_layers_slots_and_scale(dtype):
    lens, counts, slots = [77, 130], [3, 2], [5, 1]
    kv, k, v = build(128, 64, 2, lens, seed=7, slots=slots, layers=3, layer=2)
    buf = torch.randn((2, 3, 10, 128 + 3), device="cuda").to(TYPES[dtype])
    qt = buf[:, :, 1:9, 1:129]                       # odd strides, not 16-byte aligned
    obuf = torch.full((2, 8, 3, 200), 7.0, device="cuda").to(TYPES[dtype])
    out = obuf[..., 5:133].permute(0, 2, 1, 3)       # heads outside tokens
    run(kv, qt, counts, 130, slots=slots, layer=2, scale=0.3, out=out)
    compare(kv, k, v, qt, counts, lens, out, dtype, scale=0.3)
    rest = obuf.clone()
    rest[..., 5:133] = 7.0
    assert torch.equal(rest, torch.full_like(rest, 7.0))


@pytest.mark.parametrize("q_len", [1, 40])
def test_max_len_bounds_what_is_read(q_len):
    lens = [500, 90]
    kv, k, v = build(64, 32, 1, lens, seed=8)
    qt = torch.randn((2, q_len, 4, 64), device="cuda")
    out = run(kv, qt, None, 100)
    compare(kv, k[1:], v[1:], qt[1:], [q_len], [90], out[1:], "f32")
    assert torch.equal(out[0], torch.zeros_like(out[0]))  # its queries sit past max_len


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q_len,window", [(1, 0), (4, 0), (1, 1500), (300, 0)])
def test_long_caches_are_split_and_joined(q_len, window, dtype):
    lens = [9000, 4097]
    kv, k, v = build(128, 256, 2, lens, seed=9)
    qt = (torch.randn((2, q_len, 8, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) *
          2).to(TYPES[dtype])
    out = run(kv, qt, [q_len] * 2, 9000, window=window, sinks=4)
    pick = [0, 4, 7]  # a few heads: the 64-bit side is slow
    x = qt[:, :, pick].double().cpu().numpy()
    for i, n in enumerate(lens):
        for z, h in enumerate(pick):
            want, spread, logit = ref.attend(x[i, :, z:z + 1], k[i, :n, h // 4:h // 4 + 1], v[i, :n, h // 4:h // 4 + 1],
                                             n - q_len, window, 4 if window else 0)
            close(out[i, :, h:h + 1], want, spread, logit, n, 128, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q_len", [1, 50])
def test_large_scores_and_rising_maxima(q_len, dtype):
    """Scores of +-200 that rise along the cache, so the running maximum moves again and again."""
    n = 300
    kv, _, _ = build(64, 64, 1, [n], seed=10)
    k = np.zeros((1, n, 1, 64), np.float32)
    k[0, :, 0, :32] = np.linspace(-25, 25, n)[:, None].astype(np.float32)
    v = np.random.default_rng(1).standard_normal(k.shape).astype(np.float32)
    cache.qbl_kv_append(kv, 0, None, None, torch.tensor(k).cuda(), torch.tensor(v).cuda())
    k, v = ref.values(*ref.quantise(k)), ref.values(*ref.quantise(v))
    qt = torch.full((1, q_len, 2, 64), 2.0, device="cuda").to(TYPES[dtype])
    qt[:, :, 1] = -2.0
    out = run(kv, qt, None, n)
    compare(kv, k, v, qt, [q_len], [n], out, dtype)


def test_replays_of_a_captured_step_equal_eager_runs():
    """extend, append, attend, truncate in one graph, replayed with eager work in between."""
    kv, _ = make(40, 32, 2, 128, 4, 8, seed=11)
    eager, _ = make(40, 32, 2, 128, 4, 8, seed=11)
    ws, we = cache.pages_workspace(kv, 4), cache.pages_workspace(eager, 4)
    counts = dev([1, 2, 0, 2])
    qt, kt, vt = (torch.randn((4, 2, h, 128), device="cuda") for h in (4, 2, 2))
    wa = cache.attend_workspace(kv, 4, 2, 4, 256)
    out, oute = torch.zeros_like(qt), torch.zeros_like(qt)
    cut = dev([0, 0, 0, 0])

    def step(c, w, o, cut):
        cache.qbl_kv_extend(c, None, counts, w)
        cache.qbl_kv_append(c, 0, None, counts, kt, vt)
        cache.qbl_kv_attend(c, 0, None, counts, qt, o, 256, ws=wa)
        cache.qbl_kv_truncate(c, None, cut)

    cut_e = dev([0, 0, 0, 0])
    for t in (cut, cut_e):
        t.fill_(1 << 20)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kv, ws, out, cut)
    for r in range(6):
        for x in (qt, kt, vt):
            x.normal_(generator=torch.Generator(device="cuda").manual_seed(r))
        limit = 3 if r == 3 else 1 << 20
        cut.fill_(limit), cut_e.fill_(limit)
        graph.replay()
        torch.cuda.synchronize()
        step(eager, we, oute, cut_e)
        torch.cuda.synchronize()
        assert torch.equal(out, oute) and out.abs().sum() > 0
        for a, b in ((kv.refs, eager.refs), (kv.lens, eager.lens), (kv.table, eager.table), (kv.store, eager.store)):
            assert torch.equal(a, b)
        kv.check()


def test_runs_on_another_stream_and_is_deterministic():
    lens = [1000, 333, 64]
    kv, k, v = build(128, 64, 4, lens, seed=12)
    qt = torch.randn((3, 1, 16, 128), device="cuda")
    first = run(kv, qt, None, 1000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run(kv, qt, None, 1000)
    torch.cuda.synchronize()
    assert torch.equal(first, again)


def test_python_refusals():
    kv, _, _ = build(64, 32, 2, [10], seed=13)
    x = torch.zeros((1, 1, 4, 64), device="cuda")
    for bad in (x[..., :32], x.half(), x.cpu(), x.permute(0, 1, 3, 2).contiguous().permute(0, 1, 3, 2)):
        with pytest.raises(ValueError):
            cache.qbl_kv_attend(kv, 0, None, None, bad, x.clone(), 10)
    with pytest.raises(ValueError):
        cache.qbl_kv_attend(kv, 0, dev([0, 0]), None, x, x.clone(), 10)
    with pytest.raises(q.QblError):
        cache.qbl_kv_attend(kv, 1, None, None, x, x.clone(), 10)
