"""GPU tests of attention at the borders between its kernels (16, 32 and 128 query rows per workgroup)
and for queries far from 1.  Reference and tolerances are those of the other attention tests, derived
there; queries that are scaled by a power of two, with the scale taken back in `scale`, have to give the
same bits, as every kernel works on rows scaled by powers of two."""
import numpy as np
import pytest

from tests import cache_reference as ref
from tests.test_gpu_attend import build, compare, run
from tests.test_gpu_cache import TYPES, dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def queries(shape, dtype, seed, factor=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * factor).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,group,q_len", [(128, 1, 16), (128, 1, 17), (64, 4, 8), (64, 3, 11), (128, 2, 63), (128, 2, 65),
                                             (64, 1, 128), (64, 1, 129), (256, 1, 33), (256, 5, 27), (128, 7, 40)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_row_counts_at_the_kernels_borders(dim, group, q_len, window, sinks, dtype):
    lens = [q_len, q_len + 31, 333]
    counts = [q_len, max(1, q_len - 9), q_len]
    kv, k, v = build(dim, 64, 2, lens, seed=dim + q_len)
    qt = queries((3, q_len, 2 * group, dim), dtype, q_len)
    out = run(kv, qt, counts, 333, window=window, sinks=sinks)
    compare(kv, k, v, qt, counts, lens, out, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_rows_over_a_long_cache_are_split(dim, dtype):
    lens = [2500, 1300]
    kv, k, v = build(dim, 128, 1, lens, seed=21)
    qt = queries((2, 40, 2, dim), dtype, 21)
    out = run(kv, qt, [40, 37], 2500)
    compare(kv, k, v, qt, [40, 37], lens, out, dtype)
    again = run(kv, qt, [40, 37], 2500)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len", [1, 24, 70])
@pytest.mark.parametrize("power", [-90, -30, 30, 90])
def test_queries_scaled_by_powers_of_two_give_the_same(q_len, power, dtype):
    lens = [200, 77]
    kv, _, _ = build(128, 32, 2, lens, seed=22)
    qt = queries((2, q_len, 4, 128), dtype, 22)
    scale = 2.0 ** -4
    want = run(kv, qt, None, 200, scale=scale)
    got = run(kv, qt * 2.0 ** power, None, 200, scale=scale * 2.0 ** -power)
    assert torch.equal(want, got)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q_len", [1, 24, 70])
def test_a_negative_scale_and_zero_queries(q_len, dtype):
    lens = [200, 77]
    kv, k, v = build(128, 32, 2, lens, seed=23)
    qt = queries((2, q_len, 4, 128), dtype, 23)
    qt[:, :, 1] = 0
    out = run(kv, qt, None, 200, scale=-0.125)
    compare(kv, k, v, qt, [q_len] * 2, lens, out, dtype, scale=-0.125)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q_len", [2, 24, 70])
def test_a_row_that_is_not_finite_stays_alone(q_len, dtype):
    """A NaN or infinite query makes its own row NaN and no other."""
    lens = [150]
    kv, k, v = build(64, 64, 1, lens, seed=24)
    qt = queries((1, q_len, 3, 64), dtype, 24)
    clean = run(kv, qt, None, 150)
    qt[0, 0, 1, 5] = float("nan")
    qt[0, q_len - 1, 2, 9] = float("inf")
    out = run(kv, qt, None, 150)
    bad = torch.zeros((1, q_len, 3, 64), dtype=torch.bool, device="cuda")
    bad[0, 0, 1] = bad[0, q_len - 1, 2] = True
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q_len", [1, 20, 70])
def test_a_dominating_token_keeps_the_small_weights(q_len, dtype):
    """One token outweighs each other by 2^20, and there are 4000 of them: their share of 0.4 % stays."""
    n = 4000
    kv, _, _ = build(64, 128, 1, [n], seed=25)
    k = np.zeros((1, n, 1, 64), np.float32)
    k[0, 0] = 20 * np.log(2.0) / 8.0
    v = np.ones_like(k)
    v[0, 0] = 0.0
    from quantized_base_linear_amd import cache
    cache.qbl_kv_append(kv, 0, None, None, torch.tensor(k).cuda(), torch.tensor(v).cuda())
    k, v = ref.values(*ref.quantise(k)), ref.values(*ref.quantise(v))
    qt = torch.ones((1, q_len, 1, 64), device="cuda").to(TYPES[dtype])
    out = run(kv, qt, None, n)
    compare(kv, k, v, qt, [q_len], [n], out, dtype)
    assert float(out.float().min()) > 0.0035


def test_slots_counts_and_a_bounded_length_with_many_rows():
    lens, slots = [300, 90, 0], [4, 0, 2]
    kv, k, v = build(128, 64, 2, lens, seed=26, slots=slots)
    qt = queries((4, 60, 4, 128), "bf16", 26)
    out = run(kv, qt, [60, 45, 5, 60], 200, slots=slots + [99])
    assert torch.equal(out[0], torch.zeros_like(out[0]))       # its queries sit past the bound
    compare(kv, k[1:2], v[1:2], qt[1:2], [45], [90], out[1:2], "bf16")
    assert torch.equal(out[2:], torch.zeros_like(out[2:]))


@pytest.mark.parametrize("q_len", [17, 40, 100])
def test_reading_rows_by_tile_pads_with_zeros(q_len):
    """Entries with fewer, and with more, new tokens than they hold, a missing page, a slot out of range."""
    from quantized_base_linear_amd import cache
    lens, counts = [70, 9, 200, 64], [q_len, q_len, q_len - 5, 0]
    kv, k, v = build(128, 32, 2, lens, seed=27)
    hole = (200 - q_len + 5) // 32 + 1
    if hole * 32 < 200:
        kv.table[2, hole] = -1
    ko, vo = (torch.full((5, q_len, 2, 128), float("nan"), device="cuda") for _ in range(2))
    cache.qbl_kv_read(kv, 0, dev([0, 1, 2, 3, -1]), dev(counts + [q_len]), ko, vo)
    wk, wv = np.zeros((5, q_len, 2, 128)), np.zeros((5, q_len, 2, 128))
    for i, (n, c) in enumerate(zip(lens, counts)):
        for j in range(c):
            t = n - c + j
            if t >= 0 and not (i == 2 and t // 32 == hole):
                wk[i, j], wv[i, j] = k[i, t], v[i, t]
    for got, want in ((ko, wk), (vo, wv)):
        assert (np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len", [1, 24, 70])
@pytest.mark.parametrize("power", [-18, -12, 12])
def test_values_at_the_ends_of_the_scales_range(power, q_len, dtype):
    """Steps that are fp16 subnormals, and values near the largest that the cache holds.  (Not with f16 rows:
    their outputs would be subnormals, whose half step is 2^-25 and not eps/2 of the value.)"""
    from quantized_base_linear_amd import cache
    n = 150
    kv, _, _ = build(64, 32, 1, [n], seed=28)
    rng = np.random.default_rng(28)
    k = rng.standard_normal((1, n, 1, 64)).astype(np.float32)
    v = (rng.standard_normal(k.shape) * 2.0 ** power).astype(np.float32)
    cache.qbl_kv_append(kv, 0, None, None, torch.tensor(k * 2.0 ** power).float().cuda(), torch.tensor(v).cuda())
    k, v = ref.values(*ref.quantise(k * np.float32(2.0 ** power))), ref.values(*ref.quantise(v))
    qt = queries((1, q_len, 2, 64), dtype, 28)
    out = run(kv, qt, None, n, scale=2.0 ** -power / 8)
    compare(kv, k, v, qt, [q_len], [n], out, dtype, scale=2.0 ** -power / 8)


@pytest.mark.parametrize("n,kv_heads,q_len", [(8, 8, 640), (3, 3, 1500), (16, 16, 200)])
def test_many_workgroups_cover_every_row(n, kv_heads, q_len):
    """Several (entry, head) pairs per XCD, more workgroups than its CUs, and pairs left over."""
    lens = [q_len + 7 * i for i in range(n)]
    kv, k, v = build(64, 64, kv_heads, lens, seed=29)
    qt = queries((n, q_len, kv_heads, 64), "bf16", 29)
    out = run(kv, qt, None, max(lens))
    pick = [0, n - 1]
    compare(kv, k[pick], v[pick], qt[pick], [q_len] * 2, [lens[i] for i in pick], out[pick], "bf16")
    alone = [run(kv, qt[i:i + 1].contiguous(), None, max(lens), slots=[i]) for i in range(n)]
    # an entry by itself is cut along the cache where all together are not: equal up to the outputs' rounding
    for i in range(n):
        a, b = out[i].float(), alone[i][0].float()
        assert float((a - b).norm() / b.norm()) < 2 * 2.0 ** -8
