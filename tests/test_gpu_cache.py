"""GPU tests of the paged cache: pages (extend with copy-on-write, fork, truncate, compact, copy) against
sequential bookkeeping, exactly; append and read against the block quantiser, bit for bit.

Whole numbers have to be equal.  A value read back is d*code + m of fp16 d, m rounded once to float32,
so it is within half a float32 step, eps/2 = 2^-24, of the 64-bit value."""
import numpy as np
import pytest

import quantized_base_linear_amd as q
from quantized_base_linear_amd import cache
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype).cuda()


def make(n_pages, page, heads, dim, slots, max_pages, layers=1, seed=0):
    """A cache whose store holds random bytes (as fresh device memory might)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.randint(0, 256, (layers * n_pages * cache.qbl_kv_page_bytes(page, heads, dim),), generator=g,
                          device="cuda", dtype=torch.uint8)
    kv = cache.KVCache(layers, n_pages, page, heads, dim, slots, max_pages, store=store)
    return kv, ref.Pages(n_pages, page, slots, max_pages)


def same(kv, pages):
    for a, b in zip((kv.refs, kv.lens, kv.table), pages.state()):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("seed,page,n_pages", [(0, 32, 37), (1, 64, 40), (2, 256, 24), (3, 32, 20000)])
def test_page_calls_follow_the_sequential_bookkeeping(seed, page, n_pages):
    rng = np.random.default_rng(seed)
    slots, max_pages = 12, 10
    kv, pages = make(n_pages, page, 1, 64, slots, max_pages, layers=2, seed=seed)
    ws = cache.pages_workspace(kv, slots)
    model = kv.store.view(2, n_pages, -1).clone()
    if n_pages > 1000:  # free pages far from the start, so that the scan takes several steps
        busy = rng.random(n_pages) < 0.999
        pages.refs = [int(b) for b in busy]
        kv.refs.copy_(dev(pages.refs))
    done = refused = 0
    for step in range(120):
        op = rng.integers(0, 4)
        n = int(rng.integers(1, slots + 1))
        some = rng.permutation(slots)[:n]
        if op == 0:
            counts = rng.integers(-1, 2 * page, n)
            ok = pages.extend(some.tolist(), counts.tolist())
            cache.qbl_kv_extend(kv, dev(some), dev(counts), ws)
            if ok:
                done += 1
                for a, b in pages.copies:
                    model[:, b] = model[:, a]
            else:
                refused += 1
                with pytest.raises(q.QblError):
                    kv.check()
        elif op == 1:
            src = [int(s) for s in rng.integers(0, slots, n)]
            empty = [s for s in range(slots) if pages.lens[s] == 0][:n]
            if not empty:
                continue
            src = src[:len(empty)]
            prefix = None if rng.random() < 0.5 else rng.integers(-2, 4 * page, len(empty)).tolist()
            pages.fork(src, empty, prefix)
            cache.qbl_kv_fork(kv, dev(src), dev(empty), None if prefix is None else dev(prefix))
        elif op == 2:
            lens = rng.integers(-5, 3 * page, n).tolist()
            pages.truncate(some.tolist(), lens)
            cache.qbl_kv_truncate(kv, dev(some), dev(lens))
        elif n_pages < 1000 or step == 60:
            pages.compact()
            cache.qbl_kv_compact(kv, ws)
            for a, b in pages.copies:
                model[:, b] = model[:, a]
        kv.check()
        same(kv, pages)
    assert torch.equal(kv.store.view(2, n_pages, -1), model)
    assert done > 0 and (refused > 0 or n_pages > 30)


def test_identity_slots_and_many_entries():
    kv, pages = make(3000, 32, 1, 64, 1024, 4, seed=5)
    ws = cache.pages_workspace(kv, 1024)
    counts = np.random.default_rng(5).integers(0, 60, 1024)
    assert pages.extend(range(1024), counts.tolist())
    cache.qbl_kv_extend(kv, None, dev(counts), ws)
    kv.check()
    same(kv, pages)
    lens = (counts // 2).tolist()
    pages.truncate(range(1024), lens)
    cache.qbl_kv_truncate(kv, None, dev(lens))
    same(kv, pages)


def test_several_entries_share_one_partly_filled_page():
    kv, pages = make(40, 32, 2, 128, 8, 4, layers=2, seed=6)
    ws = cache.pages_workspace(kv, 8)
    cache.qbl_kv_extend(kv, dev([0]), dev([50]), ws), pages.extend([0], [50])
    cache.qbl_kv_fork(kv, dev([0] * 5), dev([1, 2, 3, 4, 5])), pages.fork([0] * 5, [1, 2, 3, 4, 5])
    model = kv.store.view(2, 40, -1).clone()
    order, counts = [3, 0, 5, 1, 2, 4], [1, 20, 0, 1, 40, 1]
    cache.qbl_kv_extend(kv, dev(order), dev(counts), ws)
    assert pages.extend(order, counts)
    for a, b in pages.copies:
        model[:, b] = model[:, a]
    same(kv, pages)
    assert torch.equal(kv.store.view(2, 40, -1), model) and len(pages.copies) == 5


@pytest.mark.parametrize("call,name", [
    (lambda kv, ws: cache.qbl_kv_extend(kv, dev([0, 9]), dev([1, 1]), ws), "QBL_E_ARG"),
    (lambda kv, ws: cache.qbl_kv_extend(kv, dev([0, -1]), dev([1, 1]), ws), "QBL_E_ARG"),
    (lambda kv, ws: cache.qbl_kv_extend(kv, dev([1, 0, 1]), dev([1, 1, 1]), ws), "QBL_E_DUPLICATE"),
    (lambda kv, ws: cache.qbl_kv_extend(kv, dev([0, 1]), dev([1, 2147483647]), ws), "QBL_E_LIMIT"),
    (lambda kv, ws: cache.qbl_kv_extend(kv, dev([1, 2, 3]), dev([96, 96, 96]), ws), "QBL_E_NOMEM"),
    (lambda kv, ws: cache.qbl_kv_fork(kv, dev([0]), dev([0])), "QBL_E_STATE"),
    (lambda kv, ws: cache.qbl_kv_fork(kv, dev([0, 0]), dev([1, 1])), "QBL_E_DUPLICATE"),
    (lambda kv, ws: cache.qbl_kv_fork(kv, dev([4]), dev([1])), "QBL_E_ARG"),
    (lambda kv, ws: cache.qbl_kv_truncate(kv, dev([0, 0]), dev([1, 1])), "QBL_E_DUPLICATE"),
    (lambda kv, ws: cache.qbl_kv_truncate(kv, dev([1 << 30]), dev([1])), "QBL_E_ARG"),
])
def test_page_calls_that_cannot_be_done_change_nothing(call, name):
    kv, pages = make(6, 32, 1, 64, 4, 3, seed=7)
    ws = cache.pages_workspace(kv, 4)
    cache.qbl_kv_extend(kv, dev([0]), dev([40]), ws), pages.extend([0], [40])
    before = kv.store.clone()
    call(kv, ws)
    with pytest.raises(q.QblError) as e:
        kv.check()
    assert e.value.name == name
    kv.check()  # reported once
    same(kv, pages)
    assert torch.equal(kv.store, before)


def test_extend_refuses_a_missing_page_and_truncate_skips_it():
    kv, _ = make(6, 32, 1, 64, 2, 3)
    ws = cache.pages_workspace(kv, 2)
    kv.lens.copy_(dev([40, 0]))
    kv.table.copy_(dev([[0, 77, -1], [-1, -1, -1]]))
    cache.qbl_kv_extend(kv, dev([0]), dev([1]), ws)
    assert int(kv.status) == q.CODE["QBL_E_STATE"]
    kv.status.zero_()
    cache.qbl_kv_truncate(kv, dev([0]), dev([32]))
    assert kv.lens.tolist() == [32, 0] and kv.table.tolist()[0] == [0, -1, -1] and kv.refs.tolist() == [0] * 6


def test_copy_pages_skips_bad_pairs():
    kv, _ = make(9, 64, 3, 128, 1, 1, layers=3, seed=8)
    s = kv.store.view(3, 9, -1)
    want = s.clone()
    want[:, 4], want[:, 0] = s[:, 1], s[:, 8]
    cache.qbl_kv_copy(kv, dev([1, 9, 2, -1, 8]), dev([4, 5, -3, 6, 0]))
    assert torch.equal(s, want)


# ------------------------------------------------------------------------------ contents ----

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def fill(kv, slots, lens, counts, seed):
    """Random shuffled pages for the given slots; returns nothing (lens, table set directly)."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(kv.n_pages).tolist()
    table = np.full((kv.n_slots, kv.max_pages), -1, np.int32)
    full = np.zeros(kv.n_slots, np.int32)
    for s, n in zip(slots, lens):
        for p in range(-(-n // kv.page_tokens)):
            table[s, p] = order.pop()
        full[s] = n
    kv.table.copy_(dev(table))
    kv.lens.copy_(dev(full))
    return table


@pytest.mark.parametrize("dim,page,heads,dtype,q_len,lens,counts", [
    (128, 64, 2, "f32", 1, [1, 40, 64, 65], [1, 1, 1, 1]),
    (64, 32, 3, "bf16", 7, [7, 33, 90, 5], [7, 3, 7, 0]),
    (256, 128, 1, "f16", 5, [5, 200, 31, 32], [5, 4, 2, 5]),
    (128, 256, 1, "bf16", 300, [300, 511, 290, 3], [300, 299, 17, 3]),
    (64, 64, 1, "f32", 65, [65, 64, 100, 128], [65, 64, 33, 65]),
])
@pytest.mark.parametrize("packed", [False, True])
def test_append_writes_the_quantisers_blocks(dim, page, heads, dtype, q_len, lens, counts, packed):
    slots = [4, 0, 2, 5]
    kv, _ = make(30, page, heads, dim, 6, 9, layers=2, seed=dim)
    table = fill(kv, slots, lens, counts, dim + q_len)
    g = torch.Generator(device="cuda").manual_seed(1)
    n = len(slots)
    wide = torch.randn((n, q_len, 3 * heads, dim), generator=g, device="cuda")
    wide[0, 0] *= 1e-3
    wide[1, 0, :, :32] = 0.0
    wide[2, 0, :, 32:64] = 0.5
    wide[3, -1] *= 1000
    wide = wide.to(TYPES[dtype])
    k, v = wide[:, :, heads:2 * heads], wide[:, :, 2 * heads:]
    if not packed:
        k, v = k.contiguous(), v.contiguous()
    before = kv.store.clone()
    cache.qbl_kv_append(kv, 1, dev(slots), dev(counts), k, v)
    ko = torch.full((n, q_len, heads, dim), float("nan"), device="cuda")
    vo = ko.clone()
    cache.qbl_kv_read(kv, 1, dev(slots), dev(counts), ko, vo)
    # what was there before stays, the rest is the quantiser's
    kc, vc = k.float().cpu().numpy(), v.float().cpu().numpy()
    size, per = 40 * dim, page // 32
    store = before.cpu().numpy().reshape(2, 30, heads, per, size).copy()
    for i, s in enumerate(slots):
        kq, vq = ref.values(*ref.quantise(kc[i])), ref.values(*ref.quantise(vc[i]))
        c = counts[i]
        for got, want in ((ko, kq), (vo, vq)):
            got = got[i].double().cpu().numpy()
            assert np.array_equal(got[c:], np.zeros_like(got[c:]))
            assert (np.abs(got[:c] - want[:c]) <= 2.0 ** -24 * np.abs(want[:c])).all()
        for t0 in range((lens[i] - c) // 32 * 32, lens[i], 32):
            if c == 0:
                break
            rows = range(max(t0, lens[i] - c), min(t0 + 32, lens[i]))
            for h in range(heads):
                tk, tv = np.zeros((32, dim), np.float32), np.zeros((32, dim), np.float32)
                for p in rows:
                    tk[p - t0], tv[p - t0] = kc[i, p - (lens[i] - c), h], vc[i, p - (lens[i] - c), h]
                new = ref.tile_bytes(tk, tv)
                ones = np.zeros((32, dim), np.float32)
                mask = tile_mask([p - t0 for p in rows], dim)
                old = store[1, table[s, t0 // page], h, t0 % page // 32]
                old[:] = (old & ~mask) | (new & mask)
    assert np.array_equal(kv.store.cpu().numpy().reshape(store.shape), store)


def tile_mask(tokens, dim):
    """The bits of a tile that belong to the given tokens."""
    nb = dim // 32
    ng = min(nb, 4)
    m = np.zeros(40 * dim, np.uint8)
    for t in tokens:
        for g in range(nb):
            at = 16 * dim + (t * nb + g) * 4
            m[at:at + 4] = 255
            s = 32 * dim + 128 * nb + ((g * 4 + t % 16 // 4) * 8 + t // 16 * 4 + t % 4) * 2
            m[s:s + 2] = m[s + 64 * nb:s + 64 * nb + 2] = 255
            for quad in range(4):
                at = ((g // ng * 32 + t) * 4 + quad) * ng * 4 + g % ng * 4
                m[at:at + 4] = 255
        for c in range(dim):
            at = 16 * dim + 128 * nb + (((c // 64 * 16 + c % 16) * 4 + t % 16 // 4) * 4 + c % 64 // 16) * 4 + t % 4
            m[at] |= 15 << (4 * (t // 16))
    return m


def test_append_tames_nan_and_large_values():
    kv, _ = make(2, 32, 1, 64, 1, 1)
    kv.lens.fill_(2)
    kv.table.fill_(1)
    x = torch.zeros((1, 2, 1, 64), device="cuda")
    x[0, 0, 0, 0], x[0, 0, 0, 33], x[0, 1, 0, 5] = float("nan"), float("inf"), -1e30
    x[0, 1, 0, 40] = 7.0
    cache.qbl_kv_append(kv, 0, None, None, x, x)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    cache.qbl_kv_read(kv, 0, None, None, ko, vo)
    want = ref.values(*ref.quantise(x.cpu().numpy()))
    assert np.isfinite(want).all() and np.array_equal(ko.double().cpu().numpy(), want)
    assert torch.equal(ko, vo)


def test_append_and_read_without_pages_or_slots():
    kv, _ = make(4, 32, 1, 64, 3, 2, seed=9)
    kv.lens.copy_(dev([40, 3, 2]))
    kv.table.copy_(dev([[2, 4], [-1, -1], [1, -1]]))  # slot 0's second page does not exist
    before = kv.store.clone()
    x = torch.randn((4, 9, 1, 64), device="cuda")
    slots, counts = dev([0, 1, 3, 2]), dev([9, 3, 4, 9])  # entry 2: no such slot; entry 3: more tokens than held
    cache.qbl_kv_append(kv, 0, slots, counts, x, x)
    ko, vo = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    cache.qbl_kv_read(kv, 0, slots, counts, ko, vo)
    want = ref.values(*ref.quantise(x.cpu().numpy()))
    want[0, 1:], want[1], want[2], want[3, :7] = 0, 0, 0, 0
    assert (np.abs(ko.double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want)).all()
    changed = (kv.store.view(4, -1) != before.view(4, -1)).any(1).tolist()
    assert changed == [False, True, True, False]


def test_cache_of_more_than_4_gib():
    kv = cache.KVCache(1, 54000, 256, 1, 256, 1, 2)
    assert kv.store.numel() > 1 << 32
    kv.lens.fill_(300)
    kv.table.copy_(dev([[53999, 53000]]))
    x = torch.randn((1, 300, 1, 256), device="cuda")
    cache.qbl_kv_append(kv, 0, None, None, x, -x)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    cache.qbl_kv_read(kv, 0, None, None, ko, vo)
    want = ref.values(*ref.quantise(x.cpu().numpy()))
    assert (np.abs(ko.double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want)).all()
    cache.qbl_kv_copy(kv, dev([53999, 53000]), dev([0, 1]))
    kv.table.copy_(dev([[0, 1]]))
    cache.qbl_kv_read(kv, 0, None, None, vo, ko)
    assert (np.abs(vo.double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want)).all()
