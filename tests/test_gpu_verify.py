"""GPU tests of draft verification against the 64-bit sequential form: whole numbers, so equal."""
import numpy as np
import pytest

from quantized_base_linear_amd import cache
from tests import cache_reference as ref
from tests.test_gpu_cache import TYPES, dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def run(target, draft, tokens, counts, u):
    n, vocab = target.shape[0], target.shape[2]
    acc, nxt = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    cache.qbl_verify(target, draft, None if tokens is None else dev(tokens), None if counts is None else dev(counts),
                     torch.tensor(u, dtype=torch.float32).cuda(), acc, nxt, cache.verify_workspace(n, vocab))
    return acc.cpu().numpy(), nxt.cpu().numpy()


def check(target, draft, tokens, counts, u, q_len):
    got = run(target, draft, tokens, counts, u)
    n = target.shape[0]
    want = ref.verify(target.double().cpu().numpy(), None if draft is None else draft.double().cpu().numpy(),
                      np.zeros((n, 0), int) if tokens is None else tokens,
                      [q_len] * n if counts is None else counts, np.asarray(u, np.float32).astype(np.float64), q_len)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (got, want)
    return got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,q_len,vocab", [(1, 1, 1), (3, 2, 2), (5, 4, 100), (2, 8, 4095), (2, 3, 4096), (4, 5, 4097),
                                           (9, 6, 32001), (2, 7, 130001)])
@pytest.mark.parametrize("with_draft", [True, False])
def test_verification_matches_the_sequential_form(n, q_len, vocab, dtype, with_draft):
    rng = np.random.default_rng(vocab + q_len)
    base = torch.tensor(rng.standard_normal((n, q_len + 1, vocab))).cuda()
    target = torch.softmax(base * 2, -1).to(TYPES[dtype])
    near = torch.softmax(base[:, :q_len] * 2 + 0.5 * torch.tensor(rng.standard_normal((n, q_len, vocab))).cuda(), -1)
    tokens = torch.multinomial(near.view(-1, vocab).float(), 1).view(n, q_len).cpu().numpy()
    draft = near.to(TYPES[dtype]) if with_draft else None
    counts = rng.integers(0, q_len + 1, n)
    counts[0] = q_len
    check(target, draft, tokens, counts, rng.random((n, q_len + 1)), q_len)


def test_acceptance_counts_cover_every_outcome():
    n, q_len, vocab = 40, 4, 500
    rng = np.random.default_rng(1)
    base = torch.tensor(rng.standard_normal((n, q_len + 1, vocab))).cuda()
    target = torch.softmax(base, -1).float()
    draft = torch.softmax(base[:, :q_len] + 0.8 * torch.tensor(rng.standard_normal((n, q_len, vocab))).cuda(), -1).float()
    tokens = torch.multinomial(draft.view(-1, vocab), 1).view(n, q_len).cpu().numpy()
    acc, _ = check(target, draft, tokens, None, rng.random((n, q_len + 1)), q_len)
    assert set(acc) == set(range(q_len + 1))


@pytest.mark.parametrize("r", [0.0, 0.24999, 0.25, 0.5, 0.9999999, 1.0, 2.0, -1.0, float("nan")])
def test_borders_of_the_cumulative_sum(r):
    """Dyadic weights: every partial sum is exact, so a number on a border has one right answer."""
    vocab = 9000
    p = np.zeros((1, 1, vocab), np.float32)
    p[0, 0, [5, 4000, 4096, 8999]] = 0.25
    check(torch.tensor(p).cuda(), None, None, None, [[r]], 0)


def test_hopeless_rows_and_odd_values():
    vocab, nan, inf = 600, float("nan"), float("inf")
    target = np.zeros((6, 2, vocab), np.float32)
    draft = np.zeros((6, 1, vocab), np.float32)
    tokens = np.array([[3], [3], [3], [3], [-1], [vocab]])
    target[1, 0, 7] = 0.5                                     # p < q at 3: rejected, draws 7
    draft[1, 0, 3] = 0.5
    target[2, 0, 3], draft[2, 0, 3] = 0.25, 0.5               # nothing left of p - q: draws from p
    target[3, 0, [1, 2, 3, 4]] = nan, inf, -1.0, 0.5          # only token 4 counts
    draft[3, 0, [1, 3, 5]] = nan, 0.5, inf
    target[4:, 0, 9] = 1.0                                    # drafted tokens outside the vocabulary
    u = np.array([[0.5, 0.5]] * 6)
    u[2, 0] = 0.75
    acc, nxt = check(torch.tensor(target).cuda(), torch.tensor(draft).cuda(), tokens, None, u, 1)
    assert acc.tolist() == [0] * 6 and nxt.tolist() == [-1, 7, 3, 4, 9, 9]
    u[:, 0] = nan                                             # never accepted
    check(torch.tensor(target).cuda(), torch.tensor(draft).cuda(), tokens, None, u, 1)
    check(torch.tensor(target).cuda(), torch.tensor(draft).cuda(), tokens, [-3, 0, 99, 1, 1, 1], u, 1)


def test_strided_rows_and_longest_draft():
    n, q_len, vocab = 2, 256, 333
    rng = np.random.default_rng(5)
    wide = torch.tensor(rng.random((n, q_len + 1, vocab + 7)), dtype=torch.float32).cuda()
    target, draft = wide[..., 3:3 + vocab], wide[:, 1:, 5:5 + vocab]
    tokens = rng.integers(0, vocab, (n, q_len))
    check(target, draft, tokens, None, rng.random((n, q_len + 1)) * 0.01, q_len)


def test_replays_of_a_captured_call():
    n, q_len, vocab = 3, 4, 9000
    rng = np.random.default_rng(6)
    target = torch.empty((n, q_len + 1, vocab), device="cuda")
    draft = torch.empty((n, q_len, vocab), device="cuda")
    tokens = dev(rng.integers(0, vocab, (n, q_len)))
    u = torch.empty((n, q_len + 1), device="cuda")
    acc, nxt = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = cache.verify_workspace(n, vocab)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.qbl_verify(target, draft, tokens, None, u, acc, nxt, ws)
    for r in range(5):
        gen = torch.Generator(device="cuda").manual_seed(r)
        for x in (target, draft, u):
            x.uniform_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.verify(target.double().cpu().numpy(), draft.double().cpu().numpy(), tokens.cpu().numpy(), [q_len] * n,
                          u.double().cpu().numpy(), q_len)
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(nxt.cpu().numpy(), want[1])
