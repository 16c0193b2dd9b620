"""GPU tests of draft verification at the sizes where the pieces of a row change: whole numbers, so equal."""
import numpy as np
import pytest

from tests.test_gpu_verify import check

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("n,vocab", [(1, 1023), (1, 1024), (1, 1025), (2, 65536), (2, 65537), (70, 29959), (70, 29960), (1, 262145),
                                     (33, 70000)])
def test_sizes_at_the_borders_of_pieces(n, vocab):
    rng = np.random.default_rng(vocab)
    base = torch.tensor(rng.standard_normal((n, 3, vocab)).astype(np.float32)).cuda()
    target = torch.softmax(base, -1)
    draft = torch.softmax(base[:, :2] + 0.7 * torch.randn((n, 2, vocab), device="cuda",
                                                          generator=torch.Generator(device="cuda").manual_seed(1)), -1)
    tokens = torch.multinomial(draft.view(-1, vocab), 1).view(n, 2).cpu().numpy()
    check(target, draft, tokens, None, rng.random((n, 3)), 2)


@pytest.mark.parametrize("vocab", [1024, 5000, 150001])
@pytest.mark.parametrize("r", [0.0, 0.125, 0.5, 0.999, 1.0])
def test_weight_in_few_pieces_only(vocab, r):
    """Pieces without any weight before, between and after those with some; borders are exact."""
    p = np.zeros((1, 1, vocab), np.float32)
    p[0, 0, [vocab // 3, vocab // 3 + 1, vocab // 2, vocab - 2]] = [0.125, 0.375, 0.25, 0.25]
    check(torch.tensor(p).cuda(), None, None, None, [[r]], 0)


@pytest.mark.parametrize("vocab", [900, 150001])
def test_draws_from_the_target_where_nothing_is_left(vocab):
    """The draft covers the target: p - q leaves nothing, and p itself is drawn from."""
    p = np.zeros((1, 2, vocab), np.float32)
    p[0, 0, [3, vocab - 5]] = 0.5
    q = np.zeros((1, 1, vocab), np.float32)
    q[0, 0, [3, vocab - 5]] = 0.75
    acc, nxt = check(torch.tensor(p).cuda(), torch.tensor(q).cuda(), np.array([[3]]), None, [[0.9, 0.75]], 1)
    assert acc[0] == 0 and nxt[0] == vocab - 5
