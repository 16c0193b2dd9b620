"""Decoding with drafted tokens over the paged 4-bit cache, on the quantised linears.

A small random model (embedding, layers of q/k/v/o projections around attention, output head; every
matrix a q8_0 base with a low-rank adapter) continues a few prompts.  Each prompt is prefilled once
and forked, so its continuations share its pages.  Every step drafts tokens with the model's first
layer alone, runs the whole model over them in one pass, keeps what verification accepts and drops the
rest from the cache.  At the end some requests are released, the pool is compacted, and one request's
cached keys and values are read back and compared with those of a fresh cache filled in one pass.

    python examples/speculative_decode.py [--steps 12]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_base_linear_amd as qbl
from quantized_base_linear_amd import cache

DIM, HEADS, KV_HEADS, HEAD_DIM, LAYERS, VOCAB = 512, 8, 2, 64, 3, 1000
WINDOW, SINKS = 96, 4
PAGE, DRAFT = 32, 3


class Model:
    """The linears of all layers in one composition: q, k, v, o per layer, then the output head."""

    def __init__(self, seed=0):
        rng = np.random.default_rng(seed)
        shapes = [(HEADS * HEAD_DIM, DIM), (KV_HEADS * HEAD_DIM, DIM), (KV_HEADS * HEAD_DIM, DIM),
                  (DIM, HEADS * HEAD_DIM)] * LAYERS + [(VOCAB, DIM)]
        descs, low_rank = [], []
        for i, (n, k) in enumerate(shapes):
            w = (rng.standard_normal((n, k)) * (1.5 / np.sqrt(k))).astype(np.float32)
            descs.append((qbl.QBL_Q8_0, n, k, qbl.qbl_quantize(qbl.QBL_Q8_0, w)))
            a = (rng.standard_normal((8, k)) / np.sqrt(k)).astype(np.float32)
            b = (rng.standard_normal((n, 8)) * 0.1).astype(np.float32)
            low_rank.append((i, a, b))
        self.base = qbl.qbl_base_load(descs)
        self.adapter = qbl.qbl_adapter_load(self.base, low_rank)
        self.comp = qbl.qbl_comp_create(self.base)
        qbl.qbl_comp_attach(self.comp, [self.adapter], [1.0])
        self.rows = [n for n, _ in shapes]
        self.ws = {(i, b): qbl.workspace(self.comp, qbl.OP_LINEAR, i, b) for i in range(len(shapes)) for b in range(1, 9)}
        self.embedding = torch.from_numpy(rng.standard_normal((VOCAB, DIM)).astype(np.float32)).cuda()

    def linear(self, i, x):
        """x [..., k] -> [..., n], eight rows per call."""
        flat = x.reshape(-1, x.shape[-1]).contiguous()
        y = torch.empty((flat.shape[0], self.rows[i]), device="cuda")
        for r in range(0, flat.shape[0], 8):
            b = min(8, flat.shape[0] - r)
            qbl.qbl_linear(self.comp, i, flat[r:r + b], y[r:r + b], b, self.ws[i, b])
        return y.view(*x.shape[:-1], self.rows[i])

    def forward(self, kv, slots, counts, tokens, max_len, layers=LAYERS):
        """Probabilities after each new token [n][q_len][VOCAB].  The tokens' room in the cache has been
        made; layers 0..layers-1 write their keys and values and attend to what the slots hold."""
        n, q_len = tokens.shape
        x = self.embedding[tokens.long()]
        out = torch.empty((n, q_len, HEADS, HEAD_DIM), device="cuda")
        ws = cache.attend_workspace(kv, n, q_len, HEADS, max_len, WINDOW, SINKS)
        for layer in range(layers):
            y = torch.nn.functional.rms_norm(x, (DIM,))
            q = self.linear(4 * layer, y).view(n, q_len, HEADS, HEAD_DIM)
            k = self.linear(4 * layer + 1, y).view(n, q_len, KV_HEADS, HEAD_DIM)
            v = self.linear(4 * layer + 2, y).view(n, q_len, KV_HEADS, HEAD_DIM)
            cache.qbl_kv_append(kv, layer, slots, counts, k, v)
            cache.qbl_kv_attend(kv, layer, slots, counts, q, out, max_len, window=WINDOW, sinks=SINKS, ws=ws)
            x = x + self.linear(4 * layer + 3, out.view(n, q_len, HEADS * HEAD_DIM))
        return torch.softmax(self.linear(4 * LAYERS, torch.nn.functional.rms_norm(x, (DIM,))) * 0.5, -1)

    def free(self):
        qbl.qbl_comp_free(self.comp)
        qbl.qbl_adapter_free(self.adapter)
        qbl.qbl_base_free(self.base)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def main(steps=12, prompts=(70, 33), copies=2, seed=0, say=print):
    torch.manual_seed(seed)
    model = Model(seed)
    n, parents = len(prompts) * copies, len(prompts)
    max_len = max(prompts) + steps * (DRAFT + 1) + DRAFT + 1
    pages = -(-max_len // PAGE)
    kv = cache.KVCache(LAYERS, (n + parents) * pages, PAGE, KV_HEADS, HEAD_DIM, n + parents, pages)
    ws = cache.pages_workspace(kv, n + parents)

    # Prefill each prompt into its own slot, then fork its continuations from it.
    longest = max(prompts)
    prompt = torch.randint(0, VOCAB, (parents, longest), dtype=torch.int32, device="cuda")
    slots, counts = ints(range(n, n + parents)), ints(prompts)
    cache.qbl_kv_extend(kv, slots, counts, ws)
    probs = model.forward(kv, slots, counts, prompt, max_len)
    first = torch.stack([probs[i, c - 1] for i, c in enumerate(prompts)])
    cache.qbl_kv_fork(kv, slots.repeat_interleave(copies), ints(range(n)))
    last = torch.multinomial(first.repeat_interleave(copies, 0), 1).to(torch.int32)   # not in the cache yet
    text = [prompt[i // copies, :prompts[i // copies]].tolist() for i in range(n)]

    accepted, following = ints([0] * n), ints([0] * n)
    check = cache.verify_workspace(n, VOCAB)
    one, kept = ints([1] * n), 0
    for _ in range(steps):
        # Draft with the first layer: the last token, then each drafted one, a token at a time.
        before = kv.lens[:n].clone()
        drafted, q_rows, token = [], [], last
        for _ in range(DRAFT):
            cache.qbl_kv_extend(kv, None, one, ws)
            q_rows.append(model.forward(kv, None, None, token, max_len, layers=1))
            token = torch.multinomial(q_rows[-1][:, 0], 1).to(torch.int32)
            drafted.append(token)
        cache.qbl_kv_truncate(kv, None, before)
        # The whole model over the last and the drafted tokens, then verification.
        drafted = torch.cat(drafted, 1)
        block = torch.cat([last, drafted], 1)
        cache.qbl_kv_extend(kv, None, one * (DRAFT + 1), ws)
        target = model.forward(kv, None, None, block, max_len)
        u = torch.rand((n, DRAFT + 1), device="cuda")
        cache.qbl_verify(target, torch.cat(q_rows, 1), drafted.contiguous(), None, u, accepted, following, check)
        cache.qbl_kv_truncate(kv, None, before + 1 + accepted)
        last = following.view(n, 1).clone()
        for i, a in enumerate(accepted.tolist()):   # the program's output, not the loop's state
            text[i] += block[i, :a + 1].tolist()
            kept += a
    kv.check()
    lens = kv.lens[:n].tolist()
    assert lens == [len(t) for t in text]
    say(f"{steps} steps of {n} requests: {kept / (steps * n):.2f} of {DRAFT} drafted tokens accepted on average")

    # Release everything but the last request, move its pages together, and compare its cache with a
    # fresh one that takes the same tokens in one pass.
    keep = n - 1
    gone = [i for i in range(n + parents) if i != keep]
    cache.qbl_kv_truncate(kv, ints(gone), ints([0] * len(gone)))
    cache.qbl_kv_compact(kv, ws)
    kv.check()
    used = int((kv.refs > 0).sum())
    assert used == -(-lens[keep] // PAGE) and bool((kv.refs[:used] == 1).all())
    other = cache.KVCache(LAYERS, pages, PAGE, KV_HEADS, HEAD_DIM, 1, pages)
    tokens = ints([text[keep]])
    cache.qbl_kv_extend(other, None, ints([lens[keep]]), ws)
    model.forward(other, None, None, tokens, max_len)
    worst = 0.0
    for layer in range(LAYERS):
        a, b, c, d = (torch.empty((1, lens[keep], KV_HEADS, HEAD_DIM), device="cuda") for _ in range(4))
        cache.qbl_kv_read(kv, layer, ints([keep]), None, a, b)
        cache.qbl_kv_read(other, layer, None, None, c, d)
        worst = max(worst, float((a - c).norm() / c.norm()), float((b - d).norm() / d.norm()))
    say(f"request {keep}: {lens[keep]} tokens in {used} pages; cached values differ by {worst:.2e} from a single pass")
    model.free()
    return kept, worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=12)
    main(parser.parse_args().steps)
