"""Plain 64-bit implementations of the cache operators (include/qbl_cache.h), on the CPU: the page
bookkeeping as sequential Python, the block quantiser in numpy, attention and draft verification in
float64.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


class Pages:
    """The bookkeeping of a cache: lists per slot, reference counts, lowest free page first."""

    def __init__(self, n_pages, page_tokens, n_slots, max_pages):
        self.n_pages, self.pt, self.n_slots, self.max_pages = n_pages, page_tokens, n_slots, max_pages
        self.refs = [0] * n_pages
        self.lens = [0] * n_slots
        self.table = [[] for _ in range(n_slots)]
        self.copies = []  # (source, destination) page pairs of the last call

    def state(self):
        t = np.full((self.n_slots, self.max_pages), -1, np.int32)
        for s, row in enumerate(self.table):
            t[s, :len(row)] = row
        return np.array(self.refs, np.int32), np.array(self.lens, np.int32), t

    def extend(self, slots, counts):
        """True if it was done; False (nothing changed) if pages lack."""
        free = [p for p in range(self.n_pages) if self.refs[p] == 0]
        refs, plan, copies = list(self.refs), [], []
        for s, c in zip(slots, counts):
            c = max(c, 0)
            row, length = list(self.table[s]), self.lens[s]
            if length + c > self.max_pages * self.pt:
                return False
            if c > 0 and length % self.pt and refs[row[-1]] > 1:
                if not free:
                    return False
                new = free.pop(0)
                refs[row[-1]] -= 1
                copies.append((row[-1], new))
                refs[new] = 1
                row[-1] = new
            while len(row) * self.pt < length + c:
                if not free:
                    return False
                new = free.pop(0)
                refs[new] = 1
                row.append(new)
            plan.append((s, row, length + c))
        for s, row, length in plan:
            self.table[s], self.lens[s] = row, length
        self.refs, self.copies = refs, copies
        return True

    def fork(self, src, dst, prefix=None):
        rows = [list(self.table[s]) for s in src]
        lens = [self.lens[s] for s in src]
        for i, d in enumerate(dst):
            n = lens[i] if prefix is None else max(0, min(prefix[i], lens[i]))
            self.table[d] = rows[i][:-(-n // self.pt)]
            self.lens[d] = n
            for p in self.table[d]:
                self.refs[p] += 1

    def truncate(self, slots, lens):
        for s, n in zip(slots, lens):
            n = max(0, min(n, self.lens[s]))
            keep = -(-n // self.pt)
            for p in self.table[s][keep:]:
                self.refs[p] -= 1
            self.table[s], self.lens[s] = self.table[s][:keep], n

    def compact(self):
        used = [p for p in range(self.n_pages) if self.refs[p] > 0]
        holes = [p for p in range(len(used)) if self.refs[p] == 0]
        self.copies = list(zip(used[len(used) - len(holes):], holes))
        to = dict(self.copies)
        for a, b in self.copies:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]


def quantise(x):
    """(codes, d, m) of the blocks of 32 along the last axis, float32 arithmetic as defined."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-32768), np.float32(32768)))
    b = x.reshape(*x.shape[:-1], -1, 32)
    m = b.min(-1, keepdims=True).astype(np.float16)
    d = ((b.max(-1, keepdims=True) - m.astype(np.float32)) / np.float32(15)).astype(np.float16)
    df = d.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(df > 0, (b - m.astype(np.float32)) / df, np.float32(0))
    code = np.clip(np.where(t > 0, np.floor(t.astype(np.float64) + 0.5), 0), 0, 15)
    return code.astype(np.uint8), d, m


def values(code, d, m):
    """float64 values of quantised blocks (exact)."""
    v = d.astype(np.float64) * code + m.astype(np.float64)
    return v.reshape(*v.shape[:-2], -1)


def tile_bytes(k, v):
    """Bytes of one tile, written code by code from the layout's definition: k, v float32 [32][D]."""
    dim = k.shape[1]
    nb = dim // 32
    ng = min(nb, 4)
    out = np.zeros(40 * dim, np.uint8)
    kc, kd, km = quantise(k)
    vc, vd, vm = quantise(v)
    half = lambda z: np.frombuffer(np.float16(z).tobytes(), np.uint8)
    for t in range(32):
        for g in range(nb):
            at = 16 * dim + (t * nb + g) * 4
            out[at:at + 2], out[at + 2:at + 4] = half(kd[t, g, 0]), half(km[t, g, 0])
            s = 32 * dim + 128 * nb + ((g * 4 + t % 16 // 4) * 8 + t // 16 * 4 + t % 4) * 2
            out[s:s + 2], out[s + 64 * nb:s + 64 * nb + 2] = half(vd[t, g, 0]), half(vm[t, g, 0])
        for c in range(dim):
            g, quad, i = c // 32, c % 32 // 8, c % 8
            at = (((g // ng * 32 + t) * 4 + quad) * ng + g % ng) * 4 + i % 4
            out[at] |= kc[t, g, c % 32] << (4 * (i // 4))
            at = 16 * dim + 128 * nb + (((c // 64 * 16 + c % 16) * 4 + t % 16 // 4) * 4 + c % 64 // 16) * 4 + t % 4
            out[at] |= vc[t, c // 32, c % 32] << (4 * (t // 16))
    return out


def attend(q, k, v, first, window=0, sinks=0, scale=0.0, hidden=None):
    """float64 attention of one entry: q [c][heads][D], k, v [len][kv heads][D], query j at position
    first + j.  hidden: bool per key, True = not there.  Returns (out, spread, logit): spread is
    sum p |v| per output, logit the largest scale * sum |q k| over a row's visible keys."""
    q, k, v = (np.asarray(z, np.float64) for z in (q, k, v))
    c, heads, dim = q.shape
    n, kv_heads = k.shape[:2]
    group = heads // kv_heads
    scale = scale or 1.0 / math.sqrt(dim)
    pos = first + np.arange(c)[:, None]
    key = np.arange(n)[None]
    seen = key <= pos
    if window:
        seen &= (pos - key < window) | (key < sinks)
    if hidden is not None:
        seen &= ~hidden[None]
    out, spread = np.zeros((c, heads, dim)), np.zeros((c, heads, dim))
    logit = np.zeros((c, heads, 1))
    rows = seen.any(1)
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        s = np.where(seen, q[:, h] @ kk.T * scale, -np.inf)
        top = np.where(rows, s.max(1, initial=-np.inf), 0.0)[:, None]
        p = np.exp(s - top)
        total = p.sum(1, keepdims=True)
        p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        out[:, h], spread[:, h] = p @ vv, p @ np.abs(vv)
        size = np.where(seen, np.abs(q[:, h]) @ np.abs(kk).T * scale, 0.0)
        logit[:, h, 0] = size.max(1, initial=0.0)
    return out, spread, logit


def verify(target, draft, tokens, counts, u, q_len):
    """(accepted, next) per request, float64, one token at a time."""
    clean = lambda z: np.where(np.isfinite(z) & (z > 0), z, 0.0)
    target = clean(np.asarray(target, np.float64))
    if draft is not None:
        draft = clean(np.asarray(draft, np.float64))
    vocab = target.shape[2]
    accepted, following = [], []
    for b in range(target.shape[0]):
        c = max(0, min(int(counts[b]), q_len))
        a = 0
        while a < c:
            x = int(tokens[b][a])
            if not 0 <= x < vocab:
                break
            q = 1.0 if draft is None else draft[b, a, x]
            if not float(u[b][a]) * q < target[b, a, x]:
                break
            a += 1
        w = target[b, a]
        if a < c:
            if draft is not None:
                rest = np.maximum(w - draft[b, a], 0.0)
            else:
                rest = w.copy()
                if 0 <= int(tokens[b][a]) < vocab:
                    rest[int(tokens[b][a])] = max(rest[int(tokens[b][a])] - 1.0, 0.0)
            if rest.sum() > 0:
                w = rest
        cum = np.cumsum(w)
        hit = np.nonzero((w > 0) & (cum > float(u[b][q_len]) * cum[-1]))[0]
        some = np.nonzero(w > 0)[0]
        following.append(int(hit[0]) if hit.size else int(some[-1]) if some.size else -1)
        accepted.append(a)
    return np.array(accepted, np.int32), np.array(following, np.int32)
