"""The serving operators around the quantized-base linear, as measured cases: the 4-bit paged
key/value cache (append, fork / extend / release, compact), attention over it (full, and with a
sliding window and sinks), and the verification of drafted tokens.

`own` selects what `run` computes: False, the operators written out in elementary torch
operations; True, the calls a user makes of quantized_base_linear_amd.cache.  Both sides work on
the same device tensors.

Layout of the cache, as both sides and `exact` read it.  A store is uint8 [page][kv head][tile]
[tile bytes]; a tile holds 32 tokens of one head, D channels in nb = D/32 blocks of 32, each with
an fp16 step d and minimum m (value = d*code + m):
  K codes   [D/64 > 1 ? D/128 : 1][32 tokens][4 quads][min(nb, 4) blocks] 32-bit words; the word of
            (token, quad, block) holds channels 32*block + 8*quad + 0..7, byte i = channel i in the
            low nibble and channel i + 4 in the high one;
  K scales  [32 tokens][nb] 32-bit words d | m << 16;
  V codes   [D/64][16 lanes][4 quads][4] words; the word of (c, lane, quad, n) holds channel
            64*c + 16*n + lane, byte j = token 4*quad + j low, token 16 + 4*quad + j high;
  V scales  d, then m, each fp16 [nb][4 quads][8]: tokens 4*quad + 0..3, then 16 + 4*quad + 0..3.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TILE = 32


# ------------------------------------------------------------------------------ cases ----

def listed():
    return [
        # One request early in a chat: the 4096-wide block's 32 heads of 128 with a key/value head
        # each, float32 as the decode linears write it.  Latency counts.
        {"name": "attend_one", "op": "attend", "n": 1, "q_len": 1, "len_max": 777, "ragged": False,
         "heads": 32, "kv_heads": 32, "dim": 128, "page": 64, "dtype": "f32", "window": 0, "sinks": 0,
         "packed": False, "shape_seed": 1},
        # A serving batch of ragged requests at the 8192-wide model's width (64 heads, 8 key/value heads).
        {"name": "attend_batch", "op": "attend", "n": 32, "q_len": 1, "len_max": 20000, "ragged": True,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "window": 0, "sinks": 0,
         "packed": True, "shape_seed": 2},
        # One very long document: few rows, so the work has to be split over the cache.
        {"name": "attend_long", "op": "attend", "n": 1, "q_len": 1, "len_max": 131071, "ragged": False,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 128, "dtype": "f32", "window": 0, "sinks": 0,
         "packed": False, "shape_seed": 3},
        # A prompt's chunk of 2048 tokens behind 6143 cached ones.
        {"name": "attend_prefill", "op": "attend", "n": 1, "q_len": 2048, "len_max": 8191, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "window": 0, "sinks": 0,
         "packed": True, "shape_seed": 4},
        # Four drafted tokens per request over long streams, read through a window with sinks.
        {"name": "window_draft", "op": "attend", "n": 16, "q_len": 4, "len_max": 32768, "ragged": True,
         "heads": 32, "kv_heads": 4, "dim": 64, "page": 32, "dtype": "f16", "window": 4096, "sinks": 4,
         "packed": False, "shape_seed": 5},
        # Prompts of two requests read through a short window with sinks, ragged.
        {"name": "window_prefill", "op": "attend", "n": 2, "q_len": 1500, "len_max": 6001, "ragged": True,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "window": 1024, "sinks": 4,
         "packed": True, "shape_seed": 6},
        # One decode step of 64 requests: a token each is quantised into its page and read back.
        {"name": "append_step", "op": "append", "n": 64, "q_len": 1, "len_max": 4096, "ragged": True,
         "kv_heads": 8, "dim": 128, "page": 64, "dtype": "f32", "packed": False, "shape_seed": 7},
        # A prompt of 4097 tokens, keys and values as slices of one projection's output.
        {"name": "append_prompt", "op": "append", "n": 1, "q_len": 4097, "len_max": 4500, "ragged": False,
         "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "packed": True, "shape_seed": 8},
        # Sampling four continuations of each of 16 prompts: the children are released, forked from
        # their parents again and extended (which copies each child's partly filled page).
        {"name": "fork_extend", "op": "fork", "parents": 16, "children": 4, "len_max": 2000, "count": 9,
         "layers": 4, "kv_heads": 8, "dim": 128, "page": 64, "spare": 200, "shape_seed": 9},
        # A pool with holes after requests ended, moved together.
        {"name": "compact", "op": "compact", "n": 48, "len_max": 3000, "layers": 4, "kv_heads": 8, "dim": 128,
         "page": 64, "spare": 1100, "shape_seed": 10},
        # One request with four drafted tokens over a 32000-token vocabulary.
        {"name": "verify_one", "op": "verify", "n": 1, "q_len": 4, "vocab": 32000, "dtype": "f32",
         "draft": True, "shape_seed": 11},
        # A batch of 64 requests with up to seven drafted tokens, a large odd vocabulary.
        {"name": "verify_batch", "op": "verify", "n": 64, "q_len": 7, "vocab": 130001, "dtype": "f32",
         "draft": True, "shape_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], {"bytes": 0, "flops": 0})
        t["bytes"], t["flops"] = max(t["bytes"], w["bytes"]), max(t["flops"], w["flops"])
    op = rng.choice(["attend", "attend", "attend", "append", "fork", "compact", "verify"])
    while True:
        seed = rng.randrange(1 << 30)
        if op == "attend":
            many = rng.random() < 0.4
            q_len = _log_int(rng, 9, 2048) if many else rng.randint(1, 8)
            length = max(q_len, _log_int(rng, 1, 131072))
            windowed = rng.random() < 0.4
            kv = rng.choice([1, 2, 4, 8, 16, 32])
            c = {"op": op, "n": _log_int(rng, 1, 32), "q_len": q_len, "len_max": length,
                 "ragged": rng.random() < 0.6, "heads": kv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]),
                 "kv_heads": kv, "dim": rng.choice([64, 128, 128, 128, 256]),
                 "page": rng.choice([32, 64, 128, 256]), "dtype": rng.choice(["f32", "bf16", "f16"]),
                 "window": _log_int(rng, 1, 8192) if windowed else 0,
                 "sinks": rng.choice([0, 1, 4, 33]) if windowed else 0, "packed": rng.random() < 0.5,
                 "shape_seed": seed}
            if c["n"] * c["q_len"] * c["heads"] > 2048 * 64:
                continue
        elif op == "append":
            q_len = _log_int(rng, 1, 4097)
            c = {"op": op, "n": _log_int(rng, 1, 128), "q_len": q_len, "len_max": max(q_len, _log_int(rng, 1, 16384)),
                 "ragged": rng.random() < 0.6, "kv_heads": rng.choice([1, 2, 4, 8, 16, 32]),
                 "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([32, 64, 128, 256]),
                 "dtype": rng.choice(["f32", "bf16", "f16"]), "packed": rng.random() < 0.5, "shape_seed": seed}
        elif op == "fork":
            c = {"op": op, "parents": _log_int(rng, 1, 32), "children": rng.randint(1, 6),
                 "len_max": _log_int(rng, 1, 4000), "count": _log_int(rng, 1, 300), "layers": rng.randint(1, 4),
                 "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128, 256]),
                 "page": rng.choice([32, 64, 128]), "spare": 0, "shape_seed": seed}
            c["spare"] = c["parents"] * c["children"] * (c["count"] // c["page"] + 2) + rng.randint(0, 50)
        elif op == "compact":
            c = {"op": op, "n": _log_int(rng, 1, 64), "len_max": _log_int(rng, 1, 4000), "layers": rng.randint(1, 4),
                 "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128, 256]),
                 "page": rng.choice([32, 64, 128]), "spare": _log_int(rng, 1, 1000), "shape_seed": seed}
        else:
            c = {"op": op, "n": _log_int(rng, 1, 64), "q_len": rng.randint(1, 8), "vocab": _log_int(rng, 100, 200000),
                 "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "draft": rng.random() < 0.8, "shape_seed": seed}
        w = work(c)
        if w["bytes"] <= top[op]["bytes"] and w["flops"] <= top[op]["flops"]:
            return c


# ------------------------------------------------- sizes that the case alone decides ----

def _shape(case):
    """Lengths (new tokens included), new-token counts and page ids of the case, as Python lists."""
    r = random.Random(case["shape_seed"])
    if case["op"] in ("attend", "append"):
        n, q_len, top = case["n"], case["q_len"], case["len_max"]
        lens, counts = [], []
        for i in range(n):
            c, t = q_len, top
            if case["ragged"] and i > 0:
                t = r.randint(1, top)
                c = min(t, q_len if q_len <= 8 else r.randint(1, q_len))
            lens.append(t)
            counts.append(c)
    elif case["op"] == "fork":
        lens = [r.randint(max(1, case["len_max"] // 2), case["len_max"]) for _ in range(case["parents"])]
        counts = []
    else:
        lens = [r.randint(1, case["len_max"]) for _ in range(case["n"])]
        counts = []
    pages = [-(-t // case["page"]) for t in lens]
    return lens, counts, pages, r


def _visible(case, lens, counts):
    """(query, key) pairs that the mask lets through, and tokens of the cache that some query reads."""
    w, s = case["window"], case["sinks"]
    pairs = tokens = 0
    for t, c in zip(lens, counts):
        first = t - c
        if w == 0:
            pairs += c * first + c * (c + 1) // 2
            tokens += t
        else:
            for i in range(first, t):
                lo = max(0, i - w + 1)
                pairs += i - lo + 1 + min(s, lo)
            lo = max(0, first - w + 1)
            tokens += t - lo + min(s, lo)
    return pairs, tokens


def _token_bytes(case):
    """Bytes of one token's keys and values over all heads of one layer."""
    return 2 * case["kv_heads"] * (case["dim"] // 2 + case["dim"] // 32 * 4)


def work(case):
    if case["op"] == "verify":
        item = 4 if case["dtype"] == "f32" else 2
        rows = case["n"] * case["vocab"]
        return {"bytes": rows * item * (2 if case["draft"] else 1) + case["n"] * (12 * case["q_len"] + 12),
                "flops": 4 * rows}
    lens, counts, pages, _ = _shape(case)
    if case["op"] == "attend":
        pairs, tokens = _visible(case, lens, counts)
        item = 4 if case["dtype"] == "f32" else 2
        rows = sum(counts) * case["heads"]
        return {"bytes": 2 * rows * case["dim"] * item + tokens * _token_bytes(case),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "append":
        item = 4 if case["dtype"] == "f32" else 2
        values = 2 * sum(counts) * case["kv_heads"] * case["dim"]
        # the input read, the cache written, its values handed back in float32
        return {"bytes": values * (item + 4) + sum(counts) * _token_bytes(case), "flops": 6 * values}
    page_bytes = case["layers"] * case["page"] * _token_bytes(case)
    if case["op"] == "fork":
        moved = case["children"] * sum(1 for t in lens if t % case["page"])
        moved += sum(0 for _ in lens)
    else:
        live, order = _compact_layout(case)
        moved = sum(1 for p in order[:live] if p >= live)
    return {"bytes": 2 * moved * page_bytes + 8 * sum(pages), "flops": sum(pages)}


def _compact_layout(case):
    _, _, pages, r = _shape(case)
    live = sum(pages)
    order = list(range(live + case["spare"]))
    r.shuffle(order)
    return live, order


# ----------------------------------------------------------------------------- inputs ----

def _tile_bytes(d):
    return TILE * d + 2 * TILE * (d // 32) * 4


def _quantise(x):
    """Codes, steps and minima of 32-value blocks, in float32: m = fp16(min), d = fp16((max - m)/15),
    code = (x - m)/d rounded half away from zero, within 0..15."""
    b = x.float().unflatten(-1, (-1, 32))
    m = b.amin(-1, keepdim=True).half()
    spread = b.amax(-1, keepdim=True) - m.float()
    d = (spread / torch.full_like(spread, 15.0)).half()   # a division by a plain number may be a product
    df = d.float()
    t = torch.where(df > 0, (b - m.float()) / torch.where(df > 0, df, torch.ones_like(df)), torch.zeros_like(b))
    t = t.clamp(-1.0, 16.0)
    whole = t.floor()
    code = (whole + (t - whole >= 0.5).float()).clamp(0.0, 15.0)
    return code, d, m


def _values(code, d, m):
    return (d.float() * code + m.float()).flatten(-2)


def _pack(k, v):
    """[tiles][32 tokens][H][D] keys and values -> bytes [tiles][H][tile bytes]."""
    n, _, h, dim = k.shape
    nb = dim // 32
    ng = min(nb, 4)
    kc, kd, km = _quantise(k)          # [n][32][h][nb][32]
    vc, vd, vm = _quantise(v)
    c = kc.to(torch.uint8).reshape(n, 32, h, nb // ng, ng, 4, 2, 4)   # ..., quad, half, byte
    c = c[..., 0, :] | (c[..., 1, :] << 4)                             # n t h chunk g quad byte
    part_kc = c.permute(0, 2, 3, 1, 5, 4, 6).reshape(n, h, -1)
    s = torch.stack([kd[..., 0], km[..., 0]], -1)                      # n t h nb 2
    part_ks = s.permute(0, 2, 1, 3, 4).contiguous().view(torch.uint8).reshape(n, h, -1)
    c = vc.to(torch.uint8).reshape(n, 2, 4, 4, h, dim // 64, 4, 16)    # n half quad j h chunk sub lane
    c = c[:, 0] | (c[:, 1] << 4)                                       # n quad j h chunk sub lane
    part_vc = c.permute(0, 3, 4, 6, 1, 5, 2).reshape(n, h, -1)
    s = torch.stack([vd[..., 0], vm[..., 0]], 1).reshape(n, 2, 2, 4, 4, h, nb)   # n dm half quad j h nb
    part_vs = s.permute(0, 5, 1, 6, 3, 2, 4).contiguous().view(torch.uint8).reshape(n, h, -1)
    return torch.cat([part_kc, part_ks, part_vc, part_vs], -1)


def _unpack(tiles, dim):
    """Bytes [tiles][H][tile bytes] -> float32 keys and values [tiles*32][H][D]."""
    n, h, _ = tiles.shape
    nb = dim // 32
    ng = min(nb, 4)
    a, b = 16 * dim, 16 * dim + 128 * nb
    e = b + 16 * dim
    c = tiles[..., :a].reshape(n, h, nb // ng, 32, 4, ng, 4)
    c = torch.stack([c & 15, c >> 4], -2)                              # n h chunk t quad g half byte
    c = c.permute(0, 3, 1, 2, 5, 4, 6, 7).reshape(n, 32, h, nb, 32)
    s = tiles[..., a:b].contiguous().view(torch.float16).reshape(n, h, 32, nb, 2).permute(0, 2, 1, 3, 4)
    k = _values(c.float(), s[..., 0:1], s[..., 1:2])
    c = tiles[..., b:e].reshape(n, h, dim // 64, 16, 4, 4, 4)          # chunk lane quad sub j
    c = torch.stack([c & 15, c >> 4], 0)                               # half n h chunk lane quad sub j
    c = c.permute(1, 0, 5, 7, 2, 3, 6, 4).reshape(n, 32, h, nb, 32)
    s = tiles[..., e:].contiguous().view(torch.float16).reshape(n, h, 2, nb, 4, 2, 4)
    s = s.permute(0, 5, 4, 6, 1, 3, 2).reshape(n, 32, h, nb, 2)
    v = _values(c.float(), s[..., 0:1], s[..., 1:2])
    return k.reshape(n * 32, h, dim), v.reshape(n * 32, h, dim)


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + salt) % (1 << 62))
    return g


def _keys_values(g, tokens, h, dim, dtype=torch.float32):
    """Keys with a few channels far from zero, as rotary-free projections have them; plain values."""
    k = torch.randn((tokens, h, dim), generator=g, device="cuda")
    k[..., ::29] += 3.0
    v = torch.randn((tokens, h, dim), generator=g, device="cuda")
    return k.to(dtype), v.to(dtype)


def _filled_store(g, layers, n_pages, case):
    h, dim, per = case["kv_heads"], case["dim"], case["page"] // TILE
    store = torch.empty((layers, n_pages, h, per, _tile_bytes(dim)), dtype=torch.uint8, device="cuda")
    flat = store.view(layers * n_pages, h, per, -1)
    step = max(1, (1 << 24) // (case["page"] * h * dim))
    for p in range(0, flat.shape[0], step):
        m = min(step, flat.shape[0] - p)
        k, v = _keys_values(g, m * case["page"], h, dim)
        t = _pack(k.view(m * per, TILE, h, dim), v.view(m * per, TILE, h, dim))
        flat[p:p + m] = t.view(m, per, h, -1).permute(0, 2, 1, 3)
    return store.view(layers, n_pages, -1)


def _table(rows, width):
    t = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, row in enumerate(rows):
        if row:
            t[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return t.cuda()


def _inputs(case, seed):
    """The device tensors of one case."""
    g = _gen(seed, case["shape_seed"])
    st = {"case": case}
    if case["op"] == "verify":
        n, j, v = case["n"], case["q_len"], case["vocab"]
        dt = DTYPES[case["dtype"]]
        base = torch.randn((n, j + 1, v), generator=g, device="cuda") * 2.0
        st["target"] = torch.softmax(base, -1).to(dt)
        near = base[:, :j] + torch.randn((n, j, v), generator=g, device="cuda") * 0.7
        near = torch.softmax(near, -1)
        pick = torch.rand((n, j, 1), generator=g, device="cuda") * near.double().sum(-1, keepdim=True)
        st["tokens"] = (near.double().cumsum(-1) <= pick).sum(-1).clamp(max=v - 1).to(torch.int32)
        st["draft"] = near.to(dt) if case["draft"] else None
        r = random.Random(case["shape_seed"])
        st["counts"] = torch.tensor([j] + [r.randint(0, j) for _ in range(n - 1)], dtype=torch.int32).cuda()
        st["u"] = torch.rand((n, j + 1), generator=g, device="cuda")
        return st
    lens, counts, pages, r = _shape(case)
    h, dim, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "compact":
        live, order = _compact_layout(case)
        n_pages, layers, slots = live + case["spare"], case["layers"], case["n"]
    elif case["op"] == "fork":
        live = sum(pages)
        n_pages, layers, slots = live + case["spare"], case["layers"], case["parents"] * (1 + case["children"])
        order = list(range(n_pages))
        r.shuffle(order)
    else:
        live = sum(pages)
        n_pages, layers, slots = live + 3, 1, case["n"]
        order = list(range(n_pages))
        r.shuffle(order)
    rows, at = [], 0
    for m in pages:
        rows.append(order[at:at + m])
        at += m
    rows += [[] for _ in range(slots - len(rows))]
    width = max(pages) + (case.get("count", 0) // page + 2 if case["op"] == "fork" else 0)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[order[:live]] = 1
    st.update(store=_filled_store(g, layers, n_pages, case), refs=refs.cuda(), table=_table(rows, width),
              lens=torch.tensor(lens + [0] * (slots - len(lens)), dtype=torch.int32).cuda(), n_pages=n_pages,
              layers=layers, slots=slots)
    if case["op"] in ("attend", "append"):
        st["counts"] = torch.tensor(counts, dtype=torch.int32).cuda()
        dt = DTYPES[case["dtype"]]
        n, q_len, heads = case["n"], case["q_len"], case.get("heads", 0)
        wide = heads + 2 * h
        if case["packed"]:
            x = torch.randn((n, q_len, wide, dim), generator=g, device="cuda").to(dt)
            st["q"], st["k"], st["v"] = x[:, :, :heads], x[:, :, heads:heads + h], x[:, :, heads + h:]
        else:
            st["q"] = torch.randn((n, q_len, heads, dim), generator=g, device="cuda").to(dt)
            st["k"] = torch.randn((n, q_len, h, dim), generator=g, device="cuda").to(dt)
            st["v"] = torch.randn((n, q_len, h, dim), generator=g, device="cuda").to(dt)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    lens, counts, pages, _ = _shape(case) if case["op"] != "verify" else (None, None, None, None)
    st["lens_host"], st["counts_host"] = lens, counts
    if case["op"] == "compact":
        st["refs0"], st["table0"] = st["refs"].clone(), st["table"].clone()
    if case["op"] == "fork":
        p, m = case["parents"], case["children"]
        st["src"] = torch.arange(p, dtype=torch.int32).repeat_interleave(m).cuda()
        st["dst"] = torch.arange(p, p * (1 + m), dtype=torch.int32).cuda()
        st["zero"] = torch.zeros(p * m, dtype=torch.int32, device="cuda")
        st["grow"] = torch.full((p * m,), case["count"], dtype=torch.int32, device="cuda")
    if own:
        from quantized_base_linear_amd import cache
        if case["op"] == "verify":
            st["accepted"] = torch.empty(case["n"], dtype=torch.int32, device="cuda")
            st["next"] = torch.empty(case["n"], dtype=torch.int32, device="cuda")
            st["ws"] = cache.verify_workspace(case["n"], case["vocab"])
            return st
        kv = cache.KVCache(st["layers"], st["n_pages"], case["page"], case["kv_heads"], case["dim"], st["slots"],
                           st["table"].shape[1], store=st["store"], refs=st["refs"], lens=st["lens"],
                           table=st["table"])
        st["kv"] = kv
        if case["op"] == "attend":
            st["out"] = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
            st["ws"] = cache.attend_workspace(kv, case["n"], case["q_len"], case["heads"], case["len_max"],
                                              window=case["window"], sinks=case["sinks"], dtype=st["q"].dtype)
        elif case["op"] == "append":
            st["k_out"] = torch.empty(st["k"].shape, dtype=torch.float32, device="cuda")
            st["v_out"] = torch.empty(st["v"].shape, dtype=torch.float32, device="cuda")
        else:
            st["ws"] = cache.pages_workspace(kv, case.get("parents", 0) * case.get("children", 0))
    return st


# -------------------------------------------------------------------------- plain forms ----

def _tokens_of(st, i, length):
    """Keys and values of the first `length` tokens of slot i, float32 [length][H][D]."""
    case = st["case"]
    per = case["page"] // TILE
    ids = st["table"][i, :-(-length // case["page"])].long()
    t = st["store"][0][ids].view(len(ids), case["kv_heads"], per, -1).permute(0, 2, 1, 3)
    k, v = _unpack(t.reshape(len(ids) * per, case["kv_heads"], -1), case["dim"])
    return k[:length], v[:length]


def _attend_plain(st):
    case = st["case"]
    heads, h, dim = case["heads"], case["kv_heads"], case["dim"]
    g = heads // h
    out = torch.zeros(st["q"].shape, dtype=st["q"].dtype, device="cuda")
    for i, (length, c) in enumerate(zip(st["lens_host"], st["counts_host"])):
        if c == 0:
            continue
        k, v = _tokens_of(st, i, length)
        q = st["q"][i, :c].float().reshape(c, h, g, dim).permute(1, 0, 2, 3).reshape(h, c * g, dim)
        s = torch.matmul(q, k.permute(1, 2, 0).contiguous()) * (1.0 / math.sqrt(dim))
        pos = torch.arange(length - c, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None]
        seen = key <= pos
        if case["window"]:
            seen &= (pos - key < case["window"]) | (key < case["sinks"])
        s = s.view(h, c, g, length).masked_fill_(~seen[None, :, None], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(h, c * g, length), v.permute(1, 0, 2).contiguous()).view(h, c, g, dim) / total
        out[i, :c] = o.permute(1, 0, 2, 3).reshape(c, heads, dim).to(out.dtype)
    return out


def _append_plain(st):
    k, v = _values(*_quantise(st["k"])), _values(*_quantise(st["v"]))
    live = torch.arange(k.shape[1], device="cuda")[None, :, None, None] < st["counts"][:, None, None, None]
    zero = torch.zeros((), device="cuda")
    return torch.where(live, k, zero), torch.where(live, v, zero)


def _release(st, slots):
    rows = st["table"][slots.long()]
    ids = rows[rows >= 0].long()
    st["refs"].index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    st["table"][slots.long()] = -1
    st["lens"][slots.long()] = 0


def _fork_plain(st):
    case = st["case"]
    page = case["page"]
    src, dst = st["src"].long(), st["dst"].long()
    _release(st, st["dst"])
    st["table"][dst] = st["table"][src]
    st["lens"][dst] = st["lens"][src]
    ids = st["table"][dst]
    ids = ids[ids >= 0].long()
    st["refs"].index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    # extend: a partly filled last page that others share is copied, then new pages are taken,
    # lowest free pages first, slot by slot
    length = st["lens"][dst].long()
    after = length + st["grow"].long()
    have, need = (length + page - 1) // page, (after + page - 1) // page
    last = st["table"][dst, (have - 1).clamp(min=0)].long()
    copy = length % page != 0        # every child shares it with its parent, who is not extended
    take = need - have + copy.long()
    free = torch.nonzero(st["refs"] == 0)[:, 0]
    start = take.cumsum(0) - take
    cols = torch.arange(st["table"].shape[1], device="cuda")[None]
    lo = have - copy.long()
    new = (cols >= lo[:, None]) & (cols < need[:, None])
    pos = (start[:, None] + cols - lo[:, None]).clamp(0, free.numel() - 1)
    rows = torch.where(new, free[pos].to(torch.int32), st["table"][dst])
    st["table"][dst] = rows
    st["lens"][dst] = after.to(torch.int32)
    st["refs"][rows[new].long()] = 1
    gone = last[copy]
    st["refs"].index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    fresh = free[start[copy]]
    for layer in range(st["layers"]):
        st["store"][layer].index_copy_(0, fresh, st["store"][layer][gone])


def _compact_plain(st):
    used = st["refs"] > 0
    live = int(used.sum())
    hole = torch.nonzero(~used[:live])[:, 0]
    tail = torch.nonzero(used[live:])[:, 0] + live
    to = torch.arange(st["n_pages"], device="cuda")
    to[tail] = hole
    st["refs"][hole] = st["refs"][tail]
    st["refs"][tail] = 0
    t = st["table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].to(torch.int32), t))
    for layer in range(st["layers"]):
        st["store"][layer].index_copy_(0, hole, st["store"][layer][tail])


def _weights(x):
    x = x.double()
    return torch.where(torch.isfinite(x) & (x > 0), x, torch.zeros_like(x))


def _verify_plain(st):
    n, j, v = st["case"]["n"], st["case"]["q_len"], st["case"]["vocab"]
    target, draft, tok = st["target"], st["draft"], st["tokens"].long()
    step = torch.arange(j, device="cuda")[None]
    p = _weights(target[:, :j].gather(2, tok[..., None])[..., 0])
    q = _weights(draft.gather(2, tok[..., None])[..., 0]) if draft is not None else torch.ones_like(p)
    ok = (st["u"][:, :j].double() * q < p) & (step < st["counts"][:, None])
    accepted = ok.long().cumprod(1).sum(1)
    row = torch.arange(n, device="cuda")
    pa = _weights(target[row, accepted])
    rejected = accepted < st["counts"]
    at = accepted.clamp(max=j - 1)
    if draft is not None:
        qa = _weights(draft[row, at])
    else:
        qa = torch.zeros_like(pa).scatter_(1, tok[row, at][:, None], 1.0)
    w = torch.where(rejected[:, None], (pa - qa).clamp(min=0.0), pa)
    w = torch.where((w.sum(1) == 0)[:, None], pa, w)
    cum = w.cumsum(1)
    total = cum[:, -1:]
    hit = (w > 0) & (cum > st["u"][:, j:].double() * total)
    index = torch.arange(v, device="cuda")[None]
    first = torch.where(hit, index, v).amin(1)
    last = torch.where(w > 0, index, -1).amax(1)
    return accepted.to(torch.int32), torch.where(first < v, first, last).to(torch.int32)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from quantized_base_linear_amd import cache
        if op == "verify":
            cache.qbl_verify(state["target"], state["draft"], state["tokens"], state["counts"], state["u"],
                             state["accepted"], state["next"], state["ws"])
            return state["accepted"], state["next"]
        kv = state["kv"]
        if op == "attend":
            cache.qbl_kv_attend(kv, 0, None, state["counts"], state["q"], state["out"], case["len_max"],
                                window=case["window"], sinks=case["sinks"], ws=state["ws"])
            return state["out"]
        if op == "append":
            cache.qbl_kv_append(kv, 0, None, state["counts"], state["k"], state["v"])
            cache.qbl_kv_read(kv, 0, None, state["counts"], state["k_out"], state["v_out"])
            return state["k_out"], state["v_out"]
        if op == "fork":
            cache.qbl_kv_truncate(kv, state["dst"], state["zero"])
            cache.qbl_kv_fork(kv, state["src"], state["dst"])
            cache.qbl_kv_extend(kv, state["dst"], state["grow"], state["ws"])
        else:
            state["refs"].copy_(state["refs0"])
            state["table"].copy_(state["table0"])
            cache.qbl_kv_compact(kv, state["ws"])
    else:
        if op == "verify":
            return _verify_plain(state)
        if op == "attend":
            return _attend_plain(state)
        if op == "append":
            return _append_plain(state)
        if op == "fork":
            _fork_plain(state)
        else:
            state["refs"].copy_(state["refs0"])
            state["table"].copy_(state["table0"])
            _compact_plain(state)
    return state["refs"], state["lens"], state["table"], state["store"].view(torch.int32)


# ------------------------------------------------------------------------------- exact ----

def _code_index(dim):
    """Byte and shift of each (token, channel) code inside a tile, for keys and for values."""
    nb = dim // 32
    ng = min(nb, 4)
    t = torch.arange(32)[:, None]
    c = torch.arange(dim)[None]
    block, quad, i = c // 32, c % 32 // 8, c % 8
    key = (((block // ng * 32 + t) * 4 + quad) * ng + block % ng) * 4 + i % 4
    key_shift = (i // 4 * 4).expand(32, dim)
    half, tt = t // 16, t % 16
    val = 16 * dim + 128 * nb + (((c // 64 * 16 + c % 16) * 4 + tt // 4) * 4 + c % 64 // 16) * 4 + tt % 4
    val_shift = (half * 4).expand(32, dim)
    key_scale = 16 * dim + (t * nb + block) * 4
    val_scale = 32 * dim + 128 * nb + ((block * 4 + tt // 4) * 8 + half * 4 + tt % 4) * 2
    return [x.reshape(-1).cuda() for x in (key, key_shift, val, val_shift, key_scale, val_scale)]


def _half_at(tiles, at):
    pair = torch.stack([tiles[:, at], tiles[:, at + 1]], -1).contiguous()
    return pair.view(torch.float16)[..., 0].double()


def _exact_tokens(st, i, head, length):
    case = st["case"]
    dim, page, per = case["dim"], case["page"], case["page"] // TILE
    key, ks, val, vs, kd, vd = _code_index(dim)
    ids = st["table"][i, :-(-length // page)].long()
    size = _tile_bytes(dim)
    tiles = st["store"][0][ids].view(len(ids), case["kv_heads"], per, size)[:, head].reshape(-1, size)
    k = _half_at(tiles, kd) * (tiles[:, key] >> ks & 15).double() + _half_at(tiles, kd + 2)
    v = _half_at(tiles, vd) * (tiles[:, val] >> vs & 15).double() + _half_at(tiles, vd + 2 * TILE * (dim // 32))
    return k.view(-1, dim)[:length], v.view(-1, dim)[:length]


def _exact_attend(case, seed):
    st = _inputs(case, seed)
    lens, counts, _, _ = _shape(case)
    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for i, (length, c) in enumerate(zip(lens, counts)):
        for head in range(case["kv_heads"]):
            k, v = _exact_tokens(st, i, head, length)
            for lo in range(0, c, 256):
                hi = min(c, lo + 256)
                x = st["q"][i, lo:hi, head * g:(head + 1) * g].double().reshape(-1, case["dim"])
                s = (x @ k.T.contiguous()) / math.sqrt(case["dim"])
                at = torch.arange(length - c + lo, length - c + hi, device="cuda").repeat_interleave(g)[:, None]
                j = torch.arange(length, device="cuda")[None]
                hidden = j > at
                if case["window"]:
                    hidden |= (j <= at - case["window"]) & (j >= case["sinks"])
                s[hidden] = -math.inf
                w = torch.softmax(s, -1)
                out[i, lo:hi, head * g:(head + 1) * g] = (w @ v).view(hi - lo, g, -1)
    return out


def _exact_round_trip(x):
    """The block quantiser's definition names its float32 and fp16 roundings; each is applied here to
    a value computed in 64 bits."""
    b = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    m = b.min(-1, keepdim=True).values.float().half().double()
    d = ((b.max(-1, keepdim=True).values - m).float().double() / 15).float().half().double()
    t = ((b - m).float().double() / torch.where(d == 0, 1.0, d)).float().double()
    code = torch.where(d == 0, 0.0, torch.trunc(t + 0.5)).clip(0, 15)
    return (d * code + m).reshape(x.shape)


def _exact_verify(case, seed):
    st = _inputs(case, seed)
    n, j = case["n"], case["q_len"]
    counts, tok, u = st["counts"].tolist(), st["tokens"].tolist(), st["u"].double().tolist()
    accepted, following = [], []
    for b in range(n):
        a = 0
        while a < counts[b]:
            x = tok[b][a]
            p = float(st["target"][b, a, x])
            q = float(st["draft"][b, a, x]) if case["draft"] else 1.0
            if u[b][a] * q >= p:
                break
            a += 1
        w = st["target"][b, a].double()
        if a < counts[b]:
            rest = w.clone()
            if case["draft"]:
                rest -= st["draft"][b, a].double()
            else:
                rest[tok[b][a]] -= 1.0
            rest[rest < 0] = 0.0
            if float(rest.sum()) > 0:
                w = rest
        total = torch.cumsum(w, 0)
        kept = torch.nonzero(w)[:, 0]
        above = kept[total[kept] > u[b][j] * total[-1]]
        following.append(int(above[0]) if above.numel() else int(kept[-1]) if kept.numel() else -1)
        accepted.append(a)
    return (torch.tensor(accepted, dtype=torch.int32, device="cuda"),
            torch.tensor(following, dtype=torch.int32, device="cuda"))


def exact(case, seed):
    if case["op"] == "attend":
        if work(case)["flops"] > 3e12:
            return None
        return _exact_attend(case, seed)
    if case["op"] == "append":
        st = _inputs(case, seed)
        live = torch.arange(case["q_len"], device="cuda")[None, :] < st["counts"][:, None]
        return tuple(_exact_round_trip(st[x]) * live[..., None, None].double() for x in ("k", "v"))
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    return None  # pages move whole numbers: there is nothing to compute in 64 bits
