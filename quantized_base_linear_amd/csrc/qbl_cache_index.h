// Index arithmetic of the cache kernels: which entry, page and tile a lane
// touches.  Everything that decides an address from device-side integers is
// here, in functions that also compile for the host, so that out-of-range
// slots, lengths, counts and pages are tested without a GPU.  Internal.
#pragma once
#include <cstdint>

#include "../../include/qbl_cache.h"

#ifdef __HIPCC__
#define QBL_HD __host__ __device__ __forceinline__
#else
#define QBL_HD inline
#endif

namespace qbl {

constexpr int kTileTokens = 32;
QBL_HD constexpr int64_t kv_tile_bytes(int dim) { return 40ll * dim; }  // codes, then 256 bytes per 32 channels

// The entries of a contents call: which slots, how many new tokens.
struct KvRows {
  const int32_t* slots;   // null: identity
  const int32_t* counts;  // null: q_len each
  int n, q_len;
};

// One entry as the kernels see it: its slot (-1: none), the tokens it holds and
// how many of them are new.
struct Entry {
  int slot, len, c;
};

QBL_HD int clamp_int(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

QBL_HD Entry load_entry(const qbl_kv& kv, const KvRows& r, int i) {
  Entry e;
  e.slot = r.slots ? r.slots[i] : i;
  if (e.slot < 0 || e.slot >= kv.n_slots) return Entry{-1, 0, 0};
  e.len = clamp_int(kv.lens[e.slot], 0, kv.max_pages * kv.page_tokens);  // <= 2^24, checked on the host
  e.c = r.counts ? clamp_int(r.counts[i], 0, r.q_len) : r.q_len;
  return e;
}

// Page of a slot's token position (0 <= pos < max_pages * page_tokens), -1 if none.
QBL_HD int page_of(const qbl_kv& kv, int slot, int pos, int page_shift) {
  const int p = kv.table[(int64_t)slot * kv.max_pages + (pos >> page_shift)];
  return p >= 0 && p < kv.n_pages ? p : -1;
}

// Byte offset in the store of the tile that holds position pos of head h in page p.
QBL_HD int64_t tile_offset(const qbl_kv& kv, int layer, int p, int h, int pos, int page_shift, int dim) {
  const int per = 1 << (page_shift - 5);
  const int64_t page = (int64_t)layer * kv.n_pages + p;
  const int64_t tile = (page * kv.n_kv_heads + h) * per + ((pos & ((1 << page_shift) - 1)) >> 5);
  return tile * kv_tile_bytes(dim);
}

// The tiles that some row of a block of query rows sees: tiles [0, sink) and
// [lo, end).  Rows are (token, query head of the group), r = token * group + head.
struct Span {
  int first, last;  // positions of the first and last valid row (last < first: none)
  int lo, end, sink;
  int tiles;
};

QBL_HD Span row_span(const Entry& e, int r0, int cols, int group, int max_len, int window, int sinks) {
  Span s{0, -1, 0, 0, 0, 0};
  const int rows = e.c * group;
  if (r0 >= rows) return s;
  const int start = e.len - e.c;
  const int r1 = r0 + cols < rows ? r0 + cols : rows;
  const int lim = e.len < max_len ? e.len : max_len;
  s.first = start + r0 / group;
  if (s.first < 0) s.first = 0;
  s.last = start + (r1 - 1) / group;
  if (s.last > lim - 1) s.last = lim - 1;
  if (s.last < s.first) return s;
  if (window > 0) {
    s.lo = s.first - window + 1;
    s.lo = s.lo < 0 ? 0 : s.lo >> 5;
    s.sink = (sinks + 31) >> 5;
    if (s.sink > s.lo) s.sink = s.lo;
  }
  s.end = (s.last >> 5) + 1;
  s.tiles = s.sink + s.end - s.lo;
  return s;
}

// Token position of the v-th visible tile's first token.
QBL_HD int span_pos(const Span& s, int v) { return (v < s.sink ? v : s.lo + v - s.sink) << 5; }

}  // namespace qbl
