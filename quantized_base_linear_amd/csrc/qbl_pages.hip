// Pages of the key/value cache: allocation with copy-on-write, forking,
// releasing and compaction, all on the device.
//
// The bookkeeping of one call is done by one workgroup: it checks everything,
// then commits, so a call that cannot be done changes nothing.  Free pages are
// found by scanning refs in index order (16 pages per thread and step), which
// keeps every result independent of scheduling.  Such a call is a chain of five or
// six dependent reads and takes 5 to 9 us whatever it does.  Page contents are
// moved by a second launch over the whole device, bound by memory.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qbl_cache_device.h"

namespace qbl {
namespace {

constexpr int kWg = 1024;
constexpr int kWaves = kWg / 64;
// Bytes of a page that one workgroup copies at a time: 16 per thread.  64 copies
// of 320 KB take 9 us so (20 us with 8 or 16 KB); 536 of them 70 us (5 TB/s,
// what a large copy reaches) with any of these.
constexpr int kPiece = 4096;

// Exclusive prefix sum over the workgroup; total receives the sum.  `red`:
// kWaves + 1 words of LDS.
__device__ __forceinline__ int block_scan(int v, int* red, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int y = __shfl_up(x, s);
    if (lane >= s) x += y;
  }
  __syncthreads();  // red may still be read by a previous scan
  if (lane == 63) red[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int r = red[w];
    if (w < wave) before += r;
    all += r;
  }
  total = all;
  return before + x - v;
}

// The smallest nonzero of the workgroup's error codes' absolute values, as a
// status (0: none); the codes are statuses, at most 15 in magnitude.
__device__ __forceinline__ int block_error(int code, unsigned* word) {
  __syncthreads();
  if (threadIdx.x == 0) *word = 0;
  __syncthreads();
  if (code != 0) atomicOr(word, 1u << (-code));
  __syncthreads();
  const unsigned w = *word;
  return w == 0 ? 0 : -(__ffs((int)w) - 1);
}

__device__ __forceinline__ void set_status(const qbl_kv& kv, int code) {
  if (threadIdx.x == 0 && *kv.status == 0) *kv.status = code;
}

// Index of the entry that flattened item x belongs to: the last i with start[i] <= x.
__device__ __forceinline__ int entry_of(const int* start, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// How many of the entries before i have value s.  Four at a time, without an
// early exit, so that the reads overlap: the list is short but every thread
// goes through it.  `list`: 16-byte aligned, kWg entries.
__device__ __forceinline__ int listed_before(const int* list, int i, int s) {
  int found = 0;
#pragma unroll 4
  for (int j = 0; j < i; j += 4) {
    const int4 v = *reinterpret_cast<const int4*>(list + j);
    found += (v.x == s) + (j + 1 < i && v.y == s) + (j + 2 < i && v.z == s) + (j + 3 < i && v.w == s);
  }
  return found;
}

// 16 consecutive refs from page p (those past n_pages read as used).
__device__ __forceinline__ unsigned free_mask16(const qbl_kv& kv, int p) {
  unsigned m = 0;
  if (p + 16 <= kv.n_pages && (reinterpret_cast<uintptr_t>(kv.refs) & 15) == 0) {
    const int4* r = reinterpret_cast<const int4*>(kv.refs + p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int4 v = r[q];
      m |= (v.x == 0 ? 1u : 0u) << (4 * q) | (v.y == 0 ? 2u : 0u) << (4 * q) | (v.z == 0 ? 4u : 0u) << (4 * q) |
           (v.w == 0 ? 8u : 0u) << (4 * q);
    }
  } else {
    for (int q = 0; q < 16; ++q)
      if (p + q < kv.n_pages && kv.refs[p + q] == 0) m |= 1u << q;
  }
  return m;
}

__global__ __launch_bounds__(kWg) void extend_kernel(qbl_kv kv, const int32_t* slots, const int32_t* counts, int n,
                                                     PagesWs ws) {
  __shared__ __align__(16) int slot_of[kWg], last_of[kWg];
  __shared__ int first_new[kWg], start[kWg];
  __shared__ int red[kWaves + 1];
  __shared__ unsigned word;
  const int i = threadIdx.x, pt = kv.page_tokens;
  const int sh = 31 - __clz(pt);
  int err = 0, s = -1, len = 0, add = 0;
  if (i < n) {
    s = slots ? slots[i] : i;
    if (s < 0 || s >= kv.n_slots) err = QBL_E_ARG, s = -1;
    else {
      len = min(max(kv.lens[s], 0), kv.max_pages * pt);
      add = max(counts[i], 0);
    }
    slot_of[i] = s;
  }
  __syncthreads();
  int have = 0, need = 0, last = -1;
  bool part = false;
  if (i < n && err == 0) {
    if (listed_before(slot_of, i, s) > 0) err = QBL_E_DUPLICATE;
    else if ((int64_t)len + add > (int64_t)kv.max_pages * pt) err = QBL_E_LIMIT;
    else {
      have = (len + pt - 1) >> sh;
      need = (len + add + pt - 1) >> sh;
      part = add > 0 && (len & (pt - 1)) != 0;
      if (part) {
        last = kv.table[(int64_t)s * kv.max_pages + have - 1];
        if (last < 0 || last >= kv.n_pages) err = QBL_E_STATE, part = false, last = -1;
      }
    }
  }
  if (i < n) last_of[i] = part ? last : -1;
  __syncthreads();
  // Of the entries that share a partly filled page each copies it as long as
  // someone else still holds it after the earlier ones have gone.
  bool copy = false;
  if (part) {
    const int r = kv.refs[last];
    if (r > 1) copy = r - listed_before(last_of, i, last) > 1;
  }
  int bad = block_error(err, &word);
  if (bad) {
    set_status(kv, bad);
    if (i == 0) ws.head[0] = 0;
    return;
  }
  const int take = need - have + (copy ? 1 : 0);
  // n_pages bounds what can be taken, so larger sums need not be exact
  int total;
  const int at = block_scan(min(take, kv.max_pages), red, total);
  int copies;
  const int cat = block_scan(copy ? 1 : 0, red, copies);
  // 1024 entries of at most max_pages <= 2^19 pages stay within 32 bits
  if (total > kv.n_pages) {
    set_status(kv, QBL_E_NOMEM);
    if (i == 0) ws.head[0] = 0;
    return;
  }
  int found = 0;
  for (int p0 = 0; p0 < kv.n_pages && found < total; p0 += kWg * 16) {
    const int p = p0 + i * 16;
    unsigned m = p < kv.n_pages ? free_mask16(kv, p) : 0;
    int got;
    int o = found + block_scan(__popc(m), red, got);
    while (m && o < total) {
      const int b = __ffs((int)m) - 1;
      m &= m - 1;
      ws.a[o++] = p + b;
    }
    found += got;
  }
  if (found < total) {
    set_status(kv, QBL_E_NOMEM);
    if (i == 0) ws.head[0] = 0;
    return;
  }
  if (i < n) {
    start[i] = at;
    first_new[i] = have - (copy ? 1 : 0);
  }
  __syncthreads();  // the list in ws.a is this workgroup's own: visible to it after the barrier
  if (i < n) {
    kv.lens[s] = len + add;
    if (copy) {
      ws.src[cat] = last;
      ws.dst[cat] = ws.a[at];
      atomicSub(kv.refs + last, 1);
    }
  }
  for (int x = i; x < total; x += kWg) {
    const int e = entry_of(start, n, x);
    const int p = ws.a[x];
    kv.refs[p] = 1;
    kv.table[(int64_t)slot_of[e] * kv.max_pages + first_new[e] + (x - start[e])] = p;
  }
  if (i == 0) ws.head[0] = copies;
}

__global__ __launch_bounds__(kWg) void fork_kernel(qbl_kv kv, const int32_t* src, const int32_t* dst,
                                                   const int32_t* prefix, int n) {
  __shared__ __align__(16) int to[kWg];
  __shared__ int from[kWg], start[kWg];
  __shared__ int red[kWaves + 1];
  __shared__ unsigned word;
  const int i = threadIdx.x, pt = kv.page_tokens;
  int err = 0, len = 0, pages = 0;
  if (i < n) from[i] = src[i], to[i] = dst[i];
  __syncthreads();
  if (i < n) {
    const int s = from[i], d = to[i];
    if (s < 0 || s >= kv.n_slots || d < 0 || d >= kv.n_slots) err = QBL_E_ARG;
    else if (listed_before(to, i, d) > 0) err = QBL_E_DUPLICATE;
    else if (kv.lens[d] > 0) err = QBL_E_STATE;
    else {
      len = min(max(kv.lens[s], 0), kv.max_pages * pt);
      if (prefix) len = min(len, max(prefix[i], 0));
      pages = (len + pt - 1) / pt;
    }
  }
  const int bad = block_error(err, &word);
  if (bad) {
    set_status(kv, bad);
    return;
  }
  int total;
  const int at = block_scan(pages, red, total);
  if (i < n) {
    start[i] = at;
    kv.lens[to[i]] = len;  // the slot was empty: as a source it is read as length 0, before the barrier in block_scan
  }
  __syncthreads();
  for (int x = i; x < total; x += kWg) {
    const int e = entry_of(start, n, x);
    const int c = x - start[e];
    const int p = kv.table[(int64_t)from[e] * kv.max_pages + c];
    kv.table[(int64_t)to[e] * kv.max_pages + c] = p;
    if (p >= 0 && p < kv.n_pages) atomicAdd(kv.refs + p, 1);
  }
}

__global__ __launch_bounds__(kWg) void truncate_kernel(qbl_kv kv, const int32_t* slots, const int32_t* lens, int n) {
  __shared__ __align__(16) int slot_of[kWg];
  __shared__ int first[kWg], start[kWg];
  __shared__ int red[kWaves + 1];
  __shared__ unsigned word;
  const int i = threadIdx.x, pt = kv.page_tokens;
  int err = 0, s = -1, len = 0, keep = 0, pages = 0;
  if (i < n) {
    s = slots ? slots[i] : i;
    if (s < 0 || s >= kv.n_slots) err = QBL_E_ARG, s = -1;
    slot_of[i] = s;
  }
  __syncthreads();
  if (i < n && err == 0) {
    if (listed_before(slot_of, i, s) > 0) err = QBL_E_DUPLICATE;
    else {
      len = min(max(kv.lens[s], 0), kv.max_pages * pt);
      keep = min(max(lens[i], 0), len);
      first[i] = (keep + pt - 1) / pt;
      pages = (len + pt - 1) / pt - first[i];
    }
  }
  const int bad = block_error(err, &word);
  if (bad) {
    set_status(kv, bad);
    return;
  }
  int total;
  const int at = block_scan(pages, red, total);
  if (i < n) {
    start[i] = at;
    kv.lens[s] = keep;
  }
  __syncthreads();
  for (int x = i; x < total; x += kWg) {
    const int e = entry_of(start, n, x);
    int32_t* t = kv.table + (int64_t)slot_of[e] * kv.max_pages + first[e] + (x - start[e]);
    const int p = *t;
    *t = -1;
    if (p >= 0 && p < kv.n_pages) atomicSub(kv.refs + p, 1);
  }
}

// Plan of a compaction.  With `used` pages in use, the h-th free page before
// index `used` receives the h-th used page at or after it; those are the last
// H used pages, H the number of such holes.
__global__ __launch_bounds__(kWg) void compact_plan_kernel(qbl_kv kv, PagesWs ws) {
  __shared__ int red[kWaves + 1];
  const int i = threadIdx.x;
  int mine = 0;
  for (int p = i * 16; p < kv.n_pages; p += kWg * 16) {
    const int m = min(16, kv.n_pages - p);
    mine += m - __popc(free_mask16(kv, p));
  }
  int used;
  (void)block_scan(mine, red, used);
  int rank = 0, holes = 0;  // used pages, holes before this step
  for (int p0 = 0; p0 < kv.n_pages; p0 += kWg * 16) {
    const int p = p0 + i * 16;
    const int m = max(0, min(16, kv.n_pages - p));
    const unsigned f = m > 0 ? free_mask16(kv, p) : 0;
    const unsigned below = used - p >= 16 ? 0xFFFFu : used > p ? (1u << (used - p)) - 1u : 0u;
    int step_used, step_holes;
    int r = rank + block_scan(m - __popc(f), red, step_used);
    int h = holes + block_scan(__popc(f & below), red, step_holes);
    for (int q = 0; q < m; ++q) {
      const bool fr = f >> q & 1u, lo = below >> q & 1u;
      if (fr) {
        if (lo) ws.a[h++] = p + q;
      } else {
        if (!lo) ws.b[used - 1 - r] = p + q;  // the e-th used page from the end, e < H
        ++r;
      }
      ws.map[p + q] = p + q;
    }
    rank += step_used;
    holes += step_holes;
  }
  __syncthreads();
  for (int h = i; h < holes; h += kWg) {
    const int from = ws.b[holes - 1 - h], to = ws.a[h];
    ws.src[h] = from;
    ws.dst[h] = to;
    ws.map[from] = to;
    kv.refs[to] = kv.refs[from];
    kv.refs[from] = 0;
  }
  if (i == 0) ws.head[0] = holes, ws.head[1] = used;
}

// Copies `count` pages (the device word if given, else n) in all layers.  With
// `map`, the tables' pages are renamed by it first (a compaction: the two touch
// different memory).
__global__ __launch_bounds__(256) void copy_pages_kernel(qbl_kv kv, const int32_t* src, const int32_t* dst,
                                                         const int32_t* count, int n, int64_t page_bytes,
                                                         const int32_t* map) {
  if (map) {
    const int64_t all = (int64_t)kv.n_slots * kv.max_pages, stride = (int64_t)gridDim.x * 256;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all; x += stride) {
      const int p = kv.table[x];
      if (p >= 0 && p < kv.n_pages) {
        const int to = map[p];
        if (to != p) kv.table[x] = to;
      }
    }
  }
  const int pairs = count ? min(*count, n) : n;
  const unsigned pieces = (unsigned)((page_bytes + kPiece - 1) / kPiece), per = pieces * (unsigned)kv.n_layers;
  const int64_t units = (int64_t)pairs * per;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    // units past 2^32 need the long division
    const int pair = units >> 32 ? (int)(u / per) : (int)((unsigned)u / per);
    const unsigned rest = (unsigned)(u - (int64_t)pair * per);
    const int layer = (int)(rest / pieces), piece = (int)(rest - layer * pieces);
    const int from = src[pair], to = dst[pair];
    if (from < 0 || from >= kv.n_pages || to < 0 || to >= kv.n_pages) continue;
    const int64_t off = (int64_t)piece * kPiece;
    const int words = (int)(min((int64_t)kPiece, page_bytes - off) / 16);
    uint8_t* store = static_cast<uint8_t*>(kv.store);
    const uint4* s = reinterpret_cast<const uint4*>(store + ((int64_t)layer * kv.n_pages + from) * page_bytes + off);
    uint4* d = reinterpret_cast<uint4*>(store + ((int64_t)layer * kv.n_pages + to) * page_bytes + off);
    uint4 v[kPiece / 16 / 256];
#pragma unroll
    for (int k = 0; k < kPiece / 16 / 256; ++k)
      if (k * 256 + (int)threadIdx.x < words) v[k] = s[k * 256 + threadIdx.x];
#pragma unroll
    for (int k = 0; k < kPiece / 16 / 256; ++k)
      if (k * 256 + (int)threadIdx.x < words) d[k * 256 + threadIdx.x] = v[k];
  }
}

}  // namespace

namespace {

hipError_t copy_pages(const qbl_kv& kv, const int32_t* src, const int32_t* dst, const int32_t* count, int n,
                      const int32_t* map, const LaunchCtx& lc) {
  const int64_t bytes = qbl_kv_page_bytes(kv.page_tokens, kv.n_kv_heads, kv.head_dim);
  const int64_t units = (int64_t)n * kv.n_layers * ((bytes + kPiece - 1) / kPiece);
  const int grid = (int)std::min<int64_t>(units, 8192);
  QBL_LAUNCH(copy_pages_kernel, dim3(grid), dim3(256), 0, lc, kv, src, dst, count, n, bytes, map);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_copy(const qbl_kv& kv, const int32_t* src, const int32_t* dst, const int32_t* count, int n,
                          const LaunchCtx& lc) {
  (void)hipGetLastError();  // drop errors left by earlier, unrelated calls
  return copy_pages(kv, src, dst, count, n, nullptr, lc);
}

hipError_t launch_kv_extend(const qbl_kv& kv, const int32_t* slots, const int32_t* counts, int n, const PagesWs& ws,
                            const LaunchCtx& lc) {
  (void)hipGetLastError();
  QBL_LAUNCH(extend_kernel, dim3(1), dim3(kWg), 0, lc, kv, slots, counts, n, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_kv_copy(kv, ws.src, ws.dst, ws.head, n, lc);
}

hipError_t launch_kv_fork(const qbl_kv& kv, const int32_t* src, const int32_t* dst, const int32_t* prefix, int n,
                          const LaunchCtx& lc) {
  (void)hipGetLastError();
  QBL_LAUNCH(fork_kernel, dim3(1), dim3(kWg), 0, lc, kv, src, dst, prefix, n);
  return hipGetLastError();
}

hipError_t launch_kv_truncate(const qbl_kv& kv, const int32_t* slots, const int32_t* lens, int n,
                              const LaunchCtx& lc) {
  (void)hipGetLastError();
  QBL_LAUNCH(truncate_kernel, dim3(1), dim3(kWg), 0, lc, kv, slots, lens, n);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const qbl_kv& kv, const PagesWs& ws, const LaunchCtx& lc) {
  (void)hipGetLastError();
  QBL_LAUNCH(compact_plan_kernel, dim3(1), dim3(kWg), 0, lc, kv, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return copy_pages(kv, ws.src, ws.dst, ws.head, kv.n_pages, ws.map, lc);
}

}  // namespace qbl
