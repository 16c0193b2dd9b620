// Attention over the paged 4-bit key/value cache (decode form, any row count).
//
//   out = softmax(c q K^T) V,  K and V in blocks of 32 channels: x = d*code + m.
//
// Both products run on the matrix cores with the integer codes as exact bf16
// operands, and the block steps and minima enter outside in float32:
//   score(t, q)  = c * sum_g [ d_K(t,g) * (sum_{k in g} code(t,k) q_k) + m_K(t,g) * sum_{k in g} q_k ]
//   out(q, c)   ~  sum_t (p_t d_V(t,g)) code(t,c) + sum_t p_t m_V(t,g),   g = c / 32
// so no key or value is ever rounded.  The other operand is split into bf16
// parts: hi + mid + lo hold a float32's 24 bits.
//
// A workgroup serves one key/value head of one entry: 16 * NT query rows (the
// query heads that share the head, times the new tokens) against a run of
// tiles, its four waves taking tiles in turn.  Tokens are the rows of the
// score product, so its result is already laid out as the second product's
// operand: lane (quad, row q) holds tokens 4 quad + 0..3 of both halves of the
// tile, which is the order that the value codes are stored in.  Codes go from
// global memory straight into operand registers, one tile ahead; only the
// scales go through LDS, as every lane needs those of 8 tokens.
//
// The softmax is one pass: each row keeps a reference maximum that is raised
// (and the sums rescaled) only when a score passes it by 8 in the exponent of
// 2, so in most tiles no cross-lane step is needed.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qbl_cache_device.h"

namespace qbl {
namespace {

typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;  // weights stay below 2^8 times the reference

__device__ __forceinline__ Span block_span(const KvAttend& a, const Entry& e, int r0, int cols) {
  return row_span(e, r0, cols, a.group, (int)a.max_len, (int)a.window, (int)a.sinks);
}

// Codes of one word as bf16, in the order channel (or token) 0..7.  A nibble n
// read as an e4m3 number is n * 2^-9 exactly (subnormal up to 7, then the first
// binade), and the conversion multiplies by 2^9.
__device__ __forceinline__ bf8v codes8(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const bf2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
  const bf2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
  const bf2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
  const bf2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
  return bf8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x as P bf16 parts, largest first; the parts of three sum to x exactly up to
// float32's range ends.
template <int P>
__device__ __forceinline__ void split8(const float (&x)[8], bf8v (&part)[P]) {
  float rest[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) rest[j] = x[j];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[p][j] = (__bf16)rest[j];
    if (p + 1 < P) {
#pragma unroll
      for (int j = 0; j < 8; ++j) rest[j] -= (float)part[p][j];
    }
  }
}

// LDS writes of this wave become visible to its own later reads; no other wave takes part.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int DIM>
struct TileRegs {
  static constexpr int kNb = DIM / 32, kNg = kNb < 4 ? kNb : 4;
  uint32_t kc[2][kNb];      // key codes of token 16 s + col
  uint32_t vc[DIM / 16];    // value codes of channel 16 n + col
  uint32_t sc[kNb];         // this lane's piece of the scales
  int pos;                  // first token position, or -1: no page
};

template <int N>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[N], int at) {
  if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[at] = v.x, w[at + 1] = v.y, w[at + 2] = v.z, w[at + 3] = v.w;
  }
}

template <int DIM>
__device__ __forceinline__ void load_tile(const KvAttend& a, const Entry& e, const Span& s, int h, int v, int page_shift,
                                          int lane, TileRegs<DIM>& t) {
  constexpr int kNb = DIM / 32, kNg = kNb < 4 ? kNb : 4;
  const int col = lane & 15, quad = lane >> 4;
  const int pos = __builtin_amdgcn_readfirstlane(span_pos(s, v));
  const int page = __builtin_amdgcn_readfirstlane(page_of(a.kv, e.slot, pos, page_shift));
  t.pos = page < 0 ? -1 : pos;
  if (page < 0) {
#pragma unroll
    for (int k = 0; k < kNb; ++k) t.kc[0][k] = t.kc[1][k] = t.sc[k] = 0;
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k) t.vc[k] = 0;
    return;
  }
  const uint8_t* p = tile_ptr<DIM>(a.kv, a.layer, page, h, pos, page_shift);
  const uint32_t* kc = reinterpret_cast<const uint32_t*>(p);
  const uint32_t* vc = reinterpret_cast<const uint32_t*>(p + 16 * DIM + 128 * kNb);
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int ch = 0; ch < kNb / kNg; ++ch)
      load_words<kNb>(kc + ((ch * 32 + half * 16 + col) * 4 + quad) * kNg, t.kc[half], 4 * ch);
#pragma unroll
  for (int ch = 0; ch < DIM / 64; ++ch) load_words<DIM / 16>(vc + ((ch * 16 + col) * 4 + quad) * 4, t.vc, 4 * ch);
  // lanes 0..31: key scales, 32..63: value scales, kNb words each
  const uint8_t* sp = p + (lane < 32 ? 16 * DIM : 32 * DIM + 128 * kNb) + (lane & 31) * 4 * kNb;
#pragma unroll
  for (int ch = 0; ch < (kNb + 3) / 4; ++ch) load_words<kNb>(reinterpret_cast<const uint32_t*>(sp) + 4 * ch, t.sc, 4 * ch);
}

template <int DIM, int T, int NT>
__global__ __launch_bounds__(kThreads) void attend_kernel(KvAttend a, int row_blocks, int chunk, int splits,
                                                          int page_shift, int64_t part_floats) {
  constexpr int kNb = DIM / 32;
  constexpr int kQp = T == QBL_T_F32 ? 3 : T == QBL_T_F16 ? 2 : 1;  // bf16 parts of q: all of its bits
  constexpr int kPp = T == QBL_T_F32 ? 3 : 2;                       // bf16 parts of the weights
  constexpr int kOut = DIM + 4;
  __shared__ __align__(16) uint32_t scales[kWaves][64 * kNb];
  __shared__ __align__(16) float obuf[kWaves][16][kOut];
  __shared__ float ml[kWaves][16][2];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, quad = lane >> 4;
  int b = blockIdx.x;
  const int split = b % splits;
  b /= splits;
  const int rb = b % row_blocks;
  b /= row_blocks;
  const int h = b % a.kv.n_kv_heads, i = b / a.kv.n_kv_heads;
  const Entry e = load_entry(a.kv, a.rows, i);
  const int r0 = rb * 16 * NT;
  const Span sp = block_span(a, e, r0, 16 * NT);
  if (splits > 1 && split * chunk >= sp.tiles) return;

  bf8v q[NT][kNb][kQp];
  float qsum[NT][kNb];
  int pos_of[NT];  // this lane's row's position, -1 for padding
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + nt * 16 + col;
    const int j = r / a.group;
    const int pos = e.len - e.c + j;
    const bool ok = r < e.c * a.group && pos >= sp.first && pos <= sp.last;
    pos_of[nt] = ok ? pos : -1;
#pragma unroll
    for (int g = 0; g < kNb; ++g) {
      float x[8];
      if (ok) {
        const int64_t at = (int64_t)i * a.qs[0] + (int64_t)j * a.qs[1] +
                           (int64_t)(h * a.group + r - j * a.group) * a.qs[2] + g * 32 + quad * 8;
        load8<T>(a.q, at, a.vec, x);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0.0f;
      }
      split8<kQp>(x, q[nt][g]);
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += x[k];
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      qsum[nt][g] = s;
    }
  }

  f4v o[NT][DIM / 16];
  float msum[NT][kNb], m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kNegInf, l[nt] = 0.0f;
#pragma unroll
    for (int n = 0; n < DIM / 16; ++n) o[nt][n] = f4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < kNb; ++g) msum[nt][g] = 0.0f;
  }
  const float c2 = a.scale * kLog2e;
  const int win = (int)a.window, sinks = (int)a.sinks;
  const int v1 = min(sp.tiles, (split + 1) * chunk);
  uint32_t* sc = scales[wave];

  TileRegs<DIM> t;
  int v = split * chunk + wave;
  if (v < v1) load_tile<DIM>(a, e, sp, h, v, page_shift, lane, t);
  for (; v < v1; v += kWaves) {
    const int pos = t.pos;
    const bool have = pos >= 0;
    const bool full = have && pos + 31 <= sp.first && (win == 0 || pos >= sp.last - win + 1 || pos + 31 < sinks);
    if (have && !full && lane >= 32) {
      // Value scales of tokens that no row sees become 0, so that whatever is
      // stored there meets a weight of 0 as a finite number.
#pragma unroll
      for (int k = 0; k < kNb; ++k) {
        const int at = (lane & 31) * 2 * kNb + 2 * k;   // half index: [d | m][block][quad][8]
        const int qd = at >> 3 & 3;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int x = (at + z) & 7;
          const int tok = pos + (x >> 2) * 16 + qd * 4 + (x & 3);
          const bool seen = tok <= sp.last && (win == 0 || tok < sinks || tok > sp.first - win);
          if (!seen) t.sc[k] &= z ? 0x0000FFFFu : 0xFFFF0000u;
        }
      }
    }
    wave_sync();
#pragma unroll
    for (int k = 0; k < kNb; ++k) sc[lane * kNb + k] = t.sc[k];
    wave_sync();
    const TileRegs<DIM> cur = t;
    if (v + kWaves < v1) load_tile<DIM>(a, e, sp, h, v + kWaves, page_shift, lane, t);
    if (!have) continue;

    float s[NT][8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t* dm = sc + (half * 16 + quad * 4) * kNb;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[nt][half * 4 + r] = 0.0f;
#pragma unroll
      for (int g = 0; g < kNb; ++g) {
        const bf8v kc = codes8(cur.kc[half][g]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f4v d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int p = kQp - 1; p >= 0; --p) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc, q[nt][g][p], d, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t w = dm[r * kNb + g];
            float x = s[nt][half * 4 + r];
            x = fmaf(half_bits(w & 0xFFFFu), d[r], x);
            s[nt][half * 4 + r] = fmaf(half_bits(w >> 16), qsum[nt][g], x);
          }
        }
      }
    }

    float p[NT][8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = kNegInf;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float x = s[nt][k] * c2;
        if (!full) {
          const int tok = pos + (k >> 2) * 16 + quad * 4 + (k & 3);
          const bool seen = tok <= pos_of[nt] && (win == 0 || pos_of[nt] - tok < win || tok < sinks);
          x = seen ? x : kNegInf;
        }
        s[nt][k] = x;
        top = fmaxf(top, x);
      }
      if (__any(top > m[nt] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float up = fmaxf(m[nt], top);
        const float f = m[nt] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[nt] - up);
        m[nt] = up;
        l[nt] *= f;
#pragma unroll
        for (int n = 0; n < DIM / 16; ++n) o[nt][n] *= f;
#pragma unroll
        for (int g = 0; g < kNb; ++g) msum[nt][g] *= f;
      }
      const float ref = m[nt] == kNegInf ? 0.0f : m[nt];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        p[nt][k] = __builtin_amdgcn_exp2f(s[nt][k] - ref);
        l[nt] += p[nt][k];
      }
    }

    const uint4* vd = reinterpret_cast<const uint4*>(sc + 32 * kNb);
#pragma unroll
    for (int g = 0; g < kNb; ++g) {
      const uint4 dw = vd[g * 4 + quad], mw = vd[(kNb + g) * 4 + quad];
      const uint32_t dws[4] = {dw.x, dw.y, dw.z, dw.w}, mws[4] = {mw.x, mw.y, mw.z, mw.w};
      const bf8v va = codes8(cur.vc[2 * g]), vb = codes8(cur.vc[2 * g + 1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pd[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t sel = k & 1 ? dws[k >> 1] >> 16 : dws[k >> 1] & 0xFFFFu;
          const uint32_t sem = k & 1 ? mws[k >> 1] >> 16 : mws[k >> 1] & 0xFFFFu;
          pd[k] = p[nt][k] * half_bits(sel);
          msum[nt][g] = fmaf(p[nt][k], half_bits(sem), msum[nt][g]);
        }
        bf8v part[kPp];
        split8<kPp>(pd, part);
#pragma unroll
        for (int x = kPp - 1; x >= 0; --x) {
          o[nt][2 * g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, part[x], o[nt][2 * g], 0, 0, 0);
          o[nt][2 * g + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, part[x], o[nt][2 * g + 1], 0, 0, 0);
        }
      }
    }
  }

  // Join the four waves, 16 rows at a time.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float ls = l[nt];
    ls += __shfl_xor(ls, 16);
    ls += __shfl_xor(ls, 32);
    if (nt > 0) __syncthreads();
#pragma unroll
    for (int g = 0; g < kNb; ++g) {
      float x = msum[nt][g];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
#pragma unroll
      for (int z = 0; z < 2; ++z)
        *reinterpret_cast<f4v*>(&obuf[wave][col][(2 * g + z) * 16 + quad * 4]) = o[nt][2 * g + z] + x;
    }
    if (quad == 0) ml[wave][col][0] = m[nt], ml[wave][col][1] = ls;
    __syncthreads();
    const int oc = tid >> 4, ch0 = (tid & 15) * (DIM / 16);
    const int r = r0 + nt * 16 + oc;
    if (r < a.rows.q_len * a.group) {
      float top = kNegInf, f[kWaves], total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[w][oc][0]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = ml[w][oc][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ml[w][oc][0] - top);
        total = fmaf(f[w], ml[w][oc][1], total);
      }
      const int j = r / a.group, hq = h * a.group + r - j * a.group;
      const int64_t row = ((int64_t)i * a.rows.q_len + j) * a.heads + hq;
      float x[DIM / 16];
#pragma unroll
      for (int k = 0; k < DIM / 16; ++k) {
        x[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) x[k] = fmaf(f[w], obuf[w][oc][ch0 + k], x[k]);
      }
      if (splits == 1) {
        const int64_t at = (int64_t)i * a.os[0] + (int64_t)j * a.os[1] + (int64_t)hq * a.os[2] + ch0;
        const int pos = e.len - e.c + j;
        const bool none = r >= e.c * a.group || pos < sp.first || pos > sp.last || top == kNegInf;
#pragma unroll
        for (int k = 0; k < DIM / 16; ++k) store_elem<T>(a.out, at + k, none ? 0.0f : x[k] / total);
      } else {
        float* dst = a.ws + (row * splits + split) * DIM + ch0;
#pragma unroll
        for (int k = 0; k < DIM / 16; ++k) dst[k] = x[k];
        if ((tid & 15) == 0) {
          float* st = a.ws + part_floats + (row * splits + split) * 2;
          st[0] = top, st[1] = total;
        }
      }
    }
  }
}

// Joins the splits: one wave per query row.
template <int DIM, int T>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(KvAttend a, int cols, int chunk, int splits,
                                                               int64_t part_floats) {
  const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= (int64_t)a.rows.n * a.rows.q_len * a.heads) return;
  const int hq = (int)(row % a.heads);
  const int64_t ij = row / a.heads;
  const int j = (int)(ij % a.rows.q_len), i = (int)(ij / a.rows.q_len);
  const Entry e = load_entry(a.kv, a.rows, i);
  const int r = j * a.group + hq % a.group;
  const Span sp = block_span(a, e, r / cols * cols, cols);
  const int pos = e.len - e.c + j;
  const int used = j < e.c && pos >= sp.first && pos <= sp.last ? (sp.tiles + chunk - 1) / chunk : 0;
  const float* st = a.ws + part_floats + row * splits * 2;
  const float* src = a.ws + row * splits * DIM + lane * (DIM / 64);
  float top = kNegInf, total = 0.0f;
  for (int s = 0; s < used; ++s) top = fmaxf(top, st[2 * s]);
  float x[DIM / 64];
#pragma unroll
  for (int k = 0; k < DIM / 64; ++k) x[k] = 0.0f;
  for (int s = 0; s < used; ++s) {
    const float f = st[2 * s] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(st[2 * s] - top);
    total = fmaf(f, st[2 * s + 1], total);
#pragma unroll
    for (int k = 0; k < DIM / 64; ++k) x[k] = fmaf(f, src[(int64_t)s * DIM + k], x[k]);
  }
  const int64_t at = (int64_t)i * a.os[0] + (int64_t)j * a.os[1] + (int64_t)hq * a.os[2] + lane * (DIM / 64);
#pragma unroll
  for (int k = 0; k < DIM / 64; ++k) store_elem<T>(a.out, at + k, top == kNegInf ? 0.0f : x[k] / total);
}

int64_t part_floats_of(const KvAttend& a, int splits) {
  return (int64_t)a.rows.n * a.rows.q_len * a.heads * splits * a.kv.head_dim;
}

template <int DIM, int T, int NT>
hipError_t launch_nt(const KvAttend& a, const AttendPlan& p, const LaunchCtx& lc) {
  const int sh = __builtin_ctz((unsigned)a.kv.page_tokens);
  const int64_t grid = (int64_t)a.rows.n * a.kv.n_kv_heads * p.row_blocks * p.splits;
  const int64_t pf = part_floats_of(a, p.splits);
  QBL_LAUNCH((attend_kernel<DIM, T, NT>), dim3((unsigned)grid), dim3(kThreads), 0, lc, a, p.row_blocks, p.chunk, p.splits,
             sh, pf);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)a.rows.n * a.rows.q_len * a.heads;
  QBL_LAUNCH((attend_join_kernel<DIM, T>), dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(kThreads), 0, lc, a, p.cols,
             p.chunk, p.splits, pf);
  return hipGetLastError();
}

template <int DIM, int T>
hipError_t launch_type(const KvAttend& a, const AttendPlan& p, const LaunchCtx& lc) {
  if constexpr (DIM <= 128)
    if (p.cols == 32) return launch_nt<DIM, T, 2>(a, p, lc);
  return launch_nt<DIM, T, 1>(a, p, lc);
}

template <int DIM>
hipError_t launch_dim(const KvAttend& a, const AttendPlan& p, const LaunchCtx& lc) {
  switch (a.dtype) {
    case QBL_T_F32: return launch_type<DIM, QBL_T_F32>(a, p, lc);
    case QBL_T_F16: return launch_type<DIM, QBL_T_F16>(a, p, lc);
    case QBL_T_BF16: return launch_type<DIM, QBL_T_BF16>(a, p, lc);
  }
  return hipErrorInvalidValue;
}

}  // namespace

AttendPlan attend_plan(const KvAttend& a) {
  AttendPlan p;
  const int64_t rows = (int64_t)a.rows.q_len * a.group;
  // Two row blocks per workgroup read the cache once for both; 256 channels
  // leave registers for one only (two spill).
  p.cols = rows <= 16 || a.kv.head_dim == 256 ? 16 : 32;
  p.row_blocks = (int)((rows + p.cols - 1) / p.cols);
  // Tiles that a block of rows can see at most.
  const int64_t len = std::min<int64_t>(a.max_len, (int64_t)a.kv.max_pages * a.kv.page_tokens);
  int64_t tiles = (len + 31) / 32;
  if (a.window > 0) {
    const int64_t span = p.cols / a.group + 2 + std::min<int64_t>(a.window, len);
    tiles = std::min<int64_t>(tiles, (span + 62) / 32 + (std::min<int64_t>(a.sinks, len) + 31) / 32);
  }
  tiles = std::max<int64_t>(tiles, 1);
  // Enough workgroups to fill the device twice over, each wave at least one tile.
  const int64_t base = (int64_t)a.rows.n * a.kv.n_kv_heads * p.row_blocks;
  const int64_t want = std::min<int64_t>(std::max<int64_t>(1, 1024 / base), (tiles + kWaves - 1) / kWaves);
  p.chunk = (int)((tiles + want - 1) / want);
  p.splits = (int)((tiles + p.chunk - 1) / p.chunk);
  const int64_t out_rows = (int64_t)a.rows.n * a.rows.q_len * a.heads;
  p.ws_bytes = p.splits == 1 ? 0 : out_rows * p.splits * (a.kv.head_dim + 2) * 4;
  return p;
}

hipError_t launch_kv_attend(const KvAttend& a, const AttendPlan& p, const LaunchCtx& lc) {
  (void)hipGetLastError();  // drop errors left by earlier, unrelated calls
  switch (a.kv.head_dim) {
    case 64: return launch_dim<64>(a, p, lc);
    case 128: return launch_dim<128>(a, p, lc);
    case 256: return launch_dim<256>(a, p, lc);
  }
  return hipErrorInvalidValue;
}

}  // namespace qbl
