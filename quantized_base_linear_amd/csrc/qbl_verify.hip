// Verification of drafted tokens against the target's probabilities.
//
// Accept while u_j q_j(x_j) < p_j(x_j); at the first rejection a (or after the
// last accepted token) draw from w = max(p_a - q_a, 0) (or w = p_c) by
// inverting its cumulative sum at u * sum w.  Only one row of p and of q is
// read per request, once, so the work is bound by memory for many requests and
// by launch latency for one.
//
// First launch: workgroups of one 4096-token piece each find a (a few loads,
// repeated by every workgroup of the request) and sum their piece of w and of p
// in float64.  Second launch: one workgroup per request finds the piece that
// the draw falls into from those sums and reads that piece again.  Differences
// of two float32 values and their products are exact in float64, and sums of a
// row are within 2^-35 of exact, so the drawn token does not depend on the
// order of summation except with that probability.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qbl_cache_device.h"

namespace qbl {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 4096;
constexpr int kPer = kPiece / kThreads;

// A usable probability: finite and positive, anything else counts as 0.
__device__ __forceinline__ double weight(float x) { return x > 0.0f && x < __builtin_inff() ? (double)x : 0.0; }

struct Draw {
  int a;         // accepted tokens
  int rejected;  // 1: token a was rejected
  int token;     // the rejected token
};

// Every thread of the workgroup receives the request's outcome (kThreads >=
// QBL_KV_MAX_DRAFT: a thread per drafted token).
template <int T>
__device__ __forceinline__ Draw accept(const VerifyArgs& v, int b) {
  __shared__ int first;
  const int c = v.counts ? min(max(v.counts[b], 0), v.q_len) : v.q_len;
  const int j = threadIdx.x;
  if (j == 0) first = c;
  __syncthreads();
  if (j < c) {
    const int x = v.tokens[(int64_t)b * v.q_len + j];
    bool ok = x >= 0 && x < v.vocab;
    if (ok) {
      const double p = weight(load_elem<T>(v.target, b * v.ts[0] + j * v.ts[1] + x));
      const double q = v.draft ? weight(load_elem<T>(v.draft, b * v.ds[0] + j * v.ds[1] + x)) : 1.0;
      ok = (double)v.u[(int64_t)b * (v.q_len + 1) + j] * q < p;
    }
    if (!ok) atomicMin(&first, j);
  }
  __syncthreads();
  Draw d;
  d.a = first;
  d.rejected = d.a < c;
  d.token = d.rejected ? v.tokens[(int64_t)b * v.q_len + d.a] : -1;
  return d;
}

// p and w at token t of the row drawn from.
template <int T>
__device__ __forceinline__ void weights(const VerifyArgs& v, int b, const Draw& d, int t, double& p, double& w) {
  p = weight(load_elem<T>(v.target, b * v.ts[0] + d.a * v.ts[1] + t));
  w = p;
  if (d.rejected) {
    const double q = v.draft ? weight(load_elem<T>(v.draft, b * v.ds[0] + d.a * v.ds[1] + t)) : t == d.token ? 1.0 : 0.0;
    w = p > q ? p - q : 0.0;
  }
}

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) x += __shfl_xor(x, s);
  return x;
}

template <int T>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(VerifyArgs v, int pieces) {
  __shared__ double red[2][kThreads / 64];
  const int b = blockIdx.y, piece = blockIdx.x;
  const Draw d = accept<T>(v, b);
  double sw = 0.0, sp = 0.0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int t = piece * kPiece + k * kThreads + threadIdx.x;
    if (t < v.vocab) {
      double p, w;
      weights<T>(v, b, d, t, p, w);
      sw += w, sp += p;
    }
  }
  sw = wave_sum64(sw), sp = wave_sum64(sp);
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = sw, red[1][threadIdx.x >> 6] = sp;
  __syncthreads();
  if (threadIdx.x < 2) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) s += red[threadIdx.x][w];
    v.ws[((int64_t)b * pieces + piece) * 2 + threadIdx.x] = s;
  }
}

template <int T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyArgs v, int pieces) {
  __shared__ double red[kThreads / 64];
  __shared__ int hit, last, chosen, which;
  __shared__ double before;
  const int b = blockIdx.x, tid = threadIdx.x;
  const Draw d = accept<T>(v, b);
  const double* sums = v.ws + (int64_t)b * pieces * 2;
  if (tid == 0) {
    double tw = 0.0, tp = 0.0;
    for (int k = 0; k < pieces; ++k) tw += sums[2 * k], tp += sums[2 * k + 1];
    const int use = tw > 0.0 ? 0 : 1;  // nothing left of p - q: draw from p
    const double goal = (double)v.u[(int64_t)b * (v.q_len + 1) + v.q_len] * (use ? tp : tw);
    double c = 0.0, at = 0.0;
    int pick = -1;
    for (int k = 0; k < pieces; ++k) {
      const double s = sums[2 * k + use];
      if (s > 0.0) pick = k, at = c;  // the last piece with any weight, if none passes the goal
      c += s;
      if (s > 0.0 && c > goal) break;
    }
    chosen = pick, which = use, before = goal - at;
    hit = v.vocab, last = -1;
  }
  __syncthreads();
  const int pick = chosen;
  if (pick >= 0) {
    const double goal = before;
    double w[kPer], mine = 0.0;
    const int t0 = pick * kPiece + tid * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      w[k] = 0.0;
      if (t0 + k < v.vocab) {
        double p, x;
        weights<T>(v, b, d, t0 + k, p, x);
        w[k] = which ? p : x;
      }
      mine += w[k];
    }
    // exclusive prefix over the workgroup
    double x = mine;
    const int lane = tid & 63;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const double y = __shfl_up(x, s);
      if (lane >= s) x += y;
    }
    if (lane == 63) red[tid >> 6] = x;
    __syncthreads();
    double c = x - mine;
    for (int k = 0; k < (tid >> 6); ++k) c += red[k];
    int first = v.vocab, end = -1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      c += w[k];
      if (w[k] > 0.0) {
        end = t0 + k;
        if (first == v.vocab && c > goal) first = t0 + k;
      }
    }
    if (first < v.vocab) atomicMin(&hit, first);
    if (end >= 0) atomicMax(&last, end);
  }
  __syncthreads();
  if (tid == 0) {
    v.accepted[b] = d.a;
    v.next[b] = hit < v.vocab ? hit : last;
  }
}

template <int T>
hipError_t launch_type(const VerifyArgs& a, const LaunchCtx& lc) {
  const int pieces = (a.vocab + kPiece - 1) / kPiece;
  QBL_LAUNCH(verify_sum_kernel<T>, dim3((unsigned)pieces, (unsigned)a.n), dim3(kThreads), 0, lc, a, pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  QBL_LAUNCH(verify_pick_kernel<T>, dim3((unsigned)a.n), dim3(kThreads), 0, lc, a, pieces);
  return hipGetLastError();
}

}  // namespace

int64_t verify_ws_bytes(int n, int vocab) { return (int64_t)n * ((vocab + kPiece - 1) / kPiece) * 2 * 8; }

hipError_t launch_verify(const VerifyArgs& a, const LaunchCtx& lc) {
  (void)hipGetLastError();  // drop errors left by earlier, unrelated calls
  switch (a.dtype) {
    case QBL_T_F32: return launch_type<QBL_T_F32>(a, lc);
    case QBL_T_F16: return launch_type<QBL_T_F16>(a, lc);
    case QBL_T_BF16: return launch_type<QBL_T_BF16>(a, lc);
  }
  return hipErrorInvalidValue;
}

}  // namespace qbl
