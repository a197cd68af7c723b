// Row kernels over logits: the label's log-probability and the entropy, the
// logits' gradient, and the policy objective that does both at once.
//
// For one row x with label y and inverse temperature s, c = s log2 e:
//   m = max x,  L_v = c (x_v - m),  e_v = exp2(L_v),
//   t = sum e,  w = sum e L,
//   z = ln t,  log p_v = s (x_v - m) - z,  H = z - ln 2 w / t,
//   dx_v = s (g (1[v = y] - p_v) - gH p_v (log p_v + H)).
// m is the maximum of the raw logits and z is kept beside it: their
// difference from a logit is exact enough for any size of logit, where
// s x - (s m + z) would lose the digits that s m holds.
//
// Sums taken against one maximum are brought to a higher one: with L' = L + d
// and f = exp2(d), t' = f t and w' = f (w + d t).
//
// HBM-bound: the forward reads each scored row once, the gradient also writes
// each row once.  Measured with a quarter of the rows not scored: the forward
// with entropy of 4096 x 32000 bf16 38.7 us (5.1 TB/s), its gradient 73.8 us
// (6.2 TB/s), the policy objective of 8192 x 32000 bf16 162 to 170 us (5.4 to
// 5.6 TB/s) and 6 us for the sums; a 1 GiB device copy moves 5.2 TB/s on the
// same card.
//
// Rows of an odd V start at any element: a row is cut into the words before its
// first 16-byte boundary, groups of 16 bytes, and the words after the last
// whole group (up to 7 of either in bf16, 3 in fp32).
#include "logits.h"

namespace qlora {
namespace {

template <bool BF16, bool ENT, int threads, int NG>
__global__ __launch_bounds__(threads) void logp_fwd_kernel(LogitRows a, float *logp,
                                                           float *stats, float *entropy) {
  __shared__ Stat red[threads / 64];
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int64_t y = a.labels[t];
  RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
  if (y >= 0 && y < a.V) {
    Held<BF16, threads, NG> h;
    r = row_stat<ENT, false>(h, row_at<BF16>(a.x, t * a.ld), int32_t(a.V), int32_t(y), a.scale,
                             red);
  }
  if (threadIdx.x == 0) {
    logp[t] = r.logp;
    stats[2 * t] = r.m;
    stats[2 * t + 1] = r.z;
    if (ENT) entropy[t] = r.ent;
  }
}

// One segment of threads * 8 * NG words of a row's gradient to a workgroup.
template <bool BF16, bool ENT, int threads, int NG>
__global__ __launch_bounds__(threads) void logp_bwd_kernel(LogitRows a, const float *stats,
                                                           const float *entropy, const float *g,
                                                           const float *g_entropy, void *dx,
                                                           int64_t ldd) {
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int32_t V = int32_t(a.V);
  const float c = a.scale * kLog2e;
  const char *row = row_at<BF16>(a.x, t * a.ld);
  char *out = row_at<BF16>(dx, t * ldd);
  const Cut<BF16> q(row, V);
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  const int32_t from = (int32_t(blockIdx.x) * threads * G + int32_t(threadIdx.x)) * W;
  const int32_t one = blockIdx.x == 0 ? q.one(int32_t(threadIdx.x)) : V;
  const int64_t y = a.labels[t];
  const float m = stats[2 * t], z = stats[2 * t + 1];
  const float gt = g[t], gh = ENT ? g_entropy[t] : 0.0f;
  if (y >= 0 && y < V && m != -INFINITY && (gt != 0.0f || gh != 0.0f)) {
    float f[G][W];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (from + i * threads * W < q.whole)
        unpack<BF16>(load_group<BF16>(row, q.head + from + i * threads * W), f[i]);
    const GradCoef k = grad_coef(a.scale, gt, gh, ENT ? entropy[t] : 0.0f, z);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int32_t v = q.head + from + i * threads * W;
      if (from + i * threads * W < q.whole) {
        grad<ENT>(f[i], int32_t(y) - v, m, c, k);
        store_group<BF16>(out, v, f[i]);
      }
    }
    if (one < V) {
      float d[1] = {load1<BF16>(row, one)};
      grad<ENT>(d, int32_t(y) - one, m, c, k);
      store1<BF16>(out, one, d[0]);
    }
  } else {
    const float e[W] = {};
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (from + i * threads * W < q.whole)
        store_group<BF16>(out, q.head + from + i * threads * W, e);
    if (one < V) store1<BF16>(out, one, 0.0f);
  }
}

// The gradient of a row.  h holds its last chunk (ONE: the row); the words
// before that are read again, each by the lane that then overwrites it.
template <bool ENT, bool ONE, bool BF16, int threads, int NG>
__device__ __forceinline__ void row_grad(Held<BF16, threads, NG> &h, const char *row, char *out,
                                         int32_t V, int32_t y, float m, float c,
                                         const GradCoef &k) {
  const Cut<BF16> q(row, V);
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  const int32_t from = ONE || q.whole <= h.words ? 0 : q.whole - h.words;
  h.keep();
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int32_t v = from + h.first(i);
    if (v < q.whole) {
      float e[W];
      unpack<BF16>(h.q[i], e);
      grad<ENT>(e, y - q.head - v, m, c, k);
      store_group<BF16>(out, q.head + v, e);
    }
    // one group's words unpacked at a time
    __builtin_amdgcn_sched_barrier(0);
  }
  if (!ONE) {
    for (int32_t v = int32_t(threadIdx.x) * W; v < from; v += threads * W) {
      float e[W];
      unpack<BF16>(load_group<BF16>(row, q.head + v), e);
      grad<ENT>(e, y - q.head - v, m, c, k);
      store_group<BF16>(out, q.head + v, e);
    }
  }
  const int32_t one = q.one(int32_t(threadIdx.x));
  if (one < V) {
    float d[1] = {ONE ? h.one : load1<BF16>(row, one)};
    grad<ENT>(d, y - one, m, c, k);
    store1<BF16>(out, one, d[0]);
  }
}

// The policy objective from a row's logits to their gradient: the row's
// coefficient depends on the row alone, so the gradient follows from the
// registers that gave the sums.  Every logit has been read before the barrier
// of the sums, so dx may be the logits.
template <bool BF16, bool ENT, bool ONE, int threads, int NG>
__global__ __launch_bounds__(threads) void policy_logits_kernel(
    LogitRows a, PolicyTokens k, PolicyParams p, float *terms, float *logp, void *dx,
    int64_t ldd) {
  __shared__ Stat red[threads / 64];
  const int32_t V = int32_t(a.V);
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int64_t y = a.labels[t];
  const float w = k.weight ? k.weight[t] : 1.0f;
  const char *row = row_at<BF16>(a.x, t * a.ld);
  char *out = row_at<BF16>(dx, t * ldd);
  RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4_t term = {0.0f, 0.0f, 0.0f, 0.0f};
  bool some = false;
  if (y >= 0 && y < V && w != 0.0f) {
    Held<BF16, threads, NG> h;
    r = row_stat<true, ONE>(h, row, V, int32_t(y), a.scale, red);
    const PolicyToken q = policy_token(p, r.logp, r.ent, k.adv ? k.adv[t] : 1.0f,
                                       k.old ? r.logp - k.old[t] : 0.0f, k.ref,
                                       k.ref ? k.ref[t] : 0.0f);
    term = f32x4_t{w * q.loss, w * q.k, w * q.bound, w * r.ent};
    const float g = w * q.dlogp, gh = -p.ent * w;
    some = r.m != -INFINITY && (g != 0.0f || gh != 0.0f);
    if (some) {
      const GradCoef kc = grad_coef(a.scale, g, gh, ENT ? r.ent : 0.0f, r.z);
      row_grad<ENT, ONE>(h, row, out, V, int32_t(y), r.m, a.scale * kLog2e, kc);
    }
  }
  if (!some) zero_row<BF16, threads>(out, V);
  if (threadIdx.x == 0) {
    reinterpret_cast<f32x4_t *>(terms)[t] = term;
    if (logp) logp[t] = r.logp;
  }
}

template <bool BF16>
__global__ __launch_bounds__(64) void logp_join_kernel(LogitRows a, const Stat *part, int segments,
                                                       float *logp, float *stats,
                                                       float *entropy) {
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int64_t y = a.labels[t];
  RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
  if (y >= 0 && y < a.V) r = join_row<BF16>(a, part, segments, t, y);
  if (threadIdx.x == 0) {
    logp[t] = r.logp;
    stats[2 * t] = r.m;
    stats[2 * t + 1] = r.z;
    if (entropy) entropy[t] = r.ent;
  }
}

// Also the token's objective: what logp_bwd_kernel needs of it, and its terms.
template <bool BF16>
__global__ __launch_bounds__(64) void policy_join_kernel(LogitRows a, PolicyTokens k,
                                                         PolicyParams p, const Stat *part,
                                                         int segments, PolicySplit o,
                                                         float *terms, float *logp) {
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int64_t y = a.labels[t];
  const float w = k.weight ? k.weight[t] : 1.0f;
  RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4_t term = {0.0f, 0.0f, 0.0f, 0.0f};
  float g = 0.0f, gh = 0.0f;
  if (y >= 0 && y < a.V && w != 0.0f) {
    r = join_row<BF16>(a, part, segments, t, y);
    const PolicyToken q = policy_token(p, r.logp, r.ent, k.adv ? k.adv[t] : 1.0f,
                                       k.old ? r.logp - k.old[t] : 0.0f, k.ref,
                                       k.ref ? k.ref[t] : 0.0f);
    term = f32x4_t{w * q.loss, w * q.k, w * q.bound, w * r.ent};
    g = w * q.dlogp;
    gh = -p.ent * w;
  }
  if (threadIdx.x == 0) {
    reinterpret_cast<f32x4_t *>(terms)[t] = term;
    if (logp) logp[t] = r.logp;
    o.stats[2 * t] = r.m;
    o.stats[2 * t + 1] = r.z;
    o.entropy[t] = r.ent;
    o.g[t] = g;
    o.gh[t] = gh;
  }
}

}  // namespace

// A second launch costs about 3 us.  Measured, us a call back to back, cut and
// whole (T = 1 / 64): V = 131072 bf16 (256 KiB a row) 10.2 / 10.2, 8.8 / 10.1;
// V = 200000 fp32 (800 KB) 10.0 / 13.5, 12.3 / 14.6.
int64_t forward_segments(int64_t T, int64_t V, bool bf16) {
  return T <= kFewRows && V * (bf16 ? 2 : 4) > (int64_t(256) << 10) ? segments_of(V) : 0;
}

// Rows that a workgroup would have to read twice.  Cut and whole (T = 1 / 64 /
// 128): V = 70000 bf16 18.7 / 18.5 / 22.1, 18.6 / 19.4 / 20.1; V = 131072 bf16
// 17.5 / 20.6 / 27.9, 22.5 / 23.9 / 25.6; V = 200000 fp32 18.0 / 34.9 / 57.9,
// 33.3 / 40.0 / 51.6.
int64_t policy_segments(int64_t T, int64_t V) {
  return T <= kFewRows && V > 65536 ? segments_of(V) : 0;
}

namespace {

// Lanes and groups to a row.  A lane wants 4 to 8 groups of 8 words in flight,
// and every wavefront of a row repeats the row's last reductions, so a row
// takes the fewest wavefronts that hold it so.  Measured, us (V, T; bf16):
//   V = 4000, T = 16384:  64 x 4 23.0   64 x 8 23.9   128 x 4 28.3
//   V = 8000, T = 8192:   128 x 8 21.2  64 x 8 22.3   256 x 4 22.8
//   V = 16000, T = 8192:  256 x 8 39.1  64 x 8 42.6   256 x 4 41.9
//   V = 32000, T = 4096:  512 x 8 37.9  64 x 8 41.0   512 x 4 40.8
template <bool BF16, bool ENT>
void logp_fwd(const LogitRows &a, float *logp, float *stats, float *entropy, float *part,
              hipStream_t s) {
  if (const int64_t n = forward_segments(a.T, a.V, BF16)) {
    Stat *q = reinterpret_cast<Stat *>(part);
    hipLaunchKernelGGL((part_kernel<BF16, ENT>), row_grid(a.T, n), dim3(kPartThreads), 0, s, a,
                       nullptr, q);
    hipLaunchKernelGGL((logp_join_kernel<BF16>), row_grid(a.T), dim3(64), 0, s, a, q, int(n),
                       logp, stats, entropy);
    return;
  }
#define ROWS(threads, NG)                                                                     \
  hipLaunchKernelGGL((logp_fwd_kernel<BF16, ENT, threads, NG>), row_grid(a.T), dim3(threads), \
                     0, s, a, logp, stats, entropy)
  if (a.V <= 4096) ROWS(64, 4);
  else if (a.V <= 8192) ROWS(128, 8);
  else if (a.V <= 16384) ROWS(256, 8);
  else ROWS(512, 8);
#undef ROWS
}

// Two groups of 16 bytes to a lane.  us, one / two / four groups: bf16, T =
// 4096, V = 32000 86.3 / 74.2 / 82.1; fp32, T = 509, V = 50001, two / four /
// eight 36.1 / 37.5 / 38.6.
template <bool BF16, bool ENT>
void logp_bwd(const LogitRows &a, const float *stats, const float *entropy, const float *g,
              const float *g_entropy, void *dx, int64_t ldd, hipStream_t s) {
  constexpr int threads = 256, NG = BF16 ? 2 : 1;
  const int64_t segments = (a.V + threads * 8 * NG - 1) / (threads * 8 * NG);
  hipLaunchKernelGGL((logp_bwd_kernel<BF16, ENT, threads, NG>), row_grid(a.T, segments),
                     dim3(threads), 0, s, a, stats, entropy, g, g_entropy, dx, ldd);
}

// As in logp_fwd, but the row has to stay in registers, up to 65536 words
// (1024 lanes of 8 groups).  Measured, us (bf16, a quarter of the rows dead):
//   V = 4000, T = 16384:  128 x 4 48.7  64 x 8 48.1   256 x 2 57.3
//   V = 8000, T = 8192:   256 x 4 45.9  128 x 8 45.7  64 x 8 49.5
//   V = 16000, T = 8192:  512 x 4 86.6  256 x 8 86.1  128 x 8 99.4
//   V = 32000, T = 4096:  512 x 8 88.6  512 x 4 90.8  1024 x 4 98.6
//   V = 60000, T = 1024:  1024 x 8 46.9, read in part twice by 512 x 8 46.0
//   V = 131072, T = 1024: 1024 x 8 102, 512 x 8 112
template <bool BF16, bool ENT>
void policy_logits(const LogitRows &a, const PolicyTokens &t, const PolicyParams &p, float *terms,
                   float *logp, void *dx, int64_t ldd, const PolicySplit &o, hipStream_t s) {
  if (const int64_t n = policy_segments(a.T, a.V)) {
    Stat *q = reinterpret_cast<Stat *>(o.part);
    hipLaunchKernelGGL((part_kernel<BF16, true>), row_grid(a.T, n), dim3(kPartThreads), 0, s, a,
                       t.weight, q);
    hipLaunchKernelGGL((policy_join_kernel<BF16>), row_grid(a.T), dim3(64), 0, s, a, t, p, q,
                       int(n), o, terms, logp);
    logp_bwd<BF16, ENT>(a, o.stats, o.entropy, o.g, o.gh, dx, ldd, s);
    return;
  }
#define ROWS(ONE, threads, NG)                                                            \
  hipLaunchKernelGGL((policy_logits_kernel<BF16, ENT, ONE, threads, NG>), row_grid(a.T), \
                     dim3(threads), 0, s, a, t, p, terms, logp, dx, ldd)
  if (a.V <= 2048) ROWS(true, 64, 4);
  else if (a.V <= 4096) ROWS(true, 128, 4);
  else if (a.V <= 8192) ROWS(true, 256, 4);
  else if (a.V <= 16384) ROWS(true, 512, 4);
  else if (a.V <= 32768) ROWS(true, 512, 8);
  else if (a.V <= 65536) ROWS(true, 1024, 8);
  else ROWS(false, 1024, 8);
#undef ROWS
}

}  // namespace

hipError_t launch_logp_fwd(const LogitRows &a, float *logp, float *stats, float *entropy,
                           float *part, hipStream_t s) {
#define GO(B) (entropy ? logp_fwd<B, true>(a, logp, stats, entropy, part, s) \
                       : logp_fwd<B, false>(a, logp, stats, entropy, part, s))
  a.bf16 ? GO(true) : GO(false);
#undef GO
  return hipGetLastError();
}

hipError_t launch_logp_bwd(const LogitRows &a, const float *stats, const float *entropy,
                           const float *g, const float *g_entropy, void *dx, int64_t ldd,
                           hipStream_t s) {
#define GO(B) (entropy ? logp_bwd<B, true>(a, stats, entropy, g, g_entropy, dx, ldd, s) \
                       : logp_bwd<B, false>(a, stats, entropy, g, g_entropy, dx, ldd, s))
  a.bf16 ? GO(true) : GO(false);
#undef GO
  return hipGetLastError();
}

hipError_t launch_policy_logits(const LogitRows &a, const PolicyTokens &t,
                                const PolicyParams &p, float *terms, float *logp, void *dx,
                                int64_t ldd, const PolicySplit &o, hipStream_t s) {
#define GO(B) (p.ent != 0.0f ? policy_logits<B, true>(a, t, p, terms, logp, dx, ldd, o, s) \
                             : policy_logits<B, false>(a, t, p, terms, logp, dx, ldd, o, s))
  a.bf16 ? GO(true) : GO(false);
#undef GO
  return hipGetLastError();
}

}  // namespace qlora
