// Row kernels over logits: the label's log-probability and the entropy, the
// logits' gradient, and the policy objective that does both at once.
//
// For one row x with label y and inverse temperature s:
//   m = max x,  z = log sum exp(s (x - m)),  log p_v = s (x_v - m) - z,
//   H = z - sum e_v s (x_v - m) / sum e_v,   e_v = exp(s (x_v - m)),
//   dx_v = s (g (1[v = y] - p_v) - gH p_v (log p_v + H)).
// m is the maximum of the raw logits and z is kept beside it: their
// difference from a logit is exact enough for any size of logit, where
// s x - (s m + z) would lose the digits that s m holds.  exp is taken as
// exp2(c (x - m)), c = s log2 e, on the hardware's exp2.
//
// One pass with the running maximum m, t = sum e and w = sum e (x - m): when
// the maximum rises by d, e shrinks by f = exp2(-c d), so
//   w <- f (w - d t),  t <- f t.
//
// HBM-bound: the forward reads each scored row once; the gradient also writes
// each row once.  Rows of an odd V start at any element, so a group of 8
// logits is loaded at its element's alignment.
#include "objective.h"

namespace qlora {
namespace {

// A launch holds less than 2^32 threads: workgroups go round the rows.
constexpr int64_t kMaxBlocks = int64_t(1) << 21;
constexpr float kLog2e = 1.44269504088896340736f;

// 8 consecutive elements at element alignment.
template <bool BF16>
struct Row {
  const char *p;
  __device__ __forceinline__ Row(const void *x, int64_t at)
      : p(static_cast<const char *>(x) + at * (BF16 ? 2 : 4)) {}
  __device__ __forceinline__ void load8(int64_t v, float (&e)[8]) const {
    if (BF16) {
      u32x4_t u;
      __builtin_memcpy(&u, p + v * 2, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[2 * i] = bf16_lo_to_f32(u[i]);
        e[2 * i + 1] = bf16_hi_to_f32(u[i]);
      }
    } else {
      __builtin_memcpy(e, p + v * 4, 32);
    }
  }
  __device__ __forceinline__ float load1(int64_t v) const {
    if (BF16) {
      uint16_t h;
      __builtin_memcpy(&h, p + v * 2, 2);
      return __uint_as_float(uint32_t(h) << 16);
    }
    float f;
    __builtin_memcpy(&f, p + v * 4, 4);
    return f;
  }
  // the group's elements, -inf past the row's end
  __device__ __forceinline__ void load(int64_t v, int64_t V, float (&e)[8]) const {
    if (v + 8 <= V) {
      load8(v, e);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = v + i < V ? load1(v + i) : -INFINITY;
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void store(void *x, int64_t at, int64_t left, const float (&e)[8]) {
  if (BF16) {
    char *p = static_cast<char *>(x) + at * 2;
    const u32x4_t u = {pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                       pack_bf16x2(e[6], e[7])};
    if (left >= 8) {
      __builtin_memcpy(p, &u, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) {
          const uint16_t h = uint16_t(u[i / 2] >> (16 * (i % 2)));
          __builtin_memcpy(p + 2 * i, &h, 2);
        }
    }
  } else {
    char *p = static_cast<char *>(x) + at * 4;
    if (left >= 8) {
      __builtin_memcpy(p, e, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) __builtin_memcpy(p + 4 * i, &e[i], 4);
    }
  }
}

struct Stat {
  float m, t, w;   // maximum, sum e, sum e (x - m)
};

// a's sums brought to the maximum `top` (>= a.m); nothing seen yet is
// m = -inf, t = w = 0 and stays so.
__device__ __forceinline__ Stat raised(const Stat &a, float top, float c) {
  const float d = a.m - top;                      // <= 0, or NaN from -inf - -inf
  if (!(a.m > -INFINITY)) return {top, a.t, a.w};
  const float f = __builtin_amdgcn_exp2f(c * d);
  // a maximum that rose by an infinite step leaves nothing (0 * inf)
  return {top, f * a.t, f > 0.0f ? f * (a.w + d * a.t) : 0.0f};
}

__device__ __forceinline__ Stat joined(const Stat &a, const Stat &b, float c) {
  const float top = fmaxf(a.m, b.m);
  const Stat x = raised(a, top, c), y = raised(b, top, c);
  return {top, x.t + y.t, x.w + y.w};
}

__device__ __forceinline__ void add8(Stat &a, const float (&e)[8], float c) {
  float top = a.m;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, e[i]);
  a = raised(a, top, c);
  // a group of nothing but -inf: differences from 0, every e is 0
  const float base = top > -INFINITY ? top : 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = e[i] - base;
    const float q = __builtin_amdgcn_exp2f(c * d);
    a.t += q;
    a.w += q > 0.0f ? q * d : 0.0f;
  }
}

// A NaN logit is skipped by the maximum but not by the sum: t becomes NaN.
template <int threads>
__device__ __forceinline__ Stat block_stat(Stat a, float c, Stat *red) {
  __syncthreads();   // the previous row's results have been read
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const Stat b = {__shfl_xor(a.m, o), __shfl_xor(a.t, o), __shfl_xor(a.w, o)};
    a = joined(a, b, c);
  }
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = a;
  __syncthreads();
  a = red[0];
#pragma unroll
  for (int w = 1; w < threads / 64; ++w) a = joined(a, red[w], c);
  return a;
}

template <bool BF16, int threads>
__device__ __forceinline__ Stat row_stat(const Row<BF16> &row, int64_t V, float c, Stat *red) {
  Stat s = {-INFINITY, 0.0f, 0.0f};
  for (int64_t v = int64_t(threadIdx.x) * 8; v < V; v += threads * 8) {
    float e[8];
    row.load(v, V, e);
    add8(s, e, c);
  }
  return block_stat<threads>(s, c, red);
}

struct RowResult {
  float m, z, logp, ent;
};

// Results of a row from its sums and its label's logit.
__device__ __forceinline__ RowResult row_result(const Stat &a, float xy, float scale) {
  if (a.t != a.t) return {a.t, a.t, a.t, a.t};
  if (!(a.m > -INFINITY)) return {-INFINITY, 0.0f, -INFINITY, 0.0f};
  const float z = logf(a.t);
  return {a.m, z, scale * (xy - a.m) - z, z - scale * (a.w / a.t)};
}

template <bool BF16, int threads>
__global__ __launch_bounds__(threads) void logp_fwd_kernel(LogitRows a, float *logp, float *stats,
                                                           float *entropy) {
  __shared__ Stat red[threads / 64];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t y = a.labels[t];
    RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
    if (y >= 0 && y < a.V) {
      const Row<BF16> row(a.x, t * a.ld);
      const Stat s = row_stat<BF16, threads>(row, a.V, a.scale * kLog2e, red);
      if (threadIdx.x == 0) r = row_result(s, row.load1(y), a.scale);
    }
    if (threadIdx.x == 0) {
      logp[t] = r.logp;
      stats[2 * t] = r.m;
      stats[2 * t + 1] = r.z;
      if (entropy) entropy[t] = r.ent;
    }
  }
}

// The gradient of 8 logits: d = s (g (1[v = y] - p) - gh p (log p + H)).
__device__ __forceinline__ void grad8(float (&e)[8], int64_t v, int64_t y, float scale, float m,
                                      float z, float g, float gh, float ent) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lp = scale * (e[i] - m) - z;
    const float p = __builtin_amdgcn_exp2f(lp * kLog2e);
    float d = (v + i == y ? g : 0.0f) - g * p;
    if (gh != 0.0f) d -= p > 0.0f ? gh * (p * (lp + ent)) : gh * p;
    e[i] = scale * d;
  }
}

template <bool BF16, int threads>
__device__ __forceinline__ void grad_row(const Row<BF16> &row, void *dx, int64_t at, int64_t V,
                                         int64_t y, float scale, float m, float z, float g,
                                         float gh, float ent, bool live) {
  for (int64_t v = int64_t(threadIdx.x) * 8; v < V; v += threads * 8) {
    float e[8] = {};
    if (live) {
      row.load(v, V, e);
      grad8(e, v, y, scale, m, z, g, gh, ent);
    }
    store<BF16>(dx, at + v, V - v, e);
  }
}

template <bool BF16, int threads>
__global__ __launch_bounds__(threads) void logp_bwd_kernel(LogitRows a, const float *stats,
                                                           const float *entropy, const float *g,
                                                           const float *g_entropy, void *dx,
                                                           int64_t ldd) {
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t y = a.labels[t];
    const float m = stats[2 * t], z = stats[2 * t + 1];
    const bool live = y >= 0 && y < a.V && m != -INFINITY;
    const Row<BF16> row(a.x, t * a.ld);
    grad_row<BF16, threads>(row, dx, t * ldd, a.V, y, a.scale, m, z, g[t],
                            g_entropy ? g_entropy[t] : 0.0f, entropy ? entropy[t] : 0.0f, live);
  }
}

// The policy objective from a row's logits to their gradient: the row's
// coefficient depends on the row alone, so the gradient follows in the same
// workgroup.
template <bool BF16, int threads>
__global__ __launch_bounds__(threads) void policy_logits_kernel(LogitRows a, PolicyTokens k,
                                                                PolicyParams p, float *terms,
                                                                float *logp, void *dx,
                                                                int64_t ldd) {
  __shared__ Stat red[threads / 64];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t y = a.labels[t];
    const float w = k.weight ? k.weight[t] : 1.0f;
    const Row<BF16> row(a.x, t * a.ld);
    bool live = y >= 0 && y < a.V && w != 0.0f;
    float g = 0.0f;
    RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4_t term = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
      // read before the workgroup's barriers, so before dx may overwrite it
      const float xy = row.load1(y);
      const Stat s = row_stat<BF16, threads>(row, a.V, a.scale * kLog2e, red);
      r = row_result(s, xy, a.scale);
      const PolicyToken q = policy_token(p, k, t, r.logp, r.ent);
      term = f32x4_t{w * q.loss, w * q.k, w * q.bound, w * r.ent};
      g = w * q.dlogp;
      live = r.m != -INFINITY;
    }
    grad_row<BF16, threads>(row, dx, t * ldd, a.V, y, a.scale, r.m, r.z, g, -p.ent * w, r.ent,
                            live);
    if (threadIdx.x == 0) {
      reinterpret_cast<f32x4_t *>(terms)[t] = term;
      if (logp) logp[t] = r.logp;
    }
  }
}

__global__ __launch_bounds__(1024) void sum4_kernel(const float *terms, int64_t n, float *out) {
  __shared__ double red[16];
  double s[4] = {};
  for (int64_t i = threadIdx.x; i < n; i += 1024) {
    const f32x4_t v = reinterpret_cast<const f32x4_t *>(terms)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += v[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double v = block_sum<1024>(s[j], red);
    if (threadIdx.x == 0) out[j] = float(v);
  }
}

}  // namespace

hipError_t launch_logp_fwd(const LogitRows &a, float *logp, float *stats, float *entropy,
                           hipStream_t s) {
  const dim3 grid{unsigned(min64(a.T, kMaxBlocks))};
  if (a.bf16)
    hipLaunchKernelGGL((logp_fwd_kernel<true, 256>), grid, dim3(256), 0, s, a, logp, stats,
                       entropy);
  else
    hipLaunchKernelGGL((logp_fwd_kernel<false, 256>), grid, dim3(256), 0, s, a, logp, stats,
                       entropy);
  return hipGetLastError();
}

hipError_t launch_logp_bwd(const LogitRows &a, const float *stats, const float *entropy,
                           const float *g, const float *g_entropy, void *dx, int64_t ldd,
                           hipStream_t s) {
  const dim3 grid{unsigned(min64(a.T, kMaxBlocks))};
  if (a.bf16)
    hipLaunchKernelGGL((logp_bwd_kernel<true, 256>), grid, dim3(256), 0, s, a, stats, entropy, g,
                       g_entropy, dx, ldd);
  else
    hipLaunchKernelGGL((logp_bwd_kernel<false, 256>), grid, dim3(256), 0, s, a, stats, entropy, g,
                       g_entropy, dx, ldd);
  return hipGetLastError();
}

hipError_t launch_policy_logits(const LogitRows &a, const PolicyTokens &t,
                                const PolicyParams &p, float *terms, float *logp, void *dx,
                                int64_t ldd, hipStream_t s) {
  const dim3 grid{unsigned(min64(a.T, kMaxBlocks))};
  if (a.bf16)
    hipLaunchKernelGGL((policy_logits_kernel<true, 256>), grid, dim3(256), 0, s, a, t, p, terms,
                       logp, dx, ldd);
  else
    hipLaunchKernelGGL((policy_logits_kernel<false, 256>), grid, dim3(256), 0, s, a, t, p, terms,
                       logp, dx, ldd);
  return hipGetLastError();
}

hipError_t launch_sum4(const float *terms, int64_t n, float *out, hipStream_t s) {
  hipLaunchKernelGGL(sum4_kernel, dim3(1), dim3(1024), 0, s, terms, n, out);
  return hipGetLastError();
}

}  // namespace qlora
