// Pieces the objectives and the dropout share: the policy objective of one
// token, stores past the caches, and workgroup sums in a fixed order.
#pragma once

#include "device.h"

namespace qlora {

__host__ __device__ __forceinline__ int64_t least64(int64_t a, int64_t b) { return a < b ? a : b; }

// 16 bytes at an element's alignment past the caches' usual order, for large
// results that are read once, later.  Alone and with a reader of the result
// behind it (us; the gradient of T x 32000 bf16 logits, T = 1024 / 2048 /
// 4096): 21.6 / 46.4 / 87.2 and 39.5 / 70.9 / 132, ordinary stores 26.8 / 47.8
// / 89.9 and 38.8 / 71.2 / 143.
__device__ __forceinline__ void store16_past(void *p, u32x4_t v) {
  typedef u32x4_t any_u32x4_t __attribute__((aligned(2)));
  __builtin_nontemporal_store(v, static_cast<any_u32x4_t *>(p));
}

// k = e^q - q - 1, em = e^q - 1.  Near 0 the difference em - q would keep only
// the digits of em past those of q, so k is summed from its series (|q| < 1/2:
// the first term left out is q^9 / 9!, 2^-24.2 of k at most); where e^q is past
// fp32 k is infinite, also for an infinite q.
__device__ __forceinline__ float kl_estimate(float q, float em) {
  float s = __builtin_fmaf(q, 1.0f / 40320.0f, 1.0f / 5040.0f);
  s = __builtin_fmaf(q, s, 1.0f / 720.0f);
  s = __builtin_fmaf(q, s, 1.0f / 120.0f);
  s = __builtin_fmaf(q, s, 1.0f / 24.0f);
  s = __builtin_fmaf(q, s, 1.0f / 6.0f);
  s = __builtin_fmaf(q, s, 0.5f);
  const float far = em < INFINITY ? em - q : em;
  return fabsf(q) < 0.5f ? q * q * s : far;
}

// v times its coefficient c: 0 where c is 0, also for an infinite or NaN v
// (one instruction; with values selected beside ordinary products the policy
// loss of 8000 tokens took 8.6 us, not 8.1).
__device__ __forceinline__ float scaled(float c, float v) {
  float r;
  asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(r) : "v"(c), "v"(v));
  return r;
}

struct PolicyToken {
  float loss, k, bound;   // -f + kl k - ent H, the KL estimate, [a bound holds]
  float dlogp;            // d loss / d logp (that of the entropy is -ent)
};

// One token of the objective (qlora_policy_loss in qlora.h has the formulas),
// d = logp - old or 0.  The branch is chosen on d against rounded logs of the
// bounds: d is one fp32 subtraction, so the choice does not hang on how exp
// rounds.
__device__ __forceinline__ PolicyToken policy_token(const PolicyParams &p, float logp, float ent,
                                                    float adv, float d, bool has_ref,
                                                    float ref) {
  PolicyToken t;
  float f = scaled(adv, logp), df = adv;
  t.bound = 0.0f;
  if (p.clip) {
    df = scaled(adv, expf(d));
    f = df;
    if (adv > 0.0f && d > p.log_hi) { f = p.hi * adv; t.bound = 1.0f; }
    if (adv < 0.0f && d < p.log_lo) { f = p.lo * adv; t.bound = 1.0f; }
    if (adv < 0.0f && d > p.log_dual) { f = p.dual * adv; t.bound = 1.0f; }
    if (t.bound != 0.0f) df = 0.0f;
  }
  t.loss = -f;
  t.dlogp = -df;
  t.k = 0.0f;
  if (has_ref) {
    const float q = ref - logp, em = expm1f(q);
    t.k = kl_estimate(q, em);
    t.loss += scaled(p.kl, t.k);
    t.dlogp -= scaled(p.kl, em);
  }
  if (p.ent != 0.0f) t.loss -= p.ent * ent;
  return t;
}

// Sum (maximum) over a wavefront's 64 lanes through data-parallel moves within
// rows of 16 lanes and broadcasts between rows: six dependent vector
// instructions, no LDS.  The total is in lane 63 and is returned as a scalar.
template <int ctrl, int rows>
__device__ __forceinline__ float dpp(float fill, float v) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_update_dpp(
      int(__float_as_uint(fill)), int(__float_as_uint(v)), ctrl, rows, 0xf, false)));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), 63)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xf>(0.0f, v);   // from 1, 2, 4 and 8 lanes below in the row
  v += dpp<0x112, 0xf>(0.0f, v);
  v += dpp<0x114, 0xf>(0.0f, v);
  v += dpp<0x118, 0xf>(0.0f, v);
  v += dpp<0x142, 0xa>(0.0f, v);   // row 0 to row 1, row 2 to row 3
  v += dpp<0x143, 0xc>(0.0f, v);   // rows 0 and 1 to rows 2 and 3
  return last_lane(v);
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x111, 0xf>(-INFINITY, v));
  v = fmaxf(v, dpp<0x112, 0xf>(-INFINITY, v));
  v = fmaxf(v, dpp<0x114, 0xf>(-INFINITY, v));
  v = fmaxf(v, dpp<0x118, 0xf>(-INFINITY, v));
  v = fmaxf(v, dpp<0x142, 0xa>(-INFINITY, v));
  v = fmaxf(v, dpp<0x143, 0xc>(-INFINITY, v));
  return last_lane(v);
}

template <int ctrl, int rows>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int low = int(uint32_t(u)), high = int(uint32_t(u >> 32));
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, low, ctrl, rows, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, high, ctrl, rows, 0xf, false);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<0x111, 0xf>(v);
  v += dpp<0x112, 0xf>(v);
  v += dpp<0x114, 0xf>(v);
  v += dpp<0x118, 0xf>(v);
  v += dpp<0x142, 0xa>(v);
  v += dpp<0x143, 0xc>(v);
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(int(uint32_t(u)), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(int(uint32_t(u >> 32)), 63);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// Sums of N values over a workgroup of `threads`, in every lane, in an order
// that `threads` alone fixes.  red: N * threads / 64 doubles of LDS, used by
// this call alone.
template <int N, int threads>
__device__ __forceinline__ void block_sums(double (&v)[N], double *red) {
  constexpr int W = threads / 64;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (W == 1) return;
  const int lane = threadIdx.x % 64;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == i) red[i * W + threadIdx.x / 64] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lane < W ? red[i * W + lane] : 0.0;
    v[i] = wave_sum(v[i]);
  }
}

}  // namespace qlora
