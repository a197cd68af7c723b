// Device pieces the objectives share: the policy objective of one token and
// workgroup sums in a fixed order.
#pragma once

#include "device.h"

namespace qlora {

struct PolicyToken {
  float loss, k, bound;   // -f + kl k - ent H, the KL estimate, [a bound holds]
  float dlogp;            // d loss / d logp (that of the entropy is -ent)
};

// One token of the objective (qlora_policy_loss in qlora.h has the formulas).
// The branch is chosen on d = logp - old against rounded logs of the bounds:
// d is one fp32 subtraction, so the choice does not hang on how exp rounds.
// k = expm1(q) - q keeps its digits where the two policies nearly agree.
__device__ __forceinline__ PolicyToken policy_token(const PolicyParams &p, const PolicyTokens &k,
                                                    int64_t i, float logp, float ent) {
  const float adv = k.adv ? k.adv[i] : 1.0f;
  PolicyToken t;
  float f = adv * logp, df = adv;
  t.bound = 0.0f;
  if (p.clip) {
    const float d = k.old ? logp - k.old[i] : 0.0f;
    df = expf(d) * adv;
    f = df;
    if (adv > 0.0f && d > p.log_hi) { f = p.hi * adv; t.bound = 1.0f; }
    if (adv < 0.0f && d < p.log_lo) { f = p.lo * adv; t.bound = 1.0f; }
    if (adv < 0.0f && d > p.log_dual) { f = p.dual * adv; t.bound = 1.0f; }
    if (t.bound != 0.0f) df = 0.0f;
  }
  t.loss = -f;
  t.dlogp = -df;
  t.k = 0.0f;
  if (k.ref) {
    const float q = k.ref[i] - logp, em = expm1f(q);
    t.k = em - q;
    t.loss += p.kl * t.k;
    t.dlogp -= p.kl * em;
  }
  if (p.ent != 0.0f) t.loss -= p.ent * ent;
  return t;
}

// Sum over a workgroup of `threads` (a multiple of 64) in a fixed order; the
// result is valid in every thread.  red: threads / 64 doubles of LDS, free
// again after the next barrier.
template <int threads>
__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  const int wave = threadIdx.x / 64;
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[wave] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < threads / 64; ++w) s += red[w];
  return s;
}

}  // namespace qlora
