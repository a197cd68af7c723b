// The objectives over token arrays: the policy loss and the preference loss,
// each with its gradient by token.  Both only stream a few fp32 arrays, so
// they are bound by HBM when long and by the launch when short.  Sums are
// fp64 and in an order that the sizes alone fix.
#include "objective.h"

namespace qlora {
namespace {

// ------------------------------------------------------------ policy loss

constexpr int kPolicyThreads = 256;
constexpr int64_t kPolicyChunk = 4096;   // tokens of one workgroup

__global__ __launch_bounds__(kPolicyThreads) void policy_kernel(
    const float *logp, const float *entropy, int64_t T, PolicyTokens k, PolicyParams p, float *out,
    float *dlogp, float *dentropy, double *partial) {
  __shared__ double red[kPolicyThreads / 64];
  double s[4] = {};
  const int64_t first = int64_t(blockIdx.x) * kPolicyChunk;
  const int64_t last = min64(first + kPolicyChunk, T);
  for (int64_t i = first + threadIdx.x; i < last; i += kPolicyThreads) {
    const float w = k.weight ? k.weight[i] : 1.0f;
    float g = 0.0f, gh = 0.0f;
    if (w != 0.0f) {
      const float h = entropy ? entropy[i] : 0.0f;
      const PolicyToken t = policy_token(p, k, i, logp[i], h);
      g = w * t.dlogp;
      gh = -w * p.ent;
      s[0] += w * t.loss; s[1] += w * t.k; s[2] += w * t.bound; s[3] += w * h;
    }
    dlogp[i] = g;
    if (dentropy) dentropy[i] = gh;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double v = block_sum<kPolicyThreads>(s[j], red);
    if (threadIdx.x == 0) {
      if (partial) partial[int64_t(blockIdx.x) * 4 + j] = v;
      else out[j] = float(v);
    }
  }
}

__global__ __launch_bounds__(1024) void policy_sum_kernel(const double *partial, int64_t n,
                                                          float *out) {
  __shared__ double red[16];
  double s[4] = {};
  for (int64_t i = threadIdx.x; i < n; i += 1024)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += partial[i * 4 + j];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double v = block_sum<1024>(s[j], red);
    if (threadIdx.x == 0) out[j] = float(v);
  }
}

// -------------------------------------------------------- preference loss
//
// With S_i the (averaged) sum of logp - ref over answer i's counted tokens and
// h = S_chosen - S_rejected, dl / dh gives every counted token of the chosen
// answer dl/dh / P (/ its number), of the rejected one the opposite.

constexpr int kPrefThreads = 256;

struct PairLoss {
  float loss, dh;
};

__device__ __forceinline__ PairLoss pair_loss(const PrefParams &p, float h) {
  if (p.kind == 1) {
    const float e = h - 0.5f / p.beta;
    return {e * e, 2.0f * e};
  }
  const float u = p.beta * h - p.margin;
  if (p.kind == 2) return u < 1.0f ? PairLoss{1.0f - u, -p.beta} : PairLoss{0.0f, 0.0f};
  // -log sigma(u) = max(-u, 0) + log1p(exp(-|u|)); sigma(-u) from the same exp
  const float e = expf(-fabsf(u)), l = log1pf(e);
  const float neg = u > 0.0f ? e / (1.0f + e) : 1.0f / (1.0f + e);
  const float down = fmaxf(-u, 0.0f) + l, up = fmaxf(u, 0.0f) + l;
  return {(1.0f - p.smoothing) * down + p.smoothing * up,
          p.beta * (p.smoothing * (1.0f - neg) - (1.0f - p.smoothing) * neg)};
}

struct Answer {
  int64_t first, last;
};

__device__ __forceinline__ Answer answer(const int64_t *cu, int64_t i, int64_t T) {
  const int64_t a = cu[i], b = cu[i + 1];
  const int64_t first = a < 0 ? 0 : min64(a, T);
  return {first, b < first ? first : min64(b, T)};
}

// Sum and number of one thread's counted tokens of [first, last).
__device__ __forceinline__ void pref_add(const float *logp, const float *ref, const uint8_t *mask,
                                         int64_t first, int64_t last, int step, int at, double &s,
                                         double &n) {
  for (int64_t t = first + at; t < last; t += step)
    if (!mask || mask[t]) {
      s += ref ? double(logp[t] - ref[t]) : double(logp[t]);
      n += 1.0;
    }
}

__global__ __launch_bounds__(kPrefThreads) void pref_sum_kernel(const float *logp,
                                                                const float *ref,
                                                                const uint8_t *mask,
                                                                const int64_t *cu, int64_t T,
                                                                double *partial) {
  __shared__ double red[kPrefThreads / 64];
  const int64_t i = blockIdx.x, j = blockIdx.y, n = gridDim.y;
  const Answer a = answer(cu, i, T);
  const int64_t len = a.last - a.first, each = (len + n - 1) / n;
  const int64_t first = a.first + min64(j * each, len), last = min64(first + each, a.last);
  double s = 0.0, c = 0.0;
  pref_add(logp, ref, mask, first, last, kPrefThreads, threadIdx.x, s, c);
  s = block_sum<kPrefThreads>(s, red);
  c = block_sum<kPrefThreads>(c, red);
  if (threadIdx.x == 0) {
    partial[(i * n + j) * 2] = s;
    partial[(i * n + j) * 2 + 1] = c;
  }
}

// S and the number of answer i from its partials.
__device__ __forceinline__ void pref_total(const PrefParams &p, const double *partial, int64_t i,
                                           int n, float &S, float &count) {
  double s = 0.0, c = 0.0;
  for (int j = 0; j < n; ++j) {
    s += partial[(i * n + j) * 2];
    c += partial[(i * n + j) * 2 + 1];
  }
  if (p.average) s = c > 0.0 ? s / c : 0.0;
  S = float(s);
  count = float(c);
}

// Zero for this workgroup's share of the tokens outside every answer.
__device__ __forceinline__ void pref_outside(const int64_t *cu, int64_t P, int64_t T,
                                             float *dlogp, int64_t b, int64_t blocks) {
  const int64_t lo = answer(cu, 0, T).first, hi = answer(cu, 2 * P - 1, T).last;
  const int64_t step = blocks * kPrefThreads;
  for (int64_t t = b * kPrefThreads + threadIdx.x; t < lo; t += step) dlogp[t] = 0.0f;
  for (int64_t t = hi + b * kPrefThreads + threadIdx.x; t < T; t += step) dlogp[t] = 0.0f;
}

// Workgroup (i, j) writes slice j of answer i's gradient; the last column's
// extra workgroups (j = n) hold the mean loss and the rewards.
__global__ __launch_bounds__(kPrefThreads) void pref_grad_kernel(
    const uint8_t *mask, const int64_t *cu, int64_t P, int64_t T, PrefParams p,
    const double *partial, int n, float *loss, float *rewards, float *dlogp) {
  __shared__ double red[kPrefThreads / 64];
  const int64_t i = blockIdx.x, j = blockIdx.y;
  if (j == n) {
    if (i != 0) return;
    double sum = 0.0;
    for (int64_t k = threadIdx.x; k < P; k += kPrefThreads) {
      float a, b, ca, cb;
      pref_total(p, partial, k, n, a, ca);
      pref_total(p, partial, P + k, n, b, cb);
      rewards[k] = p.beta * a;
      rewards[P + k] = p.beta * b;
      sum += pair_loss(p, a - b).loss;
    }
    sum = block_sum<kPrefThreads>(sum, red);
    if (threadIdx.x == 0) loss[0] = float(sum / double(P));
    return;
  }
  pref_outside(cu, P, T, dlogp, i * n + j, 2 * P * n);
  const int64_t k = i < P ? i : i - P;
  float a, b, ca, cb;
  pref_total(p, partial, k, n, a, ca);
  pref_total(p, partial, P + k, n, b, cb);
  float g = pair_loss(p, a - b).dh / float(P);
  if (i >= P) g = -g;
  const float count = i < P ? ca : cb;
  if (p.average && count > 0.0f) g /= count;
  const Answer q = answer(cu, i, T);
  const int64_t len = q.last - q.first, each = (len + n - 1) / n;
  const int64_t first = q.first + min64(j * each, len), last = min64(first + each, q.last);
  for (int64_t t = first + threadIdx.x; t < last; t += kPrefThreads)
    dlogp[t] = !mask || mask[t] ? g : 0.0f;
}

}  // namespace

int64_t policy_blocks(int64_t T) { return T > 0 ? (T + kPolicyChunk - 1) / kPolicyChunk : 1; }

hipError_t launch_policy(const float *logp, const float *entropy, int64_t T,
                         const PolicyTokens &t, const PolicyParams &p, float *out, float *dlogp,
                         float *dentropy, double *partial, hipStream_t s) {
  const int64_t n = policy_blocks(T);
  hipLaunchKernelGGL(policy_kernel, dim3(unsigned(n)), dim3(kPolicyThreads), 0, s, logp, entropy,
                     T, t, p, out, dlogp, dentropy, n > 1 ? partial : nullptr);
  if (n > 1)
    hipLaunchKernelGGL(policy_sum_kernel, dim3(1), dim3(1024), 0, s, partial, n, out);
  return hipGetLastError();
}

// Slices of an answer: enough workgroups to fill the chip for a few long
// answers, and at least a few thousand tokens each on average.
int64_t pref_splits(int64_t P, int64_t T) {
  const int64_t by_size = T / (2 * P) / 2048, by_chip = 1024 / (2 * P);
  const int64_t n = by_size < by_chip ? by_size : by_chip;
  return n < 1 ? 1 : n;
}

hipError_t launch_pref(const float *logp, const float *ref, const uint8_t *mask,
                       const int64_t *cu, int64_t P, int64_t T, const PrefParams &p, float *loss,
                       float *rewards, float *dlogp, double *partial, hipStream_t s) {
  const int64_t n = pref_splits(P, T);
  hipLaunchKernelGGL(pref_sum_kernel, dim3(unsigned(2 * P), unsigned(n)), dim3(kPrefThreads), 0,
                     s, logp, ref, mask, cu, T, partial);
  hipLaunchKernelGGL(pref_grad_kernel, dim3(unsigned(2 * P), unsigned(n) + 1),
                     dim3(kPrefThreads), 0, s, mask, cu, P, T, p, partial, int(n), loss, rewards,
                     dlogp);
  return hipGetLastError();
}

}  // namespace qlora
