// The objectives over token arrays: the policy loss and the preference loss,
// each with its gradient by token.  Both only stream a few fp32 arrays, so
// they are bound by HBM when long and by the launch when short.  Sums are
// fp64 and in an order that the sizes alone fix.  Measured: the policy loss of
// 2 M tokens with entropies 15.2 us (67 MB, 4.4 TB/s) and 3.9 us for the
// partials, of 1000 tokens 3.9 us; the preference loss of 256 pairs of 4608
// tokens 7.6 and 1.5 us, of two pairs of 147000 4.0 and 6.8 us (latency: an
// answer's place, its tokens, both answers' partials, the tokens' masks again,
// one load after the other), of four pairs of 337 5.9 us in one launch.
#include "objective.h"

namespace qlora {
namespace {

// ------------------------------------------------------------ policy loss

// Up to kPolicyLone the tokens are one workgroup's and its sums are the result;
// past that there is a second launch.  us a call, one launch and two: 5000
// tokens 7.9 and 11.6, 8000 8.7 and 11.5, 12000 10.9 and 11.2.
constexpr int kPolicyThreads = 256;
constexpr int64_t kPolicyLone = 8192;

__device__ __forceinline__ void put_sums(const double (&s)[4], float *out, double *partial) {
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (partial) partial[int64_t(blockIdx.x) * 4 + j] = s[j];
    else out[j] = float(s[j]);
  }
}

// n <= 4 values from `i` on, or `fill` where there is no array.
__device__ __forceinline__ f32x4_t take4(const float *v, int64_t i, int n, float fill) {
  f32x4_t x = {fill, fill, fill, fill};
  if (!v) return x;
  if (n == 4) {
    __builtin_memcpy(&x, v + i, 16);
  } else {
    for (int j = 0; j < n; ++j) x[j] = v[i + j];
  }
  return x;
}

__device__ __forceinline__ void give4(float *v, int64_t i, int n, const f32x4_t &x) {
  if (n == 4) {
    __builtin_memcpy(v + i, &x, 16);
  } else {
    for (int j = 0; j < n; ++j) v[i + j] = x[j];
  }
}

template <int threads>
__global__ __launch_bounds__(threads) void policy_kernel(const float *logp, const float *entropy,
                                                         int64_t T, PolicyTokens k,
                                                         PolicyParams p, float *out, float *dlogp,
                                                         float *dentropy, double *partial) {
  __shared__ double red[4 * threads / 64];
  double s[4] = {};
  const int64_t step = int64_t(gridDim.x) * threads * 4;
  for (int64_t i = (int64_t(blockIdx.x) * threads + threadIdx.x) * 4; i < T; i += step) {
    const int n = int(least64(T - i, 4));
    const f32x4_t w = take4(k.weight, i, n, 1.0f), lp = take4(logp, i, n, 0.0f);
    const f32x4_t h = take4(entropy, i, n, 0.0f), adv = take4(k.adv, i, n, 1.0f);
    const f32x4_t old = take4(k.old, i, n, 0.0f), ref = take4(k.ref, i, n, 0.0f);
    f32x4_t g, gh;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = j < n ? w[j] : 0.0f;   // 0: what the token holds is not used
      const PolicyToken t = policy_token(p, lp[j], h[j], adv[j], k.old ? lp[j] - old[j] : 0.0f,
                                         k.ref, ref[j]);
      g[j] = scaled(v, t.dlogp);
      gh[j] = scaled(v, -p.ent);
      s[0] += scaled(v, t.loss);
      s[1] += scaled(v, t.k);
      s[2] += scaled(v, t.bound);
      s[3] += scaled(v, h[j]);
    }
    give4(dlogp, i, n, g);
    if (dentropy) give4(dentropy, i, n, gh);
  }
  block_sums<4, threads>(s, red);
  put_sums(s, out, partial);
}

// Column sums of v [n x 4].  A lane's loads wait for one another, since each is
// behind its own end of the loop: 8192 rows take eight round trips, 6.3 us.
template <class F>
__global__ __launch_bounds__(1024) void sum4_kernel(const F *v, int64_t n, float *out,
                                                    double *partial) {
  __shared__ double red[4 * 16];
  double s[4] = {};
  const int64_t step = int64_t(gridDim.x) * 1024;
  for (int64_t i = int64_t(blockIdx.x) * 1024 + threadIdx.x; i < n; i += step) {
    F x[4];
    __builtin_memcpy(x, v + 4 * i, sizeof(x));
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += double(x[j]);
  }
  block_sums<4, 1024>(s, red);
  put_sums(s, out, partial);
}

constexpr int64_t kTermsLone = 8192;    // terms that one workgroup adds up alone

// -------------------------------------------------------- preference loss
//
// With S_i the (averaged) sum of logp - ref over answer i's counted tokens and
// h = S_chosen - S_rejected, dl / dh gives every counted token of the chosen
// answer dl/dh / P (/ its number), of the rejected one the opposite.

// A unit of work is one wavefront's: a slice of one answer.  The slices' sums
// and counts ("partials") join the two passes.  Few tokens: one workgroup holds
// the partials in LDS between its two passes.  Many pairs of some length: a
// workgroup to a pair, and a second launch for the mean loss.  Else: one launch
// for the sums and one for the gradients, partials in the workspace.
constexpr int kPrefThreads = 256;        // of the two launches
// One workgroup where each of its 16 wavefronts has an answer at most.  us a
// call, so and in two launches: 4 pairs of 2800 tokens 9.0 and 10.1, of 4500
// 10.4 and 10.0; 16 of 450 10.3 and 10.2; 100 of 112 44.4 and 10.1.
constexpr int64_t kPrefLoneTokens = 16384, kPrefLonePairs = 8;
// Tokens of a slice, two quads to a lane.  us a call, 256 / 512 / 1024 / 2048:
// 53 pairs of 44000 tokens 19.1 / 15.8 / 15.5 / 19.0, two of 147000 10.1 /
// 10.4 / 11.4 / 15.1, 16 of 67000 12.2 / 11.2 / 11.8 / 15.9.
constexpr int64_t kPrefSlice = 512;
constexpr int64_t kPrefMeanPairs = 512;  // past these, losses by the workspace
constexpr int64_t kPrefUnits = 16384;    // slices, when answers are cut at all

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
  // (an infinite u, from an answer that the model cannot give, has an infinite
  // `up`, of which no smoothing takes nothing)
  return {(1.0f - p.smoothing) * down + (p.smoothing > 0.0f ? p.smoothing * up : 0.0f),
          p.beta * (p.smoothing * (1.0f - neg) - (1.0f - p.smoothing) * neg)};
}

struct PrefArgs {
  const float *logp, *ref;
  const uint8_t *mask;
  const int64_t *cu;
  int64_t P, T;
  PrefParams p;
  float *loss, *rewards, *dlogp;
};

// The wavefront's number in its workgroup, as a scalar.
__device__ __forceinline__ int wave_index() {
  return __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64);
}

// Tokens number at most 2^30: a place fits 32 bits.
struct Span {
  int32_t first, last;
};

__device__ __forceinline__ Span answer(const PrefArgs &a, int32_t i) {
  const int64_t lo = a.cu[i], hi = a.cu[i + 1];
  const int64_t first = lo < 0 ? 0 : least64(lo, a.T);
  return {int32_t(first), int32_t(hi < first ? first : least64(hi, a.T))};
}

// Slice j of n of an answer, its inner ends on multiples of four tokens.
__device__ __forceinline__ Span slice(const Span &s, int32_t j, int32_t n) {
  const int32_t base = s.first & ~3;
  const uint32_t tokens = uint32_t(s.last - base), cut = uint32_t(n);
  const int32_t each = int32_t(n == 1 ? tokens : ((tokens + cut - 1) / cut + 3u) & ~3u);
  // (the last slices of a short answer are empty: j * each can pass 2^31)
  const int64_t from = base + int64_t(j) * each;
  const int32_t lo = int32_t(least64(from, s.last));
  return {lo < s.first ? s.first : lo, int32_t(least64(from + each, s.last))};
}

struct Partial {
  double sum, count;
};

// A quad's four tokens as they are loaded: from t on, or, at the end of the
// arrays, the last four, of which those before t are another quad's.
struct Quad {
  int32_t t, at;
  __device__ __forceinline__ Quad(const PrefArgs &a, int32_t from)
      : t(from), at(from + 4 <= int32_t(a.T) ? from : int32_t(a.T) - 4) {}
  // bit j: token at + j is the quad's own, lies in s and counts
  __device__ __forceinline__ uint32_t counted(const Span &s, uint32_t mask) const {
    const int32_t lo = t > s.first ? t : s.first, hi = t + 4 < s.last ? t + 4 : s.last;
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((mask >> (8 * j) & 0xffu) && at + j >= lo && at + j < hi) bits |= 1u << j;
    return bits;
  }
};

// Arrays of less than four tokens take the byte and the word one by one.  The
// test is a lane's, though all lanes agree: each load is behind a branch.
__device__ __forceinline__ uint32_t load_mask(const PrefArgs &a, const Quad &q) {
  uint32_t m = 0x01010101u;
  if (a.mask && q.at >= 0) __builtin_memcpy(&m, a.mask + q.at, 4);
  if (a.mask && q.at < 0)
    for (int j = 0; j < 4; ++j)
      if (q.at + j >= 0) m = (m & ~(0xffu << 8 * j)) | uint32_t(a.mask[q.at + j]) << 8 * j;
  return m;
}
__device__ __forceinline__ f32x4_t load_quad(const float *v, const Quad &q) {
  f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (q.at >= 0) {
    __builtin_memcpy(&x, v + q.at, 16);
  } else {
    for (int j = 0; j < 4; ++j)
      if (q.at + j >= 0) x[j] = v[q.at + j];
  }
  return x;
}

// The quads of a slice, N of a lane at a time (past the slice's end the last
// quad again, nothing of it counted), so that the loads of all N are on their
// way before the first is used.
__device__ __forceinline__ int32_t quad_at(const Span &s, int32_t t, int i) {
  return t + 256 * i < s.last ? t + 256 * i : s.last;
}

// One wavefront's sum over a slice.
template <int N>
__device__ __forceinline__ Partial slice_sum(const PrefArgs &a, const Span &s) {
  double sum = 0.0;
  int count = 0;
  for (int32_t t = (s.first & ~3) + 4 * int32_t(threadIdx.x % 64); t < s.last;
       t += 256 * N) {
    f32x4_t lp[N], rf[N] = {};
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Quad q(a, quad_at(s, t, i));
      lp[i] = load_quad(a.logp, q);
      if (a.ref) rf[i] = load_quad(a.ref, q);
      m[i] = load_mask(a, q);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t bits = Quad(a, quad_at(s, t, i)).counted(s, m[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += (bits >> j & 1u) ? lp[i][j] - rf[i][j] : 0.0f;
      count += __builtin_popcount(bits);
    }
  }
  return {wave_sum(sum), wave_sum(double(count))};
}

// dlogp of a slice: g where a token counts, 0 elsewhere in the answer.
template <int N>
__device__ __forceinline__ void slice_grad(const PrefArgs &a, const Span &s, float g) {
  for (int32_t t = (s.first & ~3) + 4 * int32_t(threadIdx.x % 64); t < s.last;
       t += 256 * N) {
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = load_mask(a, Quad(a, quad_at(s, t, i)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Quad q(a, quad_at(s, t, i));
      const uint32_t bits = q.counted(s, m[i]);
      f32x4_t d;
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = (bits >> j & 1u) ? g : 0.0f;
      if (q.t >= s.first && q.t + 4 <= s.last) {
        __builtin_memcpy(a.dlogp + q.t, &d, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (q.at + j >= q.t && q.at + j >= s.first && q.at + j < s.last) a.dlogp[q.at + j] = d[j];
      }
    }
  }
}

// Unit u: slice u % n of answer u / n.
template <int N>
__device__ __forceinline__ Partial unit_sum(const PrefArgs &a, int32_t u, int n) {
  const int32_t i = n == 1 ? u : u / n;
  return slice_sum<N>(a, slice(answer(a, i), u - i * n, n));
}

// An answer's S and count from its n partials; lane `at` of `lanes` (a power of
// two, neighbours in a wavefront) adds every lanes-th of them.
__device__ __forceinline__ Partial total(const PrefArgs &a, const Partial *partial, int32_t i,
                                         int n, int at, int lanes) {
  Partial r = {0.0, 0.0};
  // (four loads at once while four are left to a lane, the rest one by one)
#pragma unroll 4
  for (int j = at; j < n; j += lanes) {
    r.sum += partial[int64_t(i) * n + j].sum;
    r.count += partial[int64_t(i) * n + j].count;
  }
  for (int o = lanes / 2; o > 0; o >>= 1) {
    r.sum += __shfl_xor(r.sum, o);
    r.count += __shfl_xor(r.count, o);
  }
  if (a.p.average) r.sum = r.count > 0.0 ? r.sum / r.count : 0.0;
  return r;
}

__device__ __forceinline__ int lanes_for(int n) {
  return n <= 1 ? 1 : n >= 33 ? 64 : 1 << (32 - __builtin_clz(n - 1));
}

// dloss / dlogp of an answer's counted tokens.
__device__ __forceinline__ float answer_grad(const PrefArgs &a, const PairLoss &l, double count,
                                             bool rejected) {
  const float g = (rejected ? -l.dh : l.dh) / float(a.P);
  return a.p.average && count > 0.0 ? g / float(count) : g;
}

// Unit u's gradient; slice 0 also writes the answer's reward.  Its pair's loss.
template <int N>
__device__ __forceinline__ float unit_grad(const PrefArgs &a, const Partial *partial, int32_t u,
                                          int n) {
  const int32_t i = n == 1 ? u : u / n, j = u - i * n, P = int32_t(a.P);
  const Span own_slice = slice(answer(a, i), j, n);
  const int lane = threadIdx.x % 64, lanes = lanes_for(n);
  const int32_t k = i < P ? i : i - P;
  const Partial c = total(a, partial, k, n, lane % lanes, lanes);
  const Partial r = total(a, partial, P + k, n, lane % lanes, lanes);
  const Partial &own = i < P ? c : r;
  const PairLoss l = pair_loss(a.p, float(c.sum - r.sum));
  const float g = answer_grad(a, l, own.count, i >= P);
  if (j == 0 && lane == 0) a.rewards[i] = float(a.p.beta * own.sum);
  slice_grad<N>(a, own_slice, g);
  return l.loss;
}

// The mean loss, by one workgroup: a pair to so many lanes that every pair has
// some at once, up to one for each of its slices.
template <int threads>
__device__ __forceinline__ void mean_loss(const PrefArgs &a, const Partial *partial, int n,
                                          double *red) {
  int lanes = lanes_for(n);
  while (lanes > 1 && int64_t(lanes) * a.P > threads) lanes /= 2;
  const int at = threadIdx.x % lanes;
  double sum[1] = {};
  const int32_t P = int32_t(a.P);
  for (int32_t first = 0; first < P; first += threads / lanes) {
    const int32_t k = first + int32_t(threadIdx.x) / lanes;
    const int32_t kk = k < P ? k : P - 1;     // every lane takes part in the shuffles
    const Partial c = total(a, partial, kk, n, at, lanes);
    const Partial r = total(a, partial, P + kk, n, at, lanes);
    if (k < P && at == 0) sum[0] += pair_loss(a.p, float(c.sum - r.sum)).loss;
  }
  block_sums<1, threads>(sum, red);
  if (threadIdx.x == 0) a.loss[0] = float(sum[0] / double(a.P));
}

// Zeros for the tokens outside every answer, by thread `at` of `all`.
__device__ __forceinline__ void zero_outside(const PrefArgs &a, int64_t at, int64_t all) {
  const int64_t lo = answer(a, 0).first, hi = answer(a, 2 * int32_t(a.P) - 1).last;
  for (int64_t t = at; t < lo; t += all) a.dlogp[t] = 0.0f;
  for (int64_t t = hi + at; t < a.T; t += all) a.dlogp[t] = 0.0f;
}

__global__ __launch_bounds__(1024) void pref_lone_kernel(PrefArgs a, int n) {
  __shared__ Partial partial[2 * kPrefLonePairs];
  __shared__ float loss[kPrefLonePairs];
  const int units = int(2 * a.P) * n, wave = wave_index(), lane = threadIdx.x % 64;
  for (int u = wave; u < units; u += 16) {
    const Partial s = unit_sum<1>(a, u, n);
    if (lane == 0) partial[u] = s;
  }
  __syncthreads();
  for (int u = wave; u < units; u += 16) {
    const float l = unit_grad<1>(a, partial, u, n);
    if (lane == 0 && u < int(a.P) * n && u % n == 0) loss[u / n] = l;
  }
  zero_outside(a, threadIdx.x, 1024);
  __syncthreads();
  if (wave == 0) {
    double sum = 0.0;
    for (int k = lane; k < int(a.P); k += 64) sum += loss[k];
    sum = wave_sum(sum);
    if (lane == 0) a.loss[0] = float(sum / double(a.P));
  }
}

// A pair to a workgroup: half of its wavefronts to each answer.  losses [P]
// receives the pairs' losses for pref_mean_kernel.
__global__ __launch_bounds__(1024) void pref_pair_kernel(PrefArgs a, double *losses) {
  __shared__ Partial partial[16];
  const int wave = wave_index(), lane = threadIdx.x % 64, side = wave / 8;
  const int32_t k = int32_t(blockIdx.x), i = side ? int32_t(a.P) + k : k;
  const Span s = slice(answer(a, i), wave % 8, 8);
  const Partial mine = slice_sum<2>(a, s);
  if (lane == 0) partial[wave] = mine;
  __syncthreads();
  const Partial c = total(a, partial, 0, 8, lane % 8, 8), r = total(a, partial, 1, 8, lane % 8, 8);
  const PairLoss l = pair_loss(a.p, float(c.sum - r.sum));
  const Partial &own = side ? r : c;
  slice_grad<2>(a, s, answer_grad(a, l, own.count, side));
  if (wave % 8 == 0 && lane == 0) a.rewards[i] = float(a.p.beta * own.sum);
  if (threadIdx.x == 0) losses[k] = l.loss;
  zero_outside(a, int64_t(blockIdx.x) * 1024 + threadIdx.x, int64_t(gridDim.x) * 1024);
}

__global__ __launch_bounds__(1024) void pref_mean_kernel(const double *losses, int64_t P,
                                                         float *loss) {
  __shared__ double red[16];
  double s[1] = {};
#pragma unroll 4   // reached from 4096 pairs on
  for (int64_t k = threadIdx.x; k < P; k += 1024) s[0] += losses[k];
  block_sums<1, 1024>(s, red);
  if (threadIdx.x == 0) loss[0] = float(s[0] / double(P));
}

template <int N>
__global__ __launch_bounds__(kPrefThreads) void pref_sum_kernel(PrefArgs a, int n, int32_t units,
                                                                Partial *partial) {
  const int32_t u = int32_t(blockIdx.x) * (kPrefThreads / 64) + wave_index();
  if (u >= units) return;
  const Partial s = unit_sum<N>(a, u, n);
  if (threadIdx.x % 64 == 0) partial[u] = s;
}

// losses != null: the pairs' losses go there, for pref_mean_kernel; else an
// extra, last workgroup takes the mean.
template <int N>
__global__ __launch_bounds__(kPrefThreads) void pref_grad_kernel(PrefArgs a, int n, int32_t units,
                                                                 const Partial *partial,
                                                                 double *losses) {
  __shared__ double red[kPrefThreads / 64];
  const int64_t work = losses ? int64_t(gridDim.x) : int64_t(gridDim.x) - 1;
  if (blockIdx.x == work) {
    mean_loss<kPrefThreads>(a, partial, n, red);
    return;
  }
  const int32_t u = int32_t(blockIdx.x) * (kPrefThreads / 64) + wave_index();
  if (u < units) {
    const float l = unit_grad<N>(a, partial, u, n);
    if (losses && u < int32_t(a.P) * n && u % n == 0 && threadIdx.x % 64 == 0) losses[u / n] = l;
  }
  zero_outside(a, int64_t(blockIdx.x) * kPrefThreads + threadIdx.x, work * kPrefThreads);
}

}  // namespace

int64_t policy_blocks(int64_t T) {
  return T <= kPolicyLone ? 1 : least64((T + 4 * kPolicyThreads - 1) / (4 * kPolicyThreads), 2048);
}

hipError_t launch_policy(const float *logp, const float *entropy, int64_t T,
                         const PolicyTokens &t, const PolicyParams &p, float *out, float *dlogp,
                         float *dentropy, double *partial, hipStream_t s) {
  const int64_t n = policy_blocks(T);
  if (n == 1) {
    hipLaunchKernelGGL((policy_kernel<1024>), dim3(1), dim3(1024), 0, s, logp, entropy, T, t, p,
                       out, dlogp, dentropy, nullptr);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((policy_kernel<kPolicyThreads>), dim3(unsigned(n)), dim3(kPolicyThreads), 0,
                     s, logp, entropy, T, t, p, out, dlogp, dentropy, partial);
  hipLaunchKernelGGL((sum4_kernel<double>), dim3(1), dim3(1024), 0, s, partial, n, out, nullptr);
  return hipGetLastError();
}

int64_t terms_blocks(int64_t n) {
  return n <= kTermsLone ? 1 : least64((n + 1023) / 1024, 1024);
}

hipError_t launch_sum_terms(const float *terms, int64_t n, float *out, double *partial,
                            hipStream_t s) {
  const int64_t b = terms_blocks(n);
  hipLaunchKernelGGL((sum4_kernel<float>), dim3(unsigned(b)), dim3(1024), 0, s, terms, n, out,
                     b > 1 ? partial : nullptr);
  if (b > 1)
    hipLaunchKernelGGL((sum4_kernel<double>), dim3(1), dim3(1024), 0, s, partial, b, out, nullptr);
  return hipGetLastError();
}

namespace {

// Enough pairs to fill the chip with one workgroup each, and enough tokens in
// a pair for its 16 wavefronts.  Measured, us a call, by pairs and by slices:
// 256 pairs of 4608 tokens 9.6, 13.3; 64 of 18000 13.6, 14.7; 2048 of 563
// 30.6, 16.5.
bool pref_paired(int64_t P, int64_t T) {
  return P >= 64 && T / P >= 1024 && T / P <= 65536;
}

bool pref_lone(int64_t P, int64_t T) { return T <= kPrefLoneTokens && P <= kPrefLonePairs; }

int64_t pref_splits(int64_t P, int64_t T) {
  const int64_t by_size = (T / (2 * P) + kPrefSlice - 1) / kPrefSlice, most = kPrefUnits / (2 * P);
  const int64_t n = least64(by_size, most);
  return n < 1 ? 1 : n;
}

}  // namespace

int64_t pref_partials(int64_t P, int64_t T) {
  if (pref_lone(P, T)) return 0;
  if (pref_paired(P, T)) return P;
  return 4 * P * pref_splits(P, T) + (P > kPrefMeanPairs ? P : 0);
}

hipError_t launch_pref(const float *logp, const float *ref, const uint8_t *mask,
                       const int64_t *cu, int64_t P, int64_t T, const PrefParams &p, float *loss,
                       float *rewards, float *dlogp, double *partial, hipStream_t s) {
  const PrefArgs a = {logp, ref, mask, cu, P, T, p, loss, rewards, dlogp};
  if (pref_lone(P, T)) {
    // 16 wavefronts: several to an answer when there are few answers
    const int n = 2 * P >= 16 ? 1 : int(16 / (2 * P));
    hipLaunchKernelGGL(pref_lone_kernel, dim3(1), dim3(1024), 0, s, a, n);
    return hipGetLastError();
  }
  if (pref_paired(P, T)) {
    hipLaunchKernelGGL(pref_pair_kernel, dim3(unsigned(P)), dim3(1024), 0, s, a, partial);
    hipLaunchKernelGGL(pref_mean_kernel, dim3(1), dim3(1024), 0, s, partial, P, loss);
    return hipGetLastError();
  }
  const int64_t n = pref_splits(P, T), units = 2 * P * n;
  const unsigned blocks = unsigned((units + kPrefThreads / 64 - 1) / (kPrefThreads / 64));
  Partial *part = reinterpret_cast<Partial *>(partial);
  // one workgroup's mean over the partials of many pairs would outlast the rest
  // (8192 pairs of 135 tokens 53 us, through their losses 19)
  double *losses = P > kPrefMeanPairs ? partial + 2 * units : nullptr;
#define SLICES(N)                                                                               \
  do {                                                                                          \
    hipLaunchKernelGGL((pref_sum_kernel<N>), dim3(blocks), dim3(kPrefThreads), 0, s, a, int(n), \
                       int32_t(units), part);                                                   \
    hipLaunchKernelGGL((pref_grad_kernel<N>), dim3(blocks + !losses), dim3(kPrefThreads), 0, s, \
                       a, int(n), int32_t(units), part, losses);                                \
  } while (0)
  // quads of a lane in flight: as a slice of average length needs
  if (T / units <= 256) SLICES(1);
  else SLICES(kPrefSlice / 256);
#undef SLICES
  if (losses)
    hipLaunchKernelGGL(pref_mean_kernel, dim3(1), dim3(1024), 0, s, losses, P, loss);
  return hipGetLastError();
}

}  // namespace qlora
