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
#include "objective.h"

namespace qlora {
namespace {

// Rows in the y and z of a launch, a row's segments in x: neighbouring
// workgroups run through a row, and no dimension reaches its limit.
constexpr int64_t kRowsY = int64_t(1) << 15;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// exp2 is 0 from here down: an exponent of -inf, which would turn 0 L into
// NaN, is taken as this.
constexpr float kLeast = -200.0f;

template <bool BF16>
__device__ __forceinline__ const char *row_at(const void *x, int64_t at) {
  return static_cast<const char *>(x) + at * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ char *row_at(void *x, int64_t at) {
  return static_cast<char *>(x) + at * (BF16 ? 2 : 4);
}

__device__ __forceinline__ int64_t row_index() {
  return int64_t(blockIdx.z) * kRowsY + blockIdx.y;
}

// Word v of a row, at its alignment (V is at most 2^24, so a row's offsets fit
// 32 bits).
template <bool BF16>
__device__ __forceinline__ float load1(const char *row, uint32_t v) {
  if (BF16) {
    uint16_t h;
    __builtin_memcpy(&h, row + v * 2u, 2);
    return __uint_as_float(uint32_t(h) << 16);
  }
  float f;
  __builtin_memcpy(&f, row + v * 4u, 4);
  return f;
}

// A group: the 16 bytes that one load or store of a lane moves.
template <bool BF16>
constexpr int kGroup = BF16 ? 8 : 4;

template <bool BF16>
__device__ __forceinline__ void unpack(u32x4_t u, float (&e)[kGroup<BF16>]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = bf16_lo_to_f32(u[i]);
      e[2 * i + 1] = bf16_hi_to_f32(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = __uint_as_float(u[i]);
  }
}

template <bool BF16>
__device__ __forceinline__ u32x4_t load_group(const char *row, uint32_t v) {
  u32x4_t u;
  __builtin_memcpy(&u, row + v * (BF16 ? 2u : 4u), 16);
  return u;
}

template <bool BF16>
__device__ __forceinline__ void store1(char *row, uint32_t v, float e) {
  if (BF16) {
    const uint16_t h = __builtin_bit_cast(uint16_t, (__bf16)e);
    __builtin_memcpy(row + v * 2u, &h, 2);
  } else {
    __builtin_memcpy(row + v * 4u, &e, 4);
  }
}

template <bool BF16>
__device__ __forceinline__ void store_group(char *row, uint32_t v,
                                            const float (&e)[kGroup<BF16>]) {
  u32x4_t u;
  if constexpr (BF16) {
    u = u32x4_t{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                pack_bf16x2(e[6], e[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(e[i]);
  }
  store16_past(row + v * (BF16 ? 2u : 4u), u);
}

// The cut of a row of V words at address `row`: `head` words, groups from there
// on, `whole` words in all, and the rest.  Head and rest ("ones") are one word
// to a lane, the rest in lanes 0 .. 7, the head in 8 .. 15.
template <bool BF16>
struct Cut {
  int32_t head, whole, V;
  __device__ __forceinline__ Cut(const char *row, int32_t words) : V(words) {
    const int32_t off = int32_t(-reinterpret_cast<uintptr_t>(row) & 15u) / (BF16 ? 2 : 4);
    head = off < V ? off : V;
    whole = (V - head) / kGroup<BF16> * kGroup<BF16>;
  }
  // the word of lane `at` among the ones, or V
  __device__ __forceinline__ int32_t one(int32_t at) const {
    if (at < 8) return head + whole + at < V ? head + whole + at : V;
    return at - 8 < head ? at - 8 : V;
  }
};

// Words of a row in registers, 8 NG to a lane: group g of a lane is the one
// g threads + lane groups after head + from, as it lies in memory.  Groups past
// the last whole one load that one again and are masked to -inf, so every load
// is whole and none leaves the row.  The ones come with the row's first chunk.
template <bool BF16, int threads, int NG>
struct Held {
  static constexpr int32_t words = threads * 8 * NG;
  static constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  u32x4_t q[G];
  float one;

  __device__ __forceinline__ static int32_t first(int g) {
    return (g * threads + int(threadIdx.x)) * W;
  }
  // the words [from, end) of the groups of a row, at most `words` of them
  __device__ __forceinline__ void load(const char *row, const Cut<BF16> &k, int32_t from,
                                       int32_t end) {
    const int32_t last = end - W;
    if (from < end) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int32_t v = from + first(g);
        q[g] = load_group<BF16>(row, uint32_t(k.head + (v <= last ? v : last)));
      }
    }
    one = -INFINITY;
    if (from == 0) {
      const int32_t v = k.one(int32_t(threadIdx.x));
      if (v < k.V) one = load1<BF16>(row, v);
    }
    if (from + words > end) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (from + first(g) > last) {
          const uint32_t w = BF16 ? 0xff80ff80u : 0xff800000u;
          q[g] = u32x4_t{w, w, w, w};
        }
    }
  }
  // Between two passes over the registers: without it the compiler keeps the
  // unpacked words of one pass for the next, twice the registers and more.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int i = 0; i < G; ++i) asm volatile("" : "+v"(q[i]));
  }
};

struct Stat {
  float m, t, w;   // maximum, sum e, sum e L with L = c x - reference(m)
};

// L is taken as c x - M with M = c m rounded once, in one fused operation:
// whatever M is, it cancels from log p.  The rounding leaves off = c m - M, at
// most half an ulp of M, and the largest e is 2^off: below kFar it lies in
// 2^-64 .. 2^64, so that no sum of 2^24 words and no product of one with a
// difference of two references (2^32 at most) leaves fp32.  Past kFar, and
// where there is no word yet, M is 0: a lane of words so far down (a mask of
// -1e10, say) sums to 0, which is its share of any row with a maximum that is
// not far, and a row whose own maximum is far is summed again by careful_row.
constexpr float kFar = 2147483648.0f;   // 2^31

__device__ __forceinline__ bool is_near(float m, float c) { return fabsf(c * m) < kFar; }

__device__ __forceinline__ float reference(float m, float c) {
  return is_near(m, c) ? c * m : 0.0f;
}

template <bool ENT>
__device__ __forceinline__ void add(Stat &a, float x, float c, float M) {
  const float L = __builtin_fmaf(c, x, -M);
  const float p = __builtin_amdgcn_exp2f(L);   // a NaN logit leaves its mark in t
  a.t += p;
  if (ENT) a.w = __builtin_fmaf(p, fmaxf(L, kLeast), a.w);
}

// a's sums brought from their own reference to that of `top` >= a.m.
__device__ __forceinline__ Stat raised(const Stat &a, float top, float c) {
  const float d = reference(a.m, c) - reference(top, c);
  // nothing summed yet, or words far down: t and w are 0, or NaN from NaN
  // logits alone (and what a row with a far top sums to is not used)
  const float f = is_near(a.m, c) ? __builtin_amdgcn_exp2f(d) : 0.0f;
  return {top, f * a.t, f * __builtin_fmaf(d, a.t, a.w)};
}

// A lane's share of a chunk into its running sums.
template <bool ENT, bool BF16, int threads, int NG>
__device__ __forceinline__ void add_chunk(Stat &a, Held<BF16, threads, NG> &h, float c) {
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  float top = fmaxf(a.m, h.one);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float e[W];
    unpack<BF16>(h.q[g], e);
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, e[i]);
  }
  a = raised(a, top, c);
  h.keep();
  const float M = reference(top, c);
  add<ENT>(a, h.one, c, M);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float e[W];
    unpack<BF16>(h.q[g], e);
#pragma unroll
    for (int i = 0; i < W; ++i) add<ENT>(a, e[i], c, M);
  }
}

// The sums of 64 lanes as one, in every lane.
__device__ __forceinline__ Stat joined(const Stat &a, float c) {
  const float top = wave_max(a.m);
  const Stat b = raised(a, top, c);
  return {top, wave_sum(b.t), wave_sum(b.w)};
}

// The sums of a workgroup as one, in every lane, in an order that `threads`
// alone fixes.
template <int threads>
__device__ __forceinline__ Stat joined_block(Stat a, float c, Stat *red) {
  a = joined(a, c);
  if (threads == 64) return a;
  const int lane = threadIdx.x % 64;
  if (lane == 0) red[threadIdx.x / 64] = a;
  __syncthreads();
  a = lane < threads / 64 ? red[lane] : Stat{-INFINITY, 0.0f, 0.0f};
  return joined(a, c);
}

struct RowResult {
  float m, z, logp, ent;
};

// Results of a row from its sums and its label's logit.  off: c m - M, by
// which z takes the rounding of M back.
__device__ __forceinline__ RowResult row_result(const Stat &a, float off, float xy, float scale) {
  if (!(a.t < INFINITY)) {
    const float nan = a.t - a.t;
    return {nan, nan, nan, nan};
  }
  if (!(a.m > -INFINITY)) return {-INFINITY, 0.0f, -INFINITY, 0.0f};
  const float l = logf(a.t), z = l - kLn2 * off;
  return {a.m, z, scale * (xy - a.m) - z, l - kLn2 * (a.w / a.t)};
}

// The sums of a row whose maximum is far: L = c (x - m) in two steps, the row
// read again word by word.  Every word of such a row but -inf is a mask of a
// large finite value, or its logits pass 10^9: no row that a model gives, so the
// time is left as it is (scoring 4096 x 32000 bf16 118 us, not 41; rows that are
// cut, by one wavefront, 64 x 200000 fp32 785 us, not 12).
template <bool BF16, int threads>
__device__ __forceinline__ Stat careful_row(const char *row, int32_t V, float m, float c,
                                            Stat *red) {
  Stat a = {0.0f, 0.0f, 0.0f};
  for (int32_t v = int32_t(threadIdx.x) % threads; v < V; v += threads) {
    const float L = c * (load1<BF16>(row, v) - m);
    const float p = __builtin_amdgcn_exp2f(L);
    a.t += p;
    a.w = __builtin_fmaf(p, fmaxf(L, kLeast), a.w);
  }
  if (threads > 64) __syncthreads();
  return joined_block<threads>(a, c, red);
}

// Results of a row from its words' joined sums.
template <bool BF16, int threads>
__device__ __forceinline__ RowResult finished(Stat a, const char *row, int32_t V,
                                              float xy, float scale, Stat *red) {
  const float c = scale * kLog2e;
  float off = __builtin_fmaf(c, a.m, -reference(a.m, c));
  if (!is_near(a.m, c) && fabsf(a.m) < INFINITY) {
    const float m = a.m;
    a = careful_row<BF16, threads>(row, V, m, c, red);
    a.m = m;
    off = 0.0f;
  }
  return row_result(a, off, xy, scale);
}

// The first words of a row that Held takes in chunks: what remains past whole
// chunks, so that the last chunk is a full one.
template <int32_t words>
__device__ __forceinline__ int32_t first_chunk(int32_t whole) {
  return whole <= words ? whole : (whole - 1) % words + 1;
}

// A row's results: its chunks summed one after the other.  h holds the last
// chunk afterwards (ONE: the row).
template <bool ENT, bool ONE, bool BF16, int threads, int NG>
__device__ __forceinline__ RowResult row_stat(Held<BF16, threads, NG> &h, const char *row,
                                              int32_t V, int32_t y, float scale, Stat *red) {
  const float c = scale * kLog2e;
  Stat a = {-INFINITY, 0.0f, 0.0f};
  const Cut<BF16> k(row, V);
  int32_t end = ONE ? k.whole : first_chunk<Held<BF16, threads, NG>::words>(k.whole);
  h.load(row, k, 0, end);
  const float xy = load1<BF16>(row, uint32_t(y));
  add_chunk<ENT>(a, h, c);
  while (!ONE && end < k.whole) {
    h.load(row, k, end, end + h.words);
    add_chunk<ENT>(a, h, c);
    end += h.words;
  }
  a = joined_block<threads>(a, c, red);
  return finished<BF16, threads>(a, row, V, xy, scale, red);
}

// Coefficients of a row's gradient: with L = log2 p,
//   dx = s (g 1[v = y] - g p - gH p (ln 2 L + H)) = hot 1[v = y] + p (k0 + k1 L).
struct GradCoef {
  float hot, k0, k1, z2;
};

__device__ __forceinline__ GradCoef grad_coef(float scale, float g, float gh, float ent, float z) {
  // a row of NaN stays one, also where the clamp of L makes p 0
  const float nan = z != z ? z : 0.0f;
  return {scale * g, -scale * (g + gh * ent) + nan, -scale * gh * kLn2, z * kLog2e};
}

template <bool ENT, int N>
__device__ __forceinline__ void grad(float (&e)[N], int32_t label, float m, float c,
                                     const GradCoef &k) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float L = __builtin_fmaf(c, e[i] - m, -k.z2);
    if (ENT) L = fmaxf(L, kLeast);
    const float p = __builtin_amdgcn_exp2f(L);
    e[i] = p * (ENT ? __builtin_fmaf(k.k1, L, k.k0) : k.k0);
  }
  if (uint32_t(label) < uint32_t(N)) {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] += i == label ? k.hot : 0.0f;
  }
}

// Zeros, a row's gradient where there is none.
template <bool BF16, int threads>
__device__ __forceinline__ void zero_row(char *out, int32_t V) {
  constexpr int W = kGroup<BF16>;
  const float e[W] = {};
  const Cut<BF16> k(out, V);
  for (int32_t v = int32_t(threadIdx.x) * W; v < k.whole; v += threads * W)
    store_group<BF16>(out, k.head + v, e);
  const int32_t one = k.one(int32_t(threadIdx.x));
  if (one < V) store1<BF16>(out, one, 0.0f);
}

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

// ---------------------------------------------------- few, very long rows
//
// Few long rows are cut into segments: a workgroup sums a segment, a wavefront
// joins a row's segments, and the gradient is logp_bwd_kernel's, by segments
// too.

constexpr int kPartThreads = 256, kPartNG = 4;

template <bool BF16, bool ENT>
__global__ __launch_bounds__(kPartThreads) void part_kernel(LogitRows a, const float *weight,
                                                            Stat *part) {
  __shared__ Stat red[kPartThreads / 64];
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int64_t y = a.labels[t];
  if (y < 0 || y >= a.V || (weight && weight[t] == 0.0f)) return;   // nor will it be joined
  const char *row = row_at<BF16>(a.x, t * a.ld);
  const float c = a.scale * kLog2e;
  Held<BF16, kPartThreads, kPartNG> h;
  const Cut<BF16> k(row, int32_t(a.V));
  const int32_t from = int32_t(blockIdx.x) * h.words;
  Stat s = {-INFINITY, 0.0f, 0.0f};
  if (from == 0 || from < k.whole) {
    h.load(row, k, from, from + h.words < k.whole ? from + h.words : k.whole);
    add_chunk<ENT>(s, h, c);
  }
  s = joined_block<kPartThreads>(s, c, red);
  if (threadIdx.x == 0) part[t * gridDim.x + blockIdx.x] = s;
}

// A row to a wavefront.
template <bool BF16>
__device__ __forceinline__ RowResult join_row(const LogitRows &a, const Stat *part, int segments,
                                              int64_t t, int64_t y) {
  const float c = a.scale * kLog2e;
  Stat s = {-INFINITY, 0.0f, 0.0f};
  for (int j = threadIdx.x % 64; j < segments; j += 64) {
    const Stat b = part[t * segments + j];
    const float top = fmaxf(s.m, b.m);
    const Stat x = raised(s, top, c), z = raised(b, top, c);
    s = {top, x.t + z.t, x.w + z.w};
  }
  const char *row = row_at<BF16>(a.x, t * a.ld);
  return finished<BF16, 64>(joined(s, c), row, int32_t(a.V), load1<BF16>(row, uint32_t(y)),
                            a.scale, nullptr);
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

dim3 row_grid(int64_t T, int64_t segments = 1) {
  return dim3(unsigned(segments), unsigned(least64(T, kRowsY)),
              unsigned((T + kRowsY - 1) / kRowsY));
}

constexpr int64_t kFewRows = 64;

int64_t segments_of(int64_t V) {
  constexpr int64_t words = int64_t(kPartThreads) * 8 * kPartNG;
  return (V + words - 1) / words;
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
