// Pieces of the row kernels over logits: rows cut at 16-byte boundaries and held
// in registers, their maxima and sums, a row's gradient, and rows cut into
// segments.  The formulas are at the top of logits.hip.
#pragma once

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

// A lane's share of a chunk into its running sums; top: the largest word of both.
template <bool ENT, bool BF16, int threads, int NG>
__device__ __forceinline__ void add_sums(Stat &a, Held<BF16, threads, NG> &h, float c, float top) {
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
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
  add_sums<ENT>(a, h, c, top);
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

// ---------------------------------------------------- few, very long rows
//
// Few long rows are cut into segments: a workgroup sums a segment, a wavefront
// joins a row's segments, and the gradient is logp_bwd_kernel's, by segments
// too.

constexpr int kPartThreads = 256, kPartNG = 4;

// LABELS: rows that are not scored are left out, else only those without weight.
template <bool BF16, bool ENT, bool LABELS = true>
__global__ __launch_bounds__(kPartThreads) void part_kernel(LogitRows a, const float *weight,
                                                            Stat *part) {
  __shared__ Stat red[kPartThreads / 64];
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int64_t y = LABELS ? a.labels[t] : 0;
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
}  // namespace qlora
