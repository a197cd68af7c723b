// The top alternatives of rows of logits, and the loss against a teacher's.
//
// Both hold a row in registers as the other row kernels do (logits.h): each
// logit is read once, and the distillation gradient written once.
//
// Top k (k <= 64).  Words are ordered by value, then by the lower index; as
// 64-bit keys (the value's bits in an order-preserving form, then the index's
// complement) no two are equal.  No row is sorted:
//   1. a bound: the k-th largest of 64 or 128 lane maxima, to the upper 16 or
//      20 bits, by bisection with ballots (two comparisons a bit and wavefront).
//      At least k words reach it, usually few more.
//   2. the words that reach it go to a list in LDS, in any order;
//   3. each entry's place is the number of entries above it.
// A list that overflows (many equal words) is made again with the exact k-th
// key, found by bisection over all 64 bits with counts of the held words.  It is
// right for any row and slow: 4096 x 32000 of 20 words above a mask of -1e9, k = 32,
// 2.3 ms (a mask of -inf 65 us).
// Longer rows repeat this by chunks, the best k so far ahead of the list.
// 4096 x 32000 bf16, a quarter not scored, k = 32: 55 us, 3.6 TB/s of 198 MB
// (a copy 5.1; scoring alone 38.6): beside the loads there are the sums' 10
// operations a word, a maximum, and the list.  One row: 8 us, a chain of waits
// (load, bound, list, places, log p).
//
// Distillation.  With q the teacher's alternatives (their total C),
//   kl = sum_j q_j (ln q_j - log p_(i_j)),  dx_v = w s (C p_v - sum_(i_j = v) q_j);
// entry j lives in lane j of every wavefront, the gradient's ordinary part is
// formed from the registers, and the entries that fall on a wavefront's 64
// groups (a ballot) are subtracted before the group is rounded.
#include "logits.h"

namespace qlora {
namespace {

constexpr int kList = 1024;                 // entries of the list in LDS

// Value order as unsigned integers; -0 and 0 are equal.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
constexpr uint32_t kKeyLeast = 0x007fffffu;   // of -inf
__device__ __forceinline__ uint64_t entry_of(float x, uint32_t v) {
  return uint64_t(key_of(x)) << 32 | uint32_t(~v);
}
__device__ __forceinline__ uint32_t word_of(uint64_t e) { return ~uint32_t(e); }

// The k-th largest of the wavefronts' shared keys (one or two a lane), its low
// bits cut off.
template <bool BF16, bool TWO>
__device__ __forceinline__ uint32_t kth_key(uint32_t a, uint32_t b, int k) {
  constexpr int least = BF16 ? 16 : 12;
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= least; --bit) {
    const uint32_t c = t | 1u << bit;
    int n = __popcll(__ballot(a >= c));
    if (TWO) n += __popcll(__ballot(b >= c));
    t = n >= k ? c : t;
  }
  return t > kKeyLeast ? t : kKeyLeast;
}

struct TopList {
  alignas(16) uint64_t e[kList];
  int n;
};

// How many of the list's n entries are above e.
__device__ __forceinline__ int place_of(const TopList &list, int n, uint64_t e) {
  int r = 0;
  for (int j = 0; j < n; j += 8) {            // (kList is a multiple of 8)
    uint64_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = list.e[j + i];
#pragma unroll
    for (int i = 0; i < 8; ++i) r += j + i < n && v[i] > e;
  }
  return r;
}

// Number of this workgroup's words that f counts, in every lane.
template <int threads, class F>
__device__ __forceinline__ int counted(F &&f, int *sum) {
  int n = f();
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
  __syncthreads();
  if (threadIdx.x % 64 == 0) sum[threadIdx.x / 64] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < threads / 64; ++w) n += sum[w];
  return n;
}

// The largest word of each held group, and of the lane.  A signalling NaN takes the
// words before it along (a maximum makes it a quiet one, which the next drops): what
// comes out is a word of the lane or -inf, but perhaps not the largest.
template <bool BF16, int threads, int NG>
__device__ __forceinline__ float group_maxima(const Held<BF16, threads, NG> &h,
                                              float (&gm)[8 * NG / kGroup<BF16>]) {
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  float top = h.one;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float e[W];
    unpack<BF16>(h.q[g], e);
    gm[g] = e[0];
#pragma unroll
    for (int i = 1; i < W; ++i) gm[g] = fmaxf(gm[g], e[i]);
    top = fmaxf(top, gm[g]);
  }
  return fmaxf(top, -INFINITY);              // (no word but NaN)
}

// Adds a held chunk's best k words (words [from, end) of the groups, and the
// ones with the first) to the list behind its first `have` entries; end - from
// is at most the words that are held, gm and top are theirs (group_maxima), nan
// says that there may be a NaN among the lane's: it then looks into every group (a
// smaller top only lowers the bound).  Returns the new length (every lane).
template <bool BF16, int threads, int NG>
__device__ __forceinline__ int add_best(Held<BF16, threads, NG> &h, const Cut<BF16> &cut,
                                        int32_t from, int32_t end,
                                        const float (&gm)[8 * NG / kGroup<BF16>], float top,
                                        bool nan, int k, int have, TopList &list, uint32_t *keys,
                                        int *sum) {
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  constexpr int share = threads > 128 ? threads / 128 : 1;   // lanes to a key
  const int32_t one = from == 0 ? cut.one(int32_t(threadIdx.x)) : cut.V;
  const bool has_one = one < cut.V;
#pragma unroll
  for (int d = 1; d < share; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (threadIdx.x == 0) list.n = have;
  const int lane = threadIdx.x % 64;
  uint32_t bound;
  if (threads == 64) {
    bound = kth_key<BF16, false>(key_of(top), 0u, k);
    __syncthreads();
  } else {
    if (threadIdx.x % share == 0) keys[threadIdx.x / share] = key_of(top);
    __syncthreads();
    bound = kth_key<BF16, true>(keys[lane], keys[lane + 64], k);
  }
  if (have == k) {
    const uint32_t run = uint32_t(list.e[k - 1] >> 32);      // what is below cannot enter
    bound = run > bound ? run : bound;
  }
  const float least = value_of(bound), skip = nan ? -INFINITY : least;
  // All words reach -inf; of those that are -inf themselves only the first k
  // can be among the best (unless some of them are NaN: fill_masked).
  const bool all = bound == kKeyLeast;
  auto offer = [&](float x, int32_t v) {
    if (x >= least && !(all && x == least && v >= k)) {
      const int at = atomicAdd(&list.n, 1);
      if (at < kList) list.e[at] = entry_of(x, uint32_t(v));
    }
  };
  // f(value, word) of the held words of groups that reach the bound.  The
  // registers are laundered, or what is worked out of them would be kept from
  // one use for the next (four times the registers).
  auto words = [&](auto &&f) {
    h.keep();
    int32_t at = from + h.first(0);
    asm volatile("" : "+v"(at));
    if (has_one) f(h.one, one);
#pragma unroll
    for (int g = 0; g < G; ++g, at += threads * W) {
      if (at >= end || gm[g] < skip) continue;
      float e[W];
      unpack<BF16>(h.q[g], e);
#pragma unroll
      for (int i = 0; i < W; ++i) f(e[i], cut.head + at + i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  words(offer);
  __syncthreads();
  const int n = list.n;
  if (n <= kList) return n;
  // Too many: the k-th largest key of the chunk, exactly.
  __syncthreads();
  if (threadIdx.x == 0) list.n = have;
  uint64_t kth = 0;
#pragma unroll 1
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t c = kth | uint64_t(1) << bit;
    const int m = counted<threads>(
        [&] {
          int s = 0;
          words([&](float x, int32_t v) { s += x >= least && entry_of(x, uint32_t(v)) >= c; });
          return s;
        },
        sum);
    kth = m >= k ? c : kth;
  }
  words([&](float x, int32_t v) {
    const uint64_t e = entry_of(x, uint32_t(v));
    if (x >= least && e >= kth) list.e[atomicAdd(&list.n, 1)] = e;
  });
  __syncthreads();
  return list.n;
}

// A list of all the row's words but the -inf ones from word k on that is shorter
// than k (n entries): there is a NaN among the first k words.  The next -inf words
// go to its end, in order.  For one wavefront, or several that do the same; returns
// the new length.  Only such rows come here; they cost the walk to as many -inf
// words (4096 x 32000 bf16 of NaN alone, which walk to the end: 158 us, without 45).
template <bool BF16>
__device__ __forceinline__ int fill_masked(TopList &list, const char *row, int32_t V, int n,
                                           int k) {
  constexpr int N = 8;
  const int lane = threadIdx.x % 64;
  for (int32_t from = k; from < V && n < k; from += 64 * N) {
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t v = from + 64 * i + lane;
      x[i] = load1<BF16>(row, uint32_t(v < V ? v : V - 1));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t v = from + 64 * i + lane;
      const bool hit = v < V && x[i] == -INFINITY;
      const uint64_t hits = __ballot(hit);
      const int at = n + __popcll(hits & ((uint64_t(1) << lane) - 1));
      if (hit && at < k) list.e[at] = entry_of(x[i], uint32_t(v));
      n += __popcll(hits);
    }
  }
  __builtin_amdgcn_wave_barrier();
  return n < k ? n : k;
}

// The best min(n, k) of the list's n entries to its front, in order.
template <int threads>
__device__ __forceinline__ void order(TopList &list, int n, int k) {
  constexpr int per = kList / threads;
  uint64_t own[per];
  int place[per];
#pragma unroll
  for (int q = 0; q < per; ++q) {
    const int i = int(threadIdx.x) + q * threads;
    place[q] = k;
    if (i >= n) continue;
    own[q] = list.e[i];
    place[q] = place_of(list, n, own[q]);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < per; ++q)
    if (place[q] < k) list.e[place[q]] = own[q];
  __syncthreads();
}

// Alternative j of row t.
__device__ __forceinline__ void write_entry(const TopRows &o, int64_t t, int j, bool some,
                                            uint64_t e, const RowResult &r, float scale) {
  o.ids[t * o.k + j] = some ? int32_t(word_of(e)) : -1;
  const float x = value_of(uint32_t(e >> 32));
  // a row of nothing but -inf has m = -inf
  o.top[t * o.k + j] =
      r.z != r.z ? r.z : !(x > -INFINITY) ? -INFINITY : scale * (x - r.m) - r.z;
}

__device__ __forceinline__ void write_row(const TopRows &o, int64_t t, const RowResult &r) {
  if (o.logp) o.logp[t] = r.logp;
  if (o.entropy) o.entropy[t] = r.ent;
}

// A row's alternatives from its list's best n, which are in order (fewer than
// k: NaN has left no more).
template <int threads>
__device__ __forceinline__ void write_top(const TopRows &o, int64_t t, const TopList &list, int n,
                                          const RowResult &r, float scale) {
  for (int j = threadIdx.x; j < o.k; j += threads)
    write_entry(o, t, j, j < n, j < n ? list.e[j] : 0, r, scale);
  if (threadIdx.x == 0) write_row(o, t, r);
}

template <int threads>
__device__ __forceinline__ void write_unscored(const TopRows &o, int64_t t) {
  for (int j = threadIdx.x; j < o.k; j += threads) {
    o.ids[t * o.k + j] = -1;
    o.top[t * o.k + j] = 0.0f;
  }
  if (threadIdx.x == 0) {
    if (o.logp) o.logp[t] = 0.0f;
    if (o.entropy) o.entropy[t] = 0.0f;
  }
}

// The label of row t (word 0 where none are given); false: not scored.
__device__ __forceinline__ bool row_label(const LogitRows &a, int64_t t, int32_t &y) {
  const int64_t v = a.labels ? a.labels[t] : 0;
  y = int32_t(v);
  return v >= 0 && v < a.V;
}

// ONE: the row is held whole (a loop over chunks costs its invariants' registers).
// bf16 rows of one chunk: 8 wavefronts to a SIMD (64 registers; 4096 x 32000 58.2
// -> 56.6 us, though a lane spills three, 12.5 MB of writes beside 1.1 of results).
template <bool BF16, bool ENT, bool ONE, int threads, int NG>
__global__ __launch_bounds__(threads, ONE && BF16 ? 8 : 1) void top_kernel(LogitRows a, TopRows o) {
  __shared__ Stat red[threads / 64];
  __shared__ TopList list;
  __shared__ uint32_t keys[threads < 128 ? threads : 128];
  __shared__ int sum[threads / 64];
  const int64_t t = row_index();
  if (t >= a.T) return;
  int32_t y;
  if (!row_label(a, t, y)) return write_unscored<threads>(o, t);
  const char *row = row_at<BF16>(a.x, t * a.ld);
  const int32_t V = int32_t(a.V);
  const float c = a.scale * kLog2e;
  const Cut<BF16> k(row, V);
  Held<BF16, threads, NG> h;
  Stat s = {-INFINITY, 0.0f, 0.0f};
  int n = 0;
  int32_t from = 0, end = ONE ? k.whole : first_chunk<Held<BF16, threads, NG>::words>(k.whole);
  h.load(row, k, from, end);
  const float xy = load1<BF16>(row, uint32_t(y));
  for (;;) {
    float gm[8 * NG / kGroup<BF16>];
    const float top = group_maxima(h, gm);
    add_sums<ENT>(s, h, c, fmaxf(s.m, top));
    asm volatile("" : "+v"(s.t), "+v"(s.w));   // (w now, not later with all its terms)
    if (ONE) {
      // (the barriers of add_best come before the sums are read)
      s = joined(s, c);
      if (threads > 64 && threadIdx.x % 64 == 0) red[threadIdx.x / 64] = s;
    }
    n = add_best(h, k, from, end, gm, top, s.t != s.t, o.k, n, list, keys, sum);
    if (ONE) break;
    order<threads>(list, n, o.k);
    n = n < o.k ? n : o.k;
    if (end >= k.whole) break;
    from = end;
    end += h.words;
    h.load(row, k, from, end);
  }
  if (ONE) {
    // A short list, as it nearly always is, is one wavefront's: an entry a lane.
    const int lane = threadIdx.x % 64;
    const bool lone = n <= 64;
    if (lone && threadIdx.x >= 64) return;
    if (threads > 64)
      s = joined(lane < threads / 64 ? red[lane] : Stat{-INFINITY, 0.0f, 0.0f}, c);
    if (lone) {
      if (n < o.k) n = fill_masked<BF16>(list, row, V, n, o.k);
      const RowResult r = finished<BF16, 64>(s, row, V, xy, a.scale, nullptr);
      const uint64_t e = lane < n ? list.e[lane] : 0;
      const int j = lane < n ? place_of(list, n, e) : lane;
      if (j < o.k) write_entry(o, t, j, lane < n, e, r, a.scale);
      if (lane == 0) write_row(o, t, r);
      return;
    }
    order<threads>(list, n, o.k);
    n = n < o.k ? n : o.k;
  } else {
    if (n < o.k) {
      n = fill_masked<BF16>(list, row, V, n, o.k);
      __syncthreads();
    }
    s = joined_block<threads>(s, c, red);
  }
  const RowResult r = finished<BF16, threads>(s, row, V, xy, a.scale, red);
  write_top<threads>(o, t, list, n, r, a.scale);
}

// Few long rows: a segment's sums and best k; a workgroup joins a row's.
template <bool BF16, bool ENT>
__global__ __launch_bounds__(kPartThreads) void top_part_kernel(LogitRows a, int k, Stat *part,
                                                                uint64_t *best) {
  __shared__ Stat red[kPartThreads / 64];
  __shared__ TopList list;
  __shared__ uint32_t keys[128];
  __shared__ int sum[kPartThreads / 64];
  const int64_t t = row_index();
  if (t >= a.T) return;
  int32_t y;
  if (!row_label(a, t, y)) return;                         // nor will it be joined
  const char *row = row_at<BF16>(a.x, t * a.ld);
  const float c = a.scale * kLog2e;
  Held<BF16, kPartThreads, kPartNG> h;
  const Cut<BF16> cut(row, int32_t(a.V));
  const int32_t from = int32_t(blockIdx.x) * h.words;
  const int32_t end = from + h.words < cut.whole ? from + h.words : cut.whole;
  Stat s = {-INFINITY, 0.0f, 0.0f};
  int n = 0;
  if (from == 0 || from < cut.whole) {
    h.load(row, cut, from, end);
    float gm[8 * kPartNG / kGroup<BF16>];
    const float top = group_maxima(h, gm);
    add_sums<ENT>(s, h, c, top);
    asm volatile("" : "+v"(s.t), "+v"(s.w));   // (w now, not later with all its terms)
    n = add_best(h, cut, from, end, gm, top, s.t != s.t, k, 0, list, keys, sum);
    order<kPartThreads>(list, n, k);
  }
  const int64_t at = t * gridDim.x + blockIdx.x;
  for (int j = threadIdx.x; j < k; j += kPartThreads) best[at * k + j] = j < n ? list.e[j] : 0;
  s = joined_block<kPartThreads>(s, c, red);
  if (threadIdx.x == 0) part[at] = s;
}

constexpr int kJoinThreads = 512;

template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void top_join_kernel(LogitRows a, TopRows o,
                                                                const Stat *part,
                                                                const uint64_t *best,
                                                                int segments) {
  __shared__ TopList list;
  const int64_t t = row_index();
  if (t >= a.T) return;
  int32_t y;
  if (!row_label(a, t, y)) return write_unscored<kJoinThreads>(o, t);
  const int all = segments * o.k;
  const uint64_t *b = best + t * all;
  int n = 0;
  for (int at = 0; at < all;) {
    const int take = all - at < kList - n ? all - at : kList - n;
    for (int j = threadIdx.x; j < take; j += kJoinThreads) list.e[n + j] = b[at + j];
    __syncthreads();
    order<kJoinThreads>(list, n + take, o.k);
    at += take;
    // places that no segment filled are 0: all of them have the place behind
    // the last word, and what is behind that is old
    const int lane = threadIdx.x % 64;
    const uint64_t full = __ballot(lane < o.k && lane < n + take && list.e[lane] != 0);
    n = full == ~uint64_t(0) ? 64 : __ffsll((unsigned long long)~full) - 1;
    __syncthreads();
  }
  if (n < o.k) {
    n = fill_masked<BF16>(list, row_at<BF16>(a.x, t * a.ld), int32_t(a.V), n, o.k);
    __syncthreads();
  }
  const RowResult r = join_row<BF16>(a, part, segments, t, y);
  write_top<kJoinThreads>(o, t, list, n, r, a.scale);
}

// Lanes and groups as in logp_fwd, whose bits the log p and the entropy so have.
template <bool BF16, bool ENT>
void top(const LogitRows &a, const TopRows &o, float *part, uint64_t *best, hipStream_t s) {
  if (const int64_t n = forward_segments(a.T, a.V, BF16)) {
    Stat *q = reinterpret_cast<Stat *>(part);
    hipLaunchKernelGGL((top_part_kernel<BF16, ENT>), row_grid(a.T, n), dim3(kPartThreads), 0, s, a,
                       o.k, q, best);
    hipLaunchKernelGGL((top_join_kernel<BF16>), row_grid(a.T), dim3(kJoinThreads), 0, s, a, o, q,
                       best, int(n));
    return;
  }
#define ROWS(ONE, threads, NG)                                                                  \
  hipLaunchKernelGGL((top_kernel<BF16, ENT, ONE, threads, NG>), row_grid(a.T), dim3(threads), 0, \
                     s, a, o)
  if (a.V <= 2048) ROWS(true, 64, 4);
  else if (a.V <= 4096) ROWS(false, 64, 4);
  else if (a.V <= 8192) ROWS(true, 128, 8);
  else if (a.V <= 16384) ROWS(true, 256, 8);
  else if (a.V <= 32768) ROWS(true, 512, 8);
  else ROWS(false, 512, 8);
#undef ROWS
}

// --------------------------------------------------------------- distillation

// Lane j's alternative: its word (V where there is none), its probability and
// the logarithm of that; total in every lane.
struct Alternative {
  int32_t id;
  float q, lnq, total;
  bool any;                // some lane has a probability that is not 0
};

__device__ __forceinline__ Alternative alternative(const DistillRows &d, int64_t t, int32_t V) {
  const int lane = threadIdx.x % 64;
  Alternative r;
  r.id = lane < d.k ? d.ids[t * d.k + lane] : -1;
  if (r.id < 0 || r.id >= V) r.id = V;
  const float x = r.id < V ? d.logt[t * d.k + lane] : -INFINITY;
  if (d.normalize) {
    const float top = wave_max(x);
    const float e = x == -INFINITY ? 0.0f : expf(x - top);   // (top may be -inf)
    const float c = wave_sum(e);
    r.q = e == 0.0f ? 0.0f : e / c;
    r.lnq = (x - top) - logf(c);
    r.total = c == c ? 1.0f : c;
  } else {
    r.q = expf(x);
    r.lnq = x;
    r.total = wave_sum(r.q);
  }
  r.any = __ballot(r.q != 0.0f) != 0;
  return r;
}

// kl of a row whose words' logits x (each lane's own) are given.
__device__ __forceinline__ float row_kl(const Alternative &b, float x, const RowResult &r,
                                        float scale) {
  // a student that cannot give a word (x = -inf, or a row of nothing else)
  const float lp = x == -INFINITY ? (r.z != r.z ? r.z : -INFINITY) : scale * (x - r.m) - r.z;
  return wave_sum(b.q == 0.0f ? 0.0f : b.q * (b.lnq - lp));
}

// The alternatives that fall on one group of each lane of a wavefront, whose
// first word (past the row's head) is base + lane * N, subtracted from it.
template <int N>
__device__ __forceinline__ void subtract(float (&e)[N], int32_t base, int32_t end,
                                         int32_t head, const Alternative &b, float coef) {
  const int32_t rel = b.id - head - base;
  uint64_t hit = __ballot(b.id - head < end && uint32_t(rel) < uint32_t(64 * N));
  const int lane = threadIdx.x % 64;
  while (hit) {
    const int j = __ffsll((unsigned long long)hit) - 1;
    hit &= hit - 1;
    const int at = __builtin_amdgcn_readlane(rel, j);
    const float q = __uint_as_float(
        uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(b.q)), j)));
    const float v = lane == at / N ? coef * q : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] -= i == at % N ? v : 0.0f;
  }
}

// The same for the words outside the groups, one to a lane.
__device__ __forceinline__ void subtract_one(float &e, int32_t word, int32_t whole, int32_t V,
                                             int32_t head, const Alternative &b, float coef) {
  uint64_t hit = __ballot(b.id < V && uint32_t(b.id - head) >= uint32_t(whole));
  while (hit) {
    const int j = __ffsll((unsigned long long)hit) - 1;
    hit &= hit - 1;
    const int at = __builtin_amdgcn_readlane(b.id, j);
    const float q = __uint_as_float(
        uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(b.q)), j)));
    if (word == at) e -= coef * q;
  }
}

template <bool BF16, int threads, int NG>
__global__ __launch_bounds__(threads) void distill_kernel(LogitRows a, DistillRows d, float *kl,
                                                          void *dx, int64_t ldd) {
  __shared__ Stat red[threads / 64];
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int32_t V = int32_t(a.V);
  const char *row = row_at<BF16>(a.x, t * a.ld);
  char *out = row_at<BF16>(dx, t * ldd);
  const float w = d.weight ? d.weight[t] : 1.0f;
  float loss = 0.0f;
  bool some = false;
  if (w != 0.0f) {
    constexpr int W = kGroup<BF16>, G = 8 * NG / W;
    const Cut<BF16> q(row, V);
    Held<BF16, threads, NG> h;
    h.load(row, q, 0, q.whole);
    const Alternative b = alternative(d, t, V);
    if (b.any) {
      const float c = a.scale * kLog2e, coef = a.scale * w;
      float x = b.id < V ? load1<BF16>(row, uint32_t(b.id)) : -INFINITY;
      Stat s = {-INFINITY, 0.0f, 0.0f};
      add_chunk<false>(s, h, c);
      asm volatile("" : "+v"(x));              // here before the barrier: dx may be the logits
      s = joined_block<threads>(s, c, red);
      const RowResult r = finished<BF16, threads>(s, row, V, 0.0f, a.scale, red);
      loss = row_kl(b, x, r, a.scale);
      some = r.m != -INFINITY;
      if (some) {
        const GradCoef kc = grad_coef(a.scale, -w * b.total, 0.0f, 0.0f, r.z);
        h.keep();
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int32_t v = h.first(i);
          float e[W];
          unpack<BF16>(h.q[i], e);
          grad<false>(e, -1, r.m, c, kc);
          subtract<W>(e, v - int(threadIdx.x) % 64 * W, q.whole, q.head, b, coef);
          if (v < q.whole) store_group<BF16>(out, q.head + v, e);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (threadIdx.x < 64) {
          const int32_t one = q.one(int32_t(threadIdx.x));
          float e[1] = {h.one};
          grad<false>(e, -1, r.m, c, kc);
          subtract_one(e[0], one, q.whole, V, q.head, b, coef);
          if (one < V) store1<BF16>(out, one, e[0]);
        }
      }
    }
  }
  if (!some) zero_row<BF16, threads>(out, V);
  if (threadIdx.x == 0) kl[t] = loss;
}

// Longer rows: segments' sums (part_kernel), a wavefront to a row's (m, z) and
// kl, then the gradient by segments.
template <bool BF16>
__global__ __launch_bounds__(64) void distill_join_kernel(LogitRows a, DistillRows d,
                                                          const Stat *part, int segments,
                                                          float *stats, float *kl) {
  const int64_t t = row_index();
  if (t >= a.T) return;
  const float w = d.weight ? d.weight[t] : 1.0f;
  float loss = 0.0f;
  RowResult r = {-INFINITY, 0.0f, 0.0f, 0.0f};             // m = -inf: no gradient
  if (w != 0.0f) {
    const Alternative b = alternative(d, t, int32_t(a.V));
    if (b.any) {
      const char *row = row_at<BF16>(a.x, t * a.ld);
      const float x = b.id < a.V ? load1<BF16>(row, uint32_t(b.id)) : -INFINITY;
      r = join_row<BF16>(a, part, segments, t, 0);
      loss = row_kl(b, x, r, a.scale);
    }
  }
  if (threadIdx.x == 0) {
    kl[t] = loss;
    stats[2 * t] = r.m;
    stats[2 * t + 1] = r.z;
  }
}

template <bool BF16, int threads, int NG>
__global__ __launch_bounds__(threads) void distill_bwd_kernel(LogitRows a, DistillRows d,
                                                              const float *stats, void *dx,
                                                              int64_t ldd) {
  const int64_t t = row_index();
  if (t >= a.T) return;
  const int32_t V = int32_t(a.V);
  const char *row = row_at<BF16>(a.x, t * a.ld);
  char *out = row_at<BF16>(dx, t * ldd);
  const Cut<BF16> q(row, V);
  constexpr int W = kGroup<BF16>, G = 8 * NG / W;
  const int32_t from = (int32_t(blockIdx.x) * threads * G + int32_t(threadIdx.x)) * W;
  const int32_t one = blockIdx.x == 0 ? q.one(int32_t(threadIdx.x)) : V;
  const float m = stats[2 * t], z = stats[2 * t + 1];
  if (m != -INFINITY) {
    const float w = d.weight ? d.weight[t] : 1.0f;
    const Alternative b = alternative(d, t, V);
    const float c = a.scale * kLog2e, coef = a.scale * w;
    const GradCoef kc = grad_coef(a.scale, -w * b.total, 0.0f, 0.0f, z);
    float f[G][W];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int32_t v = from + i * threads * W;
#pragma unroll
      for (int e = 0; e < W; ++e) f[i][e] = 0.0f;
      if (v < q.whole) unpack<BF16>(load_group<BF16>(row, q.head + v), f[i]);
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int32_t v = from + i * threads * W;
      grad<false>(f[i], -1, m, c, kc);
      subtract<W>(f[i], v - int(threadIdx.x) % 64 * W, q.whole, q.head, b, coef);
      if (v < q.whole) store_group<BF16>(out, q.head + v, f[i]);
    }
    if (blockIdx.x == 0 && threadIdx.x < 64) {
      float e[1] = {one < V ? load1<BF16>(row, one) : 0.0f};
      grad<false>(e, -1, m, c, kc);
      subtract_one(e[0], one, q.whole, V, q.head, b, coef);
      if (one < V) store1<BF16>(out, one, e[0]);
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

template <bool BF16>
void distill(const LogitRows &a, const DistillRows &d, float *kl, void *dx, int64_t ldd,
             float *part, float *stats, hipStream_t s) {
  if (const int64_t n = distill_segments(a.V)) {
    Stat *q = reinterpret_cast<Stat *>(part);
    constexpr int threads = 256, NG = BF16 ? 2 : 1;
    hipLaunchKernelGGL((part_kernel<BF16, false, false>), row_grid(a.T, n), dim3(kPartThreads), 0,
                       s, a, d.weight, q);
    hipLaunchKernelGGL((distill_join_kernel<BF16>), row_grid(a.T), dim3(64), 0, s, a, d, q, int(n),
                       stats, kl);
    const int64_t m = (a.V + threads * 8 * NG - 1) / (threads * 8 * NG);
    hipLaunchKernelGGL((distill_bwd_kernel<BF16, threads, NG>), row_grid(a.T, m), dim3(threads), 0,
                       s, a, d, stats, dx, ldd);
    return;
  }
#define ROWS(threads, NG)                                                                      \
  hipLaunchKernelGGL((distill_kernel<BF16, threads, NG>), row_grid(a.T), dim3(threads), 0, s, a, \
                     d, kl, dx, ldd)
  if (a.V <= 2048) ROWS(64, 4);
  else if (a.V <= 4096) ROWS(128, 4);
  else if (a.V <= 8192) ROWS(256, 4);
  else if (a.V <= 16384) ROWS(512, 4);
  else if (a.V <= 32768) ROWS(512, 8);
  else ROWS(1024, 8);
#undef ROWS
}

// sum weight kl in fp64: a workgroup's share, the whole where there is one.
constexpr int kSumThreads = 1024;
constexpr int64_t kSumLone = 8192;

__device__ __forceinline__ void block_total(double v, float *out, double *partial) {
  __shared__ double red[kSumThreads / 64];
  double s[1] = {v};
  block_sums<1, kSumThreads>(s, red);
  if (threadIdx.x == 0) {
    if (partial)
      partial[blockIdx.x] = s[0];
    else
      out[0] = float(s[0]);
  }
}

__global__ __launch_bounds__(kSumThreads) void weighted_sum_kernel(const float *kl,
                                                                   const float *weight, int64_t T,
                                                                   float *out, double *partial) {
  const int64_t step = int64_t(gridDim.x) * kSumThreads;
  double s = 0.0;
  for (int64_t t = int64_t(blockIdx.x) * kSumThreads + threadIdx.x; t < T; t += 4 * step) {
    float w[4], x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = t + i * step < T ? t + i * step : t;
      w[i] = weight ? weight[at] : 1.0f;
      x[i] = kl[at];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i * step < T && w[i] != 0.0f) s += double(w[i]) * double(x[i]);
  }
  block_total(s, out, partial);
}

__global__ __launch_bounds__(kSumThreads) void last_sum_kernel(const double *partial, int n,
                                                               float *out) {
  block_total(int(threadIdx.x) < n ? partial[threadIdx.x] : 0.0, out, nullptr);
}

}  // namespace

// Rows that a workgroup does not hold are read twice, by segments.
int64_t distill_segments(int64_t V) { return V > 65536 ? segments_of(V) : 0; }

hipError_t launch_top(const LogitRows &a, const TopRows &o, float *part, uint64_t *best,
                      hipStream_t s) {
#define GO(B) (o.entropy ? top<B, true>(a, o, part, best, s) : top<B, false>(a, o, part, best, s))
  a.bf16 ? GO(true) : GO(false);
#undef GO
  return hipGetLastError();
}

hipError_t launch_distill(const LogitRows &a, const DistillRows &d, float *kl, void *dx,
                          int64_t ldd, float *part, float *stats, hipStream_t s) {
  a.bf16 ? distill<true>(a, d, kl, dx, ldd, part, stats, s)
         : distill<false>(a, d, kl, dx, ldd, part, stats, s);
  return hipGetLastError();
}

int64_t weighted_sum_blocks(int64_t T) {
  return T <= kSumLone ? 1 : least64((T + kSumThreads - 1) / kSumThreads, kSumThreads);
}

hipError_t launch_weighted_sum(const float *kl, const float *weight, int64_t T, float *out,
                               double *partial, hipStream_t s) {
  const int64_t b = weighted_sum_blocks(T);
  hipLaunchKernelGGL(weighted_sum_kernel, dim3(unsigned(b)), dim3(kSumThreads), 0, s, kl, weight,
                     T, out, b > 1 ? partial : nullptr);
  if (b > 1)
    hipLaunchKernelGGL(last_sum_kernel, dim3(1), dim3(kSumThreads), 0, s, partial, int(b), out);
  return hipGetLastError();
}

}  // namespace qlora
