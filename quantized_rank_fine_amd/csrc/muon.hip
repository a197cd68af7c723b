// The orthogonalised update of adapter matrices: momentum, Newton-Schulz
// products and the step of theta, for many matrices in a few launches.
//
//   m <- mu m + g,  u = g + mu m (Nesterov), m, or g without momentum,
//   X_0 = u / (|u| + eps),  X_(j+1) = X_j (a I + b G_j + c G_j^2),  G_j = X_j^T X_j,
//   O = X_steps,  theta <- theta - lr (scale O + wd theta),
// X taken with its short side, k <= 256, as columns.
//
// The iterations act on the k x k Gram matrix alone: with P_j = a I + b G_j +
// c G_j^2 (a polynomial of G_0, so all of them commute and are symmetric)
//   G_(j+1) = P_j G_j P_j,   O = X_0 P_0 P_1 ... = u Q / (|u| + eps),
// so a tall matrix is read twice (once for G_0, once for the last product),
// not twice an iteration.  What that costs is digits: Q reaches a^steps on the
// weak directions, and an error e of one of G's eigenvalues moves O by up to
// about 0.15 a^(2 steps) e (3.6e4 e for the usual five steps), so G and
// everything made of it are fp64 throughout (v_mfma_f64_16x16x4_f64; fp32 sums
// would leave O two decimals).  O is rounded to fp32 once.
//
// Launches: Gram partials over slabs of the long side (and the momentum); their
// sum; the k x k iterations, in one wavefront for k <= 16, in one workgroup's LDS
// for k <= 64, else by 16 x 16 tiles, one launch a product; the last product and
// the update.
//
// What bounds them (copy rate 5.1 TB/s, fp64 matrix products 74 TFLOP/s; traced):
//   64 of 4096 x 64: 173 us, of them Gram 43 (226 MB, 5.2 TB/s), iterations 38
//     (18 products of 64^3, 14 of them one after the other, on one CU a matrix:
//     about 23 by the matrix cores), update 72 (320 MB, 4.4 TB/s).
//   4 of rank 200 (11008 and 4096): 250 us, of them momentum 15 (6.3 TB/s), Gram
//     57 (fp64: 19 by the matrix cores), 14 launches of iterations 6.3 each
//     (latency), update 77 (fp64: 35 by the matrix cores, and Q from L2).
//   2 of 4096 x 16: 19 us, three launches of 6 to 7 that wait for each other.
#include <algorithm>
#include <type_traits>

#include "objective.h"
#include "qlora.h"

namespace qlora {
namespace {

// A matrix in the kernels: n long, k short; quads: 16-byte accesses.  span: long
// rows to a Gram workgroup, `splits` of them; apply: long rows to an update
// workgroup (k <= 64); area: where its fp64 scratch begins.  u: the direction, of
// k > 64 (grad, m or an array of its own).
struct MuonMat {
  const float *grad, *u;
  float *m, *theta;
  uint16_t *theta16;
  float *update;
  int64_t n, span, apply, area;
  int32_t k, wide, quads, splits;
  float scale;
};

typedef double f64x4_t __attribute__((ext_vector_type(4)));

// D += A B: lane l holds A[l % 16][l / 16] and B[l / 16][l % 16]; register r of
// D is row l / 16 + 4 r, column l % 16.
__device__ __forceinline__ f64x4_t mfma64(double a, double b, f64x4_t d) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, d, 0, 0, 0);
}

constexpr int kPad = 16;
__host__ __device__ inline int padded(int k) { return (k + kPad - 1) / kPad * kPad; }

// One value's momentum (kStep: advanced here) and the update's direction.
template <bool kStep>
__device__ __forceinline__ float direction(const MuonParams &p, bool has_m, float g, float &m) {
  if (!has_m) return g;
  if (kStep) m = p.mu * m + g;
  return p.nesterov ? g + p.mu * m : m;
}

// Where a lane's values lie: a place that is the same for the wavefront, and the
// lane's distance from it (a scalar and one 32-bit register an address).  The
// common place itself always lies in the array.
struct Place {
  int64_t base;
  uint32_t lane;
};

// The first `live` of N values at a place, the rest 0.  Q: live is 0 or N and
// the values are aligned to them (one load).  No load is conditional: what is
// not live reads the common place and is dropped.
template <int N>
struct Run {
  float v[N];
};
template <bool Q, int N>
__device__ __forceinline__ Run<N> load_run(const float *p, Place at, int live) {
  Run<N> r;
  p += at.base;
  if (Q) {
    __builtin_memcpy(&r, __builtin_assume_aligned(p + (live ? at.lane : 0u), 4 * N), 4 * N);
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = live ? r.v[i] : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = p[i < live ? at.lane + i : 0u];
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = i < live ? r.v[i] : 0.0f;
  }
  return r;
}
template <bool Q, int N>
__device__ __forceinline__ void store_run(float *p, Place at, int live, const Run<N> &r) {
  p += at.base;
  if (Q) {
    if (live) __builtin_memcpy(__builtin_assume_aligned(p + at.lane, 4 * N), &r, 4 * N);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < live) p[at.lane + i] = r.v[i];
  }
}

__device__ __forceinline__ int clamped(int64_t left, int most) {
  return left < most ? (left < 0 ? 0 : int(left)) : most;
}

// f(integral_constant<bool>), f(integral_constant<int>) for uniform values.
template <class F>
__device__ __forceinline__ void with_bool(bool v, F &&f) {
  if (v) f(std::true_type{});
  else f(std::false_type{});
}
template <class F>
__device__ __forceinline__ void with_tiles(int t, F &&f) {
  switch (t) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    default: f(std::integral_constant<int, 4>{}); break;
  }
}

// ------------------------------------------------------------ Gram partials
//
// A wavefront sums u^T u of its long rows for one pair of 64-column blocks, from
// registers: no LDS, no barrier until the end.  The 16 columns of a tile and
// the four rows of a product may be any, so they are chosen for the loads:
//   tall (a long row is k consecutive values): a block of w columns has T = 1, 2
//     or 4 tiles; lane (g, c) loads T consecutive columns T c .. of row 4 s + g,
//     one for each tile: tile t holds columns T c + t.
//   wide (a short row is n consecutive values): lane (g, c) loads four
//     consecutive long rows 4 g .. of column 16 t + c, one for each of four
//     products.
// The momentum is advanced on the way where one wavefront sees every value
// (k <= 64), else by a pass of its own before, which also leaves u.  The four
// wavefronts of a workgroup share a slab's rows and leave the sum of theirs,
// [pair][tile][register][lane] in fp64, tile = 4 ti + tj.
struct Block {
  int first, tiles, width;                     // columns first .. first + width - 1
};
__host__ __device__ __forceinline__ Block block_of(int k, int b, int wide) {
  const int w = k - 64 * b < 64 ? k - 64 * b : 64;
  const int t = (w + 15) / 16;
  return {64 * b, wide ? t : t == 3 ? 4 : t, w};
}
// Short index of element c of tile t.
__host__ __device__ __forceinline__ int column_of(const Block &b, int wide, int t, int c) {
  return b.first + (wide ? 16 * t + c : b.tiles * c + t);
}

constexpr int kGramThreads = 256;
constexpr int kGramRows = 64;                  // long rows that a workgroup takes at a time
constexpr int kPairDoubles = 16 * 256;

__host__ __device__ inline int pairs_of(int k) {
  const int nb = (k + 63) / 64;
  return nb * (nb + 1) / 2;
}

// Matrices to a launch whose arguments describe them.
constexpr int kMuonChunk = 32;
struct MuonChunk {
  int count;
  int first;               // index of mats[0] in the table
  MuonMat mats[kMuonChunk];
};

// Where the first launches find the matrices: in the table, or, of a call of a
// few, in their arguments; the Gram kernels then leave them in the table, and the
// launch that fills it is spared (2 of 4096 x 16: 21.8 -> 19.0 us).
constexpr int kMuonFew = 16;
struct MuonFew {
  MuonMat mats[kMuonFew];
  MuonMat *table;
  __device__ __forceinline__ const MuonMat &operator[](unsigned i) const { return mats[i]; }
  __device__ __forceinline__ void leave(unsigned i) const { table[i] = mats[i]; }
};
struct MuonTable {
  const MuonMat *table;
  __device__ __forceinline__ const MuonMat &operator[](unsigned i) const { return table[i]; }
  __device__ __forceinline__ void leave(unsigned) const {}
};

// A wavefront's 16 long rows of one block of T tiles as the products' operands:
// x[s][t] is tile t's of product s.
template <bool WIDE, bool Q, bool kStep, int T>
struct GramRows;

// tall: rows r .. r + 15, four to a product
template <bool Q, bool kStep, int T>
struct GramRows<false, Q, kStep, T> {
  Run<T> g[4], m[4];
  Place at[4];
  int live[4];
  __device__ __forceinline__ void request(const MuonMat &a, const MuonParams &p, const Block &b,
                                          int64_t r, int64_t end) {
    const int lane = threadIdx.x & 63, grp = lane >> 4, c = lane & 15;
    const int mine = clamped(b.width - T * c, T);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t row = r + 4 * s;
      live[s] = row + grp < end ? mine : 0;
      at[s] = {(row < end ? row : 0) * a.k + b.first, uint32_t(grp * a.k + T * c)};
      g[s] = load_run<Q, T>(kStep ? a.grad : a.u, at[s], live[s]);
      if (kStep) m[s] = a.m ? load_run<Q, T>(a.m, at[s], live[s]) : Run<T>{};
    }
  }
  __device__ __forceinline__ void finish(const MuonMat &a, const MuonParams &p, double (&x)[4][T]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int t = 0; t < T; ++t)
        x[s][t] =
            double(kStep ? direction<true>(p, a.m != nullptr, g[s].v[t], m[s].v[t]) : g[s].v[t]);
      if (kStep && a.m) store_run<Q, T>(a.m, at[s], live[s], m[s]);
    }
  }
};
// wide: long rows r .. r + 15, rows 4 g + s in product s
template <bool Q, bool kStep, int T>
struct GramRows<true, Q, kStep, T> {
  Run<4> g[T], m[T];
  Place at[T];
  int live[T];
  __device__ __forceinline__ void request(const MuonMat &a, const MuonParams &p, const Block &b,
                                          int64_t r, int64_t end) {
    const int lane = threadIdx.x & 63, grp = lane >> 4, c = lane & 15;
    const int mine = clamped(end - (r + 4 * grp), 4);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      live[t] = 16 * t + c < b.width ? mine : 0;
      at[t] = {(b.first + 16 * t) * a.n + (r < end ? r : 0), uint32_t(c * a.n) + 4 * grp};
      g[t] = load_run<Q, 4>(kStep ? a.grad : a.u, at[t], live[t]);
      if (kStep) m[t] = a.m ? load_run<Q, 4>(a.m, at[t], live[t]) : Run<4>{};
    }
  }
  __device__ __forceinline__ void finish(const MuonMat &a, const MuonParams &p, double (&x)[4][T]) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[s][t] =
            double(kStep ? direction<true>(p, a.m != nullptr, g[t].v[s], m[t].v[s]) : g[t].v[s]);
      if (kStep && a.m) store_run<Q, 4>(a.m, at[t], live[t], m[t]);
    }
  }
};

__device__ __forceinline__ void pair_of(int p, int &bi, int &bj) {
  bj = 0;
  while (p > bj) p -= ++bj;
  bi = p;
}

// The rows of a slab that are this wavefront's, for blocks of TI and TJ tiles
// (kSame: one block).  Everything that the products depend on is known here:
// a branch between two products costs the wait for their results.
template <bool kSame, bool WIDE, bool Q, bool kStep, int TI, int TJ>
__device__ __forceinline__ void gram_rows(const MuonMat &a, const MuonParams &p, const Block &bi,
                                          const Block &bj, int64_t from, int64_t end,
                                          f64x4_t (&acc)[4][4]) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  GramRows<WIDE, Q, kStep, TI> x;
  GramRows<WIDE, Q, kStep, TJ> y;
  int64_t r = from + 16 * wave;
  x.request(a, p, bi, r, end);
  if (!kSame) y.request(a, p, bj, r, end);
  for (; r < end; r += kGramRows) {
    double u[4][TI], v[4][TJ];
    x.finish(a, p, u);
    if (!kSame) y.finish(a, p, v);
    // the next rows are on their way while these are multiplied (past the end:
    // nothing is live)
    x.request(a, p, bi, r + kGramRows, end);
    if (!kSame) y.request(a, p, bj, r + kGramRows, end);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < (kSame ? j + 1 : TI); ++i)
          if constexpr (kSame) acc[i][j] = mfma64(u[s][i], u[s][j], acc[i][j]);
          else acc[i][j] = mfma64(u[s][i], v[s][j], acc[i][j]);
  }
}

// ONE: k <= 64.  Q: matrices of 16-byte accesses, or the others (whose loads take
// more registers).
template <bool ONE, bool Q, class Mats>
__global__ __launch_bounds__(kGramThreads, 2) void gram_kernel(Mats mats, MuonParams p,
                                                               double *ws) {
  __shared__ double sum[kPairDoubles];
  const MuonMat a = mats[blockIdx.z];
  if ((a.k <= 64) != ONE || bool(a.quads) != Q || int(blockIdx.x) >= a.splits ||
      int(blockIdx.y) >= pairs_of(a.k))
    return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int bi = 0, bj = 0;
  if (!ONE) pair_of(int(blockIdx.y), bi, bj);
  f64x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  const int64_t from = int64_t(blockIdx.x) * a.span;
  const int64_t end = from + a.span < a.n ? from + a.span : a.n;
  const Block b = block_of(a.k, bi, a.wide), c = block_of(a.k, bj, a.wide);
  with_bool(a.wide, [&](auto WIDE) {
    with_tiles(c.tiles, [&](auto T) {
      constexpr int TJ = decltype(T)::value;
      constexpr bool w = decltype(WIDE)::value;
      if constexpr (w || TJ != 3) {
        if (ONE || bi == bj) gram_rows<true, w, Q, ONE, TJ, TJ>(a, p, b, c, from, end, acc);
        // (all blocks but the last have four tiles)
        else if constexpr (!ONE) gram_rows<false, w, Q, ONE, 4, TJ>(a, p, b, c, from, end, acc);
      }
    });
  });
  // the four wavefronts' sums in their order
  for (int w = 0; w < 4; ++w) {
    __syncthreads();
    if (wave != w) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i >= b.tiles || j >= c.tiles || (bi == bj && i > j)) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          double *s = sum + ((4 * i + j) * 4 + r) * 64 + lane;
          *s = w == 0 ? acc[i][j][r] : *s + acc[i][j][r];
        }
      }
  }
  __syncthreads();
  double *out = ws + a.area + (int64_t(blockIdx.x) * pairs_of(a.k) + blockIdx.y) * kPairDoubles;
  for (int e = threadIdx.x; e < kPairDoubles; e += kGramThreads) {
    const int i = e >> 10, j = (e >> 8) & 3;
    if (i < b.tiles && j < c.tiles && (bi != bj || i <= j)) out[e] = sum[e];
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) mats.leave(blockIdx.z);
}

// The table of the call's matrices, which the other launches read.
__global__ __launch_bounds__(64) void table_kernel(MuonChunk c, MuonMat *table) {
  if (int(threadIdx.x) < c.count) table[c.first + threadIdx.x] = c.mats[threadIdx.x];
}

// The momentum of matrices of k > 64, whose values several wavefronts read, and
// (Nesterov) their direction.
template <class Mats>
__global__ __launch_bounds__(256) void momentum_kernel(Mats mats, MuonParams p) {
  const MuonMat a = mats[blockIdx.y];
  if (a.k <= 64 || !a.m) return;
  const int64_t all = a.n * a.k, step = int64_t(gridDim.x) * 1024;
  for (int64_t first = int64_t(blockIdx.x) * 1024; first < all; first += step) {
    const int live = clamped(all - first - 4 * int(threadIdx.x), 4);
    with_bool(a.quads, [&](auto Q) {
      constexpr bool q = decltype(Q)::value;
      const Place at = {first, 4u * threadIdx.x};
      const Run<4> g = load_run<q, 4>(a.grad, at, live);
      Run<4> m = load_run<q, 4>(a.m, at, live);
      Run<4> u;
#pragma unroll
      for (int i = 0; i < 4; ++i) u.v[i] = direction<true>(p, true, g.v[i], m.v[i]);
      store_run<q, 4>(a.m, at, live, m);
      if (p.nesterov) store_run<q, 4>(const_cast<float *>(a.u), at, live, u);
    });
  }
}

// The k x k matrices of k > 64 (kp x kp, row-major), behind the partials in the
// matrix's area: G, S, H, P and Q in two places.
struct Slots {
  double *G, *S, *H, *P, *Q0, *Q1;
  __device__ __forceinline__ Slots(double *area, int splits, int kp) {
    const int64_t n = int64_t(kp) * kp;
    G = area + int64_t(splits) * pairs_of(kp) * kPairDoubles;
    S = G + n;
    H = S + n;
    P = H + n;
    Q0 = P + n;
    Q1 = Q0 + n;
  }
  __device__ __forceinline__ double *Q(int i) const { return i & 1 ? Q1 : Q0; }
};

// Sum of a matrix's partials into the first, an element to a lane.
__global__ __launch_bounds__(256) void gram_sum_kernel(const MuonMat *table, double *ws) {
  const MuonMat a = table[blockIdx.z];
  const int pairs = pairs_of(a.k);
  if (a.k <= 16 || int(blockIdx.y) >= pairs) return;       // (one tile: tiny_kernel sums it)
  int bi, bj;
  pair_of(int(blockIdx.y), bi, bj);
  const int i = int(blockIdx.x) >> 2, j = int(blockIdx.x) & 3;
  if (i >= block_of(a.k, bi, a.wide).tiles || j >= block_of(a.k, bj, a.wide).tiles ||
      (bi == bj && i > j))
    return;
  double *x =
      ws + a.area + int64_t(blockIdx.y) * kPairDoubles + int(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = int64_t(pairs) * kPairDoubles;
  double s = 0.0;
  for (int b = 0; b < a.splits; b += 8) {
    double v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = b + i < a.splits ? x[(b + i) * n] : 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  if (a.k <= 64) {
    *x = s;
    return;
  }
  // k > 64: into G, both ways round
  const int kp = padded(a.k), e = threadIdx.x;
  const int row = column_of(block_of(a.k, bi, a.wide), a.wide, i, ((e & 63) >> 4) + 4 * (e >> 6));
  const int col = column_of(block_of(a.k, bj, a.wide), a.wide, j, e & 15);
  if (row >= kp || col >= kp) return;
  double *G = Slots(ws + a.area, a.splits, kp).G;
  G[int64_t(row) * kp + col] = s;
  G[int64_t(col) * kp + row] = s;
}

// ---------------------------------------------- k x k iterations, k <= 64
//
// Register r of a product's result is row l / 16 + 4 r, column l % 16 of its
// tile: for the product's step r that is also the layout of a B operand, and of
// an A operand whose matrix is symmetric, as all are here.  So a tile of a
// result feeds the next products as it is.
//
// k <= 16: one tile, one wavefront, no LDS after the partials are summed: 18
// products of four steps for the usual five iterations, 14 of them one after the
// other (H P and Q P need not wait for each other).
__device__ __forceinline__ f64x4_t tile_product(const f64x4_t &a, const f64x4_t &b) {
  f64x4_t d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int s = 0; s < 4; ++s) d = mfma64(a[s], b[s], d);
  return d;
}

// x + b y + c z.
__device__ __forceinline__ f64x4_t combined(f64x4_t x, double b, const f64x4_t &y, double c,
                                            const f64x4_t &z) {
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = __builtin_fma(c, z[r], __builtin_fma(b, y[r], x[r]));
  return x;
}

// 1 / (|u| + eps) from |u|^2; a zero update stays zero.
__device__ __forceinline__ double inverse_norm(double trace, double eps) {
  const double d = sqrt(trace) + eps;
  return d > 0.0 ? 1.0 / d : 0.0;
}

__global__ __launch_bounds__(256) void tiny_kernel(const MuonMat *table, MuonParams p, double *ws) {
  __shared__ double part[4][64];
  const MuonMat a = table[blockIdx.x];
  if (a.k > 16) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double *area = ws + a.area;
  double v = 0.0;                                      // register `wave` of this lane
  for (int q = 0; q < a.splits; q += 32) {
    double w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
      w[i] = area[int64_t(q + i < a.splits ? q + i : q) * kPairDoubles + threadIdx.x];
#pragma unroll
    for (int i = 0; i < 32; ++i) v += q + i < a.splits ? w[i] : 0.0;
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave) return;
  f64x4_t G, Q, I;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    G[r] = part[r][lane];
    I[r] = (lane >> 4) + 4 * r == (lane & 15) ? 1.0 : 0.0;
  }
  const double inv =
      inverse_norm(wave_sum(G[0] * I[0] + G[1] * I[1] + G[2] * I[2] + G[3] * I[3]), p.eps);
  G *= inv * inv;
  Q = I * inv;
  for (int it = 0; it < p.steps; ++it) {
    const f64x4_t S = tile_product(G, G);
    const f64x4_t P = combined(p.a * I, p.b, G, p.c, S);
    if (it + 1 < p.steps) {
      const f64x4_t H = combined(p.a * G, p.b, S, p.c, tile_product(G, S));
      G = tile_product(H, P);
    }
    Q = tile_product(Q, P);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) area[((lane >> 4) + 4 * r) * 16 + (lane & 15)] = Q[r];
}

// 16 < k <= 64: one workgroup, three matrices in LDS: G, S (then P), Q, as tiles
// of registers ([tile][register][lane ^ 4 register], tile = NT ti + tj), so that
// an operand is one contiguous read and a tile's mirror image goes to all banks
// (without the exchange it goes to 8 of 32, and storing took half the time).  A
// product's tiles of the upper triangle are dealt over the wavefronts, kept in
// registers until every read is done, and stored with their mirror images.
template <int NT>
struct Small {
  static constexpr int kp = 16 * NT, tiles = NT * (NT + 1) / 2, size = kp * kp;
  static constexpr int threads = NT == 2 ? 256 : 512, waves = threads / 64;
  static constexpr int bytes = 3 * size * 8;
};

// Register r of a lane in a tile.
__device__ __forceinline__ int in_tile(int r, int lane) { return 64 * r + (lane ^ (4 * r)); }

template <int NT>
__device__ __forceinline__ f64x4_t lds_product(const double *A, const double *B, int ti, int tj) {
  const int lane = threadIdx.x & 63;
  const double *x = A + ti * 256, *y = B + tj * 256;
  // operands four products ahead: left to itself the compiler waits for each
  // pair, and all of them first would leave the products waiting for LDS
  constexpr int N = 4 * NT, ahead = 4;
  double u[N], v[N];
  auto request = [&](int s) {
    u[s] = x[s / 4 * NT * 256 + in_tile(s % 4, lane)];
    v[s] = y[s / 4 * NT * 256 + in_tile(s % 4, lane)];
  };
#pragma unroll
  for (int s = 0; s < ahead; ++s) request(s);
  __builtin_amdgcn_sched_barrier(0);
  f64x4_t d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int s = 0; s < N; ++s) {
    if (s + ahead < N) request(s + ahead);
    __builtin_amdgcn_sched_barrier(0);
    d = mfma64(u[s], v[s], d);
  }
  return d;
}

__device__ __forceinline__ void tile_of_index(int t, int &ti, int &tj) {
  tj = 0;
  while (t > tj) t -= ++tj;
  ti = t;
}

template <int NT>
__device__ __forceinline__ void put_tile(double *M, int ti, int tj, const f64x4_t &d) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r) M[(NT * ti + tj) * 256 + in_tile(r, lane)] = d[r];
  if (ti == tj) return;
  // element (lane / 16 + 4 r, lane % 16) is (lane % 16, lane / 16 + 4 r) there
  double *T = M + (NT * tj + ti) * 256;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    T[in_tile((lane & 15) >> 2, 16 * (lane & 3) + (lane >> 4) + 4 * r)] = d[r];
}

// Element (i, j) of a matrix of tiles.
template <int NT>
__device__ __forceinline__ double &element(double *M, int i, int j) {
  return M[(NT * (i >> 4) + (j >> 4)) * 256 + in_tile((i & 15) >> 2, 16 * (i & 3) + (j & 15))];
}

template <int NT>
__global__ __launch_bounds__(Small<NT>::threads) void small_kernel(const MuonMat *table,
                                                                   MuonParams p, double *ws) {
  using S = Small<NT>;
  const MuonMat a = table[blockIdx.x];
  if ((a.k + 15) / 16 != NT) return;
  extern __shared__ __align__(16) double sq[];
  __shared__ double diagonal[S::kp];
  double *G = sq, *P = sq + S::size, *Q = sq + 2 * S::size;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  double *area = ws + a.area;
  // (a tall matrix of 33 .. 48 columns has four tiles of partials: columns 4 c + t)
  const Block b = block_of(a.k, 0, a.wide);
  constexpr int N = kPairDoubles / S::threads;
  double v[N];
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = area[threadIdx.x + q * S::threads];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int e = threadIdx.x + q * S::threads, ti = e >> 10, tj = (e >> 8) & 3;
    if (tj >= b.tiles || ti > tj) continue;                // (not written)
    const int i = column_of(b, a.wide, ti, ((e & 63) >> 4) + 4 * ((e >> 6) & 3));
    const int j = column_of(b, a.wide, tj, e & 15);
    if (i >= S::kp || j >= S::kp) continue;
    element<NT>(G, i, j) = v[q];
    if (ti < tj) element<NT>(G, j, i) = v[q];
    if (i == j) diagonal[i] = v[q];
  }
  __syncthreads();
  const double inv = inverse_norm(wave_sum(lane < S::kp ? diagonal[lane] : 0.0), p.eps);
  for (int e = threadIdx.x; e < S::size; e += S::threads) {
    G[e] *= inv * inv;
    Q[e] = 0.0;
  }
  __syncthreads();
  if (int(threadIdx.x) < S::kp) element<NT>(Q, threadIdx.x, threadIdx.x) = inv;
  __syncthreads();
  constexpr int per = (S::tiles + S::waves - 1) / S::waves;
  constexpr int both = (2 * S::tiles + S::waves - 1) / S::waves;
  f64x4_t aI;
#pragma unroll
  for (int r = 0; r < 4; ++r) aI[r] = (lane >> 4) + 4 * r == (lane & 15) ? p.a : 0.0;
  for (int it = 0; it < p.steps; ++it) {
    f64x4_t d[both], s[per];
    const bool last = it + 1 == p.steps;
    // S = G G
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int t = wave + q * S::waves;
      if (t >= S::tiles) break;
      int ti, tj;
      tile_of_index(t, ti, tj);
      s[q] = lds_product<NT>(G, G, ti, tj);
      put_tile<NT>(P, ti, tj, s[q]);
    }
    __syncthreads();
    // H = G P = a G + b S + c G S in G's place, P = a I + b G + c S in S's
    f64x4_t g[per];
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int t = wave + q * S::waves;
      if (t >= S::tiles) break;
      int ti, tj;
      tile_of_index(t, ti, tj);
#pragma unroll
      for (int r = 0; r < 4; ++r) g[q][r] = G[(NT * ti + tj) * 256 + in_tile(r, lane)];
      if (!last) d[q] = lds_product<NT>(G, P, ti, tj);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int t = wave + q * S::waves;
      if (t >= S::tiles) break;
      int ti, tj;
      tile_of_index(t, ti, tj);
      if (!last) put_tile<NT>(G, ti, tj, combined(p.a * g[q], p.b, s[q], p.c, d[q]));
      put_tile<NT>(P, ti, tj, combined(ti == tj ? aI : 0.0 * aI, p.b, g[q], p.c, s[q]));
    }
    __syncthreads();
    // G <- H P and Q <- Q P; the last time Q alone
    const int units = (last ? 1 : 2) * S::tiles;
#pragma unroll
    for (int q = 0; q < both; ++q) {
      const int t = wave + q * S::waves;
      if (t >= units) break;
      int ti, tj;
      tile_of_index(t < S::tiles ? t : t - S::tiles, ti, tj);
      d[q] = lds_product<NT>(t < S::tiles ? Q : G, P, ti, tj);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < both; ++q) {
      const int t = wave + q * S::waves;
      if (t >= units) break;
      int ti, tj;
      tile_of_index(t < S::tiles ? t : t - S::tiles, ti, tj);
      put_tile<NT>(t < S::tiles ? Q : G, ti, tj, d[q]);
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < S::size; e += S::threads)
    area[e] = element<NT>(Q, e / S::kp, e % S::kp);
}

// ------------------------------------------------ k x k iterations, k > 64
//
// A workgroup owns one 16 x 16 tile of the upper triangle of a product, its four
// wavefronts a quarter of the sum each; operands come from L2 (both symmetric, so
// every fragment is four runs of 128 bytes).  A launch is latency: 4 matrices of
// rank 200 take 4.5 to 6.3 us, of which 0.3 are products.
// kLast is the last iteration's Q P, with P formed where it is read.
enum MuonStage { kSquare, kPolynomial, kAdvance, kLast };

// A quarter of the operands of a tile of columns 16 t ..: kp / 16 steps of four
// rows, all requested before the first is used (past them the last ones again,
// which the products leave out).  kp <= 16 N; N = 8 where it does (30 of rank 128,
// a launch 9.9 -> 7.4 us).
template <int N>
struct Quarter {
  double v[N];
  __device__ __forceinline__ Quarter(const double *M, int kp, int t, int wave) {
    const int lane = threadIdx.x & 63, steps = kp / 16;
    const double *x = M + int64_t(4 * wave * steps + (lane >> 4)) * kp + 16 * t + (lane & 15);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[4 * (i < steps ? i : steps - 1) * kp];
  }
};

template <int N>
__device__ __forceinline__ f64x4_t part_product(const Quarter<N> &a, const Quarter<N> &b, int kp) {
  f64x4_t d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int i = 0; i < N; ++i) d = mfma64(i < kp / 16 ? a.v[i] : 0.0, b.v[i], d);
  return d;
}

// The wavefronts' quarters in their order; the sum's register r = wave is the
// one that this wavefront returns: its element is row lane / 16 + 4 wave.
__device__ __forceinline__ double joined_part(f64x4_t d, int wave, double (*red)[4][64]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r) red[wave][r][lane] = d[r];
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < 4; ++w) s += red[w][wave][lane];
  return s;
}

// A matrix's tiles are dealt to as few of the 8 XCDs as fill the chip (workgroups
// go round them), so that each L2 fetches only its own matrices: matrix m is on
// XCD m % 8, or on 8 / n neighbouring ones where there are fewer than 8 (4 of
// rank 200, a launch: 6.6 -> 6.4 us).
__device__ __forceinline__ void stage_job(int n, int tiles, int &which, int &t) {
  const int x = int(blockIdx.x) % 8, slot = int(blockIdx.x) / 8;
  if (n >= 8) {
    which = x + 8 * (slot / tiles);
    t = slot % tiles;
  } else {
    const int per = 8 / n;
    which = x / per;
    t = slot * per + x % per;
  }
}
int64_t stage_grid(int64_t n, int64_t tiles) {
  return n >= 8 ? 8 * tiles * ((n + 7) / 8) : 8 * ((tiles + 8 / n - 1) / (8 / n));
}

// One workgroup's tile t of a launch's product (second: of kAdvance's other one).
template <int N>
__device__ __forceinline__ void stage_tile(const MuonMat &a, const MuonParams &p, double *ws,
                                           int stage, int it, int kp, int t, bool second,
                                           double (*red)[4][64], double &norm) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int ti, tj;
  tile_of_index(t, ti, tj);
  const Slots m(ws + a.area, a.splits, kp);
  const int i = 16 * ti + (lane >> 4) + 4 * wave, j = 16 * tj + (lane & 15);
  const int64_t ij = int64_t(i) * kp + j, ji = int64_t(j) * kp + i;
  auto put = [&](double *M, double v) {
    M[ij] = v;
    if (ti < tj) M[ji] = v;
  };
  if (stage == kSquare) {
    const Quarter<N> x(m.G, kp, ti, wave), y(m.G, kp, tj, wave);
    put(m.S, joined_part(part_product(x, y, kp), wave, red));
    return;
  }
  if (stage == kPolynomial) {
    const Quarter<N> x(m.G, kp, ti, wave), y(m.S, kp, tj, wave);
    // the first G is not yet scaled: its powers take the factor here
    double f = 1.0, inv = 1.0;
    if (it == 0) {
      if (wave == 0) {
        double v = 0.0;
        for (int d = lane; d < kp; d += 64) v += m.G[int64_t(d) * (kp + 1)];
        for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
        if (lane == 0) norm = v;
      }
      __syncthreads();
      inv = inverse_norm(norm, p.eps);
      f = inv * inv;
    }
    const double g = f * m.G[ij], s = f * f * m.S[ij];
    const double v = (i == j ? p.a : 0.0) + p.b * g + p.c * s;
    put(m.P, v);
    if (it == 0) put(m.Q1, inv * v);
    if (p.steps > 1)
      put(m.H, p.a * g + p.b * s +
                   p.c * (f * f * f *
                          joined_part(part_product(x, y, kp), wave, red)));
    return;
  }
  if (stage == kLast) {
    const Quarter<N> x(m.Q(it), kp, ti, wave), g(m.G, kp, tj, wave);
    Quarter<N> y(m.S, kp, tj, wave);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const bool diagonal = 4 * (wave * (kp / 16) + e) + (lane >> 4) == 16 * tj + (lane & 15);
      y.v[e] = (diagonal ? p.a : 0.0) + p.b * g.v[e] + p.c * y.v[e];
    }
    put(m.Q(it + 1), joined_part(part_product(x, y, kp), wave, red));
    return;
  }
  // kAdvance: G <- H P or, past the first, Q' = Q P
  if (second && it == 0) return;
  const Quarter<N> x(second ? m.Q(it) : m.H, kp, ti, wave), y(m.P, kp, tj, wave);
  put(second ? m.Q(it + 1) : m.G, joined_part(part_product(x, y, kp), wave, red));
}

__global__ __launch_bounds__(256) void stage_kernel(const MuonMat *table, MuonParams p, double *ws,
                                                    int stage, int it, int n, int tiles) {
  __shared__ double red[4][4][64];
  __shared__ double norm;
  int which, t;
  stage_job(n, tiles, which, t);
  if (which >= n || t >= tiles) return;
  const MuonMat a = table[which];
  if (a.k <= 64) return;
  const int kp = padded(a.k), NT = kp / 16;
  const bool second = t >= NT * (NT + 1) / 2;              // (kAdvance: the other product)
  if (second) t -= NT * (NT + 1) / 2;
  if (t >= NT * (NT + 1) / 2 || (second && stage != kAdvance)) return;
  if (kp <= 128)
    stage_tile<8>(a, p, ws, stage, it, kp, t, second, red, norm);
  else
    stage_tile<16>(a, p, ws, stage, it, kp, t, second, red, norm);
}

// ------------------------------------------------------------ the update
//
// O = u Q and theta's step.  The operands and results of a product are again
// chosen for the memory: u comes straight into registers, four values of a lane
// at a time, and a lane's results of all tiles are neighbours.

// A value's step from its X.
__device__ __forceinline__ float stepped(const MuonParams &p, float scale, float th, float x) {
  return th - p.lr * (scale * x + p.wd * th);
}

template <bool Q, int N>
__device__ __forceinline__ void update_run(const MuonMat &a, const MuonParams &p, Place at,
                                           int live, const Run<N> &x, Run<N> th) {
  if (a.update) store_run<Q, N>(a.update, at, live, x);
  if (!a.theta) return;
#pragma unroll
  for (int i = 0; i < N; ++i) th.v[i] = stepped(p, a.scale, th.v[i], x.v[i]);
  store_run<Q, N>(a.theta, at, live, th);
  if (!a.theta16) return;
  if constexpr (Q && N > 1) {
    if (live) {
      uint32_t h[N / 2];
#pragma unroll
      for (int i = 0; i < N; i += 2) h[i / 2] = pack_bf16x2(th.v[i], th.v[i + 1]);
      __builtin_memcpy(__builtin_assume_aligned(a.theta16 + at.base + at.lane, 2 * N), h, 2 * N);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < live)
        (a.theta16 + at.base)[at.lane + i] = __builtin_bit_cast(uint16_t, (__bf16)th.v[i]);
  }
}

// k <= 64: a wavefront to 16 long rows (tall) or 32 (wide) at a time, no barrier
// between them; Q is in LDS, or of k <= 32 in registers.
//   tall: lane (g, c) loads columns 16 j + 4 g .. + 3 of row c, the operands of
//     four products; tile t has columns NT c + t.
//   wide: lane (g, c) loads long rows 2 c, 2 c + 1 of column 4 s + g, the operands
//     of two tiles; a result's rows are short.
// A lane's Q: row 16 j + 4 g + e, columns NT c .. (tall), or row 4 s + g, columns
// c, 16 + c .. (wide), as the products ask for them.
template <int NT>
struct Factor {
  static constexpr bool held = NT <= 2;
  static constexpr int K = 16 * NT, pitch = K + 2;
  double v[held ? 4 * NT : 1][held ? NT : 1];
  const double *lds;
  // Between two uses: or the compiler keeps what it has read from LDS, twice the
  // registers of everything else.
  __device__ __forceinline__ void again() {
    if constexpr (!held) asm volatile("" : "+v"(lds));
  }
  template <bool WIDE>
  __device__ __forceinline__ void init(const double *q, int kp, double *shared) {
    if constexpr (held) {
      const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
#pragma unroll
      for (int s = 0; s < 4 * NT; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int row = WIDE ? 4 * s + g : 16 * (s / 4) + 4 * g + s % 4;
          v[s][t] = q[row * kp + (WIDE ? 16 * t + c : NT * c + t)];   // (kp = K here)
        }
    } else {
      for (int e = threadIdx.x; e < K * K; e += 256) {
        const int i = e / K, j = e % K;
        shared[i * pitch + j] = i < kp && j < kp ? q[i * kp + j] : 0.0;
      }
      lds = shared;
      __syncthreads();
    }
  }
  // of product s (tall: s = 4 j + e)
  template <bool WIDE>
  __device__ __forceinline__ double at(int s, int t) const {
    if constexpr (held) return v[s][t];
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    return WIDE ? lds[(4 * s + g) * pitch + 16 * t + c]
                : lds[(16 * (s / 4) + 4 * g + s % 4) * pitch + NT * c + t];
  }
};

template <int NT, bool Q>
struct TallRows {
  Run<4> gr[NT], m[NT];
  Run<NT> th[4];
  int mine;
  __device__ __forceinline__ Place place(const MuonMat &a, int64_t r, int64_t end, int i) const {
    const int lane = threadIdx.x & 63;
    return {(r + 4 * i < end ? r + 4 * i : 0) * a.k,
            uint32_t((lane >> 4) * a.k + NT * (lane & 15))};
  }
  __device__ __forceinline__ int live(int64_t r, int64_t end, int i) const {
    return r + 4 * i + ((threadIdx.x & 63) >> 4) < end ? mine : 0;
  }
  __device__ __forceinline__ void request(const MuonMat &a, const MuonParams &p, int64_t r,
                                          int64_t end) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const bool has_m = a.m != nullptr, read_g = !has_m || p.nesterov;
    mine = clamped(a.k - NT * c, NT);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int live = r + c < end ? clamped(a.k - 16 * j - 4 * g, 4) : 0;
      const Place at = {(r < end ? r : 0) * a.k + (16 * j < a.k ? 16 * j : 0),
                        uint32_t(c * a.k + 4 * g)};
      gr[j] = read_g ? load_run<Q, 4>(a.grad, at, live) : Run<4>{};
      m[j] = has_m ? load_run<Q, 4>(a.m, at, live) : Run<4>{};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      th[i] = a.theta ? load_run<Q, NT>(a.theta, place(a, r, end, i), live(r, end, i)) : Run<NT>{};
  }
};

template <int NT, bool Q>
__device__ __forceinline__ void apply_tall(const MuonMat &a, const MuonParams &p,
                                           const Factor<NT> &f, int64_t r, int64_t end,
                                           TallRows<NT, Q> &x) {
  const bool has_m = a.m != nullptr;
  double u[4 * NT];
#pragma unroll
  for (int s = 0; s < 4 * NT; ++s)
    u[s] = double(direction<false>(p, has_m, x.gr[s / 4].v[s % 4], x.m[s / 4].v[s % 4]));
  Run<NT> th[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) th[i] = x.th[i];
  // the next rows are on their way meanwhile (past the end: nothing is live)
  x.request(a, p, r + 64, end);
  f64x4_t d[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) d[t] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  double y[2][NT];                             // a product's Q, and the next one's
#pragma unroll
  for (int t = 0; t < NT; ++t) y[0][t] = f.template at<false>(0, t);
#pragma unroll
  for (int s = 0; s < 4 * NT; ++s) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (s + 1 < 4 * NT) y[(s + 1) & 1][t] = f.template at<false>(s + 1, t);
    if (!Factor<NT>::held) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < NT; ++t) d[t] = mfma64(u[s], y[s & 1][t], d[t]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Run<NT> v;
#pragma unroll
    for (int t = 0; t < NT; ++t) v.v[t] = float(d[t][i]);
    update_run<Q, NT>(a, p, x.place(a, r, end, i), x.live(r, end, i), v, th[i]);
  }
}

template <int NT, bool Q>
struct WideRows {
  // four products' operands in hand, four on their way
  Run<2> gr[2][4], m[2][4];
  // column (row of memory) 4 s + g
  __device__ __forceinline__ Place place(const MuonMat &a, int64_t r, int64_t end, int s) const {
    const int lane = threadIdx.x & 63;
    return {(4 * s < a.k ? 4 * s : 0) * a.n + (r < end ? r : 0),
            uint32_t((lane >> 4) * a.n) + 2 * (lane & 15)};
  }
  __device__ __forceinline__ int live(const MuonMat &a, int64_t r, int64_t end, int s) const {
    const int lane = threadIdx.x & 63;
    return 4 * s + (lane >> 4) < a.k ? clamped(end - r - 2 * (lane & 15), 2) : 0;
  }
  __device__ __forceinline__ void request(const MuonMat &a, const MuonParams &p, int64_t r,
                                          int64_t end, int j) {
    const bool has_m = a.m != nullptr, read_g = !has_m || p.nesterov;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Place at = place(a, r, end, 4 * j + i);
      const int n = live(a, r, end, 4 * j + i);
      gr[j & 1][i] = read_g ? load_run<Q, 2>(a.grad, at, n) : Run<2>{};
      m[j & 1][i] = has_m ? load_run<Q, 2>(a.m, at, n) : Run<2>{};
    }
  }
};

template <int NT, bool Q>
__device__ __forceinline__ void apply_wide(const MuonMat &a, const MuonParams &p,
                                           const Factor<NT> &f, int64_t r, int64_t end,
                                           WideRows<NT, Q> &x) {
  const bool has_m = a.m != nullptr;
  f64x4_t d[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) d[t][0] = d[t][1] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  Run<2> th[4 * NT];
  double y[2][NT];                             // a product's Q, and the next one's
#pragma unroll
  for (int t = 0; t < NT; ++t) y[0][t] = f.template at<true>(0, t);
#pragma unroll
  for (int s = 0; s < 4 * NT; ++s) {
    const int j = s / 4, i = s % 4;
    if (i == 0 && j + 1 < NT) x.request(a, p, r, end, j + 1);
    if (s == 4 * NT - 4)                       // theta, behind the last of u
#pragma unroll
      for (int q = 0; q < 4 * NT; ++q)
        th[q] = a.theta ? load_run<Q, 2>(a.theta, x.place(a, r, end, q), x.live(a, r, end, q))
                        : Run<2>{};
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (s + 1 < 4 * NT) y[(s + 1) & 1][t] = f.template at<true>(s + 1, t);
    if (!Factor<NT>::held) __builtin_amdgcn_sched_barrier(0);
    double u[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      u[e] = double(direction<false>(p, has_m, x.gr[j & 1][i].v[e], x.m[j & 1][i].v[e]));
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) d[t][e] = mfma64(y[s & 1][t], u[e], d[t][e]);
  }
  x.request(a, p, r + 128, end, 0);
#pragma unroll
  for (int i = 0; i < 4 * NT; ++i) {
    const Run<2> v = {{float(d[i / 4][0][i % 4]), float(d[i / 4][1][i % 4])}};
    update_run<Q, 2>(a, p, x.place(a, r, end, i), x.live(a, r, end, i), v, th[i]);
  }
}

template <int NT, bool ALIGNED>
__global__ __launch_bounds__(256, ALIGNED ? 2 : 1) void apply_kernel(const MuonMat *table,
                                                                     MuonParams p,
                                                                     const double *ws) {
  using F = Factor<NT>;
  __shared__ __align__(16) double shared[F::held ? 1 : F::K * F::pitch];
  const MuonMat a = table[blockIdx.y];
  const int kp = padded(a.k);
  const int64_t from = int64_t(blockIdx.x) * a.apply;
  if (from >= a.n || kp > F::K || (NT > 1 && kp <= F::K / 2) || bool(a.quads) != ALIGNED) return;
  const int64_t end = from + a.apply < a.n ? from + a.apply : a.n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  F f;
  if (a.wide) {
    WideRows<NT, ALIGNED> x;
    x.request(a, p, from + 32 * wave, end, 0);
    f.template init<true>(ws + a.area, kp, shared);
    for (int64_t r = from + 32 * wave; r < end; r += 128, f.again())
      apply_wide<NT, ALIGNED>(a, p, f, r, end, x);
  } else {
    TallRows<NT, ALIGNED> x;
    x.request(a, p, from + 16 * wave, end);
    f.template init<false>(ws + a.area, kp, shared);
    for (int64_t r = from + 16 * wave; r < end; r += 64, f.again())
      apply_tall<NT, ALIGNED>(a, p, f, r, end, x);
  }
}

// k > 64: 32 long rows of u in LDS (fp32) for a workgroup, each of whose NB
// wavefronts forms a block of 64 columns of O; Q comes from L2, each value once
// a workgroup, requested a product ahead.  4 of rank 200: 77 us; with 64 rows,
// which halve the reads of Q but leave half the workgroups to a CU, 19 more.
constexpr int kLargeRows = 32, kLargeTiles = kLargeRows / 16;

// LDS row pitch (floats): 17 past a multiple of 64, so that a fragment (16 rows
// of 4) and a column written by consecutive lanes spread over the banks.
__host__ __device__ constexpr int large_pitch(int kp) { return (kp + 46) / 64 * 64 + 17; }

// The products and the update of T tiles of columns (q: the first one's Q).
template <bool WIDE, int T>
__device__ __forceinline__ void large_block(const MuonMat &a, const MuonParams &p, const float *us,
                                            int pitch, const double *q, int kp, int64_t from,
                                            int first) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  f64x4_t d[kLargeTiles][T];
#pragma unroll
  for (int i = 0; i < kLargeTiles; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) d[i][t] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  // two products of operands in hand, two on their way (kp / 4 is a multiple of
  // four; past the end the last ones again)
  double y[4][T];
  float x[4][kLargeTiles];
  const float *xs = us + c * pitch + g;
  const double *ys = q + int64_t(g) * kp + c;
  const int last = kp / 4 - 2;
  auto request = [&](int at, int s) {
    const int e = s < last ? s : last;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int t = 0; t < T; ++t) y[at + h][t] = ys[int64_t(4 * (e + h)) * kp + 16 * t];
#pragma unroll
      for (int i = 0; i < kLargeTiles; ++i) x[at + h][i] = xs[16 * i * pitch + 4 * (e + h)];
    }
  };
  auto multiply = [&](int at) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < kLargeTiles; ++i) {
          const double u = double(x[at + h][i]);
          d[i][t] = WIDE ? mfma64(y[at + h][t], u, d[i][t]) : mfma64(u, y[at + h][t], d[i][t]);
        }
  };
  request(0, 0);
  for (int s = 0; s < kp / 4; s += 4) {
    request(2, s + 2);
    __builtin_amdgcn_sched_barrier(0);
    multiply(0);
    request(0, s + 4);
    __builtin_amdgcn_sched_barrier(0);
    multiply(2);
  }
  // long row row0 + (wide: c, tall: g), column col0 + (wide: g, tall: c)
  auto row0 = [&](int i, int r) { return from + 16 * i + (WIDE ? 0 : 4 * r); };
  auto col0 = [&](int t, int r) { return first + 16 * t + (WIDE ? 4 * r : 0); };
  auto live_of = [&](int t, int i, int r) {
    return row0(i, r) + (WIDE ? c : g) < a.n && col0(t, r) + (WIDE ? g : c) < a.k;
  };
  auto place = [&](int t, int i, int r) {
    const int64_t row = row0(i, r) < a.n ? row0(i, r) : 0;
    const int col = col0(t, r) < a.k ? col0(t, r) : 0;
    return WIDE ? Place{col * a.n + row, uint32_t(g * a.n) + c}
                : Place{row * a.k + col, uint32_t(g * a.k + c)};
  };
  // (all of theta before the first store, behind which no load moves)
  Run<1> th[T][kLargeTiles][4];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < kLargeTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        th[t][i][r] = a.theta ? load_run<true, 1>(a.theta, place(t, i, r), live_of(t, i, r))
                              : Run<1>{};
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < kLargeTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        update_run<true, 1>(a, p, place(t, i, r), live_of(t, i, r), Run<1>{{float(d[i][t][r])}},
                            th[t][i][r]);
}

// u of a workgroup's long rows into LDS, four values of a lane at a time along memory.
template <bool WIDE, bool Q, int threads>
__device__ __forceinline__ void stage_rows(const MuonMat &a, int64_t from, int kp, int pitch,
                                           float *us) {
  const int per = WIDE ? kLargeRows / 4 : (a.k + 3) / 4;         // runs of a memory row
  const int items = WIDE ? a.k * per : kLargeRows * per;
  const uint32_t inv = 0xffffffffu / uint32_t(per) + 1u;         // e / per for e < 2^16
  for (int e0 = threadIdx.x; e0 < items; e0 += 4 * threads) {
    Run<4> u[4];
    int slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i * threads, hi = int(__umulhi(uint32_t(e), inv)), lo = 4 * (e - hi * per);
      const int64_t row = from + (WIDE ? lo : hi);
      const int live = e < items && row < a.n ? clamped(WIDE ? a.n - row : a.k - lo, 4) : 0;
      // (255 n + 63 and 64 k fit 32 bits)
      const Place at = WIDE ? Place{from, uint32_t(hi) * uint32_t(a.n) + lo}
                            : Place{from * a.k, uint32_t(hi * a.k + lo)};
      u[i] = load_run<Q, 4>(a.u, at, live);
      slot[i] = e >= items ? -1 : WIDE ? lo * pitch + hi : hi * pitch + lo;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (slot[i] < 0) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        us[slot[i] + e * (WIDE ? pitch : 1)] = u[i].v[e];
    }
  }
  // the columns past k (a tall row's last run has filled some)
  const int filled = WIDE ? a.k : 4 * per, pad = kp - filled;
  for (int e = threadIdx.x; e < kLargeRows * pad; e += threads)
    us[e / pad * pitch + filled + e % pad] = 0.0f;
}

template <int NB>
__global__ __launch_bounds__(64 * NB, 4) void apply_large_kernel(const MuonMat *table, MuonParams p,
                                                              double *ws) {
  extern __shared__ __align__(16) float us[];
  const MuonMat a = table[blockIdx.y];
  const int64_t from = int64_t(blockIdx.x) * kLargeRows;
  if (from >= a.n || (a.k + 63) / 64 != NB) return;
  const int kp = padded(a.k), pitch = large_pitch(kp);
  const int first = 64 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const double *q = Slots(ws + a.area, a.splits, kp).Q(p.steps) + first;
  with_bool(a.wide, [&](auto W) {
    constexpr bool wide = decltype(W)::value;
    with_bool(a.quads, [&](auto A) {
      stage_rows<wide, decltype(A)::value, 64 * NB>(a, from, kp, pitch, us);
    });
    __syncthreads();
    with_tiles((kp - first) / 16, [&](auto T) {
      large_block<wide, decltype(T)::value>(a, p, us, pitch, q, kp, from, first);
    });
  });
}

template <class F>
bool raise_lds(F *f, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void *>(f),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess;
}

// A matrix of a call: span0 as muon_span gives it for the call, o the doubles
// of the workspace that the matrices before it take.
MuonMat planned(const qlora_muon_mat &q, int64_t span0, bool nesterov, double *ws, int64_t &o) {
  MuonMat a{};
  a.grad = q.grad;
  a.m = q.m;
  a.theta = q.theta;
  a.theta16 = q.theta_bf16;
  a.update = q.update;
  a.scale = q.scale;
  a.wide = q.rows < q.cols;
  a.n = a.wide ? q.cols : q.rows;
  a.k = int32_t(a.wide ? q.rows : q.cols);
  auto ok = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  a.quads = (a.wide ? a.n : int64_t(a.k)) % 4 == 0 && ok(a.grad, 16) && ok(a.m, 16) &&
            ok(a.theta, 16) && ok(a.theta16, 8) && ok(a.update, 16);
  const int kp = padded(a.k);
  // A slab's k x k partial sums stay a small part of what it reads.  512
  // workgroups a call; of k <= 16, whose partial sums are smallest, 768, as many as
  // the chip holds (56 of rank 16, 8888 and 2000 long: 25.3 -> 20.9 us; 64 of 4096 x
  // 64 so: 43.3 -> 44.4; 1024 for rank 16: 26.9); of k > 64 a slab is a workgroup to
  // every pair of blocks.
  const int64_t most = a.k <= 16 ? span0 * 2 / 3 : a.k <= 64 ? span0 : span0 * pairs_of(a.k);
  const int64_t span = most < kp / 2 ? kp / 2 : most;
  a.span = (span + kGramRows - 1) / kGramRows * kGramRows;
  a.splits = int32_t((a.n + a.span - 1) / a.span);
  // One round of workgroups, each of which reads Q once (256 or 512 rows of 64
  // adapters of 4096 x 64: 77.4 and 70.5 us).  Q of k <= 16 is 2 KB and five times as
  // many workgroups fit (1024, 256 and 128 rows of 28 of rank 8, 4096 and 11008
  // long: 20.3, 14.5 and 11.0 us; of k <= 32, 1024 and 512: 32.7 and 33.1).
  const int64_t rows = kp <= 16 ? 128 : 1024;
  a.apply = span0 < rows ? (span0 + 127) / 128 * 128 : rows;
  a.area = o;
  const int64_t first = int64_t(pairs_of(a.k)) * kPairDoubles, sq = int64_t(kp) * kp;
  o += a.splits * first;
  if (a.k > 64) {
    o += 6 * sq;
    a.u = !a.m ? a.grad : nesterov ? reinterpret_cast<const float *>(ws + o) : a.m;
    o += (a.n * a.k + 3) / 4 * 2;
  }
  return a;
}

// Long rows to a slab of a call with 512, before a matrix's own bounds.
int64_t muon_span(const qlora_muon_mat *mats, int32_t n) {
  int64_t all = 0;
  for (int32_t i = 0; i < n; ++i)
    all += mats[i].rows < mats[i].cols ? mats[i].cols : mats[i].rows;
  return (all + 511) / 512;
}

size_t table_bytes(int32_t n) { return (size_t(n) * sizeof(MuonMat) + 255) / 256 * 256; }

}  // namespace

size_t muon_workspace_bytes(const qlora_muon_mat *mats, int32_t n) {
  const int64_t span = muon_span(mats, n);
  int64_t o = 0;
  for (int32_t i = 0; i < n; ++i) (void)planned(mats[i], span, false, nullptr, o);
  return table_bytes(n) + size_t(o) * sizeof(double);
}

hipError_t launch_muon(const qlora_muon_mat *mats, int32_t n, const MuonParams &p, void *work,
                       hipStream_t s) {
  MuonMat *table = static_cast<MuonMat *>(work);
  double *ws = reinterpret_cast<double *>(static_cast<char *>(work) + table_bytes(n));
  const int64_t span = muon_span(mats, n);
  // largest grids, by whether matrices have 16-byte accesses
  int64_t o = 0, blocks[2][5] = {}, blocks_large[5] = {}, splits[2] = {}, splits_large[2] = {};
  int64_t values = 0, values_small = 0;
  int most_k = 0;
  bool small[5] = {};
  auto raise = [](int64_t &to, int64_t v) { to = v > to ? v : to; };
  MuonChunk c;
  for (int32_t i = 0; i < n; i += kMuonChunk) {
    c.count = n - i < kMuonChunk ? n - i : kMuonChunk;
    c.first = i;
    for (int j = 0; j < c.count; ++j) {
      const MuonMat a = c.mats[j] = planned(mats[i + j], span, p.nesterov, ws, o);
      most_k = a.k > most_k ? a.k : most_k;
      const int kp = padded(a.k);
      if (a.k <= 64) {
        small[kp / 16] = true;
        values_small += a.n * a.k;
        raise(splits[a.quads], a.splits);
        const int NT = kp <= 16 ? 1 : kp <= 32 ? 2 : 4;
        raise(blocks[a.quads][NT], (a.n + a.apply - 1) / a.apply);
      } else {
        raise(splits_large[a.quads], a.splits);
        raise(blocks_large[(a.k + 63) / 64], (a.n + kLargeRows - 1) / kLargeRows);
        if (a.m) raise(values, a.n * a.k);
      }
    }
    if (n > kMuonFew) hipLaunchKernelGGL(table_kernel, dim3(1), dim3(64), 0, s, c, table);
  }
  // Matrices of both kinds of access cost a launch more of each kernel: the few of
  // a short call all go without 16-byte accesses, those of k <= 64 where they are
  // small (8 and 8 of rank 3, 82 and 1248 long: 27.4 -> 19.1 us; one adapter of 4097
  // and 11008 x 50, 0.75 M values: 112 -> 97, but of three, 2.3 M: 123 -> 134; 4 and
  // 4 of rank 150: 226 -> 219).
  if (n <= kMuonFew) {
    auto without = [&](bool small_ones) {
      for (int i = 0; i < n; ++i)
        if ((c.mats[i].k <= 64) == small_ones) c.mats[i].quads = 0;
    };
    auto join = [&](int64_t *x, int64_t *y) {
      raise(*x, *y);
      *y = 0;
    };
    if (splits[0] && splits[1] && values_small <= 3 << 19) {
      without(true);
      join(&splits[0], &splits[1]);
      for (int t = 0; t < 5; ++t) join(&blocks[0][t], &blocks[1][t]);
    }
    if (splits_large[0] && splits_large[1]) {
      without(false);
      join(&splits_large[0], &splits_large[1]);
    }
  }
  auto first = [&](auto mats) {
    using Mats = decltype(mats);
    if (values) {
      const int64_t b = (values + 1023) / 1024;
      hipLaunchKernelGGL((momentum_kernel<Mats>), dim3(unsigned(b < 1024 ? b : 1024), unsigned(n)),
                         dim3(256), 0, s, mats, p);
    }
#define QLORA_GRAM(ONE, Q, X, Y)                                                               \
  if (X)                                                                                       \
    hipLaunchKernelGGL((gram_kernel<ONE, Q, Mats>), dim3(unsigned(X), unsigned(Y), unsigned(n)), \
                       dim3(kGramThreads), 0, s, mats, p, ws)
    QLORA_GRAM(true, true, splits[1], 1);
    QLORA_GRAM(true, false, splits[0], 1);
    QLORA_GRAM(false, true, splits_large[1], pairs_of(most_k));
    QLORA_GRAM(false, false, splits_large[0], pairs_of(most_k));
#undef QLORA_GRAM
  };
  if (n <= kMuonFew) {
    MuonFew few{};
    std::copy(c.mats, c.mats + n, few.mats);
    few.table = table;
    first(few);
  } else {
    first(MuonTable{table});
  }
  const dim3 pairs(16, unsigned(pairs_of(most_k)), unsigned(n));
  if (most_k > 16) hipLaunchKernelGGL(gram_sum_kernel, pairs, dim3(256), 0, s, table, ws);
#define QLORA_SMALL(NT)                                                                 \
  if (small[NT]) {                                                                      \
    static const bool ok = raise_lds(&small_kernel<NT>, Small<NT>::bytes);              \
    if (!ok) return hipErrorInvalidValue;                                               \
    hipLaunchKernelGGL((small_kernel<NT>), dim3(unsigned(n)), dim3(Small<NT>::threads), \
                       Small<NT>::bytes, s, table, p, ws);                              \
  }
  if (small[1])
    hipLaunchKernelGGL(tiny_kernel, dim3(unsigned(n)), dim3(256), 0, s, table, p, ws);
  QLORA_SMALL(2)
  QLORA_SMALL(3)
  QLORA_SMALL(4)
#undef QLORA_SMALL
  if (most_k > 64) {
    const int NT = (most_k + 15) / 16;
    const int tiles = NT * (NT + 1) / 2;
    auto go = [&](int stage, int it) {
      const int jobs = stage == kAdvance ? 2 * tiles : tiles;
      hipLaunchKernelGGL(stage_kernel, dim3(unsigned(stage_grid(n, jobs))), dim3(256), 0, s, table,
                         p, ws, stage, it, n, jobs);
    };
    for (int it = 0; it < p.steps; ++it) {
      const bool last = it > 0 && it + 1 == p.steps;
      go(kSquare, it);
      go(last ? kLast : kPolynomial, it);
      if (p.steps > 1 && !last) go(kAdvance, it);
    }
  }
#define QLORA_APPLY(NT, Q)                                                                     \
  if (blocks[Q][NT])                                                                           \
    hipLaunchKernelGGL((apply_kernel<NT, Q>), dim3(unsigned(blocks[Q][NT]), unsigned(n)),      \
                       dim3(256), 0, s, table, p, ws)
  QLORA_APPLY(1, true);
  QLORA_APPLY(1, false);
  QLORA_APPLY(2, true);
  QLORA_APPLY(2, false);
  QLORA_APPLY(4, true);
  QLORA_APPLY(4, false);
#undef QLORA_APPLY
#define QLORA_APPLY(NB)                                                                    \
  if (blocks_large[NB]) {                                                                  \
    constexpr int lds = kLargeRows * large_pitch(64 * NB) * 4;                             \
    static const bool ok = raise_lds(&apply_large_kernel<NB>, lds);                        \
    if (!ok) return hipErrorInvalidValue;                                                  \
    hipLaunchKernelGGL((apply_large_kernel<NB>), dim3(unsigned(blocks_large[NB]), unsigned(n)), \
                       dim3(64 * NB), lds, s, table, p, ws);                               \
  }
  QLORA_APPLY(2)
  QLORA_APPLY(3)
  QLORA_APPLY(4)
#undef QLORA_APPLY
  return hipGetLastError();
}

}  // namespace qlora
