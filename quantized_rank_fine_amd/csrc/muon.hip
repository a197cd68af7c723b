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
// sum; the k x k iterations, in one workgroup's LDS for k <= 64, else by
// 16 x 16 tiles, one launch a product; the last product and the update.
#include "device.h"
#include "qlora.h"

namespace qlora {
namespace {

// A matrix in the kernels: n long, k short; quads: 16-byte loads of grad and m.
// span: long rows to a Gram workgroup, `splits` of them; apply: long rows to
// an update workgroup; area: where its fp64 scratch begins.
struct MuonMat {
  const float *grad;
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

// LDS row pitch (floats) of a slab [long][short] of kp short columns: 17 past a
// multiple of 64 (49 for 32 columns), so that both a fragment (4 rows of 16, or
// 16 rows of 4) and a column written by consecutive lanes spread over the banks.
__host__ __device__ constexpr int slab_pitch(int kp) {
  return kp == 32 ? 49 : (kp + 46) / 64 * 64 + 17;
}

// Long rows staged at a time: about 4096 values.
__host__ __device__ constexpr int slab_rows(int kp) {
  return kp <= 16 ? 256 : kp <= 32 ? 128 : kp <= 64 ? 64 : kp <= 128 ? 32 : 16;
}

constexpr int kPad = 16;
__host__ __device__ inline int padded(int k) { return (k + kPad - 1) / kPad * kPad; }

// One value's momentum and the update's direction.
template <bool kStore>
__device__ __forceinline__ float direction(const MuonParams &p, bool has_m, float g, float &m) {
  if (!has_m) return g;
  if (kStore) m = p.mu * m + g;
  return p.nesterov ? g + p.mu * m : m;
}

// `rows` long rows from `at` of a matrix into us [rows][pitch] as u; kStore: the
// momentum is advanced (else it is read as it is).  Rows past n become 0; the
// columns past k are not touched.  A thread's loads go out before the first
// value is used.
template <bool kStore, int threads, int kMost>
__device__ __forceinline__ void stage(const MuonMat &a, const MuonParams &p, int64_t at, int rows,
                                      int pitch, float *us) {
  const int t = threadIdx.x, k = a.k;
  const int64_t left = a.n - at;
  const int live = int(left < rows ? left : rows);
  const bool has_m = a.m != nullptr;
  const bool read_g = kStore || !has_m || p.nesterov;
  const uint32_t inv = k > 1 ? 0xffffffffu / uint32_t(k) + 1u : 0u;   // e / k for e < 2^16
  if (a.quads) {
    constexpr int U = (kMost / 4 + threads - 1) / threads;
    const int per = a.wide ? rows / 4 : k / 4;         // quads of a memory row
    const uint32_t pinv = per > 1 ? 0xffffffffu / uint32_t(per) + 1u : 0u;
    const int quads = a.wide ? k * per : rows * per;
    f32x4_t g[U], m[U];
    int64_t off[U];
    int row[U], col[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int e = t + i * threads;
      const int hi = per > 1 ? int(__umulhi(uint32_t(e), pinv)) : e, lo = e - hi * per;
      row[i] = a.wide ? 4 * lo : hi;
      col[i] = a.wide ? hi : 4 * lo;
      off[i] = e < quads && row[i] < live
                   ? (a.wide ? int64_t(col[i]) * a.n + at + row[i] : (at + row[i]) * k + col[i])
                   : -1;
      g[i] = m[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (off[i] >= 0) {
        if (read_g) g[i] = *reinterpret_cast<const f32x4_t *>(a.grad + off[i]);
        if (has_m) m[i] = *reinterpret_cast<const f32x4_t *>(a.m + off[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (t + i * threads >= quads) break;
      float u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float mm = m[i][e];
        u[e] = direction<kStore>(p, has_m, g[i][e], mm);
        m[i][e] = mm;
      }
      if (kStore && has_m && off[i] >= 0) *reinterpret_cast<f32x4_t *>(a.m + off[i]) = m[i];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        us[(row[i] + (a.wide ? e : 0)) * pitch + col[i] + (a.wide ? 0 : e)] = u[e];
    }
    return;
  }
  // any alignment: one value a lane at a time
  const int all = rows * k;
  const uint32_t rinv = 0xffffffffu / uint32_t(rows) + 1u;
  for (int base = 0; base < all; base += 8 * threads) {
    float g[8], m[8];
    int64_t off[8];
    int slot[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = base + i * threads + t;
      int r, c;
      if (a.wide) {
        c = int(__umulhi(uint32_t(e), rinv));
        r = e - c * rows;
      } else {
        r = k > 1 ? int(__umulhi(uint32_t(e), inv)) : e;
        c = e - r * k;
      }
      slot[i] = e < all ? r * pitch + c : -1;
      off[i] = e < all && r < live ? (a.wide ? int64_t(c) * a.n + at + r : (at + r) * k + c) : -1;
      g[i] = m[i] = 0.0f;
      if (off[i] >= 0) {
        if (read_g) g[i] = a.grad[off[i]];
        if (has_m) m[i] = a.m[off[i]];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (slot[i] < 0) continue;
      const float u = direction<kStore>(p, has_m, g[i], m[i]);
      if (kStore && has_m && off[i] >= 0) a.m[off[i]] = m[i];
      us[slot[i]] = u;
    }
  }
}

// Slabs of kp short columns hold at most this many values (quads of them, for
// k a multiple of 4, at most rows kp / 4).
constexpr int kSlabMost = 4096;

template <int threads>
__device__ __forceinline__ void clear(float *us, int n) {
  for (int i = threadIdx.x; i < n; i += threads) us[i] = 0.0f;
}

// ------------------------------------------------------------ Gram partials
//
// One slab range of a matrix to a workgroup: u goes to LDS in fp32 (advancing
// the momentum on the way) and is multiplied from there.  NB 64-column blocks:
// NB = 1: four wavefronts share the rows and hold all tiles of the upper
// triangle; else a wavefront to each pair of blocks (of the upper triangle),
// all rows each.  Partial sums: [tile][register][lane], fp64.
template <int NB>
struct Pairs {
  static constexpr int count = NB * (NB + 1) / 2;
  static constexpr int threads = NB == 1 ? 256 : count * 64;
};

__device__ __forceinline__ int tile_index(int ti, int tj) { return tj * (tj + 1) / 2 + ti; }

// Matrices to a launch whose arguments describe them.
constexpr int kMuonChunk = 32;
struct MuonChunk {
  int count;
  int first;               // index of mats[0] in the table
  MuonMat mats[kMuonChunk];
};

template <int NB>
__global__ __launch_bounds__(Pairs<NB>::threads) void gram_kernel(MuonChunk c, MuonParams p,
                                                                  MuonMat *table, double *ws) {
  constexpr int threads = Pairs<NB>::threads;
  const MuonMat &a = c.mats[blockIdx.y];
  // the later launches find the matrix in the table
  if (blockIdx.x == 0 && threadIdx.x == 0) table[c.first + blockIdx.y] = a;
  if (int(blockIdx.x) >= a.splits || (a.k + 63) / 64 != NB) return;
  extern __shared__ __align__(16) float us[];
  const int kp = padded(a.k), NT = kp / 16, pitch = slab_pitch(kp), rows = slab_rows(kp);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane >> 4, fc = lane & 15;
  int bi = 0, bj = 0;                       // this wavefront's pair of blocks
  if (NB > 1)
    for (int q = wave; q > bj; q -= ++bj) bi = q - bj - 1;
  f64x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  clear<threads>(us, rows * pitch);
  const int64_t from = int64_t(blockIdx.x) * a.span;
  const int64_t end = from + a.span < a.n ? from + a.span : a.n;
  for (int64_t at = from; at < end; at += rows) {
    __syncthreads();
    stage<true, threads, kSlabMost>(a, p, at, rows, pitch, us);
    __syncthreads();
    const int step = NB == 1 ? 16 : 4;
    for (int r = NB == 1 ? 4 * wave : 0; r < rows; r += step) {
      const float *row = us + (r + fr) * pitch + fc;
      double x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = 64 * bi + 16 * i < kp ? double(row[64 * bi + 16 * i]) : 0.0;
        if (NB > 1) y[i] = 64 * bj + 16 * i < kp ? double(row[64 * bj + 16 * i]) : 0.0;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * bj + j >= NT) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * bi + i <= 4 * bj + j) acc[i][j] = mfma64(x[i], NB > 1 ? y[j] : x[j], acc[i][j]);
      }
    }
  }
  const int tiles = NT * (NT + 1) / 2;
  double *out = ws + a.area + int64_t(blockIdx.x) * tiles * 256;
  if (NB == 1) {
    // the four wavefronts' sums in their order
    double *sum = reinterpret_cast<double *>(us);
    for (int w = 0; w < 4; ++w) {
      __syncthreads();
      if (wave == w) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i <= j; ++i)
            if (j < NT) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                double *s = sum + (tile_index(i, j) * 4 + r) * 64 + lane;
                *s = w == 0 ? acc[i][j][r] : *s + acc[i][j][r];
              }
            }
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < tiles * 256; e += threads) out[e] = sum[e];
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * bj + j < NT && 4 * bi + i <= 4 * bj + j) {
        double *o = out + tile_index(4 * bi + i, 4 * bj + j) * 256 + lane;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[64 * r] = acc[i][j][r];
      }
}

// Sum of a matrix's partials into the first, an element to a lane.
__global__ __launch_bounds__(256) void gram_sum_kernel(const MuonMat *table, double *ws) {
  const MuonMat a = table[blockIdx.y];
  if (a.k <= 16) return;                   // one tile: small_kernel sums it
  const int NT = padded(a.k) / 16, n = NT * (NT + 1) / 2 * 256;
  const int e = int(blockIdx.x) * 256 + threadIdx.x;
  if (e >= n) return;
  double *x = ws + a.area + e;
  double s = 0.0;
  for (int b = 0; b < a.splits; b += 8) {
    double v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = b + i < a.splits ? x[int64_t(b + i) * n] : 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  *x = s;
}

// ---------------------------------------------- k x k iterations, k <= 64
//
// One workgroup, three fp64 matrices in LDS: G, S (then P), Q; row pitch 16
// past a multiple of 32 doubles, so that the rows of a fragment fall on
// different halves of the banks.  A product's tiles of the upper triangle are
// dealt over the wavefronts, kept in registers until every read is done, and
// stored with their mirror images.
template <int NT>
struct Small {
  static constexpr int kp = 16 * NT, pitch = (kp + 15) / 32 * 32 + 16, tiles = NT * (NT + 1) / 2;
  static constexpr int threads = NT == 1 ? 64 : NT == 2 ? 256 : 512, waves = threads / 64;
  static constexpr int size = kp * pitch;
  static constexpr int bytes = 3 * size * 8;
};

template <int NT>
__device__ __forceinline__ f64x4_t lds_product(const double *A, const double *B, int ti, int tj) {
  constexpr int pitch = Small<NT>::pitch;
  const int lane = threadIdx.x & 63;
  const double *x = A + (lane >> 4) * pitch + (lane & 15) + 16 * ti;   // A symmetric: A[k][i]
  const double *y = B + (lane >> 4) * pitch + (lane & 15) + 16 * tj;
  f64x4_t d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int q = 0; q < 4 * NT; ++q) d = mfma64(x[4 * q * pitch], y[4 * q * pitch], d);
  return d;
}

// Tile (ti, tj) of a symmetric matrix, element by element: f(row, column, register).
template <class F>
__device__ __forceinline__ void each(int ti, int tj, F &&f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r) f(16 * ti + (lane >> 4) + 4 * r, 16 * tj + (lane & 15), r);
}

__device__ __forceinline__ void tile_of_index(int t, int &ti, int &tj) {
  tj = 0;
  while (t > tj) t -= ++tj;
  ti = t;
}

__device__ __forceinline__ double inverse_norm(double trace, double eps) {
  const double d = sqrt(trace) + eps;
  return d > 0.0 ? 1.0 / d : 0.0;          // a zero update stays zero
}

template <int NT>
__global__ __launch_bounds__(Small<NT>::threads) void small_kernel(const MuonMat *table,
                                                                   MuonParams p, double *ws) {
  using S = Small<NT>;
  const MuonMat a = table[blockIdx.x];
  if ((a.k + 15) / 16 != NT) return;
  extern __shared__ __align__(16) double sq[];
  double *G = sq, *P = sq + S::size, *Q = sq + 2 * S::size;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double *area = ws + a.area;
  for (int e = threadIdx.x; e < S::tiles * 256; e += S::threads) {
    double v = 0.0;
    if (NT == 1) {                         // one tile: its partials are summed here
      for (int b = 0; b < a.splits; b += 8) {
        double w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = b + i < a.splits ? area[(b + i) * 256 + e] : 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += w[i];
      }
    } else {
      v = area[e];
    }
    int ti, tj;
    tile_of_index(e / 256, ti, tj);
    const int i = 16 * ti + ((e & 63) >> 4) + 4 * ((e >> 6) & 3), j = 16 * tj + (e & 15);
    G[i * S::pitch + j] = v;
    if (ti < tj) G[j * S::pitch + i] = v;
  }
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < S::kp; ++i) trace += G[i * S::pitch + i];
  const double inv = inverse_norm(trace, p.eps);
  __syncthreads();
  for (int e = threadIdx.x; e < S::kp * S::kp; e += S::threads) {
    const int i = e / S::kp, j = e % S::kp;
    G[i * S::pitch + j] *= inv * inv;
    Q[i * S::pitch + j] = i == j ? inv : 0.0;
  }
  __syncthreads();
  constexpr int per = (S::tiles + S::waves - 1) / S::waves;
  constexpr int both = (2 * S::tiles + S::waves - 1) / S::waves;
  auto put = [&](double *M, int i, int j, double v, bool mirror) {
    M[i * S::pitch + j] = v;
    if (mirror) M[j * S::pitch + i] = v;
  };
  for (int it = 0; it < p.steps; ++it) {
    f64x4_t d[both];
    // S = G G
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int t = wave + q * S::waves;
      if (t >= S::tiles) break;
      int ti, tj;
      tile_of_index(t, ti, tj);
      d[q] = lds_product<NT>(G, G, ti, tj);
      each(ti, tj, [&](int i, int j, int r) { put(P, i, j, d[q][r], ti < tj); });
    }
    __syncthreads();
    // H = G P = a G + b S + c G S in G's place, P = a I + b G + c S in S's
    double g[per][4], s[per][4];
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int t = wave + q * S::waves;
      if (t >= S::tiles) break;
      int ti, tj;
      tile_of_index(t, ti, tj);
      d[q] = lds_product<NT>(G, P, ti, tj);
      each(ti, tj, [&](int i, int j, int r) {
        g[q][r] = G[i * S::pitch + j];
        s[q][r] = P[i * S::pitch + j];
      });
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < per; ++q) {
      const int t = wave + q * S::waves;
      if (t >= S::tiles) break;
      int ti, tj;
      tile_of_index(t, ti, tj);
      each(ti, tj, [&](int i, int j, int r) {
        put(G, i, j, p.a * g[q][r] + p.b * s[q][r] + p.c * d[q][r], ti < tj);
        put(P, i, j, (i == j ? p.a : 0.0) + p.b * g[q][r] + p.c * s[q][r], ti < tj);
      });
    }
    __syncthreads();
    // G <- H P and Q <- Q P; the last time Q alone
    const bool last = it + 1 == p.steps;
#pragma unroll
    for (int q = 0; q < both; ++q) {
      const int t = wave + q * S::waves;
      if (t >= (last ? 1 : 2) * S::tiles) break;
      int ti, tj;
      tile_of_index(t % S::tiles, ti, tj);
      d[q] = lds_product<NT>(t < S::tiles ? Q : G, P, ti, tj);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < both; ++q) {
      const int t = wave + q * S::waves;
      if (t >= (last ? 1 : 2) * S::tiles) break;
      int ti, tj;
      tile_of_index(t % S::tiles, ti, tj);
      each(ti, tj, [&](int i, int j, int r) { put(t < S::tiles ? Q : G, i, j, d[q][r], ti < tj); });
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < S::kp * S::kp; e += S::threads)
    area[e] = Q[e / S::kp * S::pitch + e % S::kp];
}

// ------------------------------------------------ k x k iterations, k > 64
//
// The matrices (kp x kp, row-major) follow each other in the matrix's area: G,
// S, H, P, Q, Q'.  A workgroup owns one 16 x 16 tile of the upper triangle of a
// product, its four wavefronts a quarter of the sum each; operands come from
// L2 (both symmetric, so every fragment is four runs of 128 bytes).
enum MuonStage { kUnpack, kSquare, kPolynomial, kAdvance };

struct Slots {
  double *G, *S, *H, *P, *Q[2];
  __device__ __forceinline__ Slots(double *area, int kp) {
    const int64_t n = int64_t(kp) * kp;
    G = area + n;                 // past the summed partials
    S = G + n;
    H = S + n;
    P = H + n;
    Q[0] = P + n;
    Q[1] = Q[0] + n;
  }
};

// A quarter of the sum of tile (ti, tj) of A B.
__device__ __forceinline__ f64x4_t part_product(const double *A, const double *B, int kp, int ti,
                                                int tj, int wave) {
  const int lane = threadIdx.x & 63;
  const int steps = kp / 16;               // of four rows, a quarter of kp / 4
  const int64_t at = int64_t(4 * wave * steps + (lane >> 4)) * kp + (lane & 15);
  const double *x = A + at + 16 * ti, *y = B + at + 16 * tj;
  f64x4_t d = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int q = 0; q < steps; ++q) d = mfma64(x[4 * q * kp], y[4 * q * kp], d);
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

__global__ __launch_bounds__(256) void stage_kernel(const MuonMat *table, MuonParams p, double *ws,
                                                    int stage, int it) {
  __shared__ double red[2][4][4][64];
  __shared__ double norm;
  const MuonMat a = table[blockIdx.y];
  if (a.k <= 64) return;
  const int kp = padded(a.k), NT = kp / 16, t = int(blockIdx.x);
  if (t >= NT * (NT + 1) / 2) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int ti, tj;
  tile_of_index(t, ti, tj);
  const Slots m(ws + a.area, kp);
  const int i = 16 * ti + (lane >> 4) + 4 * wave, j = 16 * tj + (lane & 15);
  const int64_t ij = int64_t(i) * kp + j, ji = int64_t(j) * kp + i;
  auto put = [&](double *M, double v) {
    M[ij] = v;
    if (ti < tj) M[ji] = v;
  };
  if (stage == kUnpack) {
    put(m.G, ws[a.area + t * 256 + 64 * wave + lane]);
    return;
  }
  if (stage == kSquare) {
    put(m.S, joined_part(part_product(m.G, m.G, kp, ti, tj, wave), wave, red[0]));
    return;
  }
  const double *q = m.Q[it & 1];
  if (stage == kPolynomial) {
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
    const bool last = it + 1 == p.steps;
    const double g = f * m.G[ij], s = f * f * m.S[ij];
    const double v = (i == j ? p.a : 0.0) + p.b * g + p.c * s;
    put(m.P, v);
    if (it == 0) put(m.Q[1], inv * v);
    if (!last)
      put(m.H, p.a * g + p.b * s +
                   p.c * (f * f * f *
                          joined_part(part_product(m.G, m.S, kp, ti, tj, wave), wave, red[0])));
    return;
  }
  // kAdvance: G <- H P (but the last time) and, past the first, Q' = Q P
  if (it + 1 < p.steps)
    put(m.G, joined_part(part_product(m.H, m.P, kp, ti, tj, wave), wave, red[0]));
  if (it > 0)
    put(m.Q[(it + 1) & 1], joined_part(part_product(q, m.P, kp, ti, tj, wave), wave, red[1]));
}

// ------------------------------------------------------------ the update
//
// O = u Q for `rows` long rows at a time: u staged in LDS as above, a wavefront
// to 16 rows, four tiles of columns at a time.  Of a tall matrix the long side
// is the rows of a tile, of a wide one its columns (the operands swapped: Q is
// symmetric), so that 16 lanes always run along memory.  kLds: Q is in LDS too.
constexpr int kApplyRows = 64;

template <bool kLds>
__global__ __launch_bounds__(256) void apply_kernel(const MuonMat *table, MuonParams p,
                                                    const double *ws) {
  const MuonMat a = table[blockIdx.y];
  const int kp = padded(a.k), NT = kp / 16, pitch = slab_pitch(kp);
  const int64_t from = int64_t(blockIdx.x) * a.apply;
  if (from >= a.n || (a.k <= 64) != kLds) return;
  extern __shared__ __align__(16) float us[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const double *Q = ws + a.area;
  if (!kLds) Q = Slots(const_cast<double *>(Q), kp).Q[p.steps & 1];
  clear<256>(us, kApplyRows * pitch);
  double *ql = reinterpret_cast<double *>(us + (kApplyRows * pitch + 3) / 4 * 4);
  if (kLds)
    for (int e = threadIdx.x; e < kp * kp; e += 256) ql[e] = Q[e];
  const double *qs = kLds ? ql : Q;
  const int64_t end = from + a.apply < a.n ? from + a.apply : a.n;
  for (int64_t at = from; at < end; at += kApplyRows) {
    __syncthreads();
    // (kSlabMost values at most are staged in one go)
    for (int r = 0; r < kApplyRows; r += slab_rows(kp) < kApplyRows ? slab_rows(kp) : kApplyRows)
      if (at + r < end)
        stage<false, 256, kSlabMost>(a, p, at + r,
                                     slab_rows(kp) < kApplyRows ? slab_rows(kp) : kApplyRows,
                                     pitch, us + r * pitch);
    __syncthreads();
    const float *x = us + (16 * wave + (lane & 15)) * pitch + (lane >> 4);
    for (int t0 = 0; t0 < NT; t0 += 4) {
      f64x4_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = f64x4_t{0.0, 0.0, 0.0, 0.0};
      for (int q = 0; q < kp / 4; ++q) {
        const double u = double(x[4 * q]);
        const double *y = qs + (4 * q + (lane >> 4)) * kp + 16 * t0 + (lane & 15);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t0 + j < NT) d[j] = a.wide ? mfma64(y[16 * j], u, d[j]) : mfma64(u, y[16 * j], d[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int over = (lane >> 4) + 4 * r, along = lane & 15;
          const int64_t i = at + 16 * wave + (a.wide ? along : over);
          const int c = 16 * (t0 + j) + (a.wide ? over : along);
          if (i >= a.n || c >= a.k) continue;
          const int64_t e = a.wide ? int64_t(c) * a.n + i : i * a.k + c;
          const float o = float(d[j][r]);
          if (a.update) a.update[e] = o;
          if (a.theta) {
            const float th = a.theta[e], v = th - p.lr * (a.scale * o + p.wd * th);
            a.theta[e] = v;
            if (a.theta16) a.theta16[e] = __builtin_bit_cast(uint16_t, (__bf16)v);
          }
        }
    }
  }
}

template <class F>
bool raise_lds(F *f, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void *>(f),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess;
}

// LDS of a Gram workgroup of NB blocks: the largest slab (NB = 1: of 32
// columns; its tiles' sums, 10 x 2 KiB, take less).
template <int NB>
constexpr int gram_lds() {
  return NB == 1 ? 128 * slab_pitch(32) * 4 : slab_rows(64 * NB) * slab_pitch(64 * NB) * 4;
}
static_assert(gram_lds<1>() >= 10 * 2048 && gram_lds<1>() >= 256 * slab_pitch(16) * 4 &&
                  gram_lds<1>() >= 64 * slab_pitch(64) * 4,
              "Gram LDS");

constexpr int kApplyLds = kApplyRows * slab_pitch(64) * 4 + 64 * 64 * 8;
constexpr int kApplyLdsLarge = kApplyRows * slab_pitch(256) * 4;

// A matrix of a call: span0 as muon_span gives it for the call, o the doubles
// of the workspace that the matrices before it take.
MuonMat planned(const qlora_muon_mat &q, int64_t span0, int64_t &o) {
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
  auto ok16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  a.quads = ok16(a.grad) && ok16(a.m) && (a.wide ? a.n : int64_t(a.k)) % 4 == 0;
  const int kp = padded(a.k), rows = slab_rows(kp);
  // a slab's k x k partial sums stay a small part of what it reads
  const int64_t span = span0 < kp / 2 ? kp / 2 : span0;
  a.span = (span + rows - 1) / rows * rows;
  a.splits = int32_t((a.n + a.span - 1) / a.span);
  a.apply = a.k <= 64 && a.span > kApplyRows ? a.span / kApplyRows * kApplyRows : kApplyRows;
  a.area = o;
  const int64_t sq = int64_t(kp) * kp, tiles = int64_t(kp / 16) * (kp / 16 + 1) / 2 * 256;
  const int64_t squares = (a.k <= 64 ? 1 : 7) * sq, partials = a.splits * tiles;
  o += squares > partials ? squares : partials;
  return a;
}

// Long rows to a slab, before a matrix's own bounds: 512 workgroups a call.
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
  for (int32_t i = 0; i < n; ++i) (void)planned(mats[i], span, o);
  return table_bytes(n) + size_t(o) * sizeof(double);
}

hipError_t launch_muon(const qlora_muon_mat *mats, int32_t n, const MuonParams &p, void *work,
                       hipStream_t s) {
  MuonMat *table = static_cast<MuonMat *>(work);
  double *ws = reinterpret_cast<double *>(static_cast<char *>(work) + table_bytes(n));
  const int64_t span = muon_span(mats, n);
  int64_t o = 0, blocks = 0, blocks_large = 0;
  int most_k = 0;
  bool small[5] = {};
  for (int32_t i = 0; i < n; i += kMuonChunk) {
    MuonChunk c;
    c.count = n - i < kMuonChunk ? n - i : kMuonChunk;
    c.first = i;
    bool any[5] = {};
    int32_t most = 0;
    for (int j = 0; j < c.count; ++j) {
      const MuonMat a = c.mats[j] = planned(mats[i + j], span, o);
      any[(a.k + 63) / 64] = true;
      most = a.splits > most ? a.splits : most;
      most_k = a.k > most_k ? a.k : most_k;
      int64_t &b = a.k <= 64 ? blocks : blocks_large;
      const int64_t need = (a.n + a.apply - 1) / a.apply;
      b = need > b ? need : b;
      if (a.k <= 64) small[(a.k + 15) / 16] = true;
    }
#define QLORA_GRAM(NB)                                                                         \
  if (any[NB])                                                                                 \
    hipLaunchKernelGGL((gram_kernel<NB>), dim3(unsigned(most), unsigned(c.count)),             \
                       dim3(Pairs<NB>::threads), gram_lds<NB>(), s, c, p, table, ws)
    QLORA_GRAM(1);
    QLORA_GRAM(2);
    QLORA_GRAM(3);
    QLORA_GRAM(4);
#undef QLORA_GRAM
  }
  const int NT = (most_k + 15) / 16;
  const dim3 tiles(unsigned(NT * (NT + 1) / 2), unsigned(n));
  if (most_k > 16) hipLaunchKernelGGL(gram_sum_kernel, tiles, dim3(256), 0, s, table, ws);
#define QLORA_SMALL(NT)                                                                 \
  if (small[NT]) {                                                                      \
    static const bool ok = raise_lds(&small_kernel<NT>, Small<NT>::bytes);              \
    if (!ok) return hipErrorInvalidValue;                                               \
    hipLaunchKernelGGL((small_kernel<NT>), dim3(unsigned(n)), dim3(Small<NT>::threads), \
                       Small<NT>::bytes, s, table, p, ws);                              \
  }
  QLORA_SMALL(1)
  QLORA_SMALL(2)
  QLORA_SMALL(3)
  QLORA_SMALL(4)
#undef QLORA_SMALL
  if (most_k > 64) {
    auto go = [&](int stage, int it) {
      hipLaunchKernelGGL(stage_kernel, tiles, dim3(256), 0, s, table, p, ws, stage, it);
    };
    go(kUnpack, 0);
    for (int it = 0; it < p.steps; ++it) {
      go(kSquare, it);
      go(kPolynomial, it);
      if (p.steps > 1) go(kAdvance, it);
    }
  }
  if (blocks)
    hipLaunchKernelGGL((apply_kernel<true>), dim3(unsigned(blocks), unsigned(n)), dim3(256),
                       kApplyLds, s, table, p, ws);
  if (blocks_large) {
    static const bool ok = raise_lds(&apply_kernel<false>, kApplyLdsLarge);
    if (!ok) return hipErrorInvalidValue;
    hipLaunchKernelGGL((apply_kernel<false>), dim3(unsigned(blocks_large), unsigned(n)),
                       dim3(256), kApplyLdsLarge, s, table, p, ws);
  }
  return hipGetLastError();
}

}  // namespace qlora
