// The gradient of a linear's epilogue y = residual + act(z) mul:
//   dZ = dY mul act'(Z),  dmul = dY act(Z),  dbias = column sums of dZ
// (the residual's gradient is dY itself).  One pass, HBM-bound: Z, dY and mul
// read once, dZ and dmul written once.  A workgroup takes a slab of rows of one
// run of columns, 16 bytes a lane, four rows in flight; its column sums (fp32
// over 16 rows of a lane, fp64 from there on) leave as partials that a
// second launch adds in a fixed order, or as dbias where there is one slab.
// dZ enters the sums before it is rounded.
// 2048 x 11008 bf16, SiLU with a factor: 36 us, 6.3 TB/s of 226 MB (a copy
// reaches 5.1), 43 with the launch's own; 509 x 4096 fp32, GELU with a bias: 7.0
// and 2.4, 25 MB, latency.
#include "epilogue.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;
constexpr int kTurns = 4;            // of them, summed in fp32

template <bool BF16, int kCols>     // kCols: lanes along a row
__global__ __launch_bounds__(kThreads) void ep_bwd_kernel(EpBwdArgs a) {
  constexpr int W = kWide<BF16>, kRows = kThreads / kCols;
  __shared__ double red[kRows][kCols * W + 1];
  const int cl = threadIdx.x % kCols, rl = threadIdx.x / kCols;
  const int64_t col = (int64_t(blockIdx.x) * kCols + cl) * W;
  const int64_t from = int64_t(blockIdx.y) * a.slab;
  const int64_t end = from + a.slab < a.M ? from + a.slab : a.M;
  const bool in = col < a.out;
  float sum[W];
  double total[W];
#pragma unroll
  for (int i = 0; i < W; ++i) total[i] = sum[i] = 0.0f;
  auto collect = [&] {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      total[i] += double(sum[i]);
      sum[i] = 0.0f;
    }
  };
  constexpr int es = BF16 ? 2 : 4;
  auto at = [&](const void *p, int64_t r) {
    return reinterpret_cast<const u32x4_t *>(static_cast<const char *>(p) + (r * a.out + col) * es);
  };
  auto to = [&](void *p, int64_t r) {
    return reinterpret_cast<u32x4_t *>(static_cast<char *>(p) + (r * a.out + col) * es);
  };
  with_act(a.act, [&](auto A) {
    constexpr int act = decltype(A)::value;
    int turn = 0;
    for (int64_t r0 = from + rl; r0 < end && in; r0 += kRows * kRowsAhead) {
      u32x4_t z[kRowsAhead], dy[kRowsAhead], mu[kRowsAhead];
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i) {
        // (past the end: the last row again, not used)
        const int64_t r = r0 + i * kRows < end ? r0 + i * kRows : end - 1;
        dy[i] = *at(a.dY, r);
        if (a.Z) z[i] = *at(a.Z, r);
        if (a.mul) mu[i] = *at(a.mul, r);
      }
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i) {
        const int64_t r = r0 + i * kRows;
        if (r >= end) break;
        float d[W], x[W], g[W], h[W];
        widen<BF16>(dy[i], d);
        if (a.Z) widen<BF16>(z[i], x);
        if (a.mul) widen<BF16>(mu[i], g);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          float f = 0.0f, df = 1.0f;
          if (a.Z) activated<act, BF16>(x[e], f, df);
          h[e] = d[e] * f;
          d[e] = d[e] * df;
          if (a.mul) d[e] *= g[e];
          sum[e] += d[e];
        }
        if (a.dZ) *to(a.dZ, r) = narrow<BF16>(d);
        if (a.dmul) *to(a.dmul, r) = narrow<BF16>(h);
      }
      if (++turn % kTurns == 0) collect();
    }
  });
  if (!a.dbias) return;
  collect();
#pragma unroll
  for (int e = 0; e < W; ++e) red[rl][cl * W + e] = total[e];
  __syncthreads();
  for (int c = threadIdx.x; c < kCols * W; c += kThreads) {
    const int64_t n = int64_t(blockIdx.x) * kCols * W + c;
    if (n >= a.out) break;
    double s = 0.0;
    for (int r = 0; r < kRows; ++r) s += red[r][c];
    if (a.partial)
      a.partial[int64_t(blockIdx.y) * a.out + n] = s;
    else
      a.dbias[n] = float(s);
  }
}

// 64 columns to a workgroup, four lanes to a column.
__global__ __launch_bounds__(kThreads) void bias_sum_kernel(const double *partial, int64_t slabs,
                                                            int64_t out, float *dbias) {
  __shared__ double red[4][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t n = int64_t(blockIdx.x) * 64 + c;      // out is a multiple of 64
  double s = 0.0;
  for (int64_t b = q; b < slabs; b += 32) {
    double v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = b + 4 * i < slabs ? partial[(b + 4 * i) * out + n] : 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  red[q][c] = s;
  __syncthreads();
  if (q == 0) dbias[n] = float(((red[0][c] + red[1][c]) + red[2][c]) + red[3][c]);
}

}  // namespace

// 64 rows of up to 128 (one or two slabs), else 32, or more where there would be
// more than 256 slabs (509 x 4096 fp32 with 64: 13.0 us, with 32: 9.8).
int64_t ep_bwd_slab(int64_t M) {
  if (M <= 128) return 64;
  const int64_t most = ((M + 255) / 256 + 31) / 32 * 32;
  return most < 32 ? 32 : most;
}

int64_t ep_bwd_slabs(int64_t M) { return (M + ep_bwd_slab(M) - 1) / ep_bwd_slab(M); }

hipError_t launch_ep_bwd(EpBwdArgs a, bool bf16, hipStream_t s) {
  a.slab = ep_bwd_slab(a.M);
  const int64_t slabs = ep_bwd_slabs(a.M);
  if (slabs == 1) a.partial = nullptr;
  // 32 lanes along a row where it has as many, so that a row's run is 512 bytes
  const bool wide = a.out >= 32 * (bf16 ? 8 : 4);
  const int64_t cols = (wide ? 32 : 8) * (bf16 ? 8 : 4);
  const dim3 grid(unsigned((a.out + cols - 1) / cols), unsigned(slabs));
#define QLORA_EP(B, C) hipLaunchKernelGGL((ep_bwd_kernel<B, C>), grid, dim3(kThreads), 0, s, a)
  if (bf16) {
    if (wide) QLORA_EP(true, 32);
    else QLORA_EP(true, 8);
  } else {
    if (wide) QLORA_EP(false, 32);
    else QLORA_EP(false, 8);
  }
#undef QLORA_EP
  if (a.dbias && slabs > 1)
    hipLaunchKernelGGL(bias_sum_kernel, dim3(unsigned(a.out / 64)), dim3(kThreads), 0, s,
                       a.partial, slabs, a.out, a.dbias);
  return hipGetLastError();
}

}  // namespace qlora
