// Dropout whose mask is a function of the element's place: nothing is stored
// and the backward draws the same mask again.
//
// y = residual + keep x c, c = 65536 / (65536 - p16).  The mask comes from
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3"): a 128-bit counter (n, counter) and a 64-bit key (seed) go
// through ten rounds of two 32 x 32 -> 64 bit products,
//   (a, b, c, d) <- (hi(M1 c) ^ b ^ k0, lo(M1 c), hi(M0 a) ^ d ^ k1, lo(M0 a)),
//   (k0, k1) <- (k0 + W0, k1 + W1),
// and give 128 bits, 16 for each of the 8 elements of group n of the row-wise
// grouping (a row always starts a new group).  16 bits an element halve the
// generator's work against 32; p is rounded to a multiple of 2^-16 and c uses
// the rounded p, so the mean is kept.
#include "device.h"

namespace qlora {
namespace {

__device__ __forceinline__ u32x4_t philox(uint64_t n, uint64_t counter, uint64_t seed) {
  uint32_t a = uint32_t(n), b = uint32_t(n >> 32);
  uint32_t c = uint32_t(counter), d = uint32_t(counter >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t u = uint64_t(a) * 0xD2511F53u, v = uint64_t(c) * 0xCD9E8D57u;
    a = uint32_t(v >> 32) ^ b ^ k0;
    b = uint32_t(v);
    c = uint32_t(u >> 32) ^ d ^ k1;
    d = uint32_t(u);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{a, b, c, d};
}

template <bool BF16>
__device__ __forceinline__ float load1(const void *x, int64_t at) {
  if (BF16)
    return __uint_as_float(uint32_t(static_cast<const uint16_t *>(x)[at]) << 16);
  return static_cast<const float *>(x)[at];
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *x, int64_t at, float (&e)[8]) {
  if (BF16) {
    u32x4_t u;
    __builtin_memcpy(&u, static_cast<const uint16_t *>(x) + at, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = bf16_lo_to_f32(u[i]);
      e[2 * i + 1] = bf16_hi_to_f32(u[i]);
    }
  } else {
    __builtin_memcpy(e, static_cast<const float *>(x) + at, 32);
  }
}

template <bool BF16>
__device__ __forceinline__ void dropout8(const DropoutArgs &a, int64_t groups, int64_t n) {
  const int64_t row = n / groups, j = (n - row * groups) * 8;
  const u32x4_t w = philox(uint64_t(n), a.counter, a.seed);
  const int64_t ix = row * a.ldx + j, ir = row * a.ldr + j, iy = row * a.ldy + j;
  const int left = int(a.cols - j < 8 ? a.cols - j : 8);
  float e[8] = {}, r[8] = {};
  if (left == 8) {
    load8<BF16>(a.x, ix, e);
    if (a.res) load8<BF16>(a.res, ir, r);
  } else {
    for (int i = 0; i < left; ++i) {
      e[i] = load1<BF16>(a.x, ix + i);
      if (a.res) r[i] = load1<BF16>(a.res, ir + i);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bits = (w[i / 2] >> (16 * (i % 2))) & 0xffffu;
    e[i] = (bits >= a.p16 ? a.c * e[i] : 0.0f) + r[i];
  }
  if (BF16) {
    uint16_t *y = static_cast<uint16_t *>(a.y) + iy;
    const u32x4_t u = {pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                       pack_bf16x2(e[6], e[7])};
    if (left == 8)
      __builtin_memcpy(y, &u, 16);
    else
      for (int i = 0; i < left; ++i) y[i] = uint16_t(u[i / 2] >> (16 * (i % 2)));
  } else {
    float *y = static_cast<float *>(a.y) + iy;
    if (left == 8)
      __builtin_memcpy(y, e, 32);
    else
      for (int i = 0; i < left; ++i) y[i] = e[i];
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, int64_t groups) {
  const int64_t all = a.rows * groups, step = int64_t(gridDim.x) * 256;
  for (int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x; n < all; n += step)
    dropout8<BF16>(a, groups, n);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, bool bf16, hipStream_t s) {
  const int64_t groups = (a.cols + 7) / 8;
  // a launch holds less than 2^32 threads: larger arrays go round
  const dim3 grid{unsigned(min64((a.rows * groups + 255) / 256, int64_t(1) << 22))};
  if (bf16)
    hipLaunchKernelGGL((dropout_kernel<true>), grid, dim3(256), 0, s, a, groups);
  else
    hipLaunchKernelGGL((dropout_kernel<false>), grid, dim3(256), 0, s, a, groups);
  return hipGetLastError();
}

}  // namespace qlora
