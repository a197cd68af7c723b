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
//
// HBM-bound: 16384 x 4096 bf16 45.1 us (6.0 TB/s), with a residual 69 us (5.9
// TB/s); 8192 x 4096 fp32 49.7 us (5.4 TB/s).  Rows off the 16-byte boundary
// (odd widths) move 3.8 TB/s: a lane's 8 elements are those of its draws, not
// those of an aligned line.
#include "objective.h"

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

// 8 elements from `p` on, of which n are there (n < 8 at a row's end only).
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t at, int n, float (&e)[8]) {
  if (BF16) {
    const uint16_t *x = static_cast<const uint16_t *>(p) + at;
    if (n >= 8) {
      u32x4_t u;
      __builtin_memcpy(&u, x, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[2 * i] = bf16_lo_to_f32(u[i]);
        e[2 * i + 1] = bf16_hi_to_f32(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < n ? __uint_as_float(uint32_t(x[i]) << 16) : 0.0f;
    }
  } else {
    const float *x = static_cast<const float *>(p) + at;
    if (n >= 8) {
      __builtin_memcpy(e, x, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < n ? x[i] : 0.0f;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t at, int n, const float (&e)[8]) {
  if (BF16) {
    uint16_t *y = static_cast<uint16_t *>(p) + at;
    const u32x4_t u = {pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                       pack_bf16x2(e[6], e[7])};
    if (n >= 8) {
      __builtin_memcpy(y, &u, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) y[i] = uint16_t(u[i / 2] >> (16 * (i % 2)));
    }
  } else {
    float *y = static_cast<float *>(p) + at;
    if (n >= 8) {
      __builtin_memcpy(y, e, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) y[i] = e[i];
    }
  }
}

// Group n of `count` to a lane, the first of them the matrix's group `base`.
// FLAT: dense rows of a multiple of 8, group n is elements 8 n .. 8 n + 7 (the
// division by the groups of a row is about a quarter of the lane's work).
template <bool BF16, bool RES, bool FLAT>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, uint32_t groups,
                                                      uint32_t count, uint64_t base) {
  const uint32_t n = blockIdx.x * 256 + threadIdx.x;
  if (n >= count) return;
  const uint32_t row = FLAT ? 0 : n / groups;
  const int64_t j = FLAT ? int64_t(n) * 8 : int64_t(n - row * groups) * 8;
  const int left = FLAT ? 8 : int(least64(a.cols - j, 8));
  float e[8], r[8];
  load8<BF16>(a.x, row * a.ldx + j, left, e);
  if (RES) load8<BF16>(a.res, row * a.ldr + j, left, r);
  const u32x4_t w = philox(base + n, a.counter, a.seed);
  // a half h is kept where h >= p16, compared in a word's upper half
  const uint32_t least = a.p16 << 16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool keep = i % 2 ? w[i / 2] >= least : w[i / 2] << 16 >= least;
    e[i] = keep ? a.c * e[i] : 0.0f;
    if (RES) e[i] += r[i];
  }
  store8<BF16>(a.y, row * a.ldy + j, left, e);
}

template <bool BF16, bool RES>
void dropout(DropoutArgs a, hipStream_t s) {
  const int64_t groups = (a.cols + 7) / 8;
  const bool flat = a.cols % 8 == 0 && a.ldx == a.cols && a.ldy == a.cols &&
                    (!RES || a.ldr == a.cols);
  // a launch counts its groups in 32 bits, and holds less than 2^32 threads
  const int64_t rows_each = ((int64_t(1) << 31) / groups);
  const int64_t size = BF16 ? 2 : 4;
  for (int64_t row = 0; row < a.rows; row += rows_each) {
    const int64_t count = least64(a.rows - row, rows_each) * groups;
    DropoutArgs b = a;
    b.x = static_cast<const char *>(a.x) + row * a.ldx * size;
    b.y = static_cast<char *>(a.y) + row * a.ldy * size;
    if (RES) b.res = static_cast<const char *>(a.res) + row * a.ldr * size;
    const dim3 grid{unsigned((count + 255) / 256)};
    if (flat)
      hipLaunchKernelGGL((dropout_kernel<BF16, RES, true>), grid, dim3(256), 0, s, b,
                         uint32_t(groups), uint32_t(count), uint64_t(row * groups));
    else
      hipLaunchKernelGGL((dropout_kernel<BF16, RES, false>), grid, dim3(256), 0, s, b,
                         uint32_t(groups), uint32_t(count), uint64_t(row * groups));
  }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, bool bf16, hipStream_t s) {
  if (bf16)
    a.res ? dropout<true, true>(a, s) : dropout<true, false>(a, s);
  else
    a.res ? dropout<false, true>(a, s) : dropout<false, false>(a, s);
  return hipGetLastError();
}

}  // namespace qlora
