// The bias gradient of the grouped products, for gfx950.
//
//   group_colsum_kernel  db[e, n] = sum of dz[r, n] over the rows of group e:
//                        reads dz once.  A block owns 128 columns of one group
//                        (16 lanes of 16 bytes, 64 row slots); slots are added
//                        in slot order through LDS, so the sum's order depends
//                        on nothing but the group's rows.  Long groups at few
//                        columns are latency bound: 64 rows in flight per
//                        block, 4 deep.
#include <algorithm>

#include "common.h"
#include "gemm_train.h"

namespace fmlp {

namespace {

constexpr int kSlots = 64, kLanes = 16;   // row slots and 8-column lanes of a colsum block

__global__ void __launch_bounds__(kSlots* kLanes) group_colsum_kernel(const uint16_t* __restrict__ dz,
                                                                      const int32_t* __restrict__ group_off, int32_t R,
                                                                      int64_t N, uint16_t* __restrict__ db) {
  __shared__ int32_t tops[kSlots * kLanes / 64];
  __shared__ float part[kSlots][kLanes * 8 + 4];
  const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int64_t n = (int64_t)blockIdx.x * (kLanes * 8) + lane * 8;
  const int e = blockIdx.y;
  // the group's clamped ends: the maximum of the offsets up to its first, and
  // of that and its last
  static_assert(kSlots * kLanes == kMaxGroups, "an offset per thread");
  int32_t top = (int)threadIdx.x <= e ? min(max(group_off[threadIdx.x], 0), R) : 0;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max(top, __shfl_xor(top, d, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  for (int w = 0; w < kSlots * kLanes / 64; ++w) top = max(top, tops[w]);
  const int64_t r0 = top, r1 = min(max(group_off[e + 1], top), R);
  float acc[8] = {};
  if (n < N) {   // N % 8 == 0: a lane's columns are all in or all out
    int64_t r = r0 + slot;
    for (; r + 3 * kSlots < r1; r += 4 * kSlots) {
      u32x4_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = ld16(dz + (r + i * kSlots) * N + n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[8];
        unpack_bf16x8(v[i], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] += f[c];
      }
    }
    for (; r < r1; r += kSlots) {
      float f[8];
      unpack_bf16x8(ld16(dz + r * N + n), f);
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += f[c];
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) part[slot][lane * 8 + c] = acc[c];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < kLanes * 8 && (int64_t)blockIdx.x * (kLanes * 8) + c < N) {
    float s = 0.f;
    for (int i = 0; i < kSlots; ++i) s += part[i][c];
    const __bf16 b = (__bf16)s;
    db[(int64_t)e * N + (int64_t)blockIdx.x * (kLanes * 8) + c] = __builtin_bit_cast(uint16_t, b);
  }
}

}  // namespace

hipError_t launch_group_colsum(const uint16_t* dz, const int32_t* group_off, int64_t R, int E, int64_t N, uint16_t* db,
                               hipStream_t s) {
  if (E < 1 || E > kMaxGroups || R < 0 || R > 0x7fffffff || N < 8 || N % 8 != 0) return hipErrorInvalidValue;
  const int64_t bx = (N + kLanes * 8 - 1) / (kLanes * 8);
  hipLaunchKernelGGL(group_colsum_kernel, dim3((unsigned)bx, (unsigned)E), dim3(kSlots * kLanes), 0, s, dz, group_off,
                     (int32_t)R, N, db);
  return hipGetLastError();
}

}  // namespace fmlp
