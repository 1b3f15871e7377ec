// Helpers of the grouped products, for gfx950: the plan a call's GEMM kernels
// read about its groups, and the bias gradient.
//
//   group_plan_kernel    one block scans the caller's E + 1 offsets: a running
//                        maximum (clamped into the rows there are), then the
//                        prefix sums of row tiles and of 64-row stages.  E is
//                        at most 1024, so one thread per group and two levels
//                        of wave scans do; it is bound by one launch (2 us).
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

constexpr int kPlanThreads = 1024;
constexpr int kSlots = 64, kLanes = 16;   // row slots and 8-column lanes of a colsum block

template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, Op op) {   // inclusive, lanes 0 .. 63
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_up(v, d, 64);
    if (lane >= d) v = op(o, v);
  }
  return v;
}
// Inclusive over the block's threads; tmp holds one T per wave.
template <class T, class Op>
__device__ __forceinline__ T block_scan(T v, Op op, T* tmp) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  v = wave_scan(v, op);
  if (lane == 63) tmp[wave] = v;
  __syncthreads();
  for (int w = wave - 1; w >= 0; --w) v = op(tmp[w], v);   // op is max or +: any order, exact
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) group_plan_kernel(const int32_t* __restrict__ off, int32_t R, int E,
                                                                  int bm, int split, GroupPlan p) {
  __shared__ int32_t t32[kPlanThreads / 64];
  __shared__ int64_t t64[kPlanThreads / 64];
  const int g = threadIdx.x;   // one thread per group (the block has at least E threads)
  const int32_t first = min(max(off[0], 0), R);
  const int32_t mine = g < E ? min(max(off[g + 1], first), R) : first;
  const int32_t end = block_scan(mine, [](int32_t a, int32_t b) { return max(a, b); }, t32);
  // the group's first row is the previous thread's end
  int32_t begin = __shfl_up(end, 1, 64);
  if ((threadIdx.x & 63) == 63) t32[threadIdx.x >> 6] = end;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) begin = threadIdx.x == 0 ? first : t32[(threadIdx.x >> 6) - 1];
  __syncthreads();
  const int32_t rows = g < E ? end - begin : 0;
  const int32_t tiles = block_scan((rows + bm - 1) / bm, [](int32_t a, int32_t b) { return a + b; }, t32);
  const int64_t work = block_scan((int64_t)max((rows + 63) / 64, split), [](int64_t a, int64_t b) { return a + b; }, t64);
  if (g == 0) {
    p.group_off[0] = first;
    p.tile_off[0] = 0;
    p.work_off[0] = 0;
  }
  if (g < E) {
    p.group_off[g + 1] = end;
    p.tile_off[g + 1] = tiles;
    p.work_off[g + 1] = work;
  }
}

__global__ void __launch_bounds__(kSlots* kLanes) group_colsum_kernel(const uint16_t* __restrict__ dz,
                                                                      const int32_t* __restrict__ group_off, int64_t N,
                                                                      uint16_t* __restrict__ db) {
  __shared__ float part[kSlots][kLanes * 8 + 4];
  const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int64_t n = (int64_t)blockIdx.x * (kLanes * 8) + lane * 8;
  const int e = blockIdx.y;
  const int64_t r1 = group_off[e + 1];
  float acc[8] = {};
  if (n < N) {   // N % 8 == 0: a lane's columns are all in or all out
    int64_t r = group_off[e] + slot;
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

hipError_t launch_group_plan(const int32_t* off, int64_t R, int E, int bm, int split, const GroupPlan& plan,
                             hipStream_t s) {
  if (E < 1 || E > kPlanThreads || R < 0 || R > 0x7fffffff || bm < 1 || split < 1) return hipErrorInvalidValue;
  const int threads = (E + 63) / 64 * 64;
  hipLaunchKernelGGL(group_plan_kernel, dim3(1), dim3((unsigned)threads), 0, s, off, (int32_t)R, E, bm, split, plan);
  return hipGetLastError();
}

hipError_t launch_group_colsum(const uint16_t* dz, const int32_t* group_off, int E, int64_t N, uint16_t* db,
                               hipStream_t s) {
  if (E < 1 || E > 65535 || N < 8 || N % 8 != 0) return hipErrorInvalidValue;
  const int64_t bx = (N + kLanes * 8 - 1) / (kLanes * 8);
  hipLaunchKernelGGL(group_colsum_kernel, dim3((unsigned)bx, (unsigned)E), dim3(kSlots * kLanes), 0, s, dz, group_off, N,
                     db);
  return hipGetLastError();
}

}  // namespace fmlp
