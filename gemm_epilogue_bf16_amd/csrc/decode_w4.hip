// Decode path with 4-bit weights and group scales (M <= 16 tokens) for gfx950.
//
//   W[n, k] = s[n, k / G] * (q[n, k] - z[n, k / G]),   y = act(x W^T + b),
//
// q in 0 .. 15, two codes a byte (code 2j in the low half of byte j), s and z
// bf16, z = 8 where no zero points are given, G = 32, 64 or 128.  A decode layer
// is bound by reading its weights once: 1/2 + 2/G bytes each (+ 2/G with zero
// points).
//
// Arithmetic.  A byte 0x0q read as E4M3 is q * 2^-9 for every q (codes below 8
// are its subnormals, 8 .. 15 its first binade), so the hardware's scaled
// conversion with 2^9 turns two codes at a time into the bf16 integers q,
// exactly.  Within a group
//   sum_k x (q - z) = sum_k x q + sum_k x (-z),
// both on v_mfma_f32_16x16x32_bf16 into one fp32 accumulator (the second with a
// constant weight operand; without zero points it is the same for every weight
// row and computed once); the group's scale multiplies the finished sum, in
// fp32.  Nothing is rounded to fewer bits before the output's bf16.  A token
// that holds an infinity or a NaN gets NaN or infinite outputs; others do not
// see it (tokens are rows of the matrix product).
//
// Layout.  The activations are the MFMA's row operand and 16 weight rows its
// column operand, so a lane's four results are four tokens of ONE weight row
// and need one scale.  A 16-byte load gives a lane 32 consecutive codes of its
// row and the wave 128 codes ("a chunk") of 16 rows.  With G = 128 the four
// words of a lane feed four MFMAs as they are: the contraction is order-free
// within a group.  With G = 32 or 64 an MFMA's 32 k must be consecutive, and
// four half-wave swaps (permlane32 / permlane16) exchange words between the
// four lanes of a row.  8 waves share a block's rows and split k in runs of U
// chunks; partial sums meet in LDS in wave order (deterministic).  Weight
// batches are double-buffered in registers.
//
// Activations: up to 64 KB of them are staged in LDS once per block (16 weight
// rows a block); a larger set is read from L2 beside the weights, where a
// block takes twice the rows so that half of those reads serve.  Every token's
// row of the operand is independent, so rows past M need no masking.
#include <algorithm>

#include "common.h"
#include "decode_w4.h"
#include "lds_dma.h"

namespace fmlp {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kChunk = 128;   // k of one 16-byte load of the 4 lanes of a row

__device__ __forceinline__ __amdgpu_buffer_rsrc_t w4_desc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t d, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(d, (int)off, 0, 0));
}
// weights are read exactly once: non-temporal
__device__ __forceinline__ u32x4_t load16_stream(__amdgpu_buffer_rsrc_t d, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(d, (int)off, 0, 2));
}

// words w[i] of lane group g -> w[g] of lane group i (4 x 4 over the 16-lane groups)
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void exchange_words(uint32_t w[4]) {
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
}

// 8 codes of a word -> 8 bf16 integers, in k order
__device__ __forceinline__ u32x4_t expand(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;   // even codes, odd codes
  const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u);      // codes 0 1 2 3
  const uint32_t b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);      // codes 4 5 6 7
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true));
  return r;
}

// one bf16 in all 8 places of an operand, sign flipped
__device__ __forceinline__ u32x4_t minus_all(uint32_t bf) {
  const uint32_t v = (bf | (bf << 16)) ^ 0x80008000u;
  u32x4_t r;
  r[0] = r[1] = r[2] = r[3] = v;
  return r;
}

// n bf16 values of a row at byte offset off; NW words.  WHOLE: off is a
// multiple of the vector's size; else each value is loaded by itself, those
// at or past `have` as zeros.
template <int NV, bool WHOLE>
struct Values {
  static constexpr int kWords = WHOLE ? (NV + 1) / 2 : NV;
  uint32_t v[kWords];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t d, uint32_t off, int have) {
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        v[i] = __builtin_amdgcn_raw_buffer_load_b16(d, (int)(i < have ? off + 2u * i : kOutOfRange), 0, 0);
    } else if constexpr (NV == 2) {
      v[0] = __builtin_amdgcn_raw_buffer_load_b32(d, (int)off, 0, 0);
    } else if constexpr (NV == 4) {
      const auto r = __builtin_amdgcn_raw_buffer_load_b64(d, (int)off, 0, 0);
      v[0] = r[0];
      v[1] = r[1];
    } else {
      static_assert(NV % 8 == 0, "values of a batch");
#pragma unroll
      for (int i = 0; i < NV / 8; ++i) {
        const u32x4_t r = load16(d, off + 16u * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = r[j];
      }
    }
  }
  __device__ __forceinline__ uint32_t bits(int i) const {   // the bf16's 16 bits
    if constexpr (WHOLE) return (i & 1) ? v[i / 2] >> 16 : v[i / 2] & 0xFFFFu;
    else return v[i];
  }
  __device__ __forceinline__ float f32(int i) const {
    if constexpr (WHOLE) return (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
    else return __uint_as_float(v[i] << 16);
  }
  __device__ __forceinline__ void hold() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(v[i]));
  }
};

// NS weight streams (row tiles, gate and up), U chunks each
template <int NS, int U, int NV, bool WHOLE, bool ZEROS, bool XL>
struct Batch {
  u32x4_t w[NS][U];
  Values<NV, WHOLE> s[NS];
  Values<ZEROS ? NV : 2, WHOLE> z[ZEROS ? NS : 1];
  u32x4_t x[XL ? 1 : U][4];
};

// GS: log2 of the group size.  WHOLE: K is a multiple of U chunks, so no load
// needs a mask and scales come as aligned vectors.  XL: activations in LDS.
template <bool DUAL, int RT, int U, int GS, bool ZEROS, bool WHOLE, bool XL>
__global__ __launch_bounds__(kThreads) void decode_w4_kernel(W4Layer L, int M) {
  constexpr int SETS = DUAL ? 2 : 1;
  constexpr int NS = RT * SETS;            // stream s: row tile s / SETS, set s % SETS
  constexpr int GPC = kChunk >> GS;        // groups per chunk
  constexpr int IPG = 4 / GPC;             // MFMAs per group
  constexpr int NV = U * GPC;              // scales of a batch
  constexpr bool FINE = GPC > 1;
  using B = Batch<NS, U, NV, WHOLE, ZEROS, XL>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15;   // weight row of a tile; token of the activation operand
  const int g = lane >> 4;
  const int K = (int)L.K;
  const int groups = K >> GS;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
  const int rows = (int)min<int64_t>(16 * RT, L.N - n0);
  const int chunks = (K + kChunk - 1) / kChunk;
  const int nb = (chunks + kWaves * U - 1) / (kWaves * U);   // batches of the first wave

  __amdgpu_buffer_rsrc_t dw[SETS], ds[SETS], dz[SETS];
#pragma unroll
  for (int t = 0; t < SETS; ++t) {
    dw[t] = w4_desc((t ? L.q1 : L.q0) + n0 * (K / 2), (uint32_t)rows * (uint32_t)(K / 2));
    ds[t] = w4_desc((t ? L.s1 : L.s0) + n0 * groups, (uint32_t)rows * (uint32_t)groups * 2u);
    if constexpr (ZEROS) dz[t] = w4_desc((t ? L.z1 : L.z0) + n0 * groups, (uint32_t)rows * (uint32_t)groups * 2u);
  }
  const __amdgpu_buffer_rsrc_t dx = w4_desc(L.x, (uint32_t)(M * K) * 2u);
  // codes 32 g .. of a chunk; the MFMA's k of lane group g: 8 g .. (FINE) or 32 g ..
  const uint32_t wlane = (uint32_t)(r * (K / 2) + g * 16);
  const uint32_t slane = (uint32_t)(r * groups) * 2u;
  const int xk = FINE ? 8 * g : 32 * g;
  constexpr int kXStep = FINE ? 32 : 8;   // k between an operand's four MFMAs
  const int xstride = 2 * (chunks * kChunk) + 16;   // bytes of a staged row; + 16: rows in different banks
  const uint8_t* xl = lds + (r < M ? r : 0) * xstride + 2 * xk;
  const uint32_t xg = r < M ? (uint32_t)(r * K + xk) * 2u : kOutOfRange;

  auto issue = [&](B& b, int i) {
    const int c0 = (i * kWaves + wave) * U;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint32_t row = (uint32_t)((s / SETS) * 16);
      const int left = WHOLE ? U : chunks - c0;   // chunks from c0 on
#pragma unroll
      for (int j = 0; j < U; ++j)
        b.w[s][j] = load16_stream(dw[s % SETS],
                                  WHOLE || j < left ? wlane + row * (uint32_t)(K / 2) + (uint32_t)(c0 + j) * 64u : kOutOfRange);
      const uint32_t so = slane + row * (uint32_t)groups * 2u + (uint32_t)(c0 * GPC) * 2u;
      const int have = WHOLE ? NV : groups - c0 * GPC;
      b.s[s].load(ds[s % SETS], so, have);
      if constexpr (ZEROS) b.z[s].load(dz[s % SETS], so, have);
    }
    if constexpr (!XL) {
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k = (c0 + j) * kChunk + kXStep * q;
          b.x[j][q] = load16(dx, WHOLE || k + xk < K ? xg + (uint32_t)k * 2u : kOutOfRange);
        }
    }
  };
  auto hold = [&](B& b) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int j = 0; j < U; ++j) asm volatile("" : "+v"(b.w[s][j]));
      b.s[s].hold();
      if constexpr (ZEROS) b.z[s].hold();
    }
    if constexpr (!XL) {
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(b.x[j][q]));
    }
  };
  f32x4_t tot[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) tot[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const u32x4_t minus8 = minus_all(0x4100u);

  auto consume = [&](const B& b, int i) {
    const int c0 = (i * kWaves + wave) * U;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!WHOLE && c0 + j >= chunks) break;   // wave-uniform
      u32x4_t x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x[q] = XL ? *reinterpret_cast<const u32x4_t*>(xl + (c0 + j) * (2 * kChunk) + 2 * kXStep * q) : b.x[XL ? 0 : j][q];
      f32x4_t corr[GPC];
      if constexpr (!ZEROS) {
#pragma unroll
        for (int t = 0; t < GPC; ++t) {
          corr[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < IPG; ++q) corr[t] = mfma_16x16x32(x[t * IPG + q], minus8, corr[t]);
        }
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        uint32_t w[4] = {b.w[s][j][0], b.w[s][j][1], b.w[s][j][2], b.w[s][j][3]};
        if constexpr (FINE) exchange_words(w);
#pragma unroll
        for (int t = 0; t < GPC; ++t) {
          f32x4_t acc;
          if constexpr (ZEROS) {
            acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
            const u32x4_t z = minus_all(b.z[s].bits(j * GPC + t));
#pragma unroll
            for (int q = 0; q < IPG; ++q) acc = mfma_16x16x32(x[t * IPG + q], z, acc);
          } else {
            acc = corr[t];
          }
#pragma unroll
          for (int q = 0; q < IPG; ++q) acc = mfma_16x16x32(x[t * IPG + q], expand(w[t * IPG + q]), acc);
          const float sc = b.s[s].f32(j * GPC + t);
#pragma unroll
          for (int v = 0; v < 4; ++v) tot[s][v] = fmaf(sc, acc[v], tot[s][v]);
        }
      }
    }
  };

  // this wave's batches: those whose first chunk exists
  int mine = 0;
  if (wave * U < chunks) mine = (chunks - wave * U + kWaves * U - 1) / (kWaves * U);
  (void)nb;
  B A, C;
  if (mine > 0) issue(A, 0);
  if constexpr (XL) {
    // rows of x straight into LDS, 1 KB per instruction, all in flight before
    // one wait; zeros behind a row whose K ends inside a chunk
    const int per_row = K / 8;   // 16-byte pieces
    const int ipr = (per_row + 63) / 64;
    const i32x4_t xd = make_desc(reinterpret_cast<uint64_t>(L.x), (uint32_t)(M * K) * 2u);
    const uint32_t xs = lds_addr(lds);
    for (int t = wave; t < M * ipr; t += kWaves) {   // wave-uniform
      const int m = t / ipr, q = t - m * ipr;
      const int c = q * 64 + lane;
      if (c < per_row) asm_load_lds(xd, uniform32(xs + (uint32_t)(m * xstride + q * 1024)), (uint32_t)(m * K + c * 8) * 2u);
    }
    if constexpr (!WHOLE) {
      const int pad = (chunks * kChunk - K) / 8;
      for (int t = threadIdx.x; t < M * pad; t += kThreads) {
        const int m = t / pad;
        *reinterpret_cast<u32x4_t*>(lds + m * xstride + 2 * K + 16 * (t - m * pad)) = zero4();
      }
    }
    wait_vm<0>();
    __syncthreads();
  }
  int i = 0;
  for (; i + 2 < mine; i += 2) {
    issue(C, i + 1);
    hold(A);
    consume(A, i);
    issue(A, i + 2);
    hold(C);
    consume(C, i + 1);
  }
  if (i + 1 < mine) {
    issue(C, i + 1);
    hold(A);
    consume(A, i);
    hold(C);
    consume(C, i + 1);
  } else if (i < mine) {
    hold(A);
    consume(A, i);
  }

  // the waves' partial sums, added in wave order
  if constexpr (XL) __syncthreads();   // every wave has read its activations
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);   // [wave][stream][lane]
#pragma unroll
  for (int s = 0; s < NS; ++s) red[(wave * NS + s) * 64 + lane] = tot[s];
  __syncthreads();
  for (int o = threadIdx.x; o < RT * 256; o += kThreads) {
    const int ln = o & 63, v = (o >> 6) & 3, t = o >> 8;
    const int m = 4 * (ln >> 4) + v, row = 16 * t + (ln & 15);
    if (m >= M || row >= rows) continue;
    float z[SETS];
#pragma unroll
    for (int e = 0; e < SETS; ++e) {
      z[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) z[e] += reinterpret_cast<const float*>(red + (w * NS + t * SETS + e) * 64 + ln)[v];
    }
    float out;
    if constexpr (DUAL) {
      out = apply_act(z[0], L.act) * z[SETS - 1];
    } else {
      out = z[0];
      if (L.bias) out += bf16_to_f32(L.bias[n0 + row]);
      out = apply_act(out, L.act);
    }
    const __bf16 ob = (__bf16)out;
    L.y[(int64_t)m * L.N + n0 + row] = __builtin_bit_cast(uint16_t, ob);
  }
}

constexpr int kXMax = 64 * 1024;   // staged activations of a block

template <bool DUAL, int GS, bool ZEROS>
hipError_t launch_w4(const W4Layer& L, int M, hipStream_t s) {
  constexpr int SETS = DUAL ? 2 : 1;
  const int64_t chunks = (L.K + kChunk - 1) / kChunk;
  const int64_t xbytes = (int64_t)M * (2 * chunks * kChunk + 16);
  auto go = [&](auto kernel, int rt, int64_t xb) {
    const int64_t red = (int64_t)kWaves * rt * SETS * 64 * 16;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((L.N + 16 * rt - 1) / (16 * rt))), dim3(kThreads),
                       (unsigned)std::max(xb, red), s, L, M);
    return hipGetLastError();
  };
  constexpr int UL = DUAL && GS < 7 ? 2 : 4;
  if (xbytes <= kXMax) {
    if (L.K % (UL * kChunk) == 0) return go(decode_w4_kernel<DUAL, 1, UL, GS, ZEROS, true, true>, 1, xbytes);
    return go(decode_w4_kernel<DUAL, 1, UL, GS, ZEROS, false, true>, 1, xbytes);
  }
  if (L.K % (2 * kChunk) == 0) return go(decode_w4_kernel<DUAL, 2, 2, GS, ZEROS, true, false>, 2, 0);
  return go(decode_w4_kernel<DUAL, 2, 2, GS, ZEROS, false, false>, 2, 0);
}

template <bool DUAL, int GS>
hipError_t by_zeros(const W4Layer& L, int M, hipStream_t s) {
  return L.z0 ? launch_w4<DUAL, GS, true>(L, M, s) : launch_w4<DUAL, GS, false>(L, M, s);
}
template <bool DUAL>
hipError_t by_group(const W4Layer& L, int M, hipStream_t s) {
  switch (L.G) {
    case 32: return by_zeros<DUAL, 5>(L, M, s);
    case 64: return by_zeros<DUAL, 6>(L, M, s);
    case 128: return by_zeros<DUAL, 7>(L, M, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_decode_w4(const W4Layer& L, int M, hipStream_t s) {
  if (M < 1 || M > 16 || L.K < 32 || L.K % L.G != 0 || L.N < 1) return hipErrorInvalidValue;
  if (L.q1 != nullptr && (L.z0 == nullptr) != (L.z1 == nullptr)) return hipErrorInvalidValue;
  return L.q1 ? by_group<true>(L, M, s) : by_group<false>(L, M, s);
}

}  // namespace fmlp
