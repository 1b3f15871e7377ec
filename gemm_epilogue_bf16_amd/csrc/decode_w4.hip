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
// are its subnormals, 8 .. 15 its first binade), so a mask and a shift turn 8
// codes into 8 matrix operands, with nothing to convert.  The activations meet
// them as a sum of two E4M3 values: of a token's 128 k ("a chunk"), 2^e is the
// least power of two that brings the largest magnitude to 448 or less, and
//   x = 2^e hi + 2^(e-4) lo,  hi = e4m3(x 2^-e),  lo = e4m3(16 (x 2^-e - hi)).
// A bf16 has 8 significant bits and hi and lo take 4 each, so this is exact for
// every x within 14 binades of the chunk's largest, and off by at most 2^-21 of
// that largest below.  v_mfma_scale_f32_16x16x128_f8f6f4 multiplies a whole
// chunk, with 2^e and 2^9 as its block scales.  (bf16 operands need four
// 16x16x32 MFMAs and a conversion of every code: 97 ns and 134 ns a KB of codes
// and SIMD, against 17 or 33 ns and about 50 ns, and made the kernel compute
// bound.)  The instruction adds its 128 products and the accumulator in fp32,
// but was seen to align neighbouring products before that to 13 bits below the
// larger one: a relative 2^-13 of a product, where the output rounds at 2^-9.
//   sum_k x (q - z) = sum_k x q - z sum_k x,
// the second sum in fp32 once per token and group.  The group's scale multiplies
// the finished sum in fp32.  A token that holds an infinity or a NaN gets NaN;
// others do not see it (tokens are rows of the matrix product).
//
// Groups smaller than a chunk.  The MFMA sums over 128 k; with G = 64 or 32 it
// runs 2 or 4 times, each with the block scales of the other groups at 2^-127
// on both operands (their products underflow).  A block of the instruction is
// half of the registers of two lane groups, so with G = 32 two words change
// places between neighbouring lane groups first (permlane16_swap).
//
// Layout.  The activations are the MFMA's row operand and 16 weight rows its
// column operand, so a lane's four results are four rows of ONE weight row and
// need one scale.  Up to 8 tokens, rows 0-7 are their hi and 8-15 their lo parts
// and one MFMA does both (the two results of a token are added at the end, and
// each carries half of the zero point's sum); beyond, a second MFMA takes lo.
// A 16-byte load gives a lane 32 consecutive codes of its row.
//
// A block has 16 waves and a CU to itself (the grid is persistent); they share a
// tile of 16 rows (gate and up rows for a gated layer), U chunks of k each a
// step.  A block's work is one stream of steps through its tiles, with two
// steps' weights in flight in registers, across tiles.  The 16 waves' sums meet in
// LDS in wave order (deterministic).
//
// Activations live in LDS as records, one per chunk: hi and lo of every token in
// operand order, their exponents, and the groups' sums.  Up to 160 of them
// (tokens x chunks) a block makes its own from x, while its first weights are
// in flight; more are made once per call by a small kernel into the workspace
// and copied to LDS.  Where all records do not fit, k is cut into slices that
// do: each slice has its share of the blocks, the slices' sums go to the
// workspace in fp32 and a last small kernel adds them in order.  (Streaming the
// records through LDS beside the weights, a step at a time, made every step
// wait for its records: 60 us against 55 us for 16 tokens through 8192 -> 28672.)
//
// What it reaches (GPU time in a replayed graph).  A call of many tiles takes about
// 8 us (start, records, first loads, last sums) and then reads 5.7 TB/s, where a
// copy moves 5.15.  One token through 4096 -> 4096 takes 4.6 us, through the gated
// 8192 -> 28672 -> 8192 block 80 us (363 MB, 4.5 TB/s), 16 tokens through
// 8192 -> 28672 47 to 55 us (148 MB; two slices of k, three launches).
#include <algorithm>

#include "common.h"
#include "decode_w4.h"
#include "lds_dma.h"

namespace fmlp {

namespace {

constexpr int kWaves = 16;   // one block a CU
constexpr int kThreads = kWaves * 64;
constexpr int kChunk = 128;   // k of one 16-byte load of the 4 lanes of a row
// Tokens x chunks whose records a block makes itself, up to three passes of its
// threads, all of x's values requested before the weights.  Against the small kernel's
// launch: 96 units 5.6 us (6.8), 128 11.4 (12.4), 160 12.3 (13.2), but 192 8.1
// (7.7) and 8.8 (8.2).
constexpr int kUnitsInside = 160;

// A raw buffer of `bytes` at base, both wave-uniform: readfirstlane says so to
// the compiler, which computes tile addresses on the vector unit and would
// issue every load in a loop over the lanes' descriptors (and drain all loads
// before it).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t w4_desc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint64_t u = (uint64_t)uniform32((uint32_t)(a >> 32)) << 32 | uniform32((uint32_t)a);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), (short)0, (int)uniform32(bytes), 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t d, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(d, (int)off, 0, 0));
}

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Records: one per chunk.  Operand bytes of 2 M slots (token m's hi in slot m, lo
// in slot M + m) as [half][lane group][slot][16], the slots' exponents (+ 127,
// one byte each), then [group][tokens] fp32 sums.
// ---------------------------------------------------------------------------
struct Record {
  int slots, exps, sums, tokens, bytes;
};
__host__ __device__ __forceinline__ Record record_of(int M, int gs) {
  Record r;
  r.slots = 2 * M;
  r.exps = r.slots * 128;
  r.sums = r.exps + (M <= 8 ? 16 : 32);
  r.tokens = M <= 4 ? 4 : M <= 8 ? 8 : 16;
  r.bytes = r.sums + (kChunk >> gs) * r.tokens * 4;
  return r;
}

// v of another lane of the row of 16 (the DPP control says which)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// 16 lanes (i = 0 .. 15) put one token's chunk into its record: lane i has k
// 8 i .. 8 i + 7 (zeros past K).
template <int GS, bool ZEROS>
__device__ __forceinline__ void put_record(uint8_t* rec, const Record& R, const u32x4_t& xv, int m, int M, int i) {
  float v[8];
  unpack_bf16x8(xv, v);
  float top = 0.f, sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(v[j]);
    top = fmaxf(top, a < __builtin_inff() ? a : 0.f);
    sum += v[j];
  }
  top = fmaxf(top, dpp<0xB1>(top));    // quad_perm 1 0 3 2
  top = fmaxf(top, dpp<0x4E>(top));    // quad_perm 2 3 0 1
  top = fmaxf(top, dpp<0x141>(top));   // row_half_mirror: the other quad of 8
  top = fmaxf(top, dpp<0x140>(top));   // row_mirror: the other 8 of 16
  sum += dpp<0xB1>(sum);
  sum += dpp<0x4E>(sum);
  if constexpr (GS > 5) sum += dpp<0x141>(sum);
  if constexpr (GS > 6) sum += dpp<0x140>(sum);
  const uint32_t bits = __float_as_uint(top);
  // at least -122: the lo part's exponent byte stays positive
  const int e = max((int)(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), -122);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t hi[2], lo[2];   // even k, odd k: the order of a word's low and high halves
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    float a[4], h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = v[2 * j + o] * inv;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a[0], a[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a[2], a[3], w, true);
    hi[o] = (uint32_t)w;
    const auto h0 = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), h1 = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    h[0] = h0[0];
    h[1] = h0[1];
    h[2] = h1[0];
    h[3] = h1[1];
    int l = __builtin_amdgcn_cvt_pk_fp8_f32(16.f * (a[0] - h[0]), 16.f * (a[1] - h[1]), 0, false);
    l = __builtin_amdgcn_cvt_pk_fp8_f32(16.f * (a[2] - h[2]), 16.f * (a[3] - h[3]), l, true);
    lo[o] = (uint32_t)l;
  }
  // word d of lane group g of the weights: its place in the operand
  const int g = i >> 2, d = i & 3;
  const int half = GS == 5 ? g & 1 : d >> 1;
  const int lg = GS == 5 ? (g & 2) | (d >> 1) : g;
  uint8_t* at = rec + (half * 4 + lg) * (R.slots * 16) + (d & 1) * 8;
  *reinterpret_cast<uint2*>(at + m * 16) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(at + (M + m) * 16) = make_uint2(lo[0], lo[1]);
  if (i == 0) {
    rec[R.exps + m] = (uint8_t)(e + 127);
    rec[R.exps + M + m] = (uint8_t)(e + 123);
  }
  constexpr int kPer = (1 << GS) / 8;   // lanes of a group
  if (i % kPer == 0)
    reinterpret_cast<float*>(rec + R.sums)[(i / kPer) * R.tokens + m] = (ZEROS ? -1.f : -8.f) * (M <= 8 ? 0.5f : 1.f) * sum;
}

constexpr int kPutThreads = 256;
template <int GS, bool ZEROS>
__global__ __launch_bounds__(kPutThreads) void w4_records_kernel(const uint16_t* x, int M, int K, int chunks,
                                                                 uint8_t* out) {
  const int u = blockIdx.x * (kPutThreads / 16) + (threadIdx.x >> 4);   // chunk u / M, token u % M
  const int i = threadIdx.x & 15;
  if (u >= M * chunks) return;   // 16 lanes together
  const Record R = record_of(M, GS);
  const int c = u / M, m = u - c * M;
  const int k = c * kChunk + i * 8;
  put_record<GS, ZEROS>(out + (int64_t)c * R.bytes, R, k < K ? ld16(x + (int64_t)m * K + k) : zero4(), m, M, i);
}

// the 32 codes of a lane's 4 words as operand bytes, words 0 and 1 in the first
// half of the registers (G = 32: neighbouring lane groups exchange words first)
template <int GS>
__device__ __forceinline__ i32x8_t expand(const u32x4_t& q) {
  uint32_t w[4] = {q[0], q[1], q[2], q[3]};
  if constexpr (GS == 5) {
    const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(w[1], w[3], false, false);
    w[0] = a[0];
    w[2] = a[1];
    w[1] = b[0];
    w[3] = b[1];
  }
  i32x8_t r;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    r[2 * d] = (int)(w[d] & 0x0F0F0F0Fu);
    r[2 * d + 1] = (int)((w[d] >> 4) & 0x0F0F0F0Fu);
  }
  return r;
}

// n bf16 values of a row at byte offset off; NW words.  WHOLE: off is a
// multiple of the vector's size; else each value is loaded by itself, those
// at or past `have` as zeros.
template <int NV, bool WHOLE>
struct Values {
  static constexpr int kWords = WHOLE ? (NV + 1) / 2 : NV;
  static constexpr int kLoads = !WHOLE ? NV : NV <= 8 ? 1 : NV / 8;
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

// A wave's step: NS weight streams (gate and up) of U chunks, and the bias of the
// tile's 16 rows with its last step (nothing is read in the others).
template <int NS, int U, int NV, bool WHOLE, bool ZEROS>
struct Batch {
  u32x4_t w[NS][U];
  Values<NV, WHOLE> s[NS];
  Values<ZEROS ? NV : 2, WHOLE> z[ZEROS ? NS : 1];
  uint32_t bias;
};

// How a call is cut: k slices of `chunks` chunks each (the last may have fewer),
// with per_slice blocks each; parts: [slice][set][M][N] fp32, or nullptr (one slice).
struct W4Cut {
  int slices, chunks, per_slice;
  float* parts;
};

// GS: log2 of the group size.  WHOLE: a slice is a multiple of U chunks, so a
// step exists in full or not at all and scales come as aligned vectors.  M8: at
// most 8 tokens.
template <bool DUAL, int U, int GS, bool ZEROS, bool WHOLE, bool M8>
__global__ __launch_bounds__(kThreads) void decode_w4_kernel(W4Layer L, int M, W4Cut cut) {
  constexpr int NS = DUAL ? 2 : 1;
  constexpr int GPC = kChunk >> GS;        // groups per chunk
  constexpr int NV = U * GPC;              // scales of a step
  constexpr int SC = kWaves * U;           // chunks of a block's step
  using B = Batch<NS, U, NV, WHOLE, ZEROS>;
  // load instructions of a step's weights, scales and zero points
  constexpr int kLoads = NS * (U + (ZEROS ? 2 : 1) * Values<NV, WHOLE>::kLoads) + (DUAL ? 0 : 1);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15;   // weight row of a tile; row of the activation operand
  const int g = lane >> 4;
  const int K = (int)L.K;
  const int groups = K >> GS;
  const int slice = blockIdx.x % cut.slices, first = blockIdx.x / cut.slices;   // the block's slice, its first tile
  const int cb = slice * cut.chunks;                                              // first chunk of the slice
  const int chunks = min((K + kChunk - 1) / kChunk - cb, cut.chunks);
  const int steps = (chunks + SC - 1) / SC;   // of a tile
  const int tiles = (int)((L.N + 15) / 16);
  const int total = (tiles - first + cut.per_slice - 1) / cut.per_slice * steps;   // per_slice <= tiles
  const Record R = record_of(M, GS);

  const uint32_t wlane = (uint32_t)(r * (K / 2) + g * 16);
  const uint32_t slane = (uint32_t)(r * groups) * 2u;
  // the lane's slot (rows without a token read slot 0; their results are not used)
  const int slot = M8 ? ((r & 7) < M ? (r & 7) + (r >> 3) * M : 0) : (r < M ? r : 0);
  const int xop = g * (R.slots * 16) + slot * 16;    // the lane's operand bytes in a record, first half
  const int xsum = R.sums + 16 * (M8 ? (R.tokens == 8 ? g & 1 : 0) : g);   // the sums of its 4 result rows' tokens

  const __amdgpu_buffer_rsrc_t dbias = w4_desc(L.bias ? L.bias : L.x, L.bias ? (uint32_t)L.N * 2u : 0u);
  int it = first, is = 0;   // tile and step of the next weights issued
  auto issue = [&](B& b) {
    const int64_t n0 = (int64_t)it * 16;
    const int rows = (int)max<int64_t>(min<int64_t>(16, L.N - n0), 0);
    const int c0 = (is * kWaves + wave) * U;   // within the slice
    const bool any = c0 < chunks;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const __amdgpu_buffer_rsrc_t dw = w4_desc((s ? L.q1 : L.q0) + n0 * (K / 2), (uint32_t)rows * (uint32_t)(K / 2));
      const __amdgpu_buffer_rsrc_t ds = w4_desc((s ? L.s1 : L.s0) + n0 * groups, (uint32_t)rows * (uint32_t)groups * 2u);
      const uint32_t wo = wlane + (any ? (uint32_t)(cb + c0) * 64u : kOutOfRange);
#pragma unroll
      for (int j = 0; j < U; ++j) b.w[s][j] = load16(dw, WHOLE || c0 + j < chunks ? wo + 64u * j : kOutOfRange);
      const uint32_t so = slane + (any ? (uint32_t)((cb + c0) * GPC) * 2u : kOutOfRange);
      b.s[s].load(ds, so, min(groups - cb * GPC, chunks * GPC) - c0 * GPC);
      if constexpr (ZEROS)
        b.z[s].load(w4_desc((s ? L.z1 : L.z0) + n0 * groups, (uint32_t)rows * (uint32_t)groups * 2u), so, min(groups - cb * GPC, chunks * GPC) - c0 * GPC);
    }
    if constexpr (!DUAL)
      b.bias = __builtin_amdgcn_raw_buffer_load_b16(dbias, is + 1 == steps ? (int)((uint32_t)(it * 16 + r) * 2u) : (int)kOutOfRange, 0, 0);
    if (++is == steps) {
      is = 0;
      it += cut.per_slice;
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
    if constexpr (!DUAL) asm volatile("" : "+v"(b.bias));
  };
  f32x4_t tot[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) tot[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // block scales of the weights: 2^9 where the lane's block belongs to group t
  int bscale[GPC];
  bool mine_t[GPC];
#pragma unroll
  for (int t = 0; t < GPC; ++t) {
    mine_t[t] = GS == 7 || (GS == 6 ? (g & 1) == t : g == (t & 1) * 2 + (t >> 1));
    bscale[t] = mine_t[t] ? 136 : 0;
  }
  auto operand = [&](const uint8_t* rec, int at) {
    const u32x4_t a = *reinterpret_cast<const u32x4_t*>(rec + at);
    const u32x4_t b = *reinterpret_cast<const u32x4_t*>(rec + at + 4 * (R.slots * 16));
    i32x8_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = (int)a[j];
      v[4 + j] = (int)b[j];
    }
    return v;
  };
  auto consume = [&](const B& b, int step) {
    const int c0 = (step * kWaves + wave) * U;
    const uint8_t* recs = lds + c0 * R.bytes;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (WHOLE ? c0 >= chunks : c0 + j >= chunks) break;   // wave-uniform
      const uint8_t* rec = recs + j * R.bytes;
      const i32x8_t xh = operand(rec, xop);
      const int eh = rec[R.exps + slot];
      i32x8_t xl;
      if constexpr (!M8) xl = operand(rec, xop + M * 16);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const i32x8_t w = expand<GS>(b.w[s][j]);
        f32x4_t acc[GPC];
#pragma unroll
        for (int t = 0; t < GPC; ++t) {
          const f32x4_t sums = *reinterpret_cast<const f32x4_t*>(rec + xsum + t * (R.tokens * 4));
          const int ea = mine_t[t] ? eh : 0;
          if constexpr (ZEROS) {
            const float z = b.z[s].f32(j * GPC + t);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[t][v] = z * sums[v];
          } else {
            acc[t] = sums;
          }
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xh, w, acc[t], 0, 0, 0, ea, 0, bscale[t]);
          if constexpr (!M8) {
            const int el = mine_t[t] ? eh - 4 : 0;
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xl, w, acc[t], 0, 0, 0, el, 0, bscale[t]);
          }
        }
#pragma unroll
        for (int t = 0; t < GPC; ++t) {
          const float sc = b.s[s].f32(j * GPC + t);
#pragma unroll
          for (int v = 0; v < 4; ++v) tot[s][v] = fmaf(sc, acc[t][v], tot[s][v]);
        }
      }
    }
  };
  constexpr int kRedLanes = M8 ? 32 : 64;
  // One output of a tile per thread o < 256: weight row o % 16, token
  // 4 ((o / 16) % 4) + (o / 64) % 4.
  const int ov = (threadIdx.x >> 6) & 3, om = 4 * g + ov;
  // A finished tile: the waves' partial sums, added in wave order.  (Two
  // buffers with one barrier a tile took LDS from the records, a third slice of
  // k at 16 tokens and K = 8192, and measured no faster.)
  auto finish = [&](int tile, float bias) {
    f32x4_t* red = reinterpret_cast<f32x4_t*>(lds + chunks * R.bytes);   // [wave][stream][lane]
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if constexpr (M8) {   // rows m and m + 8 are one token's: the lower half wave takes both
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint32_t t = __float_as_uint(tot[s][v]);
          const auto h = __builtin_amdgcn_permlane32_swap(t, t, false, false);
          tot[s][v] = __uint_as_float(h[0]) + __uint_as_float(h[1]);
        }
      }
      if (!M8 || lane < 32) red[(wave * NS + s) * kRedLanes + lane] = tot[s];
      tot[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    lds_barrier();
    const int64_t n = (int64_t)tile * 16 + r;
    if (threadIdx.x < 256 && om < M && n < L.N) {
      float z[NS];
#pragma unroll
      for (int e = 0; e < NS; ++e) {
        z[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          z[e] += reinterpret_cast<const float*>(red + (w * NS + e) * kRedLanes + lane)[ov];
        }
      }
      if (cut.parts) {
#pragma unroll
        for (int e = 0; e < NS; ++e) cut.parts[((int64_t)(slice * NS + e) * M + om) * L.N + n] = z[e];
      } else {
        const float out = DUAL ? apply_act(z[0], L.act) * z[NS - 1] : apply_act(z[0] + bias, L.act);
        const __bf16 ob = (__bf16)out;
        L.y[(int64_t)om * L.N + n] = __builtin_bit_cast(uint16_t, ob);
      }
    }
    lds_barrier();   // the sums are read before the next tile's are written
  };

  B A, C;
  int ct = first, cs = 0;   // tile and step being consumed
  // A step's weights are multiplied and their registers take those of the step
  // after the next.
  auto step = [&](B& now) {
    hold(now);
    consume(now, cs);
    const float bias = DUAL ? 0.f : __uint_as_float(now.bias << 16);
    issue(now);   // past the last step: descriptors of no rows, nothing is read
    if (++cs == steps) {
      finish(ct, bias);
      cs = 0;
      ct += cut.per_slice;
    }
  };
  // The first step's weights go out before the records are made, the second's
  // after: a CU takes only so many requests, and with both ahead every wave
  // stood in its second step's issue until the first had arrived (7 us).
  if (L.records) {   // made by the kernel before
    const uint32_t xlds = lds_addr(lds);
    const int bytes = chunks * R.bytes;
    const i32x4_t rd = make_desc(reinterpret_cast<uint64_t>(L.records + (int64_t)cb * R.bytes), (uint32_t)bytes);
    for (int t = wave; t * 1024 < bytes; t += kWaves)   // wave-uniform; the last piece's lanes past the end write nothing
      if (t * 1024 + lane * 16 < bytes) asm_load_lds(rd, uniform32(xlds + (uint32_t)(t * 1024)), (uint32_t)(t * 1024 + lane * 16));
    issue(A);
    wait_vm<kLoads < 63 ? kLoads : 63>();   // loads return in order: all but the weights have landed
  } else {
    // 16 lanes a unit (chunk u / M, token u % M)
    constexpr int kUnits = kThreads / 16;
    static_assert(kUnitsInside <= 3 * kUnits, "three passes");
    const int i16 = threadIdx.x & 15;
    auto fetch = [&](int u) {
      const int c = u / M, k = (cb + c) * kChunk + i16 * 8;
      return u < M * chunks && k < K ? ld16(L.x + (int64_t)(u - c * M) * K + k) : zero4();
    };
    int u = threadIdx.x >> 4;
    u32x4_t xv = fetch(u), xn = fetch(u + kUnits), xo = fetch(u + 2 * kUnits);
    issue(A);
#pragma clang loop unroll(disable)
    for (; u < M * chunks; u += kUnits) {
      const int c = u / M;
      put_record<GS, ZEROS>(lds + c * R.bytes, R, xv, u - c * M, M, i16);
      xv = xn;
      xn = xo;
    }
  }
  lds_barrier();
  issue(C);
  int i = 0;
  for (; i + 1 < total; i += 2) {
    step(A);
    step(C);
  }
  if (i < total) step(A);
  wait_vm<0>();
}

// y = act(sum of the slices + bias), or act(gate) * up: one thread per output.
template <bool DUAL>
__global__ __launch_bounds__(256) void w4_sum_kernel(W4Layer L, int M, W4Cut cut) {
  const int64_t MN = (int64_t)M * L.N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= MN) return;
  float z = 0.f, u = 0.f;
  for (int s = 0; s < cut.slices; ++s) {
    z += cut.parts[(int64_t)s * (DUAL ? 2 : 1) * MN + i];
    if (DUAL) u += cut.parts[((int64_t)s * 2 + 1) * MN + i];
  }
  if (!DUAL && L.bias) z += bf16_to_f32(L.bias[i % L.N]);
  const __bf16 o = (__bf16)(DUAL ? apply_act(z, L.act) * u : apply_act(z, L.act));
  L.y[i] = __builtin_bit_cast(uint16_t, o);
}

constexpr int64_t kLdsMax = 160 * 1024;   // of a block, one a CU

int log2_group(int G) { return G == 32 ? 5 : G == 64 ? 6 : 7; }
int64_t red_bytes(int64_t M, bool dual) { return (int64_t)kWaves * (dual ? 2 : 1) * (M <= 8 ? 32 : 64) * 16; }

// The k slices of a call: as few as have records that fit in LDS, of equal
// numbers of chunks (a multiple of 4, so that every slice starts on whole steps).
W4Cut cut_of(int64_t M, int64_t K, int G, bool dual) {
  const int64_t chunks = (K + kChunk - 1) / kChunk;
  const int64_t fit = (kLdsMax - red_bytes(M, dual)) / record_of((int)M, log2_group(G)).bytes / 4 * 4;
  W4Cut c{};
  const int64_t slices = (chunks + fit - 1) / fit;
  c.chunks = (int)(((chunks + slices - 1) / slices + 3) / 4 * 4);
  c.slices = (int)((chunks + c.chunks - 1) / c.chunks);
  return c;
}
bool made_inside(int64_t M, const W4Cut& c) { return M * c.chunks <= kUnitsInside; }
size_t records_bytes(int64_t M, int64_t K, int G, const W4Cut& c) {
  const size_t b = (size_t)((K + kChunk - 1) / kChunk) * (size_t)record_of((int)M, log2_group(G)).bytes;
  return made_inside(M, c) ? 0 : (b + 255) / 256 * 256;
}

template <bool DUAL, int GS, bool ZEROS, bool M8>
hipError_t launch_w4(const W4Layer& L, int M, int cus, hipStream_t s) {
  const int chunks = (int)((L.K + kChunk - 1) / kChunk);
  W4Cut cut = cut_of(M, L.K, L.G, DUAL);
  const size_t records = records_bytes(M, L.K, L.G, cut);
  if ((records || cut.slices > 1) && L.scratch == nullptr) return hipErrorInvalidValue;
  W4Layer P = L;
  P.records = records ? L.scratch : nullptr;
  if (records) {
    const int units = M * chunks;
    hipLaunchKernelGGL((w4_records_kernel<GS, ZEROS>), dim3((unsigned)((units + kPutThreads / 16 - 1) / (kPutThreads / 16))),
                       dim3(kPutThreads), 0, s, L.x, M, (int)L.K, chunks, P.records);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const int64_t tiles = (L.N + 15) / 16;
  if (cut.slices > 1) cut.parts = reinterpret_cast<float*>(L.scratch + records);
  cut.per_slice = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, cus / cut.slices));
  const int64_t lds = std::min(chunks, cut.chunks) * (int64_t)record_of(M, GS).bytes + red_bytes(M, DUAL);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(cut.per_slice * cut.slices)), dim3(kThreads), (unsigned)lds, s, P, M, cut);
    return hipGetLastError();
  };
  constexpr int U = (DUAL || (GS == 5 && ZEROS && !M8)) && GS < 7 ? 2 : 4;
  hipError_t e;
  if (U == 4 && cut.chunks >= kWaves * 4 && L.K % (4 * kChunk) == 0)
    e = go(decode_w4_kernel<DUAL, U, GS, ZEROS, true, M8>);
  else if (L.K % (2 * kChunk) == 0)
    e = go(decode_w4_kernel<DUAL, 2, GS, ZEROS, true, M8>);
  else
    e = go(decode_w4_kernel<DUAL, 2, GS, ZEROS, false, M8>);
  if (e != hipSuccess || cut.slices == 1) return e;
  hipLaunchKernelGGL((w4_sum_kernel<DUAL>), dim3((unsigned)(((int64_t)M * L.N + 255) / 256)), dim3(256), 0, s, P, M, cut);
  return hipGetLastError();
}

template <bool DUAL, int GS>
hipError_t by_zeros(const W4Layer& L, int M, int cus, hipStream_t s) {
  if (M <= 8) return L.z0 ? launch_w4<DUAL, GS, true, true>(L, M, cus, s) : launch_w4<DUAL, GS, false, true>(L, M, cus, s);
  return L.z0 ? launch_w4<DUAL, GS, true, false>(L, M, cus, s) : launch_w4<DUAL, GS, false, false>(L, M, cus, s);
}
template <bool DUAL>
hipError_t by_group(const W4Layer& L, int M, int cus, hipStream_t s) {
  switch (L.G) {
    case 32: return by_zeros<DUAL, 5>(L, M, cus, s);
    case 64: return by_zeros<DUAL, 6>(L, M, cus, s);
    case 128: return by_zeros<DUAL, 7>(L, M, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

size_t decode_w4_scratch_bytes(int64_t M, int64_t K, int64_t N, int G, bool dual) {
  const W4Cut c = cut_of(M, K, G, dual);
  return records_bytes(M, K, G, c) + (c.slices > 1 ? (size_t)c.slices * (dual ? 2 : 1) * (size_t)M * (size_t)N * 4 : 0);
}

hipError_t launch_decode_w4(const W4Layer& L, int M, int cus, hipStream_t s) {
  if (cus < 1 || M < 1 || M > 16 || L.K < 32 || L.K % L.G != 0 || L.N < 1) return hipErrorInvalidValue;
  if (L.q1 != nullptr && (L.z0 == nullptr) != (L.z1 == nullptr)) return hipErrorInvalidValue;
  return L.q1 ? by_group<true>(L, M, cus, s) : by_group<false>(L, M, cus, s);
}

}  // namespace fmlp
