// Large-token bf16 GEMM with a register epilogue, for gfx950.
//
//   C[rows, N] = epilogue(A[rows, K] . B[N, K]^T),  fp32 accumulate
//
// Both operands are K-contiguous (the weight is read as stored, [out, in]):
// "Profiling in PyTorch (Part 2): From nn.Linear to a Fused MLP", section
// "Where did the transpose go? Kernel layouts and pre-ops".  The epilogue runs
// on the fp32 accumulator in registers and writes only the final tile
// (section "Why are there no separate mul and add kernels?"):
//   GEMM_OUT_BF16        bias add + activation (none / exact GELU / tanh GELU /
//                        ReLU / SiLU)
//   GEMM_OUT_GEGLU       gate and up projections share every A tile; the block
//                        holds matching g and u accumulators and writes only
//                        m = act(g) * u, act = tanh GELU for GeGLU (section
//                        "The fused Triton kernel": the intermediate never
//                        makes an HBM round trip) or another gate activation
//   GEMM_OUT_F32_SCALED  fp32 output scaled per row (expert combine weights;
//                        no scale: 1), optionally split over K into parts
//                        that each write their own copy (summed in order by
//                        the caller: the MoE combine, or the backward's
//                        weight gradients)
//   GEMM_OUT_DACT        backward of a Linear + activation: the forward GEMM
//                        recomputes z = x W^T + b in registers and writes only
//                        dz = dy * act'(z)
//   GEMM_OUT_DGLU        backward of the gated block: the gate+up GEMM
//                        recomputes g and u and, with the incoming dm, writes
//                        m = act(g) * u, dg = dm * u * act'(g) and du = dm * act(g)
//   GEMM_OUT_GLU_SAVE    GEMM_OUT_GEGLU that also keeps g and u for the
//                        backward pass as E4M3 codes with a power-of-two scale
//                        for each row and 32 columns
//   GEMM_OUT_DGLU_SAVED  backward from those codes: the accumulator is dm, and
//                        m, dg and du follow from the stored g and u
//
// Structure: a block computes a BM x BN tile with WAVES_M x WAVES_N waves
// (256 x 256 with 8 waves of 128 x 64 for large inputs: two waves per SIMD,
// so one issues MFMAs while the other waits, each with 128 fp32 accumulators
// in AGPRs).  K advances in stages of BK (64 for the
// large tile: 128-byte LDS rows, two ring slots; 32 for the small one:
// 64-byte rows, four slots).  Stages stream from memory straight into the
// LDS ring with buffer loads that write LDS, R - 1 stages ahead of the MFMAs
// and with no register staging; each wave waits only for its own loads of
// the stage it is about to read, and one workgroup barrier per stage
// publishes the stage and frees the slot the next loads go to.  Each 1 KB
// load instruction fills 1 KB of LDS in lane order, a lane fetching the
// global chunk whose permuted home (swz_a, swz_b below) is its own LDS
// position, so the 16-byte fragment reads are bank-conflict free.  Rows past
// the tile's end and chunks past K are requested out of range and arrive as
// zeros.  The loop is issued in a fixed order: MFMAs of a k-step run from
// registers while the next k-step's fragments are read from LDS and the next
// stage's loads are issued, one such instruction after each MFMA.
// v_mfma_f32_16x16x32_bf16 is fed with the weight as the row operand and the
// activation as the column operand; the weight rows of a fragment pair are
// interleaved so each lane ends with 8 consecutive output columns of one row,
// stored as one 16-byte write.
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include "common.h"
#include "gemm_train.h"
#include "kernels.h"
#include "lds_dma.h"

namespace fmlp {

namespace {

// LDS layout.  A stage holds BK k of every tile row: rows of BK * 2 bytes
// (CH = BK / 8 chunks of 16 B).  A ds_read_b128 takes four LDS cycles of 16
// lanes (measured on gfx950): the cycle of lane l is set by its half-wave
// (l >> 5) and the parity of its quad index bits ((l >> 2) & 7), and within
// a cycle the lanes must hit distinct 16-byte bank groups (unit index mod 16).
// A fragment read puts k group lg = l >> 4 and row offset li = l & 15 on each
// lane, so a cycle holds two k groups, each with half of the row offsets.
// Chunk c of row r sits at slot c ^ swz(r), with one permutation for
// activation fragments (16 consecutive rows) and one for weight fragments
// (rows interleaved in groups of 4: 8*(l/4) + (l%4)), chosen so every cycle
// of both kinds of read is conflict free:
//   64-byte rows:  q = bits 2-3 (activation) or 3-4 (weight) of r, slot
//                  permutation {0, 2, 3, 1}[q] (the plain q pairs lanes);
//   128-byte rows: bits 1-3 of r (activation), bits 1, 3, 4 (weight).
template <int CH>
__host__ __device__ constexpr int swz_a(int r) {
  if constexpr (CH == 4) return (0x78 >> (2 * ((r >> 2) & 3))) & 3;
  else return (r >> 1) & 7;
}
template <int CH>
__host__ __device__ constexpr int swz_b(int r) {
  if constexpr (CH == 4) return (0x78 >> (2 * ((r >> 3) & 3))) & 3;
  else return ((r >> 1) & 1) | ((r >> 2) & 6);
}

// Weight fragment f of a wave covers tile rows w_lane_row + w_delta(f), with
// the rows permuted so that every lane ends up holding runs of 8 consecutive
// output columns (one 16-byte store each):
//   16x16x32 (M32 = false): the rows of a fragment pair interleave, so lane
//     group g holds columns 8g .. 8g+7 of the pair's 32 columns;
//   32x32x16 (M32 = true): fragment row i (= lane % 32) reads weight row
//     rho(i) = 16 (i >> 4) + 8 ((i >> 2) & 1) + 4 ((i >> 3) & 1) + (i & 3), so
//     the 16 results of lane half h (accumulator registers 0-7 and 8-15) are
//     columns 8h .. 8h+7 and 16+8h .. 16+8h+7 of the fragment's 32.
// With two weight sets, fragments [0, FN/2) read the first and [FN/2, FN) the
// second.
__host__ __device__ constexpr int rho32(int i) {
  return 16 * (i >> 4) + 8 * ((i >> 2) & 1) + 4 * ((i >> 3) & 1) + (i & 3);
}
__host__ __device__ constexpr int w_delta(int f, int FN, int BN, bool dual, bool m32) {
  const int half = FN / 2;
  const int set = dual ? f / half : 0;
  const int fl = dual ? f % half : f;
  return set * (BN / 2) + (m32 ? fl * 32 : (fl >> 1) * 32 + 4 * (fl & 1));
}
__host__ __device__ constexpr int w_lane_row(int wn, int li, int TN, bool dual, bool m32) {
  return wn * (dual ? TN / 2 : TN) + (m32 ? rho32(li) : 8 * (li >> 2) + (li & 3));
}
// The swizzles read only bits 1-4 of a row, so every fragment of a wave has
// the same chunk permutation as its first one and its LDS address is the
// first one's plus a constant.  Checked exhaustively at compile time.
template <int CH, int TM, int TN, int FM, int FN, int BN, int WAVES_M, int WAVES_N, bool DUAL, bool M32>
constexpr bool fragment_swizzle_is_uniform() {
  constexpr int MR = M32 ? 32 : 16;
  for (int li = 0; li < MR; ++li) {
    for (int wm = 0; wm < WAVES_M; ++wm)
      for (int f = 0; f < FM; ++f)
        if (swz_a<CH>(wm * TM + f * MR + li) != swz_a<CH>(wm * TM + li)) return false;
    for (int wn = 0; wn < WAVES_N; ++wn) {
      const int r0 = w_lane_row(wn, li, TN, DUAL, M32);
      for (int f = 0; f < FN; ++f)
        if (swz_b<CH>(r0 + w_delta(f, FN, BN, DUAL, M32)) != swz_b<CH>(r0)) return false;
    }
  }
  return true;
}
// The 32-row fragment reads are bank-conflict free under the measured model
// of a ds_read_b128 (four 16-lane cycles; cycle of lane l: l >> 5 and the
// parity of the bits of (l >> 2) & 7; units within a cycle distinct mod 16):
// checked exhaustively at compile time for both operands' row maps.
template <int CH>
constexpr bool m32_reads_conflict_free(bool weights) {
  if (CH != 8) return false;
  for (int c0 = 0; c0 < CH; c0 += 2)
    for (int base = 0; base < 256; base += 32)
      for (int cyc = 0; cyc < 4; ++cyc) {
        bool seen[16] = {};
        for (int l = 0; l < 64; ++l) {
          const int q = (l >> 2) & 7;
          const int par = (q ^ (q >> 1) ^ (q >> 2)) & 1;
          if (((l >> 5) << 1 | par) != cyc) continue;
          const int i = l & 31;
          const int r = base + (weights ? rho32(i) : i);
          const int c = c0 + (l >> 5);
          const int slot = c ^ (weights ? swz_b<CH>(r) : swz_a<CH>(r));
          const int unit = (r * CH + slot) & 15;
          if (seen[unit]) return false;
          seen[unit] = true;
        }
      }
  return true;
}
static_assert(m32_reads_conflict_free<8>(false) && m32_reads_conflict_free<8>(true),
              "32-row fragment reads of 128-byte rows");

// k-major operand tiles (the backward's contractions over the rows of both
// operands, read without a transpose copy).  A stage holds 64 k-rows of the
// tile's 256 columns: rows of 512 bytes, 32 chunks of 16 B, chunk c of row k
// at slot c ^ kswz(k) (128 columns: rows of 256 bytes, 16 chunks).  A fragment (16 columns x 32 k) is two transposing
// reads (ds_read_b64_tr_b16): within each 16-lane group, lane 4 r + q points
// at 4 consecutive columns of k-row kbase + r, and lane j gets column group
// j / 4, element j % 4 of all four rows, i.e. 4 consecutive k of one column;
// kbase = 32 ks + 8 (lane / 16) and + 4 give a lane the 8 consecutive k of the
// 16x16x32 operand, in the order the row-major reads give them.  kswz moves
// chunk bits 1-3: the 8 k-rows of a half-wave's read land on 8 distinct chunk
// pairs (an activation fragment's 16 consecutive columns are one chunk pair
// per row), so those reads are conflict free.  A weight fragment keeps the
// pair permutation that gives each lane runs of 8 output columns (16-byte
// stores): its 16 columns are 4 half chunks, all in the same half, so its
// reads take two passes.  (Weight columns kept in order instead, 4-column
// runs with 8-byte stores and conflict-free reads, measured 1 % slower on the
// large backward.)
__host__ __device__ constexpr int kswz(int k) { return 2 * ((k & 7) ^ (((k >> 3) & 1) << 2)); }
typedef short v4i16_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4_t lds_read_tr_pair(uint32_t addr0, uint32_t addr1) {
  typedef __attribute__((address_space(3))) v4i16_t lds_v4;
  const v4i16_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)(uintptr_t)addr0);
  const v4i16_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)(uintptr_t)addr1);
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_shufflevector(a, a, 0, 1));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_shufflevector(a, a, 2, 3));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_shufflevector(b, b, 0, 1));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_shufflevector(b, b, 2, 3));
  return r;
}

// The main loop interleaves MFMAs with loads and LDS reads in a fixed order.
// Instruction selection moves an MFMA builtin freely (it touches no memory),
// so the loop issues them as volatile asm, which keeps its place among the
// other volatile asm (loads into LDS, waits, barriers); the accumulator is
// pinned in AGPRs and updated in place.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void mfma_ordered(f32x4_t& acc, const u32x4_t& a, const u32x4_t& b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b) : "memory");
}
// D[32x32] += A[32x16] B[16x32]: lane l supplies row (l % 32) of A and column
// (l % 32) of B, each as 8 consecutive k of k-group l / 32, and receives
// column l % 32 of D, rows 8 (r / 4) + 4 (l / 32) + r % 4 in register r.
__device__ __forceinline__ void mfma_ordered(f32x16_t& acc, const u32x4_t& a, const u32x4_t& b) {
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b) : "memory");
}
// A copy of v the compiler cannot see through: what is computed from it
// stays where it is written instead of being hoisted out of the tile loop and
// kept live (in registers the main loop needs) across it.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
// materialise a value in AGPRs at this point of the instruction stream
__device__ __forceinline__ void pin_agpr(f32x4_t& acc) { asm volatile("" : "+a"(acc)); }
__device__ __forceinline__ void pin_agpr(f32x16_t& acc) { asm volatile("" : "+a"(acc)); }
// the same, also ordered after every memory access before it: reads of the
// accumulator cannot be hoisted above the preceding output stores (which
// would have every accumulator copied to VGPRs at once)
__device__ __forceinline__ void pin_agpr_ordered(f32x4_t& acc) { asm volatile("" : "+a"(acc) : : "memory"); }
__device__ __forceinline__ void pin_agpr_ordered(f32x16_t& acc) { asm volatile("" : "+a"(acc) : : "memory"); }
// wait states between the last MFMA of the loop and the first read of its
// accumulators by ordinary code (the hazard check cannot see into asm)
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory"); }
#pragma clang diagnostic pop

// ---------------------------------------------------------------------------
// 8-bit checkpoints of g and u
// ---------------------------------------------------------------------------
// The 8 values a lane holds of a row's block of 32 columns (lanes l, l ^ 16,
// l ^ 32 and l ^ 48 hold the block): E4M3 codes of v * 2^-e, round to nearest
// even, with e the least exponent (at least -126) that brings the block's
// largest finite magnitude to at most 448, E4M3's largest.  A power of two, so
// scaling rounds nothing and each value is rounded once, by at most 2^-4 of
// itself above 2^-6 of the block's scale.  Infinities and NaN do not enter the
// scale and are stored as NaN.  Returns e + 127.
__device__ __forceinline__ uint32_t ckpt_encode(const float v[8], uint32_t code[2]) {
  float a = 0.f;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const float m = fabsf(v[r]);
    a = fmaxf(a, m < __builtin_inff() ? m : 0.f);
  }
  a = fmaxf(a, __shfl_xor(a, 16, 64));
  a = fmaxf(a, __shfl_xor(a, 32, 64));
  const uint32_t bits = __float_as_uint(a);
  const int e = max((int)(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
    code[h] = (uint32_t)w;
  }
  return (uint32_t)(e + 127);
}
// and back: code * 2^e, exact in fp32 but for subnormal results
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void ckpt_decode(const uint32_t code[2], uint32_t e127, float v[8]) {
  const float sc = __uint_as_float(e127 << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[h], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[h], true);
    v[4 * h] = lo[0] * sc;
    v[4 * h + 1] = lo[1] * sc;
    v[4 * h + 2] = hi[0] * sc;
    v[4 * h + 3] = hi[1] * sc;
  }
}

// The kernels of gemm_train.hip take GemmTrainParams: the checkpoint outputs,
// grouped products with a bias of their own per group, ragged weight gradients.
template <int OUT, bool GROUPED, int KM>
constexpr bool gemm_is_train() {
  return OUT == GEMM_OUT_GLU_SAVE || OUT == GEMM_OUT_DGLU_SAVED || (KM & (kKmajorRagged | kList | kSplitB | kTail)) != 0 ||
         (GROUPED && (OUT == GEMM_OUT_BF16 || OUT == GEMM_OUT_DACT));
}
template <int OUT, bool GROUPED, int KM>
using gemm_params_t =
    typename std::conditional<gemm_is_train<OUT, GROUPED, KM>(), GemmTrainParams, GemmParams>::type;

// ---------------------------------------------------------------------------
// Groups of the grouped and ragged products
// ---------------------------------------------------------------------------
// What a block knows about its groups, made from the caller's offsets at its
// start: offsets clamped into [0, R] and to a running maximum (a bad table gives
// wrong rows, never an access outside the buffers), the prefix of the groups'
// row tiles, and for ragged products the prefix of one tile's 64-k stages.  One
// wave scans 64 groups at a time (under 1 us for 64 groups); a table made once
// by a kernel of its own cost a launch (4.6 us), and searching it in memory a
// round trip per halving, per tile.
template <bool RAGGED>
struct GroupTables {
  int32_t off[kMaxGroups + 1];
  int32_t tile[RAGGED ? 1 : kMaxGroups + 1];
  int64_t work[RAGGED ? kMaxGroups + 1 : 1];
};
template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, int lane, Op op) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_up(v, d, 64);
    if (lane >= d) v = op(o, v);
  }
  return v;
}
// Called by every thread of the block.  bm: rows of a tile; split: parts of a
// ragged product's k range (a tile costs at least one stage for each).
template <bool RAGGED>
__device__ __forceinline__ void make_group_tables(GroupTables<RAGGED>& t, const int32_t* off, int groups, int32_t R, int bm,
                                                  int split) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int32_t end0 = min(max(off[0], 0), R);   // the previous 64 groups' end, tiles and stages
    int32_t tile0 = 0;
    int64_t work0 = 0;
    if (lane == 0) {
      t.off[0] = end0;
      t.tile[0] = 0;
      t.work[0] = 0;
    }
    for (int base = 0; base < groups; base += 64) {
      const int g = base + lane;
      const int32_t mine = g < groups ? min(max(off[g + 1], end0), R) : end0;
      const int32_t end = wave_scan(mine, lane, [](int32_t a, int32_t b) { return max(a, b); });
      int32_t begin = __shfl_up(end, 1, 64);
      if (lane == 0) begin = end0;
      const int32_t rows = end - begin;   // 0 past the last group
      if (g < groups) t.off[g + 1] = end;
      if constexpr (RAGGED) {
        const int64_t w = work0 + wave_scan((int64_t)max((rows + 63) / 64, split), lane, [](int64_t a, int64_t b) { return a + b; });
        if (g < groups) t.work[g + 1] = w;
        work0 = __shfl(w, 63, 64);
      } else {
        const int32_t n = tile0 + wave_scan((rows + bm - 1) / bm, lane, [](int32_t a, int32_t b) { return a + b; });
        if (g < groups) t.tile[g + 1] = n;
        tile0 = __shfl(n, 63, 64);
      }
      end0 = __shfl(end, 63, 64);
    }
  }
  __syncthreads();
}

// The blocks of a persistent grid of G on XCDs 0 .. x - 1 (block b is on XCD b mod 8).
__device__ __forceinline__ int blocks_before_xcd(int G, int x) {
  const int q = G / kNumXcd, r = G % kNumXcd;
  return x * q + min(x, r);
}
// kTail: how an XCD's n tiles of `stages` 64-k stages run on its nb blocks: whole
// rounds, then `rest` tiles in `parts` parts of the k range each, of kTailStages or
// more, one per block (1: the rest runs unsplit).
struct TailCut {
  int full, rest, parts;
};
__device__ __forceinline__ TailCut tail_cut(int n, int nb, int stages) {
  TailCut c;
  c.full = n / nb * nb;
  c.rest = n - c.full;
  c.parts = c.rest > 0 ? max(min(nb / c.rest, min(stages / kTailStages, kMaxTailParts)), 1) : 1;
  return c;
}

// GACT: the gate activation of a gated (GEMM_OUT_GEGLU, GEMM_OUT_DGLU) kernel,
// or the activation of a GEMM_OUT_DACT kernel, fixed per kernel so each
// carries one epilogue: with several epilogue copies behind a
// runtime switch, the register allocator copied accumulator lanes out of AGPRs
// inside the main loop, a few wait states after the (asm) MFMA that wrote them.
// M32: the wave tile runs on v_mfma_f32_32x32x16_bf16 (32x32 fragments, 16 k
// per MFMA) instead of v_mfma_f32_16x16x32_bf16: half the MFMA instructions
// and half the operand register reads per flop, the same LDS bytes.
// KM: bit 0 A, bit 1 B stored k-major, bit 2 a k range of its own for every
// group, bit 3 a list of products, bit 4 two padded right operands, bit 5 the last
// round's tiles split over K (GemmParams::kmajor).
template <int BM, int BN, int WAVES_M, int WAVES_N, int BK, int R, int OUT, bool GATHER, bool GROUPED,
          int GACT = ACT_NONE, bool M32 = false, int KM = 0>
__global__ void __launch_bounds__(WAVES_M * WAVES_N * 64)
gemm_bf16_kernel(gemm_params_t<OUT, GROUPED, KM> p) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int TM = BM / WAVES_M;   // wave tile rows (activation rows)
  constexpr int TN = BN / WAVES_N;   // wave tile width in B-tile rows
  constexpr int MR = M32 ? 32 : 16;  // rows (and columns) of one MFMA's output
  constexpr int KSTEP = M32 ? 16 : 32;   // k per MFMA
  typedef typename std::conditional<M32, f32x16_t, f32x4_t>::type acc_t;
  constexpr int NACC = M32 ? 16 : 4;     // accumulator registers per MFMA tile
  constexpr int FM = TM / MR;
  constexpr int FN = TN / MR;
  constexpr bool DUAL = (OUT == GEMM_OUT_GEGLU || OUT == GEMM_OUT_DGLU || OUT == GEMM_OUT_GLU_SAVE);
  constexpr int HALF = FN / 2;       // DUAL: gate fragments [0,HALF), up [HALF,FN)
  constexpr int CH = BK / 8;         // 16-byte chunks per LDS row
  constexpr int KS = BK / KSTEP;     // MFMA k-steps per stage
  constexpr int RPI = 64 / CH;       // rows filled by one 1 KB load instruction
  constexpr int A_INS = BM / (RPI * NW);   // load instructions per wave and stage
  constexpr int B_INS = BN / (RPI * NW);
  constexpr int LOADS = A_INS + B_INS;
  constexpr int SLOT = (BM + BN) * CH;     // 16-byte chunks per ring slot
  constexpr int OUT_N = DUAL ? BN / 2 : BN;   // output columns per block
  static_assert(BK == 32 || BK == 64, "stage depth");
  static_assert(A_INS >= 1 && B_INS >= 1 && BM % (RPI * NW) == 0 && BN % (RPI * NW) == 0, "load mapping");
  static_assert(!DUAL || (BN / 2) % (RPI * NW) == 0, "a load instruction stays in one weight set");
  static_assert(TM % MR == 0 && TN % MR == 0 && FM % 2 == 0, "wave tile");
  static_assert(M32 || (DUAL ? (HALF % 2 == 0) : (FN % 2 == 0)), "fragment pairs");
  static_assert(!DUAL || HALF >= 1, "gate and up fragments");
  static_assert(KS == 1 || KS % 2 == 0, "k-steps per stage");
  static_assert(R >= 2 && LOADS * (R - 2) < 64, "ring depth");
  constexpr bool KMA = (KM & 1) != 0, KMB = (KM & 2) != 0;
  constexpr bool RAGK = (KM & kKmajorRagged) != 0;
  constexpr bool TRAIN = gemm_is_train<OUT, GROUPED, KM>();
  static_assert(KM == 0 || (!DUAL && !GATHER && !M32 && BM % 128 == 0 && BN % 128 == 0 && BM <= 256 && BN <= 256 &&
                            BK == 64 && (TM == 32 || TM == 64 || TM == 128) && TN == 64),
                "k-major operands: tiles of 128 or 256 columns, wave tiles 64 wide, 16x16x32 MFMAs, one weight set");
  constexpr bool TAIL = (KM & kTail) != 0;
  static_assert(!GROUPED || (KM & ~kTail) == 0 || (KM & ~kTail) == 2, "grouped rows: only the weights k-major");
  static_assert(!TAIL || (GROUPED && (OUT == GEMM_OUT_BF16 || OUT == GEMM_OUT_DACT)), "split last round: grouped rows");
  static_assert(!RAGK || (KMA && KMB && !GROUPED), "ragged k ranges: both operands k-major");
  static_assert(!(OUT == GEMM_OUT_GLU_SAVE && M32) && kCkptBlock == 32, "a checkpoint block is one run of 4 lane groups");

  __shared__ u32x4_t ring[R * SLOT];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WAVES_N;
  const int wn = wave % WAVES_N;

  const int64_t K = p.K, N = p.N;
  const int Kc = (int)K;                       // < 2^22
  const int li = lane & (MR - 1);   // fragment row (weight) / column (activation)
  const int lg = lane / MR;         // k group: 8 consecutive k

  constexpr bool OWN_TABLES = RAGK || (GROUPED && TRAIN);
  __shared__ typename std::conditional<OWN_TABLES, GroupTables<RAGK>, int>::type tables;
  if constexpr (OWN_TABLES)
    make_group_tables(tables, p.group_off, p.groups, (int32_t)p.group_rows, BM, RAGK && p.ksplit > 1 ? p.ksplit : 1);

  // ---- this block's tiles ----------------------------------------------------
  // The grid is persistent (at most one block per CU).  Logical tiles (in
  // grouped order) are split into one contiguous range per XCD, in
  // proportion to its blocks, and the blocks of an XCD take its range
  // round-robin, so at any time the blocks sharing an L2 work on
  // neighbouring tiles.  Grouped mode counts only the tiles that exist.
  auto group_off = [&](int g) -> int { if constexpr (OWN_TABLES) return tables.off[g]; else return p.group_off[g]; };
  auto tile_off = [&](int g) -> int { if constexpr (OWN_TABLES) return tables.tile[g]; else return p.tile_off[g]; };
  const int tiles_m = GROUPED ? __builtin_amdgcn_readfirstlane(tile_off(p.groups)) : p.tiles_m;
  // split-K (fp32 output only): every tile appears KSP times, once per part
  // of the K range, each writing its own output copy
  constexpr bool SPLITK = OUT == GEMM_OUT_F32_SCALED;
  const int KSP = SPLITK && p.ksplit > 1 ? p.ksplit : 1;
  constexpr bool LIST = (KM & kList) != 0;   // products over the same k range, their tiles one after another
  static_assert(!LIST || (KMA && KMB && !SPLITK && !RAGK && OUT == GEMM_OUT_BF16), "list: dense k-major products, bf16");
  auto tiles_of = [&](int i) -> int {   // of product i
    if constexpr (LIST) return (int)(((p.list[i].M + BM - 1) / BM) * ((p.list[i].N + BN - 1) / BN));
    else return 0;
  };
  int total = (RAGK ? p.groups : 1) * tiles_m * p.tiles_n * KSP;
  if constexpr (LIST) {
    total = 0;
    for (int i = 0; i < p.products; ++i) total += tiles_of(i);
  }
  const int G = gridDim.x, bid = blockIdx.x;
  const int xcd = bid % kNumXcd, xj = bid / kNumXcd;
  auto blocks_before = [&](int x) { return blocks_before_xcd(G, x); };   // blocks on XCDs 0 .. x-1
  const int nbx = blocks_before(xcd + 1) - blocks_before(xcd);
  // Ragged k ranges: tiles cost what their group's k rows are, so the XCDs'
  // ranges are cut at equal stages instead of equal tiles (8 groups over 8
  // XCDs would otherwise give each XCD one group, the longest one last).
  auto range_end = [&](int x) -> int {   // the first logical tile past the ranges of XCDs 0 .. x - 1
    const int64_t nb = blocks_before(x);
    if constexpr (RAGK) {
      const int64_t tt = (int64_t)tiles_m * p.tiles_n;
      const int64_t w = tables.work[p.groups] * tt * nb / G;   // in stages
      int lo = 0, hi = p.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tables.work[mid] * tt <= w) lo = mid; else hi = mid;
      }
      const int64_t in = (w - tables.work[lo] * tt) * KSP / (tables.work[lo + 1] - tables.work[lo]);
      return (int)(lo * tt * KSP + in);
    } else {
      return (int)((int64_t)total * nb / G);
    }
  };
  const int t_lo = range_end(xcd);
  const int t_hi = range_end(xcd + 1);
  int nmine = xj < t_hi - t_lo ? (t_hi - t_lo - xj + nbx - 1) / nbx : 0;
  TailCut cut{0, 0, 1};
  if constexpr (TAIL) {
    cut = tail_cut(t_hi - t_lo, nbx, (Kc + BK - 1) / BK);
    nmine = cut.full / nbx + (xj < cut.rest * cut.parts ? 1 : 0);
  }
  if (nmine == 0) return;   // block-uniform: no barrier has been reached

  struct Tile {
    int64_t row_begin, row_end, n0;
    int kp;   // part of the K range (split-K)
    int parts;   // tail: of so many
    const uint16_t* b0;
    const uint16_t* b1;
    const uint16_t* bias;
    int64_t k_begin, c_off;   // ragged: the group's first k row, its output
    int kc;                   //   and its k rows
    int product;              // list: which
    int64_t rows, cols;       //   its size
    uint16_t* c;              //   and its output
  };
  auto tile_at = [&](int i) -> Tile {   // this block's i-th tile
    int tm, tn;
    int lt = t_lo + xj + i * nbx;
    const bool tail = TAIL && cut.parts > 1 && i * nbx == cut.full;
    if (tail) lt = t_lo + cut.full + xj / cut.parts;
    const int lg_t = RAGK ? lt / (tiles_m * p.tiles_n * KSP) : 0;   // ragged: the tile's group
    Tile t;
    t.product = 0;
    t.rows = p.M;
    t.cols = N;
    if constexpr (LIST) {
      int at = lt;
      while (t.product + 1 < p.products && at >= tiles_of(t.product)) at -= tiles_of(t.product++);
      t.rows = p.list[t.product].M;
      t.cols = p.list[t.product].N;
      t.c = p.list[t.product].C;
      grouped_tile(at, (int)((t.rows + BM - 1) / BM), (int)((t.cols + BN - 1) / BN), p.group_m, tm, tn);
    } else {
      grouped_tile((lt - lg_t * (tiles_m * p.tiles_n * KSP)) / KSP, tiles_m, p.tiles_n, p.group_m, tm, tn);
    }
    t.b0 = p.B0;
    t.b1 = p.B1;
    t.bias = p.bias;
    t.k_begin = 0;
    t.c_off = 0;
    t.kc = Kc;
    if constexpr (RAGK) {
      t.k_begin = group_off(lg_t);
      t.kc = group_off(lg_t + 1) - group_off(lg_t);
      t.c_off = (int64_t)lg_t * p.stride_c;
    }
    if constexpr (GROUPED) {
      int lo = 0, hi = p.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tile_off(mid) <= tm) lo = mid; else hi = mid;
      }
      t.row_begin = (int64_t)group_off(lo) + (int64_t)(tm - tile_off(lo)) * BM;
      t.row_end = min(t.row_begin + BM, (int64_t)group_off(lo + 1));
      t.b0 += (int64_t)lo * p.strideB;
      if constexpr (TRAIN) {
        if (p.bias) t.bias += (int64_t)lo * p.stride_bias;
      }
      if constexpr (DUAL) t.b1 += (int64_t)lo * p.strideB;
    } else {
      t.row_begin = (int64_t)tm * BM;
      t.row_end = min(t.row_begin + BM, LIST ? t.rows : p.M);
    }
    t.n0 = (int64_t)tn * OUT_N;
    t.kp = lt % KSP;
    t.parts = 1;
    if (tail) {
      t.kp = xj % cut.parts;
      t.parts = cut.parts;
    }
    return t;
  };

  // ---- load descriptors and per-lane offsets (of the tile being issued) -----
  // Load instruction i of this wave fills tile rows RPI * (i * NW + wave) +
  // lane / CH; the lane's LDS position in its row is lane % CH and it fetches
  // the chunk that belongs there.  RPI * NW is a multiple of 32 and the
  // swizzles read bits 1-4 of a row, so that chunk is the same for every load
  // instruction of the lane.  Byte spans fit 31 bits (checked by the caller),
  // so 32-bit offsets suffice and kOutOfRange is past every descriptor's end.
  // A tile's descriptors end at its last valid row, so rows past the end of
  // the activation or weight arrive as zeros with no per-lane test; gathered
  // rows past a group's end get an out-of-range offset once per tile.  Only
  // chunks past K need a mask per stage: they would read the next row.
  static_assert((RPI * NW) % 32 == 0, "one chunk permutation per lane");
  const int ra = RPI * wave + lane / CH;      // tile row of the lane's load 0 (activation and weight)
  const int a_k = 8 * ((lane % CH) ^ swz_a<CH>(ra));   // k of the lane's chunk in a stage
  const int b_k = 8 * ((lane % CH) ^ swz_b<CH>(ra));
  uint32_t lda2 = (uint32_t)p.lda * 2u;   // list: of the product being issued, as is ldb2
  const uint32_t K2 = (uint32_t)Kc * 2u;
  // offsets of the lane's load 0 within a tile (load i adds a constant number of rows)
  const uint32_t a_lane = (uint32_t)ra * lda2 + (uint32_t)a_k * 2u;
  const uint32_t b_lane = (uint32_t)ra * K2 + (uint32_t)b_k * 2u;
  // k-major: a row of the stage has CR = columns / 8 chunks and one instruction
  // fills 64 / CR of them (256 columns: 2 rows of 512 B); load i of this wave
  // fills k-rows KR i + (64 / CR) wave + lane / CR, the lane's slot lane % CR of
  // its row holding chunk slot ^ kswz(row) (kswz reads row bits 0-3, the same
  // for every i)
  constexpr int CRA = BM / 8, CRB = BN / 8;
  constexpr int KRA = 64 / CRA * NW, KRB = 64 / CRB * NW;   // k-rows between a wave's loads
  static_assert(KM == 0 || (KRA % 16 == 0 && KRB % 16 == 0), "one chunk permutation per lane");
  const int kra0 = 64 / CRA * wave + lane / CRA, krb0 = 64 / CRB * wave + lane / CRB;
  uint32_t ldb2 = (uint32_t)(KMB ? p.ldb : 0) * 2u;
  uint32_t a_lane_km = (uint32_t)kra0 * lda2 + (uint32_t)(((lane % CRA) ^ kswz(kra0)) * 16);
  uint32_t b_lane_km = (uint32_t)krb0 * ldb2 + (uint32_t)(((lane % CRB) ^ kswz(krb0)) * 16);
  i32x4_t da, db0, db1;
  uint32_t a_gat[GATHER ? A_INS : 1];   // gather: the lane's source-row offsets in this tile
  auto issue_tile = [&](const Tile& t) {
    const int a_rows_here = (int)(t.row_end - t.row_begin);
    if constexpr (LIST) {
      const GemmProduct& q = p.list[t.product];
      lda2 = (uint32_t)q.lda * 2u;
      ldb2 = (uint32_t)q.ldb * 2u;
      a_lane_km = (uint32_t)kra0 * lda2 + (uint32_t)(((lane % CRA) ^ kswz(kra0)) * 16);
      b_lane_km = (uint32_t)krb0 * ldb2 + (uint32_t)(((lane % CRB) ^ kswz(krb0)) * 16);
      da = make_desc(reinterpret_cast<uint64_t>(q.A + t.row_begin),
                     (uint32_t)((((int64_t)Kc - 1) * q.lda + q.M - t.row_begin) * 2));
      db0 = make_desc(reinterpret_cast<uint64_t>(q.B + t.n0), (uint32_t)((((int64_t)Kc - 1) * q.ldb + q.N - t.n0) * 2));
      db1 = db0;
      return;
    }
    // k-major descriptors end at the operand's last element ((K - 1) ld +
    // width): columns past the width read the next row's (in the operand, and
    // only into accumulators that are never stored), past the last row zeros
    if constexpr (KMA)   // the tile's rows are columns row_begin .. of A [K, lda], p.M wide
      da = make_desc(reinterpret_cast<uint64_t>(p.A + (RAGK ? t.k_begin * p.lda : 0) + t.row_begin),
                     RAGK && t.kc <= 0 ? 0u : (uint32_t)((((int64_t)t.kc - 1) * p.lda + p.M - t.row_begin) * 2));
    else
      da = GATHER ? make_desc(reinterpret_cast<uint64_t>(p.A), (uint32_t)(p.a_src_rows * p.lda * 2))
                  : make_desc(reinterpret_cast<uint64_t>(p.A + t.row_begin * p.lda), (uint32_t)a_rows_here * lda2);
    const int n_here = (int)min((int64_t)OUT_N, N - t.n0);   // weight rows of each set in this tile
    if constexpr (KMB) {   // the tile's columns are columns n0 .. of B0 [K0, ldb] (and B1 [K - K0, ldb]), N wide
      int64_t k0rows = p.kb_split > 0 ? p.kb_split : (int64_t)t.kc;
      if constexpr ((KM & kSplitB) != 0) k0rows = p.kb_rows;   // rows from there to the split load zeros
      db0 = make_desc(reinterpret_cast<uint64_t>(t.b0 + (RAGK ? t.k_begin * p.ldb : 0) + t.n0),
                      RAGK && t.kc <= 0 ? 0u : (uint32_t)(((k0rows - 1) * p.ldb + N - t.n0) * 2));
      if constexpr ((KM & kSplitB) != 0)
        db1 = make_desc(reinterpret_cast<uint64_t>(t.b1 + t.n0), (uint32_t)(((k0rows - 1) * p.ldb + N - t.n0) * 2));
      else
        db1 = p.kb_split > 0 ? make_desc(reinterpret_cast<uint64_t>(t.b1 + t.n0),
                                         (uint32_t)((((int64_t)Kc - p.kb_split - 1) * p.ldb + N - t.n0) * 2))
                             : db0;
    } else {
      db0 = make_desc(reinterpret_cast<uint64_t>(t.b0 + t.n0 * K), (uint32_t)n_here * K2);
      db1 = DUAL ? make_desc(reinterpret_cast<uint64_t>(t.b1 + t.n0 * K), (uint32_t)n_here * K2) : db0;
    }
    if constexpr (GATHER) {
      const int rt = RPI * wave + opaque(lane) / CH;
      const int ak = 8 * ((opaque(lane) % CH) ^ swz_a<CH>(rt));
#pragma unroll
      for (int i = 0; i < A_INS; ++i) {
        const int r = RPI * i * NW + rt;
        const uint32_t src = (uint32_t)p.a_rows[t.row_begin + min(r, a_rows_here - 1)];
        a_gat[i] = r < a_rows_here ? src * lda2 + (uint32_t)ak * 2u : kOutOfRange;
      }
    }
  };
  static_assert(RPI * NW <= BN / 2, "weight row of a load");
  const uint32_t ring_lds = lds_addr(&ring[0]) + (uint32_t)wave * 1024u;
  // Stages of one tile; the loop runs k-steps in pairs (the fragment register
  // sets alternate), so with one k-step per stage an odd count gets one
  // all-zero stage more, which adds nothing.  The block's stream is its
  // tiles' stages back to back: stream stage q is stage q % NS of tile q / NS.
  // Split over K: part kp of a tile takes stages [kp nk / KSP, (kp + 1) nk /
  // KSP) (shares that differ by at most one stage; with one k-step per stage
  // the caller keeps every share even).
  const int nk = (Kc + BK - 1) / BK;
  const int NS = KSP > 1 ? nk / KSP : (KS % 2 == 0 ? nk : (nk + 1) & ~1);   // stages of an unsplit tile
  auto part_first = [&](int kp) { return (int)((int64_t)kp * nk / KSP); };
  auto part_stages = [&](int kp) { return SPLITK ? part_first(kp + 1) - part_first(kp) : NS; };
  // Ragged: the stages of a tile's part are those of its group's k rows; a
  // part without any (an empty group, or fewer stages than parts) runs one
  // stage of zeros, so its output is written.
  auto rag_first = [&](const Tile& t, int kp) { return (int)((int64_t)kp * ((t.kc + BK - 1) / BK) / KSP); };
  auto tail_first = [&](const Tile& t, int kp) { return kp * nk / t.parts; };
  auto stages_of = [&](const Tile& t) -> int {
    if constexpr (TAIL) return tail_first(t, t.kp + 1) - tail_first(t, t.kp);
    else if constexpr (RAGK) return max(rag_first(t, t.kp + 1) - rag_first(t, t.kp), 1);
    else return part_stages(t.kp);
  };
  int iss_kp = 0;   // K part of the tile whose stages are being issued
  int iss_ns = NS;  // and its stage count
  int iss_kc = Kc;  // ragged: the k rows of its group (none for a part of zeros); ragged, tail: its first stage
  int iss_first = 0;
  auto iss_begin = [&](const Tile& t) {
    issue_tile(t);
    iss_kp = t.kp;
    iss_ns = stages_of(t);
    if constexpr (TAIL) iss_first = tail_first(t, t.kp);
    if constexpr (RAGK) {
      iss_first = rag_first(t, t.kp);
      iss_kc = rag_first(t, t.kp + 1) > iss_first ? t.kc : 0;
    }
  };
  iss_begin(tile_at(0));

  // How this wave loads the next stage of its stream (stages are issued once
  // each, in order): the lane's chunks are out of range past K (the k tail,
  // the padding stage) and for stages past the end of the stream; kb is the
  // byte offset of the stage's k range (the loads' soffset).  The first stage
  // of a tile switches the descriptors and offsets over to it.
  int iss_t = 0, iss_s = 0;   // tile and stage within the tile of the next stage issued
  struct StageIssue {
    bool a_in, b_in;
    uint32_t kb;      // soffset of the stage's k range: row-major operands
    uint32_t kb_a;    // A's (its rows past a k-major stage's first)
    uint32_t kb_b;    // B's
    int k0;           // the stage's first k (K when past the end)
    bool b1;          // k-major B: the stage's rows come from B1
    int kc;           // k rows past this one load zeros (k-major operands)
  };
  auto stage_begin = [&]() -> StageIssue {
    const bool live = iss_t < nmine;   // block-uniform
    if (live && iss_s == 0 && iss_t > 0) iss_begin(tile_at(iss_t));
    const int first = RAGK || TAIL ? iss_first : SPLITK ? part_first(iss_kp) : 0;
    const int ks0 = __builtin_amdgcn_readfirstlane(live ? first + iss_s : 0);   // stage index within K
    const int kc = RAGK ? iss_kc : Kc;
    const int k0 = live ? ks0 * BK : kc;
    const uint32_t kb = (uint32_t)ks0 * (BK * 2);
    const bool b1 = KMB && p.kb_split > 0 && k0 >= p.kb_split;   // block-uniform
    const StageIssue st{k0 + a_k < Kc, k0 + b_k < Kc, kb,
                        KMA ? (uint32_t)(ks0 * BK) * lda2 : kb,
                        KMB ? (uint32_t)(ks0 * BK - (b1 ? (int)p.kb_split : 0)) * ldb2 : kb, k0, b1, kc};
    if (++iss_s == iss_ns) {
      iss_s = 0;
      ++iss_t;
    }
    return st;
  };
  // load i (of LOADS) of a stage into the slot at LDS byte address `base`
  auto dma = [&](int i, uint32_t base, const StageIssue& st) {
    if (i < A_INS) {
      if constexpr (KMA) {   // k-rows past K load zeros
        const uint32_t off = a_lane_km + (uint32_t)(KRA * i) * lda2;
        asm_load_lds(da, base + (uint32_t)(i * NW) * 1024u, st.k0 + kra0 + KRA * i < (RAGK ? st.kc : Kc) ? off : kOutOfRange, st.kb_a);
      } else {
        const uint32_t off = GATHER ? a_gat[GATHER ? i : 0] : a_lane + (uint32_t)(RPI * i * NW) * lda2;
        asm_load_lds(da, base + (uint32_t)(i * NW) * 1024u, st.a_in ? off : kOutOfRange, st.kb_a);
      }
    } else {
      const int b = i - A_INS;
      if constexpr (KMB) {
        const uint32_t off = b_lane_km + (uint32_t)(KRB * b) * ldb2;
        asm_load_lds(st.b1 ? db1 : db0, base + (uint32_t)(BM * CH * 16 + b * NW * 1024),
                     st.k0 + krb0 + KRB * b < (RAGK ? st.kc : Kc) ? off : kOutOfRange, st.kb_b);
      } else {
        const bool up = DUAL && RPI * (b * NW) >= BN / 2;   // compile-time per i
        const uint32_t off = b_lane + (uint32_t)((RPI * b * NW) % (DUAL ? BN / 2 : BN)) * K2;
        asm_load_lds(up ? db1 : db0, base + (uint32_t)(BM * CH * 16 + b * NW * 1024),
                     st.b_in ? off : kOutOfRange, st.kb_b);
      }
    }
  };
  auto issue_all = [&](int slot) {
    const StageIssue st = stage_begin();
#pragma unroll
    for (int i = 0; i < LOADS; ++i) dma(i, ring_lds + (uint32_t)slot * (SLOT * 16), st);
  };
  // ---- LDS fragment addresses (16-byte units within a slot) -----------------
  // Activation fragment f: rows wm * TM + 16 f + li; weight fragment f: rows
  // w_lane_row + w_delta(f).  One base per k-step, the rest compile-time.
  static_assert(fragment_swizzle_is_uniform<CH, TM, TN, FM, FN, BN, WAVES_M, WAVES_N, DUAL, M32>(),
                "fragment addresses are affine");
  const int wr0 = w_lane_row(wn, li, TN, DUAL, M32);
  int x_idx[KS], w_idx[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int c = ks * (KSTEP / 8) + lg;
    x_idx[ks] = (wm * TM + li) * CH + (c ^ swz_a<CH>(wm * TM + li));
    w_idx[ks] = BM * CH + wr0 * CH + (c ^ swz_b<CH>(wr0));
  }

  acc_t acc[FM][FN];
  // The zeros are pinned into the accumulators here: the loop's MFMAs are
  // asm, so the hazard check cannot see them read a register that a plain
  // write set just before, and the compiler would otherwise sink each write
  // to right before its MFMA.
  auto zero_acc = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
#pragma unroll
        for (int r = 0; r < NACC; ++r) acc[i][j][r] = 0.f;
        pin_agpr(acc[i][j]);
      }
  };
  zero_acc();

  // Fragment registers: two sets, alternating by k-step.  Read n of a k-step
  // is x0, w0 .. w(FN-1), x1 .. x(FM-1): the order its MFMAs consume them.
  constexpr int NREADS = FM + FN;
  u32x4_t xf[2][FM], wf[2][FN];
  // k-major: the lane's byte offset in the operand's region for k-step 0,
  // half 0 (k-row 8 (lane / 16) + (lane % 16) / 4) and fragment 0.  The rest
  // are compile-time: k-step 1 is 32 rows on (the swizzle reads row bits 0-3:
  // only + 32 rows), half 1 is 4 rows on (row bit 2 set: swizzle bit 3 flips,
  // XOR 128, then + 4 rows), and a fragment XORs chunk bits the lane's own part
  // leaves zero (activation f: 2 f; weight f: 4 (f / 2), plus half chunk
  // f % 2).  One register per operand.
  uint32_t km_x = 0, km_w = 0;
  if constexpr (KM != 0) {
    const int kq = lane >> 4, s16 = lane & 15;
    const int row = 8 * kq + (s16 >> 2);
    km_x = (uint32_t)(row * (2 * BM) + (((wm * (TM / 8) + ((s16 & 3) >> 1)) ^ kswz(row)) << 4) + ((s16 & 1) << 3));
    km_w = (uint32_t)(BM * CH * 16 + row * (2 * BN) + (((wn * 8 + (s16 & 3)) ^ kswz(row)) << 4));
  }
  auto km_pair = [&](const u32x4_t* sl, uint32_t a0, uint32_t rowb, int ks, uint32_t half) -> u32x4_t {
    const uint32_t b = lds_addr(sl) + 32u * rowb * (uint32_t)ks + half;   // rowb: bytes of an LDS row
    return lds_read_tr_pair(b + a0, b + ((a0 ^ 128u) + 4u * rowb));
  };
  auto frag_x = [&](const u32x4_t* sl, int ks, int f) -> u32x4_t {
    if constexpr (KMA) {
      return km_pair(sl, km_x ^ (uint32_t)(32 * f), 2 * BM, ks, 0u);
    } else {
      return sl[x_idx[ks] + f * MR * CH];
    }
  };
  auto frag_w = [&](const u32x4_t* sl, int ks, int f) -> u32x4_t {
    if constexpr (KMB) {   // the pair permutation: columns 32 (f / 2) + 8 g + 4 (f % 2) .. + 3, g = 0..3
      return km_pair(sl, km_w ^ (uint32_t)(64 * (f >> 1)), 2 * BN, ks, (uint32_t)(8 * (f & 1)));
    } else {
      return sl[w_idx[ks] + w_delta(f, FN, BN, DUAL, M32) * CH];
    }
  };
  auto frag_read = [&](int n, const u32x4_t* sl, int ks, auto set_c) {
    constexpr int set = decltype(set_c)::value;
    if (n == 0) {
      xf[set][0] = frag_x(sl, ks, 0);
    } else if (n <= FN) {
      wf[set][n - 1] = frag_w(sl, ks, n - 1);
    } else {
      xf[set][n - FN] = frag_x(sl, ks, n - FN);
    }
  };
  auto mfma_t = [&](int t, auto set_c) {   // MFMA t of a k-step: row t / FN, column t % FN
    constexpr int set = decltype(set_c)::value;
    mfma_ordered(acc[t / FN][t % FN], wf[set][t % FN], xf[set][t / FN]);
  };
  using Set0 = std::integral_constant<int, 0>;
  using Set1 = std::integral_constant<int, 1>;

  // ---- epilogue of a finished tile ------------------------------------------
  // Global-address-space accesses: a store through a generic pointer is a flat
  // store, which would also hold lgkmcnt and stall the next tile's fragment
  // reads behind the write.
  typedef __attribute__((address_space(1))) u32x4_t gu32x4_t;
  auto gst16 = [](void* ptr, const u32x4_t& v) { *(gu32x4_t*)ptr = v; };
  auto gld16 = [](const void* ptr) -> u32x4_t { return *(const gu32x4_t*)ptr; };
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(1))) u32x2_t gu32x2_t;
  typedef __attribute__((address_space(1))) uint8_t gu8_t;
  auto gst8 = [](void* ptr, const uint32_t v[2]) { *(gu32x2_t*)ptr = u32x2_t{v[0], v[1]}; };
  auto gld8 = [](const void* ptr, uint32_t v[2]) {
    const u32x2_t r = *(const gu32x2_t*)ptr;
    v[0] = r[0];
    v[1] = r[1];
  };
  // Runs of 8 consecutive output columns a lane holds for activation fragment
  // i, RUNS per weight set (the weight-row permutation above makes them
  // consecutive):
  //   16x16x32: run q is accumulator pair (2q, 2q+1), 4 values each, columns
  //             32 q + 8 lg of the wave's columns;
  //   32x32x16: run q is registers 8 (q % 2) .. +7 of accumulator q / 2,
  //             columns 32 (q / 2) + 16 (q % 2) + 8 lg.
  constexpr int SETF = DUAL ? HALF : FN;   // fragments per weight set
  constexpr int RUNS = M32 ? 2 * SETF : SETF / 2;
  auto run_col = [](int q, int lgv) { return M32 ? (q >> 1) * 32 + 16 * (q & 1) + 8 * lgv : q * 32 + 8 * lgv; };
  auto run_vals = [&](int i, int q, int set, float v[8]) {   // set 0: gate (or the only set), 1: up
    if constexpr (M32) {
      const int f = set * HALF + (q >> 1);
      pin_agpr_ordered(acc[i][f]);
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = acc[i][f][8 * (q & 1) + r];
    } else {
      const int f0 = set * HALF + 2 * q;
      pin_agpr_ordered(acc[i][f0]);
      pin_agpr_ordered(acc[i][f0 + 1]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[r] = acc[i][f0][r];
        v[4 + r] = acc[i][f0 + 1][r];
      }
    }
  };
  // What the DGLU_SAVED and grouped DACT epilogues read beside the accumulator
  // (dy, or the checkpoint's codes and exponents), for one activation fragment:
  // requested a fragment ahead, since the accumulator reads are ordered after the
  // stores before them and a load left where it is used would wait out a round
  // trip per run.  (Worth 95 -> 94.5 us on the 2047 tokens of 2048 -> 5640.)
  struct Ahead {
    u32x4_t v[RUNS];     // dy; or g's codes (words 0, 1) and u's (2, 3)
    uint32_t e[RUNS];    // the exponents of g (low byte) and u
  };
  constexpr bool AHEAD = OUT == GEMM_OUT_DGLU_SAVED || (OUT == GEMM_OUT_DACT && TRAIN);
  auto ahead = [&](const Tile& t, int i, int li, int lg, Ahead& a) {
    if constexpr (AHEAD) {
      const int64_t lrow = t.row_begin + wm * TM + i * MR + li;
#pragma unroll
      for (int q = 0; q < RUNS; ++q) {
        const int64_t n = t.n0 + wn * TN + run_col(q, lg);
        if (!(lrow < t.row_end && n < N)) continue;
        if constexpr (OUT == GEMM_OUT_DACT) {
          a.v[q] = gld16(p.E + lrow * p.lde + n);
        } else {
          const int64_t nb = (N + kCkptBlock - 1) / kCkptBlock;
          const uint8_t* code = p.codes + lrow * 2 * N + n;
          const uint8_t* sc = p.qscale + lrow * 2 * nb + n / kCkptBlock;
          uint32_t c[4];
          gld8(code, c);
          gld8(code + N, c + 2);
          a.v[q] = u32x4_t{c[0], c[1], c[2], c[3]};
          a.e[q] = (uint32_t)*(const gu8_t*)sc | (uint32_t)*(const gu8_t*)(sc + nb) << 8;
        }
      }
    }
  };
  // The activation is a template argument so each copy of the epilogue is
  // straight-line code (a per-element switch would branch around every value).
  auto epilogue_act = [&](const Tile& t, auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
    const int el = opaque(lane);
    const int li = el & (MR - 1), lg = el / MR;
    Ahead now, next;
    ahead(t, 0, li, lg, next);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      now = next;
      if (i + 1 < FM) ahead(t, i + 1, li, lg, next);
      const int64_t lrow = t.row_begin + wm * TM + i * MR + li;
      const bool row_ok = lrow < t.row_end;
      if constexpr (OUT == GEMM_OUT_GEGLU) {
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
          const int64_t n = t.n0 + wn * (TN / 2) + run_col(q, lg);
          float g[8], u[8], v[8];
          run_vals(i, q, 0, g);
          run_vals(i, q, 1, u);
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = act_of<ACT>(g[r]) * u[r];
          if (row_ok && n < N) gst16(static_cast<uint16_t*>(p.C) + lrow * p.ldc + n, pack_bf16x8(v));
        }
      } else if constexpr (OUT == GEMM_OUT_GLU_SAVE) {
        // as GEMM_OUT_GEGLU, and g and u themselves in 8 bits.  Every lane
        // takes part in a block's maximum, so only the stores are masked;
        // columns past N are zeros (weight rows past the end) or, for a row
        // that holds one, not finite: neither enters a scale.
        const int64_t nb = (N + kCkptBlock - 1) / kCkptBlock;
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
          const int64_t n = t.n0 + wn * (TN / 2) + run_col(q, lg);
          float g[8], u[8], v[8];
          run_vals(i, q, 0, g);
          run_vals(i, q, 1, u);
          uint32_t cg[2], cu[2];
          const uint32_t eg = ckpt_encode(g, cg), eu = ckpt_encode(u, cu);
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = act_of<ACT>(g[r]) * u[r];
          if (row_ok && n < N) {
            gst16(static_cast<uint16_t*>(p.C) + lrow * p.ldc + n, pack_bf16x8(v));
            uint8_t* code = p.codes + lrow * 2 * N + n;
            gst8(code, cg);
            gst8(code + N, cu);
            if (lg == 0) {   // the block's first lane group: n is the block's first column
              uint8_t* sc = p.qscale + lrow * 2 * nb + n / kCkptBlock;
              *(gu8_t*)sc = (uint8_t)eg;
              *(gu8_t*)(sc + nb) = (uint8_t)eu;
            }
          }
        }
      } else if constexpr (OUT == GEMM_OUT_DGLU_SAVED) {
        // the accumulator is dm = dy Wd, in fp32; g and u as the forward kept them
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
          const int64_t n = t.n0 + wn * TN + run_col(q, lg);
          float dm[8];
          run_vals(i, q, 0, dm);
          const int64_t np = p.ldc2 >> 1;   // columns of dg, and of du: N rounded up to a stage of the product that reads them
          if (!(row_ok && n < np)) continue;
          uint16_t* d2 = static_cast<uint16_t*>(p.C2) + lrow * p.ldc2 + n;
          if (n >= N) {
            gst16(d2, zero4());
            gst16(d2 + np, zero4());
            continue;
          }
          const uint32_t cg[2] = {now.v[q][0], now.v[q][1]}, cu[2] = {now.v[q][2], now.v[q][3]};
          float g[8], u[8], m[8], dg[8], du[8];
          ckpt_decode(cg, now.e[q] & 255u, g);
          ckpt_decode(cu, now.e[q] >> 8, u);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            float a, da;
            act_and_grad<ACT>(g[r], a, da);
            m[r] = a * u[r];
            dg[r] = dm[r] * u[r] * da;
            du[r] = dm[r] * a;
          }
          gst16(static_cast<uint16_t*>(p.C) + lrow * p.ldc + n, pack_bf16x8(m));
          gst16(d2, pack_bf16x8(dg));
          gst16(d2 + np, pack_bf16x8(du));
        }
      } else if constexpr (OUT == GEMM_OUT_DGLU) {
        // recomputed g and u with the incoming dm: m for the down projection's
        // weight gradient, dg and du for the input and gate/up weight gradients
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
          const int64_t n = t.n0 + wn * (TN / 2) + run_col(q, lg);
          float g[8], u[8];
          run_vals(i, q, 0, g);
          run_vals(i, q, 1, u);
          if (!(row_ok && n < N)) continue;
          float dm[8];
          unpack_bf16x8(gld16(p.E + lrow * p.lde + n), dm);
          float m[8], dg[8], du[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            float a, da;
            act_and_grad<ACT>(g[r], a, da);
            m[r] = a * u[r];
            dg[r] = dm[r] * u[r] * da;
            du[r] = dm[r] * a;
          }
          gst16(static_cast<uint16_t*>(p.C) + lrow * p.ldc + n, pack_bf16x8(m));
          uint16_t* d2 = static_cast<uint16_t*>(p.C2) + lrow * p.ldc2 + n;
          gst16(d2, pack_bf16x8(dg));
          gst16(d2 + N, pack_bf16x8(du));
        }
      } else {
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
          const int64_t n = t.n0 + wn * TN + run_col(q, lg);
          float v[8];
          run_vals(i, q, 0, v);
          if (!(row_ok && n < (LIST ? t.cols : N))) continue;
          if constexpr (TAIL) {   // a part of a tail tile: its fp32 sum, for gemm_tail_kernel
            if (t.parts > 1) {
              float* dst = p.tail + (int64_t)bid * (BM * BN) + (lrow - t.row_begin) * BN + (n - t.n0);
              u32x4_t lo, hi;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                lo[r] = __float_as_uint(v[r]);
                hi[r] = __float_as_uint(v[4 + r]);
              }
              gst16(dst, lo);
              gst16(dst + 4, hi);
              continue;
            }
          }
          if constexpr (OUT == GEMM_OUT_F32_SCALED) {
            const float sc = p.row_scale ? p.row_scale[lrow] : 1.f;
            float* dst = static_cast<float*>(p.C) + (int64_t)t.kp * p.c_kstride + (RAGK ? t.c_off : 0) + lrow * p.ldc + n;
            u32x4_t lo, hi;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              lo[r] = __float_as_uint(v[r] * sc);
              hi[r] = __float_as_uint(v[4 + r] * sc);
            }
            gst16(dst, lo);
            gst16(dst + 4, hi);
          } else {
            if (p.bias) {
              float b[8];
              unpack_bf16x8(gld16((TRAIN ? t.bias : p.bias) + n), b);
#pragma unroll
              for (int r = 0; r < 8; ++r) v[r] += b[r];
            }
            if constexpr (OUT == GEMM_OUT_DACT) {
              // the recomputed pre-activation z: dz = dy * act'(z)
              float dy[8];
              unpack_bf16x8(TRAIN ? now.v[q] : gld16(p.E + lrow * p.lde + n), dy);
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                float a, da;
                act_and_grad<ACT>(v[r], a, da);
                v[r] = dy[r] * da;
              }
            } else {
#pragma unroll
              for (int r = 0; r < 8; ++r) v[r] = act_of<ACT>(v[r]);
            }
            if constexpr (LIST) {
              gst16(t.c + lrow * t.cols + n, pack_bf16x8(v));
            } else {
              gst16(static_cast<uint16_t*>(p.C) + (RAGK ? t.c_off : 0) + lrow * p.ldc + n, pack_bf16x8(v));
            }
          }
        }
      }
    }
  };
  auto epilogue = [&](const Tile& t) {
    mfma_drain();
    if constexpr (OUT == GEMM_OUT_GEGLU || OUT == GEMM_OUT_DGLU || OUT == GEMM_OUT_DACT ||
                  OUT == GEMM_OUT_GLU_SAVE || OUT == GEMM_OUT_DGLU_SAVED) {
      epilogue_act(t, std::integral_constant<int, GACT>{});   // the (gate's) activation
    } else if constexpr (OUT == GEMM_OUT_BF16) {
      if (p.act == ACT_GELU_ERF) epilogue_act(t, std::integral_constant<int, ACT_GELU_ERF>{});
      else if (p.act == ACT_GELU_TANH) epilogue_act(t, std::integral_constant<int, ACT_GELU_TANH>{});
      else if (p.act == ACT_RELU) epilogue_act(t, std::integral_constant<int, ACT_RELU>{});
      else if (p.act == ACT_SILU) epilogue_act(t, std::integral_constant<int, ACT_SILU>{});
      else epilogue_act(t, std::integral_constant<int, ACT_NONE>{});
    } else {
      epilogue_act(t, std::integral_constant<int, ACT_NONE>{});
    }
    zero_acc();
  };

  // Prologue: stages 0 .. R-2 in flight, stage 0 published, R-1 issued.
  // Every stage up to the last one read plus R - 1 is issued (past the end
  // they load nothing), so every wait below is the same.
#pragma unroll
  for (int q = 0; q < R - 1; ++q) issue_all(q);
  wait_vm<LOADS * (R - 2)>();
  lds_barrier();
  issue_all(R - 1);
#pragma unroll
  for (int n = 0; n < NREADS; ++n) frag_read(n, ring, 0, Set0{});

  // One k-step (ks of the stage q in slot `slot`), register set CUR.
  //  * Not the stage's last k-step: its MFMAs, each followed by at most one
  //    fragment read of the next k-step (same slot) into the other set.
  //  * The last one: the first half of its MFMAs; hand-off (wait for this
  //    wave's loads of stage q + 1, then a barrier: stage q + 1 is in LDS for
  //    every wave, and every wave has finished reading `slot`); the second
  //    half, each MFMA followed by at most one instruction of the hand-off
  //    stream: the loads of stage q + R into `slot` (the first LNOW of them;
  //    the rest lead the next stage's first k-step), then the fragment reads
  //    of stage q + 1 into the other set.  The matrix core never waits for a
  //    run of memory instructions.  At the end of a tile (LAST) the fragment
  //    reads wait until the epilogue has freed its registers.  After an
  //    epilogue (whose stores count in vmcnt) the hand-off waits for every
  //    access, so no wait count depends on how loads and stores retire
  //    relative to each other.
  //  * Issue priority falls as a wave moves through a stage: 2 from the
  //    hand-off barrier to the end of the hand-off window, 1 through the next
  //    stage's first k-step, 0 up to the next barrier.  Of the two waves on a
  //    SIMD, the one behind gets the issue slots first, and the pair reaches
  //    the next barrier closer together (measured: the 8192/28672 GeGLU at
  //    4096 tokens 3 % faster, the 768/3072 one 2 %; a fixed priority per
  //    wave gained nothing).
  constexpr int NMA = (FM / 2) * FN;          // MFMAs per half k-step
  constexpr int NPRE = NMA;                   // MFMAs of the last k-step before the hand-off
  constexpr int NPOST = 2 * NMA - NPRE;
  static_assert(NPRE >= 1 && NPOST >= 1, "hand-off inside the last k-step");
  // Loads of stage q + R issued in the hand-off window.  With two k-steps per
  // stage half of them go out during the next stage's first k-step instead:
  // every wave reaches the hand-off together, and eight loads each in a
  // quarter of a stage queue behind one another in the address unit (measured
  // 3-4 % faster on the large shapes; a quarter or none in the window is
  // slower again).
  constexpr int LNOW = KS >= 2 ? LOADS / 2 : LOADS;
  StageIssue pend_st{false, false, 0};
  uint32_t pend_base = 0;
  bool pend = false;   // block-uniform: the first stage has none
  bool stored = false;   // an epilogue has stored since the last hand-off
  auto next_slot = [&](int sl) { return sl + 1 == R ? 0 : sl + 1; };
  auto kstep = [&](auto ks_c, int slot, auto cur_c, auto last_c) {
    constexpr int ks = decltype(ks_c)::value;
    constexpr int CUR = decltype(cur_c)::value;
    constexpr bool LAST = decltype(last_c)::value;
    using Nxt = std::integral_constant<int, CUR ^ 1>;
    if constexpr (ks + 1 < KS) {
      const u32x4_t* sl = ring + slot * SLOT;
      // the stage's first k-step leads with the loads deferred from the
      // hand-off window, then every k-step reads the next one's fragments
      constexpr int DEF = ks == 0 ? LOADS - LNOW : 0;
      constexpr int OPS0 = NREADS + DEF;
#pragma unroll
      for (int t = 0; t < 2 * NMA; ++t) {
        mfma_t(t, cur_c);
#pragma unroll
        for (int n = t * OPS0 / (2 * NMA); n < (t + 1) * OPS0 / (2 * NMA); ++n) {
          if (n < DEF) {
            if (pend) dma(LNOW + n, pend_base, pend_st);
          }
          else frag_read(n - DEF, sl, ks + 1, Nxt{});
        }
      }
      if constexpr (ks == 0) __builtin_amdgcn_s_setprio(0);
      return;
    }
    const StageIssue st = stage_begin();   // stage q + R
#pragma unroll
    for (int t = 0; t < NPRE; ++t) mfma_t(t, cur_c);
    if (R > 2 && stored) wait_vm<0>(); else wait_vm<LOADS * (R - 2)>();
    stored = false;
    lds_barrier();
    __builtin_amdgcn_s_setprio(2);
    const uint32_t base = ring_lds + (uint32_t)slot * (SLOT * 16);
    const u32x4_t* sl = ring + next_slot(slot) * SLOT;
    constexpr int OPS = LAST ? LNOW : LNOW + NREADS;
#pragma unroll
    for (int t = 0; t < NPOST; ++t) {
      mfma_t(NPRE + t, cur_c);
#pragma unroll
      for (int n = t * OPS / NPOST; n < (t + 1) * OPS / NPOST; ++n) {
        if (n < LNOW) dma(n, base, st);
        else frag_read(n - LNOW, sl, 0, Nxt{});
      }
    }
    __builtin_amdgcn_s_setprio(1);
    pend_st = st;
    pend_base = base;
    pend = true;
  };
  using Mid = std::false_type;
  using Last = std::true_type;
  // the end of this block's tile ti (its last k-step done): epilogue, then the
  // first fragments of the next tile, from the next slot
  auto tile_end = [&](int ti, int slot) {
    epilogue(tile_at(ti));
    stored = true;
    const u32x4_t* sl = ring + next_slot(slot) * SLOT;
#pragma unroll
    for (int n = 0; n < NREADS; ++n) frag_read(n, sl, 0, Set0{});
  };
  // every k-step of one stage (KS even: the register sets alternate within it)
  auto stage = [&](int slot, auto last_c) {
    auto step = [&](auto self, auto k_c) {
      constexpr int K = decltype(k_c)::value;
      if constexpr (K < KS) {
        kstep(k_c, slot, std::integral_constant<int, K & 1>{},
              std::integral_constant<bool, decltype(last_c)::value && K + 1 == KS>{});
        self(self, std::integral_constant<int, K + 1>{});
      }
    };
    step(step, std::integral_constant<int, 0>{});
  };
  using K0 = std::integral_constant<int, 0>;
  int slot = 0;
  for (int ti = 0; ti < nmine; ++ti) {
    const int ns = SPLITK || RAGK || TAIL ? stages_of(tile_at(ti)) : NS;
    if constexpr (KS >= 2) {
      for (int q = 0; q < ns - 1; ++q) {
        stage(slot, Mid{});
        slot = next_slot(slot);
      }
      stage(slot, Last{});
    } else {
      for (int q = 0; q < ns - 2; q += 2) {   // ns is even
        kstep(K0{}, slot, Set0{}, Mid{});
        slot = next_slot(slot);
        kstep(K0{}, slot, Set1{}, Mid{});
        slot = next_slot(slot);
      }
      kstep(K0{}, slot, Set0{}, Mid{});
      slot = next_slot(slot);
      kstep(K0{}, slot, Set1{}, Last{});
    }
    tile_end(ti, slot);
    slot = next_slot(slot);
  }
  wait_vm<0>();   // the stages issued past the end (loads of nothing) land before LDS is released
}

// kTail's second launch, with the first one's grid: the block that made part kp of a
// split tile adds a share of the tile's rows over its parts, in their order, and
// applies the epilogue's bias and activation (or its derivative) and rounds once.
template <int BM, int BN, int OUT, int GACT>
__global__ void __launch_bounds__(512) gemm_tail_kernel(GemmTrainParams p) {
  __shared__ GroupTables<false> tables;
  make_group_tables(tables, p.group_off, p.groups, (int32_t)p.group_rows, BM, 1);
  const int G = gridDim.x, bid = blockIdx.x;
  const int xcd = bid % kNumXcd, xj = bid / kNumXcd;
  const int tiles_m = tables.tile[p.groups];
  const int64_t total = (int64_t)tiles_m * p.tiles_n;
  const int b0 = blocks_before_xcd(G, xcd), b1 = blocks_before_xcd(G, xcd + 1);
  const int t_lo = (int)(total * b0 / G), t_hi = (int)(total * b1 / G);
  const TailCut cut = tail_cut(t_hi - t_lo, b1 - b0, (int)((p.K + 63) / 64));
  if (cut.parts == 1 || xj >= cut.rest * cut.parts) return;
  int tm, tn;
  grouped_tile(t_lo + cut.full + xj / cut.parts, tiles_m, p.tiles_n, p.group_m, tm, tn);
  int lo = 0, hi = p.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tables.tile[mid] <= tm) lo = mid; else hi = mid;
  }
  const int64_t row0 = (int64_t)tables.off[lo] + (int64_t)(tm - tables.tile[lo]) * BM;
  const int rows = (int)min((int64_t)BM, tables.off[lo + 1] - row0);
  const int kp = xj % cut.parts, first = xj - kp;   // the tile's parts: blocks first .. of this XCD
  const int c = (threadIdx.x % (BN / 8)) * 8;
  const int64_t n = (int64_t)tn * BN + c;
  if (n >= p.N) return;   // N % 8 == 0
  const int end = min(rows, (kp + 1) * BM / cut.parts);
  float bias[8] = {};
  if (p.bias) unpack_bf16x8(ld16(p.bias + lo * p.stride_bias + n), bias);
  for (int r = kp * BM / cut.parts + threadIdx.x / (BN / 8); r < end; r += 512 / (BN / 8)) {
    float v[8] = {};
    for (int j = 0; j < cut.parts; ++j) {
      const float* src = p.tail + (int64_t)(xcd + kNumXcd * (first + j)) * (BM * BN) + r * BN + c;
      const u32x4_t a = ld16(src), b = ld16(src + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] += __uint_as_float(a[e]);
        v[4 + e] += __uint_as_float(b[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += bias[e];
    if constexpr (OUT == GEMM_OUT_DACT) {
      float dy[8];
      unpack_bf16x8(ld16(p.E + (row0 + r) * p.lde + n), dy);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a, da;
        act_and_grad<GACT>(v[e], a, da);
        v[e] = dy[e] * da;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = apply_act(v[e], p.act);
    }
    st16(static_cast<uint16_t*>(p.C) + (row0 + r) * p.ldc + n, pack_bf16x8(v));
  }
}

template <int BM, int BN, int WM, int WN, int BK, int R, int OUT, bool GATHER, bool GROUPED, int GACT,
          bool M32 = false, int KM = 0>
hipError_t launch_cfg(gemm_params_t<OUT, GROUPED, KM> p, hipStream_t s) {
  constexpr int OUT_N = (OUT == GEMM_OUT_GEGLU || OUT == GEMM_OUT_DGLU || OUT == GEMM_OUT_GLU_SAVE) ? BN / 2 : BN;
  if (!GROUPED) p.tiles_m = (int)((p.M + BM - 1) / BM);
  p.tiles_n = (int)((p.N + OUT_N - 1) / OUT_N);
  p.group_m = 4;
  int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * ((KM & kKmajorRagged) ? p.groups : 1) *   // grouped: an upper bound
                        ((OUT == GEMM_OUT_F32_SCALED && p.ksplit > 1) ? p.ksplit : 1);
  if constexpr ((KM & kList) != 0) {
    if (p.products < 1 || p.products > kMaxProducts) return hipErrorInvalidValue;
    tiles = 0;
    for (int i = 0; i < p.products; ++i) {
      const GemmProduct& q = p.list[i];
      if (std::max(q.lda, q.ldb) * p.K * 2 >= (int64_t(1) << 31) || q.lda < q.M || q.ldb < q.N) return hipErrorInvalidValue;
      tiles += ((q.M + BM - 1) / BM) * ((q.N + BN - 1) / BN);
    }
  }
  if (tiles <= 0) return hipSuccess;
  if (tiles > 0x7fffffff || p.cus <= 0) return hipErrorInvalidValue;
  // A 32-k stage tile consumes its stages two at a time, so it needs an even
  // stage count per tile; the parts of a split K range can be odd.
  if (OUT == GEMM_OUT_F32_SCALED && BK < 64 && p.ksplit > 1) return hipErrorInvalidValue;
  if (KM != p.kmajor) return hipErrorInvalidValue;
  if constexpr (KM != 0) {   // the byte spans of k-major operands fit the 31-bit offsets
    if ((KM & 1) && p.K * p.lda * 2 >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    if (KM & 2) {
      if (p.kb_split < 0 || p.kb_split >= p.K || p.kb_split % BK != 0) return hipErrorInvalidValue;
      if (p.kb_split > 0 && p.B1 == nullptr) return hipErrorInvalidValue;
      const int64_t rows = p.kb_split > 0 ? std::max(p.kb_split, p.K - p.kb_split) : p.K;
      if (rows * p.ldb * 2 >= (int64_t(1) << 31) || p.ldb < p.N) return hipErrorInvalidValue;
    }
  } else if (p.kb_split != 0) {
    return hipErrorInvalidValue;
  }
  // persistent: as many blocks as fit on the chip at once, each looping over
  // its tiles
  auto kernel = gemm_bf16_kernel<BM, BN, WM, WN, BK, R, OUT, GATHER, GROUPED, GACT, M32, KM>;
  static const int per_cu = [&] {
    int o = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&o, kernel, WM * WN * 64, 0) != hipSuccess) o = 1;
    return std::max(o, 1);
  }();
  const int64_t blocks = std::min<int64_t>(tiles * ((KM & kTail) ? kMaxTailParts : 1), (int64_t)p.cus * per_cu);
  if constexpr ((KM & kTail) != 0) {   // every block has a tile of `tail`
    static_assert(BK == 64, "64-k stages");
    if (p.tail == nullptr || blocks > kMaxTailBlocks) return hipErrorInvalidValue;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(WM * WN * 64), 0, s, p);
  if constexpr ((KM & kTail) != 0) {
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL((gemm_tail_kernel<BM, BN, OUT, GACT>), dim3((unsigned)blocks), dim3(512), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace

}  // namespace fmlp
