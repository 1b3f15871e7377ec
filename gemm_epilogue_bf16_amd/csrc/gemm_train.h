// Launch interface of the GEMM forms behind the grouped products and the gated
// block with an 8-bit checkpoint (gemm_train.hip).  Internal to the library,
// like kernels.h; not part of the public ABI.
#pragma once

#include "kernels.h"

namespace fmlp {

// Output kinds beyond GemmOut.
constexpr int GEMM_OUT_GLU_SAVE = 5;     // GEMM_OUT_GEGLU that also writes g and u as E4M3 codes with block scales
constexpr int GEMM_OUT_DGLU_SAVED = 6;   // acc = dm; g and u come from those codes: C = m = act(g) * u,
                                         // C2 = [dm * u * act'(g) | dm * act(g)], each ldc2 / 2 columns
                                         // wide (N and zeros)

// Hidden units of one row that share a checkpoint scale.
constexpr int kCkptBlock = 32;

// GemmParams::kmajor bit 2: ragged weight gradient.  Both operands are k-major
// and every group has its own range of k rows, [group_off[g], group_off[g+1]):
// C[g] [M, N] = A[rows of g]^T . B[rows of g], zeros for a group without rows.
constexpr int kKmajorRagged = 4;
constexpr int kMaxGroups = 1024;

// bit 3: a list of products over the same k rows (K), each with operands, sizes and
// a bf16 output [M, N] of its own: weight gradients of one step in one launch.
constexpr int kList = 8;
constexpr int kMaxProducts = 3;
struct GemmProduct {
  const uint16_t *A, *B;   // k-major [K, lda] (the output's rows are columns of A), [K, ldb]
  uint16_t* C;             // row stride N
  int64_t lda, ldb, M, N;
};
// bit 4, with kb_split: B0 and B1 have kb_rows (at most kb_split) rows each, and
// the k rows from there to the split (or to K) are zeros.
constexpr int kSplitB = 16;

// bit 5: tiles left over after the last whole round of an XCD's blocks, where two or
// more blocks are there for each, are split over k; the parts go to `tail` in fp32
// (256 x 256 for each of kMaxTailBlocks blocks at most) and a second launch adds them.
constexpr int kTail = 32;
constexpr int kMaxTailParts = 32, kTailStages = 4, kMaxTailBlocks = 256;
constexpr size_t kTailBytes = (size_t)kMaxTailBlocks * 256 * 256 * 4;

struct GemmTrainParams : GemmParams {
  uint8_t* codes;              // checkpoint: E4M3 codes [rows, 2N], g in columns [0, N), u in [N, 2N)
  uint8_t* qscale;             // and scale exponents (+ 127) [rows, 2 ceil(N / kCkptBlock)]
  int64_t stride_bias;         // grouped: elements between consecutive groups' biases
  int products;                // kList
  GemmProduct list[kMaxProducts];
  int64_t kb_rows;             // kSplitB
  float* tail;                 // kTail
  int64_t stride_c;            // ragged: elements between consecutive groups' outputs
  int64_t group_rows;          // grouped, ragged: the rows there are; group_off is the caller's table, unchecked
};

// Every form below runs on TILE_128x128 or TILE_256x256.
// y = act(x W[g]^T + b[g]) over each group's rows (GEMM_OUT_BF16), its dz
// (GEMM_OUT_DACT), or dx = dz W[g] (GEMM_OUT_BF16 with kmajor = 2); on 256x256
// tiles also with kmajor | kTail.
hipError_t launch_gemm_grouped(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s);
// The ragged weight gradient (kmajor = 3 | kKmajorRagged), bf16 or split fp32.
hipError_t launch_gemm_ragged(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s);
// Dense products on either tile, bf16 or split fp32: kmajor = 0, 2 | kSplitB, 3 or
// 3 | kList (bf16 only).
hipError_t launch_gemm_kmajor(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s);
// GEMM_OUT_GLU_SAVE, and GEMM_OUT_DGLU_SAVED (kmajor 0 or 2).
hipError_t launch_gemm_ckpt(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s);

// ---------------------------------------------------------------------------
// Helpers of the grouped products (grouped.hip).
// ---------------------------------------------------------------------------
// db[e, n] = bf16(sum of dz[r, n] over group e's rows), fp32, a fixed order.
// group_off: the caller's table for R rows, unchecked.
hipError_t launch_group_colsum(const uint16_t* dz, const int32_t* group_off, int64_t R, int E, int64_t N, uint16_t* db,
                               hipStream_t s);

}  // namespace fmlp
