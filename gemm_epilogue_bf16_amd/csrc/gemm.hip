// The dense, gathered and grouped forms of the bf16 GEMM (gemm_kernel.h) behind
// launch_gemm: which output, tile and operand layout runs as which kernel.
// Forms of the training and grouped calls are in gemm_train.hip.
#include "gemm_kernel.h"

namespace fmlp {

namespace {

// The 256x256 tile's MFMA shape (see gemm_bf16_kernel's M32).  The 32x32x16
// form halves MFMA instructions and operand register reads, but was measured
// 6 % slower on the large GeGLU (4295-4300 us against 4055-4061 us for the
// 16x16x32 form, same sources and box); 16x16x32 stays the default and the
// 32x32x16 form is built only with -DFMLP_TILE256_M32=1.
#ifndef FMLP_TILE256_M32
#define FMLP_TILE256_M32 0
#endif
constexpr bool kTile256M32 = FMLP_TILE256_M32 != 0;


template <int OUT, bool GATHER, bool GROUPED, int GACT = ACT_NONE>
hipError_t launch_tile(int tile, const GemmParams& p, hipStream_t s) {
  if constexpr ((OUT == GEMM_OUT_GEGLU || OUT == GEMM_OUT_DGLU || OUT == GEMM_OUT_DACT) && GACT == ACT_NONE) {
    // one kernel per (gate) activation
    switch (p.act) {
      case ACT_GELU_TANH: return launch_tile<OUT, GATHER, GROUPED, ACT_GELU_TANH>(tile, p, s);
      case ACT_GELU_ERF: return launch_tile<OUT, GATHER, GROUPED, ACT_GELU_ERF>(tile, p, s);
      case ACT_RELU: return launch_tile<OUT, GATHER, GROUPED, ACT_RELU>(tile, p, s);
      case ACT_SILU: return launch_tile<OUT, GATHER, GROUPED, ACT_SILU>(tile, p, s);
      case ACT_NONE: break;
      default: return hipErrorInvalidValue;
    }
  }
  if constexpr ((OUT == GEMM_OUT_BF16 || OUT == GEMM_OUT_F32_SCALED) && !GATHER && !GROUPED) {
    if (p.kmajor != 0) {   // k-major operands: 256x256 tiles only
      if (tile != TILE_256x256) return hipErrorInvalidValue;
      switch (p.kmajor) {
        case 1: return launch_cfg<256, 256, 2, 4, 64, 2, OUT, false, false, GACT, false, 1>(p, s);
        case 2: return launch_cfg<256, 256, 2, 4, 64, 2, OUT, false, false, GACT, false, 2>(p, s);
        case 3: return launch_cfg<256, 256, 2, 4, 64, 2, OUT, false, false, GACT, false, 3>(p, s);
        default: return hipErrorInvalidValue;
      }
    }
  } else {
    if (p.kmajor != 0) return hipErrorInvalidValue;
  }
  switch (tile) {
    case TILE_128x128: return launch_cfg<128, 128, 2, 2, 32, 4, OUT, GATHER, GROUPED, GACT>(p, s);
    case TILE_256x256: return launch_cfg<256, 256, 2, 4, 64, 2, OUT, GATHER, GROUPED, GACT, kTile256M32>(p, s);
    case TILE_128x192:
      // 4 ring slots of 40 KB: all 160 KB of LDS.  These shapes run about one
      // tile per CU over a long K, bound by the bytes each CU has in flight
      // (the 768/3072 GeGLU's down GEMM: 1.5 % faster forward than 3 slots)
      if constexpr (OUT == GEMM_OUT_BF16 && !GATHER && !GROUPED)
        return launch_cfg<128, 192, 4, 2, 64, 4, OUT, GATHER, GROUPED, GACT>(p, s);
      else
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

int gemm_tile_bm(int tile) { return tile == TILE_256x256 ? 256 : 128; }
int gemm_tile_bn(int tile) { return tile == TILE_256x256 ? 256 : tile == TILE_128x192 ? 192 : 128; }

hipError_t launch_gemm(int out_kind, bool gather, bool grouped, int tile, GemmParams p,
                       hipStream_t s) {
  if (out_kind == GEMM_OUT_BF16 && !gather && !grouped) return launch_tile<GEMM_OUT_BF16, false, false>(tile, p, s);
  if (out_kind == GEMM_OUT_GEGLU && !gather && !grouped) return launch_tile<GEMM_OUT_GEGLU, false, false>(tile, p, s);
  if (out_kind == GEMM_OUT_GEGLU && gather && grouped) return launch_tile<GEMM_OUT_GEGLU, true, true>(tile, p, s);
  if (out_kind == GEMM_OUT_F32_SCALED && !gather && grouped) return launch_tile<GEMM_OUT_F32_SCALED, false, true>(tile, p, s);
  if (out_kind == GEMM_OUT_F32_SCALED && !gather && !grouped && tile == TILE_256x256)
    return launch_tile<GEMM_OUT_F32_SCALED, false, false>(tile, p, s);
  if (out_kind == GEMM_OUT_DACT && !gather && !grouped && tile != TILE_128x192)
    return launch_tile<GEMM_OUT_DACT, false, false>(tile, p, s);
  if (out_kind == GEMM_OUT_DGLU && !gather && !grouped) return launch_tile<GEMM_OUT_DGLU, false, false>(tile, p, s);
  return hipErrorInvalidValue;
}

}  // namespace fmlp
