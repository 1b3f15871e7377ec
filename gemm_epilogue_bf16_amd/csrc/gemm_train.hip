// The GEMM forms of the grouped products and of the gated block with an 8-bit
// checkpoint: instantiations of gemm_kernel.h.
#include "gemm_kernel.h"

namespace fmlp {

namespace {

// one kernel per activation (see GACT in gemm_kernel.h)
template <class F>
hipError_t by_act(int act, F f) {
  switch (act) {
    case ACT_NONE: return f(std::integral_constant<int, ACT_NONE>{});
    case ACT_GELU_ERF: return f(std::integral_constant<int, ACT_GELU_ERF>{});
    case ACT_GELU_TANH: return f(std::integral_constant<int, ACT_GELU_TANH>{});
    case ACT_RELU: return f(std::integral_constant<int, ACT_RELU>{});
    case ACT_SILU: return f(std::integral_constant<int, ACT_SILU>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_gemm_grouped(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s) {
  if (p.groups < 1 || p.groups > kMaxGroups) return hipErrorInvalidValue;
  const bool big = tile == TILE_256x256;
  if (!big && tile != TILE_128x128) return hipErrorInvalidValue;
  if (out_kind == GEMM_OUT_BF16 && p.kmajor == 2) {
    if (p.bias != nullptr || p.act != ACT_NONE) return hipErrorInvalidValue;
    return big ? launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_BF16, false, true, ACT_NONE, false, 2>(p, s)
               : launch_cfg<128, 128, 4, 2, 64, 2, GEMM_OUT_BF16, false, true, ACT_NONE, false, 2>(p, s);
  }
  if (out_kind == GEMM_OUT_BF16 && p.kmajor == (2 | kTail) && big) {
    if (p.bias != nullptr || p.act != ACT_NONE) return hipErrorInvalidValue;
    return launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_BF16, false, true, ACT_NONE, false, 2 | kTail>(p, s);
  }
  if (p.kmajor == kTail && big) {
    if (out_kind == GEMM_OUT_BF16) return launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_BF16, false, true, ACT_NONE, false, kTail>(p, s);
    if (out_kind == GEMM_OUT_DACT)
      return by_act(p.act, [&](auto a) {
        return launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_DACT, false, true, a.value, false, kTail>(p, s);
      });
  }
  if (p.kmajor != 0) return hipErrorInvalidValue;
  if (out_kind == GEMM_OUT_BF16)
    return big ? launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_BF16, false, true, ACT_NONE>(p, s)
               : launch_cfg<128, 128, 4, 2, 64, 2, GEMM_OUT_BF16, false, true, ACT_NONE>(p, s);
  if (out_kind == GEMM_OUT_DACT)
    return by_act(p.act, [&](auto a) {
      return big ? launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_DACT, false, true, a.value>(p, s)
                 : launch_cfg<128, 128, 4, 2, 64, 2, GEMM_OUT_DACT, false, true, a.value>(p, s);
    });
  return hipErrorInvalidValue;
}

// 256x256 tiles, or 128x128 (two blocks a CU), both of 8 waves with 64-k stages.
// (128x128 tiles of 4 waves: a 1001-token step of the 768 -> 2056 block 118 us
// against 109; a ring of 4 stages, one block a CU, 3001 expert rows' gradients
// 124 against 109.)
template <int OUT, int KM, bool GROUPED = false>
static hipError_t launch_km(int tile, const gemm_params_t<OUT, GROUPED, KM>& p, hipStream_t s) {
  if (tile == TILE_256x256) return launch_cfg<256, 256, 2, 4, 64, 2, OUT, false, GROUPED, ACT_NONE, false, KM>(p, s);
  if (tile == TILE_128x128) return launch_cfg<128, 128, 4, 2, 64, 2, OUT, false, GROUPED, ACT_NONE, false, KM>(p, s);
  return hipErrorInvalidValue;
}

hipError_t launch_gemm_ragged(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s) {
  constexpr int KM = 3 | kKmajorRagged;
  if (p.kmajor != KM || p.groups < 1 || p.groups > kMaxGroups) return hipErrorInvalidValue;
  if (out_kind == GEMM_OUT_BF16 && p.ksplit <= 1 && p.act == ACT_NONE && p.bias == nullptr)
    return launch_km<GEMM_OUT_BF16, KM>(tile, p, s);
  if (out_kind == GEMM_OUT_F32_SCALED && p.row_scale == nullptr) return launch_km<GEMM_OUT_F32_SCALED, KM>(tile, p, s);
  return hipErrorInvalidValue;
}

hipError_t launch_gemm_kmajor(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s) {
  if (p.bias != nullptr || p.act != ACT_NONE || p.row_scale != nullptr) return hipErrorInvalidValue;
  if ((p.kmajor & kSplitB) && (p.kb_split <= 0 || p.K != 2 * p.kb_split || p.kb_rows < 1 || p.kb_rows > p.kb_split))
    return hipErrorInvalidValue;
  if (out_kind == GEMM_OUT_BF16 && p.ksplit <= 1) {
    if (p.kmajor == 0) return launch_km<GEMM_OUT_BF16, 0>(tile, p, s);
    if (p.kmajor == (2 | kSplitB)) return launch_km<GEMM_OUT_BF16, 2 | kSplitB>(tile, p, s);
    if (p.kmajor == 3) return launch_km<GEMM_OUT_BF16, 3>(tile, p, s);
    if (p.kmajor == (3 | kList)) return launch_km<GEMM_OUT_BF16, 3 | kList>(tile, p, s);
  }
  if (out_kind == GEMM_OUT_F32_SCALED) {
    if (p.kmajor == 0) return launch_km<GEMM_OUT_F32_SCALED, 0>(tile, p, s);
    if (p.kmajor == (2 | kSplitB)) return launch_km<GEMM_OUT_F32_SCALED, 2 | kSplitB>(tile, p, s);
    if (p.kmajor == 3) return launch_km<GEMM_OUT_F32_SCALED, 3>(tile, p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_gemm_ckpt(int out_kind, int tile, const GemmTrainParams& p, hipStream_t s) {
  const bool big = tile == TILE_256x256;
  if (!big && tile != TILE_128x128) return hipErrorInvalidValue;
  if (p.codes == nullptr || p.qscale == nullptr) return hipErrorInvalidValue;
  if (out_kind == GEMM_OUT_GLU_SAVE && p.kmajor == 0)
    return by_act(p.act, [&](auto a) {
      return big ? launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_GLU_SAVE, false, false, a.value>(p, s)
                 : launch_cfg<128, 128, 4, 2, 64, 2, GEMM_OUT_GLU_SAVE, false, false, a.value>(p, s);
    });
  if (out_kind == GEMM_OUT_DGLU_SAVED && p.kmajor == 2)
    return by_act(p.act, [&](auto a) {
      return big ? launch_cfg<256, 256, 2, 4, 64, 2, GEMM_OUT_DGLU_SAVED, false, false, a.value, false, 2>(p, s)
                 : launch_cfg<128, 128, 4, 2, 64, 2, GEMM_OUT_DGLU_SAVED, false, false, a.value, false, 2>(p, s);
    });
  if (out_kind == GEMM_OUT_DGLU_SAVED && p.kmajor == 0 && !big)   // weights past the k-major span, transposed
    return by_act(p.act, [&](auto a) {
      return launch_cfg<128, 128, 4, 2, 64, 2, GEMM_OUT_DGLU_SAVED, false, false, a.value>(p, s);
    });
  return hipErrorInvalidValue;
}

}  // namespace fmlp
