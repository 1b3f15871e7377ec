// What the C entry points share: argument checks and their error text, the
// device check, the plain GEMM calls and their tile choice.  Internal to the
// library, like kernels.h; not part of the public ABI.
#pragma once

#include "../../include/fmlp.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "kernels.h"

namespace fmlp {

constexpr int kPathAuto = 0, kPathDecode = 1, kPathGemm = 2, kPathSmall = 3, kPathFused = 4;
constexpr int64_t kDecodeMaxM = 16;
constexpr int64_t kSmallMaxDim = 128;
constexpr int64_t kMaxDim = int64_t(1) << 31;   // bound on a token count
constexpr int64_t kMaxInner = int64_t(1) << 22; // bound on an inner dimension: a 256-row
                                                // operand tile spans < 2^31 bytes
constexpr size_t kHeader = kWorkspaceHeaderBytes;  // barrier / error words

// fmlp_last_error's text, and the status to return
fmlp_status fail(fmlp_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fmlp_status ok();
// ok(), or the launch error as FMLP_E_HIP
fmlp_status launched(hipError_t e, const char* what);
// The current device is a gfx950 (probed once per device); its compute units.
fmlp_status check_device(int* cus_out = nullptr);

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE_PTR(p)                                                      \
  do {                                                                      \
    if ((p) == nullptr) return fail(FMLP_E_NULL, "%s is NULL", #p);         \
    if (!aligned16(p)) return fail(FMLP_E_ALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)

// Token-sized buffers (activations, outputs, routes) hold nothing when there
// are no tokens: NULL is then accepted, a misaligned pointer is still not.
#define TOKEN_PTR(p, rows)                                                  \
  do {                                                                      \
    if ((rows) > 0) REQUIRE_PTR(p);                                         \
    else if ((p) != nullptr && !aligned16(p))                               \
      return fail(FMLP_E_ALIGN, "%s is not 16-byte aligned", #p);           \
  } while (0)

#define OPTIONAL_PTR(p)                                                     \
  do {                                                                      \
    if ((p) != nullptr && !aligned16(p))                                    \
      return fail(FMLP_E_ALIGN, "%s is not 16-byte aligned", #p);           \
  } while (0)

#define SCALE_PTR(p)                                                        \
  do {                                                                      \
    if ((p) == nullptr) return fail(FMLP_E_NULL, "%s is NULL", #p);         \
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0)                         \
      return fail(FMLP_E_ALIGN, "%s is not 4-byte aligned", #p);            \
  } while (0)

inline fmlp_status check_rows(const char* name, int64_t v) {
  if (v < 0 || v >= kMaxDim) return fail(FMLP_E_SHAPE, "%s=%lld is out of range", name, (long long)v);
  return FMLP_OK;
}

inline fmlp_status check_inner(const char* name, int64_t v) {
  if (v <= 0 || v >= kMaxInner)
    return fail(FMLP_E_SHAPE, "%s=%lld must be in [8, 2^22)", name, (long long)v);
  if (v % 8 != 0) return fail(FMLP_E_ALIGN, "%s=%lld is not a multiple of 8", name, (long long)v);
  return FMLP_OK;
}

inline fmlp_status check_act(int act, const char* name = "act") {
  if (act != FMLP_ACT_NONE && act != FMLP_ACT_GELU_ERF && act != FMLP_ACT_GELU_TANH &&
      act != FMLP_ACT_RELU && act != FMLP_ACT_SILU)
    return fail(FMLP_E_ARG, "%s=%d is not an fmlp_act", name, act);
  return FMLP_OK;
}

#define TRY(expr)                              \
  do {                                         \
    fmlp_status s_ = (expr);                   \
    if (s_ != FMLP_OK) return s_;              \
  } while (0)

#define HIP_TRY(expr, what)                               \
  do {                                                    \
    hipError_t e_ = (expr);                               \
    if (e_ != hipSuccess) return launched(e_, what);      \
  } while (0)

inline fmlp_status check_workspace(void* workspace, size_t workspace_bytes, size_t need) {
  if (need == 0) return FMLP_OK;
  if (workspace == nullptr) return fail(FMLP_E_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
  if (!aligned16(workspace)) return fail(FMLP_E_ALIGN, "workspace is not 16-byte aligned");
  if (workspace_bytes < need) return fail(FMLP_E_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  return FMLP_OK;
}

// Token counts of a backward call bound the contraction over tokens, which the
// GEMM reads with 32-bit offsets like any inner dimension.
constexpr int64_t kBwdMaxTokens = kMaxInner;

inline size_t ws_bf16(int64_t rows, int64_t cols) { return round_up((size_t)rows * (size_t)cols * 2, 256); }
inline int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }

// ---- GEMM calls (abi.cpp) ---------------------------------------------------
GemmParams dense_params(const uint16_t* A, int64_t lda, const uint16_t* B0, const uint16_t* B1,
                        const uint16_t* bias, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                        int act, int cus);
int choose_tile(int64_t M, int64_t out_cols_per_256_tile_n, int cus);
int choose_tile_linear(int64_t M, int64_t N, int cus);
hipError_t gemm_linear(const uint16_t* x, const uint16_t* W, const uint16_t* b, int act, int64_t M,
                       int64_t K, int64_t N, uint16_t* y, int cus, hipStream_t s);
hipError_t gemm_glu_gateup(const uint16_t* x, const uint16_t* Wg, const uint16_t* Wu, int gate_act,
                           int64_t M, int64_t D, int64_t H, uint16_t* m, int cus, hipStream_t s);
int wgrad_split(int64_t R, int64_t T, int64_t Cc);
size_t wgrad_parts_bytes(int64_t R, int64_t T, int64_t Cc);
hipError_t gemm_wgrad(const uint16_t* A, const uint16_t* B, int64_t R, int64_t T, int64_t Cc, uint16_t* C,
                      float* parts, int cus, hipStream_t s);
bool gemm_bkmajor_ok(int64_t M, int64_t N, int64_t K, int64_t kb_split, int cus);
hipError_t gemm_bkmajor(const uint16_t* A, const uint16_t* B0, const uint16_t* B1, int64_t kb_split, int64_t M,
                        int64_t N, int64_t K, uint16_t* C, int cus, hipStream_t s);
bool wgrad_kmajor_ok(int64_t R, int64_t T, int64_t Cc, int64_t lda, int64_t ldb, int cus);
hipError_t gemm_wgrad_kmajor(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, int64_t R, int64_t T,
                             int64_t Cc, uint16_t* C, float* parts, int cus, hipStream_t s);
bool kmajor_fits(int64_t rows, int64_t ld);
size_t glu_products_scratch(int64_t M, int64_t D, int64_t H);
fmlp_status glu_bwd_products(const uint16_t* x, const uint16_t* dy, const uint16_t* Wg, const uint16_t* Wu,
                             const uint16_t* m, const uint16_t* dgdu, int64_t M, int64_t D, int64_t H, uint16_t* dx,
                             uint16_t* dWg, uint16_t* dWu, uint16_t* dWd, void* scratch, int cus, hipStream_t s);

}  // namespace fmlp
