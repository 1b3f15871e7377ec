// C entry points of the grouped products and of the gated block with an 8-bit
// checkpoint.  See include/fmlp.h for the contract.
#include <cstring>

#include "abi_calls.h"
#include "gemm_train.h"

using namespace fmlp;

namespace {

constexpr int kMaxGroups = 1024;
constexpr int64_t kMaxSpan = int64_t(1) << 30;   // elements of an operand read k-major: 2^31 bytes

fmlp_status check_groups(int32_t E) {
  if (E < 1 || E > kMaxGroups) return fail(FMLP_E_ARG, "E=%d must be in [1, %d]", E, kMaxGroups);
  return FMLP_OK;
}

struct PlanLayout {
  size_t group_off, tile_off, work_off, end;
};
PlanLayout plan_layout(int32_t E) {
  PlanLayout L;
  size_t o = kHeader;   // the decode header stays untouched
  L.group_off = o; o += round_up(((size_t)E + 1) * 4, 256);
  L.tile_off = o;  o += round_up(((size_t)E + 1) * 4, 256);
  L.work_off = o;  o += round_up(((size_t)E + 1) * 8, 256);
  L.end = o;
  return L;
}
GroupPlan plan_at(void* workspace, const PlanLayout& L) {
  char* ws = static_cast<char*>(workspace);
  return {reinterpret_cast<int32_t*>(ws + L.group_off), reinterpret_cast<int32_t*>(ws + L.tile_off),
          reinterpret_cast<int64_t*>(ws + L.work_off)};
}

GemmTrainParams train_params(const GemmParams& p) {
  GemmTrainParams t;
  std::memset(&t, 0, sizeof t);
  static_cast<GemmParams&>(t) = p;
  return t;
}

// Row tiles of a grouped product.  256 rows need groups that fill them (the
// rows are on the device: the mean of R / E stands for them) and enough tiles
// for the chip; else 128.
bool grouped_big(int64_t R, int64_t N, int32_t E, int cus) {
  const int64_t tiles = (R / 256 + E / 2) * ((N + 255) / 256);
  return R >= (int64_t)192 * E && tiles >= cus;
}

void set_groups(GemmTrainParams& p, const GroupPlan& plan, int32_t E, int64_t R, bool big) {
  const int bm = big ? 256 : 128;
  p.group_off = plan.group_off;
  p.tile_off = plan.tile_off;
  p.groups = E;
  p.tiles_m = (int)(R / bm + E);   // at most one partial tile per group
}

// Parts of the rows that a weight gradient is split in, as for the dense one:
// when all groups' tiles leave compute units idle.
int grouped_split(int64_t R, int64_t N, int64_t K, int32_t E) {
  const int64_t tiles = ((N + 255) / 256) * ((K + 255) / 256) * E;
  if (tiles >= 256) return 1;
  const int64_t P = std::min<int64_t>({256 / tiles, 8, R / E / 512});
  return P > 1 ? (int)P : 1;
}

struct GroupedBwdLayout {
  PlanLayout plan;
  size_t dz, parts, total;
  int split;
};
GroupedBwdLayout grouped_bwd_layout(int64_t R, int64_t K, int64_t N, int32_t E, int act) {
  GroupedBwdLayout L;
  L.plan = plan_layout(E);
  L.split = grouped_split(R, N, K, E);
  size_t o = L.plan.end;
  L.dz = o;    o += act != FMLP_ACT_NONE ? ws_bf16(R, N) : 0;
  L.parts = o; o += L.split > 1 ? round_up((size_t)L.split * (size_t)E * (size_t)N * (size_t)K * 4, 256) : 0;
  L.total = o;
  return L;
}

}  // namespace

extern "C" {

size_t fmlp_grouped_linear_workspace_size(int32_t E) {
  return E < 1 || E > kMaxGroups ? 0 : plan_layout(E).end;
}

fmlp_status fmlp_grouped_linear(const fmlp_bf16* x, const int32_t* group_off, const fmlp_bf16* W, const fmlp_bf16* b,
                                int act, int64_t R, int64_t K, int64_t N, int32_t E, fmlp_bf16* y, void* workspace,
                                size_t workspace_bytes, fmlp_stream stream) {
  TRY(check_rows("R", R));
  TRY(check_inner("K", K));
  TRY(check_inner("N", N));
  TRY(check_groups(E));
  TRY(check_act(act));
  TOKEN_PTR(x, R);
  SCALE_PTR(group_off);
  REQUIRE_PTR(W);
  OPTIONAL_PTR(b);
  TOKEN_PTR(y, R);
  const PlanLayout L = plan_layout(E);
  TRY(check_workspace(workspace, workspace_bytes, L.end));
  if (R == 0) return ok();
  int cus = 0;
  TRY(check_device(&cus));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const GroupPlan plan = plan_at(workspace, L);
  const bool big = grouped_big(R, N, E, cus);
  HIP_TRY(launch_group_plan(group_off, R, E, big ? 256 : 128, 1, plan, s), "grouped_linear plan launch");
  GemmTrainParams p = train_params(dense_params(x, K, W, nullptr, b, y, N, R, N, K, act, cus));
  set_groups(p, plan, E, R, big);
  p.strideB = N * K;
  p.stride_bias = N;
  return launched(launch_gemm_grouped(GEMM_OUT_BF16, big ? TILE_256x256 : TILE_128x128, p, s), "grouped_linear launch");
}

size_t fmlp_grouped_linear_bwd_workspace_size(int64_t R, int64_t K, int64_t N, int32_t E, int act) {
  if (R < 0 || K <= 0 || N <= 0 || E < 1 || E > kMaxGroups) return 0;
  return grouped_bwd_layout(R, K, N, E, act).total;
}

fmlp_status fmlp_grouped_linear_bwd(const fmlp_bf16* x, const int32_t* group_off, const fmlp_bf16* W,
                                    const fmlp_bf16* b, int act, const fmlp_bf16* dy, int64_t R, int64_t K, int64_t N,
                                    int32_t E, fmlp_bf16* dx, fmlp_bf16* dW, fmlp_bf16* db, void* workspace,
                                    size_t workspace_bytes, fmlp_stream stream) {
  TRY(check_rows("R", R));
  TRY(check_inner("K", K));
  TRY(check_inner("N", N));
  TRY(check_groups(E));
  TRY(check_act(act));
  if (R * K >= kMaxSpan || R * N >= kMaxSpan)
    return fail(FMLP_E_SHAPE, "R=%lld: R*K and R*N must be below 2^30 for the backward pass", (long long)R);
  if (N * K >= kMaxSpan)
    return fail(FMLP_E_SHAPE, "N*K=%lld must be below 2^30 for the backward pass", (long long)(N * K));
  TOKEN_PTR(x, R);
  SCALE_PTR(group_off);
  REQUIRE_PTR(W);
  OPTIONAL_PTR(b);
  TOKEN_PTR(dy, R);
  TOKEN_PTR(dx, R);
  REQUIRE_PTR(dW);
  OPTIONAL_PTR(db);
  const GroupedBwdLayout L = grouped_bwd_layout(R, K, N, E, act);
  TRY(check_workspace(workspace, workspace_bytes, L.total));
  int cus = 0;
  TRY(check_device(&cus));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (R == 0) {   // no rows: the weight and bias gradients are sums over nothing
    HIP_TRY(launch_fill_zero(dW, E * N * K, s), "grouped_linear_bwd zero dW");
    if (db) HIP_TRY(launch_fill_zero(db, E * N, s), "grouped_linear_bwd zero db");
    return ok();
  }
  char* ws = static_cast<char*>(workspace);
  const GroupPlan plan = plan_at(workspace, L.plan);
  // one plan serves dz and dx: both run on row tiles of the same height
  const bool big = grouped_big(R, K, E, cus);
  const int tile = big ? TILE_256x256 : TILE_128x128;
  HIP_TRY(launch_group_plan(group_off, R, E, big ? 256 : 128, L.split, plan, s), "grouped_linear_bwd plan launch");
  const uint16_t* dz = dy;
  if (act != FMLP_ACT_NONE) {   // dz = dy * act'(x W^T + b), z recomputed
    uint16_t* dzw = reinterpret_cast<uint16_t*>(ws + L.dz);
    GemmTrainParams p = train_params(dense_params(x, K, W, nullptr, b, dzw, N, R, N, K, act, cus));
    set_groups(p, plan, E, R, big);
    p.strideB = N * K;
    p.stride_bias = N;
    p.E = dy;
    p.lde = N;
    HIP_TRY(launch_gemm_grouped(GEMM_OUT_DACT, tile, p, s), "grouped_linear_bwd dz launch");
    dz = dzw;
  }
  {   // dx = dz W[e]: the contraction runs over W's rows, read k-major
    GemmTrainParams p = train_params(dense_params(dz, N, W, nullptr, nullptr, dx, K, R, K, N, FMLP_ACT_NONE, cus));
    set_groups(p, plan, E, R, big);
    p.strideB = N * K;
    p.kmajor = 2;
    p.ldb = K;
    HIP_TRY(launch_gemm_grouped(GEMM_OUT_BF16, tile, p, s), "grouped_linear_bwd dx launch");
  }
  {   // dW[e] = dz^T x over the group's rows, both read k-major
    float* parts = reinterpret_cast<float*>(ws + L.parts);
    const bool split = L.split > 1;
    GemmTrainParams p = train_params(dense_params(dz, N, x, nullptr, nullptr, split ? static_cast<void*>(parts) : dW, K, N,
                                                  K, R, FMLP_ACT_NONE, cus));
    p.kmajor = 3 | kKmajorRagged;
    p.ldb = K;
    p.group_off = plan.group_off;
    p.work_off = plan.work_off;
    p.groups = E;
    p.stride_c = N * K;
    if (split) {
      p.ksplit = L.split;
      p.c_kstride = E * N * K;
    }
    HIP_TRY(launch_gemm_ragged(split ? GEMM_OUT_F32_SCALED : GEMM_OUT_BF16, p, s), "grouped_linear_bwd dW launch");
    if (split) HIP_TRY(launch_sum_parts(parts, L.split, E * N * K, E * N * K, dW, s), "grouped_linear_bwd dW sum");
  }
  if (db) HIP_TRY(launch_group_colsum(dz, plan.group_off, E, N, db, s), "grouped_linear_bwd db launch");
  return ok();
}

// ---------------------------------------------------------------------------
// The gated block with an 8-bit checkpoint
// ---------------------------------------------------------------------------
size_t fmlp_glu_ckpt_workspace_size(int64_t M, int64_t D, int64_t H) {
  if (M < 0 || D <= 0 || H <= 0) return 0;
  return kHeader + ws_bf16(M, H);
}

size_t fmlp_glu_ckpt_codes_size(int64_t M, int64_t H) { return M < 0 || H <= 0 ? 0 : (size_t)M * (size_t)H * 2; }

size_t fmlp_glu_ckpt_scales_size(int64_t M, int64_t H) {
  return M < 0 || H <= 0 ? 0 : (size_t)M * (size_t)((H + kCkptBlock - 1) / kCkptBlock) * 2;
}

fmlp_status fmlp_glu_ckpt(const fmlp_bf16* x, const fmlp_bf16* Wg, const fmlp_bf16* Wu, const fmlp_bf16* Wd, int gate_act,
                          int64_t M, int64_t D, int64_t H, fmlp_bf16* y, fmlp_fp8* codes, uint8_t* scales,
                          void* workspace, size_t workspace_bytes, fmlp_stream stream) {
  TRY(check_rows("M", M));
  TRY(check_inner("D", D));
  TRY(check_inner("H", H));
  TRY(check_act(gate_act, "gate_act"));
  TOKEN_PTR(x, M);
  REQUIRE_PTR(Wg);
  REQUIRE_PTR(Wu);
  REQUIRE_PTR(Wd);
  TOKEN_PTR(y, M);
  TOKEN_PTR(codes, M);
  TOKEN_PTR(scales, M);
  TRY(check_workspace(workspace, workspace_bytes, fmlp_glu_ckpt_workspace_size(M, D, H)));
  if (M == 0) return ok();
  int cus = 0;
  TRY(check_device(&cus));
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint16_t* m = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + kHeader);
  GemmTrainParams p = train_params(dense_params(x, D, Wg, Wu, nullptr, m, H, M, H, D, gate_act, cus));
  p.codes = codes;
  p.qscale = scales;
  HIP_TRY(launch_gemm_ckpt(GEMM_OUT_GLU_SAVE, choose_tile(M, (H + 127) / 128, cus), p, s), "glu_ckpt gate+up launch");
  return launched(gemm_linear(m, Wd, nullptr, FMLP_ACT_NONE, M, H, D, y, cus, s), "glu_ckpt down launch");
}

namespace {
// m and [dg | du], then scratch that the steps use in turn: Wd^T for dm; the
// transposes of glu_bwd_products; the split weight gradients' parts.
struct CkptBwdLayout {
  size_t m, dgdu, scratch, total;
};
CkptBwdLayout ckpt_bwd_layout(int64_t M, int64_t D, int64_t H) {
  CkptBwdLayout L;
  size_t o = kHeader;
  L.m = o;       o += ws_bf16(M, H);
  L.dgdu = o;    o += ws_bf16(M, 2 * H);
  L.scratch = o; o += std::max(ws_bf16(H, D), glu_products_scratch(M, D, H));
  L.total = o;
  return L;
}
}  // namespace

size_t fmlp_glu_ckpt_bwd_workspace_size(int64_t M, int64_t D, int64_t H) {
  if (M < 0 || D <= 0 || H <= 0) return 0;
  return ckpt_bwd_layout(M, D, H).total;
}

fmlp_status fmlp_glu_ckpt_bwd(const fmlp_bf16* x, const fmlp_fp8* codes, const uint8_t* scales, const fmlp_bf16* Wg,
                              const fmlp_bf16* Wu, const fmlp_bf16* Wd, int gate_act, const fmlp_bf16* dy, int64_t M,
                              int64_t D, int64_t H, fmlp_bf16* dx, fmlp_bf16* dWg, fmlp_bf16* dWu, fmlp_bf16* dWd,
                              void* workspace, size_t workspace_bytes, fmlp_stream stream) {
  TRY(check_rows("M", M));
  if (M >= kBwdMaxTokens) return fail(FMLP_E_SHAPE, "M=%lld must be below 2^22 for the backward pass", (long long)M);
  TRY(check_inner("D", D));
  TRY(check_inner("H", H));
  if (2 * H >= kMaxInner) return fail(FMLP_E_SHAPE, "H=%lld: 2H must be below 2^22", (long long)H);
  TRY(check_act(gate_act, "gate_act"));
  TOKEN_PTR(x, M);
  TOKEN_PTR(codes, M);
  TOKEN_PTR(scales, M);
  REQUIRE_PTR(Wg);
  REQUIRE_PTR(Wu);
  REQUIRE_PTR(Wd);
  TOKEN_PTR(dy, M);
  TOKEN_PTR(dx, M);
  REQUIRE_PTR(dWg);
  REQUIRE_PTR(dWu);
  REQUIRE_PTR(dWd);
  const CkptBwdLayout L = ckpt_bwd_layout(M, D, H);
  TRY(check_workspace(workspace, workspace_bytes, L.total));
  int cus = 0;
  TRY(check_device(&cus));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (M == 0) {
    HIP_TRY(launch_fill_zero(dWg, H * D, s), "glu_ckpt_bwd zero dWg");
    HIP_TRY(launch_fill_zero(dWu, H * D, s), "glu_ckpt_bwd zero dWu");
    HIP_TRY(launch_fill_zero(dWd, D * H, s), "glu_ckpt_bwd zero dWd");
    return ok();
  }
  char* ws = static_cast<char*>(workspace);
  uint16_t* m = reinterpret_cast<uint16_t*>(ws + L.m);
  uint16_t* dgdu = reinterpret_cast<uint16_t*>(ws + L.dgdu);
  uint16_t* scratch = reinterpret_cast<uint16_t*>(ws + L.scratch);
  // dm = dy Wd with the derivative epilogue on the stored g and u: m and
  // [dg | du]; dm stays in registers.  The contraction runs over Wd's rows.
  GemmTrainParams p = train_params(dense_params(dy, D, Wd, nullptr, nullptr, m, H, M, H, D, gate_act, cus));
  p.C2 = dgdu;
  p.ldc2 = 2 * H;
  p.codes = const_cast<fmlp_fp8*>(codes);
  p.qscale = const_cast<uint8_t*>(scales);
  if (gemm_bkmajor_ok(M, H, D, 0, cus)) {
    p.kmajor = 2;
    p.ldb = H;
    HIP_TRY(launch_gemm_ckpt(GEMM_OUT_DGLU_SAVED, TILE_256x256, p, s), "glu_ckpt_bwd dm launch");
  } else {
    HIP_TRY(launch_transpose(Wd, D, H, H, scratch, D, D, s), "glu_ckpt_bwd transpose Wd");
    p.B0 = scratch;
    HIP_TRY(launch_gemm_ckpt(GEMM_OUT_DGLU_SAVED, TILE_128x128, p, s), "glu_ckpt_bwd dm launch");
  }
  return glu_bwd_products(x, dy, Wg, Wu, m, dgdu, M, D, H, dx, dWg, dWu, dWd, scratch, cus, s);
}

}  // extern "C"
