// C entry points of the grouped products and of the gated block with an 8-bit
// checkpoint.  See include/fmlp.h for the contract.
#include <cstring>

#include "abi_calls.h"
#include "gemm_train.h"

using namespace fmlp;

namespace {

constexpr int64_t kMaxSpan = int64_t(1) << 30;   // elements of an operand read k-major: 2^31 bytes

fmlp_status check_groups(int32_t E) {
  if (E < 1 || E > kMaxGroups) return fail(FMLP_E_ARG, "E=%d must be in [1, %d]", E, kMaxGroups);
  return FMLP_OK;
}

GemmTrainParams train_params(const GemmParams& p) {
  GemmTrainParams t;
  std::memset(&t, 0, sizeof t);
  static_cast<GemmParams&>(t) = p;
  return t;
}

// ---- tile and split of a product ------------------------------------------------
// A product runs in rounds of one 256x256 tile per compute unit (of 256: the
// workspace is sized without a device) or two 128x128 ones, for as many 64-k
// stages as a tile has; splitting k in P parts makes more, shorter tiles, and
// costs the parts' fp32 round trip and a launch.  The estimate of a candidate in
// us, fitted to the k-major forms over ten shapes from 256x256x8192 to
// 14336x4096x4096 (2047x2048x11264: 98 us as 256 tiles in 4 parts, estimate 106;
// 201 unsplit, 106 as 128 tiles in 2 parts; 4112x768x1001: 17 us as 128 tiles,
// 29 as 256 tiles):
constexpr double kPartsLaunch = 5.0, kPartsBytesPerUs = 5.0e6;
// full rounds of 256 tiles, and a last one that runs faster the emptier it is
double rounds256(int64_t tiles, int64_t stages) {
  const int64_t full = tiles / 256, rest = tiles % 256;
  return (double)full * (1.45 * (double)stages + 10) + (rest ? (1.10 + 0.35 * (double)rest / 256) * (double)stages + 8 : 0);
}
// full rounds of 512 tiles, two to a compute unit; up to 256 have one each
double rounds128(int64_t tiles, int64_t stages) {
  const int64_t full = tiles / 512, rest = tiles % 512;
  return (double)full * ((double)stages + 4) + (rest == 0 ? 0 : (rest <= 256 ? 0.50 + 0.17 * (double)rest / 256 : 1.0) * (double)stages + 4);
}

struct ProductPlan {
  int tile, split;
  double us;
};
// tiles256, tiles128: the product's tiles of either size, `stages` of 64 k each;
// out: its output elements; max_split: 1 where k cannot be split.
ProductPlan plan_product(int64_t tiles256, int64_t tiles128, int64_t stages, int64_t out, int max_split) {
  ProductPlan best{TILE_256x256, 1, 0};
  for (int P = 1; P <= max_split; ++P) {
    if (P > 1 && stages / P < 4) break;
    const double parts = P > 1 ? kPartsLaunch + 8.0 * P * (double)out / kPartsBytesPerUs : 0;
    for (int tile : {TILE_256x256, TILE_128x128}) {
      const int64_t st = (stages + P - 1) / P;
      const double t = (tile == TILE_256x256 ? rounds256(tiles256 * P, st) : rounds128(tiles128 * P, st)) + parts;
      if (best.us == 0 || t < best.us) best = {tile, P, t};
    }
  }
  return best;
}
int64_t tiles_of(int64_t rows, int64_t cols, int t) { return ((rows + t - 1) / t) * ((cols + t - 1) / t); }
constexpr int kMaxSplit = 8;
ProductPlan plan_dense(int64_t rows, int64_t cols, int64_t K, int max_split = kMaxSplit) {
  return plan_product(tiles_of(rows, cols, 256), tiles_of(rows, cols, 128), (K + 63) / 64, rows * cols, max_split);
}
size_t parts_bytes(const ProductPlan& p, int64_t out) {
  return p.split > 1 ? round_up((size_t)p.split * (size_t)out * 4, 256) : 0;
}

// A product on its plan: C [M, N] = A . B with the operands of `kmajor`.
hipError_t run_product(const ProductPlan& plan, GemmTrainParams p, uint16_t* C, float* parts, hipStream_t s) {
  if (plan.split == 1) {
    p.C = C;
    return launch_gemm_kmajor(GEMM_OUT_BF16, plan.tile, p, s);
  }
  p.C = parts;
  p.ksplit = plan.split;
  p.c_kstride = p.M * p.N;
  const hipError_t e = launch_gemm_kmajor(GEMM_OUT_F32_SCALED, plan.tile, p, s);
  return e != hipSuccess ? e : launch_sum_parts(parts, plan.split, p.M * p.N, p.M * p.N, C, s);
}

// Tiles over E ragged groups' rows: the sizes are on the device, so the mean R / E
// stands for them, with half a tile wasted per group.
int64_t grouped_tiles(int64_t R, int64_t N, int32_t E, int t) { return (R / t + (E + 1) / 2) * ((N + t - 1) / t); }
bool grouped_big(int64_t R, int64_t N, int64_t K, int32_t E) {
  return plan_product(grouped_tiles(R, N, E, 256), grouped_tiles(R, N, E, 128), (K + 63) / 64, R * N, 1).tile == TILE_256x256;
}

// 256 tiles with the last round's split over a long contraction (kTail): one
// more launch and the parts' round trip, against up to three quarters of a round.
// Where the estimated tiles leave two or more blocks for each of that round's.
// (The three gradients, unsplit in brackets: 8192 rows in 8 groups through
// 4096 <- 14336, 2.25 rounds, 1848 us (1974); 4096 rows 1136 (1375); the forward of
// 210 rows, 8192 -> 992, 32 us (80), of 40 rows in 4 groups, 8192 -> 4096, 60 (114).)
constexpr int64_t kTailK = 1024;
bool grouped_tail(int64_t R, int64_t N, int64_t K, int32_t E) {
  const int64_t tiles = grouped_tiles(R, N, E, 256), rest = tiles % 256, stages = (K + 63) / 64;
  const int64_t P = rest > 0 ? std::min<int64_t>({256 / rest, stages / kTailStages, kMaxTailParts}) : 1;
  if (K < kTailK || P < 2) return false;
  const double t = rounds256(tiles - rest, stages) + kPartsLaunch + rounds256(rest * P, (stages + P - 1) / P) +
                   8.0 * (double)(P * rest * 256 * 256) / kPartsBytesPerUs;
  return t < std::min(rounds256(tiles, stages), rounds128(grouped_tiles(R, N, E, 128), stages));
}

// Tile of a grouped product over K, and whether its last round is split.
struct GroupedPlan {
  bool big, tail;
};
GroupedPlan plan_grouped(int64_t R, int64_t N, int64_t K, int32_t E) {
  const bool tail = grouped_tail(R, N, K, E);
  return {tail || grouped_big(R, N, K, E), tail};
}
hipError_t run_grouped(int out_kind, const GroupedPlan& plan, GemmTrainParams p, float* tail, hipStream_t s) {
  if (plan.tail && p.cus <= kMaxTailBlocks) {
    p.kmajor |= kTail;
    p.tail = tail;
  }
  return launch_gemm_grouped(out_kind, plan.big ? TILE_256x256 : TILE_128x128, p, s);
}

void set_groups(GemmTrainParams& p, const int32_t* group_off, int32_t E, int64_t R, bool big) {
  const int bm = big ? 256 : 128;
  p.group_off = group_off;
  p.groups = E;
  p.group_rows = R;
  p.tiles_m = (int)(R / bm + E);   // at most one partial tile per group
}

// The weight gradient of E groups: each its own rows, the mean stands for them.
ProductPlan plan_grouped_dw(int64_t R, int64_t N, int64_t K, int32_t E) {
  return plan_product(E * tiles_of(N, K, 256), E * tiles_of(N, K, 128), (R / E + 63) / 64, E * N * K, kMaxSplit);
}

struct GroupedBwdLayout {
  size_t dz, parts, total;
  ProductPlan dw;
  GroupedPlan dzp, dxp;
};
GroupedBwdLayout grouped_bwd_layout(int64_t R, int64_t K, int64_t N, int32_t E, int act) {
  GroupedBwdLayout L;
  L.dw = plan_grouped_dw(R, N, K, E);
  L.dzp = plan_grouped(R, N, K, E);
  L.dxp = plan_grouped(R, K, N, E);
  size_t o = kHeader;   // the decode header stays untouched
  L.dz = o;    o += act != FMLP_ACT_NONE ? ws_bf16(R, N) : 0;
  L.parts = o; o += std::max(parts_bytes(L.dw, E * N * K), L.dxp.tail || (act != FMLP_ACT_NONE && L.dzp.tail) ? kTailBytes : 0);   // of one product at a time
  L.total = o;
  return L;
}

}  // namespace

extern "C" {

size_t fmlp_grouped_linear_workspace_size(int64_t R, int64_t K, int64_t N, int32_t E) {
  if (R <= 0 || K <= 0 || N <= 0 || E < 1 || E > kMaxGroups) return 0;
  return plan_grouped(R, N, K, E).tail ? kHeader + kTailBytes : 0;
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
  if (const size_t need = fmlp_grouped_linear_workspace_size(R, K, N, E)) TRY(check_workspace(workspace, workspace_bytes, need));
  if (R == 0) return ok();
  int cus = 0;
  TRY(check_device(&cus));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const GroupedPlan plan = plan_grouped(R, N, K, E);
  GemmTrainParams p = train_params(dense_params(x, K, W, nullptr, b, y, N, R, N, K, act, cus));
  set_groups(p, group_off, E, R, plan.big);
  p.strideB = N * K;
  p.stride_bias = N;
  float* tail = plan.tail ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader) : nullptr;
  return launched(run_grouped(GEMM_OUT_BF16, plan, p, tail, s), "grouped_linear launch");
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
  float* parts = reinterpret_cast<float*>(ws + L.parts);
  const uint16_t* dz = dy;
  if (act != FMLP_ACT_NONE) {   // dz = dy * act'(x W^T + b), z recomputed
    uint16_t* dzw = reinterpret_cast<uint16_t*>(ws + L.dz);
    GemmTrainParams p = train_params(dense_params(x, K, W, nullptr, b, dzw, N, R, N, K, act, cus));
    set_groups(p, group_off, E, R, L.dzp.big);
    p.strideB = N * K;
    p.stride_bias = N;
    p.E = dy;
    p.lde = N;
    HIP_TRY(run_grouped(GEMM_OUT_DACT, L.dzp, p, parts, s), "grouped_linear_bwd dz launch");
    dz = dzw;
  }
  {   // dx = dz W[e]: the contraction runs over W's rows, read k-major
    GemmTrainParams p = train_params(dense_params(dz, N, W, nullptr, nullptr, dx, K, R, K, N, FMLP_ACT_NONE, cus));
    set_groups(p, group_off, E, R, L.dxp.big);
    p.strideB = N * K;
    p.kmajor = 2;
    p.ldb = K;
    HIP_TRY(run_grouped(GEMM_OUT_BF16, L.dxp, p, parts, s), "grouped_linear_bwd dx launch");
  }
  {   // dW[e] = dz^T x over the group's rows, both read k-major
    const bool split = L.dw.split > 1;
    GemmTrainParams p = train_params(dense_params(dz, N, x, nullptr, nullptr, split ? static_cast<void*>(parts) : dW, K, N,
                                                  K, R, FMLP_ACT_NONE, cus));
    p.kmajor = 3 | kKmajorRagged;
    p.ldb = K;
    p.group_off = group_off;
    p.groups = E;
    p.group_rows = R;
    p.stride_c = N * K;
    if (split) {
      p.ksplit = L.dw.split;
      p.c_kstride = E * N * K;
    }
    HIP_TRY(launch_gemm_ragged(split ? GEMM_OUT_F32_SCALED : GEMM_OUT_BF16, L.dw.tile, p, s), "grouped_linear_bwd dW launch");
    if (split) HIP_TRY(launch_sum_parts(parts, L.dw.split, E * N * K, E * N * K, dW, s), "grouped_linear_bwd dW sum");
  }
  if (db) HIP_TRY(launch_group_colsum(dz, group_off, R, E, N, db, s), "grouped_linear_bwd db launch");
  return ok();
}

// ---------------------------------------------------------------------------
// The gated block with an 8-bit checkpoint
// ---------------------------------------------------------------------------
size_t fmlp_glu_ckpt_workspace_size(int64_t M, int64_t D, int64_t H) {
  if (M < 0 || D <= 0 || H <= 0) return 0;
  return kHeader + ws_bf16(M, H) + parts_bytes(plan_dense(M, D, H), M * D);
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
  HIP_TRY(launch_gemm_ckpt(GEMM_OUT_GLU_SAVE, plan_dense(M, 2 * H, D, 1).tile, p, s), "glu_ckpt gate+up launch");
  p = train_params(dense_params(m, H, Wd, nullptr, nullptr, nullptr, D, M, D, H, FMLP_ACT_NONE, cus));
  float* parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader + ws_bf16(M, H));
  return launched(run_product(plan_dense(M, D, H), p, y, parts, s), "glu_ckpt down launch");
}

namespace {
// The products of the checkpoint's backward, all with operands as stored (read
// k-major): dm [M, H] over D, dx [M, D] over 2H, dWd [D, H], dWg and dWu [H, D] over
// the tokens.  The weight gradients run as one list of tiles in one launch where
// that saves rounds, else dWd and a list of dWg and dWu, or each by itself where few
// tiles over many tokens are better split.  `stored`: the spans fit (operands below 2^30 elements);
// else the transposing form of fmlp_glu_bwd's last steps.
// dg and du are Hp columns wide, H rounded up to the 64-k stages of dx's product,
// with zeros in between.
struct CkptBwdLayout {
  bool stored;
  int64_t Hp;
  ProductPlan dm, dx, dw3, dw2, dwd, dwgu;   // dw3: a list of all three gradients; dw2: of dWg and dWu
  int listed;                                 // 3, 2 (dWd by itself) or 0
  size_t m, dgdu, scratch, total;
};
CkptBwdLayout ckpt_bwd_layout(int64_t M, int64_t D, int64_t H) {
  CkptBwdLayout L;
  L.Hp = (H + 63) / 64 * 64;
  L.stored = D * L.Hp < kMaxSpan && M * D < kMaxSpan && 2 * M * L.Hp < kMaxSpan;
  if (!L.stored) L.Hp = H;
  L.dm = plan_dense(M, H, D, 1);   // its epilogue needs the whole sum
  L.dx = plan_dense(M, D, 2 * L.Hp);
  L.dwd = plan_dense(D, H, M);
  L.dwgu = plan_dense(H, D, M);
  L.dw2 = plan_product(2 * tiles_of(H, D, 256), 2 * tiles_of(H, D, 128), (M + 63) / 64, 2 * D * H, 1);
  L.dw3 = plan_product(tiles_of(D, H, 256) + 2 * tiles_of(H, D, 256), tiles_of(D, H, 128) + 2 * tiles_of(H, D, 128),
                       (M + 63) / 64, 3 * D * H, 1);
  // us of a launch's start and end.  A list's sizes and pointers change from tile to
  // tile, and the long one has all five operands in flight at once on different
  // XCDs and reads them more often: at 4096 tokens of 8192 -> 28672, where every
  // form has the same rounds, 9.06 ms as one list of three and 9.0 with a list of
  // two, 8.9 without; at 1001 tokens of 768 -> 2056 one list takes 98 us, two launches 109.
  constexpr double kLaunch = 3.0, kList2 = 1.02, kList3 = 1.1;
  const double one = 2 * L.dwgu.us + kLaunch, two = kList2 * L.dw2.us;
  L.listed = kList3 * L.dw3.us < L.dwd.us + kLaunch + std::min(one, two) ? 3 : two < one ? 2 : 0;
  size_t o = kHeader;
  L.m = o;       o += ws_bf16(M, H);
  L.dgdu = o;    o += ws_bf16(M, 2 * L.Hp);
  L.scratch = o;   // the parts of split products, one at a time, or the transposes
  o += L.stored ? std::max({parts_bytes(L.dx, M * D), L.listed == 3 ? 0 : parts_bytes(L.dwd, D * H),
                          L.listed ? 0 : parts_bytes(L.dwgu, H * D)})
                : std::max(ws_bf16(H, D), glu_products_scratch(M, D, H));
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
  p.ldc2 = 2 * L.Hp;
  p.codes = const_cast<fmlp_fp8*>(codes);
  p.qscale = const_cast<uint8_t*>(scales);
  if (!L.stored) {
    HIP_TRY(launch_transpose(Wd, D, H, H, scratch, D, D, s), "glu_ckpt_bwd transpose Wd");
    p.B0 = scratch;
    HIP_TRY(launch_gemm_ckpt(GEMM_OUT_DGLU_SAVED, TILE_128x128, p, s), "glu_ckpt_bwd dm launch");
    return glu_bwd_products(x, dy, Wg, Wu, m, dgdu, M, D, H, dx, dWg, dWu, dWd, scratch, cus, s);
  }
  p.kmajor = 2;
  p.ldb = H;
  HIP_TRY(launch_gemm_ckpt(GEMM_OUT_DGLU_SAVED, L.dm.tile, p, s), "glu_ckpt_bwd dm launch");
  float* parts = reinterpret_cast<float*>(scratch);
  // dx = [dg | du] [Wg ; Wu]: one product over 2 Hp
  GemmTrainParams q = train_params(dense_params(dgdu, 2 * L.Hp, Wg, Wu, nullptr, nullptr, D, M, D, 2 * L.Hp, FMLP_ACT_NONE, cus));
  q.kmajor = 2 | kSplitB;
  q.ldb = D;
  q.kb_split = L.Hp;
  q.kb_rows = H;
  HIP_TRY(run_product(L.dx, q, dx, parts, s), "glu_ckpt_bwd dx launch");
  const GemmProduct dw[3] = {{dy, m, dWd, D, H, D, H},
                             {dgdu, x, dWg, 2 * L.Hp, D, H, D},
                             {dgdu + L.Hp, x, dWu, 2 * L.Hp, D, H, D}};
  for (int i = 0; i < 3 - L.listed; ++i) {
    const GemmProduct& w = dw[i];
    q = train_params(dense_params(w.A, w.lda, w.B, nullptr, nullptr, nullptr, w.N, w.M, w.N, M, FMLP_ACT_NONE, cus));
    q.kmajor = 3;
    q.ldb = w.ldb;
    HIP_TRY(run_product(i == 0 ? L.dwd : L.dwgu, q, w.C, parts, s), "glu_ckpt_bwd weight gradient launch");
  }
  if (L.listed) {
    const GemmProduct& w = dw[3 - L.listed];
    q = train_params(dense_params(w.A, w.lda, w.B, nullptr, nullptr, nullptr, w.N, w.M, w.N, M, FMLP_ACT_NONE, cus));
    q.kmajor = 3 | kList;
    q.ldb = w.ldb;
    q.products = L.listed;
    std::copy(dw + 3 - L.listed, dw + 3, q.list);
    HIP_TRY(launch_gemm_kmajor(GEMM_OUT_BF16, L.listed == 3 ? L.dw3.tile : L.dw2.tile, q, s),
            "glu_ckpt_bwd weight gradients launch");
  }
  return ok();
}

}  // extern "C"
