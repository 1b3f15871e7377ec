// C entry points of decode with 4-bit weights.  See include/fmlp.h for the
// contract.
#include "abi_calls.h"
#include "decode_w4.h"

using namespace fmlp;

namespace {

fmlp_status check_w4(int64_t M, int group) {
  TRY(check_rows("M", M));
  if (M > kDecodeMaxM)
    return fail(FMLP_E_ARG, "4-bit-weight calls take M <= %lld tokens (M=%lld)", (long long)kDecodeMaxM, (long long)M);
  if (group != 32 && group != 64 && group != 128) return fail(FMLP_E_ARG, "group=%d is not 32, 64 or 128", group);
  return FMLP_OK;
}

fmlp_status check_w4_inner(const char* name, int64_t v, int group) {
  TRY(check_inner(name, v));
  if (v % group != 0) return fail(FMLP_E_ALIGN, "%s=%lld is not a multiple of the group size %d", name, (long long)v, group);
  return FMLP_OK;
}

// sizes that a workspace is computed for (1 <= M <= 16)
bool w4_sizes_ok(int64_t M, int64_t K, int group) {
  return M > 0 && M <= kDecodeMaxM && K > 0 && K < kMaxInner && (group == 32 || group == 64 || group == 128);
}

uint8_t* scratch_at(void* workspace, size_t off) {
  return workspace == nullptr ? nullptr : static_cast<uint8_t*>(workspace) + off;
}

}  // namespace

extern "C" {

size_t fmlp_linear_w4_workspace_size(int64_t M, int64_t K, int64_t N, int group) {
  if (!w4_sizes_ok(M, K, group) || N <= 0 || N >= kMaxInner) return 0;
  const size_t scratch = decode_w4_scratch_bytes(M, K, N, group, false);
  return scratch ? kHeader + scratch : 0;
}

fmlp_status fmlp_linear_w4(const fmlp_bf16* x, const uint8_t* Wq, const fmlp_bf16* scales, const fmlp_bf16* zeros,
                           const fmlp_bf16* b, int act, int64_t M, int64_t K, int64_t N, int group, fmlp_bf16* y,
                           void* workspace, size_t workspace_bytes, fmlp_stream stream) {
  TRY(check_w4(M, group));
  TRY(check_w4_inner("K", K, group));
  TRY(check_inner("N", N));
  TRY(check_act(act));
  TOKEN_PTR(x, M);
  REQUIRE_PTR(Wq);
  REQUIRE_PTR(scales);
  OPTIONAL_PTR(zeros);
  OPTIONAL_PTR(b);
  TOKEN_PTR(y, M);
  TRY(check_workspace(workspace, workspace_bytes, fmlp_linear_w4_workspace_size(M, K, N, group)));
  if (M == 0) return ok();
  int cus = 0;
  TRY(check_device(&cus));
  const W4Layer L{x, Wq, scales, zeros, nullptr, nullptr, nullptr, b, y, K, N, group, act, scratch_at(workspace, kHeader), nullptr};
  return launched(launch_decode_w4(L, (int)M, cus, static_cast<hipStream_t>(stream)), "linear (4-bit weights) launch");
}

size_t fmlp_glu_w4_workspace_size(int64_t M, int64_t D, int64_t H, int group) {
  if (!w4_sizes_ok(M, D, group) || !w4_sizes_ok(M, H, group)) return 0;
  return kHeader + ws_bf16(M, H) +
         std::max(decode_w4_scratch_bytes(M, D, H, group, true), decode_w4_scratch_bytes(M, H, D, group, false));
}

fmlp_status fmlp_glu_w4(const fmlp_bf16* x, const uint8_t* Wgq, const fmlp_bf16* sg, const fmlp_bf16* zg,
                        const uint8_t* Wuq, const fmlp_bf16* su, const fmlp_bf16* zu, const uint8_t* Wdq,
                        const fmlp_bf16* sd, const fmlp_bf16* zd, int gate_act, int64_t M, int64_t D, int64_t H,
                        int group, fmlp_bf16* y, void* workspace, size_t workspace_bytes, fmlp_stream stream) {
  TRY(check_w4(M, group));
  TRY(check_w4_inner("D", D, group));
  TRY(check_w4_inner("H", H, group));
  TRY(check_act(gate_act, "gate_act"));
  TOKEN_PTR(x, M);
  REQUIRE_PTR(Wgq);
  REQUIRE_PTR(sg);
  OPTIONAL_PTR(zg);
  REQUIRE_PTR(Wuq);
  REQUIRE_PTR(su);
  OPTIONAL_PTR(zu);
  REQUIRE_PTR(Wdq);
  REQUIRE_PTR(sd);
  OPTIONAL_PTR(zd);
  if ((zg == nullptr) != (zu == nullptr)) return fail(FMLP_E_ARG, "zg and zu must both be given or both be NULL");
  TOKEN_PTR(y, M);
  TRY(check_workspace(workspace, workspace_bytes, fmlp_glu_w4_workspace_size(M, D, H, group)));
  if (M == 0) return ok();
  int cus = 0;
  TRY(check_device(&cus));
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint16_t* m = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + kHeader);
  uint8_t* scratch = scratch_at(workspace, kHeader + ws_bf16(M, H));   // of the first layer, then of the second
  const W4Layer L1{x, Wgq, sg, zg, Wuq, su, zu, nullptr, m, D, H, group, gate_act, scratch, nullptr};
  const W4Layer L2{m, Wdq, sd, zd, nullptr, nullptr, nullptr, nullptr, y, H, D, group, FMLP_ACT_NONE, scratch, nullptr};
  HIP_TRY(launch_decode_w4(L1, (int)M, cus, s), "glu (4-bit weights) gate+up launch");
  return launched(launch_decode_w4(L2, (int)M, cus, s), "glu (4-bit weights) down launch");
}

}  // extern "C"
