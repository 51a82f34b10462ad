// C entry points of the block operators: host-side validation, plan choice
// and launch.  As everywhere in the library, every check runs on the host
// before anything is enqueued.
#include <algorithm>

#include "../api_util.h"
#include "block.h"

using nvfp4::aligned;
using nvfp4::check_k;
using nvfp4::EpilogueLaunch;
using nvfp4::fail;
using nvfp4::GemmPlan;
using nvfp4::hip_status;
using nvfp4::ok;

namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Row stride of a [rows][cols] matrix: 0 stands for cols.
bool stride_ok(int64_t* ld, int64_t cols) {
  if (*ld == 0) *ld = cols;
  return *ld >= cols;
}

// Fewer than 2^24 tiles of 64 x 32 outputs (M N up to about 2^35): a launch has
// fewer than 2^32 threads.
bool sizes_ok(int64_t M, int64_t N) {
  const int64_t kMax = int64_t(1) << 36;
  return M <= kMax && N <= kMax && (M + 63) / 64 < (int64_t(1) << 24) / ((N + 31) / 32);
}

// The checks shared by the GEMM entry points; cols are the output columns and
// nb the rows of B.  Returns NVFP4_OK and *empty when there is nothing to do.
nvfp4_status check_gemm(const char* fn, const void* a, const void* a_sf, const void* b, const void* b_sf,
                        const float* alpha, const void* bias, int32_t act, int64_t M, int64_t cols, const char* cname,
                        int64_t K, bool* empty) {
  *empty = false;
  if (M < 0 || cols < 0)
    return fail(NVFP4_ERR_SHAPE, "%s: M = %lld, %s = %lld must be >= 0", fn, (long long)M, cname, (long long)cols);
  if (act < 0 || act > NVFP4_ACT_SILU) return fail(NVFP4_ERR_SHAPE, "%s: act = %d is not an nvfp4_activation", fn, act);
  const nvfp4_status s = check_k(K);
  if (s != NVFP4_OK) return s;
  if (M == 0 || cols == 0) {
    *empty = true;
    return ok();
  }
  if (!a || !a_sf || !b || !b_sf) return fail(NVFP4_ERR_NULL, "%s: a, a_sf, b and b_sf must not be NULL", fn);
  if (!aligned(a, 16) || !aligned(a_sf, 16) || !aligned(b, 16) || !aligned(b_sf, 16))
    return fail(NVFP4_ERR_ALIGN, "%s: a, a_sf, b and b_sf must be 16-byte aligned", fn);
  if (!aligned(alpha, 4) || !aligned(bias, 2))
    return fail(NVFP4_ERR_ALIGN, "%s: alpha must be 4-byte and bias 2-byte aligned", fn);
  if (!sizes_ok(M, cols))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: %lld x %lld outputs: fewer than 2^24 tiles of 64 x 32 are supported", fn, (long long)M, (long long)cols);
  return NVFP4_OK;
}

nvfp4_status check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (need == 0) return NVFP4_OK;
  if (!ws || have < need)
    return fail(NVFP4_ERR_WORKSPACE, "%s: the workspace must hold %zu bytes (%zu given)", fn, need, ws ? have : 0);
  if (!aligned(ws, 256)) return fail(NVFP4_ERR_ALIGN, "%s: the workspace must be 256-byte aligned", fn);
  return NVFP4_OK;
}

bool gemm_sizes(int64_t M, int64_t cols, int64_t K) {
  return M > 0 && cols > 0 && K > 0 && K % 256 == 0 && K <= (int64_t(1) << 22) && sizes_ok(M, cols);
}

EpilogueLaunch launch_of(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                         const float* alpha, const uint16_t* bias, int32_t act, int64_t M, int64_t nb, int64_t cols,
                         int64_t K, void* ws) {
  EpilogueLaunch p = {};
  p.g.a = a;
  p.g.a_sf = a_sf;
  p.g.b = b;
  p.g.b_sf = b_sf;
  p.g.alpha = alpha;
  p.g.ws = (float*)ws;
  p.g.M = M;
  p.g.N = nb;
  p.g.K = K;
  p.bias = bias;
  p.act = act;
  p.cols = cols;
  return p;
}

nvfp4_status check_residual(const char* fn, const uint16_t* residual, int64_t* ldr, const uint16_t* d, int64_t* ldd,
                            int64_t N) {
  if (!d) return fail(NVFP4_ERR_NULL, "%s: d must not be NULL", fn);
  if (!aligned(d, 2) || !aligned(residual, 2)) return fail(NVFP4_ERR_ALIGN, "%s: d and residual must be 2-byte aligned", fn);
  if (!stride_ok(ldd, N)) return fail(NVFP4_ERR_SHAPE, "%s: ldd = %lld is below N = %lld", fn, (long long)*ldd, (long long)N);
  if (!residual) *ldr = N;
  if (!stride_ok(ldr, N)) return fail(NVFP4_ERR_SHAPE, "%s: ldr = %lld is below N = %lld", fn, (long long)*ldr, (long long)N);
  return NVFP4_OK;
}

hipError_t run_epilogue(const GemmPlan& plan, EpilogueLaunch p, const uint16_t* residual, int64_t ldr, float beta,
                        uint16_t* d, int64_t ldd, hipStream_t stream) {
  p.res = residual;
  p.ldr = ldr;
  p.beta = beta;
  p.g.d = d;
  p.ldd = ldd;
  return nvfp4::launch_gemm_epilogue(plan, p, stream);
}

}  // namespace

size_t nvfp4_gemm_epilogue_workspace_size(int64_t M, int64_t N, int64_t K) {
  return gemm_sizes(M, N, K) ? nvfp4::choose_epilogue_plan(M, N, K).workspace : 0;
}

const char* nvfp4_gemm_epilogue_plan(int64_t M, int64_t N, int64_t K) {
  return gemm_sizes(M, N, K) ? nvfp4::choose_epilogue_plan(M, N, K).name : "none";
}

nvfp4_status nvfp4_gemm_epilogue(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                                 const float* alpha, const uint16_t* bias, int32_t act, const uint16_t* residual,
                                 int64_t ldr, float beta, uint16_t* d, int64_t ldd, int64_t M, int64_t N, int64_t K,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "nvfp4_gemm_epilogue";
  bool empty;
  nvfp4_status s = check_gemm(fn, a, a_sf, b, b_sf, alpha, bias, act, M, N, "N", K, &empty);
  if (s != NVFP4_OK || empty) return s;
  if ((s = check_residual(fn, residual, &ldr, d, &ldd, N)) != NVFP4_OK) return s;
  const GemmPlan plan = nvfp4::choose_epilogue_plan(M, N, K);
  if ((s = check_workspace(fn, workspace, workspace_bytes, plan.workspace)) != NVFP4_OK) return s;
  const EpilogueLaunch p = launch_of(a, a_sf, b, b_sf, alpha, bias, act, M, N, N, K, workspace);
  return hip_status(run_epilogue(plan, p, residual, ldr, beta, d, ldd, (hipStream_t)stream), fn);
}

size_t nvfp4_gemm_gated_workspace_size(int64_t M, int64_t I, int64_t K) {
  if (!gemm_sizes(M, I, K)) return 0;
  return std::max(nvfp4::choose_gated_plan(M, I, K, false).workspace, nvfp4::choose_gated_plan(M, I, K, true).workspace);
}

const char* nvfp4_gemm_gated_plan(int64_t M, int64_t I, int64_t K) {
  return gemm_sizes(M, I, K) ? nvfp4::choose_gated_plan(M, I, K, false).name : "none";
}

nvfp4_status nvfp4_gemm_gated(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                              const float* alpha, const uint16_t* bias, int32_t act, uint16_t* h, int64_t ldh,
                              int64_t M, int64_t I, int64_t K, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const char* fn = "nvfp4_gemm_gated";
  bool empty;
  nvfp4_status s = check_gemm(fn, a, a_sf, b, b_sf, alpha, bias, act, M, I, "I", K, &empty);
  if (s != NVFP4_OK || empty) return s;
  if (!h) return fail(NVFP4_ERR_NULL, "%s: h must not be NULL", fn);
  if (!aligned(h, 2)) return fail(NVFP4_ERR_ALIGN, "%s: h must be 2-byte aligned", fn);
  if (!stride_ok(&ldh, I)) return fail(NVFP4_ERR_SHAPE, "%s: ldh = %lld is below I = %lld", fn, (long long)ldh, (long long)I);
  const GemmPlan plan = nvfp4::choose_gated_plan(M, I, K, false);
  if ((s = check_workspace(fn, workspace, workspace_bytes, plan.workspace)) != NVFP4_OK) return s;
  EpilogueLaunch p = launch_of(a, a_sf, b, b_sf, alpha, bias, act, M, 2 * I, I, K, workspace);
  p.g.d = h;
  p.ldd = ldh;
  return hip_status(nvfp4::launch_gemm_gated(plan, p, false, (hipStream_t)stream), fn);
}

nvfp4_status nvfp4_gemm_gated_quantize(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                                       const float* alpha, const uint16_t* bias, int32_t act, const float* gs,
                                       uint8_t* q, uint8_t* sf, int64_t M, int64_t I, int64_t K, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const char* fn = "nvfp4_gemm_gated_quantize";
  if (I % 16 != 0) return fail(NVFP4_ERR_SHAPE, "%s: I = %lld is not a multiple of the block size 16", fn, (long long)I);
  bool empty;
  nvfp4_status s = check_gemm(fn, a, a_sf, b, b_sf, alpha, bias, act, M, I, "I", K, &empty);
  if (s != NVFP4_OK || empty) return s;
  if (!q || !sf) return fail(NVFP4_ERR_NULL, "%s: q and sf must not be NULL", fn);
  if (!aligned(q, 8) || !aligned(gs, 4)) return fail(NVFP4_ERR_ALIGN, "%s: q must be 8-byte and gs 4-byte aligned", fn);
  const GemmPlan plan = nvfp4::choose_gated_plan(M, I, K, true);
  if ((s = check_workspace(fn, workspace, workspace_bytes, plan.workspace)) != NVFP4_OK) return s;
  EpilogueLaunch p = launch_of(a, a_sf, b, b_sf, alpha, bias, act, M, 2 * I, I, K, workspace);
  p.gs = gs;
  p.q = q;
  p.sf = sf;
  return hip_status(nvfp4::launch_gemm_gated(plan, p, true, (hipStream_t)stream), fn);
}

namespace {

// Workspace of nvfp4_ffn: the two GEMMs' split-K area (always its counters'
// block, so that no hidden layer ever lies on counters), then the hidden
// layer's codes and scales.
struct FfnSpace {
  GemmPlan gated, down;
  size_t codes, scales, bytes;
};

FfnSpace ffn_space(int64_t M, int64_t H, int64_t I) {
  FfnSpace f;
  f.gated = nvfp4::choose_gated_plan(M, I, H, true);
  f.down = nvfp4::choose_epilogue_plan(M, H, I);
  size_t split = 4096;
  if (f.gated.workspace > split) split = f.gated.workspace;
  if (f.down.workspace > split) split = f.down.workspace;
  f.codes = align256(split);
  f.scales = f.codes + align256((size_t)M * (size_t)(I / 2));
  f.bytes = f.scales + align256((size_t)M * (size_t)(I / 16));
  return f;
}

}  // namespace

size_t nvfp4_ffn_workspace_size(int64_t M, int64_t H, int64_t I) {
  if (!gemm_sizes(M, I, H) || !gemm_sizes(M, H, I)) return 0;
  return ffn_space(M, H, I).bytes;
}

nvfp4_status nvfp4_ffn(const uint8_t* a, const uint8_t* a_sf, const uint8_t* w_gu, const uint8_t* w_gu_sf,
                       const float* alpha_gu, const uint16_t* bias_gu, int32_t act, const float* gs_h,
                       const uint8_t* w_d, const uint8_t* w_d_sf, const float* alpha_d, const uint16_t* bias_d,
                       const uint16_t* residual, int64_t ldr, float beta, uint16_t* d, int64_t ldd, int64_t M,
                       int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "nvfp4_ffn";
  bool empty;
  nvfp4_status s = check_k(I);
  if (s != NVFP4_OK) return s;
  s = check_gemm(fn, a, a_sf, w_gu, w_gu_sf, alpha_gu, bias_gu, act, M, I, "I", H, &empty);
  if (s != NVFP4_OK || empty) return s;
  // h stands in for the down projection's first operand, which is the workspace's
  s = check_gemm(fn, a, a_sf, w_d, w_d_sf, alpha_d, bias_d, NVFP4_ACT_NONE, M, H, "H", I, &empty);
  if (s != NVFP4_OK) return s;
  if ((s = check_residual(fn, residual, &ldr, d, &ldd, H)) != NVFP4_OK) return s;
  if (!aligned(gs_h, 4)) return fail(NVFP4_ERR_ALIGN, "%s: gs_h must be 4-byte aligned", fn);
  const FfnSpace f = ffn_space(M, H, I);
  if ((s = check_workspace(fn, workspace, workspace_bytes, f.bytes)) != NVFP4_OK) return s;
  uint8_t* base = (uint8_t*)workspace;
  EpilogueLaunch p = launch_of(a, a_sf, w_gu, w_gu_sf, alpha_gu, bias_gu, act, M, 2 * I, I, H, workspace);
  p.gs = gs_h;
  p.q = base + f.codes;
  p.sf = base + f.scales;
  const hipError_t e = nvfp4::launch_gemm_gated(f.gated, p, true, (hipStream_t)stream);
  if (e != hipSuccess) return hip_status(e, fn);
  p = launch_of(base + f.codes, base + f.scales, w_d, w_d_sf, alpha_d, bias_d, NVFP4_ACT_NONE, M, H, H, I, workspace);
  return hip_status(run_epilogue(f.down, p, residual, ldr, beta, d, ldd, (hipStream_t)stream), fn);
}

nvfp4_status nvfp4_residual_norm(const uint16_t* x, int64_t ldx, const uint16_t* post_weight,
                                 const uint16_t* post_bias, const uint16_t* gate, int64_t gate_group,
                                 const uint16_t* residual, int64_t ldres, float beta, const uint16_t* weight,
                                 const uint16_t* bias, float eps, int32_t kind, uint16_t* r, int64_t ldr,
                                 uint16_t* y, int64_t ldy, const float* gs, uint8_t* q, uint8_t* sf, int64_t T,
                                 int64_t H, void* stream) {
  const char* fn = "nvfp4_residual_norm";
  if (T < 0 || H < 1) return fail(NVFP4_ERR_SHAPE, "%s: T = %lld must be >= 0 and H = %lld >= 1", fn, (long long)T, (long long)H);
  if (kind != NVFP4_NORM_RMS && kind != NVFP4_NORM_LAYER)
    return fail(NVFP4_ERR_SHAPE, "%s: kind = %d is not an nvfp4_norm_kind", fn, kind);
  if (gate_group < 0) return fail(NVFP4_ERR_SHAPE, "%s: gate_group = %lld must be >= 0", fn, (long long)gate_group);
  if (!(eps >= 0.0f)) return fail(NVFP4_ERR_SHAPE, "%s: eps must be >= 0", fn);
  if (q && H % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "%s: H = %lld is not a multiple of the block size 16", fn, (long long)H);
  if (!stride_ok(&ldx, H) || !stride_ok(&ldres, H) || !stride_ok(&ldr, H) || !stride_ok(&ldy, H))
    return fail(NVFP4_ERR_SHAPE, "%s: a row stride is below H = %lld", fn, (long long)H);
  if (T > INT32_MAX || H > (int64_t(1) << 30))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: T = %lld rows, H = %lld: at most 2^31 - 1 rows of 2^30", fn, (long long)T, (long long)H);
  if (T == 0) return ok();
  if (!x) return fail(NVFP4_ERR_NULL, "%s: x must not be NULL", fn);
  if (!r && !y && !q) return fail(NVFP4_ERR_NULL, "%s: no output: r, y and q are all NULL", fn);
  if ((q == nullptr) != (sf == nullptr)) return fail(NVFP4_ERR_NULL, "%s: q and sf go together", fn);
  if (post_bias && !post_weight) return fail(NVFP4_ERR_NULL, "%s: post_bias without post_weight", fn);
  const void* two[] = {x, post_weight, post_bias, gate, residual, weight, bias, r, y};
  for (const void* v : two)
    if (!aligned(v, 2)) return fail(NVFP4_ERR_ALIGN, "%s: bf16 pointers must be 2-byte aligned", fn);
  if (!aligned(q, 8) || !aligned(gs, 4)) return fail(NVFP4_ERR_ALIGN, "%s: q must be 8-byte and gs 4-byte aligned", fn);
  nvfp4::NormLaunch p = {};
  p.x = x;
  p.post_w = post_weight;
  p.post_b = post_bias;
  p.gate = gate;
  p.res = residual;
  p.w = weight;
  p.b = bias;
  p.r = r;
  p.y = y;
  p.gs = gs;
  p.q = q;
  p.sf = sf;
  p.T = T;
  p.H = H;
  p.ldx = ldx;
  p.ldres = ldres;
  p.ldr = ldr;
  p.ldy = ldy;
  p.gate_group = gate_group;
  p.beta = beta;
  p.eps = eps;
  p.inv_h = 1.0 / (double)H;
  p.layer = kind == NVFP4_NORM_LAYER;
  return hip_status(nvfp4::launch_residual_norm(p, (hipStream_t)stream), fn);
}
