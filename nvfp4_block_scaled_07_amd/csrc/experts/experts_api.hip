// C entry points of the mixture-of-experts operators on MXFP4 operands:
// host-side validation and launch.  As everywhere in the library, every check
// runs on the host before anything is enqueued.
#include "../api_util.h"
#include "experts.h"

using nvfp4::aligned;
using nvfp4::fail;
using nvfp4::hip_status;
using nvfp4::MxGroupedLaunch;
using nvfp4::ok;

namespace {

typedef long long ll;

constexpr int64_t kMaxRows = int64_t(1) << 30;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

nvfp4_status check_rule(const char* fn, int32_t rule) {
  if (rule != NVFP4_MX_FLOOR && rule != NVFP4_MX_CEIL)
    return fail(NVFP4_ERR_SHAPE, "%s: rule = %d is not an nvfp4_mx_rule", fn, rule);
  return NVFP4_OK;
}

// K of a quantisation: whole blocks, and chunk counts of a row in 32 bits.
nvfp4_status check_blocks(const char* fn, int64_t K) {
  if (K < 0 || K % 32 != 0)
    return fail(NVFP4_ERR_SHAPE, "%s: K = %lld must be >= 0 and a multiple of the block size 32", fn, (ll)K);
  if (K > (int64_t(1) << 30)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: K = %lld is above 2^30", fn, (ll)K);
  return NVFP4_OK;
}

// K of a product.
nvfp4_status check_product_k(const char* fn, const char* name, int64_t K) {
  if (K < 0 || K % 32 != 0)
    return fail(NVFP4_ERR_SHAPE, "%s: %s = %lld must be >= 0 and a multiple of the block size 32", fn, name, (ll)K);
  if (K == 0 || K % 256 != 0 || K > (int64_t(1) << 22))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: %s = %lld: the library needs 0 < %s <= 4194304 and %s %% 256 == 0", fn, name, (ll)K,
                name, name);
  return NVFP4_OK;
}

// Sizes of a grouped product with N weight rows per expert.
nvfp4_status check_sizes(const char* fn, int64_t rows, int64_t T, int64_t N, const char* nname, int64_t K, int32_t E,
                         bool gather) {
  if (rows < 0 || T < 0 || N < 0 || E < 0)
    return fail(NVFP4_ERR_SHAPE, "%s: rows = %lld, T = %lld, %s = %lld, E = %d must be >= 0", fn, (ll)rows, (ll)T, nname,
                (ll)N, E);
  if (!gather && rows > T)
    return fail(NVFP4_ERR_SHAPE, "%s: rows = %lld > T = %lld with row_token NULL (row r is row r of a)", fn, (ll)rows, (ll)T);
  const nvfp4_status s = check_product_k(fn, "K", K);
  if (s != NVFP4_OK) return s;
  if (rows > kMaxRows || N > kMaxRows || E > 65535)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: rows and %s up to 2^30 and E up to 65535 are supported", fn, nname);
  // row offsets of a in 32 bits; a launch has fewer than 2^32 threads
  if (T > ((int64_t(1) << 32) - 1) / K)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: T = %lld rows of K = %lld: T K < 2^32 is supported", fn, (ll)T, (ll)K);
  if ((rows / 16 + (rows < E ? rows : E)) * ((N + 63) / 64) >= (int64_t(1) << 24))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: rows = %lld of %d experts, %s = %lld: fewer than 2^24 tiles of 16 x 64 are supported",
                fn, (ll)rows, E, nname, (ll)N);
  return NVFP4_OK;
}

nvfp4_status check_pointers(const char* fn, const MxGroupedLaunch& p, const int32_t* status) {
  if (!p.offsets && p.E > 0) return fail(NVFP4_ERR_NULL, "%s: offsets must not be NULL", fn);
  if (!aligned(p.offsets, 4) || !aligned(p.row_token, 4) || !aligned(status, 4) || !aligned(p.alpha, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: offsets, row_token, alpha and status must be 4-byte aligned", fn);
  return NVFP4_OK;
}

nvfp4_status check_operands(const char* fn, const MxGroupedLaunch& p) {
  if (!p.a || !p.a_sf || !p.b || !p.b_sf) return fail(NVFP4_ERR_NULL, "%s: a, a_sf, b and b_sf must not be NULL", fn);
  if (!aligned(p.a, 16) || !aligned(p.a_sf, 16) || !aligned(p.b, 16) || !aligned(p.b_sf, 16))
    return fail(NVFP4_ERR_ALIGN, "%s: a, a_sf, b and b_sf must be 16-byte aligned", fn);
  if (!aligned(p.bias, 2)) return fail(NVFP4_ERR_ALIGN, "%s: bias must be 2-byte aligned", fn);
  return NVFP4_OK;
}

nvfp4_status report(const char* fn, const MxGroupedLaunch& p, int32_t* status, hipStream_t stream) {
  if (!status) return ok();
  return hip_status(nvfp4::launch_expert_status(p.offsets, p.E, p.row_token, p.rows, p.T, status, stream), fn);
}

nvfp4_status check_act(const char* fn, int32_t act) {
  if (act < 0 || act > NVFP4_ACT_SILU) return fail(NVFP4_ERR_SHAPE, "%s: act = %d is not an nvfp4_activation", fn, act);
  return NVFP4_OK;
}

nvfp4_status check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (need == 0) return NVFP4_OK;
  if (!ws || have < need)
    return fail(NVFP4_ERR_WORKSPACE, "%s: the workspace must hold %zu bytes (%zu given)", fn, need, ws ? have : 0);
  if (!aligned(ws, 256)) return fail(NVFP4_ERR_ALIGN, "%s: the workspace must be 256-byte aligned", fn);
  return NVFP4_OK;
}

}  // namespace

nvfp4_status nvfp4_moe_route(const void* logits, int32_t logits_type, int64_t ldl, const float* bias, int32_t score,
                             int32_t n_group, int32_t topk_group, int32_t group_top, int32_t top_k,
                             int32_t renormalize, float scale, int32_t* ids, float* weights, int64_t T, int32_t E,
                             void* stream) {
  const char* fn = "nvfp4_moe_route";
  if (T < 0 || E < 1 || top_k < 1)
    return fail(NVFP4_ERR_SHAPE, "%s: T = %lld must be >= 0, E = %d and top_k = %d >= 1", fn, (ll)T, E, top_k);
  if (logits_type != NVFP4_LOGITS_F32 && logits_type != NVFP4_LOGITS_BF16)
    return fail(NVFP4_ERR_SHAPE, "%s: logits_type = %d is not an nvfp4_logits_type", fn, logits_type);
  if (score != NVFP4_SCORE_SOFTMAX && score != NVFP4_SCORE_SIGMOID)
    return fail(NVFP4_ERR_SHAPE, "%s: score = %d is not an nvfp4_score", fn, score);
  if (n_group < 1 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
    return fail(NVFP4_ERR_SHAPE, "%s: n_group = %d must divide E = %d and topk_group = %d lie in 1 .. n_group", fn, n_group,
                E, topk_group);
  if (group_top != 1 && group_top != 2) return fail(NVFP4_ERR_SHAPE, "%s: group_top = %d must be 1 or 2", fn, group_top);
  if (top_k > topk_group * (int64_t)(E / n_group))
    return fail(NVFP4_ERR_SHAPE, "%s: top_k = %d of %lld experts", fn, top_k, (ll)(topk_group * (int64_t)(E / n_group)));
  if (ldl == 0) ldl = E;
  if (ldl < E) return fail(NVFP4_ERR_SHAPE, "%s: ldl = %lld is below E = %d", fn, (ll)ldl, E);
  if (E > nvfp4::kMaxRouteExperts || top_k > nvfp4::kMaxRouteTop || n_group > 64 || T > kMaxRows)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: E = %d, top_k = %d, n_group = %d, T = %lld: at most %d, %d, 64 and 2^30", fn, E,
                top_k, n_group, (ll)T, nvfp4::kMaxRouteExperts, nvfp4::kMaxRouteTop);
  if (T == 0) return ok();
  if (!logits || !ids || !weights) return fail(NVFP4_ERR_NULL, "%s: logits, ids and weights must not be NULL", fn);
  const bool bf16 = logits_type == NVFP4_LOGITS_BF16;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: logits must be aligned to their type, bias, ids and weights to 4 bytes", fn);
  nvfp4::RouteLaunch p = {};
  p.logits = logits;
  p.ldl = ldl;
  p.bf16 = bf16;
  p.bias = bias;
  p.score = score;
  p.groups = n_group;
  p.top_groups = topk_group;
  p.group_top = E / n_group == 1 ? 1 : group_top;  // a group of one has no second
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  p.scale = scale;
  p.ids = ids;
  p.weights = weights;
  p.T = T;
  p.E = E;
  return hip_status(nvfp4::launch_moe_route(p, (hipStream_t)stream), fn);
}

size_t nvfp4_moe_sort_workspace_size(int64_t T, int32_t E, int32_t top_k) {
  if (T <= 0 || E < 1 || E > 65535 || top_k <= 0 || T > kMaxRows / top_k) return 0;
  return nvfp4::moe_sort_workspace(T * top_k, E);
}

nvfp4_status nvfp4_moe_sort(const int32_t* ids, int32_t first, int32_t* offsets, int32_t* row_token,
                            int32_t* token_rows, int64_t T, int32_t E, int32_t top_k, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const char* fn = "nvfp4_moe_sort";
  if (T < 0 || E < 1 || top_k < 0 || first < 0)
    return fail(NVFP4_ERR_SHAPE, "%s: T = %lld, top_k = %d, first = %d must be >= 0 and E = %d >= 1", fn, (ll)T, top_k, first, E);
  // the kernels compare id - first with E in wrapping 32 bits: no negative id may land below E
  if (first - 1 > INT32_MAX - E) return fail(NVFP4_ERR_SHAPE, "%s: first = %d, E = %d: first + E is above 2^31", fn, first, E);
  if (E > 65535 || (top_k > 0 && T > kMaxRows / top_k))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: E = %d, T = %lld, top_k = %d: E up to 65535 and T top_k up to 2^30", fn, E, (ll)T, top_k);
  // a work-group an expert goes through all ids
  if (E > nvfp4::kMostSorted && T * top_k > (1 << 20))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: T = %lld, top_k = %d: T top_k up to 2^20 above %d experts (E = %d)", fn, (ll)T, top_k,
                nvfp4::kMostSorted, E);
  const int64_t n = T * top_k;
  if (!offsets || (n > 0 && (!ids || !row_token || !token_rows)))
    return fail(NVFP4_ERR_NULL, "%s: ids, offsets, row_token and token_rows must not be NULL", fn);
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(token_rows, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: all pointers must be 4-byte aligned", fn);
  const nvfp4_status s = check_workspace(fn, workspace, workspace_bytes, nvfp4_moe_sort_workspace_size(T, E, top_k));
  if (s != NVFP4_OK) return s;
  nvfp4::SortLaunch p = {};
  p.ids = ids;
  p.first = first;
  p.offsets = offsets;
  p.row_token = row_token;
  p.token_rows = token_rows;
  p.n = n;
  p.top_k = top_k;
  p.E = E;
  p.ws = (uint16_t*)workspace;
  return hip_status(nvfp4::launch_moe_sort(p, (hipStream_t)stream), fn);
}

nvfp4_status nvfp4_mx_quantize(const float* x, int64_t R, int64_t K, int32_t rule, uint8_t* q, uint8_t* sf,
                               void* stream) {
  const char* fn = "nvfp4_mx_quantize";
  if (R < 0) return fail(NVFP4_ERR_SHAPE, "%s: R = %lld must be >= 0", fn, (ll)R);
  nvfp4_status s = check_blocks(fn, K);
  if (s != NVFP4_OK || (s = check_rule(fn, rule)) != NVFP4_OK) return s;
  if (R > INT64_MAX / 4 / (K > 0 ? K : 1)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: R = %lld rows are too many", fn, (ll)R);
  if (R == 0 || K == 0) return ok();
  if (!x || !q || !sf) return fail(NVFP4_ERR_NULL, "%s: x, q and sf must not be NULL", fn);
  if (!aligned(x, 16) || !aligned(q, 16)) return fail(NVFP4_ERR_ALIGN, "%s: x and q must be 16-byte aligned", fn);
  return hip_status(nvfp4::launch_mx_quantize(x, R * K, rule, q, sf, (hipStream_t)stream), fn);
}

nvfp4_status nvfp4_mx_quantize_rows_bf16(const uint16_t* x, const int32_t* row_token, int32_t rule, uint8_t* q,
                                         uint8_t* sf, int64_t rows, int64_t T, int64_t K, void* stream) {
  const char* fn = "nvfp4_mx_quantize_rows_bf16";
  if (rows < 0 || T < 0) return fail(NVFP4_ERR_SHAPE, "%s: rows = %lld and T = %lld must be >= 0", fn, (ll)rows, (ll)T);
  nvfp4_status s = check_blocks(fn, K);
  if (s != NVFP4_OK || (s = check_rule(fn, rule)) != NVFP4_OK) return s;
  if (!row_token && rows > T)
    return fail(NVFP4_ERR_SHAPE, "%s: rows = %lld > T = %lld with row_token NULL", fn, (ll)rows, (ll)T);
  const int64_t most = INT64_MAX / 4 / (K > 0 ? K : 1);
  if (rows > most || T > most) return fail(NVFP4_ERR_UNSUPPORTED, "%s: rows = %lld, T = %lld are too many", fn, (ll)rows, (ll)T);
  if (rows == 0 || K == 0) return ok();
  if ((!x && T > 0) || !q || !sf) return fail(NVFP4_ERR_NULL, "%s: x, q and sf must not be NULL", fn);
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(row_token, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: x and q must be 16-byte, row_token 4-byte aligned", fn);
  return hip_status(nvfp4::launch_mx_quantize_rows(x, row_token, rows, T, K, rule, q, sf, (hipStream_t)stream), fn);
}

nvfp4_status nvfp4_mx_grouped_gemm(const uint8_t* a, const uint8_t* a_sf, const int32_t* row_token, const uint8_t* b,
                                   const uint8_t* b_sf, const int32_t* offsets, const float* alpha,
                                   const uint16_t* bias, uint16_t* d, int64_t rows, int64_t T, int64_t N, int64_t K,
                                   int32_t E, int32_t* status, void* stream) {
  const char* fn = "nvfp4_mx_grouped_gemm";
  nvfp4_status s = check_sizes(fn, rows, T, N, "N", K, E, row_token != nullptr);
  if (s != NVFP4_OK) return s;
  MxGroupedLaunch p = {};
  p.a = a;
  p.a_sf = a_sf;
  p.row_token = row_token;
  p.b = b;
  p.b_sf = b_sf;
  p.offsets = offsets;
  p.alpha = alpha;
  p.bias = bias;
  p.d = d;
  p.rows = rows;
  p.T = T;
  p.N = N;
  p.K = K;
  p.E = E;
  if ((s = check_pointers(fn, p, status)) != NVFP4_OK) return s;
  if (rows == 0 || N == 0 || E == 0) return report(fn, p, status, (hipStream_t)stream);
  if ((s = check_operands(fn, p)) != NVFP4_OK) return s;
  if (!d) return fail(NVFP4_ERR_NULL, "%s: d must not be NULL", fn);
  if (!aligned(d, 2)) return fail(NVFP4_ERR_ALIGN, "%s: d must be 2-byte aligned", fn);
  if ((s = report(fn, p, status, (hipStream_t)stream)) != NVFP4_OK) return s;
  return hip_status(nvfp4::launch_mx_grouped(p, false, (hipStream_t)stream), fn);
}

nvfp4_status nvfp4_mx_grouped_gated_quantize(const uint8_t* a, const uint8_t* a_sf, const int32_t* row_token,
                                             const uint8_t* b, const uint8_t* b_sf, const int32_t* offsets,
                                             const float* alpha, const uint16_t* bias, int32_t act, int32_t rule,
                                             uint8_t* q, uint8_t* sf, int64_t rows, int64_t T, int64_t I, int64_t K,
                                             int32_t E, int32_t* status, void* stream) {
  const char* fn = "nvfp4_mx_grouped_gated_quantize";
  if (I < 0 || I % 32 != 0)
    return fail(NVFP4_ERR_SHAPE, "%s: I = %lld must be >= 0 and a multiple of the block size 32", fn, (ll)I);
  nvfp4_status s = check_sizes(fn, rows, T, I, "I", K, E, row_token != nullptr);
  if (s != NVFP4_OK || (s = check_act(fn, act)) != NVFP4_OK || (s = check_rule(fn, rule)) != NVFP4_OK) return s;
  MxGroupedLaunch p = {};
  p.a = a;
  p.a_sf = a_sf;
  p.row_token = row_token;
  p.b = b;
  p.b_sf = b_sf;
  p.offsets = offsets;
  p.alpha = alpha;
  p.bias = bias;
  p.q = q;
  p.sf = sf;
  p.rows = rows;
  p.T = T;
  p.N = 2 * I;
  p.K = K;
  p.E = E;
  p.act = act;
  p.rule = rule;
  if ((s = check_pointers(fn, p, status)) != NVFP4_OK) return s;
  if (rows == 0 || I == 0 || E == 0) return report(fn, p, status, (hipStream_t)stream);
  if ((s = check_operands(fn, p)) != NVFP4_OK) return s;
  if (!q || !sf) return fail(NVFP4_ERR_NULL, "%s: q and sf must not be NULL", fn);
  if (!aligned(q, 2)) return fail(NVFP4_ERR_ALIGN, "%s: q must be 2-byte aligned", fn);
  if ((s = report(fn, p, status, (hipStream_t)stream)) != NVFP4_OK) return s;
  return hip_status(nvfp4::launch_mx_grouped(p, true, (hipStream_t)stream), fn);
}

namespace {

// Workspace of nvfp4_mx_moe_ffn: the quantised tokens, the hidden rows and the
// down projection's rows.
struct MoeSpace {
  size_t xq, xsf, hq, hsf, down, bytes;
};

MoeSpace moe_space(int64_t T, int64_t H, int64_t I, int32_t top_k) {
  const size_t rows = (size_t)T * (size_t)top_k;
  MoeSpace w;
  w.xq = 0;
  w.xsf = w.xq + align256((size_t)T * (size_t)(H / 2));
  w.hq = w.xsf + align256((size_t)T * (size_t)(H / 32));
  w.hsf = w.hq + align256(rows * (size_t)(I / 2));
  w.down = w.hsf + align256(rows * (size_t)(I / 32));
  w.bytes = w.down + align256(rows * (size_t)H * 2);
  return w;
}

// Whether the products of a layer take these sizes (E experts aside).
bool moe_sizes(int64_t T, int64_t H, int64_t I, int32_t top_k) {
  const int64_t kMaxK = int64_t(1) << 22;
  if (T < 0 || top_k < 0 || H <= 0 || I <= 0 || H % 256 || I % 256 || H > kMaxK || I > kMaxK) return false;
  const int64_t most = ((int64_t(1) << 32) - 1);
  if (T > most / H || (top_k > 0 && T > kMaxRows / top_k)) return false;
  return T * (int64_t)top_k <= most / I;
}

}  // namespace

size_t nvfp4_mx_moe_ffn_workspace_size(int64_t T, int64_t H, int64_t I, int32_t top_k) {
  return moe_sizes(T, H, I, top_k) ? moe_space(T, H, I, top_k).bytes : 0;
}

nvfp4_status nvfp4_mx_moe_ffn(const uint16_t* x, const int32_t* row_token, const int32_t* offsets,
                              const uint8_t* w_gu, const uint8_t* w_gu_sf, const float* alpha_gu,
                              const uint16_t* bias_gu, int32_t act, int32_t rule, const uint8_t* w_d,
                              const uint8_t* w_d_sf, const float* alpha_d, const uint16_t* bias_d,
                              const int32_t* token_rows, const float* token_weight, uint16_t* out, int64_t T,
                              int64_t H, int64_t I, int32_t E, int32_t top_k, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream) {
  const char* fn = "nvfp4_mx_moe_ffn";
  if (T < 0 || E < 0 || top_k < 0)
    return fail(NVFP4_ERR_SHAPE, "%s: T = %lld, E = %d, top_k = %d must be >= 0", fn, (ll)T, E, top_k);
  nvfp4_status s = check_product_k(fn, "H", H);
  if (s != NVFP4_OK || (s = check_product_k(fn, "I", I)) != NVFP4_OK) return s;
  if ((s = check_act(fn, act)) != NVFP4_OK || (s = check_rule(fn, rule)) != NVFP4_OK) return s;
  if (top_k > 0 && E == 0) return fail(NVFP4_ERR_SHAPE, "%s: top_k = %d routed rows need E >= 1 experts", fn, top_k);
  if (!moe_sizes(T, H, I, top_k))
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: T = %lld, top_k = %d: T top_k up to 2^30, T H and T top_k I below 2^32", fn, (ll)T, top_k);
  const int64_t rows = T * (int64_t)top_k;
  if ((s = check_sizes(fn, rows, T, I, "I", H, E, true)) != NVFP4_OK) return s;
  if ((s = check_sizes(fn, rows, rows, H, "H", I, E, false)) != NVFP4_OK) return s;
  if (T == 0) return ok();
  if (!x || !out) return fail(NVFP4_ERR_NULL, "%s: x and out must not be NULL", fn);
  if (rows > 0 && (!row_token || !token_rows || !token_weight))
    return fail(NVFP4_ERR_NULL, "%s: row_token, token_rows and token_weight must not be NULL", fn);
  if (!aligned(x, 16) || !aligned(out, 16)) return fail(NVFP4_ERR_ALIGN, "%s: x and out must be 16-byte aligned", fn);
  if (!aligned(token_rows, 4) || !aligned(token_weight, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: token_rows and token_weight must be 4-byte aligned", fn);
  const MoeSpace w = moe_space(T, H, I, top_k);
  if ((s = check_workspace(fn, workspace, workspace_bytes, w.bytes)) != NVFP4_OK) return s;
  uint8_t* ws = (uint8_t*)workspace;
  hipStream_t st = (hipStream_t)stream;
  MxGroupedLaunch gu = {};
  gu.a = ws + w.xq;
  gu.a_sf = ws + w.xsf;
  gu.row_token = row_token;
  gu.b = w_gu;
  gu.b_sf = w_gu_sf;
  gu.offsets = offsets;
  gu.alpha = alpha_gu;
  gu.bias = bias_gu;
  gu.q = ws + w.hq;
  gu.sf = ws + w.hsf;
  gu.rows = rows;
  gu.T = T;
  gu.N = 2 * I;
  gu.K = H;
  gu.E = E;
  gu.act = act;
  gu.rule = rule;
  MxGroupedLaunch dn = {};
  dn.a = ws + w.hq;
  dn.a_sf = ws + w.hsf;
  dn.b = w_d;
  dn.b_sf = w_d_sf;
  dn.offsets = offsets;
  dn.alpha = alpha_d;
  dn.bias = bias_d;
  // bf16 rows, as in nvfp4_moe_ffn, so that the four calls one by one give the same
  // bits: 0.0024 from the 64-bit layer, where fp32 rows would be 0.0017 (the output's
  // own rounding).  fp32 rows would double what the combine reads (4096 tokens, 8 rows
  // of 6144 each: 403 MB in 84 us) and the projection writes, some 150 us of 1100.
  dn.d = (uint16_t*)(ws + w.down);
  dn.rows = rows;
  dn.T = rows;
  dn.N = H;
  dn.K = I;
  dn.E = E;
  if ((s = check_pointers(fn, gu, status)) != NVFP4_OK || (s = check_pointers(fn, dn, status)) != NVFP4_OK) return s;
  if (rows > 0 && ((s = check_operands(fn, gu)) != NVFP4_OK || (s = check_operands(fn, dn)) != NVFP4_OK)) return s;
  if ((s = report(fn, gu, status, st)) != NVFP4_OK) return s;
  hipError_t e = hipSuccess;
  if (rows > 0) {
    e = nvfp4::launch_mx_quantize_rows(x, nullptr, T, T, H, rule, ws + w.xq, ws + w.xsf, st);
    if (e == hipSuccess) e = nvfp4::launch_mx_grouped(gu, true, st);
    if (e == hipSuccess) e = nvfp4::launch_mx_grouped(dn, false, st);
  }
  if (e == hipSuccess) e = nvfp4::launch_moe_combine(dn.d, token_rows, token_weight, out, T, H, top_k, rows, st);
  return hip_status(e, fn);
}
