// Internal interfaces of the mixture-of-experts operators on MXFP4 operands:
// routing (moe_route.hip), row order (moe_sort.hip), quantisation
// (mx_quantize.hip) and the grouped products (mx_grouped.hip), between their
// kernels and their C entry points (experts_api.hip).
#pragma once
#include "../internal.h"

namespace nvfp4 {

// Experts and weights of T tokens from their router logits.
struct RouteLaunch {
  const void* logits;  // fp32 or bf16 [T][E], row stride ldl
  int64_t ldl;
  bool bf16;
  const float* bias;  // [E] or NULL
  int score;          // 0: softmax, 1: sigmoid
  int groups, top_groups, group_top, top_k;
  bool renormalize;
  float scale;
  int32_t* ids;
  float* weights;
  int64_t T;
  int E;
};
constexpr int kMaxRouteExperts = 1024, kMaxRouteTop = 64;
hipError_t launch_moe_route(const RouteLaunch& p, hipStream_t stream);

// Rows of T tokens of top_k experts each, in expert order.
struct SortLaunch {
  const int32_t* ids;  // [T top_k]
  int32_t first;       // expert e of the output is id first + e
  int32_t* offsets;    // [E + 1]
  int32_t* row_token;  // [T top_k]
  int32_t* token_rows; // [T top_k]
  int64_t n;           // T top_k
  int top_k, E;
  uint16_t* ws;
};
constexpr int kMostSorted = 1024;  // experts of the form for many ids
size_t moe_sort_workspace(int64_t n, int E);
hipError_t launch_moe_sort(const SortLaunch& p, hipStream_t stream);

hipError_t launch_mx_quantize(const float* x, int64_t n, int rule, uint8_t* q, uint8_t* sf, hipStream_t stream);
// bf16 rows x[row_token[i]] (x[i] if row_token is NULL)
hipError_t launch_mx_quantize_rows(const uint16_t* x, const int32_t* row_token, int64_t rows, int64_t T, int64_t K,
                                   int rule, uint8_t* q, uint8_t* sf, hipStream_t stream);

// Products of each expert's rows with its weights.  Row r of A is row
// row_token[r] of a (r itself if NULL); B is [E][N][K].
//   plain: d[r][n] = alpha[e] s + bias[e][n], bf16 [rows][N]
//   gated: h = act(alpha[2e] s_gate + bias) (alpha[2e + 1] s_up + bias), N = 2 I
//          (I gate rows, then I up rows), to MXFP4 [rows][I]
struct MxGroupedLaunch {
  const uint8_t* a;
  const uint8_t* a_sf;
  const int32_t* row_token;
  const uint8_t* b;
  const uint8_t* b_sf;
  const int32_t* offsets;
  const float* alpha;
  const uint16_t* bias;
  uint16_t* d;
  uint8_t* q;
  uint8_t* sf;
  int64_t rows, T, N, K;
  int E, act, rule;
};
// status: 0, 1 + first bad expert, or -(1 + first row whose token is outside [0, T))
hipError_t launch_expert_status(const int32_t* offsets, int E, const int32_t* row_token, int64_t rows, int64_t T,
                                int32_t* status, hipStream_t stream);
hipError_t launch_mx_grouped(const MxGroupedLaunch& p, bool gated, hipStream_t stream);
// ... by the 256 x 256 tiles for experts of many rows (mx_grouped_tile.hip)
void launch_mx_grouped_tile(const MxGroupedLaunch& p, bool gated, hipStream_t stream);

}  // namespace nvfp4
