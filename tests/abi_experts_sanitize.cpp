// Host-layer driver of the mixture-of-experts operators for the
// AddressSanitizer / UndefinedBehaviorSanitizer build
// (tests/test_abi_experts_sanitized.py).  No GPU is touched: every call is a
// query, a no-op or is refused on the host before anything is enqueued (the
// last pointer looked at is misaligned or missing).  It walks sizes, ranges,
// groups and workspaces over a grid, and every entry point's refusals at
// ordinary and extreme arguments.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "nvfp4.h"

static int g_fail = 0;

static void check(bool good, const char* what, int64_t a = 0, int64_t b = 0, int64_t c = 0) {
  if (good) return;
  fprintf(stderr, "FAIL %s (%lld, %lld, %lld): %s\n", what, (long long)a, (long long)b, (long long)c, nvfp4_last_error());
  g_fail = 1;
}

// an aligned non-NULL address that is never dereferenced, and one that no call takes
static uint8_t* const F = (uint8_t*)(uintptr_t)0x10000;
static uint8_t* const ODD = F + 1;
static uint16_t* const D = (uint16_t*)F;
static int32_t* const I32 = (int32_t*)F;
static float* const F32 = (float*)F;

// each ends in a refusal of its last pointer where everything else is in order
static int route(int64_t T, int32_t E, int32_t k, int32_t groups = 1, int32_t kept = 1, int32_t top = 1, int64_t ldl = 0,
                 int32_t type = 0, int32_t score = 0) {
  return nvfp4_moe_route(F, type, ldl, F32, score, groups, kept, top, k, 1, 1.0f, I32, (float*)ODD, T, E, NULL);
}
static int sort(int64_t T, int32_t E, int32_t k, int32_t first = 0, int32_t* rows = (int32_t*)ODD, void* ws = NULL, size_t wsb = 0) {
  return nvfp4_moe_sort(I32, first, I32, I32, rows, T, E, k, ws, wsb, NULL);
}
static int quantize(int64_t R, int64_t K, int32_t rule = 0) { return nvfp4_mx_quantize(F32, R, K, rule, ODD, F, NULL); }
static int rows_bf16(int64_t rows, int64_t T, int64_t K, const int32_t* tok = I32, int32_t rule = 0) {
  return nvfp4_mx_quantize_rows_bf16(D, tok, rule, ODD, F, rows, T, K, NULL);
}
static int gemm(int64_t rows, int64_t T, int64_t N, int64_t K, int32_t E, const int32_t* tok = I32) {
  return nvfp4_mx_grouped_gemm(F, F, tok, F, F, I32, NULL, NULL, (uint16_t*)ODD, rows, T, N, K, E, NULL, NULL);
}
static int gated(int64_t rows, int64_t T, int64_t I, int64_t K, int32_t E, int32_t act = 4, int32_t rule = 0) {
  return nvfp4_mx_grouped_gated_quantize(F, F, I32, F, F, I32, NULL, NULL, act, rule, ODD, F, rows, T, I, K, E, NULL, NULL);
}
static int ffn(int64_t T, int64_t H, int64_t I, int32_t E, int32_t k, void* ws, size_t wsb, int32_t act = 4) {
  return nvfp4_mx_moe_ffn(D, I32, I32, F, F, NULL, NULL, act, 0, F, F, NULL, NULL, I32, F32, D, T, H, I, E, k, ws, wsb,
                          (int32_t*)ODD, NULL);
}

int main() {
  const int64_t kHuge = INT64_MAX;

  // routing: every division into groups
  for (int32_t E : {1, 2, 7, 60, 64, 65, 256, 1000, 1024})
    for (int32_t groups = 1; groups <= E && groups <= 80; ++groups)
      for (int32_t kept = 1; kept <= groups; kept += groups > 8 ? 7 : 1) {
        const int32_t most = E % groups ? 0 : kept * (E / groups);
        for (int32_t k : {1, 2, 8, 63, 64, 65}) {
          const int got = route(5, E, k, groups, kept, 1 + k % 2);
          const int want = E % groups || k > most ? NVFP4_ERR_SHAPE : k > 64 || groups > 64 ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
          check(got == want, "route", E, groups, k);
        }
      }
  for (int64_t v : {int64_t(7), int64_t(-1), -kHuge - 1}) check(route(4, 8, 2, 1, 1, 1, v) == NVFP4_ERR_SHAPE, "ldl", v);
  check(route(4, 8, 2, 1, 1, 1, kHuge) == NVFP4_ERR_ALIGN, "ldl");
  for (int64_t v : {kHuge, (int64_t(1) << 30) + 1}) check(route(v, 8, 2) == NVFP4_ERR_UNSUPPORTED, "route T", v);
  for (int32_t v : {INT32_MIN, -1, INT32_MAX}) {
    check(route(4, v, 2) != NVFP4_OK && route(4, v, v) != NVFP4_OK && route(4, 8, v) == NVFP4_ERR_SHAPE, "route", v);
    check(route(4, 8, 2, v) == NVFP4_ERR_SHAPE && route(4, 8, 2, 4, v) == NVFP4_ERR_SHAPE && route(4, 8, 2, 4, 2, v) == NVFP4_ERR_SHAPE, "groups", v);
    check(route(4, INT32_MAX, 2, INT32_MAX, v) != NVFP4_OK, "groups", v);
    check(route(4, 8, 2, 1, 1, 1, 0, v) == NVFP4_ERR_SHAPE && route(4, 8, 2, 1, 1, 1, 0, 0, v) == NVFP4_ERR_SHAPE, "enum", v);
  }
  check(route(0, 8, 2) == NVFP4_OK, "no tokens");

  // row order: workspaces over the sizes of both forms, ranges up to the largest id
  for (int64_t T : {int64_t(1), int64_t(5120), int64_t(5121), int64_t(1) << 17, int64_t(1) << 20, int64_t(1) << 27, int64_t(1) << 30})
    for (int32_t E : {1, 64, 65, 1024, 1025, 65535})
      for (int32_t k : {1, 8}) {
        const size_t ws = nvfp4_moe_sort_workspace_size(T, E, k);
        const bool too_many = T > (int64_t(1) << 30) / k || (E > 1024 && T * k > (1 << 20));
        if (too_many) {
          check(sort(T, E, k, 0, I32) == NVFP4_ERR_UNSUPPORTED, "too many ids", T, E, k);
          continue;
        }
        check(ws <= (size_t(1) << 26), "sort workspace", T, E, k);
        check(sort(T, E, k) == NVFP4_ERR_ALIGN, "rows", T, E, k);
        if (ws) check(sort(T, E, k, 0, I32) == NVFP4_ERR_WORKSPACE && sort(T, E, k, 0, I32, F, ws - 1) == NVFP4_ERR_WORKSPACE &&
                          sort(T, E, k, 0, I32, F + 128, ws) == NVFP4_ERR_ALIGN, "sort workspace", T, E, k);
      }
  for (int32_t v : {INT32_MIN, -1}) check(sort(4, v, 2) == NVFP4_ERR_SHAPE && sort(4, 8, v) == NVFP4_ERR_SHAPE && sort(4, 8, 2, v) == NVFP4_ERR_SHAPE, "sort", v);
  for (int32_t E : {2, 8, 65535, 65536, INT32_MAX}) {
    check(sort(4, E, 2, INT32_MAX) == NVFP4_ERR_SHAPE && sort(4, E, 2, INT32_MAX - E + 2) == NVFP4_ERR_SHAPE, "range", E);
    check(sort(4, E, 2, INT32_MAX - E + 1) == (E > 65535 ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN), "range", E);
  }
  for (int64_t v : {kHuge, int64_t(1) << 62, (int64_t(1) << 30) + 1}) {
    check(sort(v, 8, 1) == NVFP4_ERR_UNSUPPORTED && sort(v, 8, INT32_MAX) == NVFP4_ERR_UNSUPPORTED, "sort T", v);
    check(nvfp4_moe_sort_workspace_size(v, 8, 1) == 0 && nvfp4_moe_sort_workspace_size(v, 8, INT32_MAX) == 0, "query", v);
    check(sort(v, 8, 0) == NVFP4_ERR_ALIGN, "no choices", v);
  }
  for (int64_t v : {int64_t(-1), -kHuge - 1}) check(sort(v, 8, 2) == NVFP4_ERR_SHAPE && nvfp4_moe_sort_workspace_size(v, 8, 2) == 0, "sort T", v);

  // quantisation
  for (int64_t v : {kHuge, kHuge - 31, int64_t(1) << 62}) {
    check(quantize(v, 32) == NVFP4_ERR_UNSUPPORTED && quantize(4, v / 32 * 32) == NVFP4_ERR_UNSUPPORTED, "quantize", v);
    check(rows_bf16(v, 4, 32) == NVFP4_ERR_UNSUPPORTED && rows_bf16(4, v, 32) == NVFP4_ERR_UNSUPPORTED && rows_bf16(4, 4, v / 32 * 32) == NVFP4_ERR_UNSUPPORTED, "rows", v);
  }
  for (int64_t v : {int64_t(-1), -kHuge - 1, -kHuge}) {
    check(quantize(v, 32) == NVFP4_ERR_SHAPE && quantize(4, v) == NVFP4_ERR_SHAPE, "quantize", v);
    check(rows_bf16(v, 4, 32) == NVFP4_ERR_SHAPE && rows_bf16(4, v, 32) == NVFP4_ERR_SHAPE && rows_bf16(4, 4, v) == NVFP4_ERR_SHAPE, "rows", v);
  }
  check(rows_bf16(5, 4, 32, NULL) == NVFP4_ERR_SHAPE && rows_bf16(4, 4, 32, NULL) == NVFP4_ERR_ALIGN && quantize(4, 32) == NVFP4_ERR_ALIGN, "rows");
  for (int32_t v : {INT32_MIN, -1, 2, INT32_MAX}) check(quantize(4, 32, v) == NVFP4_ERR_SHAPE && rows_bf16(4, 4, 32, I32, v) == NVFP4_ERR_SHAPE && gated(4, 4, 32, 256, 2, 4, v) == NVFP4_ERR_SHAPE, "rule", v);

  // grouped products
  for (int64_t rows : {int64_t(1), int64_t(16), int64_t(1000), int64_t(1) << 20, int64_t(1) << 30})
    for (int64_t N : {int64_t(1), int64_t(64), int64_t(2048), int64_t(1) << 20, int64_t(1) << 30})
      for (int32_t E : {1, 256, 65535}) {
        const int64_t tiles = (rows / 16 + (rows < E ? rows : E)) * ((N + 63) / 64);
        const int want = tiles >= (1 << 24) ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
        check(gemm(rows, 100, N, 256, E) == want, "tiles", rows, N, E);
        if (N % 32 == 0) check(gated(rows, 100, N, 256, E) == want, "tiles", rows, N, E);
      }
  for (int64_t K : {int64_t(256), int64_t(6144), int64_t(1) << 22}) {
    const int64_t most = ((int64_t(1) << 32) - 1) / K;
    check(gemm(4, most, 64, K, 2) == NVFP4_ERR_ALIGN && gemm(4, most + 1, 64, K, 2) == NVFP4_ERR_UNSUPPORTED, "T K", K, most);
  }
  for (int64_t v : {kHuge, kHuge - 255, int64_t(1) << 62}) {
    check(gemm(v, 4, 64, 256, 2) == NVFP4_ERR_UNSUPPORTED && gemm(4, v, 64, 256, 2) == NVFP4_ERR_UNSUPPORTED && gemm(4, 4, v, 256, 2) == NVFP4_ERR_UNSUPPORTED, "gemm", v);
    check(gemm(4, 4, 64, v / 32 * 32, 2) == NVFP4_ERR_UNSUPPORTED && gated(4, 4, v / 32 * 32, 256, 2) == NVFP4_ERR_UNSUPPORTED, "gemm", v);
  }
  for (int64_t v : {int64_t(-1), -kHuge - 1, -kHuge}) {
    check(gemm(v, 4, 64, 256, 2) == NVFP4_ERR_SHAPE && gemm(4, v, 64, 256, 2) == NVFP4_ERR_SHAPE && gemm(4, 4, v, 256, 2) == NVFP4_ERR_SHAPE, "gemm", v);
    check(gemm(4, 4, 64, v, 2) == NVFP4_ERR_SHAPE && gated(4, 4, v, 256, 2) == NVFP4_ERR_SHAPE, "gemm", v);
  }
  for (int32_t v : {INT32_MIN, -1}) check(gemm(4, 4, 64, 256, v) == NVFP4_ERR_SHAPE && gated(4, 4, 64, 256, 2, v) == NVFP4_ERR_SHAPE, "gemm", v);
  for (int32_t v : {65536, INT32_MAX}) check(gemm(4, 4, 64, 256, v) == NVFP4_ERR_UNSUPPORTED && gated(4, 4, 64, 256, 2, v) == NVFP4_ERR_SHAPE, "gemm", v);
  check(gemm(5, 4, 64, 256, 2, NULL) == NVFP4_ERR_SHAPE && gemm(0, 4, 64, 256, 2) == NVFP4_OK && gemm(4, 4, 0, 256, 2) == NVFP4_OK && gemm(4, 4, 64, 256, 0) == NVFP4_OK, "no-ops");

  // the layer
  for (int64_t T : {int64_t(1), int64_t(16), int64_t(4096), int64_t(1) << 20, int64_t(1) << 32, kHuge})
    for (int64_t H : {int64_t(256), int64_t(6144), int64_t(1) << 22})
      for (int64_t I : {int64_t(256), int64_t(2048), int64_t(1) << 22})
        for (int32_t k : {1, 8, INT32_MAX}) {
          const size_t ws = nvfp4_mx_moe_ffn_workspace_size(T, H, I, k);
          if (ws == 0) {
            check(ffn(T, H, I, 8, k, F, SIZE_MAX) == NVFP4_ERR_UNSUPPORTED, "layer size", T, H, I);
            continue;
          }
          check(ws >= size_t(T) * size_t(H / 2) + size_t(T * k) * size_t(I / 2 + 2 * H), "layer workspace", T, H, I);
          const int none = ffn(T, H, I, 8, k, NULL, 0);
          if (none == NVFP4_ERR_UNSUPPORTED) continue;  // too many tiles
          check(none == NVFP4_ERR_WORKSPACE && ffn(T, H, I, 8, k, F, ws - 1) == NVFP4_ERR_WORKSPACE, "layer workspace", T, H, I);
          check(ffn(T, H, I, 8, k, F + 16, ws) == NVFP4_ERR_ALIGN && ffn(T, H, I, 8, k, F, ws) == NVFP4_ERR_ALIGN, "layer pointers", T, H, I);
        }
  for (int64_t v : {int64_t(-1), -kHuge - 1}) {
    check(ffn(v, 256, 256, 8, 2, F, SIZE_MAX) == NVFP4_ERR_SHAPE && ffn(4, v, 256, 8, 2, F, SIZE_MAX) == NVFP4_ERR_SHAPE && ffn(4, 256, v, 8, 2, F, SIZE_MAX) == NVFP4_ERR_SHAPE, "layer", v);
    check(nvfp4_mx_moe_ffn_workspace_size(v, 256, 256, 2) == 0 && nvfp4_mx_moe_ffn_workspace_size(4, v, 256, 2) == 0 && nvfp4_mx_moe_ffn_workspace_size(4, 256, v, 2) == 0, "query", v);
  }
  for (int32_t v : {INT32_MIN, -1}) check(ffn(4, 256, 256, v, 2, F, SIZE_MAX) == NVFP4_ERR_SHAPE && ffn(4, 256, 256, 8, v, F, SIZE_MAX) == NVFP4_ERR_SHAPE && ffn(4, 256, 256, 8, 2, F, SIZE_MAX, v) == NVFP4_ERR_SHAPE, "layer", v);
  check(ffn(0, 256, 256, 8, 2, NULL, 0) == NVFP4_OK && nvfp4_last_error()[0] == 0, "no tokens");
  if (g_fail) return 1;
  printf("all host checks passed\n");
  return 0;
}
