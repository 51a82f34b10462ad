// Host-layer driver of the block operators for the AddressSanitizer /
// UndefinedBehaviorSanitizer build (tests/test_abi_block_sanitized.py).  No GPU
// is touched: every call is a query or is refused on the host before anything
// is enqueued.  It walks plan choice and workspace sizes over a grid of shapes
// (the library's own choice and every forced kind and split count), and every
// entry point's refusals at ordinary and extreme arguments.
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

// an aligned non-NULL address that is never dereferenced
static uint8_t* const F = (uint8_t*)(uintptr_t)0x10000;
static uint16_t* const D = (uint16_t*)F;

static int epilogue(int64_t M, int64_t N, int64_t K, size_t wsb, int64_t ldd = 0, int64_t ldr = 0, int32_t act = 0) {
  return nvfp4_gemm_epilogue(F, F, F, F, NULL, D, act, D, ldr, 1.0f, D, ldd, M, N, K, wsb ? F : NULL, wsb, NULL);
}
static int gated(int64_t M, int64_t I, int64_t K, size_t wsb, int64_t ldh = 0) {
  return nvfp4_gemm_gated(F, F, F, F, NULL, D, 4, D, ldh, M, I, K, wsb ? F : NULL, wsb, NULL);
}
static int gated_quantize(int64_t M, int64_t I, int64_t K, size_t wsb) {
  return nvfp4_gemm_gated_quantize(F, F, F, F, NULL, D, 4, NULL, F, F, M, I, K, wsb ? F : NULL, wsb, NULL);
}
static int ffn(int64_t M, int64_t H, int64_t I, size_t wsb, int64_t ldd = 0) {
  return nvfp4_ffn(F, F, F, F, NULL, NULL, 4, NULL, F, F, NULL, NULL, D, 0, 1.0f, D, ldd, M, H, I, wsb ? F : NULL, wsb, NULL);
}
static int norm(int64_t T, int64_t H, int64_t group, int64_t ldx, int32_t kind, float eps, uint16_t* y = D) {
  return nvfp4_residual_norm(D, ldx, D, D, D, group, D, 0, 1.0f, D, D, eps, kind, NULL, 0, y, 0, NULL, NULL, NULL, T, H, NULL);
}

int main() {
  const int64_t kHuge = INT64_MAX;
  const int64_t Ms[] = {1, 15, 16, 17, 64, 128, 300, 1000, 2048, 8192, 1 << 20, int64_t(1) << 29};
  const int64_t Ns[] = {1, 16, 17, 256, 336, 768, 2048, 6144, 1 << 20, int64_t(1) << 34};
  const int64_t Ks[] = {256, 512, 768, 1536, 6144, 6400, 1 << 16, 1 << 22};
  int kinds_seen = 0;
  const char* last = "";
  for (int kind = -1; kind < 40; ++kind)
    for (int splits = 0; splits <= 16; splits += kind < 0 ? 17 : 4) {
      check(nvfp4_force_plan(0, kind, splits) == NVFP4_OK, "force_plan", kind, splits);
      for (int64_t M : Ms)
        for (int64_t N : Ns)
          for (int64_t K : Ks) {
            const char* name = nvfp4_gemm_epilogue_plan(M, N, K);
            const char* gname = nvfp4_gemm_gated_plan(M, N, K);
            check(name && name[0] && gname && gname[0], "plan name", M, N, K);
            if (strcmp(name, last)) ++kinds_seen;
            last = name;
            const bool none = !strcmp(name, "none");
            check(none == !strcmp(gname, "none"), "the same sizes are served", M, N, K);
            if (none) {
              check(nvfp4_gemm_epilogue_workspace_size(M, N, K) == 0 && epilogue(M, N, K, 0) == NVFP4_ERR_UNSUPPORTED &&
                        gated(M, N, K, 0) == NVFP4_ERR_UNSUPPORTED,
                    "too large", M, N, K);
              continue;
            }
            // a plan that needs a workspace refuses a call without one, or with one byte less
            if (const size_t ws = nvfp4_gemm_epilogue_workspace_size(M, N, K)) {
              check(ws < (size_t(1) << 30), "workspace size", M, N, K);
              check(epilogue(M, N, K, 0) == NVFP4_ERR_WORKSPACE && epilogue(M, N, K, ws - 1) == NVFP4_ERR_WORKSPACE, "epilogue workspace", M, N, K);
            }
            if (const size_t ws = nvfp4_gemm_gated_workspace_size(M, N, K)) {
              check(ws < (size_t(1) << 30), "workspace size", M, N, K);
              // (the 16 x 8 tiles serve only one of the two forms, so their need may be the other's)
              if (strncmp(gname, "gatedreg16x8", 12)) {
                check(gated(M, N, K, 0) == NVFP4_ERR_WORKSPACE && gated(M, N, K, ws - 1) == NVFP4_ERR_WORKSPACE, "gated workspace", M, N, K);
                if (N % 16 == 0) check(gated_quantize(M, N, K, ws - 1) == NVFP4_ERR_WORKSPACE, "gated workspace", M, N, K);
              }
            }
            if (N % 256 == 0) {
              const size_t ws = nvfp4_ffn_workspace_size(M, K, N);
              if (N > (1 << 22)) {
                check(ws == 0 && ffn(M, K, N, 1 << 30) == NVFP4_ERR_UNSUPPORTED, "ffn too long", M, K, N);
              } else if (ws) {
                check(ws >= 4096 + size_t(M) * size_t(N / 2) + size_t(M) * size_t(N / 16), "ffn workspace size", M, K, N);
                check(ffn(M, K, N, 0) == NVFP4_ERR_WORKSPACE && ffn(M, K, N, ws - 1) == NVFP4_ERR_WORKSPACE, "ffn workspace", M, K, N);
              }
            }
          }
    }
  check(kinds_seen > 20, "plans seen", kinds_seen);
  check(nvfp4_force_plan(0, -1, 0) == NVFP4_OK, "force_plan reset");

  // extreme sizes and strides
  for (int64_t v : {kHuge, kHuge - 63, int64_t(1) << 62, (int64_t(1) << 36) + 1}) {
    check(epilogue(v, 16, 256, 0) == NVFP4_ERR_UNSUPPORTED && epilogue(16, v, 256, 0) == NVFP4_ERR_UNSUPPORTED, "epilogue size", v);
    check(epilogue(v, v, 256, 0) == NVFP4_ERR_UNSUPPORTED, "epilogue size", v);
    check(gated(v, 16, 256, 0) == NVFP4_ERR_UNSUPPORTED && gated(16, v, 256, 0) == NVFP4_ERR_UNSUPPORTED, "gated size", v);
    check(gated_quantize(16, v / 16 * 16, 256, 0) == NVFP4_ERR_UNSUPPORTED || v < (int64_t(1) << 40), "gated size", v);
    check(ffn(v, 256, 256, 1 << 20) == NVFP4_ERR_UNSUPPORTED, "ffn size", v);
    check(nvfp4_gemm_epilogue_workspace_size(v, v, v) == 0 && nvfp4_gemm_gated_workspace_size(v, 16, 256) == 0 &&
              nvfp4_ffn_workspace_size(v, 256, 256) == 0,
          "queries", v);
    check(norm(v, 64, 0, 0, 0, 0.0f) == NVFP4_ERR_UNSUPPORTED && norm(4, v, 0, 0, 0, 0.0f) == NVFP4_ERR_UNSUPPORTED, "norm size", v);
  }
  for (int64_t v : {-kHuge - 1, -kHuge, int64_t(-1)}) {
    check(epilogue(v, 16, 256, 0) == NVFP4_ERR_SHAPE && epilogue(16, v, 256, 0) == NVFP4_ERR_SHAPE, "negative", v);
    check(epilogue(16, 16, v, 0) != NVFP4_OK && epilogue(16, 16, 256, 0, v) == NVFP4_ERR_SHAPE, "negative", v);
    check(epilogue(16, 16, 256, 0, 0, v) == NVFP4_ERR_SHAPE && gated(16, 16, 256, 0, v) == NVFP4_ERR_SHAPE, "negative stride", v);
    check(gated(v, 16, 256, 0) == NVFP4_ERR_SHAPE && gated_quantize(16, v, 256, 0) == NVFP4_ERR_SHAPE, "negative", v);
    check(ffn(v, 256, 256, 1 << 20) == NVFP4_ERR_SHAPE && ffn(16, v, 256, 1 << 20) != NVFP4_OK && ffn(16, 256, v, 1 << 20) != NVFP4_OK, "negative", v);
    check(ffn(16, 256, 256, 1 << 20, v) == NVFP4_ERR_SHAPE, "negative stride", v);
    check(norm(v, 64, 0, 0, 0, 0.0f) == NVFP4_ERR_SHAPE && norm(4, v, 0, 0, 0, 0.0f) == NVFP4_ERR_SHAPE, "negative", v);
    check(norm(4, 64, v, 0, 0, 0.0f) == NVFP4_ERR_SHAPE && norm(4, 64, 0, v, 0, 0.0f) == NVFP4_ERR_SHAPE, "negative", v);
    check(nvfp4_gemm_epilogue_workspace_size(v, 16, 256) == 0 && nvfp4_gemm_gated_workspace_size(16, 16, v) == 0 &&
              nvfp4_ffn_workspace_size(16, v, 256) == 0 && !strcmp(nvfp4_gemm_gated_plan(16, v, 256), "none"),
          "queries", v);
  }
  for (int32_t v : {INT32_MIN, -1, 5, INT32_MAX}) check(epilogue(16, 16, 256, 0, 0, 0, v) == NVFP4_ERR_SHAPE, "act", v);
  for (int32_t v : {INT32_MIN, -1, 2, INT32_MAX}) check(norm(4, 64, 0, 0, v, 0.0f) == NVFP4_ERR_SHAPE, "kind", v);
  const float nan = __builtin_nanf("");
  for (float v : {-1.0f, -__builtin_inff(), nan}) check(norm(4, 64, 0, 0, 0, v) == NVFP4_ERR_SHAPE, "eps");
  check(norm(4, 64, 0, 0, 0, 0.0f, NULL) == NVFP4_ERR_NULL && strstr(nvfp4_last_error(), "no output"), "no output");
  check(epilogue(0, 16, 256, 0) == NVFP4_OK && gated(16, 0, 256, 0) == NVFP4_OK && ffn(0, 256, 256, 0) == NVFP4_OK &&
            norm(0, 64, 0, 0, 0, 0.0f) == NVFP4_OK && nvfp4_last_error()[0] == 0,
        "no-ops");
  if (g_fail) return 1;
  printf("all host checks passed\n");
  return 0;
}
