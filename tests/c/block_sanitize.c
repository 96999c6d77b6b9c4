/*
 * The host code of kt_block.h's entry points under AddressSanitizer and
 * UndefinedBehaviorSanitizer: every call here is answered on the host before
 * any GPU work.  It sweeps the workspace sizes up to the limits (multiples of
 * 256 bytes that grow with the token count) and drives every entry point through
 * its argument errors.  Exits nonzero on a failed check; a sanitizer report
 * aborts the run.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kt_block.h"

#define FAKE ((void*)(uintptr_t)(1u << 20)) /* 256-byte aligned, never dereferenced */
#define ODD ((void*)(uintptr_t)((1u << 20) + 2))

static int fails = 0, checks = 0;
static void check(int ok, const char* what) {
  ++checks;
  if (!ok) {
    printf("FAIL %s (%s)\n", what, kt_rawint4_last_error());
    ++fails;
  }
}
static void refused(int rc, const char* what) { check(rc == KT_RAWINT4_EINVAL && kt_rawint4_last_error()[0], what); }

static void sweep_sizes(void) {
  const int ks[] = {8, 136, 1024, 7168, 65536}, ns[] = {1, 7, 384, 4096, 65536};
  const int ts[] = {0, 1, 16, 17, 64, 65, 128, 129, 1000, 4096, 16384, 1 << 17, 1 << 20};
  for (size_t a = 0; a < sizeof ks / sizeof *ks; ++a)
    for (size_t b = 0; b < sizeof ns / sizeof *ns; ++b)
      for (int act = KT_ACT_NONE; act <= KT_ACT_GELU_TANH; ++act) {
        const kt_linear l = {ks[a], ns[b], act, FAKE, FAKE};
        size_t fwd = 0, bwd = 0, ck = 0;
        for (size_t c = 0; c < sizeof ts / sizeof *ts; ++c) {
          const size_t f = kt_linear_workspace_bytes(&l, ts[c]), g = kt_linear_bwd_workspace_bytes(&l, ts[c], 0),
                       h = kt_linear_bwd_workspace_bytes(&l, ts[c], 1);
          check(f % 256 == 0 && g % 256 == 0 && h % 256 == 0, "sizes are multiples of 256");
          check(f >= fwd && g >= bwd && h >= ck && h >= g, "sizes grow with the tokens");
          fwd = f, bwd = g, ck = h;
        }
      }
}

static void linear_errors(void) {
  const int bad[][3] = {{0, 8, 0}, {12, 8, 0}, {65544, 8, 0}, {-8, 8, 0}, {INT32_MIN, 8, 0}, {8, 0, 0},
                        {8, 65537, 0}, {8, -1, 0}, {8, 8, -1}, {8, 8, 5}, {8, 8, INT32_MAX}};
  for (size_t i = 0; i < sizeof bad / sizeof *bad; ++i) {
    const kt_linear l = {bad[i][0], bad[i][1], bad[i][2], FAKE, NULL};
    check(kt_linear_workspace_bytes(&l, 4) == 0 && kt_rawint4_last_error()[0], "size of an invalid layer");
    check(kt_linear_bwd_workspace_bytes(&l, 4, 1) == 0 && kt_rawint4_last_error()[0], "size of an invalid layer");
    refused(kt_linear_fwd(&l, 4, FAKE, NULL, FAKE, KT_TYPE_BF16, NULL, FAKE, 1u << 20, NULL), "an invalid layer");
    refused(kt_linear_bwd(&l, 4, FAKE, NULL, NULL, FAKE, KT_TYPE_BF16, NULL, FAKE, FAKE, FAKE, 0, 1.f, FAKE, 1u << 20,
                          NULL), "an invalid layer");
  }
  const kt_linear l = {7168, 384, KT_ACT_NONE, FAKE, NULL}, act = {7168, 384, KT_ACT_SILU, FAKE, NULL};
  const int32_t counts[] = {-1, INT32_MIN, (1 << 20) + 1, INT32_MAX};
  for (size_t i = 0; i < sizeof counts / sizeof *counts; ++i) {
    refused(kt_linear_fwd(&l, counts[i], FAKE, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, (size_t)-1, NULL), "tokens");
    refused(kt_linear_bwd(&l, counts[i], FAKE, NULL, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, FAKE, 0, 1.f, FAKE,
                          (size_t)-1, NULL), "tokens");
  }
  refused(kt_linear_fwd(NULL, 4, FAKE, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, 0, NULL), "no layer");
  refused(kt_linear_fwd(&l, 4, NULL, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, 0, NULL), "no inputs");
  refused(kt_linear_fwd(&l, 4, FAKE, ODD, FAKE, KT_TYPE_F32, NULL, FAKE, 0, NULL), "an odd residual");
  refused(kt_linear_fwd(&l, 4, FAKE, NULL, FAKE, 2, NULL, FAKE, 0, NULL), "an output type");
  const size_t fwd = kt_linear_workspace_bytes(&l, 300), bwd = kt_linear_bwd_workspace_bytes(&l, 300, 1);
  check(kt_linear_fwd(&l, 300, FAKE, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, fwd - 256, NULL) == KT_RAWINT4_EWORKSPACE,
        "a small workspace");
  refused(kt_linear_fwd(&l, 300, FAKE, NULL, FAKE, KT_TYPE_F32, NULL, ODD, fwd, NULL), "an odd workspace");
  const kt_ckpt8 c = {KT_CKPT8_E4M3, FAKE, FAKE}, odd = {KT_CKPT8_INT8, ODD, FAKE}, none = {KT_CKPT8_INT8, FAKE, NULL},
                 fmt = {7, FAKE, FAKE};
  check(kt_linear_bwd(&act, 300, NULL, &c, FAKE, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, FAKE, 0, 1.f, FAKE, 0, NULL) ==
            KT_RAWINT4_EWORKSPACE, "no room for the backward");
  const kt_ckpt8* cks[] = {&odd, &none, &fmt};
  for (int i = 0; i < 3; ++i)
    refused(kt_linear_bwd(&act, 300, NULL, cks[i], FAKE, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, FAKE, 0, 1.f, FAKE, bwd,
                          NULL), "a checkpoint");
  refused(kt_linear_bwd(&act, 300, FAKE, NULL, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, FAKE, 0, 1.f, FAKE, bwd, NULL),
          "no preact");
  refused(kt_linear_bwd(&l, 300, FAKE, NULL, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, FAKE, 0, NAN, FAKE, bwd, NULL),
          "a scale of NaN");
}

static void router_errors(void) {
  const kt_router bad[] = {
      {0, 1, 1, 1, 1, 0, 1, 1.f, 1},       {INT32_MAX, 1, 1, 1, 1, 0, 1, 1.f, 1}, {64, 0, 1, 1, 1, 0, 1, 1.f, 1},
      {64, 65, 1, 1, 1, 0, 1, 1.f, 1},     {64, 4, 0, 1, 1, 0, 1, 1.f, 1},        {64, 4, -4, 1, 1, 0, 1, 1.f, 1},
      {64, 4, 65, 1, 1, 0, 1, 1.f, 1},     {64, 4, 4, 5, 1, 0, 1, 1.f, 1},        {64, 4, 4, 2, 3, 0, 1, 1.f, 1},
      {64, 40, 4, 2, 1, 0, 1, 1.f, 1},     {64, 4, 4, 2, 1, 2, 1, 1.f, 1},        {64, 4, 4, 2, 1, 0, 1, INFINITY, 1},
      {64, 4, 4, 2, 1, 0, 1, 1.f, 2},      {64, 4, 4, INT32_MIN, 1, 0, 1, 1.f, 1}};
  for (size_t i = 0; i < sizeof bad / sizeof *bad; ++i) {
    refused(kt_router_fwd(&bad[i], 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, NULL), "an invalid router");
    refused(kt_router_bwd(&bad[i], 4, FAKE, FAKE, FAKE, FAKE, NULL), "an invalid router");
  }
  const kt_router r = {64, 4, 4, 2, 2, KT_SCORE_SIGMOID, 1, 2.5f, KT_TYPE_BF16};
  const int32_t counts[] = {-1, INT32_MIN, (1 << 23) + 1, INT32_MAX};
  for (size_t i = 0; i < sizeof counts / sizeof *counts; ++i) {
    refused(kt_router_fwd(&r, counts[i], FAKE, NULL, NULL, FAKE, FAKE, NULL, 0, NULL), "tokens");
    refused(kt_router_bwd(&r, counts[i], FAKE, FAKE, FAKE, FAKE, NULL), "tokens");
  }
  refused(kt_router_fwd(&r, 4, ODD, NULL, NULL, FAKE, FAKE, NULL, 0, NULL), "odd logits");
  refused(kt_router_fwd(&r, 4, FAKE, NULL, NULL, ODD, FAKE, NULL, 0, NULL), "odd ids");
  refused(kt_router_bwd(&r, 4, FAKE, FAKE, FAKE, ODD, NULL), "an odd gradient");
  refused(kt_router_update_bias(FAKE, FAKE, 0, 0.1f, NULL), "no experts");
  refused(kt_router_update_bias(FAKE, FAKE, INT32_MAX, 0.1f, NULL), "too many experts");
  refused(kt_router_update_bias(FAKE, ODD, 8, INFINITY, NULL), "a rate");
  check(kt_router_fwd(&r, 0, NULL, NULL, NULL, NULL, NULL, NULL, 1, NULL) == KT_RAWINT4_OK, "no tokens");
}

static void checkpoint_errors(void) {
  const int64_t sizes[][2] = {{-1, 4}, {4, -1}, {INT64_MIN, INT64_MIN}, {INT64_MAX, INT64_MAX}, {2, INT64_MAX},
                              {INT64_MAX, 1}, {((int64_t)1 << 32) + 1, 32}, {(int64_t)1 << 31, 65}};
  for (size_t i = 0; i < sizeof sizes / sizeof *sizes; ++i) {
    refused(kt_ckpt8_pack(FAKE, sizes[i][0], sizes[i][1], 0, FAKE, FAKE, NULL), "sizes");
    refused(kt_ckpt8_unpack(FAKE, FAKE, sizes[i][0], sizes[i][1], 1, FAKE, NULL), "sizes");
  }
  refused(kt_ckpt8_pack(FAKE, 4, 4, -1, FAKE, FAKE, NULL), "a format");
  refused(kt_ckpt8_pack(NULL, 4, 4, 0, FAKE, FAKE, NULL), "no rows");
  refused(kt_ckpt8_unpack(ODD, FAKE, 4, 4, 0, FAKE, NULL), "odd codes");
  check(kt_ckpt8_pack(NULL, INT64_MAX, 0, 0, NULL, NULL, NULL) == KT_RAWINT4_OK, "rows without columns");
  check(kt_ckpt8_unpack(NULL, NULL, 0, 1 << 20, 1, NULL, NULL) == KT_RAWINT4_OK, "columns without rows");
}

int main(void) {
  sweep_sizes();
  linear_errors();
  router_errors();
  checkpoint_errors();
  printf("%d checks, %d failed\n", checks, fails);
  return fails != 0;
}
