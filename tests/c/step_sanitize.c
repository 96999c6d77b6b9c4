/*
 * The host code of kt_step.h's entry points under AddressSanitizer and
 * UndefinedBehaviorSanitizer: every call here is answered on the host before
 * any GPU work.  Exits nonzero on a failed check; a sanitizer report aborts the run.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "kt_step.h"

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

static void norms(void) {
  const int32_t hs[] = {0, -1, INT32_MIN, KT_NORM_MAX_HIDDEN + 1, INT32_MAX};
  for (size_t i = 0; i < sizeof hs / sizeof *hs; ++i) {
    const kt_norm n = {hs[i], 0, 0, 0, 0.f, 1.f, 0, 0, 0, 0, 0};
    check(kt_norm_bwd_workspace_bytes(&n, 4) == 0 && kt_rawint4_last_error()[0], "hidden");
    refused(kt_norm_fwd(&n, 4, FAKE, 0, 0, 0, FAKE, 0), "hidden");
  }
  const int32_t ts[] = {-1, INT32_MIN, (1 << 23) + 1, INT32_MAX};
  const kt_norm n = {KT_NORM_MAX_HIDDEN, KT_NORM_LAYER, KT_TYPE_F32, 1, 1e-6f, 1.f, FAKE, FAKE, FAKE, FAKE, FAKE};
  for (size_t i = 0; i < sizeof ts / sizeof *ts; ++i) {
    refused(kt_norm_fwd(&n, ts[i], FAKE, FAKE, FAKE, FAKE, FAKE, 0), "tokens");
    refused(kt_norm_bwd(&n, ts[i], FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 1.f, FAKE, (size_t)-1, 0),
            "tokens");
  }
  check(kt_norm_bwd_workspace_bytes(&n, 1 << 23) % 256 == 0, "a size");
  check(kt_norm_bwd(&n, 1 << 23, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 1.f, FAKE, 4096, 0) ==
            KT_RAWINT4_EWORKSPACE, "a small workspace");
  refused(kt_norm_bwd(&n, 4, ODD, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 1.f, FAKE, (size_t)-1, 0), "odd h");
  refused(kt_norm_fwd(0, 4, FAKE, FAKE, 0, FAKE, FAKE, 0), "no norm");
  check(kt_norm_fwd(&n, 0, 0, 0, 0, 0, 0, 0) == KT_RAWINT4_OK, "no tokens");
}

static void steps(void) {
  kt_adamw h = {1e-3, 0.9, 0.999, 1e-8, 0.01, 0.0, 1.0, KT_ADAMW_STATES_E4M3};
  kt_adamw_tensor t[3] = {{8, 1, 0, 1, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE}, {0, 1, 1, 0, 0, 0, 0, 0, 0, 0, 0}, {8, 0, 1, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE}};
  const int32_t counts[] = {-1, INT32_MIN, KT_ADAMW_MAX_TENSORS + 1, INT32_MAX};
  for (size_t i = 0; i < sizeof counts / sizeof *counts; ++i) {
    check(kt_adamw_workspace_bytes(counts[i]) == 0, "num_tensors");
    refused(kt_adamw_step(&h, t, counts[i], FAKE, 0, 0, FAKE, (size_t)-1, 0), "num_tensors");
  }
  check(kt_adamw_step(&h, t, 3, FAKE, FAKE, FAKE, FAKE, 256, 0) == KT_RAWINT4_EWORKSPACE, "a small workspace");
  t[2].count = INT64_MAX;
  refused(kt_adamw_step(&h, t, 3, FAKE, 0, 0, FAKE, (size_t)-1, 0), "a count");
  t[2].count = INT64_MIN;
  refused(kt_adamw_step(&h, t, 3, FAKE, 0, 0, FAKE, (size_t)-1, 0), "a count");
  t[2].count = 8, t[2].v_scale = ODD;
  refused(kt_adamw_step(&h, t, 3, FAKE, 0, 0, FAKE, (size_t)-1, 0), "an odd scale");
  h.beta2 = NAN;
  refused(kt_adamw_step(&h, t, 1, FAKE, 0, 0, FAKE, (size_t)-1, 0), "beta2");
  check(kt_adamw_workspace_bytes(KT_ADAMW_MAX_TENSORS) % 256 == 0, "a size");
}

static void experts(void) {
  kt_rawint4_moe_layer l = {384, 8, 7168, 2048, 16, 1.f, 0.f, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0};
  const int32_t ts[] = {-1, INT32_MIN, KT_MOE_DECODE_MAX_TOKENS + 1, INT32_MAX};
  for (size_t i = 0; i < sizeof ts / sizeof *ts; ++i) {
    check(kt_moe_decode_workspace_bytes(&l, ts[i]) == 0, "tokens");
    refused(kt_moe_decode(&l, ts[i], FAKE, FAKE, FAKE, FAKE, FAKE, (size_t)-1, 0), "tokens");
  }
  size_t last = 0;
  for (int32_t t = 0; t <= KT_MOE_DECODE_MAX_TOKENS; ++t) {
    const size_t n = kt_moe_decode_workspace_bytes(&l, t);
    check(n >= last && n % 256 == 0, "sizes grow");
    last = n;
  }
  check(kt_moe_decode(&l, 4, FAKE, FAKE, FAKE, FAKE, FAKE, 4096, 0) == KT_RAWINT4_EWORKSPACE, "a small workspace");
  l.top_k = 17;
  refused(kt_moe_decode(&l, 61, FAKE, FAKE, FAKE, FAKE, FAKE, (size_t)-1, 0), "slots");
  l.top_k = 0;
  refused(kt_moe_decode(&l, 4, FAKE, FAKE, FAKE, FAKE, FAKE, (size_t)-1, 0), "top_k");
}

int main(void) {
  norms();
  steps();
  experts();
  printf("%d checks, %d failed\n", checks, fails);
  return fails != 0;
}
