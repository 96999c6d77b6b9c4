/*
 * A plain C consumer of include/kt_block.h: compiled with gcc, linked to
 * libkt_rawint4.so.  It only makes calls that the host answers before any GPU
 * work (sizes, argument errors, calls without tokens), so it runs on a machine
 * without a GPU.  Prints one line per check and exits nonzero after a failure.
 */
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "kt_block.h"

#define FAKE ((void*)(uintptr_t)(1u << 20)) /* 256-byte aligned, never dereferenced */

static int fails = 0;
static void check(int ok, const char* what) {
  printf("%s %s\n", ok ? "ok  " : "FAIL", what);
  if (!ok) ++fails;
}
static int says(int rc, int want, const char* word) { return rc == want && strstr(kt_rawint4_last_error(), word); }

int main(void) {
  kt_router r = {.num_experts = 8, .top_k = 2, .num_groups = 1, .top_groups = 1, .group_top = 1,
                 .score = KT_SCORE_SIGMOID, .renormalize = 1, .scale = 2.5f, .logits_type = KT_TYPE_F32};
  check(kt_router_fwd(&r, 0, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL) == KT_RAWINT4_OK, "routing no tokens");
  check(kt_router_bwd(&r, 0, NULL, NULL, NULL, NULL, NULL) == KT_RAWINT4_OK, "gradient of no tokens");
  check(says(kt_router_fwd(&r, 4, NULL, NULL, NULL, FAKE, FAKE, NULL, 0, NULL), KT_RAWINT4_EINVAL, "non-NULL"),
        "routing without logits refused");
  check(says(kt_router_fwd(NULL, 4, FAKE, NULL, NULL, FAKE, FAKE, NULL, 0, NULL), KT_RAWINT4_EINVAL, "router"),
        "routing without a router refused");
  r.num_groups = 3;
  check(says(kt_router_bwd(&r, 4, FAKE, FAKE, FAKE, FAKE, NULL), KT_RAWINT4_EINVAL, "num_groups"),
        "groups that do not divide the experts refused");
  check(says(kt_router_update_bias(FAKE, FAKE, 8, NAN, NULL), KT_RAWINT4_EINVAL, "rate"), "a rate of NaN refused");

  check(kt_ckpt8_pack(NULL, 0, 64, KT_CKPT8_INT8, NULL, NULL, NULL) == KT_RAWINT4_OK, "packing no rows");
  check(says(kt_ckpt8_unpack(FAKE, FAKE, 4, 64, 2, FAKE, NULL), KT_RAWINT4_EINVAL, "format"), "a third format refused");
  check(says(kt_ckpt8_pack(FAKE, -1, 64, KT_CKPT8_E4M3, FAKE, FAKE, NULL), KT_RAWINT4_EINVAL, "rows"),
        "negative rows refused");

  kt_linear l = {.in_features = 2048, .out_features = 384, .activation = KT_ACT_SILU, .weight = FAKE, .bias = NULL};
  const size_t fwd = kt_linear_workspace_bytes(&l, 300), rows = kt_linear_bwd_workspace_bytes(&l, 300, 0),
               ck = kt_linear_bwd_workspace_bytes(&l, 300, 1);
  check(fwd > 0 && fwd % 256 == 0 && rows > 0, "workspaces of a dense layer");
  check(ck == rows + 300u * 2048u * 2u, "a checkpoint's rows lie behind the rest");
  check(kt_linear_workspace_bytes(&l, 1) == 0 && kt_rawint4_last_error()[0] == 0, "one token needs no workspace");
  check(kt_linear_fwd(&l, 0, NULL, NULL, NULL, KT_TYPE_BF16, NULL, NULL, 0, NULL) == KT_RAWINT4_OK, "no tokens");
  check(says(kt_linear_fwd(&l, 300, FAKE, NULL, FAKE, KT_TYPE_BF16, NULL, FAKE, fwd - 256, NULL),
             KT_RAWINT4_EWORKSPACE, "smaller"),
        "a small workspace refused");
  const kt_ckpt8 c = {.format = KT_CKPT8_INT8, .codes = FAKE, .scales = FAKE};
  check(says(kt_linear_bwd(&l, 300, FAKE, &c, FAKE, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, NULL, 0, 1.f, FAKE, ck, NULL),
             KT_RAWINT4_EINVAL, "not both"),
        "inputs given twice refused");
  check(says(kt_linear_bwd(&l, 300, FAKE, NULL, NULL, FAKE, KT_TYPE_F32, NULL, FAKE, FAKE, NULL, 0, 1.f, FAKE, ck, NULL),
             KT_RAWINT4_EINVAL, "preact"),
        "an activation's gradient without its inputs refused");
  l.in_features = 12;
  check(kt_linear_workspace_bytes(&l, 300) == 0 && strstr(kt_rawint4_last_error(), "in_features"),
        "rows that are no multiple of 16 bytes refused");
  return fails != 0;
}
