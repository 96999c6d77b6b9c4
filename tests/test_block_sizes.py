"""The operators around the experts on the CPU: a workspace sized for the longest
batch serves every shorter one."""

import pytest

import int4_quantized_moe_amd as kt

FAKE = 1 << 20  # a non-null, 256-aligned address; never dereferenced by the size functions


@pytest.mark.parametrize("k,n", [(64, 24), (512, 384), (1024, 1), (2048, 2048), (7168, 384), (7168, 2048), (2048, 7168),
                                 (65536, 8), (8, 65536)])
@pytest.mark.parametrize("act", [0, 2])
def test_workspaces_grow_with_the_tokens(k, n, act):
    lin = kt.kt_linear(k, n, act, FAKE, None)
    tokens = [*range(0, 400), *range(400, 9000, 61), *(128 * r for r in range(1, 160)), *(128 * r + 1 for r in range(1, 160)),
              1 << 15, 1 << 18, 1 << 20]
    last = [0, 0, 0]
    for t in sorted(set(tokens)):
        sizes = [kt.kt_linear_workspace_bytes(lin, t), kt.kt_linear_bwd_workspace_bytes(lin, t),
                 kt.kt_linear_bwd_workspace_bytes(lin, t, True)]
        assert all(a >= b for a, b in zip(sizes, last)), (t, sizes, last)
        last = sizes
