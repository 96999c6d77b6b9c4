"""GPU: equal rows of a dense product's inputs give equal rows of its outputs,
wherever they stand in a batch: what a token gets does not depend on its place.
Each case prints its name first."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[places]", *a, flush=True)


# one-launch tiles of both sizes, tiles with splits, the form for few tokens
@pytest.mark.parametrize("t,k,n", [(16384, 1024, 384), (8192, 2048, 2048), (4096, 1024, 256), (1000, 7168, 384), (40, 512, 384),
                                   (16, 7168, 384), (61, 1024, 100)])
def test_equal_rows_give_equal_rows(dev, t, k, n):
    _say(t, k, n)
    g = torch.Generator().manual_seed(t)
    kinds = 7
    which = (torch.arange(t) % kinds).cuda()
    rows = torch.randn(kinds, k, generator=g).to(BF16).cuda()
    w = (torch.randn(n, k, generator=g) * k**-0.5).to(BF16).cuda()
    lin = dev.DeviceLinear(w)
    y = lin.forward(rows[which].contiguous(), lin.workspace(t), dtype=F32)
    assert torch.equal(y, y[:kinds][which])
    dy = torch.randn(kinds, n, generator=g).cuda()[which].contiguous()
    dx = lin.backward(rows[which].contiguous(), dy, lin.backward_workspace(t), {})
    assert torch.equal(dx, dx[:kinds][which])
