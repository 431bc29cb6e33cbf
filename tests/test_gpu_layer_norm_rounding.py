"""The 8-bit norm divides: a value that lies on the border of two 8-bit values once divided by its block's scale goes to
the even one, which a product with a rounded reciprocal misses in one case of a few."""
import pytest
import torch

from test_gpu_layer import DT, gdr  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def borders():
    """The borders between neighbouring e4m3 values, subnormal ones included, as exact numbers of five bits."""
    values = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return (values[1:] + values[:-1]) / 2


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [2048, 8192, 2043, 16384])
def test_borders_go_to_the_even_value(gdr, D, dt):  # noqa: F811
    # x = 1 and eps = 0: rstd is 1 and y the weights.  A block's weights are its scale (17 bits, odd) times 448 and
    # times borders, both exact in fp32, so that the scale comes out exact and y / scale is a border.
    gen = torch.Generator().manual_seed(D)
    blocks = -(-D // 128)
    scale = (2 * torch.randint(1 << 15, 1 << 16, (blocks,), generator=gen).double() + 1) * 2.0 ** -17
    line = borders()
    pick = line[torch.randint(0, line.numel(), (blocks, 128), generator=gen)]
    pick[:, 0] = 448
    w64 = (pick * scale[:, None]).flatten()[:D]
    w = w64.float()
    assert torch.equal(w.double(), w64)
    x = torch.ones(3, D, dtype=DT[dt], device="cuda")
    q, scales, _ = gdr.residual_rms_norm_fp8(x, w.cuda(), eps=0.0)
    assert torch.equal(scales.cpu().double(), scale[:, None].expand(blocks, 3))
    want = pick.flatten()[:D].float().to(torch.float8_e4m3fn)
    got = q.cpu()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8).expand(3, D)), int((got[0].view(torch.uint8) != want.view(torch.uint8)).sum())
