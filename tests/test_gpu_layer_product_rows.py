"""The product takes what the 8-bit norm returns, whatever dimensions the norm's input had."""
import pytest
import torch

from test_gpu_layer import gdr, gen_of, operands, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lead", [(), (3,), (2, 5), (2, 3, 4), (2, 0)])
def test_rows_of_any_dimensions(gdr, lead):  # noqa: F811
    gen = gen_of(50)
    x, w = rand(gen, *lead, 272, dt=torch.bfloat16), rand(gen, 272)
    _, _, b, sb = operands(gen, 1, 200, 272)
    q, scales, _ = gdr.residual_rms_norm_fp8(x, w)
    out = gdr.block_matmul_fp8(q, scales, b, sb)
    assert out.shape == (*lead, 200)
    assert torch.equal(out.reshape(-1, 200), gdr.block_matmul_fp8(q.reshape(-1, 272), scales, b, sb))


def test_refusals_of_shapes(gdr):  # noqa: F811
    a, sa, b, sb = operands(gen_of(51), 6, 64, 256)
    with pytest.raises(gdr.GdrError):
        gdr.block_matmul_fp8(a.view(2, 3, 256), sa[:, :3].contiguous(), b, sb)  # scales of three rows for six
    with pytest.raises(gdr.GdrError):
        gdr.block_matmul_fp8(a.view(2, 3, 256).transpose(0, 1), sa, b, sb)  # not contiguous
    with pytest.raises(gdr.GdrError):
        gdr.block_matmul_fp8(a.view(2, 3, 256)[..., :128], sa, b, sb)
    with pytest.raises(gdr.GdrError):
        gdr.block_matmul_fp8(a[0, 0], sa, b, sb)
    with pytest.raises(gdr.GdrError):
        gdr.block_matmul_fp8(a, sa, b[None], sb)
    with pytest.raises(gdr.GdrError):
        gdr.block_matmul_fp8(a, sa, b[:0], sb[:0])  # no columns
