"""The block-scaled product over enough k blocks and tiles that every ring of every tile form goes round: operand stages,
accumulators, scale slots, and the walk from tile to tile.  Forms at 152 SMs beside the sizes.

Bound: half a step of the output's type and c of the terms' magnitudes: 2^-20 for a block's MMAs and scales, 2^-24 for
each block added and each part of a split."""
import pytest
import torch

from test_gpu_layer import DT, U, gdr, gen_of, operands  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

LONG = [
    (16, 1000, 32784),   # 16 tokens, eight CTAs on a tile's 257 blocks
    (20, 300, 33008),    # 32 tokens, eight CTAs on 258 blocks
    (64, 40000, 2064),   # 64 tokens, 313 tiles of 17 blocks on 304 CTAs
    (128, 512, 4112),    # 128 x 64, 33 blocks
    (19500, 64, 4112),   # 128 x 64, two CTAs an SM
    (511, 4096, 4112),   # 128 x 128, 33 blocks
    (300, 10100, 2064),  # 128 x 128, 237 tiles of 17 blocks on 152 CTAs
    (700, 4000, 4112),   # pairs on 256 x 256, 33 blocks
    (2300, 5000, 2064),  # pairs, 180 tiles of 17 blocks on at most 76
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", LONG)
def test_product_goes_round_its_rings(gdr, M, N, K, out):  # noqa: F811
    a, sa, b, sb = operands(gen_of(M + N + K), M, N, K)
    got = gdr.block_matmul_fp8(a, sa, b, sb, out_dtype=DT[out])
    torch.cuda.synchronize()
    gdr.check_status()
    blocks = -(-K // 128)
    af = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :K]
    c = 2.0 ** -20 + (blocks + 4) * 2.0 ** -24
    for n in range(0, N, 4096):  # a part of the weights at a time: 64-bit operands are large
        part = slice(n, min(n + 4096, N))
        bf = b[part].double() * sb.double().repeat_interleave(128, 0)[part].repeat_interleave(128, 1)[:, :K]
        ref, mag = af @ bf.t(), af.abs() @ bf.abs().t()
        off = (got[:, part].double() - ref).abs()
        assert (off <= U[DT[out]] * ref.abs() + c * mag).all(), float((off / mag).max())
