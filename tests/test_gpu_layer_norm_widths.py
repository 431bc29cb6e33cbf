"""The norm at the widths next to its greatest: a row that begins inside a piece of eight then needs one piece more than
16384 channels do.  Nine rows, so that every shift occurs; what the outputs' memory held before is NaN."""
import pytest
import torch

import test_gpu_layer as G
from test_gpu_layer import DT, gdr  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

WIDTHS = [16376, 16377, 16379, 16380, 16381, 16382, 16383, 16384]


def poison(M, D, dt):
    """Memory of the calls' sizes goes back to the allocator full of NaN."""
    for size in (M * D * 4, M * D * DT[dt].itemsize, M * D, 4096 * D):
        held = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del held


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("added", [True, False])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm_of_the_widest_rows(gdr, D, added, dt):  # noqa: F811
    poison(9, D, dt)
    G.test_norm(gdr, 9, D, added, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("added", [True, False])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm_fp8_of_the_widest_rows(gdr, D, added, dt):  # noqa: F811
    poison(9, D, dt)
    G.test_norm_fp8(gdr, 9, D, added, dt)
