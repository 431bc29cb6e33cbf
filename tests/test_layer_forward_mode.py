"""The layer operators refuse inputs with forward-mode tangents, before they look at anything else, and take inputs
without one inside the same level as always."""
import pytest
import torch
from torch.autograd import forward_ad

import gated_deltanet_chunked_delta_gb300 as gdr

x, w, vec = torch.zeros(1, 8, 16), torch.zeros(16, 4), torch.zeros(16)
A, BC, state = torch.zeros(16, 16), torch.zeros(1, 8, 1, 16), torch.zeros(8, 16, 16)

CALLS = {
    "short_conv": (gdr.short_conv, [x, w, vec]),
    "short_conv_step": (gdr.short_conv_step, [x[0], w, torch.zeros(8, 3, 16), vec]),
    "state_space_scan": (gdr.state_space_scan, [x, x, A, BC, BC, vec, x, vec]),
    "state_space_step": (gdr.state_space_step, [x[0], x[0], A, BC[0], BC[0], state, vec, x[0], vec]),
    "residual_rms_norm": (gdr.residual_rms_norm, [x, vec, x]),
    "residual_rms_norm_fp8": (gdr.residual_rms_norm_fp8, [x, vec, x]),
    "block_matmul_fp8": (gdr.block_matmul_fp8, [torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.zeros(1, 4),
                                                torch.zeros(8, 128).to(torch.float8_e4m3fn), torch.zeros(1, 1)]),
}


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_tangents_are_refused(name, grad):
    call, args = CALLS[name]
    with forward_ad.dual_level():
        for i, t in enumerate(args):
            if t.dtype != torch.float32:
                continue
            t = t.clone().requires_grad_(grad)
            with pytest.raises(gdr.GdrError, match="forward-mode"):
                call(*args[:i], forward_ad.make_dual(t, torch.ones_like(t)), *args[i + 1:])
        with pytest.raises(gdr.GdrError, match="GPU"):  # no tangent: the next check speaks
            call(*args)
