"""A recurrent layer served in 8 bits, and trained: the layer operators run together.

    python examples/recurrent_block.py

``StateSpaceBlock`` is one layer of a recurrent language model:

    residual stream -> norm in 8 bits -> input projection -> short convolution -> state space scan -> norm in 8 bits
    -> output projection

``prompt`` runs it over packed prompts and fills a cache of recurrent states; ``token`` advances running requests by one
token from that cache; ``train_step`` runs the differentiable forms with 16-bit projections.  ``delta_prompt`` is the
same layer around the chunked gated delta rule, whose q, k and v come from the same convolution.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_chunked_delta_gb300 as gdr  # noqa: E402


def quantise_weight(w):
    """A weight [N, K] once and for all in 8 bits with a scale for each 128 x 128 block."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    big = torch.zeros(nb * 128, kb * 128, device=w.device)
    big[:n, :k] = w
    blocks = big.view(nb, 128, kb, 128)
    scales = blocks.abs().amax((1, 3)).clamp_min(1e-30) / 448
    q = (blocks / scales[:, None, :, None]).reshape(nb * 128, kb * 128)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), scales


class StateSpaceBlock:
    def __init__(self, width=1024, inner=2048, state=16, taps=4, slots=8, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def randn(*s):
            return torch.randn(*s, device=device, generator=gen)

        self.width, self.inner, self.state = width, inner, state
        self.cuts = [inner, inner, inner, state, state]  # x, z, dt, B, C of the input projection
        self.w_in = (randn(sum(self.cuts), width) * width ** -0.5).bfloat16()
        self.w_out = (randn(width, inner) * inner ** -0.5).bfloat16()
        self.norm_in, self.norm_out = torch.ones(width, device=device), torch.ones(inner, device=device)
        self.conv_w, self.conv_b = randn(inner, taps) * taps ** -0.5, torch.zeros(inner, device=device)
        self.A = -torch.arange(1, state + 1, device=device, dtype=torch.float32).repeat(inner, 1)
        self.D = torch.ones(inner, device=device)
        self.dt_bias = torch.full((inner,), -4.0, device=device)
        self.q_in, self.q_out = quantise_weight(self.w_in.float()), quantise_weight(self.w_out.float())
        self.conv_cache = torch.zeros(slots, taps - 1, inner, device=device, dtype=torch.bfloat16)
        self.scan_cache = torch.zeros(slots, inner, state, device=device)

    def _project(self, h, residual):
        a, scales, residual = gdr.residual_rms_norm_fp8(h, self.norm_in, residual)
        x, z, dt, B, C = gdr.block_matmul_fp8(a, scales, *self.q_in).split(self.cuts, dim=-1)  # slices, not copies
        return x, z, dt, B.unsqueeze(-2), C.unsqueeze(-2), residual

    def _out(self, y):
        a, scales, _ = gdr.residual_rms_norm_fp8(y, self.norm_out)
        return gdr.block_matmul_fp8(a, scales, *self.q_out)

    @torch.no_grad()
    def prompt(self, h, residual, cu_seqlens, slots):
        """h, residual [tokens, width] of packed prompts; slots [n_seqs] (long) take their states."""
        x, z, dt, B, C, residual = self._project(h, residual)
        x, conv_state = gdr.short_conv(x[None], self.conv_w, self.conv_b, output_final_state=True, cu_seqlens=cu_seqlens)
        y, scan_state = gdr.state_space_scan(x, dt[None], self.A, B[None], C[None], self.D, z[None], self.dt_bias,
                                             output_final_state=True, cu_seqlens=cu_seqlens)
        self.conv_cache[slots], self.scan_cache[slots] = conv_state, scan_state
        return self._out(y[0]), residual

    @torch.no_grad()
    def token(self, h, residual, slots):
        """h, residual [rows, width]: one token of each running request; slots [rows] int32, negative for an idle row."""
        x, z, dt, B, C, residual = self._project(h, residual)
        x = gdr.short_conv_step(x, self.conv_w, self.conv_cache, self.conv_b, slots=slots)
        y = gdr.state_space_step(x, dt, self.A, B, C, self.scan_cache, self.D, z, self.dt_bias, slots=slots)
        return self._out(y), residual

    def train_step(self, h, residual, target):
        """Gradients of a squared error with 16-bit projections: (loss, {name: gradient})."""
        leaves = {k: getattr(self, k).detach().clone().requires_grad_() for k in
                  ("w_in", "w_out", "norm_in", "norm_out", "conv_w", "conv_b", "A", "D", "dt_bias")}
        p = type("P", (), leaves)
        a, residual = gdr.residual_rms_norm(h, p.norm_in, residual)
        x, z, dt, B, C = (a @ p.w_in.t()).split(self.cuts, dim=-1)
        x, _ = gdr.short_conv(x, p.conv_w, p.conv_b)
        y, _ = gdr.state_space_scan(x, dt, p.A, B.unsqueeze(-2), C.unsqueeze(-2), p.D, z, p.dt_bias)
        y, _ = gdr.residual_rms_norm(y, p.norm_out)
        loss = (residual + y @ p.w_out.t() - target).float().square().mean()
        return loss.detach(), dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


@torch.no_grad()
def delta_prompt(h, weight, gates, conv_w, norm_w, heads, cu_seqlens):
    """Packed prompts through the chunked gated delta rule: q, k, v from one 8-bit projection and the convolution.
    h [tokens, width]; weight, the quantised [3 heads 128, width]; gates (g, beta) [tokens, heads] fp32."""
    a, scales, _ = gdr.residual_rms_norm_fp8(h, norm_w)
    qkv, _ = gdr.short_conv(gdr.block_matmul_fp8(a, scales, *weight)[None], conv_w, cu_seqlens=cu_seqlens)
    q, k, v = (t.unflatten(-1, (heads, 128)).contiguous() for t in qkv.chunk(3, dim=-1))
    q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
    return gdr.chunk_gated_delta_rule(q, k, v, gates[0][None], gates[1][None], output_final_state=True, cu_seqlens=cu_seqlens)


def main():
    block = StateSpaceBlock()
    gen = torch.Generator(device="cuda").manual_seed(1)
    lengths = [37, 1, 90]
    cu = torch.tensor([0, 37, 38, 128], dtype=torch.int32, device="cuda")
    h, residual = (torch.randn(128, block.width, device="cuda", generator=gen).bfloat16() for _ in range(2))
    whole, _ = block.prompt(h, residual, cu, torch.arange(3, device="cuda"))

    # the same prompts without their last token, which then comes as a step: the outputs of the last tokens agree
    last = torch.tensor([n - 1 for n in (37, 38, 128)], device="cuda")
    keep = torch.ones(128, dtype=torch.bool, device="cuda")
    keep[last] = False
    short = torch.tensor([0, 36, 36, 125], dtype=torch.int32, device="cuda")
    block.prompt(h[keep], residual[keep], short, torch.arange(3, device="cuda"))
    step, _ = block.token(h[last], residual[last], torch.arange(3, dtype=torch.int32, device="cuda"))
    off = float((step.float() - whole[last].float()).norm() / whole[last].float().norm())
    print(f"prompts of {lengths} tokens; last tokens as steps: relative difference {off:.1e}")

    loss, grads = block.train_step(*(torch.randn(2, 64, block.width, device="cuda", generator=gen).bfloat16() for _ in range(3)))
    print(f"training step: loss {float(loss):.4f}, gradient norms " + ", ".join(f"{k} {float(g.float().norm()):.2e}" for k, g in grads.items()))

    heads, width = 4, block.width
    weight = quantise_weight(torch.randn(3 * heads * 128, width, device="cuda", generator=gen) * width ** -0.5)
    g = -torch.rand(128, heads, device="cuda", generator=gen)
    o, state = delta_prompt(h, weight, (g, torch.sigmoid(torch.randn(128, heads, device="cuda", generator=gen))),
                            torch.randn(3 * heads * 128, 4, device="cuda", generator=gen) * 0.5, torch.ones(width, device="cuda"), heads, cu)
    gdr.check_status()
    print(f"delta rule over the same prompts: output {tuple(o.shape)}, states {tuple(state.shape)}")
    return off, loss, grads, o


if __name__ == "__main__":
    main()
