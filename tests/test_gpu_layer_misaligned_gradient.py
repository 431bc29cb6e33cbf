"""A gradient of the final state that lies anywhere in memory: autograd hands it over as the loss made it."""
import pytest
import torch

from test_gpu_layer import gdr, rand, gen_of, scan_inputs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [1, 2, 3])
def test_scan_takes_a_misaligned_gradient_of_its_state(gdr, off):  # noqa: F811
    v, dy, dht = scan_inputs((2, 40, 24, 1, 16, None, True, True, True, True, True), "f32")
    leaves = [t.requires_grad_() for t in v.values()]
    flat = torch.zeros(dht.numel() + 4, device="cuda")
    moved = flat[off:off + dht.numel()].view(dht.shape)
    moved.copy_(dht)
    assert moved.data_ptr() % 16 and moved.is_contiguous()
    got, want = (torch.autograd.grad(gdr.state_space_scan(**v, output_final_state=True), leaves, [dy, g]) for g in (moved, dht))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("off", [1, 3])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_conv_and_norm_take_misaligned_gradients(gdr, off, dt):  # noqa: F811
    gen = gen_of(60)
    x, w, n = rand(gen, 2, 9, 32, dt=dt), rand(gen, 32, 4), rand(gen, 32)
    h0 = rand(gen, 2, 3, 32, dt=dt)
    dy, dht = rand(gen, 2, 9, 32, dt=dt), rand(gen, 2, 3, 32, dt=dt)

    def move(t):
        flat = torch.zeros(t.numel() + 4, device="cuda", dtype=dt)
        flat[off:off + t.numel()] = t.flatten()
        return flat[off:off + t.numel()].view(t.shape)

    leaves = [t.requires_grad_() for t in (x, w, h0)]
    got, want = (torch.autograd.grad(gdr.short_conv(x, w, initial_state=h0, output_final_state=True), leaves, g)
                 for g in ([move(dy), move(dht)], [dy, dht]))
    # four channels a thread and one sum the weights' gradient in another order: sums of 18 tokens
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert (got[1] - want[1]).norm() <= 18 * 2.0 ** -24 * 18 ** 0.5 * want[1].norm()
    leaves = [t.detach().requires_grad_() for t in (x, n)]
    got, want = (torch.autograd.grad(gdr.residual_rms_norm(*leaves), leaves, g) for g in ([move(dy), move(dy)], [dy, dy]))
    for a, b, u in zip(got, want, (2.0 ** -7 if dt is torch.bfloat16 else 2.0 ** -20, 2.0 ** -20)):
        assert (a.float() - b.float()).norm() <= u * b.float().norm()  # sums of a row in another order, rounded once
