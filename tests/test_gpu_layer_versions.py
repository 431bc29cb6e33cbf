"""The steps write their state as torch's in-place operations do: a backward that saved it raises instead of reading
what the step left there."""
import pytest
import torch

from test_gpu_layer import gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def parts(gen):
    x, BC = rand(gen, 2, 5, 16), rand(gen, 2, 5, 1, 16)
    return x, rand(gen, 16, 4), -1 - rand(gen, 16, 16).abs(), BC, rand(gen, 2, 3, 16), rand(gen, 2, 16, 16)


@pytest.mark.parametrize("view", [False, True])
def test_a_stepped_cache_is_no_longer_the_saved_initial_state(gdr, view):  # noqa: F811
    x, w, A, BC, conv_state, scan_state = parts(gen_of(40))
    if view:  # the steps go through a view of the cache
        conv_step, scan_step = conv_state.view(conv_state.shape), scan_state.view(scan_state.shape)
    else:
        conv_step, scan_step = conv_state, scan_state
    for run, step in (
            (lambda v: gdr.short_conv(v, w, initial_state=conv_state)[0], lambda: gdr.short_conv_step(x[:, 0], w, conv_step)),
            (lambda v: gdr.state_space_scan(v, x, A, BC, BC, initial_state=scan_state)[0],
             lambda: gdr.state_space_step(x[:, 0], x[:, 0], A, BC[:, 0], BC[:, 0], scan_step))):
        v = x.clone().requires_grad_()
        want = torch.autograd.grad(run(v).sum(), v)[0]  # not stepped in between: nothing to complain of
        assert torch.isfinite(want).all()
        y = run(v)
        step()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            torch.autograd.grad(y.sum(), v)


def test_steps_in_inference_mode(gdr):  # noqa: F811
    x, w, A, BC, conv_state, scan_state = parts(gen_of(41))
    want = conv_state.clone(), scan_state.clone()
    y = gdr.short_conv_step(x[:, 0], w, want[0]), gdr.state_space_step(x[:, 0], x[:, 0], A, BC[:, 0], BC[:, 0], want[1])
    with torch.inference_mode():
        for held in ((conv_state.clone(), scan_state.clone()), (conv_state, scan_state)):  # inference tensors, and not
            got = (gdr.short_conv_step(x[:, 0], w, held[0]), gdr.state_space_step(x[:, 0], x[:, 0], A, BC[:, 0], BC[:, 0], held[1]))
            assert all(torch.equal(a, b) for a, b in zip((*held, *got), (*want, *y)))


def test_reading_calls_leave_versions_alone(gdr):  # noqa: F811
    x, w, A, BC, conv_state, scan_state = parts(gen_of(42))
    gdr.short_conv(x, w, initial_state=conv_state, output_final_state=True)
    gdr.state_space_scan(x, x, A, BC, BC, initial_state=scan_state, output_final_state=True)
    assert all(t._version == 0 for t in (x, w, conv_state, scan_state, BC))
