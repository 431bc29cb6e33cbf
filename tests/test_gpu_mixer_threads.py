"""Two host threads in the same kernel with calls of very different shared memory: neither call may fail, nor change.

The calls go through the C interface with their arguments laid out beforehand (a call releases the interpreter's lock), as
a program without an interpreter makes them."""
import threading

import pytest
import torch

from gated_deltanet_chunked_delta_gb300 import layer as L
from test_gpu_layer import gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
CALLS = 4000


def both(lib_call, calls):
    """Each of `calls` (arguments, outputs) over and over on a stream and a thread of its own."""
    for args, _ in calls:
        assert lib_call(args, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, outs in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    start, codes = threading.Barrier(len(calls)), [None] * len(calls)

    def run(i):
        args, stream = calls[i][0], streams[i].cuda_stream
        start.wait()
        codes[i] = sum(lib_call(args, stream) != 0 for _ in range(CALLS))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [0] * len(calls)  # calls that failed
    for w, (_, outs) in zip(want, calls):
        assert all(torch.equal(a, b) for a, b in zip(w, outs))


def linear_call(gen, T, D, backward):
    x, i, r, dy = (rand(gen, 1, T, D) for _ in range(4))
    decay = rand(gen, D) - 3
    head = L._linear_head(x, i, r, decay, None, 8.0, None, None, 1)
    lib = L._calls()
    size = max(lib.gdr_linear_fwd_workspace_size(1, T, D), lib.gdr_linear_bwd_workspace_size(1, T, D))
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    y, states = torch.empty_like(x), torch.empty(1, -(-T // L.LINEAR_STRIDE), D, device="cuda")
    args = L._LINEAR.pack(*head, y.data_ptr(), 0, states.data_ptr(), *[0] * 8, ws.data_ptr(), ws.numel())
    if not backward:
        return args, [y, states], (x, i, r, decay, ws)
    assert lib.gdr_linear_fwd(args, torch.cuda.current_stream().cuda_stream) == 0
    outs = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(decay)]
    args = L._LINEAR.pack(*head, 0, 0, states.data_ptr(), dy.data_ptr(), 0, *(t.data_ptr() for t in outs[:3]), 0, outs[3].data_ptr(), 0,
                          ws.data_ptr(), ws.numel())
    return args, outs, (x, i, r, dy, decay, ws, states)


@pytest.mark.parametrize("backward", [False, True])
def test_scans_of_two_threads(gdr, backward):  # noqa: F811
    """One warp with tokens in a CTA, and twelve with two or three tiles each."""
    gen = gen_of(101)
    calls = [linear_call(gen, T, 512, backward) for T in (5, 3000)]
    lib = L._calls()
    both(lib.gdr_linear_bwd if backward else lib.gdr_linear_fwd, [c[:2] for c in calls])


def test_norm_gradients_of_two_threads(gdr):  # noqa: F811
    """CTAs of 64 threads and of 256, which run the same kernel."""
    gen, lib, calls, kept = gen_of(102), L._calls(), [], []
    for M, D in ((40, 1024), (400, 4096)):
        x, gate, res, dy, dr = (rand(gen, M, D).bfloat16() for _ in range(5))
        w, w2 = 1 + 0.1 * rand(gen, D), 1 + 0.1 * rand(gen, D)
        head = L._block_head(x, w, gate, res, w2, 0.5, 1e-6)
        y, r = torch.empty_like(x), torch.empty_like(x)
        stats = torch.empty(M, 2, device="cuda")
        assert lib.gdr_block_norm_fwd(L._BLOCK_NORM.pack(*head, r.data_ptr(), y.data_ptr(), stats.data_ptr(), *[0] * 9),
                                      torch.cuda.current_stream().cuda_stream) == 0
        size = lib.gdr_block_norm_bwd_workspace_size(M, D)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(w) for _ in range(2)]
        calls.append((L._BLOCK_NORM.pack(*head, 0, 0, stats.data_ptr(), dr.data_ptr(), dy.data_ptr(), *(t.data_ptr() for t in outs),
                                         ws.data_ptr(), size), outs))
        kept.append((x, gate, res, dy, dr, w, w2, stats, ws))
    both(lib.gdr_block_norm_bwd, calls)
