"""The waits of the block-scaled product (csrc/gdr_fp8.cu), as a model on the CPU: every order in which its warps can
run, for every depth of its rings.  No order may leave a warp waiting for ever, overwrite a stage whose MMAs are not
done, or overwrite scales that have not been read.

Roles, each with the number of blocks it is through: the feeding warp (f) waits for a free stage and copies operands;
the scales' warp (s) waits for the same stage, arrives on it where the kernel counts it, and copies scales; the MMA
warp (m) waits for operands and a free accumulator; the tensor core (c) finishes blocks in order; the accumulating
warps (t) wait for the block and its scales, and free the accumulator; they read the last scales (r) after that.
"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_chunked_delta_gb300", "csrc", "gdr_fp8.cu")
DEPTHS = [(6, 2), (6, 4), (3, 2), (4, 2), (5, 2)]  # operand stages, accumulators


def arrivals():
    """How many arrivals free a stage, and whether the scales' warp makes one of them."""
    text = open(SOURCE).read()
    count = int(re.search(r"bar_init\(&empty\[i\], (\d+)\)", text).group(1))
    return count, "bar_arrive(&empty[it % kStages])" in text


def slots():
    return int(re.search(r"kScaleSlots = (\d+)", open(SOURCE).read()).group(1))


def of(done, stage, stages):
    """Blocks 0 .. done - 1 that used the stage."""
    return (done - stage + stages - 1) // stages if done > stage else 0


def explore(stages, bufs, ring, count, scales_arrive, blocks):
    """None, or what goes wrong in some order."""
    def phases(stage, c, s):
        return (of(c, stage, stages) + (of(s, stage, stages) if scales_arrive else 0)) // count

    def free(block, c, s):  # a wait by parity for the stage's turn before this block's
        return block < stages or (phases(block % stages, c, s) & 1) != ((block // stages - 1) & 1)

    start = (0, 0, 0, 0, 0, 0)
    seen, todo = {start}, [start]
    while todo:
        f, s, m, c, t, r = todo.pop()
        nexts = []
        if f < blocks and free(f, c, s):
            if f - stages >= c:
                return f"operands of block {f} over block {f - stages}"
            nexts.append((f + 1, s, m, c, t, r))
        if s < blocks and free(s, c, s):
            if s - ring >= r:
                return f"scales of block {s} over block {s - ring}"
            nexts.append((f, s + 1, m, c, t, r))
        if m < f and (m < bufs or t > m - bufs):
            nexts.append((f, s, m + 1, c, t, r))
        if c < m:
            nexts.append((f, s, m, c + 1, t, r))
        if t < c and t < s and r == t:
            nexts.append((f, s, m, c, t + 1, r))
        if r < t:
            nexts.append((f, s, m, c, t, r + 1))
        if not nexts and (f, s, m, c, t, r) != (blocks,) * 6:
            return f"stuck with {f} blocks fed, {s} scaled, {m} issued, {c} multiplied, {t} taken"
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return None


@pytest.mark.parametrize("stages,bufs", DEPTHS)
def test_no_order_goes_wrong(stages, bufs):
    assert explore(stages, bufs, slots(), *arrivals(), blocks=slots() + 2 * stages) is None


def test_the_model_finds_the_order_that_does():
    """Without the scales' warp's arrival a stage can be emptied twice before that warp looks; with a ring of scales as
    deep as the accumulators a block's scales are overwritten."""
    assert "stuck" in explore(6, 4, 16, 1, False, 24)
    assert "scales" in explore(6, 2, 4, 2, True, 24)
