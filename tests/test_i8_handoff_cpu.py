"""The hand-over of filled slots in the 8-bit product of CTA pairs, as a model of its two warps' barriers: every
order in which their steps can follow one another is gone through.

A named barrier of two warps completes at its second arrival, whoever made them, and is then as new.  One warp
announces slot i, the other takes it; they meet at one barrier, where both wait.  A slot is filled only after it
was taken a turn before, unless a wait has given up: then the announcing warp goes on at once.
"""
import ctypes

import pytest

import diffusion_transformer_text_block_b200 as moss

S = 3  # slots


def steps(two_sided, total):
    """(announcing warp, taking warp): lists of (kind, barrier, slot).  One-sided: a barrier for each slot of the
    ring, where the announcing warp does not wait."""
    ann, take = [], []
    for i in range(total):
        ann.append(("fill", None, i))
        ann.append(("sync", 0, i) if two_sided else ("arrive", i % S, i))
        take.append(("sync", 0 if two_sided else i % S, i))
    return ann, take


def stuck(two_sided, total, gives_up_at):
    """Whether some order of steps ends with a warp that waits for good, or with two arrivals of one warp at one
    barrier.  From slot gives_up_at on the announcing warp waits for nothing to be filled."""
    warps = steps(two_sided, total)
    taken_after = {}  # slot -> number of steps of the taking warp behind which it is taken
    for n, (kind, bar, i) in enumerate(warps[1]):
        taken_after[i] = n + 1
    # A state: the warps' positions, whether each waits in a barrier, the barriers' arrivals.
    first = (0, 0, None, None, frozenset())
    seen, todo = {first}, [first]
    while todo:
        pos0, pos1, wait0, wait1, bars = todo.pop()
        pos, wait = [pos0, pos1], [wait0, wait1]
        nexts = []
        for w in (0, 1):
            if wait[w] is not None or pos[w] == len(warps[w]):
                continue
            kind, bar, i = warps[w][pos[w]]
            p, q, b = list(pos), list(wait), dict(bars)
            if kind == "fill":
                if i < gives_up_at and i >= S and pos[1] < taken_after[i - S]:
                    continue
                p[w] += 1
            elif bar in b:
                if b[bar] == w:
                    return True  # two arrivals of one warp complete it without the other
                del b[bar]
                p[w] += 1
                if q[1 - w] == bar:
                    q[1 - w] = None
                    p[1 - w] += 1
            else:
                b[bar] = w
                if kind == "sync":
                    q[w] = bar
                else:
                    p[w] += 1
            nexts.append((p[0], p[1], q[0], q[1], frozenset(b.items())))
        if not nexts and (pos[0], pos[1]) != (len(warps[0]), len(warps[1])):
            return True
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return False


@pytest.mark.parametrize("total", [1, S, S + 1, 2 * S, 3 * S + 1])
def test_no_order_of_steps_is_stuck(total):
    for gives_up_at in range(total + 1):
        assert not stuck(True, total, gives_up_at)


def test_the_model_finds_what_a_one_sided_hand_over_does():
    """Without an answer the announcing warp, once a wait has given up, runs a turn ahead: two of its arrivals
    complete a barrier, and the taking warp waits at it for good."""
    assert not stuck(False, 3 * S + 1, 3 * S + 1)
    assert stuck(False, 3 * S + 1, S + 1)


def test_selftest_refusals():
    """Sizes that do not reach the failure, and unknown ones, launch nothing."""
    f, at = moss.lib().moss_selftest_gemm_i8_timeout, [ctypes.c_void_p((i + 1) << 24) for i in range(5)]
    before = moss.launch_count()
    for failure, M, N, K in ((0, 300, 300, 512), (4, 300, 300, 512), (1, 16, 300, 512), (1, 0, 300, 512), (1, 300, 0, 512),
                             (1, 300, 300, 128), (1, 3840, 3840, 512), (2, 300, 300, 512), (3, 2048, 2048, 512)):
        assert f(failure, *at, M, N, K, None) == 1, (failure, M, N, K)
    assert moss.launch_count() == before
