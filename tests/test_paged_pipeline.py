"""The row-tile kernel's waits, on the CPU: a model of its warps (tile copies, products, the warp that answers for landed
tiles, softmax) with the ring's slots and the barriers between them, run until nobody can go on; and the rule that a
warp's lanes act on one outcome of a wait."""

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_matmul_lwq_b200",
                      "csrc", "lwq_paged_tile.cuh")


def source():
    with open(SOURCE) as f:
        return f.read()


def pipeline_ends(stages, cnt):
    """True when every agent ends; cnt: key tiles of the two row tiles.  A copy i is tile i // 2's keys (even) or values;
    events are strings in a set, each agent a generator that yields the event it waits for."""
    n, done = max(cnt), set()

    def copies():
        for i in range(2 * n):
            if i >= stages:
                yield f"empty {i - stages}"
            done.add(f"full {i}")

    def answers():
        for j in range(n):
            yield f"full {2 * j + 1}"
            if j + 1 < n:
                yield f"full {2 * j + 2}"
            for t in (0, 1):
                if j < cnt[t]:
                    if j > 0:
                        yield f"first {t} {j - 1}"
                    done.add(f"answer {t} {j}")

    def softmax(t):
        for j in range(cnt[t]):
            yield f"scores {t} {j}"
            done.add(f"first {t} {j}")
            done.add(f"second {t} {j}")
        if cnt[t]:
            yield f"result {t}"

    def products():
        if not n:
            return
        yield "full 0"
        for t in (0, 1):
            if cnt[t]:
                done.add(f"scores {t} 0")
        back = [0]
        for j in range(n):
            for t in (0, 1):
                if j >= cnt[t]:
                    continue
                yield f"first {t} {j}"
                yield f"answer {t} {j}"
                for i in back:
                    done.add(f"empty {i}")
                back = []
                yield f"second {t} {j}"
                done.add(f"scores {t} {j + 1}" if j + 1 < cnt[t] else f"result {t}")
            back = [2 * j + 1] + ([2 * j + 2] if j + 1 < n else [])

    agents = {a: None for a in (copies(), answers(), softmax(0), softmax(1), products())}
    for a in agents:
        agents[a] = next(a, "end")
    moved = True
    while moved:
        moved = False
        for a, want in agents.items():
            while want != "end" and want in done:
                want = next(a, "end")
                moved = True
            agents[a] = want
    return all(want == "end" for want in agents.values())


COUNTS = [(0, 0), (1, 0), (1, 1), (2, 1), (1, 2), (2, 2), (3, 5), (5, 3), (9, 9), (9, 0), (40, 41)]


def test_three_slots_are_too_few():
    """V_j and K_(j+1) have to land before tile j's products, which alone hand back the slot of V_(j-1)."""
    assert not all(pipeline_ends(3, c) for c in COUNTS)


@pytest.mark.parametrize("stages", [4, 5, 6, 7, 8])
def test_four_slots_and_more_end(stages):
    assert all(pipeline_ends(stages, c) for c in COUNTS)


def test_the_least_number_of_slots_that_is_compiled_ends():
    least = int(re.search(r"static_assert\(SM::STAGES >= (\d+)", source()).group(1))
    assert all(pipeline_ends(least, c) for c in COUNTS)


def test_a_softmax_warp_acts_on_one_outcome_of_a_wait():
    """A wait that runs out ends with a result, in each lane its own: between the softmax warps' start and end only the
    two waits whose outcome the warp shares are made, or lanes that gave up would leave the others in instructions of
    the whole warp."""
    text = source()
    softmax = text[text.index("regs_inc<TILE_REGS_SOFTMAX>();"):]
    softmax = softmax[:softmax.index("    __syncthreads();\n    if (warp == 1) {")]
    waits = re.findall(r"\b(\w*_wait(?:_near)?)\(", softmax)
    assert waits and set(waits) == {"all_wait", "warp_wait"}
    body = text[text.index("auto all_wait ="):]
    assert "return __all_sync(0xffffffffu, mbar_wait_near(" in body[:body.index("};")]
    body = text[text.index("auto warp_wait ="):]
    assert "if (lane == 0) ok =" in body[:body.index("};")] and "return __shfl_sync(" in body[:body.index("};")]
