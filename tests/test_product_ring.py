"""The E4M3 product's ring of steps (afx_ring.h, afx_fp8.cu), on the CPU: every
order in which a CTA's copies, products and sums can come.

A CTA's loads go into a ring of slots, one after the other; two warps issue the
products, each every second step, into four buffers of sums.  A warp tests the
barriers of its step's copy and of its buffer side by side, so neither's
result is behind the other's.  A wait for a barrier knows a phase by its parity
alone: it also passes while the phase before the one that is meant is open.
"""
import os
import shutil
import subprocess

import pytest

BUFS, WARPS = 4, 2
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_streaming_canonical_gb300", "csrc")


def _reads_an_unloaded_slot(stages, steps):
    """Whether some order of events lets a product be issued on a slot whose copy has not come.

    A state: loads begun; loads done (bits), each warp's step, which of its two waits it has through (bits), products
    done (bits), sums read.  Copies and products end in any order; sums are read step by step."""
    start = (0, 0, (0, 1), (0, 0), 0, 0)
    seen, todo = {start}, [start]
    put = lambda pair, w, v: (v, pair[1]) if w == 0 else (pair[0], v)  # noqa: E731
    while todo:
        begun, done, at, through, multiplied, read = todo.pop()
        after = []
        # a load begins once its slot's last product is done
        if begun < steps and (begun < stages or multiplied >> (begun - stages) & 1):
            after.append((begun + 1, done, at, through, multiplied, read))
        for s in range(begun):  # a copy comes
            if not done >> s & 1:
                after.append((begun, done | 1 << s, at, through, multiplied, read))
        for s in range(steps):  # a product is done: it was issued if its warp is past it
            if at[s % WARPS] > s and not multiplied >> s & 1:
                after.append((begun, done, at, through, multiplied | 1 << s, read))
        if read < steps and multiplied >> read & 1:
            after.append((begun, done, at, through, multiplied, read + 1))
        for w in range(WARPS):
            it = at[w]
            if it >= steps:
                continue
            if through[w] == 3:
                if not done >> it & 1:
                    return True
                after.append((begun, done, put(at, w, it + WARPS), put(through, w, 0), multiplied, read))
                continue
            loaded = sum(done >> s & 1 for s in range(it % stages, steps, stages))  # phases that the slot has been through
            emptied = sum(1 for s in range(it % BUFS, read, BUFS))
            if not through[w] & 1 and loaded % 2 != it // stages % 2:
                after.append((begun, done, at, put(through, w, through[w] | 1), multiplied, read))
            if not through[w] & 2 and (it < BUFS or emptied % 2 != (it // BUFS - 1) % 2):
                after.append((begun, done, at, put(through, w, through[w] | 2), multiplied, read))
        for state in after:
            if state not in seen:
                seen.add(state)
                todo.append(state)
    return False


def _counts(tmp_path):
    """The stages of every ring that a product of 1 to 128 tokens' tiles gets, by the library's own rule."""
    compiler = shutil.which("g++")
    if not compiler:
        pytest.skip("g++ not available")
    src = tmp_path / "ring.cpp"
    src.write_text("""#include "afx_ring.h"
#include <cstdio>
#include <initializer_list>
int main() {  // W's rows of a tile, rows of staging or none, tokens of a tile
    for (unsigned n : {64u, 128u})
        for (unsigned staging : {0u, 8u * 32 * 33 * 4})
            for (unsigned box = 8; box <= 128; box += 8)
                std::printf("%u\\n", afx::serve::ring_stages(232448 - 1024 - 5120 - (128 - box) * 128 - staging, (n + box) * 128, 16, 2));
}
""")
    exe = str(tmp_path / "ring")
    subprocess.run([compiler, "-std=c++17", "-I", CSRC, str(src), "-o", exe], check=True)
    return sorted({int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()})


def test_products_wait_for_their_copies(tmp_path):
    counts = _counts(tmp_path)
    assert counts[0] >= 2
    for stages in sorted({min(n, 8) for n in counts}):  # more are like eight: the buffers of sums hold the warps back
        assert not _reads_an_unloaded_slot(stages, 2 * stages + 3), stages


def test_a_ring_of_five_does_not():
    assert _reads_an_unloaded_slot(5, 9)
