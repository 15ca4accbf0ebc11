"""Numbers that are asked for once (afx_known.h): a call that fails is asked again."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_streaming_canonical_gb300", "csrc")

PROGRAM = """#include "afx_known.h"
#include <cstdio>
#include <thread>
#include <vector>
int main() {
    static afx::serve::Known known, none;
    int asked = 0;
    uint64_t v = 5;
    auto fails = [&](uint64_t* to) { ++asked; *to = 77; return false; };
    auto tells = [&](uint64_t* to) { ++asked; *to = 152; return true; };
    auto say = [&](bool told) { std::printf("%d %d %d\\n", told, (int)v, asked); };
    say(known.get(&v, fails));
    say(known.get(&v, fails));
    say(known.get(&v, tells));
    v = 0;
    say(known.get(&v, fails));
    // an answer of none is an answer
    say(none.get(&v, [](uint64_t* to) { *to = 0; return true; }));
    say(none.get(&v, fails));
    static afx::serve::Known shared;
    std::vector<std::thread> threads;
    std::atomic<int> wrong{0};
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] {
            for (int i = 0; i < 1000; ++i) {
                uint64_t got = 0;
                const bool told = shared.get(&got, [&](uint64_t* to) { *to = 9; return (i + t) % 7 == 0; });
                wrong += told ? got != 9 : got != 0;
            }
        });
    for (auto& t : threads) t.join();
    std::printf("%d\\n", wrong.load());
}
"""


def test_a_failure_is_not_kept(tmp_path):
    compiler = shutil.which("g++")
    if not compiler:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "known.cpp", str(tmp_path / "known")
    src.write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", exe], check=True)
    got = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert got == "0 0 1  0 0 2  1 152 3  1 152 3  1 0 3  1 0 3  0".split()
