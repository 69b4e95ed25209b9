"""Which tile counters a launch with claims takes (csrc/rgg_counters.h, plain host code): launches that may overlap on
the GPU never share a set."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ragged_grouped_gemm_02_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <memory>
#include <set>
#include <thread>
#include <vector>
#include "rgg_counters.h"
using namespace rgg;
#define EXPECT(c) do { if (!(c)) { std::printf("failed: %s (line %d)\n", #c, __LINE__); return 1; } } while (0)
int main() {
    auto sets = std::make_unique<CounterSets>();
    // a stream keeps its set; other streams, and captures of the same stream, have their own
    const int a = sets->set_of(7, 0), b = sets->set_of(8, 0), c = sets->set_of(7, 1), d = sets->set_of(7, 2);
    EXPECT(a >= 0 && b >= 0 && c >= 0 && d >= 0);
    EXPECT((std::set<int>{a, b, c, d}.size()) == 4);
    EXPECT(sets->set_of(7, 0) == a && sets->set_of(8, 0) == b && sets->set_of(7, 1) == c && sets->set_of(7, 2) == d);
    EXPECT(sets->set_of(0, 0) >= 0 && sets->set_of(0, 0) == sets->set_of(0, 0));
    // every set goes to one owner; past the last there is none, and the owners keep theirs
    sets = std::make_unique<CounterSets>();
    std::set<int> seen;
    for (int i = 0; i < kCounterSets; ++i) {
        const int s = sets->set_of(1000 + i / 3, i % 3);
        EXPECT(s >= 0 && s < kCounterSets && seen.insert(s).second);
    }
    EXPECT(sets->set_of(5, 0) == -1 && sets->set_of(1000, 9) == -1);
    for (int i = 0; i < kCounterSets; ++i) EXPECT(seen.count(sets->set_of(1000 + i / 3, i % 3)));
    // from several threads at a time
    sets = std::make_unique<CounterSets>();
    std::vector<std::vector<int>> got(8, std::vector<int>(400));
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] { for (int i = 0; i < 400; ++i) got[t][i] = sets->set_of(i, 0); });
    for (auto& t : threads) t.join();
    for (int t = 1; t < 8; ++t) EXPECT(got[t] == got[0]);
    EXPECT((std::set<int>(got[0].begin(), got[0].end()).size()) == 400);
    std::printf("ok\n");
    return 0;
}
"""


def test_counter_sets(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "sets.cc").write_text(PROGRAM)
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(tmp_path / "sets.cc"), "-o",
                        str(tmp_path / "sets")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(tmp_path / "sets")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
