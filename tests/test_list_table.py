"""The table that finds tokens listed twice (csrc/ce_list_table.h), on the host: entered by threads at once, with
16-bit compare-and-swaps, the only way in which its slots are changed."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vocabulary_cross_entropy_pass_gb300", "csrc")
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <atomic>
#include <map>
#include <random>
#include <thread>
#include <vector>
#include "ce_list_table.h"
using namespace gbce;
int main(int, char** v) {
    const int entries = atoi(v[1]), columns = atoi(v[2]), threads = 8;
    for (int seed = 0; seed < atoi(v[3]); ++seed) {
        std::mt19937 g(seed);
        uint32_t n = 64;
        while (n < 2u * entries) n *= 2;
        std::vector<uint16_t> slots(n, (uint16_t)kSlotFree);
        std::vector<std::atomic<int>> col(entries);
        std::vector<int> was(entries), again(entries, 0);
        for (int k = 0; k < entries; ++k) col[k] = was[k] = (int)(g() % columns) * 977;
        std::atomic<int> begin{0};
        auto work = [&](int t) {
            ++begin;
            while (begin < threads) {}
            auto cas = [&](uint16_t* s, uint32_t expected, uint32_t value) -> uint32_t {
                uint16_t e = (uint16_t)expected;
                __atomic_compare_exchange_n(s, &e, (uint16_t)value, false, __ATOMIC_RELAXED, __ATOMIC_RELAXED);
                return e;
            };
            for (int k = t; k < entries; k += threads)
                if (list_enter(slots.data(), n, k, was[k], [&](int j) { return col[j].load(); }, cas)) {
                    again[k] = 1;
                    col[k] = -2 - was[k];
                }
        };
        std::vector<std::thread> all;
        for (int t = 0; t < threads; ++t) all.emplace_back(work, t);
        for (auto& t : all) t.join();
        std::map<int, int> listed, first;
        for (int k = 0; k < entries; ++k) {
            ++listed[was[k]];
            first[was[k]] += !again[k];
        }
        size_t held = 0;
        for (uint32_t s : slots) {
            if (s == kSlotFree) continue;
            ++held;
            const int k = slot_entry(s);
            if (k >= entries || again[k] || slot_twice(s) != (listed[was[k]] > 1)) return printf("slot of %d\n", k), 1;
        }
        for (auto& f : first)
            if (f.second != 1) return printf("column %d stands %d times\n", f.first, f.second), 1;
        if (held != listed.size()) return printf("%zu slots of %zu columns\n", held, listed.size()), 1;
    }
    puts("ok");
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("table")
    (d / "table.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-pthread", f"-I{CSRC}", str(d / "table.cpp"), "-o", str(d / "table")],
                   check=True)
    return str(d / "table")


@pytest.mark.parametrize("entries,columns", [(1, 1), (2, 1), (65, 3), (300, 40000), (1024, 1), (1024, 61),
                                             (1024, 1500), (1024, 32000)])
def test_entered_at_once(program, entries, columns):
    r = subprocess.run([program, str(entries), str(columns), "150"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_one_width():
    """The kernels reach the slots through list_enter and its compare-and-swap of one slot."""
    for name in ("ce_softgrad.cu", "ce_distill.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert "list_enter(" in text and "slot_cas" in text
        for line in text.splitlines():
            assert not ("atomic" in line and "slot" in line), line
