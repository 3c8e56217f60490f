"""How the logits operator cuts its rows (csrc/ce_logits_plan.h), on the host: the
list kernel's shared memory stays within what a CTA can have, and the tables hold
every column that the lists can touch, whatever the sizes."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include "ce_logits_plan.h"
using namespace gbce;
int main() {
    LogitSizes a;
    long long N, V, hist, bias;
    int es;
    while (scanf("%lld %lld %lld %lld %d", &N, &V, &hist, &bias, &es) == 5) {
        a = LogitSizes();
        a.N = N; a.V = V; a.hist_max = hist; a.bias_max = bias;
        const int tables = plan_logits(a, es);
        printf("%d %d %d %d %d %d %d %d %zu\n", tables, a.cols, a.runs, a.parts, a.part_runs, a.entries, a.slots,
               a.sums, tables ? list_bytes(a) : (size_t)0);
    }
}
"""
OPT_IN = 227 * 1024  # shared memory a CTA can have, its static part included


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    csrc = os.path.join(ROOT, "vocabulary_cross_entropy_pass_gb300", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{csrc}", str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


def cases():
    rows = [1, 3, 16, 17, 33, 100, 304, 512, 700, 1400, 2048, 4096, 70001, 4294836225]
    widths = [1, 100, 4096, 32000, 50257, 128000, 256000, 1 << 20, (1 << 31) - 1]
    lists = [(0, 0), (1, 0), (0, 1), (4096, 64), (0, 300), (8192, 300), (0, 4097), (0, 8192), (0, 8193), (0, 20000),
             (8192, 8192), (32768, 1025), (70000, 2048), (70000, 0), (65533, 0), (0, 128000), (500000, 500000),
             (1 << 30, 0), (0, 1 << 30), (1 << 30, 1 << 30)]
    return [(n, v, h, b, es) for n in rows for v in widths for h, b in lists for es in (2, 4)]


def test_plan_fits_and_holds_every_column(plan):
    given = cases()
    got = plan(given)
    assert len(got) == len(given)
    seen = set()
    for (n, v, hist, bias, es), (tables, cols, runs, parts, part_runs, entries, slots, sums, size) in zip(given, got):
        at = (n, v, hist, bias, es)
        assert cols % 128 == 0 and cols & (cols - 1) == 0 and 1024 <= cols <= 65536, at
        assert (runs - 1) * cols < v <= runs * cols, at
        assert part_runs >= 1 and (parts - 1) * part_runs < runs <= parts * part_runs, at
        if not tables:
            assert hist + bias == 0 or n * v <= 1 << 21, at
            continue
        assert hist + bias > 0 and n * v > 1 << 21, at
        assert 0 < size <= OPT_IN - 1024, at
        assert entries % 4 == 0 and entries <= 65535, at
        assert entries >= min(hist + bias, part_runs * cols), at
        if bias == 0:
            assert slots == sums == 0, at
        elif slots:
            # room for every biased entry and an empty slot to stop at
            assert slots & (slots - 1) == 0 and slots == sums and slots > min(bias, part_runs * cols), at
        else:
            assert sums == entries, at
        seen.add((parts > 1, bool(slots), bool(sums)))
    assert {(False, True, True), (True, True, True), (False, False, True), (True, False, True)} <= seen


def test_plan_of_ordinary_lists(plan):
    # a decoding batch: one table a row, the few biases by their keys
    (got,) = plan([(512, 128000, 4096, 64, 2)])
    assert got[0] == 1 and got[3] == 1 and got[5] == 4160 and got[6] == got[7] == 128


def test_workspace_follows_the_plan(plan):
    from vocabulary_cross_entropy_pass_gb300 import _lib, build
    build.build()
    lib = _lib.load()
    for n, v, hist, bias, es in cases()[::7]:
        if n > 1 << 20:  # more bytes than 64 bits count
            continue
        (p,) = plan([(n, v, hist, bias, es)])
        need = lib.ce_logits_workspace_bytes(n, v, 0 if es == 4 else 1, hist, bias)
        pad = lambda x: -(-x // 256) * 256  # noqa: E731
        table = pad(n * p[3] * p[5] * 8)
        assert need == (pad(n * p[2] * 8) + table + (table // 2 if bias else 0) if p[0] else 0)
    assert lib.ce_logits_workspace_bytes(65535 * 65535 + 1, 10, 1, 5, 0) == 0
    assert lib.ce_logits_workspace_bytes(100, 128000, 1, (1 << 30) + 1, 0) == 0
