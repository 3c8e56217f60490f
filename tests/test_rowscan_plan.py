"""How the log-probabilities' pass cuts its rows (csrc/ce_rowscan_plan.h), on the host:
segments hold every vector, the groups' maxima have room at every place of the queue,
and what a call without room is told."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include "ce_rowscan_plan.h"
using namespace gbce;
int main() {
    printf("%d %d %d %d %d %d\n", kMainThreads, kTileVecs, kTopHeads, kHeadsRoom, kQueue, kSideWarps);
    long long N, V;
    int es, k;
    while (scanf("%lld %lld %d %d", &N, &V, &es, &k) == 4) {
        const ScanPlan p = plan_scan(N, V, es, k);
        printf("%d %lld %d %d\n", p.segs, (long long)p.per, p.places, p.heads);
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    csrc = os.path.join(ROOT, "vocabulary_cross_entropy_pass_gb300", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{csrc}", str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        lines = [tuple(map(int, line.split())) for line in out.splitlines()]
        return lines[0], lines[1:]

    return run


WIDTHS = [1, 3, 7, 8, 100, 300, 4095, 4096, 9001, 16383, 16384, 16385, 16392, 32000, 32768, 32776, 50257, 65536, 100277,
          128000, 131072, 131073, 131080, 151937, 256000, 1 << 20, 1 << 27, (1 << 27) + 8, (1 << 31) - 1]


def test_segments_hold_every_vector_and_every_group(plan):
    cases = [(n, v, es, k) for n in (1, 2, 4, 16, 151, 304, 305, 4096, 70001, (1 << 31) - 1) for v in WIDTHS
             for es in (2, 4) for k in (0, 1, 8, 64, 128, 129, 256) if k <= v]
    (threads, tile, most, room, queue, sides), got = plan(cases)
    assert len(got) == len(cases) and tile == 8 * threads
    refused = 0
    for (n, v, es, k), (segs, per, places, heads) in zip(cases, got):
        at = (n, v, es, k)
        if segs == 0:  # only a list of likeliest tokens needs room, and 1024 segments of 2048 groups have it
            assert k > 0 and v * es // 16 > 1024 * (most // threads) * tile, at
            refused += 1
            continue
        assert 1 <= segs <= 1024 and per >= 1, at
        nv = v * es // 16  # of a row that begins at a 16-byte boundary; no row has more
        assert segs * per >= nv and (segs == 1 or (segs - 1) * per < nv), at
        # a row in the stream beside one with each side warp, and no more than there are
        assert sides < places <= queue, at
        if k == 0:
            continue
        assert heads * places <= room and heads <= most and heads % 8 == 0, at
        # any segment, shorter ones too: a group for each thread of a tile, or, where these are fewer
        # than 2 k and the vectors fit, the vectors up to a multiple of 256
        for have in {per, per - 1, per // 2, min(per, tile), min(per, tile + 1), 1, 0}:
            groups = -(-have // tile) * threads
            assert groups <= heads, (at, have)
            if groups < 2 * k and have <= most:
                assert -(-have // 256) * 256 <= max(heads, groups), (at, have)
    assert refused


def test_few_rows_are_cut_and_many_are_not(plan):
    _, ((few, *_), (many, *_), (one, *_)) = plan([(4, 32000, 2, 20), (4096, 128000, 2, 64), (1, 100, 2, 8)])
    assert few > 1 and many == 1 and one == 1
