// ce_rowscan_plan.h -- how a pass over rows of logits cuts them into segments, and
// the limits of its lists.  Host arithmetic on sizes alone, without CUDA: the
// workspace's size, the launches and the tests go by the same plan.
#pragma once

#include <stdint.h>

namespace gbce {

constexpr int kScanThreads = 256;                            // threads that read a tile
constexpr int kScanVecs = 4;                                 // 16-byte vectors of it a thread takes
constexpr int kScanTileVecs = kScanThreads * kScanVecs;      // 16 KB
constexpr int kTopCap = 4096;                                // candidates held at a time
constexpr int kMaxTop = 256;                                 // likeliest tokens a call may ask for
constexpr int kMaxListed = 1024;                             // given or teacher's tokens of a row
constexpr int kMaxSegments = 64;
constexpr int64_t kScanSlots = 304;                          // CTAs that run at a time: two on each of 152 SMs

struct ScanPlan {
    int segs;      // segments of a row
    int64_t per;   // whole vectors in a segment
};

// Few rows are cut so that every SM has a part; from four rounds of whole rows on
// a row stays in one piece.
inline ScanPlan plan_scan(int64_t N, int64_t V, int es) {
    const int64_t nv = V * es / 16;
    const int64_t tiles = (nv + kScanTileVecs - 1) / kScanTileVecs;
    int64_t segs = 1;
    if (N > 0 && N < 4 * kScanSlots) segs = (4 * kScanSlots + N - 1) / N;
    if (segs > tiles) segs = tiles;
    if (segs > kMaxSegments) segs = kMaxSegments;
    if (segs < 1) segs = 1;
    ScanPlan p;
    p.per = (nv + segs - 1) / segs;
    if (p.per < 1) p.per = 1;
    p.segs = (int)segs;
    return p;
}

}  // namespace gbce
