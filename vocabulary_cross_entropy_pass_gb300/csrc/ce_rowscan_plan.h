// ce_rowscan_plan.h -- how a pass over rows of logits cuts them into segments, and
// the limits of its lists.  Host arithmetic on sizes alone, without CUDA: the
// workspace's size, the launches and the tests go by the same plan.
#pragma once

#include <stdint.h>

namespace gbce {

constexpr int kMainThreads = 256;                            // threads that read a tile
constexpr int kSideWarps = 3;                                // warps beside them
constexpr int kSideThreads = 32 * kSideWarps;
constexpr int kRowThreads = kMainThreads + 32 + kSideThreads;  // and the copying warp
constexpr int kTileVecs = kMainThreads * 8;                  // 16-byte vectors of a tile: 32 KB
constexpr int kTopCap = 1024;                                // candidates held at a time
constexpr int kTopHeads = 2048;                              // groups' maxima of a row or segment at most
constexpr int kQueue = 6;                                    // rows or segments a CTA has begun at most
constexpr int kHeadsRoom = 4 * kTopHeads;                    // for theirs
constexpr int kMaxTop = 256;                                 // likeliest tokens a call may ask for
constexpr int kMaxListed = 1024;                             // given or teacher's tokens of a row
constexpr int kMaxSegments = 1024;
constexpr int64_t kSMs = 152;
constexpr int64_t kScanSlots = 2 * kSMs;                     // CTAs that run at a time

struct ScanPlan {
    int segs;      // segments of a row
    int64_t per;   // whole vectors in a segment
    int places;    // of the queue of rows or segments that are begun
    int heads;     // room for groups' maxima at each
};

// Rows are cut where that ends sooner: the rounds of kScanSlots CTAs times a segment's
// tiles and what it costs beside them (four tenths of a tile's time), and one tile's time
// for putting segments together.  A segment's groups' maxima have to have room; segs is 0
// where they have none.
inline ScanPlan plan_scan(int64_t N, int64_t V, int es, int top_k) {
    const int64_t nv = V * es / 16;
    const int64_t parts = nv / (kTileVecs / 2);  // of 16 KB at least
    int64_t segs = 1;
    double least = 0;
    for (int64_t s = 1; s <= 64 && s <= (parts > 1 ? parts : 1) && N > 0 && N < 64 * kScanSlots; ++s) {
        const double rounds = (double)((N * s + kScanSlots - 1) / kScanSlots);
        const double time = rounds * ((double)nv / kTileVecs / s + 0.4) + (s > 1 ? 1 : 0);
        if (s == 1 || time < least) {
            least = time;
            segs = s;
        }
    }
    const int64_t room = top_k <= 0 ? nv : (int64_t)(kTopHeads / kMainThreads) * kTileVecs;
    if (nv > segs * room) segs = (nv + room - 1) / room;
    ScanPlan p;
    p.per = (nv + segs - 1) / segs;
    if (p.per < 1) p.per = 1;
    p.segs = segs > kMaxSegments ? 0 : (int)segs;
    // A group for each main thread of a tile; where these may be too few for top_k, a short
    // row's vectors are groups.  As many places as the maxima leave: three rows are with the side
    // warps, and one alone to stream ahead leaves the main warps waiting.
    p.heads = 0;
    p.places = kQueue;
    if (top_k > 0 && p.segs > 0) {
        p.heads = 2 * top_k > kMainThreads ? kTopHeads : (int)((p.per + kTileVecs - 1) / kTileVecs) * kMainThreads;
        if (p.places > kHeadsRoom / p.heads) p.places = kHeadsRoom / p.heads;
    }
    return p;
}

}  // namespace gbce
