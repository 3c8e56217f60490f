// ce_logits_plan.h -- how the logits operator cuts its rows, and what its list
// kernel holds in shared memory.  Host arithmetic on sizes alone, without CUDA: the
// workspace's size, the launches and the tests go by the same plan.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gbce {

constexpr int kLogitThreads = 256;
constexpr int kFusedCols = 4096;       // columns of a CTA that reads the lists itself, at most
// Up to 2^21 columns the CTAs read the lists themselves: 16 rows of 128000 under a
// mask with histories of 1000 / 8000 tokens 6.8 / 11.8 us against 10.3 / 14.1
// with tables; 30 rows 10.9 / 19.2 against 11.2 / 15.9.
constexpr int64_t kFusedColumns = 1 << 21;
constexpr size_t kListBytes = 200 * 1024;  // shared memory of the list kernel, at most

struct LogitSizes {
    int64_t N, V, hist_max, bias_max;
    int cols, runs;        // a CTA's run of columns (a multiple of 128) and the runs of a row
    int parts, part_runs;  // parts of a row with a table each (one but for the longest lists), runs in a part
    int entries;           // room of a table: min(history + biases, the part's columns), a multiple of 4
    int slots;             // list kernel: keys of biased entries, a power of two, or 0: sums go by entry
    int sums;              // list kernel: summed biases, one to a slot or to an entry
};

inline size_t list_bytes(const LogitSizes& a) {
    const int64_t words = (int64_t)a.part_runs * a.cols / 32;
    return (size_t)(words + a.entries + a.slots + a.sums) * 4 + (size_t)(words + a.entries) * 2;
}

// The parts of a row at the present runs; whether a part's table fits.
inline bool plan_parts(LogitSizes& a) {
    const int64_t list = a.hist_max + a.bias_max;
    a.runs = (int)((a.V + a.cols - 1) / a.cols);
    for (int64_t per = a.runs;; per = (per + 1) / 2) {
        a.part_runs = (int)per;
        a.parts = (int)((a.runs + per - 1) / per);
        const int64_t cols = per * a.cols, most = list < cols ? list : cols;
        if (most <= 65532) {
            a.entries = (int)((most + 3) / 4 * 4);  // what follows them holds vectors
            // few biases beside many entries are found by a key; else each entry has a
            // sum of its own, which takes less
            const int64_t biased = a.bias_max < cols ? a.bias_max : cols;
            int slots = 32;
            while (slots < 2 * biased) slots *= 2;
            const bool keyed = biased > 0 && 2 * slots < a.entries;
            a.slots = keyed ? slots : 0;
            a.sums = biased > 0 ? (keyed ? slots : a.entries) : 0;
            if (list_bytes(a) <= kListBytes) return true;
        }
        if (per == 1) return false;
    }
}

// The runs of columns and, for many columns in all, the tables: whether there are any.
inline bool plan_logits(LogitSizes& a, int es) {
    const int64_t list = a.hist_max + a.bias_max;
    const bool tables = list > 0 && a.N * a.V > kFusedColumns;
    a.parts = 1;
    a.entries = a.slots = a.sums = 0;
    // a run of eight vectors a thread; sixteen where that still fills the GPU's
    // places several times over (gradient of 4096 rows of 50257 columns 182 ->
    // 179 us; 512 rows of 128000, twice, 77 -> 81 us)
    a.cols = list > 0 && !tables ? kFusedCols : kLogitThreads * 8 * 16 / es;
    if (a.N * ((a.V + 2 * a.cols - 1) / (2 * a.cols)) >= 6 * 912 && a.cols != kFusedCols) a.cols *= 2;
    // few columns in all: shorter runs on more SMs
    while (a.cols > 1024 && a.N * ((a.V + a.cols - 1) / a.cols) < 304) a.cols /= 2;
    a.part_runs = a.runs = (int)((a.V + a.cols - 1) / a.cols);
    if (!tables) return false;
    // a table of a run's every column takes ten bytes each: shorter runs where that
    // does not fit (16384 columns do)
    while (!plan_parts(a)) a.cols /= 2;
    return true;
}

}  // namespace gbce
