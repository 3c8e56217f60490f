// ce_list_table.h -- which entries of a row's list name one column.
//
// An open table of 16-bit slots in shared memory, at least twice as many as entries and a power
// of two.  The first entry to take a slot for its column stands for the column; one that finds it
// there marks the slot.  Slots are changed by 16-bit compare-and-swap alone: atomics of another
// width on a slot's word would not be atomic towards them.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GBCE_TABLE_FN __device__ __forceinline__
#else
#define GBCE_TABLE_FN inline
#endif

namespace gbce {

constexpr uint32_t kSlotFree = 0xffffu;
constexpr uint32_t kSlotTwice = 0x8000u;  // beside the number of the entry that stands for the column

GBCE_TABLE_FN bool slot_twice(uint32_t slot) { return slot != kSlotFree && (slot & kSlotTwice) != 0u; }
GBCE_TABLE_FN int slot_entry(uint32_t slot) { return (int)(slot & (kSlotTwice - 1u)); }

// Entry k, of column `col`; column_of(j): the column of an entry that stands for one; cas(slot, expected,
// value): what the slot held.  True: another entry stands for the column.
template <typename Column, typename Cas>
GBCE_TABLE_FN bool list_enter(uint16_t* slots, uint32_t n, int k, int col, Column column_of, Cas cas) {
    for (uint32_t h = ((uint32_t)col * 2654435761u) >> 7;; ++h) {
        h &= n - 1u;
        const uint32_t was = cas(slots + h, kSlotFree, (uint32_t)k);
        if (was == kSlotFree) return false;
        const uint32_t first = was & (kSlotTwice - 1u);
        if (column_of((int)first) != col) continue;
        if (was == first) (void)cas(slots + h, first, first | kSlotTwice);
        return true;
    }
}

}  // namespace gbce
