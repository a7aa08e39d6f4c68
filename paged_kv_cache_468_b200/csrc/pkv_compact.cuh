// pkv_compact.cuh -- kept cells of each sequence moved together, in place.
//
// Cell start + keep[i] of a sequence goes to cell start + i, K and V, in
// every layer's caches, for i = 0 .. keep_lens - 1; keep ascends, so keep[i]
// >= i and a cell is read before a later one is written over it when the
// moves run in order.
#pragma once

#include "pkv_kernels.cuh"

namespace pkv {

constexpr int kCompactMaxLayers = 128;   // layers per launch (pointers travel as kernel arguments)

struct CompactArgs {
    const int32_t *block_tables;     // [batch, max_blocks]
    const int32_t *start_lens;       // [batch]
    const int32_t *keep;             // [batch, max_keep]
    const int32_t *keep_lens;        // [batch]
    int max_blocks;
    int max_keep;
    int block_size;
    int num_blocks;
    int vec_per_cell;                // 16-byte vectors of a cell (all kv heads)
    uint4 *cache[2 * kCompactMaxLayers];   // K caches, then V caches
};

// One CTA per (sequence, cache, slice of a cell's 16-byte vectors): a thread
// moves one vector column of the sequence's cells in order.
constexpr int kCompactThreads = 64;
__global__ void __launch_bounds__(kCompactThreads)
compact_kernel(const __grid_constant__ CompactArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int b = blockIdx.z;
    const int v = blockIdx.x * kCompactThreads + threadIdx.x;
    uint4 *cache = a.cache[blockIdx.y];
    const int start = __ldg(a.start_lens + b);
    int n = __ldg(a.keep_lens + b);
    const int64_t span = (int64_t)a.max_blocks * a.block_size;
    if (start < 0 || n < 0 || n > a.max_keep || start + (int64_t)n > span) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
        return;                                    // the sequence is skipped
    }
    if (v >= a.vec_per_cell)
        return;
    const int32_t *keep = a.keep + (size_t)b * a.max_keep;
    const int32_t *table = a.block_tables + (size_t)b * a.max_blocks;
    auto cell = [&](int64_t pos, bool *ok) -> uint4 * {
        const int blk = __ldg(table + pos / a.block_size);
        *ok = (unsigned)blk < (unsigned)a.num_blocks;
        return cache + ((size_t)(*ok ? blk : 0) * a.block_size + pos % a.block_size) * a.vec_per_cell + v;
    };
    int before = -1;
    for (int i = 0; i < n; ++i) {
        const int k = __ldg(keep + i);
        if (k <= before || start + (int64_t)k >= span) {
            raise_flag(PKV_DEVFLAG_INDEX_RANGE);
            continue;
        }
        before = k;
        if (k == i)
            continue;
        bool ok_s, ok_d;
        const uint4 *src = cell(start + (int64_t)k, &ok_s);
        uint4 *dst = cell(start + (int64_t)i, &ok_d);
        if (ok_s && ok_d)
            *dst = *src;
        else
            raise_flag(PKV_DEVFLAG_BLOCK_RANGE);
    }
}

}  // namespace pkv
