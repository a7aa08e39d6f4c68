// pkv_compact.cuh -- kept cells of each sequence moved together, in place.
//
// Cell start + keep[i] of a sequence goes to cell start + i, K and V, in
// every layer's caches, for i = 0 .. keep_lens - 1; keep ascends, so keep[i]
// >= i.  Bound by memory: every moved cell is read and written once.
//
// Work.  A chunk is a run of `rows` consecutive entries of one sequence, for
// one cache and one slice of a cell; all its cells are read before any is
// written.  Leading entries that stay where they are (keep[i] == i) are not
// touched.
//
// Short lists (an accepted path) are one chunk.  In longer ones chunk c writes
// the cells of positions c rows .. (c + 1) rows - 1, and the entries that read
// them (keep[i] in that range, so i <= keep[i]: chunks up to c) must have been
// read before.  Being at most `rows` entries in a row they lie in two chunks
// at most.  So a chunk loads its cells, marks that in a flag, waits for the
// flags of these (at most two) earlier chunks, and stores.  Chunks are handed
// out in order by a counter, a warp does its own in order, and a chunk only
// waits for loads of earlier ones: no circle of waits can form.  One pass over
// the data; through a second buffer it would be two.
#pragma once

#include "pkv_kernels.cuh"

namespace pkv {

constexpr int kCompactMaxLayers = 128;   // layers per launch (pointers travel as kernel arguments)
constexpr int kCompactThreads = 256;     // short lists: threads of a CTA, and the longest list
// Longer lists: bytes of a warp's chunk in shared memory, and warps per SM.  A
// list of half of 16-32 K cells of 4 KB, 8 sequences (765 MB moved): 137 us so
// (5.6 TB/s), 141 with 13 x 16 KB, 163 with 24 x 8 KB.
constexpr int kCompactStage = 32768;
constexpr int kCompactPerSm = 6;

struct CompactArgs {
    const int32_t *block_tables;     // [batch, max_blocks]
    const int32_t *start_lens;       // [batch]
    const int32_t *keep;             // [batch, max_keep]
    const int32_t *keep_lens;        // [batch]
    unsigned int *flags;             // longer lists: [0] the counter, then one per chunk
    int batch;
    int max_blocks;
    int max_keep;
    int block_size;
    int num_blocks;
    int vec_per_cell;                // 16-byte vectors of a cell (all kv heads)
    int slice_vec;                   // vectors of a slice (the last one may have fewer)
    int slices;
    int rows;                        // entries per chunk
    int caches;                      // 2 * layers
    uint4 *cache[2 * kCompactMaxLayers];   // K caches, then V caches
};

__device__ __forceinline__ unsigned int load_acquire(const unsigned int *p)
{
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(unsigned int *p, unsigned int v)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The first entry with keep >= x among entries 0 .. n - 1 (n if none), by a
// 32-way search of one warp.  keep ascends.
__device__ __forceinline__ int compact_lower_bound(const int32_t *keep, int n, int x)
{
    const int lane = threadIdx.x & 31;
    int lo = 0;                                   // entries before lo are < x
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = lane * step;                // probes lo + i
        const int below = __popc(__ballot_sync(0xffffffffu, i < n && __ldg(keep + lo + i) < x));
        if (step == 1)
            return lo + below;
        if (below == 0)
            return lo;
        lo += (below - 1) * step + 1;
        n = min(step - 1, n - (below - 1) * step - 1);
    }
    return lo;
}

// Entries of sequence b: 0 (and PKV_DEVFLAG_CONTEXT_RANGE, where `tell`) for
// one that contradicts itself.
__device__ __forceinline__ int compact_entries(const CompactArgs &a, int b, bool tell)
{
    const int start = __ldg(a.start_lens + b), n = __ldg(a.keep_lens + b);
    if (start < 0 || n < 0 || n > a.max_keep || start + (int64_t)n > (int64_t)a.max_blocks * a.block_size) {
        if (tell)
            raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
        return 0;                                 // the sequence is skipped
    }
    return n;
}

// The source and target cell of entry i of sequence b; false: it does not move.
__device__ __forceinline__ bool compact_lookup(const CompactArgs &a, int b, int start, int i, int *src, int *dst)
{
    const int32_t *keep = a.keep + (size_t)b * a.max_keep;
    const int32_t *table = a.block_tables + (size_t)b * a.max_blocks;
    const int k = __ldg(keep + i), before = i > 0 ? __ldg(keep + i - 1) : -1;
    *src = *dst = -1;
    if (k < i || k <= before || start + (int64_t)k >= (int64_t)a.max_blocks * a.block_size) {
        raise_flag(PKV_DEVFLAG_INDEX_RANGE);
        return false;
    }
    if (k == i)
        return false;
    const int sb = (start + k) / a.block_size, db = (start + i) / a.block_size;
    const int sp = __ldg(table + sb), dp = __ldg(table + db);
    if ((unsigned)sp >= (unsigned)a.num_blocks || (unsigned)dp >= (unsigned)a.num_blocks) {
        raise_flag(PKV_DEVFLAG_BLOCK_RANGE);
        return false;
    }
    *src = sp * a.block_size + (start + k) - sb * a.block_size;   // below 2^31: cells of the pool
    *dst = dp * a.block_size + (start + i) - db * a.block_size;
    return true;
}

// A thread's vectors: the first is (tid / slice_vec, tid % slice_vec) of the
// chunk, each next one 256 vectors on.
template <int VEC, typename F>
__device__ __forceinline__ void compact_vectors(const CompactArgs &a, F &&f)
{
    int r = (int)threadIdx.x / a.slice_vec, v = (int)threadIdx.x - r * a.slice_vec;
    const int row_step = kCompactThreads / a.slice_vec, v_step = kCompactThreads - row_step * a.slice_vec;
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
        f(u, r, v);
        r += row_step;
        v += v_step;
        if (v >= a.slice_vec) {
            v -= a.slice_vec;
            ++r;
        }
    }
}

// Lists of one chunk: CTA x is (sequence, cache, slice) x; a slice is narrow
// enough for the longest list, VEC of its vectors to a thread.
template <int VEC>
__global__ void __launch_bounds__(kCompactThreads)
compact_short_kernel(const __grid_constant__ CompactArgs a)
{
    __shared__ int s_src[kCompactThreads], s_dst[kCompactThreads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int bc = (int)blockIdx.x / a.slices, slice = (int)blockIdx.x - bc * a.slices;
    const int b = bc / a.caches, cache_i = bc - b * a.caches;
    const int cnt = compact_entries(a, b, threadIdx.x == 0 && cache_i == 0 && slice == 0);   // at most a.rows
    bool moves = false;
    if ((int)threadIdx.x < cnt)
        moves = compact_lookup(a, b, __ldg(a.start_lens + b), threadIdx.x, &s_src[threadIdx.x], &s_dst[threadIdx.x]);
    if (!__syncthreads_or(moves))
        return;
    uint4 *at = a.cache[cache_i] + slice * a.slice_vec;
    const int vec = min(a.slice_vec, a.vec_per_cell - slice * a.slice_vec);
    uint4 x[VEC];
    unsigned int all = 0u;
    compact_vectors<VEC>(a, [&](int u, int r, int v) {
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < cnt && v < vec && s_src[r] >= 0)
            x[u] = at[(size_t)s_src[r] * a.vec_per_cell + v];
        all |= x[u].x | x[u].y | x[u].z | x[u].w;
    });
    // in place: the barrier sees every thread's values, so all cells have been
    // read when the first is written
    __syncthreads_or(all != 0u);
    compact_vectors<VEC>(a, [&](int u, int r, int v) {
        if (r < cnt && v < vec && s_src[r] >= 0)
            at[(size_t)s_dst[r] * a.vec_per_cell + v] = x[u];
    });
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}

// Longer lists: a warp to a CTA, a chunk at a time, a lane to an entry.  A
// lane's piece of a cell comes into shared memory and leaves it by bulk copies
// (nothing passes through registers), so a warp's chain of waits (indices,
// cells, flags) costs few instructions and six warps per SM overlap.
// Equal lists, cells of 8 x 128 bf16: 8 us and 6.1 TB/s (0.93 of a plain copy's
// rate; 8 x 12000 cells, 786 MB: 137 us).  Random, page-wise or contiguous kept
// cells and scattered or ascending pages are within 5 % of each other; lists of
// unequal length cost 5 to 7 % more.
__global__ void __launch_bounds__(32)
compact_long_kernel(const __grid_constant__ CompactArgs a)
{
    extern __shared__ __align__(128) uint8_t s_stage[];
    __shared__ __align__(8) uint64_t s_bar;
    const uint32_t stage = smem_addr(s_stage), bar = smem_addr(&s_bar);
    const int lane = threadIdx.x;
    if (lane == 0)
        mbar_init(bar, 1);
    fence_mbar_init();
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // tickets: chunk after chunk, each over all (sequence, cache, slice)
    // columns; the longest list bounds the chunks
    int longest = 0;
    for (int b = lane; b < a.batch; b += 32)
        longest = max(longest, compact_entries(a, b, blockIdx.x == 0));
    longest = __reduce_max_sync(0xffffffffu, longest);
    const unsigned int columns = (unsigned int)a.batch * a.caches * a.slices;
    const unsigned int tickets = (unsigned int)((longest + a.rows - 1) / a.rows) * columns;
    unsigned int ticket = 0u;
    if (lane == 0)
        ticket = atomicAdd(a.flags, 1u);
    ticket = __shfl_sync(0xffffffffu, ticket, 0);
    uint32_t phase = 0u;
    while (ticket < tickets) {
        const int chunk = (int)(ticket / columns);
        const int col = (int)(ticket - (unsigned int)chunk * columns);
        const int bc = col / a.slices, slice = col - bc * a.slices;
        const int b = bc / a.caches, cache_i = bc - b * a.caches;
        const int i0 = chunk * a.rows;
        const int cnt = min(a.rows, compact_entries(a, b, false) - i0);
        int src, dst;
        const bool mine = lane < cnt && compact_lookup(a, b, __ldg(a.start_lens + b), i0 + lane, &src, &dst);
        const unsigned int moving = __ballot_sync(0xffffffffu, mine);
        uint4 *cache = a.cache[cache_i] + slice * a.slice_vec;
        const uint32_t bytes = 16u * (uint32_t)min(a.slice_vec, a.vec_per_cell - slice * a.slice_vec);
        const uint32_t at = stage + (uint32_t)(lane * a.slice_vec) * 16u;
        if (moving) {
            // the lane's last store has been read out of shared memory
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            if (lane == 0)
                mbar_arrive_expect_tx(bar, bytes * (uint32_t)__popc(moving));
            __syncwarp();
            if (mine)
                bulk_load(at, cache + (size_t)src * a.vec_per_cell, bytes, bar);
        }
        unsigned int next = 0u;
        if (lane == 0)
            next = atomicAdd(a.flags, 1u);
        unsigned int *flag = a.flags + 1 + ticket;
        bool ok = true;
        if (moving) {
            // (while the loads are under way) the chunks that read what this one writes
            const int lo = compact_lower_bound(a.keep + (size_t)b * a.max_keep, i0, i0) / a.rows;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase, kWaitLimitNs));
            phase ^= 1u;
            if (lane == 0 && ok) {
                __threadfence();
                store_release(flag, 1u);
            }
            if (ok && lane < 2 && lo + lane < chunk) {
                const unsigned int *f = flag - (size_t)(chunk - lo - lane) * columns;
                if (load_acquire(f) == 0u) {
                    const uint64_t t0 = global_timer_ns();
                    while (!(ok = load_acquire(f) != 0u) && global_timer_ns() - t0 < kWaitLimitNs)
                        __nanosleep(64);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            if (mine) {
                asm volatile("fence.proxy.async;" ::: "memory");
                bulk_store(cache + (size_t)dst * a.vec_per_cell, at, bytes);
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        } else if (lane == 0) {
            store_release(flag, 1u);
        }
        ticket = __shfl_sync(0xffffffffu, next, 0);
    }
    if (ticket < tickets && lane == 0) {          // a wait gave up
        raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
        mbar_wait_bounded(bar, phase ^ 1u, kWaitLimitNs / 8);   // loads in flight land
    }
    __syncwarp();
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace pkv
