// pkv_tree.cuh -- kernels of a speculative step with drafted token trees:
// the tree's ancestor bits, attention of the drafted tokens over the paged
// cache, and the greedy acceptance of a path.
//
// Sequence b drafts n_b = query_start[b+1] - query_start[b] nodes, which are
// the last n_b of its context_lens[b] cached tokens (written through
// slot_mapping beforehand, "大模型推理框架VLLM-0.7.3源码", sections 2.1 / 3.3).
// parents[] holds each node's parent as an index within its sequence, a
// smaller one than its own, or -1.
#pragma once

#include "pkv_prefill.cuh"

namespace pkv {

// A sequence's drafted rows: first row and count, and its length.  False (and
// PKV_DEVFLAG_CONTEXT_RANGE) where they contradict the call's sizes: such a
// sequence is skipped.
struct TreeSeq {
    int q0, n, len;
};
__device__ __forceinline__ bool tree_seq(const int32_t *query_start, const int32_t *context_lens, int b,
                                         int num_tokens, int max_query_len, int span, TreeSeq *s)
{
    s->q0 = __ldg(query_start + b);
    const int q1 = __ldg(query_start + b + 1);
    s->len = context_lens ? __ldg(context_lens + b) : 0;
    s->n = 0;
    if (s->q0 < 0 || q1 < s->q0 || q1 > num_tokens || q1 - s->q0 > max_query_len)
        return false;
    if (context_lens && (s->len < q1 - s->q0 || s->len > span))
        return false;
    s->n = q1 - s->q0;
    return true;
}

// ---------------------------------------------------------------------------
// Ancestor bits and positions
// ---------------------------------------------------------------------------
// bits(i) = {i} + bits(parent(i)); position(i) = context_lens[b] - n_b + depth(i).
//
// Nodes are taken 32 at a time (a word of the mask).  Within a word the
// ancestors of a node are found by pointer doubling between the lanes of a
// warp (five rounds whatever the tree's depth); what is left per node is its
// word's bits and the ancestor through which its path leaves the word.  A
// node's whole row then takes one step per word that its path touches, at
// most 32, instead of one per ancestor.  A CTA takes 32 * NW nodes of one
// sequence; every CTA of a sequence works out all words (4 KB of parents at
// most), which costs less than a second launch.
constexpr int kTreeMaxNodes = 1024;
template <int NW>
__global__ void __launch_bounds__(NW * 32)
tree_mask_kernel(const int32_t *__restrict__ parents, int num_tokens, const int32_t *__restrict__ query_start,
                 int max_query_len, const int32_t *__restrict__ context_lens, int words,
                 int32_t *__restrict__ tree_mask, int32_t *__restrict__ positions)
{
    __shared__ uint32_t s_bits[kTreeMaxNodes];
    __shared__ int16_t s_exit[kTreeMaxNodes];
    __shared__ uint32_t s_row[NW][32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TreeSeq s;
    if (!tree_seq(query_start, context_lens, blockIdx.y, num_tokens, max_query_len, 0x7fffffff, &s)) {
        if (threadIdx.x == 0 && blockIdx.x == 0)
            raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
        return;
    }
    const int first = blockIdx.x * NW * 32;       // this CTA's nodes
    if (first >= s.n)
        return;
    const int upto = min(s.n, first + NW * 32);   // earlier nodes are their only ancestors
    bool bad = false;
    for (int i0 = warp * 32; i0 < upto; i0 += NW * 32) {
        const int i = i0 + lane;
        int p = -1;
        if (i < s.n) {
            p = __ldg(parents + s.q0 + i);
            if (p < -1 || p >= i) {
                bad = true;
                p = -1;                           // taken as a root
            }
        }
        uint32_t m = 1u << lane;
        int up = p;                               // the next ancestor not in m yet
#pragma unroll
        for (int r = 0; r < 5; ++r) {
            const uint32_t mu = __shfl_sync(0xffffffffu, m, up & 31);
            const int uu = __shfl_sync(0xffffffffu, up, up & 31);
            if (up >= i0) {                       // still within the word (negative: none)
                m |= mu;
                up = uu;
            }
        }
        s_bits[i] = m;
        s_exit[i] = (int16_t)up;
    }
    if (bad)
        raise_flag(PKV_DEVFLAG_INDEX_RANGE);
    __syncthreads();
    const int i0 = first + warp * 32;
    if (i0 >= s.n)
        return;                                   // whole warp
#pragma unroll 4
    for (int w = 0; w < words; ++w)
        s_row[warp][lane][w] = 0u;
    int depth = -1;
    if (i0 + lane < s.n)
        for (int c = i0 + lane; c >= 0; c = s_exit[c]) {
            const uint32_t m = s_bits[c];
            s_row[warp][lane][c >> 5] = m;
            depth += __popc(m);
        }
    __syncwarp();
    const int rows = min(32, s.n - i0);
    if (lane < rows)
        positions[s.q0 + i0 + lane] = s.len - s.n + depth;
    // rows of `words` words are contiguous: lane after lane over the warp's rows
    int32_t *out = tree_mask + (size_t)(s.q0 + i0) * words;
    for (int e = lane; e < rows * words; e += 32)
        out[e] = (int32_t)s_row[warp][e / words][e % words];
}

// ---------------------------------------------------------------------------
// Greedy acceptance
// ---------------------------------------------------------------------------
// From node 0 on: the accepted node's next one is its lowest child whose
// drafted token is the target's answer at the node; the path ends where no
// child has it.  Each node offers itself to its parent (an atomic minimum in
// shared memory: the result does not depend on the order), one thread follows
// the winners.  A CTA per sequence; bound by launch and two round trips to
// memory.
constexpr int kAcceptThreads = 128;
__global__ void __launch_bounds__(kAcceptThreads)
tree_accept_kernel(const int64_t *__restrict__ draft, const int64_t *__restrict__ target,
                   const int32_t *__restrict__ parents, int num_tokens,
                   const int32_t *__restrict__ query_start, int max_query_len,
                   int32_t *__restrict__ path, int32_t *__restrict__ lens, int64_t *__restrict__ next_tokens)
{
    __shared__ int s_next[kTreeMaxNodes];
    __shared__ int16_t s_path[kTreeMaxNodes];
    __shared__ int s_len;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int b = blockIdx.x;
    TreeSeq s;
    if (!tree_seq(query_start, nullptr, b, num_tokens, max_query_len, 0, &s) && threadIdx.x == 0)
        raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);    // s.n is 0: an empty path
    for (int i = threadIdx.x; i < s.n; i += kAcceptThreads)
        s_next[i] = kTreeMaxNodes;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += kAcceptThreads) {
        const int p = __ldg(parents + s.q0 + i);
        if (p < -1 || p >= i)
            raise_flag(PKV_DEVFLAG_INDEX_RANGE);   // never accepted
        else if (p >= 0 && __ldg(draft + s.q0 + i) == __ldg(target + s.q0 + p))
            atomicMin(&s_next[p], i);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int k = 0, last = -1;
        for (int c = 0; c < s.n; c = s_next[c]) { // a child's index is above its parent's: the walk ends
            s_path[k++] = (int16_t)c;
            last = c;
        }
        s_len = k;
        lens[b] = k;
        next_tokens[b] = last >= 0 ? __ldg(target + s.q0 + last) : -1;
    }
    __syncthreads();
    const int k = s_len;
    for (int i = threadIdx.x; i < max_query_len; i += kAcceptThreads)
        path[(size_t)b * max_query_len + i] = i < k ? (int)s_path[i] : -1;
}

// ---------------------------------------------------------------------------
// Attention of the drafted tokens
// ---------------------------------------------------------------------------
// Per (sequence, kv head) the rows are the (node, head of the group) pairs,
// 128 to a row tile; the keys are taken 64 at a time.  On the tensor cores
// (tcgen05, as the prefill: pkv_prefill.cuh holds the barriers' reasoning):
//
//   S_j = Q K_j^T,   P_j = 2^(S_j scale log2 e - m),   O += P_j V_j
//
// with P over S in tensor memory, S double-buffered, and the running maximum m
// moved only when a tile exceeds it by 2^8.  Only the last key tiles of a
// sequence hold drafted keys: they alone are masked, by 64 bits per row cut
// from the row's mask words.
//
// Work.  The keys are read once per (sequence, kv head) if one row tile covers
// its rows, so the floor of such calls is the cache's bytes over the memory
// rate, and every SM has to stream all the time.  Lengths and tree sizes are
// on the device and ragged, so the work is cut into equal shares there: the
// key tiles of all (sequence, kv head, row tile) items form one sequence of
// units, and CTA c of n takes units [W c / n, W (c+1) / n), two CTAs to an SM.
// An item that lies in one CTA's share is written out by it; a part of an
// item becomes a record (running maximum, sum, O row), and tree_merge_kernel
// joins the records of such an item.  A CTA holds two parts at most, so the
// records' size does not depend on the call.
//
// Row tiles beyond the first would read the keys again.  They are therefore
// taken in pairs by two CTAs that walk the same keys side by side (the second
// read comes from L2); an odd last row tile joins the single ones.  Pairs and
// singles are two such sequences of units, shared out one after the other.
//
// A masked tile is the only one whose V rows some row may not see: such a row
// gives them weight 0, and 0 times an infinity or a NaN would poison it.  The
// softmax warps look through the V rows of masked tiles; where one holds such
// a value, they zero it in shared memory and add it to the rows that do see it.
struct TreeArgs {
    const int32_t *query_start;      // [batch + 1]
    const int32_t *tree_mask;        // [T, words]
    const uint16_t *value_cache;     // [num_blocks, bs, Hkv, D]
    const int32_t *block_tables;     // [batch, max_blocks]
    const int32_t *context_lens;     // [batch]
    uint16_t *out;                   // [T, Hq, D]
    int4 *desc;                      // [CTAs][2]: the item whose records start before this CTA's share
    float2 *rec_ml;                  // [CTAs][2 shares][2 parts][128]
    float *rec_o;                    // [CTAs][2][2][128][D]
    int batch;
    int num_tokens;
    int max_query_len;
    int words;                       // mask words per row
    int max_blocks;
    int num_heads;
    int num_kv_heads;
    int group;
    int num_blocks;
    int shares;                      // 2: pairs of row tiles, then single ones; 1: single ones only
    float scale_log2;
};

constexpr int kTreeThreads = 256;
constexpr int kTreeRows = 128;           // query rows per tile (MMA M)
constexpr int kTreeKeys = 64;            // keys per tile
constexpr int kTreeItemCost = 2;         // an item's start and end, in key tiles
constexpr int kTreeMinUnits = 2;         // a CTA's share is not cut below this

template <int D>
struct TreeShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kQHalf = kTreeRows * 128;
    static constexpr int kKVHalf = kTreeKeys * 128;
    static constexpr int kQBytes = kHalves * kQHalf;
    static constexpr int kKVBytes = kHalves * kKVHalf;
    // two CTAs per SM: 112 KB each (D = 128: 32 + 80, D = 64: 16 + 80)
    static constexpr int kKStages = D == 128 ? 3 : 6;
    static constexpr int kVStages = D == 128 ? 2 : 4;
    static constexpr int kKOff = kQBytes;
    static constexpr int kVOff = kKOff + kKStages * kKVBytes;
    static constexpr int kDataBytes = kVOff + kVStages * kKVBytes;
    static constexpr int kSmemBytes = kDataBytes + 1024;
    // barriers
    static constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kKEmpty = kKFull + kKStages, kVFull = kKEmpty + kKStages,
                         kVEmpty = kVFull + kVStages, kSFull = kVEmpty + kVStages, kPFull = kSFull + 2,
                         kODone = kPFull + 2, kDrain = kODone + 1, kScan = kDrain + 1, kNumBars = kScan + 1;
};

// One sequence of units: a share [g, end) of it, walked item by item.
struct TreeSegment {
    int b;            // sequence
    int kvh;
    int rt;           // row tile
    int q0, n, len;   // the sequence's rows and length
    int tiles;        // key tiles of the item
    int k0, k1;       // this part's key tiles
};
struct TreeWalk {
    int64_t g, end;   // units left
    int64_t seq0;     // first unit of sequence b
    int b;
};

// Units of a sequence: single items (pair = false) or pairs of row tiles.
__device__ __forceinline__ int tree_items(int n, int G, bool single_only, bool pair)
{
    const int tt = kTreeRows / G;
    const int rt = (n + tt - 1) / tt;
    return pair ? rt / 2 : (single_only ? rt : rt & 1);
}
__device__ __forceinline__ int64_t tree_units(int items, int len, int kv_heads)
{
    return (int64_t)items * kv_heads * ((len + kTreeKeys - 1) / kTreeKeys + kTreeItemCost);
}

template <int BS>
__device__ __forceinline__ bool tree_next(TreeWalk &w, const TreeArgs &a, int share, int member, TreeSegment *s)
{
    const bool pair = a.shares == 2 && share == 0;
    while (w.g < w.end) {
        TreeSeq q;
        // contradicting sequences have no units
        const bool ok = tree_seq(a.query_start, a.context_lens, w.b, a.num_tokens, a.max_query_len,
                                 a.max_blocks * BS, &q);
        const int items = ok ? tree_items(q.n, a.group, a.shares == 1, pair) : 0;
        const int64_t units = tree_units(items, q.len, a.num_kv_heads);
        const int64_t off = w.g - w.seq0;
        if (off >= units) {
            w.seq0 += units;
            ++w.b;
            continue;
        }
        const int tiles = (q.len + kTreeKeys - 1) / kTreeKeys;
        const int cost = tiles + kTreeItemCost;
        const int item = (int)(off / cost);
        const int k0 = (int)(off - (int64_t)item * cost);
        const int step = (int)min((int64_t)(cost - k0), w.end - w.g);
        w.g += step;
        if (k0 >= tiles)
            continue;
        s->b = w.b;
        s->kvh = item % a.num_kv_heads;
        const int r = item / a.num_kv_heads;
        // pairs: row tiles 2 r and 2 r + 1; singles: row tile r, or the odd last one
        s->rt = pair ? 2 * r + member : (a.shares == 1 ? r : (q.n + kTreeRows / a.group - 1) / (kTreeRows / a.group) - 1);
        s->q0 = q.q0;
        s->n = q.n;
        s->len = q.len;
        s->tiles = tiles;
        s->k0 = k0;
        s->k1 = min(tiles, k0 + step);
        return true;
    }
    return false;
}

__device__ __forceinline__ int64_t tree_cut(int64_t total, int c, int n)   // the first unit of CTA (or pair) c
{
    return total / n * c + total % n * c / n;
}
__device__ __forceinline__ int tree_ctas(int64_t total, int most)          // CTAs (or pairs) that share the units
{
    const int64_t want = (total + kTreeMinUnits - 1) / kTreeMinUnits;
    return (int)min((int64_t)most, max((int64_t)1, want));
}

// Row r's visible positions p0 .. p0 + 63 as bits: committed cells, and the
// drafted ones that its mask row names.
__device__ __forceinline__ uint64_t tree_bits(const int32_t *mask, int words, int base, int n, int p0)
{
    int j0 = p0 - base;
    uint64_t ones = 0ull;
    int sh = 0;
    if (j0 < 0) {
        if (j0 <= -64)
            return ~0ull;
        sh = -j0;
        ones = (1ull << sh) - 1ull;
        j0 = 0;
    }
    const int left = n - j0;                 // drafted cells from j0 on
    if (left <= 0)
        return ones;
    const int w = j0 >> 5, o = j0 & 31;
    const uint32_t w0 = (uint32_t)__ldg(mask + w);
    const uint32_t w1 = w + 1 < words ? (uint32_t)__ldg(mask + w + 1) : 0u;
    const uint32_t w2 = w + 2 < words ? (uint32_t)__ldg(mask + w + 2) : 0u;
    uint64_t v = (uint64_t)__funnelshift_r(w0, w1, o) | ((uint64_t)__funnelshift_r(w1, w2, o) << 32);
    if (left < 64)
        v &= (1ull << left) - 1ull;
    return ones | (v << sh);
}

// Infinities and NaN among the 16-bit values of a word (all exponent bits set).
template <bool BF16>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x)   // bit 0: low half, bit 16: high half
{
    constexpr uint32_t e = BF16 ? 0x7f807f80u : 0x7c007c00u;
    const uint32_t y = x & e;
    return ((y & 0xffffu) == (e & 0xffffu) ? 1u : 0u) | ((y >> 16) == (e >> 16) ? 0x10000u : 0u);
}

template <int D, int BS, bool BF16>
__global__ void __launch_bounds__(kTreeThreads, 2)
tree_attend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k4,
                   const __grid_constant__ CUtensorMap tm_v4, const TreeArgs a)
{
    using Sh = TreeShape<D>;
    constexpr int KS = D / 16, KV_STEPS = kTreeKeys / 16, BPT = kTreeKeys / BS;
    constexpr uint32_t kTmemCols = 256;          // S/P: 2 x 64 columns, O: D columns at 128
    // The tiles start on a 1024-byte boundary; what else the CTA keeps lies in
    // whichever end of the 1024 bytes of slack has room (with 1 KB more two
    // CTAs would not fit an SM).
    struct Local {
        uint64_t bars[Sh::kNumBars];
        TreeWalk walk[2];
        int64_t scan[kTreeThreads / 32];
        uint32_t bad[2][4];
        uint32_t tmem;
    };
    static_assert(sizeof(Local) <= 512, "fits one end of the slack");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t front = ((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw);
    uint8_t *data = smem_raw + front;
    const uint32_t data_s = smem_addr(data);
    Local *loc = reinterpret_cast<Local *>(front >= 512u ? smem_raw : data + Sh::kDataBytes);
    TreeWalk *s_walk = loc->walk;
    int64_t *s_scan = loc->scan;
    uint32_t(*s_bad)[4] = loc->bad;
    const uint32_t bars_s = smem_addr(loc->bars);
    auto bar = [&](int i) { return bars_s + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group, TT = kTreeRows / G, R = TT * G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kNumBars; ++i)
            mbar_init(bar(i), i == Sh::kPFull || i == Sh::kPFull + 1 || i == Sh::kScan ? 4 : 1);
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_k4);
        prefetch_tensormap(&tm_v4);
    }
    fence_mbar_init();
    if (warp == 5) {
        tmem_alloc(smem_addr(&loc->tmem), kTmemCols);
        tmem_relinquish();
    }
    // masked columns of a tile may meet V rows that no load has filled
    {
        uint4 *vr = reinterpret_cast<uint4 *>(data + Sh::kVOff);
        for (int i = threadIdx.x; i < Sh::kVStages * Sh::kKVBytes / 16; i += kTreeThreads)
            vr[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&loc->tmem);

    // ---- this CTA's shares: a thread adds up a run of sequences, the block
    // their totals; the thread whose run holds the share's start finds it ----
    for (int share = 0; share < a.shares; ++share) {
        const bool pair = a.shares == 2 && share == 0;
        const int per = (a.batch + kTreeThreads - 1) / kTreeThreads;
        const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) {
            TreeSeq q;
            if (tree_seq(a.query_start, a.context_lens, b, a.num_tokens, a.max_query_len, a.max_blocks * BS, &q))
                mine += tree_units(tree_items(q.n, G, a.shares == 1, pair), q.len, a.num_kv_heads);
            else if (blockIdx.x == 0 && share == 0)
                raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
        }
        int64_t upto = mine;                         // inclusive prefix over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += x;
        }
        if (lane == 31)
            s_scan[warp] = upto;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int i = 0; i < kTreeThreads / 32; ++i) {
            if (i < warp)
                upto += s_scan[i];
            total += s_scan[i];
        }
        const int n = tree_ctas(total, pair ? gridDim.x / 2 : gridDim.x);
        const int c = pair ? blockIdx.x >> 1 : blockIdx.x;
        const int64_t g0 = c < n ? tree_cut(total, c, n) : total;
        const int64_t g1 = c < n ? tree_cut(total, c + 1, n) : total;
        if (threadIdx.x == 0)
            s_walk[share] = TreeWalk{0, 0, 0, 0};    // an empty share
        __syncthreads();
        if (g0 < g1 && g0 >= upto - mine && g0 < upto) {
            int64_t at = upto - mine;
            int b = b0;
            for (;; ++b) {
                TreeSeq q;
                int64_t u = 0;
                if (tree_seq(a.query_start, a.context_lens, b, a.num_tokens, a.max_query_len, a.max_blocks * BS, &q))
                    u = tree_units(tree_items(q.n, G, a.shares == 1, pair), q.len, a.num_kv_heads);
                if (g0 < at + u)
                    break;
                at += u;
            }
            s_walk[share] = TreeWalk{g0, g1, at, b};
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            // An item that started in the share before and goes on here: its
            // second part.  The merge finds the item's records through it.
            int4 d = make_int4(0, 0, 0, 0);
            TreeWalk w = s_walk[share];
            TreeSeq q;
            if (c > 0 && w.g < w.end &&
                tree_seq(a.query_start, a.context_lens, w.b, a.num_tokens, a.max_query_len, a.max_blocks * BS, &q)) {
                const int tiles = (q.len + kTreeKeys - 1) / kTreeKeys;
                const int k0 = (int)((w.g - w.seq0) % (tiles + kTreeItemCost));
                const int64_t start = w.g - k0;      // the item's first unit
                TreeSegment s;
                if (k0 > 0 && k0 < tiles && start >= tree_cut(total, c - 1, n) &&
                    tree_next<BS>(w, a, share, blockIdx.x & 1, &s)) {
                    int last = c;                    // the last CTA (or pair) with keys of the item
                    while (last + 1 < n && tree_cut(total, last + 1, n) < start + tiles)
                        ++last;
                    d = make_int4(s.q0 + s.rt * TT, min(R, s.n * G - s.rt * R), s.kvh, last - c + 2);
                }
            }
            a.desc[blockIdx.x * 2 + share] = d;
        }
    }

    const uint32_t sQ = data_s, sK = data_s + Sh::kKOff, sV = data_s + Sh::kVOff;
    const uint32_t tO = tmem + 2 * kTreeKeys;
    const int member = blockIdx.x & 1;

    // every role walks the same parts; key tiles are numbered on across them (J)
    int w_share = 0;
    TreeWalk walk = s_walk[0];
    auto next_part = [&](TreeSegment *s) -> bool {
        for (;;) {
            if (tree_next<BS>(walk, a, w_share, member, s))
                return true;
            if (++w_share >= a.shares)
                return false;
            walk = s_walk[w_share];
        }
    };

    if (warp == 4 || warp == 6) {
        // ---- loads: warp 4 the K ring, warp 6 the V ring ----
        const bool is_k = warp == 4;
        const CUtensorMap *tm = is_k ? &tm_k : &tm_v;
        const CUtensorMap *tm4 = is_k ? &tm_k4 : &tm_v4;
        const int full0 = is_k ? Sh::kKFull : Sh::kVFull;
        const int empty0 = is_k ? Sh::kKEmpty : Sh::kVEmpty;
        const uint32_t ring = is_k ? sK : sV;
        const int NS = is_k ? Sh::kKStages : Sh::kVStages;
        const uint64_t once = policy_evict_first(), again = policy_evict_normal();
        int J = 0, st = 0, round = 0;
        bool ok = true;
        TreeSegment s;
        while (ok && next_part(&s)) {
            const uint64_t policy = a.shares == 2 && w_share == 0 ? again : once;
            const int nblk = (s.len + BS - 1) / BS;
            const int tail = s.len % BS;
            const int32_t *trow = a.block_tables + (size_t)s.b * a.max_blocks;
            int ids = 0, have = -1;                  // block ids of the 32-entry window `have`
            for (int t = s.k0; t < s.k1; ++t, ++J) {
                if (J >= NS) {
                    const bool free_ = mbar_wait_bounded(bar(empty0 + st), (uint32_t)((round - 1) & 1), kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, free_)) {
                        ok = false;
                        break;
                    }
                }
                const int kb0 = t * BPT;             // a tile's ids lie in one window
                const int nb = min(BPT, nblk - kb0);
                if ((kb0 & ~31) != have) {
                    have = kb0 & ~31;
                    ids = have + lane < nblk ? __ldg(trow + have + lane) : 0;
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(full0 + st), (uint32_t)(nb * BS * D * 2));
                __syncwarp();
                const int i = lane / Sh::kHalves, h = lane % Sh::kHalves;
                int blk = __shfl_sync(0xffffffffu, ids, (kb0 + min(i, BPT - 1)) & 31);
                if (i < nb) {
                    if ((unsigned)blk >= (unsigned)a.num_blocks) {
                        if (h == 0)
                            raise_flag(PKV_DEVFLAG_BLOCK_RANGE);
                        blk = 0;
                    }
                    // a partly filled last block ends at its slot's last row; the rows before read as zero
                    const int shift = tail && kb0 + i == nblk - 1 ? tail - BS : 0;
                    const uint32_t dst = ring + st * Sh::kKVBytes + h * Sh::kKVHalf + i * BS * 128;
                    if (shift)
                        tma_load_4d(dst, tm4, bar(full0 + st), h * 64, s.kvh, shift, blk, policy);
                    else
                        tma_load_3d(dst, tm, bar(full0 + st), h * 64, s.kvh, blk * BS, policy);
                }
                if (++st == NS) {
                    st = 0;
                    ++round;
                }
            }
        }
        if (!ok && lane == 0)
            raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
        // copies still in flight land before the CTA can exit
        if (lane == 0)
            for (int j = J > NS ? J - NS : 0; j < J; ++j)
                mbar_wait_bounded(bar(full0 + j % NS), (uint32_t)((j / NS) & 1), kWaitLimitNs / 8);
    } else if (warp == 7) {
        // ---- Q of each part, once the previous part's last S has completed ----
        if (lane == 0) {
            const uint64_t policy = policy_evict_normal();
            TreeSegment s;
            int u = 0;
            while (next_part(&s)) {
                if (u > 0 && !mbar_wait_bounded(bar(Sh::kQEmpty), (uint32_t)((u - 1) & 1), kWaitLimitNs)) {
                    raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
                    break;
                }
                mbar_arrive_expect_tx(bar(Sh::kQFull), (uint32_t)(Sh::kHalves * R * 128));
#pragma unroll
                for (int h = 0; h < Sh::kHalves; ++h)
                    tma_load_3d(sQ + h * Sh::kQHalf, &tm_q, bar(Sh::kQFull), h * 64, s.kvh * G, s.q0 + s.rt * TT, policy);
                ++u;
            }
            if (u > 0)
                mbar_wait_bounded(bar(Sh::kQFull), (uint32_t)((u - 1) & 1), kWaitLimitNs / 8);
        }
    } else if (warp == 5) {
        // ---- MMA issue: one thread ----
        if (lane == 0) {
            constexpr uint32_t idS = f16_idesc<BF16>(kTreeRows, kTreeKeys, false);
            constexpr uint32_t idO = f16_idesc<BF16>(kTreeRows, D, true);
            int ks_ = 0, kround = 0;                 // K stage of the next S
            auto issue_s = [&](int J) -> bool {
                if (!mbar_wait_bounded(bar(Sh::kKFull + ks_), (uint32_t)(kround & 1), kWaitLimitNs))
                    return false;
                tc_fence_after();
                const uint32_t kt = sK + ks_ * Sh::kKVBytes;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t koff = (uint32_t)((ks & 3) * 32);
                    tc_mma_f16(tmem + (J & 1) * kTreeKeys, sw128_desc(sQ + (ks >> 2) * Sh::kQHalf + koff, 16, 1024),
                               sw128_desc(kt + (ks >> 2) * Sh::kKVHalf + koff, 16, 1024), idS, ks > 0 ? 1u : 0u);
                }
                tc_commit(bar(Sh::kSFull + (J & 1)));
                tc_commit(bar(Sh::kKEmpty + ks_));
                if (++ks_ == Sh::kKStages) {
                    ks_ = 0;
                    ++kround;
                }
                return true;
            };
            TreeSegment s, nx;
            bool has = next_part(&s), has_nx = has && next_part(&nx);
            bool ok = true;
            int J = 0, u = 0, vs = 0, vround = 0;
            if (has) {
                ok = mbar_wait_bounded(bar(Sh::kQFull), 0u, kWaitLimitNs) && issue_s(0);
                if (ok && s.k1 - s.k0 == 1)
                    tc_commit(bar(Sh::kQEmpty));     // the part's last S
            }
            while (ok && has) {
                const int cnt = s.k1 - s.k0;
                for (int j = 0; j < cnt; ++j, ++J) {
                    if (j + 1 < cnt) {
                        // S_{J+1} overwrites the buffer that P_{J-1} V_{J-1} reads
                        if (J >= 1 && !(ok = mbar_wait_bounded(bar(Sh::kODone), (uint32_t)((J - 1) & 1), kWaitLimitNs)))
                            break;
                        if (!(ok = issue_s(J + 1)))
                            break;
                        if (j + 2 == cnt)
                            tc_commit(bar(Sh::kQEmpty));
                    }
                    ok = mbar_wait_bounded(bar(Sh::kPFull + (J & 1)), (uint32_t)((J >> 1) & 1), kWaitLimitNs) &&
                         mbar_wait_bounded(bar(Sh::kVFull + vs), (uint32_t)(vround & 1), kWaitLimitNs);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t vt = sV + vs * Sh::kKVBytes;
                    const uint32_t tp = tmem + (J & 1) * kTreeKeys;
#pragma unroll
                    for (int kk = 0; kk < KV_STEPS; ++kk)
                        tc_mma_f16_ts(tO, tp + kk * 8, sw128_desc(vt + kk * 16 * 128, Sh::kKVHalf, 1024), idO,
                                      (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(bar(Sh::kODone));
                    tc_commit(bar(Sh::kVEmpty + vs));
                    if (++vs == Sh::kVStages) {
                        vs = 0;
                        ++vround;
                    }
                }
                if (!ok)
                    break;
                if (has_nx) {
                    // the next part's first S: its buffer was read by P_{J-2} V_{J-2},
                    // which completed before P_{J-1} V_{J-1} (waited for here)
                    if (!(ok = mbar_wait_bounded(bar(Sh::kODone), (uint32_t)((J - 1) & 1), kWaitLimitNs) &&
                               mbar_wait_bounded(bar(Sh::kQFull), (uint32_t)((u + 1) & 1), kWaitLimitNs) && issue_s(J)))
                        break;
                    ++u;
                    if (nx.k1 - nx.k0 == 1)
                        tc_commit(bar(Sh::kQEmpty));
                }
                s = nx;
                has = has_nx;
                has_nx = has && next_part(&nx);
            }
            if (!ok)
                raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
            tc_commit(bar(Sh::kDrain));
            mbar_wait_bounded(bar(Sh::kDrain), 0u, kWaitLimitNs);
        }
    } else {
        // ---- softmax and epilogue: thread = row r of the tile = TMEM lane r ----
        const int r = warp * 32 + lane;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const int q = lane & 3;
        const int r_tok = r / G, r_head = r - r_tok * G;
        int rq_tok = r_tok, rq_head = r_head - q;    // the first row of this lane's quad
        while (rq_head < 0) {
            rq_head += G;
            --rq_tok;
        }
        const float sc = a.scale_log2;
        const bool fold = sc > 0.f;                  // a positive scale joins the exponent's fma
        const float sm = fold ? 1.f : sc, se = fold ? sc : 1.f;
        bool ok = true;
        int J = 0, scans = 0, vs = 0, vround = 0;
        TreeSegment s;
        while (ok && next_part(&s)) {
            const int rows = min(R, s.n * G - s.rt * R);      // rows of this tile
            const bool warp_on = warp * 32 < rows;
            const bool real = r < rows;
            const int tok = s.q0 + s.rt * TT + (real ? r_tok : 0);   // this row's node
            const int base = s.len - s.n;
            const int tail = s.len % BS;
            float m_used = kNegInf, l = 0.f;
            for (int t = s.k0; t < s.k1; ++t, ++J) {
                const int t0 = t * kTreeKeys;
                const int sb = J & 1;
                const bool masked = t0 + kTreeKeys > base;
                uint64_t vis = ~0ull;
                if (masked) {
                    vis = tree_bits(a.tree_mask + (size_t)tok * a.words, a.words, base, s.n, t0);
                    if (t + 1 == s.tiles && tail) {
                        // the partly filled last block was loaded to end its slot
                        const int lo = s.len - tail - t0;
                        const uint64_t low = (1ull << lo) - 1ull;
                        vis = (vis & low) | ((vis & ~low) << (BS - tail));
                    }
                }
                ok = mbar_wait_bounded(bar(Sh::kSFull + sb), (uint32_t)((J >> 1) & 1), kWaitLimitNs);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                bool bad = false;                    // the tile's V holds an infinity or a NaN
                if (masked) {
                    ok = mbar_wait_bounded(bar(Sh::kVFull + vs), (uint32_t)(vround & 1), kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    uint4 *vt = reinterpret_cast<uint4 *>(data + Sh::kVOff + vs * Sh::kKVBytes);
                    uint32_t any = 0u;
#pragma unroll
                    for (int i = 0; i < Sh::kKVBytes / 16 / 128; ++i) {
                        const uint4 x = vt[i * 128 + r];
                        any |= nonfinite2<BF16>(x.x) | nonfinite2<BF16>(x.y) | nonfinite2<BF16>(x.z) | nonfinite2<BF16>(x.w);
                    }
                    const bool here = __any_sync(0xffffffffu, any != 0u);
                    if (lane == 0) {
                        s_bad[scans & 1][warp] = here;
                        mbar_arrive(bar(Sh::kScan));
                    }
                    ok = mbar_wait_bounded(bar(Sh::kScan), (uint32_t)(scans & 1), kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const volatile uint32_t *sb4 = s_bad[scans & 1];
                    bad = (sb4[0] | sb4[1] | sb4[2] | sb4[3]) != 0u;
                    ++scans;
                    if (here) {
#pragma unroll 1
                        for (int i = 0; i < Sh::kKVBytes / 16 / 128; ++i) {
                            uint4 x = vt[i * 128 + r];
                            uint32_t *w = &x.x;
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t f = nonfinite2<BF16>(w[e]);
                                w[e] &= ~(f * 0xffffu);
                            }
                            vt[i * 128 + r] = x;
                        }
                        fence_proxy_async_smem();
                    }
                }
                bool resc = false;
                float alpha = 1.f;
                uint32_t pk[32];
                if (warp_on) {
                    uint32_t raw[64];
                    tmem_ld64(tmem + lane_base + sb * kTreeKeys, raw);
                    float x[64];
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        x[c] = fold ? __uint_as_float(raw[c]) : __uint_as_float(raw[c]) * sm;
                    if (masked) {
                        const uint32_t vlo = (uint32_t)vis, vhi = (uint32_t)(vis >> 32);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            x[c] = (((c < 32 ? vlo : vhi) >> (c & 31)) & 1u) ? x[c] : kNegInf;
                    }
                    float mx[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mx[i] = fmaxf(x[2 * i], x[2 * i + 1]);
#pragma unroll
                    for (int c = 16; c < 64; c += 2)
                        mx[(c >> 1) & 7] = fmax3(mx[(c >> 1) & 7], x[c], x[c + 1]);
                    const float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * se;
                    resc = real && mt > m_used + 8.f;
                    const float m_new = resc ? mt : m_used;
                    alpha = resc ? ex2(m_used - m_new) : 1.f;
                    const float msub = m_new == kNegInf ? 0.f : m_new;
                    const uint64_t se2 = f2(se, se), nm2 = f2(-msub, -msub);
                    uint64_t rsv[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const uint64_t e = fma2(f2(x[2 * c], x[2 * c + 1]), se2, nm2);
                        pk[c] = pack2<BF16>(ex2(f2_lo(e)), ex2(f2_hi(e)));
                        const float2 pr = unpack2<BF16>(pk[c]);
                        rsv[c & 3] = add2(rsv[c & 3], f2(pr.x, pr.y));
                    }
                    const uint64_t r2 = add2(add2(rsv[0], rsv[1]), add2(rsv[2], rsv[3]));
                    l = l * alpha + (f2_lo(r2) + f2_hi(r2));
                    m_used = m_new;
                }
                if (t > s.k0) {
                    // P_{J-1} V_{J-1} has completed: O is stable, and O_DONE within one phase
                    ok = mbar_wait_bounded(bar(Sh::kODone), (uint32_t)((J - 1) & 1), kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + lane_base + c0, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(tO + lane_base + c0, o);
                        }
                    }
                }
                if (warp_on) {
                    tmem_st32(tmem + lane_base + sb * kTreeKeys, pk);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(Sh::kPFull + sb));
                if (++vs == Sh::kVStages) {
                    vs = 0;
                    ++vround;
                }
                if (bad) {
                    // rare: add the values taken out of V to the rows that see their keys
                    ok = mbar_wait_bounded(bar(Sh::kODone), (uint32_t)(J & 1), kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (warp_on) {
                        const int nblk = (s.len + BS - 1) / BS;
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + lane_base + c0, o);
#pragma unroll 1
                            for (int c = 0; c < kTreeKeys; ++c) {
                                const int bi = t * BPT + c / BS;
                                if (bi >= nblk)
                                    break;
                                const int shift = tail && bi == nblk - 1 ? BS - tail : 0;
                                const int cell = c % BS - shift;
                                if (cell < 0)
                                    continue;
                                int blk = __ldg(a.block_tables + (size_t)s.b * a.max_blocks + bi);
                                blk = (unsigned)blk < (unsigned)a.num_blocks ? blk : 0;
                                const uint32_t *v = reinterpret_cast<const uint32_t *>(
                                    a.value_cache + (((size_t)blk * BS + cell) * a.num_kv_heads + s.kvh) * D + c0);
                                const bool see = real && ((vis >> c) & 1ull);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const uint32_t x = __ldg(v + i);
                                    const uint32_t f = nonfinite2<BF16>(x);
                                    const float2 y = unpack2<BF16>(x);
                                    if (see && (f & 1u))
                                        o[2 * i] = __float_as_uint(__uint_as_float(o[2 * i]) + y.x);
                                    if (see && (f >> 16))
                                        o[2 * i + 1] = __float_as_uint(__uint_as_float(o[2 * i + 1]) + y.y);
                                }
                            }
                            tmem_st32(tO + lane_base + c0, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
            }
            if (ok)
                ok = mbar_wait_bounded(bar(Sh::kODone), (uint32_t)((J - 1) & 1), kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !warp_on)
                continue;
            tc_fence_after();
            if (s.k0 == 0 && s.k1 == s.tiles) {
                // the whole item: output rows.  The four lanes of a quad trade
                // 16-byte chunks, so that a store covers 64 bytes of a row.
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint4 *orow[4];
                int tk = rq_tok, hd = rq_head;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    orow[h] = r - q + h < rows
                                  ? reinterpret_cast<uint4 *>(a.out + ((size_t)(s.q0 + s.rt * TT + tk) * a.num_heads +
                                                                       (size_t)s.kvh * G + hd) * D)
                                  : nullptr;
                    if (++hd == G) {
                        hd = 0;
                        ++tk;
                    }
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 64) {
                    uint32_t o[64];
                    tmem_ld64(tO + lane_base + c0, o);
#pragma unroll
                    for (int g2 = 0; g2 < 2; ++g2) {
                        uint4 ch[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack2<BF16>(__uint_as_float(o[32 * g2 + 8 * v + 2 * e]) * inv,
                                                   __uint_as_float(o[32 * g2 + 8 * v + 2 * e + 1]) * inv);
                            ch[v] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        quad_transpose(ch, q);
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            if (orow[h] != nullptr)
                                orow[h][(c0 + 32 * g2) / 8 + q] = ch[h];
                    }
                }
            } else {
                // a part of an item: a record (m, l, O), part 1 if the item starts here
                const size_t rec = (((size_t)blockIdx.x * 2 + w_share) * 2 + (s.k0 > 0 ? 0 : 1)) * kTreeRows + r;
                float4 *orec = reinterpret_cast<float4 *>(a.rec_o + rec * D);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + lane_base + c0, o);
                    if (real) {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            orec[c0 / 4 + v] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                           __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                    }
                }
                if (real)
                    a.rec_ml[rec] = make_float2(m_used, l);
            }
            // the next part's first P V overwrites O after this warp's next P
        }
        if (!ok && lane == 0)
            raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The records of an item that several CTAs shared, joined by log-sum-exp:
//   out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k,   M = max_k m_k.
// CTA (c, x, share) takes rows 32 x .. 32 x + 31 of the item whose second part
// opens CTA c's share; a warp takes a row, a lane D / 32 of its columns.
template <int D, bool BF16>
__global__ void __launch_bounds__(256)
tree_merge_kernel(const TreeArgs a)
{
    constexpr int V = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int c = blockIdx.x, share = blockIdx.z;
    const int4 d = __ldg(a.desc + c * 2 + share);
    const int step = a.shares == 2 && share == 0 ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (d.w == 0)
        return;
    for (int r = blockIdx.y * 32 + warp; r < min(d.y, (int)(blockIdx.y + 1) * 32); r += 8) {
        // record k: CTA c + (k - 1) step; part 1 of the first, part 0 of the others
        auto rec = [&](int k) {
            return (((size_t)(c + (k - 1) * step) * 2 + share) * 2 + (k == 0 ? 1 : 0)) * kTreeRows + r;
        };
        float M = kNegInf;
        for (int k = lane; k < d.w; k += 32)
            M = fmaxf(M, __ldg(&a.rec_ml[rec(k)].x));
#pragma unroll
        for (int o = 16; o; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float den = 0.f, acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = 0.f;
#pragma unroll 4
        for (int k = 0; k < d.w; ++k) {
            const float2 ml = __ldg(a.rec_ml + rec(k));
            float v[V];
            load_slice<D>(a.rec_o + rec(k) * D + lane * V, v);
            const float f = ml.x == kNegInf ? 1.f : ex2(ml.x - M);   // (1: a part without keys, or all NaN)
            den += f * ml.y;
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[i] += f * v[i];
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        uint16_t *o = a.out + ((size_t)(d.x + r / a.group) * a.num_heads + (size_t)d.z * a.group + r % a.group) * D + lane * V;
        if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv),
                                                       pack2<BF16>(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t *>(o) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
    }
}

}  // namespace pkv
