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

#include <type_traits>

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
    const int r_step = 32 / words, w_step = 32 - r_step * words;
    int r = lane / words, w = lane - r * words;
#pragma unroll 4
    for (int e = lane; e < rows * words; e += 32) {
        out[e] = (int32_t)s_row[warp][r][w];
        r += r_step;
        w += w_step;
        if (w >= words) {
            w -= words;
            ++r;
        }
    }
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
template <int NT>
__global__ void __launch_bounds__(NT)
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
    for (int i = threadIdx.x; i < s.n; i += NT)
        s_next[i] = kTreeMaxNodes;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += NT) {
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
    for (int i = threadIdx.x; i < max_query_len; i += NT)
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
// with P over S in tensor memory, S double-buffered, and the reference m (the
// running maximum, for bf16 raised by tree_headroom) moved only when a tile's
// maximum exceeds the one it was taken from by 2^8.  Only the last key tiles of a
// sequence hold drafted keys: they alone are masked, by 64 bits per row cut
// from the row's mask words.  A tile's scores are read twice, for the maximum
// and, 32 at a time by a loop, for the weights: less code and no spills, since
// the warps' different work fills the instruction cache (256 sequences of 512
// .. 640 tokens, 32/8 heads, 8 and 32 nodes: 120 and 166 us with the weights of
// 64 keys unrolled, 117 and 160 so; 8 of 16-32 K tokens and 64 nodes 283, 285).
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
// Calls with little to do in all are bound by latency: working out the shares
// and a second kernel would cost as much as the attention.  There (CL) a
// cluster of 1, 2, 4 or 8 CTAs takes an item, a CTA an equal run of its key
// tiles, and the partial results are joined through the cluster's shared
// memory: one kernel, no workspace.
//
// A masked tile is the only one whose V rows some row may not see: such a row
// gives them weight 0, and 0 times an infinity or a NaN would poison it.  Warp 7
// looks through the V rows of masked tiles; where one holds such a value, it
// zeroes it in shared memory and the softmax warps add it to the rows that do
// see it.
//
// Up to 64 rows over long contexts (TR, head_dim 128) half of a 128-row tile's
// products and weights and more would be for rows that do not exist, and
// in a power-limited run they cost clock.  There the products are transposed:
//
//   S^T[keys x rows] = K_j Q^T,   O^T[D x rows] += V_j^T P_j^T
//
// 128 keys to a tile and 64 rows as the products' N.  A softmax thread is a
// key, so a row's maximum is the CTA's: it lies in shared memory, all weights
// of a tile are taken against it, and the four warps vote whether a score lies
// more than 2^14 above it; only then (seldom: a part starts with its first
// key's scores) the true maxima are worked out by exchanges.  Row sums stay
// spread over the threads, by mma.sync products of the weights' registers with
// ones.  P^T goes through shared memory as the second product's B; V^T is its
// A, with head_dim along the rows as it lies.  A part's end is dearer than
// with 128-row tiles (2-byte stores, a column of the head per thread), the
// tile half as dear: 32 sequences of 3-4 K tokens, 32/8 heads, 8 nodes 88 us
// against 94, 16 nodes 94 against 119 (sustained 99, 113); 8 of 16-32 K and 16
// nodes 140 against 149 (sustained 154, 178); at 512 .. 640 tokens and 10 nodes
// 170 against 127, level near 1000 tokens.
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
    int row_tiles;                   // of the largest tree (CL: items are (sequence, kv head, row tile))
    int shares;                      // 2: pairs of row tiles, then single ones; 1: single ones only
    int q_box;                       // query tokens that a Q copy brings
    int q_slots;                     // 2: two Q buffers of 64 rows (no item has more), 1: one of 128
    float scale_log2;
};

constexpr int kTreeThreads = 256;
constexpr int kTreeRows = 128;           // query rows per tile (MMA M)
constexpr int kTreeKeys = 64;            // keys per tile
constexpr int kTreeItemCost = 2;         // an item's start and end, in key tiles (1 to 5: within 4 %, 1 and 2 ahead)
constexpr int kTreeMinUnits = 2;         // a CTA's share is not cut below this

constexpr int kTreeParts = 6;            // queue of parts between a CTA's warps
constexpr int kTreeScans = 8;            // masked tiles whose scan result is kept

// Shared memory and barriers of a CTA; TR: of the transposed products.
template <int D, bool TR>
struct TreeShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kKeys = TR ? 128 : kTreeKeys;           // keys per tile; V comes 64 at a time
    // two Q buffers of 64 rows: one after the other TR, else the halves of each 64-column half
    static constexpr int kQHalf = (TR ? 64 : kTreeRows) * 128;
    static constexpr int kQSlot = TR ? kHalves * kQHalf : 64 * 128;
    static constexpr int kQBytes = kHalves * kTreeRows * 128;
    static constexpr int kKHalf = kKeys * 128;
    static constexpr int kKBytes = kHalves * kKHalf;
    static constexpr int kVHalf = kTreeKeys * 128;
    static constexpr int kVBytes = kHalves * kVHalf;
    // two CTAs per SM: 112 KB each for D = 128 (32 + 80), 96 KB for D = 64 (16 + 80)
    static constexpr int kKStages = TR ? 1 : (D == 128 ? 3 : 6);
    static constexpr int kVStages = D == 128 ? 2 : 4;
    static constexpr int kKOff = kQBytes;
    static constexpr int kVOff = kKOff + kKStages * kKBytes;
    static constexpr int kPOff = kVOff + kVStages * kVBytes;     // TR: the weights, 128 keys x 64 rows
    static constexpr int kDataBytes = kPOff + (TR ? 128 * 128 : 0);
    static constexpr int kSmemBytes = kDataBytes + 1024;
    // barriers
    static constexpr int kQFull = 0, kQEmpty = 2, kKFull = 4, kKEmpty = kKFull + kKStages, kVFull = kKEmpty + kKStages,
                         kVEmpty = kVFull + kVStages, kScanReq = kVEmpty + kVStages, kScanned = kScanReq + 1, kSFull = kScanned + 1,
                         kPFull = kSFull + 2, kODone = kPFull + 2, kDrain = kODone + 1, kVote = kDrain + 1, kShare = kVote + 1,
                         kPartFull = kShare + 1, kPartEmpty = kPartFull + kTreeParts, kNumBars = kPartEmpty + kTreeParts;
};

// A part of an item: key tiles k0 .. k1 - 1 of `tiles` for one row tile of a
// (sequence, kv head).  k1 = 0 ends a CTA's parts.
struct TreePart {
    int b, kvh, rt, share;
    int q0, n, len;   // the sequence's rows and length
    int tiles;        // key tiles of the item
    int k0, k1;
};
// Units g .. end - 1 of a sequence of units, sequence b's first unit being seq0.
struct TreeWalk {
    int g, end, seq0, b;
};

// Items of a sequence: single row tiles, or pairs of them.
__device__ __forceinline__ int tree_items(int n, int G, int shares, int share)
{
    const int tt = kTreeRows / G;
    const int rt = (n + tt - 1) / tt;
    return shares == 1 ? rt : (share == 0 ? rt / 2 : rt & 1);
}
// Units of sequence b (0 where it contradicts itself).  The host keeps the
// total below 2^31.
template <int BS, int KEYS>
__device__ __forceinline__ int tree_units(const TreeArgs &a, int b, int share, TreeSeq *s)
{
    if (!tree_seq(a.query_start, a.context_lens, b, a.num_tokens, a.max_query_len, a.max_blocks * BS, s))
        return -1;
    return tree_items(s->n, a.group, a.shares, share) * a.num_kv_heads *
           ((s->len + KEYS - 1) / KEYS + kTreeItemCost);
}

template <int BS, int KEYS>
__device__ __forceinline__ bool tree_next(TreeWalk &w, const TreeArgs &a, int share, int member, TreePart *p)
{
    while (w.g < w.end) {
        TreeSeq q;
        const int units = max(0, tree_units<BS, KEYS>(a, w.b, share, &q));
        const int off = w.g - w.seq0;
        if (off >= units) {
            w.seq0 += units;
            ++w.b;
            continue;
        }
        const int tiles = (q.len + KEYS - 1) / KEYS;
        const int cost = tiles + kTreeItemCost;
        const int item = off / cost;
        const int k0 = off - item * cost;
        const int step = min(cost - k0, w.end - w.g);
        w.g += step;
        if (k0 >= tiles)
            continue;
        const int r = item / a.num_kv_heads;
        p->b = w.b;
        p->kvh = item - r * a.num_kv_heads;
        // pairs: row tiles 2 r and 2 r + 1; beside pairs, the odd last row tile
        const int tt = kTreeRows / a.group;
        p->rt = a.shares == 1 ? r : (share == 0 ? 2 * r + member : (q.n + tt - 1) / tt - 1);
        p->share = share;
        p->q0 = q.q0;
        p->n = q.n;
        p->len = q.len;
        p->tiles = tiles;
        p->k0 = k0;
        p->k1 = min(tiles, k0 + step);
        return true;
    }
    return false;
}

__device__ __forceinline__ int tree_cut(int total, int c, int n)   // the first unit of CTA (or pair) c of n
{
    const int q = total / n;
    return q * c + (total - q * n) * c / n;
}
__device__ __forceinline__ int tree_ctas(int total, int most)      // CTAs (or pairs) that share the units
{
    return min(most, max(1, (total + kTreeMinUnits - 1) / kTreeMinUnits));
}

// How far (in powers of two) the reference that a row's weights are taken
// against lies above the row's maximum.  The weights are summed unnormalised,
// and reach 2^move over the maximum that they were first taken against; bf16
// values reach 2^128, so `len` such products would overflow the 32-bit
// accumulator where their average does not.  With the reference this much
// higher the weights of a row add up to less than one.  bf16 has the range for
// it, and weights that vanish now are below 2^-80 of the largest.  What it costs
// are bits of sums of the smallest values, as 32-bit subnormals: over 1300 keys
// the outputs are as exact as ever for values from 2^-118 (transposed: 2^-112)
// to 2^128, and lose bits below (values of 2^-124: 0.6 %, transposed 20 %).
// Times stay within 1 % (one user's 4000 tokens, few rows: 15.6 to 16.0 us).  f16
// has neither such values nor the range for such weights.
template <bool BF16>
__device__ __forceinline__ float tree_headroom(int len, int move)
{
    return BF16 ? (float)(33 - __clz(len) + move) : 0.f;
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

// acc stays 0 until a value is an infinity or a NaN (0 times it is NaN).
template <bool BF16>
__device__ __forceinline__ uint32_t fma_zero2(uint32_t x, uint32_t acc)
{
    if constexpr (BF16)
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
}

// (a NaN stays)
__device__ __forceinline__ float fmax3_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// TR: the query rows (bit c: row c) that see the key in cell `cell` of the
// block whose first position is p0 (no row: a cell that holds none).
template <int BS, int UNROLL>
__device__ __forceinline__ uint64_t tree_rows_that_see(const int32_t *mask, int words, int G, int n, int len, int p0, int cell)
{
    const int tail = len % BS;
    if (p0 >= len)
        return 0ull;
    if (tail && p0 + BS > len)
        cell -= BS - tail;                   // a partly filled last block ends its slot
    if (cell < 0)
        return 0ull;
    const int j = p0 + cell - (len - n);
    if (j < 0)
        return ~0ull;
    mask += j >> 5;
    const uint64_t rows = (1ull << G) - 1ull;            // (G <= 8)
    uint64_t v = 0ull;
#pragma unroll UNROLL
    for (int i = 0; i < n; ++i)
        v |= ((uint32_t)__ldg(mask + (size_t)i * words) >> (j & 31)) & 1u ? rows << (i * G) : 0ull;
    return v;
}

// O_row += the infinities and NaN of V's rows of key tile t that the row sees
// (they were zeroed in shared memory).  Rare, so simple: one key at a time,
// read from the cache again.
template <int D, int BS, bool BF16>
__device__ __noinline__ void tree_add_nonfinite(const uint16_t *value_cache, const int32_t *table, int num_blocks,
                                                int num_kv_heads, int kvh, int len, int t, uint64_t vis, uint32_t tO)
{
    const int nblk = (len + BS - 1) / BS, tail = len % BS;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c0, o);
#pragma unroll 1
        for (int c = 0; c < kTreeKeys; ++c) {
            const int bi = t * (kTreeKeys / BS) + c / BS;
            if (bi >= nblk)
                break;
            const int cell = c % BS - (tail && bi == nblk - 1 ? BS - tail : 0);
            if (cell < 0)
                continue;
            int blk = __ldg(table + bi);
            blk = (unsigned)blk < (unsigned)num_blocks ? blk : 0;
            const uint32_t *v = reinterpret_cast<const uint32_t *>(
                value_cache + (((size_t)blk * BS + cell) * num_kv_heads + kvh) * D + c0);
            const bool see = (vis >> c) & 1ull;
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
        tmem_st32(tO + c0, o);
    }
    tmem_wait_st();
}

// The same for the transposed products: thread = column `col` of the head, the
// tile's 128 keys one at a time, query row c in TMEM column c.  (Inline and
// few registers: a call here had the key loop's registers spilled.)
template <int BS, bool BF16>
__device__ __forceinline__ void tree_add_nonfinite_t(const uint16_t *value_cache, const int32_t *table, int num_blocks, int kvs, int kvh,
                                                     const int32_t *mask, int words, int G, int n, int len, int t, int col, uint32_t tO)
{
#pragma unroll 1
    for (int k = 0; k < 128; ++k) {
        const int p0 = t * 128 + k / BS * BS;
        uint64_t vis = tree_rows_that_see<BS, 1>(mask, words, G, n, len, p0, k % BS) & (~0ull >> (64 - n * G));
        if (vis == 0ull)
            continue;
        const int tail = len % BS;
        const int cell = k % BS - (tail && p0 + BS > len ? BS - tail : 0);
        int blk = __ldg(table + p0 / BS);
        blk = (unsigned)blk < (unsigned)num_blocks ? blk : 0;
        const uint32_t x = __ldg(value_cache + (((size_t)blk * BS + cell) * kvs + kvh) * 128 + col);
        const bool bad = nonfinite2<BF16>(x) & 1u;
        if (!__any_sync(0xffffffffu, bad))
            continue;
        const float y = bad ? unpack2<BF16>(x).x : 0.f;
        for (; vis; vis &= vis - 1ull) {
            const uint32_t at = tO + (uint32_t)__ffsll((long long)vis) - 1u;
            const float o = tmem_ld1(at);
            tmem_st1(at, bad ? o + y : o);
            tmem_wait_st();
        }
    }
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `addr` (own shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Warps: 0-3 softmax and output (warp w owns TMEM lanes 32 w ..), 4 K loads,
// 5 MMA issue, 6 V loads, 7 the parts' queue, Q loads and the scan of masked
// tiles' V rows.
template <int D, int BS, bool BF16, bool CL, bool TR>
__global__ void __launch_bounds__(kTreeThreads, 2)
tree_attend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k4,
                   const __grid_constant__ CUtensorMap tm_v4, const __grid_constant__ TreeArgs a)
{
    using Sh = TreeShape<D, TR>;
    static_assert(!TR || (D == 128 && !CL), "the transposed products have head_dim as M; clusters have few tiles");
    constexpr int KEYS = Sh::kKeys;
    constexpr int KS = D / 16, KV_STEPS = kTreeKeys / 16;
    constexpr uint32_t kTmemCols = 256;          // S/P: 2 x 64 columns, O: D columns at 128
    // The dynamic shared memory is all that the kernel has, so it starts on the
    // 1024-byte boundary that the swizzled tiles need; what else the CTA keeps
    // follows them (with 1 KB more two CTAs would not fit an SM).
    struct Local {
        uint64_t bars[Sh::kNumBars];
        TreeWalk walk[2];
        int total[2];
        int scan[kTreeThreads / 32];
        uint32_t bad[kTreeScans];
        uint32_t vote[2][4];
        alignas(16) float m[TR ? 64 : 4];
        uint32_t tmem;
        TreePart part[kTreeParts];
    };
    static_assert(sizeof(Local) <= 1024, "fits behind the tiles");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *data = smem_raw;
    const uint32_t data_s = smem_addr(data);
    Local *loc = reinterpret_cast<Local *>(data + Sh::kDataBytes);
    TreePart *s_part = loc->part;
    if (data_s & 1023u) {                            // (never seen: fail loudly, not by wrong tiles)
        if (threadIdx.x == 0)
            raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
        return;
    }
    const uint32_t bars_s = smem_addr(loc->bars);
    auto bar = [&](int i) { return bars_s + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group, TT = kTreeRows / G, R = TT * G;

    if (threadIdx.x < Sh::kNumBars) {
        const int i = threadIdx.x;
        // P: one arrival per softmax warp; a part is read by K, V and MMA warps and the softmax warps
        const int count = (i >= Sh::kPFull && i < Sh::kPFull + 2) || i == Sh::kVote || i == Sh::kShare
                              ? 4 : (i >= Sh::kPartEmpty ? 7 : 1);
        mbar_init(bar(i), count);
    }
    if (threadIdx.x == 128) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_k4);
        prefetch_tensormap(&tm_v4);
    }
    fence_mbar_init();
    // masked columns of a tile may meet V rows that no load has filled; TR: so
    // may Q rows and weights past the tree's rows, and zeros cost least power
    {
        uint4 *vr = reinterpret_cast<uint4 *>(data + Sh::kVOff);
        for (int i = threadIdx.x; i < (Sh::kDataBytes - Sh::kVOff) / 16; i += kTreeThreads)
            vr[i] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (TR) {
            uint4 *qr = reinterpret_cast<uint4 *>(data);
            for (int i = threadIdx.x; i < Sh::kQBytes / 16; i += kTreeThreads)
                qr[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // (after the wait: a kernel before this one may still be taking its own)
    if (warp == 5) {
        tmem_alloc(smem_addr(&loc->tmem), kTmemCols);
        tmem_relinquish();
    }

    int cl_tiles = 0, cl_rows = 0, cl_q0 = 0, cl_kvh = 0;   // CL: the item, if it is joined (else cl_rows is 0)
    if constexpr (CL) {
        // ---- the CTA's one part: key tiles tiles x / P .. tiles (x + 1) / P - 1 of item y ----
        const int item = blockIdx.y, P = gridDim.x;
        const int bh = item / a.row_tiles, rt = item - bh * a.row_tiles;
        const int b = bh / a.num_kv_heads, kvh = bh - b * a.num_kv_heads;
        TreeSeq q;
        const bool good = tree_seq(a.query_start, a.context_lens, b, a.num_tokens, a.max_query_len, a.max_blocks * BS, &q);
        if (!good && threadIdx.x == 0 && blockIdx.x == 0 && rt == 0 && kvh == 0)
            raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
        const int rows = good ? min(R, q.n * G - rt * R) : 0;
        const int tiles = rows > 0 ? (q.len + KEYS - 1) / KEYS : 0;
        if (threadIdx.x == 0) {
            TreePart p{b, kvh, rt, 0, q.q0, q.n, q.len, tiles, tiles * (int)blockIdx.x / P, tiles * ((int)blockIdx.x + 1) / P};
            if (p.k0 == p.k1)
                p.k1 = 0;
            loc->part[0] = p;
            loc->part[1].k1 = 0;
        }
        if (P > 1 && tiles > 1) {                    // (a single tile is one CTA's alone)
            cl_tiles = tiles;
            cl_rows = rows;
            cl_q0 = q.q0 + rt * TT;
            cl_kvh = kvh;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        // (behind the block's barrier: other threads initialised these two)
        if (threadIdx.x == 0) {
            mbar_arrive(bar(Sh::kPartFull));
            mbar_arrive(bar(Sh::kPartFull + 1));
        }
    }
    // ---- this CTA's shares: a thread adds up a run of sequences, the block
    // their totals; the thread whose run holds the share's start finds it ----
    for (int share = 0; !CL && share < a.shares; ++share) {
        const bool pair = a.shares == 2 && share == 0;
        const int per = (a.batch + kTreeThreads - 1) / kTreeThreads;
        const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            TreeSeq q;
            const int u = tree_units<BS, KEYS>(a, b, share, &q);
            if (u < 0 && blockIdx.x == 0 && share == 0)
                raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
            mine += max(u, 0);
        }
        int upto = mine;                             // inclusive prefix over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += x;
        }
        if (lane == 31)
            loc->scan[warp] = upto;
        if (threadIdx.x == 0)
            loc->walk[share] = TreeWalk{0, 0, 0, 0}; // an empty share
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int i = 0; i < kTreeThreads / 32; ++i) {
            const int x = loc->scan[i];
            if (i < warp)
                upto += x;
            total += x;
        }
        const int n = tree_ctas(total, pair ? gridDim.x / 2 : gridDim.x);
        const int c = pair ? blockIdx.x >> 1 : blockIdx.x;
        const int g0 = c < n ? tree_cut(total, c, n) : total;
        if (g0 >= upto - mine && g0 < upto) {
            int at = upto - mine, b = b0;
            for (;; ++b) {
                TreeSeq q;
                const int u = max(0, tree_units<BS, KEYS>(a, b, share, &q));
                if (g0 < at + u)
                    break;
                at += u;
            }
            loc->walk[share] = TreeWalk{g0, tree_cut(total, c + 1, n), at, b};
        }
        if (threadIdx.x == 0)
            loc->total[share] = total;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&loc->tmem);

    const uint32_t sQ = data_s, sK = data_s + Sh::kKOff, sV = data_s + Sh::kVOff;
    const uint32_t tO = tmem + 2 * kTreeKeys;
    const bool two_q = a.q_slots == 2;               // at most 64 rows: two Q buffers of 64 rows

    // The parts in order, from the queue that warp 7 fills (used by whole
    // warps, or by one thread with one = true); false at their end.
    int part_i = 0;
    auto next_part = [&](TreePart *p, bool one) -> bool {
        const int slot = part_i % kTreeParts;
        bool got = mbar_wait_tries(bar(Sh::kPartFull + slot), (uint32_t)((part_i / kTreeParts) & 1));
        if (!one)
            got = __all_sync(0xffffffffu, got);
        if (!got) {
            if (one || lane == 0)
                raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
            return false;
        }
        *p = s_part[slot];
        if (!one)
            __syncwarp();
        if (one || lane == 0)
            mbar_arrive(bar(Sh::kPartEmpty + slot));
        ++part_i;
        return p->k1 > 0;
    };

    if (warp == 4 || warp == 6) {
        // ---- loads: warp 4 the K ring, warp 6 the V ring ----
        const bool is_k = warp == 4;
        const CUtensorMap *tm = is_k ? &tm_k : &tm_v;        // 3-D view: whole blocks
        const CUtensorMap *tm4 = is_k ? &tm_k4 : &tm_v4;     // 4-D view: shifted last blocks
        const int full0 = is_k ? Sh::kKFull : Sh::kVFull;
        const int empty0 = is_k ? Sh::kKEmpty : Sh::kVEmpty;
        const uint32_t ring = is_k ? sK : sV;
        const int NS = is_k ? Sh::kKStages : Sh::kVStages;
        const uint64_t once = policy_evict_first(), again = policy_evict_normal();
        int J = 0, st = 0, round = 0;
        bool ok = true;
        TreePart s;
        while (ok && next_part(&s, false)) {
            // a pair's keys are read a second time, by the other CTA
            const uint64_t policy = (CL ? a.row_tiles > 1 : a.shares == 2 && s.share == 0) ? again : once;
            const int nblk = (s.len + BS - 1) / BS;
            const int tail = s.len % BS;
            const int32_t *trow = a.block_tables + (size_t)s.b * a.max_blocks;
            int ids = 0, have = -1;                  // block ids of the 32-entry window `have`
            // K by tiles, V by 64 keys
            const int bpt = (is_k ? KEYS : kTreeKeys) / BS;
            const int per = is_k ? 1 : KEYS / kTreeKeys;
            const int t1 = is_k ? s.k1 : min(s.k1 * per, (s.len + kTreeKeys - 1) / kTreeKeys);
            for (int t = s.k0 * per; t < t1; ++t, ++J) {
                const int kb0 = t * bpt;             // a tile's ids lie in one window
                const int nb = min(bpt, nblk - kb0);
                if ((kb0 & ~31) != have) {
                    have = kb0 & ~31;
                    ids = have + lane < nblk ? __ldg(trow + have + lane) : 0;
                }
                if (J >= NS) {
                    const bool free_ = mbar_wait_tries(bar(empty0 + st), (uint32_t)((round - 1) & 1));
                    if (!__all_sync(0xffffffffu, free_)) {
                        ok = false;
                        break;
                    }
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(full0 + st), (uint32_t)(nb * BS * D * 2));
                __syncwarp();
                const int i = lane / Sh::kHalves, h = lane % Sh::kHalves;
                int blk = __shfl_sync(0xffffffffu, ids, (kb0 + min(i, bpt - 1)) & 31);
                if (i < nb) {
                    if ((unsigned)blk >= (unsigned)a.num_blocks) {
                        if (h == 0)
                            raise_flag(PKV_DEVFLAG_BLOCK_RANGE);
                        blk = 0;
                    }
                    // a partly filled last block ends at its slot's last row; the rows before read as zero
                    const int shift = tail && kb0 + i == nblk - 1 ? tail - BS : 0;
                    const uint32_t dst = ring + st * (is_k ? Sh::kKBytes : Sh::kVBytes) + h * (is_k ? Sh::kKHalf : Sh::kVHalf) + i * BS * 128;
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
                mbar_wait_tries(bar(full0 + j % NS), (uint32_t)((j / NS) & 1));
        if (!CL && is_k && lane < a.shares) {
            // An item that started in the share before and goes on in this one:
            // the merge finds its records through this share.
            const int share = lane;
            const bool pair = a.shares == 2 && share == 0;
            const int total = loc->total[share];
            const int n = tree_ctas(total, pair ? gridDim.x / 2 : gridDim.x);
            const int c = pair ? blockIdx.x >> 1 : blockIdx.x;
            int4 d = make_int4(0, 0, 0, 0);
            TreeWalk w = loc->walk[share];
            TreeSeq q;
            if (c > 0 && w.g < w.end && tree_units<BS, KEYS>(a, w.b, share, &q) > 0) {
                const int tiles = (q.len + KEYS - 1) / KEYS;
                const int k0 = (w.g - w.seq0) % (tiles + kTreeItemCost);
                const int start = w.g - k0;          // the item's first unit
                TreePart p;
                if (k0 > 0 && k0 < tiles && start >= tree_cut(total, c - 1, n) &&
                    tree_next<BS, KEYS>(w, a, share, blockIdx.x & 1, &p)) {
                    // the last CTA (or pair) with keys of the item: about (its end) n / total
                    int last = (int)min((int64_t)(n - 1), (int64_t)(start + tiles) * n / total);
                    while (tree_cut(total, last, n) >= start + tiles)
                        --last;
                    while (last + 1 < n && tree_cut(total, last + 1, n) < start + tiles)
                        ++last;
                    d = make_int4(p.q0 + p.rt * TT, min(R, p.n * G - p.rt * R), p.kvh, last - c + 2);
                }
            }
            a.desc[blockIdx.x * 2 + share] = d;
        }
    } else if (warp == 7) {
        // ---- the queue, Q, and the scan of masked tiles ----
        // Parts are queued up to four ahead of the one whose tiles are scanned
        // here: the loaders run at most their rings ahead of the MMAs.
        constexpr int kAhead = 4;
        const uint64_t policy = policy_evict_normal();
        TreeWalk walk = CL ? TreeWalk{} : loc->walk[0];
        int share = 0, made = CL ? 2 : 0, scans = 0, vs = 0, vround = 0;
        bool ok = true, done = CL;
        auto make = [&]() {                          // queue part `made`
            const int slot = made % kTreeParts;
            if (made >= kTreeParts &&
                !__all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kPartEmpty + slot),
                                                           (uint32_t)((made / kTreeParts - 1) & 1)))) {
                ok = false;
                return;
            }
            TreePart p;
            while (!tree_next<BS, KEYS>(walk, a, share, blockIdx.x & 1, &p)) {
                if (++share >= a.shares) {
                    done = true;
                    p.k1 = 0;
                    break;
                }
                walk = loc->walk[share];
            }
            if (lane == 0) {
                s_part[slot] = p;
                mbar_arrive(bar(Sh::kPartFull + slot));
            }
            __syncwarp();
            ++made;
        };
        auto load_q = [&](int u, const TreePart &p) {
            const int slot = two_q ? u & 1 : 0;
            const int turn = two_q ? u >> 1 : u;
            if (turn > 0 && !__all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kQEmpty + slot), (uint32_t)((turn - 1) & 1)))) {
                ok = false;
                return;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(Sh::kQFull + slot), (uint32_t)(Sh::kHalves * a.q_box * G * 128));
#pragma unroll
                for (int h = 0; h < Sh::kHalves; ++h)
                    tma_load_3d(sQ + h * Sh::kQHalf + slot * Sh::kQSlot, &tm_q, bar(Sh::kQFull + slot), h * 64, p.kvh * G,
                                p.q0 + p.rt * TT, policy);
            }
            __syncwarp();
        };
        int u = 0, loaded = 0;                       // part scanned; Q loads issued
        while (ok) {
            while (ok && !done && made <= u + kAhead)
                make();
            if (!ok)
                break;
            const TreePart s = s_part[u % kTreeParts];   // (rewritten only by this warp, when made reaches u + kTreeParts)
            if (s.k1 == 0)
                break;
            if (loaded == u) {
                load_q(u, s);
                ++loaded;
            }
            if (two_q && ok) {
                const TreePart nx = s_part[(u + 1) % kTreeParts];   // made > u + 1, or the end marker
                if (nx.k1 > 0) {
                    load_q(u + 1, nx);
                    ++loaded;
                }
            }
            for (int t = s.k0; ok && t < s.k1; ++t) {
                const bool masked = (t + 1) * KEYS > s.len - s.n;
                // the MMA thread asks for it when the tile's V has landed: this
                // warp's place in the tiles says nothing of the V ring's
                if (masked && !__all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kScanReq), (uint32_t)(scans & 1)))) {
                    ok = false;
                    break;
                }
                bool bad = false;
                for (int v = t * (KEYS / kTreeKeys); v < (t + 1) * (KEYS / kTreeKeys) && v * kTreeKeys < s.len; ++v) {
                    if (masked) {
                        mbar_wait_tries(bar(Sh::kVFull + vs), (uint32_t)(vround & 1));   // (has landed)
                        // V rows that some query row may not see: from the first drafted
                        // key on (a shifted last block puts it further on), four at a time
                        const int i0 = max(0, s.len - s.n - v * kTreeKeys) / 4;
                        uint4 *vt = reinterpret_cast<uint4 *>(data + Sh::kVOff + vs * Sh::kVBytes) + lane;
                        uint32_t any[4] = {0u, 0u, 0u, 0u};
#pragma unroll 4
                        for (int i = i0 * Sh::kHalves; i < Sh::kVBytes / 512; ++i) {
                            // (the rows of the 64-column halves in turn)
                            const int row4 = i / Sh::kHalves, h = i - row4 * Sh::kHalves;
                            const uint4 x = vt[h * (Sh::kVHalf / 16) + row4 * 32];
                            any[0] = fma_zero2<BF16>(x.x, any[0]);
                            any[1] = fma_zero2<BF16>(x.y, any[1]);
                            any[2] = fma_zero2<BF16>(x.z, any[2]);
                            any[3] = fma_zero2<BF16>(x.w, any[3]);
                        }
                        // (a sum of zeros is 0 or -0)
                        if (__any_sync(0xffffffffu, ((any[0] | any[1] | any[2] | any[3]) & 0x7fff7fffu) != 0u)) {
                            bad = true;
                            uint32_t *w = reinterpret_cast<uint32_t *>(data + Sh::kVOff + vs * Sh::kVBytes) + lane;
#pragma unroll 1
                            for (int i = 0; i < Sh::kVBytes / 128; ++i)
                                w[i * 32] &= ~(nonfinite2<BF16>(w[i * 32]) * 0xffffu);
                            fence_proxy_async_smem();
                        }
                    }
                    if (++vs == Sh::kVStages) {
                        vs = 0;
                        ++vround;
                    }
                }
                if (masked) {
                    __syncwarp();
                    if (lane == 0) {
                        loc->bad[scans % kTreeScans] = bad;
                        mbar_arrive(bar(Sh::kScanned));
                    }
                    ++scans;
                }
            }
            ++u;
        }
        if (!ok && lane == 0)
            raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
        // the last Q loads land before the CTA can exit
        if (lane == 0)
            for (int i = max(0, loaded - (two_q ? 2 : 1)); i < loaded; ++i)
                mbar_wait_tries(bar(Sh::kQFull + (two_q ? i & 1 : 0)), (uint32_t)((two_q ? i >> 1 : i) & 1));
    } else if (!TR && warp == 5) {
        // ---- MMA issue: one thread ----
        if (lane == 0) {
            constexpr uint32_t idS = f16_idesc<BF16>(kTreeRows, kTreeKeys, false);
            constexpr uint32_t idO = f16_idesc<BF16>(kTreeRows, D, true);
            int ks_ = 0, kround = 0;                 // K stage of the next S
            // S of global tile J; u: its part (Q buffer); last: the part's last S
            auto k_ready = [&]() -> bool {
                return mbar_wait_tries(bar(Sh::kKFull + ks_), (uint32_t)(kround & 1));
            };
            auto issue_s = [&](int J, int u, bool last) {
                tc_fence_after();
                const uint32_t kt = sK + ks_ * Sh::kKBytes;
                // with two Q buffers the rows past a buffer's 64 read what lies
                // behind it: rows that nobody reads
                const uint32_t qt = sQ + (two_q ? (u & 1) * 64 * 128 : 0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t koff = (uint32_t)((ks & 3) * 32);
                    tc_mma_f16(tmem + (J & 1) * kTreeKeys, sw128_desc(qt + (ks >> 2) * Sh::kQHalf + koff, 16, 1024),
                               sw128_desc(kt + (ks >> 2) * Sh::kKHalf + koff, 16, 1024), idS, ks > 0 ? 1u : 0u);
                }
                tc_commit(bar(Sh::kSFull + (J & 1)));
                tc_commit(bar(Sh::kKEmpty + ks_));
                if (last)
                    tc_commit(bar(Sh::kQEmpty + (two_q ? u & 1 : 0)));
                if (++ks_ == Sh::kKStages) {
                    ks_ = 0;
                    ++kround;
                }
            };
            auto q_ready = [&](int u) -> bool {
                return mbar_wait_tries(bar(Sh::kQFull + (two_q ? u & 1 : 0)), (uint32_t)((two_q ? u >> 1 : u) & 1));
            };
            TreePart s, nx;
            bool has = next_part(&s, true), has_nx = has && next_part(&nx, true);
            bool ok = true;
            int J = 0, u = 0, vs = 0, vround = 0;
            int scans = 0;
            if (has && (ok = q_ready(0) && k_ready()))
                issue_s(0, 0, s.k1 - s.k0 == 1);
            while (ok && has) {
                const int cnt = s.k1 - s.k0;
                const int first_masked = (s.len - s.n) / kTreeKeys - s.k0;   // (tiles of this part)
                for (int j = 0; j < cnt; ++j, ++J) {
                    const bool last = j + 1 == cnt;
                    // The next S, of this part or the next one, before this
                    // tile's P V: it overwrites the buffer that P_{J-1} V_{J-1}
                    // reads.  With one Q buffer the next part's first S comes
                    // after P V: its Q may still be on the way.
                    const bool ahead = !last || (has_nx && two_q);
                    // what has landed long since is looked at first: each look
                    // costs 100-200 cycles, and P_{J-1} V_{J-1} runs meanwhile
                    ok = mbar_wait_tries(bar(Sh::kVFull + vs), (uint32_t)(vround & 1));
                    const bool scan = j >= first_masked;
                    if (ok && scan)
                        mbar_arrive(bar(Sh::kScanReq));      // warp 7 scans V while the softmax works
                    if (ok && ahead) {
                        ok = (!last || q_ready(u + 1)) && k_ready() &&
                             (J == 0 || mbar_wait_tries(bar(Sh::kODone), (uint32_t)((J - 1) & 1)));
                        if (ok)
                            issue_s(J + 1, last ? u + 1 : u, last ? nx.k1 - nx.k0 == 1 : j + 2 == cnt);
                    }
                    if (ok && scan) {
                        ok = mbar_wait_tries(bar(Sh::kScanned), (uint32_t)(scans & 1));
                        ++scans;
                    }
                    ok = ok && mbar_wait_tries(bar(Sh::kPFull + (J & 1)), (uint32_t)((J >> 1) & 1));
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t vt = sV + vs * Sh::kVBytes;
                    const uint32_t tp = tmem + (J & 1) * kTreeKeys;
#pragma unroll
                    for (int kk = 0; kk < KV_STEPS; ++kk)
                        tc_mma_f16_ts(tO, tp + kk * 8, sw128_desc(vt + kk * 16 * 128, Sh::kVHalf, 1024), idO,
                                      (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(bar(Sh::kODone));
                    tc_commit(bar(Sh::kVEmpty + vs));
                    if (++vs == Sh::kVStages) {
                        vs = 0;
                        ++vround;
                    }
                    if (last && has_nx && !two_q) {
                        // O_DONE of this tile: it completes after the MMAs that read
                        // the buffer, and a wait for the phase before could miss it
                        if (!(ok = q_ready(u + 1) && k_ready() &&
                                   mbar_wait_tries(bar(Sh::kODone), (uint32_t)(J & 1))))
                            break;
                        issue_s(J + 1, u + 1, nx.k1 - nx.k0 == 1);
                    }
                }
                if (!ok)
                    break;
                ++u;
                s = nx;
                has = has_nx;
                has_nx = has && next_part(&nx, true);
            }
            if (!ok)
                raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
            tc_commit(bar(Sh::kDrain));
            mbar_wait_tries(bar(Sh::kDrain), 0u);
        }
    } else if (warp == 5) {
        // ---- TR: MMA issue, one thread ----
        if (lane == 0) {
            constexpr uint32_t idS = f16_idesc<BF16>(128, 64, false);
            constexpr uint32_t idO = f16_idesc<BF16>(128, 64, true) | (1u << 15);   // A = V^T: M (head_dim) along its rows
            TreePart s, nx;
            bool has = next_part(&s, true), has_nx = has && next_part(&nx, true);
            bool ok = true;
            int J = 0, u = 0, vs = 0, vround = 0, scans = 0;
            auto q_ready = [&](int u) -> bool {
                return mbar_wait_tries(bar(Sh::kQFull + (u & 1)), (uint32_t)((u >> 1) & 1));
            };
            auto k_ready = [&](int J) -> bool { return mbar_wait_tries(bar(Sh::kKFull), (uint32_t)(J & 1)); };
            // S^T of global tile J (part u; last: the part's last): buffer J & 1
            auto issue_s = [&](int J, int u, bool last) {
                tc_fence_after();
                const uint32_t qt = sQ + (u & 1) * Sh::kQSlot;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t koff = (uint32_t)((ks & 3) * 32);
                    tc_mma_f16(tmem + (J & 1) * 64, sw128_desc(sK + (ks >> 2) * Sh::kKHalf + koff, 16, 1024),
                               sw128_desc(qt + (ks >> 2) * Sh::kQHalf + koff, 16, 1024), idS, ks > 0 ? 1u : 0u);
                }
                tc_commit(bar(Sh::kSFull + (J & 1)));
                tc_commit(bar(Sh::kKEmpty));
                if (last)
                    tc_commit(bar(Sh::kQEmpty + (u & 1)));
            };
            if (has && (ok = q_ready(0) && k_ready(0)))
                issue_s(0, 0, s.k1 - s.k0 == 1);
            while (ok && has) {
                const int first_masked = (s.len - s.n) / KEYS;
                for (int t = s.k0; t < s.k1; ++t, ++J) {
                    const bool last = t + 1 == s.k1;
                    const int subs = min(2, (s.len - t * KEYS + kTreeKeys - 1) / kTreeKeys);   // 64-key halves with keys
                    if (!last || has_nx) {
                        // the next S^T: its buffer was read before P_{J-1} was handed over
                        ok = (!last || q_ready(u + 1)) && k_ready(J + 1);
                        if (!ok)
                            break;
                        issue_s(J + 1, last ? u + 1 : u, last ? nx.k1 - nx.k0 == 1 : t + 2 == s.k1);
                    }
                    for (int h = 0; ok && h < subs; ++h) {
                        const int st = (vs + h) % Sh::kVStages, round = vround + (vs + h) / Sh::kVStages;
                        ok = mbar_wait_tries(bar(Sh::kVFull + st), (uint32_t)(round & 1));
                    }
                    if (ok && t >= first_masked) {
                        mbar_arrive(bar(Sh::kScanReq));      // warp 7 scans V while the softmax works
                        ok = mbar_wait_tries(bar(Sh::kScanned), (uint32_t)(scans & 1));
                        ++scans;
                    }
                    ok = ok && mbar_wait_tries(bar(Sh::kPFull), (uint32_t)(J & 1));
                    if (!ok)
                        break;
                    tc_fence_after();
                    // O^T += V^T P^T, 16 keys per step: V^T (head_dim along the rows
                    // of V, halves kVHalf apart) and P^T (query rows along its rows)
                    for (int h = 0; h < subs; ++h) {
                        const uint32_t vt = sV + vs * Sh::kVBytes, pt = data_s + Sh::kPOff + h * 64 * 128;
#pragma unroll
                        for (int kk = 0; kk < KV_STEPS; ++kk)
                            tc_mma_f16(tO, sw128_desc(vt + kk * 16 * 128, Sh::kVHalf, 1024),
                                       sw128_desc(pt + kk * 16 * 128, 1024, 1024), idO, (t > s.k0 || h > 0 || kk > 0) ? 1u : 0u);
                        tc_commit(bar(Sh::kVEmpty + vs));
                        if (++vs == Sh::kVStages) {
                            vs = 0;
                            ++vround;
                        }
                    }
                    tc_commit(bar(Sh::kODone));
                }
                if (!ok)
                    break;
                ++u;
                s = nx;
                has = has_nx;
                has_nx = has && next_part(&nx, true);
            }
            if (!ok)
                raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
            tc_commit(bar(Sh::kDrain));
            mbar_wait_tries(bar(Sh::kDrain), 0u);
        }
    } else if constexpr (TR) {
        // ---- TR: softmax, thread = key of the tile = TMEM lane; output, thread
        // = column of the head = TMEM lane.  Query row c is TMEM column c. ----
        const int key = warp * 32 + lane;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const float sc = a.scale_log2;
        const bool fold = sc > 0.f;
        const float sm = fold ? 1.f : sc, se = fold ? sc : 1.f;
        uint8_t *sp = data + Sh::kPOff;
        // B[k][n] of the sums' products, k = row parity within 8 (+ 8: next register
        // but one), n = lane / 4: outputs 0 .. 3 of even groups, 4 .. 7 of odd ones
        constexpr float kMove = 14.f;                // f16 weights stay below 2^14 (bf16 ones below tree_headroom)
        const uint32_t one = BF16 ? 0x3f80u : 0x3c00u;
        const uint32_t pick = (lane & 4) ? one << 16 : one;
        uint32_t ones0[2], ones1[2];
        ones0[0] = (lane >> 3) == 0 ? pick : 0u, ones0[1] = (lane >> 3) == 1 ? pick : 0u;
        ones1[0] = (lane >> 3) == 2 ? pick : 0u, ones1[1] = (lane >> 3) == 3 ? pick : 0u;
        float *scratch = reinterpret_cast<float *>(sp);      // while no P V runs: [4][64], [64]
        bool ok = true;
        int J = 0, scans = 0, shares_ = 0, votes = 0, u = 0;
        // exchange between the four warps through shared memory written before
        auto all_four = [&](int b, int &count) -> bool {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(b));
            const bool got = mbar_wait_tries(bar(b), (uint32_t)(count & 1));
            ++count;
            return __all_sync(0xffffffffu, got);
        };
        for (; ok; ++u) {
            const int slot = u % kTreeParts;
            ok = __all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kPartFull + slot), (uint32_t)((u / kTreeParts) & 1)));
            const volatile TreePart &s = s_part[slot];
            const int k0 = s.k0, k1 = s.k1;
            if (!ok || k1 == 0)
                break;
            const int rows = s.n * G;                    // <= 64
            const int chunks = rows > 32 ? 2 : 1;
            const int first_masked = (s.len - s.n) / KEYS;
            auto up = [&]() -> float { return tree_headroom<BF16>(s.len, (int)kMove); };   // (no register to keep it in)
            float m_own[2] = {kNegInf, kNegInf};     // references (maximum + up) of rows lane and lane + 32
            // sums[q][e]: row 16 q + 4 (lane & 3) + e, over the keys 4 (lane >> 2) .. + 3 of the warp's 32
            float sums[4][4];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sums[i >> 2][i & 3] = 0.f;
            bool was_masked = false;
            auto mend = [&](int t) -> bool {
                const bool bad = was_masked && *reinterpret_cast<volatile uint32_t *>(&loc->bad[(scans - 1) % kTreeScans]);
                if (bad) {
                    tree_add_nonfinite_t<BS, BF16>(a.value_cache, a.block_tables + (size_t)s.b * a.max_blocks, a.num_blocks,
                                                   a.num_kv_heads, s.kvh, a.tree_mask + (size_t)s.q0 * a.words, a.words, G, s.n,
                                                   s.len, t, key, tO + lane_base);
                    __syncwarp();
                }
                return bad;
            };
            for (int t = k0; t < k1; ++t, ++J) {
                const int sb = J & 1;
                const bool masked = t >= first_masked;
                uint64_t vis = ~0ull;                    // the rows that see this thread's key
                if (masked)
                    vis = tree_rows_that_see<BS, 8>(a.tree_mask + (size_t)s.q0 * a.words, a.words, G, s.n, s.len, t * KEYS + key / BS * BS,
                                                 key % BS);
                ok = __all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kSFull + sb), (uint32_t)((J >> 1) & 1)));
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t se2 = f2(se, se);
                uint32_t pk[2][16];
                float over[2] = {kNegInf, kNegInf};      // how far a score lies above its row's reference
                // weights of 32 rows against the references in loc->m
                auto weigh = [&](int cc) {
                    uint32_t raw[32];
                    tmem_ld32(tmem + lane_base + sb * 64 + cc * 32, raw);
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = __uint_as_float(raw[i]);
                    if (!fold) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] *= sm;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(loc->m + cc * 32 + i);
                        const uint64_t lo = fma2(f2(x[i], x[i + 1]), se2, f2(-m.x, -m.y));
                        const uint64_t hi = fma2(f2(x[i + 2], x[i + 3]), se2, f2(-m.z, -m.w));
                        x[i] = f2_lo(lo);
                        x[i + 1] = f2_hi(lo);
                        x[i + 2] = f2_lo(hi);
                        x[i + 3] = f2_hi(hi);
                    }
                    if (masked) {
                        const uint32_t w = (uint32_t)(vis >> (cc * 32));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = (w >> i) & 1u ? x[i] : kNegInf;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        over[0] = fmax3_nan(over[0], x[i], x[i + 1]);
                        over[1] = fmax3_nan(over[1], x[i + 2], x[i + 3]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[cc][i] = pack2<BF16>(ex2(x[2 * i]), ex2(x[2 * i + 1]));
                };
                // A part's first maxima: the scores of its first key, if every row
                // sees it (not above the true ones, and seldom far below them);
                // infinities and NaN there are voted out.
                const bool lead = t == k0 && !masked;
                if (lead) {
                    if (warp == 0) {
#pragma unroll 1
                        for (int cc = 0; cc < chunks; ++cc) {
                            uint32_t raw[32];
                            tmem_ld32(tmem + lane_base + sb * 64 + cc * 32, raw);
                            if (lane == 0) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    loc->m[cc * 32 + i] = __uint_as_float(raw[i]) * sc + up();
                            }
                        }
                    }
                    if (!(ok = all_four(Sh::kShare, shares_)))
                        break;
                    m_own[0] = loc->m[lane];
                    m_own[1] = loc->m[lane + 32];
                }
                bool move = t == k0 && !lead, weighed = false;
                if (!move) {
                    weigh(0);
                    if (chunks > 1)
                        weigh(1);
                    const bool v = __any_sync(0xffffffffu, !(fmax3_nan(over[0], over[1], kNegInf) <= kMove - up()));
                    if (lane == 0)
                        loc->vote[sb][warp] = v;
                    // the maxima are the CTA's: any warp's vote moves them
                    if (!(ok = all_four(Sh::kVote, votes)))
                        break;
                    const volatile uint32_t *vt = loc->vote[sb];
                    move = (vt[0] | vt[1] | vt[2] | vt[3]) != 0u;
                    weighed = !move;
                }
                if (t > k0) {
                    // P_{J-1} V_{J-1} has completed: the weights' buffer is free, O stable
                    ok = __all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kODone), (uint32_t)((J - 1) & 1)));
                    if (!ok)
                        break;
                    tc_fence_after();
                    weighed = !mend(t - 1) && weighed;       // (the weights do not outlive its call)
                }
                if (move) {
                    // The rows' maxima over this tile: per warp by exchanges in which
                    // a lane keeps one row, then over the warps.
#pragma unroll 1
                    for (int cc = 0; cc < chunks; ++cc) {
                        uint32_t raw[32];
                        tmem_ld32(tmem + lane_base + sb * 64 + cc * 32, raw);
                        const uint32_t w = (uint32_t)(vis >> (cc * 32));
                        float x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float v = __uint_as_float(raw[i]) * sc;
                            x[i] = (w >> i) & 1u ? v : kNegInf;
                        }
#pragma unroll
                        for (int k = 16; k; k >>= 1) {
                            const bool up = (lane & k) != 0;
#pragma unroll
                            for (int i = 0; i < k; ++i) {
                                const float send = up ? x[i] : x[i + k], stay = up ? x[i + k] : x[i];
                                x[i] = fmaxf(stay, __shfl_xor_sync(0xffffffffu, send, k));
                            }
                        }
                        scratch[warp * 64 + cc * 32 + lane] = x[0];
                    }
                    if (!(ok = all_four(Sh::kShare, shares_)))
                        break;
                    float *s_alpha = scratch + 256;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        if (cc >= chunks)
                            break;
                        const int c = cc * 32 + lane;
                        float M = fmaxf(fmaxf(scratch[c], scratch[64 + c]), fmaxf(scratch[128 + c], scratch[192 + c])) + up();
                        if (lead)
                            m_own[cc] = kNegInf;
                        M = M > m_own[cc] + kMove ? M : m_own[cc];
                        const float alpha = M == m_own[cc] ? 1.f : ex2(m_own[cc] - M);
                        m_own[cc] = M;
                        // (every warp writes the same values)
                        loc->m[c] = M == kNegInf ? 0.f : M;
                        s_alpha[c] = alpha;
                    }
                    __syncwarp();
                    if (t > k0) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                sums[q][e] *= s_alpha[16 * q + 4 * (lane & 3) + e];   // (past the rows: 0, or not used)
#pragma unroll 1
                        for (int cc = 0; cc < chunks; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(tO + lane_base + cc * 32, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * s_alpha[cc * 32 + i]);
                            tmem_st32(tO + lane_base + cc * 32, o);
                        }
                        tmem_wait_st();
                    }
                    // the scratch is the weights' buffer: all have read it
                    if (!(ok = all_four(Sh::kShare, shares_)))
                        break;
                }
                if (!weighed) {
                    weigh(0);
                    if (chunks > 1)
                        weigh(1);
                }
                // P^T: key's row of 64 query rows, 128-byte swizzle
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
                    if (cc < chunks) {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            *reinterpret_cast<uint4 *>(sp + key * 128 + (((cc * 4 + v) ^ (key & 7)) << 4)) =
                                make_uint4(pk[cc][4 * v], pk[cc][4 * v + 1], pk[cc][4 * v + 2], pk[cc][4 * v + 3]);
                    }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(Sh::kPFull));
                // The rows' sums, of the rounded weights that the products take: a
                // register holds a key (the lane's) of two rows, which as A of an
                // mma is 4 keys x 2 rows along k; B's ones (b0, b1) keep the rows apart.
                // A NaN weight would reach the others of its product and is left
                // out: its row's O is NaN whatever the sum.
                const bool nan = __any_sync(0xffffffffu, over[0] != over[0] || over[1] != over[1]);
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    if (g < 4 * chunks) {
                        const uint32_t *p = &pk[g >> 2][4 * (g & 3)];
                        uint32_t A[4] = {p[0], p[1], p[2], p[3]};
                        if (nan) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                A[e] &= ~(nonfinite2<BF16>(A[e]) * 0xffffu);
                        }
                        mma_16816<BF16>(sums[g >> 1], A, g & 1 ? ones1[0] : ones0[0], g & 1 ? ones1[1] : ones0[1]);
                    }
                was_masked = masked;
                scans += masked ? 1 : 0;
            }
            if (!ok)
                break;
            ok = __all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kODone), (uint32_t)((J - 1) & 1)));
            if (!ok)
                break;
            tc_fence_after();
            mend(k1 - 1);
            // the rows' sums over the four warps
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = sums[q][e];
                    v += __shfl_xor_sync(0xffffffffu, v, 4);
                    v += __shfl_xor_sync(0xffffffffu, v, 8);
                    v += __shfl_xor_sync(0xffffffffu, v, 16);
                    if (lane < 4)
                        scratch[warp * 64 + 16 * q + 4 * lane + e] = v;
                }
            if (!(ok = all_four(Sh::kShare, shares_)))
                break;
            const bool item = k0 == 0 && k1 == s.tiles;
            float l_own[2];
            float *s_inv = scratch + 256 + warp * 64;    // each warp's own copy
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                const int c = cc * 32 + lane;
                const float l = (scratch[c] + scratch[64 + c]) + (scratch[128 + c] + scratch[192 + c]);
                l_own[cc] = l;
                s_inv[c] = l == 0.f ? 0.f : __frcp_rn(l);
            }
            __syncwarp();
            const uint32_t div_g = (65536u + G - 1) / G;     // c / G = c div_g >> 16 (c < 64)
#pragma unroll 1
            for (int cc = 0; cc < chunks; ++cc) {
                uint32_t o[32];
                tmem_ld32(tO + lane_base + cc * 32, o);
                const int cnt = min(32, rows - cc * 32);
                if (item) {
                    // row by row: token cc * 32 / G, then on by heads and tokens
                    const uint32_t c0 = cc * 32, tok = c0 * div_g >> 16;
                    int left = (int)(G - (c0 - tok * G));            // rows left of the token
                    uint16_t *at = a.out + ((size_t)(s.q0 + (int)tok) * a.num_heads + (size_t)s.kvh * G + (c0 - tok * G)) * D + key;
                    const size_t hop = (size_t)(a.num_heads - G) * D;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < cnt) {
                            *at = to_storage<BF16>(__uint_as_float(o[i]) * s_inv[c0 + i]);
                            at += D;
                            if (--left == 0) {
                                at += hop;
                                left = G;
                            }
                        }
                } else {
                    const size_t rec = (((size_t)blockIdx.x * 2 + s.share) * 2 + (k0 > 0 ? 0 : 1)) * kTreeRows + cc * 32;
                    float *orec = a.rec_o + rec * D + key;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < cnt)
                            orec[(size_t)i * D] = __uint_as_float(o[i]);
                    if (warp == 0 && lane < cnt)
                        a.rec_ml[rec + lane] = make_float2(m_own[cc], l_own[cc]);
                }
            }
            // the scratch becomes weights again: all have read it
            if (!(ok = all_four(Sh::kShare, shares_)))
                break;
            if (lane == 0)
                mbar_arrive(bar(Sh::kPartEmpty + slot));
        }
        if (!ok && lane == 0)
            raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
    } else {
        // ---- softmax and epilogue: thread = row r of the tile = TMEM lane r ----
        const int r = warp * 32 + lane;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const int r_tok = r / G, r_head = r - r_tok * G;
        const float sc = a.scale_log2;
        const bool fold = sc > 0.f;                  // a positive scale joins the exponent's fma
        const float sm = fold ? 1.f : sc, se = fold ? sc : 1.f;
        bool ok = true;
        int J = 0, scans = 0, u = 0;
        for (; ok; ++u) {
            // The part's fields stay in its slot of the queue, which this warp
            // gives back when it is done: the key loop needs the registers.
            const int slot = u % kTreeParts;
            ok = __all_sync(0xffffffffu, mbar_wait_tries(bar(Sh::kPartFull + slot), (uint32_t)((u / kTreeParts) & 1)));
            const volatile TreePart &s = s_part[slot];
            const int k1 = s.k1;
            if (!ok || k1 == 0)
                break;
            const int k0 = s.k0;
            const int first_masked = (s.len - s.n) / kTreeKeys;
            const int mine = min(R, s.n * G - s.rt * R) - warp * 32;   // this warp's rows of the tile
            const bool warp_on = mine > 0, real = lane < mine;
            const float up = tree_headroom<BF16>(s.len, 8);
            float m_used = kNegInf, l = 0.f;         // the row's reference (maximum + up), its weights' sum
            uint64_t vis = 0ull;                     // of the last masked tile
            bool was_masked = false;
            // after P V of tile t - 1 (or the last one): what the scan took out of its V
            auto mend = [&](int t) {
                if (was_masked && *reinterpret_cast<volatile uint32_t *>(&loc->bad[(scans - 1) % kTreeScans])) {
                    if (warp_on)
                        tree_add_nonfinite<D, BS, BF16>(a.value_cache, a.block_tables + (size_t)s.b * a.max_blocks, a.num_blocks,
                                                        a.num_kv_heads, s.kvh, s.len, t, real ? vis : 0ull, tO + lane_base);
                    __syncwarp();
                }
            };
            for (int t = k0; t < k1; ++t, ++J) {
                const int sb = J & 1;
                const bool masked = t >= first_masked;
                uint64_t vis_now = ~0ull;
                if (masked && warp_on) {
                    const int t0 = t * kTreeKeys, len = s.len, base = len - s.n;
                    vis_now = tree_bits(a.tree_mask + (size_t)(s.q0 + s.rt * TT + (real ? r_tok : 0)) * a.words, a.words,
                                        base, len - base, t0);
                    const int tail = len % BS;
                    if (t0 + kTreeKeys >= len && tail) {
                        // the partly filled last block was loaded to end its slot
                        const int lo = len - tail - t0;
                        const uint64_t low = (1ull << lo) - 1ull;
                        vis_now = (vis_now & low) | ((vis_now & ~low) << (BS - tail));
                    }
                }
                ok = mbar_wait_tries(bar(Sh::kSFull + sb), (uint32_t)((J >> 1) & 1));
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                bool resc = false;
                float alpha = 1.f;
                if (warp_on) {
                    // 32 keys at a time, by loops that are not unrolled: once for the
                    // maximum, once for the weights, which take the place of the scores
                    const uint32_t ts = tmem + lane_base + sb * kTreeKeys;
                    const uint32_t vis2[2] = {(uint32_t)vis_now, (uint32_t)(vis_now >> 32)};
                    float x[32];
                    auto scores = [&](int h) {
                        uint32_t raw[32];
                        tmem_ld32(ts + h * 32, raw);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            x[c] = __uint_as_float(raw[c]);
                        if (!fold) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                x[c] *= sm;
                        }
                        if (masked) {
                            const uint32_t w = h ? vis2[1] : vis2[0];
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                x[c] = ((w >> c) & 1u) ? x[c] : kNegInf;
                        }
                    };
                    float mt;
                    {
                        uint32_t raw[64];
                        tmem_ld64(ts, raw);
                        if (!fold) {
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                raw[c] = __float_as_uint(__uint_as_float(raw[c]) * sm);
                        }
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                raw[c] = (vis2[c >> 5] >> (c & 31)) & 1u ? raw[c] : 0xff800000u;
                        }
                        float mx[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mx[i] = fmaxf(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1]));
#pragma unroll
                        for (int c = 16; c < 64; c += 2)
                            mx[(c >> 1) & 7] = fmax3(mx[(c >> 1) & 7], __uint_as_float(raw[c]), __uint_as_float(raw[c + 1]));
                        mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                    }
                    mt = BF16 ? fmaf(mt, se, up) : mt * se;
                    resc = real && mt > m_used + 8.f;
                    const float m_new = resc ? mt : m_used;
                    alpha = resc ? ex2(m_used - m_new) : 1.f;
                    const float msub = m_new == kNegInf ? 0.f : m_new;
                    // the row sum is taken over the rounded weights the MMA multiplies
                    const uint64_t se2 = f2(se, se), nm2 = f2(-msub, -msub);
                    uint64_t rsv[2] = {0ull, 0ull};
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        scores(h);
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const uint64_t e = fma2(f2(x[2 * c], x[2 * c + 1]), se2, nm2);
                            pk[c] = pack2<BF16>(ex2(f2_lo(e)), ex2(f2_hi(e)));
                            const float2 pr = unpack2<BF16>(pk[c]);
                            rsv[c & 1] = add2(rsv[c & 1], f2(pr.x, pr.y));
                        }
                        tmem_st16(ts + h * 16, pk);
                    }
                    const uint64_t r2 = add2(rsv[0], rsv[1]);
                    l = l * alpha + (f2_lo(r2) + f2_hi(r2));
                    m_used = m_new;
                }
                if (t > k0) {
                    // P_{J-1} V_{J-1} has completed: O is stable, and O_DONE within one phase
                    ok = mbar_wait_tries(bar(Sh::kODone), (uint32_t)((J - 1) & 1));
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mend(t - 1);
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
                if (warp_on)
                    tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(Sh::kPFull + sb));
                vis = vis_now;
                was_masked = masked;
                scans += masked ? 1 : 0;
            }
            if (!ok)
                break;
            const bool item = k0 == 0 && k1 == s.tiles;
            const size_t orow = (size_t)(s.q0 + s.rt * TT + r_tok) * a.num_heads + (size_t)s.kvh * G + r_head;
            const float inv = l == 0.f ? 0.f : __frcp_rn(l);
            ok = mbar_wait_tries(bar(Sh::kODone), (uint32_t)((J - 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
            if (ok && warp_on) {
                tc_fence_after();
                mend(k1 - 1);
                if (item) {
                    // the whole item: output rows
                    uint4 *o16 = reinterpret_cast<uint4 *>(a.out + orow * D);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 64) {
                        uint32_t o[64];
                        tmem_ld64(tO + lane_base + c0, o);
                        if (real) {
#pragma unroll
                            for (int v = 0; v < 8; ++v) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = pack2<BF16>(__uint_as_float(o[8 * v + 2 * e]) * inv,
                                                       __uint_as_float(o[8 * v + 2 * e + 1]) * inv);
                                o16[c0 / 8 + v] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                } else {
                    // a part of an item: a record (m, l, O); CL: in shared memory, over
                    // the K and V rings (every copy and product is done), 16-byte
                    // chunks of a row swizzled by the row
                    if constexpr (CL) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + lane_base + c0, o);
#pragma unroll
                            for (int v = 0; v < 8; ++v)
                                *reinterpret_cast<uint4 *>(data + Sh::kKOff + r * D * 4 + (((c0 / 4 + v) ^ (r & 7)) << 4)) =
                                    make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                        }
                        *reinterpret_cast<float2 *>(data + r * 8) = make_float2(m_used, l);   // (over Q)
                        __syncwarp();
                        continue;
                    }
                    // (part 1 if the item starts here)
                    const size_t rec = (((size_t)blockIdx.x * 2 + s.share) * 2 + (k0 > 0 ? 0 : 1)) * kTreeRows + r;
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
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(Sh::kPartEmpty + slot));
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
    if constexpr (CL) {
        if (cl_rows == 0)
            return;                                  // (so for the whole cluster)
        // ---- join the cluster's parts by log-sum-exp: a warp to a row, a lane
        // to D / 32 of its columns, all parts' loads at once ----
        cluster_barrier();
        constexpr int V = D / 32;
        const int P = gridDim.x, rank = blockIdx.x;
        for (int r = rank * 8 + warp; r < cl_rows; r += P * 8) {
            const uint32_t at_ml = data_s + r * 8;
            const uint32_t at_o = data_s + Sh::kKOff + r * D * 4 + (((lane * V / 4) ^ (r & 7)) << 4) + (lane * V % 4) * 4;
            float2 ml[8];
            float v[8][V];
            float M = kNegInf;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // part k has keys
                if (k < P && cl_tiles * k / P < cl_tiles * (k + 1) / P) {
                    ml[k] = cluster_load2(cluster_map(at_ml, k));
                    if constexpr (V == 4) {
                        const float4 x = cluster_load4(cluster_map(at_o, k));
                        v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
                    } else {
                        const float2 x = cluster_load2(cluster_map(at_o, k));
                        v[k][0] = x.x, v[k][1] = x.y;
                    }
                } else {
                    ml[k] = make_float2(kNegInf, 0.f);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        v[k][i] = 0.f;
                }
                M = fmaxf(M, ml[k].x);
            }
            float den = 0.f, acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // (1: no keys seen, or all NaN)
                const float f = ml[k].x == kNegInf ? 1.f : ex2(ml[k].x - M);
                den += f * ml[k].y;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] += f * v[k][i];
            }
            const float inv = den == 0.f ? 0.f : 1.f / den;
            uint16_t *o = a.out + ((size_t)(cl_q0 + r / G) * a.num_heads + (size_t)cl_kvh * G + r % G) * D + lane * V;
            if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(o) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv),
                                                           pack2<BF16>(acc[2] * inv, acc[3] * inv));
            else
                *reinterpret_cast<uint32_t *>(o) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
        }
        cluster_barrier();                           // no CTA leaves while its memory is read
    }
}

// The records of an item that several CTAs shared, joined by log-sum-exp:
//   out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k,   M = max_k m_k.
// The CTAs (c, y) take the rows of the items whose second parts open CTA c's
// shares, sixteen to a CTA at a time; a warp takes two rows side by side, a
// lane D / 32 of their columns.  Bound by the round trips, so four records are
// loaded at a time; many of the CTAs have nothing to join.
constexpr int kTreeMergeThreads = 256;
template <int D, bool BF16>
__global__ void __launch_bounds__(kTreeMergeThreads, 4)
tree_merge_kernel(const TreeArgs a)
{
    constexpr int V = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int share = 0; share < a.shares; ++share) {
        const int4 d = __ldg(a.desc + c * 2 + share);
        const int step = a.shares == 2 && share == 0 ? 2 : 1;
        for (int r0 = ((int)blockIdx.y * 8 + warp) * 2; r0 < d.y; r0 += (int)gridDim.y * 16) {   // (no records: d.y is 0)
            // record k: CTA c + (k - 1) step; part 1 of the first, part 0 of the others
            auto rec = [&](int k) {
                return (((size_t)(c + (k - 1) * step) * 2 + share) * 2 + (k == 0 ? 1 : 0)) * kTreeRows + r0;
            };
            const int second = r0 + 1 < d.y ? 1 : 0;      // (an odd last row is taken twice)
            float M[2] = {kNegInf, kNegInf};
            for (int k = lane; k < d.w; k += 32) {
                M[0] = fmaxf(M[0], __ldg(&a.rec_ml[rec(k)].x));
                M[1] = fmaxf(M[1], __ldg(&a.rec_ml[rec(k) + second].x));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                M[0] = fmaxf(M[0], __shfl_xor_sync(0xffffffffu, M[0], o));
                M[1] = fmaxf(M[1], __shfl_xor_sync(0xffffffffu, M[1], o));
            }
            float den[2] = {0.f, 0.f}, acc[2][V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[0][i] = acc[1][i] = 0.f;
            auto batch = [&](auto count, int k0) {           // records k0 .. k0 + N - 1
                constexpr int N = decltype(count)::value;
                float2 ml[N][2];
                float v[N][2][V];
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const size_t at = rec(k0 + j) + (q ? second : 0);
                        ml[j][q] = __ldg(a.rec_ml + at);
                        load_slice<D>(a.rec_o + at * D + lane * V, v[j][q]);
                    }
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        // (1: a part without keys, or all NaN)
                        const float f = ml[j][q].x == kNegInf ? 1.f : ex2(ml[j][q].x - M[q]);
                        den[q] += f * ml[j][q].y;
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            acc[q][i] += f * v[j][q][i];
                    }
            };
            int k0 = 0;
            for (; k0 + 4 <= d.w; k0 += 4)
                batch(std::integral_constant<int, 4>{}, k0);
            if (d.w - k0 == 3)
                batch(std::integral_constant<int, 3>{}, k0);
            else if (d.w - k0 == 2)
                batch(std::integral_constant<int, 2>{}, k0);
            else if (d.w - k0 == 1)
                batch(std::integral_constant<int, 1>{}, k0);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = r0 + q;
                if (r >= d.y)
                    break;
                const float inv = den[q] == 0.f ? 0.f : 1.f / den[q];
                uint16_t *o = a.out + ((size_t)(d.x + r / a.group) * a.num_heads + (size_t)d.z * a.group + r % a.group) * D +
                              lane * V;
                if constexpr (V == 4)
                    *reinterpret_cast<uint2 *>(o) = make_uint2(pack2<BF16>(acc[q][0] * inv, acc[q][1] * inv),
                                                               pack2<BF16>(acc[q][2] * inv, acc[q][3] * inv));
                else
                    *reinterpret_cast<uint32_t *>(o) = pack2<BF16>(acc[q][0] * inv, acc[q][1] * inv);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows: up to 16 per (sequence, kv head)
// ---------------------------------------------------------------------------
// Small trees (or few heads to a group) leave the 128-row tiles above mostly
// empty, and their calls are bound by the cache's bytes alone.  Here a warp
// keeps 16 rows in its own registers and streams pages, as the decode kernel
// does: no hand-over between warps per tile, many independent streams per SM.
//   S[rows x keys] = Q K^T      mma.sync m16n8k16, Q as A, K rows as B
//   O[rows x D]   += P V        P straight from S's registers as A, V as B
// P is split into a 16-bit high part and a 16-bit remainder, each multiplied
// by V: the weights keep about 16 bits (bf16) or 22.  A CTA takes part_tokens keys
// of a (sequence, kv head), a warp every other page of them.  An item of one
// part is written out, of several as records that tree_rows_merge_kernel joins.
// Bound by the cache's bytes: 256 x 512 .. 640 tokens, 8 kv heads of 128, 2
// nodes x 4 heads take 107 us, 4 nodes 112 (0.86 of the measured copy rate;
// the 128-row tiles 110 and 120, sustained 130 and 131 against 107 and 111).
// With 32 rows the legacy matrix instructions bound it (174 us against 117), so
// more rows go to the tiles above.
struct TreeRowsArgs {
    const uint16_t *query;           // [T, Hq, D]
    const int32_t *query_start;      // [batch + 1]
    const int32_t *tree_mask;        // [T, words]
    const uint16_t *value_cache;
    const int32_t *block_tables;     // [batch, max_blocks]
    const int32_t *context_lens;     // [batch]
    uint16_t *out;                   // [T, Hq, D]
    float2 *rec_ml;                  // [T * Hq, num_parts]
    float *rec_o;                    // [T * Hq, num_parts, D]
    int num_tokens;
    int max_query_len;
    int words;
    int max_blocks;
    int num_heads;
    int num_kv_heads;
    int group;
    int num_blocks;
    int part_tokens;                 // a multiple of the block size
    int num_parts;
    float scale_log2;
};

template <int D, int BS>
struct TreeRowsShape {
    static constexpr int kWarps = 2, kStages = 2;            // as the decode kernel
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = BS * 128;
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = kWarps * 16 * (D + 2) * 4;
    static constexpr int kSmemBytes = (kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes) + 1024;
    static constexpr int kCtas = 6;                          // per SM, by registers (168)
};

template <int D, int BS, bool BF16>
__global__ void __launch_bounds__(TreeRowsShape<D, BS>::kWarps * 32, TreeRowsShape<D, BS>::kCtas)
tree_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const TreeRowsArgs a)
{
    using Sh = TreeRowsShape<D, BS>;
    constexpr int KW = Sh::kWarps, S = Sh::kStages, NT = KW * 32;
    constexpr int KS = D / 16, NB = BS / 8, DT = D / 8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[KW * S];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int part = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (threadIdx.x < KW * S)
        mbar_init(smem_addr(&s_full[threadIdx.x]), 1);
    fence_mbar_init();
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // this warp's first 32 table entries do not wait for the length
    const int blk0 = part * (a.part_tokens / BS);
    const int32_t *trow = a.block_tables + (size_t)b * a.max_blocks + blk0 + warp;
    int ids;
    {
        const int lb = warp + lane * KW;
        ids = lb < a.part_tokens / BS && blk0 + lb < a.max_blocks ? __ldg(trow + (size_t)lane * KW) : 0;
    }
    TreeSeq s;
    const bool good = tree_seq(a.query_start, a.context_lens, b, a.num_tokens, a.max_query_len, a.max_blocks * BS, &s);
    if (!good && threadIdx.x == 0 && part == 0 && kvh == 0)
        raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
    const int rows = s.n * G;                     // <= 16 (0 for a sequence that contradicts itself)
    const int tok0 = part * a.part_tokens;
    const int tok1 = min(s.len, tok0 + a.part_tokens);
    if (rows == 0 || tok1 <= tok0)
        return;
    const bool split = s.len > a.part_tokens;
    const int base = s.len - s.n;
    const int nblk = (tok1 - tok0 + BS - 1) / BS;
    const int nk = nblk > warp ? (nblk - warp + KW - 1) / KW : 0;   // this warp's blocks
    uint8_t *ring = smem + (size_t)warp * S * Sh::kStageBytes;
    const uint32_t ring_s = smem_addr(ring);
    const uint32_t full0 = smem_addr(&s_full[warp * S]);
    const uint64_t policy = policy_evict_first();
    auto issue = [&](int k) {
        if ((k & 31) == 0 && k > 0)
            ids = k + lane < nk ? __ldg(trow + (size_t)(k + lane) * KW) : 0;
        int blk = __shfl_sync(0xffffffffu, ids, k & 31);
        if ((unsigned)blk >= (unsigned)a.num_blocks) {
            if (lane == 0)
                raise_flag(PKV_DEVFLAG_BLOCK_RANGE);
            blk = 0;
        }
        if (lane == 0) {
            const uint32_t bar = full0 + 8u * (k % S);
            const uint32_t dk = ring_s + (uint32_t)((k % S) * Sh::kStageBytes), dv = dk + Sh::kTileBytes;
            mbar_arrive_expect_tx(bar, Sh::kStageBytes);
#pragma unroll
            for (int h = 0; h < Sh::kHalves; ++h) {
                tma_load_3d(dk + h * Sh::kHalfBytes, &tm_k, bar, h * 64, kvh, blk * BS, policy);
                tma_load_3d(dv + h * Sh::kHalfBytes, &tm_v, bar, h * 64, kvh, blk * BS, policy);
            }
        }
    };
    int issued = 0, consumed = 0;
    for (; issued < (nk < S ? nk : S); ++issued)
        issue(issued);

    // ---- Q fragments: row r of the item is (node r / G, head r % G) ----
    const int g0 = lane >> 2, c2 = (lane & 3) * 2;
    const int ra = g0, rb = g0 + 8;               // this lane's rows
    auto q_row = [&](int r) {
        r = r < rows ? r : 0;
        return reinterpret_cast<const uint32_t *>(
            a.query + ((size_t)(s.q0 + r / G) * a.num_heads + (size_t)kvh * G + r % G) * D + c2);
    };
    uint32_t qf[KS][4];
    {
        const uint32_t *qa = q_row(ra), *qb = q_row(rb);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            qf[ks][0] = __ldg(qa + ks * 8);
            qf[ks][1] = __ldg(qb + ks * 8);
            qf[ks][2] = __ldg(qa + ks * 8 + 4);
            qf[ks][3] = __ldg(qb + ks * 8 + 4);
        }
    }
    const float up = tree_headroom<BF16>(s.len, 8);
    float m_run[2] = {kNegInf, kNegInf}, l_run[2] = {0.f, 0.f}, acc[DT][4];   // (references: maximum + up)
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[d][i] = 0.f;
    for (int k = 0; k < nk; ++k) {
        const int st = k % S;
        const bool got = mbar_wait_tries(full0 + 8u * st, (uint32_t)((k / S) & 1));
        if (!__all_sync(0xffffffffu, got)) {
            if (lane == 0)
                raise_flag(PKV_DEVFLAG_WAIT_TIMEOUT);
            break;
        }
        consumed = k + 1;
        const uint32_t sk = ring_s + (uint32_t)(st * Sh::kStageBytes), sv = sk + Sh::kTileBytes;
        const int p0 = (blk0 + warp + k * KW) * BS;        // the block's first position
        const bool masked = p0 + BS > base;
        bool bad = false;
        if (masked) {
            // Cells past the end may hold anything: zero.  Infinities and NaN
            // of drafted cells are zeroed too and added below to the rows that
            // see them (weight 0 times such a value would not be 0).
            uint8_t *vt = ring + (size_t)st * Sh::kStageBytes + Sh::kTileBytes;
            const int valid = min(BS, s.len - p0);
            uint32_t any = 0u;
#pragma unroll
            for (int i = 0; i < Sh::kTileBytes / 512; ++i) {
                const int v = i * 32 + lane;
                const int row = (v >> 3) % BS;
                uint4 *at = reinterpret_cast<uint4 *>(vt) + v;
                const uint4 x = *at;
                if (row >= valid)
                    *at = make_uint4(0u, 0u, 0u, 0u);
                else
                    any = fma_zero2<BF16>(x.x, fma_zero2<BF16>(x.y, fma_zero2<BF16>(x.z, fma_zero2<BF16>(x.w, any))));
            }
            bad = __any_sync(0xffffffffu, (any & 0x7fff7fffu) != 0u);
            if (bad) {
#pragma unroll 1
                for (int i = 0; i < Sh::kTileBytes / 4 / 32; ++i) {
                    uint32_t *at = reinterpret_cast<uint32_t *>(vt) + i * 32 + lane;
                    *at &= ~(nonfinite2<BF16>(*at) * 0xffffu);
                }
            }
            // order these generic stores before any later TMA (async proxy) write
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        }
        // ---- scores ----
        float sc[NB][4];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sc[j][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
                const int key = j * 8 + (lane >> 4) * 8 + (lane & 7);
                const int chunk = (ks & 3) * 2 + ((lane >> 3) & 1);
                uint32_t kf[4];
                ldsm_x4(sk + (uint32_t)((ks >> 2) * Sh::kHalfBytes + key * 128 + ((chunk ^ (key & 7)) << 4)), kf);
                mma_16816<BF16>(sc[j], qf[ks], kf[0], kf[1]);
                mma_16816<BF16>(sc[j + 1], qf[ks], kf[2], kf[3]);
            }
        // ---- mask, online softmax (base 2) ----
        uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
        float alpha[2];
        bool any_resc = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (masked) {
                const int r = h ? rb : ra;
                vis[h] = (uint32_t)tree_bits(a.tree_mask + (size_t)(s.q0 + (r < rows ? r / G : 0)) * a.words, a.words,
                                             base, s.n, p0);
            }
            float mx = kNegInf;
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float &x = sc[j][2 * h + i];
                    x *= a.scale_log2;
                    if (masked)
                        x = (vis[h] >> (j * 8 + c2 + i)) & 1u ? x : kNegInf;
                    mx = fmaxf(mx, x);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // the reference moves when a block's maximum exceeds the last by 2^8
            mx += up;
            const bool move = mx > m_run[h] + 8.f;
            const float mnew = move ? mx : m_run[h];
            alpha[h] = move ? ex2(m_run[h] - mnew) : 1.f;
            any_resc |= move;
            m_run[h] = mnew;
            const float msub = mnew == kNegInf ? 0.f : mnew;
            float ls = 0.f;
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float &x = sc[j][2 * h + i];
                    x = ex2(x - msub);
                    ls += x;
                }
            l_run[h] = l_run[h] * alpha[h] + ls;
        }
        if (__any_sync(0xffffffffu, any_resc)) {
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                acc[d][0] *= alpha[0];
                acc[d][1] *= alpha[0];
                acc[d][2] *= alpha[1];
                acc[d][3] *= alpha[1];
            }
        }
        // ---- O += P V, 16 keys at a time ----
#pragma unroll
        for (int kb = 0; kb < BS / 16; ++kb) {
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *x = &sc[2 * kb + (i >> 1)][2 * (i & 1)];
                ph[i] = pack2<BF16>(x[0], x[1]);
                const float2 f = unpack2<BF16>(ph[i]);
                pl[i] = pack2<BF16>(x[0] - f.x, x[1] - f.y);
            }
            const int key = kb * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int d = 0; d < DT; d += 2) {
                const int chunk = (d & 7) + (lane >> 4);
                uint32_t vf[4];
                ldsm_x4_trans(sv + (uint32_t)((d >> 3) * Sh::kHalfBytes + key * 128 + ((chunk ^ (key & 7)) << 4)), vf);
                mma_16816<BF16>(acc[d], ph, vf[0], vf[1]);
                mma_16816<BF16>(acc[d + 1], ph, vf[2], vf[3]);
                mma_16816<BF16>(acc[d], pl, vf[0], vf[1]);
                mma_16816<BF16>(acc[d + 1], pl, vf[2], vf[3]);
            }
        }
        if (bad) {
            int blk = __ldg(a.block_tables + (size_t)b * a.max_blocks + p0 / BS);
            blk = (unsigned)blk < (unsigned)a.num_blocks ? blk : 0;
#pragma unroll 1
            for (int c = 0; c < min(BS, s.len - p0); ++c) {
                const uint32_t *v = reinterpret_cast<const uint32_t *>(
                    a.value_cache + (((size_t)blk * BS + c) * a.num_kv_heads + kvh) * D + c2);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const uint32_t x = __ldg(v + d * 4);
                    const uint32_t f = nonfinite2<BF16>(x);
                    const float2 y = unpack2<BF16>(x);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if ((vis[h] >> c) & 1u) {
                            if (f & 1u)
                                acc[d][2 * h] += y.x;
                            if (f >> 16)
                                acc[d][2 * h + 1] += y.y;
                        }
                }
            }
        }
        __syncwarp();
        if (k + S < nk) {
            issue(k + S);
            issued = k + S + 1;
        }
    }
    // a wait gave up: copies in flight land (bounded) before the memory is reused
    for (int k = consumed; k < issued; ++k)
        mbar_wait_tries(full0 + 8u * (k % S), (uint32_t)((k / S) & 1));

    // ---- merge the warps by log-sum-exp through shared memory ----
    __syncthreads();
    float *so = reinterpret_cast<float *>(smem);                      // [warps][16][D]
    float2 *sml = reinterpret_cast<float2 *>(so + KW * 16 * D);   // [warps][16]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = h * 8 + g0;
        float l = l_run[h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if ((lane & 3) == 0)
            sml[warp * 16 + r] = make_float2(m_run[h], l);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<float2 *>(so + (warp * 16 + r) * D + d * 8 + c2) =
                make_float2(acc[d][2 * h], acc[d][2 * h + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += NT) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < KW; ++w)
            M = fmaxf(M, sml[w * 16 + r].x);
        float den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const float2 ml = sml[w * 16 + r];
            const float e = ml.x == kNegInf ? 1.f : ex2(ml.x - M);   // (1: no keys seen, or all NaN)
            const float4 o = *reinterpret_cast<const float4 *>(so + (w * 16 + r) * D + d);
            den += e * ml.y;
            num.x += e * o.x;
            num.y += e * o.y;
            num.z += e * o.z;
            num.w += e * o.w;
        }
        const size_t row = (size_t)(s.q0 + r / G) * a.num_heads + (size_t)kvh * G + r % G;
        if (!split) {
            const float inv = den == 0.f ? 0.f : 1.f / den;
            *reinterpret_cast<uint2 *>(a.out + row * D + d) =
                make_uint2(pack2<BF16>(num.x * inv, num.y * inv), pack2<BF16>(num.z * inv, num.w * inv));
        } else {
            const size_t rec = row * a.num_parts + part;
            *reinterpret_cast<float4 *>(a.rec_o + rec * D + d) = num;
            if (d == 0)
                a.rec_ml[rec] = make_float2(M, den);
        }
    }
}

// Records of the items of several parts, a warp per row: grid (eights of the
// rows, kv heads, sequences).
template <int D, bool BF16>
__global__ void __launch_bounds__(256)
tree_rows_merge_kernel(const TreeRowsArgs a, int block_size)
{
    constexpr int V = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TreeSeq s;
    if (!tree_seq(a.query_start, a.context_lens, blockIdx.z, a.num_tokens, a.max_query_len,
                  a.max_blocks * block_size, &s))
        return;
    const int r = blockIdx.x * 8 + warp;
    const int np = (s.len + a.part_tokens - 1) / a.part_tokens;
    if (np <= 1 || r >= s.n * a.group)
        return;
    const size_t row = (size_t)(s.q0 + r / a.group) * a.num_heads + (size_t)blockIdx.y * a.group + r % a.group;
    const float2 *ml = a.rec_ml + row * a.num_parts;
    float M = kNegInf;
    for (int k = lane; k < np; k += 32)
        M = fmaxf(M, __ldg(&ml[k].x));
#pragma unroll
    for (int o = 16; o; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float den = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.f;
#pragma unroll 8
    for (int k = 0; k < np; ++k) {
        const float2 x = __ldg(ml + k);
        float v[V];
        load_slice<D>(a.rec_o + (row * a.num_parts + k) * D + lane * V, v);
        const float f = x.x == kNegInf ? 1.f : ex2(x.x - M);         // (1: no keys seen, or all NaN)
        den += f * x.y;
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] += f * v[i];
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint16_t *o = a.out + row * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(o) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv),
                                                   pack2<BF16>(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(o) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
}

}  // namespace pkv
