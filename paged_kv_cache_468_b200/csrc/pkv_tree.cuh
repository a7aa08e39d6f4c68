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

#include "pkv_kernels.cuh"

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
struct TreeArgs {
    const uint16_t *query;           // [T, Hq, D]
    const int32_t *query_start;      // [batch + 1]
    const int32_t *tree_mask;        // [T, words]
    const uint16_t *key_cache;       // [num_blocks, bs, Hkv, D]
    const uint16_t *value_cache;
    const int32_t *block_tables;     // [batch, max_blocks]
    const int32_t *context_lens;     // [batch]
    uint16_t *out;                   // [T, Hq, D]
    int batch;
    int num_tokens;
    int max_query_len;
    int words;                       // mask words per row
    int max_blocks;
    int block_size;
    int num_heads;
    int num_kv_heads;
    int group;
    int num_blocks;
    float scale_log2;
};

// One CTA per (drafted token, kv head): its four warps take every fourth key
// each, all heads of the group at once, with a running maximum and sum.
template <int D, bool BF16>
__global__ void __launch_bounds__(128)
tree_attend_kernel(const TreeArgs a)
{
    constexpr int V = D / 32;
    __shared__ float s_m[4][8], s_l[4][8], s_o[4][8][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, kvh = blockIdx.y;
    int lo = 0, hi = a.batch;                      // the last sequence that starts at or before row t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.query_start + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    TreeSeq s;
    if (!tree_seq(a.query_start, a.context_lens, lo, a.num_tokens, a.max_query_len,
                  a.max_blocks * a.block_size, &s)) {
        if (threadIdx.x == 0)
            raise_flag(PKV_DEVFLAG_CONTEXT_RANGE);
        return;
    }
    if (t < s.q0 || t >= s.q0 + s.n)
        return;                                    // a row of no sequence
    const int base = s.len - s.n;
    float q[8][V], m[8], l[8], o[8][V];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        m[g] = kNegInf;
        l[g] = 0.f;
        const uint32_t *qp = reinterpret_cast<const uint32_t *>(
            a.query + ((size_t)t * a.num_heads + (size_t)kvh * a.group + (g < a.group ? g : 0)) * D + lane * V);
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const float2 f = unpack2<BF16>(__ldg(qp + v / 2));
            q[g][v] = f.x * a.scale_log2;
            q[g][v + 1] = f.y * a.scale_log2;
            o[g][v] = o[g][v + 1] = 0.f;
        }
    }
    for (int j = warp; j < s.len; j += 4) {
        if (j >= base && !((__ldg(a.tree_mask + (size_t)t * a.words + ((j - base) >> 5)) >> ((j - base) & 31)) & 1))
            continue;
        int blk = __ldg(a.block_tables + (size_t)lo * a.max_blocks + j / a.block_size);
        if ((unsigned)blk >= (unsigned)a.num_blocks) {
            if (lane == 0)
                raise_flag(PKV_DEVFLAG_BLOCK_RANGE);
            blk = 0;
        }
        const size_t cell = ((size_t)blk * a.block_size + j % a.block_size) * a.num_kv_heads + kvh;
        const uint32_t *kp = reinterpret_cast<const uint32_t *>(a.key_cache + cell * D + lane * V);
        const uint32_t *vp = reinterpret_cast<const uint32_t *>(a.value_cache + cell * D + lane * V);
        float k[V], x[V];
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            const float2 f = unpack2<BF16>(__ldg(kp + v / 2)), h = unpack2<BF16>(__ldg(vp + v / 2));
            k[v] = f.x; k[v + 1] = f.y;
            x[v] = h.x; x[v + 1] = h.y;
        }
#pragma unroll
        for (int g = 0; g < 8; ++g)
            if (g < a.group) {
                float d = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    d += q[g][v] * k[v];
#pragma unroll
                for (int off = 16; off; off >>= 1)
                    d += __shfl_xor_sync(0xffffffffu, d, off);
                const float mn = fmaxf(m[g], d);
                const float e = mn == kNegInf ? 1.f : ex2(m[g] - mn), p = ex2(d - (mn == kNegInf ? 0.f : mn));   // NaN stays NaN
                m[g] = mn;
                l[g] = l[g] * e + p;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    o[g][v] = o[g][v] * e + p * x[v];
            }
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        s_m[warp][g] = m[g];
        s_l[warp][g] = l[g];
#pragma unroll
        for (int v = 0; v < V; ++v)
            s_o[warp][g][lane * V + v] = o[g][v];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.group * D; e += 128) {
        const int g = e / D, d = e % D;
        const float M = fmaxf(fmaxf(s_m[0][g], s_m[1][g]), fmaxf(s_m[2][g], s_m[3][g]));
        float den = 0.f, num = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = s_m[w][g] == kNegInf ? 1.f : ex2(s_m[w][g] - M);   // (1: sums of 0, or NaN)
            den += f * s_l[w][g];
            num += f * s_o[w][g][d];
        }
        a.out[((size_t)t * a.num_heads + (size_t)kvh * a.group + g) * D + d] =
            to_storage<BF16>(den == 0.f ? 0.f : num / den);
    }
}

}  // namespace pkv
