// tree_nodes.cuh -- the nodes of a drafted tree in shared memory, and what a node reads of its ancestors, for the kernels that
// work out gates (k_tree.cu, k_tree_tc.cu).
#pragma once

#include "paged.cuh"

namespace mc {

struct Nodes {
    uint64_t anc[kMaxTree];      // a node's ancestors and itself
    uint64_t seg_set[kMaxTree];  // the nodes of a segment (0: the one that the cache has begun)
    int up[kMaxTree], seg[kMaxTree];
    float2 cum[kMaxTree];        // log_alpha summed along the path within the segment, in two parts (delta_parts)
    float la[kMaxTree], be[kMaxTree];
};

// Sequence b's m nodes; in0 tokens are in the begun segment.  The whole block calls it, with at least 64 threads.
template <typename E>
__device__ void make_nodes(const TreeArgs &a, Nodes &s, int b, int bh, int m, int in0)
{
    const int tid = threadIdx.x;
    uint64_t set = 0;
    int f = -1;
    if (tid < kMaxTree) {
        if (tid < m) {
            set = 1ull << tid;
            f = a.parent ? a.parent[(size_t)b * a.T + tid] : -1;
            if (f < -1 || f >= tid) {
                atomicOr(a.c.status, MC_PAGES_INDEX);
                f = -1;
            }
            if (a.delta) {
                s.la[tid] = delta_log(to_f(static_cast<const E *>(a.la)[(size_t)bh * a.T + tid]));
                s.be[tid] = to_f(static_cast<const E *>(a.be)[(size_t)bh * a.T + tid]);
            }
        }
        s.anc[tid] = set;
        s.up[tid] = f;
        s.seg_set[tid] = 0;
    }
    __syncthreads();
#pragma unroll 1
    for (int x = 1; x < m; x *= 2) {  // by doubling: after this turn a node knows its ancestors up to 2x above it
        if (tid < m && f >= 0) {
            set |= s.anc[f];
            f = s.up[f];
        }
        __syncthreads();
        if (tid < m) {
            s.anc[tid] = set;
            s.up[tid] = f;
        }
        __syncthreads();
    }
    if (tid < kMaxTree) {  // (two whole warps, each with its half of the sets)
        const int j = tid < m ? (in0 + __popcll(set) - 1) / a.c.C : -1;
        s.seg[tid] = j;
        const unsigned same = __match_any_sync(0xffffffffu, j);
        if (j >= 0 && (same & ((1u << (tid % 32)) - 1)) == 0) reinterpret_cast<unsigned *>(&s.seg_set[j])[tid / 32] = same;
    }
    if (!a.delta) {
        __syncthreads();
        return;
    }
    // sums along the path, by doubling again: up to the segment's first node
    float2 sum = make_float2(0.f, 0.f);
    if (tid < m) {
        sum = delta_parts(s.la[tid]);
        f = a.parent ? a.parent[(size_t)b * a.T + tid] : -1;
        if (f < -1 || f >= tid) f = -1;
        s.cum[tid] = sum;
    }
    __syncthreads();
    if (tid < m) {
        if (f >= 0 && s.seg[f] != s.seg[tid]) f = -1;
        s.up[tid] = f;
    }
    __syncthreads();
#pragma unroll 1
    for (int x = 1; x < m; x *= 2) {
        if (tid < m && f >= 0) {
            sum.x += s.cum[f].x;
            sum.y += s.cum[f].y;
            f = s.up[f];
        }
        __syncthreads();
        if (tid < m) {
            s.cum[tid] = sum;
            s.up[tid] = f;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ float decay(const Nodes &s, int to, int from)
{
    return expf((s.cum[to].x - s.cum[from].x) + (s.cum[to].y - s.cum[from].y));
}
// From the cache to node n's deepest ancestor in the begun segment.
__device__ __forceinline__ float decay_from_cache(const Nodes &s, int n)
{
    const float2 z = s.cum[63 - __clzll(s.anc[n] & s.seg_set[0])];
    return expf(z.x + z.y);
}
// P_{n,x} (with gate w of x's segment and qk = k_x . q_n) and A_{n,x} (kk = k_x . k_n) for an ancestor x of n.
__device__ __forceinline__ float path_read(const TreeArgs &a, const Nodes &s, int n, int x, float w, float qk)
{
    const float p = w * qk;
    return a.delta ? p * (decay(s, 63 - __clzll(s.anc[n] & s.seg_set[s.seg[x]]), x) * s.be[x]) : p;
}
__device__ __forceinline__ float path_meet(const Nodes &s, int n, int x, float kk)
{
    return x != n && s.seg[x] == s.seg[n] ? decay(s, n, x) * s.be[x] * kk : 0.f;
}

// The ancestors' columns of P and A for tokens n0 .. n0 + G - 1, transposed: row x, column n.  gate(t, j), qk(t, x) and
// kk(t, x) give token n0 + t's gate of path segment j and its products with node x.
template <int G, typename F, typename Q, typename K>
__device__ __forceinline__ void write_path(const TreeArgs &a, const Nodes &s, int bh, int n0, int m, F gate, Q qk, K kk)
{
    for (int i = threadIdx.x; i < m * G; i += blockDim.x) {
        const int t = i % G, x = i / G, n = n0 + t;
        float p = 0.f, q = 0.f;
        if (n < m && (s.anc[n] >> x) & 1) {
            p = path_read(a, s, n, x, gate(t, s.seg[x]), qk(t, x));
            if (a.delta) q = path_meet(s, n, x, kk(t, x));
        }
        if (n < a.Tp) {
            a.P[((size_t)bh * a.T + x) * a.Tp + n] = p;
            if (a.delta) a.A[((size_t)bh * a.T + x) * a.Tp + n] = q;
        }
    }
    if (n0 + (int)threadIdx.x < m && threadIdx.x < G && bh % a.c.H == 0)
        a.anc[(size_t)(bh / a.c.H) * kMaxTree + n0 + threadIdx.x] = s.anc[n0 + threadIdx.x];
}

}  // namespace mc
