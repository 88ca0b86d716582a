// paged.cuh -- argument blocks and device helpers of decoding over a paged cache (mc_pages.cu, k_pages.cu, k_tree.cu,
// k_tree_tc.cu).
//
// Every call over a batch begins with a plan (one CTA): which row of the cache each batch row works on, its position, and
// what it needs of the pool.  The kernels after it read positions from the plan alone, so that the last of them may write
// the cache's.
#pragma once

#include "mc_internal.cuh"

namespace mc {

constexpr int kMaxTree = 64;    // nodes of a draft: a set of them is one 64-bit word
constexpr int kMaxRows = 1024;  // sequences of a cache, rows of a batch
constexpr int kMaxPaged = 1024; // segments of a sequence
constexpr int kMaxPos = 1 << 30;

// Device pointers as in mc_paged_cache.
struct Paged {
    float *pages, *kbar;   // [P][H][d][d], [P][H][d]
    int32_t *refs;         // [P]
    float *online, *ksum;  // [S][H][d][d], [S][H][d]
    int32_t *table;        // [S][nmax]
    int32_t *pos;          // [S]
    int32_t *row;          // [S]
    int32_t *status;       // [1]
    int P, S, H, d, C, nmax;
};

// What a call does with the batch rows' sequences.
struct Plan {
    int32_t *act;      // [B] the cache's row, -1: nothing to do
    int32_t *pos;      // [B] position before the call
    int32_t *len;      // [B] tokens added (accept: the path's length)
    uint64_t *path;    // [B] accept: the nodes of the path
    int32_t *fresh;    // [B + 1] where a batch row's new pages begin in list
    int32_t *list;     // new pages in order of batch row and time, -1 where none was free
    int32_t *units;    // [B + 1] memories to read before those of batch row b, per head
};

struct TreeArgs {
    Paged c;
    Plan p;
    const void *q, *k, *v, *u, *la, *be;  // [B][H][T][d]; la, be [B][H][T] or null
    const int32_t *parent;                // [B][T], or null (T = 1)
    const int32_t *count;                 // [B] nodes, or null (T)
    const int32_t *slots;                 // [B], or null (batch row b is slot b)
    const int32_t *last;                  // [B] accept: the last node of the path
    void *y;                              // [B][H][T][d]
    float *gates;                         // [BH][nmax + 2][Tp] gates of the cached memories, then what nodes read of the begun
                                          // segment's with their queries (gate and decay) and with their keys (decay)
    float *P, *A;                         // [BH][T][Tp] what a node reads of what its ancestors wrote; what they meet in its key
    float *f0;                            // [BH][Tp] a step: the online memory's gate
    float *Z;                             // [BH][Tp][d] the begun segment's memory read with the nodes' keys, decayed
    float *part;                          // [ranges + BH][Tp][d] partial reads
    int B, T, Tp, mode, topk;
    int ranges, groups;                   // shares of the memories; of the tokens
    bool bf16, delta, step, accept;
};

// The U memories that a call reads are cut into R = ranges_of(U) ranges, none of them empty: memory x is in range
// range_of(x), and range j begins at range_begin(j).
__device__ __forceinline__ long long ranges_of(long long U, int most) { return U < most ? U : most; }
__device__ __forceinline__ long long range_begin(long long j, long long U, long long R) { return j * U / R; }
__device__ __forceinline__ int range_of(long long x, long long U, long long R) { return (int)(((x + 1) * R - 1) / U); }

__device__ __forceinline__ int valid_page(const Paged &c, int p) { return (unsigned)p < (unsigned)c.P ? p : -1; }

// Completed segments of a sequence at pos that its table has room for, and the memories that a read goes over: those and,
// in a tree's reads, that of a segment begun, for the queries and (gated delta memory) for the keys.
__device__ __forceinline__ int cached_segments(const Paged &c, int pos) { return min(pos / c.C, c.nmax); }
__device__ __forceinline__ int units_of(const TreeArgs &a, int pos)
{
    return cached_segments(a.c, pos) + (!a.step && pos % a.c.C ? (a.delta ? 2 : 1) : 0);
}
__device__ __forceinline__ int nodes_of(const TreeArgs &a, int b)
{
    return a.count ? max(0, min(a.count[b], a.T)) : a.T;
}

__device__ __forceinline__ float dot4(const float4 &a, const float4 &b)
{
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}
__device__ __forceinline__ float4 fma4(float s, const float4 &a, const float4 &b)
{
    return make_float4(fmaf(s, a.x, b.x), fmaf(s, a.y, b.y), fmaf(s, a.z, b.z), fmaf(s, a.w, b.w));
}
__device__ __forceinline__ float4 scale4(float s, const float4 &a) { return make_float4(s * a.x, s * a.y, s * a.z, s * a.w); }
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.x));
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.y));
    return make_float4(x.x, x.y, y.x, y.y);
}

// Sums of N values over groups of LANES lanes, N a power of two: the exchange halves the values a lane keeps while it can
// (log2(N) steps), so N values cost N - 1 + log2(LANES / N) shuffles instead of N log2(LANES).  A lane is left with the sums
// kept<N, LANES>() values from first<N, LANES>(lane).
template <int N, int LANES>
__device__ __forceinline__ constexpr int kept() { return N > LANES ? N / LANES : 1; }
template <int N, int LANES>
__device__ __forceinline__ int first(int lane)
{
    int at = 0, half = N / 2;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        if (half >= 1) at += lane & o ? half : 0;
        half >>= 1;
    }
    return at;
}
// Whether this lane is the one of those with the same sums that stores them.
template <int N, int LANES>
__device__ __forceinline__ bool stores(int lane) { return LANES <= N || lane % (LANES / N > 0 ? LANES / N : 1) == 0; }
template <int N, int LANES>
__device__ __forceinline__ void sum_groups(float (&p)[N], int lane)
{
    int keep = N;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        if (keep > 1) {
            const int half = keep / 2;
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < half) {
                    const float give = up ? p[i] : p[i + half], stay = up ? p[i + half] : p[i];
                    p[i] = stay + __shfl_xor_sync(0xffffffffu, give, o);
                }
            keep = half;
        } else {
            p[0] += __shfl_xor_sync(0xffffffffu, p[0], o);
        }
    }
}

cudaError_t launch_plan(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_gates(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_read(const TreeArgs &a, cudaStream_t s);
bool tree_tc_supported(const TreeArgs &a);
cudaError_t launch_tree_read_tc(const TreeArgs &a, cudaStream_t s);
cudaError_t take_tree_abort(int *was_set);
cudaError_t launch_tree_finish(const TreeArgs &a, cudaStream_t s);  // a step's end too
cudaError_t launch_accept(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_fork(const Paged &c, const int32_t *src, int32_t *plan, cudaStream_t s);
cudaError_t launch_pages_compact(const Paged &dst, const Paged &src, int32_t *plan, cudaStream_t s);
cudaError_t launch_pages_load(const Paged &c, int slot, const void *k, const float *states, int L, bool bf16, int32_t *plan,
                              cudaStream_t s);

}  // namespace mc
