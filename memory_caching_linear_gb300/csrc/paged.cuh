// paged.cuh -- argument blocks and device helpers of decoding over a paged cache (mc_pages.cu, k_pages.cu, k_step.cu, k_tree.cu,
// k_tree_tc.cu).
//
// The acceptance of a path, a fork, a compaction and a prompt's loading begin with a plan (one CTA): which rows of the cache
// are worked on, and what is needed of the pool.  The kernel after it takes positions from the plan alone, so that it may write
// the cache's.  A step and a tree's reads need no plan.
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

// What the acceptance of paths does with the batch rows' sequences.
struct Plan {
    int32_t *act;      // [B] the cache's row, -1: nothing to do
    int32_t *pos;      // [B] position before the call
    uint64_t *path;    // [B] the nodes of the path
    int32_t *fresh;    // [B + 1] where a batch row's new pages begin in list
    int32_t *list;     // new pages in order of batch row and time, -1 where none was free
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
    // Scratch.  In what follows a split read is one whose cached memories are weighed as they are read, without what the path
    // adds to the softmax (k_tree_tc.cu); otherwise the gates are worked out first (k_tree.cu).
    int32_t *line;                        // the batch's seats (Line)
    float *gates;                         // [BH][nmax + 2][Tp] gates of the cached memories, then what nodes read of the begun
                                          // segment's with their queries (gate and decay) and with their keys (decay); split:
                                          // [BH][nmax][Tp] scores
    float *top;                           // [BH][Tp] split: the largest of a node's
    float *P, *A;                         // [BH][T][Tp] per ancestor: what nodes read of what it wrote (a split read's without
                                          // the gates); what it meets in their keys
    float *score;                         // [BH][path_segments()][Tp] split: nodes' scores of their paths' segments
    float *into;                          // [BH][Tp] split: decay from the cache to a node's deepest ancestor in the begun segment
    uint64_t *anc;                        // [B][64] a node's ancestors and itself
    int32_t *seg;                         // [B][64] its segment, counted from the one begun
    float *Y0, *Z;                        // [BH][Tp][d] the begun segment's memory read with the nodes' queries (split, without gate
                                          // and decay) and with their keys (decayed; split: without)
    float *part;                          // [ranges + BH][Tp][d] partial reads (split at d = 64: twice, the sums of every other memory)
    float2 *weight;                       // [ranges + BH][Tp] split: top, or 0 without a router, and the sum of exp(score - top)
    int B, T, Tp, mode, topk;
    int ranges, groups;                   // shares of the memories; of the tokens
    int rest;                             // what a head's end costs, in memories (sum_line)
    bool scored;                          // split: tree_scores_tc comes first
    bool bf16, delta, whole;              // whole: tree_gates does all (a tree of up to 8 nodes over few heads)
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
    return cached_segments(a.c, pos) + (pos % a.c.C ? (a.delta ? 2 : 1) : 0);
}
// A batch row's place: the cache's row (-1: nobody's), its position, and its nodes.  tell: what is out of range is reported.
struct Seat {
    int row, pos, m;
};
__device__ __forceinline__ Seat seat_of(const TreeArgs &a, int b, bool tell)
{
    Seat s{-1, 0, a.T};
    const Paged &c = a.c;
    const int slot = a.slots ? a.slots[b] : b;
    bool bad = slot < -1 || slot >= c.S;
    if (!bad && slot >= 0) {
        s.row = c.row[slot];
        if ((unsigned)s.row >= (unsigned)c.S || (unsigned)(s.pos = c.pos[s.row]) > (unsigned)kMaxPos) {
            bad = true;
            s.row = -1;
        } else if (a.count) {
            const int n = a.count[b];
            s.m = max(0, min(n, a.T));
            bad = s.m != n;
        }
    }
    if (bad && tell) atomicOr(c.status, MC_PAGES_INDEX);
    return s;
}
__device__ __forceinline__ int units_of(const TreeArgs &a, const Seat &s) { return s.row < 0 || s.m == 0 ? 0 : units_of(a, s.pos); }

// The whole batch's seats and where their memories begin in the line of all (per head): 4 B + 1 ints.  Finding them takes four
// loads that wait for one another, so a kernel does it once, and a kernel at a call's end is left them in memory.
struct Line {
    int *row, *pos, *nodes, *units;
    __host__ __device__ static size_t ints(int B) { return 4 * (size_t)B + 1; }
};
__host__ __device__ inline Line line_in(int *space, int B) { return Line{space, space + B, space + 2 * B, space + 3 * B}; }
// units[b + 1] are row b's own memories: makes them sums.  Where there is a memory for every range, a.rest more, which nobody
// reads, come after those of a head.  The whole block calls it.
__device__ inline void sum_line(const TreeArgs &a, const Line &l)
{
    constexpr unsigned kSum = (1u << 21) - 1;  // rows with memories are counted above it
    __syncthreads();
    if (threadIdx.x < 32) {
        unsigned sum = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + (int)threadIdx.x;
            unsigned x = b < a.B ? (unsigned)l.units[b + 1] : 0;
            if (x) x += kSum + 1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                if ((int)threadIdx.x >= o) x += y;
            }
            if (b < a.B) l.units[b + 1] = (int)(sum + x);
            sum += __shfl_sync(0xffffffffu, x, 31);
        }
        const unsigned rest = (long long)(sum & kSum) * a.c.H >= a.ranges ? a.rest : 0;
        __syncwarp();
        for (int b = threadIdx.x; b < a.B; b += 32) {
            const unsigned x = (unsigned)l.units[b + 1];
            l.units[b + 1] = (int)((x & kSum) + rest * (x >> 21));
        }
        if (threadIdx.x == 0) l.units[0] = 0;
    }
    __syncthreads();
}
// The batch's line in shared memory; the whole block calls it.  tell as for seat_of.
__device__ inline Line make_line(const TreeArgs &a, int *space, bool tell)
{
    const Line l = line_in(space, a.B);
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const Seat s = seat_of(a, b, tell);
        l.row[b] = s.row;
        l.pos[b] = s.pos;
        l.nodes[b] = s.m;
        l.units[b + 1] = units_of(a, s);
    }
    sum_line(a, l);
    return l;
}
// To memory, for tree_finish.
__device__ inline void leave_line(const TreeArgs &a, int *space)
{
    make_line(a, space, true);
    for (size_t i = threadIdx.x; i < Line::ints(a.B); i += blockDim.x) a.line[i] = space[i];
}

// CTAs of tree_read that share a range, each with a part of the rows: four rows to a lane at d = 128 (and 64), two CTAs an SM.
// With 16 rows there is one (fp32, 16 heads: 4 sequences of 30 to 63 segments, 24 nodes 226 -> 157 us; 2 of up to 63, 4 heads, 16
// nodes 57 -> 36), with two what goes with a memory outweighs its products (157 -> 232; d = 64, 84 -> 113).
__host__ __device__ constexpr int read_blocks(int d) { return d == 128 ? 4 : 1; }

// Segments that a path of T nodes can touch.
inline int path_segments(const TreeArgs &a) { return (int)(((long long)a.c.C - 1 + a.T - 1) / a.c.C) + 1; }

// Kernels of a call come up while the one before still runs its last CTAs.  after_previous() waits for all that came
// before; what a kernel does ahead of it must not depend on that.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename K, typename... A>
cudaError_t launch_early(K *kern, size_t grid, int block, size_t smem, cudaStream_t s, const A &...args)
{
    cudaError_t e = smem > 16 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
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
bool tree_whole(const TreeArgs &a);
cudaError_t launch_tree_gates(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_read(const TreeArgs &a, cudaStream_t s);
bool tree_tc_supported(const TreeArgs &a);  // the split read on the tensor cores
cudaError_t launch_tree_scores_tc(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_path_tc(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_tree_read_tc(const TreeArgs &a, cudaStream_t s);
cudaError_t take_tree_abort(int *was_set);
cudaError_t launch_tree_finish(const TreeArgs &a, cudaStream_t s);
// A step's memory in the cache (mc_paged_cache's work): tickets, zero between calls, and partial reads.
struct StepWork {
    int32_t *turns;  // [S H + 1]
    float *part;     // [ranges + S H][d + 2] a range's read, its largest score and sum of weights
    float *online;   // [S H][d + 1] the online memory's read and score
};
cudaError_t launch_step(const TreeArgs &a, const StepWork &work, cudaStream_t s);
cudaError_t take_step_abort(int *was_set);
cudaError_t launch_accept(const TreeArgs &a, cudaStream_t s);
cudaError_t launch_fork(const Paged &c, const int32_t *src, int32_t *plan, cudaStream_t s);
cudaError_t launch_pages_compact(const Paged &dst, const Paged &src, int32_t *plan, cudaStream_t s);
cudaError_t launch_pages_load(const Paged &c, int slot, const void *k, const float *states, int L, bool bf16, int32_t *plan,
                              cudaStream_t s);

}  // namespace mc
