// k_tree_tc.cu -- what a drafted tree reads of the cached memories, on the tensor cores (bf16 tokens, d = 64 or 128, every cached
// memory read by every node: no SSC).
//
// The reads (tree_read_tc).  A memory's products with a head's queries, D[r][t] = M[r][:] . q_t, are made by tcgen05.mma in bf16: the
// queries are bf16 as they come, and the fp32 memory, which comes by TMA, is split into two bf16 terms, each rounded to
// nearest, that go through tensor memory (together within 2^-18 of every value, to either side; the sums are fp32).  The
// softmax weights are applied to D in fp32, so a read is as accurate as an fp32 one.  A third term would make the split exact; it
// cost 297 us against 279 where both were tried (64 nodes, 12 sequences, gated delta; neither without spills), and no output
// shows it.  kind::tf32 takes the memory as it comes, but cuts it off after 11 bits: up to 2^-10 of a value, and always
// towards zero.  With what is cut off as a second operand it is as accurate too, in twice the products (8 columns each, not
// 16), which one thread issues, 60 to 80 clocks each: 264 us, bound by that, against 217 as it is.
// A memory of 64 KB is read from HBM once for all nodes, 1.5 us of an SM's share of the bandwidth; eight warps need about that for
// the split, the weights and the sums, one thread 0.6 us for the products of 64 nodes.  So the memories stream through a ring
// of 32-column panels (144 KB on an SM; 160 and 176 give nothing), and the split of one tile (a memory of 128 rows, two of 64)
// runs beside the products of the one before and the sums of the one before that.  With most of an SM's memory shared, what a
// thread spills goes to L2: the kernel keeps within its registers.
//
// The memories of all heads and sequences form one line, cut into one range per CTA whatever the sequences' lengths.  A range
// leaves the sum of its weights with its partial read, and tree_finish joins them, as a softmax over parts; the begun segment's
// memory, whose weight hangs on the path, is read without one.
//
// The scores of the cached segments (tree_scores_tc) come first: the reads' CTAs come up beside them and fill their rings.
// The path's own products (tree_path_tc) are a small kernel that comes up beside the reads once these are under way.
// It needs nothing of them, but ends after them, so that what follows has both.
//
// 16 heads of d = 128, bf16: 12 sequences of up to 96 segments, 64 nodes, gated delta 200 us (scores 13, reads 165 at 5.9 TB/s,
// path 53 beside them, finish 29); 8 of up to 63, 32 nodes, linear 102 (8, 79, 18, 12; cold, each alone).
#include <cfloat>
#include <cstdint>

#include "mma_sync.cuh"
#include "paged.cuh"
#include "sm100.cuh"
#include "tensormap.cuh"
#include "tree_nodes.cuh"

namespace mc {

using namespace sm100;

namespace {

__device__ int g_tree_abort;

// Warp-level products (m16n8k16) take the columns of their operands in an order that makes a lane's four of every 16 adjacent:
// tokens and keys come straight from global memory, 8 bytes a lane, and mean keys, in fp32, 16.
// Rows g and g + 8 (g = lane / 4) of an A operand at columns 16 ks + 4 (lane % 4) .. + 3; null rows are zeros.
__device__ __forceinline__ void rows_of(const __nv_bfloat16 *lo, const __nv_bfloat16 *hi, int col, uint32_t (&f)[4])
{
    const uint2 x = lo ? __ldg(reinterpret_cast<const uint2 *>(lo + col)) : make_uint2(0, 0);
    const uint2 y = hi ? __ldg(reinterpret_cast<const uint2 *>(hi + col)) : make_uint2(0, 0);
    f[0] = x.x;
    f[1] = y.x;
    f[2] = x.y;
    f[3] = y.y;
}

// ------------------------------------------------------------------------------------------------ the scores

constexpr int kSpan = 32, kPathThreads = 256, kCol = kSpan + 1;

// Scores of a head's cached segments for 32 nodes, and every node's largest.  Eight segments a warp at a time; a mean key takes
// part in three bf16 terms (2^-25 of it).  A chain of loads bounds it (slot, row, position,
// page, mean key).
template <int D>
__global__ void __launch_bounds__(256, 3) tree_scores_tc(TreeArgs a, int spans)
{
    constexpr int KS = D / 16, LINE = 2 * D + 32;  // router inputs in rows eight banks apart
    __shared__ __align__(16) uint8_t us[kSpan * LINE];
    __shared__ float top[8][kSpan];
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / spans, n0 = (int)blockIdx.x % spans * kSpan, b = bh / c.H, h = bh % c.H;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c4 = lane % 4;
    after_previous();
    let_next_start();
    const uint4 *U = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.u) + ((size_t)bh * a.T + n0) * D);
    const int here = min(kSpan, a.T - n0);
    uint4 inputs[kSpan * (D / 8) / 256];
#pragma unroll
    for (int x = 0; x < kSpan * (D / 8) / 256; ++x) inputs[x] = tid + 256 * x < here * (D / 8) ? __ldg(U + tid + 256 * x) : make_uint4(0, 0, 0, 0);
    const Seat seat = seat_of(a, b, false);
    if (seat.row < 0 || n0 >= seat.m) return;
    const int nb = cached_segments(c, seat.pos);
    const int32_t *table = c.table + (size_t)seat.row * c.nmax;
    int page = 8 * warp + g < nb ? table[8 * warp + g] : -1;
#pragma unroll
    for (int x = 0; x < kSpan * (D / 8) / 256; ++x) {
        const int y = tid + 256 * x;
        *reinterpret_cast<uint4 *>(us + y / (D / 8) * LINE + y % (D / 8) * 16) = inputs[x];
    }
    __syncthreads();
    const float low = __int_as_float(0xff800000);
    float *scores = a.gates + (size_t)bh * a.c.nmax * a.Tp + n0, most[4] = {low, low, low, low};  // of rows g, g + 8, g + 16, g + 24
    for (int i0 = 8 * warp; i0 < nb; i0 += 64) {
        page = valid_page(c, page);
        const float *src = c.kbar + ((size_t)max(page, 0) * c.H + h) * D;
        float4 v[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) v[ks] = page >= 0 ? load4(src + 16 * ks + 4 * c4) : make_float4(0.f, 0.f, 0.f, 0.f);
        const bool there[2] = {__shfl_sync(0xffffffffu, page, 8 * c4) >= 0, __shfl_sync(0xffffffffu, page, 8 * c4 + 4) >= 0};
        page = i0 + 64 + g < nb ? table[i0 + 64 + g] : -1;
        float s[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t hi[2], mid[2], lo[2];
            mma::split3(v[ks].x, v[ks].y, hi[0], mid[0], lo[0]);
            mma::split3(v[ks].z, v[ks].w, hi[1], mid[1], lo[1]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                const uint8_t *first = us + (16 * mt + g) * LINE + 8 * c4 + 32 * ks, *second = first + 8 * LINE;
                const uint2 x = *reinterpret_cast<const uint2 *>(first), y = *reinterpret_cast<const uint2 *>(second);
                const uint32_t f[4] = {x.x, y.x, x.y, y.y};
                mma::mma16816(s[mt], f, hi[0], hi[1]);
                mma::mma16816(s[mt], f, mid[0], mid[1]);
                mma::mma16816(s[mt], f, lo[0], lo[1]);
            }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {  // segment i0 + 2 c4 (+ 1), node n0 + t
                const int seg = i0 + 2 * c4 + (y & 1), t = 16 * mt + g + (y & 2 ? 8 : 0);
                const float x = there[y & 1] ? s[mt][y] : low;
                most[2 * mt + (y >> 1)] = fmaxf(most[2 * mt + (y >> 1)], x);
                if (seg < nb && n0 + t < seat.m) scores[(size_t)seg * a.Tp + t] = x;
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        most[x] = fmaxf(most[x], __shfl_xor_sync(0xffffffffu, most[x], 1));
        most[x] = fmaxf(most[x], __shfl_xor_sync(0xffffffffu, most[x], 2));
        if (c4 == 0) top[warp][8 * x + g] = most[x];
    }
    __syncthreads();
    if (tid < kSpan && n0 + tid < seat.m) {
        float best = -FLT_MAX;  // (no segment may have a page)
#pragma unroll
        for (int x = 0; x < 8; ++x) best = fmaxf(best, top[x][tid]);
        a.top[(size_t)bh * a.Tp + n0 + tid] = best;
    }
}

// ------------------------------------------------------------------------------------------------ the path
// Registers a thread, so that a CTA of each runs on an SM: a quarter of it, with 512 registers a lane, has up to three of the
// reads' ten warps and two of the path's eight.  Neither spills (64 nodes, 12 sequences, gated delta: 217 us; at 112 and 80 the
// reads do, 234, at 104 and 96 267).
constexpr int kPathRegs = 64, kReadRegs = 128;

// Scores of the path's segments, P without the gates, and A, for 32 nodes of a head at a time.  A CTA goes over its
// share of the heads: little enough in registers and shared memory to run beside a CTA of tree_read_tc.
template <int D>
__global__ void __maxnreg__(kPathRegs) tree_path_tc(TreeArgs a, int spans, int segments)
{
    constexpr int KS = D / 16;
    __shared__ Nodes nodes;
    __shared__ float uk[kMaxTree * kCol], us[kSpan];  // u . k [node][token], u . key sum
    extern __shared__ int space[];
    const Paged &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c4 = lane % 4;
    const bool routed = a.mode == MC_GRM;
    let_next_start();
    if (blockIdx.x == gridDim.x - 1) {  // one CTA more, for tree_finish
        leave_line(a, space);
        after_previous();
        return;
    }
    const Line line = make_line(a, space, false);
    for (long long item = blockIdx.x; item < (long long)a.B * c.H * spans; item += gridDim.x - 1) {
        const int bh = (int)(item / spans), n0 = (int)(item % spans) * kSpan, b = bh / c.H, h = bh % c.H;
        const int row = line.row[b], m = line.nodes[b], in0 = line.pos[b] % c.C;
        if (row < 0 || n0 >= m) continue;
        __syncthreads();  // the item before has read nodes and products
        make_nodes<__nv_bfloat16>(a, nodes, b, bh, m, in0);
        const __nv_bfloat16 *U = static_cast<const __nv_bfloat16 *>(a.u) + (size_t)bh * a.T * D;
        const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(a.q) + (size_t)bh * a.T * D;
        const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(a.k) + (size_t)bh * a.T * D;
        if (routed && in0) {  // the begun segment's keys
            const float *sum = c.ksum + ((size_t)row * c.H + h) * D;
            for (int t = warp; t < kSpan && n0 + t < m; t += 8) {
                float x = 0.f;
                if (lane < D / 4) x = dot4(load4(U + (size_t)(n0 + t) * D + 4 * lane), load4(sum + 4 * lane));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (lane == 0) us[t] = x;
            }
        }
        // sixteen tokens and sixteen nodes a warp
        const int x0 = warp / 2 * 16, lo = n0 + warp % 2 * 16 + g, hi = lo + 8;
        if (x0 < m) {
            float uf[2][4] = {}, qf[2][4] = {}, kf[2][4] = {};
            auto row_of = [&](const __nv_bfloat16 *x, int n) { return n < m ? x + (size_t)n * D : nullptr; };
#pragma unroll 2
            for (int ks = 0; ks < KS; ++ks) {
                const int col = 16 * ks + 4 * c4;
                uint32_t key[4], f[4];
                rows_of(row_of(K, x0 + g), row_of(K, x0 + 8 + g), col, key);  // B of two tiles: {0, 2} and {1, 3}
                if (routed) {
                    rows_of(row_of(U, lo), row_of(U, hi), col, f);
                    mma::mma16816(uf[0], f, key[0], key[2]);
                    mma::mma16816(uf[1], f, key[1], key[3]);
                }
                rows_of(row_of(Q, lo), row_of(Q, hi), col, f);
                mma::mma16816(qf[0], f, key[0], key[2]);
                mma::mma16816(qf[1], f, key[1], key[3]);
                if (a.delta) {
                    rows_of(row_of(K, lo), row_of(K, hi), col, f);
                    mma::mma16816(kf[0], f, key[0], key[2]);
                    mma::mma16816(kf[1], f, key[1], key[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int x = x0 + 8 * nt + 2 * c4 + (y & 1), n = y & 2 ? hi : lo;
                    uk[x * kCol + n - n0] = uf[nt][y];
                    if (x >= m || n >= a.Tp) continue;
                    const bool above = n < m && (nodes.anc[n] >> x) & 1;
                    a.P[((size_t)bh * a.T + x) * a.Tp + n] = above ? path_read(a, nodes, n, x, 1.f, qf[nt][y]) : 0.f;
                    if (a.delta) a.A[((size_t)bh * a.T + x) * a.Tp + n] = above ? path_meet(nodes, n, x, kf[nt][y]) : 0.f;
                }
        }
        __syncthreads();
        for (int t = warp; t < kSpan && n0 + t < m; t += 8) {
            const int n = n0 + t, last = nodes.seg[n];
            const uint64_t mine = nodes.anc[n];
            float *score = a.score + (size_t)bh * segments * a.Tp + n;
            if (routed) {
                for (int j = 0; j <= last; ++j) {
                    const uint64_t w = mine & nodes.seg_set[j];
                    float x = ((w >> lane) & 1 ? uk[lane * kCol + t] : 0.f) + ((w >> (lane + 32)) & 1 ? uk[(lane + 32) * kCol + t] : 0.f);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    if (j == 0 && in0) x += us[t];
                    if (lane == 0) score[(size_t)j * a.Tp] = x / (float)(j < last ? c.C : (in0 + __popcll(mine) - 1) % c.C + 1);
                }
            } else {
                for (int j = lane; j <= last; j += 32) score[(size_t)j * a.Tp] = 0.f;
            }
            if (lane == 0) {
                a.into[(size_t)bh * a.Tp + n] = a.delta ? decay_from_cache(nodes, n) : 1.f;
                if (h == 0) {
                    a.anc[(size_t)b * kMaxTree + n] = mine;
                    a.seg[(size_t)b * kMaxTree + n] = last;
                }
            }
        }
    }
    after_previous();
}

// ------------------------------------------------------------------------------------------------ the reads

constexpr int kWorkers = 8, kThreads = 32 * (kWorkers + 2);
constexpr int kPanels = 9;                    // of the ring: 128 rows (a memory's, or two memories' of 64) by 32 columns
constexpr int kPanelBytes = 128 * 128;
// Columns of tensor memory: of a tile's sums (two tiles), then of every 64 columns' two terms (two tiles again).
constexpr int kSums = 64, kTerm = 32, kTerms = 2 * kTerm;
// The ring and two heads' queries.
template <int D> struct ReadSmem {
    static constexpr int B = kMaxTree * D * 2, BYTES = 1024 + kPanels * kPanelBytes + 2 * B;
};
// With the line of a full batch and up to 4 KB of static memory an SM has room for it.
static_assert(ReadSmem<128>::BYTES + 4 * (4 * kMaxRows + 1) + 4096 <= 227 * 1024);

// A panel of the ring and how often it has been used, modulo 2.
struct Place {
    uint32_t s = 0, phase = 0;
    __device__ __forceinline__ void advance(uint32_t by)
    {
        s += by;
        if (s >= kPanels) {
            s -= kPanels;
            phase ^= 1;
        }
    }
};

// Pairs of fp32 in one instruction: x - y.
__device__ __forceinline__ float2 minus(float2 x, float2 y)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, m;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 m, {%6, %6};\n\t"
        "fma.rn.f32x2 x, y, m, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(-1.f));
    return r;
}
// The largest magnitude; NaN if any is.
__device__ __forceinline__ float most(float x, float y, float z)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

enum { kCached, kBegunQ, kBegunK };
// Memories of one head that follow each other in a CTA's range: cached ones, or the begun one for the queries or the keys.
struct Run {
    int h, bh, row, nb, m, i0, i1, kind;
};
// The runs of a range, in order; every role walks the same ones.
struct Runs {
    long long x, end;
    int b;
    __device__ Runs(const TreeArgs &a, const Line &l)
    {
        const long long U = (long long)l.units[a.B] * a.c.H, R = ranges_of(U, a.ranges);
        const bool in = blockIdx.x < R;
        x = in ? range_begin(blockIdx.x, U, R) : 0;
        end = in ? range_begin(blockIdx.x + 1, U, R) : 0;
        b = 0;
    }
    __device__ bool next(const TreeArgs &a, const Line &l, Run &r)
    {
        int nu, read;
        long long in_b;
        while (true) {
            if (x >= end) return false;
            while (x >= (long long)l.units[b + 1] * a.c.H) ++b;
            nu = l.units[b + 1] - l.units[b];
            in_b = x - (long long)l.units[b] * a.c.H;
            r.i0 = (int)(in_b % nu);
            read = units_of(a, l.pos[b]);
            if (r.i0 < read) break;
            x += nu - r.i0;  // past what comes after a head's memories
        }
        r.h = (int)(in_b / nu);
        r.bh = b * a.c.H + r.h;
        r.row = l.row[b];
        r.nb = cached_segments(a.c, l.pos[b]);
        r.m = l.nodes[b];
        r.kind = r.i0 < r.nb ? kCached : r.i0 == r.nb ? kBegunQ : kBegunK;
        const int stop = r.kind == kCached ? r.nb : r.i0 + 1;
        const long long left = end - x;
        r.i1 = left < stop - r.i0 ? r.i0 + (int)left : stop;
        x += r.i1 - r.i0;
        return true;
    }
};

template <int D>
__global__ void __maxnreg__(kReadRegs)
tree_read_tc(const __grid_constant__ CUtensorMap pages, const __grid_constant__ CUtensorMap online, TreeArgs a)
{
    constexpr int PANELS = D / 32, BLOCKS = D / 64, BATCH = 128 / D;  // of a tile: panels, pairs of them, and memories
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bs = ring + kPanels * kPanelBytes;
    int *space = reinterpret_cast<int *>(raw + ReadSmem<D>::BYTES);
    __shared__ uint64_t full[kPanels], empty[kPanels], terms[2], b_full[2], d_full[2], d_empty[2], drain;
    __shared__ __align__(16) float weights[kWorkers][2][32];
    __shared__ struct { float *out; int nodes; } done[kWorkers];  // the run before
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const Paged &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (!a.scored) after_previous();  // (else the scores' kernel has waited for what came before)
    const int NT = (a.T + 15) / 16 * 16;  // columns of D
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kPanels; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWorkers / 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&terms[i], kWorkers);
            mbar_init(&b_full[i], kWorkers);
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], kWorkers);
        }
        mbar_init(&drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    const Line line = make_line(a, space, false);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base;
    Runs runs(a, line);
    Run r{};

    if (warp == kWorkers) {
        if (lane == 0) {
            prefetch_tensormap(&pages);
            prefetch_tensormap(&online);
            Place p;
            uint32_t used = 0;  // panels, as far as the ring's number of them
            bool ok = true;
            while (ok && runs.next(a, line, r)) {
                prefetch_l2(static_cast<const __nv_bfloat16 *>(r.kind == kBegunK ? a.k : a.q) + (size_t)r.bh * a.T * D, a.T * D * 2);
                const int32_t *table = c.table + (size_t)r.row * c.nmax;
                const bool cached = r.kind == kCached;
                int page[BATCH];
#pragma unroll
                for (int y = 0; y < BATCH; ++y) page[y] = cached && r.i0 + y < r.i1 ? table[r.i0 + y] : 0;
                for (int i = r.i0; ok && i < r.i1; i += BATCH) {
                    int at[BATCH];
#pragma unroll
                    for (int y = 0; y < BATCH; ++y) {
                        const int was = page[y];
                        if (cached && i + BATCH + y < r.i1) page[y] = table[i + BATCH + y];
                        // a segment without a page is one past the pool: zeros
                        at[y] = cached ? (valid_page(c, was) < 0 ? c.P * c.H : was * c.H + r.h) : r.row * c.H + r.h;
                    }
                    const int here = min(BATCH, r.i1 - i);
                    for (int x = 0; x < PANELS; ++x) {
                        if (!(ok = mbar_wait(&empty[p.s], p.phase ^ 1, &abort_flag))) break;
                        mbar_arrive_expect_tx(&full[p.s], here * (kPanelBytes / BATCH));
#pragma unroll
                        for (int y = 0; y < BATCH; ++y)
                            if (y < here)
                                tma_load_3d(ring + p.s * kPanelBytes + y * (kPanelBytes / BATCH), cached ? &pages : &online, 32 * x, 0, at[y], &full[p.s]);
                        p.advance(1);
                        used = min(used + 1, (uint32_t)kPanels);
                    }
                }
            }
            for (; used > 0; --used) {  // no copy lands after the CTA has left
                int gave_up = 0;
                const uint32_t s = p.s >= used ? p.s - used : p.s + kPanels - used;
                mbar_wait_limit(&full[s], p.s >= used ? p.phase : p.phase ^ 1, &gave_up, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == kWorkers + 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16(128, NT, false, false);
            uint32_t u = 0, n = 0;
            bool ok = true;
            while (ok && runs.next(a, line, r)) {
                ok = mbar_wait(&b_full[u & 1], (u >> 1) & 1, &abort_flag);
                const uint32_t b0 = smem_u32(bs + (u & 1) * ReadSmem<D>::B);
                for (int i = r.i0; ok && i < r.i1; i += BATCH, ++n) {
                    if (!(ok = mbar_wait(&d_empty[n & 1], ((n >> 1) & 1) ^ 1, &abort_flag) &&
                               mbar_wait(&terms[n & 1], (n >> 1) & 1, &abort_flag)))
                        break;
                    tc_fence_after();
                    const uint32_t d = tb + kSums * (n & 1), a0 = tb + 2 * kSums + BLOCKS * kTerms * (n & 1);
                    const uint64_t bx = make_desc_sw128(b0, 0, 1024);
#pragma unroll
                    for (int x = 0; x < BLOCKS; ++x)
#pragma unroll
                        for (int y = 0; y < 8; ++y) mma_ts(d, a0 + kTerms * x + 8 * y, bx + (uint64_t)(x * NT * 8 + 2 * (y % 4)), idesc, x > 0 || y > 0);
                    mma_commit(&d_full[n & 1]);
                }
                ++u;
            }
            if (n > 0) {  // the products under way end before tensor memory is freed, whoever has given up
                int gave_up = 0;
                mma_commit(&drain);
                mbar_wait_limit(&drain, 0, &gave_up, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else {
        // this thread's row of a tile, the warp's panels (every other) and columns of D (16 of every 32); the node whose weights
        // the lane forms
        const int quarter = warp % 4, side = warp / 4, row = 32 * quarter + lane, half = row / D, t = 16 * side + lane % 16 + (lane & 16) * 2;
        uint32_t u = 0, n = 0;
        Place at;
        at.advance(side);
        bool ok = true, counts = false;  // counts: the half's memory is there in the tile before
        float acc[2][16];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < 16; ++x) acc[y][x] = 0.f;
        // tile i's sums, weighted
        auto add_up = [&](uint32_t i) {
            if (!mbar_wait(&d_full[i & 1], (i >> 1) & 1, &abort_flag)) return false;
            tc_fence_after();
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (16 * side + 32 * y >= NT) break;
                float x[16];
                tmem_ld16f(tmem_addr(tb + kSums * (i & 1), 32 * quarter, 16 * side + 32 * y), x);
                tmem_wait_ld();
                if (!counts) continue;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float4 w = load4(&weights[warp][i & 1][16 * y + 4 * z]);
                    acc[y][4 * z] = fmaf(w.x, x[4 * z], acc[y][4 * z]);
                    acc[y][4 * z + 1] = fmaf(w.y, x[4 * z + 1], acc[y][4 * z + 1]);
                    acc[y][4 * z + 2] = fmaf(w.z, x[4 * z + 2], acc[y][4 * z + 2]);
                    acc[y][4 * z + 3] = fmaf(w.w, x[4 * z + 3], acc[y][4 * z + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[i & 1]);
            return true;
        };
        // a run's sums to where they belong, in eights of nodes, for which there is room
        auto bring_out = [&]() {
            const int nodes = done[warp].nodes;
            float *out = done[warp].out + row % D;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int node = 16 * side + 32 * (y / 2) + 8 * (y % 2);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (node < nodes) out[(size_t)(node + x) * D] = acc[y / 2][8 * (y % 2) + x];
                    acc[y / 2][8 * (y % 2) + x] = 0.f;
                }
            }
        };
        for (bool more = true; ok && more;) {
            more = runs.next(a, line, r);
            if (!more) {  // one turn more, for the last tile's sums
                r.i0 = r.m = 0;
                r.i1 = 1;
                r.kind = kBegunQ;
            }
            if (more) {
                // B: the head's queries (or keys).  Its slot is free: every warp has seen the end of the run before the last one.
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(r.kind == kBegunK ? a.k : a.q) + (size_t)r.bh * a.T * D);
                uint8_t *b = bs + (u & 1) * ReadSmem<D>::B;
#pragma unroll 4
                for (int x = tid; x < NT * (D / 8); x += 32 * kWorkers) {
                    const int node = x / (D / 8), piece = x % (D / 8);
                    const uint4 w = node < r.m ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(b + piece / 8 * NT * 128 + node * 128 + (((piece % 8) ^ (node & 7)) << 4)) = w;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_full[u & 1]);
            }
            if (u == 0) {
                after_previous();  // the scores
                let_next_start();
            }
            const bool in = t < r.m, scored = r.kind == kCached && a.scored && in;
            const float best = scored ? a.top[(size_t)r.bh * a.Tp + t] : 0.f;
            const float *next = a.gates + ((size_t)r.bh * c.nmax + r.i0) * a.Tp + t;
            // the weight's logarithm: a score, or 0 (what has no page is read as zeros)
            auto load = [&](int i) {
                const float x = scored && i < r.i1 ? *next : 0.f;
                next += a.Tp;
                return x;
            };
            float ahead[2 * BATCH];  // scores come from L2, whose latency is some memories' time
#pragma unroll
            for (int x = 0; x < 2 * BATCH; ++x) ahead[x] = load(r.i0 + x);
            float z = 0.f;
            for (int i = r.i0; i < r.i1; i += BATCH, ++n) {
                const bool there = i + half < r.i1;
                if (more) {
                    const uint32_t to = tmem_addr(tb + 2 * kSums + BLOCKS * kTerms * (n & 1) + 16 * side, 32 * quarter, 0);
#pragma unroll 1
                    for (int x = 0; x < BLOCKS; ++x) {
                        if (!(ok = mbar_wait(&full[at.s], at.phase, &abort_flag))) break;
                        if (there) {  // (what lies in the rows of a memory that is not there goes into sums that nobody takes)
                            const uint8_t *from = ring + at.s * kPanelBytes + row * 128;
                            float4 all[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) all[y] = *reinterpret_cast<const float4 *>(from + ((y ^ (row & 7)) << 4));
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                uint32_t hi[8], lo[8];
                                float big = 0.f;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const float4 w = all[4 * z + y];
                                    hi[2 * y] = mma::pack2(w.x, w.y);
                                    hi[2 * y + 1] = mma::pack2(w.z, w.w);
                                    const float2 p = minus(make_float2(w.x, w.y), make_float2(mma::low_f(hi[2 * y]), mma::high_f(hi[2 * y])));
                                    const float2 q = minus(make_float2(w.z, w.w), make_float2(mma::low_f(hi[2 * y + 1]), mma::high_f(hi[2 * y + 1])));
                                    lo[2 * y] = mma::pack2(p.x, p.y);
                                    lo[2 * y + 1] = mma::pack2(q.x, q.y);
                                    big = most(most(big, p.x, p.y), q.x, q.y);
                                }
                                // not finite, or rounded to what is not: the first term cut off; of what is not finite it is all
                                if (!(big < FLT_MAX)) {
#pragma unroll
                                    for (int y = 0; y < 8; ++y) {
                                        const uint2 w = *reinterpret_cast<const uint2 *>(from + (((4 * z + y / 2) ^ (row & 7)) << 4) + y % 2 * 8);
                                        const float p = __uint_as_float(w.x), q = __uint_as_float(w.y);
                                        const uint32_t p0 = w.x & 0xffff0000u, q0 = w.y & 0xffff0000u;
                                        hi[y] = p0 >> 16 | q0 | (isnan(p) ? 0x40u : 0u) | (isnan(q) ? 0x400000u : 0u);
                                        lo[y] = mma::pack2(isfinite(p) ? p - __uint_as_float(p0) : 0.f, isfinite(q) ? q - __uint_as_float(q0) : 0.f);
                                    }
                                }
                                __syncwarp();
                                tmem_st8(to + kTerms * x + 8 * z, hi);
                                tmem_st8(to + kTerms * x + kTerm + 8 * z, lo);
                            }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&empty[at.s]);
                        at.advance(2);
                    }
                    if (!ok) break;
                    float mine = 0.f;
#pragma unroll
                    for (int y = 0; y < BATCH; ++y) {
                        const float w = in && i + y < r.i1 ? expf(ahead[y] - best) : 0.f;
                        z += w;
                        if (y == half) mine = w;
                        ahead[y] = ahead[y + BATCH];
                        ahead[y + BATCH] = load(i + y + 2 * BATCH);
                    }
                    weights[warp][n & 1][lane] = mine;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&terms[n & 1]);
                }
                if (n > 0) {  // a tile behind the products
                    if (!(ok = add_up(n - 1))) break;
                    if (i == r.i0) bring_out();
                }
                counts = there;
            }
            if (!ok || !more) break;
            const size_t part = (size_t)blockIdx.x + r.bh;
            if (r.kind == kCached && !a.scored) {  // nothing is scored: the pages that there are
                z = 0.f;
                for (int i = r.i0; i < r.i1; ++i) z += valid_page(c, c.table[(size_t)r.row * c.nmax + i]) >= 0 ? 1.f : 0.f;
            }
            if (r.kind == kCached && in && quarter == 0) a.weight[part * a.Tp + t] = make_float2(best, z);
            if (lane == 0) {  // of the cached memories both halves' sums, which tree_finish adds
                const bool cached = r.kind == kCached;
                done[warp].out = cached ? a.part + (part + (half ? a.ranges + (size_t)a.B * c.H : 0)) * a.Tp * D
                                        : (r.kind == kBegunQ ? a.Y0 : a.Z) + (size_t)r.bh * a.Tp * D;
                done[warp].nodes = half && !cached ? 0 : r.m;
            }
            __syncwarp();
            ++u;
        }
    }
    __syncwarp();
    tmem_wait_st();  // (of a conversion that was given up)
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
    if (tid == 0 && abort_flag) atomicExch(&g_tree_abort, 1);
}

template <int D>
cudaError_t scores_impl(const TreeArgs &a, cudaStream_t s)
{
    const int spans = (a.T + kSpan - 1) / kSpan;
    cudaError_t e = cudaFuncSetAttribute(tree_scores_tc<D>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    return e == cudaSuccess ? launch_early(tree_scores_tc<D>, (size_t)a.B * a.c.H * spans, 256, 0, s, a, spans) : e;
}

template <int D>
cudaError_t path_impl(const TreeArgs &a, cudaStream_t s)
{
    const int spans = (a.T + kSpan - 1) / kSpan;
    const long long items = (long long)a.B * a.c.H * spans;
    // the SM's shared memory is divided for the CTA of reads that comes beside this one
    cudaError_t e = cudaFuncSetAttribute(tree_path_tc<D>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    // one CTA an SM beside the reads of many segments; where there is room for few, most of the path comes after them, and three
    // fit: 16 heads of d = 128, gated delta, 64 nodes, 32 sequences of 5 to 10 segments 230 -> 198 us, 12 of up to 96 189 -> 206;
    // of up to 16 nodes there is too little for that: d = 64, 32 sequences of up to 10 segments 48 -> 52.  The host knows the
    // room, not what is cached: the same short sequences in a table of 17 or 1024 take the 230
    const long long most = (long long)a.ranges * (a.c.nmax <= 16 && a.T > 16 ? 3 : 1);
    return launch_early(tree_path_tc<D>, (size_t)(items < most ? items : most) + 1, kPathThreads, sizeof(int) * Line::ints(a.B), s, a, spans,
                        path_segments(a));
}

// A [matrices][D][D] fp32 tensor in boxes of 32 columns of one matrix, 128-byte swizzled.
bool make_map(CUtensorMap *map, const float *base, unsigned long long matrices, int D)
{
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)D, matrices};
    cuuint64_t strides[2] = {(cuuint64_t)D * 4, (cuuint64_t)D * D * 4};
    cuuint32_t box[3] = {32, (cuuint32_t)D, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool tree_tc_supported(const TreeArgs &a)
{
    // every page and row of a head as a coordinate, and one past them
    return a.bf16 && (a.c.d == 64 || a.c.d == 128) && a.mode != MC_SSC && (long long)a.c.P * a.c.H < (1ll << 31) - 1;
}

cudaError_t launch_tree_scores_tc(const TreeArgs &a, cudaStream_t s)
{
    return a.c.d == 128 ? scores_impl<128>(a, s) : scores_impl<64>(a, s);
}

cudaError_t launch_tree_path_tc(const TreeArgs &a, cudaStream_t s)
{
    return a.c.d == 128 ? path_impl<128>(a, s) : path_impl<64>(a, s);
}

cudaError_t launch_tree_read_tc(const TreeArgs &a, cudaStream_t s)
{
    CUtensorMap pages, online;
    if (!make_map(&pages, a.c.pages, (unsigned long long)a.c.P * a.c.H, a.c.d) ||
        !make_map(&online, a.c.online, (unsigned long long)a.c.S * a.c.H, a.c.d))
        return cudaErrorInvalidValue;
    return launch_early(a.c.d == 128 ? tree_read_tc<128> : tree_read_tc<64>, (size_t)a.ranges, kThreads,
                        (a.c.d == 128 ? ReadSmem<128>::BYTES : ReadSmem<64>::BYTES) + sizeof(int) * Line::ints(a.B), s, pages, online, a);
}

cudaError_t take_tree_abort(int *was_set)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_abort, sizeof(int));
    if (e != cudaSuccess) return e;
    *was_set = v;
    if (v) {
        v = 0;
        e = cudaMemcpyToSymbol(g_tree_abort, &v, sizeof(int));
    }
    return e;
}

}  // namespace mc
