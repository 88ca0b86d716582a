// k_tree_tc.cu -- what a drafted tree reads of the cached memories, on the tensor cores (bf16 tokens, d = 64 or 128, every cached
// memory read by every node: no SSC).
//
// The reads (tree_read_tc).  For the head at hand, D[r][t] = sum over memories i of M^(i)[r][:] . (g_{t,i} q_t): the fp32 memory is
// the A operand as it comes by TMA (kind::tf32 takes 11 significant bits of it: 2^-11 of every product against the 2^-9 of
// y's own rounding), the weighted queries are B, rounded to tf32, and the sum over a head's memories stays in tensor memory.
// A memory of 64 KB is read from HBM once for all nodes, 1.5 us of an SM's share of the bandwidth, against 0.3 us of products
// at 64 nodes: HBM is the bound, so the memories stream through a ring of 32-column panels (144 KB on an SM) and
// everything else is made to keep up: a head's sums are brought out while the next one's panels and B are on their way.
//
// The memories of all heads and sequences form one line, cut into one range per CTA whatever the sequences' lengths.  A range
// leaves the sum of its weights with its partial read, and tree_finish joins them, as a softmax over parts; the begun segment's
// memory, whose weight hangs on the path, is read without one.
//
// The scores of the cached segments (tree_scores_tc) come first: the reads' CTAs come up beside them and fill their rings.
// The path's own products (tree_path_tc) are a small kernel that comes up beside the reads once these are under way.
// It needs nothing of them, but ends after them, so that what follows has both.
//
// 16 heads of d = 128, bf16: 12 sequences of up to 96 segments, 64 nodes, gated delta 189 us (scores 12, reads 155 at 6.2 TB/s,
// path 51 beside them, finish 30); 8 of up to 63, 32 nodes, linear 98 (8, 78, 18, 14; cold, each alone).
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

// kind::tf32: as idesc_bf16 with both formats tf32.
__host__ __device__ constexpr uint32_t idesc_tf32(int M, int N)
{
    return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ float to_tf32(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return __uint_as_float(r);
}

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
// part in two bf16 terms (2^-17 of it, for weights that are not ranked).  A chain of loads bounds it (slot, row, position,
// page, mean key).
template <int D>
__global__ void __launch_bounds__(256) tree_scores_tc(TreeArgs a, int spans)
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
        uint32_t hi[KS][2], lo[KS][2];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const float4 v = page >= 0 ? load4(src + 16 * ks + 4 * c4) : make_float4(0.f, 0.f, 0.f, 0.f);
            mma::split2(v.x, v.y, hi[ks][0], lo[ks][0]);
            mma::split2(v.z, v.w, hi[ks][1], lo[ks][1]);
        }
        const bool there[2] = {__shfl_sync(0xffffffffu, page, 8 * c4) >= 0, __shfl_sync(0xffffffffu, page, 8 * c4 + 4) >= 0};
        page = i0 + 64 + g < nb ? table[i0 + 64 + g] : -1;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            const uint8_t *first = us + (16 * mt + g) * LINE + 8 * c4, *second = first + 8 * LINE;
            float s[4] = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint2 x = *reinterpret_cast<const uint2 *>(first + 32 * ks), y = *reinterpret_cast<const uint2 *>(second + 32 * ks);
                const uint32_t f[4] = {x.x, y.x, x.y, y.y};
                mma::mma16816(s, f, hi[ks][0], hi[ks][1]);
                mma::mma16816(s, f, lo[ks][0], lo[ks][1]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {  // segment i0 + 2 c4 (+ 1), node n0 + t
                const int seg = i0 + 2 * c4 + (y & 1), t = 16 * mt + g + (y & 2 ? 8 : 0);
                const float x = there[y & 1] ? s[y] : low;
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
// reads' ten warps and two of the path's eight.
constexpr int kPathRegs = 96, kReadRegs = 104;

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
#pragma unroll 4
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
constexpr int kRingBytes = 147456;            // nine panels of 128 rows, eighteen of 64
constexpr int kMaxPanels = 18;
constexpr int kBSlot = kMaxTree * 128 * 4;    // weighted queries of one memory
constexpr int kReadSmem = 1024 + kRingBytes + 2 * kBSlot;

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
    constexpr int PANELS = D / 32, kPanelBytes = D * 128, RING = kRingBytes / kPanelBytes;
    constexpr int BATCH = 4 / PANELS;  // memories whose B share a slot and its handshake
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bs = ring + kRingBytes;  // (a 64-row panel's second half, which nobody reads, may be of the next one or of B)
    int *space = reinterpret_cast<int *>(raw + kReadSmem);
    __shared__ uint64_t full[kMaxPanels], empty[kMaxPanels], b_full[2], b_empty[2], d_full[2], d_empty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const Paged &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (!a.scored) after_previous();  // (else the scores' kernel has waited for what came before)
    const int NT = (a.T + 15) / 16 * 16;                           // columns of D
    const int groups = (NT + 31) / 32, writers = PANELS * BATCH * groups;  // warps that make B: 32 tokens of one panel each
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < RING; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b_full[i], writers);
            mbar_init(&b_empty[i], 1);
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], kWorkers);
        }
        mbar_init(&drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base, 128);
        tmem_relinquish();
    }
    const Line line = make_line(a, space, false);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base;
    Runs runs(a, line);
    Run r;

    if (warp == kWorkers) {
        if (lane == 0) {
            prefetch_tensormap(&pages);
            prefetch_tensormap(&online);
            uint32_t g = 0;
            bool ok = true;
            while (ok && runs.next(a, line, r)) {
                const int32_t *table = c.table + (size_t)r.row * c.nmax;
                const bool cached = r.kind == kCached;
                int page = cached ? table[r.i0] : 0;
                for (int i = r.i0; ok && i < r.i1; ++i) {
                    const int p = page;
                    if (cached && i + 1 < r.i1) page = table[i + 1];
                    // a segment without a page is one past the pool: zeros
                    const int at = cached ? (valid_page(c, p) < 0 ? c.P * c.H : p * c.H + r.h) : r.row * c.H + r.h;
                    for (int x = 0; x < PANELS; ++x, ++g) {
                        const uint32_t s = g % RING;
                        if (!(ok = mbar_wait(&empty[s], ((g / RING) & 1) ^ 1, &abort_flag))) break;
                        mbar_arrive_expect_tx(&full[s], kPanelBytes);
                        tma_load_3d(ring + s * kPanelBytes, cached ? &pages : &online, 32 * x, 0, at, &full[s]);
                    }
                }
            }
            for (uint32_t x = g > (uint32_t)RING ? g - RING : 0; x < g; ++x) {  // no copy lands after the CTA has left
                int gave_up = 0;
                mbar_wait_limit(&full[x % RING], (x / RING) & 1, &gave_up, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == kWorkers + 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_tf32(128, NT);
            uint32_t g = 0, u = 0, n = 0;
            bool ok = true;
            while (ok && runs.next(a, line, r)) {
                const uint32_t d = tb + 64 * (n & 1);
                ok = mbar_wait(&d_empty[n & 1], ((n >> 1) & 1) ^ 1, &abort_flag);
                for (int i = r.i0; ok && i < r.i1; i += BATCH, ++u) {
                    if (!(ok = mbar_wait(&b_full[u & 1], (u >> 1) & 1, &abort_flag))) break;
                    const uint32_t b0 = smem_u32(bs + (u & 1) * kBSlot);
#pragma unroll
                    for (int y = 0; y < BATCH; ++y) {
                        if (!ok || i + y >= r.i1) break;
                        for (int x = 0; x < PANELS; ++x, ++g) {
                            const uint32_t s = g % RING;
                            if (!(ok = mbar_wait(&full[s], (g / RING) & 1, &abort_flag))) break;
                            tc_fence_after();
                            const uint32_t a0 = smem_u32(ring + s * kPanelBytes), bx = b0 + (y * PANELS + x) * NT * 128;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_tf32(d, make_desc_sw128(a0 + 32 * k, 0, 1024), make_desc_sw128(bx + 32 * k, 0, 1024), idesc,
                                         i + y > r.i0 || x > 0 || k > 0);
                            mma_commit(&empty[s]);
                        }
                    }
                    if (ok) mma_commit(&b_empty[u & 1]);
                }
                if (ok) mma_commit(&d_full[n & 1]);
                ++n;
            }
            if (!ok) {  // the products under way end before tensor memory is freed
                int gave_up = 0;
                mma_commit(&drain);
                mbar_wait_limit(&drain, 0, &gave_up, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else {
        // this thread's memory of a slot's, 32 columns of B, and token
        const int sub = warp / PANELS % BATCH, panel = warp % PANELS, t = warp / (PANELS * BATCH) * 32 + lane;
        const bool writes = warp < writers, routed = a.mode == MC_GRM;
        uint32_t u = 0, n = 0;
        bool ok = true;
        after_previous();  // the scores
        // the sums of run `i` to out: rows 32 (warp % 4) + lane of D; the two warps of a quarter take every other 16 columns
        float *out = nullptr;
        int nodes = 0;
        auto bring_out = [&](uint32_t i) {
            if (!mbar_wait(&d_full[i & 1], (i >> 1) & 1, &abort_flag)) return false;
            tc_fence_after();
            const int quarter = warp % 4, row = 32 * quarter + lane;
            for (int t0 = 16 * (warp / 4); t0 < NT; t0 += 32) {
                float x[16];
                tmem_ld16f(tmem_addr(tb + 64 * (i & 1), 32 * quarter, t0), x);
                tmem_wait_ld();
                if (row < D) {
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        if (t0 + y < nodes) out[(size_t)(t0 + y) * D + row] = x[y];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[i & 1]);
            return true;
        };
        while (ok && runs.next(a, line, r)) {
            const float *scores = a.gates + (size_t)r.bh * c.nmax * a.Tp;
            const bool in = writes && t < r.m, cached = r.kind == kCached;
            const float best = cached && in && routed ? a.top[(size_t)r.bh * a.Tp + t] : 0.f;
            uint32_t q[16];
            if (in) {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(r.kind == kBegunK ? a.k : a.q) +
                                                                   ((size_t)r.bh * a.T + t) * D + 32 * panel);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint4 w = __ldg(src + x);
                    q[4 * x] = w.x;
                    q[4 * x + 1] = w.y;
                    q[4 * x + 2] = w.z;
                    q[4 * x + 3] = w.w;
                }
            }
            if (n == 0) let_next_start();
            float z = 0.f;
            bool brought = false;
            if (writes) {
                const int32_t *table = c.table + (size_t)r.row * c.nmax;
                // the weight's logarithm: a score; 0 for a page where nothing is scored
                auto load = [&](int i) {
                    if (!in || i >= r.i1) return 0.f;
                    if (!cached) return 0.f;
                    return routed ? scores[(size_t)i * a.Tp + t] : valid_page(c, table[i]) >= 0 ? 0.f : __int_as_float(0xff800000);
                };
                float ahead[2 * BATCH];  // scores come from L2, whose latency is some memories' time
#pragma unroll
                for (int x = 0; x < 2 * BATCH; ++x) ahead[x] = load(r.i0 + x);
                for (int i = r.i0; i < r.i1; i += BATCH, ++u) {
                    float g = 0.f;
#pragma unroll
                    for (int y = 0; y < BATCH; ++y) {
                        const float w = i + y < r.i1 ? expf(ahead[y] - best) : 0.f;
                        z += w;
                        if (y == sub) g = w;
                        ahead[y] = ahead[y + BATCH];
                        ahead[y + BATCH] = load(i + y + 2 * BATCH);
                    }
                    if (!(ok = mbar_wait(&b_empty[u & 1], ((u >> 1) & 1) ^ 1, &abort_flag))) break;
                    uint8_t *row = bs + (u & 1) * kBSlot + (sub * PANELS + panel) * NT * 128 + t * 128;
                    if (t < NT && i + sub < r.i1) {
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (in) {
                                w.x = to_tf32(g * __uint_as_float(q[2 * x] << 16));
                                w.y = to_tf32(g * __uint_as_float(q[2 * x] & 0xffff0000u));
                                w.z = to_tf32(g * __uint_as_float(q[2 * x + 1] << 16));
                                w.w = to_tf32(g * __uint_as_float(q[2 * x + 1] & 0xffff0000u));
                            }
                            *reinterpret_cast<float4 *>(row + ((x ^ (t & 7)) << 4)) = w;
                        }
                        fence_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b_full[u & 1]);
                    if (i == r.i0 + BATCH && n > 0) {  // two slots ahead of the products
                        if (!(ok = bring_out(n - 1))) break;
                        brought = true;
                    }
                }
            }
            if (ok && n > 0 && !brought) ok = bring_out(n - 1);
            if (!ok) break;
            const size_t part = (size_t)blockIdx.x + r.bh;
            if (cached && in && panel == 0 && sub == 0) a.weight[part * a.Tp + t] = make_float2(best, z);
            out = cached ? a.part + part * a.Tp * D : (r.kind == kBegunQ ? a.Y0 : a.Z) + (size_t)r.bh * a.Tp * D;
            nodes = r.m;
            ++n;
        }
        if (ok && n > 0) bring_out(n - 1);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, 128);
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
    // fit: 16 heads of d = 128, gated delta, 64 nodes, 32 sequences of 5 to 10 segments 227 -> 198 us, 12 of up to 96 189 -> 206;
    // of up to 16 nodes there is too little for that: d = 64, 32 sequences of up to 10 segments 48 -> 52
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
                        kReadSmem + sizeof(int) * Line::ints(a.B), s, pages, online, a);
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
