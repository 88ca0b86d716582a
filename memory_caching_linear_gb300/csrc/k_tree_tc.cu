// k_tree_tc.cu -- the cached memories' reads of a drafted tree on the tensor cores (bf16 tokens, d = 64 or 128, more than 8
// nodes, every cached memory read by every node: no SSC).
//
// For the head at hand, D[r][t] = sum over memories i of M^(i)[r][:] . (g_{t,i} q_t): the fp32 memory is the A operand as it
// comes by TMA (kind::tf32 takes 11 significant bits of it: 2^-11 of every product against the 2^-9 of y's own rounding), the
// gate-scaled queries are B, rounded to tf32, and the sum over a head's memories stays in tensor memory.  A memory of 64 KB
// is read from HBM once for all nodes, 1.5 us of an SM's share of the bandwidth, against 0.3 us of products at 64 nodes: HBM
// is the bound, so the memories stream through a ring of 32-column panels (144 KB in flight on an SM) and everything else is
// made to keep up.
//
// The memories of all heads and sequences form one line, cut into one range per CTA whatever the sequences' lengths; a head
// that crosses a cut leaves partial sums, which tree_finish adds in their order.
//
// Warps 0-7 make B and drain D, warp 8 brings the panels, warp 9 issues the products.
#include <cstdint>

#include "paged.cuh"
#include "sm100.cuh"
#include "tensormap.cuh"

namespace mc {

using namespace sm100;

namespace {

__device__ int g_tree_abort;

constexpr int kWorkers = 8, kThreads = 32 * (kWorkers + 2);
constexpr int kRingBytes = 147456;            // nine panels of 128 rows, eighteen of 64
constexpr int kMaxPanels = 18;
constexpr int kBSlot = kMaxTree * 128 * 4;    // gate-scaled queries of one memory
constexpr int kSmem = 1024 + kRingBytes + 2 * kBSlot;

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

// One head's memories (or its begun memory for the keys) within a CTA's range.
struct Run {
    int b, h, bh, row, nb, m, i0, i1;
    bool keys;
};
// The runs of a range, in order; every role walks the same ones.
struct Runs {
    long long x, end;
    int b;
    __device__ Runs(const TreeArgs &a)
    {
        const long long U = (long long)a.p.units[a.B] * a.c.H, R = ranges_of(U, a.ranges);
        const bool in = blockIdx.x < R;
        x = in ? range_begin(blockIdx.x, U, R) : 0;
        end = in ? range_begin(blockIdx.x + 1, U, R) : 0;
        b = 0;
    }
    __device__ bool next(const TreeArgs &a, Run &r)
    {
        if (x >= end) return false;
        while (x >= (long long)a.p.units[b + 1] * a.c.H) ++b;
        const int u0 = a.p.units[b], nu = a.p.units[b + 1] - u0;
        const long long in_b = x - (long long)u0 * a.c.H;
        r.b = b;
        r.h = (int)(in_b / nu);
        r.bh = b * a.c.H + r.h;
        r.row = a.p.act[b];
        r.nb = cached_segments(a.c, a.p.pos[b]);
        r.m = nodes_of(a, b);
        r.i0 = (int)(in_b % nu);
        r.keys = r.i0 > r.nb;
        const long long left = end - x;
        const int stop = r.keys || nu <= r.nb + 1 ? nu : r.nb + 1;  // the keys' read is a run of its own
        r.i1 = left < stop - r.i0 ? r.i0 + (int)left : stop;
        x += r.i1 - r.i0;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_read_tc(const __grid_constant__ CUtensorMap pages, const __grid_constant__ CUtensorMap online, TreeArgs a)
{
    constexpr int PANELS = D / 32, kPanelBytes = D * 128, RING = kRingBytes / kPanelBytes;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bs = ring + kRingBytes;  // (a 64-row panel's second half, which nobody reads, may be of the next one or of B)
    __shared__ uint64_t full[kMaxPanels], empty[kMaxPanels], b_full[2], b_empty[2], d_full[2], d_empty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const Paged &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int NT = (a.T + 15) / 16 * 16;                       // columns of D
    const int groups = (NT + 31) / 32, writers = PANELS * groups;  // warps that make B: 32 tokens of one panel each
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base;
    Runs runs(a);
    Run r;

    if (warp == kWorkers) {
        if (lane == 0) {
            prefetch_tensormap(&pages);
            prefetch_tensormap(&online);
            uint32_t g = 0;
            bool ok = true;
            while (ok && runs.next(a, r)) {
                const int32_t *table = c.table + (size_t)r.row * c.nmax;
                int page = r.i0 < r.nb ? table[r.i0] : 0;
                for (int i = r.i0; ok && i < r.i1; ++i) {
                    const int p = page;
                    if (i + 1 < r.nb && i + 1 < r.i1) page = table[i + 1];
                    // a segment without a page is one past the pool: zeros
                    const bool cached = i < r.nb;
                    const int at = cached ? (valid_page(c, p) < 0 ? c.P * c.H : p * c.H + r.h) : r.row * c.H + r.h;
                    for (int x = 0; x < PANELS; ++x, ++g) {
                        const uint32_t s = g % RING;
                        if (!(ok = mbar_wait(&empty[s], ((g / RING) & 1) ^ 1, &abort_flag))) break;
                        mbar_arrive_expect_tx(&full[s], kPanelBytes);
                        tma_load_3d(ring + s * kPanelBytes, cached ? &pages : &online, 32 * x, 0, at, &full[s]);
                    }
                }
            }
            if (!ok) {  // the copies under way land before the CTA leaves
                for (uint32_t x = g > (uint32_t)RING ? g - RING : 0; x < g; ++x) {
                    int gave_up = 0;
                    mbar_wait_limit(&full[x % RING], (x / RING) & 1, &gave_up, kWaitLimitNs);
                }
            }
        }
        __syncwarp();
    } else if (warp == kWorkers + 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_tf32(128, NT);
            uint32_t g = 0, u = 0, n = 0;
            bool ok = true;
            while (ok && runs.next(a, r)) {
                const uint32_t d = tb + 64 * (n & 1);
                ok = mbar_wait(&d_empty[n & 1], ((n >> 1) & 1) ^ 1, &abort_flag);
                for (int i = r.i0; ok && i < r.i1; ++i, ++u) {
                    if (!(ok = mbar_wait(&b_full[u & 1], (u >> 1) & 1, &abort_flag))) break;
                    const uint32_t b0 = smem_u32(bs + (u & 1) * kBSlot);
                    for (int x = 0; x < PANELS; ++x, ++g) {
                        const uint32_t s = g % RING;
                        if (!(ok = mbar_wait(&full[s], (g / RING) & 1, &abort_flag))) break;
                        tc_fence_after();
                        const uint32_t a0 = smem_u32(ring + s * kPanelBytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_tf32(d, make_desc_sw128(a0 + 32 * k, 0, 1024), make_desc_sw128(b0 + x * NT * 128 + 32 * k, 0, 1024),
                                     idesc, i > r.i0 || x > 0 || k > 0);
                        mma_commit(&empty[s]);
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
        const int panel = warp % PANELS, t = warp / PANELS * 32 + lane;  // this thread's token and 32 columns of B
        const bool writes = warp < writers;
        uint32_t u = 0, n = 0;
        bool ok = true;
        while (ok && runs.next(a, r)) {
            if (writes) {
                uint32_t q[16];
                const bool in = t < r.m;
                if (in) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(r.keys ? a.k : a.q) +
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
                const float *gates = a.gates + (size_t)r.bh * (c.nmax + 2) * a.Tp + t;
                float g = in ? gates[(size_t)r.i0 * a.Tp] : 0.f;
                for (int i = r.i0; i < r.i1; ++i, ++u) {
                    const float next = in && i + 1 < r.i1 ? gates[(size_t)(i + 1) * a.Tp] : 0.f;
                    if (!(ok = mbar_wait(&b_empty[u & 1], ((u >> 1) & 1) ^ 1, &abort_flag))) break;
                    uint8_t *row = bs + (u & 1) * kBSlot + panel * NT * 128 + t * 128;
                    if (t < NT) {
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
                    g = next;
                }
            }
            if (!ok || !(ok = mbar_wait(&d_full[n & 1], (n >> 1) & 1, &abort_flag))) break;
            tc_fence_after();
            // rows 32 (warp % 4) + lane of D; the two warps of a quarter take every other 16 columns
            const int quarter = warp % 4, row = 32 * quarter + lane;
            float *out = r.keys ? a.Z + (size_t)r.bh * a.Tp * D : a.part + ((size_t)blockIdx.x + r.bh) * a.Tp * D;
            for (int t0 = 16 * (warp / 4); t0 < NT; t0 += 32) {
                float x[16];
                tmem_ld16f(tmem_addr(tb + 64 * (n & 1), 32 * quarter, t0), x);
                tmem_wait_ld();
                if (row < D) {
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        if (t0 + y < r.m) out[(size_t)(t0 + y) * D + row] = x[y];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[n & 1]);
            ++n;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, 128);
    }
    if (tid == 0 && abort_flag) atomicExch(&g_tree_abort, 1);
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
    return a.bf16 && (a.c.d == 64 || a.c.d == 128) && a.T > 8 && a.mode != MC_SSC && (long long)a.c.P * a.c.H < (1ll << 31) - 1;
}

cudaError_t launch_tree_read_tc(const TreeArgs &a, cudaStream_t s)
{
    CUtensorMap pages, online;
    if (!make_map(&pages, a.c.pages, (unsigned long long)a.c.P * a.c.H, a.c.d) ||
        !make_map(&online, a.c.online, (unsigned long long)a.c.S * a.c.H, a.c.d))
        return cudaErrorInvalidValue;
    auto kern = a.c.d == 128 ? tree_read_tc<128> : tree_read_tc<64>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)a.ranges, kThreads, kSmem, s>>>(pages, online, a);
    return cudaGetLastError();
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
