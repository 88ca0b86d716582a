// k_delta_tc.cu -- tensor-core kernels of the gated delta memory for bf16 inputs, d = 64 or 128, any
// segment length (the formulas are in k_delta_simt.cu).
//
// Within a chunk of 64 tokens, with c_i the running sum of log_alpha, D_ij = exp(c_i - c_j), S the
// memory before the chunk and A_ij = D_ij (k_i . k_j) beta_j for j < i (else 0):
//   (1 + A) E = V - diag(exp c) K S^T         every error of the chunk at once
//   O   = diag(exp c) Q S^T + P diag(beta) E,  P_ij = D_ij (q_i . k_j), j <= i
//   S'  = exp(c_end) S + (diag(beta exp(c_end - c)) E)^T K
// delta_prep_tc forms (1 + A)^-1 and P for all chunks at once; delta_walk_tc then goes through a
// segment's chunks.  A warp of the walk owns 16 value rows of S in registers and works on S K^T, R T^T and
// U^T K transposed (rows: values, columns: tokens or keys), where every result is the next product's
// left operand as it lies: the warps of a head never exchange anything, so the rows of one head can be
// spread over CTAs.  This is why the products are warp-level ones: the chunk's chain of four products is
// short and each is small, and an accumulator in tensor memory would have to be read back, split and
// written to shared memory between any two of them.
//
// Precision: the memory is held in fp32, and what is not an input enters the products in two bf16 terms, products of two
// lows left out: 2^-17 of a term (the inverse in three, 2^-25).  The errors e_j of keys that resemble each other are large
// and cancel in S, in O and in the gradients' sums over pairs, so one term (2^-9) would show: at keys with a cosine of 0.8 it
// leaves the memory 7e-3 and y 9e-3 off, as against 2e-5 and 1.4e-3, the last bf16 rounding, and at all but parallel ones
// dq and dbeta 5e-2.  One term's are readings in which nothing cancels and whose results are bf16: O's of S, and in the
// gradients' kernels S and R at a chunk's ends; E's of S in their own walk leaves S 4e-4 off there (135 instead of 150 us at
// L = 2048, 96 heads, d = 128).
#include <atomic>
#include <cstdint>

#include "mc_internal.cuh"
#include "mma_sync.cuh"
#include "sm100.cuh"
#include "tensormap.cuh"

namespace mc {
namespace {

using namespace mma;
using namespace sm100;

__device__ int g_delta_abort;
std::atomic<int> g_give_up{0};  // waits to be taken for ones that gave up, in later launches

constexpr int kCH = kDeltaChunk;

// Lower-triangular B operands by 16 x 8 tiles: column tile nt (8 tokens) needs row tiles kt <= nt / 2.
constexpr int kTiles = 20;
__host__ __device__ constexpr int tile_base(int nt) { return nt / 2 * (nt / 2 + 1) + (nt & 1) * (nt / 2 + 1); }
static_assert(tile_base(7) + 4 == kTiles, "tiles of a lower triangle");

// A chunk's record (DeltaTcArgs::rec): T - 1 as {hi, lo} operand tiles; 256 floats: exp(c_i), beta_i exp(c_end - c_i),
// beta_i, and [192] exp(c_end); P as {hi, lo} tiles.
constexpr int kRecT = kTiles * 32 * 16, kRecV = 1024;
constexpr int kRec = kDeltaRecBytes;
static_assert(2 * kRecT + kRecV == kRec, "record");

// The other way round, rows m >= columns i: column tile nt needs row tiles kt = nt / 2 .. 3.
__host__ __device__ constexpr int rev_base(int nt) { return 8 * (nt / 2) - nt / 2 * (nt / 2 - 1) + (nt & 1) * (4 - nt / 2); }
static_assert(rev_base(7) + 1 == kTiles, "tiles of an upper triangle");
// The reverse walk's record: exp(c_i), exp(c_end - c_i), beta_i, [192] exp(c_end); T - 1 and P as {hi, lo} tiles.
static_assert(2 * kRecT + kRecV == kDeltaRRecBytes, "record");

struct Where {
    int bh, seg, ch, tb, cnt;
};
__device__ __forceinline__ Where chunk_at(const DeltaTcArgs &a, long long id)
{
    Where w;
    w.ch = (int)(id % a.NCH);
    const long long r = id / a.NCH;
    w.seg = (int)(r % a.N);
    w.bh = (int)(r / a.N);
    w.tb = w.seg * a.C + w.ch * kCH;
    w.cnt = min(min(w.tb + kCH, (w.seg + 1) * a.C), a.L) - w.tb;
    return w;
}

// Tiles of tokens come by TMA: 64 x 64 panels of q and k, and a walk's columns of v (or dy).
struct DeltaMaps {
    CUtensorMap k, q, v;
};
constexpr int kPanel = kCH * 128;
__device__ __forceinline__ uint32_t panel_off(int r, int c) { return (uint32_t)((c >> 3) * kPanel) + tile_off<128>(r, c & 7); }

// A kernel's CTAs may come up while the one before it, whose work they need, still runs its last ones: what a kernel reads
// or writes in global memory comes after after_previous().  let_next_start() stands at a kernel's end: called at its
// start the next one's CTAs crowd onto the SMs that are free by then (L = 4096, 32 heads: gradients 466 instead of 404 us).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename K, typename... A>
cudaError_t launch_early(K *kern, long long grid, int block, int smem, cudaStream_t s, const A &...args)
{
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// A bounded wait; `refused` says that the caller is to take it for one that gave up (mc_selftest_delta_give_up).
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort_flag, bool refused)
{
    return !refused && mbar_wait(bar, parity, abort_flag);
}
// A CTA that gives up: the thread that issued the copies waits (with a limit again) until those under way have landed, so
// that none writes shared memory that is another CTA's by then.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity)
{
    int gave_up = 0;
    mbar_wait_limit(bar, parity, &gave_up, kWaitLimitNs);
}

// What follows the tiles in shared memory: a barrier per stage, one for the single buffer, and whether a wait gave up.
struct WalkSync {
    uint64_t full[2], single;
    int abort_flag, pad;
};
__device__ __forceinline__ bool walk_sync_init(WalkSync *y, const void *sm, int tid)
{
    if (tid == 0) {
        y->abort_flag = (smem_addr(sm) & 1023) != 0;  // (the panels' swizzle counts from 1024-byte boundaries)
        mbar_init(&y->full[0], 1);
        mbar_init(&y->full[1], 1);
        mbar_init(&y->single, 1);
        fence_mbar_init();
    }
    __syncthreads();
    return y->abort_flag == 0;
}
// A walk that gives up after `stages` loads of stages (number j went to full[b(j)], its use j / 2 of that barrier) and
// `singles` of the single buffer: none was issued where walk_sync_init said no.
template <typename F>
__device__ __forceinline__ void walk_gives_up(WalkSync *y, const void *sm, int stages, int singles, F b)
{
    if ((smem_addr(sm) & 1023) == 0) {
        for (int j = max(stages - 2, 0); j < stages; ++j) wait_out(&y->full[b(j)], j / 2 & 1);
        if (singles > 0) wait_out(&y->single, (singles - 1) & 1);
    }
    atomicExch(&g_delta_abort, 1);
}
// Rows from cnt on of a tile of ROW bytes a row: a chunk's last tokens may be another segment's.
template <int ROW, int ROWS, int NT>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int cnt, int tid)
{
    for (int e = cnt * (ROW / 16) + tid; e < ROWS * (ROW / 16); e += NT) reinterpret_cast<uint4 *>(tile)[e] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// delta_prep_tc: one warp per chunk, no barrier between warps.  K K^T (and Q K^T) in registers, exact bf16
// products; then X = (1 + A)^-1 by 16 x 16 blocks: the four diagonal blocks by substitution in fp32, all at once (a lane
// per column, two blocks on each half of the warp), and the others from them as products of 16 x 16 blocks with every
// operand in three bf16 terms (2^-25):
//   X10 = -X11 A10 X00, X32 = -X33 A32 X22, and [X20 X21; X30 X31] = -[X22 0; X32 X33] [A20 A21; A30 A31] [X00 0; X10 X11].
// A product's result is a left operand as it lies, its 8 x 8 transposes are a right one, and a block of X (or P) is, as it
// lies, also the walk's operand of rows j, columns i: nothing but the diagonal blocks passes through shared memory.
// 16 heads of 65536 tokens, d = 128: 164 us for 0.89 GB of keys and queries read and records written, 5.4 TB/s (without P
// 102 us; substitution over all 64 rows, two columns a lane: 156); with P and the reverse record 62 us for 4096 chunks,
// 5.0 TB/s, without P 34 us for 2048 chunks, where a chunk's own chain of small products, 8 us, is what a warp waits for.
// ---------------------------------------------------------------------------
constexpr int kXP = 20, kXB = 16 * kXP + 8;  // row and block pitch of the diagonal blocks, in words

struct Terms {  // an operand in three bf16 terms: left 4 registers each, right 2 x 2
    uint32_t h[4], m[4], l[4];
};
// 16 x 16 results: [column half][accumulator]
__device__ __forceinline__ Terms left_of(const float (&x)[2][4])
{
    Terms t;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) split3(x[h][2 * r], x[h][2 * r + 1], t.h[2 * h + r], t.m[2 * h + r], t.l[2 * h + r]);
    return t;
}
__device__ __forceinline__ Terms right_of(const Terms &left)
{
    Terms t;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        t.h[q] = movm_t(left.h[q]);
        t.m[q] = movm_t(left.m[q]);
        t.l[q] = movm_t(left.l[q]);
    }
    return t;
}
// acc += left x right
__device__ __forceinline__ void block_mma(float (&acc)[2][4], const Terms &a, const Terms &b)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        mma16816(acc[h], a.l, b.h[2 * h], b.h[2 * h + 1]);
        mma16816(acc[h], a.h, b.l[2 * h], b.l[2 * h + 1]);
        mma16816(acc[h], a.m, b.m[2 * h], b.m[2 * h + 1]);
        mma16816(acc[h], a.m, b.h[2 * h], b.h[2 * h + 1]);
        mma16816(acc[h], a.h, b.m[2 * h], b.m[2 * h + 1]);
        mma16816(acc[h], a.h, b.h[2 * h], b.h[2 * h + 1]);
    }
}

template <int D, bool QK>
__host__ __device__ constexpr int prep_smem()
{
    constexpr int tiles = (kCH + (QK ? 32 : 0)) * D * 2;
    return (tiles > 8 * kXB * 4 ? tiles : 8 * kXB * 4) + 3 * kCH * 4 + (int)sizeof(WalkSync);
}

template <int D, bool READ, bool REV>
__global__ void __launch_bounds__(32) delta_prep_tc(DeltaTcArgs a, const __grid_constant__ DeltaMaps maps)
{
    constexpr int KS = D / 16;
    constexpr bool QK = READ || REV;
    extern __shared__ __align__(1024) uint8_t sm[];
    float *Ad = reinterpret_cast<float *>(sm), *Xd = Ad + 4 * kXB;  // over the tiles once these are read
    WalkSync *sync = reinterpret_cast<WalkSync *>(sm + prep_smem<D, QK>() - sizeof(WalkSync));
    float *bet = reinterpret_cast<float *>(sync) - kCH, *cum = bet - kCH, *cul = cum - kCH;
    const Where w = chunk_at(a, blockIdx.x);
    if (w.cnt <= 0) return;
    const int lane = threadIdx.x, g = lane / 4, c = lane % 4;
    const size_t row0 = (size_t)w.bh * a.L + w.tb;
    // K, and 16 rows of Q at a time in two buffers: with all of Q an SM would hold six chunks, not eight
    constexpr int QB = 16 * D * 2;
    uint8_t *Qs = sm + kCH * D * 2;
    const uint32_t Kt = smem_addr(sm);
    const bool refused = a.give_up & kGiveUpTiles;
    int under_way = 0;  // (lane 0) K and how many blocks of Q
    auto load_q = [&](int b) {
        ++under_way;
        mbar_arrive_expect_tx(&sync->full[b & 1], QB);
#pragma unroll
        for (int p = 0; p < D / 64; ++p)
            tma_load_3d(Qs + (b & 1) * QB + p * 2048, &maps.q, 64 * p, w.tb + 16 * b, w.bh, &sync->full[b & 1]);
    };
    bool ok = walk_sync_init(sync, sm, lane);
    auto give_up = [&]() {
        if (lane != 0) return;
        if (under_way > 0) wait_out(&sync->single, 0);
        for (int b = max(under_way - 3, 0); b < under_way - 1; ++b) wait_out(&sync->full[b & 1], b / 2);
        atomicExch(&g_delta_abort, 1);
    };
    if (ok && lane == 0) {
        under_way = 1;
        mbar_arrive_expect_tx(&sync->single, kCH * D * 2);
#pragma unroll
        for (int p = 0; p < D / 64; ++p) tma_load_3d(sm + p * kPanel, &maps.k, 64 * p, w.tb, w.bh, &sync->single);
        if (QK) {
            load_q(0);
            load_q(1);
        }
    }
    __syncwarp();
    {  // running sums of the chunk's decays as cum + cul (delta_parts), two tokens per lane
        const int i = 2 * lane;
        const float2 x0 = delta_parts(i < w.cnt ? delta_log(__bfloat162float(a.la[row0 + i])) : 0.f);
        const float2 x1 = delta_parts(i + 1 < w.cnt ? delta_log(__bfloat162float(a.la[row0 + i + 1])) : 0.f);
        float s = x0.x + x1.x, r = x0.y + x1.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float n = __shfl_up_sync(0xffffffffu, s, o), m = __shfl_up_sync(0xffffffffu, r, o);
            if (lane >= o) {
                s += n;
                r += m;
            }
        }
        cum[i] = s - x1.x;
        cum[i + 1] = s;
        cul[i] = r - x1.y;
        cul[i + 1] = r;
        bet[i] = i < w.cnt ? __bfloat162float(a.be[row0 + i]) : 0.f;
        bet[i + 1] = i + 1 < w.cnt ? __bfloat162float(a.be[row0 + i + 1]) : 0.f;
    }
    if (ok) ok = wait_for(&sync->single, 0, &sync->abort_flag, refused);
    if (__any_sync(0xffffffffu, !ok)) {
        give_up();
        return;
    }
    if (w.cnt < kCH)
#pragma unroll
        for (int p = 0; p < D / 64; ++p) clear_rows<128, kCH, 32>(sm + p * kPanel, w.cnt, lane);
    __syncwarp();
    uint8_t *rec = a.rec + (size_t)blockIdx.x * kRec, *rrec = REV ? a.rrec + (size_t)blockIdx.x * kDeltaRRecBytes : nullptr;
    const float ce = cum[kCH - 1], cel = cul[kCH - 1];  // tokens past the end add nothing
    {
        float *vec = reinterpret_cast<float *>(rec + kRecT);
        float *rvec = reinterpret_cast<float *>(rrec);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            const float ea = __expf(cum[i] + cul[i]), eb = __expf((ce - cum[i]) + (cel - cul[i]));
            vec[i] = ea;
            vec[64 + i] = bet[i] * eb;
            vec[128 + i] = bet[i];
            if (REV) {
                rvec[i] = ea;
                rvec[64 + i] = eb;
                rvec[128 + i] = bet[i];
            }
        }
        if (lane == 0) {
            vec[192] = __expf(ce + cel);
            if (REV) rvec[192] = __expf(ce + cel);
        }
    }
    const int ar = lane & 15, ac = lane >> 4, br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;
    float kk[10][2][4];  // 16 x 16 blocks (b, n2 <= b) of K K^T
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint8_t *Qb = Qs + (b & 1) * QB;
        if (QK) {
            if (ok) ok = wait_for(&sync->full[b & 1], b / 2, &sync->abort_flag, refused);
            if (__any_sync(0xffffffffu, !ok)) {
                give_up();
                return;
            }
            if (w.cnt < 16 * b + 16)
#pragma unroll
                for (int p = 0; p < D / 64; ++p) clear_rows<128, 16, 32>(Qb + p * 2048, max(w.cnt - 16 * b, 0), lane);
            __syncwarp();
        }
        float qk[4][2][4];
#pragma unroll
        for (int n2 = 0; n2 <= b; ++n2)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) kk[b * (b + 1) / 2 + n2][h][e] = qk[n2][h][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t ak[4], aq[4];
            ldsm4(ak, Kt + panel_off(16 * b + ar, 2 * ks + ac));
            if (QK) ldsm4(aq, smem_addr(Qb) + (2 * ks + ac) / 8 * 2048 + tile_off<128>(ar, (2 * ks + ac) & 7));
#pragma unroll
            for (int n2 = 0; n2 <= b; ++n2) {
                uint32_t bf[4];
                ldsm4(bf, Kt + panel_off(16 * n2 + br, 2 * ks + bc));
                mma16816(kk[b * (b + 1) / 2 + n2][0], ak, bf[0], bf[1]);
                mma16816(kk[b * (b + 1) / 2 + n2][1], ak, bf[2], bf[3]);
                if (QK) {
                    mma16816(qk[n2][0], aq, bf[0], bf[1]);
                    mma16816(qk[n2][1], aq, bf[2], bf[3]);
                }
            }
        }
        if (QK && b < 2) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) load_q(b + 2);
        }
        const float c0 = cum[16 * b + g], c1 = cum[16 * b + g + 8], r0 = cul[16 * b + g], r1 = cul[16 * b + g + 8];
#pragma unroll
        for (int n2 = 0; n2 <= b; ++n2) {
            uint32_t p[2][2], pl[2][2];  // [columns half][rows half] 8 x 8 tiles of P, two terms
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 cj = *reinterpret_cast<const float2 *>(cum + 16 * n2 + 8 * h + 2 * c);
                const float2 rj = *reinterpret_cast<const float2 *>(cul + 16 * n2 + 8 * h + 2 * c);
                const float2 bj = *reinterpret_cast<const float2 *>(bet + 16 * n2 + 8 * h + 2 * c);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int il = g + 8 * (e >> 1), jl = 8 * h + 2 * c + (e & 1);
                    const float dec = __expf(((e >> 1 ? c1 : c0) - (e & 1 ? cj.y : cj.x)) + ((e >> 1 ? r1 : r0) - (e & 1 ? rj.y : rj.x)));
                    float &x = kk[b * (b + 1) / 2 + n2][h][e];
                    x = n2 < b || jl < il ? x * (dec * (e & 1 ? bj.y : bj.x)) : 0.f;  // A
                    v[e] = n2 < b || jl <= il ? qk[n2][h][e] * dec : 0.f;
                }
                if (QK) {
                    split2(v[0], v[1], p[h][0], pl[h][0]);
                    split2(v[2], v[3], p[h][1], pl[h][1]);
                }
            }
            if (READ) {
                uint4 *pt = reinterpret_cast<uint4 *>(rec + kRecT + kRecV) + lane;
                pt[(tile_base(2 * b) + n2) * 32] = make_uint4(p[0][0], p[1][0], pl[0][0], pl[1][0]);
                pt[(tile_base(2 * b + 1) + n2) * 32] = make_uint4(p[0][1], p[1][1], pl[0][1], pl[1][1]);
            }
            if (REV) {
                uint4 *pt = reinterpret_cast<uint4 *>(rrec + kRecV + kRecT) + lane;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    pt[(rev_base(2 * n2 + h) + b - n2) * 32] =
                        make_uint4(movm_t(p[h][0]), movm_t(p[h][1]), movm_t(pl[h][0]), movm_t(pl[h][1]));
            }
        }
    }
    __syncwarp();  // the tiles have been read
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)  // the diagonal blocks of A: column j as a row
                Ad[b * kXB + (8 * h + 2 * c + (e & 1)) * kXP + g + 8 * (e >> 1)] = kk[b * (b + 3) / 2][h][e];
    __syncwarp();
    {
        const int hw = lane / 16, col = lane % 16;
        float x[2][16];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[s][r] = r == col ? 1.f : 0.f;
#pragma unroll
        for (int k = 0; k < 15; ++k)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r4 = (k + 1) / 4; r4 < 4; ++r4) {
                    const float4 av = *reinterpret_cast<const float4 *>(Ad + (2 * s + hw) * kXB + k * kXP + 4 * r4);
                    const float al[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (4 * r4 + q > k) x[s][4 * r4 + q] = fmaf(-al[q], x[s][k], x[s][4 * r4 + q]);
                }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 16; ++r) Xd[(2 * s + hw) * kXB + r * kXP + col] = x[s][r];
    }
    __syncwarp();
    auto diag = [&](int b, float (&x)[2][4]) {  // a diagonal block as a result
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 v = *reinterpret_cast<const float2 *>(Xd + b * kXB + (g + 8 * r) * kXP + 8 * h + 2 * c);
                x[h][2 * r] = v.x;
                x[h][2 * r + 1] = v.y;
            }
    };
    auto out = [&](int bi, int bj, const Terms &t) {  // block (bi, bj) of T - 1
        uint4 *tt = reinterpret_cast<uint4 *>(rec) + lane;
#pragma unroll
        for (int r = 0; r < 2; ++r) tt[(tile_base(2 * bi + r) + bj) * 32] = make_uint4(t.h[r], t.h[2 + r], t.m[r], t.m[2 + r]);
        if (REV) {
            uint4 *lt = reinterpret_cast<uint4 *>(rrec + kRecV) + lane;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                lt[(rev_base(2 * bj + h) + bi - bj) * 32] =
                    make_uint4(movm_t(t.h[2 * h]), movm_t(t.h[2 * h + 1]), movm_t(t.m[2 * h]), movm_t(t.m[2 * h + 1]));
        }
    };
    auto negate = [](float (&x)[2][4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[h][e] = -x[h][e];
    };
    auto clear = [](float (&x)[2][4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[h][e] = 0.f;
    };
    Terms D0, D1, D2, D3;
    {
        float x[2][4];
        Terms *const to[4] = {&D0, &D1, &D2, &D3};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            diag(b, x);
            *to[b] = left_of(x);
#pragma unroll
            for (int h = 0; h < 2; ++h)  // T - 1: the diagonal out
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (8 * h + 2 * c + (e & 1) >= g + 8 * (e >> 1)) x[h][e] = 0.f;
            out(b, b, left_of(x));
        }
    }
    // A_bn is kk[b (b + 1) / 2 + n]
    Terms X10r, X32l;
    {
        float y[2][4], x[2][4];
        clear(y);
        block_mma(y, left_of(kk[1]), right_of(D0));
        clear(x);
        block_mma(x, D1, right_of(left_of(y)));
        negate(x);
        const Terms t = left_of(x);
        out(1, 0, t);
        X10r = right_of(t);
        clear(y);
        block_mma(y, left_of(kk[8]), right_of(D2));
        clear(x);
        block_mma(x, D3, right_of(left_of(y)));
        negate(x);
        X32l = left_of(x);
        out(3, 2, X32l);
    }
    const Terms D0r = right_of(D0), D1r = right_of(D1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // block columns 0 and 1
        float y2[2][4], y3[2][4], x[2][4];
        clear(y2);
        clear(y3);
        if (j == 0) {
            block_mma(y2, left_of(kk[3]), D0r);
            block_mma(y3, left_of(kk[6]), D0r);
            block_mma(y2, left_of(kk[4]), X10r);
            block_mma(y3, left_of(kk[7]), X10r);
        } else {
            block_mma(y2, left_of(kk[4]), D1r);
            block_mma(y3, left_of(kk[7]), D1r);
        }
        const Terms y2r = right_of(left_of(y2)), y3r = right_of(left_of(y3));
        clear(x);
        block_mma(x, D2, y2r);
        negate(x);
        out(2, j, left_of(x));
        clear(x);
        block_mma(x, X32l, y2r);
        block_mma(x, D3, y3r);
        negate(x);
        out(3, j, left_of(x));
    }
    let_next_start();
}

// A warp's own 32 bytes of every row of the V (or dy) tile: once read, its staging area for what it writes.
template <int NW>
__device__ __forceinline__ uint32_t own_off(int r, int pc, int warp)
{
    // 16-byte pieces of a row, exchanged as the copies of 64-byte and of 128-byte rows leave them
    return (uint32_t)(r * NW * 32 + (((2 * warp + pc) ^ (NW == 4 ? r & 7 : r >> 1 & 3)) << 4));
}

// 16 values x 64 tokens in operand registers to rows of 16 values.  Where two warps hold the same values (KP = 2), each
// writes half of the tokens.
template <int NW, int KP, int D>
__device__ __forceinline__ void put_tokens(__nv_bfloat16 *dst, const uint32_t (&f)[4][4], uint8_t *vt, int cnt, int wr, int kp, int lane)
{
    const uint32_t at = smem_addr(vt);
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4)
        if (KP == 1 || k4 / 2 == kp)
            stsm4t(at + own_off<NW>(16 * k4 + (lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1, wr), f[k4][0], f[k4][1], f[k4][2], f[k4][3]);
    __syncwarp();
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int r = 16 * x + lane / 2, pc = lane % 2;
        if ((KP == 1 || x / 2 == kp) && r < cnt)
            *reinterpret_cast<uint4 *>(dst + (size_t)r * D + 8 * pc) = *reinterpret_cast<const uint4 *>(vt + own_off<NW>(r, pc, wr));
    }
    __syncwarp();
}

// f times a warp's 16 rows in bf16: neighbouring lanes exchange halves of two tiles, so that a row's four lanes hold 32
// bytes in a run.  `put` takes (row, tile of 8 columns, byte within the tile's 16, 8 bytes).
template <int NT, typename F>
__device__ __forceinline__ void put_rows(const float (&S)[NT][4], float f, int lane, F put)
{
    const int g = lane / 4, c = lane % 4;
#pragma unroll
    for (int n = 0; n < NT; n += 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t p0 = pack2(f * S[n][2 * h], f * S[n][2 * h + 1]), p1 = pack2(f * S[n + 1][2 * h], f * S[n + 1][2 * h + 1]);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, c & 1 ? p0 : p1, 1);
            put(g + 8 * h, n + (c & 1), 8 * (c >> 1), c & 1 ? make_uint2(got, p1) : make_uint2(p0, got));
        }
}

// Two warps that hold the two halves of the keys of 16 rows add their partial products: each leaves its own in xb,
// and adds the other's (tiles with `mine` only).
template <int TILES, typename F, typename G>
__device__ __forceinline__ void pair_sum(float4 *xb, int warp, int lane, F each, G add)
{
    each([&](int i, const float (&x)[4]) { xb[(warp * TILES + i) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]); });
    asm volatile("bar.sync %0, 64;" ::"r"(1 + warp / 2) : "memory");
    add([&](int i, float (&x)[4]) {
        const float4 y = xb[((warp ^ 1) * TILES + i) * 32 + lane];
        x[0] += y.x;
        x[1] += y.y;
        x[2] += y.z;
        x[3] += y.w;
    });
}

// ---------------------------------------------------------------------------
// delta_walk_tc: one CTA per (bh, segment, 16 NW value rows); NW warps of 16 rows.  Two stages of
// the chunk's K, V columns, (Q,) and record, filled by TMA one chunk ahead: copied by the threads, 16 bytes at a
// time, they took a fifth of the time (shared memory's pipe is what the products wait for, too).  16 heads of 65536
// tokens, segments of 1024, d = 128: 571 us, 413 TFLOP/s of warp-level products against 600 that these reach when nothing
// else is done (420 us without the online reads, which the readout would then form in one term).  One memory of 4096
// tokens, 32 heads (recomputed, one term, e in two for the gradients): 126 us, 2.0 us for a chunk, half of which are one warp's own products one after
// the other.
// ---------------------------------------------------------------------------
template <int D, int NW, int KP, bool READ>
struct WalkSmem {
    static constexpr int kK = kCH * D * 2, kV = kCH * NW * 32;
    static constexpr bool kLate = READ && KP == 1;  // P is needed late in a chunk: one buffer, where two CTAs share an SM
    static constexpr int kR = kRecT + kRecV + (READ && !kLate ? kRecT : 0);
    static constexpr int kStage = kK * (READ ? 2 : 1) + kV + kR;
    static constexpr int kP = kLate ? kRecT : 0;
    static constexpr int kTotal = 2 * kStage + kP;
};

template <int D, int NW, int KP, bool READ, bool FULL>
__global__ void __launch_bounds__(32 * NW * KP, KP == 1 ? 2 : 1) delta_walk_tc(DeltaTcArgs a, const __grid_constant__ DeltaMaps maps)
{
    using W = WalkSmem<D, NW, KP, READ>;
    constexpr int NT = 32 * NW * KP, KS = D / 16 / KP;
    extern __shared__ __align__(1024) uint8_t sm[];
    WalkSync *sync = reinterpret_cast<WalkSync *>(sm + W::kTotal);
    constexpr int splits = D / (16 * NW);
    const int rs = (int)blockIdx.x % splits;
    const long long sid = blockIdx.x / splits;
    const int seg = (int)(sid % a.N), bh = (int)(sid / a.N);
    const int t0 = seg * a.C, len = min((seg + 1) * a.C, a.L) - t0, nch = (len + kCH - 1) / kCH;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int vbase = rs * 16 * NW;  // the CTA's first value row
    const int wr = warp / KP, kp = KP == 1 ? 0 : warp % KP, k0 = kp * KS;  // the warp's rows, its share of the keys

    auto load = [&](int ch) {  // one thread
        uint8_t *st = sm + (ch & 1) * W::kStage;
        uint64_t *bar = &sync->full[ch & 1];
        mbar_arrive_expect_tx(bar, W::kStage);
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
            tma_load_3d(st + p * kPanel, &maps.k, 64 * p, t0 + ch * kCH, bh, bar);
            if (READ) tma_load_3d(st + W::kK + W::kV + p * kPanel, &maps.q, 64 * p, t0 + ch * kCH, bh, bar);
        }
        tma_load_3d(st + W::kK, &maps.v, vbase, t0 + ch * kCH, bh, bar);
        bulk_load(st + W::kStage - W::kR, a.rec + ((size_t)sid * a.NCH + ch) * kRec, W::kR, bar);
    };
    bool ok = walk_sync_init(sync, sm, tid);
    auto give_up = [&](int stages, int singles) {
        if (tid == 0) walk_gives_up(sync, sm, stages, W::kLate ? singles : 0, [](int j) { return j & 1; });
    };

    float S[2 * KS][4];  // 16 rows x D / KP keys: tile n holds keys 16 k0 + 8 n ..
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = 0.f;

    after_previous();
    if (ok && tid == 0) load(0);
    for (int ch = 0; ch < nch; ++ch) {
        if (ok) ok = wait_for(&sync->full[ch & 1], ch / 2 & 1, &sync->abort_flag, a.give_up & kGiveUpTiles);
        fence_async_smem();  // what was staged in the other stage goes before what will come there
        if (__syncthreads_or(!ok)) {
            give_up(ch + 1, ch);
            return;
        }
        if (tid == 0) {
            if (W::kLate) {
                mbar_arrive_expect_tx(&sync->single, kRecT);
                bulk_load(sm + 2 * W::kStage, a.rec + ((size_t)sid * a.NCH + ch) * kRec + kRecT + kRecV, kRecT, &sync->single);
            }
            if (ch + 1 < nch) load(ch + 1);
        }
        __syncwarp();
        uint8_t *st = sm + (ch & 1) * W::kStage, *vown = st + W::kK;
        const uint32_t kt = smem_addr(st), vt = kt + W::kK, qt = vt + W::kV;
        const uint8_t *rec = st + W::kStage - W::kR;
        const float *vec = reinterpret_cast<const float *>(rec + kRecT);
        const size_t row0 = (size_t)bh * a.L + t0 + ch * kCH;
        const int cnt = min(kCH, len - ch * kCH);
        const size_t cidx = (size_t)sid * a.NCH + ch;
        if (cnt < kCH) {
#pragma unroll
            for (int p = 0; p < D / 64; ++p) {
                clear_rows<128, kCH, NT>(st + p * kPanel, cnt, tid);
                if (READ) clear_rows<128, kCH, NT>(st + W::kK + W::kV + p * kPanel, cnt, tid);
            }
            clear_rows<NW * 32, kCH, NT>(vown, cnt, tid);
            __syncthreads();
        }

        // (S K^T) and (S Q^T): rows values, columns tokens
        float X[8][4], O[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[n][e] = O[n][e] = 0.f;
        const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t hi[4], lo[4];
            split2(S[2 * ks][0], S[2 * ks][1], hi[0], lo[0]);
            split2(S[2 * ks][2], S[2 * ks][3], hi[1], lo[1]);
            split2(S[2 * ks + 1][0], S[2 * ks + 1][1], hi[2], lo[2]);
            split2(S[2 * ks + 1][2], S[2 * ks + 1][3], hi[3], lo[3]);
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                uint32_t b[4];
                ldsm4(b, kt + panel_off(16 * n2 + br, 2 * (k0 + ks) + bc));
                mma16816(X[2 * n2], hi, b[0], b[1]);
                mma16816(X[2 * n2 + 1], hi, b[2], b[3]);
                if (FULL) {
                    mma16816(X[2 * n2], lo, b[0], b[1]);
                    mma16816(X[2 * n2 + 1], lo, b[2], b[3]);
                }
                if (READ) {  // the output is bf16 and nothing cancels here: one term
                    ldsm4(b, qt + panel_off(16 * n2 + br, 2 * (k0 + ks) + bc));
                    mma16816(O[2 * n2], hi, b[0], b[1]);
                    mma16816(O[2 * n2 + 1], hi, b[2], b[3]);
                }
            }
        }
        uint32_t v4[4][4];
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
            ldsm4t(v4[k4], vt + own_off<NW>(16 * k4 + (lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1, wr));
        if (KP == 2)
            pair_sum<READ ? 12 : 8>(reinterpret_cast<float4 *>(sm + W::kTotal + sizeof(WalkSync)), warp, lane,
                     [&](auto leave) {
#pragma unroll
                         for (int n = 0; n < 8; ++n) {
                             leave(n, X[n]);
                             if (READ && n / 4 != kp) leave(8 + n % 4, O[n]);
                         }
                     },
                     [&](auto add) {
#pragma unroll
                         for (int n = 0; n < 8; ++n) {
                             add(n, X[n]);
                             if (READ && n / 4 == kp) add(8 + n % 4, O[n]);
                         }
                     });
        else __syncwarp();  // the warp's part of V is free
        // R = V - diag(exp c) K S^T, then E = R + (T - 1) R
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const uint32_t lo2 = v4[n / 2][2 * (n & 1)], hi2 = v4[n / 2][2 * (n & 1) + 1];
            const float2 ga = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * c);
            X[n][0] = low_f(lo2) - ga.x * X[n][0];
            X[n][1] = high_f(lo2) - ga.y * X[n][1];
            X[n][2] = low_f(hi2) - ga.x * X[n][2];
            X[n][3] = high_f(hi2) - ga.y * X[n][3];
            if (READ) {
                O[n][0] *= ga.x;
                O[n][1] *= ga.y;
                O[n][2] *= ga.x;
                O[n][3] *= ga.y;
            }
        }
        if (a.S_c) {  // the memory before the chunk
            __nv_bfloat16 *dst = a.S_c + (cidx * D + vbase + 16 * wr) * D + 16 * k0;
            put_rows(S, 1.f, lane, [&](int r, int n, int at, const uint2 &x) { *reinterpret_cast<uint2 *>(dst + (size_t)r * D + 8 * n + at / 2) = x; });
        }
        {
            uint32_t rh[4][4], rl[4][4];
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
                split2(X[2 * k4][0], X[2 * k4][1], rh[k4][0], rl[k4][0]);
                split2(X[2 * k4][2], X[2 * k4][3], rh[k4][1], rl[k4][1]);
                split2(X[2 * k4 + 1][0], X[2 * k4 + 1][1], rh[k4][2], rl[k4][2]);
                split2(X[2 * k4 + 1][2], X[2 * k4 + 1][3], rh[k4][3], rl[k4][3]);
            }
            const uint4 *tt = reinterpret_cast<const uint4 *>(rec) + lane;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
                for (int n = 2 * k4; n < 8; ++n) {
                    const uint4 b = tt[(tile_base(n) + k4) * 32];
                    mma16816(X[n], rh[k4], b.x, b.y);
                    mma16816(X[n], rl[k4], b.x, b.y);
                    mma16816(X[n], rh[k4], b.z, b.w);
                }
        }
        // U = diag(beta) E for the read; U' = diag(beta exp(c_end - c)) E for the memory
        const float dec = vec[192];
        uint32_t uh[4][4], ul[4][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 be = *reinterpret_cast<const float2 *>(vec + 128 + 8 * n + 2 * c);
            split2(be.x * X[n][0], be.y * X[n][1], uh[n / 2][2 * (n & 1)], ul[n / 2][2 * (n & 1)]);
            split2(be.x * X[n][2], be.y * X[n][3], uh[n / 2][2 * (n & 1) + 1], ul[n / 2][2 * (n & 1) + 1]);
        }
        if (READ) {
            if (W::kLate) {
                if (ok) ok = wait_for(&sync->single, ch & 1, &sync->abort_flag, a.give_up & kGiveUpLate);
                __syncwarp();
            }
            const uint4 *pt = reinterpret_cast<const uint4 *>(W::kLate ? sm + 2 * W::kStage : rec + kRecT + kRecV) + lane;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
                for (int n = 2 * k4; n < 8; ++n) {
                    if (KP == 2 && n / 4 != kp) continue;
                    const uint4 b = pt[(tile_base(n) + k4) * 32];
                    mma16816(O[n], ul[k4], b.x, b.y);
                    mma16816(O[n], uh[k4], b.z, b.w);
                    mma16816(O[n], uh[k4], b.x, b.y);
                }
        }
        auto put = [&](__nv_bfloat16 *dst, const uint32_t (&f)[4][4]) {
            put_tokens<NW, KP, D>(dst + row0 * D + vbase + 16 * wr, f, vown, cnt, wr, kp, lane);
        };
        if (READ) {
            uint32_t of[4][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                of[n / 2][2 * (n & 1)] = pack2(O[n][0], O[n][1]);
                of[n / 2][2 * (n & 1) + 1] = pack2(O[n][2], O[n][3]);
            }
            if (a.y) put(a.y, of);
            if (a.O_on) {
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 8 * n + 2 * c + (e & 1), r = vbase + 16 * wr + g + 8 * (e >> 1);
                        if ((KP == 1 || n / 4 == kp) && t < cnt) a.O_on[(row0 + t) * D + r] = O[n][e];
                    }
            }
        }
        if (a.E) {
            uint32_t eh[4][4], el[4][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                split2(X[n][0], X[n][1], eh[n / 2][2 * (n & 1)], el[n / 2][2 * (n & 1)]);
                split2(X[n][2], X[n][3], eh[n / 2][2 * (n & 1) + 1], el[n / 2][2 * (n & 1) + 1]);
            }
            put(a.E, eh);
            put(a.E_lo, el);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 w = *reinterpret_cast<const float2 *>(vec + 64 + 8 * n + 2 * c);
            split2(w.x * X[n][0], w.y * X[n][1], uh[n / 2][2 * (n & 1)], ul[n / 2][2 * (n & 1)]);
            split2(w.x * X[n][2], w.y * X[n][3], uh[n / 2][2 * (n & 1) + 1], ul[n / 2][2 * (n & 1) + 1]);
        }
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[n][e] *= dec;
        const int tr = ((lane >> 3) & 1) * 8 + (lane & 7), tc = lane >> 4;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
            for (int n2 = 0; n2 < KS; ++n2) {
                uint32_t b[4];
                ldsm4t(b, kt + panel_off(16 * k4 + tr, 2 * (k0 + n2) + tc));
                mma16816(S[2 * n2], uh[k4], b[0], b[1]);
                mma16816(S[2 * n2 + 1], uh[k4], b[2], b[3]);
                mma16816(S[2 * n2], ul[k4], b[0], b[1]);
                mma16816(S[2 * n2 + 1], ul[k4], b[2], b[3]);
            }
    }
    if (W::kLate && __syncthreads_or(!ok)) {  // the last chunk's wait
        give_up(nch, nch);
        return;
    }
    let_next_start();
    if (a.states_img) {
        uint8_t *img = a.states_img + (size_t)sid * (D * D * 2) + (vbase + 16 * wr) * 128;
        put_rows(S, 1.f, lane, [&](int r, int n, int at, const uint2 &x) {
            *reinterpret_cast<uint2 *>(img + (2 * k0 + n) / 8 * (D * 128) + tile_off<128>(r, (2 * k0 + n) % 8) + at) = x;
        });
    }
    if (a.states) {
        float *dst = a.states + ((size_t)sid * D + vbase + 16 * wr) * D + 16 * k0;
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
            *reinterpret_cast<float2 *>(dst + (size_t)g * D + 8 * n + 2 * c) = make_float2(S[n][0], S[n][1]);
            *reinterpret_cast<float2 *>(dst + (size_t)(g + 8) * D + 8 * n + 2 * c) = make_float2(S[n][2], S[n][3]);
        }
    }
}

// ---------------------------------------------------------------------------
// delta_rwalk_tc: the walk backwards over the adjoint, with the layout of delta_walk_tc.  Per chunk,
// with p_i = g_i dy_i and R the adjoint after the chunk:
//   X   = diag(exp(c_end - c)) K R^T + P^T p,   W = T^T diag(beta) X            (dv = W)
//   R' = exp(c_end) R + sum_i exp(c_i) (p_i q_i^T - w_i k_i^T)
// R is held in fp32 and read in two bf16 terms, as T, P, X and w are: for keys that resemble each other X gathers what later
// tokens ask of every one of them, and w is the small difference that is left (all in one term: dv 3e-2 off at all but
// parallel keys; R alone: dv and dbeta 1.2e-2).  p is rounded once.  One memory of 4096 tokens, 32 heads, d = 128: 155 us,
// 2.4 us for a chunk, its chain as in delta_walk_tc; 16 heads of 16384, segments of 1024: 199 us.
// ---------------------------------------------------------------------------
template <int D, int NW, int KP>
struct RWalkSmem {
    static constexpr int kK = kCH * D * 2, kV = kCH * NW * 32;
    static constexpr bool kLate = KP == 1;  // T and P are needed late in a chunk, as P above
    static constexpr int kR = kRecV + (kLate ? 0 : 2 * kRecT);
    static constexpr int kStage = 2 * kK + kV + kR;  // K, Q, dy columns, record
    static constexpr int kGates = 2 * kStage + (kLate ? 2 * kRecT : 0);
    static constexpr int kTotal = kGates + 2 * kCH * 4;  // two chunks' gates
};

template <int D, int NW, int KP>
__global__ void __launch_bounds__(32 * NW * KP, KP == 1 ? 2 : 1) delta_rwalk_tc(DeltaTcArgs a, const __grid_constant__ DeltaMaps maps)
{
    using W = RWalkSmem<D, NW, KP>;
    constexpr int NT = 32 * NW * KP, KS = D / 16 / KP;
    extern __shared__ __align__(1024) uint8_t sm[];
    WalkSync *sync = reinterpret_cast<WalkSync *>(sm + W::kTotal);
    float *gates = reinterpret_cast<float *>(sm + W::kGates);
    constexpr int splits = D / (16 * NW);
    const int rs = (int)blockIdx.x % splits;
    const long long sid = blockIdx.x / splits;
    const int seg = (int)(sid % a.N), bh = (int)(sid / a.N);
    const int t0 = seg * a.C, len = min((seg + 1) * a.C, a.L) - t0, nch = (len + kCH - 1) / kCH;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int vbase = rs * 16 * NW;
    const int wr = warp / KP, kp = KP == 1 ? 0 : warp % KP, k0 = kp * KS;

    auto load = [&](int ch) {  // one thread
        uint8_t *st = sm + (ch & 1) * W::kStage;
        uint64_t *bar = &sync->full[ch & 1];
        mbar_arrive_expect_tx(bar, W::kStage);
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
            tma_load_3d(st + p * kPanel, &maps.k, 64 * p, t0 + ch * kCH, bh, bar);
            tma_load_3d(st + W::kK + p * kPanel, &maps.q, 64 * p, t0 + ch * kCH, bh, bar);
        }
        tma_load_3d(st + 2 * W::kK, &maps.v, vbase, t0 + ch * kCH, bh, bar);
        bulk_load(st + 2 * W::kK + W::kV, a.rrec + ((size_t)sid * a.NCH + ch) * kDeltaRRecBytes, W::kR, bar);
    };
    auto gate = [&](int ch) {
        return a.gon && ch * kCH + tid < len ? a.gon[((size_t)bh * a.L + t0 + ch * kCH + tid) * a.gw_stride] : 1.f;
    };
    bool ok = walk_sync_init(sync, sm, tid);
    auto give_up = [&](int stages, int singles) {
        if (tid == 0) walk_gives_up(sync, sm, stages, W::kLate ? singles : 0, [&](int j) { return (nch - 1 - j) & 1; });
    };
    after_previous();
    if (ok && tid == 0) load(nch - 1);
    __syncwarp();
    if (tid < kCH) gates[(nch - 1 & 1) * kCH + tid] = gate(nch - 1);

    float R[2 * KS][4];
    if (a.G && seg < a.N - 1) {  // partial sums, in order
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) R[n][0] = R[n][1] = R[n][2] = R[n][3] = 0.f;
        for (int part = 0; part < a.g_parts; ++part) {
            const float *src = a.G + (((size_t)part * a.BH * a.N + sid) * D + vbase + 16 * wr) * D + 16 * k0;
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n) {
                const float2 x = *reinterpret_cast<const float2 *>(src + (size_t)g * D + 8 * n + 2 * c);
                const float2 y = *reinterpret_cast<const float2 *>(src + (size_t)(g + 8) * D + 8 * n + 2 * c);
                R[n][0] += x.x; R[n][1] += x.y; R[n][2] += y.x; R[n][3] += y.y;
            }
        }
    } else {
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) R[n][e] = 0.f;
    }

    for (int ch = nch - 1; ch >= 0; --ch) {
        const int turn = nch - 1 - ch;
        if (ok) ok = wait_for(&sync->full[ch & 1], turn / 2 & 1, &sync->abort_flag, a.give_up & kGiveUpTiles);
        fence_async_smem();  // what was staged in the other stage goes before what will come there
        if (__syncthreads_or(!ok)) {
            give_up(turn + 1, turn);
            return;
        }
        if (tid == 0) {
            if (W::kLate) {
                mbar_arrive_expect_tx(&sync->single, 2 * kRecT);
                bulk_load(sm + 2 * W::kStage, a.rrec + ((size_t)sid * a.NCH + ch) * kDeltaRRecBytes + kRecV, 2 * kRecT, &sync->single);
            }
            if (ch > 0) load(ch - 1);
        }
        __syncwarp();
        const float next_gate = ch > 0 && tid < kCH ? gate(ch - 1) : 1.f;
        uint8_t *st = sm + (ch & 1) * W::kStage, *vown = st + 2 * W::kK;
        const uint32_t kt = smem_addr(st), qt = kt + W::kK, vt = qt + W::kK;
        const uint8_t *rec = st + 2 * W::kK + W::kV;
        const float *vec = reinterpret_cast<const float *>(rec);
        const float *gs = gates + (ch & 1) * kCH;
        const size_t row0 = (size_t)bh * a.L + t0 + ch * kCH;
        const int cnt = min(kCH, len - ch * kCH);
        if (cnt < kCH) {
#pragma unroll
            for (int p = 0; p < 2 * (D / 64); ++p) clear_rows<128, kCH, NT>(st + p * kPanel, cnt, tid);
            clear_rows<NW * 32, kCH, NT>(vown, cnt, tid);
            __syncthreads();
        }
        float X[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[n][e] = 0.f;
        const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t rf[4], rl[4];
            split2(R[2 * ks][0], R[2 * ks][1], rf[0], rl[0]);
            split2(R[2 * ks][2], R[2 * ks][3], rf[1], rl[1]);
            split2(R[2 * ks + 1][0], R[2 * ks + 1][1], rf[2], rl[2]);
            split2(R[2 * ks + 1][2], R[2 * ks + 1][3], rf[3], rl[3]);
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                uint32_t b[4];
                ldsm4(b, kt + panel_off(16 * n2 + br, 2 * (k0 + ks) + bc));
                mma16816(X[2 * n2], rf, b[0], b[1]);
                mma16816(X[2 * n2 + 1], rf, b[2], b[3]);
                mma16816(X[2 * n2], rl, b[0], b[1]);
                mma16816(X[2 * n2 + 1], rl, b[2], b[3]);
            }
        }
        uint32_t v4[4][4];
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
            ldsm4t(v4[k4], vt + own_off<NW>(16 * k4 + (lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1, wr));
        if (KP == 1) __syncwarp();  // the warp's part of dy is free
        uint32_t pf[4][4], pg[4][4];  // p, and exp(c) p
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 re = *reinterpret_cast<const float2 *>(vec + 64 + 8 * n + 2 * c);
            const float2 ga = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * c);
            const float2 go = *reinterpret_cast<const float2 *>(gs + 8 * n + 2 * c);
            X[n][0] *= re.x;
            X[n][1] *= re.y;
            X[n][2] *= re.x;
            X[n][3] *= re.y;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int q = 2 * (n & 1) + z;
                const float p0 = go.x * low_f(v4[n / 2][q]), p1 = go.y * high_f(v4[n / 2][q]);
                pf[n / 2][q] = pack2(p0, p1);
                pg[n / 2][q] = pack2(ga.x * p0, ga.y * p1);
            }
        }
        {  // the adjoint after the chunk
            __nv_bfloat16 *dst = a.R_c + (((size_t)sid * a.NCH + ch) * D + vbase + 16 * wr) * D + 16 * k0;
            put_rows(R, 1.f, lane, [&](int r, int n, int at, const uint2 &x) { *reinterpret_cast<uint2 *>(dst + (size_t)r * D + 8 * n + at / 2) = x; });
        }
        if (W::kLate) {
            if (ok) ok = wait_for(&sync->single, turn & 1, &sync->abort_flag, a.give_up & kGiveUpLate);
            __syncwarp();
        }
        const uint4 *lt = reinterpret_cast<const uint4 *>(W::kLate ? sm + 2 * W::kStage : rec + kRecV) + lane;
        const uint4 *pt = lt + kRecT / 16;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (KP == 2 && (k4 == 1 || k4 == 2) != (kp == 1)) continue;  // ten of the twenty tiles to each of two warps
#pragma unroll
            for (int n = 0; n < 2 * k4 + 2; ++n) {
                const uint4 b = pt[(rev_base(n) + k4 - n / 2) * 32];
                mma16816(X[n], pf[k4], b.z, b.w);
                mma16816(X[n], pf[k4], b.x, b.y);
            }
        }
        if (KP == 2)
            pair_sum<8>(reinterpret_cast<float4 *>(sm + W::kTotal + sizeof(WalkSync)), warp, lane,
                     [&](auto leave) {
#pragma unroll
                         for (int n = 0; n < 8; ++n) leave(n, X[n]);
                     },
                     [&](auto add) {
#pragma unroll
                         for (int n = 0; n < 8; ++n) add(n, X[n]);
                     });
        uint32_t wf[4][4], wl[4][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 be = *reinterpret_cast<const float2 *>(vec + 128 + 8 * n + 2 * c);
            X[n][0] *= be.x;
            X[n][1] *= be.y;
            X[n][2] *= be.x;
            X[n][3] *= be.y;
            split2(X[n][0], X[n][1], wf[n / 2][2 * (n & 1)], wl[n / 2][2 * (n & 1)]);
            split2(X[n][2], X[n][3], wf[n / 2][2 * (n & 1) + 1], wl[n / 2][2 * (n & 1) + 1]);
        }
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
            for (int n = 0; n < 2 * k4 + 2; ++n) {
                const uint4 b = lt[(rev_base(n) + k4 - n / 2) * 32];
                mma16816(X[n], wf[k4], b.x, b.y);
                mma16816(X[n], wl[k4], b.x, b.y);
                mma16816(X[n], wf[k4], b.z, b.w);
            }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            split2(X[n][0], X[n][1], wf[n / 2][2 * (n & 1)], wl[n / 2][2 * (n & 1)]);
            split2(X[n][2], X[n][3], wf[n / 2][2 * (n & 1) + 1], wl[n / 2][2 * (n & 1) + 1]);
        }
        put_tokens<NW, KP, D>(a.dv + row0 * D + vbase + 16 * wr, wf, vown, cnt, wr, kp, lane);
        put_tokens<NW, KP, D>(a.W_lo + row0 * D + vbase + 16 * wr, wl, vown, cnt, wr, kp, lane);
#pragma unroll
        for (int n = 0; n < 8; ++n) {  // -exp(c) w
            const float2 ga = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * c);
            split2(-ga.x * X[n][0], -ga.y * X[n][1], wf[n / 2][2 * (n & 1)], wl[n / 2][2 * (n & 1)]);
            split2(-ga.x * X[n][2], -ga.y * X[n][3], wf[n / 2][2 * (n & 1) + 1], wl[n / 2][2 * (n & 1) + 1]);
        }
        const float dec = vec[192];
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) R[n][e] *= dec;
        const int tr = ((lane >> 3) & 1) * 8 + (lane & 7), tc = lane >> 4;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
            for (int n2 = 0; n2 < KS; ++n2) {
                uint32_t b[4];
                ldsm4t(b, kt + panel_off(16 * k4 + tr, 2 * (k0 + n2) + tc));
                mma16816(R[2 * n2], wf[k4], b[0], b[1]);
                mma16816(R[2 * n2 + 1], wf[k4], b[2], b[3]);
                mma16816(R[2 * n2], wl[k4], b[0], b[1]);
                mma16816(R[2 * n2 + 1], wl[k4], b[2], b[3]);
                ldsm4t(b, qt + panel_off(16 * k4 + tr, 2 * (k0 + n2) + tc));
                mma16816(R[2 * n2], pg[k4], b[0], b[1]);
                mma16816(R[2 * n2 + 1], pg[k4], b[2], b[3]);
            }
        if (ch > 0 && tid < kCH) gates[(ch - 1 & 1) * kCH + tid] = next_gate;
    }
    if (W::kLate && __syncthreads_or(!ok)) {  // the last chunk's wait
        give_up(nch, nch);
        return;
    }
    let_next_start();
}

// ---------------------------------------------------------------------------
// delta_grads_tc: one CTA per chunk, everything that sums over value rows (k_delta_simt.cu's header).
// Eight warps: warp % 4 takes 16 tokens, warp / 4 half of the dimensions.  The warps of one half form B1, those of the
// other B2 (16 rows each), and leave them in shared memory as 16 x 16 blocks of the lower triangle in two bf16 terms, from
// which both read them as they lie (with beta_j) and transposed.  A chunk is a chain of loads and small products, so two
// CTAs share an SM, a load is under way while what is there is worked on, and tiles that have been read make room: q and k
// come where the second terms of e and w were, the pairs' second terms go where e was (d = 128), S's second block where the
// first was, R where p and w were, e comes again in S's place, u in R's.  2048 chunks, d = 128: 147 us for 0.52 GB (3.5 TB/s)
// and 33 GFLOP of products; 4096 chunks with gates and pooled keys 317 us.  Bound by the latency of loads and products
// within a chunk, with 16 warps on an SM.
// e, w and the weighted pairs enter the sums over pairs in two terms: for keys that resemble each other these sums cancel
// (one term: dq and dbeta up to 5e-2 off, 117 us).  p, S, R and e's and w's products with these are one term's: the gradients
// come out 1.7e-3 to 2.5e-3 off in the 2-norm, of which their own last rounding is 1.7e-3.
// The decay's gradient is a running sum of pair terms of which each enters and leaves with the same value.
constexpr int kGradThreads = 256;

struct GradMaps {
    CUtensorMap dy, e, e_lo, w, w_lo, q, k, u, S, R;  // tokens (e and w in two terms); the memories and adjoints by chunk
};
struct GradSync {
    uint64_t tiles, S0, qk, S1, R, u;
    int abort_flag, used;  // used: the barriers, in this order, that copies were sent to
};

template <int D>
struct GradSmem {
    static constexpr int kT = kCH * D * 2;   // a 64-token tile
    static constexpr int kM = 64 * D * 2;    // 64 rows of S or R
    static constexpr int kVec = 4 * (22 * kCH + 16);
    static constexpr int kB = 2 * 10 * 512;  // B1 and B2: ten 16 x 16 blocks each, their first terms
    static constexpr int kBl = kT < kB ? kB : 0;  // their second terms (else over e's tile)
    static constexpr int kSync = 5 * kT + kM + kB + kBl + kVec;
    static constexpr int kTotal = kSync + (int)sizeof(GradSync);
};

template <int D>
__global__ void __launch_bounds__(kGradThreads, 2) delta_grads_tc(DeltaTcArgs a, const __grid_constant__ GradMaps maps)
{
    using G = GradSmem<D>;
    constexpr int PIECES = D / 8, KS = D / 16, HD = D / 2, HN = HD / 8;  // HN column tiles per warp
    constexpr int MB = D / 64;                                                         // blocks of S and R
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t *Qt = sm, *Kt = Qt + G::kT, *Pt = Kt + G::kT, *Et = Pt + G::kT, *Wt = Et + G::kT, *Mt = Wt + G::kT;
    uint8_t *Bt = Mt + G::kM, *Bl = G::kBl ? Bt + G::kB : Et;
    float *cum = reinterpret_cast<float *>(Bt + G::kB + G::kBl), *bet = cum + kCH, *gs = bet + kCH, *pw = gs + kCH;
    float *rowsum = pw + kCH;                      // [4][2][64] by half: Y.k, exp(c) p S q, D R e k, exp(c) w S k
    float *rowf = rowsum + 8 * kCH, *colf = rowf + 5 * kCH;  // [2][10][16] sums of F's blocks over their columns, rows
    float *red = colf + 5 * kCH;
    const Where w = chunk_at(a, blockIdx.x);
    if (w.cnt <= 0) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int wm = warp & 3, m0 = 16 * wm, half = warp >> 2, d0 = half * HD;
    const size_t row0 = (size_t)w.bh * a.L + w.tb;
    const __nv_bfloat16 *S = a.S_c + (size_t)blockIdx.x * D * D;
    GradSync *sync = reinterpret_cast<GradSync *>(sm + G::kSync);

    // one thread's
    auto load_tokens = [&](uint8_t *dst, const CUtensorMap &map, uint64_t *bar) {
#pragma unroll
        for (int p = 0; p < D / 64; ++p) tma_load_3d(dst + p * kPanel, &map, 64 * p, w.tb, w.bh, bar);
    };
    auto load_rows = [&](uint8_t *dst, const CUtensorMap &map, int b, uint64_t *bar) {  // rows 64 b .. of S or R
#pragma unroll
        for (int p = 0; p < D / 64; ++p) tma_load_3d(dst + p * kPanel, &map, 64 * p, 64 * b, (int)blockIdx.x, bar);
    };
    // the chunk's last tokens may be another segment's
    auto clear_tokens = [&](uint8_t *tile) {
#pragma unroll
        for (int p = 0; p < D / 64; ++p) clear_rows<128, kCH, kGradThreads>(tile + p * kPanel, w.cnt, tid);
    };
    if (tid == 0) {
        sync->abort_flag = (smem_addr(sm) & 1023) != 0;
        sync->used = 0;
        mbar_init(&sync->tiles, 1);
        mbar_init(&sync->S0, 1);
        mbar_init(&sync->qk, 1);
        mbar_init(&sync->S1, 1);
        mbar_init(&sync->R, 1);
        mbar_init(&sync->u, 1);
        fence_mbar_init();
    }
    after_previous();
    // the gates' loads first, or they would queue behind the tiles
    const int gt = warp == 0 ? 2 * lane : tid - kCH;
    const bool in_chunk = gt >= 0 && gt < w.cnt;
    float g0 = 0.f, g1 = 1.f, g2 = 0.f;
    if (warp == 0) {
        if (in_chunk) g0 = delta_log(__bfloat162float(a.la[row0 + gt]));
        g1 = gt + 1 < w.cnt ? delta_log(__bfloat162float(a.la[row0 + gt + 1])) : 0.f;
    } else if (in_chunk) {
        g0 = __bfloat162float(a.be[row0 + gt]);
        if (a.gon) g1 = a.gon[(row0 + gt) * a.gw_stride];
        if (a.pw) g2 = a.pw[(row0 + gt) * a.gw_stride];
    }
    __syncthreads();
    bool ok = sync->abort_flag == 0;
    auto wait = [&](uint64_t *bar, int kind) {
        if (ok) ok = wait_for(bar, 0, &sync->abort_flag, a.give_up & kind);
    };
    auto give_up = [&]() {
        if (tid != 0) return;
        for (uint64_t *bar : {&sync->tiles, &sync->S0, &sync->qk, &sync->S1, &sync->R, &sync->u})
            if (sync->used >> (bar - &sync->tiles) & 1) wait_out(bar, 0);
        atomicExch(&g_delta_abort, 1);
    };
    if (ok && tid == 0) {
        sync->used = 3;
        mbar_arrive_expect_tx(&sync->tiles, 5 * G::kT);
        load_tokens(Pt, maps.dy, &sync->tiles);
        load_tokens(Et, maps.e, &sync->tiles);
        load_tokens(Wt, maps.w, &sync->tiles);
        load_tokens(Kt, maps.e_lo, &sync->tiles);  // (q and k take the places of the second terms, which the pairs alone need)
        load_tokens(Qt, maps.w_lo, &sync->tiles);
        mbar_arrive_expect_tx(&sync->S0, G::kM);
        load_rows(Mt, maps.S, 0, &sync->S0);
    }
    __syncwarp();
    if (warp == 0) {
        float s = g0 + g1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float n = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += n;
        }
        cum[gt] = s - g1;
        cum[gt + 1] = s;
    } else if (gt >= 0 && gt < kCH) {
        bet[gt] = g0;
        gs[gt] = g1;
        pw[gt] = g2;
    }
    wait(&sync->tiles, kGiveUpTiles);
    if (__syncthreads_or(!ok)) {
        give_up();
        return;
    }
    if (w.cnt < kCH) {
        for (uint8_t *t : {Qt, Kt, Pt, Et, Wt}) clear_tokens(t);
        __syncthreads();
    }
    if (a.gon) {  // p = g dy, in place
        for (int e = tid; e < kCH * PIECES; e += kGradThreads) {
            const int r = e / PIECES;
            uint4 *x = reinterpret_cast<uint4 *>(Pt + panel_off(r, e % PIECES));
            uint4 y = *x;
            uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
            for (int z = 0; z < 4; ++z) yw[z] = pack2(gs[r] * low_f(yw[z]), gs[r] * high_f(yw[z]));
            *x = y;
        }
        __syncthreads();
    }

    const int ar = m0 + (lane & 15), ac = lane >> 4;                       // A operand of a token tile
    const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;     // B, columns = rows of the tile
    const int tr = ((lane >> 3) & 1) * 8 + (lane & 7), tc = lane >> 4;     // B, rows = rows of the tile
    const float c_lo = cum[m0 + g], c_hi = cum[m0 + g + 8], ce = cum[kCH - 1];
    auto zero = [](auto &x) {
#pragma unroll
        for (int n = 0; n < (int)(sizeof(x) / sizeof(x[0])); ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
    };
    auto scale = [&](float (&x)[HN][4], float e0, float e1) {
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            x[n][0] *= e0; x[n][1] *= e0; x[n][2] *= e1; x[n][3] *= e1;
        }
    };
    // the warp's 16 rows of `tile` times 64 rows of S or R (block b of its columns)
    auto times_rows = [&](float (&x)[HN][4], const uint8_t *tile, const uint8_t *rows, int b) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t af[4];
            ldsm4(af, smem_addr(tile) + panel_off(ar, 2 * (4 * b + ks) + ac));
#pragma unroll
            for (int n2 = 0; n2 < HN / 2; ++n2) {
                uint32_t bf[4];
                ldsm4t(bf, smem_addr(rows) + panel_off(16 * ks + tr, d0 / 8 + 2 * n2 + tc));
                mma16816(x[2 * n2], af, bf[0], bf[1]);
                mma16816(x[2 * n2 + 1], af, bf[2], bf[3]);
            }
        }
    };
    // x += (the weighted pairs) times the tokens of `tile`
    auto times_tokens = [&](float (&x)[HN][4], const uint32_t (&f)[4], const uint8_t *tile, int k4) {
#pragma unroll
        for (int n2 = 0; n2 < HN / 2; ++n2) {
            uint32_t bf[4];
            ldsm4t(bf, smem_addr(tile) + panel_off(16 * k4 + tr, d0 / 8 + 2 * n2 + tc));
            mma16816(x[2 * n2], f, bf[0], bf[1]);
            mma16816(x[2 * n2 + 1], f, bf[2], bf[3]);
        }
    };
    auto row_dot = [&](const float (&x)[HN][4], const uint8_t *tile, int what) {  // per token, over this half
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            const uint32_t a0 = *reinterpret_cast<const uint32_t *>(tile + panel_off(m0 + g, d0 / 8 + n) + 4 * c);
            const uint32_t a1 = *reinterpret_cast<const uint32_t *>(tile + panel_off(m0 + g + 8, d0 / 8 + n) + 4 * c);
            s0 = fmaf(x[n][0], low_f(a0), fmaf(x[n][1], high_f(a0), s0));
            s1 = fmaf(x[n][2], low_f(a1), fmaf(x[n][3], high_f(a1), s1));
        }
        s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
        s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
        s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
        s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
        if (c == 0) {
            rowsum[(2 * what + half) * kCH + m0 + g] = s0;
            rowsum[(2 * what + half) * kCH + m0 + g + 8] = s1;
        }
    };
    // Block (r, q) of B1 (which = 0) or B2: 16 rows of 32 bytes, their two pieces exchanged every four rows.
    auto block = [&](int which, int r, int q) { return (uint32_t)((which * 10 + r * (r + 1) / 2 + q) * 512); };
    const uint32_t bh_at = smem_addr(Bt), bl_at = smem_addr(Bl);  // first, second terms
    auto block_off = [](int r, int pc) { return (uint32_t)(r * 32 + ((pc ^ ((r >> 2) & 1)) << 4)); };
    // The ten blocks of a half go round its warps, three or two to each, five to an SM's quarter.
    auto block_at = [&](int x, int &r, int &q) {
        const int blk = (half ? 3 - wm : wm) + 4 * x;
        r = (blk >= 1) + (blk >= 3) + (blk >= 6);
        q = blk - r * (r + 1) / 2;
        return blk;
    };
    // x += 16 tokens of `rows` against 16 of `cols`
    auto pairs = [&](float (&x)[2][4], const uint8_t *rows, int r, const uint8_t *cols, int q) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t af[4], bf[4];
            ldsm4(af, smem_addr(rows) + panel_off(16 * r + (lane & 15), 2 * ks + ac));
            ldsm4(bf, smem_addr(cols) + panel_off(16 * q + br, 2 * ks + bc));
            mma16816(x[0], af, bf[0], bf[1]);
            mma16816(x[1], af, bf[2], bf[3]);
        }
    };
    // a block of B weighted with D_ij; w_i . e_i is kept
    float *we = gs;  // (the gates have been read)
    auto weigh = [&](float (&x)[2][4], int r, int q) {
        const float c0 = cum[16 * r + g], c1 = cum[16 * r + g + 8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 cj = *reinterpret_cast<const float2 *>(cum + 16 * q + 8 * h + 2 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int il = g + 8 * (e >> 1), jl = 8 * h + 2 * c + (e & 1);
                if (half == 1 && r == q && jl == il) we[16 * r + il] = x[h][e];
                x[h][e] = r > q || jl < il || (half == 0 && jl == il) ? x[h][e] * __expf((e >> 1 ? c1 : c0) - (e & 1 ? cj.y : cj.x)) : 0.f;
            }
        }
    };
    // into shared memory in two terms, and back
    auto put_block = [&](const float (&x)[2][4], int r, int q) {
        uint32_t f[4], l[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            split2(x[h][0], x[h][1], f[2 * h], l[2 * h]);
            split2(x[h][2], x[h][3], f[2 * h + 1], l[2 * h + 1]);
        }
        const uint32_t at = block(half, r, q) + block_off(lane & 15, lane >> 4);
        stsm4(bh_at + at, f[0], f[1], f[2], f[3]);
        stsm4(bl_at + at, l[0], l[1], l[2], l[3]);
    };
    // block (r, q) of B as pairs of values: register x holds (row g + 8 (x % 2), columns 8 (x / 2) + 2 c, + 1)
    auto get_block = [&](float2 (&v)[4], int which, int r, int q) {
        uint32_t f[4], l[4];
        const uint32_t at = block(which, r, q) + block_off(lane & 15, lane >> 4);
        ldsm4(f, bh_at + at);
        ldsm4(l, bl_at + at);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = make_float2(low_f(f[x]) + low_f(l[x]), high_f(f[x]) + high_f(l[x]));
    };
    // F_ij = beta_j B_ij (rows_i . k_j) for j < i: the sums over a block's columns and rows
    auto pair_sums = [&](const uint8_t *rows, float sign, int blk, int r, int q) {
        float kk[2][4], f0 = 0.f, f1 = 0.f, col[2][2];
        float2 b[4];
        zero(kk);
        pairs(kk, rows, r, Kt, q);
        get_block(b, half, r, q);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 bj = *reinterpret_cast<const float2 *>(bet + 16 * q + 8 * h + 2 * c);
            col[h][0] = col[h][1] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int il = g + 8 * (e >> 1), jl = 8 * h + 2 * c + (e & 1);
                const float f = r > q || jl < il ? sign * (e & 1 ? bj.y : bj.x) * kk[h][e] * (e & 1 ? b[2 * h + (e >> 1)].y : b[2 * h + (e >> 1)].x) : 0.f;
                col[h][e & 1] += f;
                if (e >> 1) f1 += f;
                else f0 += f;
            }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                col[h][0] += __shfl_xor_sync(0xffffffffu, col[h][0], o);
                col[h][1] += __shfl_xor_sync(0xffffffffu, col[h][1], o);
            }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            f0 += __shfl_xor_sync(0xffffffffu, f0, o);
            f1 += __shfl_xor_sync(0xffffffffu, f1, o);
        }
        float *rf = rowf + (half * 10 + blk) * 16, *cf = colf + (half * 10 + blk) * 16;
        if (c == 0) {
            rf[g] = f0;
            rf[g + 8] = f1;
        }
        if (g == 0)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                cf[8 * h + 2 * c] = col[h][0];
                cf[8 * h + 2 * c + 1] = col[h][1];
            }
    };
    // x += (this warp's rows of B, with beta_j) times the keys
    auto times_keys = [&](float (&x)[HN][4], int which) {
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (k4 > wm) continue;
            float2 v[4];
            get_block(v, which, wm, k4);
            uint32_t f[4], l[4];
#pragma unroll
            for (int x2 = 0; x2 < 4; ++x2) {
                const float2 be = *reinterpret_cast<const float2 *>(bet + 16 * k4 + 8 * (x2 / 2) + 2 * c);
                split2(v[x2].x * be.x, v[x2].y * be.y, f[x2], l[x2]);
            }
            times_tokens(x, l, Kt, k4);
            times_tokens(x, f, Kt, k4);
        }
    };
    // 16 x HD results to global memory: neighbouring lanes exchange halves of two tiles, so that a row's four lanes
    // write 32 bytes in a run
    auto store = [&](__nv_bfloat16 *dst, const float (&x)[HN][4]) {
#pragma unroll
        for (int n = 0; n < HN; n += 2)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t p0 = pack2(x[n][2 * h], x[n][2 * h + 1]), p1 = pack2(x[n + 1][2 * h], x[n + 1][2 * h + 1]);
                const uint32_t got = __shfl_xor_sync(0xffffffffu, c & 1 ? p0 : p1, 1);
                const int t = m0 + g + 8 * h;
                if (t < w.cnt)
                    *reinterpret_cast<uint2 *>(dst + (row0 + t) * D + d0 + 8 * (n + (c & 1)) + 4 * (c >> 1)) =
                        c & 1 ? make_uint2(got, p1) : make_uint2(p0, got);
            }
    };

    {
        float b[3][2][4];
        int r, q;
#pragma unroll
        for (int x = 0; x < 3; ++x)
            if (block_at(x, r, q) < 10) {
                zero(b[x]);
                pairs(b[x], half ? Wt : Pt, r, Kt, q);  // e's second term
                if (half) pairs(b[x], Qt, r, Et, q);    // w's second term
                pairs(b[x], half ? Wt : Pt, r, Et, q);
                weigh(b[x], r, q);
            }
        fence_async_smem();  // (what was cleared in the tiles, before the copies over them)
        __syncthreads();     // the second terms have been read, and e
        if (tid == 0) {
            sync->used |= 4;
            mbar_arrive_expect_tx(&sync->qk, 2 * G::kT);
            load_tokens(Qt, maps.q, &sync->qk);
            load_tokens(Kt, maps.k, &sync->qk);
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 3; ++x)
            if (block_at(x, r, q) < 10) put_block(b[x], r, q);
    }
    wait(&sync->S0, kGiveUpLate);
    __syncwarp();
    float z[HN][4];
    zero(z);
    {
        float dq[HN][4];
        zero(dq);
        times_rows(dq, Pt, Mt, 0);
        times_rows(z, Wt, Mt, 0);
        wait(&sync->qk, kGiveUpLate);
        if (__syncthreads_or(!ok)) {  // the blocks are there, S's first rows have been read
            give_up();
            return;
        }
        if (MB > 1 && tid == 0) {
            sync->used |= 8;
            mbar_arrive_expect_tx(&sync->S1, G::kM);
            load_rows(Mt, maps.S, 1, &sync->S1);
        }
        __syncwarp();
        if (w.cnt < kCH) {
            clear_tokens(Qt);
            clear_tokens(Kt);
            __syncthreads();
        }
        {
            int r, q;
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                const int blk = block_at(x, r, q);
                if (blk < 10) pair_sums(half ? Kt : Qt, half ? -1.f : 1.f, blk, r, q);
            }
        }
        if (MB > 1) {
            wait(&sync->S1, kGiveUpLate);
            __syncwarp();
            times_rows(dq, Pt, Mt, 1);
            times_rows(z, Wt, Mt, 1);
        }
        fence_async_smem();
        if (__syncthreads_or(!ok)) {  // p and w have been read: their tiles take R, and S's takes e
            give_up();
            return;
        }
        if (tid == 0) {
            sync->used |= 16;
            mbar_arrive_expect_tx(&sync->R, MB * G::kM + (MB > 1 ? G::kT : 0));
            load_rows(Wt, maps.R, 0, &sync->R);
            if (MB > 1) {
                load_rows(Pt, maps.R, 1, &sync->R);
                load_tokens(Mt, maps.e, &sync->R);
            }
        }
        __syncwarp();
        const float e0 = __expf(c_lo), e1 = __expf(c_hi);
        scale(dq, e0, e1);
        scale(z, e0, e1);
        row_dot(dq, Qt, 1);
        row_dot(z, Kt, 3);
        float2 add[HN / 2][2];  // half of the cached memories' share at once, on its way under the products
        auto fetch = [&](int hf) {
#pragma unroll
            for (int n = 0; n < HN / 2; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int t = m0 + g + 8 * x;
                    add[n][x] = t < w.cnt ? *reinterpret_cast<const float2 *>(a.dq_add + (row0 + t) * D + d0 + 8 * (hf * (HN / 2) + n) + 2 * c)
                                          : make_float2(0.f, 0.f);
                }
        };
        auto join = [&](int hf) {
#pragma unroll
            for (int n = 0; n < HN / 2; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    dq[hf * (HN / 2) + n][2 * x] += add[n][x].x;
                    dq[hf * (HN / 2) + n][2 * x + 1] += add[n][x].y;
                }
        };
        if (a.dq_add) fetch(0);
        times_keys(z, 1);
        if (a.dq_add) {
            join(0);
            fetch(1);
        }
        times_keys(dq, 0);
        if (a.dq_add) join(1);
        store(a.dq, dq);
    }
    float y[HN][4];
    zero(y);
    uint8_t *const E2 = MB > 1 ? Mt : Et;
    float in = 0.f;  // <R, S>; S's rows are still there where they are one block
    constexpr int X4 = 64 * PIECES / kGradThreads;
    uint4 s4[MB][X4];
    if (MB > 1)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int x = 0; x < X4; ++x) s4[mb][x] = *reinterpret_cast<const uint4 *>(S + (size_t)(tid + (mb * X4 + x) * kGradThreads) * 8);
    wait(&sync->R, kGiveUpEnd);
    __syncwarp();
    if (MB > 1 && w.cnt < kCH) {
        clear_tokens(E2);
        __syncthreads();
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int x = 0; x < X4; ++x) {
            const int e = tid + x * kGradThreads;
            const uint32_t o = panel_off(e / PIECES, e % PIECES);
            const uint4 r4 = *reinterpret_cast<const uint4 *>((mb ? Pt : Wt) + o);
            const uint4 m4 = MB > 1 ? s4[mb][x] : *reinterpret_cast<const uint4 *>(Mt + o);
            const uint32_t *rw = reinterpret_cast<const uint32_t *>(&r4), *sw = reinterpret_cast<const uint32_t *>(&m4);
#pragma unroll
            for (int q = 0; q < 4; ++q) in = fmaf(low_f(rw[q]), low_f(sw[q]), fmaf(high_f(rw[q]), high_f(sw[q]), in));
        }
    times_rows(y, E2, Wt, 0);
    if (MB > 1) times_rows(y, E2, Pt, 1);
    if (a.pw) {  // u for the pooled keys' share, in R's place
        __syncthreads();
        if (ok && tid == 0) {
            sync->used |= 32;
            mbar_arrive_expect_tx(&sync->u, G::kT);
            load_tokens(Wt, maps.u, &sync->u);
        }
        __syncwarp();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) in += __shfl_xor_sync(0xffffffffu, in, o);
    if (lane == 0) red[warp] = in;
    scale(y, __expf(ce - c_lo), __expf(ce - c_hi));
    row_dot(y, Kt, 2);
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {  // the transposed blocks: rows j, columns i >= j
        if (k4 < wm) continue;
        const uint32_t off = block_off(((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1);
#pragma unroll
        for (int term = 1; term >= 0; --term) {
            const uint32_t at = (term ? bl_at : bh_at) + off;
            uint32_t f[4];
            ldsm4t(f, at + block(0, k4, wm));
            times_tokens(y, f, Qt, k4);
            ldsm4t(f, at + block(1, k4, wm));
#pragma unroll
            for (int q = 0; q < 4; ++q) f[q] ^= 0x80008000u;
            times_tokens(y, f, Kt, k4);
        }
    }
    row_dot(y, Kt, 0);
    {
        const float be0 = bet[m0 + g], be1 = bet[m0 + g + 8];
#pragma unroll
        for (int n = 0; n < HN; ++n) {  // dk
            y[n][0] = fmaf(be0, y[n][0], -z[n][0]);
            y[n][1] = fmaf(be0, y[n][1], -z[n][1]);
            y[n][2] = fmaf(be1, y[n][2], -z[n][2]);
            y[n][3] = fmaf(be1, y[n][3], -z[n][3]);
        }
    }
    if (a.pw) wait(&sync->u, kGiveUpEnd);
    if (__syncthreads_or(!ok)) {  // the sums are there
        give_up();
        return;
    }
    if (a.pw && w.cnt < kCH) {
        clear_tokens(Wt);
        __syncthreads();
    }
    if (a.pw) {  // the pooled keys' share: rho after the chunk + sum over the chunk's tokens t >= j of pw_t u_t
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (k4 < wm) continue;
            uint32_t fh[4], fl[4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = m0 + g + 8 * x, t = 8 * (2 * k4 + h) + 2 * c;
                    split2(t >= j ? pw[t] : 0.f, t + 1 >= j ? pw[t + 1] : 0.f, fh[2 * h + x], fl[2 * h + x]);
                }
            times_tokens(y, fh, Wt, k4);
            times_tokens(y, fl, Wt, k4);
        }
        const float *rho = a.rho + (size_t)blockIdx.x * D + d0 + 2 * c;
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            const float2 x = *reinterpret_cast<const float2 *>(rho + 8 * n);
            y[n][0] += x.x; y[n][1] += x.y; y[n][2] += x.x; y[n][3] += x.y;
        }
    }
    store(a.dk, y);
    if (warp == 0) {
        // dbeta, and h_t = <adjoint, memory> before token t: exp(c_end) <R, S>, the reads of S by tokens i >= t, the
        // writes of tokens j < t into R, and the pairs F_ij on either side of t.  As a running sum from the end every
        // pair enters with one value and leaves with the same, so nothing of the pairs on one side stays behind.
        const int i = 2 * lane;
        float in = 0.f, fr = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) in += red[x];
        float h0 = 0.f, h1 = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int t = i + x;
            const float f = bet[t] * (rowsum[4 * kCH + t] + rowsum[5 * kCH + t]);
            float r = (rowsum[2 * kCH + t] + rowsum[3 * kCH + t]) - (rowsum[6 * kCH + t] + rowsum[7 * kCH + t]) - f;
#pragma unroll
            for (int y = 0; y < 8; ++y) {  // block (t's, y) of its row, (y, t's) of its column, of B1 and B2
                const int b0 = t / 16, b1 = y % 4, base = y / 4 * 10;
                if (b1 <= b0) r += rowf[(base + b0 * (b0 + 1) / 2 + b1) * 16 + t % 16];
                if (b1 >= b0) r -= colf[(base + b1 * (b1 + 1) / 2 + b0) * 16 + t % 16];
            }
            (x ? h1 : h0) = r;
            fr += f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) fr += __shfl_xor_sync(0xffffffffu, fr, o);
        float s = h0 + h1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float n = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += n;
        }
        const float end = __expf(ce) * in + fr;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (i + x >= w.cnt) continue;
            const float h = end + s - (x ? h0 : 0.f);
            a.dla[row0 + i + x] = __float2bfloat16_rn(w.ch == 0 && i + x == 0 ? 0.f : h);  // the first decay meets an empty memory
            // w_t . e_t / beta_t; without a beta_t, e_t . (N_t k_t) through the pairs, whose terms may cancel
            const int t = i + x;
            a.dbe[row0 + t] = __float2bfloat16_rn(fabsf(bet[t]) > 1e-20f ? we[t] / bet[t] : rowsum[t] + rowsum[kCH + t]);
        }
    }
}

template <int D, int NW>
bool make_maps(DeltaMaps *m, const Problem &p, const DeltaTcArgs &a, const void *v, int q_rows = kCH)
{
    const auto sw = NW == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    return make_tmap_bf16_3d_sw128(&m->k, a.k, p.BH, p.L, D, kCH) && make_tmap_bf16_3d_sw128(&m->q, a.q, p.BH, p.L, D, q_rows) &&
           make_tmap_bf16_3d(&m->v, v, p.BH, p.L, D, 16 * NW, kCH, sw);
}

// Few walkers leave most of the card idle, and a chunk's products on a walker's way to the next chunk are what counts: then
// two warps share 16 rows, half of the keys each.  KP = 2 with two row groups per CTA as long as every CTA has an SM to
// itself, else four row groups and whole rows.  L = 2048, d = 128, one memory (forward, recomputed, reverse walk), KP = 2
// against 1: 32 heads (128 CTAs) 80 66 82 against 103 83 113 us; 48 heads (192 CTAs) 155 97 156 against 103 82 113 us.
inline bool split_keys(const Problem &p) { return (long long)p.BH * p.N * (p.d / 32) <= 152; }

template <int D, int NW, int KP>
cudaError_t rwalk_launch(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    constexpr int smem = RWalkSmem<D, NW, KP>::kTotal + (int)sizeof(WalkSync) + (KP == 2 ? 2 * NW * 8 * 512 : 0);
    DeltaMaps maps;
    if (!make_maps<D, NW>(&maps, p, a, a.dy)) return cudaErrorUnknown;
    auto kern = delta_rwalk_tc<D, NW, KP>;
    return launch_early(kern, (long long)p.BH * p.N * (D / (16 * NW)), 32 * NW * KP, smem, s, a, maps);
}

template <int D>
cudaError_t grads_tc_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    cudaError_t e = split_keys(p) ? rwalk_launch<D, 2, 2>(p, a, s) : rwalk_launch<D, 4, 1>(p, a, s);
    if (e != cudaSuccess) return e;
    profile_after_kernel(s, "delta_rwalk_tc");
    constexpr int smem = GradSmem<D>::kTotal;
    GradMaps maps;
    const unsigned long long chunks = (unsigned long long)p.BH * p.N * a.NCH;
    auto tokens = [&](CUtensorMap *m, const void *x) { return make_tmap_bf16_3d_sw128(m, x, p.BH, p.L, D, kCH); };
    if (!tokens(&maps.dy, a.dy) || !tokens(&maps.e, a.E) || !tokens(&maps.w, a.dv) || !tokens(&maps.e_lo, a.E_lo) ||
        !tokens(&maps.w_lo, a.W_lo) || !tokens(&maps.q, a.q) || !tokens(&maps.k, a.k) ||
        !tokens(&maps.u, a.pw ? a.u : a.k) || !make_tmap_bf16_3d_sw128(&maps.S, a.S_c, chunks, D, D, 64) ||
        !make_tmap_bf16_3d_sw128(&maps.R, a.R_c, chunks, D, D, 64))
        return cudaErrorUnknown;
    auto kern = delta_grads_tc<D>;
    e = launch_early(kern, (long long)p.BH * p.N * a.NCH, kGradThreads, smem, s, a, maps);
    profile_after_kernel(s, "delta_grads_tc");
    return e;
}

// dy_t . O_t per token (the gradient of the online gate): d / 8 lanes per token.
__global__ void __launch_bounds__(256) delta_dgon(const __nv_bfloat16 *dy, const __nv_bfloat16 *O, float *dgon, long long tokens, int d)
{
    const int pieces = d / 8;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    const bool ok = e / pieces < tokens;
    float s = 0.f;
    if (ok) {
        const uint4 y = reinterpret_cast<const uint4 *>(dy)[e], o = reinterpret_cast<const uint4 *>(O)[e];
        const uint32_t *yw = reinterpret_cast<const uint32_t *>(&y), *ow = reinterpret_cast<const uint32_t *>(&o);
#pragma unroll
        for (int q = 0; q < 4; ++q) s = fmaf(low_f(yw[q]), low_f(ow[q]), fmaf(high_f(yw[q]), high_f(ow[q]), s));
    }
    for (int o = pieces / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (ok && e % pieces == 0) dgon[e / pieces] = s;
}

template <int D, bool READ, bool REV>
cudaError_t prep_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    constexpr int smem = prep_smem<D, READ || REV>();
    DeltaMaps maps;
    if (!make_maps<D, 4>(&maps, p, a, a.v, 16)) return cudaErrorUnknown;
    auto kern = delta_prep_tc<D, READ, REV>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * p.N * a.NCH), 32, smem, s>>>(a, maps);
    return cudaGetLastError();
}

template <int D, int NW, int KP, bool READ, bool FULL>
cudaError_t walk_launch(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    constexpr int smem = WalkSmem<D, NW, KP, READ>::kTotal + (int)sizeof(WalkSync) + (KP == 2 ? 2 * NW * (READ ? 12 : 8) * 512 : 0);
    DeltaMaps maps;
    if (!make_maps<D, NW>(&maps, p, a, a.v)) return cudaErrorUnknown;
    auto kern = delta_walk_tc<D, NW, KP, READ, FULL>;
    return launch_early(kern, (long long)p.BH * p.N * (D / (16 * NW)), 32 * NW * KP, smem, s, a, maps);
}

template <int D, bool READ, bool FULL>
cudaError_t walk_kp(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    return split_keys(p) ? walk_launch<D, 2, 2, READ, FULL>(p, a, s) : walk_launch<D, 4, 1, READ, FULL>(p, a, s);
}

template <int D, bool READ>
cudaError_t walk_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    // (the forward always reads, and only it walks in full terms and without the reverse walk's record)
    cudaError_t e = !READ || a.rrec ? prep_impl<D, READ, true>(p, a, s) : prep_impl<D, true, false>(p, a, s);
    if (e != cudaSuccess) return e;
    profile_after_kernel(s, "delta_prep_tc");
    e = READ && a.full ? walk_kp<D, true, true>(p, a, s) : walk_kp<D, READ, false>(p, a, s);
    profile_after_kernel(s, "delta_walk_tc");
    return e;
}

}  // namespace

cudaError_t take_delta_abort(int *was_set)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_delta_abort, sizeof(int));
    if (e != cudaSuccess) return e;
    *was_set = v;
    if (v) {
        v = 0;
        e = cudaMemcpyToSymbol(g_delta_abort, &v, sizeof(int));
    }
    return e;
}

cudaError_t launch_delta_dgon(const Problem &p, const void *dy, const void *O, float *dgon, cudaStream_t s)
{
    const long long n = (long long)p.BH * p.L;
    delta_dgon<<<(unsigned)((n * (p.d / 8) + 255) / 256), 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(dy),
                                                                   static_cast<const __nv_bfloat16 *>(O), dgon, n, p.d);
    return cudaGetLastError();
}

void set_delta_give_up(int waits) { g_give_up = waits; }

cudaError_t launch_delta_grads_tc(const Problem &p, const DeltaTcArgs &args, cudaStream_t s)
{
    DeltaTcArgs a = args;
    a.give_up = g_give_up;
    return p.d == 64 ? grads_tc_impl<64>(p, a, s) : grads_tc_impl<128>(p, a, s);
}

bool delta_tc_supported(const Problem &p) { return p.bf16 && (p.d == 64 || p.d == 128); }

cudaError_t launch_delta_walk_tc(const Problem &p, const DeltaTcArgs &args, bool read, cudaStream_t s)
{
    DeltaTcArgs a = args;
    a.give_up = g_give_up;
    if (p.d == 64) return read ? walk_impl<64, true>(p, a, s) : walk_impl<64, false>(p, a, s);
    return read ? walk_impl<128, true>(p, a, s) : walk_impl<128, false>(p, a, s);
}

}  // namespace mc
