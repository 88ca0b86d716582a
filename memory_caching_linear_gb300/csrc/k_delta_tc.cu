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
// Precision: the memory, the errors and T carry fp32 accuracy (every operand that is not an input is
// split into two bf16 terms, products of two lows left out: 2^-17 of a term); rounding T, R or S to
// one bf16 would put 2^-9 of the memory into every later error.  P is one bf16 term, since it only
// reaches the bf16 output.
#include <cstdint>

#include "mc_internal.cuh"
#include "mma_sync.cuh"

namespace mc {
namespace {

using namespace mma;

constexpr int kCH = kDeltaChunk;
constexpr int kPrepThreads = 128;
constexpr int kAP = kCH + 1;  // padded row of the 64 x 64 matrices

// Lower-triangular B operands by 16 x 8 tiles: column tile nt (8 tokens) needs row tiles kt <= nt / 2.
constexpr int kTiles = 20;
__host__ __device__ constexpr int tile_base(int nt) { return nt / 2 * (nt / 2 + 1) + (nt & 1) * (nt / 2 + 1); }
static_assert(tile_base(7) + 4 == kTiles, "tiles of a lower triangle");

// A chunk's record (DeltaTcArgs::rec): T - 1 as {hi, lo} operand tiles, P tiles, and 256 floats:
// exp(c_i), beta_i exp(c_end - c_i), beta_i, and [192] exp(c_end).
constexpr int kRecT = kTiles * 32 * 16, kRecP = kTiles * 32 * 8, kRecV = 1024;
constexpr int kRec = kDeltaRecBytes;
static_assert(kRecT + kRecP + kRecV == kRec, "record");

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

// ---------------------------------------------------------------------------
// delta_prep_tc: one CTA per chunk.  K K^T (exact bf16 products) on the tensor cores, 16 rows per
// warp; (1 + A)^-1 in fp32 by 16 x 16 blocks: each warp inverts a diagonal block by substitution (a lane
// per column), then X_ij = -X_ii sum_k A_ik X_kj, one block diagonal after the other.
// ---------------------------------------------------------------------------
template <int D, bool READ>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_tc(DeltaTcArgs a)
{
    constexpr int ROW = D * 2, PIECES = D / 8;
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t *Kt = sm, *Qt = Kt + kCH * ROW;
    float *A = reinterpret_cast<float *>(Qt + (READ ? kCH * ROW : 0)), *X = A + kCH * kAP, *Y = X + kCH * kAP;
    __shared__ float cum[kCH], bet[kCH];
    const Where w = chunk_at(a, blockIdx.x);
    if (w.cnt <= 0) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const size_t row0 = (size_t)w.bh * a.L + w.tb;
    for (int e = tid; e < kCH * PIECES; e += kPrepThreads) {
        const int r = e / PIECES, pc = e % PIECES;
        const size_t off = (row0 + (r < w.cnt ? r : 0)) * D + pc * 8;
        cp16(smem_addr(Kt) + tile_off<ROW>(r, pc), a.k + off, r < w.cnt);
        if (READ) cp16(smem_addr(Qt) + tile_off<ROW>(r, pc), a.q + off, r < w.cnt);
    }
    cp_commit();
    if (warp == 0) {  // running sums of the chunk's decays, two tokens per lane
        const int i = 2 * lane;
        const float x0 = i < w.cnt ? delta_log(__bfloat162float(a.la[row0 + i])) : 0.f;
        const float x1 = i + 1 < w.cnt ? delta_log(__bfloat162float(a.la[row0 + i + 1])) : 0.f;
        float s = x0 + x1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float n = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += n;
        }
        cum[i] = s - x1;
        cum[i + 1] = s;
        bet[i] = i < w.cnt ? __bfloat162float(a.be[row0 + i]) : 0.f;
        bet[i + 1] = i + 1 < w.cnt ? __bfloat162float(a.be[row0 + i + 1]) : 0.f;
    }
    cp_wait<0>();
    __syncthreads();
    uint8_t *rec = a.rec + (size_t)blockIdx.x * kRec;
    {
        // rows 16 warp .. + 15, columns up to the diagonal
        float kk[8][4], qk[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
        const int ar = 16 * warp + (lane & 15), ac = lane >> 4;
        const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t ak[4], aq[4];
            ldsm4(ak, smem_addr(Kt) + tile_off<ROW>(ar, 2 * ks + ac));
            if (READ) ldsm4(aq, smem_addr(Qt) + tile_off<ROW>(ar, 2 * ks + ac));
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                if (n2 > warp) break;
                uint32_t b[4];
                ldsm4(b, smem_addr(Kt) + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(kk[2 * n2], ak, b[0], b[1]);
                mma16816(kk[2 * n2 + 1], ak, b[2], b[3]);
                if (READ) {
                    mma16816(qk[2 * n2], aq, b[0], b[1]);
                    mma16816(qk[2 * n2 + 1], aq, b[2], b[3]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * warp + g + 8 * (e >> 1), j = 8 * n + 2 * c + (e & 1);
                const float dec = j <= i ? expf(cum[i] - cum[j]) : 0.f;
                A[i * kAP + j] = j < i ? kk[n][e] * dec * bet[j] : 0.f;
                if (READ) Y[i * kAP + j] = qk[n][e] * dec;
                X[i * kAP + j] = 0.f;
            }
    }
    __syncthreads();
    {  // diagonal blocks: lane j < 16 has column j
        float *Xd = X + (16 * warp) * kAP + 16 * warp;
        const float *Ad = A + (16 * warp) * kAP + 16 * warp;
        if (lane < 16) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < i; ++k) {
                    if (k & 1) s1 = fmaf(-Ad[i * kAP + k], x[k], s1);
                    else s0 = fmaf(-Ad[i * kAP + k], x[k], s0);
                }
                x[i] = s0 + s1;
                Xd[i * kAP + lane] = x[i];
            }
        }
    }
    __syncthreads();
    if (READ) {  // P tiles while the blocks settle (nothing below touches Y until the next barrier)
        uint2 *pt = reinterpret_cast<uint2 *>(rec + kRecT);
        for (int e = tid; e < kTiles * 32; e += kPrepThreads) {
            const int t = e / 32, l = e % 32;
            int nt = 0;
            while (nt < 7 && tile_base(nt + 1) <= t) ++nt;
            const float *y = Y + (8 * nt + l / 4) * kAP + 16 * (t - tile_base(nt)) + 2 * (l % 4);
            pt[e] = make_uint2(pack2(y[0], y[1]), pack2(y[8], y[9]));
        }
        __syncthreads();
    }
    for (int diag = 1; diag < 4; ++diag) {
        // blocks (i, j) with i - j = diag: Y_ij = sum_{j <= k < i} A_ik X_kj, then X_ij = -X_ii Y_ij
        const int nb = 4 - diag;
        for (int e = tid; e < nb * 64; e += kPrepThreads) {  // four entries of a row each
            const int b = e / 64, r = (e % 64) / 4, cc = (e % 4) * 4, i = b + diag;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 16 * b; k < 16 * i; ++k) {
                const float av = A[(16 * i + r) * kAP + k];
#pragma unroll
                for (int x = 0; x < 4; ++x) s[x] = fmaf(av, X[k * kAP + 16 * b + cc + x], s[x]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) Y[(16 * i + r) * kAP + 16 * b + cc + x] = s[x];
        }
        __syncthreads();
        for (int e = tid; e < nb * 64; e += kPrepThreads) {
            const int b = e / 64, r = (e % 64) / 4, cc = (e % 4) * 4, i = b + diag;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float xv = X[(16 * i + r) * kAP + 16 * i + k];
#pragma unroll
                for (int x = 0; x < 4; ++x) s[x] = fmaf(-xv, Y[(16 * i + k) * kAP + 16 * b + cc + x], s[x]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) X[(16 * i + r) * kAP + 16 * b + cc + x] = s[x];
        }
        __syncthreads();
    }
    uint4 *tt = reinterpret_cast<uint4 *>(rec);
    for (int e = tid; e < kTiles * 32; e += kPrepThreads) {
        const int t = e / 32, l = e % 32;
        int nt = 0;
        while (nt < 7 && tile_base(nt + 1) <= t) ++nt;
        const int i = 8 * nt + l / 4, j = 16 * (t - tile_base(nt)) + 2 * (l % 4);
        const float *x = X + i * kAP + j;
        uint4 o;
        split2(j < i ? x[0] : 0.f, j + 1 < i ? x[1] : 0.f, o.x, o.z);
        split2(j + 8 < i ? x[8] : 0.f, j + 9 < i ? x[9] : 0.f, o.y, o.w);
        tt[e] = o;
    }
    if (tid < kCH) {
        float *vec = reinterpret_cast<float *>(rec + kRecT + kRecP);
        const float ce = cum[kCH - 1];  // tokens past the end add nothing
        vec[tid] = expf(cum[tid]);
        vec[64 + tid] = bet[tid] * expf(ce - cum[tid]);
        vec[128 + tid] = bet[tid];
        if (tid == 0) vec[192] = expf(ce);
    }
}

// ---------------------------------------------------------------------------
// delta_walk_tc: one CTA per (bh, segment, 16 NW value rows); NW warps of 16 rows.  Two stages of
// the chunk's K, V columns, (Q,) and record, filled by asynchronous copies one chunk ahead.
// ---------------------------------------------------------------------------
template <int D, int NW, bool READ>
struct WalkSmem {
    static constexpr int kK = kCH * D * 2, kV = kCH * NW * 32;
    static constexpr int kStage = kK * (READ ? 2 : 1) + kV + kRec;
    static constexpr int kOut = NW * 2048;  // a warp's 64 tokens x 16 values on their way out
    static constexpr int kTotal = 2 * kStage + kOut;
};

template <int D, int NW, bool READ>
__global__ void __launch_bounds__(32 * NW) delta_walk_tc(DeltaTcArgs a)
{
    using W = WalkSmem<D, NW, READ>;
    constexpr int ROW = D * 2, PIECES = D / 8, NT = 32 * NW, KS = D / 16, VROW = NW * 32, VP = NW * 2;
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr int splits = D / (16 * NW);
    const int rs = (int)blockIdx.x % splits;
    const long long sid = blockIdx.x / splits;
    const int seg = (int)(sid % a.N), bh = (int)(sid / a.N);
    const int t0 = seg * a.C, len = min((seg + 1) * a.C, a.L) - t0, nch = (len + kCH - 1) / kCH;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int vbase = rs * 16 * NW;  // the CTA's first value row

    auto load = [&](int ch) {
        uint8_t *st = sm + (ch & 1) * W::kStage;
        const int cnt = min(kCH, len - ch * kCH);
        const size_t row0 = (size_t)bh * a.L + t0 + ch * kCH;
        for (int e = tid; e < kCH * PIECES; e += NT) {
            const int r = e / PIECES, pc = e % PIECES;
            const size_t off = (row0 + (r < cnt ? r : 0)) * D + pc * 8;
            cp16(smem_addr(st) + tile_off<ROW>(r, pc), a.k + off, r < cnt);
            if (READ) cp16(smem_addr(st) + W::kK + W::kV + tile_off<ROW>(r, pc), a.q + off, r < cnt);
        }
        for (int e = tid; e < kCH * VP; e += NT) {
            const int r = e / VP, pc = e % VP;
            // rows of VROW bytes; the pieces of a row turn with it
            cp16(smem_addr(st) + W::kK + r * VROW + ((pc ^ (r & (VP < 8 ? VP - 1 : 7))) << 4),
                 a.v + (row0 + (r < cnt ? r : 0)) * D + vbase + pc * 8, r < cnt);
        }
        const uint8_t *rec = a.rec + ((size_t)sid * a.NCH + ch) * kRec;
        const uint32_t dst = smem_addr(st) + W::kStage - kRec;
        for (int e = tid; e < kRec / 16; e += NT)
            if (READ || e < kRecT / 16 || e >= (kRecT + kRecP) / 16) cp16(dst + e * 16, rec + e * 16, true);
        cp_commit();
    };

    float S[2 * KS][4];  // 16 rows x D keys: tile n holds keys 8n ..
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = 0.f;

    uint8_t *outb = sm + 2 * W::kStage + warp * 2048;
    load(0);
    for (int ch = 0; ch < nch; ++ch) {
        cp_wait<0>();
        __syncthreads();  // the chunk has come, and the stage of the one before is free
        if (ch + 1 < nch) load(ch + 1);
        const uint8_t *st = sm + (ch & 1) * W::kStage;
        const uint32_t kt = smem_addr(st), vt = kt + W::kK, qt = vt + W::kV;
        const uint8_t *rec = st + W::kStage - kRec;
        const float *vec = reinterpret_cast<const float *>(rec + kRecT + kRecP);
        const size_t row0 = (size_t)bh * a.L + t0 + ch * kCH;
        const int cnt = min(kCH, len - ch * kCH);
        const size_t cidx = (size_t)sid * a.NCH + ch;

        if (a.S_c) {  // the memory before the chunk, in bf16, through the warp's staging area
            __nv_bfloat16 *dst = a.S_c + (cidx * D + vbase + 16 * warp) * D;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {  // 64 keys at a time: 16 rows of 128 bytes
#pragma unroll
                for (int n = 0; n < 8; n += 2)
                    stsm4(smem_addr(outb) + tile_off<128>(lane & 15, n + (lane >> 4)), pack2(S[8 * h + n][0], S[8 * h + n][1]),
                          pack2(S[8 * h + n][2], S[8 * h + n][3]), pack2(S[8 * h + n + 1][0], S[8 * h + n + 1][1]),
                          pack2(S[8 * h + n + 1][2], S[8 * h + n + 1][3]));
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = x * 4 + lane / 8, pc = lane % 8;
                    *reinterpret_cast<uint4 *>(dst + (size_t)r * D + 64 * h + pc * 8) =
                        *reinterpret_cast<const uint4 *>(outb + tile_off<128>(r, pc));
                }
                __syncwarp();
            }
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
                ldsm4(b, kt + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(X[2 * n2], hi, b[0], b[1]);
                mma16816(X[2 * n2 + 1], hi, b[2], b[3]);
                mma16816(X[2 * n2], lo, b[0], b[1]);
                mma16816(X[2 * n2 + 1], lo, b[2], b[3]);
                if (READ) {  // the output is bf16: one term
                    ldsm4(b, qt + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                    mma16816(O[2 * n2], hi, b[0], b[1]);
                    mma16816(O[2 * n2 + 1], hi, b[2], b[3]);
                }
            }
        }
        // R = V - diag(exp c) K S^T, then E = R + (T - 1) R
#pragma unroll
        for (int kt4 = 0; kt4 < 4; ++kt4) {
            uint32_t v4[4];
            {
                const int r = 16 * kt4 + (lane >> 4) * 8 + (lane & 7), pc = 2 * warp + ((lane >> 3) & 1);
                ldsm4t(v4, vt + r * VROW + ((pc ^ (r & (VP < 8 ? VP - 1 : 7))) << 4));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * kt4 + h;
                const float2 ga = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * c);
                X[n][0] = low_f(v4[2 * h]) - ga.x * X[n][0];
                X[n][1] = high_f(v4[2 * h]) - ga.y * X[n][1];
                X[n][2] = low_f(v4[2 * h + 1]) - ga.x * X[n][2];
                X[n][3] = high_f(v4[2 * h + 1]) - ga.y * X[n][3];
                if (READ) {
                    O[n][0] *= ga.x;
                    O[n][1] *= ga.y;
                    O[n][2] *= ga.x;
                    O[n][3] *= ga.y;
                }
            }
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
        // U = diag(beta) E for the read and the readout; U' = diag(beta exp(c_end - c)) E for the memory
        const float dec = vec[192];
        uint32_t uh[4][4], ul[4][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 be = *reinterpret_cast<const float2 *>(vec + 128 + 8 * n + 2 * c);
            const uint32_t u0 = pack2(be.x * X[n][0], be.y * X[n][1]), u1 = pack2(be.x * X[n][2], be.y * X[n][3]);
            uh[n / 2][2 * (n & 1)] = u0;
            uh[n / 2][2 * (n & 1) + 1] = u1;
        }
        if (READ) {
            const uint2 *pt = reinterpret_cast<const uint2 *>(rec + kRecT) + lane;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
                for (int n = 2 * k4; n < 8; ++n) {
                    const uint2 b = pt[(tile_base(n) + k4) * 32];
                    mma16816(O[n], uh[k4], b.x, b.y);
                }
        }
        auto put = [&](__nv_bfloat16 *dst, const uint32_t (&f)[4][4]) {  // f: an operand of values x tokens
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
                const int r = 16 * k4 + (lane >> 4) * 8 + (lane & 7), pc = (lane >> 3) & 1;
                stsm4t(smem_addr(outb) + r * 32 + ((pc ^ ((r >> 2) & 1)) << 4), f[k4][0], f[k4][1], f[k4][2], f[k4][3]);
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = 16 * x + lane / 2, pc = lane % 2;
                if (r < cnt)
                    *reinterpret_cast<uint4 *>(dst + (row0 + r) * D + vbase + 16 * warp + 8 * pc) =
                        *reinterpret_cast<const uint4 *>(outb + r * 32 + ((pc ^ ((r >> 2) & 1)) << 4));
            }
            __syncwarp();
        };
        if (a.U) put(a.U, uh);
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
                        const int t = 8 * n + 2 * c + (e & 1), r = vbase + 16 * warp + g + 8 * (e >> 1);
                        if (t < cnt) a.O_on[(row0 + t) * D + r] = O[n][e];
                    }
            }
        }
        if (a.E) {
            uint32_t ef[4][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                ef[n / 2][2 * (n & 1)] = pack2(X[n][0], X[n][1]);
                ef[n / 2][2 * (n & 1) + 1] = pack2(X[n][2], X[n][3]);
            }
            put(a.E, ef);
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
                ldsm4t(b, kt + tile_off<ROW>(16 * k4 + tr, 2 * n2 + tc));
                mma16816(S[2 * n2], uh[k4], b[0], b[1]);
                mma16816(S[2 * n2 + 1], uh[k4], b[2], b[3]);
                mma16816(S[2 * n2], ul[k4], b[0], b[1]);
                mma16816(S[2 * n2 + 1], ul[k4], b[2], b[3]);
            }
    }
    if (a.states) {
        float *dst = a.states + ((size_t)sid * D + vbase + 16 * warp) * D;
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
            *reinterpret_cast<float2 *>(dst + (size_t)g * D + 8 * n + 2 * c) = make_float2(S[n][0], S[n][1]);
            *reinterpret_cast<float2 *>(dst + (size_t)(g + 8) * D + 8 * n + 2 * c) = make_float2(S[n][2], S[n][3]);
        }
    }
}

// The scalars of the window update that the readout's kernels take (mc_forward_swla's alpha, beta, lambda):
// over the written values beta_t e_t the delta memory is the one with alpha = exp(log_alpha), beta = 0, lambda = 1.
__global__ void __launch_bounds__(256) delta_scalars(const __nv_bfloat16 *la, float *alpha, float *zero, float *one, long long n)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    alpha[i] = delta_decay(__bfloat162float(la[i]));
    zero[i] = 0.f;
    one[i] = 1.f;
}

template <int D, bool READ>
cudaError_t prep_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    const size_t smem = (READ ? 2 : 1) * kCH * D * 2 + 3 * sizeof(float) * kCH * kAP;
    auto kern = delta_prep_tc<D, READ>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * p.N * a.NCH), kPrepThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D, int NW, bool READ>
cudaError_t walk_launch(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    constexpr int smem = WalkSmem<D, NW, READ>::kTotal;
    auto kern = delta_walk_tc<D, NW, READ>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * p.N * (D / (16 * NW))), 32 * NW, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool READ>
cudaError_t walk_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    cudaError_t e = prep_impl<D, READ>(p, a, s);
    if (e != cudaSuccess) return e;
    profile_after_kernel(s, "delta_prep_tc");
    e = walk_launch<D, 4, READ>(p, a, s);
    profile_after_kernel(s, "delta_walk_tc");
    return e;
}

}  // namespace

bool delta_tc_supported(const Problem &p) { return p.bf16 && (p.d == 64 || p.d == 128); }

cudaError_t launch_delta_scalars(const Problem &p, const void *la, float *alpha, float *zero, float *one, cudaStream_t s)
{
    const long long n = (long long)p.BH * p.L;
    delta_scalars<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(la), alpha, zero, one, n);
    return cudaGetLastError();
}

cudaError_t launch_delta_walk_tc(const Problem &p, const DeltaTcArgs &a, bool read, cudaStream_t s)
{
    if (p.d == 64) return read ? walk_impl<64, true>(p, a, s) : walk_impl<64, false>(p, a, s);
    return read ? walk_impl<128, true>(p, a, s) : walk_impl<128, false>(p, a, s);
}

}  // namespace mc
