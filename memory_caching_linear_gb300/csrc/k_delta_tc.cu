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

// The other way round, rows m >= columns i: column tile nt needs row tiles kt = nt / 2 .. 3.
__host__ __device__ constexpr int rev_base(int nt) { return 8 * (nt / 2) - nt / 2 * (nt / 2 - 1) + (nt & 1) * (4 - nt / 2); }
static_assert(rev_base(7) + 1 == kTiles, "tiles of an upper triangle");
__device__ __forceinline__ void rev_tile(int t, int &nt, int &kt)
{
    nt = 0;
    while (nt < 7 && rev_base(nt + 1) <= t) ++nt;
    kt = nt / 2 + t - rev_base(nt);
}
// The reverse walk's record: T - 1 (one term), P, and exp(c_i), exp(c_end - c_i), beta_i, [192] exp(c_end).
static_assert(2 * kRecP + kRecV == kDeltaRRecBytes, "record");

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
template <int D, bool READ, bool REV>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_tc(DeltaTcArgs a)
{
    constexpr int ROW = D * 2, PIECES = D / 8;
    constexpr bool QK = READ || REV;
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t *Kt = sm, *Qt = Kt + kCH * ROW;
    float *A = reinterpret_cast<float *>(Qt + (QK ? kCH * ROW : 0)), *X = A + kCH * kAP, *Y = X + kCH * kAP;
    __shared__ float cum[kCH], bet[kCH];
    const Where w = chunk_at(a, blockIdx.x);
    if (w.cnt <= 0) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const size_t row0 = (size_t)w.bh * a.L + w.tb;
    for (int e = tid; e < kCH * PIECES; e += kPrepThreads) {
        const int r = e / PIECES, pc = e % PIECES;
        const size_t off = (row0 + (r < w.cnt ? r : 0)) * D + pc * 8;
        cp16(smem_addr(Kt) + tile_off<ROW>(r, pc), a.k + off, r < w.cnt);
        if (QK) cp16(smem_addr(Qt) + tile_off<ROW>(r, pc), a.q + off, r < w.cnt);
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
            if (QK) ldsm4(aq, smem_addr(Qt) + tile_off<ROW>(ar, 2 * ks + ac));
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                if (n2 > warp) break;
                uint32_t b[4];
                ldsm4(b, smem_addr(Kt) + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(kk[2 * n2], ak, b[0], b[1]);
                mma16816(kk[2 * n2 + 1], ak, b[2], b[3]);
                if (QK) {
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
                if (QK) Y[i * kAP + j] = qk[n][e] * dec;
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
    if (REV) {  // the same P as an operand of rows i, columns j
        uint2 *pt = reinterpret_cast<uint2 *>(a.rrec + (size_t)blockIdx.x * kDeltaRRecBytes + kRecP);
        for (int e = tid; e < kTiles * 32; e += kPrepThreads) {
            int nt, kt;
            rev_tile(e / 32, nt, kt);
            const int l = e % 32;
            const float *y = Y + (16 * kt + 2 * (l % 4)) * kAP + 8 * nt + l / 4;
            pt[e] = make_uint2(pack2(y[0], y[kAP]), pack2(y[8 * kAP], y[9 * kAP]));
        }
        if (!READ) __syncthreads();
    }
    if (READ) {  // P tiles (nothing below touches Y until the next barrier)
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
    if (REV) {
        uint8_t *rrec = a.rrec + (size_t)blockIdx.x * kDeltaRRecBytes;
        uint2 *lt = reinterpret_cast<uint2 *>(rrec);
        for (int e = tid; e < kTiles * 32; e += kPrepThreads) {
            int nt, kt;
            rev_tile(e / 32, nt, kt);
            const int l = e % 32, i = 8 * nt + l / 4, m = 16 * kt + 2 * (l % 4);  // T_mi, m > i
            const float *x = X + m * kAP + i;
            lt[e] = make_uint2(pack2(m > i ? x[0] : 0.f, m + 1 > i ? x[kAP] : 0.f),
                               pack2(m + 8 > i ? x[8 * kAP] : 0.f, m + 9 > i ? x[9 * kAP] : 0.f));
        }
        if (tid < kCH) {
            float *vec = reinterpret_cast<float *>(rrec + 2 * kRecP);
            const float ce = cum[kCH - 1];
            vec[tid] = expf(cum[tid]);
            vec[64 + tid] = expf(ce - cum[tid]);
            vec[128 + tid] = bet[tid];
            if (tid == 0) vec[192] = expf(ce);
        }
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

// A warp's 16 rows of f S into an operand image (D / 64 panels of D rows), through its 2 KB staging area.
template <int NT>
__device__ __forceinline__ void put_image(const float (&S)[NT][4], uint8_t *img, float f, uint8_t *outb, int row, int lane)
{
#pragma unroll
    for (int h = 0; h < NT / 8; ++h) {
#pragma unroll
        for (int n = 8 * h; n < 8 * h + 8; n += 2)
            stsm4(smem_addr(outb) + tile_off<128>(lane & 15, (n & 7) + (lane >> 4)), pack2(f * S[n][0], f * S[n][1]),
                  pack2(f * S[n][2], f * S[n][3]), pack2(f * S[n + 1][0], f * S[n + 1][1]), pack2(f * S[n + 1][2], f * S[n + 1][3]));
        __syncwarp();
        uint4 *dst = reinterpret_cast<uint4 *>(img + h * (NT * 8 * 128) + row * 128);
#pragma unroll
        for (int x = 0; x < 4; ++x) dst[32 * x + lane] = reinterpret_cast<const uint4 *>(outb)[32 * x + lane];
        __syncwarp();
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

        // an image's panels: 64 columns of all D rows, rows of 128 bytes with their pieces exchanged by row % 8
        if (a.spre_img && ch > 0 && !(ch & 1))
            put_image(S, a.spre_img + ((size_t)sid * (a.C / 128) + ch / 2) * (D * D * 2), vec[0], outb, vbase + 16 * warp, lane);
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
    if (a.states_img) put_image(S, a.states_img + (size_t)sid * (D * D * 2), 1.f, outb, vbase + 16 * warp, lane);
    if (a.states) {
        float *dst = a.states + ((size_t)sid * D + vbase + 16 * warp) * D;
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
// R itself enters the products in two bf16 terms, the rest in one: the results are bf16 gradients.
// ---------------------------------------------------------------------------
template <int D, int NW>
struct RWalkSmem {
    static constexpr int kK = kCH * D * 2, kV = kCH * NW * 32;
    static constexpr int kStage = 2 * kK + kV + kDeltaRRecBytes + 256;  // K, Q, dy columns, record, gates
    static constexpr int kTotal = 2 * kStage + NW * 2048;
};

template <int D, int NW>
__global__ void __launch_bounds__(32 * NW) delta_rwalk_tc(DeltaTcArgs a)
{
    using W = RWalkSmem<D, NW>;
    constexpr int ROW = D * 2, PIECES = D / 8, NT = 32 * NW, KS = D / 16, VROW = NW * 32, VP = NW * 2;
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr int splits = D / (16 * NW);
    const int rs = (int)blockIdx.x % splits;
    const long long sid = blockIdx.x / splits;
    const int seg = (int)(sid % a.N), bh = (int)(sid / a.N);
    const int t0 = seg * a.C, len = min((seg + 1) * a.C, a.L) - t0, nch = (len + kCH - 1) / kCH;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int vbase = rs * 16 * NW;

    auto load = [&](int ch) {
        uint8_t *st = sm + (ch & 1) * W::kStage;
        const int cnt = min(kCH, len - ch * kCH);
        const size_t row0 = (size_t)bh * a.L + t0 + ch * kCH;
        for (int e = tid; e < kCH * PIECES; e += NT) {
            const int r = e / PIECES, pc = e % PIECES;
            const size_t off = (row0 + (r < cnt ? r : 0)) * D + pc * 8;
            cp16(smem_addr(st) + tile_off<ROW>(r, pc), a.k + off, r < cnt);
            cp16(smem_addr(st) + W::kK + tile_off<ROW>(r, pc), a.q + off, r < cnt);
        }
        for (int e = tid; e < kCH * VP; e += NT) {
            const int r = e / VP, pc = e % VP;
            cp16(smem_addr(st) + 2 * W::kK + r * VROW + ((pc ^ (r & (VP < 8 ? VP - 1 : 7))) << 4),
                 a.dy + (row0 + (r < cnt ? r : 0)) * D + vbase + pc * 8, r < cnt);
        }
        const uint8_t *rec = a.rrec + ((size_t)sid * a.NCH + ch) * kDeltaRRecBytes;
        const uint32_t dst = smem_addr(st) + 2 * W::kK + W::kV;
        for (int e = tid; e < kDeltaRRecBytes / 16; e += NT) cp16(dst + e * 16, rec + e * 16, true);
        float *gs = reinterpret_cast<float *>(st + 2 * W::kK + W::kV + kDeltaRRecBytes);
        for (int e = tid; e < kCH; e += NT) gs[e] = a.gon && e < cnt ? a.gon[(row0 + e) * a.gw_stride] : 1.f;
        cp_commit();
    };

    float R[2 * KS][4];
    if (a.G_img && seg < a.N - 1) {  // 128 x 128 image: two panels of 128 rows
        const uint8_t *img = a.G_img + (size_t)sid * 32768;
        const int r = vbase + 16 * warp + g;
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
            const uint8_t *at = img + (n / 8) * 16384 + r * 128 + (((n & 7) ^ (r & 7)) << 4) + 4 * c;
            const uint32_t x = *reinterpret_cast<const uint32_t *>(at), y = *reinterpret_cast<const uint32_t *>(at + 8 * 128);
            R[n][0] = low_f(x); R[n][1] = high_f(x); R[n][2] = low_f(y); R[n][3] = high_f(y);
        }
    } else if (a.G && seg < a.N - 1) {
        const float *src = a.G + ((size_t)sid * D + vbase + 16 * warp) * D;
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
            const float2 x = *reinterpret_cast<const float2 *>(src + (size_t)g * D + 8 * n + 2 * c);
            const float2 y = *reinterpret_cast<const float2 *>(src + (size_t)(g + 8) * D + 8 * n + 2 * c);
            R[n][0] = x.x; R[n][1] = x.y; R[n][2] = y.x; R[n][3] = y.y;
        }
    } else {
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) R[n][e] = 0.f;
    }

    uint8_t *outb = sm + 2 * W::kStage + warp * 2048;
    load(nch - 1);
    for (int ch = nch - 1; ch >= 0; --ch) {
        cp_wait<0>();
        __syncthreads();
        if (ch > 0) load(ch - 1);
        const uint8_t *st = sm + (ch & 1) * W::kStage;
        const uint32_t kt = smem_addr(st), qt = kt + W::kK, vt = qt + W::kK;
        const uint8_t *rec = st + 2 * W::kK + W::kV;
        const float *vec = reinterpret_cast<const float *>(rec + 2 * kRecP);
        const float *gs = reinterpret_cast<const float *>(rec + kDeltaRRecBytes);
        const size_t row0 = (size_t)bh * a.L + t0 + ch * kCH;
        const int cnt = min(kCH, len - ch * kCH);
        {
            __nv_bfloat16 *dst = a.R_c + (((size_t)sid * a.NCH + ch) * D + vbase + 16 * warp) * D;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
#pragma unroll
                for (int n = 0; n < 8; n += 2)
                    stsm4(smem_addr(outb) + tile_off<128>(lane & 15, n + (lane >> 4)), pack2(R[8 * h + n][0], R[8 * h + n][1]),
                          pack2(R[8 * h + n][2], R[8 * h + n][3]), pack2(R[8 * h + n + 1][0], R[8 * h + n + 1][1]),
                          pack2(R[8 * h + n + 1][2], R[8 * h + n + 1][3]));
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
        float X[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[n][e] = 0.f;
        const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t hi[4], lo[4];
            split2(R[2 * ks][0], R[2 * ks][1], hi[0], lo[0]);
            split2(R[2 * ks][2], R[2 * ks][3], hi[1], lo[1]);
            split2(R[2 * ks + 1][0], R[2 * ks + 1][1], hi[2], lo[2]);
            split2(R[2 * ks + 1][2], R[2 * ks + 1][3], hi[3], lo[3]);
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                uint32_t b[4];
                ldsm4(b, kt + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(X[2 * n2], hi, b[0], b[1]);
                mma16816(X[2 * n2 + 1], hi, b[2], b[3]);
                mma16816(X[2 * n2], lo, b[0], b[1]);
                mma16816(X[2 * n2 + 1], lo, b[2], b[3]);
            }
        }
        uint32_t pf[4][4], pg[4][4];  // p, and exp(c) p
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            uint32_t v4[4];
            const int r = 16 * k4 + (lane >> 4) * 8 + (lane & 7), pc = 2 * warp + ((lane >> 3) & 1);
            ldsm4t(v4, vt + r * VROW + ((pc ^ (r & (VP < 8 ? VP - 1 : 7))) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * k4 + h;
                const float2 re = *reinterpret_cast<const float2 *>(vec + 64 + 8 * n + 2 * c);
                const float2 ga = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * c);
                const float2 go = *reinterpret_cast<const float2 *>(gs + 8 * n + 2 * c);
                X[n][0] *= re.x;
                X[n][1] *= re.y;
                X[n][2] *= re.x;
                X[n][3] *= re.y;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float p0 = go.x * low_f(v4[2 * h + z]), p1 = go.y * high_f(v4[2 * h + z]);
                    pf[k4][2 * h + z] = pack2(p0, p1);
                    pg[k4][2 * h + z] = pack2(ga.x * p0, ga.y * p1);
                }
            }
        }
        const uint2 *lt = reinterpret_cast<const uint2 *>(rec) + lane;
        const uint2 *pt = reinterpret_cast<const uint2 *>(rec + kRecP) + lane;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
            for (int n = 0; n < 2 * k4 + 2; ++n) {
                const uint2 b = pt[(rev_base(n) + k4 - n / 2) * 32];
                mma16816(X[n], pf[k4], b.x, b.y);
            }
        {
            uint32_t yh[4][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const float2 be = *reinterpret_cast<const float2 *>(vec + 128 + 8 * n + 2 * c);
                X[n][0] *= be.x;
                X[n][1] *= be.y;
                X[n][2] *= be.x;
                X[n][3] *= be.y;
                yh[n / 2][2 * (n & 1)] = pack2(X[n][0], X[n][1]);
                yh[n / 2][2 * (n & 1) + 1] = pack2(X[n][2], X[n][3]);
            }
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
                for (int n = 0; n < 2 * k4 + 2; ++n) {
                    const uint2 b = lt[(rev_base(n) + k4 - n / 2) * 32];
                    mma16816(X[n], yh[k4], b.x, b.y);
                }
        }
        uint32_t wf[4][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            wf[n / 2][2 * (n & 1)] = pack2(X[n][0], X[n][1]);
            wf[n / 2][2 * (n & 1) + 1] = pack2(X[n][2], X[n][3]);
        }
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            const int r = 16 * k4 + (lane >> 4) * 8 + (lane & 7), pc = (lane >> 3) & 1;
            stsm4t(smem_addr(outb) + r * 32 + ((pc ^ ((r >> 2) & 1)) << 4), wf[k4][0], wf[k4][1], wf[k4][2], wf[k4][3]);
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = 16 * x + lane / 2, pc = lane % 2;
            if (r < cnt)
                *reinterpret_cast<uint4 *>(a.dv + (row0 + r) * D + vbase + 16 * warp + 8 * pc) =
                    *reinterpret_cast<const uint4 *>(outb + r * 32 + ((pc ^ ((r >> 2) & 1)) << 4));
        }
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 8; ++n) {  // -exp(c) w
            const float2 ga = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * c);
            wf[n / 2][2 * (n & 1)] = pack2(-ga.x * X[n][0], -ga.y * X[n][1]);
            wf[n / 2][2 * (n & 1) + 1] = pack2(-ga.x * X[n][2], -ga.y * X[n][3]);
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
                ldsm4t(b, kt + tile_off<ROW>(16 * k4 + tr, 2 * n2 + tc));
                mma16816(R[2 * n2], wf[k4], b[0], b[1]);
                mma16816(R[2 * n2 + 1], wf[k4], b[2], b[3]);
                ldsm4t(b, qt + tile_off<ROW>(16 * k4 + tr, 2 * n2 + tc));
                mma16816(R[2 * n2], pg[k4], b[0], b[1]);
                mma16816(R[2 * n2 + 1], pg[k4], b[2], b[3]);
            }
    }
}

// ---------------------------------------------------------------------------
// delta_grads_tc: one CTA per chunk, everything that sums over value rows (k_delta_simt.cu's header).
// Eight warps: warp % 4 takes 16 tokens, warp / 4 half of the dimensions.  B1, B2 and their transposes
// are formed by each warp for its own tokens straight into operand registers.  S and R share a buffer,
// so that two CTAs fit on an SM (d = 128) and one's loads run under the other's products.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 256;

template <int D>
struct GradSmem {
    static constexpr int kT = kCH * D * 2;         // a 64-token tile
    static constexpr int kM = D * D * 2;           // S, then R
    static constexpr int kVec = 4 * (22 * kCH + 16);
    static constexpr int kTotal = 5 * kT + kM + kVec;
};

template <int D>
__global__ void __launch_bounds__(kGradThreads, D == 128 ? 1 : 2) delta_grads_tc(DeltaTcArgs a)
{
    using G = GradSmem<D>;
    constexpr int ROW = D * 2, PIECES = D / 8, KS = D / 16, HD = D / 2, HN = HD / 8;  // HN column tiles per warp
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t *Qt = sm, *Kt = Qt + G::kT, *Pt = Kt + G::kT, *Et = Pt + G::kT, *Wt = Et + G::kT, *Mt = Wt + G::kT;
    float *cum = reinterpret_cast<float *>(Mt + G::kM), *bet = cum + kCH, *gs = bet + kCH, *pw = gs + kCH;
    float *rowsum = pw + kCH;                      // [4][2][64] by half: Y.k, exp(c) p S q, D R e k, exp(c) w S k
    float *rowf = rowsum + 8 * kCH, *colf = rowf + 2 * kCH;  // [2][64], [2][4][64]: sums of F over its rows, columns
    float *red = colf + 8 * kCH;
    const Where w = chunk_at(a, blockIdx.x);
    if (w.cnt <= 0) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const int m0 = 16 * (warp & 3), half = warp >> 2, d0 = half * HD;
    const size_t row0 = (size_t)w.bh * a.L + w.tb;
    const __nv_bfloat16 *S = a.S_c + (size_t)blockIdx.x * D * D, *R = a.R_c + (size_t)blockIdx.x * D * D;

    for (int e = tid; e < kCH * PIECES; e += kGradThreads) {
        const int r = e / PIECES, pc = e % PIECES;
        const bool ok = r < w.cnt;
        const size_t off = (row0 + (ok ? r : 0)) * D + pc * 8;
        const uint32_t o = tile_off<ROW>(r, pc);
        cp16(smem_addr(Qt) + o, a.q + off, ok);
        cp16(smem_addr(Kt) + o, a.k + off, ok);
        cp16(smem_addr(Pt) + o, a.dy + off, ok);
        cp16(smem_addr(Et) + o, a.E + off, ok);
        cp16(smem_addr(Wt) + o, a.dv + off, ok);
    }
    for (int e = tid; e < D * PIECES; e += kGradThreads)
        cp16(smem_addr(Mt) + tile_off<ROW>(e / PIECES, e % PIECES), S + (size_t)e * 8, true);
    cp_commit();
    if (warp == 0) {
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
    }
    if (tid < kCH) {
        const bool ok = tid < w.cnt;
        bet[tid] = ok ? __bfloat162float(a.be[row0 + tid]) : 0.f;
        gs[tid] = ok && a.gon ? a.gon[(row0 + tid) * a.gw_stride] : 1.f;
        pw[tid] = ok && a.pw ? a.pw[(row0 + tid) * a.gw_stride] : 0.f;
    }
    cp_wait<0>();
    __syncthreads();
    if (a.gon) {  // p = g dy, in place
        for (int e = tid; e < kCH * PIECES; e += kGradThreads) {
            const int r = e / PIECES;
            uint4 *x = reinterpret_cast<uint4 *>(Pt + tile_off<ROW>(r, e % PIECES));
            uint4 y = *x;
            uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
            for (int z = 0; z < 4; ++z) yw[z] = pack2(gs[r] * low_f(yw[z]), gs[r] * high_f(yw[z]));
            *x = y;
        }
    }
    auto inner = [](const uint4 &x, const uint4 &y, float s) {
        const uint32_t *xw = reinterpret_cast<const uint32_t *>(&x), *yw = reinterpret_cast<const uint32_t *>(&y);
#pragma unroll
        for (int q = 0; q < 4; ++q) s = fmaf(low_f(xw[q]), low_f(yw[q]), fmaf(high_f(xw[q]), high_f(yw[q]), s));
        return s;
    };
    uint4 sk[D * PIECES / kGradThreads];  // this thread's pieces of S, for <R, S>
#pragma unroll
    for (int x = 0; x < D * PIECES / kGradThreads; ++x) {
        const int e = tid + x * kGradThreads;
        sk[x] = *reinterpret_cast<const uint4 *>(Mt + tile_off<ROW>(e / PIECES, e % PIECES));
    }
    __syncthreads();

    const int ar = m0 + (lane & 15), ac = lane >> 4;                       // A operand of a token tile
    const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;     // B, columns = rows of the tile
    const int tr = ((lane >> 3) & 1) * 8 + (lane & 7), tc = lane >> 4;     // B, rows = rows of the tile
    float dq[HN][4], y[HN][4], z[HN][4];
#pragma unroll
    for (int n = 0; n < HN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[n][e] = y[n][e] = z[n][e] = 0.f;
    // p S and w S
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        uint32_t ap[4], aw[4];
        ldsm4(ap, smem_addr(Pt) + tile_off<ROW>(ar, 2 * ks + ac));
        ldsm4(aw, smem_addr(Wt) + tile_off<ROW>(ar, 2 * ks + ac));
#pragma unroll
        for (int n2 = 0; n2 < HN / 2; ++n2) {
            uint32_t b[4];
            ldsm4t(b, smem_addr(Mt) + tile_off<ROW>(16 * ks + tr, d0 / 8 + 2 * n2 + tc));
            mma16816(dq[2 * n2], ap, b[0], b[1]);
            mma16816(dq[2 * n2 + 1], ap, b[2], b[3]);
            mma16816(z[2 * n2], aw, b[0], b[1]);
            mma16816(z[2 * n2 + 1], aw, b[2], b[3]);
        }
    }
    __syncthreads();  // S has been read
    for (int e = tid; e < D * PIECES; e += kGradThreads)
        cp16(smem_addr(Mt) + tile_off<ROW>(e / PIECES, e % PIECES), R + (size_t)e * 8, true);
    cp_commit();
    const float c_lo = cum[m0 + g], c_hi = cum[m0 + g + 8], ce = cum[kCH - 1];
    {
        const float e0 = expf(c_lo), e1 = expf(c_hi);
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            dq[n][0] *= e0; dq[n][1] *= e0; dq[n][2] *= e1; dq[n][3] *= e1;
            z[n][0] *= e0; z[n][1] *= e0; z[n][2] *= e1; z[n][3] *= e1;
        }
    }
    auto row_dot = [&](const float (&x)[HN][4], const uint8_t *tile, int what) {  // per token, over this half
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            const uint32_t a0 = *reinterpret_cast<const uint32_t *>(tile + tile_off<ROW>(m0 + g, d0 / 8 + n) + 4 * c);
            const uint32_t a1 = *reinterpret_cast<const uint32_t *>(tile + tile_off<ROW>(m0 + g + 8, d0 / 8 + n) + 4 * c);
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
    row_dot(dq, Qt, 1);
    row_dot(z, Kt, 3);
    // rows i of B1 beta and B2 beta (columns j <= i): dq += B1 K, z += B2 K.  F_ij = beta_j (B1_ij q_i.k_j - B2_ij k_i.k_j)
    // for j < i, the first term on the warps of half 0, the second on those of half 1
    {
        float b1[8][4], b2[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) b1[n][e] = b2[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t ap[4], aw[4];
            ldsm4(ap, smem_addr(Pt) + tile_off<ROW>(ar, 2 * ks + ac));
            ldsm4(aw, smem_addr(Wt) + tile_off<ROW>(ar, 2 * ks + ac));
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                if (n2 > (warp & 3)) break;
                uint32_t b[4];
                ldsm4(b, smem_addr(Et) + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(b1[2 * n2], ap, b[0], b[1]);
                mma16816(b1[2 * n2 + 1], ap, b[2], b[3]);
                mma16816(b2[2 * n2], aw, b[0], b[1]);
                mma16816(b2[2 * n2 + 1], aw, b[2], b[3]);
            }
        }
        float f0 = 0.f, f1s = 0.f;  // row sums of F
#pragma unroll
        for (int n2 = 0; n2 < 4; ++n2) {
            float *cf = colf + (4 * half + (warp & 3)) * kCH + 16 * n2;
            if (n2 > (warp & 3)) {
                if (lane < 16) cf[lane] = 0.f;
                continue;
            }
            float kk[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) kk[h][e] = 0.f;
            const uint32_t at = smem_addr(half ? Kt : Qt);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t aq[4], b[4];
                ldsm4(aq, at + tile_off<ROW>(ar, 2 * ks + ac));
                ldsm4(b, smem_addr(Kt) + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(kk[0], aq, b[0], b[1]);
                mma16816(kk[1], aq, b[2], b[3]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * n2 + h, j = 8 * n + 2 * c;
                float col[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = m0 + g + 8 * (e >> 1), jj = j + (e & 1);
                    const float f = jj < i ? expf((e >> 1 ? c_hi : c_lo) - cum[jj]) * bet[jj] * kk[h][e] * (half ? -b2[n][e] : b1[n][e]) : 0.f;
                    col[e & 1] += f;
                    if (e >> 1) f1s += f;
                    else f0 += f;
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    col[0] += __shfl_xor_sync(0xffffffffu, col[0], o);
                    col[1] += __shfl_xor_sync(0xffffffffu, col[1], o);
                }
                if (g == 0) {
                    cf[8 * h + 2 * c] = col[0];
                    cf[8 * h + 2 * c + 1] = col[1];
                }
            }
        }
        f0 += __shfl_xor_sync(0xffffffffu, f0, 1);
        f0 += __shfl_xor_sync(0xffffffffu, f0, 2);
        f1s += __shfl_xor_sync(0xffffffffu, f1s, 1);
        f1s += __shfl_xor_sync(0xffffffffu, f1s, 2);
        if (c == 0) {
            rowf[half * kCH + m0 + g] = f0;
            rowf[half * kCH + m0 + g + 8] = f1s;
        }
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (k4 > (warp & 3)) break;
            uint32_t f1[4], f2[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * k4 + h;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = m0 + g + 8 * (e >> 1), j = 8 * n + 2 * c + (e & 1);
                    const float f = j <= i ? expf((e >> 1 ? c_hi : c_lo) - cum[j]) * bet[j] : 0.f;
                    b1[n][e] *= f;
                    b2[n][e] *= j < i ? f : 0.f;
                }
                f1[2 * h] = pack2(b1[n][0], b1[n][1]);
                f1[2 * h + 1] = pack2(b1[n][2], b1[n][3]);
                f2[2 * h] = pack2(b2[n][0], b2[n][1]);
                f2[2 * h + 1] = pack2(b2[n][2], b2[n][3]);
            }
#pragma unroll
            for (int n2 = 0; n2 < HN / 2; ++n2) {
                uint32_t b[4];
                ldsm4t(b, smem_addr(Kt) + tile_off<ROW>(16 * k4 + tr, d0 / 8 + 2 * n2 + tc));
                mma16816(dq[2 * n2], f1, b[0], b[1]);
                mma16816(dq[2 * n2 + 1], f1, b[2], b[3]);
                mma16816(z[2 * n2], f2, b[0], b[1]);
                mma16816(z[2 * n2 + 1], f2, b[2], b[3]);
            }
        }
    }
    cp_wait<0>();
    __syncthreads();  // R has come
    {
        float in = 0.f;
#pragma unroll
        for (int x = 0; x < D * PIECES / kGradThreads; ++x) {
            const int e = tid + x * kGradThreads;
            in = inner(sk[x], *reinterpret_cast<const uint4 *>(Mt + tile_off<ROW>(e / PIECES, e % PIECES)), in);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) in += __shfl_xor_sync(0xffffffffu, in, o);
        if (lane == 0) red[warp] = in;
    }
    // E R
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        uint32_t ae[4];
        ldsm4(ae, smem_addr(Et) + tile_off<ROW>(ar, 2 * ks + ac));
#pragma unroll
        for (int n2 = 0; n2 < HN / 2; ++n2) {
            uint32_t b[4];
            ldsm4t(b, smem_addr(Mt) + tile_off<ROW>(16 * ks + tr, d0 / 8 + 2 * n2 + tc));
            mma16816(y[2 * n2], ae, b[0], b[1]);
            mma16816(y[2 * n2 + 1], ae, b[2], b[3]);
        }
    }
    {
        const float e0 = expf(ce - c_lo), e1 = expf(ce - c_hi);
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            y[n][0] *= e0; y[n][1] *= e0; y[n][2] *= e1; y[n][3] *= e1;
        }
    }
    row_dot(y, Kt, 2);
    // rows j of B1^T and B2^T (columns i >= j): y += B1^T Q - B2^T K
    {
        float b1[8][4], b2[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) b1[n][e] = b2[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t ae[4];
            ldsm4(ae, smem_addr(Et) + tile_off<ROW>(ar, 2 * ks + ac));
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                if (n2 < (warp & 3)) continue;
                uint32_t b[4];
                ldsm4(b, smem_addr(Pt) + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(b1[2 * n2], ae, b[0], b[1]);
                mma16816(b1[2 * n2 + 1], ae, b[2], b[3]);
                ldsm4(b, smem_addr(Wt) + tile_off<ROW>(16 * n2 + br, 2 * ks + bc));
                mma16816(b2[2 * n2], ae, b[0], b[1]);
                mma16816(b2[2 * n2 + 1], ae, b[2], b[3]);
            }
        }
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (k4 < (warp & 3)) continue;
            uint32_t f1[4], f2[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 2 * k4 + h;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = m0 + g + 8 * (e >> 1), i = 8 * n + 2 * c + (e & 1);
                    const float f = i >= j ? expf(cum[i] - (e >> 1 ? c_hi : c_lo)) : 0.f;
                    b1[n][e] *= f;
                    b2[n][e] *= i > j ? -f : 0.f;
                }
                f1[2 * h] = pack2(b1[n][0], b1[n][1]);
                f1[2 * h + 1] = pack2(b1[n][2], b1[n][3]);
                f2[2 * h] = pack2(b2[n][0], b2[n][1]);
                f2[2 * h + 1] = pack2(b2[n][2], b2[n][3]);
            }
#pragma unroll
            for (int n2 = 0; n2 < HN / 2; ++n2) {
                uint32_t b[4];
                ldsm4t(b, smem_addr(Qt) + tile_off<ROW>(16 * k4 + tr, d0 / 8 + 2 * n2 + tc));
                mma16816(y[2 * n2], f1, b[0], b[1]);
                mma16816(y[2 * n2 + 1], f1, b[2], b[3]);
                ldsm4t(b, smem_addr(Kt) + tile_off<ROW>(16 * k4 + tr, d0 / 8 + 2 * n2 + tc));
                mma16816(y[2 * n2], f2, b[0], b[1]);
                mma16816(y[2 * n2 + 1], f2, b[2], b[3]);
            }
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
    __syncthreads();  // the tiles have been read
    if (a.pw) {  // the pooled keys' share: rho after the chunk + sum over the chunk's tokens t >= j of pw_t u_t
        for (int e = tid; e < kCH * PIECES; e += kGradThreads) {
            const int r = e / PIECES, pc = e % PIECES;
            cp16(smem_addr(Et) + tile_off<ROW>(r, pc), a.u + (row0 + (r < w.cnt ? r : 0)) * D + pc * 8, r < w.cnt);
        }
        cp_commit();
        cp_wait<0>();
        __syncthreads();
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            if (k4 < (warp & 3)) continue;
            uint32_t fh[4], fl[4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = m0 + g + 8 * x, t = 8 * (2 * k4 + h) + 2 * c;
                    split2(t >= j ? pw[t] : 0.f, t + 1 >= j ? pw[t + 1] : 0.f, fh[2 * h + x], fl[2 * h + x]);
                }
#pragma unroll
            for (int n2 = 0; n2 < HN / 2; ++n2) {
                uint32_t b[4];
                ldsm4t(b, smem_addr(Et) + tile_off<ROW>(16 * k4 + tr, d0 / 8 + 2 * n2 + tc));
                mma16816(y[2 * n2], fh, b[0], b[1]);
                mma16816(y[2 * n2 + 1], fh, b[2], b[3]);
                mma16816(y[2 * n2], fl, b[0], b[1]);
                mma16816(y[2 * n2 + 1], fl, b[2], b[3]);
            }
        }
        const float *rho = a.rho + (size_t)blockIdx.x * D + d0 + 2 * c;
#pragma unroll
        for (int n = 0; n < HN; ++n) {
            const float2 x = *reinterpret_cast<const float2 *>(rho + 8 * n);
            y[n][0] += x.x; y[n][1] += x.y; y[n][2] += x.x; y[n][3] += x.y;
        }
    }
    if (a.dq_add) {
#pragma unroll
        for (int n = 0; n < HN; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = m0 + g + 8 * x;
                if (t >= w.cnt) continue;
                const float2 f = *reinterpret_cast<const float2 *>(a.dq_add + (row0 + t) * D + d0 + 8 * n + 2 * c);
                dq[n][2 * x] += f.x;
                dq[n][2 * x + 1] += f.y;
            }
    }
    // out through this warp's own part of two tiles
#pragma unroll
    for (int n = 0; n < HN; n += 2) {
        const uint32_t o = tile_off<ROW>(m0 + (lane & 15), d0 / 8 + n + (lane >> 4));
        stsm4(smem_addr(Qt) + o, pack2(dq[n][0], dq[n][1]), pack2(dq[n][2], dq[n][3]), pack2(dq[n + 1][0], dq[n + 1][1]),
              pack2(dq[n + 1][2], dq[n + 1][3]));
        stsm4(smem_addr(Kt) + o, pack2(y[n][0], y[n][1]), pack2(y[n][2], y[n][3]), pack2(y[n + 1][0], y[n + 1][1]),
              pack2(y[n + 1][2], y[n + 1][3]));
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < 16 * (HD / 8) / 32; ++x) {
        const int e = x * 32 + lane, r = m0 + e / (HD / 8), pc = d0 / 8 + e % (HD / 8);
        if (r < w.cnt) {
            *reinterpret_cast<uint4 *>(a.dq + (row0 + r) * D + pc * 8) = *reinterpret_cast<const uint4 *>(Qt + tile_off<ROW>(r, pc));
            *reinterpret_cast<uint4 *>(a.dk + (row0 + r) * D + pc * 8) = *reinterpret_cast<const uint4 *>(Kt + tile_off<ROW>(r, pc));
        }
    }
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
            r += rowf[t] + rowf[kCH + t];
#pragma unroll
            for (int q = 0; q < 8; ++q) r -= colf[q * kCH + t];
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
        const float end = expf(ce) * in + fr;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (i + x >= w.cnt) continue;
            const float h = end + s - (x ? h0 : 0.f);
            a.dla[row0 + i + x] = __float2bfloat16_rn(w.ch == 0 && i + x == 0 ? 0.f : h);  // the first decay meets an empty memory
            a.dbe[row0 + i + x] = __float2bfloat16_rn(rowsum[i + x] + rowsum[kCH + i + x]);
        }
    }
}

template <int D, int NW>
cudaError_t rwalk_launch(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    constexpr int smem = RWalkSmem<D, NW>::kTotal;
    auto kern = delta_rwalk_tc<D, NW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * p.N * (D / (16 * NW))), 32 * NW, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t grads_tc_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    cudaError_t e = rwalk_launch<D, 4>(p, a, s);
    if (e != cudaSuccess) return e;
    profile_after_kernel(s, "delta_rwalk_tc");
    constexpr int smem = GradSmem<D>::kTotal;
    auto kern = delta_grads_tc<D>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * p.N * a.NCH), kGradThreads, smem, s>>>(a);
    e = cudaGetLastError();
    profile_after_kernel(s, "delta_grads_tc");
    return e;
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

// dy_t . O_t per token (the gradient of the online gate): one warp per token.
__global__ void __launch_bounds__(256) delta_dgon(const __nv_bfloat16 *dy, const float *O, float *dgon, long long tokens, int d)
{
    const long long t = (long long)blockIdx.x * 8 + threadIdx.x / 32;
    if (t >= tokens) return;
    const int lane = threadIdx.x % 32;
    float s = 0.f;
    for (int i = 2 * lane; i < d; i += 64) {
        const uint32_t y = *reinterpret_cast<const uint32_t *>(dy + t * d + i);
        const float2 o = *reinterpret_cast<const float2 *>(O + t * d + i);
        s = fmaf(low_f(y), o.x, fmaf(high_f(y), o.y, s));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) dgon[t] = s;
}

template <int D, bool READ, bool REV>
cudaError_t prep_impl(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    const size_t smem = (READ || REV ? 2 : 1) * kCH * D * 2 + 3 * sizeof(float) * kCH * kAP;
    auto kern = delta_prep_tc<D, READ, REV>;
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
    cudaError_t e = a.rrec ? prep_impl<D, READ, true>(p, a, s) : prep_impl<D, READ, false>(p, a, s);
    if (e != cudaSuccess) return e;
    profile_after_kernel(s, "delta_prep_tc");
    e = walk_launch<D, 4, READ>(p, a, s);
    profile_after_kernel(s, "delta_walk_tc");
    return e;
}

}  // namespace

cudaError_t launch_delta_dgon(const Problem &p, const void *dy, const float *O_on, float *dgon, cudaStream_t s)
{
    const long long n = (long long)p.BH * p.L;
    delta_dgon<<<(unsigned)((n + 7) / 8), 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(dy), O_on, dgon, n, p.d);
    return cudaGetLastError();
}

cudaError_t launch_delta_grads_tc(const Problem &p, const DeltaTcArgs &a, cudaStream_t s)
{
    return p.d == 64 ? grads_tc_impl<64>(p, a, s) : grads_tc_impl<128>(p, a, s);
}

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
