// k_compact.cu -- from a prefill of many segments to a decoding cache of a few slots: the gate
// weight that every cached segment gathered over the prefill, the segments that are kept, and
// their move into the cache.
//
//   mass_i = sum over the tokens t of the later segments of g_{t,i}, with mc_forward's gates:
//            softmax over <u_t, kbar_i> (i < s_t; SSC: the topk largest) and the online score.
// Kept are the `protect` newest complete segments and, of the others, those with the most mass
// (equal mass: the newer), in order of time; the last, incomplete segment becomes the online memory.
//
// Kernels: the pooled-key sums (k_delta_simt.cu), gate_mass (per tile of 64 or 128 tokens, the gates and their
// sums over the tile's tokens), mass_reduce (the tiles' sums in a fixed order), compact_select (per head, the
// ranking), compact_gather (copies, bound by HBM).  Partial sums instead of atomics keep the mass,
// and with it the choice, the same from run to run.  A head has at most 512 of them (and no more than a state has
// numbers): row r of `part` takes tile tiles - shares + r and every shares-th one before it, summed in that order, so the
// scratch grows with the number of segments alone; up to 32768 tokens (65536 in gate_mass_tc; half of that
// for d = 16) a row is a tile.
#include <cfloat>
#include <cstdint>

#include "mc_internal.cuh"
#include "mma_sync.cuh"

namespace mc {
namespace {

constexpr int kMT = 64;   // tokens per tile
constexpr int kMS = 64;   // segments per block of scores
constexpr int kMThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kMThreads) gate_mass_simt(CompactArgs a)
{
    constexpr int P = D + 4;  // rows stay 16-byte aligned; eight rows apart by 4 words touch every bank
    extern __shared__ float sm[];
    float *Us = sm;               // kMT x P
    float *Kb = Us + kMT * P;     // kMS x P
    float *Sc = Kb + kMS * P;     // kMT x (kMS + 1)
    float *mx = Sc + kMT * (kMS + 1), *zs = mx + kMT, *thr = zs + kMT;
    int *thi = reinterpret_cast<int *>(thr + kMT), *nsel = thi + kMT;
    float *selv = reinterpret_cast<float *>(nsel + kMT);            // SSC: kMT x topk
    int *seli = reinterpret_cast<int *>(selv + (size_t)kMT * a.topk);
    const int last = a.tiles - a.shares + (int)blockIdx.x % a.shares, bh = (int)blockIdx.x / a.shares;
    const size_t base = (size_t)bh * a.L * D;
    const T *u = static_cast<const T *>(a.u) + base;
    const float *kbar = a.kbar_all + (size_t)bh * a.N * D;
    float *out = a.part + (size_t)blockIdx.x * a.N;
    const int tid = threadIdx.x;
    for (int tile = last; tile >= 0; tile -= a.shares) {
        const bool first = tile == last;  // (a tile reads no segment that a later one does not)
        const int tb = tile * kMT, cnt = min(kMT, a.L - tb);
        const int smax = (tb + cnt - 1) / a.C;  // the newest segment in the tile: segments before it are read
        __syncthreads();
        for (int e = tid; e < kMT * D; e += kMThreads)
            Us[(e / D) * P + e % D] = e / D < cnt ? to_f(u[(size_t)tb * D + e]) : 0.f;
        const bool ssc = a.mode == MC_SSC;
        if (tid < kMT) {
            mx[tid] = tid < cnt ? a.r_on[(size_t)bh * a.L + tb + tid] : 0.f;
            zs[tid] = 1.f;
            nsel[tid] = 0;
        }
        // Four tokens (tx + 16 x) by four segments (ty + 16 y) per thread, each score in gate_score's order of sums, so that
        // the router ranks as everywhere else.  Columns past the last segment that the tile reads are left out.
        auto scores = [&](int s0) {
            __syncthreads();
            for (int e = tid; e < kMS * D; e += kMThreads)
                Kb[(e / D) * P + e % D] = s0 + e / D < smax ? kbar[(size_t)s0 * D + e] : 0.f;
            __syncthreads();
            const int tx = tid % 16, ty = tid / 16;
#pragma unroll 1
            for (int y = 0; y < 4; ++y) {
                const int i = ty + 16 * y;
                if (s0 + 16 * y >= smax) break;
                float p[4][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) p[x][0] = p[x][1] = p[x][2] = p[x][3] = 0.f;
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    const float4 kv = *reinterpret_cast<const float4 *>(Kb + i * P + c);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 uv = *reinterpret_cast<const float4 *>(Us + (tx + 16 * x) * P + c);
                        p[x][0] = fmaf(uv.x, kv.x, p[x][0]);
                        p[x][1] = fmaf(uv.y, kv.y, p[x][1]);
                        p[x][2] = fmaf(uv.z, kv.z, p[x][2]);
                        p[x][3] = fmaf(uv.w, kv.w, p[x][3]);
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) Sc[(tx + 16 * x) * (kMS + 1) + i] = (p[x][0] + p[x][1]) + (p[x][2] + p[x][3]);
            }
            __syncthreads();
        };
        for (int s0 = 0; s0 < smax; s0 += kMS) {
            scores(s0);
            if (tid < cnt) {
                const int n = min((tb + tid) / a.C - s0, kMS);  // cached segments of this token in the block
                if (ssc) {
                    int c = nsel[tid];
                    for (int i = 0; i < n; ++i)
                        topk_insert(selv + (size_t)tid * a.topk, seli + (size_t)tid * a.topk, c, a.topk, Sc[tid * (kMS + 1) + i], s0 + i);
                    nsel[tid] = c;
                } else {
                    float m = mx[tid], z = zs[tid];
                    for (int i = 0; i < n; ++i) {
                        const float r = Sc[tid * (kMS + 1) + i];
                        if (r > m) {
                            z = z * expf(m - r) + 1.f;
                            m = r;
                        } else {
                            z += expf(r - m);
                        }
                    }
                    mx[tid] = m;
                    zs[tid] = z;
                }
            }
        }
        if (ssc && tid < cnt) {
            const float ron = mx[tid];
            const int c = nsel[tid];
            const float *vals = selv + (size_t)tid * a.topk;
            float m = ron;
            if (c > 0) m = fmaxf(m, vals[0]);
            float z = expf(ron - m);
            for (int i = 0; i < c; ++i) z += expf(vals[i] - m);
            mx[tid] = m;
            zs[tid] = z;
            thr[tid] = c > 0 ? vals[c - 1] : FLT_MAX;  // a segment is selected if its score is above the last one's,
            thi[tid] = c > 0 ? seli[(size_t)tid * a.topk + c - 1] : -1;  // or equal with an index up to it
        }
        __shared__ float part[4][kMS];
        for (int s0 = 0; s0 < smax; s0 += kMS) {
            if (smax > kMS) scores(s0);  // a single block's scores are still there
            else __syncthreads();
            const int q = tid / kMS, i = s0 + tid % kMS;  // a quarter of the tokens
            float sum = 0.f;
            if (i < smax)
                for (int t = q * (kMT / 4); t < min(cnt, (q + 1) * (kMT / 4)); ++t) {
                    if (i >= (tb + t) / a.C) continue;
                    const float r = Sc[t * (kMS + 1) + tid % kMS];
                    if (ssc && !(r > thr[t] || (r == thr[t] && i <= thi[t]))) continue;
                    sum += expf(r - mx[t]) / zs[t];
                }
            part[q][tid % kMS] = sum;
            __syncthreads();
            if (tid < kMS && s0 + tid < a.N) {
                const float x = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
                out[s0 + tid] = first ? x : out[s0 + tid] + x;
            }
        }
        if (first)
            for (int i = ((smax + kMS - 1) / kMS) * kMS + tid; i < a.N; i += kMThreads) out[i] = 0.f;
    }
}

// ---------------------------------------------------------------------------
// gate_mass_tc: the same for bf16 inputs and the softmax gates.  A CTA takes 128 tokens, a warp 16; the scores
// against 32 segments at a time are warp-level products of u with the key means as three bf16 terms
// (launch_kbar_images: every product is exact, only the fp32 sum rounds), the next 32 segments' means on their way
// meanwhile.  Up to 128 segments the scores stay in registers between the softmax's sums and the gates; beyond, they are
// formed a second time.  16 heads of 65536 tokens, 128 segments, d = 128: 222 us (gate_mass_simt 7.2 ms); the products alone
// would take 90 us and the matrix loads in front of them, one for every two, 87 us of shared memory's time.  256 tokens
// and 16 warps per CTA halve the key means' way through L2 and are slower, 259 us: one CTA on an SM waits at its barriers.
// ---------------------------------------------------------------------------
constexpr int kTM = 128;

template <int D>
struct MassSmem {
    static constexpr int PN = D > 64 ? 2 : 1;                   // 64-column panels
    static constexpr int UR = D * 2 < 128 ? 128 : D * 2;        // row of the token tile
    static constexpr int kHalf = 3 * PN * 32 * 128;             // three terms of 32 segments
    static constexpr int kTotal = kTM * UR + 2 * kHalf;
};

template <int D>
__global__ void __launch_bounds__(256, 2) gate_mass_tc(CompactArgs a)
{
    using namespace mma;
    using M = MassSmem<D>;
    constexpr int KS = D / 16, PN = M::PN, UR = M::UR;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *Ut = smem_raw, *Kt = smem_raw + kTM * UR;
    __shared__ float cols[8][32];
    const int row = a.shares - 1 - (int)(blockIdx.x / a.BH), bh = (int)(blockIdx.x % a.BH);  // the longest first
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
    const __nv_bfloat16 *u = static_cast<const __nv_bfloat16 *>(a.u);
    float *out = a.part + ((size_t)bh * a.shares + row) * a.N;
    for (int tile = a.tiles - a.shares + row; tile >= 0; tile -= a.shares) {
        const bool first = tile == a.tiles - a.shares + row;  // (a tile reads no segment that a later one does not)
        const int tb = tile * kTM, cnt = min(kTM, a.L - tb);
        const int smax = (tb + cnt - 1) / a.C, nh = (smax + 31) / 32;
        const size_t row0 = (size_t)bh * a.L + tb;
        if (first)
            for (int i = nh * 32 + tid; i < a.N; i += 256) out[i] = 0.f;
        if (nh == 0) break;  // (nor do the tiles before it read any)
        if (!first) __syncthreads();
        const uint8_t *img = a.kbar_img + (size_t)bh * ((a.N + 63) / 64) * 49152;
        int it = 0;  // loads so far: half h goes to buffer it % 2
        auto issue = [&](int h) {
            const uint32_t dst = smem_addr(Kt) + (it & 1) * M::kHalf;
            const uint8_t *src = img + (size_t)(h / 2) * 49152 + (h & 1) * 32 * 128;
            for (int e = tid; e < 3 * PN * 256; e += 256) {
                const int tp = e / 256, r = e % 256;  // term and panel; 16-byte piece
                cp16(dst + e * 16, src + (tp / PN) * 16384 + (tp % PN) * 8192 + r * 16, true);
            }
            cp_commit();
            ++it;
        };
        for (int e = tid; e < kTM * (D / 8); e += 256) {
            const int r = e / (D / 8), pc = e % (D / 8);
            cp16(smem_addr(Ut) + tile_off<UR>(r, pc), u + (row0 + (r < cnt ? r : 0)) * D + pc * 8, r < cnt);
        }
        issue(0);
        // rows g and g + 8 of the warp's tokens: cached segments, online score
        const int t0 = 16 * warp + g, t1 = t0 + 8;
        const int lim0 = t0 < cnt ? (tb + t0) / a.C : 0, lim1 = t1 < cnt ? (tb + t1) / a.C : 0;
        float m0 = t0 < cnt ? a.r_on[row0 + t0] : 0.f, m1 = t1 < cnt ? a.r_on[row0 + t1] : 0.f, z0 = c == 0 ? 1.f : 0.f, z1 = z0;
        uint32_t au[KS][4];

        // Half h's scores, -inf where a token does not read the segment; `next` is loaded meanwhile (-1: nothing).
        auto scores = [&](int h, int next, float (&S)[4][4]) {
            cp_wait<0>();
            __syncthreads();  // the half has come, and the other buffer has been read
            const uint32_t kt = smem_addr(Kt) + ((it - 1) & 1) * M::kHalf;
            if (it == 1) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    ldsm4(au[ks], smem_addr(Ut) + tile_off<UR>(16 * warp + (lane & 15), 2 * ks + (lane >> 4)));
            }
            if (next >= 0) issue(next);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[n][e] = 0.f;
            const int br = (lane >> 4) * 8 + (lane & 7), bc = (lane >> 3) & 1;
#pragma unroll
            for (int term = 2; term >= 0; --term)  // the small terms first
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int n2 = 0; n2 < 2; ++n2) {
                        if (32 * h + 16 * n2 >= smax) break;
                        uint32_t bf[4];
                        ldsm4(bf, kt + (term * PN + ks / 4) * 4096 + tile_off<128>(16 * n2 + br, 2 * (ks & 3) + bc));
                        mma16816(S[2 * n2], au[ks], bf[0], bf[1]);
                        mma16816(S[2 * n2 + 1], au[ks], bf[2], bf[3]);
                    }
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (32 * h + 8 * n + 2 * c + (e & 1) >= (e >> 1 ? lim1 : lim0)) S[n][e] = -INFINITY;
        };
        auto softmax = [&](const float (&S)[4][4]) {  // running maximum and sum (each lane its own columns)
            float x0 = m0, x1 = m1;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                x0 = fmaxf(x0, fmaxf(S[n][0], S[n][1]));
                x1 = fmaxf(x1, fmaxf(S[n][2], S[n][3]));
            }
            z0 *= __expf(m0 - x0);
            z1 *= __expf(m1 - x1);
            m0 = x0;
            m1 = x1;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                z0 += __expf(S[n][0] - m0) + __expf(S[n][1] - m0);
                z1 += __expf(S[n][2] - m1) + __expf(S[n][3] - m1);
            }
        };
        auto join = [&]() {  // the four lanes of a row
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const float y0 = __shfl_xor_sync(0xffffffffu, m0, o), y1 = __shfl_xor_sync(0xffffffffu, m1, o);
                const float w0 = __shfl_xor_sync(0xffffffffu, z0, o), w1 = __shfl_xor_sync(0xffffffffu, z1, o);
                const float x0 = fmaxf(m0, y0), x1 = fmaxf(m1, y1);
                z0 = z0 * __expf(m0 - x0) + w0 * __expf(y0 - x0);
                z1 = z1 * __expf(m1 - x1) + w1 * __expf(y1 - x1);
                m0 = x0;
                m1 = x1;
            }
            z0 = 1.f / z0;
            z1 = 1.f / z1;
        };
        auto gates = [&](int h, const float (&S)[4][4]) {  // sums over the tile's tokens
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float s0 = __expf(S[n][0] - m0) * z0 + __expf(S[n][2] - m1) * z1;
                float s1 = __expf(S[n][1] - m0) * z0 + __expf(S[n][3] - m1) * z1;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                }
                if (g == 0) {
                    cols[warp][8 * n + 2 * c] = s0;
                    cols[warp][8 * n + 2 * c + 1] = s1;
                }
            }
            __syncthreads();
            if (tid < 32 && 32 * h + tid < a.N) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) s += cols[w][tid];
                out[32 * h + tid] = first ? s : out[32 * h + tid] + s;
            }
            __syncthreads();
        };
        if (nh <= 4) {
            float S[4][4][4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (h < nh) {
                    scores(h, h + 1 < nh ? h + 1 : -1, S[h]);
                    softmax(S[h]);
                }
            join();
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (h < nh) gates(h, S[h]);
        } else {
            float S[4][4];
            for (int h = 0; h < nh; ++h) {
                scores(h, h + 1 < nh ? h + 1 : 0, S);
                softmax(S);
            }
            join();
            for (int h = 0; h < nh; ++h) {
                scores(h, h + 1 < nh ? h + 1 : -1, S);
                gates(h, S);
            }
        }
    }
}

// mass_i: the rows' sums, 32 strided shares of the rows, joined in a fixed order.
__global__ void __launch_bounds__(1024) mass_reduce(CompactArgs a)
{
    __shared__ float part[32][33];
    const int blocks = (a.N + 31) / 32, bh = (int)blockIdx.x / blocks, lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const int i = ((int)blockIdx.x % blocks) * 32 + lane;
    float s = 0.f;
    if (i < a.N) {
        const float *p = a.part + (size_t)bh * a.shares * a.N + i;
        // no token before the segment's end reads it: the first row with a tile that does
        int t = max(0, (int)((long long)(i + 1) * a.C / a.tile_len) - (a.tiles - a.shares));
        t += (w - t % 32 + 32) % 32;
#pragma unroll 4
        for (; t < a.shares; t += 32) s += p[(size_t)t * a.N];
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && i < a.N) {
#pragma unroll
        for (int x = 1; x < 32; ++x) s += part[x][lane];
        a.mass_all[(size_t)bh * a.N + i] = s;
    }
}

// One CTA per head: which complete segments are kept.
// order[bh][slot] is the segment of each slot, -1 for an empty one.
__global__ void __launch_bounds__(kMThreads) compact_select(CompactArgs a)
{
    extern __shared__ float ms[];  // N masses, then N flags
    int *kept = reinterpret_cast<int *>(ms + a.N);
    __shared__ int total;
    const int bh = (int)blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    for (int i = tid; i < a.N; i += kMThreads) {
        ms[i] = a.mass_all[(size_t)bh * a.N + i];
    }
    __syncthreads();
    const int done = a.done, nkeep = min(a.nmax, done), loose = done - a.protect;  // segments below `loose` compete
    for (int i = warp; i < done; i += kMThreads / 32) {  // how many competitors go before segment i
        int before = 0;
        for (int j = lane; j < loose; j += 32) before += ms[j] < ms[i] || (ms[j] == ms[i] && j < i) ? 1 : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (lane == 0) kept[i] = i >= loose || before >= done - nkeep;
    }
    __syncthreads();
    int32_t *order = a.order + (size_t)bh * a.nmax;
    for (int i = tid; i < done; i += kMThreads) {
        if (!kept[i]) continue;
        int slot = 0;
        for (int j = 0; j < i; ++j) slot += kept[j];
        if (slot >= a.nmax) continue;  // (masses that are not numbers)
        order[slot] = i;
        a.mass[(size_t)bh * a.nmax + slot] = ms[i];
    }
    if (tid == 0) total = 0;
    __syncthreads();
    int n = 0;
    for (int j = tid; j < done; j += kMThreads) n += kept[j];
    if (n) atomicAdd(&total, n);
    __syncthreads();
    for (int s = min(total, a.nmax) + tid; s < a.nmax; s += kMThreads) {
        order[s] = -1;
        a.mass[(size_t)bh * a.nmax + s] = 0.f;
    }
}

// One CTA per (head, slot or the online memory): the state, key mean and segment id of a slot; empty
// slots and an absent online memory are zeroed.
__global__ void __launch_bounds__(kMThreads) compact_gather(CompactArgs a)
{
    const int slot = (int)blockIdx.x % (a.nmax + 1), bh = (int)blockIdx.x / (a.nmax + 1), tid = threadIdx.x;
    const int d = a.d, dd4 = d * d / 4;
    const bool online = slot == a.nmax;
    const int seg = online ? (a.done < a.N ? a.N - 1 : -1) : a.order[(size_t)bh * a.nmax + slot];
    float4 *dst = reinterpret_cast<float4 *>(online ? a.online + (size_t)bh * d * d
                                                    : a.states + ((size_t)bh * a.nmax + slot) * d * d);
    const float4 *src = reinterpret_cast<const float4 *>(a.states_all + ((size_t)bh * a.N + (seg < 0 ? 0 : seg)) * d * d);
    if (seg >= 0) {
#pragma unroll 4
        for (int i = tid; i < dd4; i += kMThreads) dst[i] = __ldcs(src + i);
    } else {
        for (int i = tid; i < dd4; i += kMThreads) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < d) {
        const float kb = seg >= 0 ? a.kbar_all[((size_t)bh * a.N + seg) * d + tid] : 0.f;
        if (online)
            a.ksum[(size_t)bh * d + tid] = kb * (float)(a.L - a.done * a.C);  // the sum behind the mean
        else
            a.kbar[((size_t)bh * a.nmax + slot) * d + tid] = kb;
    }
    if (tid == 0 && !online) a.slot_seg[(size_t)bh * a.nmax + slot] = seg;
}

template <typename T, int D>
cudaError_t mass_impl(const Problem &p, const CompactArgs &a, cudaStream_t s)
{
    const size_t smem = sizeof(float) * ((kMT + kMS) * (D + 4) + kMT * (kMS + 1) + 5 * kMT + 2 * (size_t)kMT * a.topk);
    auto kern = gate_mass_simt<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * a.shares), kMThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t mass_tc_impl(const Problem &p, const CompactArgs &a, cudaStream_t s)
{
    constexpr int smem = MassSmem<D>::kTotal;
    auto kern = gate_mass_tc<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * a.shares), 256, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

int gate_mass_tile(const Problem &p) { return p.bf16 && p.mode == MC_GRM ? kTM : kMT; }

cudaError_t launch_gate_mass(const Problem &p, const CompactArgs &a, cudaStream_t s)
{
    if (p.bf16 && p.mode == MC_GRM) {
        switch (p.d) {
        case 16: return mass_tc_impl<16>(p, a, s);
        case 32: return mass_tc_impl<32>(p, a, s);
        case 64: return mass_tc_impl<64>(p, a, s);
        case 128: return mass_tc_impl<128>(p, a, s);
        default: return cudaErrorInvalidValue;
        }
    }
    switch (p.d) {
    case 16: return p.bf16 ? mass_impl<__nv_bfloat16, 16>(p, a, s) : mass_impl<float, 16>(p, a, s);
    case 32: return p.bf16 ? mass_impl<__nv_bfloat16, 32>(p, a, s) : mass_impl<float, 32>(p, a, s);
    case 64: return p.bf16 ? mass_impl<__nv_bfloat16, 64>(p, a, s) : mass_impl<float, 64>(p, a, s);
    case 128: return p.bf16 ? mass_impl<__nv_bfloat16, 128>(p, a, s) : mass_impl<float, 128>(p, a, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_compact(const Problem &p, const CompactArgs &a, cudaStream_t s)
{
    const size_t smem = 2 * sizeof(float) * a.N;
    cudaError_t e = cudaFuncSetAttribute(compact_select, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    mass_reduce<<<(unsigned)((long long)p.BH * ((a.N + 31) / 32)), 1024, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    compact_select<<<(unsigned)p.BH, kMThreads, smem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    compact_gather<<<(unsigned)((long long)p.BH * (a.nmax + 1)), kMThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mc
