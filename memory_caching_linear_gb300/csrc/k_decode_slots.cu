// k_decode_slots.cu -- one recurrent decoding step over a cache of memory slots: the gated delta
// memory, and eviction by accumulated gate weight.
//
// For the token at position t of segment s (t0 the segment's first token), per (b,h):
//   online:  e = v - a M k,  M <- a M + beta e k^T  (a = exp(log_alpha); without log_alpha and
//            beta the linear memory's e = v, a = beta = 1), M empty at t0
//   gates:   as mc_decode_step over the cached segments: the first s slots, or with eviction
//            every slot that holds a segment (slot_seg >= 0)
//   read:    y = g_on M q + sum_i g_i M_i q
//   mass:    mass_i += g_i (eviction only), rounded up or down so that small gates count in a large mass (add_mass)
//   at the segment's last token M and the mean key become a cached segment: in slot s, or with
//   eviction in the first empty slot, else in that of the segment with the least mass (this
//   token's weight included) among those that are not the `protect` newest; equal mass: the oldest.
//
// Row r of a memory is written by v_r and read into y_r alone, so a CTA takes 16 rows of one
// head and reads them from every memory: one launch, bound by the cached memories' bytes.  The
// CTAs of a head form a cluster; each works the gates out for itself (N dot products from L2, two
// orders of magnitude below its rows' bytes), and the first one writes the head's small state after
// all have read it.  Rows are read past the caches, four in flight for every lane group, and five CTAs share an SM:
// 128 heads, d = 128, 63 slots 94 us a token, 5.9 TB/s (a plain sum over the same bytes reads 5.6); deeper asynchronous
// copies through shared memory and four CTAs with more registers were slower.  One user, 4 heads, 5 slots, d = 64: 4.3 us.
#include <cfloat>
#include <cstdint>

#include "mc_internal.cuh"

namespace mc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;   // rows per CTA
constexpr int kMaxN = 64;   // slots

__device__ __forceinline__ float4 fma4(float s, const float4 &a, const float4 &b)
{
    return make_float4(fmaf(s, a.x, b.x), fmaf(s, a.y, b.y), fmaf(s, a.z, b.z), fmaf(s, a.w, b.w));
}
__device__ __forceinline__ float dot4(const float4 &a, const float4 &b)
{
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}

// m + g for a sum without end.  To the nearest fp32, a gate below half a unit in the last place would add nothing from some
// mass on (0.004 at 65536), and the ranking would go by what was lost.  So the sum goes to the fp32 below it or above it:
// above if its distance from the one below, in units, exceeds r.  With r the multiples of the golden ratio modulo 1, which are
// spread as evenly as a sequence can be, the sum of n gates is a few units off, not n halves.  r is a function of the
// position alone, so that runs repeat and equal masses with equal gates stay equal.
__device__ __forceinline__ float add_mass(float m, float g, float r)
{
    const float s = m + g, b = s - m, e = (m - (s - b)) + (g - b);  // m + g = s + e exactly
    if (!(e != 0.f) || !(s < FLT_MAX)) return s;
    const float o = __int_as_float(__float_as_int(s) + (e > 0.f ? 1 : -1));  // the fp32 on the other side of m + g (s > 0)
    const float up = e / (o - s);  // how far towards it
    return e > 0.f ? (up > r ? o : s) : (1.f - up > r ? s : o);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 5) decode_slots(SlotArgs a)
{
    constexpr int LPR = D / 4;                   // lanes per row (a 16-byte piece each)
    constexpr int RPW = 32 / LPR;                // rows of a warp at once
    constexpr int SPLIT = kWarps * RPW / kRows < 1 ? 1 : kWarps * RPW / kRows;  // warps that share a row, by memories
    constexpr int PASS = kRows * SPLIT / (kWarps * RPW);                        // rows of a warp one after the other
    const int bh = (int)blockIdx.x / (D / kRows), rb = (int)blockIdx.x % (D / kRows);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const bool evict = a.mass != nullptr, delta = a.la != nullptr;
    const int s = a.t / a.C, t0 = s * a.C;
    const bool seg_start = a.t == t0, seg_end = a.t - t0 == a.C - 1;
    const int n = evict ? a.nmax : s;  // slots looked at
    const bool routed = a.mode == MC_GRM || a.mode == MC_SSC;
    __shared__ __align__(16) float qs[D], ks[D], us[D], ps[D];
    __shared__ float sc[kMaxN + 1], gv[kMaxN];
    __shared__ int gi[kMaxN], ids[kMaxN];
    __shared__ float g_on, red[kRows][kWarps];
    __shared__ int n_list, put;

    // This warp's rows, and its share of the memories where several warps share a row.  Every slot is read in its
    // order, the first four already while the gates are worked out, unless the router keeps a few only.
    const int part = SPLIT == 1 ? 0 : (warp * RPW) / kRows;
    const int rl0 = SPLIT == 1 ? warp * RPW * PASS + lane / LPR : (warp * RPW) % kRows + lane / LPR;
    const float4 *st = reinterpret_cast<const float4 *>(a.states + ((size_t)bh * a.nmax * D + rb * kRows + rl0) * D) + lane % LPR;
    const bool all = a.mode != MC_SSC;
    float4 m4[4];
    if (all && part + 3 * SPLIT < n) {
#pragma unroll
        for (int y = 0; y < 4; ++y) m4[y] = __ldcs(st + (size_t)(part + y * SPLIT) * (D * D / 4));
    }

    for (int i = tid; i < D; i += kThreads) {
        const size_t at = (size_t)bh * D + i;
        qs[i] = to_f(static_cast<const T *>(a.q)[at]);
        ks[i] = to_f(static_cast<const T *>(a.k)[at]);
        us[i] = routed ? to_f(static_cast<const T *>(a.u)[at]) : 0.f;
        ps[i] = (seg_start ? 0.f : a.ksum[at]) + ks[i];
    }
    for (int i = tid; i < n; i += kThreads) ids[i] = evict ? a.slot_seg[(size_t)bh * a.nmax + i] : i;
    __syncthreads();
    if (routed) {  // scores: LPR lanes per key mean, the online one last
        const float4 uv = reinterpret_cast<const float4 *>(us)[lane % LPR];
        const float *kb = a.kbar + (size_t)bh * a.nmax * D;
#pragma unroll 4
        for (int i0 = warp * RPW; i0 <= n; i0 += kWarps * RPW) {
            const int i = i0 + lane / LPR;
            float p = 0.f;
            if (i < n) p = dot4(uv, reinterpret_cast<const float4 *>(kb + (size_t)i * D)[lane % LPR]);
            else if (i == n) p = dot4(uv, reinterpret_cast<const float4 *>(ps)[lane % LPR]);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
            if (lane % LPR == 0 && i <= n) sc[i] = i < n ? p : p / (float)(a.t - t0 + 1);
        }
        __syncthreads();
    }
    if (warp == 0) {  // gates: slots lane and lane + 32 on each lane
        const int i0 = lane, i1 = lane + 32;
        const bool v0 = i0 < n && ids[i0] >= 0, v1 = i1 < n && ids[i1] >= 0;
        bool c0 = v0, c1 = v1;
        float g0 = 1.f, g1 = 1.f, go = 1.f;
        if (routed) {
            const float r0 = v0 ? sc[i0] : -FLT_MAX, r1 = v1 ? sc[i1] : -FLT_MAX, ron = sc[n];
            const int held = __popc(__ballot_sync(0xffffffffu, v0)) + __popc(__ballot_sync(0xffffffffu, v1));
            if (a.mode == MC_SSC && a.topk < held) {  // the topk largest; equal scores: the older segment
                c0 = c1 = false;
                for (int r = 0; r < a.topk; ++r) {
                    const bool f0 = v0 && !c0, f1 = v1 && !c1;
                    const bool second = f1 && (!f0 || r1 > r0 || (r1 == r0 && ids[i1] < ids[i0]));
                    float bv = second ? r1 : r0;
                    int bi = second ? i1 : i0, bs = f0 || f1 ? ids[second ? i1 : i0] : 0x7fffffff;
                    if (!f0 && !f1) bv = -FLT_MAX;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
                        const int oi = __shfl_xor_sync(0xffffffffu, bi, o), os = __shfl_xor_sync(0xffffffffu, bs, o);
                        if (ov > bv || (ov == bv && os < bs)) { bv = ov; bi = oi; bs = os; }
                    }
                    bi = __shfl_sync(0xffffffffu, bi, 0);
                    if (bi == i0) c0 = v0;
                    if (bi == i1) c1 = v1;
                }
            }
            float m = fmaxf(ron, fmaxf(c0 ? r0 : -FLT_MAX, c1 ? r1 : -FLT_MAX));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            g0 = c0 ? expf(r0 - m) : 0.f;
            g1 = c1 ? expf(r1 - m) : 0.f;
            go = expf(ron - m);
            float z = g0 + g1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            const float inv = 1.f / (z + go);
            g0 *= inv;
            g1 *= inv;
            go *= inv;
        } else if (a.mode == MC_MEAN) {
            g0 = g1 = go = 1.f / (float)(s + 1);
        }
        const unsigned b0 = __ballot_sync(0xffffffffu, c0), b1 = __ballot_sync(0xffffffffu, c1);
        const unsigned below = (1u << lane) - 1;
        if (all) {
            gv[i0] = c0 ? g0 : 0.f;
            gv[i1] = c1 ? g1 : 0.f;
        } else if (c0) {
            gv[__popc(b0 & below)] = g0;
            gi[__popc(b0 & below)] = i0;
        }
        if (!all && c1) {
            const int at = __popc(b0) + __popc(b1 & below);
            gv[at] = g1;
            gi[at] = i1;
        }
        int where = s;
        if (evict) {
            float *mass = a.mass + (size_t)bh * a.nmax;
            const float r = (float)((unsigned)a.t * 2654435769u >> 8) * 0x1p-24f;  // 2^32 / golden ratio
            const float m0 = i0 < n ? add_mass(mass[i0], c0 ? g0 : 0.f, r) : 0.f, m1 = i1 < n ? add_mass(mass[i1], c1 ? g1 : 0.f, r) : 0.f;
            sc[lane] = m0;  // the head's new masses (the scores are spent)
            if (i1 < n) sc[i1] = m1;
            if (seg_end) {
                // in order of: empty, not protected, protected; then the mass; then the age
                auto rank_of = [&](int i, bool v) { return i >= n ? 3 : !v ? 0 : ids[i] < s - a.protect ? 1 : 2; };
                const int k0 = rank_of(i0, v0), k1 = rank_of(i1, v1);
                const int d0 = i0 < n ? ids[i0] : 0, d1 = i1 < n ? ids[i1] : 0;
                const bool second = k1 < k0 || (k1 == k0 && k0 != 0 && k0 != 3 && (m1 < m0 || (m1 == m0 && d1 < d0)));
                int bk = second ? k1 : k0, bi = second ? i1 : i0, bd = second ? d1 : d0;
                float bm = second ? m1 : m0;
                if (bk == 0) {  // empty slots: the first one
                    bm = 0.f;
                    bd = bi;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const int ok = __shfl_xor_sync(0xffffffffu, bk, o), oi = __shfl_xor_sync(0xffffffffu, bi, o);
                    const int od = __shfl_xor_sync(0xffffffffu, bd, o);
                    const float om = __shfl_xor_sync(0xffffffffu, bm, o);
                    if (ok < bk || (ok == bk && (om < bm || (om == bm && od < bd)))) { bk = ok; bi = oi; bd = od; bm = om; }
                }
                where = __shfl_sync(0xffffffffu, bi, 0);
                where = where < n ? where : 0;
            }
        }
        if (lane == 0) {
            g_on = go;
            n_list = all ? n : __popc(b0) + __popc(b1);
            put = where;
        }
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA has read the head's key sum, key means, masses and slots

    // the rows
    const int nl = n_list;
    const float4 qv = reinterpret_cast<const float4 *>(qs)[lane % LPR];
    const float4 kv = reinterpret_cast<const float4 *>(ks)[lane % LPR];
    const float dec = delta ? delta_decay(to_f(static_cast<const T *>(a.la)[bh])) : 1.f;
    const float bet = delta ? to_f(static_cast<const T *>(a.be)[bh]) : 1.f;
    float4 on[PASS];
#pragma unroll
    for (int x = 0; x < PASS; ++x) {
        const int rl = rl0 + x * RPW, r = rb * kRows + rl;
        float acc = 0.f;
        if (part == 0) {
            float4 *row = reinterpret_cast<float4 *>(a.online + ((size_t)bh * D + r) * D) + lane % LPR;
            float e = to_f(static_cast<const T *>(a.v)[(size_t)bh * D + r]);
            float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!seg_start) {
                m = *row;
                m = make_float4(dec * m.x, dec * m.y, dec * m.z, dec * m.w);
            }
            if (delta) {
                float p = dot4(m, kv);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
                e = bet * (e - p);
            }
            m = fma4(e, kv, m);
            *row = m;
            on[x] = m;
            acc = g_on * dot4(m, qv);
        }
        const float4 *src = st + x * RPW * (D / 4);
        // an empty slot's gate is 0 and its memory anything, so a gate of 0 is not multiplied
        auto add = [&](int j, const float4 &m) {
            const float gj = gv[j];
            if (gj != 0.f) acc = fmaf(gj, dot4(m, qv), acc);
        };
        int j = part;
        for (; j + 3 * SPLIT < nl; j += 4 * SPLIT) {  // four rows in flight
            if (!(all && x == 0 && j == part)) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int i = j + y * SPLIT;
                    m4[y] = __ldcs(src + (size_t)(all ? i : gi[i]) * (D * D / 4));
                }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) add(j + y * SPLIT, m4[y]);
        }
        for (; j < nl; j += SPLIT) add(j, __ldcs(src + (size_t)(all ? j : gi[j]) * (D * D / 4)));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane % LPR == 0) red[rl][part] = acc;
    }
    __syncthreads();  // every read of the cached rows is done: the new segment may take a slot's place
    if (tid < kRows) {
        float y = red[tid][0];
#pragma unroll
        for (int p = 1; p < SPLIT; ++p) y += red[tid][p];
        static_cast<T *>(a.y)[(size_t)bh * D + rb * kRows + tid] = from_f<T>(y);
    }
    if (seg_end && part == 0) {
#pragma unroll
        for (int x = 0; x < PASS; ++x) {
            const int r = rb * kRows + rl0 + x * RPW;
            reinterpret_cast<float4 *>(a.states + (((size_t)bh * a.nmax + put) * D + r) * D)[lane % LPR] = on[x];
        }
    }
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (rb == 0) {
        for (int i = tid; i < D; i += kThreads) {
            a.ksum[(size_t)bh * D + i] = ps[i];
            if (seg_end) a.kbar[((size_t)bh * a.nmax + put) * D + i] = ps[i] / (float)a.C;
        }
        if (evict && tid < n) {
            const bool fresh = seg_end && tid == put;
            a.mass[(size_t)bh * a.nmax + tid] = fresh ? 0.f : sc[tid];
            if (fresh) a.slot_seg[(size_t)bh * a.nmax + tid] = s;
        }
    }
}

template <typename T, int D>
cudaError_t slots_impl(const SlotArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.BH * (D / kRows)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = D / kRows;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_slots<T, D>, a);
}

}  // namespace

cudaError_t launch_decode_slots(const SlotArgs &a, cudaStream_t s)
{
    switch (a.d) {
    case 16: return a.bf16 ? slots_impl<__nv_bfloat16, 16>(a, s) : slots_impl<float, 16>(a, s);
    case 32: return a.bf16 ? slots_impl<__nv_bfloat16, 32>(a, s) : slots_impl<float, 32>(a, s);
    case 64: return a.bf16 ? slots_impl<__nv_bfloat16, 64>(a, s) : slots_impl<float, 64>(a, s);
    case 128: return a.bf16 ? slots_impl<__nv_bfloat16, 128>(a, s) : slots_impl<float, 128>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mc
