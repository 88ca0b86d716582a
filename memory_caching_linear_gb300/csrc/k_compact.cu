// k_compact.cu -- from a prefill of many segments to a decoding cache of a few slots: the gate
// weight that every cached segment gathered over the prefill, the segments that are kept, and
// their move into the cache.
//
//   mass_i = sum over the tokens t of the later segments of g_{t,i}, with mc_forward's gates:
//            softmax over <u_t, kbar_i> (i < s_t; SSC: the topk largest) and the online score.
// Kept are the `protect` newest complete segments and, of the others, those with the most mass
// (equal mass: the newer), in order of time; the last, incomplete segment becomes the online memory.
//
// Kernels: the pooled-key sums (k_delta_simt.cu), gate_mass (per 64-token tile, the gates and their
// sums over the tile's tokens), compact_select (per head: the tiles' sums in a fixed order, the
// ranking), compact_gather (copies, bound by HBM).  Partial sums instead of atomics keep the mass,
// and with it the choice, the same from run to run.
#include <cfloat>
#include <cstdint>

#include "mc_internal.cuh"

namespace mc {
namespace {

constexpr int kMT = 64;   // tokens per tile
constexpr int kMS = 64;   // segments per block of scores
constexpr int kMThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kMThreads) gate_mass_simt(CompactArgs a)
{
    constexpr int P = D + 1;
    extern __shared__ float sm[];
    float *Us = sm;               // kMT x P
    float *Kb = Us + kMT * P;     // kMS x P
    float *Sc = Kb + kMS * P;     // kMT x (kMS + 1)
    float *mx = Sc + kMT * (kMS + 1), *zs = mx + kMT, *thr = zs + kMT;
    int *thi = reinterpret_cast<int *>(thr + kMT), *nsel = thi + kMT;
    float *selv = reinterpret_cast<float *>(nsel + kMT);            // SSC: kMT x topk
    int *seli = reinterpret_cast<int *>(selv + (size_t)kMT * a.topk);
    const int tile = (int)blockIdx.x % a.tiles, bh = (int)blockIdx.x / a.tiles;
    const int tb = tile * kMT, cnt = min(kMT, a.L - tb);
    const int smax = (tb + cnt - 1) / a.C;  // the newest segment in the tile: segments before it are read
    const size_t base = (size_t)bh * a.L * D;
    const T *u = static_cast<const T *>(a.u) + base;
    const float *kbar = a.kbar_all + (size_t)bh * a.N * D;
    float *out = a.part + (size_t)blockIdx.x * a.N;
    const int tid = threadIdx.x;
    for (int e = tid; e < kMT * D; e += kMThreads)
        Us[(e / D) * P + e % D] = e / D < cnt ? to_f(u[(size_t)tb * D + e]) : 0.f;
    const bool ssc = a.mode == MC_SSC;
    if (tid < kMT) {
        mx[tid] = tid < cnt ? a.r_on[(size_t)bh * a.L + tb + tid] : 0.f;
        zs[tid] = 1.f;
        nsel[tid] = 0;
    }
    auto scores = [&](int s0) {
        __syncthreads();
        for (int e = tid; e < kMS * D; e += kMThreads)
            Kb[(e / D) * P + e % D] = s0 + e / D < smax ? kbar[(size_t)s0 * D + e] : 0.f;
        __syncthreads();
        for (int e = tid; e < kMT * kMS; e += kMThreads)
            Sc[(e / kMS) * (kMS + 1) + e % kMS] = gate_score(Us + (e / kMS) * P, Kb + (e % kMS) * P, D);
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
    for (int s0 = 0; s0 < smax; s0 += kMS) {
        scores(s0);
        if (tid < kMS && s0 + tid < a.N) {
            const int i = s0 + tid;
            float sum = 0.f;
            for (int t = 0; t < cnt; ++t) {
                if (i >= (tb + t) / a.C) continue;
                const float r = Sc[t * (kMS + 1) + tid];
                if (ssc && !(r > thr[t] || (r == thr[t] && i <= thi[t]))) continue;
                sum += expf(r - mx[t]) / zs[t];
            }
            out[i] = sum;
        }
    }
    for (int i = ((smax + kMS - 1) / kMS) * kMS + tid; i < a.N; i += kMThreads) out[i] = 0.f;
}

// One CTA per head: mass_i = the tiles' sums in order, then which complete segments are kept.
// order[bh][slot] is the segment of each slot, -1 for an empty one.
__global__ void __launch_bounds__(kMThreads) compact_select(CompactArgs a)
{
    extern __shared__ float ms[];  // N masses, then N flags
    int *kept = reinterpret_cast<int *>(ms + a.N);
    __shared__ int total;
    const int bh = (int)blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    for (int i = tid; i < a.N; i += kMThreads) {
        // four chains of tiles, joined in a fixed order
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const float *p = a.part + (size_t)bh * a.tiles * a.N + i;
        int t = (int)((long long)(i + 1) * a.C / kMT);  // no token before the segment's end reads it
        for (; t + 4 <= a.tiles; t += 4)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[x] += p[(size_t)(t + x) * a.N];
        for (; t < a.tiles; ++t) s[0] += p[(size_t)t * a.N];
        const float m = (s[0] + s[1]) + (s[2] + s[3]);
        ms[i] = m;
        if (a.mass_all) a.mass_all[(size_t)bh * a.N + i] = m;
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
    const size_t smem = sizeof(float) * ((kMT + kMS) * (D + 1) + kMT * (kMS + 1) + 5 * kMT + 2 * (size_t)kMT * a.topk);
    auto kern = gate_mass_simt<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * a.tiles), kMThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gate_mass(const Problem &p, const CompactArgs &a, cudaStream_t s)
{
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
    compact_select<<<(unsigned)p.BH, kMThreads, smem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    compact_gather<<<(unsigned)((long long)p.BH * (a.nmax + 1)), kMThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mc
