// k_step.cu -- one decoding step over a paged cache: a token for every sequence of the batch, each at its own position, in one
// launch without scratch.
//
// As in a tree's split read (k_tree_tc.cu) the memories of all heads and sequences form one line that is cut evenly over the
// SMs, each range weighing its cached memories against its own largest score, so sequences of unlike lengths keep every SM as
// busy as any.  The end of a head -- its online memory, and the scores of the next one -- takes as long as 1024 / d memories
// (512 KB at d = 128), and has that much room in the line, or the ranges with most ends would run on alone: 16 heads of
// d = 128, 16 sequences of 2 to 63 segments 120 -> 88 us, 32 of up to 10 93 -> 55.  The online memory is the last of its head's: whoever has it updates it (e = v - a M k, M <- a M + beta e k^T),
// writes it, and reads it.  Nothing waits for another CTA: the last one to come to a head's end joins the partial reads, in
// their order, and the last one of all moves positions on and gives out pages (a CTA that needs to know its page before
// looks it up as the last one will).
//
// The memories, 4 d^2 bytes each, come by bulk copies through a ring of 192 KB (d >= 64) and are read from there, a lane
// holding four columns of every row that it adds up.  HBM bounds a batch, a chain of loads (slot, row, position, page, mean
// key, memory) and two rounds of counting a single user.  16 heads of d = 128, bf16, gated delta: 8 sequences of up to 63
// segments 83 us a token (5.2 TB/s), one of 5 segments 12.5 and of 40 15.7.
#include <cfloat>
#include <cstdint>

#include "paged.cuh"
#include "sm100.cuh"

namespace mc {

using namespace sm100;

namespace {

__device__ int g_step_abort;

constexpr int kWorkers = 8, kThreads = 32 * (kWorkers + 1), kMaxStages = 24;

template <int D>
struct StepShape {
    static constexpr int BYTES = D * D * 4, STAGES = D == 128 ? 3 : D == 64 ? 12 : 24;
    static constexpr int LPR = D / 4, RPW = 32 / LPR, PASS = D / (kWorkers * RPW) < 1 ? 1 : D / (kWorkers * RPW);
};
// After the ring: seats (Line), slots' takers, and a head's scores and pages.
template <int D>
size_t step_smem(const TreeArgs &a)
{
    return 128 + (size_t)StepShape<D>::STAGES * StepShape<D>::BYTES + sizeof(int) * (Line::ints(a.B) + a.c.S + 2 * (size_t)a.c.nmax);
}

// The seats of a call that writes: a slot that several batch rows name is the first one's.
__device__ Line make_line_once(const TreeArgs &a, int *space, int *taker, bool tell)
{
    const Paged &c = a.c;
    const Line l = line_in(space, a.B);
    for (int r = threadIdx.x; r < c.S; r += blockDim.x) taker[r] = 0x7fffffff;
    __syncthreads();
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const Seat s = seat_of(a, b, tell);
        l.row[b] = s.row;
        l.pos[b] = s.pos;
        if (s.row >= 0) atomicMin(&taker[s.row], b);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int row = l.row[b];
        if (row >= 0 && taker[row] != b) {
            l.row[b] = -1;
            if (tell) atomicOr(c.status, MC_PAGES_INDEX);
        }
        l.units[b + 1] = l.row[b] >= 0 ? cached_segments(c, l.pos[b]) + 1 : 0;
    }
    sum_line(a, l);
    return l;
}

// Whether the sparse router keeps a memory: those up to the last that it chose, in order of score and age, or (kAll) every one.
constexpr int kAll = 0x7fffffff;
__device__ __forceinline__ bool keeps(float score, int i, float cut, int cut_at)
{
    return cut_at == kAll || score > cut || (score == cut && i <= cut_at);
}

// Whether row b's token completes a segment that the table has room for.
__device__ __forceinline__ bool wants_page(const Paged &c, const Line &l, int b)
{
    return l.row[b] >= 0 && l.pos[b] % c.C == c.C - 1 && l.pos[b] / c.C < c.nmax;
}

// The rank-th free page of the pool, -1 if there are fewer; one warp, 128 references a turn, from the first one: where a segment
// ends the pages in use before the lowest free one are looked through, for every head and once more at the call's end.  60
// sequences of one head, 32 of which end a segment: 41 -> 96 us with 4400 pages in use, 123 -> 819 with 49 400.
__device__ int free_page(const Paged &c, int rank)
{
    const int lane = threadIdx.x % 32;
    for (int p0 = 0; p0 < c.P; p0 += 128) {
        unsigned open[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int p = p0 + 32 * x + lane;
            open[x] = __ballot_sync(0xffffffffu, p < c.P && __ldcg(c.refs + p) == 0);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int n = __popc(open[x]);
            if (rank < n) return p0 + 32 * x + (int)__fns(open[x], 0, rank + 1);
            rank -= n;
        }
    }
    return -1;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1) step_paged(TreeArgs a, StepWork work)
{
    using S = StepShape<D>;
    constexpr int LPR = S::LPR, RPW = S::RPW, PASS = S::PASS, STAGES = S::STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    int *space = reinterpret_cast<int *>(raw + 128 + STAGES * S::BYTES), *taker = space + Line::ints(a.B);
    float *score = reinterpret_cast<float *>(taker + a.c.S);  // [nmax]
    int *page = reinterpret_cast<int *>(score + a.c.nmax);    // [nmax]
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], meet, chosen, issued;
    __shared__ int abort_flag, last, mine, cut_at;
    __shared__ float cut;
    const Paged &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWorkers);
        }
        mbar_init(&meet, kWorkers);
        mbar_init(&chosen, kWorkers);
        mbar_init(&issued, 1);
        fence_mbar_init();
    }
    after_previous();
    const Line line = make_line_once(a, space, taker, blockIdx.x == 0);
    const long long U = (long long)line.units[a.B] * c.H, R = ranges_of(U, a.ranges);
    // a CTA without a range counts at the end too: it has read positions, from which all must work out the same line
    const bool in = blockIdx.x < R;
    const long long begin = in ? range_begin(blockIdx.x, U, R) : 0, end = in ? range_begin(blockIdx.x + 1, U, R) : 0;
    const bool routed = a.mode == MC_GRM || a.mode == MC_SSC, sparse = a.mode == MC_SSC;

    if (warp == kWorkers) {
        if (lane > 0 && routed) {  // the range's mean keys, as far as L2: scores are wanted at once where a head begins
            int b = 0;
            for (long long x = begin + lane - 1; x < end; x += 31) {
                while (x >= (long long)line.units[b + 1] * c.H) ++b;
                const int nu = line.units[b + 1] - line.units[b];
                const int in_b = (int)(x - (long long)line.units[b] * c.H), h = in_b / nu, i = in_b % nu;
                const int p = i < cached_segments(c, line.pos[b]) ? valid_page(c, c.table[(size_t)line.row[b] * c.nmax + i]) : -1;
                if (p >= 0)
                    for (int y = 0; y < D * 4; y += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(c.kbar + ((size_t)p * c.H + h) * D + y / 4));
            }
        }
        if (lane == 0) {
            uint32_t g = 0, picks = 0;
            bool ok = true;
            int b = 0;
            for (long long x = begin; ok && x < end;) {
                while (x >= (long long)line.units[b + 1] * c.H) ++b;
                const int nu = line.units[b + 1] - line.units[b], nb = cached_segments(c, line.pos[b]), row = line.row[b], in0 = line.pos[b] % c.C;
                const int in_b = (int)(x - (long long)line.units[b] * c.H);
                const int h = in_b / nu, i0 = in_b % nu, i1 = min((int)(end - x < nu - i0 ? i0 + (end - x) : nu), nb + 1);
                x += (end - x < nu - i0 ? end - x : nu - i0);
                if (i0 > nb) continue;
                if (sparse && i0 < nb) {  // which of them the router keeps
                    if (!(ok = mbar_wait(&chosen, picks & 1, &abort_flag))) break;
                    ++picks;
                }
                int next = i0 < nb ? c.table[(size_t)row * c.nmax + i0] : 0;
                for (int i = i0; i < i1; ++i) {
                    const int p = next;
                    if (i + 1 < i1 && i + 1 < nb) next = c.table[(size_t)row * c.nmax + i + 1];
                    const float *src = c.online + ((size_t)row * c.H + h) * D * D;
                    if (i < nb) {
                        if (valid_page(c, p) < 0) continue;
                        if (sparse && !keeps(score[i], i, cut, cut_at)) continue;
                        src = c.pages + ((size_t)p * c.H + h) * D * D;
                    } else if (!in0) {
                        continue;
                    }
                    const uint32_t s = g % STAGES;
                    if (!(ok = mbar_wait(&empty[s], ((g / STAGES) & 1) ^ 1, &abort_flag))) break;
                    mbar_arrive_expect_tx(&full[s], S::BYTES);
                    constexpr int PIECE = S::BYTES < 16384 ? S::BYTES : 16384;
#pragma unroll
                    for (int y = 0; y < S::BYTES / PIECE; ++y)
                        bulk_load(ring + s * S::BYTES + y * PIECE, reinterpret_cast<const uint8_t *>(src) + y * PIECE, PIECE, &full[s]);
                    ++g;
                }
                if (sparse && i0 < nb) mbar_arrive(&issued);  // the scores may go
            }
            for (uint32_t x = g > (uint32_t)STAGES ? g - STAGES : 0; x < g; ++x) {  // no copy lands after the CTA has left
                int gave_up = 0;
                mbar_wait_limit(&full[x % STAGES], (x / STAGES) & 1, &gave_up, kWaitLimitNs);
            }
        }
        return;
    }

    // workers meet without the producer, and without waiting for ever
    uint32_t meetings = 0;
    auto gather = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&meet);
        return mbar_wait(&meet, meetings++ & 1, &abort_flag);
    };
    const int c0 = lane % LPR * 4, r0 = warp * RPW * PASS + lane / LPR;
    const bool rows = warp * RPW * PASS < D;
    uint32_t g = 0, picks = 0;
    bool ok = true;
    int b = 0;
    for (long long x = begin; ok && x < end;) {
        while (x >= (long long)line.units[b + 1] * c.H) ++b;
        const int nu = line.units[b + 1] - line.units[b], row = line.row[b], pos = line.pos[b], nb = cached_segments(c, pos), in0 = pos % c.C;
        const long long u0 = (long long)line.units[b] * c.H;
        const int in_b = (int)(x - u0), h = in_b / nu, i0 = in_b % nu, i1 = min((int)(end - x < nu - i0 ? i0 + (end - x) : nu), nb + 1);
        x += (end - x < nu - i0 ? end - x : nu - i0);
        if (i0 > nb) continue;
        const int bh = b * c.H + h, stop = min(i1, nb);
        const size_t at = (size_t)bh * D;
        const float4 q = load4(static_cast<const E *>(a.q) + at + c0);
        const float4 u = routed ? load4(static_cast<const E *>(a.u) + at + c0) : q;
        float *part = work.part + ((size_t)blockIdx.x + bh) * (D + 2);
        if (i0 < nb) {
            // scores: of the range's memories, or, for the sparse router, of all that are cached
            const int s0 = sparse ? 0 : i0, s1 = sparse ? nb : stop;
            const int32_t *table = c.table + (size_t)row * c.nmax;
            float best = -FLT_MAX;
            if (sparse && picks++ > 0 && !(ok = mbar_wait(&issued, picks & 1, &abort_flag))) break;
            for (int j0 = s0 + warp * RPW; j0 < s1; j0 += 4 * kWorkers * RPW) {
                int p[4];
                float4 k[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int i = j0 + y * kWorkers * RPW + lane / LPR;
                    p[y] = i < s1 ? valid_page(c, table[i]) : -1;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    k[y] = routed && p[y] >= 0 ? load4(c.kbar + ((size_t)p[y] * c.H + h) * D + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    float r = dot4(u, k[y]);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
                    const int i = j0 + y * kWorkers * RPW + lane / LPR;
                    if (i < s1 && lane % LPR == 0) {
                        score[i] = routed ? r : 0.f;
                        page[i] = p[y];
                    }
                }
            }
            if (!(ok = gather())) break;
            if (sparse) {
                // the topk largest; equal scores: the older segment.  One warp's work, in topk turns, and that of every range that has
                // a part of the head: this and not the memories bounds a large topk (8 heads of d = 64, 4 sequences of 512 segments:
                // topk 4 55 us, 64 178, 256 565; all of them 76 without the router's choice)
                if (warp == 0) {
                    int held = 0;
                    for (int i = lane; i < nb; i += 32) held += page[i] >= 0;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) held += __shfl_xor_sync(0xffffffffu, held, o);
                    float lim = 0.f;
                    int lim_at = kAll;
                    if (a.topk < held) {
                        lim = __int_as_float(0x7f800000);
                        lim_at = -1;
                        for (int t = 0; t < a.topk; ++t) {
                            float bv = 0.f;
                            int bi = 0x7fffffff;
                            for (int i = lane; i < nb; i += 32) {
                                const float v = score[i];
                                if (page[i] < 0 || !(v < lim || (v == lim && i > lim_at))) continue;
                                if (bi == 0x7fffffff || v > bv) { bv = v; bi = i; }
                            }
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) {
                                const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
                                const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
                                if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) { bv = ov; bi = oi; }
                            }
                            if (bi == 0x7fffffff) break;
                            lim = bv;
                            lim_at = bi;
                        }
                    }
                    if (lane == 0) {
                        cut = lim;
                        cut_at = lim_at;
                    }
                }
                if (!(ok = gather())) break;
                if (lane == 0) mbar_arrive(&chosen);
            }
            const float lim = cut;
            const int lim_at = cut_at;
            auto takes = [&](int i) { return page[i] >= 0 && (!sparse || keeps(score[i], i, lim, lim_at)); };
            for (int i = i0 + lane; i < stop; i += 32)
                if (takes(i)) best = fmaxf(best, score[i]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
            float acc[PASS], z = 0.f;
#pragma unroll
            for (int y = 0; y < PASS; ++y) acc[y] = 0.f;
            for (int i = i0; i < stop; ++i) {
                if (!takes(i)) continue;
                const float w = expf(score[i] - best);
                z += w;
                const float4 wq = scale4(w, q);
                const uint32_t s = g % STAGES;
                if (!(ok = mbar_wait(&full[s], (g / STAGES) & 1, &abort_flag))) break;
                if (rows) {
                    const float *M = reinterpret_cast<const float *>(ring + s * S::BYTES) + r0 * D + c0;
#pragma unroll
                    for (int y = 0; y < PASS; ++y) {
                        const float4 m = load4(M + y * RPW * D);
                        acc[y] = fmaf(m.x, wq.x, fmaf(m.y, wq.y, fmaf(m.z, wq.z, fmaf(m.w, wq.w, acc[y]))));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                ++g;
            }
            if (!ok) break;
            sum_groups<PASS, LPR>(acc, lane);
            if (rows && stores<PASS, LPR>(lane)) part[r0 + first<PASS, LPR>(lane) * RPW] = acc[0];
            if (tid == 0) {
                part[D] = best;
                part[D + 1] = z;
            }
        }
        if (i1 > nb) {  // the online memory
            const bool ends = in0 == c.C - 1;
            const float4 k = load4(static_cast<const E *>(a.k) + at + c0);
            if (ends && warp == 0) {  // the page that the last CTA will give this row
                int before = 0;
                for (int y = lane; y < b; y += 32) before += wants_page(c, line, y);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
                const int p = wants_page(c, line, b) ? free_page(c, before) : -1;
                if (lane == 0) mine = p;
            }
            if (ends && !(ok = gather())) break;
            const int to = ends ? mine : -1;
            if (warp == 0) {
                float4 sum = in0 ? load4(c.ksum + ((size_t)row * c.H + h) * D + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
                sum = fma4(1.f, k, sum);
                float r = dot4(u, sum);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
                if (lane < LPR) {
                    *reinterpret_cast<float4 *>(c.ksum + ((size_t)row * c.H + h) * D + c0) = sum;
                    const float n = (float)c.C;
                    if (to >= 0) *reinterpret_cast<float4 *>(c.kbar + ((size_t)to * c.H + h) * D + c0) = make_float4(sum.x / n, sum.y / n, sum.z / n, sum.w / n);
                }
                if (lane == 0) work.online[(size_t)bh * (D + 1) + D] = routed ? r / (float)(in0 + 1) : 0.f;
            }
            const float dec = a.delta ? delta_decay(to_f(static_cast<const E *>(a.la)[bh])) : 1.f;
            const float bet = a.delta ? to_f(static_cast<const E *>(a.be)[bh]) : 1.f;
            const uint32_t s = g % STAGES;
            if (in0 && !(ok = mbar_wait(&full[s], (g / STAGES) & 1, &abort_flag))) break;
            if (rows) {
                const float *M = reinterpret_cast<const float *>(ring + s * S::BYTES) + r0 * D + c0;
                float *out = c.online + (((size_t)row * c.H + h) * D + r0) * D + c0, *keep = c.pages + (((size_t)max(to, 0) * c.H + h) * D + r0) * D + c0;
                auto old = [&](int y) { return in0 ? scale4(dec, load4(M + y * RPW * D)) : make_float4(0.f, 0.f, 0.f, 0.f); };
                const E *v = static_cast<const E *>(a.v) + at + r0;
                float p[PASS], yv[PASS], e[PASS];
#pragma unroll
                for (int y = 0; y < PASS; ++y) e[y] = to_f(v[y * RPW]);
                if (a.delta) {
#pragma unroll
                    for (int y = 0; y < PASS; ++y) p[y] = dot4(old(y), k);
                    sum_groups<PASS, LPR>(p, lane);  // a lane is left with one row's: hand them round
#pragma unroll
                    for (int y = 0; y < PASS; ++y) {
                        int from = lane / LPR * LPR;  // the first of the lanes with row y's
#pragma unroll
                        for (int o = LPR / 2, half = PASS / 2; half >= 1; o >>= 1, half >>= 1) from += y & half ? o : 0;
                        e[y] = bet * (e[y] - __shfl_sync(0xffffffffu, p[0], from));
                    }
                }
#pragma unroll
                for (int y = 0; y < PASS; ++y) {
                    const float4 m = fma4(e[y], k, old(y));
                    *reinterpret_cast<float4 *>(out + y * RPW * D) = m;
                    if (to >= 0) *reinterpret_cast<float4 *>(keep + y * RPW * D) = m;
                    yv[y] = dot4(m, q);
                }
                sum_groups<PASS, LPR>(yv, lane);
                if (stores<PASS, LPR>(lane)) work.online[(size_t)bh * (D + 1) + r0 + first<PASS, LPR>(lane) * RPW] = yv[0];
            }
            if (in0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                ++g;
            }
        }
        // the head's last CTA joins what all of them left
        const long long head0 = u0 + (long long)h * nu;
        const int j0 = range_of(head0, U, R), j1 = range_of(head0 + nb, U, R);
        bool joins = j0 == j1;
        if (!joins) {
            __threadfence();
            if (!(ok = gather())) break;
            if (tid == 0) last = atomicAdd(work.turns + bh, 1) == j1 - j0;
            if (!(ok = gather())) break;
            joins = last;
            __threadfence();
        } else if (!(ok = gather())) {
            break;
        }
        if (joins) {
            const int jc = nb > 0 ? range_of(head0 + nb - 1, U, R) : j0 - 1;  // (the last range with cached memories)
            const float *own = work.online + (size_t)bh * (D + 1);
            float top = __ldcg(own + D), zs = 0.f;
            for (int j = j0; j <= jc; ++j) top = fmaxf(top, __ldcg(work.part + ((size_t)j + bh) * (D + 2) + D));
            const float w_on = expf(__ldcg(own + D) - top);
            for (int j = j0; j <= jc; ++j) {
                const float2 w = __ldcg(reinterpret_cast<const float2 *>(work.part + ((size_t)j + bh) * (D + 2) + D));
                zs += w.y * expf(w.x - top);
            }
            const float inv = a.mode == MC_RESIDUAL ? 1.f : 1.f / (zs + w_on);
            for (int r = tid; r < D; r += 32 * kWorkers) {
                float y = w_on * __ldcg(own + r);
                for (int j = j0; j <= jc; ++j) {
                    const float *p = work.part + ((size_t)j + bh) * (D + 2);
                    y = fmaf(expf(__ldcg(p + D) - top), __ldcg(p + r), y);
                }
                static_cast<E *>(a.y)[at + r] = from_f<E>(y * inv);
            }
            if (tid == 0) work.turns[bh] = 0;
        }
    }
    if (ok) {
        __threadfence();
        ok = gather();
    }
    if (ok && tid == 0) last = atomicAdd(work.turns + (size_t)c.S * c.H, 1) == (int)gridDim.x - 1;
    if (ok) ok = gather();
    if (ok && last) {
        __threadfence();
        if (tid == 0) work.turns[(size_t)c.S * c.H] = 0;
        for (int y = tid; y < a.B; y += 32 * kWorkers)
            if (line.row[y] >= 0) {
                c.pos[line.row[y]] = line.pos[y] + 1;
                if (line.pos[y] % c.C == c.C - 1 && !wants_page(c, line, y)) atomicOr(c.status, MC_PAGES_TABLE_FULL);
            }
        if (warp == 0) {  // free pages in order, to the batch's rows in order
            int y = 0;
            while (y < a.B && !wants_page(c, line, y)) ++y;
            for (int p0 = 0; p0 < c.P && y < a.B; p0 += 32) {
                unsigned open = __ballot_sync(0xffffffffu, p0 + lane < c.P && __ldcg(c.refs + p0 + lane) == 0);
                for (; open && y < a.B; open &= open - 1) {
                    const int p = p0 + __ffs(open) - 1;
                    if (lane == 0) {
                        c.table[(size_t)line.row[y] * c.nmax + line.pos[y] / c.C] = p;
                        c.refs[p] = 1;
                    }
                    do ++y;
                    while (y < a.B && !wants_page(c, line, y));
                }
            }
            for (; y < a.B; ++y)
                if (lane == 0 && wants_page(c, line, y)) {
                    c.table[(size_t)line.row[y] * c.nmax + line.pos[y] / c.C] = -1;
                    atomicOr(c.status, MC_PAGES_NONE_FREE);
                }
        }
    }
    if (tid == 0 && abort_flag) atomicExch(&g_step_abort, 1);
}

template <typename E, int D>
cudaError_t step_impl(TreeArgs a, const StepWork &work, cudaStream_t s)
{
    a.rest = 1024 / D;
    return launch_early(step_paged<E, D>, (size_t)a.ranges, kThreads, step_smem<D>(a), s, a, work);
}
template <typename E>
cudaError_t step_by_d(const TreeArgs &a, const StepWork &w, cudaStream_t s)
{
    switch (a.c.d) {
    case 16: return step_impl<E, 16>(a, w, s);
    case 32: return step_impl<E, 32>(a, w, s);
    case 64: return step_impl<E, 64>(a, w, s);
    default: return step_impl<E, 128>(a, w, s);
    }
}

}  // namespace

cudaError_t launch_step(const TreeArgs &a, const StepWork &work, cudaStream_t s)
{
    return a.bf16 ? step_by_d<__nv_bfloat16>(a, work, s) : step_by_d<float>(a, work, s);
}

cudaError_t take_step_abort(int *was_set)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_step_abort, sizeof(int));
    if (e != cudaSuccess) return e;
    *was_set = v;
    if (v) {
        v = 0;
        e = cudaMemcpyToSymbol(g_step_abort, &v, sizeof(int));
    }
    return e;
}

}  // namespace mc
