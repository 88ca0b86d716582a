// k_pages.cu -- the bookkeeping of a paged cache and the copies that follow from it: the plan of a call over a batch, the
// acceptance of a drafted path, forks, compaction into another pool, and the loading of a prompt.
//
// Counts of pages and sequences are small, so every plan is one CTA with a thread per sequence (at most 1024) that scans
// the pool's reference counts 1024 at a time: the lowest free pages are found by a prefix sum, in the same order in every run.
// What follows a plan moves the bytes, on the whole GPU.
#include <cstdint>

#include "paged.cuh"

namespace mc {
namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void report(const Paged &c, int bits) { atomicOr(c.status, bits); }

// Exclusive prefix sum over the block's threads; total gets the sum.  Every thread of the block calls it.
__device__ int block_scan(int x, int *total)
{
    __shared__ int sums[kPlanThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int s = lane < kPlanThreads / 32 ? sums[lane] : 0;
        int si = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, si, o);
            if (lane >= o) si += y;
        }
        sums[lane] = si;
    }
    __syncthreads();
    const int before = warp ? sums[warp - 1] : 0;
    *total = sums[kPlanThreads / 32 - 1];
    __syncthreads();
    return before + incl - x;
}

// The lowest `want` free pages of the pool to list, in order, each with one reference; -1 where there are no more.  head: the
// references of page threadIdx.x.
__device__ void take_pages(const Paged &c, int want, int32_t *list, int head)
{
    int found = 0;
    for (int p0 = 0; p0 < c.P && found < want; p0 += kPlanThreads) {
        const int p = p0 + (int)threadIdx.x;
        const bool free = p < c.P && (p0 ? __ldcg(c.refs + p) : head) == 0;
        int here;
        const int at = found + block_scan(free, &here);
        if (free && at < want) {
            list[at] = p;
            c.refs[p] = 1;
        }
        found += here;
    }
    for (int j = found + (int)threadIdx.x; j < want; j += kPlanThreads) list[j] = -1;
    if (found < want && threadIdx.x == 0) report(c, MC_PAGES_NONE_FREE);
    __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads) plan_rows(TreeArgs a)
{
    const Paged &c = a.c;
    const int tid = threadIdx.x, lane = tid % 32;
    __shared__ int taker[kMaxRows], lens[kMaxRows];
    taker[tid] = 0x7fffffff;
    after_previous();
    let_next_start();
    const int head = tid < c.P ? __ldcg(c.refs + tid) : 1;  // the first references, wanted last
    __syncthreads();
    // which row: the slot's; a slot that several batch rows name is the first one's where it is written
    const bool in = tid < a.B;
    int slot = -1, row = -1, pos = 0;
    if (in) {
        slot = a.slots ? a.slots[tid] : tid;
        if (slot < -1 || slot >= c.S) {
            report(c, MC_PAGES_INDEX);
            slot = -1;
        }
        if (slot >= 0) {
            row = c.row[slot];
            if ((unsigned)row >= (unsigned)c.S || (unsigned)(pos = c.pos[row]) > (unsigned)kMaxPos) {
                report(c, MC_PAGES_INDEX);
                row = -1;
            }
        }
        if (row >= 0) atomicMin(&taker[row], tid);
    }
    __syncthreads();
    if (row >= 0 && taker[row] != tid) {
        report(c, MC_PAGES_INDEX);
        row = -1;
    }
    lens[tid] = row < 0 ? -1 : 0;
    __syncthreads();
    // the path to the last node, a warp to a batch row with two nodes' parents on each lane; a row of nobody has none
    for (int b = tid / 32; b < a.B; b += kPlanThreads / 32) {
        if (lens[b] < 0) continue;
        const int32_t *par = a.parent + (size_t)b * a.T;
        const int lo = lane < a.T ? par[lane] : -1, hi = lane + 32 < a.T ? par[lane + 32] : -1;
        int x = a.last[b];
        bool bad = x < -1 || x >= a.T;
        if (bad) x = -1;
        uint64_t path = 0;
        while (x >= 0) {  // parents come before their nodes: at most 64 turns
            path |= 1ull << x;
            const int f0 = __shfl_sync(0xffffffffu, lo, x & 31), f1 = __shfl_sync(0xffffffffu, hi, x & 31);
            const int f = x < 32 ? f0 : f1;
            if (f < -1 || f >= x) bad = true;
            x = f >= -1 && f < x ? f : -1;
        }
        if (lane == 0) {
            if (bad) report(c, MC_PAGES_INDEX);
            lens[b] = __popcll(path);
            a.p.path[b] = path;
        }
    }
    __syncthreads();
    const int len = row < 0 ? 0 : lens[tid];
    const int s0 = pos / c.C, s1 = (pos + len) / c.C;
    const int more = row < 0 ? 0 : min(s1, c.nmax) - min(s0, c.nmax);
    if (row >= 0 && s1 > s0 && s1 > c.nmax) report(c, MC_PAGES_TABLE_FULL);
    if (in) {
        a.p.act[tid] = row;
        a.p.pos[tid] = pos;
    }
    int want;
    const int fb = block_scan(more, &want);
    if (in) a.p.fresh[tid] = fb;
    if (tid == 0) a.p.fresh[a.B] = want;
    if (want == 0) return;
    take_pages(c, want, a.p.list, head);
    for (int i = 0; i < more; ++i) c.table[(size_t)row * c.nmax + s0 + i] = __ldcg(a.p.list + fb + i);
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair_of(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 of_pair(uint64_t p)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The accepted tokens, one after the other, into the memory of the begun segment; what completes goes to its page.  A row of
// a memory sees its own value's entry alone, so the memory stays in registers: it is read and written once, and a
// CTA takes up to 64 rows of a head.  Instructions bound it, 4 d^2 products a token and what goes with them, so a lane holds
// 16 columns of its rows (d / 16 lanes to a row, three exchanges for a key's dot product at d = 128) as pairs, several rows share
// what is loaded of a token, and the memory is kept as M = s M': a token costs M' a dot product and an update, and only s,
// the decays' product, its decay (M' takes s over when it falls below 2^-30).  What a token does to s, and where a segment
// ends, is worked out once, ahead of the chain.
// What the plan does not say -- tokens, where the memory lies -- is fetched while it is made.
// 16 heads of d = 128, 16 sequences, 32 tokens, bf16: 33 us with the plan (gated delta; linear 24), of which a CTA's chain is 12,
// 0.4 us a token; one user 16.  Four CTAs an SM at 128 registers instead of three at 161: 33, and 94 -> 100 at twice both.
template <int D> struct AcceptShape {
    static constexpr int ROWS = D < 64 ? D : 64, LANES = D / 16, GROUPS = 32 / LANES, R = D == 16 ? 1 : D == 32 ? 2 : 4;
    static constexpr int PER_WARP = GROUPS * R, WARPS = ROWS < PER_WARP ? 1 : ROWS / PER_WARP;
    static size_t smem(int T) { return sizeof(float) * T * (D + ROWS + 2); }
};

template <typename E, int D>
__global__ void __launch_bounds__(32 * AcceptShape<D>::WARPS) accept_rows(TreeArgs a)
{
    using S = AcceptShape<D>;
    constexpr int R = S::R, THREADS = 32 * S::WARPS;
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / (D / S::ROWS), rb = (int)blockIdx.x % (D / S::ROWS), b = bh / c.H, h = bh % c.H;
    extern __shared__ __align__(16) float dyn[];
    float *ks = dyn, *vs = ks + a.T * D, *dec = vs + a.T * S::ROWS, *bet = dec + a.T;  // [node][column], [node][row], [node]
    __shared__ float4 turn[kMaxTree];  // of the path's tokens: M' is multiplied by (0: emptied), s, beta / s, page to write (as bits)
    __shared__ int node[kMaxTree];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, l = lane % S::LANES;
    const int r0 = warp * S::PER_WARP + lane / S::LANES;  // and, a group's rows apart, r0 + GROUPS, ...
    const bool rows = r0 < S::ROWS;
    const int slot = a.slots ? a.slots[b] : b;
    int guess = (unsigned)slot < (unsigned)c.S ? c.row[slot] : -1;  // (its position another CTA may have moved on)
    if ((unsigned)guess >= (unsigned)c.S) guess = -1;
    uint64_t m[R][8];
    float4 *const mem = reinterpret_cast<float4 *>(c.online + (((size_t)max(guess, 0) * c.H + h) * D + rb * S::ROWS + r0) * D) + l;
    constexpr int APART = S::GROUPS * (D / 4);
    if (guess >= 0 && rows) {
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 w = mem[x * APART + i * S::LANES];
                m[x][2 * i] = pair_of(w.x, w.y);
                m[x][2 * i + 1] = pair_of(w.z, w.w);
            }
    }
    const size_t at = (size_t)bh * a.T;
#pragma unroll 4
    for (int i = tid; i < a.T * (D / 4); i += THREADS)
        *reinterpret_cast<float4 *>(ks + 4 * i) = load4(static_cast<const E *>(a.k) + at * D + 4 * i);
#pragma unroll 4
    for (int i = tid; i < a.T * (S::ROWS / 4); i += THREADS)
        *reinterpret_cast<float4 *>(vs + 4 * i) =
            load4(static_cast<const E *>(a.v) + (at + i / (S::ROWS / 4)) * D + rb * S::ROWS + i % (S::ROWS / 4) * 4);
    if (a.delta)
        for (int i = tid; i < a.T; i += THREADS) {
            dec[i] = delta_decay(to_f(static_cast<const E *>(a.la)[at + i]));
            bet[i] = to_f(static_cast<const E *>(a.be)[at + i]);
        }
    after_previous();
    const int row = a.p.act[b];
    const uint64_t path = a.p.path[b];
    if (row < 0 || path == 0) return;  // (else it is the row guessed)
    const int pos = a.p.pos[b], in0 = pos % c.C, s0 = pos / c.C, n = __popcll(path);
    const int32_t *list = a.p.list + a.p.fresh[b];
    for (int x = tid; x < kMaxTree; x += THREADS)
        if ((path >> x) & 1) node[__popcll(path & ((1ull << x) - 1))] = x;
    __syncthreads();
    for (int j = tid; j < n; j += THREADS) {
        const int in = in0 + j, seg = in / c.C;  // counted from s0
        int page = -1;
        if ((in + 1) % c.C == 0 && s0 + seg < c.nmax) page = list[seg];
        turn[j] = make_float4(in % c.C ? 1.f : 0.f, a.delta ? dec[node[j]] : 1.f, a.delta ? bet[node[j]] : 1.f, __int_as_float(page));
    }
    __syncthreads();
    if (a.delta) {
        if (tid == 0) {
            float s = 1.f;
            for (int j = 0; j < n; ++j) {
                const float2 w = *reinterpret_cast<const float2 *>(&turn[j]);
                s = w.x == 0.f ? 1.f : s * w.y;
                if (s < 0x1p-30f) {
                    turn[j].x = s;
                    s = 1.f;
                }
                turn[j].y = s;
            }
        }
        __syncthreads();
        for (int j = tid; j < n; j += THREADS) turn[j].z /= turn[j].y;
        __syncthreads();
    }
    if (rows) {
        if (!in0) {
#pragma unroll
            for (int x = 0; x < R; ++x)
#pragma unroll
                for (int i = 0; i < 8; ++i) m[x][i] = 0;
        }
        auto store = [&](float4 *to, float s) {
#pragma unroll
            for (int x = 0; x < R; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 lo = of_pair(m[x][2 * i]), hi = of_pair(m[x][2 * i + 1]);
                    to[x * APART + i * S::LANES] = make_float4(s * lo.x, s * lo.y, s * hi.x, s * hi.y);
                }
        };
        for (int j = 0; j < n; ++j) {
            const float4 t = turn[j];
            const float *kj = ks + node[j] * D + 4 * l, *vj = vs + node[j] * S::ROWS + r0;
            if (t.x != 1.f) {
                const uint64_t ss = pair_of(t.x, t.x);
#pragma unroll
                for (int x = 0; x < R; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) m[x][i] = t.x == 0.f ? 0 : mul_pair(m[x][i], ss);
            }
            uint64_t k[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 kv = *reinterpret_cast<const ulonglong2 *>(kj + 4 * i * S::LANES);
                k[2 * i] = kv.x;
                k[2 * i + 1] = kv.y;
            }
            float e[R];
#pragma unroll
            for (int x = 0; x < R; ++x) e[x] = vj[x * S::GROUPS];
            if (a.delta) {
                float p[R];
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    uint64_t p0 = mul_pair(m[x][0], k[0]);
#pragma unroll
                    for (int i = 1; i < 8; ++i) p0 = fma_pair(m[x][i], k[i], p0);
                    const float2 q = of_pair(p0);
                    p[x] = q.x + q.y;
                }
#pragma unroll
                for (int o = S::LANES / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int x = 0; x < R; ++x) p[x] += __shfl_xor_sync(0xffffffffu, p[x], o);
#pragma unroll
                for (int x = 0; x < R; ++x) e[x] = t.z * fmaf(-t.y, p[x], e[x]);
            }
#pragma unroll
            for (int x = 0; x < R; ++x) {
                const uint64_t ee = pair_of(e[x], e[x]);
#pragma unroll
                for (int i = 0; i < 8; ++i) m[x][i] = fma_pair(ee, k[i], m[x][i]);
            }
            const int page = __float_as_int(t.w);
            if (page >= 0) store(reinterpret_cast<float4 *>(c.pages + (((size_t)page * c.H + h) * D + rb * S::ROWS + r0) * D) + l, t.y);
        }
        store(mem, turn[n - 1].y);
    }
    if (rb == 0) {
        for (int x = tid; x < D; x += THREADS) {
            float *sum = c.ksum + ((size_t)row * c.H + h) * D + x;
            float t = in0 ? *sum : 0.f;
            int in = in0;
            for (int j = 0; j < n; ++j) {
                t = (in ? t : 0.f) + ks[node[j] * D + x];
                if (++in == c.C) {
                    const int page = __float_as_int(turn[j].w);
                    if (page >= 0) c.kbar[((size_t)page * c.H + h) * D + x] = t / (float)c.C;
                    in = 0;
                }
            }
            *sum = t;
        }
        if (h == 0 && tid == 0) c.pos[row] = pos + n;
    }
}

constexpr int kCopyFloats = 8192;  // floats that a CTA of 256 threads copies: eight 16-byte pieces a thread, all in flight

__device__ __forceinline__ void copy_piece(float *to, const float *from, size_t floats, int piece)
{
    const size_t n4 = floats / 4, i0 = (size_t)piece * (kCopyFloats / 4) + threadIdx.x;
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i0 + i * 256 < n4) x[i] = __ldcs(reinterpret_cast<const float4 *>(from) + i0 + i * 256);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i0 + i * 256 < n4) __stcs(reinterpret_cast<float4 *>(to) + i0 + i * 256, x[i]);
}

// A fork in two steps.  A row that some slot goes on from stays where it is and becomes that slot's (its own if it stays,
// else the lowest's); the other slots take the rows that nobody goes on from, in order.  So what is read is never written,
// and only true copies move: a permutation of the slots moves nothing.  from [S]: the row to copy to to[S]; -1 none (the
// slot is freed), -2 nothing to do.
// Two launches and their chains of loads bound it: 8.5 us for four samples of one user, 11.4 for 28 copies of 1 MB.
__global__ void __launch_bounds__(kPlanThreads) plan_fork(Paged c, const int32_t *src, int32_t *from, int32_t *to)
{
    __shared__ int keeper[kMaxRows], rows[kMaxRows], spare[kMaxRows];
    __shared__ unsigned char kept[kMaxRows];
    const int x = threadIdx.x;
    const bool in = x < c.S;
    keeper[x] = 0x7fffffff;
    kept[x] = 0;
    spare[x] = -1;
    after_previous();
    let_next_start();
    rows[x] = in ? c.row[x] : -1;
    int f = -1;
    if (in) {
        f = src[x];
        if (f < -1 || f >= c.S) {
            report(c, MC_PAGES_INDEX);
            f = x;
        }
        if ((unsigned)rows[x] >= (unsigned)c.S) {
            report(c, MC_PAGES_INDEX);
            rows[x] = -1;
        }
    }
    __syncthreads();
    if (in && f >= 0) atomicMin(&keeper[f], f == x ? 0 : 1 + x);
    __syncthreads();
    const bool keeps = in && f >= 0 && keeper[f] == (f == x ? 0 : 1 + x) && rows[f] >= 0;
    if (keeps) kept[rows[f]] = 1;
    __syncthreads();
    int n_spare, n_need;
    const int at = block_scan(in && !kept[x], &n_spare);
    if (in && !kept[x]) spare[at] = x;
    const int mine = block_scan(in && !keeps, &n_need);
    if (!in) return;
    const int r = keeps ? rows[f] : mine < n_spare ? spare[mine] : -1;
    from[x] = keeps || r < 0 ? -2 : f >= 0 ? rows[f] : -1;
    to[x] = r;
    if (r >= 0) c.row[x] = r;
}

__global__ void __launch_bounds__(256) fork_rows(Paged c, const int32_t *from, const int32_t *to, int pieces)
{
    after_previous();
    const int x = (int)(blockIdx.x / pieces), piece = (int)(blockIdx.x % pieces), f = from[x], t = to[x];
    if (f == -2) return;
    const size_t mem = (size_t)c.H * c.d * c.d, key = (size_t)c.H * c.d;
    if (f >= 0) copy_piece(c.online + t * mem, c.online + f * mem, mem, piece);
    if (piece) return;
    for (int i = threadIdx.x; i < c.nmax; i += 256) {
        const int gone = valid_page(c, c.table[(size_t)t * c.nmax + i]);
        const int now = f >= 0 ? valid_page(c, c.table[(size_t)f * c.nmax + i]) : -1;
        c.table[(size_t)t * c.nmax + i] = now;
        if (gone == now) continue;
        if (gone >= 0) atomicSub(c.refs + gone, 1);
        if (now >= 0) atomicAdd(c.refs + now, 1);
    }
    if (f >= 0)
        for (int i = threadIdx.x; i < (int)key; i += 256) c.ksum[t * key + i] = c.ksum[f * key + i];
    if (threadIdx.x == 0) c.pos[t] = f >= 0 ? c.pos[f] : 0;
}

// Compaction: the live pages of src, in order, to the first pages of dst.  from [dst.P]: the page of src that comes here;
// map [src.P]: where a page goes, -1 if it is free or there is no room; live [1]: pages to move.  HBM bounds it: 0.96 GB
// read and written in 139 us, 6.9 TB/s; a small pool is two launches, 8 us.
__global__ void __launch_bounds__(kPlanThreads) plan_compact(Paged dst, Paged src, int32_t *from, int32_t *map, int32_t *live)
{
    int n = 0;
    after_previous();
    let_next_start();
    for (int p0 = 0; p0 < src.P; p0 += kPlanThreads) {
        const int p = p0 + (int)threadIdx.x, refs = p < src.P ? src.refs[p] : 0;
        int here;
        const int at = n + block_scan(refs != 0, &here);
        if (p < src.P) map[p] = refs && at < dst.P ? at : -1;
        if (refs && at < dst.P) {
            from[at] = p;
            dst.refs[at] = refs;
        }
        n += here;
    }
    if (threadIdx.x == 0) {
        *live = min(n, dst.P);
        if (n > dst.P) report(dst, MC_PAGES_NONE_FREE);
    }
    for (int p = n + (int)threadIdx.x; p < dst.P; p += kPlanThreads) dst.refs[p] = 0;
}

__global__ void __launch_bounds__(256) compact_move(Paged dst, Paged src, const int32_t *from, const int32_t *map,
                                                    const int32_t *live, int places, int pieces)
{
    after_previous();
    const size_t mem = (size_t)dst.H * dst.d * dst.d, key = (size_t)dst.H * dst.d;
    const int y = (int)(blockIdx.x / pieces), piece = (int)(blockIdx.x % pieces);
    if (y < places) {
        if (y >= *live) return;
        const int p = from[y];
        copy_piece(dst.pages + y * mem, src.pages + p * mem, mem, piece);
        if (piece == 0)
            for (int i = threadIdx.x; i < (int)key; i += 256) dst.kbar[y * key + i] = src.kbar[p * key + i];
        return;
    }
    const int x = y - places;
    int r = x < src.S ? src.row[x] : -1;
    const bool bad = x < src.S && (unsigned)r >= (unsigned)src.S;
    if (bad) r = -1;
    if (r >= 0) copy_piece(dst.online + x * mem, src.online + r * mem, mem, piece);
    if (piece) return;
    for (int i = threadIdx.x; i < dst.nmax; i += 256) {
        const int p = r >= 0 && i < src.nmax ? valid_page(src, src.table[(size_t)r * src.nmax + i]) : -1;
        dst.table[(size_t)x * dst.nmax + i] = p >= 0 ? map[p] : -1;
    }
    if (r >= 0)
        for (int i = threadIdx.x; i < (int)key; i += 256) dst.ksum[x * key + i] = src.ksum[r * key + i];
    if (threadIdx.x == 0) {
        dst.pos[x] = r >= 0 ? src.pos[r] : 0;
        dst.row[x] = x;
        if (bad) report(dst, MC_PAGES_INDEX);
    }
}

// A prompt into a slot: its old pages go back, its complete segments get the lowest free ones.
__global__ void __launch_bounds__(kPlanThreads) plan_load(Paged c, int slot, int L, int done, int32_t *list)
{
    after_previous();
    let_next_start();
    const int row = c.row[slot];
    if ((unsigned)row >= (unsigned)c.S) {
        if (threadIdx.x == 0) {
            report(c, MC_PAGES_INDEX);
            list[done] = -1;
        }
        return;
    }
    int32_t *table = c.table + (size_t)row * c.nmax;
    for (int i = threadIdx.x; i < c.nmax; i += kPlanThreads) {
        const int p = valid_page(c, table[i]);
        if (p >= 0) atomicSub(c.refs + p, 1);
    }
    __syncthreads();
    take_pages(c, done, list, (int)threadIdx.x < c.P ? __ldcg(c.refs + threadIdx.x) : 1);
    for (int i = threadIdx.x; i < c.nmax; i += kPlanThreads) table[i] = i < done ? __ldcg(list + i) : -1;
    if (threadIdx.x == 0) {
        c.pos[row] = L;
        list[done] = row;
    }
}

// One head of one segment: its memory from the prefill's states [H][N][d][d], and its keys' mean (of the last, incomplete
// segment the sum).  The sums of a segment are taken by 1024 / d threads for every column and added in their order.
template <typename E, int D>
__global__ void __launch_bounds__(256) load_segment(Paged c, const E *k, const float *states, int L, int done,
                                                    const int32_t *list)
{
    constexpr int PARTS = 256 / (D / 4);
    const int n = (int)blockIdx.x / c.H, h = (int)blockIdx.x % c.H, N = (L - 1) / c.C + 1;  // (L + C need not fit)
    after_previous();
    const bool tail = n == done;
    const int at = list[done] < 0 ? -1 : list[tail ? done : n];
    if (at < 0) return;
    const int len = min(c.C, L - n * c.C);  // 0: no segment is begun
    float *to = (tail ? c.online : c.pages) + ((size_t)at * c.H + h) * D * D;
    const float *from = states + ((size_t)h * N + n) * D * D;
#pragma unroll 8
    for (int i = threadIdx.x; i < D * D / 4; i += 256)
        reinterpret_cast<float4 *>(to)[i] = len > 0 ? reinterpret_cast<const float4 *>(from)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    __shared__ float4 sums[256];
    const int part = threadIdx.x / (D / 4), x = threadIdx.x % (D / 4);
    const E *kp = k + ((size_t)h * L + (size_t)n * c.C) * D + x * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int t = part; t < len; t += PARTS) s = fma4(1.f, load4(kp + (size_t)t * D), s);
    sums[threadIdx.x] = s;
    __syncthreads();
    if (part == 0) {
        for (int p = 1; p < PARTS; ++p) s = fma4(1.f, sums[p * (D / 4) + x], s);
        float *key = (tail ? c.ksum : c.kbar) + ((size_t)at * c.H + h) * D + x * 4;
        if (!tail) s = make_float4(s.x / c.C, s.y / c.C, s.z / c.C, s.w / c.C);
        *reinterpret_cast<float4 *>(key) = s;
    }
}

template <typename E, int D>
cudaError_t accept_impl(const TreeArgs &a, cudaStream_t s)
{
    using S = AcceptShape<D>;
    return launch_early(accept_rows<E, D>, (size_t)a.B * a.c.H * (D / S::ROWS), 32 * S::WARPS, S::smem(a.T), s, a);
}
template <typename E>
cudaError_t accept_by_d(const TreeArgs &a, cudaStream_t s)
{
    switch (a.c.d) {
    case 16: return accept_impl<E, 16>(a, s);
    case 32: return accept_impl<E, 32>(a, s);
    case 64: return accept_impl<E, 64>(a, s);
    default: return accept_impl<E, 128>(a, s);
    }
}

template <typename E>
cudaError_t load_impl(const Paged &c, const void *k, const float *states, int L, const int32_t *list, cudaStream_t s)
{
    const int done = L / c.C;
    const unsigned ctas = (unsigned)((done + 1) * c.H);
    const E *kk = static_cast<const E *>(k);
    switch (c.d) {
    case 16: return launch_early(load_segment<E, 16>, ctas, 256, 0, s, c, kk, states, L, done, list);
    case 32: return launch_early(load_segment<E, 32>, ctas, 256, 0, s, c, kk, states, L, done, list);
    case 64: return launch_early(load_segment<E, 64>, ctas, 256, 0, s, c, kk, states, L, done, list);
    default: return launch_early(load_segment<E, 128>, ctas, 256, 0, s, c, kk, states, L, done, list);
    }
}

unsigned copy_pieces(const Paged &c) { return (unsigned)(((size_t)c.H * c.d * c.d + kCopyFloats - 1) / kCopyFloats); }

}  // namespace

cudaError_t launch_plan(const TreeArgs &a, cudaStream_t s)
{
    return launch_early(plan_rows, 1, kPlanThreads, 0, s, a);
}

cudaError_t launch_accept(const TreeArgs &a, cudaStream_t s)
{
    return a.bf16 ? accept_by_d<__nv_bfloat16>(a, s) : accept_by_d<float>(a, s);
}

cudaError_t launch_fork(const Paged &c, const int32_t *src, int32_t *plan, cudaStream_t s)
{
    const int32_t *from = plan, *to = plan + c.S;
    const unsigned pieces = copy_pieces(c);
    cudaError_t e = launch_early(plan_fork, 1, kPlanThreads, 0, s, c, src, plan, plan + c.S);
    return e == cudaSuccess ? launch_early(fork_rows, (size_t)pieces * c.S, 256, 0, s, c, from, to, (int)pieces) : e;
}

cudaError_t launch_pages_compact(const Paged &dst, const Paged &src, int32_t *plan, cudaStream_t s)
{
    int32_t *live = plan, *from = plan + 1, *map = from + dst.P;
    cudaError_t e = launch_early(plan_compact, 1, kPlanThreads, 0, s, dst, src, from, map, live);
    if (e != cudaSuccess) return e;
    const int places = dst.P < src.P ? dst.P : src.P;
    const unsigned pieces = copy_pieces(dst);
    return launch_early(compact_move, (size_t)pieces * (places + dst.S), 256, 0, s, dst, src, (const int32_t *)from, (const int32_t *)map,
                        (const int32_t *)live, places, (int)pieces);
}

cudaError_t launch_pages_load(const Paged &c, int slot, const void *k, const float *states, int L, bool bf16, int32_t *plan,
                              cudaStream_t s)
{
    cudaError_t e = launch_early(plan_load, 1, kPlanThreads, 0, s, c, slot, L, L / c.C, plan);
    if (e != cudaSuccess) return e;
    return bf16 ? load_impl<__nv_bfloat16>(c, k, states, L, plan, s) : load_impl<float>(c, k, states, L, plan, s);
}

}  // namespace mc
