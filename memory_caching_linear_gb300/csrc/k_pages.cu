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

// The lowest `want` free pages of the pool to list, in order, each with one reference; -1 where there are no more.
__device__ void take_pages(const Paged &c, int want, int32_t *list)
{
    int found = 0;
    for (int p0 = 0; p0 < c.P && found < want; p0 += kPlanThreads) {
        const int p = p0 + (int)threadIdx.x;
        const bool free = p < c.P && __ldcg(c.refs + p) == 0;
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
    const bool accept = a.accept;
    __shared__ int taker[kMaxRows], lens[kMaxRows];
    taker[tid] = 0x7fffffff;
    lens[tid] = 0;
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
    if (accept) {  // the path to the last node, a warp to a batch row with two nodes' parents on each lane
        for (int b = tid / 32; b < a.B; b += kPlanThreads / 32) {
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
    }
    const int len = row < 0 ? 0 : a.step ? 1 : accept ? lens[tid] : 0;
    const int s0 = pos / c.C, s1 = (pos + len) / c.C;
    const int more = row < 0 ? 0 : min(s1, c.nmax) - min(s0, c.nmax);
    if (row >= 0 && s1 > s0 && s1 > c.nmax) report(c, MC_PAGES_TABLE_FULL);
    if (in) {
        a.p.act[tid] = row;
        a.p.pos[tid] = pos;
        a.p.len[tid] = len;
    }
    int want;
    const int fb = block_scan(more, &want);
    if (in) a.p.fresh[tid] = fb;
    if (tid == 0) a.p.fresh[a.B] = want;
    if (want == 0) return;
    take_pages(c, want, a.p.list);
    for (int i = 0; i < more; ++i) c.table[(size_t)row * c.nmax + s0 + i] = __ldcg(a.p.list + fb + i);
}

// The accepted tokens, one after the other, into the memory of the begun segment; what completes goes to its page.  A row of
// a memory sees its own value's entry alone, so a CTA takes up to 32 rows of a head, a group of d / 4 lanes each, in
// registers: the memory is read and written once.  The chain of a token is its key's dot product (five exchanges at d = 128)
// and the update.
template <typename E, int D>
__global__ void __launch_bounds__(256) accept_rows(TreeArgs a)
{
    constexpr int RB = D < 32 ? D : 32, LPR = D / 4, RPW = 32 / LPR, PASS = RB / (8 * RPW) < 1 ? 1 : RB / (8 * RPW);
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / (D / RB), rb = (int)blockIdx.x % (D / RB), b = bh / c.H, h = bh % c.H;
    const int row = a.p.act[b], n = a.p.len[b];
    if (row < 0 || n == 0) return;
    __shared__ __align__(16) float ks[kMaxTree][D];
    __shared__ float vs[kMaxTree][RB], dec[kMaxTree], bet[kMaxTree];
    __shared__ int node[kMaxTree];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint64_t path = a.p.path[b];
    if (tid < kMaxTree && (path >> tid) & 1) node[__popcll(path & ((1ull << tid) - 1))] = tid;
    __syncthreads();
    const size_t at = (size_t)bh * a.T;
    for (int i = tid; i < n * (D / 4); i += 256) {
        const int j = i / (D / 4), x = i % (D / 4) * 4;
        *reinterpret_cast<float4 *>(&ks[j][x]) = load4(static_cast<const E *>(a.k) + (at + node[j]) * D + x);
    }
    for (int i = tid; i < n * RB; i += 256)
        vs[i / RB][i % RB] = to_f(static_cast<const E *>(a.v)[(at + node[i / RB]) * D + rb * RB + i % RB]);
    if (a.delta && tid < n) {
        dec[tid] = delta_decay(to_f(static_cast<const E *>(a.la)[at + node[tid]]));
        bet[tid] = to_f(static_cast<const E *>(a.be)[at + node[tid]]);
    }
    __syncthreads();
    const int pos = a.p.pos[b], in0 = pos % c.C, s0 = pos / c.C;
    const int32_t *list = a.p.list + a.p.fresh[b];
    const int r0 = warp * RPW * PASS + lane / LPR;
    if (warp * RPW * PASS < RB) {
        float4 m[PASS];
        float4 *mem = reinterpret_cast<float4 *>(c.online + (((size_t)row * c.H + h) * D + rb * RB + r0) * D) + lane % LPR;
#pragma unroll
        for (int x = 0; x < PASS; ++x) m[x] = in0 ? mem[x * RPW * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
        int in = in0, s = s0;
        for (int j = 0; j < n; ++j) {
            const float4 kv = *reinterpret_cast<const float4 *>(&ks[j][lane % LPR * 4]);
            float e[PASS];
#pragma unroll
            for (int x = 0; x < PASS; ++x) e[x] = vs[j][r0 + x * RPW];
            if (a.delta) {
                const float d = in ? dec[j] : 0.f, be = bet[j];  // an empty memory has nothing to decay
#pragma unroll
                for (int x = 0; x < PASS; ++x) {
                    m[x] = in ? scale4(d, m[x]) : make_float4(0.f, 0.f, 0.f, 0.f);
                    float p = dot4(m[x], kv);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
                    e[x] = be * (e[x] - p);
                }
            } else if (!in) {
#pragma unroll
                for (int x = 0; x < PASS; ++x) m[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int x = 0; x < PASS; ++x) m[x] = fma4(e[x], kv, m[x]);
            if (++in == c.C) {
                const int page = s < c.nmax ? list[s - s0] : -1;
                if (page >= 0) {
                    float4 *to = reinterpret_cast<float4 *>(c.pages + (((size_t)page * c.H + h) * D + rb * RB + r0) * D) + lane % LPR;
#pragma unroll
                    for (int x = 0; x < PASS; ++x) to[x * RPW * (D / 4)] = m[x];
                }
                in = 0;
                ++s;
            }
        }
#pragma unroll
        for (int x = 0; x < PASS; ++x) mem[x * RPW * (D / 4)] = m[x];
    }
    if (rb == 0 && tid < D) {
        float *sum = c.ksum + ((size_t)row * c.H + h) * D + tid;
        float x = in0 ? *sum : 0.f;
        int in = in0, s = s0;
        for (int j = 0; j < n; ++j) {
            x = (in ? x : 0.f) + ks[j][tid];
            if (++in == c.C) {
                const int page = s < c.nmax ? list[s - s0] : -1;
                if (page >= 0) c.kbar[((size_t)page * c.H + h) * D + tid] = x / (float)c.C;
                in = 0;
                ++s;
            }
        }
        *sum = x;
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
__global__ void __launch_bounds__(kPlanThreads) plan_fork(Paged c, const int32_t *src, int32_t *from, int32_t *to)
{
    __shared__ int keeper[kMaxRows], rows[kMaxRows], spare[kMaxRows];
    __shared__ unsigned char kept[kMaxRows];
    const int x = threadIdx.x;
    const bool in = x < c.S;
    keeper[x] = 0x7fffffff;
    kept[x] = 0;
    spare[x] = -1;
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

__global__ void __launch_bounds__(256) fork_rows(Paged c, const int32_t *from, const int32_t *to)
{
    const int x = blockIdx.y, f = from[x], t = to[x];
    if (f == -2) return;
    const size_t mem = (size_t)c.H * c.d * c.d, key = (size_t)c.H * c.d;
    if (f >= 0) copy_piece(c.online + t * mem, c.online + f * mem, mem, blockIdx.x);
    if (blockIdx.x) return;
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
// map [src.P]: where a page goes, -1 if it is free or there is no room; live [1]: pages to move.
__global__ void __launch_bounds__(kPlanThreads) plan_compact(Paged dst, Paged src, int32_t *from, int32_t *map, int32_t *live)
{
    int n = 0;
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
    take_pages(c, done, list);
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
    const int n = (int)blockIdx.x / c.H, h = (int)blockIdx.x % c.H, N = (L + c.C - 1) / c.C;
    const bool tail = n == done;
    const int at = list[done] < 0 ? -1 : list[tail ? done : n];
    if (at < 0) return;
    const int len = min(c.C, L - n * c.C);  // 0: no segment is begun
    float *to = (tail ? c.online : c.pages) + ((size_t)at * c.H + h) * D * D;
    const float *from = states + ((size_t)h * N + n) * D * D;
    for (int i = threadIdx.x; i < D * D / 4; i += 256)
        reinterpret_cast<float4 *>(to)[i] = len > 0 ? reinterpret_cast<const float4 *>(from)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    __shared__ float4 sums[256];
    const int part = threadIdx.x / (D / 4), x = threadIdx.x % (D / 4);
    const E *kp = k + ((size_t)h * L + (size_t)n * c.C) * D + x * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
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

template <typename E>
cudaError_t accept_impl(const TreeArgs &a, cudaStream_t s)
{
    const unsigned heads = (unsigned)(a.B * a.c.H);
    switch (a.c.d) {
    case 16: accept_rows<E, 16><<<heads, 256, 0, s>>>(a); break;
    case 32: accept_rows<E, 32><<<heads, 256, 0, s>>>(a); break;
    case 64: accept_rows<E, 64><<<heads * 2, 256, 0, s>>>(a); break;
    default: accept_rows<E, 128><<<heads * 4, 256, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

template <typename E>
cudaError_t load_impl(const Paged &c, const void *k, const float *states, int L, const int32_t *list, cudaStream_t s)
{
    const int done = L / c.C;
    const unsigned ctas = (unsigned)((done + 1) * c.H);
    const E *kk = static_cast<const E *>(k);
    switch (c.d) {
    case 16: load_segment<E, 16><<<ctas, 256, 0, s>>>(c, kk, states, L, done, list); break;
    case 32: load_segment<E, 32><<<ctas, 256, 0, s>>>(c, kk, states, L, done, list); break;
    case 64: load_segment<E, 64><<<ctas, 256, 0, s>>>(c, kk, states, L, done, list); break;
    default: load_segment<E, 128><<<ctas, 256, 0, s>>>(c, kk, states, L, done, list); break;
    }
    return cudaGetLastError();
}

unsigned copy_pieces(const Paged &c) { return (unsigned)(((size_t)c.H * c.d * c.d + kCopyFloats - 1) / kCopyFloats); }

}  // namespace

cudaError_t launch_plan(const TreeArgs &a, cudaStream_t s)
{
    plan_rows<<<1, kPlanThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_accept(const TreeArgs &a, cudaStream_t s)
{
    return a.bf16 ? accept_impl<__nv_bfloat16>(a, s) : accept_impl<float>(a, s);
}

cudaError_t launch_fork(const Paged &c, const int32_t *src, int32_t *plan, cudaStream_t s)
{
    plan_fork<<<1, kPlanThreads, 0, s>>>(c, src, plan, plan + c.S);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    fork_rows<<<dim3(copy_pieces(c), (unsigned)c.S), 256, 0, s>>>(c, plan, plan + c.S);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const Paged &dst, const Paged &src, int32_t *plan, cudaStream_t s)
{
    int32_t *live = plan, *from = plan + 1, *map = from + dst.P;
    plan_compact<<<1, kPlanThreads, 0, s>>>(dst, src, from, map, live);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int places = dst.P < src.P ? dst.P : src.P;
    const unsigned pieces = copy_pieces(dst);
    compact_move<<<pieces * (unsigned)(places + dst.S), 256, 0, s>>>(dst, src, from, map, live, places, (int)pieces);
    return cudaGetLastError();
}

cudaError_t launch_pages_load(const Paged &c, int slot, const void *k, const float *states, int L, bool bf16, int32_t *plan,
                              cudaStream_t s)
{
    plan_load<<<1, kPlanThreads, 0, s>>>(c, slot, L, L / c.C, plan);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return bf16 ? load_impl<__nv_bfloat16>(c, k, states, L, plan, s) : load_impl<float>(c, k, states, L, plan, s);
}

}  // namespace mc
