// k_tree.cu -- what the tokens of a draft read: a tree of up to 64 nodes that goes on from a sequence of a paged cache (a
// single token is a tree of one node).
//
// Node n at depth e is the token at position pos + e; its ancestors and itself are the tokens that the memories it reads have
// seen beyond the cache.  With seg(a) the segment of node a, counted from the one that the cache has begun (0), and, per
// segment j, l the deepest ancestor of n in it,
//     M_j = D(0, l) M_begun [j = 0] + sum over ancestors a in j of D(a, l) beta_a e_a k_a^T,   D(a, l) = exp(c_l - c_a)
//     e_n = v_n - D(0, n) M_begun k_n [seg(n) = 0] - sum over a above n in seg(n) of D(a, n) beta_a (k_a . k_n) e_a
// (c: log_alpha summed along the path within a segment; the linear memory has D = beta = 1 and e = v), and
//     y_n = sum_i g_{n,i} M^(i) q_n + g_{n,0} D(0, l) M_begun q_n + sum over ancestors a of P_{n,a} e_a,
//     P_{n,a} = g_{n,seg(a)} D(a, l) beta_a (k_a . q_n).
// tree_gates works out the gates, P, and A_{n,a} = D(a, n) beta_a (k_a . k_n); tree_read (or tree_read_tc) goes over the
// cached memories; tree_finish solves for e and adds up.  The cached memories' bytes, read once for all nodes, bound all.
#include <cfloat>
#include <cstdint>

#include "paged.cuh"

namespace mc {
namespace {

constexpr int kGroup = 8;  // tokens that a CTA of the gates and of the CUDA-core read works on

// ------------------------------------------------------------------------------------------------ gates

constexpr int kGateThreads = 256;

size_t gates_smem(const Paged &c)
{
    return sizeof(float) * (kGroup * (size_t)(c.nmax + 1 + kMaxTree) + c.nmax);
}

template <typename E, int D>
__global__ void __launch_bounds__(kGateThreads) tree_gates(TreeArgs a)
{
    constexpr int LPR = D / 4, RPW = 32 / LPR, WARPS = kGateThreads / 32;
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / a.groups, n0 = (int)blockIdx.x % a.groups * kGroup, b = bh / c.H, h = bh % c.H;
    const int row = a.p.act[b], m = nodes_of(a, b);
    if (row < 0 || n0 >= m) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int pos = a.p.pos[b], nb = cached_segments(c, pos), in0 = pos % c.C;
    const bool routed = a.mode == MC_GRM || a.mode == MC_SSC;
    const int stride = c.nmax + 1 + kMaxTree;
    extern __shared__ __align__(16) float dyn[];
    float *sc = dyn;                                         // [kGroup][stride] scores: cached, key sum, nodes; then gates
    int *page = reinterpret_cast<int *>(dyn + kGroup * stride);  // [nmax]
    __shared__ uint64_t anc[kMaxTree], seg_set[kMaxTree];
    __shared__ int up[kMaxTree], seg[kMaxTree];
    __shared__ __align__(16) float tok[3][kGroup][D];  // u, q, k of the group's tokens
    __shared__ float kq[kGroup][kMaxTree], kk[kGroup][kMaxTree], gp[kGroup][kMaxTree];
    __shared__ float2 cum[kMaxTree];
    __shared__ float la[kMaxTree], be[kMaxTree];

    // ancestors by doubling: after turn x a node knows those up to 2^x above it
    uint64_t set = 0;
    int f = -1;
    if (tid < kMaxTree) {
        if (tid < m) {
            set = 1ull << tid;
            f = a.parent ? a.parent[(size_t)b * a.T + tid] : -1;
            if (f < -1 || f >= tid) {
                atomicOr(c.status, MC_PAGES_INDEX);
                f = -1;
            }
            if (a.delta) {
                la[tid] = delta_log(to_f(static_cast<const E *>(a.la)[(size_t)bh * a.T + tid]));
                be[tid] = to_f(static_cast<const E *>(a.be)[(size_t)bh * a.T + tid]);
            }
        }
        anc[tid] = set;
        up[tid] = f;
        seg_set[tid] = 0;
    }
    for (int i = tid; i < nb; i += kGateThreads) page[i] = valid_page(c, c.table[(size_t)row * c.nmax + i]);
    for (int i = tid; i < kGroup * D; i += kGateThreads) {
        const int t = i / D, x = i % D;
        const size_t at = ((size_t)bh * a.T + n0 + t) * D + x;
        const bool in = n0 + t < m;
        if (routed) tok[0][t][x] = in ? to_f(static_cast<const E *>(a.u)[at]) : 0.f;
        tok[1][t][x] = in ? to_f(static_cast<const E *>(a.q)[at]) : 0.f;
        if (a.delta) tok[2][t][x] = in ? to_f(static_cast<const E *>(a.k)[at]) : 0.f;
    }
    __syncthreads();
#pragma unroll 1
    for (int x = 1; x < m; x *= 2) {
        if (tid < m && f >= 0) {
            set |= anc[f];
            f = up[f];
        }
        __syncthreads();
        if (tid < m) {
            anc[tid] = set;
            up[tid] = f;
        }
        __syncthreads();
    }
    if (tid < m) {
        const int s = (in0 + __popcll(set) - 1) / c.C;
        seg[tid] = s;
        atomicOr(reinterpret_cast<unsigned long long *>(&seg_set[s]), 1ull << tid);
    }
    __syncthreads();
    if (a.delta && tid < m) {
        float2 s = make_float2(0.f, 0.f);
        for (uint64_t w = set & seg_set[seg[tid]]; w; w &= w - 1) {
            const float2 x = delta_parts(la[__ffsll(w) - 1]);
            s.x += x.x;
            s.y += x.y;
        }
        cum[tid] = s;
    }

    // dot products of the group's tokens (tok[which]) with rows: LPR lanes to a row
    auto dots = [&](int which, int rows, auto load, auto store) {
        float4 t4[kGroup];
#pragma unroll
        for (int t = 0; t < kGroup; ++t) t4[t] = reinterpret_cast<const float4 *>(tok[which][t])[lane % LPR];
        for (int i0 = warp * RPW; i0 < rows; i0 += WARPS * RPW) {
            const int i = i0 + lane / LPR;
            const float4 r = i < rows ? load(i, lane % LPR * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            float p[kGroup];
#pragma unroll
            for (int t = 0; t < kGroup; ++t) p[t] = dot4(r, t4[t]);
            sum_groups<kGroup, LPR>(p, lane);
            const int t0 = first<kGroup, LPR>(lane);
            if (i < rows && stores<kGroup, LPR>(lane)) {
#pragma unroll
                for (int x = 0; x < kept<kGroup, LPR>(); ++x) store(t0 + x, i, p[x]);
            }
        }
    };
    const E *keys = static_cast<const E *>(a.k) + (size_t)bh * a.T * D;
    const float *sum = c.ksum + ((size_t)row * c.H + h) * D;
    if (routed) {
        dots(0, nb + 1 + m,
             [&](int i, int x) {
                 if (i < nb) return page[i] >= 0 ? load4(c.kbar + ((size_t)page[i] * c.H + h) * D + x) : make_float4(0.f, 0.f, 0.f, 0.f);
                 if (i == nb) return in0 ? load4(sum + x) : make_float4(0.f, 0.f, 0.f, 0.f);
                 return load4(keys + (size_t)(i - nb - 1) * D + x);
             },
             [&](int t, int i, float p) { sc[t * stride + i] = p; });
    }
    dots(1, m, [&](int i, int x) { return load4(keys + (size_t)i * D + x); }, [&](int t, int i, float p) { kq[t][i] = p; });
    if (a.delta)
        dots(2, m, [&](int i, int x) { return load4(keys + (size_t)i * D + x); }, [&](int t, int i, float p) { kk[t][i] = p; });
    __syncthreads();

    // gates: a warp to a token
    const int n = n0 + warp;
    if (n < m) {
        float *s = sc + warp * stride;
        const uint64_t mine = anc[n];
        const int last = seg[n];
        float top = -FLT_MAX;
        if (routed) {
            for (int j = lane; j <= last; j += 32) {  // the path's segments: keys of the cache and of the path
                float x = j == 0 && in0 ? s[nb] : 0.f;
                for (uint64_t w = mine & seg_set[j]; w; w &= w - 1) x += s[nb + __ffsll(w)];
                gp[warp][j] = x / (float)(j < last ? c.C : (in0 + __popcll(mine) - 1) % c.C + 1);
            }
            __syncwarp();
        }
        // a memory that takes part: a cached one that has a page, one that the path completed, the online one
        float cut = FLT_MAX;  // SSC: the last score chosen and its place (a page i, or nmax + j)
        int cut_at = 0x7fffffff, held = 0;
        for (int i = lane; i < nb; i += 32) held += page[i] >= 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) held += __shfl_xor_sync(0xffffffffu, held, o);
        held += last;
        const bool sparse = a.mode == MC_SSC && a.topk < held;
        if (sparse) {  // the topk largest; equal scores: the older segment
            cut = __int_as_float(0x7f800000);
            cut_at = -1;
            for (int r = 0; r < a.topk; ++r) {
                float bv = 0.f;
                int bi = 0x7fffffff;
                auto offer = [&](float v, int i) {
                    if (!(v < cut || (v == cut && i > cut_at))) return;
                    if (bi == 0x7fffffff || v > bv || (v == bv && i < bi)) { bv = v; bi = i; }
                };
                for (int i = lane; i < nb; i += 32)
                    if (page[i] >= 0) offer(s[i], i);
                for (int j = lane; j < last; j += 32) offer(gp[warp][j], c.nmax + j);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
                    const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
                    if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) { bv = ov; bi = oi; }
                }
                if (bi == 0x7fffffff) break;
                cut = bv;
                cut_at = bi;
            }
        }
        auto chosen = [&](float v, int i) { return !sparse || v > cut || (v == cut && i <= cut_at); };
        if (routed) {
            top = gp[warp][last];
            for (int i = lane; i < nb; i += 32)
                if (page[i] >= 0 && chosen(s[i], i)) top = fmaxf(top, s[i]);
            for (int j = lane; j < last; j += 32)
                if (chosen(gp[warp][j], c.nmax + j)) top = fmaxf(top, gp[warp][j]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float z = 0.f;
            for (int i = lane; i < nb; i += 32) {
                const float g = page[i] >= 0 && chosen(s[i], i) ? expf(s[i] - top) : 0.f;
                s[i] = g;
                z += g;
            }
            __syncwarp();
            for (int j = lane; j <= last; j += 32) {
                const float g = j == last || chosen(gp[warp][j], c.nmax + j) ? expf(gp[warp][j] - top) : 0.f;
                gp[warp][j] = g;
                z += g;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            const float inv = 1.f / z;
            for (int i = lane; i < nb; i += 32) s[i] *= inv;
            for (int j = lane; j <= last; j += 32) gp[warp][j] *= inv;
        } else {
            const float g = a.mode == MC_MEAN ? 1.f / (float)(held + 1) : 1.f;
            for (int i = lane; i < nb; i += 32) s[i] = page[i] >= 0 ? g : 0.f;
            for (int j = lane; j <= last; j += 32) gp[warp][j] = g;
        }
        __syncwarp();
        // what the node reads of what its ancestors wrote, and what they meet in its key
        float *Pr = a.P + ((size_t)bh * a.T + n) * a.Tp, *Ar = a.delta ? a.A + ((size_t)bh * a.T + n) * a.Tp : nullptr;
        auto decay = [&](int to, int from) { return expf((cum[to].x - cum[from].x) + (cum[to].y - cum[from].y)); };
        for (int x = lane; x < a.Tp; x += 32) {
            const bool above = x < m && (mine >> x) & 1;
            float p = 0.f, q = 0.f;
            if (above) {
                const int sx = seg[x];
                p = gp[warp][sx] * kq[warp][x];
                if (a.delta) {
                    const int deepest = 63 - __clzll(mine & seg_set[sx]);
                    p *= decay(deepest, x) * be[x];
                    if (sx == last && x != n) q = decay(n, x) * be[x] * kk[warp][x];
                }
            }
            Pr[x] = p;
            if (a.delta) Ar[x] = q;
        }
        if (lane == 0) {
            float into = 1.f;  // of the begun segment's memory
            if (a.delta) {
                const float2 z = cum[63 - __clzll(mine & seg_set[0])];
                into = expf(z.x + z.y);
            }
            s[nb + 1] = in0 && last == 0 ? into : 0.f;
            s[nb] = in0 ? gp[warp][0] * into : 0.f;
            if (a.step) a.f0[(size_t)bh * a.Tp] = gp[warp][0];  // a step's end reads the memory after the token
        }
    }
    __syncthreads();
    float *out = a.gates + (size_t)bh * (c.nmax + 2) * a.Tp + n0;
    for (int i = tid; i < (nb + 2) * kGroup; i += kGateThreads) {
        const int t = i % kGroup;
        out[(size_t)(i / kGroup) * a.Tp + t] = n0 + t < m ? sc[t * stride + i / kGroup] : 0.f;
    }
}

// ------------------------------------------------------------------------------------------------ read

// One memory after the other for up to 8 tokens on the CUDA cores.  A lane holds four columns of its rows and adds
// M[r][c..] . (g q)[c..] over the memories of a head; the lanes are joined once per head.
template <typename E, int D, int TG>
__global__ void __launch_bounds__(256) tree_read(TreeArgs a)
{
    constexpr int LPR = D / 4, RPW = 32 / LPR, PASS = D / (8 * RPW) < 1 ? 1 : D / (8 * RPW);
    const Paged &c = a.c;
    const int range = (int)blockIdx.x / a.groups, n0 = (int)blockIdx.x % a.groups * kGroup;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const long long U = (long long)a.p.units[a.B] * c.H;
    const long long R = ranges_of(U, a.ranges);
    if (range >= R || warp * RPW * PASS >= D) return;
    long long x = range_begin(range, U, R);
    const long long end = range_begin(range + 1, U, R);
    const int r0 = warp * RPW * PASS + lane / LPR, c0 = lane % LPR * 4;
    int b = 0;
    while (x < end) {
        while (x >= (long long)a.p.units[b + 1] * c.H) ++b;
        const int nu = a.p.units[b + 1] - a.p.units[b];
        const long long in_b = x - (long long)a.p.units[b] * c.H;
        const int bh = b * c.H + (int)(in_b / nu), h = (int)(in_b / nu), row = a.p.act[b], nb = cached_segments(c, a.p.pos[b]);
        const int i0 = (int)(in_b % nu);
        const bool for_keys = i0 > nb;
        const int stop = for_keys || nu <= nb + 1 ? nu : nb + 1;  // the keys' read is apart
        const int i1 = (int)(end - x < stop - i0 ? i0 + (end - x) : stop);
        x += i1 - i0;
        const int m = nodes_of(a, b);
        if (n0 >= m) continue;
        float4 q[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t)
            q[t] = n0 + t < m ? load4(static_cast<const E *>(for_keys ? a.k : a.q) + ((size_t)bh * a.T + n0 + t) * D + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
        float acc[PASS][TG];
#pragma unroll
        for (int y = 0; y < PASS; ++y)
#pragma unroll
            for (int t = 0; t < TG; ++t) acc[y][t] = 0.f;
        for (int i = i0; i < i1; ++i) {
            const float *g = a.gates + ((size_t)bh * (c.nmax + 2) + i) * a.Tp + n0;
            float gv[TG];
            bool any = false;
#pragma unroll
            for (int t = 0; t < TG; ++t) any |= (gv[t] = g[t]) != 0.f;
            if (!any) continue;
            const int p = i < nb ? valid_page(c, c.table[(size_t)row * c.nmax + i]) : 0;
            if (p < 0) continue;
            const float *M = (i < nb ? c.pages + ((size_t)p * c.H + h) * D * D : c.online + ((size_t)row * c.H + h) * D * D) + (size_t)r0 * D + c0;
#pragma unroll
            for (int y = 0; y < PASS; ++y) {
                const float4 w = __ldg(reinterpret_cast<const float4 *>(M + y * RPW * D));
#pragma unroll
                for (int t = 0; t < TG; ++t)
                    if (gv[t] != 0.f) acc[y][t] = fmaf(gv[t], dot4(w, q[t]), acc[y][t]);
            }
        }
        float *out = (for_keys ? a.Z + (size_t)bh * a.Tp * D : a.part + ((size_t)range + bh) * a.Tp * D) + (size_t)n0 * D;
#pragma unroll
        for (int y = 0; y < PASS; ++y) {
            sum_groups<TG, LPR>(acc[y], lane);
            const int t0 = first<TG, LPR>(lane);
            if (stores<TG, LPR>(lane)) {
#pragma unroll
                for (int t = 0; t < kept<TG, LPR>(); ++t) out[(size_t)(t0 + t) * D + r0 + y * RPW] = acc[y][t];
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------ finish

// The partial reads of head bh at (token, row), in their order.
__device__ __forceinline__ float sum_parts(const TreeArgs &a, int bh, int b, int h, int D, int n, int r)
{
    const long long U = (long long)a.p.units[a.B] * a.c.H;
    const int all = a.p.units[b + 1] - a.p.units[b];  // (the last of which, of a begun delta memory, is the keys' read)
    const int nu = all - (a.delta && !a.step && a.p.pos[b] % a.c.C ? 1 : 0);
    float y = 0.f;
    if (nu == 0) return y;
    const long long u0 = (long long)a.p.units[b] * a.c.H + (long long)h * all;
    const long long R = ranges_of(U, a.ranges);
    const int j0 = range_of(u0, U, R), j1 = range_of(u0 + nu - 1, U, R);
    for (int j = j0; j <= j1; ++j) y += a.part[(((size_t)j + bh) * a.Tp + n) * D + r];
    return y;
}

// Solves for e node by node (each node's is taken from all of its descendants' at once) and adds everything up: 32 rows of a
// head, a lane to a row, a warp to every eighth node.
template <typename E, int D>
__global__ void __launch_bounds__(256) tree_finish(TreeArgs a)
{
    constexpr int RB = D < 32 ? D : 32;
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / (D / RB), rb = (int)blockIdx.x % (D / RB), b = bh / c.H, h = bh % c.H;
    const int row = a.p.act[b], m = nodes_of(a, b);
    if (row < 0 || m == 0) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, r = lane % RB;
    const int in0 = a.p.pos[b] % c.C;
    extern __shared__ __align__(16) float dyn[];
    float *Ps = dyn, *As = Ps + kMaxTree * kMaxTree;  // [m][Tp]
    __shared__ float es[kMaxTree][RB];
    const size_t at = (size_t)bh * a.T;
    for (int i = tid; i < m * a.Tp; i += 256) {
        Ps[i] = a.P[at * a.Tp + i];
        if (a.delta) As[i] = a.A[at * a.Tp + i];
    }
    const float *into = a.gates + ((size_t)bh * (c.nmax + 2) + cached_segments(c, a.p.pos[b]) + 1) * a.Tp;
    float e[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int n = warp + 8 * x;
        e[x] = n < m ? to_f(static_cast<const E *>(a.v)[(at + n) * D + rb * RB + r]) : 0.f;
        if (a.delta && in0 && n < m && into[n] != 0.f) e[x] -= a.Z[((size_t)bh * a.Tp + n) * D + rb * RB + r];
    }
    __syncthreads();
    if (a.delta) {
#pragma unroll 1
        for (int j = 0; j < m; ++j) {
            if (warp == j % 8 && lane < RB) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (x == j / 8) es[j][r] = e[x];
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int n = warp + 8 * x;
                if (n > j && n < m) {
                    const float w = As[n * a.Tp + j];
                    if (w != 0.f) e[x] = fmaf(-w, es[j][r], e[x]);
                }
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (warp + 8 * x < m && lane < RB) es[warp + 8 * x][r] = e[x];
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int n = warp + 8 * x;
        if (n >= m) continue;
        float y = sum_parts(a, bh, b, h, D, n, rb * RB + r);
        for (int j = 0; j <= n; ++j) {
            const float w = Ps[n * a.Tp + j];
            if (w != 0.f) y = fmaf(w, es[j][r], y);  // a node that is no ancestor is not multiplied, whatever it holds
        }
        if (lane < RB) static_cast<E *>(a.y)[(at + n) * D + rb * RB + r] = from_f<E>(y);
    }
}

// The end of a step: the token's update of the online memory, its read, and what it completes.  32 rows of a head.
template <typename E, int D>
__global__ void __launch_bounds__(256) step_finish(TreeArgs a)
{
    constexpr int RB = D < 32 ? D : 32, LPR = D / 4, RPW = 32 / LPR, PASS = RB / (8 * RPW) < 1 ? 1 : RB / (8 * RPW);
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / (D / RB), rb = (int)blockIdx.x % (D / RB), b = bh / c.H, h = bh % c.H;
    const int row = a.p.act[b];
    if (row < 0) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int pos = a.p.pos[b], in0 = pos % c.C;
    const int32_t *fresh = a.p.fresh + b;
    const bool ends = in0 == c.C - 1;
    const int page = ends && fresh[1] > fresh[0] ? a.p.list[fresh[0]] : -1;
    const size_t at = (size_t)bh * D;
    if (warp * RPW * PASS < RB) {
        const int r0 = rb * RB + warp * RPW * PASS + lane / LPR, c0 = lane % LPR * 4;
        const float4 kv = load4(static_cast<const E *>(a.k) + at + c0), qv = load4(static_cast<const E *>(a.q) + at + c0);
        const float dec = a.delta ? delta_decay(to_f(static_cast<const E *>(a.la)[bh])) : 1.f;
        const float bet = a.delta ? to_f(static_cast<const E *>(a.be)[bh]) : 1.f;
        const float g_on = a.f0[(size_t)bh * a.Tp];
        float4 *mem = reinterpret_cast<float4 *>(c.online + (((size_t)row * c.H + h) * D + r0) * D) + lane % LPR;
        float4 m[PASS];
#pragma unroll
        for (int x = 0; x < PASS; ++x) m[x] = in0 ? mem[x * RPW * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < PASS; ++x) {
            const int r = r0 + x * RPW;
            float e = to_f(static_cast<const E *>(a.v)[at + r]);
            if (a.delta) {
                if (in0) m[x] = scale4(dec, m[x]);
                float p = dot4(m[x], kv);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
                e = bet * (e - p);
            }
            m[x] = fma4(e, kv, m[x]);
            mem[x * RPW * (D / 4)] = m[x];
            if (page >= 0) reinterpret_cast<float4 *>(c.pages + (((size_t)page * c.H + h) * D + r) * D)[lane % LPR] = m[x];
            float y = dot4(m[x], qv);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            if (lane % LPR == 0) static_cast<E *>(a.y)[at + r] = from_f<E>(sum_parts(a, bh, b, h, D, 0, r) + g_on * y);
        }
    }
    if (rb == 0 && tid < D) {
        float *sum = c.ksum + ((size_t)row * c.H + h) * D + tid;
        const float x = (in0 ? *sum : 0.f) + to_f(static_cast<const E *>(a.k)[at + tid]);
        *sum = x;
        if (page >= 0) c.kbar[((size_t)page * c.H + h) * D + tid] = x / (float)c.C;
        if (h == 0 && tid == 0) c.pos[row] = pos + 1;
    }
}

// ------------------------------------------------------------------------------------------------ launchers

template <typename E, int D>
cudaError_t gates_impl(const TreeArgs &a, cudaStream_t s)
{
    const size_t smem = gates_smem(a.c);
    cudaError_t e = cudaFuncSetAttribute(tree_gates<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    tree_gates<E, D><<<(unsigned)(a.B * a.c.H * ((a.T + kGroup - 1) / kGroup)), kGateThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t read_impl(const TreeArgs &a, cudaStream_t s)
{
    const unsigned grid = (unsigned)(a.ranges * a.groups);
    if (a.T == 1) tree_read<E, D, 1><<<grid, 256, 0, s>>>(a);
    else if (a.T == 2) tree_read<E, D, 2><<<grid, 256, 0, s>>>(a);
    else if (a.T <= 4) tree_read<E, D, 4><<<grid, 256, 0, s>>>(a);
    else tree_read<E, D, 8><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t finish_impl(const TreeArgs &a, cudaStream_t s)
{
    constexpr int RB = D < 32 ? D : 32;
    const unsigned grid = (unsigned)(a.B * a.c.H * (D / RB));
    if (a.step) {
        step_finish<E, D><<<grid, 256, 0, s>>>(a);
        return cudaGetLastError();
    }
    const size_t smem = sizeof(float) * 2 * kMaxTree * kMaxTree;
    cudaError_t e = cudaFuncSetAttribute(tree_finish<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    tree_finish<E, D><<<grid, 256, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t by_d(const TreeArgs &a, cudaStream_t s, int what)
{
    switch (a.c.d) {
    case 16: return what == 0 ? gates_impl<E, 16>(a, s) : what == 1 ? read_impl<E, 16>(a, s) : finish_impl<E, 16>(a, s);
    case 32: return what == 0 ? gates_impl<E, 32>(a, s) : what == 1 ? read_impl<E, 32>(a, s) : finish_impl<E, 32>(a, s);
    case 64: return what == 0 ? gates_impl<E, 64>(a, s) : what == 1 ? read_impl<E, 64>(a, s) : finish_impl<E, 64>(a, s);
    default: return what == 0 ? gates_impl<E, 128>(a, s) : what == 1 ? read_impl<E, 128>(a, s) : finish_impl<E, 128>(a, s);
    }
}

cudaError_t run(const TreeArgs &a, cudaStream_t s, int what)
{
    return a.bf16 ? by_d<__nv_bfloat16>(a, s, what) : by_d<float>(a, s, what);
}

}  // namespace

cudaError_t launch_tree_gates(const TreeArgs &a, cudaStream_t s) { return run(a, s, 0); }
cudaError_t launch_tree_read(const TreeArgs &a, cudaStream_t s)
{
    return tree_tc_supported(a) ? launch_tree_read_tc(a, s) : run(a, s, 1);
}
cudaError_t launch_tree_finish(const TreeArgs &a, cudaStream_t s) { return run(a, s, 2); }

}  // namespace mc
