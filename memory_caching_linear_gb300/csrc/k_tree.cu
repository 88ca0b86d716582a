// k_tree.cu -- what the tokens of a draft read: a tree of up to 64 nodes that goes on from a sequence of a paged cache.
//
// Node n at depth e is the token at position pos + e; its ancestors and itself are the tokens that the memories it reads have
// seen beyond the cache.  With seg(a) the segment of node a, counted from the one that the cache has begun (0), and, per
// segment j, l the deepest ancestor of n in it,
//     M_j = D(0, l) M_begun [j = 0] + sum over ancestors a in j of D(a, l) beta_a e_a k_a^T,   D(a, l) = exp(c_l - c_a)
//     e_n = v_n - D(0, n) M_begun k_n [seg(n) = 0] - sum over a above n in seg(n) of D(a, n) beta_a (k_a . k_n) e_a
// (c: log_alpha summed along the path within a segment; the linear memory has D = beta = 1 and e = v), and
//     y_n = sum_i g_{n,i} M^(i) q_n + g_{n,0} D(0, l) M_begun q_n + sum over ancestors a of P_{n,a} e_a,
//     P_{n,a} = g_{n,seg(a)} D(a, l) beta_a (k_a . q_n).
// tree_gates works out the gates, P, and A_{n,a} = D(a, n) beta_a (k_a . k_n); tree_read goes over the cached memories;
// tree_finish solves for e and adds up.  On the tensor cores (k_tree_tc.cu) scores come first, the reads next, P and A beside
// them, and tree_finish last; a draft of up to 8 nodes over little room is tree_gates' alone (tree_whole).  The cached
// memories' bytes, read once for all nodes, bound a batch, launches and chains of loads everything small.
// On the CUDA cores (fp32, d < 64, SSC): 3 sequences, 6 heads of d = 64, 29 segments of 7, 13 nodes, SSC, fp32 31 us in three
// launches; 8 sequences of 2 to 63 segments, 16 heads of d = 128, 32 nodes, delta, fp32 234 us (30 of bytes), bound by products.
#include <cfloat>
#include <cstdint>

#include "mma_sync.cuh"
#include "paged.cuh"
#include "tree_nodes.cuh"

namespace mc {
namespace {

constexpr int kGroup = 8;  // tokens that a CTA of the gates and of the CUDA-core read works on

// ------------------------------------------------------------------------------------------------ gates

constexpr int kGateThreads = 256;

size_t gates_smem(const TreeArgs &a)
{
    const size_t ints = Line::ints(a.B), floats = kGroup * (size_t)(a.c.nmax + 1 + kMaxTree) + a.c.nmax;
    return 4 * (ints > floats ? ints : floats);
}

// WHOLE: the rest too, for drafts of up to 8 nodes over few heads: a CTA has 8 (d = 128), 16 (64) or all rows of a head, a lane
// group to each, and goes over all memories with the gates that it has worked out for itself.  One launch and no scratch.
template <int D> struct WholeRows { static constexpr int PER_CTA = 8 * (32 / (D / 4)), CTAS = D / PER_CTA < 1 ? 1 : D / PER_CTA; };

template <typename E, int D, bool WHOLE>
__global__ void __launch_bounds__(kGateThreads) tree_gates(TreeArgs a)
{
    constexpr int LPR = D / 4, RPW = 32 / LPR, WARPS = kGateThreads / 32;
    const Paged &c = a.c;
    extern __shared__ __align__(16) float dyn[];
    after_previous();
    if (!WHOLE && blockIdx.x == gridDim.x - 1) {  // one CTA more, for those that come after
        leave_line(a, reinterpret_cast<int *>(dyn));
        return;
    }
    const int per_head = WHOLE ? WholeRows<D>::CTAS : a.groups, bh = (int)blockIdx.x / per_head, part = (int)blockIdx.x % per_head;
    const int n0 = WHOLE ? 0 : part * kGroup, b = bh / c.H, h = bh % c.H;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const Seat seat = seat_of(a, b, WHOLE && h == 0 && part == 0 && tid == 0);
    const int row = seat.row, m = seat.m;
    if (row < 0 || n0 >= m) return;
    const int nb = cached_segments(c, seat.pos), in0 = seat.pos % c.C;
    const bool routed = a.mode == MC_GRM || a.mode == MC_SSC;
    const int stride = c.nmax + 1 + kMaxTree;
    float *sc = dyn;                                         // [kGroup][stride] scores: cached, key sum, nodes; then gates
    int *page = reinterpret_cast<int *>(dyn + kGroup * stride);  // [nmax]
    __shared__ Nodes nodes;
    __shared__ __align__(16) float tok[3][kGroup][D];  // u, q, k of the group's tokens
    __shared__ float kq[kGroup][kMaxTree], kk[kGroup][kMaxTree], gp[kGroup][kMaxTree];

    for (int i = tid; i < nb; i += kGateThreads) page[i] = valid_page(c, c.table[(size_t)row * c.nmax + i]);
    for (int i = tid; i < kGroup * D; i += kGateThreads) {
        const int t = i / D, x = i % D;
        const size_t at = ((size_t)bh * a.T + n0 + t) * D + x;
        const bool in = n0 + t < m;
        if (routed) tok[0][t][x] = in ? to_f(static_cast<const E *>(a.u)[at]) : 0.f;
        tok[1][t][x] = in ? to_f(static_cast<const E *>(a.q)[at]) : 0.f;
        if (a.delta) tok[2][t][x] = in ? to_f(static_cast<const E *>(a.k)[at]) : 0.f;
    }
    make_nodes<E>(a, nodes, b, bh, m, in0);

    // WHOLE: this lane's row, and the first memories' entries under way
    const int r = part * WholeRows<D>::PER_CTA + warp * RPW + lane / LPR, c0 = lane % LPR * 4;
    const bool reads = WHOLE && warp * RPW + part * WholeRows<D>::PER_CTA < D;
    const int count = nb + (in0 ? 1 : 0);  // memories to read
    auto entry = [&](int i) {
        if (i > nb || (i < nb && page[i] < 0) || (i == nb && !in0)) return make_float4(0.f, 0.f, 0.f, 0.f);
        const float *M = i < nb ? c.pages + ((size_t)page[i] * c.H + h) * D * D : c.online + ((size_t)row * c.H + h) * D * D;
        return __ldcs(reinterpret_cast<const float4 *>(M + (size_t)r * D + c0));
    };
    float4 ahead[4];
    if (reads && a.mode != MC_SSC) {
#pragma unroll
        for (int x = 0; x < 4; ++x) ahead[x] = entry(x);
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
        const uint64_t mine = nodes.anc[n];
        const int last = nodes.seg[n];
        float top = -FLT_MAX;
        if (routed) {
            for (int j = lane; j <= last; j += 32) {  // the path's segments: keys of the cache and of the path
                float x = j == 0 && in0 ? s[nb] : 0.f;
                for (uint64_t w = mine & nodes.seg_set[j]; w; w &= w - 1) x += s[nb + __ffsll(w)];
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
        if (lane == 0) {
            const float into = a.delta ? decay_from_cache(nodes, n) : 1.f;  // of the begun segment's memory
            s[nb + 1] = in0 && last == 0 ? into : 0.f;
            s[nb] = in0 ? gp[warp][0] * into : 0.f;
        }
    }
    __syncthreads();
    if constexpr (WHOLE) {
        __shared__ float P[kGroup][kGroup], A[kGroup][kGroup];  // [node][ancestor]
        __shared__ float base[WholeRows<D>::PER_CTA][2 * kGroup];
        if (tid < kGroup * kGroup) {
            const int n = tid / kGroup, x = tid % kGroup;
            const bool above = n < m && (nodes.anc[n] >> x) & 1;
            P[n][x] = above ? path_read(a, nodes, n, x, gp[n][nodes.seg[x]], kq[n][x]) : 0.f;
            A[n][x] = above && a.delta ? path_meet(nodes, n, x, kk[n][x]) : 0.f;
        }
        __syncthreads();
        if (!reads) return;
        float y[kGroup] = {}, z[kGroup] = {};
        float4 q[kGroup];
#pragma unroll
        for (int t = 0; t < kGroup; ++t) q[t] = *reinterpret_cast<const float4 *>(&tok[1][t][c0]);
        for (int i0 = 0; i0 < count; i0 += 4) {
            float4 w[4];
            if (i0 == 0 && a.mode != MC_SSC) {
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = ahead[x];
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    bool any = false;
                    if (a.mode == MC_SSC && i0 + x < count)
#pragma unroll
                        for (int t = 0; t < kGroup; ++t) any |= t < m && sc[t * stride + i0 + x] != 0.f;
                    w[x] = a.mode != MC_SSC || any || i0 + x == nb ? entry(i0 + x) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (i0 + x >= count) break;
#pragma unroll
                for (int t = 0; t < kGroup; ++t) {
                    const float g = t < m ? sc[t * stride + i0 + x] : 0.f;
                    if (g != 0.f) y[t] = fmaf(g, dot4(w[x], q[t]), y[t]);
                }
                if (a.delta && i0 + x == nb) {  // what the begun memory answers to the keys
#pragma unroll
                    for (int t = 0; t < kGroup; ++t) {
                        const float f = t < m ? sc[t * stride + nb + 1] : 0.f;
                        if (f != 0.f) z[t] = f * dot4(w[x], *reinterpret_cast<const float4 *>(&tok[2][t][c0]));
                    }
                }
            }
        }
        const int rl = warp * RPW + lane / LPR;
        sum_groups<kGroup, LPR>(y, lane);
        sum_groups<kGroup, LPR>(z, lane);
        if (stores<kGroup, LPR>(lane)) {
#pragma unroll
            for (int x = 0; x < kept<kGroup, LPR>(); ++x) {
                base[rl][first<kGroup, LPR>(lane) + x] = y[x];
                base[rl][kGroup + first<kGroup, LPR>(lane) + x] = z[x];
            }
        }
        __syncwarp();
        const int mine = warp * RPW + lane, mr = part * WholeRows<D>::PER_CTA + mine;  // a lane to a row: e in the nodes' order
        if (lane >= RPW || mr >= D) return;
        const size_t at = (size_t)bh * a.T;
        float e[kGroup], out[kGroup];
#pragma unroll
        for (int t = 0; t < kGroup; ++t) {
            e[t] = t < m ? to_f(static_cast<const E *>(a.v)[(at + t) * D + mr]) - base[mine][kGroup + t] : 0.f;
            out[t] = base[mine][t];
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            if (j >= m) break;
#pragma unroll
            for (int t = j; t < kGroup; ++t)
                if (t < m && (nodes.anc[t] >> j) & 1) {
                    out[t] = fmaf(P[t][j], e[j], out[t]);
                    if (A[t][j] != 0.f) e[t] = fmaf(-A[t][j], e[j], e[t]);
                }
        }
#pragma unroll
        for (int t = 0; t < kGroup; ++t)
            if (t < m) static_cast<E *>(a.y)[(at + t) * D + mr] = from_f<E>(out[t]);
        return;
    }
    float *out = a.gates + (size_t)bh * (c.nmax + 2) * a.Tp + n0;
    for (int i = tid; i < (nb + 2) * kGroup; i += kGateThreads) {
        const int t = i % kGroup;
        out[(size_t)(i / kGroup) * a.Tp + t] = n0 + t < m ? sc[t * stride + i / kGroup] : 0.f;
    }
    write_path<kGroup>(a, nodes, bh, n0, m, [&](int t, int j) { return gp[t][j]; }, [&](int t, int x) { return kq[t][x]; },
                           [&](int t, int x) { return kk[t][x]; });
}

// ------------------------------------------------------------------------------------------------ read

// One memory after the other for up to 8 tokens on the CUDA cores.  A lane holds four columns of its rows and adds
// M[r][c..] . (g q)[c..] over the memories of a head; the lanes are joined once per head.  Several CTAs share a range, each with
// a part of a memory's rows (read_blocks).
template <typename E, int D, int TG>
__global__ void __launch_bounds__(256, 2) tree_read(TreeArgs a)
{
    constexpr int BLOCKS = read_blocks(D);
    constexpr int LPR = D / 4, RPW = 32 / LPR, PASS = D / (8 * RPW * BLOCKS) < 1 ? 1 : D / (8 * RPW * BLOCKS);
    const Paged &c = a.c;
    const int range = (int)blockIdx.x / (a.groups * BLOCKS), n0 = (int)blockIdx.x / BLOCKS % a.groups * kGroup;
    const int from = (int)blockIdx.x % BLOCKS * (8 * RPW * PASS);  // the CTA's first row
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    extern __shared__ int space[];
    after_previous();
    const Line line = make_line(a, space, false);
    const long long U = (long long)line.units[a.B] * c.H;
    const long long R = ranges_of(U, a.ranges);
    if (range >= R || warp * RPW * PASS >= D) return;
    long long x = range_begin(range, U, R);
    const long long end = range_begin(range + 1, U, R);
    const int r0 = from + warp * RPW * PASS + lane / LPR, c0 = lane % LPR * 4;
    int b = 0;
    while (x < end) {
        while (x >= (long long)line.units[b + 1] * c.H) ++b;
        const int nu = line.units[b + 1] - line.units[b];
        const long long in_b = x - (long long)line.units[b] * c.H;
        const int bh = b * c.H + (int)(in_b / nu), h = (int)(in_b / nu), row = line.row[b], nb = cached_segments(c, line.pos[b]);
        const int i0 = (int)(in_b % nu), all = units_of(a, line.pos[b]);
        if (i0 >= all) {  // past what comes after a head's memories
            x += nu - i0;
            continue;
        }
        const bool for_keys = i0 > nb;
        const int stop = for_keys || all <= nb + 1 ? all : nb + 1;  // the keys' read is apart
        const int i1 = (int)(end - x < stop - i0 ? i0 + (end - x) : stop);
        x += i1 - i0;
        const int m = line.nodes[b];
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

// The partial reads of a head's `count` memories lie in ranges j0 .. j1, in the order of the memories.
struct Parts {
    int j0, j1;
    __device__ Parts(const TreeArgs &a, const Line &l, int b, int h, int count)
    {
        const int before = l.units[b], all = l.units[b + 1] - before;
        const long long U = (long long)l.units[a.B] * a.c.H, R = ranges_of(U, a.ranges), u0 = (long long)before * a.c.H + (long long)h * all;
        j0 = count > 0 ? range_of(u0, U, R) : 0;
        j1 = count > 0 ? range_of(u0 + count - 1, U, R) : -1;
    }
};

// Solves for e and adds everything up: 64 rows of a head (32 for d = 32, 16 for 16), two to a lane, and eight nodes to a warp,
// whose e and y it keeps in registers.  A row needs its own e alone, so lanes share nothing but P and A.  The e come in turns of
// eight: the warp at hand works its own out (a triangle) and leaves them in shared memory, the later ones take them up.
// The linear memory's e are the values: no turns.  What is read of them, P e, follows for all warps at once.
//   SPLIT: a split read.  With s the scores, a part's largest L_p and sum z_p, top = max(L_p, path scores) and
//   Z = sum_p z_p exp(L_p - top) + sum_j exp(s_j - top), a part counts exp(L_p - top) / Z and path segment j, whose P and (j = 0)
//   read of the begun memory wait for it, exp(s_j - top) / Z (Residual: 1 and 1; Mean: all scores 0).
// Instructions and latency bound it: what a warp loads of P and A serves both rows, an e that is nobody's ancestor costs a
// branch, and loads that do not hang on one another are all under way before the first is used.  64 nodes, 12 sequences,
// 16 heads of d = 128, gated delta 30 us; 32 nodes, 8 sequences, linear 12.
// A split read's finish wants 128 registers (at 80 it spills, and what is spilled goes to L2): so it runs where all CTAs are on
// the SMs at once with them (8 sequences, 16 heads, 32 nodes: the call 105 -> 101 us, d = 64 70 -> 66), and at 80 where they
// are not (12 sequences, 64 nodes: 199 against 204).
template <int D> struct FinishRows { static constexpr int BLOCK = D < 64 ? D : 64, LANE = D < 64 ? 1 : 2; };

template <typename E, int D, bool SPLIT, int PER_SM>
__global__ void __launch_bounds__(256, PER_SM) tree_finish(TreeArgs a, int segments)
{
    constexpr int RB = FinishRows<D>::BLOCK, R = FinishRows<D>::LANE;
    const Paged &c = a.c;
    const int bh = (int)blockIdx.x / (D / RB), rb = (int)blockIdx.x % (D / RB), b = bh / c.H, h = bh % c.H;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, row = rb * RB + lane % RB, n0 = 8 * warp;  // (and row + 32)
    extern __shared__ __align__(16) float dyn[];
    float *Ps = dyn, *As = Ps + a.T * a.Tp;          // [m][Tp]
    float *ws = As + (a.delta ? a.T * a.Tp : 0);     // SPLIT: [segment][Tp] path weights; a path has path_segments() of them
    __shared__ float es[kMaxTree][32 * R];
    __shared__ uint64_t anc[kMaxTree];
    __shared__ uint64_t seg_set[kMaxTree];
    __shared__ int seg[kMaxTree];
    __shared__ float share[kMaxTree], into[kMaxTree], first[kMaxTree], tops[kMaxTree], invs[kMaxTree];
    const size_t at = (size_t)bh * a.T;
    after_previous();
    const Line line = line_in(a.line, a.B);
    const int where = line.row[b], pos = line.pos[b], m = line.nodes[b];
    // rows of V, Z and the begun memory's read: not all of them count, but all are there
    float e[8][R], z[8][R], y[8][R];
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = n0 + x < a.T;
            const size_t there = ((size_t)bh * a.Tp + n0 + x) * D + row + 32 * r;
            e[x][r] = in ? to_f(static_cast<const E *>(a.v)[(at + n0 + x) * D + row + 32 * r]) : 0.f;
            z[x][r] = in && a.delta ? a.Z[there] : 0.f;
            y[x][r] = in && SPLIT ? a.Y0[there] : 0.f;
        }
    for (int i = tid; i < a.T * a.Tp / 4; i += blockDim.x) {
        mma::cp16(mma::smem_addr(Ps + 4 * i), a.P + at * a.Tp + 4 * i, true);
        if (a.delta) mma::cp16(mma::smem_addr(As + 4 * i), a.A + at * a.Tp + 4 * i, true);
    }
    mma::cp_commit();
    if (where < 0 || m == 0) {
        mma::cp_wait<0>();
        return;
    }
    const int nb = cached_segments(c, pos), in0 = pos % c.C;
    const Parts parts(a, line, b, h, SPLIT ? nb : nb + (in0 ? 1 : 0));
    constexpr bool HALVES = SPLIT && D == 64;  // two memories of 64 rows go through the tensor cores at once: a read is two sums
    const size_t second = (a.ranges + (size_t)a.B * c.H) * a.Tp * D;
    float p2[8][R] = {};  // (of the second halves)
    float p[8][R];  // partial reads: the next ones, under way
    auto fetch = [&](int j) {
        const float *src = a.part + (((size_t)j + bh) * a.Tp + n0) * D + row;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool there = j <= parts.j1 && n0 + x < m;
                p[x][r] = there ? src[(size_t)x * D + 32 * r] : 0.f;
                if (HALVES) p2[x][r] = there ? src[second + (size_t)x * D + 32 * r] : 0.f;
            }
    };
    fetch(parts.j0);
    for (int n = tid; n < kMaxTree; n += blockDim.x) {
        const bool in = n < m;
        const uint64_t set = in ? a.anc[(size_t)b * kMaxTree + n] : 0;
        if (!SPLIT) {
            anc[n] = set;
            into[n] = in ? a.gates[((size_t)bh * (c.nmax + 2) + nb + 1) * a.Tp + n] : 0.f;
        } else if (in) {
            // two path segments and four parts are the rule: their loads do not wait for one another
            const float *score = a.score + (size_t)bh * segments * a.Tp + n;
            const float2 *weight = a.weight + (size_t)bh * a.Tp + n;
            const int last = a.seg[(size_t)b * kMaxTree + n];
            float d = a.into[(size_t)bh * a.Tp + n];
            const float s0 = score[0], s1 = score[segments > 1 ? a.Tp : 0];
            float2 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = parts.j0 + j <= parts.j1 ? weight[(size_t)(parts.j0 + j) * a.Tp] : make_float2(-FLT_MAX, 0.f);
            auto path = [&](int j) { return j == 0 ? s0 : j == 1 ? s1 : score[(size_t)j * a.Tp]; };
            if (!in0) d = 0.f;
            float top = fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x));
            for (int j = parts.j0 + 4; j <= parts.j1; ++j) top = fmaxf(top, weight[(size_t)j * a.Tp].x);
            for (int j = 0; j <= last; ++j) top = fmaxf(top, path(j));
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += w[j].y * expf(w[j].x - top);
            for (int j = parts.j0 + 4; j <= parts.j1; ++j) sum += weight[(size_t)j * a.Tp].y * expf(weight[(size_t)j * a.Tp].x - top);
            for (int j = 0; j <= last; ++j) sum += ws[j * a.Tp + n] = expf(path(j) - top);
            const float inv = a.mode == MC_RESIDUAL ? 1.f : 1.f / sum;
            for (int j = 0; j <= last; ++j) ws[j * a.Tp + n] *= inv;
            anc[n] = set;
            seg[n] = last;
            tops[n] = top;
            invs[n] = inv;
            first[n] = ws[n] * d;           // of the begun memory's read
            into[n] = last == 0 ? d : 0.f;  // of what it answers to the key
        } else {
            anc[n] = 0;
        }
    }
    mma::cp_wait<0>();
    __syncthreads();
    if (SPLIT) {  // the path segments' nodes
        if (tid < segments) seg_set[tid] = 0;
        __syncthreads();
        if (tid < m) atomicOr(reinterpret_cast<unsigned *>(&seg_set[seg[tid]]) + tid / 32, 1u << (tid % 32));
    }
    uint64_t above = 0;  // ancestors of any of the warp's nodes
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int n = n0 + x;
        if (n < m) above |= anc[n];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (n >= m) e[x][r] = y[x][r] = 0.f;
            else {
                if (a.delta && into[n] != 0.f) e[x][r] -= SPLIT ? into[n] * z[x][r] : z[x][r];
                y[x][r] = SPLIT && in0 ? first[n] * y[x][r] : 0.f;
            }
        }
    }
    for (int j = parts.j0; j <= parts.j1; ++j) {
        if (SPLIT) {
            __syncthreads();
            for (int n = tid; n < m; n += blockDim.x) share[n] = expf(a.weight[((size_t)j + bh) * a.Tp + n].x - tops[n]) * invs[n];
            __syncthreads();
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (n0 + x < m) {
                const float w = SPLIT ? share[n0 + x] : 1.f;
#pragma unroll
                for (int r = 0; r < R; ++r) y[x][r] = fmaf(w, HALVES ? p[x][r] + p2[x][r] : p[x][r], y[x][r]);
            }
        if (j < parts.j1) fetch(j + 1);
    }
    // to[x] += sign W_{j,x} ej for this warp's nodes x: W of one that j is no ancestor of is 0, but ej may not be finite, and
    // then it is not multiplied
    auto take = [&](const float *W, float sign, int j, const float (&ej)[R], float (&to)[8][R]) {
        const float4 w0 = load4(W + j * a.Tp + n0), w1 = load4(W + j * a.Tp + n0 + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        bool finite = true;
#pragma unroll
        for (int r = 0; r < R; ++r) finite &= isfinite(ej[r]);
        if (finite) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
                for (int r = 0; r < R; ++r) to[x][r] = fmaf(sign * w[x], ej[r], to[x][r]);
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (w[x] != 0.f)
#pragma unroll
                    for (int r = 0; r < R; ++r) to[x][r] = fmaf(sign * w[x], ej[r], to[x][r]);
        }
    };
    __syncthreads();
    const bool mine = n0 < m;
    if (a.delta) {
        for (int k = 0; 8 * k < m; ++k) {
            if (warp == k) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n0 + j < m) {
                        float ej[R];
#pragma unroll
                        for (int r = 0; r < R; ++r) es[n0 + j][lane + 32 * r] = ej[r] = e[j][r];
                        take(As, -1.f, n0 + j, ej, e);
                    }
            }
            __syncthreads();
            if (warp > k && mine && ((above >> (8 * k)) & 255)) {
#pragma unroll 4
                for (int j = 8 * k; j < 8 * k + 8; ++j) {
                    if (!((above >> j) & 1)) continue;
                    float ej[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) ej[r] = es[j][lane + 32 * r];
                    take(As, -1.f, j, ej, e);
                }
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int r = 0; r < R; ++r) es[n0 + x][lane + 32 * r] = e[x][r];
        __syncthreads();
    }
    if (mine) {
        auto read = [&](uint64_t of, float (&to)[8][R]) {
#pragma unroll 4
            for (int j = 0; j < min(n0 + 8, m); ++j) {
                if (!((of >> j) & 1)) continue;
                float ej[R];
#pragma unroll
                for (int r = 0; r < R; ++r) ej[r] = es[j][lane + 32 * r];
                take(Ps, 1.f, j, ej, to);
            }
        };
        if (!SPLIT) {
            read(above, y);
        } else {
            for (int k = 0; k < segments; ++k) {
                const uint64_t of = above & seg_set[k];
                if (!of) continue;
                float part[8][R] = {};
                read(of, part);
#pragma unroll
                for (int x = 0; x < 8; ++x)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (n0 + x < m && seg[n0 + x] >= k) y[x][r] = fmaf(ws[k * a.Tp + n0 + x], part[x][r], y[x][r]);
            }
        }
    }
    if (lane < RB) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (n0 + x < m) static_cast<E *>(a.y)[(at + n0 + x) * D + row + 32 * r] = from_f<E>(y[x][r]);
    }
}

// ------------------------------------------------------------------------------------------------ launchers

template <typename E, int D>
cudaError_t gates_impl(const TreeArgs &a, cudaStream_t s)
{
    const size_t heads = (size_t)a.B * a.c.H;
    return a.whole ? launch_early(tree_gates<E, D, true>, heads * WholeRows<D>::CTAS, kGateThreads, gates_smem(a), s, a)
                   : launch_early(tree_gates<E, D, false>, heads * a.groups + 1, kGateThreads, gates_smem(a), s, a);
}

template <typename E, int D>
cudaError_t read_impl(const TreeArgs &a, cudaStream_t s)
{
    const size_t grid = (size_t)a.ranges * a.groups * read_blocks(D), smem = sizeof(int) * Line::ints(a.B);
    return a.T == 1   ? launch_early(tree_read<E, D, 1>, grid, 256, smem, s, a)
           : a.T == 2 ? launch_early(tree_read<E, D, 2>, grid, 256, smem, s, a)
           : a.T <= 4 ? launch_early(tree_read<E, D, 4>, grid, 256, smem, s, a)
                      : launch_early(tree_read<E, D, 8>, grid, 256, smem, s, a);
}

template <typename E, int D>
cudaError_t finish_impl(const TreeArgs &a, cudaStream_t s)
{
    const size_t grid = (size_t)a.B * a.c.H * (D / FinishRows<D>::BLOCK);
    const bool split = tree_tc_supported(a);
    const size_t smem = sizeof(float) * ((size_t)(a.delta ? 2 : 1) * a.T + (split ? path_segments(a) : 0)) * a.Tp;
    const int block = 32 * a.groups;  // a warp to eight nodes
    if constexpr (sizeof(E) == 2 && D >= 64) {
        if (split) {
            const bool room = grid * block <= 152 * 512;
            return room ? launch_early(tree_finish<E, D, true, 2>, grid, block, smem, s, a, path_segments(a))
                        : launch_early(tree_finish<E, D, true, 3>, grid, block, smem, s, a, path_segments(a));
        }
    }
    return launch_early(tree_finish<E, D, false, 3>, grid, block, smem, s, a, path_segments(a));
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

// While the memories that there is room for come to no more than 40 MB: 4 heads of d = 64 over 5 segments, 8 nodes, 11 us in one
// launch and 17 in three; 16 heads of d = 128 over 20, 18 and 28; over 63 (66 MB) 48 and 39.  The host knows the room, not
// what is cached: in a table of 1024 the first of these takes the three launches (34 us cold against 16).
bool tree_whole(const TreeArgs &a)
{
    return a.T <= kGroup && (long long)a.B * a.c.H * (a.c.nmax + 1) * a.c.d * a.c.d * 4 <= 40 << 20;
}
cudaError_t launch_tree_gates(const TreeArgs &a, cudaStream_t s) { return run(a, s, 0); }
cudaError_t launch_tree_read(const TreeArgs &a, cudaStream_t s) { return run(a, s, 1); }
cudaError_t launch_tree_finish(const TreeArgs &a, cudaStream_t s) { return run(a, s, 2); }

}  // namespace mc
