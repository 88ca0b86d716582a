// k_delta_simt.cu -- CUDA-core (FFMA) kernels of the gated delta memory: its forward scan, its
// reverse scan and the gradients, for fp32 inputs and for d in {16, 32} (fp32 arithmetic end to
// end), and the pooled-key sums that every delta path needs.
//
// Per (b,h) and segment, from an empty memory, with a_t = exp(log_alpha_t):
//   e_t = v_t - a_t M_{t-1} k_t            the error of the decayed memory at the new key
//   M_t = a_t M_{t-1} + beta_t e_t k_t^T   the write,   o_t = M_t q_t   the read
// Value row r of M depends on row r of v alone, so the rows are independent walkers.
//
// Adjoint, with N_t the gradient of M_t through o_t and every later step, p_t = g_t dy_t:
//   N_t += p_t q_t^T,  z_t = N_t k_t,  w_t = beta_t z_t,  N_{t-1} = a_t (N_t - w_t k_t^T)
//   dv_t = w_t,  dbeta_t = z_t . e_t,  dq_t = M_t^T p_t,  dk_t = beta_t N_t^T e_t - a_t M_{t-1}^T w_t
//   dlog_alpha_t = <N_{t-1}, M_{t-1}> = h_t,  and since o_t and e_t are linear in M,
//   h_t = h_{t+1} + p_t . o_t - w_t . v_t  (p_t . o_t = dq_t . q_t), restarted from
//   <N, M> at every 64-token chunk's end so that no rounding runs along a whole segment.
// The rows of N are independent walkers too.  What sums over rows (dq, dk, dbeta, dlog_alpha) is
// formed per 64-token chunk from the states at the chunk's two ends: with S the memory before the
// chunk, R the adjoint after it, c_i the running sum of log_alpha in the chunk, D_ij = exp(c_i - c_j),
//   B1_ij = D_ij p_i.e_j (i >= j),  B2_ij = D_ij w_i.e_j (i > j)
//   Y_j   = sum_i B1_ij q_i + D_Cj R^T e_j - sum_i B2_ij k_i          (= N_j^T e_j)
//   dk_j  = beta_j Y_j - exp(c_j) S^T w_j - sum_i B2_ji beta_i k_i,   dbeta_j = Y_j . k_j
//   dq_i  = exp(c_i) S^T p_i + sum_j B1_ij beta_j k_j
#include <cstdint>

#include "mc_internal.cuh"
#include "mma_sync.cuh"

namespace mc {
namespace {

constexpr int kCH = kDeltaChunk;  // 64 tokens

template <typename F>
cudaError_t set_smem(F *kern, size_t bytes)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// A row of M lies on G neighbouring lanes, KPL keys each: lane g holds the 16-byte pieces
// g, g + G, ... of the row, so that the lanes of a row read one run of shared memory.
template <int D>
struct RowSplit {
    static constexpr int KPL = D >= 64 ? 16 : 8;
    static constexpr int G = D / KPL;
    static constexpr int RW = 32 / G;                          // rows per warp
    static constexpr int W = D / RW < 4 ? D / RW : 4;          // warps per CTA
    static constexpr int RC = RW * W;                          // rows per CTA
    static constexpr int TT = 16;                              // tokens staged at once
};

template <int D>
__device__ __forceinline__ void load_keys(float (&x)[RowSplit<D>::KPL], const float *row, int g)
{
    constexpr int G = RowSplit<D>::G;
#pragma unroll
    for (int m = 0; m < RowSplit<D>::KPL / 4; ++m) {
        const float4 f = reinterpret_cast<const float4 *>(row)[g + G * m];
        x[4 * m] = f.x; x[4 * m + 1] = f.y; x[4 * m + 2] = f.z; x[4 * m + 3] = f.w;
    }
}

template <int D>
__device__ __forceinline__ void store_keys(float *row, const float (&x)[RowSplit<D>::KPL], int g)
{
    constexpr int G = RowSplit<D>::G;
#pragma unroll
    for (int m = 0; m < RowSplit<D>::KPL / 4; ++m)
        reinterpret_cast<float4 *>(row)[g + G * m] = make_float4(x[4 * m], x[4 * m + 1], x[4 * m + 2], x[4 * m + 3]);
}

template <int D>
__device__ __forceinline__ float dot_keys(const float (&x)[RowSplit<D>::KPL], const float (&y)[RowSplit<D>::KPL])
{
    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RowSplit<D>::KPL; ++i) p[i & 3] = fmaf(x[i], y[i], p[i & 3]);
    float s = (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
    for (int o = RowSplit<D>::G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The row with two vectors at once: their lanes' sums go side by side.
template <int D>
__device__ __forceinline__ float2 dot2_keys(const float (&m)[RowSplit<D>::KPL], const float (&x)[RowSplit<D>::KPL],
                                            const float (&y)[RowSplit<D>::KPL])
{
    float p[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RowSplit<D>::KPL; ++i) {
        p[i & 3] = fmaf(m[i], x[i], p[i & 3]);
        q[i & 3] = fmaf(m[i], y[i], q[i & 3]);
    }
    float2 s = make_float2((p[0] + p[1]) + (p[2] + p[3]), (q[0] + q[1]) + (q[2] + q[3]));
#pragma unroll
    for (int o = RowSplit<D>::G / 2; o > 0; o >>= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, s.x, o), b = __shfl_xor_sync(0xffffffffu, s.y, o);
        s.x += a;
        s.y += b;
    }
    return s;
}

// ---------------------------------------------------------------------------
// delta_scan_simt: one CTA per (bh, segment, RC value rows).  Bound by the chain of one token to the next; the row
// stays in registers, its read by q_t and by the next key go side by side, and the rows, heads and segments run in
// parallel.  4 heads of 1024 tokens, fp32, d = 64: 186 us, 0.18 us a token (208 with the two reads one after the other; a
// row over twice as many lanes 202; the reverse scan with its next vectors loaded ahead 171 instead of 162).
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(32 * RowSplit<D>::W) delta_scan_simt(DeltaArgs a)
{
    using R = RowSplit<D>;
    constexpr int NT = 32 * R::W;
    __shared__ __align__(16) float Ks[(R::TT + 1) * D], Qs[R::TT * D], Vs[R::TT * R::RC];
    __shared__ float As[R::TT], Bs[R::TT];
    constexpr int splits = D / R::RC;
    const int rs = blockIdx.x % splits;
    const int seg = (int)(blockIdx.x / splits) % a.N, bh = (int)(blockIdx.x / splits) / a.N;
    const int t0 = seg * a.C, t1 = min(t0 + a.C, a.L);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane % R::G;
    const int rl = warp * R::RW + lane / R::G, row = rs * R::RC + rl;
    const size_t base = (size_t)bh * a.L * D, sbase = (size_t)bh * a.L;
    const T *q = static_cast<const T *>(a.q) + base, *k = static_cast<const T *>(a.k) + base;
    const T *v = static_cast<const T *>(a.v) + base;
    const T *la = static_cast<const T *>(a.la) + sbase, *be = static_cast<const T *>(a.be) + sbase;
    float M[R::KPL], x[R::KPL];
#pragma unroll
    for (int i = 0; i < R::KPL; ++i) M[i] = 0.f;
    constexpr int NL = (R::TT * D + NT - 1) / NT, NV = (R::TT * R::RC + NT - 1) / NT;
    T kn[NL], qn[NL], vn[NV], an, bn;  // the next tile, on its way while this one is worked on
    auto fetch = [&](int c0) {
        const int cnt = min(R::TT, t1 - c0);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = tid + i * NT;
            if (e < cnt * D) {
                kn[i] = k[(size_t)c0 * D + e];
                qn[i] = q[(size_t)c0 * D + e];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + i * NT;
            if (e < cnt * R::RC) vn[i] = v[(size_t)(c0 + e / R::RC) * D + rs * R::RC + e % R::RC];
        }
        if (tid < cnt) {
            an = la[c0 + tid];
            bn = be[c0 + tid];
        }
    };
    for (int e = tid; e < D; e += NT) Ks[R::TT * D + e] = 0.f;  // (read, not used)
    fetch(t0);
    for (int c0 = t0; c0 < t1; c0 += R::TT) {
        const int cnt = min(R::TT, t1 - c0);
        if (a.S_c && (c0 - t0) % kCH == 0)
            store_keys<D>(a.S_c + (((size_t)bh * a.N + seg) * a.NCH + (c0 - t0) / kCH) * D * D + (size_t)row * D, M, g);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = tid + i * NT;
            if (e < cnt * D) {
                Ks[e] = to_f(kn[i]);
                Qs[e] = to_f(qn[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * NT < cnt * R::RC) Vs[tid + i * NT] = to_f(vn[i]);
        if (tid < cnt) {
            As[tid] = delta_decay(to_f(an));
            Bs[tid] = to_f(bn);
        }
        if (c0 + R::TT < t1) fetch(c0 + R::TT);
        __syncthreads();
        float z[R::KPL], y[R::KPL];
        load_keys<D>(x, Ks, g);
        float mk = dot_keys<D>(M, x);  // M_{t-1} k_t
        size_t at_ = base + (size_t)c0 * D + row;
        auto token = [&](int t, const float (&kt)[R::KPL], float (&kn)[R::KPL]) {
            const float at = As[t];
            load_keys<D>(y, Qs + t * D, g);
            load_keys<D>(kn, Ks + (t + 1) * D, g);
            const float e = Vs[t * R::RC + rl] - at * mk;
            const float ue = Bs[t] * e;
#pragma unroll
            for (int i = 0; i < R::KPL; ++i) M[i] = fmaf(ue, kt[i], at * M[i]);
            const float2 oz = dot2_keys<D>(M, y, kn);
            mk = oz.y;
            if (g == 0) {
                if (a.y) static_cast<T *>(a.y)[at_] = from_f<T>(oz.x);
                if (a.O_on) a.O_on[at_] = oz.x;
                if (a.E) a.E[at_] = e;
            }
            at_ += D;
        };
        for (int t = 0; t < cnt; t += 2) {
            token(t, x, z);
            if (t + 1 < cnt) token(t + 1, z, x);
        }
    }
    if (a.states) store_keys<D>(a.states + ((size_t)bh * a.N + seg) * D * D + (size_t)row * D, M, g);
}

// The same walk backwards over the adjoint N: dv_t = w_t (and fp32 w for the chunks), R at every chunk's end.
template <typename T, int D>
__global__ void __launch_bounds__(32 * RowSplit<D>::W) delta_rscan_simt(DeltaArgs a)
{
    using R = RowSplit<D>;
    constexpr int NT = 32 * R::W;
    __shared__ __align__(16) float Ks[R::TT * D], Qs[R::TT * D], Ps[R::TT * R::RC];
    __shared__ float As[R::TT], Bs[R::TT], Gs[R::TT];
    constexpr int splits = D / R::RC;
    const int rs = blockIdx.x % splits;
    const int seg = (int)(blockIdx.x / splits) % a.N, bh = (int)(blockIdx.x / splits) / a.N;
    const int t0 = seg * a.C, t1 = min(t0 + a.C, a.L);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane % R::G;
    const int rl = warp * R::RW + lane / R::G, row = rs * R::RC + rl;
    const size_t base = (size_t)bh * a.L * D, sbase = (size_t)bh * a.L;
    const T *q = static_cast<const T *>(a.q) + base, *k = static_cast<const T *>(a.k) + base;
    const T *dy = static_cast<const T *>(a.dy) + base;
    const T *la = static_cast<const T *>(a.la) + sbase, *be = static_cast<const T *>(a.be) + sbase;
    T *dv = static_cast<T *>(a.dv) + base;
    float N[R::KPL], kx[R::KPL], qx[R::KPL];
#pragma unroll
    for (int i = 0; i < R::KPL; ++i) N[i] = 0.f;
    if (a.G && seg < a.N - 1)
        for (int part = 0; part < a.g_parts; ++part) {
            load_keys<D>(kx, a.G + (((size_t)part * a.BH + bh) * a.N + seg) * D * D + (size_t)row * D, g);
#pragma unroll
            for (int i = 0; i < R::KPL; ++i) N[i] += kx[i];
        }
    const int nt = (t1 - t0 + R::TT - 1) / R::TT;
    constexpr int NL = (R::TT * D + NT - 1) / NT, NV = (R::TT * R::RC + NT - 1) / NT;
    T kn[NL], qn[NL], pn[NV], an, bn;
    float gn = 1.f;
    auto fetch = [&](int c0) {
        const int cnt = min(R::TT, t1 - c0);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = tid + i * NT;
            if (e < cnt * D) {
                kn[i] = k[(size_t)c0 * D + e];
                qn[i] = q[(size_t)c0 * D + e];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + i * NT;
            if (e < cnt * R::RC) pn[i] = dy[(size_t)(c0 + e / R::RC) * D + rs * R::RC + e % R::RC];
        }
        if (tid < cnt) {
            an = la[c0 + tid];
            bn = be[c0 + tid];
            if (a.tok) gn = a.tok[(sbase + c0 + tid) * kBwdTokWords + 2];
        }
    };
    fetch(t0 + (nt - 1) * R::TT);
    for (int ti = nt - 1; ti >= 0; --ti) {
        const int c0 = t0 + ti * R::TT, cnt = min(R::TT, t1 - c0);
        if (c0 + cnt == t1 || (c0 + cnt - t0) % kCH == 0)
            store_keys<D>(a.R_c + (((size_t)bh * a.N + seg) * a.NCH + (c0 - t0) / kCH) * D * D + (size_t)row * D, N, g);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = tid + i * NT;
            if (e < cnt * D) {
                Ks[e] = to_f(kn[i]);
                Qs[e] = to_f(qn[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * NT < cnt * R::RC) Ps[tid + i * NT] = to_f(pn[i]);
        if (tid < cnt) {
            As[tid] = delta_decay(to_f(an));
            Bs[tid] = to_f(bn);
            Gs[tid] = gn;
        }
        if (ti > 0) fetch(c0 - R::TT);
        __syncthreads();
        for (int t = cnt - 1; t >= 0; --t) {
            load_keys<D>(qx, Qs + t * D, g);
            load_keys<D>(kx, Ks + t * D, g);
            const float p = Gs[t] * Ps[t * R::RC + rl];
#pragma unroll
            for (int i = 0; i < R::KPL; ++i) N[i] = fmaf(p, qx[i], N[i]);
            const float w = Bs[t] * dot_keys<D>(N, kx);
            const float at = As[t];
#pragma unroll
            for (int i = 0; i < R::KPL; ++i) N[i] = at * fmaf(-w, kx[i], N[i]);
            if (g == 0) {
                const size_t at_ = (size_t)(c0 + t) * D + row;
                dv[at_] = from_f<T>(w);
                a.W[base + at_] = w;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// delta_grads_simt: one CTA per (bh, segment, 64-token chunk): everything that sums over value
// rows, as in the header.  Tiles of q, k, p, e, w in shared memory (fp32, rows padded by one word);
// S and R come through in blocks of 32 rows.  tx = tid % 16, ty = tid / 16: a thread owns tokens
// ty + 16 p and dimensions tx + 16 r.
// ---------------------------------------------------------------------------
constexpr int kGT = 256;
constexpr int kGB = 32;  // rows of S and R at once (16 for d = 16)

template <int D>
constexpr size_t grads_smem()
{
    return sizeof(float) * (5 * kCH * (D + 1) + 2 * kCH * (kCH + 1) + (D < kGB ? D : kGB) * (D + 1) + 7 * kCH + 32);
}

template <typename T, int D>
__global__ void __launch_bounds__(kGT) delta_grads_simt(DeltaArgs a)
{
    constexpr int P = D + 1, BP = kCH + 1, RB = D / 16, TP = kCH / 16, GB = D < kGB ? D : kGB;
    extern __shared__ float sm[];
    float *Qs = sm, *Ks = Qs + kCH * P, *Ps = Ks + kCH * P, *Es = Ps + kCH * P, *Ws = Es + kCH * P;
    float *B1 = Ws + kCH * P, *B2 = B1 + kCH * BP, *Ms = B2 + kCH * BP;
    float *cum = Ms + GB * P, *bet = cum + kCH, *hd = bet + kCH, *hb = hd + kCH, *dbe = hb + kCH, *cul = dbe + kCH, *red = cul + kCH;

    const int ch = (int)blockIdx.x % a.NCH;
    const int seg = (int)(blockIdx.x / a.NCH) % a.N, bh = (int)(blockIdx.x / a.NCH) / a.N;
    const int t0 = seg * a.C, tb = t0 + ch * kCH, te = min(min(tb + kCH, t0 + a.C), a.L);
    if (tb >= te) return;
    const int cnt = te - tb, last = cnt - 1;
    const size_t base = (size_t)bh * a.L * D, sbase = (size_t)bh * a.L;
    const T *q = static_cast<const T *>(a.q) + base, *k = static_cast<const T *>(a.k) + base;
    const T *v = static_cast<const T *>(a.v) + base, *dy = static_cast<const T *>(a.dy) + base;
    const T *u = a.rho ? static_cast<const T *>(a.u) + base : nullptr;
    const T *la = static_cast<const T *>(a.la) + sbase, *be = static_cast<const T *>(a.be) + sbase;
    const size_t cidx = ((size_t)bh * a.N + seg) * a.NCH + ch;
    const float *S = a.S_c + cidx * D * D, *Rc = a.R_c + cidx * D * D;
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;

    for (int e = tid; e < kCH * D; e += kGT) {
        const int r = e / D, c = e % D;
        const bool ok = r < cnt;
        const size_t gi = (size_t)(tb + r) * D + c;
        const float gon = ok && a.tok ? a.tok[(sbase + tb + r) * kBwdTokWords + 2] : 1.f;
        Qs[r * P + c] = ok ? to_f(q[gi]) : 0.f;
        Ks[r * P + c] = ok ? to_f(k[gi]) : 0.f;
        Ps[r * P + c] = ok ? gon * to_f(dy[gi]) : 0.f;
        Es[r * P + c] = ok ? a.E[base + gi] : 0.f;
        Ws[r * P + c] = ok ? a.W[base + gi] : 0.f;
    }
    if (tid < kCH) {
        const float2 x = delta_parts(tid < cnt ? delta_log(to_f(la[tb + tid])) : 0.f);
        cum[tid] = x.x;
        cul[tid] = x.y;
        bet[tid] = tid < cnt ? to_f(be[tb + tid]) : 0.f;
        hd[tid] = hb[tid] = dbe[tid] = 0.f;
    }
    __syncthreads();
    if (tid == 0)
        for (int i = 1; i < kCH; ++i) {
            cum[i] += cum[i - 1];
            cul[i] += cul[i - 1];
        }
    __syncthreads();
    auto decay = [&](int i, int j) { return expf((cum[i] - cum[j]) + (cul[i] - cul[j])); };  // D_ij
    for (int e = tid; e < kCH * kCH; e += kGT) {
        const int i = e / kCH, j = e % kCH;
        float b1 = 0.f, b2 = 0.f;
        if (j <= i && i < cnt) {
            for (int c = 0; c < D; ++c) {
                b1 = fmaf(Ps[i * P + c], Es[j * P + c], b1);
                b2 = fmaf(Ws[i * P + c], Es[j * P + c], b2);
            }
            const float dec = decay(i, j);
            b1 *= dec;
            b2 = j < i ? b2 * dec : 0.f;
        }
        B1[i * BP + j] = b1;
        B2[i * BP + j] = b2;
    }
    // P S, W S, E R (rows of S and R by blocks)
    float xs[TP][RB], ws[TP][RB], er[TP][RB];
#pragma unroll
    for (int p = 0; p < TP; ++p)
#pragma unroll
        for (int r = 0; r < RB; ++r) xs[p][r] = ws[p][r] = er[p][r] = 0.f;
    float inner = 0.f;  // <R, S>, by element
    for (int b = 0; b < D; b += GB) {
        __syncthreads();
        for (int e = tid; e < GB * D; e += kGT) {
            const float s = S[(size_t)b * D + e];
            inner = fmaf(s, Rc[(size_t)b * D + e], inner);
            Ms[(e / D) * P + e % D] = s;
        }
        __syncthreads();
        for (int c = 0; c < GB; ++c) {
            float m[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) m[r] = Ms[c * P + tx + 16 * r];
#pragma unroll
            for (int p = 0; p < TP; ++p) {
                const float pv = Ps[(ty + 16 * p) * P + b + c], wv = Ws[(ty + 16 * p) * P + b + c];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    xs[p][r] = fmaf(pv, m[r], xs[p][r]);
                    ws[p][r] = fmaf(wv, m[r], ws[p][r]);
                }
            }
        }
        __syncthreads();
        for (int e = tid; e < GB * D; e += kGT) Ms[(e / D) * P + e % D] = Rc[(size_t)b * D + e];
        __syncthreads();
        for (int c = 0; c < GB; ++c) {
            float m[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) m[r] = Ms[c * P + tx + 16 * r];
#pragma unroll
            for (int p = 0; p < TP; ++p) {
                const float ev = Es[(ty + 16 * p) * P + b + c];
#pragma unroll
                for (int r = 0; r < RB; ++r) er[p][r] = fmaf(ev, m[r], er[p][r]);
            }
        }
    }
    // <R, S> of the chunk over the CTA, in a fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
    if (tid % 32 == 0) red[tid / 32] = inner;
    T *dqo = static_cast<T *>(a.dq) + base, *dko = static_cast<T *>(a.dk) + base;
    float dk[TP][RB];
#pragma unroll
    for (int p = 0; p < TP; ++p) {
        const int t = ty + 16 * p;
        const float ge = expf(cum[t] + cul[t]), gr = decay(last, t);
        float dq[RB], y[RB], kk[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            dq[r] = ge * xs[p][r];
            y[r] = gr * er[p][r];
            kk[r] = -ge * ws[p][r];
        }
        float hpart = 0.f;  // beta_t D_Ct (R^T e_t) . k_t, the chunk's own share of <R, M at its end>
#pragma unroll
        for (int r = 0; r < RB; ++r) hpart = fmaf(y[r], Ks[t * P + tx + 16 * r], hpart);
        for (int j = 0; j <= t; ++j) {
            const float b1 = B1[t * BP + j] * bet[j], b2 = B2[t * BP + j] * bet[j];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const float kj = Ks[j * P + tx + 16 * r];
                dq[r] = fmaf(b1, kj, dq[r]);
                kk[r] = fmaf(-b2, kj, kk[r]);
            }
        }
        for (int i = t; i < cnt; ++i) {
            const float b1 = B1[i * BP + t], b2 = B2[i * BP + t];
#pragma unroll
            for (int r = 0; r < RB; ++r)
                y[r] = fmaf(b1, Qs[i * P + tx + 16 * r], fmaf(-b2, Ks[i * P + tx + 16 * r], y[r]));
        }
        float dbp = 0.f, hq = 0.f, hv = 0.f;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int c = tx + 16 * r;
            dk[p][r] = fmaf(bet[t], y[r], kk[r]);
            dbp = fmaf(y[r], Ks[t * P + c], dbp);
            hq = fmaf(dq[r], Qs[t * P + c], hq);
            if (t < cnt) {
                const size_t gi = (size_t)(tb + t) * D + c;
                hv = fmaf(Ws[t * P + c], to_f(v[gi]), hv);
                dqo[gi] = from_f<T>(dq[r] + (a.dq_add ? a.dq_add[base + gi] : 0.f));
            }
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            dbp += __shfl_xor_sync(0xffffffffu, dbp, o);
            hq += __shfl_xor_sync(0xffffffffu, hq, o);
            hv += __shfl_xor_sync(0xffffffffu, hv, o);
            hpart += __shfl_xor_sync(0xffffffffu, hpart, o);
        }
        if (tx == 0) {
            dbe[t] = dbp;
            hd[t] = hq - hv;
            hb[t] = bet[t] * hpart;
        }
    }
    __syncthreads();
    if (tid == 0) {  // h backwards over the chunk
        float in = 0.f;
        for (int w = 0; w < kGT / 32; ++w) in += red[w];
        float h = expf(cum[last] + cul[last]) * in;
        for (int t = 0; t < cnt; ++t) h += hb[t];
        for (int t = last; t >= 0; --t) {
            h += hd[t];
            hd[t] = h;
        }
    }
    // the pooled keys' share of dk: sum over the segment's tokens from t on of w_t' u_t' (word 4 of tok)
    if (a.rho) {
        __syncthreads();
        if (tid < D) {
            float acc = a.rho[cidx * D + tid];
            for (int t = last; t >= 0; --t) {
                acc = fmaf(a.tok[(sbase + tb + t) * kBwdTokWords + 4], to_f(u[(size_t)(tb + t) * D + tid]), acc);
                Ps[t * P + tid] = acc;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < TP; ++p) {
        const int t = ty + 16 * p;
        if (t >= cnt) continue;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int c = tx + 16 * r;
            dko[(size_t)(tb + t) * D + c] = from_f<T>(dk[p][r] + (a.rho ? Ps[t * P + c] : 0.f));
        }
    }
    if (tid < cnt) {
        static_cast<T *>(a.dbe)[sbase + tb + tid] = from_f<T>(dbe[tid]);
        // a segment's first decay meets an empty memory
        static_cast<T *>(a.dla)[sbase + tb + tid] = from_f<T>(tb + tid == t0 ? 0.f : hd[tid]);
    }
}

// ---------------------------------------------------------------------------
// Pooled sums over the 64-token chunks of every segment: x_t, or s_t x_t.
//   pool_sums : per chunk, the sum over its tokens                       -> out [BH][N][NCH][d]
//   pool_scan : per segment, exclusive prefix (keys; and the key mean) or exclusive suffix
//               plus dkbar / segment length (the gradient), in place
//   pool_score: r_on[t] = <u_t, keys of the segment up to t> / their number
// ---------------------------------------------------------------------------
// A chunk's rows in 16-byte pieces: thread (lane tl, piece pc) takes the TPL tokens from tl TPL on.
template <typename T, int D>
struct PoolTile {
    static constexpr int V = 16 / (int)sizeof(T), PC = D / V;
    static constexpr int TL = 256 / PC < kCH ? 256 / PC : kCH;
    static constexpr int TPL = kCH / TL;
    static constexpr int NT = TL * PC;  // threads at work
};
template <typename T, int V>
__device__ __forceinline__ void load_piece(float (&x)[V], const T *src)
{
    const uint4 q = *reinterpret_cast<const uint4 *>(src);
    const T *t = reinterpret_cast<const T *>(&q);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f(t[i]);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) pool_sums(DeltaArgs a, const T *x, const float *pw, float *out)
{
    using P = PoolTile<T, D>;
    __shared__ float part[P::TL * (D + 1)];
    const int ch = (int)(blockIdx.x % a.NCH);
    const int seg = (int)(blockIdx.x / a.NCH) % a.N, bh = (int)(blockIdx.x / a.NCH) / a.N;
    const int t0 = seg * a.C, tb = t0 + ch * kCH, cnt = min(min(tb + kCH, t0 + a.C), a.L) - tb;
    if (cnt <= 0) return;
    const int tid = threadIdx.x, pc = tid % P::PC, tl = tid / P::PC;
    const size_t row0 = (size_t)bh * a.L + tb;
    if (tid < P::NT) {
        float s[P::V];
#pragma unroll
        for (int i = 0; i < P::V; ++i) s[i] = 0.f;
#pragma unroll
        for (int j = 0; j < P::TPL; ++j) {
            const int t = tl * P::TPL + j;
            if (t >= cnt) break;
            float v[P::V];
            load_piece<T, P::V>(v, x + (row0 + t) * D + pc * P::V);
            const float f = pw ? pw[(row0 + t) * a.gw_stride] : 1.f;
#pragma unroll
            for (int i = 0; i < P::V; ++i) s[i] = fmaf(f, v[i], s[i]);
        }
#pragma unroll
        for (int i = 0; i < P::V; ++i) part[tl * (D + 1) + pc * P::V + i] = s[i];
    }
    __syncthreads();
    if (tid < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < P::TL; ++i) s += part[i * (D + 1) + tid];
        out[(size_t)blockIdx.x * D + tid] = s;
    }
}

template <int D>
__global__ void __launch_bounds__(D) pool_scan(DeltaArgs a, float *sums, float *kbar, const float *dkbar)
{
    const int seg = (int)blockIdx.x % a.N, bh = (int)blockIdx.x / a.N, c = threadIdx.x;
    const int len = min((seg + 1) * a.C, a.L) - seg * a.C, n = (len + kCH - 1) / kCH;
    float *s = sums + (size_t)blockIdx.x * a.NCH * D + c;
    if (!dkbar) {
        float acc = 0.f;
        for (int i = 0; i < n; ++i) {
            const float x = s[(size_t)i * D];
            s[(size_t)i * D] = acc;
            acc += x;
        }
        if (kbar) kbar[((size_t)bh * a.N + seg) * D + c] = acc / (float)len;
        return;
    }
    float acc = dkbar[((size_t)bh * a.N + seg) * D + c] / (float)len;
    for (int i = n - 1; i >= 0; --i) {
        const float x = s[(size_t)i * D];
        s[(size_t)i * D] = acc;
        acc += x;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) pool_score(DeltaArgs a, const float *kpre, float *r_on)
{
    using P = PoolTile<T, D>;
    __shared__ float part[P::TL * (D + 1)];
    const int ch = (int)(blockIdx.x % a.NCH);
    const int seg = (int)(blockIdx.x / a.NCH) % a.N, bh = (int)(blockIdx.x / a.NCH) / a.N;
    const int t0 = seg * a.C, tb = t0 + ch * kCH, cnt = min(min(tb + kCH, t0 + a.C), a.L) - tb;
    if (cnt <= 0) return;
    const int tid = threadIdx.x, pc = tid % P::PC, tl = tid / P::PC;
    const size_t row0 = (size_t)bh * a.L + tb;
    const T *k = static_cast<const T *>(a.k), *u = static_cast<const T *>(a.u);
    float x[P::TPL][P::V];  // running key sums over the lane's tokens
#pragma unroll
    for (int j = 0; j < P::TPL; ++j) {
        const int t = tl * P::TPL + j;
        if (tid < P::NT && t < cnt) {
            load_piece<T, P::V>(x[j], k + (row0 + t) * D + pc * P::V);
        } else {
#pragma unroll
            for (int i = 0; i < P::V; ++i) x[j][i] = 0.f;
        }
        if (j > 0)
#pragma unroll
            for (int i = 0; i < P::V; ++i) x[j][i] += x[j > 0 ? j - 1 : 0][i];
    }
    if (tid < P::NT)
#pragma unroll
        for (int i = 0; i < P::V; ++i) part[tl * (D + 1) + pc * P::V + i] = x[P::TPL - 1][i];
    __syncthreads();
    if (tid < D) {  // keys of the segment before each lane's tokens
        float s = kpre[(size_t)blockIdx.x * D + tid];
#pragma unroll
        for (int i = 0; i < P::TL; ++i) {
            const float own = part[i * (D + 1) + tid];
            part[i * (D + 1) + tid] = s;
            s += own;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < P::TPL; ++j) {
        const int t = tl * P::TPL + j;
        float s = 0.f;
        if (tid < P::NT && t < cnt) {
            float v[P::V];
            load_piece<T, P::V>(v, u + (row0 + t) * D + pc * P::V);
#pragma unroll
            for (int i = 0; i < P::V; ++i) s = fmaf(v[i], x[j][i] + part[tl * (D + 1) + pc * P::V + i], s);
        }
#pragma unroll
        for (int o = P::PC / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (pc == 0 && tid < P::NT && t < cnt) r_on[row0 + t] = s / (float)(tb + t - t0 + 1);
    }
}

// The three passes in one, for many segments: one CTA per (bh, segment) goes through the chunks with the running key
// sum in shared memory, so k and u come from HBM once.  A thread copies the pieces that it will read itself, the
// next chunk's asynchronously, so the copies need no barrier; three CTAs on an SM (bf16, d = 128) keep 96 KB on their way.
// 16 heads of 65536 tokens: 109 us for 0.54 GB, 4.9 TB/s (three passes 158 us).
constexpr int kPoolStages = 2;
template <typename T, int D>
constexpr int pool_walk_smem(bool score) { return kPoolStages * (score ? 2 : 1) * PoolTile<T, D>::TPL * 256 * 16; }

template <typename T, int D, bool SCORE>
__global__ void __launch_bounds__(256) pool_walk(DeltaArgs a, float *kpre, float *kbar, float *r_on)
{
    using P = PoolTile<T, D>;
    constexpr int NS = kPoolStages, OPS = SCORE ? 2 : 1;
    extern __shared__ __align__(16) uint8_t fifo[];
    __shared__ float part[P::TL * (D + 1)];
    const int seg = (int)blockIdx.x % a.N, bh = (int)blockIdx.x / a.N;
    const int t0 = seg * a.C, len = min((seg + 1) * a.C, a.L) - t0, nch = (len + kCH - 1) / kCH;
    const int tid = threadIdx.x, pc = tid % P::PC, tl = tid / P::PC;
    const size_t row0 = (size_t)bh * a.L + t0;
    const T *k = static_cast<const T *>(a.k) + row0 * D + pc * P::V, *u = SCORE ? static_cast<const T *>(a.u) + row0 * D + pc * P::V : nullptr;
    const bool scored = SCORE && seg > 0;  // the first segment's gate is 1 whatever its score
    auto slot = [&](int ch, int op, int j) { return fifo + ((((ch % NS) * OPS + op) * P::TPL + j) * 256 + tid) * 16; };
    auto load = [&](int ch) {
        if (ch < nch && tid < P::NT) {
#pragma unroll
            for (int j = 0; j < P::TPL; ++j) {
                const int t = ch * kCH + tl * P::TPL + j;
                mma::cp16(mma::smem_addr(slot(ch, 0, j)), k + (size_t)(t < len ? t : 0) * D, t < len);
                if (scored) mma::cp16(mma::smem_addr(slot(ch, 1, j)), u + (size_t)(t < len ? t : 0) * D, t < len);
            }
        }
        mma::cp_commit();
    };
    float run = 0.f;  // (threads below D) the segment's sum of column tid so far
#pragma unroll
    for (int ch = 0; ch < NS - 1; ++ch) load(ch);
    for (int ch = 0; ch < nch; ++ch) {
        load(ch + NS - 1);
        mma::cp_wait<NS - 1>();
        float x[P::TPL][P::V];
        if (tid < P::NT) {
#pragma unroll
            for (int j = 0; j < P::TPL; ++j) {
                load_piece<T, P::V>(x[j], reinterpret_cast<const T *>(slot(ch, 0, j)));
                if (j > 0)
#pragma unroll
                    for (int i = 0; i < P::V; ++i) x[j][i] += x[j > 0 ? j - 1 : 0][i];
            }
#pragma unroll
            for (int i = 0; i < P::V; ++i) part[tl * (D + 1) + pc * P::V + i] = x[P::TPL - 1][i];
        }
        __syncthreads();
        if (tid < D) {
            float own[P::TL], s = run;
#pragma unroll
            for (int i = 0; i < P::TL; ++i) own[i] = part[i * (D + 1) + tid];
            if (kpre) kpre[((size_t)blockIdx.x * a.NCH + ch) * D + tid] = s;
#pragma unroll
            for (int i = 0; i < P::TL; ++i) {
                part[i * (D + 1) + tid] = s;
                s += own[i];
            }
            run = s;
            if (ch + 1 == nch) kbar[(size_t)blockIdx.x * D + tid] = s / (float)len;
        }
        __syncthreads();
        if (!SCORE) continue;
        float before[P::V];
        if (tid < P::NT)
#pragma unroll
            for (int i = 0; i < P::V; ++i) before[i] = part[tl * (D + 1) + pc * P::V + i];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < P::TPL; ++j) {
            const int t = ch * kCH + tl * P::TPL + j;
            float s = 0.f;
            if (scored && tid < P::NT) {
                float v[P::V];
                load_piece<T, P::V>(v, reinterpret_cast<const T *>(slot(ch, 1, j)));
#pragma unroll
                for (int i = 0; i < P::V; ++i) s = fmaf(v[i], x[j][i] + before[i], s);
            }
#pragma unroll
            for (int o = P::PC / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (pc == 0 && tid < P::NT && t < len) r_on[row0 + t] = s / (float)(t + 1);
        }
    }
    mma::cp_wait<0>();
}

template <typename T, int D>
cudaError_t scan_impl(const Problem &p, const DeltaArgs &a, cudaStream_t s)
{
    constexpr int splits = D / RowSplit<D>::RC;
    delta_scan_simt<T, D><<<(unsigned)((long long)p.BH * p.N * splits), 32 * RowSplit<D>::W, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t rscan_impl(const Problem &p, const DeltaArgs &a, cudaStream_t s)
{
    constexpr int splits = D / RowSplit<D>::RC;
    delta_rscan_simt<T, D><<<(unsigned)((long long)p.BH * p.N * splits), 32 * RowSplit<D>::W, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t grads_impl(const Problem &p, const DeltaArgs &a, cudaStream_t s)
{
    const size_t smem = grads_smem<D>();
    auto kern = delta_grads_simt<T, D>;
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)((long long)p.BH * p.N * a.NCH), kGT, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t pool_impl(const Problem &p, const DeltaArgs &a, float *sums, float *kbar, float *r_on, cudaStream_t s)
{
    const unsigned chunks = (unsigned)((long long)p.BH * p.N * a.NCH);
    // One pass where most SMs have a segment.  16 heads, segments of 1024, d = 128, one pass against three: 4 segments
    // 30 against 27 us (fp32 50 against 34), 8 segments 31 against 42 (50 against 60), 32 segments 70 against 121.
    if ((long long)p.BH * p.N >= 128) {
        auto kern = r_on ? pool_walk<T, D, true> : pool_walk<T, D, false>;
        const int smem = pool_walk_smem<T, D>(r_on != nullptr);
        cudaError_t e = set_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)(p.BH * p.N), 256, smem, s>>>(a, sums, kbar, r_on);
        return cudaGetLastError();
    }
    pool_sums<T, D><<<chunks, 256, 0, s>>>(a, static_cast<const T *>(a.k), nullptr, sums);
    pool_scan<D><<<(unsigned)((long long)p.BH * p.N), D, 0, s>>>(a, sums, kbar, nullptr);
    if (r_on) pool_score<T, D><<<chunks, 256, 0, s>>>(a, sums, r_on);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t pool_grad_impl(const Problem &p, const DeltaArgs &a, const float *pw, float *rho, const float *dkbar, cudaStream_t s)
{
    pool_sums<T, D><<<(unsigned)((long long)p.BH * p.N * a.NCH), 256, 0, s>>>(a, static_cast<const T *>(a.u), pw, rho);
    pool_scan<D><<<(unsigned)((long long)p.BH * p.N), D, 0, s>>>(a, rho, nullptr, dkbar);
    return cudaGetLastError();
}

#define MC_DELTA_DISPATCH(FN, p, ...)                                                               \
    do {                                                                                            \
        switch ((p).d) {                                                                            \
        case 16: return (p).bf16 ? FN<__nv_bfloat16, 16>(p, __VA_ARGS__) : FN<float, 16>(p, __VA_ARGS__);    \
        case 32: return (p).bf16 ? FN<__nv_bfloat16, 32>(p, __VA_ARGS__) : FN<float, 32>(p, __VA_ARGS__);    \
        case 64: return (p).bf16 ? FN<__nv_bfloat16, 64>(p, __VA_ARGS__) : FN<float, 64>(p, __VA_ARGS__);    \
        case 128: return (p).bf16 ? FN<__nv_bfloat16, 128>(p, __VA_ARGS__) : FN<float, 128>(p, __VA_ARGS__); \
        default: return cudaErrorInvalidValue;                                                      \
        }                                                                                           \
    } while (0)

}  // namespace

cudaError_t launch_delta_scan_simt(const Problem &p, const DeltaArgs &a, cudaStream_t s) { MC_DELTA_DISPATCH(scan_impl, p, a, s); }
cudaError_t launch_delta_rscan_simt(const Problem &p, const DeltaArgs &a, cudaStream_t s) { MC_DELTA_DISPATCH(rscan_impl, p, a, s); }
cudaError_t launch_delta_grads_simt(const Problem &p, const DeltaArgs &a, cudaStream_t s) { MC_DELTA_DISPATCH(grads_impl, p, a, s); }
cudaError_t launch_pool_simt(const Problem &p, const DeltaArgs &a, float *sums, float *kbar, float *r_on, cudaStream_t s)
{
    MC_DELTA_DISPATCH(pool_impl, p, a, sums, kbar, r_on, s);
}
cudaError_t launch_pool_grad_simt(const Problem &p, const DeltaArgs &a, const float *pw, float *rho, const float *dkbar, cudaStream_t s)
{
    MC_DELTA_DISPATCH(pool_grad_impl, p, a, pw, rho, dkbar, s);
}

}  // namespace mc
