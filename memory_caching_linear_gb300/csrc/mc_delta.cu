// mc_delta.cu -- the entry points of the gated delta memory and of the evicting decode cache
// (include/mc.h): argument checks, scratch, and the choice of kernels.
#include <algorithm>
#include <cstdint>

#include "mc_internal.cuh"

namespace mc {
namespace {

// A block of stream-ordered scratch handed out in 256-byte aligned pieces: a first walk with a null
// base adds the sizes up, a second one hands out the pointers.
struct Carver {
    char *base;
    size_t used;
    template <typename T>
    T *take(size_t count, bool want = true)
    {
        if (!want) return nullptr;
        char *p = base ? base + used : nullptr;
        used += round_up(sizeof(T) * count);
        return reinterpret_cast<T *>(p);
    }
};

int fail(cudaError_t e)
{
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? MC_ERR_ALLOC : MC_ERR_CUDA;
}

struct Call {
    Problem p;
    int NCH;
    bool uses_u;
};

int check_call(Call &c, int B, int H, int L, int d, int seg_len, int agg_mode, int topk, bool bf16)
{
    int st = check_shape(B, H, L, d, seg_len);
    if (st != MC_OK) return st;
    if (L > (1 << 30)) return MC_ERR_SHAPE;  // a segment's end, up to L + seg_len, is an int in the kernels
    if (seg_len > L) seg_len = L;
    Problem &p = c.p;
    p = Problem{};
    p.B = B; p.H = H; p.L = L; p.d = d; p.C = seg_len;
    p.N = (L + seg_len - 1) / seg_len;
    p.BH = B * H;
    p.bf16 = bf16;
    c.NCH = (seg_len + kDeltaChunk - 1) / kDeltaChunk;
    // one CTA per 64-token chunk, up to eight per segment
    if ((long long)p.BH * p.N * (c.NCH > 8 ? c.NCH : 8) >= (1ll << 31)) return MC_ERR_SHAPE;
    if (agg_mode < MC_RESIDUAL || agg_mode > MC_MEAN) return MC_ERR_MODE;
    c.uses_u = mode_uses_u(agg_mode) && p.N > 1;  // a single memory has nothing to weigh
    p.mode = agg_mode == MC_SOUP ? MC_GRM : agg_mode;  // the same function for a matrix memory
    if (agg_mode == MC_SSC) {
        if (topk < 0) return MC_ERR_TOPK;
        if (topk >= p.N - 1) p.mode = MC_GRM;
        else if (topk > kMaxTopk) return MC_ERR_TOPK;
    }
    p.topk = p.mode == MC_SSC ? topk : 0;
    return MC_OK;
}

bool any_null(std::initializer_list<const void *> ptrs)
{
    for (const void *x : ptrs)
        if (!x) return true;
    return false;
}

// NULL pointers are left to any_null.
bool any_misaligned(std::initializer_list<const void *> ptrs)
{
    for (const void *x : ptrs)
        if (!aligned16(x)) return true;
    return false;
}

DeltaArgs delta_args(const Call &c)
{
    DeltaArgs a{};
    a.BH = c.p.BH; a.L = c.p.L; a.C = c.p.C; a.N = c.p.N; a.NCH = c.NCH;
    return a;
}

DeltaTcArgs delta_tc_args(const Call &c, const void *q, const void *k, const void *v, const void *la, const void *be)
{
    DeltaTcArgs t{};
    t.q = static_cast<const __nv_bfloat16 *>(q);
    t.k = static_cast<const __nv_bfloat16 *>(k);
    t.v = static_cast<const __nv_bfloat16 *>(v);
    t.la = static_cast<const __nv_bfloat16 *>(la);
    t.be = static_cast<const __nv_bfloat16 *>(be);
    t.BH = c.p.BH; t.L = c.p.L; t.C = c.p.C; t.N = c.p.N; t.NCH = c.NCH;
    return t;
}

// bf16, d = 64 or 128.  One memory: the walk writes y.  Several: the walk writes the states and, in fp32, the online reads,
// whose terms may cancel and which it forms in two bf16 terms (at all but parallel keys one term left y 4e-2 off); the
// readout adds the cached memories, on the tensor cores where it takes the shape.
int forward_delta_tc(const Call &c, const void *q, const void *k, const void *v, const void *u, const void *la,
                     const void *be, void *y, float *states, cudaStream_t s)
{
    const Problem &p = c.p;
    const size_t BH = p.BH, N = p.N, L = p.L, d = p.d;
    const bool one = N == 1, routed = mode_uses_u(p.mode), tc = !one && tc_fused_gates(p);
    DeltaTcArgs t = delta_tc_args(c, q, k, v, la, be);
    t.states = states;
    t.full = true;
    FwdArgs f{};
    float *kbar = nullptr, *r_on = nullptr, *sums = nullptr;
    char *tc_scratch = nullptr;
    void *scratch = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Carver cv{static_cast<char *>(scratch), 0};
        t.rec = cv.take<uint8_t>(BH * N * c.NCH * kDeltaRecBytes);
        if (!one) {
            float *own_states = cv.take<float>(BH * N * d * d, !states);
            t.states = states ? states : own_states;
        }
        t.O_on = cv.take<float>(BH * L * d, !one);
        tc_scratch = cv.take<char>(tc ? tc_scratch_bytes(p, true) : 0, tc);
        r_on = cv.take<float>(BH * L, !one && !tc && routed);
        kbar = cv.take<float>(BH * N * d, !one && routed);
        sums = cv.take<float>(BH * N * c.NCH * d, !one && routed);
        if (pass == 0 && scratch_alloc(&scratch, cv.used, s) != cudaSuccess) {
            cudaGetLastError();
            return MC_ERR_ALLOC;
        }
    }
    if (one) t.y = static_cast<__nv_bfloat16 *>(y);
    f.q = q; f.k = k; f.u = routed ? u : nullptr; f.y = y;
    f.BH = p.BH; f.L = p.L; f.C = p.C; f.N = p.N; f.mode = p.mode; f.topk = p.topk;
    TcForwardImages img{};
    if (tc) {
        img = tc_forward_images(p, tc_scratch);
        t.states_img = img.states_img;
        r_on = img.r_on;
    }
    profile_call_start(s);
    cudaError_t e = launch_delta_walk_tc(p, t, true, s);
    if (e == cudaSuccess && !one && routed) {
        DeltaArgs a = delta_args(c);
        a.k = k; a.u = f.u;
        e = launch_pool_simt(p, a, sums, kbar, r_on, s);
        profile_after_kernel(s, "pool_simt");
    }
    f.states = t.states;
    f.O_on = t.O_on;
    if (e == cudaSuccess && tc) {
        f.v = v;
        f.given = true;
        if (routed) {
            e = launch_kbar_images(p, kbar, img.kbar_img, s);
            profile_after_kernel(s, "kbar_images");
        }
        if (e == cudaSuccess) e = launch_forward_tc(p, f, tc_scratch, s);
    } else if (e == cudaSuccess && !one) {
        f.r_on = r_on; f.kbar = kbar;
        e = launch_readout_simt(p, f, s);
        profile_after_kernel(s, "readout_simt");
    }
    cudaError_t ef = cudaFreeAsync(scratch, s);
    return e == cudaSuccess && ef == cudaSuccess ? MC_OK : fail(e != cudaSuccess ? e : ef);
}

int forward_delta(const void *q, const void *k, const void *v, const void *u, const void *la, const void *be, int B,
                  int H, int L, int d, int seg_len, int agg_mode, int topk, void *y, float *states, bool bf16,
                  cudaStream_t s)
{
    Call c;
    int st = check_call(c, B, H, L, d, seg_len, agg_mode, topk, bf16);
    if (st != MC_OK) return st;
    if (any_null({q, k, v, la, be, y}) || (c.uses_u && !u)) return MC_ERR_NULL;
    if (any_misaligned({q, k, v, u, la, be, y, states})) return MC_ERR_ALIGN;
    if ((st = check_device()) != MC_OK) return st;
    const Problem &p = c.p;
    const size_t BH = p.BH, N = p.N;
    const bool routed = mode_uses_u(p.mode);
    if (delta_tc_supported(p)) return forward_delta_tc(c, q, k, v, u, la, be, y, states, s);
    DeltaArgs a = delta_args(c);
    a.q = q; a.k = k; a.v = v; a.la = la; a.be = be;
    a.u = routed ? u : nullptr;
    a.states = states;
    if (N == 1) {  // one memory, every gate is 1: the scan writes y
        a.y = y;
        profile_call_start(s);
        cudaError_t e = launch_delta_scan_simt(p, a, s);
        profile_after_kernel(s, "delta_scan_simt");
        return e == cudaSuccess ? MC_OK : fail(e);
    }
    float *sums = nullptr, *kbar = nullptr, *r_on = nullptr;
    void *scratch = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Carver cv{static_cast<char *>(scratch), 0};
        float *own_states = cv.take<float>(BH * N * d * d, !states);
        a.states = states ? states : own_states;
        a.O_on = cv.take<float>(BH * L * d);
        kbar = cv.take<float>(BH * N * d, routed);
        r_on = cv.take<float>(BH * L, routed);
        sums = cv.take<float>(BH * N * c.NCH * d, routed);
        if (pass == 0 && scratch_alloc(&scratch, cv.used, s) != cudaSuccess) {
            cudaGetLastError();
            return MC_ERR_ALLOC;
        }
    }
    profile_call_start(s);
    cudaError_t e = launch_delta_scan_simt(p, a, s);
    profile_after_kernel(s, "delta_scan_simt");
    if (e == cudaSuccess && routed) {
        e = launch_pool_simt(p, a, sums, kbar, r_on, s);
        profile_after_kernel(s, "pool_simt");
    }
    if (e == cudaSuccess) {
        FwdArgs f{};
        f.q = q; f.u = a.u; f.y = y;
        f.states = a.states; f.O_on = a.O_on; f.r_on = r_on; f.kbar = kbar;
        f.BH = p.BH; f.L = L; f.C = p.C; f.N = p.N; f.mode = p.mode; f.topk = p.topk;
        e = launch_readout_simt(p, f, s);
        profile_after_kernel(s, "readout_simt");
    }
    cudaError_t ef = cudaFreeAsync(scratch, s);
    return e == cudaSuccess && ef == cudaSuccess ? MC_OK : fail(e != cudaSuccess ? e : ef);
}

// Shares of the tokens for the CUDA-core G: two CTAs for every SM where there are few heads and segments (4 heads of 1000
// tokens, 4 segments, d = 64: 18 us in eight shares, 100 in one).  The summands are added in their order.
int simt_G_parts(const Problem &p)
{
    const long long ctas = (long long)p.BH * (p.N - 1);
    return ctas >= 304 ? 1 : (int)std::min<long long>(8, (304 + ctas - 1) / ctas);
}

int backward_delta(const void *q, const void *k, const void *v, const void *u, const void *la, const void *be,
                   const void *dy, int B, int H, int L, int d, int seg_len, int agg_mode, int topk, void *dq, void *dk,
                   void *dv, void *du, void *dla, void *dbe, bool bf16, cudaStream_t s)
{
    Call c;
    int st = check_call(c, B, H, L, d, seg_len, agg_mode, topk, bf16);
    if (st != MC_OK) return st;
    if (any_null({q, k, v, la, be, dy, dq, dk, dv, dla, dbe}) || (c.uses_u && (!u || !du))) return MC_ERR_NULL;
    if (any_misaligned({q, k, v, u, la, be, dy, dq, dk, dv, du, dla, dbe})) return MC_ERR_ALIGN;
    if ((st = check_device()) != MC_OK) return st;
    const Problem &p = c.p;
    const size_t BH = p.BH, N = p.N, NCH = c.NCH;
    const bool many = N > 1, routed = many && mode_uses_u(p.mode);
    DeltaArgs a = delta_args(c);
    a.q = q; a.k = k; a.v = v; a.la = la; a.be = be; a.dy = dy;
    a.u = routed ? u : nullptr;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dla = dla; a.dbe = dbe;
    const bool tc = delta_tc_supported(p), rtc = tc && many && bwd_tc_supported(p);  // rtc: the gate work too
    DeltaTcArgs t = delta_tc_args(c, q, k, v, la, be);
    t.dy = static_cast<const __nv_bfloat16 *>(dy);
    t.u = static_cast<const __nv_bfloat16 *>(a.u);
    t.dq = static_cast<__nv_bfloat16 *>(dq);
    t.dk = static_cast<__nv_bfloat16 *>(dk);
    t.dv = static_cast<__nv_bfloat16 *>(dv);
    t.dla = static_cast<__nv_bfloat16 *>(dla);
    t.dbe = static_cast<__nv_bfloat16 *>(dbe);
    BwdArgs b{};
    float *sums = nullptr, *kbar = nullptr, *r_on = nullptr, *G = nullptr, *dkbar = nullptr, *tok = nullptr,
          *dq_add = nullptr, *gam = nullptr, *dg = nullptr, *dgon = nullptr;
    uint8_t *states_img = nullptr, *kbar_img = nullptr;
    void *scratch = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Carver cv{static_cast<char *>(scratch), 0};
        a.E = cv.take<float>(BH * L * d, !tc);
        a.W = cv.take<float>(BH * L * d, !tc);
        a.S_c = cv.take<float>(BH * N * NCH * d * d, !tc);
        a.R_c = cv.take<float>(BH * N * NCH * d * d, !tc);
        t.rec = cv.take<uint8_t>(BH * N * NCH * kDeltaRecBytes, tc);
        t.rrec = cv.take<uint8_t>(BH * N * NCH * kDeltaRRecBytes, tc);
        t.E = cv.take<__nv_bfloat16>(BH * L * d, tc);
        t.E_lo = cv.take<__nv_bfloat16>(BH * L * d, tc);
        t.W_lo = cv.take<__nv_bfloat16>(BH * L * d, tc);
        t.S_c = cv.take<__nv_bfloat16>(BH * N * NCH * d * d, tc);
        t.R_c = cv.take<__nv_bfloat16>(BH * N * NCH * d * d, tc);
        a.states = cv.take<float>(BH * N * d * d, many);
        a.O_on = cv.take<float>(BH * L * d, many && !rtc);
        t.y = cv.take<__nv_bfloat16>(BH * L * d, rtc);
        b.g_parts = a.g_parts = t.g_parts = rtc ? bwd_G_parts(p) : many ? simt_G_parts(p) : 1;
        G = cv.take<float>(t.g_parts * BH * N * d * d, many);
        tok = cv.take<float>(BH * L * kBwdTokWords, many);
        dq_add = cv.take<float>(BH * L * d, many);
        kbar = cv.take<float>(BH * N * d, many);
        dkbar = cv.take<float>(BH * N * d, many);
        r_on = cv.take<float>(BH * L, routed);
        sums = cv.take<float>(BH * N * NCH * d, routed);
        b.sel_idx = cv.take<int32_t>(BH * L * p.topk, routed && !rtc && p.mode == MC_SSC);
        b.sel_g = cv.take<float>(BH * L * p.topk, routed && !rtc && p.mode == MC_SSC);
        b.Np = (int)((N + 15) & ~(size_t)15);
        states_img = cv.take<uint8_t>(BH * N * 32768, rtc);
        kbar_img = cv.take<uint8_t>(BH * ((N + 63) / 64) * 49152, rtc && routed);
        gam = cv.take<float>(BH * N * L, rtc && routed);
        dg = cv.take<float>(2 * BH * N * L, rtc);
        dgon = cv.take<float>(BH * L, rtc);
        b.kv_gw = cv.take<float>(2 * BH * L, rtc);
        b.dr_hi = cv.take<__nv_bfloat16>(BH * b.Np * L, rtc && routed);
        b.dr_lo = cv.take<__nv_bfloat16>(BH * b.Np * L, rtc && routed);
        if (pass == 0 && scratch_alloc(&scratch, cv.used, s) != cudaSuccess) {
            cudaGetLastError();
            return MC_ERR_ALLOC;
        }
    }
    cudaError_t e = cudaSuccess;
    if (du && !routed) e = cudaMemsetAsync(du, 0, BH * L * d * (bf16 ? 2 : 4), s);  // no score has a weight to move
    profile_call_start(s);
    if (tc) {
        t.states = a.states;
        t.O_on = a.O_on;
        if (e == cudaSuccess) e = launch_delta_walk_tc(p, t, many, s);
    } else {
        if (e == cudaSuccess) e = launch_delta_scan_simt(p, a, s);
        profile_after_kernel(s, "delta_scan_simt");
    }
    if (e == cudaSuccess && many) {
        if (routed) {
            e = launch_pool_simt(p, a, sums, kbar, r_on, s);
            profile_after_kernel(s, "pool_simt");
            if (e == cudaSuccess) e = cudaMemsetAsync(dkbar, 0, sizeof(float) * BH * N * d, s);
        }
        b.q = q; b.k = k; b.v = v; b.u = a.u; b.dy = dy;
        b.dq_f32 = dq_add; b.du = routed ? du : nullptr;
        b.states = a.states; b.kbar = kbar; b.r_on = r_on; b.O_on = a.O_on;
        b.G = G; b.dkbar = dkbar; b.tok = tok;
        b.BH = p.BH; b.L = L; b.C = p.C; b.N = p.N; b.mode = p.mode; b.topk = p.topk;
        t.gon = tok + 2;
        t.gw_stride = kBwdTokWords;
        const float *pw = tok + 4;
        if (rtc) {
            // the tensor-core backward's gate kernels over images of these states: gates, the cached memories' dg and
            // dq, dg of the online reads, the score gradients, G
            b.dq_f32 = nullptr;
            b.gam = gam;
            b.dg_in = dg; b.dg_in2 = dg + BH * N * L;
            b.dgon_in = dgon;
            b.kpre_tiles = sums;
            TcImages img{};
            img.states_img = states_img; img.kbar_img = kbar_img; img.r_on = r_on;
            if (e == cudaSuccess) e = launch_state_images(p, a.states, states_img, s);
            if (e == cudaSuccess && routed) e = launch_kbar_images(p, kbar, kbar_img, s);
            profile_after_kernel(s, "images");
            if (e == cudaSuccess && routed) {
                e = launch_bwd_gates_tc(p, u, img, gam, tok, s);
                profile_after_kernel(s, "gate_tiles_tc");
            }
            if (e == cudaSuccess) e = launch_bwd_cached_only_tc(p, q, dy, states_img, gam, dq_add, dg, s);
            profile_after_kernel(s, "bwd_cached_tc");
            if (e == cudaSuccess) e = launch_delta_dgon(p, dy, t.y, dgon, s);
            profile_after_kernel(s, "delta_dgon");
            if (e == cudaSuccess) e = launch_bwd_route(p, b, s);
            if (e == cudaSuccess) e = launch_bwd_G_parts_tc(p, dy, q, gam, G, s);
            profile_after_kernel(s, "bwd_G_tc");
            t.gon = b.kv_gw;
            pw = b.kv_gw + BH * L;
            t.gw_stride = 1;
        } else {
            if (e == cudaSuccess) e = launch_bwd_router_simt(p, b, s);
        }
        t.G = G;
        if (e == cudaSuccess && routed) {
            a.gw_stride = t.gw_stride;
            e = launch_pool_grad_simt(p, a, pw, sums, dkbar, s);
            profile_after_kernel(s, "pool_grad_simt");
            a.rho = sums;
            t.rho = sums;
            t.pw = pw;
        }
        a.tok = tok;
        a.G = G;
        a.dq_add = dq_add;
        t.dq_add = dq_add;
    }
    if (tc) {
        if (e == cudaSuccess) e = launch_delta_grads_tc(p, t, s);
    } else {
        if (e == cudaSuccess) e = launch_delta_rscan_simt(p, a, s);
        profile_after_kernel(s, "delta_rscan_simt");
        if (e == cudaSuccess) e = launch_delta_grads_simt(p, a, s);
        profile_after_kernel(s, "delta_grads_simt");
    }
    cudaError_t ef = cudaFreeAsync(scratch, s);
    return e == cudaSuccess && ef == cudaSuccess ? MC_OK : fail(e != cudaSuccess ? e : ef);
}

int decode_slots(SlotArgs a, int B, int H, int seg_len, int agg_mode, int topk, bool evict, cudaStream_t s)
{
    int st = check_shape(B, H, 1, a.d, seg_len);
    if (st != MC_OK) return st;
    if (a.t < 0 || a.nmax < 1 || a.nmax > kDecMaxN - 1) return MC_ERR_SHAPE;
    if (evict ? a.protect < 0 || a.protect >= a.nmax : a.t / seg_len >= a.nmax) return MC_ERR_SHAPE;
    if (agg_mode < MC_RESIDUAL || agg_mode > MC_MEAN) return MC_ERR_MODE;
    const bool routed = mode_uses_u(agg_mode);
    if (evict && !routed) return MC_ERR_MODE;  // constant gates tell no segment from another
    if (agg_mode == MC_SSC && topk < 0) return MC_ERR_TOPK;
    if (any_null({a.q, a.k, a.v, a.y, a.states, a.kbar, a.online, a.ksum}) || (routed && !a.u)) return MC_ERR_NULL;
    if (evict && any_null({a.mass, a.slot_seg})) return MC_ERR_NULL;
    if (evict ? !a.la != !a.be : !a.la || !a.be) return MC_ERR_NULL;
    if (any_misaligned({a.q, a.k, a.v, a.u, a.y, a.states, a.kbar, a.online, a.ksum, a.mass, a.slot_seg})) return MC_ERR_ALIGN;
    // one number per head: a token's, wherever it lies in a sequence's [B][H][L]
    if ((reinterpret_cast<uintptr_t>(a.la) | reinterpret_cast<uintptr_t>(a.be)) & (a.bf16 ? 1u : 3u)) return MC_ERR_ALIGN;
    if ((st = check_device()) != MC_OK) return st;
    a.BH = B * H;
    a.C = seg_len;
    a.mode = agg_mode == MC_SOUP ? MC_GRM : agg_mode;
    a.topk = agg_mode == MC_SSC ? topk : 0;
    if (!routed) a.u = nullptr;
    profile_call_start(s);
    cudaError_t e = launch_decode_slots(a, s);
    profile_after_kernel(s, "decode_slots");
    return e == cudaSuccess ? MC_OK : fail(e);
}

int cache_compact(const void *k, const void *u, const float *states_all, int B, int H, int L, int d, int seg_len,
                  int agg_mode, int topk, int protect, float *states, float *kbar, float *mass, int32_t *slot_seg,
                  float *online, float *ksum, int n_max, float *mass_all, bool bf16, cudaStream_t s)
{
    Call c;
    int st = check_shape(B, H, L, d, seg_len);
    if (st != MC_OK) return st;
    if (n_max < 1 || n_max > kDecMaxN - 1 || protect < 0 || protect > n_max) return MC_ERR_SHAPE;
    if ((st = check_call(c, B, H, L, d, seg_len, agg_mode, topk, bf16)) != MC_OK) return st;
    if (!mode_uses_u(agg_mode)) return MC_ERR_MODE;  // constant gates tell no segment from another
    Problem &p = c.p;
    const int tile_len = gate_mass_tile(p);
    const long long tiles = ((long long)L + tile_len - 1) / tile_len;
    if (p.N > 16384 || (long long)p.BH * ((p.N + 63) / 64) * 64 >= (1ll << 31) || (long long)p.BH * tiles >= (1ll << 31) || (long long)p.BH * (n_max + 1) >= (1ll << 31))
        return MC_ERR_SHAPE;
    if (any_null({k, u, states_all, states, kbar, mass, slot_seg, online, ksum})) return MC_ERR_NULL;
    if (any_misaligned({k, u, states_all, states, kbar, mass, slot_seg, online, ksum, mass_all})) return MC_ERR_ALIGN;
    if ((st = check_device()) != MC_OK) return st;
    const size_t BH = p.BH, N = p.N;
    DeltaArgs a = delta_args(c);
    a.k = k; a.u = u;
    CompactArgs m{};
    m.u = u; m.states_all = states_all; m.mass_all = mass_all;
    m.states = states; m.kbar = kbar; m.mass = mass; m.online = online; m.ksum = ksum; m.slot_seg = slot_seg;
    m.BH = p.BH; m.L = L; m.C = p.C; m.N = p.N; m.d = d; m.mode = p.mode; m.topk = p.topk; m.tiles = (int)tiles;
    m.tile_len = tile_len;
    m.shares = (int)std::min<long long>(tiles, std::min(512, d * d));
    const bool tc = tile_len == 128;
    m.done = L / seg_len; m.nmax = n_max;
    m.protect = protect < m.done ? protect : m.done;
    float *sums = nullptr, *kbar_all = nullptr, *r_on = nullptr;
    uint8_t *kbar_img = nullptr;
    void *scratch = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Carver cv{static_cast<char *>(scratch), 0};
        if (!mass_all) m.mass_all = cv.take<float>(BH * N);
        kbar_img = cv.take<uint8_t>(BH * ((N + 63) / 64) * 49152, tc);
        kbar_all = cv.take<float>(BH * N * d);
        r_on = cv.take<float>(BH * L);
        sums = cv.take<float>(BH * N * c.NCH * d);
        m.part = cv.take<float>(BH * m.shares * N);
        m.order = cv.take<int32_t>(BH * n_max);
        if (pass == 0 && scratch_alloc(&scratch, cv.used, s) != cudaSuccess) {
            cudaGetLastError();
            return MC_ERR_ALLOC;
        }
    }
    m.kbar_all = kbar_all;
    m.r_on = r_on;
    profile_call_start(s);
    cudaError_t e = launch_pool_simt(p, a, sums, kbar_all, r_on, s);
    profile_after_kernel(s, "pool_simt");
    if (e == cudaSuccess && tc) e = launch_kbar_images(p, kbar_all, kbar_img, s);
    m.kbar_img = kbar_img;
    if (e == cudaSuccess) {
        e = launch_gate_mass(p, m, s);
        profile_after_kernel(s, "gate_mass");
    }
    if (e == cudaSuccess) {
        e = launch_compact(p, m, s);
        profile_after_kernel(s, "compact");
    }
    cudaError_t ef = cudaFreeAsync(scratch, s);
    return e == cudaSuccess && ef == cudaSuccess ? MC_OK : fail(e != cudaSuccess ? e : ef);
}

}  // namespace
}  // namespace mc

extern "C" {

int mc_forward_delta(const void *q, const void *k, const void *v, const void *u, const void *log_alpha,
                     const void *beta, int B, int H, int L, int d, int seg_len, int agg_mode, int topk, void *y,
                     float *states, int is_bf16, mc_stream_t stream)
{
    return mc::forward_delta(q, k, v, u, log_alpha, beta, B, H, L, d, seg_len, agg_mode, topk, y, states, is_bf16 != 0,
                             reinterpret_cast<cudaStream_t>(stream));
}

int mc_backward_delta(const void *q, const void *k, const void *v, const void *u, const void *log_alpha,
                      const void *beta, const void *dy, int B, int H, int L, int d, int seg_len, int agg_mode, int topk,
                      void *dq, void *dk, void *dv, void *du, void *dlog_alpha, void *dbeta, int is_bf16,
                      mc_stream_t stream)
{
    return mc::backward_delta(q, k, v, u, log_alpha, beta, dy, B, H, L, d, seg_len, agg_mode, topk, dq, dk, dv, du,
                              dlog_alpha, dbeta, is_bf16 != 0, reinterpret_cast<cudaStream_t>(stream));
}

int mc_decode_step_delta(const void *q, const void *k, const void *v, const void *u, const void *log_alpha,
                         const void *beta, int B, int H, int d, int seg_len, int agg_mode, int topk, int t,
                         float *states, float *kbar, float *online, float *ksum, int n_max, void *y, int is_bf16,
                         mc_stream_t stream)
{
    mc::SlotArgs a{};
    a.q = q; a.k = k; a.v = v; a.u = u; a.la = log_alpha; a.be = beta; a.y = y;
    a.states = states; a.kbar = kbar; a.online = online; a.ksum = ksum;
    a.d = d; a.t = t; a.nmax = n_max; a.bf16 = is_bf16 != 0;
    return mc::decode_slots(a, B, H, seg_len, agg_mode, topk, false, reinterpret_cast<cudaStream_t>(stream));
}

int mc_decode_step_evict(const void *q, const void *k, const void *v, const void *u, const void *log_alpha,
                         const void *beta, int B, int H, int d, int seg_len, int agg_mode, int topk, int t, int protect,
                         float *states, float *kbar, float *mass, int32_t *slot_seg, float *online, float *ksum,
                         int n_max, void *y, int is_bf16, mc_stream_t stream)
{
    mc::SlotArgs a{};
    a.q = q; a.k = k; a.v = v; a.u = u; a.la = log_alpha; a.be = beta; a.y = y;
    a.states = states; a.kbar = kbar; a.online = online; a.ksum = ksum; a.mass = mass; a.slot_seg = slot_seg;
    a.d = d; a.t = t; a.nmax = n_max; a.protect = protect; a.bf16 = is_bf16 != 0;
    return mc::decode_slots(a, B, H, seg_len, agg_mode, topk, true, reinterpret_cast<cudaStream_t>(stream));
}

int mc_cache_compact(const void *k, const void *u, const float *prefill_states, int B, int H, int L, int d, int seg_len,
                     int agg_mode, int topk, int protect, float *states, float *kbar, float *mass, int32_t *slot_seg,
                     float *online, float *ksum, int n_max, float *prefill_mass, int is_bf16, mc_stream_t stream)
{
    return mc::cache_compact(k, u, prefill_states, B, H, L, d, seg_len, agg_mode, topk, protect, states, kbar, mass,
                             slot_seg, online, ksum, n_max, prefill_mass, is_bf16 != 0,
                             reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
