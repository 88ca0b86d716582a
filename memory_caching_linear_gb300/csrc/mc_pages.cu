// mc_pages.cu -- the entry points of decoding over a paged cache (include/mc.h): argument checks, scratch, and the
// kernels of each call.
#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "paged.cuh"

namespace mc {
namespace {

constexpr int kSms = 152;

// A block of stream-ordered scratch handed out in 256-byte aligned pieces (a first walk with a null base adds the sizes up).
struct Carver {
    char *base;
    size_t used;
    template <typename T>
    T *take(size_t count)
    {
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

bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

bool has_width(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

int check_cache(const mc_paged_cache *c, Paged &p)
{
    if (!c) return MC_ERR_NULL;
    if (!has_width(c->d)) return MC_ERR_SHAPE;
    if (c->H < 1 || c->seg_len < 1 || c->n_seqs < 1 || c->n_seqs > kMaxRows || c->n_max < 1 || c->n_max > kMaxPaged ||
        c->n_pages < 1 || c->n_pages > (1 << 20))
        return MC_ERR_SHAPE;
    // a CTA for every 32 KB of the pool and of the rows, and one for every head of a sequence's segments
    const long long pieces = ((long long)c->H * c->d * c->d + 8191) / 8192;
    if (c->H > (1 << 20) || pieces * (c->n_pages + c->n_seqs) >= (1ll << 31) || (long long)c->H * kMaxRows * 8 >= (1ll << 31))
        return MC_ERR_SHAPE;
    if ((long long)c->n_seqs * c->H >= (1ll << 30)) return MC_ERR_SHAPE;
    p = Paged{c->pages, c->kbar, c->refs, c->online, c->ksum, c->table, c->pos, c->row, c->status,
              c->n_pages, c->n_seqs, c->H, c->d, c->seg_len, c->n_max};
    return MC_OK;
}

// A step's memory: tickets, then partial reads.
struct StepPlan {
    size_t part, online, total;
};
StepPlan step_plan(size_t S, size_t H, size_t d)
{
    StepPlan p;
    p.part = round_up(sizeof(int32_t) * (S * H + 1));
    p.online = p.part + round_up(sizeof(float) * (kSms + S * H) * (d + 2));
    p.total = p.online + round_up(sizeof(float) * S * H * (d + 1));
    return p;
}

int check_cache_pointers(const Paged &p, const void *work)
{
    if (!work) return MC_ERR_NULL;
    if (!aligned(work, 16)) return MC_ERR_ALIGN;
    for (const void *x : {(const void *)p.pages, (const void *)p.kbar, (const void *)p.refs, (const void *)p.online,
                          (const void *)p.ksum, (const void *)p.table, (const void *)p.pos, (const void *)p.row, (const void *)p.status})
        if (!x) return MC_ERR_NULL;
    for (const void *x : {p.pages, p.kbar, p.online, p.ksum})
        if (!aligned(x, 16)) return MC_ERR_ALIGN;
    for (const void *x : {p.refs, p.table, p.pos, p.row, p.status})
        if (!aligned(x, 4)) return MC_ERR_ALIGN;
    return MC_OK;
}

int check_pointers(std::initializer_list<const void *> wanted, std::initializer_list<const void *> words,
                   std::initializer_list<const void *> elements, size_t element)
{
    for (const void *x : wanted)
        if (!x) return MC_ERR_NULL;
    for (const void *x : wanted)
        if (!aligned(x, 16)) return MC_ERR_ALIGN;
    for (const void *x : words)
        if (!aligned(x, 4)) return MC_ERR_ALIGN;
    for (const void *x : elements)
        if (!aligned(x, element)) return MC_ERR_ALIGN;
    return MC_OK;
}

enum Call { kStep, kTree, kAccept };

int run_batch(const mc_paged_cache *cache, TreeArgs a, Call call, int agg_mode, cudaStream_t s)
{
    int st = check_cache(cache, a.c);
    if (st != MC_OK) return st;
    const Paged &c = a.c;
    const bool accept = call == kAccept;
    if (a.B < 1 || a.B > c.S || a.T < 1 || a.T > kMaxTree) return MC_ERR_SHAPE;
    if (agg_mode < MC_RESIDUAL || agg_mode > MC_MEAN) return MC_ERR_MODE;
    a.mode = agg_mode == MC_SOUP ? MC_GRM : agg_mode;  // the same function for a matrix memory
    if (a.mode == MC_SSC && a.topk < 0) return MC_ERR_TOPK;
    if ((st = check_cache_pointers(c, cache->work)) != MC_OK) return st;
    if ((a.la == nullptr) != (a.be == nullptr)) return MC_ERR_NULL;
    a.delta = a.la != nullptr;
    const bool routed = !accept && mode_uses_u(a.mode);
    if ((!a.parent && (a.T > 1 || accept)) || (accept && !a.last)) return MC_ERR_NULL;
    const size_t element = a.bf16 ? 2 : 4;
    st = accept ? check_pointers({a.k, a.v}, {a.parent, a.last, a.slots}, {a.la, a.be}, element)
                : check_pointers({a.q, a.k, a.v, routed ? a.u : a.q, a.y}, {a.parent, a.count, a.slots}, {a.la, a.be}, element);
    if (st != MC_OK) return st;
    if ((st = check_device()) != MC_OK) return st;
    if (call == kStep) {
        const StepPlan plan = step_plan(c.S, c.H, c.d);
        char *work = static_cast<char *>(cache->work);
        a.ranges = kSms;
        profile_call_start(s);
        const cudaError_t e = launch_step(a, StepWork{reinterpret_cast<int32_t *>(work), reinterpret_cast<float *>(work + plan.part),
                                                      reinterpret_cast<float *>(work + plan.online)}, s);
        profile_after_kernel(s, "step_paged");
        return e == cudaSuccess ? MC_OK : fail(e);
    }
    if (call == kTree && tree_whole(a)) {
        a.whole = true;
        profile_call_start(s);
        const cudaError_t e = launch_tree_gates(a, s);
        profile_after_kernel(s, "tree_whole");
        return e == cudaSuccess ? MC_OK : fail(e);
    }
    const size_t BH = (size_t)a.B * c.H, T = a.T, B = a.B;
    a.Tp = (a.T + 7) / 8 * 8;
    a.groups = a.Tp / 8;
    const bool split = tree_tc_supported(a);
    a.scored = split && routed;
    a.ranges = split ? kSms : std::max(1, 4 * kSms / (a.groups * read_blocks(c.d)));
    // a head's end, on the tensor cores: 16 heads of d = 128, 16 sequences of 2 to 62 segments, 16 nodes 145 -> 125 us (caches
    // flushed), d = 64, 8 of up to 63, 32 nodes 82 -> 65; twice as much 125 and 59, four times 131 and 61.  None on the CUDA
    // cores, whose ranges are a quarter as long and bound by products: 16 sequences of 2 to 63 segments, d = 64, 16 nodes in
    // fp32, 84 without and 86 with it
    a.rest = split ? 256 / c.d : 0;
    void *scratch = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Carver cv{static_cast<char *>(scratch), 0};
        if (accept) {
            a.p.path = cv.take<uint64_t>(B);
            a.p.act = cv.take<int32_t>(B);
            a.p.pos = cv.take<int32_t>(B);
            a.p.fresh = cv.take<int32_t>(B + 1);
            a.p.list = cv.take<int32_t>(B * T);
        }
        else {
            a.line = cv.take<int32_t>(Line::ints(a.B));
            a.gates = cv.take<float>(BH * (c.nmax + 2) * a.Tp);
            a.Z = cv.take<float>(a.delta ? BH * a.Tp * c.d : 0);
            if (split) {
                a.top = cv.take<float>(BH * a.Tp);
                a.Y0 = cv.take<float>(BH * a.Tp * c.d);
                a.score = cv.take<float>(BH * path_segments(a) * a.Tp);
                a.into = cv.take<float>(BH * a.Tp);
                a.seg = cv.take<int32_t>(B * kMaxTree);
                a.weight = cv.take<float2>((a.ranges + BH) * a.Tp);
            }
            a.anc = cv.take<uint64_t>(B * kMaxTree);
            a.P = cv.take<float>(BH * T * a.Tp);
            a.A = cv.take<float>(a.delta ? BH * T * a.Tp : 0);
            a.part = cv.take<float>((a.ranges + BH) * a.Tp * c.d * (split && c.d == 64 ? 2 : 1));
        }
        if (pass == 0 && scratch_alloc(&scratch, cv.used, s) != cudaSuccess) {
            cudaGetLastError();
            return MC_ERR_ALLOC;
        }
    }
    profile_call_start(s);
    cudaError_t e;
    if (accept) {
        e = launch_plan(a, s);
        profile_after_kernel(s, "plan_rows");
        if (e == cudaSuccess) e = launch_accept(a, s);
        profile_after_kernel(s, "accept_rows");
    } else {
        e = a.scored ? launch_tree_scores_tc(a, s) : cudaSuccess;
        if (a.scored) profile_after_kernel(s, "tree_scores_tc");
        if (e == cudaSuccess) e = split ? launch_tree_read_tc(a, s) : launch_tree_gates(a, s);
        profile_after_kernel(s, split ? "tree_read_tc" : "tree_gates");
        if (e == cudaSuccess) e = split ? launch_tree_path_tc(a, s) : launch_tree_read(a, s);
        profile_after_kernel(s, split ? "tree_path_tc" : "tree_read");
        if (e == cudaSuccess) e = launch_tree_finish(a, s);
        profile_after_kernel(s, "tree_finish");
    }
    cudaError_t ef = cudaFreeAsync(scratch, s);
    return e == cudaSuccess && ef == cudaSuccess ? MC_OK : fail(e != cudaSuccess ? e : ef);
}

template <typename F>
int with_plan(size_t ints, cudaStream_t s, F &&work)
{
    void *plan = nullptr;
    if (scratch_alloc(&plan, sizeof(int32_t) * ints, s) != cudaSuccess) {
        cudaGetLastError();
        return MC_ERR_ALLOC;
    }
    cudaError_t e = work(static_cast<int32_t *>(plan)), ef = cudaFreeAsync(plan, s);
    return e == cudaSuccess && ef == cudaSuccess ? MC_OK : fail(e != cudaSuccess ? e : ef);
}

}  // namespace
}  // namespace mc

extern "C" {

size_t mc_paged_work_bytes(int n_seqs, int H, int d)
{
    if (n_seqs < 1 || n_seqs > mc::kMaxRows || H < 1 || H > (1 << 20) || !mc::has_width(d)) return 0;
    return mc::step_plan(n_seqs, H, d).total;
}

int mc_decode_step_paged(const mc_paged_cache *cache, const void *q, const void *k, const void *v, const void *u,
                         const void *log_alpha, const void *beta, const int32_t *slots, int B, int agg_mode, int topk,
                         void *y, int is_bf16, mc_stream_t stream)
{
    mc::TreeArgs a{};
    a.q = q; a.k = k; a.v = v; a.u = u; a.la = log_alpha; a.be = beta; a.slots = slots; a.y = y;
    a.B = B; a.T = 1; a.topk = topk; a.bf16 = is_bf16 != 0;
    return mc::run_batch(cache, a, mc::kStep, agg_mode, reinterpret_cast<cudaStream_t>(stream));
}

int mc_decode_tree(const mc_paged_cache *cache, const void *q, const void *k, const void *v, const void *u,
                   const void *log_alpha, const void *beta, const int32_t *parent, const int32_t *count,
                   const int32_t *slots, int B, int T, int agg_mode, int topk, void *y, int is_bf16, mc_stream_t stream)
{
    mc::TreeArgs a{};
    a.q = q; a.k = k; a.v = v; a.u = u; a.la = log_alpha; a.be = beta; a.slots = slots; a.y = y;
    a.parent = parent; a.count = count;
    a.B = B; a.T = T; a.topk = topk; a.bf16 = is_bf16 != 0;
    return mc::run_batch(cache, a, mc::kTree, agg_mode, reinterpret_cast<cudaStream_t>(stream));
}

int mc_tree_accept(const mc_paged_cache *cache, const void *k, const void *v, const void *log_alpha, const void *beta,
                   const int32_t *parent, const int32_t *last, const int32_t *slots, int B, int T, int is_bf16,
                   mc_stream_t stream)
{
    mc::TreeArgs a{};
    a.k = k; a.v = v; a.la = log_alpha; a.be = beta; a.slots = slots; a.parent = parent; a.last = last;
    a.B = B; a.T = T; a.bf16 = is_bf16 != 0;
    return mc::run_batch(cache, a, mc::kAccept, MC_RESIDUAL, reinterpret_cast<cudaStream_t>(stream));
}

int mc_pages_fork(const mc_paged_cache *cache, const int32_t *src, mc_stream_t stream)
{
    mc::Paged c;
    int st = mc::check_cache(cache, c);
    if (st == MC_OK) st = mc::check_cache_pointers(c, cache->work);
    if (st != MC_OK) return st;
    if (!src) return MC_ERR_NULL;
    if (!mc::aligned(src, 4)) return MC_ERR_ALIGN;
    if ((st = mc::check_device()) != MC_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return mc::with_plan(2 * (size_t)c.S, s, [&](int32_t *plan) { return mc::launch_fork(c, src, plan, s); });
}

int mc_pages_compact(const mc_paged_cache *dst, const mc_paged_cache *src, mc_stream_t stream)
{
    mc::Paged to, from;
    int st = mc::check_cache(dst, to);
    if (st == MC_OK) st = mc::check_cache(src, from);
    if (st != MC_OK) return st;
    if (to.H != from.H || to.d != from.d || to.C != from.C || to.S < from.S || to.nmax < from.nmax) return MC_ERR_SHAPE;
    if ((st = mc::check_cache_pointers(to, dst->work)) != MC_OK || (st = mc::check_cache_pointers(from, src->work)) != MC_OK) return st;
    if (to.pages == from.pages || to.kbar == from.kbar || to.refs == from.refs || to.online == from.online || to.ksum == from.ksum ||
        to.table == from.table || to.pos == from.pos || to.row == from.row)
        return MC_ERR_SHAPE;
    if ((st = mc::check_device()) != MC_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return mc::with_plan(1 + (size_t)to.P + from.P, s, [&](int32_t *plan) { return mc::launch_pages_compact(to, from, plan, s); });
}

int mc_pages_load(const mc_paged_cache *cache, int slot, const void *k, const float *states, int L, int is_bf16,
                  mc_stream_t stream)
{
    mc::Paged c;
    int st = mc::check_cache(cache, c);
    if (st != MC_OK) return st;
    if (slot < 0 || slot >= c.S || L < 1 || L > mc::kMaxPos || L / c.C > c.nmax) return MC_ERR_SHAPE;
    if ((long long)(L / c.C + 1) * c.H >= (1ll << 31)) return MC_ERR_SHAPE;
    if ((st = mc::check_cache_pointers(c, cache->work)) != MC_OK) return st;
    if ((st = mc::check_pointers({k, states}, {}, {}, 4)) != MC_OK) return st;
    if ((st = mc::check_device()) != MC_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return mc::with_plan((size_t)(L / c.C) + 1, s, [&](int32_t *plan) {
        return mc::launch_pages_load(c, slot, k, states, L, is_bf16 != 0, plan, s);
    });
}

}  // extern "C"
