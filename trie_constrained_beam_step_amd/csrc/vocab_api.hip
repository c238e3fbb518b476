// vocab_api.hip -- the C ABI of the embedding (gr_embed) and the head
// (gr_head): argument checks, workspace ownership and launches.
#include <math.h>

#include <new>

#include "errors.h"
#include "gr.h"
#include "vocab.h"

using gr::fail;

namespace {

constexpr int32_t kMaxVocab = 1 << 30, kMaxDim = 65536, kMaxTokens = 1 << 24, kMaxRows = 1 << 20;
constexpr int64_t kMaxStride = 1 << 22;

// Makes the handle's device current for a call and restores the caller's.
struct OnDevice {
    int prev = -1;
    hipError_t err;
    explicit OnDevice(int dev) {
        err = hipGetDevice(&prev);
        if (err != hipSuccess || prev == dev) prev = -1;
        else err = hipSetDevice(dev);
    }
    ~OnDevice() {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

template <typename T>
hipError_t dalloc(T** p, size_t count) {
    *p = nullptr;
    return hipMalloc((void**)p, (count ? count : 1) * sizeof(T));
}

gr_status check_common(int32_t vocab, int32_t dim, int32_t dtype, float scale) {
    if (vocab < 1 || vocab > kMaxVocab) return fail(GR_ERR_INVALID_ARG, "vocab %d outside [1, 2^30]", vocab);
    if (dim < 1 || dim > kMaxDim) return fail(GR_ERR_INVALID_ARG, "dim %d outside [1, %d]", dim, kMaxDim);
    if (dtype != GR_F32 && dtype != GR_BF16) return fail(GR_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (!isfinite(scale) || scale == 0.0f) return fail(GR_ERR_INVALID_ARG, "scale must be finite and not zero");
    return GR_OK;
}

// A row stride: 0 stands for dim.
gr_status check_stride(int64_t* stride, int32_t dim, const char* what) {
    if (*stride == 0) *stride = dim;
    if (*stride < dim || *stride > kMaxStride)
        return fail(GR_ERR_INVALID_ARG, "%s row stride %lld outside [dim %d, 2^22]", what, (long long)*stride, dim);
    return GR_OK;
}

gr_status check_count(int32_t n, int32_t most) {
    if (n < 0 || n > most) return fail(GR_ERR_INVALID_ARG, "count %d outside [0, %d]", n, most);
    return GR_OK;
}

// dtype of the elements; GR_F32 stands for any 32-bit type
gr_status check_aligned(const void* p, int32_t dtype, const char* what) {
    if ((uintptr_t)p % (dtype == GR_BF16 ? 2 : 4)) return fail(GR_ERR_INVALID_ARG, "%s is not aligned to its elements", what);
    return GR_OK;
}

gr_status init_fail(hipError_t e, const char* what) {
    (void)hipGetLastError();  // an allocation's error is reported here, not by the next launch
    if (e == hipErrorOutOfMemory) return fail(GR_ERR_OUT_OF_MEMORY, "%s: %s", what, hipGetErrorString(e));
    return gr::hip_fail(e, what);
}

}  // namespace

struct gr_embed {
    gr_embed_config cfg{};
    int device = 0;
    gr::EmbedSpace ws{};
};

struct gr_head {
    gr_head_config cfg{};
    int device = 0;
    gr::HeadPlan plan{};
    gr::HeadSpace ws{};
};

#define GR_TRY(expr)                          \
    do {                                      \
        if (gr_status s_ = (expr)) return s_; \
    } while (0)

// ------------------------------------------------------------- embedding

static int32_t embed_width(int32_t dim) { return (dim + 7) / 8 * 8; }

static void embed_release(gr_embed* h) {
    const gr::EmbedSpace& w = h->ws;
    void* all[] = {w.keys[0], w.keys[1], w.pos[0], w.pos[1], w.table, w.totals, w.parts};
    for (void* p : all) (void)hipFree(p);
    delete h;
}

extern "C" gr_status gr_embed_init(const gr_embed_config* cfg, gr_stream stream, gr_embed** out) {
    if (!cfg || !out) return fail(GR_ERR_INVALID_ARG, "NULL config or out");
    GR_TRY(check_common(cfg->vocab, cfg->dim, cfg->dtype, cfg->scale));
    if (cfg->max_tokens < 1 || cfg->max_tokens > kMaxTokens)
        return fail(GR_ERR_INVALID_ARG, "max_tokens %d outside [1, 2^24]", cfg->max_tokens);
    int dev = 0;
    HIP_TRY(hipGetDevice(&dev), "get device");
    gr_embed* h = new (std::nothrow) gr_embed();
    if (!h) return fail(GR_ERR_OUT_OF_MEMORY, "host allocation failed");
    h->cfg = *cfg;
    h->device = dev;
    (void)stream;
    hipError_t e = hipSuccess;
    if (cfg->max_tokens > gr::kEmbedFew) {
        // a smaller call's sort has fewer workgroups; its sums may have more
        // (smaller) tiles than the largest call's, but no more than the limits here
        const size_t n = cfg->max_tokens;
        const gr::EmbedPlan p = gr::embed_plan(n, cfg->vocab, 256);
        const size_t tiles = n / 8 + 1 < gr::kSumTiles ? n / 8 + 1 : gr::kSumTiles;
        for (int i = 0; i < 2 && e == hipSuccess; ++i) {
            e = dalloc(&h->ws.keys[i], n);
            if (e == hipSuccess) e = dalloc(&h->ws.pos[i], n);
        }
        if (e == hipSuccess) e = dalloc(&h->ws.table, ((size_t)1 << p.bits) * p.blocks);
        if (e == hipSuccess) e = dalloc(&h->ws.totals, (size_t)1 << p.bits);
        if (e == hipSuccess) e = dalloc(&h->ws.parts, tiles * 2 * embed_width(cfg->dim));
    }
    if (e != hipSuccess) {
        embed_release(h);
        return init_fail(e, "embedding workspace");
    }
    *out = h;
    return GR_OK;
}

extern "C" gr_status gr_embed_lookup(gr_embed* h, const int32_t* d_tokens, int32_t n, const void* d_weight,
                                     int64_t weight_row_stride, void* d_out, int64_t out_row_stride,
                                     gr_stream stream) {
    if (!h || !d_weight || (n != 0 && (!d_tokens || !d_out))) return fail(GR_ERR_INVALID_ARG, "NULL argument");
    const gr_embed_config& c = h->cfg;
    GR_TRY(check_count(n, c.max_tokens));
    GR_TRY(check_stride(&weight_row_stride, c.dim, "weight"));
    GR_TRY(check_stride(&out_row_stride, c.dim, "out"));
    GR_TRY(check_aligned(d_weight, c.dtype, "weight"));
    GR_TRY(check_aligned(d_out, c.dtype, "out"));
    GR_TRY(check_aligned(d_tokens, GR_F32, "tokens"));
    gr::EmbedLookupArgs a;
    a.tokens = d_tokens;
    a.n = n;
    a.V = c.vocab;
    a.D = c.dim;
    a.scale = c.scale;
    a.weight = d_weight;
    a.wstride = weight_row_stride;
    a.out = d_out;
    a.ostride = out_row_stride;
    OnDevice on(h->device);
    HIP_TRY(on.err, "set device");
    HIP_TRY(gr::launch_embed_lookup(a, c.dtype, (hipStream_t)stream), "embedding lookup launch");
    return GR_OK;
}

extern "C" gr_status gr_embed_backward(gr_embed* h, const int32_t* d_tokens, int32_t n, const void* d_grad,
                                       int64_t grad_row_stride, void* d_grad_weight, int64_t grad_weight_row_stride,
                                       int32_t accumulate, gr_stream stream) {
    if (!h || !d_grad_weight || (n != 0 && (!d_tokens || !d_grad))) return fail(GR_ERR_INVALID_ARG, "NULL argument");
    const gr_embed_config& c = h->cfg;
    GR_TRY(check_count(n, c.max_tokens));
    GR_TRY(check_stride(&grad_row_stride, c.dim, "grad"));
    GR_TRY(check_stride(&grad_weight_row_stride, c.dim, "grad_weight"));
    GR_TRY(check_aligned(d_grad, c.dtype, "grad"));
    GR_TRY(check_aligned(d_grad_weight, c.dtype, "grad_weight"));
    GR_TRY(check_aligned(d_tokens, GR_F32, "tokens"));
    gr::EmbedBackwardArgs a;
    a.tokens = d_tokens;
    a.n = n;
    a.V = c.vocab;
    a.D = c.dim;
    a.scale = c.scale;
    a.grad = d_grad;
    a.gstride = grad_row_stride;
    a.gweight = d_grad_weight;
    a.wstride = grad_weight_row_stride;
    a.accumulate = accumulate != 0;
    a.Dp = embed_width(c.dim);
    a.ws = h->ws;
    OnDevice on(h->device);
    HIP_TRY(on.err, "set device");
    HIP_TRY(gr::launch_embed_backward(a, c.dtype, (hipStream_t)stream), "embedding backward launch");
    return GR_OK;
}

extern "C" void gr_embed_free(gr_embed* h) {
    if (!h) return;
    OnDevice on(h->device);
    (void)hipDeviceSynchronize();
    embed_release(h);
}

// ------------------------------------------------------------------ head

static void head_release(gr_head* h) {
    const gr::HeadSpace& w = h->ws;
    void* all[] = {w.count, w.target, w.source, w.place, w.gscale, w.lse, w.zt, w.H, w.Hh, w.hdown, w.Wh, w.wdown, w.parts, w.W, w.G, w.gh, w.gw};
    for (void* p : all) (void)hipFree(p);
    delete h;
}

extern "C" gr_status gr_head_init(const gr_head_config* cfg, gr_stream stream, gr_head** out) {
    if (!cfg || !out) return fail(GR_ERR_INVALID_ARG, "NULL config or out");
    GR_TRY(check_common(cfg->vocab, cfg->dim, cfg->dtype, cfg->scale));
    if (cfg->max_rows < 1 || cfg->max_rows > kMaxRows)
        return fail(GR_ERR_INVALID_ARG, "max_rows %d outside [1, 2^20]", cfg->max_rows);
    int dev = 0;
    HIP_TRY(hipGetDevice(&dev), "get device");
    gr_head* h = new (std::nothrow) gr_head();
    if (!h) return fail(GR_ERR_OUT_OF_MEMORY, "host allocation failed");
    h->cfg = *cfg;
    h->device = dev;
    (void)stream;
    const gr::HeadPlan p = gr::head_plan(cfg->max_rows, cfg->vocab, cfg->dim, cfg->dtype, !cfg->score_only);
    h->plan = p;
    gr::HeadSpace& w = h->ws;
    hipError_t e = dalloc(&w.count, 1);
    if (e == hipSuccess) e = dalloc(&w.target, p.packed);
    if (e == hipSuccess) e = dalloc(&w.source, p.packed);
    if (e == hipSuccess) e = dalloc(&w.place, p.packed);
    if (e == hipSuccess) e = dalloc(&w.zt, p.packed);
    // fp32: the logits take the halves, the gradients the planes
    const bool planes = !p.halves || !cfg->score_only;
    if (e == hipSuccess && planes) e = dalloc(&w.H, (size_t)p.planes * p.packed * p.Dp);
    if (e == hipSuccess && planes) e = dalloc(&w.W, p.W);
    if (p.halves) {
        if (e == hipSuccess) e = dalloc(&w.Hh, (size_t)p.halves * p.packed * p.Dp);
        if (e == hipSuccess) e = dalloc(&w.hdown, p.packed);
        if (e == hipSuccess) e = dalloc(&w.Wh, (size_t)p.halves * p.Vw * p.Dp);
        if (e == hipSuccess) e = dalloc(&w.wdown, p.Vw);
    }
    if (e == hipSuccess) e = dalloc(&w.parts, p.parts);
    if (!cfg->score_only) {
        if (e == hipSuccess) e = dalloc(&w.gscale, p.packed);
        if (e == hipSuccess) e = dalloc(&w.lse, p.packed);
        if (e == hipSuccess) e = dalloc(&w.G, p.G);
        if (e == hipSuccess) e = dalloc(&w.gh, p.gh);
        if (e == hipSuccess) e = dalloc(&w.gw, p.gw);
    }
    if (e != hipSuccess) {
        head_release(h);
        return init_fail(e, "head workspace");
    }
    *out = h;
    return GR_OK;
}

static gr::HeadArgs head_args(const gr_head* h, int32_t n) {
    gr::HeadArgs a{};
    a.N = n;
    a.V = h->cfg.vocab;
    a.D = h->cfg.dim;
    a.scale = h->cfg.scale;
    a.plan = h->plan;
    a.ws = h->ws;
    return a;
}

extern "C" gr_status gr_head_loss(gr_head* h, const void* d_hidden, int64_t hidden_row_stride, const void* d_weight,
                                  int64_t weight_row_stride, const int32_t* d_targets, int32_t n, float* d_loss,
                                  float* d_lse, gr_stream stream) {
    if (!h || !d_weight || (n != 0 && (!d_hidden || !d_targets || !d_loss || !d_lse)))
        return fail(GR_ERR_INVALID_ARG, "NULL argument");
    const gr_head_config& c = h->cfg;
    GR_TRY(check_count(n, c.max_rows));
    GR_TRY(check_stride(&hidden_row_stride, c.dim, "hidden"));
    GR_TRY(check_stride(&weight_row_stride, c.dim, "weight"));
    GR_TRY(check_aligned(d_hidden, c.dtype, "hidden"));
    GR_TRY(check_aligned(d_weight, c.dtype, "weight"));
    GR_TRY(check_aligned(d_targets, GR_F32, "targets"));
    GR_TRY(check_aligned(d_loss, GR_F32, "loss"));
    GR_TRY(check_aligned(d_lse, GR_F32, "lse"));
    gr::HeadArgs a = head_args(h, n);
    a.hidden = d_hidden;
    a.hstride = hidden_row_stride;
    a.weight = d_weight;
    a.wstride = weight_row_stride;
    a.targets = d_targets;
    a.loss = d_loss;
    a.lse = d_lse;
    OnDevice on(h->device);
    HIP_TRY(on.err, "set device");
    HIP_TRY(gr::launch_head_loss(a, c.dtype, (hipStream_t)stream), "head loss launch");
    return GR_OK;
}

extern "C" gr_status gr_head_backward(gr_head* h, const void* d_hidden, int64_t hidden_row_stride,
                                      const void* d_weight, int64_t weight_row_stride, const int32_t* d_targets,
                                      int32_t n, const float* d_lse, const float* d_grad_loss, void* d_grad_hidden,
                                      int64_t grad_hidden_row_stride, void* d_grad_weight,
                                      int64_t grad_weight_row_stride, int32_t accumulate, gr_stream stream) {
    if (!h || !d_weight || (n != 0 && (!d_hidden || !d_targets || !d_lse || !d_grad_loss)))
        return fail(GR_ERR_INVALID_ARG, "NULL argument");
    if (n != 0 && !d_grad_hidden && !d_grad_weight) return fail(GR_ERR_INVALID_ARG, "neither gradient asked for");
    const gr_head_config& c = h->cfg;
    if (c.score_only) return fail(GR_ERR_UNSUPPORTED, "the head was made for scoring only");
    GR_TRY(check_count(n, c.max_rows));
    GR_TRY(check_stride(&hidden_row_stride, c.dim, "hidden"));
    GR_TRY(check_stride(&weight_row_stride, c.dim, "weight"));
    GR_TRY(check_stride(&grad_hidden_row_stride, c.dim, "grad_hidden"));
    GR_TRY(check_stride(&grad_weight_row_stride, c.dim, "grad_weight"));
    GR_TRY(check_aligned(d_hidden, c.dtype, "hidden"));
    GR_TRY(check_aligned(d_weight, c.dtype, "weight"));
    GR_TRY(check_aligned(d_grad_hidden, c.dtype, "grad_hidden"));
    GR_TRY(check_aligned(d_grad_weight, c.dtype, "grad_weight"));
    GR_TRY(check_aligned(d_targets, GR_F32, "targets"));
    GR_TRY(check_aligned(d_lse, GR_F32, "lse"));
    GR_TRY(check_aligned(d_grad_loss, GR_F32, "grad_loss"));
    gr::HeadArgs a = head_args(h, n);
    a.hidden = d_hidden;
    a.hstride = hidden_row_stride;
    a.weight = d_weight;
    a.wstride = weight_row_stride;
    a.targets = d_targets;
    a.lse_in = d_lse;
    a.grad_loss = d_grad_loss;
    a.ghidden = d_grad_hidden;
    a.ghstride = grad_hidden_row_stride;
    a.gweight = d_grad_weight;
    a.gwstride = grad_weight_row_stride;
    a.accumulate = accumulate != 0;
    OnDevice on(h->device);
    HIP_TRY(on.err, "set device");
    HIP_TRY(gr::launch_head_backward(a, c.dtype, (hipStream_t)stream), "head backward launch");
    return GR_OK;
}

extern "C" void gr_head_free(gr_head* h) {
    if (!h) return;
    OnDevice on(h->device);
    (void)hipDeviceSynchronize();
    head_release(h);
}
