// Paged KV cache: the C ABI of include/arl2.h (arl2_paged_*).  Arguments are
// checked here; what lies in device memory (lengths, offsets, page numbers)
// is checked by the kernels before it becomes an address.
//
// Kernels per call: write 1, read 1, attend 1, forward 3 (2 without rotary).
#include "arl2.h"
#include "paged.h"

#include <climits>
#include <cmath>
#include <cstdint>
#include <new>

namespace arl2 {
int rotary_head_dim(const arl2_rotary* r);  // rotary.cu
}

struct arl2_paged_handle {
    int device = -1;
    arl2::PagedGeom g{};
    arl2_dtype dtype = ARL2_BF16;
    bool e4m3 = false, use_tc = false;
    float scale = 0.f;
    int max_ctas = 0, sms = 0;
    size_t bytes = 0;
    arl2::PagedWork work{};
    int* err = nullptr;
    unsigned long long launches = 0;
};

namespace {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadDim = 128;
constexpr int kMaxGroup = 64;
constexpr int kMaxCtasPerSm = 8;
constexpr int kFewRows = 16;  // query rows of a key head up to which the transposed kernel runs
constexpr long long kMaxKeys = 1ll << 30;
constexpr int kMaxTokens = 1 << 30;  // (with what a kernel's blocks take on top it still fits an int)

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

arl2_status check_device(const arl2_paged_handle* h) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ARL2_ERR_CUDA;
    return dev == h->device ? ARL2_OK : ARL2_ERR_INVALID_ARG;
}

template <typename T>
arl2_status dalloc(arl2_paged_handle* h, T** p, size_t bytes) {
    void* q = nullptr;
    if (cudaMalloc(&q, bytes) != cudaSuccess) {
        cudaGetLastError();
        return ARL2_ERR_OOM;
    }
    *p = static_cast<T*>(q);
    h->bytes += bytes;
    return ARL2_OK;
}

void release(arl2_paged_handle* h) {
    if (!h) return;
    void* ptrs[] = {h->work.o, h->work.ml, h->work.arrived, h->err};
    for (void* p : ptrs)
        if (p) cudaFree(p);
    delete h;
}

size_t esize(const arl2_paged_handle* h) { return h->dtype == ARL2_BF16 ? 2 : 4; }

arl2_status check_pool(const arl2_paged_handle* h, const arl2_paged_pool* p) {
    if (!p || !p->k || !p->v) return ARL2_ERR_INVALID_ARG;
    if (h->e4m3 != (p->k_scale != nullptr) || h->e4m3 != (p->v_scale != nullptr)) return ARL2_ERR_INVALID_ARG;
    if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_scale, 16) || !aligned(p->v_scale, 16))
        return ARL2_ERR_ALIGN;
    return ARL2_OK;
}

arl2_status check_tables(const arl2_paged_handle* h, int seqs, int tokens, int max_pages) {
    if (seqs < 0 || seqs > arl2::kPagedMaxSeqs || tokens < 0 || tokens > kMaxTokens || max_pages < 0 ||
        ((long long)max_pages << h->g.page_log2) > kMaxKeys)
        return ARL2_ERR_SHAPE;
    return ARL2_OK;
}

arl2_status check_batch(const arl2_paged_handle* h, const arl2_paged_batch* b) {
    if (!b) return ARL2_ERR_INVALID_ARG;
    const arl2_status s = check_tables(h, b->seqs, b->tokens, b->max_pages);
    if (s != ARL2_OK) return s;
    if (b->max_new < 0) return ARL2_ERR_SHAPE;
    if (b->seqs > 0 && b->tokens > 0) {
        if (!b->q_offsets || !b->kv_lens || (b->max_pages > 0 && !b->page_table)) return ARL2_ERR_INVALID_ARG;
        if (!aligned(b->q_offsets, 4) || !aligned(b->kv_lens, 4) || !aligned(b->page_table, 4)) return ARL2_ERR_ALIGN;
    }
    return ARL2_OK;
}

// Stride between tokens (0: dense); 0 if the given one is too small.
long long token_stride(long long given, int heads, int d) {
    const long long dense = (long long)heads * d;
    return given == 0 ? dense : given >= dense ? given : 0;
}

// The tensor-core kernels load 16 bytes at a time; the SIMT ones take single
// elements where a tensor does not fit that.
arl2_status check_tokens(const arl2_paged_handle* h, const void* p, long long stride, bool wide) {
    if (!p) return ARL2_ERR_INVALID_ARG;
    if (stride == 0) return ARL2_ERR_SHAPE;
    const size_t esz = esize(h);
    if (!aligned(p, wide ? 16 : esz) || (wide && (stride * (long long)esz) % 16)) return ARL2_ERR_ALIGN;
    return ARL2_OK;
}

arl2::PagedPool pool_of(const arl2_paged_pool* p) { return arl2::PagedPool{p->k, p->v, p->k_scale, p->v_scale}; }

arl2::PagedSeqs seqs_of(const arl2_paged_batch* b) {
    return arl2::PagedSeqs{b->seqs, b->tokens, b->max_pages, b->q_offsets, b->kv_lens, b->page_table};
}

arl2_status check_mask(int block, int window, int sinks) {
    return block < 1 || window < 0 || sinks < 0 ? ARL2_ERR_INVALID_ARG : ARL2_OK;
}

arl2_status write_now(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* b, const void* k,
                      long long ks, const void* v, long long vs, cudaStream_t stream) {
    ++h->launches;
    return arl2::launch_paged_write(h->dtype == ARL2_BF16, h->e4m3, h->g, pool_of(pool), seqs_of(b), k, ks, v, vs,
                                    h->err, stream) == cudaSuccess
               ? ARL2_OK
               : ARL2_ERR_CUDA;
}

arl2_status attend_now(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* b, int block,
                       int window, int sinks, const void* q, long long qs, void* out, cudaStream_t stream) {
    arl2::PagedAttend a{};
    a.g = h->g;
    a.pool = pool_of(pool);
    a.seqs = seqs_of(b);
    // positions stay below 2^30: a longer block, window or run of sinks holds
    // them all just the same
    const long long bl = block < kMaxKeys ? block : kMaxKeys;
    const long long w = (long long)window * bl, s = (long long)sinks * bl;
    a.mask = arl2::PagedMask{(int)bl, (int)(w < INT_MAX ? w : INT_MAX), (int)(s < INT_MAX ? s : INT_MAX)};
    a.work = h->work;
    a.q = q;
    a.q_stride = qs;
    a.out = out;
    a.scale = h->scale;
    a.err = h->err;
    // (unknown: the average; any choice is right, the wrong one slower)
    const int known = b->max_new > 0 ? b->max_new : (b->tokens + b->seqs - 1) / b->seqs;
    const int max_new = known < b->tokens ? known : b->tokens;
    ++h->launches;
    cudaError_t e;
    const long long rows = (long long)max_new * h->g.G;
    if (!h->use_tc)
        e = arl2::launch_paged_simt(h->dtype == ARL2_BF16, h->e4m3, a, max_new, h->max_ctas, stream);
    else if (rows <= kFewRows)  // 48 streams' tokens (12000 keys, 4 rows): 237 us, 294 with 128-row tiles
        e = arl2::launch_paged_few(h->e4m3, a, (int)rows, h->max_ctas, stream);
    else
        e = arl2::launch_paged_tc(h->e4m3, a, h->max_ctas, stream);
    return e == cudaSuccess ? ARL2_OK : ARL2_ERR_CUDA;
}

}  // namespace

extern "C" {

arl2_status arl2_paged_create(const arl2_paged_config* cfg, cudaStream_t stream, arl2_paged_handle** out) {
    if (!cfg || !out) return ARL2_ERR_INVALID_ARG;
    *out = nullptr;
    if (cfg->dtype != ARL2_BF16 && cfg->dtype != ARL2_FP32) return ARL2_ERR_INVALID_ARG;
    if (cfg->format != ARL2_CACHE_NATIVE && cfg->format != ARL2_CACHE_E4M3) return ARL2_ERR_INVALID_ARG;
    if (cfg->impl != ARL2_IMPL_AUTO && cfg->impl != ARL2_IMPL_SIMT) return ARL2_ERR_INVALID_ARG;
    if (!(cfg->softmax_scale >= 0.f) || std::isinf(cfg->softmax_scale)) return ARL2_ERR_INVALID_ARG;
    if (cfg->max_ctas < 0) return ARL2_ERR_INVALID_ARG;
    if (cfg->kv_heads < 1 || cfg->q_heads < 1 || cfg->q_heads > kMaxHeads || cfg->q_heads % cfg->kv_heads ||
        cfg->q_heads / cfg->kv_heads > kMaxGroup || cfg->head_dim < 1 || cfg->head_dim > kMaxHeadDim ||
        cfg->pages < 1 || (long long)cfg->pages * cfg->kv_heads >= 1ll << 31)
        return ARL2_ERR_SHAPE;
    int log2 = 4;
    while (log2 <= 8 && (1 << log2) != cfg->page_tokens) ++log2;
    if (log2 > 8) return ARL2_ERR_SHAPE;
    const bool use_tc = cfg->impl == ARL2_IMPL_AUTO && cfg->dtype == ARL2_BF16;
    if (use_tc && cfg->head_dim != 128) return ARL2_ERR_UNSUPPORTED;

    arl2_paged_handle* h = new (std::nothrow) arl2_paged_handle();
    if (!h) return ARL2_ERR_OOM;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return ARL2_ERR_CUDA;
    }
    h->g = arl2::PagedGeom{cfg->q_heads, cfg->kv_heads, cfg->q_heads / cfg->kv_heads, cfg->head_dim, cfg->pages, log2};
    h->dtype = cfg->dtype;
    h->e4m3 = cfg->format == ARL2_CACHE_E4M3;
    h->use_tc = use_tc;
    h->scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.f / std::sqrt((float)cfg->head_dim);
    h->max_ctas = cfg->max_ctas;
    const size_t rows = (size_t)h->sms * arl2::kPagedRowsPerSm;
    const size_t counters = (size_t)h->sms * kMaxCtasPerSm;
    arl2_status s = dalloc(h, &h->work.o, rows * kMaxHeadDim * sizeof(float));
    if (s == ARL2_OK) s = dalloc(h, &h->work.ml, rows * sizeof(float2));
    if (s == ARL2_OK) s = dalloc(h, &h->work.arrived, counters * sizeof(int));
    if (s == ARL2_OK) s = dalloc(h, &h->err, sizeof(int));
    if (s == ARL2_OK && arl2::paged_simt_init() != cudaSuccess) s = ARL2_ERR_CUDA;
    if (s == ARL2_OK && use_tc && !(arl2::paged_tc_init() && arl2::paged_few_init())) s = ARL2_ERR_CUDA;
    if (s == ARL2_OK && (cudaMemsetAsync(h->work.arrived, 0, counters * sizeof(int), stream) != cudaSuccess ||
                         cudaMemsetAsync(h->err, 0, sizeof(int), stream) != cudaSuccess))
        s = ARL2_ERR_CUDA;
    if (s != ARL2_OK) {
        cudaGetLastError();
        cudaStreamSynchronize(stream);
        release(h);
        return s;
    }
    *out = h;
    return ARL2_OK;
}

arl2_status arl2_paged_write(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* batch,
                             const void* k, long long k_stride, const void* v, long long v_stride,
                             cudaStream_t stream) {
    if (!h) return ARL2_ERR_INVALID_ARG;
    arl2_status s = check_pool(h, pool);
    if (s == ARL2_OK) s = check_batch(h, batch);
    if (s != ARL2_OK) return s;
    if (batch->seqs == 0 || batch->tokens == 0) return ARL2_OK;
    k_stride = token_stride(k_stride, h->g.Hk, h->g.d);
    v_stride = token_stride(v_stride, h->g.Hk, h->g.d);
    s = check_tokens(h, k, k_stride, h->use_tc);
    if (s == ARL2_OK) s = check_tokens(h, v, v_stride, h->use_tc);
    if (s == ARL2_OK) s = check_device(h);
    return s == ARL2_OK ? write_now(h, pool, batch, k, k_stride, v, v_stride, stream) : s;
}

arl2_status arl2_paged_read(arl2_paged_handle* h, const arl2_paged_pool* pool, int seqs, int tokens,
                            int max_pages, const int* offsets, const int* starts, const int* page_table,
                            void* k_dst, void* v_dst, cudaStream_t stream) {
    if (!h) return ARL2_ERR_INVALID_ARG;
    arl2_status s = check_pool(h, pool);
    if (s == ARL2_OK) s = check_tables(h, seqs, tokens, max_pages);
    if (s != ARL2_OK) return s;
    if (seqs == 0 || tokens == 0) return ARL2_OK;
    if (!offsets || (max_pages > 0 && !page_table)) return ARL2_ERR_INVALID_ARG;
    if (!aligned(offsets, 4) || !aligned(starts, 4) || !aligned(page_table, 4)) return ARL2_ERR_ALIGN;
    s = check_tokens(h, k_dst, 1 << 4, h->use_tc);
    if (s == ARL2_OK) s = check_tokens(h, v_dst, 1 << 4, h->use_tc);
    if (s == ARL2_OK) s = check_device(h);
    if (s != ARL2_OK) return s;
    ++h->launches;
    const arl2::PagedSeqs b{seqs, tokens, max_pages, offsets, nullptr, page_table};
    return arl2::launch_paged_read(h->dtype == ARL2_BF16, h->e4m3, h->g, pool_of(pool), b, starts, k_dst, v_dst,
                                   h->err, stream) == cudaSuccess
               ? ARL2_OK
               : ARL2_ERR_CUDA;
}

arl2_status arl2_paged_attend(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* batch,
                              int block, int window, int sinks, const void* q, long long q_stride, void* out,
                              cudaStream_t stream) {
    if (!h) return ARL2_ERR_INVALID_ARG;
    arl2_status s = check_pool(h, pool);
    if (s == ARL2_OK) s = check_batch(h, batch);
    if (s == ARL2_OK) s = check_mask(block, window, sinks);
    if (s != ARL2_OK) return s;
    if (batch->seqs == 0 || batch->tokens == 0) return ARL2_OK;
    q_stride = token_stride(q_stride, h->g.Hq, h->g.d);
    s = check_tokens(h, q, q_stride, h->use_tc);
    if (s == ARL2_OK) s = check_tokens(h, out, 1 << 4, h->use_tc);
    if (s == ARL2_OK && out == q) s = ARL2_ERR_INVALID_ARG;
    if (s == ARL2_OK) s = check_device(h);
    return s == ARL2_OK ? attend_now(h, pool, batch, block, window, sinks, q, q_stride, out, stream) : s;
}

arl2_status arl2_paged_forward(arl2_paged_handle* h, const arl2_paged_pool* pool, const arl2_paged_batch* batch,
                               const arl2_rotary* rotary, const int* positions, int block, int window, int sinks,
                               const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                               long long v_stride, void* turned, void* out, cudaStream_t stream) {
    if (!h) return ARL2_ERR_INVALID_ARG;
    const arl2::PagedGeom& g = h->g;
    arl2_status s = check_pool(h, pool);
    if (s == ARL2_OK) s = check_batch(h, batch);
    if (s == ARL2_OK) s = check_mask(block, window, sinks);
    if (s == ARL2_OK && rotary && arl2::rotary_head_dim(rotary) != g.d) s = ARL2_ERR_SHAPE;
    if (s != ARL2_OK) return s;
    if (batch->seqs == 0 || batch->tokens == 0) return ARL2_OK;
    q_stride = token_stride(q_stride, g.Hq, g.d);
    k_stride = token_stride(k_stride, g.Hk, g.d);
    v_stride = token_stride(v_stride, g.Hk, g.d);
    s = check_tokens(h, q, q_stride, h->use_tc);
    if (s == ARL2_OK) s = check_tokens(h, k, k_stride, h->use_tc);
    if (s == ARL2_OK) s = check_tokens(h, v, v_stride, h->use_tc);
    if (s == ARL2_OK) s = check_tokens(h, out, 1 << 4, h->use_tc);
    if (s == ARL2_OK && rotary) s = check_tokens(h, turned, 1 << 4, h->use_tc);
    if (s == ARL2_OK && (out == q || out == k || out == v || (rotary && (turned == out || !positions))))
        s = ARL2_ERR_INVALID_ARG;
    if (s == ARL2_OK) s = check_device(h);
    if (s != ARL2_OK) return s;
    if (rotary) {
        const long long stride = (long long)(g.Hq + g.Hk) * g.d;
        void* k_turned = static_cast<char*>(turned) + (size_t)g.Hq * g.d * esize(h);
        ++h->launches;
        s = arl2_rotary_apply(rotary, h->dtype, batch->tokens, positions, g.Hq, q, q_stride, turned, stride, g.Hk, k,
                              k_stride, k_turned, stride, 0, stream);
        if (s != ARL2_OK) return s;
        q = turned;
        k = k_turned;
        q_stride = k_stride = stride;
    }
    s = write_now(h, pool, batch, k, k_stride, v, v_stride, stream);
    return s == ARL2_OK ? attend_now(h, pool, batch, block, window, sinks, q, q_stride, out, stream) : s;
}

arl2_status arl2_paged_device_status(arl2_paged_handle* h, cudaStream_t stream) {
    if (!h) return ARL2_ERR_INVALID_ARG;
    const arl2_status s = check_device(h);
    if (s != ARL2_OK) return s;
    int word = 0;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return ARL2_ERR_CUDA;
    if (cudaMemcpy(&word, h->err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return ARL2_ERR_CUDA;
    if (word == 0) return ARL2_OK;
    if (cudaMemset(h->err, 0, sizeof(int)) != cudaSuccess) return ARL2_ERR_CUDA;
    if (word & arl2::kErrPagedTimeout) {
        // a kernel that gave up may have left arrivals behind
        if (cudaMemset(h->work.arrived, 0, (size_t)h->sms * kMaxCtasPerSm * sizeof(int)) != cudaSuccess)
            return ARL2_ERR_CUDA;
        return ARL2_ERR_TIMEOUT;
    }
    return ARL2_ERR_INVALID_ARG;
}

size_t arl2_paged_device_bytes(const arl2_paged_handle* h) { return h ? h->bytes : 0; }

unsigned long long arl2_paged_kernel_launches(const arl2_paged_handle* h) { return h ? h->launches : 0; }

void arl2_paged_destroy(arl2_paged_handle* h) {
    if (!h) return;
    const int dev = h->device;
    int prev = -1;
    cudaGetDevice(&prev);
    if (prev != dev) cudaSetDevice(dev);
    cudaDeviceSynchronize();
    release(h);
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
}

}  // extern "C"
