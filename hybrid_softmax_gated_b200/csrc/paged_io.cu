// Writing new keys and values into the pages of a paged KV cache, as they
// are or quantised to e4m3 with one fp32 scale per token and head, and
// reading them back.
//
// Both are memory bound: a row (the d features of one token and head) is
// read once and written once.  A row is held by 16 lanes (bf16, d = 128) or
// 32 (fp32), 16 bytes each, so its largest magnitude takes four or five
// shuffles and never leaves the registers.  Widths that do not fit take the
// generic form, a warp per row.  A block takes a few tokens with all their
// heads of both tensors: the sequence a token belongs to and its page are
// looked up once per token.
#include "paged.cuh"

namespace arl2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;  // tokens per block
constexpr float kCodeMax = 448.f, kScaleMin = 0x1p-126f;

// Sequence of row `tok`: the number of offsets in (offsets[0], offsets[S]]
// that are <= tok, counted by the whole block (offsets ascend).
__device__ __forceinline__ int owner_of(const int* __restrict__ offsets, int S, int tok) {
    int s = 0;
    for (int i0 = 0; i0 < S; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        s += __syncthreads_count(i < S && offsets[i + 1] <= tok);
    }
    return s;
}

// Place of each of the block's tokens: page and key position, or page -1.
struct Places {
    int page[kMaxTok], key[kMaxTok];
};

// Writing: row i of a sequence's n is its position total - n + i; reading:
// starts[s] + i (starts == nullptr: i).
__device__ __forceinline__ void find_places(const PagedGeom& g, const PagedSeqs& b, const int* starts, bool reading,
                                            int tok0, int n_tok, Places& pl, int* err) {
    int s = 0;  // thread t looks up the block's token t
    for (int t = 0; t < n_tok; ++t) {
        const int o = owner_of(b.q_off, b.S, tok0 + t);
        if ((int)threadIdx.x == t) s = o;
    }
    if ((int)threadIdx.x < n_tok) {
        const int tok = tok0 + threadIdx.x;
        int page = -1, key = 0;
        if (s < b.S && tok >= b.q_off[0]) {
            const long long cap = (long long)b.max_pages << g.page_log2;
            const int q0 = b.q_off[s], q1 = b.q_off[s + 1];
            long long at;
            bool bad = q0 < 0 || q1 < q0 || q1 > b.tokens;
            if (reading) {
                at = (long long)(starts ? starts[s] : 0) + (tok - q0);
                bad = bad || at < 0 || at >= cap;
            } else {
                const int total = b.kv_len[s];
                bad = bad || total < 0 || total > cap;
                at = (long long)total - (q1 - q0) + (tok - q0);
            }
            if (bad) {
                paged::report(err, kErrPagedTable);
            } else if (at >= 0) {  // (before position 0: a chunk padded on the left)
                key = (int)at;
                page = b.table[(size_t)s * b.max_pages + (key >> g.page_log2)];
                if ((unsigned)page >= (unsigned)g.pages) {
                    paged::report(err, kErrPagedTable);
                    page = -1;
                }
            }
        }
        pl.page[threadIdx.x] = page;
        pl.key[threadIdx.x] = key;
    }
    __syncthreads();
}

template <typename T>
struct Lane16;  // elements of 16 bytes
template <>
struct Lane16<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void load(const void* p, float (&x)[8]) {
        const uint4 u = __ldcs(static_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(void* p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
};
template <>
struct Lane16<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void load(const void* p, float (&x)[4]) {
        const float4 u = __ldcs(static_cast<const float4*>(p));
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
    static __device__ __forceinline__ void store(void* p, const float (&x)[4]) {
        __stcs(static_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    }
};

__device__ __forceinline__ unsigned char code_of(float y) {
    return (unsigned char)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float value_of(unsigned char c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(__half(h));
}

// Scale of a row with largest magnitude `amax` and whether it is finite.
__device__ __forceinline__ float scale_of(float amax, bool finite) {
    return finite ? fmaxf(amax / kCodeMax, kScaleMin) : __int_as_float(0x7fffffff);
}

// kLanes lanes hold a row (d = kLanes * Lane16<T>::n); 0: the generic form.
template <typename T, bool kCodes, int kLanes>
__global__ void __launch_bounds__(kThreads) write_kernel(PagedGeom g, PagedPool pool, PagedSeqs b, const T* k,
                                                         long long k_stride, const T* v, long long v_stride,
                                                         int per_block, int* err) {
    __shared__ Places pl;
    const int tok0 = blockIdx.x * per_block;
    const int n_tok = min(per_block, b.tokens - tok0);
    find_places(g, b, nullptr, false, tok0, n_tok, pl, err);
    constexpr int kRow = kLanes ? kLanes : 32;
    const int lane = threadIdx.x % kRow;
    const int rows = n_tok * 2 * g.Hk;
    for (int r0 = 0; r0 < rows; r0 += kThreads / kRow) {  // (whole warps: the shuffles need every lane)
        const int r = r0 + threadIdx.x / kRow;
        const int t = r < rows ? r / (2 * g.Hk) : 0;
        const int hh = r - t * 2 * g.Hk;
        const bool is_v = hh >= g.Hk;
        const int h = is_v ? hh - g.Hk : hh;
        const bool on = r < rows && pl.page[t] >= 0;
        const T* src = (is_v ? v + (long long)(tok0 + t) * v_stride : k + (long long)(tok0 + t) * k_stride) + h * g.d;
        const size_t row = on ? paged::pool_row(g, pl.page[t], h, pl.key[t]) : 0;
        void* dst = is_v ? pool.v : pool.k;
        float* sc = is_v ? pool.vs : pool.ks;
        if constexpr (kLanes > 0) {
            constexpr int n = Lane16<T>::n;
            if constexpr (!kCodes) {
                if (on)
                    reinterpret_cast<uint4*>(dst)[row * kLanes + lane] =
                        __ldcs(reinterpret_cast<const uint4*>(src) + lane);
            } else {
                float x[n];
#pragma unroll
                for (int i = 0; i < n; ++i) x[i] = 0.f;
                if (on) Lane16<T>::load(reinterpret_cast<const uint4*>(src) + lane, x);
                float amax = 0.f;
                bool finite = true;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    amax = fmaxf(amax, fabsf(x[i]));
                    finite = finite && fabsf(x[i]) < INFINITY;
                }
                if (!finite) amax = INFINITY;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                finite = amax < INFINITY;
                const float s = scale_of(amax, finite);
                const float inv = finite ? 1.f / s : 0.f;
                if (on) {
                    uint32_t w[n / 4];
#pragma unroll
                    for (int i = 0; i < n / 4; ++i) {
                        uint32_t c = 0;
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const float2 y = make_float2(x[4 * i + j] * inv, x[4 * i + j + 1] * inv);
                            c |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (8 * j);
                        }
                        w[i] = finite ? c : 0u;
                    }
                    uint32_t* to = reinterpret_cast<uint32_t*>(dst) + (row * kLanes + lane) * (n / 4);
                    if constexpr (n == 8)
                        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                    else
                        *to = w[0];
                    if (lane == 0) sc[row] = s;
                }
            }
        } else {
            if constexpr (!kCodes) {
                if (on)
                    for (int c = lane; c < g.d; c += 32) static_cast<T*>(dst)[row * g.d + c] = src[c];
            } else {
                float amax = 0.f;
                if (on)
                    for (int c = lane; c < g.d; c += 32) {
                        const float a = fabsf(paged::to_float(src[c]));
                        amax = a < INFINITY ? fmaxf(amax, a) : INFINITY;
                    }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const bool finite = amax < INFINITY;
                const float s = scale_of(amax, finite);
                if (on) {
                    const float inv = 1.f / s;
                    for (int c = lane; c < g.d; c += 32)
                        static_cast<unsigned char*>(dst)[row * g.d + c] =
                            finite ? code_of(paged::to_float(src[c]) * inv) : (unsigned char)0;
                    if (lane == 0) sc[row] = s;
                }
            }
        }
    }
}

template <typename T, bool kCodes, int kLanes>
__global__ void __launch_bounds__(kThreads) read_kernel(PagedGeom g, PagedPool pool, PagedSeqs b, const int* starts,
                                                        T* k, T* v, int per_block, int* err) {
    __shared__ Places pl;
    const int tok0 = blockIdx.x * per_block;
    const int n_tok = min(per_block, b.tokens - tok0);
    find_places(g, b, starts, true, tok0, n_tok, pl, err);
    constexpr int kRow = kLanes ? kLanes : 32;
    const int lane = threadIdx.x % kRow;
    const int rows = n_tok * 2 * g.Hk;
#pragma unroll 4
    for (int r = threadIdx.x / kRow; r < rows; r += kThreads / kRow) {
        const int t = r / (2 * g.Hk);
        const int hh = r - t * 2 * g.Hk;
        const bool is_v = hh >= g.Hk;
        const int h = is_v ? hh - g.Hk : hh;
        if (pl.page[t] < 0) continue;
        const size_t row = paged::pool_row(g, pl.page[t], h, pl.key[t]);
        const void* src = is_v ? pool.v : pool.k;
        T* dst = (is_v ? v : k) + ((size_t)(tok0 + t) * g.Hk + h) * g.d;
        const float s = kCodes ? __ldg((is_v ? pool.vs : pool.ks) + row) : 1.f;
        if constexpr (kLanes > 0) {
            constexpr int n = Lane16<T>::n;
            if constexpr (!kCodes) {
                __stcs(reinterpret_cast<uint4*>(dst) + lane, __ldcs(static_cast<const uint4*>(src) + row * kLanes + lane));
            } else {
                uint32_t w[n / 4];
                const uint32_t* from = static_cast<const uint32_t*>(src) + (row * kLanes + lane) * (n / 4);
                if constexpr (n == 8) {
                    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(from));
                    w[0] = u.x, w[1] = u.y;
                } else {
                    w[0] = __ldcs(from);
                }
                float x[n];
#pragma unroll
                for (int i = 0; i < n; i += 2) {
                    const __half2_raw hr =
                        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(hr));
                    x[i] = f.x * s;
                    x[i + 1] = f.y * s;
                }
                Lane16<T>::store(reinterpret_cast<uint4*>(dst) + lane, x);
            }
        } else {
            for (int c = lane; c < g.d; c += 32) {
                if constexpr (kCodes)
                    paged::store_as(dst + c, value_of(static_cast<const unsigned char*>(src)[row * g.d + c]) * s);
                else
                    dst[c] = static_cast<const T*>(src)[row * g.d + c];
            }
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// As many tokens per block as still leave several blocks per SM.
int tokens_per_block(int tokens) { return tokens >= 148 * 8 * 8 ? 8 : tokens >= 148 * 4 * 4 ? 4 : tokens >= 148 * 4 ? 2 : 1; }

template <typename T, bool kCodes>
cudaError_t write_as(const PagedGeom& g, const PagedPool& pool, const PagedSeqs& b, const void* k, long long ks,
                     const void* v, long long vs, int* err, cudaStream_t st) {
    constexpr int n = Lane16<T>::n;
    const int per = tokens_per_block(b.tokens), grid = (b.tokens + per - 1) / per;
    const bool fits = aligned16(k) && aligned16(v) && ks % n == 0 && vs % n == 0;
    auto go = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, st>>>(g, pool, b, static_cast<const T*>(k), ks, static_cast<const T*>(v), vs, per,
                                          err);
        return cudaGetLastError();
    };
    if (fits && g.d == 128) return go(write_kernel<T, kCodes, 128 / n>);
    if (fits && g.d == 64) return go(write_kernel<T, kCodes, 64 / n>);
    return go(write_kernel<T, kCodes, 0>);
}

template <typename T, bool kCodes>
cudaError_t read_as(const PagedGeom& g, const PagedPool& pool, const PagedSeqs& b, const int* starts, void* k, void* v,
                    int* err, cudaStream_t st) {
    constexpr int n = Lane16<T>::n;
    const int per = tokens_per_block(b.tokens), grid = (b.tokens + per - 1) / per;
    const bool fits = aligned16(k) && aligned16(v);
    auto go = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, st>>>(g, pool, b, starts, static_cast<T*>(k), static_cast<T*>(v), per, err);
        return cudaGetLastError();
    };
    if (fits && g.d == 128) return go(read_kernel<T, kCodes, 128 / n>);
    if (fits && g.d == 64) return go(read_kernel<T, kCodes, 64 / n>);
    return go(read_kernel<T, kCodes, 0>);
}

}  // namespace

cudaError_t launch_paged_write(bool bf16, bool e4m3, const PagedGeom& g, const PagedPool& pool, const PagedSeqs& b,
                               const void* k, long long ks, const void* v, long long vs, int* err, cudaStream_t st) {
    if (bf16)
        return e4m3 ? write_as<__nv_bfloat16, true>(g, pool, b, k, ks, v, vs, err, st)
                    : write_as<__nv_bfloat16, false>(g, pool, b, k, ks, v, vs, err, st);
    return e4m3 ? write_as<float, true>(g, pool, b, k, ks, v, vs, err, st)
                : write_as<float, false>(g, pool, b, k, ks, v, vs, err, st);
}

cudaError_t launch_paged_read(bool bf16, bool e4m3, const PagedGeom& g, const PagedPool& pool, const PagedSeqs& b,
                              const int* starts, void* k, void* v, int* err, cudaStream_t st) {
    if (bf16)
        return e4m3 ? read_as<__nv_bfloat16, true>(g, pool, b, starts, k, v, err, st)
                    : read_as<__nv_bfloat16, false>(g, pool, b, starts, k, v, err, st);
    return e4m3 ? read_as<float, true>(g, pool, b, starts, k, v, err, st)
                : read_as<float, false>(g, pool, b, starts, k, v, err, st);
}

}  // namespace arl2
