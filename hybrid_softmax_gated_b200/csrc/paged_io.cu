// Writing new keys and values into the pages of a paged KV cache, as they
// are or quantised to e4m3 with one fp32 scale per token and head, and
// reading them back.
//
// Both are memory bound: a row (the d features of one token and head) is
// read once and written once.  A row is held by 16 lanes (bf16, d = 128) or
// 32 (fp32), 16 bytes each, so its largest magnitude takes four or five
// shuffles and never leaves the registers.  Widths that do not fit take the
// generic form, a warp per row.  A warp takes a few rows of one token, all
// their loads in flight together; it finds the token's sequence by a 32-way
// search of the offsets (one load for up to 32 sequences, two for 1024).  A
// history of 3 x 9360 tokens of 12 heads read back from codes: 31.5 us, 5.9 TB/s;
// four frames of 1560 tokens quantised: 10.2 us, 3.4 TB/s, most of it the chain from
// a token's offsets to its page and the conversion's instructions.
#include "paged.cuh"
#include "ptx.cuh"

#include <type_traits>

namespace arl2 {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // rows a lane has in flight
constexpr float kCodeMax = 448.f, kScaleMin = 0x1p-126f;

// Sequence of row `tok`: how many of the ascending offsets[1 .. S] are <= tok.
// The whole warp, S <= 1024.
__device__ __forceinline__ int owner_of(const int* __restrict__ offsets, int S, int tok) {
    const int lane = threadIdx.x & 31;
    int first = 0;
    if (S > 32) {  // the group of 32 that the answer lies in
        const int i = 32 * lane + 32;
        first = 32 * __popc(__ballot_sync(0xffffffffu, i <= S && offsets[i] <= tok));
    }
    const int i = first + lane + 1;
    return first + __popc(__ballot_sync(0xffffffffu, i <= S && offsets[i] <= tok));
}

// Place of a token in the cache: page and key position, or page -1.
struct Place {
    int page, key;
};

// Writing: row i of a sequence's n is its position total - n + i; reading:
// starts[s] + i (starts == nullptr: i).  The whole warp.  owner_of is right for
// ascending offsets only: among others the row may lie outside the sequence it
// names, and then it has no position.
__device__ __forceinline__ Place find_place(const PagedGeom& g, const PagedSeqs& b, const int* starts, bool reading,
                                            int tok, int* err) {
    const int s = owner_of(b.q_off, b.S, tok);
    Place pl{-1, 0};
    if (s >= b.S || tok < b.q_off[0]) return pl;
    const long long cap = (long long)b.max_pages << g.page_log2;
    const int q0 = b.q_off[s], q1 = b.q_off[s + 1];
    long long at;
    bool bad = q0 < 0 || tok < q0 || tok >= q1 || q1 > b.tokens;
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
        const int page = b.table[(size_t)s * b.max_pages + ((int)at >> g.page_log2)];
        if ((unsigned)page < (unsigned)g.pages)
            pl = Place{page, (int)at};
        else
            paged::report(err, kErrPagedTable);
    }
    return pl;
}

// The grid's last block has no rows: it looks at all sequences' entries, those
// that no row leads to as well.  (Beside the rows' blocks, it costs them nothing.)
__device__ __forceinline__ bool check_block(const PagedGeom& g, const PagedSeqs& b, int* err) {
    if (blockIdx.x + 1 < gridDim.x) return false;
    const long long cap = (long long)b.max_pages << g.page_log2;
    for (int s = threadIdx.x; s < b.S; s += kThreads) {
        const int q0 = b.q_off[s], q1 = b.q_off[s + 1], total = b.kv_len ? b.kv_len[s] : 0;
        if (q0 < 0 || q1 < q0 || q1 > b.tokens || total < 0 || total > cap) paged::report(err, kErrPagedTable);
    }
    return true;
}

// The warp's share of the tokens' rows (K's heads, then V's): kSteps steps of
// kPer rows of one token.
struct Share {
    int tok, r0;  // token, first row
};
__device__ __forceinline__ Share share_of(int rows, int per_warp) {
    const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int parts = (rows + per_warp - 1) / per_warp;
    const long long tok = w / parts;
    return Share{(int)tok, (int)(w - tok * parts) * per_warp};
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename T>
struct Lane16;  // elements of 16 bytes
template <>
struct Lane16<__nv_bfloat16> {
    static constexpr int n = 8;
    // largest magnitude of the 16 bytes, NaN if one is
    static __device__ __forceinline__ float amax(const uint4& u) {
        auto b = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(b(u.x), b(u.y)), __hmax2_nan(b(u.z), b(u.w)));
        return __bfloat162float(__hmax_nan(m.x, m.y));
    }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
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
    static __device__ __forceinline__ float amax(const uint4& u) {
        float x[4];
        unpack(u, x);
        return max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3])));
    }
    static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
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
                                                         long long k_stride, const T* v, long long v_stride, int* err) {
    ptx::pdl_wait_then_trigger();
    if (check_block(g, b, err)) return;
    constexpr int kRow = kLanes ? kLanes : 32, kPer = 32 / kRow;
    const int rows = 2 * g.Hk;
    const Share sh = share_of(rows, kSteps * kPer);
    if (sh.tok >= b.tokens) return;
    const int lane = threadIdx.x & 31, c = lane % kRow, sub = lane / kRow;
    auto source = [&](int r) {
        return r >= g.Hk ? v + sh.tok * v_stride + (long long)(r - g.Hk) * g.d : k + sh.tok * k_stride + (long long)r * g.d;
    };
    if constexpr (kLanes > 0) {
        constexpr int n = Lane16<T>::n;
        uint4 raw[kSteps];  // (the rows' loads do not wait for their place)
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int r = sh.r0 + u * kPer + sub;
            raw[u] = r < rows ? __ldcs(reinterpret_cast<const uint4*>(source(r)) + c) : make_uint4(0u, 0u, 0u, 0u);
        }
        const Place pl = find_place(g, b, nullptr, false, sh.tok, err);
        if (pl.page < 0) return;
        // The scales of the rows, the two divisions of each in one lane only
        float scale = 0.f, inverse = 0.f;
        if constexpr (kCodes) {
            float mine = 0.f;
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                float m = Lane16<T>::amax(raw[u]);
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                mine = c == u ? m : mine;
            }
            const bool finite = mine < INFINITY;
            scale = scale_of(mine, finite);
            inverse = finite ? 1.f / scale : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int r = sh.r0 + u * kPer + sub;
            const bool on = r < rows, is_v = r >= g.Hk;
            const size_t row = on ? paged::pool_row(g, pl.page, is_v ? r - g.Hk : r, pl.key) : 0;
            void* dst = is_v ? pool.v : pool.k;
            if constexpr (!kCodes) {
                if (on) reinterpret_cast<uint4*>(dst)[row * kLanes + c] = raw[u];
            } else {
                const float s = __shfl_sync(0xffffffffu, scale, u, kLanes);
                const float inv = __shfl_sync(0xffffffffu, inverse, u, kLanes);
                if (on) {
                    float x[n];
                    Lane16<T>::unpack(raw[u], x);
                    uint32_t w[n / 4];
#pragma unroll
                    for (int i = 0; i < n / 4; ++i) {
                        uint32_t code = 0;
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const float2 y = make_float2(x[4 * i + j] * inv, x[4 * i + j + 1] * inv);
                            code |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (8 * j);
                        }
                        w[i] = inv != 0.f ? code : 0u;  // (a row that is not finite)
                    }
                    uint32_t* to = reinterpret_cast<uint32_t*>(dst) + (row * kLanes + c) * (n / 4);
                    if constexpr (n == 8)
                        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                    else
                        *to = w[0];
                    if (c == 0) (is_v ? pool.vs : pool.ks)[row] = s;
                }
            }
        }
    } else {
        const Place pl = find_place(g, b, nullptr, false, sh.tok, err);
        if (pl.page < 0) return;
        for (int r = sh.r0; r < sh.r0 + kSteps && r < rows; ++r) {
            const bool is_v = r >= g.Hk;
            const T* src = source(r);
            const size_t row = paged::pool_row(g, pl.page, is_v ? r - g.Hk : r, pl.key);
            void* dst = is_v ? pool.v : pool.k;
            if constexpr (!kCodes) {
                for (int i = lane; i < g.d; i += 32) static_cast<T*>(dst)[row * g.d + i] = src[i];
            } else {
                float amax = 0.f;
                for (int i = lane; i < g.d; i += 32) {
                    const float x = fabsf(paged::to_float(src[i]));
                    amax = x < INFINITY ? fmaxf(amax, x) : INFINITY;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const bool finite = amax < INFINITY;
                const float s = scale_of(amax, finite);
                const float inv = 1.f / s;
                for (int i = lane; i < g.d; i += 32)
                    static_cast<unsigned char*>(dst)[row * g.d + i] =
                        finite ? code_of(paged::to_float(src[i]) * inv) : (unsigned char)0;
                if (lane == 0) (is_v ? pool.vs : pool.ks)[row] = s;
            }
        }
    }
}

template <typename T, bool kCodes, int kLanes>
__global__ void __launch_bounds__(kThreads) read_kernel(PagedGeom g, PagedPool pool, PagedSeqs b, const int* starts,
                                                        T* k, T* v, int* err) {
    ptx::pdl_wait_then_trigger();
    if (check_block(g, b, err)) return;
    constexpr int kRow = kLanes ? kLanes : 32, kPer = 32 / kRow;
    const int rows = 2 * g.Hk;
    const Share sh = share_of(rows, kSteps * kPer);
    if (sh.tok >= b.tokens) return;
    const int lane = threadIdx.x & 31, c = lane % kRow, sub = lane / kRow;
    const Place pl = find_place(g, b, starts, true, sh.tok, err);
    if (pl.page < 0) return;
    auto row_at = [&](int r) { return paged::pool_row(g, pl.page, r >= g.Hk ? r - g.Hk : r, pl.key); };
    auto target = [&](int r) {
        return r >= g.Hk ? v + ((size_t)sh.tok * g.Hk + r - g.Hk) * g.d : k + ((size_t)sh.tok * g.Hk + r) * g.d;
    };
    if constexpr (kLanes > 0) {
        constexpr int n = Lane16<T>::n;
        using Raw = typename std::conditional<!kCodes, uint4, typename std::conditional<n == 8, uint2, uint32_t>::type>::type;
        Raw raw[kSteps];
        float s[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int r = sh.r0 + u * kPer + sub;
            if (r < rows) {
                const bool is_v = r >= g.Hk;
                raw[u] = __ldcs(static_cast<const Raw*>(is_v ? pool.v : pool.k) + row_at(r) * kLanes + c);
                s[u] = kCodes ? __ldg((is_v ? pool.vs : pool.ks) + row_at(r)) : 1.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int r = sh.r0 + u * kPer + sub;
            if (r >= rows) continue;
            uint4* to = reinterpret_cast<uint4*>(target(r)) + c;
            if constexpr (!kCodes) {
                __stcs(to, raw[u]);
            } else {
                uint32_t w[n / 4];
                if constexpr (n == 8)
                    w[0] = raw[u].x, w[1] = raw[u].y;
                else
                    w[0] = raw[u];
                float x[n];
#pragma unroll
                for (int i = 0; i < n; i += 2) {
                    const __half2_raw hr =
                        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(hr));
                    x[i] = f.x * s[u];
                    x[i + 1] = f.y * s[u];
                }
                Lane16<T>::store(to, x);
            }
        }
    } else {
        for (int r = sh.r0; r < sh.r0 + kSteps && r < rows; ++r) {
            const size_t row = row_at(r);
            const bool is_v = r >= g.Hk;
            const void* src = is_v ? pool.v : pool.k;
            const float s = kCodes ? (is_v ? pool.vs : pool.ks)[row] : 1.f;
            T* dst = target(r);
            for (int i = lane; i < g.d; i += 32) {
                if constexpr (kCodes)
                    paged::store_as(dst + i, value_of(static_cast<const unsigned char*>(src)[row * g.d + i]) * s);
                else
                    dst[i] = static_cast<const T*>(src)[row * g.d + i];
            }
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Blocks for the tokens' rows, `per` rows a step, and the one that checks.
unsigned blocks_for(int tokens, int Hk, int per) {
    const int parts = (2 * Hk + kSteps * per - 1) / (kSteps * per);
    return (unsigned)(((long long)tokens * parts + kThreads / 32 - 1) / (kThreads / 32) + 1);
}

template <typename T, bool kCodes>
cudaError_t write_as(const PagedGeom& g, const PagedPool& pool, const PagedSeqs& b, const void* k, long long ks,
                     const void* v, long long vs, int* err, cudaStream_t st) {
    constexpr int n = Lane16<T>::n;
    const bool fits = aligned16(k) && aligned16(v) && ks % n == 0 && vs % n == 0;
    auto go = [&](auto kernel, int lanes) {
        return launch_pdl(kernel, blocks_for(b.tokens, g.Hk, 32 / lanes), kThreads, 0, st, g, pool, b,
                          static_cast<const T*>(k), ks, static_cast<const T*>(v), vs, err);
    };
    if (fits && g.d == 128) return go(write_kernel<T, kCodes, 128 / n>, 128 / n);
    if (fits && g.d == 64) return go(write_kernel<T, kCodes, 64 / n>, 64 / n);
    return go(write_kernel<T, kCodes, 0>, 32);
}

template <typename T, bool kCodes>
cudaError_t read_as(const PagedGeom& g, const PagedPool& pool, const PagedSeqs& b, const int* starts, void* k, void* v,
                    int* err, cudaStream_t st) {
    constexpr int n = Lane16<T>::n;
    const bool fits = aligned16(k) && aligned16(v);
    auto go = [&](auto kernel, int lanes) {
        return launch_pdl(kernel, blocks_for(b.tokens, g.Hk, 32 / lanes), kThreads, 0, st, g, pool, b, starts,
                          static_cast<T*>(k), static_cast<T*>(v), err);
    };
    if (fits && g.d == 128) return go(read_kernel<T, kCodes, 128 / n>, 128 / n);
    if (fits && g.d == 64) return go(read_kernel<T, kCodes, 64 / n>, 64 / n);
    return go(read_kernel<T, kCodes, 0>, 32);
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
