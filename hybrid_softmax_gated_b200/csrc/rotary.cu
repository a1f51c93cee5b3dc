// Rotary positions with up to four axes: the C ABI of include/arl2.h
// (arl2_rotary_*) and its kernel.
//
// Pair p of a head turns by angle = pos[axis(p)] f_p.  The frequency is kept
// in turns as a 64-bit fraction F_p = f_p / (2 pi) * 2^64, so the product
// pos * F_p mod 2^64 IS the angle reduced to one turn, exact but for F_p's
// own rounding (2^-65 turns per position step): no range reduction, and a
// position of 10^6 costs no accuracy.  Its top part goes through sincospif.
//
// Memory bound: q and k are read once and written once.  A thread has one
// place of a head (16 bytes of features, or two) and up to four heads of one
// token; its loads are on their way while the block works out its tokens'
// sines, once each, into shared memory.  14400 tokens of 24 heads: 32 us, 5.5
// TB/s.
#include "arl2.h"
#include "internal.h"
#include "ptx.cuh"

#include <cmath>
#include <cstdint>
#include <new>

namespace arl2 {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kThreads = 256;
constexpr int kMaxTokensPerBlock = 32;
constexpr int kMaxTokens = 1 << 30;  // (with a block's tokens on top it still fits an int)
constexpr int kInFlight = 4;  // heads of an item, all their loads on their way together

// The plan as the kernel gets it (1.2 KB of launch parameters).
struct Plan {
    unsigned long long freq[kMaxPairs];  // turns per position, as a fraction of 2^64
    unsigned char axis[kMaxPairs];
    int d, axes, rot;                    // rot = R: turned features
};

struct Side {
    const void* in;
    void* out;
    long long in_stride, out_stride;     // elements between tokens
    int heads;
};

// A place of a head: what an item turns, 16 bytes of it (kHalves: 16 bytes of
// each half), or, with kWide = false, one pair in single elements: the form
// for heads, strides or pointers that 16-byte vectors do not fit.  kHalves:
// pair p = features (p, p + R/2), else (2p, 2p + 1).
template <typename T, bool kHalves, bool kWide>
struct Form {
    static constexpr int kBytes = kWide ? 16 : (int)sizeof(T);  // of a load
    static constexpr int NP = kWide ? (kHalves ? 16 : 8) / (int)sizeof(T) : 1;
    static constexpr int kLoads = !kWide ? 2 : kHalves ? 2 : 1;
    static constexpr int kStep = kHalves || !kWide ? kBytes / (int)sizeof(T) : 2 * NP;  // features from place to place
    static constexpr int kTail = kBytes / (int)sizeof(T);  // untouched features of an item behind the turned ones
};
template <int kBytes>
struct RawOf;
template <>
struct RawOf<16> {
    using type = uint4;
};
template <>
struct RawOf<4> {
    using type = uint32_t;
};
template <>
struct RawOf<2> {
    using type = uint16_t;
};

// (written out, so that every form of the kernel rounds alike)
__device__ __forceinline__ float2 turn1(float x, float y, float2 cs) {
    return make_float2(__fmaf_rn(x, cs.x, -__fmul_rn(y, cs.y)), __fmaf_rn(x, cs.y, __fmul_rn(y, cs.x)));
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The two words of a pair's features (fp32), or of two pairs' (bf16).
template <typename T>
__device__ __forceinline__ void turn_halves(uint32_t& a, uint32_t& b, const float2* cs) {
    if constexpr (sizeof(T) == 4) {
        const float2 z = turn1(__uint_as_float(a), __uint_as_float(b), cs[0]);
        a = __float_as_uint(z.x), b = __float_as_uint(z.y);
    } else {
        const float2 z = turn1(low_bf16(a), low_bf16(b), cs[0]), w = turn1(high_bf16(a), high_bf16(b), cs[1]);
        a = pack_bf16(z.x, w.x), b = pack_bf16(z.y, w.y);
    }
}
template <typename T, bool kHalves>
__device__ __forceinline__ void turn16(uint4& a, uint4& b, const float2* cs) {
    if constexpr (kHalves) {
        constexpr int n = 4 / (int)sizeof(T);
        turn_halves<T>(a.x, b.x, cs);
        turn_halves<T>(a.y, b.y, cs + n);
        turn_halves<T>(a.z, b.z, cs + 2 * n);
        turn_halves<T>(a.w, b.w, cs + 3 * n);
    } else if constexpr (sizeof(T) == 4) {
        turn_halves<T>(a.x, a.y, cs);
        turn_halves<T>(a.z, a.w, cs + 1);
    } else {
        uint32_t* w[4] = {&a.x, &a.y, &a.z, &a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = turn1(low_bf16(*w[i]), high_bf16(*w[i]), cs[i]);
            *w[i] = pack_bf16(z.x, z.y);
        }
    }
}
// One pair in single elements.
template <typename T, typename R>
__device__ __forceinline__ void turn_single(R& a, R& b, float2 cs) {
    if constexpr (sizeof(T) == 4) {
        const float2 z = turn1(__uint_as_float(a), __uint_as_float(b), cs);
        a = __float_as_uint(z.x), b = __float_as_uint(z.y);
    } else {
        const float2 z = turn1(low_bf16(a), low_bf16(b), cs);
        const uint32_t w = pack_bf16(z.x, z.y);
        a = (R)w, b = (R)(w >> 16);
    }
}

// An item is a place of up to `group` heads of q or of k, of one token.
template <typename T, bool kHalves, bool kWide>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Plan plan, Side q, Side k,
                                                          const int* __restrict__ positions, int tokens, int per_block,
                                                          int group, float sign) {
    using F = Form<T, kHalves, kWide>;
    using R = typename RawOf<F::kBytes>::type;
    extern __shared__ float2 cs[];  // [token][pair]
    ptx::pdl_wait_then_trigger();
    const int half = plan.rot >> 1, d = plan.d;
    const int tok0 = blockIdx.x * per_block;
    const int n_tok = min(per_block, tokens - tok0);
    const int turned = half / F::NP;  // places that turn
    const int per_head = turned + (d - plan.rot) / F::kTail;
    const int q_groups = (q.heads + group - 1) / group, groups = q_groups + (k.heads + group - 1) / group;
    const int items = n_tok * groups * per_head;
    const int other = kHalves ? half : 1;  // from a pair's first feature to its second
    int t = 0, e = 0, n = 0;
    const T* in = nullptr;
    T* out = nullptr;
    R a[kInFlight], b[kInFlight];
    auto open = [&](int i) {  // item i's place; its loads
        const int tg = i / per_head;
        e = i - tg * per_head;
        t = tg / groups;
        int gr = tg - t * groups;
        const bool is_k = gr >= q_groups;
        if (is_k) gr -= q_groups;
        const Side& sd = is_k ? k : q;
        const int h0 = gr * group;
        n = min(group, sd.heads - h0);
        const int off = h0 * d + (e < turned ? e * (kWide || kHalves ? F::kStep : 2) : plan.rot + (e - turned) * F::kTail);
        in = static_cast<const T*>(sd.in) + (tok0 + t) * sd.in_stride + off;
        out = static_cast<T*>(sd.out) + (tok0 + t) * sd.out_stride + off;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (u < n) {
                a[u] = *reinterpret_cast<const R*>(in + u * d);
                if (F::kLoads == 2 && e < turned) b[u] = *reinterpret_cast<const R*>(in + u * d + other);
            }
    };
    int i = threadIdx.x;
    if (i < items) open(i);
    for (int p = threadIdx.x; p < n_tok * half; p += kThreads) {
        const int pt = p / half, pp = p - pt * half;
        const long long pos = positions[(size_t)(tok0 + pt) * plan.axes + plan.axis[pp]];
        const long long phase = (long long)((unsigned long long)pos * plan.freq[pp]);
        float s, c;
        sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &c);
        cs[p] = make_float2(c, s * sign);
    }
    __syncthreads();
    for (; i < items; i += kThreads) {
        if (i >= kThreads) open(i);
        const bool turns = e < turned;
        float2 c[F::NP];
        if (turns) {
#pragma unroll
            for (int j = 0; j < F::NP; ++j) c[j] = cs[t * half + e * F::NP + j];
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (u < n) {
                if (turns) {
                    if constexpr (kWide)
                        turn16<T, kHalves>(a[u], b[u], c);
                    else
                        turn_single<T>(a[u], b[u], c[0]);
                    if (F::kLoads == 2) *reinterpret_cast<R*>(out + u * d + other) = b[u];
                }
                *reinterpret_cast<R*>(out + u * d) = a[u];
            }
    }
}

template <typename T, bool kHalves, bool kWide>
cudaError_t launch_as(const Plan& p, const Side& q, const Side& k, const int* pos, int tokens, float sign,
                      cudaStream_t st) {
    using F = Form<T, kHalves, kWide>;
    const int per_head = p.rot / 2 / F::NP + (p.d - p.rot) / F::kTail;
    // Heads of an item: as many as are in flight, fewer when the items would not
    // be two blocks of threads on each of a B200's 148 SMs (a token's heads then
    // spread over the block's threads); tokens of a block: what its threads
    // have one item each for
    int group = kInFlight, groups;
    while (true) {
        groups = (q.heads + group - 1) / group + (k.heads + group - 1) / group;
        if (group == 1 || (long long)tokens * per_head * groups >= 148 * 512) break;
        group /= 2;
    }
    int per_block = kThreads / (per_head * groups);
    per_block = per_block < 1 ? 1 : per_block > kMaxTokensPerBlock ? kMaxTokensPerBlock : per_block;
    const int grid = (tokens + per_block - 1) / per_block;
    return launch_pdl(rotary_kernel<T, kHalves, kWide>, grid, kThreads, (size_t)per_block * (p.rot / 2) * sizeof(float2),
                      st, p, q, k, pos, tokens, per_block, group, sign);
}

template <typename T, bool kHalves>
cudaError_t launch(const Plan& p, const Side& q, const Side& k, const int* pos, int tokens, float sign, bool wide,
                   cudaStream_t st) {
    return wide ? launch_as<T, kHalves, true>(p, q, k, pos, tokens, sign, st)
                : launch_as<T, kHalves, false>(p, q, k, pos, tokens, sign, st);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace arl2

struct arl2_rotary {
    arl2::Plan plan;
    arl2_pairs pairs;
};

namespace arl2 {

int rotary_head_dim(const arl2_rotary* r) { return r->plan.d; }

}  // namespace arl2

extern "C" {

arl2_status arl2_rotary_create(const arl2_rotary_config* cfg, arl2_rotary** out) {
    if (!cfg || !out) return ARL2_ERR_INVALID_ARG;
    *out = nullptr;
    if (cfg->pairs != ARL2_PAIRS_ADJACENT && cfg->pairs != ARL2_PAIRS_HALVES) return ARL2_ERR_INVALID_ARG;
    if (cfg->freqs != ARL2_FREQS_PER_AXIS && cfg->freqs != ARL2_FREQS_SHARED) return ARL2_ERR_INVALID_ARG;
    if (!(cfg->base >= 1.0) || std::isinf(cfg->base)) return ARL2_ERR_INVALID_ARG;
    if (cfg->head_dim < 2 || cfg->head_dim > 2 * arl2::kMaxPairs || cfg->axes < 1 || cfg->axes > 4)
        return ARL2_ERR_SHAPE;
    long long rot = 0;
    for (int a = 0; a < cfg->axes; ++a) {
        if (cfg->axis_dim[a] < 0 || cfg->axis_dim[a] % 2) return ARL2_ERR_SHAPE;
        rot += cfg->axis_dim[a];
    }
    if (rot < 2 || rot > cfg->head_dim) return ARL2_ERR_SHAPE;
    arl2_rotary* r = new (std::nothrow) arl2_rotary();
    if (!r) return ARL2_ERR_OOM;
    r->pairs = cfg->pairs;
    r->plan.d = cfg->head_dim;
    r->plan.axes = cfg->axes;
    r->plan.rot = (int)rot;
    int p = 0;
    for (int a = 0; a < cfg->axes; ++a) {
        for (int i = 0; i < cfg->axis_dim[a] / 2; ++i, ++p) {
            const long double x = cfg->freqs == ARL2_FREQS_SHARED ? 2.0L * p / (long double)rot
                                                                  : 2.0L * i / (long double)cfg->axis_dim[a];
            const long double turns = powl((long double)cfg->base, -x) / 6.283185307179586476925286766559005768L;
            r->plan.freq[p] = (unsigned long long)(ldexpl(turns, 64) + 0.5L);
            r->plan.axis[p] = (unsigned char)a;
        }
    }
    *out = r;
    return ARL2_OK;
}

arl2_status arl2_rotary_apply(const arl2_rotary* r, arl2_dtype dtype, int tokens, const int* positions,
                              int q_heads, const void* q, long long q_stride, void* q_out,
                              long long q_out_stride, int k_heads, const void* k, long long k_stride,
                              void* k_out, long long k_out_stride, int inverse, cudaStream_t stream) {
    if (!r || (dtype != ARL2_BF16 && dtype != ARL2_FP32)) return ARL2_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > arl2::kMaxTokens || q_heads < 0 || k_heads < 0 || q_heads > 1024 || k_heads > 1024) return ARL2_ERR_SHAPE;
    if (tokens == 0 || q_heads + k_heads == 0) return ARL2_OK;
    if (!positions || (q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out))) return ARL2_ERR_INVALID_ARG;
    const int d = r->plan.d;
    const size_t esz = dtype == ARL2_BF16 ? 2 : 4;
    if (!q_heads) q_stride = q_out_stride = 0, q = q_out = nullptr;
    if (!k_heads) k_stride = k_out_stride = 0, k = k_out = nullptr;
    arl2::Side sq{q, q_out, q_stride ? q_stride : (long long)q_heads * d,
                  q_out_stride ? q_out_stride : (long long)q_heads * d, q_heads};
    arl2::Side sk{k, k_out, k_stride ? k_stride : (long long)k_heads * d,
                  k_out_stride ? k_out_stride : (long long)k_heads * d, k_heads};
    const bool halves = r->pairs == ARL2_PAIRS_HALVES;
    const int vec = 16 / (int)esz;
    // 16-byte vectors need whole vectors in each half, head and token step
    bool wide = (halves ? r->plan.rot / 2 : r->plan.rot) % vec == 0 && d % vec == 0;
    for (const arl2::Side* s : {&sq, &sk}) {
        if (s->in_stride < (long long)s->heads * d || s->out_stride < (long long)s->heads * d)
            return ARL2_ERR_SHAPE;
        if (!arl2::aligned(s->in, esz) || !arl2::aligned(s->out, esz)) return ARL2_ERR_ALIGN;
        wide = wide && arl2::aligned(s->in, 16) && arl2::aligned(s->out, 16) && s->in_stride % vec == 0 &&
               s->out_stride % vec == 0;
    }
    if (!arl2::aligned(positions, 4)) return ARL2_ERR_ALIGN;
    const float sign = inverse ? -1.f : 1.f;
    cudaError_t e;
    if (dtype == ARL2_BF16)
        e = halves ? arl2::launch<__nv_bfloat16, true>(r->plan, sq, sk, positions, tokens, sign, wide, stream)
                   : arl2::launch<__nv_bfloat16, false>(r->plan, sq, sk, positions, tokens, sign, wide, stream);
    else
        e = halves ? arl2::launch<float, true>(r->plan, sq, sk, positions, tokens, sign, wide, stream)
                   : arl2::launch<float, false>(r->plan, sq, sk, positions, tokens, sign, wide, stream);
    return e == cudaSuccess ? ARL2_OK : ARL2_ERR_CUDA;
}

void arl2_rotary_destroy(arl2_rotary* r) { delete r; }

}  // extern "C"
