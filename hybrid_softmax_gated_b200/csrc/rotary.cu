// Rotary positions with up to four axes: the C ABI of include/arl2.h
// (arl2_rotary_*) and its kernel.
//
// Pair p of a head turns by angle = pos[axis(p)] f_p.  The frequency is kept
// in turns as a 64-bit fraction F_p = f_p / (2 pi) * 2^64, so the product
// pos * F_p mod 2^64 IS the angle reduced to one turn, exact but for F_p's
// own rounding (2^-65 turns per position step): no range reduction, and a
// position of 10^6 costs no accuracy.  Its top part goes through sincospif.
//
// Memory bound: q and k are read once and written once.  A thread keeps one
// place of a head (a 16-byte vector of features) and one token, works out its
// few pairs' sines once, in registers, and turns that place of the token's
// heads, four loads in flight.  Few tokens: a token's heads are split over
// more threads.  14400 tokens of 24 heads (177 MB in all): 32 us, 5.5 TB/s.
#include "arl2.h"
#include "internal.h"

#include <cmath>
#include <cstdint>
#include <new>

namespace arl2 {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kThreads = 256;
constexpr int kInFlight = 4;  // heads a thread loads before it turns them

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

template <typename T>
__device__ __forceinline__ float to_f(T x) {
    return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T, int N, int kAlign>
struct __align__(kAlign) Vec {
    T v[N];
};

// A thread's place of a head: NP pairs, or (past the turned features) kTail
// elements copied through.  kHalves: pair p = features (p, p + R/2).  NP = 1
// is the form for heads, strides or pointers that 16-byte vectors do not
// fit: it touches single elements.  `split` threads share the heads of a place.
template <typename T, bool kHalves, int NP>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Plan plan, Side q, Side k,
                                                          const int* __restrict__ positions, int tokens, int split,
                                                          float sign) {
    constexpr int N = kHalves ? NP : 2 * NP;  // elements of one vector
    constexpr int kTail = NP == 1 ? 1 : N;
    using V = Vec<T, N, NP == 1 ? sizeof(T) : 16>;
    using Tail = Vec<T, kTail, NP == 1 ? sizeof(T) : 16>;
    const int half = plan.rot >> 1;
    const int turned = half / NP;  // places that turn
    const int per_head = turned + (plan.d - plan.rot) / kTail;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    // (a division of 64-bit numbers costs more than all of a place's sines)
    const bool small = i < (1ll << 32);
    const long long hs = small ? (unsigned)i / (unsigned)per_head : i / per_head;
    const int e = (int)(i - hs * per_head);
    const long long tok = small ? (unsigned)hs / (unsigned)split : hs / split;
    const int h0 = (int)(hs - tok * split);
    if (tok >= tokens) return;
    const int heads = q.heads + k.heads;
    const bool turns = e < turned;
    float c[NP], s[NP];
    if (turns) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int p = e * NP + j;
            const long long pos = positions[tok * plan.axes + plan.axis[p]];
            const long long phase = (long long)((unsigned long long)pos * plan.freq[p]);
            sincospif(__ll2float_rn(phase) * 0x1p-63f, &s[j], &c[j]);
            s[j] *= sign;
        }
    }
    const int off = turns ? e * N : plan.rot + (e - turned) * kTail;
    const T* qi = static_cast<const T*>(q.in) + tok * q.in_stride + off;
    const T* ki = static_cast<const T*>(k.in) + tok * k.in_stride + off;
    T* qo = static_cast<T*>(q.out) + tok * q.out_stride + off;
    T* ko = static_cast<T*>(k.out) + tok * k.out_stride + off;
    auto in_at = [&](int h) { return h < q.heads ? qi + h * plan.d : ki + (h - q.heads) * plan.d; };
    auto out_at = [&](int h) { return h < q.heads ? qo + h * plan.d : ko + (h - q.heads) * plan.d; };
    for (int h1 = h0; h1 < heads; h1 += kInFlight * split) {
        if (turns) {
            V a[kInFlight], b[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int h = h1 + u * split;
                if (h < heads) {
                    a[u] = *reinterpret_cast<const V*>(in_at(h));
                    if constexpr (kHalves) b[u] = *reinterpret_cast<const V*>(in_at(h) + half);
                }
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int h = h1 + u * split;
                if (h < heads) {
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        T& xt = kHalves ? a[u].v[j] : a[u].v[2 * j];
                        T& yt = kHalves ? b[u].v[j] : a[u].v[2 * j + 1];
                        const float x = to_f(xt), y = to_f(yt);
                        xt = from_f<T>(x * c[j] - y * s[j]);
                        yt = from_f<T>(x * s[j] + y * c[j]);
                    }
                    *reinterpret_cast<V*>(out_at(h)) = a[u];
                    if constexpr (kHalves) *reinterpret_cast<V*>(out_at(h) + half) = b[u];
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int h = h1 + u * split;
                if (h < heads) *reinterpret_cast<Tail*>(out_at(h)) = *reinterpret_cast<const Tail*>(in_at(h));
            }
        }
    }
}

template <typename T, bool kHalves, int NP>
cudaError_t launch_as(const Plan& p, const Side& q, const Side& k, const int* pos, int tokens, float sign,
                      cudaStream_t st) {
    constexpr int kTail = NP == 1 ? 1 : kHalves ? NP : 2 * NP;
    const long long places = (long long)tokens * (p.rot / 2 / NP + (p.d - p.rot) / kTail);
    const int heads = q.heads + k.heads;
    // Threads per place: one while that fills the GPU (1000 threads per SM);
    // with fewer tokens each thread takes fewer heads, down to one
    long long split = (148 * 1000 + places - 1) / places;
    if (split > heads) split = heads;
    const long long blocks = (places * split + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    rotary_kernel<T, kHalves, NP><<<(unsigned)blocks, kThreads, 0, st>>>(p, q, k, pos, tokens, (int)split, sign);
    return cudaGetLastError();
}

template <typename T, bool kHalves>
cudaError_t launch(const Plan& p, const Side& q, const Side& k, const int* pos, int tokens, float sign, bool wide,
                   cudaStream_t st) {
    constexpr int kWide = (kHalves ? 16 : 8) / (int)sizeof(T);  // pairs per 16-byte vector
    return wide ? launch_as<T, kHalves, kWide>(p, q, k, pos, tokens, sign, st)
                : launch_as<T, kHalves, 1>(p, q, k, pos, tokens, sign, st);
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
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || q_heads > 1024 || k_heads > 1024) return ARL2_ERR_SHAPE;
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
