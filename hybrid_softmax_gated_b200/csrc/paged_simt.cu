// Attention of a batch's new tokens over the paged cache in fp32 arithmetic:
// any head width up to 128, fp32 or bf16 tensors, pools as they are or e4m3.
// It serves the fp32 handles and cross-checks the tensor-core kernels.
//
// One CTA works on tiles of 16 RM query rows (new tokens x the query heads of
// one key head) against blocks of 64 keys, with the online softmax: a block's
// scores S = Q K^T in 16 x 16 threads of RM x 4 each, the rows' running
// maximum and sum, then O += P V with O in registers.  A masked key's weight
// is marked (-1) and its value is not multiplied, so it has no effect
// whatever it holds; a weight that rounds to 0 is multiplied (0 x NaN is NaN).  The CTAs split all tiles' blocks evenly and merge a cut
// tile's partials (paged.cuh).  Bound by the fp32 pipes: per 4 features of
// the products a thread loads RM + 4 vectors from shared memory for 16 RM
// multiply-adds (12 to 16 TFLOP/s on long chunks); short calls by one block's
// latency, 14 to 25 us.
#include "paged.cuh"
#include "ptx.cuh"

#include <cmath>
#include <type_traits>

namespace arl2 {
namespace {

constexpr int kThreads = 256;
constexpr int kKB = 64;
constexpr int kPitch = 132;  // floats between rows of Q, K, V in shared memory (d <= 128)

template <int RM>
struct Smem {
    float q[16 * RM][kPitch];
    float k[kKB][kPitch];
    float v[kKB][kPitch];
    float p[16 * RM][kKB + 1];
    float m[16 * RM], l[16 * RM], corr[16 * RM];
    paged::Sight see[16 * RM];
    float ks[kKB], vs[kKB];
    long long row[kKB];  // pool row of each key of the block, -1: not there
    int last;
    int tiles[kPagedMaxSeqs + 1];
    paged::PlanSmem plan;
};

// Four consecutive elements.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const __nv_fp8_e4m3* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3)));
    const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3)));
    return make_float4(a.x, a.y, b.x, b.y);
}

// kVec: heads, strides and pointers take four elements at a time.
template <typename T, typename C, int RM, bool kVec>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(PagedAttend a, float scale_log2) {
    constexpr int R = 16 * RM;
    constexpr int kPerRow = kThreads / R;  // threads that share a row's statistics
    constexpr bool kCodes = std::is_same<C, __nv_fp8_e4m3>::value;
    extern __shared__ float4 smem_raw[];
    Smem<RM>& sm = *reinterpret_cast<Smem<RM>*>(smem_raw);
    const PagedGeom& g = a.g;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    ptx::pdl_wait_then_trigger();
    const paged::Tiling tl{R / g.G, R / g.G, 1, 1, 1, 0, 1};
    const paged::Plan pl = paged::make_plan<kKB>(g, a.seqs, a.mask, tl, 1, sm.plan, sm.tiles, a.err);
    if (pl.u1 == pl.u0) return;
    const T* q = static_cast<const T*>(a.q);
    const C* kp = static_cast<const C*>(a.pool.k);
    const C* vp = static_cast<const C*>(a.pool.v);
    paged::Cursor cur = pl.first;
    while (true) {
        const paged::Piece pc = paged::piece_at<kKB>(a.mask, sm.plan, pl, cur, tl);
        const int rows = pc.n * g.G;
        __syncthreads();  // the previous tile is done with shared memory
        if constexpr (kVec) {
#pragma unroll
            for (int i0 = 0; i0 < R * 32; i0 += kThreads) {
                const int r = (i0 + tid) >> 5, c = 4 * ((i0 + tid) & 31), t = r / g.G;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < rows && c < g.d)
                    x = load4(q + (long long)(pc.q.q0 + pc.i0 + t) * a.q_stride + (cur.h * g.G + r - t * g.G) * g.d + c);
                *reinterpret_cast<float4*>(&sm.q[r][c]) = x;
            }
        }
        for (int i = kVec ? R * 128 : tid; i < R * 128; i += kThreads) {
            const int r = i >> 7, c = i & 127;
            float x = 0.f;
            if (r < rows && c < g.d)
                x = paged::to_float(q[(long long)(pc.q.q0 + pc.i0 + r / g.G) * a.q_stride +
                                      (cur.h * g.G + r % g.G) * g.d + c]);
            sm.q[r][c] = x;
        }
        for (int r = tid; r < R; r += kThreads) {
            sm.m[r] = -INFINITY;
            sm.l[r] = 0.f;
            sm.see[r] = r < rows ? paged::sight(a.mask, pc.q.total - pc.q.n + pc.i0 + r / g.G, pc.q.total)
                                 : paged::Sight{0, 0, 0};
        }
        float4 o[RM][2];
#pragma unroll
        for (int i = 0; i < RM; ++i) o[i][0] = o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int at0 = pc.q.total - pc.q.n + pc.i0;
        const paged::Sight hi = paged::sight(a.mask, at0 + pc.n - 1, pc.q.total);
        const int lo = paged::sight(a.mask, at0 < 0 ? 0 : at0, pc.q.total).lo;
        for (int bi = pc.b0; bi < pc.b1; ++bi) {
            const int key0 = pc.blocks.at(bi) * kKB;
            __syncthreads();
            if (tid < kKB) {
                long long row = -1;
                const int key = key0 + tid;  // (a page that no query of the tile sees is not looked up)
                if (key < hi.end && (key >= lo || key < hi.sink))
                    row = (long long)paged::pool_row(g, paged::page_at(a.seqs, g, cur.s, key0 + tid, a.err), cur.h,
                                                     key0 + tid);
                sm.row[tid] = row;
                if (kCodes) {
                    sm.ks[tid] = row >= 0 ? a.pool.ks[row] : 0.f;
                    sm.vs[tid] = row >= 0 ? a.pool.vs[row] : 0.f;
                }
            }
            __syncthreads();
            if constexpr (kVec) {
#pragma unroll
                for (int i0 = 0; i0 < kKB * 32; i0 += kThreads) {
                    const int j = (i0 + tid) >> 5, c = 4 * ((i0 + tid) & 31);
                    const long long row = sm.row[j];
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                    if (row >= 0 && c < g.d) {
                        x = load4(kp + row * g.d + c);
                        y = load4(vp + row * g.d + c);
                        if (kCodes) {
                            const float ks = sm.ks[j], vs = sm.vs[j];
                            x = make_float4(x.x * ks, x.y * ks, x.z * ks, x.w * ks);
                            y = make_float4(y.x * vs, y.y * vs, y.z * vs, y.w * vs);
                        }
                    }
                    *reinterpret_cast<float4*>(&sm.k[j][c]) = x;
                    *reinterpret_cast<float4*>(&sm.v[j][c]) = y;
                }
            }
            for (int i = kVec ? kKB * 128 : tid; i < kKB * 128; i += kThreads) {
                const int j = i >> 7, c = i & 127;
                const long long row = sm.row[j];
                float x = 0.f, y = 0.f;
                if (row >= 0 && c < g.d) {
                    x = paged::to_float(kp[row * g.d + c]);
                    y = paged::to_float(vp[row * g.d + c]);
                    if (kCodes) x *= sm.ks[j], y *= sm.vs[j];
                }
                sm.k[j][c] = x;
                sm.v[j][c] = y;
            }
            __syncthreads();
            float s[RM][4];
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
            for (int c = 0; c < g.d; c += 4) {  // (features past d are zeros)
                float4 kk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][c]);
#pragma unroll
                for (int i = 0; i < RM; ++i) {
                    const float4 qq = *reinterpret_cast<const float4*>(&sm.q[ty * RM + i][c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(qq.x, kk[j].x, s[i][j]);
                        s[i][j] = fmaf(qq.y, kk[j].y, s[i][j]);
                        s[i][j] = fmaf(qq.z, kk[j].z, s[i][j]);
                        s[i][j] = fmaf(qq.w, kk[j].w, s[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const paged::Sight see = sm.see[ty * RM + i];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sm.p[ty * RM + i][tx + 16 * j] =
                        paged::sees(see, key0 + tx + 16 * j) ? s[i][j] * scale_log2 : -INFINITY;
            }
            __syncthreads();
            {
                const int r = tid / kPerRow, part = tid % kPerRow;
                float mx = -INFINITY;
                for (int j = part; j < kKB; j += kPerRow) mx = fmaxf(mx, sm.p[r][j]);
#pragma unroll
                for (int off = kPerRow / 2; off > 0; off >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float m_old = sm.m[r], m_new = fmaxf(m_old, mx);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                float sum = 0.f;
                for (int j = part; j < kKB; j += kPerRow) {
                    const float x = sm.p[r][j];
                    const float e = exp2f(x - base);  // (x = -inf: 0)
                    // (a visible score may be -inf, too)
                    sm.p[r][j] = x == -INFINITY && !paged::sees(sm.see[r], key0 + j) ? -1.f : e;
                    sum += e;
                }
#pragma unroll
                for (int off = kPerRow / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (part == 0) {
                    const float corr = exp2f(m_old - base);  // (m_old = -inf: 0)
                    sm.corr[r] = corr;
                    sm.m[r] = m_new;
                    sm.l[r] = sm.l[r] * corr + sum;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const float corr = sm.corr[ty * RM + i];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    o[i][c].x *= corr;
                    o[i][c].y *= corr;
                    o[i][c].z *= corr;
                    o[i][c].w *= corr;
                }
            }
            for (int j = 0; j < kKB; ++j) {
                float4 vv[2];
                vv[0] = *reinterpret_cast<const float4*>(&sm.v[j][tx * 4]);
                vv[1] = *reinterpret_cast<const float4*>(&sm.v[j][64 + tx * 4]);
#pragma unroll
                for (int i = 0; i < RM; ++i) {
                    const float p = sm.p[ty * RM + i][j];
                    if (!(p < 0.f)) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            o[i][c].x = fmaf(p, vv[c].x, o[i][c].x);
                            o[i][c].y = fmaf(p, vv[c].y, o[i][c].y);
                            o[i][c].z = fmaf(p, vv[c].z, o[i][c].z);
                            o[i][c].w = fmaf(p, vv[c].w, o[i][c].w);
                        }
                    }
                }
            }
        }
        __syncthreads();
        bool write = true;
        if (pc.c0 != pc.c1) {
            const int slot = paged::partial_slot(pl, blockIdx.x, cur.base);
            float4* po = reinterpret_cast<float4*>(a.work.o) + (size_t)slot * R * 32;
            float2* pm = a.work.ml + (size_t)slot * R;
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                po[(ty * RM + i) * 32 + tx] = o[i][0];
                po[(ty * RM + i) * 32 + 16 + tx] = o[i][1];
            }
            for (int r = tid; r < R; r += kThreads) pm[r] = make_float2(sm.m[r], sm.l[r]);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atomicAdd(a.work.arrived + pc.c0, 1);
                sm.last = n == pc.c1 - pc.c0;
                if (sm.last) a.work.arrived[pc.c0] = 0;
            }
            __syncthreads();
            write = sm.last != 0;
            if (write) {  // every piece of the tile is there: merge in order
                __threadfence();
                for (int r = tid; r < R; r += kThreads) {
                    float m = -INFINITY;
                    for (int c = pc.c0; c <= pc.c1; ++c)
                        m = fmaxf(m, __ldcg(a.work.ml + (size_t)paged::partial_slot(pl, c, cur.base) * R + r).x);
                    float l = 0.f;
                    for (int c = pc.c0; c <= pc.c1; ++c) {
                        const float2 ml = __ldcg(a.work.ml + (size_t)paged::partial_slot(pl, c, cur.base) * R + r);
                        l += ml.x == -INFINITY ? ml.y : ml.y * exp2f(ml.x - m);
                    }
                    sm.m[r] = m;
                    sm.l[r] = l;
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < RM; ++i) o[i][0] = o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = pc.c0; c <= pc.c1; ++c) {
                    const size_t sl = (size_t)paged::partial_slot(pl, c, cur.base);
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        const int r = ty * RM + i;
                        const float mc = __ldcg(a.work.ml + sl * R + r).x;
                        const float w = mc == -INFINITY ? 1.f : exp2f(mc - sm.m[r]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.work.o) + (sl * R + r) * 32 +
                                                    16 * e + tx);
                            o[i][e].x = fmaf(w, x.x, o[i][e].x);
                            o[i][e].y = fmaf(w, x.y, o[i][e].y);
                            o[i][e].z = fmaf(w, x.z, o[i][e].z);
                            o[i][e].w = fmaf(w, x.w, o[i][e].w);
                        }
                    }
                }
            }
        }
        if (write) {
            T* out = static_cast<T*>(a.out);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const int r = ty * RM + i;
                if (r >= rows) continue;
                T* to = out + ((size_t)(pc.q.q0 + pc.i0 + r / g.G) * g.Hq + cur.h * g.G + r % g.G) * g.d;
                const float l = sm.l[r];
                const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: zeros
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x[4] = {o[i][e].x, o[i][e].y, o[i][e].z, o[i][e].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (64 * e + tx * 4 + c < g.d) paged::store_as(to + 64 * e + tx * 4 + c, x[c] * inv);
                }
            }
        }
        if (!paged::advance(sm.plan, pl, a.seqs, tl, pc.units, cur)) break;
    }
}

template <typename T, typename C, int RM, bool kVec>
cudaError_t launch_as(const PagedAttend& a, int max_ctas, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int per_sm = RM == 4 ? 1 : 2;
    int grid = sms * per_sm;
    static_assert(2 * 16 * 4 <= kPagedRowsPerSm && 2 * 2 * 16 <= kPagedRowsPerSm, "workspace rows");
    if (max_ctas > 0 && max_ctas < grid) grid = max_ctas;
    return launch_pdl(paged_simt_kernel<T, C, RM, kVec>, grid, kThreads, sizeof(Smem<RM>), st, a,
                      a.scale * 1.4426950408889634f);
}

template <typename T, typename C, int RM>
cudaError_t launch(const PagedAttend& a, int max_ctas, cudaStream_t st) {
    const bool vec = a.g.d % 4 == 0 && a.q_stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.q) % (4 * sizeof(T)) == 0;
    return vec ? launch_as<T, C, RM, true>(a, max_ctas, st) : launch_as<T, C, RM, false>(a, max_ctas, st);
}

template <typename T, typename C>
cudaError_t launch_rows(const PagedAttend& a, int max_new, int max_ctas, cudaStream_t st) {
    // 16-row tiles when that holds every sequence's rows of a key head, or
    // the group alone fills them; 64-row tiles read a key block once for
    // four times the rows
    const long long tiles = ((long long)a.seqs.tokens * a.g.G + 63) / 64 * a.g.Hk;
    const long long keys = (long long)a.seqs.max_pages << a.g.page_log2;
    // (also when 64-row tiles would give work to half of a B200's 148 SMs at most:
    // 34 tokens of 8 heads on 43 keys 21 -> 16 us; 160 of 24 on 98 keys, above that
    // border, would take 33, not 27)
    if (a.g.G <= 16 && ((long long)max_new * a.g.G <= 16 || tiles * ((keys + kKB - 1) / kKB) <= 74))
        return launch<T, C, 1>(a, max_ctas, st);
    return launch<T, C, 4>(a, max_ctas, st);
}

template <typename T, typename C, int RM, bool kVec>
cudaError_t allow() {
    return cudaFuncSetAttribute(paged_simt_kernel<T, C, RM, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Smem<RM>));
}
template <typename T, typename C>
cudaError_t init_one() {
    cudaError_t e = allow<T, C, 1, false>();
    if (e == cudaSuccess) e = allow<T, C, 1, true>();
    if (e == cudaSuccess) e = allow<T, C, 4, false>();
    return e == cudaSuccess ? allow<T, C, 4, true>() : e;
}

}  // namespace

cudaError_t paged_simt_init() {
    cudaError_t e = init_one<float, float>();
    if (e == cudaSuccess) e = init_one<float, __nv_fp8_e4m3>();
    if (e == cudaSuccess) e = init_one<__nv_bfloat16, __nv_bfloat16>();
    if (e == cudaSuccess) e = init_one<__nv_bfloat16, __nv_fp8_e4m3>();
    return e;
}

cudaError_t launch_paged_simt(bool bf16, bool e4m3, const PagedAttend& a, int max_new, int max_ctas, cudaStream_t st) {
    if (bf16)
        return e4m3 ? launch_rows<__nv_bfloat16, __nv_fp8_e4m3>(a, max_new, max_ctas, st)
                    : launch_rows<__nv_bfloat16, __nv_bfloat16>(a, max_new, max_ctas, st);
    return e4m3 ? launch_rows<float, __nv_fp8_e4m3>(a, max_new, max_ctas, st)
                : launch_rows<float, float>(a, max_new, max_ctas, st);
}

}  // namespace arl2
