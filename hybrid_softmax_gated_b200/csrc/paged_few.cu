// Attention over the paged cache for tiles of at most 16 query rows (the next
// tokens of many streams: new tokens x the query heads of one key head): the
// products transposed, so that the keys are the tensor cores' 128 rows and the
// queries their columns.  bf16 queries and outputs, head width 128, pages of
// bf16 or of e4m3 codes with one scale per token and head.
//
//   S^T [128 keys x 16]  = K Q^T      (K from the page, as it lies)
//   O^T [128 features x 16] += V^T P^T  (V from the page, as it lies)
//
// The products cost an eighth of what 128-row query tiles would, most of
// their rows empty; what is left is the pages' way from memory to shared
// memory, which is the bound.  Pages of codes are not converted at all:
//   Q = the sum of two e4m3 terms, q 2^k = hi + lo (see paged_tc.cu), 16 columns each;
//   P = the sum of three e4m3 terms, 16 columns each: a weight w (times the
//     value's scale, and scaled so that the largest of a row lies in [2^7,
//     448]) = t_0 + t_1 / 16 + t_2 / 256, each term the e4m3 of what the ones
//     before leave.  A term's error is half a step of its 4 bits, so the next
//     one, times 16, fits; the last is off by at most 2^-10 / 256, 2^-25 of
//     the row's largest weight, and by 2^-12 of the weight itself otherwise.
// Scores, weights, sums and accumulators are fp32; with bf16 pages the weights
// are rounded to bf16, the type of that product.
//
// One softmax thread has one key of a block (a TMEM lane of S^T) and all rows'
// scores against it.  A row's maximum over the block takes a reduction in each
// warp and one exchange between the four warps of the warpgroup.  It is a
// lazy base c: weights are 2^(score - c), and c moves only when a weight would
// pass the terms' range, which rescales O.  With codes O has a base of its own,
// o: it differs from c only where all values that weigh in a row have scales
// below 2^-93, whose weights alone would not fit fp32 at the terms' range (down
// to 2^-126 they are 2^133).  The two warpgroups take alternate
// blocks, with their own bases and accumulators; the epilogue combines them.
// 48 streams of up to 12000 keys (32 heads on 8): 236 to 242 us, 6.5 TB/s, the
// rate of a copy; 64 streams with a window of 8192 keys over e4m3 pages: 182 to
// 194 us (170 in the first launches), 5.5 to 5.8 TB/s.
//
// Schedule, loads and what keeps hidden values that are not finite out of the
// products: paged_tc.cuh.
#include "paged_tc.cuh"

#include <cmath>

namespace arl2 {
namespace {

using paged::Desc;
using paged::kCodeTile;
using paged::kD;
using paged::kDescs;
using paged::kKB;
using paged::kSoftmaxWarps;
using paged::kTileBytes;
using paged::kWaitLimitNs;
using paged::kWgWarps;

constexpr int kThreads = 384;
constexpr int kN = 16;                    // columns of a term (query rows)
// For the schedule, in blocks: what a tile costs on top of its blocks, up to
// what it is not cut, and how much a CTA has at least.  (With no cost for a tile
// and short ones cut, four streams of 300 keys take 16.7 us, not 12.4; with the
// cost but short ones cut, 16 streams of 1000 keys 26.0, not 16.8.)
constexpr int kTileCost = 4, kWhole = 16, kMinUnits = 8;
static_assert(kMinUnits > kTileCost, "one border at most in what a tile costs for itself");
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS = 0, kColO = 128;  // four S buffers of 32 columns; O_0, O_1 of 64
constexpr float kTopBits = 7.f;           // codes: the largest weight is 2^7 when c is set ...
constexpr float kLazyCodes = 1.75f;       // ... and may grow to 2^8.75 (e4m3 ends at 448 = 2^8.8)
constexpr float kLazyBf16 = 8.f;
constexpr float kLeastScale = -100.f;     // c: weights up to 2^(100 + kLazyCodes), whose sums fit fp32
constexpr float kLeastCode = -126.f - kTopBits;  // o: of the least scale of a row

template <bool kCodes>
struct __align__(1024) Smem {
    // enough tiles on their way to keep HBM busy
    static constexpr int kK = kCodes ? 6 : 3, kKBytes = kCodes ? kCodeTile : (int)kTileBytes;
    static constexpr int kVLoads = kCodes ? 5 : 3;
    static constexpr int kTerms = kCodes ? 3 : 1;
    static constexpr uint32_t kQHalf = kN * 128;
    static constexpr bool kClean = true;
    uint8_t k[kK][kKBytes];
    uint8_t v[kVLoads][kKBytes];
    uint8_t q[2][2 * kQHalf];                 // two halves of 64 features; codes: then the two terms
    uint8_t p[2][kCodes ? 3 * kN * 128 : 2 * kN * 128];
    // scratch of the plan, then (codes) the blocks' scales: K of block j is
    // loaded when S of block j - kK is done, which comes after P V of block
    // j - kK - 4: the slots of those in between may be in use
    static constexpr int kScaleSlots = kK + 4;
    __align__(16) int scratch[kCodes ? kScaleSlots * 2 * kKB : kPagedMaxSeqs + 4];
    static_assert(kScaleSlots * 2 * kKB > kPagedMaxSeqs, "scratch");
    __device__ float* ks(int blk) { return reinterpret_cast<float*>(scratch) + blk % kScaleSlots * 2 * kKB; }
    __device__ float* vs(int blk) { return ks(blk) + kKB; }
    float row_scale[4][kN];
    float top[2][2][kWgWarps][kN];            // [warpgroup][item & 1][warp][row]: block maxima for c
    float o_top[kCodes ? 2 : 1][2][kWgWarps][kN];  // and for o, where they differ in some row:
    __align__(4) uint8_t o_apart[2][2][kWgWarps];
    float red_l[kSoftmaxWarps][kN], red_c[2][kN], red_o[2][kN];
    uint64_t d_full[kDescs], d_empty[kDescs];
    uint64_t q_raw[2], q_full[2], q_empty[2];
    uint64_t k_full[kK], k_empty[kK];
    uint64_t v_full[kVLoads], v_empty[kVLoads];
    uint64_t v_edge[kVLoads];  // a block of V that some query does not see all of: landed, not cleaned yet
    uint64_t s_full[4], s_taken[4];  // by item & 3: S in TMEM; read (4 warp arrivals)
    uint64_t p_full[2], pv_done[2];  // by warpgroup: 4 warp arrivals; one commit per item
    uint64_t o_free, ebar, wbar[2], drain;
    Desc desc[kDescs];
    uint32_t tmem_base;
    int abort;
    int last;
    paged::Plan pl;
    paged::PlanSmem plan;
    __device__ uint64_t* q_landed(int s) { return kCodes ? &q_raw[s] : &q_full[s]; }
    __device__ uint64_t* v_landed(int s) { return &v_full[s]; }
    __device__ uint64_t* v_taken(int s) { return &v_empty[s]; }
    __device__ uint8_t* v_load(int s) { return v[s]; }
};

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_of(float x) {
    return (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float of_e4m3(uint32_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// What rows first .. first + 7 of a piece that had values taken out get of them
// (lane l knows what row l sees): feature `at`.
static __device__ __noinline__ void give_rows_back(const PagedAttend& a, const Desc& d, paged::Sight mine, int first, int at,
                                                   float (&sum)[8]) {
    const paged::Seen seen = paged::seen_by(a.mask, d);
#pragma unroll
    for (int r = 0; r < 8; ++r) sum[r] = 0.f;
    paged::for_edge_keys(a, d, seen, [&](const __nv_bfloat16* v, int j) {
#pragma unroll 8
        for (int u = 0; u < paged::kEdgeKeys; ++u) {
            const float x = __bfloat162float(v[u * kD + at]);
            const uint32_t rows =
                __ballot_sync(0xffffffffu, paged::sees(mine, j + u) && !paged::sees(seen.all, j + u)) >> first;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if ((rows >> r & 1u) && !(fabsf(x) < INFINITY)) sum[r] += x;
        }
    });
}

// NR: rows of a tile (4, 8 or 16).
template <bool kCodes, int NR>
__global__ void __launch_bounds__(kThreads, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttend a,
                     float scale_log2) {
    using S = Smem<kCodes>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    if (ptx::smem_u32(smem_raw) & 1023u) {  // (the swizzled tiles need it)
        if (threadIdx.x == 0) atomicOr(a.err, kErrPagedTimeout);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedGeom& g = a.g;
    volatile int* abort = &sm.abort;
    const int no_abort = 0;
    if (threadIdx.x == 0) {
        auto init = [](uint64_t* b, int n) { ptx::mbar_init(ptx::smem_u32(b), n); };
        for (int i = 0; i < kDescs; ++i) {
            init(&sm.d_full[i], 1);
            init(&sm.d_empty[i], 1 + kSoftmaxWarps + 2);
            init(&sm.s_full[i], 1);
            init(&sm.s_taken[i], kWgWarps);
        }
        for (int i = 0; i < S::kK; ++i) {
            init(&sm.k_full[i], paged::kKArrivals<kCodes>);
            init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < S::kVLoads; ++i) {
            init(&sm.v_full[i], 1);
            init(&sm.v_empty[i], 1);
            init(&sm.v_edge[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            init(&sm.q_raw[i], 1);
            init(&sm.q_full[i], 1);
            init(&sm.q_empty[i], 1);
            init(&sm.p_full[i], kWgWarps);
            init(&sm.pv_done[i], 1);
            init(&sm.wbar[i], kWgWarps);
        }
        init(&sm.o_free, kSoftmaxWarps);
        init(&sm.ebar, kSoftmaxWarps);
        init(&sm.drain, 1);
        sm.abort = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_u32(&sm.tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::pdl_wait_then_trigger();  // (nothing before this touches global memory)
    const paged::Tiling tl{NR / g.G, NR / g.G, 1, 1, 1, kTileCost, kWhole};
    const paged::Plan pl = paged::make_plan<kKB>(g, a.seqs, a.mask, tl, kMinUnits, sm.plan, sm.scratch, a.err);
    if (threadIdx.x == 0) sm.pl = pl;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    auto fail = [&]() {
        atomicOr(a.err, kErrPagedTimeout);
        *abort = 1;
    };
    auto wwait = [&](uint64_t* bar, uint32_t parity) {
        return ptx::mbar_wait_warp(ptx::smem_u32(bar), parity, abort, kWaitLimitNs);
    };
    auto arrive1 = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(bar));
    };
    auto get_desc = [&](int si, Desc& d) -> bool {
        if (!wwait(&sm.d_full[si % kDescs], (si / kDescs) & 1)) return false;
        d = sm.desc[si % kDescs];
        arrive1(&sm.d_empty[si % kDescs]);
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------------ loader --
        if (!paged::load_pieces<kCodes, false>(sm, tm_q, tm_k, tm_v, a, pl, tl, wwait)) fail();
    } else if (warp == 1) {
        // ------------------------------------------------------ issuer --
        // A: K (K-major) or V (MN-major), 128 rows; B: Q or P (K-major), 16 rows a term
        constexpr uint32_t idesc_s = kCodes ? ptx::idesc_e4m3_f32(128, 2 * kN) : ptx::idesc_bf16_f32(128, kN, false, false);
        constexpr uint32_t idesc_pv =
            kCodes ? ptx::idesc_e4m3_f32(128, 3 * kN) | (1u << 15) : ptx::idesc_bf16_f32(128, kN, true, false);
        constexpr uint32_t sbo = 1024u;
        int kn = 0, vn = 0, qn = 0, pieces = 0, items = 0;
        uint32_t p_par = 0;
        bool ok = true;
        for (int si = 0; ok; ++si) {
            Desc d;
            if (!get_desc(si, d)) {
                ok = false;
                break;
            }
            if (d.done) break;
            const int n = d.b1 - d.b0;
            if (n <= 0) continue;
            const int qs = qn & 1;
            ok = wwait(&sm.q_full[qs], (qn >> 1) & 1);
            ++qn;
            const uint32_t q_s = ptx::smem_u32(sm.q[qs]);
            // S of the piece's item i into the buffer (items + i) & 3; an
            // item's warpgroup is i & 1
            auto score = [&](int i) -> bool {
                const int b = (items + i) & 3, s = kn % S::kK;
                // the buffer's previous S has been read
                if (items + i >= 4 && !wwait(&sm.s_taken[b], (((items + i) >> 2) - 1) & 1)) return false;
                if (!wwait(&sm.k_full[s], (kn / S::kK) & 1)) return false;
                ptx::tc_fence_after();
                const uint32_t k_s = ptx::smem_u32(sm.k[s]), to = tmem + kColS + 32u * b;
                if constexpr (kCodes) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::umma_e4m3_ss_w(to, ptx::sdesc_sw128(k_s + 32u * kk, 16u, sbo),
                                            ptx::sdesc_sw128(q_s + 32u * kk, 16u, sbo), idesc_s, kk > 0);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::umma_f16_ss_w(to, ptx::kmajor_desc(k_s, kk),
                                           ptx::sdesc_sw128(q_s + (kk >> 2) * S::kQHalf + 32u * (kk & 3), 16u, sbo), idesc_s,
                                           kk > 0);
                }
                ptx::umma_commit_w(ptx::smem_u32(&sm.s_full[b]));
                ptx::umma_commit_w(ptx::smem_u32(&sm.k_empty[s]));
                if (i == n - 1) ptx::umma_commit_w(ptx::smem_u32(&sm.q_empty[qs]));
                ++kn;
                return true;
            };
            for (int i = 0; ok && i < 4 && i < n; ++i) ok = score(i);
            // O_0 and O_1 are free once the previous piece has been read out
            if (ok && pieces > 0) ok = wwait(&sm.o_free, (pieces - 1) & 1);
            ++pieces;
            for (int i = 0; ok && i < n; ++i) {
                const int w = i & 1, s = vn % S::kVLoads;
                ok = wwait(&sm.v_full[s], (vn / S::kVLoads) & 1) && wwait(&sm.p_full[w], (p_par >> w) & 1);
                p_par ^= 1u << w;
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t v_s = ptx::smem_u32(sm.v[s]), p_s = ptx::smem_u32(sm.p[w]);
                const uint32_t to = tmem + kColO + 64u * w;
                if constexpr (kCodes) {
                    // V^T: 128 features along a row, a k-step 32 keys = 4 KB on
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::umma_e4m3_ss_w(to, ptx::sdesc_sw128(v_s + 4096u * kk, kCodeTile, sbo),
                                            ptx::sdesc_sw128(p_s + 32u * kk, 16u, sbo), idesc_pv, i >= 2 || kk > 0);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        ptx::umma_f16_ss_w(to, ptx::mnmajor_desc(v_s, kk),
                                           ptx::sdesc_sw128(p_s + (kk >> 2) * (kN * 128u) + 32u * (kk & 3), 16u, sbo),
                                           idesc_pv, i >= 2 || kk > 0);
                }
                ptx::umma_commit_w(ptx::smem_u32(&sm.pv_done[w]));
                ptx::umma_commit_w(ptx::smem_u32(&sm.v_empty[s]));
                ++vn;
                if (i + 4 < n) ok = score(i + 4);
            }
            items += n;
        }
        if (!ok) {
            fail();
            // nothing may still run on the tensor cores when TMEM is released
            ptx::umma_commit_w(ptx::smem_u32(&sm.drain));
            ptx::mbar_wait_bounded(ptx::smem_u32(&sm.drain), 0, &no_abort, kWaitLimitNs);
        }
    } else if (warp == 2) {
        // -------------------------- what is hidden in V and not finite --
        if (!paged::clean_pieces<kCodes>(sm, a.mask, get_desc, wwait)) fail();
    } else if (warp == 3) {
        // ------------------------- V's loader; codes: Q in two terms --
        // (one warp for all loads would take 1560 cycles a block of codes: more
        // than the block's way from memory)
        ptx::tma_prefetch_desc(&tm_v);
        paged::Loader<kCodes, S> ld{sm, a, tm_q, tm_k, tm_v};
        int qn = 0;
        bool ok = true;
        for (int si = 0; ok; ++si) {
            Desc d;
            if (!get_desc(si, d)) {
                ok = false;
                break;
            }
            if (d.done) break;
            const int n = d.b1 - d.b0;
            if (n <= 0) continue;
            paged::Places at(a, d);
            auto split = [&]() -> bool {
                const int qs = qn & 1;
                if (!wwait(&sm.q_raw[qs], (qn >> 1) & 1)) return false;
                paged::split_q<S::kQHalf>(sm.q[qs], sm.row_scale[qn & 3], d.n * g.G, 0, 1, scale_log2);
                ptx::fence_proxy_async_smem();
                arrive1(&sm.q_full[qs]);
                ++qn;
                return true;
            };
            for (int j = 0; ok && j < n; ++j) {
                ok = ld.load_v(at, j, wwait);
                at.done(j);
                // (Q has landed by the time the first blocks are on their way)
                if (kCodes && ok && (j == 1 || j == n - 1 && j < 1)) ok = split();
            }
        }
        ld.drain();
        if (!ok) fail();
    } else if (warp >= 4) {
        // ------------------------------------------ softmax, epilogue --
        const int wg = (warp - 4) >> 2, ww = warp & 3;  // ww: TMEM lanes 32 ww ..
        const int at = 32 * ww + lane;                  // this thread's key of a block, feature of O^T
        const uint32_t lane_base = (uint32_t)(ww * 32) << 16;
        const uint32_t obuf = tmem + lane_base + kColO + 64u * wg;
        uint32_t e_uses = 0, w_uses = 0, pv_uses = 0;
        int blk = 0, qn = 0, items = 0;
        bool ok = true;
        auto meet = [&]() -> bool {  // all 8 softmax warps
            arrive1(&sm.ebar);
            return wwait(&sm.ebar, (e_uses++) & 1);
        };
        for (int si = 0; ok; ++si) {
            ok = wwait(&sm.d_full[si % kDescs], (si / kDescs) & 1);
            if (!ok) break;
            const Desc& d = sm.desc[si % kDescs];
            if (d.done) break;
            const int n = d.b1 - d.b0;
            const int rows = d.n * g.G;
            // lane r looks after row r: what it sees, its base
            paged::Sight see{1 << 30, 0, 0};
            if (lane < rows) see = paged::sight(a.mask, d.at0 + lane / g.G, d.total);
            float c = -INFINITY, ob = -INFINITY;
            float l[NR], row_mul[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                l[r] = 0.f;
                row_mul[r] = scale_log2;
            }
            for (int j = wg; j < n; j += 2) {
                const int b = (items + j) & 3;
                ok = wwait(&sm.s_full[b], ((items + j) >> 2) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t sbuf = tmem + lane_base + kColS + 32u * b;
                uint32_t y[16], y2[16];
                ptx::tmem_ld16(sbuf, y);
                if (kCodes) ptx::tmem_ld16(sbuf + kN, y2);
                if (kCodes && j == wg) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) row_mul[r] = sm.row_scale[qn & 3][r];
                }
                const int key0 = d.key0(j);
                const bool open = key0 + kKB <= see.end && (key0 >= see.lo || key0 + kKB <= see.sink);
                const bool masked = __any_sync(0xffffffffu, !open);
                float ks = 1.f, vs = 1.f, grow = 0.f, o_grow = 0.f;
                bool small = false;  // (warp-uniform) some scale is below what c can follow
                if constexpr (kCodes) {
                    ks = sm.ks(blk + j)[at];
                    vs = sm.vs(blk + j)[at];
                    // a weight's size against its score's: the terms' range, and the sum's
                    o_grow = fmaxf(__log2f(vs) - kTopBits, kLeastCode);
                    grow = fmaxf(o_grow, kLeastScale);
                    small = __any_sync(0xffffffffu, vs > 0.f && o_grow < kLeastScale);
                }
                ptx::tmem_wait_ld();
                ptx::reg_fence16(y);
                if (kCodes) ptx::reg_fence16(y2);
                ptx::tc_fence_before();
                arrive1(&sm.s_taken[b]);
                float x[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float s = __uint_as_float(y[r]);
                    if constexpr (kCodes) s = (s + __uint_as_float(y2[r])) * ks;
                    x[r] = s * row_mul[r];
                }
                if (masked) {
                    const int key = key0 + at;
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        paged::Sight t;
                        t.end = __shfl_sync(0xffffffffu, see.end, r);
                        t.lo = __shfl_sync(0xffffffffu, see.lo, r);
                        t.sink = __shfl_sync(0xffffffffu, see.sink, r);
                        if (!paged::sees(t, key)) x[r] = -INFINITY;
                    }
                }
                // the block's largest weight of each row
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float m = warp_max(kCodes ? x[r] + grow : x[r]);
                    if (lane == r) top = m;
                }
                float(&tops)[kWgWarps][kN] = sm.top[wg][(j >> 1) & 1];
                float(&o_tops)[kWgWarps][kN] = sm.o_top[kCodes ? wg : 0][(j >> 1) & 1];
                if (lane < NR) tops[ww][lane] = top;
                if constexpr (kCodes) {
                    if (lane == 0) sm.o_apart[wg][(j >> 1) & 1][ww] = small;
                    float o_top = top;
                    if (__builtin_expect(small, 0)) {
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            const float m = warp_max(x[r] + o_grow);
                            if (lane == r) o_top = m;
                        }
                    }
                    if (lane < NR) o_tops[ww][lane] = o_top;
                }
                arrive1(&sm.wbar[wg]);
                ok = wwait(&sm.wbar[wg], (w_uses++) & 1);
                if (!ok) break;
                constexpr float kLazy = kCodes ? kLazyCodes : kLazyBf16;
                const int mine = lane & (NR - 1);
                auto highest = [&](const float(&t)[kWgWarps][kN]) {
                    return ptx::max3(t[0][mine], t[1][mine], fmaxf(t[2][mine], t[3][mine]));
                };
                const float z = highest(tops);
                bool need = z > c + kLazy;
                const float fac = need ? ptx::ex2(c - z) : 1.f;  // of the sums
                c = need ? z : c;
                float o_fac = fac;                                // of O
                if constexpr (kCodes) {
                    float zo = z;
                    if (*reinterpret_cast<const uint32_t*>(sm.o_apart[wg][(j >> 1) & 1])) zo = highest(o_tops);
                    const bool o_need = zo > ob + kLazy;
                    o_fac = o_need ? ptx::ex2(ob - zo) : 1.f;
                    ob = o_need ? zo : ob;
                    need = need || o_need;
                }
                const bool rescale = __any_sync(0xffffffffu, need);
                const float base = c == -INFINITY ? 0.f : c;  // nothing seen yet: weights 2^-inf
                // P and O of the warpgroup's previous item are done with
                if (j > wg) {
                    ok = wwait(&sm.pv_done[wg], (pv_uses++) & 1);
                    if (!ok) break;
                }
                if (rescale) {
                    if (j > wg) {
                        ptx::tc_fence_after();
#pragma unroll
                        for (int t = 0; t < S::kTerms; ++t) {
                            uint32_t o[16];
                            ptx::tmem_ld16(obuf + 16u * t, o);
                            ptx::tmem_wait_ld();
                            ptx::reg_fence16(o);
#pragma unroll
                            for (int r = 0; r < NR; ++r)
                                o[r] = __float_as_uint(__uint_as_float(o[r]) * __shfl_sync(0xffffffffu, o_fac, r));
                            ptx::tmem_st16(obuf + 16u * t, o);
                        }
                        ptx::tmem_wait_st();
                    }
#pragma unroll
                    for (int r = 0; r < NR; ++r) l[r] *= __shfl_sync(0xffffffffu, fac, r);
                }
                // weights -> P^T, K-major rows of 128 keys
                uint8_t* pt = sm.p[wg];
                const uint32_t spot = kCodes ? (uint32_t)at : (uint32_t)((at >> 6) * (kN * 128) + (at & 63) * 2);
                // (always: a branch, which the compiler makes two loops of, costs 0.7 us of
                // instruction fetches in a short call)
                const float up = c != ob ? ptx::ex2(c - ob) : 1.f;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float p = ptx::ex2(x[r] - __shfl_sync(0xffffffffu, base, r));
                    l[r] += p;
                    uint8_t* to = pt + r * 128 + (spot ^ ((r & 7) << 4));
                    if constexpr (kCodes) {
                        float w = p * vs;
                        w *= __shfl_sync(0xffffffffu, up, r);
                        if (masked && x[r] == -INFINITY) w = 0.f;  // (a hidden value's scale may be anything)
#pragma unroll
                        for (int t = 0; t < 3; ++t) {
                            const uint32_t code = e4m3_of(w);
                            to[t * kN * 128] = (uint8_t)code;
                            w = (w - of_e4m3(code)) * 16.f;
                        }
                    } else {
                        *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16_rn(p);
                    }
                }
                ptx::tc_fence_before();
                ptx::fence_proxy_async_smem();
                arrive1(&sm.p_full[wg]);
            }
            if (!ok) break;
            blk += n;
            items += n;
            if (n > 0) ++qn;
            // ------------------------------------------------ epilogue --
            const bool has0 = n > 0, has1 = n > 1;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
                if (lane == 0) sm.red_l[warp - 4][r] = l[r];
            }
            if (ww == 0 && lane < NR) {
                sm.red_c[wg][lane] = c;
                sm.red_o[wg][lane] = kCodes ? ob : c;
            }
            // the last P V of each warpgroup (its own is waited for here, the
            // other's by the meeting)
            if (wg < n) {
                ok = wwait(&sm.pv_done[wg], (pv_uses++) & 1);
                if (!ok) break;
            }
            ptx::tc_fence_after();
            ptx::tc_fence_before();
            ok = meet();
            if (!ok) break;
            ptx::tc_fence_after();
            const bool cut = d.c0 != d.c1;
            const int slot = cut ? paged::partial_slot(sm.pl, blockIdx.x, d.base) : 0;
            float acc[NR / 2];
            // this warpgroup's half of the rows, feature `at`
            const int r0 = wg * (NR / 2);
            {
                uint32_t o[2][S::kTerms][16];
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int t = 0; t < S::kTerms; ++t)
                        ptx::tmem_ld16(tmem + lane_base + kColO + 64u * w + 16u * t, o[w][t]);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int t = 0; t < S::kTerms; ++t) ptx::reg_fence16(o[w][t]);
                auto pick = [&](int w, int r) -> float {  // O_w of row r0 + r
                    float x = 0.f;
#pragma unroll
                    for (int t = S::kTerms - 1; t >= 0; --t) {
                        const float y = __uint_as_float(wg == 0 ? o[w][t][r] : o[w][t][NR / 2 + r]);
                        x = t == S::kTerms - 1 ? y : fmaf(x, 1.f / 16.f, y);
                    }
                    return x;
                };
#pragma unroll
                for (int r = 0; r < NR / 2; ++r) {
                    const float c0 = sm.red_c[0][r0 + r], c1 = sm.red_c[1][r0 + r];
                    const float m = fmaxf(c0, c1);
                    const float o0 = sm.red_o[0][r0 + r], o1 = sm.red_o[1][r0 + r];
                    const float f0 = c0 == -INFINITY ? 1.f : ptx::ex2(o0 - m), f1 = c1 == -INFINITY ? 1.f : ptx::ex2(o1 - m);
                    acc[r] = (has0 ? f0 * pick(0, r) : 0.f) + (has1 ? f1 * pick(1, r) : 0.f);
                }
            }
            ptx::tc_fence_before();
            if (n > 0) arrive1(&sm.o_free);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
            auto out_at = [&](int r) -> size_t {  // row r of the tile
                const int token = r / g.G;
                return ((size_t)(d.row0 + token) * g.Hq + d.h * g.G + r - token * g.G) * kD;
            };
            float* part = a.work.o + (size_t)slot * kN * kD;
            if constexpr (!kCodes) {
                if (d.taken) {
                    float back[8];
                    give_rows_back(a, d, lane < rows ? see : paged::Sight{0, 0, 0}, r0, at, back);
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r) acc[r] += back[r];
                }
            }
#pragma unroll
            for (int r = 0; r < NR / 2; ++r) {
                const int row = r0 + r;
                if (row >= rows) continue;
                // (a row before the sequence sees nothing, whatever the values that all others see hold)
                if (d.at0 + row / g.G < 0) acc[r] = 0.f;
                const float c0 = sm.red_c[0][row], c1 = sm.red_c[1][row];
                const float m = fmaxf(c0, c1);
                const float f0 = c0 == -INFINITY ? 1.f : ptx::ex2(c0 - m), f1 = c1 == -INFINITY ? 1.f : ptx::ex2(c1 - m);
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int w = 0; w < kWgWarps; ++w) {
                    l0 += sm.red_l[w][row];
                    l1 += sm.red_l[kWgWarps + w][row];
                }
                const float lsum = f0 * l0 + f1 * l1;
                const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // nothing seen: zeros
                if (cut) {
                    part[row * kD + at] = acc[r];
                    if (at == 0) a.work.ml[(size_t)slot * kN + row] = make_float2(m, lsum);
                } else {
                    out[out_at(row) + at] = __float2bfloat16_rn(acc[r] * inv);
                }
            }
            if (cut) {
                // The last CTA to arrive merges the tile's partials, in order.
                __threadfence();
                ok = meet();
                if (!ok) break;
                if (threadIdx.x == 128) {
                    const int arrived = atomicAdd(a.work.arrived + d.c0, 1);
                    sm.last = arrived == d.c1 - d.c0;
                    if (sm.last) a.work.arrived[d.c0] = 0;
                    __threadfence();
                }
                ok = meet();
                if (!ok) break;
                if (sm.last) {
                    __threadfence();
                    // one pass over the pieces, all rows' loads in flight together
                    constexpr int R = NR / 2;
                    float mm[R], ll[R], oo[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        mm[r] = -INFINITY;
                        ll[r] = oo[r] = 0.f;
                    }
#pragma unroll 2
                    for (int i = d.c0; i <= d.c1; ++i) {
                        const size_t at_row = (size_t)paged::partial_slot(sm.pl, i, d.base) * kN + r0;
                        float2 ml[R];
                        float o[R];
#pragma unroll
                        for (int r = 0; r < R; ++r) {  // (rows past the tile's: of earlier use, not written out)
                            ml[r] = __ldcg(a.work.ml + at_row + r);
                            o[r] = __ldcg(a.work.o + (at_row + r) * kD + at);
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float m = fmaxf(mm[r], ml[r].x);
                            // (weights without a maximum are NaN or none)
                            const float w0 = mm[r] == -INFINITY ? 1.f : ptx::ex2(mm[r] - m);
                            const float w1 = ml[r].x == -INFINITY ? 1.f : ptx::ex2(ml[r].x - m);
                            ll[r] = ll[r] * w0 + ml[r].y * w1;
                            oo[r] = oo[r] * w0 + o[r] * w1;
                            mm[r] = m;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (r0 + r < rows)
                            out[out_at(r0 + r) + at] = __float2bfloat16_rn(oo[r] * (ll[r] == 0.f ? 0.f : 1.f / ll[r]));
                }
            } else {
                // (red_l and red_c have been read: the next piece may write them)
                ok = meet();
                if (!ok) break;
            }
            arrive1(&sm.d_empty[si % kDescs]);
        }
        if (!ok) fail();
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool kCodes, int NR>
bool ready() {
    static_assert(sizeof(Smem<kCodes>) <= 232448, "shared memory");
    if (cudaFuncSetAttribute(paged_few_kernel<kCodes, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Smem<kCodes>)) == cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}

template <bool kCodes, int NR>
cudaError_t launch(const PagedAttend& a, int max_ctas, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int page = 1 << a.g.page_log2, box = page < kKB ? page : kKB;
    const long long outer = (long long)a.g.pages * a.g.Hk;
    CUtensorMap q, k, v;
    if (!tma_encode_head_rows(&q, a.q, a.g.Hq, a.seqs.tokens, a.q_stride, a.g.G, NR / a.g.G) ||
        !tma_encode_pages(&k, a.pool.k, kCodes, page, outer, box) ||
        !tma_encode_pages(&v, a.pool.v, kCodes, page, outer, box))
        return cudaErrorInvalidValue;
    const int grid = max_ctas > 0 && max_ctas < sms ? max_ctas : sms;
    static_assert(2 * kN <= kPagedRowsPerSm, "workspace rows");
    return launch_pdl(paged_few_kernel<kCodes, NR>, grid, kThreads, sizeof(Smem<kCodes>), st, q, k, v, a,
                      a.scale * 1.4426950408889634f);
}

template <bool kCodes>
cudaError_t launch_rows(const PagedAttend& a, int rows, int max_ctas, cudaStream_t st) {
    if (rows <= 4) return launch<kCodes, 4>(a, max_ctas, st);
    if (rows <= 8) return launch<kCodes, 8>(a, max_ctas, st);
    return launch<kCodes, 16>(a, max_ctas, st);
}

}  // namespace

bool paged_few_init() {
    return tma_available() && ready<false, 4>() && ready<false, 8>() && ready<false, 16>() && ready<true, 4>() &&
           ready<true, 8>() && ready<true, 16>();
}

cudaError_t launch_paged_few(bool e4m3, const PagedAttend& a, int rows, int max_ctas, cudaStream_t st) {
    return e4m3 ? launch_rows<true>(a, rows, max_ctas, st) : launch_rows<false>(a, rows, max_ctas, st);
}

}  // namespace arl2
