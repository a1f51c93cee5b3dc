// Attention of a batch's new tokens over the paged cache on the tensor cores
// (tcgen05): bf16 queries and outputs, head width 128, pages of bf16 or of
// e4m3 codes with one scale per token and head.
//
// A tile is up to 256 query rows (new tokens x the G query heads of one key
// head), two halves of 128 rows = TMEM lanes, against blocks of 128 keys; the
// schedule of paged.cuh splits all tiles' blocks evenly over one CTA per SM.
// Softmax warpgroup w owns the S/P buffer w and the accumulator O_w:
//   a tile of two halves: half w against every block of keys;
//   a tile of one half (its rows fit 128): the half against every second
//   block, so both warpgroups and the tensor core stay busy; O_0 and O_1 are
//   combined at the end.
// In both, item i of a piece (i = 0, 1, ...) belongs to warpgroup i & 1, and
// the issue order is S_0, S_1, then P V_i followed by S_{i+2}: one
// warpgroup's softmax runs beside the other's products.
//
// Roles: warp 0 loads (TMA: Q tiles, and each block's pages, found through
// the page table, into the rings of K and V tiles), warp 1 issues the products,
// warp 2 holds the TMEM, warp 3 (bf16 pages) cleans V's blocks at the mask's
// edges, warps 4-11 are the two softmax warpgroups and write the outputs.
//
// Pages of codes.  S takes K's codes as they are, with Q as the sum of two e4m3
// terms: q 2^k = hi + lo, k per row so that the largest element lies in [2^7,
// 2^8).  An element's 8 bits fit the two terms' 4 + 4 exactly down to 2^-2; below,
// lo is a subnormal and off by at most 2^-10, 2^-17 of the row's largest
// element.  e4m3 products run at twice the rate of bf16 ones, so two terms cost
// what one bf16 product does, and K needs no conversion.  P has no such split
// (its small weights would need bf16's exponents): V's codes become bf16 tiles,
// exactly, in warps 2 and 3, which also split Q.  The keys' scales multiply their
// scores and the values' scales the weights, in fp32.
//
// Softmax statistics, sums and accumulators are fp32.  The weights are
// rounded to bf16, the type of the product with V; the sum they are divided
// by is of the unrounded ones.  The running maximum moves only when it grows
// by more than 2^8, which rescales O.
//
// Masked scores become -inf before the maximum: a weight of exactly 0.  What
// a masked V row holds still enters 0 x v: warp 3 takes what is not finite out of
// blocks that some query of the tile does not see all of (clean_block), and
// the queries that do see it get it back at the end (give_back).
//
// Bound by the softmax's chain per block (scores from TMEM, maximum, weights,
// half a P V, the next S: about 3400 cycles for two halves, of which the
// products take 2048).  With codes it is about 6200 cycles, tile starts and ends
// included, in which no unit is busy much more than half the time (issue slots 47
// %, tensor pipe 35 %, SFU 33 %; shared memory 1350 wavefronts of loads and
// stores and about 2050 of operands and copies): the chain of V's conversion in
// two warps, P V and the next S.  One 480p frame over 24 frames (12 heads): 415 to
// 455 us (355 to 400 in the first launches), 790 to 865 TFLOP/s, at 1.45 GHz
// under the power cap; five chunks of prompts (32 heads on 8): 272 to 300 us, 815
// to 900 TFLOP/s; two streams' frames over e4m3 pages: 360 to 370 us, 655 to 675.
#include "paged_tc.cuh"

#include <cmath>

namespace arl2 {
namespace {

using paged::Desc;
using paged::kCodeTile;
using paged::kD;
using paged::kDescs;
using paged::kHalfBytes;
using paged::kKB;
using paged::kSoftmaxWarps;
using paged::kTileBytes;
using paged::kWaitLimitNs;
using paged::kWgWarps;

constexpr int kRows = 128;  // rows of a half tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // S/P buffers at 0, 128; O_0, O_1 at 256, 384
constexpr float kRescaleLog2 = 8.0f;
constexpr int kThreads = 384;
constexpr int kConvWarps = 2;
// Registers per thread at launch (one CTA per SM) and after the split: warps
// 0-3 hand theirs to the two softmax warpgroups.
constexpr int kRegsLaunch = 168, kRegsLow = 96, kRegsHigh = 200;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * kRegsLaunch, "register split");
// For the schedule, in quarters of a block of two halves: the cost of a block,
// of a tile on top of its blocks, up to what a tile is not cut, and how much a
// CTA has at least.  (With no cost for a tile prompts take 314 us, not 281, a
// frame over 24 frames 424, not 437; with the same cost for a half and a quarter
// of a half as for two halves, two streams' frames over codes 392, not 363.)
constexpr int kPairCost = 4, kSingleCost = 3, kSmallCost = 2, kTileCost = 6, kWhole = 16, kMinUnits = 8;
static_assert(kMinUnits > kTileCost, "one border at most in what a tile costs for itself");

template <bool kCodes>
struct Cfg {
    static constexpr int kK = kCodes ? 3 : 2;       // K tiles in their ring
    static constexpr int kKBytes = kCodes ? kCodeTile : (int)kTileBytes;
    static constexpr int kV = 2;                    // V tiles (bf16) in theirs
    static constexpr int kStaged = 2;               // blocks of V's codes on their way
};

template <bool kCodes>
struct __align__(1024) Smem {
    using C = Cfg<kCodes>;
    uint8_t q[2][kTileBytes];
    uint8_t k[C::kK][C::kKBytes];
    uint8_t v[C::kV][kTileBytes];
    uint8_t st[kCodes ? C::kStaged : 1][kCodes ? kCodeTile : 16];
    // scratch of the plan, then (codes) the blocks' key and value scales: K of
    // block j is loaded when S of block j - 3 is done, and with two warpgroups
    // on alternate blocks the one before may still be in use
    static constexpr int kScaleSlots = 5;
    __align__(16) int scratch[kCodes ? kScaleSlots * 2 * kKB : kPagedMaxSeqs + 4];
    static_assert(kScaleSlots * 2 * kKB > kPagedMaxSeqs, "scratch");
    __device__ float* ks(int blk) { return reinterpret_cast<float*>(scratch) + blk % kScaleSlots * 2 * kKB; }
    __device__ float* vs(int blk) { return ks(blk) + kKB; }
    float ones[kCodes ? kKB : 4];
    float row_scale[kCodes ? 4 : 1][kRows];  // 2^-k of Q's rows times the softmax scale (log2 units)
    uint64_t d_full[kDescs], d_empty[kDescs];
    uint64_t q_raw[2], q_full[2], q_empty[2];  // (q_raw: before the split in two terms)
    uint64_t k_full[3], k_empty[3];
    uint64_t v_full[2], v_empty[2];
    uint64_t st_full[2], st_empty[2];
    // (for the loading warp)
    static constexpr int kK = C::kK, kKBytes = C::kKBytes, kVLoads = 2;
    static constexpr uint32_t kQHalf = kHalfBytes;
    static constexpr bool kClean = !kCodes;  // (a code, NaN's too, becomes a finite bf16)
    __device__ uint64_t* q_landed(int s) { return kCodes ? &q_raw[s] : &q_full[s]; }
    __device__ uint64_t* v_landed(int s) { return kCodes ? &st_full[s] : &v_full[s]; }
    __device__ uint64_t* v_taken(int s) { return kCodes ? &st_empty[s] : &v_empty[s]; }
    __device__ uint8_t* v_load(int s) { return kCodes ? st[s] : v[s]; }
    uint64_t v_edge[kVLoads];    // a block of V that some query does not see all of has landed, not cleaned yet
    uint64_t s_full[2];          // S of warpgroup w's item is in TMEM
    uint64_t p_half[2], p_full[2];  // 4 warp arrivals: P of the last / first 64 keys written
    uint64_t pv_half[2];         // an item's first half of P V is in O_w
    uint64_t pv_done[2];         // the piece's last P V of warpgroup w
    uint64_t o_free;             // 8 warp arrivals per piece: O_0, O_1 read out
    uint64_t ebar;               // 8 warp arrivals: the softmax warps meet
    uint64_t drain;
    float red_m[2][kRows], red_l[2][kRows];  // [warpgroup][row]
    Desc desc[kDescs];
    uint32_t tmem_base;
    int abort;
    int last;
    paged::Plan pl;
    paged::PlanSmem plan;
};

// A block of codes -> the two 128-byte-swizzled halves of a bf16 tile.  A code
// s eeee mmm becomes the bf16 s 0000eeee mmm0000, its value times 2^-120
// (subnormal codes are subnormal there too), and the product with 2^120 is
// exact.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    const uint32_t x = ((a >> 4) & 0x07f007f0u) | (a & 0x80008000u);
    const uint32_t y = ((b >> 4) & 0x07f007f0u) | (b & 0x80008000u);
    constexpr uint32_t k2p120 = 0x7b807b80u;  // 2^120 twice
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(k2p120));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(k2p120));
}

// A staged block of V's codes -> a bf16 tile; warp ww of two does rows 64 ww ..
__device__ __forceinline__ void convert_v(const uint8_t* st, uint32_t v, int ww) {
    const int lane = threadIdx.x & 31;
    // lanes of a quarter warp take eight rows: loads and stores
    // of the swizzled tiles then touch every bank once
    const int r7 = lane & 7, c = lane >> 3;
    const uint8_t* from = st + (ww * 64 + r7) * 128 + ((c ^ r7) << 4);
    const uint32_t to = v + (uint32_t)((ww * 64 + r7) * 128 + (((2 * c) ^ r7) << 4));
    const uint32_t to2 = to ^ 16u;
    const uint8_t* from2 = st + (ww * 64 + r7) * 128 + (((c + 4) ^ r7) << 4);
    // (two at a time: the products' operands come first at the shared memory;
    // four at a time 380 us, eight 423, one 367, two 356, at two streams' frames)
#pragma unroll 1
    for (int i0 = 0; i0 < 16; i0 += 2) {
        uint4 u[2];  // 16 codes each: features 64 half + 16 c ..., of rows 8 apart
#pragma unroll
        for (int i = 0; i < 2; ++i)
            u[i] = *reinterpret_cast<const uint4*>((i & 1 ? from2 : from) + ((i0 + i) >> 1) * 1024);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t y[8];
            codes_to_bf16(u[i].x, y[0], y[1]);
            codes_to_bf16(u[i].y, y[2], y[3]);
            codes_to_bf16(u[i].z, y[4], y[5]);
            codes_to_bf16(u[i].w, y[6], y[7]);
            const uint32_t at = (i & 1) * kHalfBytes + ((i0 + i) >> 1) * 1024;
            ptx::st_shared_v4(to + at, y[0], y[1], y[2], y[3]);
            ptx::st_shared_v4(to2 + at, y[4], y[5], y[6], y[7]);
        }
    }
    ptx::fence_proxy_async_smem();
}

// Row `row` of warpgroup wg's half tile: token of the tile and query head.
struct RowOf {
    int token, head;
    bool valid;
};
__device__ __forceinline__ RowOf row_of(const Desc& d, int row, int wg, int G, int HT) {
    const int i = row / G;
    RowOf r;
    r.token = (d.pair ? wg * HT : 0) + i;
    r.head = d.h * G + row - i * G;
    r.valid = i < HT && r.token < d.n;
    return r;
}

// The softmax warp's rows (one a thread) of the piece in a slot of sm.desc that
// had values taken out, after their outputs or partials were written: first
// which features hold such values at all, then their sums over the keys that
// the row sees.  (All of it worked out again, and few registers: what the main
// loop keeps for it, or moves out of its way, costs prompts 250 -> 288 us.)
static __device__ __noinline__ void give_rows_back(const PagedAttend& a, Smem<false>& sm, int desc) {
    const Desc& d = sm.desc[desc];
    const int lane = threadIdx.x & 31, wg = (threadIdx.x >> 7) - 1, row = threadIdx.x & 127;
    const bool pair = d.pair != 0, cut = d.c0 != d.c1;
    const RowOf r = row_of(d, row, wg, a.g.G, kRows / a.g.G);
    const paged::Seen seen = paged::seen_by(a.mask, d);
    paged::Sight mine{0, 0, 0};
    if (r.valid) mine = paged::sight(a.mask, d.at0 + r.token, d.total);
    uint32_t hit = 0u;
    paged::for_edge_keys(a, d, seen, [&](const __nv_bfloat16* v, int) {
#pragma unroll 8
        for (int u = 0; u < paged::kEdgeKeys; ++u) {
            const uint2 w = *reinterpret_cast<const uint2*>(v + u * kD + 4 * lane);
            hit |= paged::not_finite_bf16(w.x) | paged::not_finite_bf16(w.y);
        }
    });
    uint32_t quads = __ballot_sync(0xffffffffu, hit != 0u);  // of four features
    if (!pair) quads &= wg ? 0xffff0000u : 0x0000ffffu;       // (a tile of one half: this warpgroup's columns)
    for (; quads; quads &= quads - 1) {
        const int quad = __ffs(quads) - 1;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        paged::for_edge_keys(a, d, seen, [&](const __nv_bfloat16* v, int j) {
#pragma unroll 8
            for (int u = 0; u < paged::kEdgeKeys; ++u) {
                const uint2 w = *reinterpret_cast<const uint2*>(v + u * kD + 4 * quad);
                const uint32_t x = paged::not_finite_bf16(w.x), y = paged::not_finite_bf16(w.y);
                if ((x | y) && paged::sees(mine, j + u) && !paged::sees(seen.all, j + u)) {
                    if (x & 0x8000u) sum[0] += __uint_as_float(w.x << 16);
                    if (x >> 16) sum[1] += __uint_as_float(w.x & 0xffff0000u);
                    if (y & 0x8000u) sum[2] += __uint_as_float(w.y << 16);
                    if (y >> 16) sum[3] += __uint_as_float(w.y & 0xffff0000u);
                }
            }
        });
        if (sum[0] == 0.f && sum[1] == 0.f && sum[2] == 0.f && sum[3] == 0.f) continue;
        if (cut) {
            const size_t slot = (size_t)paged::partial_slot(sm.pl, blockIdx.x, d.base) * 2 + (pair ? wg : 0);
            float4& o = reinterpret_cast<float4*>(a.work.o)[(slot * 32 + quad) * kRows + row];
            o = make_float4(o.x + sum[0], o.y + sum[1], o.z + sum[2], o.w + sum[3]);
        } else {
            __nv_bfloat16* o =
                static_cast<__nv_bfloat16*>(a.out) + ((size_t)(d.row0 + r.token) * a.g.Hq + r.head) * kD + 4 * quad;
            for (int c = 0; c < 4; ++c) o[c] = __float2bfloat16_rn(__bfloat162float(o[c]) + sum[c]);
        }
    }
}

template <bool kCodes>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttend a,
                    float scale_log2) {
    using C = Cfg<kCodes>;
    // (the swizzled tiles need 1024-byte boundaries; there is no room to align by hand)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<kCodes>& sm = *reinterpret_cast<Smem<kCodes>*>(smem_raw);
    if (ptx::smem_u32(smem_raw) & 1023u) {
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
            init(&sm.d_empty[i], 1 + kSoftmaxWarps + (kCodes ? kConvWarps : 1));
        }
        for (int i = 0; i < 3; ++i) {
            init(&sm.k_full[i], paged::kKArrivals<kCodes>);
            init(&sm.k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            init(&sm.v_full[i], kCodes ? kConvWarps : 1);
            init(&sm.v_empty[i], 1);
            init(&sm.v_edge[i], 1);
            init(&sm.st_full[i], 1);
            init(&sm.st_empty[i], kConvWarps);
            init(&sm.q_raw[i], 1);
            init(&sm.q_full[i], kCodes ? kConvWarps : 1);
            init(&sm.q_empty[i], 1);
            init(&sm.s_full[i], 1);
            init(&sm.p_half[i], kWgWarps);
            init(&sm.p_full[i], kWgWarps);
            init(&sm.pv_half[i], 1);
            init(&sm.pv_done[i], 1);
        }
        init(&sm.o_free, kSoftmaxWarps);
        init(&sm.ebar, kSoftmaxWarps);
        init(&sm.drain, 1);
        sm.abort = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (kCodes && threadIdx.x < kKB) sm.ones[threadIdx.x] = 1.f;
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_u32(&sm.tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::pdl_wait_then_trigger();  // (nothing before this touches global memory)
    const int HT = kRows / g.G;  // tokens of a half tile
    const paged::Tiling tl{2 * HT, HT, kPairCost, kSingleCost, kSmallCost, kTileCost, kWhole};
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
    // bounded wait with a warp-uniform result (every role runs as whole warps)
    auto wwait = [&](uint64_t* bar, uint32_t parity) {
        return ptx::mbar_wait_warp(ptx::smem_u32(bar), parity, abort, kWaitLimitNs);
    };
    auto arrive1 = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(bar));
    };
    // piece si's descriptor, copied; its slot is free again once all have
    auto get_desc = [&](int si, Desc& d) -> bool {
        if (!wwait(&sm.d_full[si % kDescs], (si / kDescs) & 1)) return false;
        d = sm.desc[si % kDescs];
        arrive1(&sm.d_empty[si % kDescs]);
        return true;
    };

    if (warp < 4) ptx::setmaxnreg_dec<kRegsLow>();
    if (warp == 0) {
        // ------------------------------------------------------ loader --
        if (!paged::load_pieces<kCodes, true>(sm, tm_q, tm_k, tm_v, a, pl, tl, wwait)) fail();
    } else if (warp == 1) {
        // ------------------------------------------------------ issuer --
        const uint32_t idesc_s = kCodes ? ptx::idesc_e4m3_f32(kRows, kKB) : ptx::idesc_bf16_f32(kRows, kKB, false, false);
        const uint32_t idesc_pv = ptx::idesc_bf16_f32(kRows, kD, false, true);  // V: MN-major
        int kn = 0, vn = 0, qn = 0, pieces = 0;
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
            const bool pair = d.pair != 0;
            const int N = pair ? 2 * n : n;
            const int q0 = qn, nq = pair ? 2 : 1;
            for (int t = 0; ok && t < nq; ++t, ++qn) ok = wwait(&sm.q_full[qn & 1], (qn >> 1) & 1);
            int ks = 0, vs = 0;       // ring stages of the K and V tile in use
            const bool keep = pair;   // a tile serves two items
            auto s_ready = [&](int i) -> bool {
                if (keep && (i & 1)) return true;
                ks = kn % C::kK;
                return wwait(&sm.k_full[ks], (kn++ / C::kK) & 1);
            };
            auto s_issue = [&](int i) {
                ptx::tc_fence_after();
                const uint32_t q_s = ptx::smem_u32(sm.q[(q0 + (pair ? i & 1 : 0)) & 1]);
                const uint32_t k_s = ptx::smem_u32(sm.k[ks]);
                const uint32_t s_t = tmem + kColS + (uint32_t)(i & 1) * kKB;
                if constexpr (kCodes)
                    ptx::umma_e4m3_two_terms(s_t, ptx::kmajor_desc(q_s, 0), ptx::kmajor_desc(k_s, 0), idesc_s);
                else
                    ptx::umma_ss8_kk(s_t, ptx::kmajor_desc(q_s, 0), ptx::kmajor_desc(k_s, 0), idesc_s, 0u);
                ptx::umma_commit_w(ptx::smem_u32(&sm.s_full[i & 1]));
                if (!keep || (i & 1)) ptx::umma_commit_w(ptx::smem_u32(&sm.k_empty[ks]));
                if (i == N - 1)
                    for (int t = 0; t < nq; ++t) ptx::umma_commit_w(ptx::smem_u32(&sm.q_empty[(q0 + t) & 1]));
            };
            for (int i = 0; ok && i < 2 && i < N; ++i) {
                ok = s_ready(i);
                if (ok) s_issue(i);
            }
            // O_0 and O_1 are free once the previous piece has been read out
            if (ok && pieces > 0) ok = wwait(&sm.o_free, (pieces - 1) & 1);
            ++pieces;
            for (int i = 0; ok && i < N; ++i) {
                const int w = i & 1;
                const uint32_t par = (p_par >> w) & 1;
                p_par ^= 1u << w;
                if (!keep || w == 0) {
                    vs = vn & 1;
                    ok = wwait(&sm.v_full[vs], (vn++ >> 1) & 1);
                }
                ok = ok && wwait(&sm.p_half[w], par);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t p_t = tmem + kColS + (uint32_t)w * kKB + 64u;
                const uint32_t o_t = tmem + kColO + (uint32_t)w * kD;
                const uint32_t v_s = ptx::smem_u32(sm.v[vs]);
                // O_w += P V in two halves of 64 keys, the last 64 first: they
                // run while the softmax warps work on the other half's P
                ptx::umma_ts4_mn(o_t, p_t + 32u, ptx::mnmajor_desc(v_s, 4), idesc_pv, i >= 2 ? 1u : 0u);
                ptx::umma_commit_w(ptx::smem_u32(&sm.pv_half[w]));
                const bool next = i + 2 < N;
                ok = (!next || s_ready(i + 2)) && wwait(&sm.p_full[w], par);
                if (!ok) break;
                ptx::tc_fence_after();
                ptx::umma_ts4_mn(o_t, p_t, ptx::mnmajor_desc(v_s, 0), idesc_pv, 1u);
                if (!keep || w == 1) ptx::umma_commit_w(ptx::smem_u32(&sm.v_empty[vs]));
                if (next)
                    s_issue(i + 2);
                else
                    ptx::umma_commit_w(ptx::smem_u32(&sm.pv_done[w]));
            }
        }
        if (!ok) {
            fail();
            // nothing may still run on the tensor cores when TMEM is released
            ptx::umma_commit_w(ptx::smem_u32(&sm.drain));
            ptx::mbar_wait_bounded(ptx::smem_u32(&sm.drain), 0, &no_abort, kWaitLimitNs);
        }
    } else if (!kCodes && warp == 3) {
        // -------------------------- what is hidden in V and not finite --
        if constexpr (!kCodes)
            if (!paged::clean_pieces<false>(sm, a.mask, get_desc, wwait)) fail();
    } else if (kCodes && warp < 4) {
        // ----------------- Q in two terms, V's codes -> bf16 tiles --
        if constexpr (kCodes) {
            const int cw = warp - 2;
            int vn = 0;
            int qn = 0;
            bool ok = true;
            for (int si = 0; ok; ++si) {
                Desc d;
                if (!get_desc(si, d)) {
                    ok = false;
                    break;
                }
                if (d.done) break;
                if (d.b1 <= d.b0) continue;
                for (int t = 0; ok && t < (d.pair ? 2 : 1); ++t, ++qn) {
                    const int qs = qn & 1;
                    ok = wwait(&sm.q_raw[qs], (qn >> 1) & 1);
                    if (!ok) break;
                    const int tokens = d.n - t * HT < HT ? d.n - t * HT : HT;
                    paged::split_q<kHalfBytes>(sm.q[qs], sm.row_scale[qn & 3], tokens * g.G, cw, kConvWarps, scale_log2);
                    ptx::fence_proxy_async_smem();
                    arrive1(&sm.q_full[qs]);
                }
                for (int j = d.b0; ok && j < d.b1; ++j, ++vn) {
                    const int s = vn & 1;
                    ok = wwait(&sm.st_full[s], (vn >> 1) & 1) && (vn < 2 || wwait(&sm.v_empty[s], ((vn >> 1) - 1) & 1));
                    if (!ok) break;
                    convert_v(sm.st[s], ptx::smem_u32(sm.v[s]), cw);
                    arrive1(&sm.v_full[s]);
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.st_empty[s]));
                }
            }
            if (!ok) fail();
        }
    } else if (warp >= 4) {
        // ------------------------------------------ softmax, epilogue --
        ptx::setmaxnreg_inc<kRegsHigh>();
        const int wg = (warp - 4) >> 2;                // S/P buffer and accumulator
        const int row = ((warp & 3) << 5) + lane;      // row of the half tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sbuf = tmem + lane_base + kColS + (uint32_t)wg * kKB;
        const uint32_t obuf = tmem + lane_base + kColO + (uint32_t)wg * kD;
        uint32_t s_par = 0, e_uses = 0, pv_par = 0;
        int blk = 0, it = 0;  // blocks, items of this warpgroup so far
        bool ok = true;
        // all 8 softmax warps meet (arrive, then a bounded wait)
        auto meet = [&]() -> bool {
            arrive1(&sm.ebar);
            return wwait(&sm.ebar, (e_uses++) & 1);
        };
        int qn = 0;
        for (int si = 0; ok; ++si) {
            // (read where it is, and given back at the piece's end: registers are short)
            ok = wwait(&sm.d_full[si % kDescs], (si / kDescs) & 1);
            if (!ok) break;
            const Desc& d = sm.desc[si % kDescs];
            if (d.done) break;
            const int n = d.b1 - d.b0;
            const bool pair = d.pair != 0;
            // what this thread's row sees (a row of no query: whatever there is)
            paged::Sight see{1 << 30, 0, 0};
            bool busy;  // else nobody reads this warp's rows
            {
                const RowOf r = row_of(d, row, wg, g.G, HT);
                if (r.valid) see = paged::sight(a.mask, d.at0 + r.token, d.total);
                busy = __any_sync(0xffffffffu, r.valid);
            }
            float m_run = -INFINITY, l_run = 0.f;
            const float row_mul = scale_log2;  // scores -> log2 units
            // Codes: a thread has four rows (lane / 4 + 8 r of the warp's 32) and a
            // quarter of the columns, so that it needs a quarter of the scales: as
            // one row a thread, their broadcast loads and the products' operands
            // wait for each other at the shared memory.
            float qm[4], ql[4], qmul[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                qm[r] = -INFINITY;
                ql[r] = 0.f;
                qmul[r] = 0.f;
            }
            const int step = pair ? 1 : 2, j0 = pair ? 0 : wg;
            for (int j = j0; j < n; j += step) {
                ok = wwait(&sm.s_full[wg], s_par);
                s_par ^= 1u;
                if (!ok) break;
                if (!busy) {
                    arrive1(&sm.p_half[wg]);
                    arrive1(&sm.p_full[wg]);
                    ++it;
                    continue;
                }
                ptx::tc_fence_after();
                const int key0 = d.key0(j);
                const float* kscale = sm.ks(blk + j);
                const float* vscale = kscale + kKB;
                if (kCodes && j == j0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        qmul[r] = sm.row_scale[(qn + (pair ? wg : 0)) & 3][(warp & 3) * 32 + (lane >> 2) + 8 * r];
                }
                // nothing of the block is hidden from this row
                const bool open = key0 + kKB <= see.end && (key0 >= see.lo || key0 + kKB <= see.sink);
                const bool masked = __any_sync(0xffffffffu, !open);
                if (masked) {
                    // hidden scores become -inf where they are: a pass of its
                    // own, for the few blocks at the mask's edges, costs the
                    // other blocks no registers
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t y[32];
                        ptx::tmem_ld32(sbuf + (uint32_t)c * 32, y);
                        const int k = key0 + 32 * c;
                        const uint32_t seen = paged::bits_below(see.end - k) & (~paged::bits_below(see.lo - k) | paged::bits_below(see.sink - k));
                        ptx::tmem_wait_ld();
                        ptx::reg_fence(y);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            // (after the key's scale, which may be anything where the key is hidden;
                            // a value's scale that is not finite makes the score NaN, and with it the row)
                            if constexpr (kCodes)
                                y[i] = __float_as_uint(fmaf(vscale[32 * c + i], 0.f, __uint_as_float(y[i]) * kscale[32 * c + i]));
                            y[i] = (seen >> i) & 1u ? y[i] : 0xff800000u;
                        }
                        ptx::tmem_st32(sbuf + (uint32_t)c * 32, y);
                    }
                    ptx::tmem_wait_st();
                }
                if (kCodes && masked) kscale = sm.ones;  // (they are scaled already)
                auto top = [](const uint32_t(&y)[32]) {  // 3-input max tree
                    float m8[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        auto f = [&](int k) { return __uint_as_float(y[8 * i + k]); };
                        m8[i] = ptx::max3(ptx::max3(f(0), f(1), f(2)), ptx::max3(f(3), f(4), f(5)), fmaxf(f(6), f(7)));
                    }
                    return ptx::max3(m8[0], m8[1], fmaxf(m8[2], m8[3]));
                };
                // The weights' base: the running maximum, which moves only when
                // a half block's scores pass it by more than 2^8.  A warp that
                // has such a row rescales O_w and the sums.
                auto rescale_o = [&](float corr) {
#pragma unroll 1
                    for (int b = 0; b < 8; ++b) {
                        uint32_t o[16];
                        ptx::tmem_ld16(obuf + (uint32_t)b * 16, o);
                        ptx::tmem_wait_ld();
                        ptx::reg_fence16(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                        ptx::tmem_st16(obuf + (uint32_t)b * 16, o);
                    }
                };
                // P is handed to the issuer in two halves of 64 keys, the last 64
                // first, each half's maximum taken just before its weights: the
                // first products start early (a frame over 24 frames: 422 us,
                // against 437 with the maximum of all first).
                if constexpr (kCodes) {
                    const int q2 = 2 * (lane & 3);
                    auto half_block = [&](int h, bool has_o) -> bool {  // keys 64 h ..
                        uint32_t y[2][32];  // lanes 0-15 (rows r = 0, 1), 16-31 (rows 2, 3)
                        ptx::tmem_ld_quads(sbuf + 64u * h, y[0]);
                        ptx::tmem_ld_quads(sbuf + (16u << 16) + 64u * h, y[1]);
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        ptx::tmem_wait_ld();
                        ptx::reg_fence(y[0]);
                        ptx::reg_fence(y[1]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 k2 = *reinterpret_cast<const float2*>(kscale + 64 * h + 8 * i + q2);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                uint32_t &a0 = y[r >> 1][4 * i + 2 * (r & 1)], &a1 = y[r >> 1][4 * i + 2 * (r & 1) + 1];
                                const float2 x = ptx::mul2(make_float2(__uint_as_float(a0), __uint_as_float(a1)), k2);
                                a0 = __float_as_uint(x.x), a1 = __float_as_uint(x.y);
                                mx[r] = ptx::max3(mx[r], x.x, x.y);
                            }
                        }
                        bool need = false;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2)) * qmul[r];
                            need = need || mx[r] > qm[r] + kRescaleLog2;
                        }
                        if (__any_sync(0xffffffffu, need)) {
                            float mine = 1.f;  // of the row of O_w that is this lane's
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const bool moves = mx[r] > qm[r] + kRescaleLog2;
                                const float corr = moves ? ptx::ex2(qm[r] - mx[r]) : 1.f;
                                qm[r] = moves ? mx[r] : qm[r];
                                ql[r] *= corr;
                                const float c = __shfl_sync(0xffffffffu, corr, (lane & 7) * 4);
                                mine = (lane >> 3) == r ? c : mine;
                            }
                            if (has_o) {
                                if (h == 0) {  // the other half's P V must be in O_w
                                    if (!wwait(&sm.pv_half[wg], it & 1)) return false;
                                    ptx::tc_fence_after();
                                }
                                rescale_o(mine);
                            }
                        }
                        uint32_t pk[2][16];
                        float2 qs[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 v2 = *reinterpret_cast<const float2*>(vscale + 64 * h + 8 * i + q2);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float base = qm[r] == -INFINITY ? 0.f : qm[r];  // nothing seen yet: weights 2^-inf
                                const float2 x = make_float2(__uint_as_float(y[r >> 1][4 * i + 2 * (r & 1)]),
                                                             __uint_as_float(y[r >> 1][4 * i + 2 * (r & 1) + 1]));
                                const float2 e = ptx::fma2(x, make_float2(qmul[r], qmul[r]), make_float2(-base, -base));
                                const float2 p = make_float2(ptx::ex2(e.x), ptx::ex2(e.y));
                                qs[r] = ptx::add2(qs[r], p);
                                float2 w = ptx::mul2(p, v2);
                                if (masked) {  // (a hidden value's scale may be anything)
                                    w.x = p.x == 0.f ? 0.f : w.x;
                                    w.y = p.y == 0.f ? 0.f : w.y;
                                }
                                pk[r >> 1][2 * i + (r & 1)] = ptx::pack_bf16x2(w.x, w.y);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) ql[r] += qs[r].x + qs[r].y;
                        // (behind the scores that are still to be read)
                        ptx::tmem_st_quads(sbuf + 64u + 32u * h, pk[0]);
                        ptx::tmem_st_quads(sbuf + (16u << 16) + 64u + 32u * h, pk[1]);
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                        return true;
                    };
                    ok = half_block(1, j > j0);
                    arrive1(&sm.p_half[wg]);
                    ok = ok && half_block(0, true);
                    if (!ok) break;
                    arrive1(&sm.p_full[wg]);
                    ++it;
                    continue;
                }
                float2 nm;
                auto set_base = [&]() {
                    const float base = m_run == -INFINITY ? 0.f : m_run;  // nothing seen yet: weights 2^-inf
                    nm = make_float2(-base, -base);
                };
                auto over = [&](float mx) { return __any_sync(0xffffffffu, mx > m_run + kRescaleLog2); };
                auto move_base = [&](float mx, bool has_o) {
                    const bool need = mx > m_run + kRescaleLog2;
                    const float corr = need ? ptx::ex2(m_run - mx) : 1.f;
                    l_run *= corr;
                    m_run = need ? mx : m_run;
                    if (has_o) rescale_o(corr);
                };
                // columns 32 c ... -> P, bf16 pairs in columns 64 + 16 c ... of the
                // buffer (behind the scores that are still to be loaded again)
                auto weigh = [&](const uint32_t(&y)[32], int c) {
                    uint32_t pk[16];
                    float2 sum4[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 xi = make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
                        const float2 e = ptx::fma2(xi, make_float2(row_mul, row_mul), nm);
                        float2 p;
                        p.x = ptx::ex2(e.x);
                        p.y = ptx::ex2(e.y);
                        sum4[i & 3] = ptx::add2(sum4[i & 3], p);
                        pk[i] = ptx::pack_bf16x2(p.x, p.y);
                    }
                    ptx::tmem_st16(sbuf + 64u + 16u * c, pk);
                    const float2 s2 = ptx::add2(ptx::add2(sum4[0], sum4[1]), ptx::add2(sum4[2], sum4[3]));
                    l_run += s2.x + s2.y;
                };
                uint32_t ya[32], yb[32];
                ptx::tmem_ld32(sbuf + 64, ya);
                ptx::tmem_ld32(sbuf + 96, yb);
                ptx::tmem_wait_ld();
                ptx::reg_fence(ya);
                ptx::reg_fence(yb);
                float mx = fmaxf(top(ya), top(yb)) * row_mul;
                // (S of this item was committed after the P V of the previous one: O_w is still)
                if (over(mx)) move_base(mx, j > j0);
                set_base();
                weigh(ya, 2);
                ptx::tmem_ld32(sbuf, ya);
                weigh(yb, 3);
                ptx::tmem_ld32(sbuf + 32, yb);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                arrive1(&sm.p_half[wg]);
                ptx::tmem_wait_ld();
                ptx::reg_fence(ya);
                ptx::reg_fence(yb);
                mx = fmaxf(top(ya), top(yb)) * row_mul;
                if (over(mx)) {
                    ok = wwait(&sm.pv_half[wg], it & 1);  // the first half's P V is in O_w
                    if (!ok) break;
                    ptx::tc_fence_after();
                    move_base(mx, true);
                    set_base();
                }
                weigh(ya, 0);
                weigh(yb, 1);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                arrive1(&sm.p_full[wg]);
                ++it;
            }
            if (!ok) break;
            blk += n;
            if (n > 0) qn += pair ? 2 : 1;
            // ------------------------------------------------ epilogue --
            // (the row's place again, from a number the compiler cannot see
            // through: kept over the loop it would cost its registers)
            int row_again = row;
            asm volatile("" : "+r"(row_again));
            const RowOf r = row_of(d, row_again, wg, g.G, HT);
            const int token = r.token, head = r.head;
            const bool valid = r.valid;
            const bool has[2] = {n > 0, pair ? n > 0 : n > 1};
            if constexpr (kCodes) {  // to one row a lane
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ql[r] += __shfl_xor_sync(0xffffffffu, ql[r], 1);
                    ql[r] += __shfl_xor_sync(0xffffffffu, ql[r], 2);
                    const float mr = __shfl_sync(0xffffffffu, qm[r], (lane & 7) * 4);
                    const float lr = __shfl_sync(0xffffffffu, ql[r], (lane & 7) * 4);
                    m_run = (lane >> 3) == r ? mr : m_run;
                    l_run = (lane >> 3) == r ? lr : l_run;
                }
            }
            // the row's statistics over the piece, and what O_0 and O_1 count
            float m = m_run, l = l_run, f0 = 1.f, f1 = 1.f;
            if (!pair) {
                sm.red_m[wg][row] = m_run;
                sm.red_l[wg][row] = l_run;
                ok = meet();
                if (!ok) break;
                const float m0 = sm.red_m[0][row], m1 = sm.red_m[1][row];
                m = fmaxf(m0, m1);
                // (weights without a maximum are NaN or none)
                f0 = m0 == -INFINITY ? 1.f : ptx::ex2(m0 - m);
                f1 = m1 == -INFINITY ? 1.f : ptx::ex2(m1 - m);
                l = f0 * sm.red_l[0][row] + f1 * sm.red_l[1][row];
                ok = meet();  // (all have read: the next piece may write)
                if (!ok) break;
            }
            // A row before the sequence sees nothing, whatever its query (NaN makes
            // hidden scores of codes NaN) and the values that all others see hold.
            const bool before = d.at0 + token < 0;
            if (before) l = 0.f;
            for (int w = 0; ok && w < 2; ++w) {
                if (!has[w]) continue;
                if (!pair || w == wg) ok = wwait(&sm.pv_done[w], (pv_par >> w) & 1);
                pv_par ^= 1u << w;
            }
            if (!ok) break;
            ptx::tc_fence_after();
            // this thread's columns of the row: all of O_wg, or half of both
            const int col0 = pair ? 0 : 64 * wg, chunks = pair ? 4 : 2;
            const bool use0 = pair ? wg == 0 && n > 0 : has[0], use1 = pair ? wg == 1 && n > 0 : has[1];
            const bool cut = d.c0 != d.c1;
            const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: zeros
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                 ((size_t)(d.row0 + token) * g.Hq + head) * kD;
            const int slot = cut ? paged::partial_slot(sm.pl, blockIdx.x, d.base) : 0;
            const int half = pair ? wg : 0;
            float4* part = reinterpret_cast<float4*>(a.work.o) + (size_t)slot * 2 * 32 * kRows + half * 32 * kRows + row;
            if (busy) {
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    uint32_t o0[32], o1[32];
                    const uint32_t at = tmem + lane_base + kColO + (uint32_t)(col0 + 32 * c);
                    if (use0) ptx::tmem_ld32(at, o0);
                    if (use1) ptx::tmem_ld32(at + kD, o1);
                    ptx::tmem_wait_ld();
                    ptx::reg_fence(o0);
                    ptx::reg_fence(o1);
                    float acc[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float x0 = use0 && !before ? f0 * __uint_as_float(o0[i]) : 0.f;
                        acc[i] = use1 && !before ? fmaf(f1, __uint_as_float(o1[i]), x0) : x0;
                    }
                    if (valid && cut) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            part[(size_t)(col0 / 4 + 8 * c + i) * kRows] =
                                make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                    } else if (valid) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = ptx::pack_bf16x2(acc[8 * i + 2 * e] * inv, acc[8 * i + 2 * e + 1] * inv);
                            *reinterpret_cast<uint4*>(out + col0 + 32 * c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (cut && valid && (pair || wg == 0)) a.work.ml[(size_t)slot * 2 * kRows + half * kRows + row] = make_float2(m, l);
            }
            ptx::tc_fence_before();
            if (n > 0) arrive1(&sm.o_free);
            if constexpr (!kCodes) {
                if (d.taken && busy) give_rows_back(a, sm, si % kDescs);
            }
            if (!cut) {
                arrive1(&sm.d_empty[si % kDescs]);
                continue;
            }
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
            if (sm.last && valid) {
                __threadfence();
                const float2* ml = a.work.ml + half * kRows + row;
                auto slot_of = [&](int c) { return (size_t)paged::partial_slot(sm.pl, c, d.base); };
                float mm = -INFINITY;
#pragma unroll 4
                for (int c = d.c0; c <= d.c1; ++c) mm = fmaxf(mm, __ldcg(ml + slot_of(c) * 2 * kRows).x);
                const float4* po = reinterpret_cast<const float4*>(a.work.o) + (size_t)half * 32 * kRows +
                                   (size_t)(col0 / 4) * kRows + row;
                // 64 columns a time, a piece's loads all in flight together
#pragma unroll 1
                for (int c16 = 0; c16 < chunks / 2; ++c16) {
                    float acc[64], ll = 0.f;
#pragma unroll
                    for (int i = 0; i < 64; ++i) acc[i] = 0.f;
#pragma unroll 1
                    for (int c = d.c0; c <= d.c1; ++c) {
                        const float2 x = __ldcg(ml + slot_of(c) * 2 * kRows);
                        const float4* from = po + slot_of(c) * 2 * 32 * kRows + (size_t)(16 * c16) * kRows;
                        float4 y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __ldcg(from + (size_t)i * kRows);
                        const float w = x.x == -INFINITY ? 1.f : ptx::ex2(x.x - mm);
                        ll = fmaf(w, x.y, ll);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            acc[4 * i] = fmaf(w, y[i].x, acc[4 * i]);
                            acc[4 * i + 1] = fmaf(w, y[i].y, acc[4 * i + 1]);
                            acc[4 * i + 2] = fmaf(w, y[i].z, acc[4 * i + 2]);
                            acc[4 * i + 3] = fmaf(w, y[i].w, acc[4 * i + 3]);
                        }
                    }
                    const float inv_l = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = ptx::pack_bf16x2(acc[8 * i + 2 * e] * inv_l, acc[8 * i + 2 * e + 1] * inv_l);
                        *reinterpret_cast<uint4*>(out + col0 + 64 * c16 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
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

template <bool kCodes>
bool ready() {
    const auto kernel = paged_tc_kernel<kCodes>;
    static_assert(sizeof(Smem<kCodes>) <= 232448, "shared memory");
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<kCodes>)) !=
        cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    // the warpgroups' register split needs the launch count it was sized for
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != kRegsLaunch) {
        cudaGetLastError();
        return false;
    }
    return true;
}

template <bool kCodes>
cudaError_t launch(const PagedAttend& a, int max_ctas, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int page = 1 << a.g.page_log2, box = page < kKB ? page : kKB;
    const long long outer = (long long)a.g.pages * a.g.Hk;
    const int HT = kRows / a.g.G;
    CUtensorMap q, k, v;
    if (!tma_encode_head_rows(&q, a.q, a.g.Hq, a.seqs.tokens, a.q_stride, a.g.G, HT) ||
        !tma_encode_pages(&k, a.pool.k, kCodes, page, outer, box) ||
        !tma_encode_pages(&v, a.pool.v, kCodes, page, outer, box))
        return cudaErrorInvalidValue;
    const int grid = max_ctas > 0 && max_ctas < sms ? max_ctas : sms;
    static_assert(2 * 2 * kRows <= kPagedRowsPerSm, "workspace rows");
    return launch_pdl(paged_tc_kernel<kCodes>, grid, kThreads, sizeof(Smem<kCodes>), st, q, k, v, a,
                      a.scale * 1.4426950408889634f);
}

}  // namespace

bool paged_tc_init() { return tma_available() && ready<false>() && ready<true>(); }

cudaError_t launch_paged_tc(bool e4m3, const PagedAttend& a, int max_ctas, cudaStream_t st) {
    return e4m3 ? launch<true>(a, max_ctas, st) : launch<false>(a, max_ctas, st);
}

}  // namespace arl2
