// Parts shared by the tensor-core kernels over the paged cache: the pieces of
// work as their roles see them, the loading warp, and the repair of rows that a
// hidden value which is not finite has spoilt.
#pragma once

#include "paged.cuh"
#include "ptx.cuh"
#include "tma.h"

namespace arl2 {
namespace paged {

using ptx::kHalfBytes;
using ptx::kTileBytes;

constexpr int kKB = 128;  // keys per block
constexpr int kD = 128;
constexpr int kCodeTile = kKB * kD;  // bytes of a block of codes
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr int kSoftmaxWarps = 8, kWgWarps = 4;
constexpr int kDescs = 4;
// Arrivals on a K tile's barrier: the loader's and, with codes, its lanes'
// copies of the scales.
template <bool kCodes>
constexpr int kKArrivals = kCodes ? 33 : 1;

// What every role needs of a piece of work.
struct Desc {
    int done;
    int s, h, row0, n;       // sequence, key head, first token row, tokens
    int at0, total;          // position of the first token, keys of the sequence
    int ns, w0, b0, b1;      // blocks (see Blocks), this CTA's
    int pair;                // the tile has two halves
    int c0, c1;              // CTAs that share the tile
    long long base;
    // first key of this CTA's block j
    __device__ int key0(int j) const {
        const int i = b0 + j;
        return (i < ns ? i : w0 + i - ns) * kKB;
    }
};

__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// One output row again, by a whole warp, with plain loads: O = sum over the
// keys it sees of the blocks [b0, b1) of exp2(score - m) v, lane l holding
// features 4 l .. 4 l + 3.
template <bool kCodes>
static __device__ __noinline__ float4 repair_row(const PagedAttend& a, const Desc& d, int token, int head, float m,
                                                 float scale_log2) {
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16* q =
        static_cast<const __nv_bfloat16*>(a.q) + (long long)(d.row0 + token) * a.q_stride + head * kD + 4 * lane;
    float qf[4];
    for (int c = 0; c < 4; ++c) qf[c] = to_float(q[c]);
    const Sight see = sight(a.mask, d.at0 + token, d.total);
    const float base = m == -INFINITY ? 0.f : m;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int bi = d.b0; bi < d.b1; ++bi) {
        const int key0 = d.key0(bi - d.b0);
        for (int j = key0; j < key0 + kKB; ++j) {
            if (!sees(see, j)) continue;
            const int page = a.seqs.table[(size_t)d.s * a.seqs.max_pages + (j >> a.g.page_log2)];
            if ((unsigned)page >= (unsigned)a.g.pages) continue;  // (reported by the loader)
            const size_t row = pool_row(a.g, page, d.h, j), at = row * kD + 4 * lane;
            float k[4], v[4];
            for (int c = 0; c < 4; ++c) {
                if constexpr (kCodes) {
                    k[c] = to_float(static_cast<const __nv_fp8_e4m3*>(a.pool.k)[at + c]) * a.pool.ks[row];
                    v[c] = to_float(static_cast<const __nv_fp8_e4m3*>(a.pool.v)[at + c]) * a.pool.vs[row];
                } else {
                    k[c] = to_float(static_cast<const __nv_bfloat16*>(a.pool.k)[at + c]);
                    v[c] = to_float(static_cast<const __nv_bfloat16*>(a.pool.v)[at + c]);
                }
            }
            float s = 0.f;
            for (int c = 0; c < 4; ++c) s = fmaf(qf[c], k[c], s);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const float p = ptx::ex2(fmaf(s, scale_log2, -base));
            for (int c = 0; c < 4; ++c) acc[c] = fmaf(p, v[c], acc[c]);
        }
    }
    return make_float4(acc[0], acc[1], acc[2], acc[3]);
}

// The slots of the block at key0 behind the sequence's last key, in a tile of
// `halves` x 128 rows of 128 bytes: zeros (what lies in a page there may be NaN,
// and 0 x NaN is not 0).  By one warp.
__device__ __forceinline__ void clear_tail(uint8_t* tile, int halves, int key0, int total) {
    const int first = total > key0 ? total - key0 : 0;
    for (int half = 0; half < halves; ++half)
        for (int at = first * 128 + (threadIdx.x & 31) * 16; at < (int)kHalfBytes; at += 512)
            *reinterpret_cast<uint4*>(tile + half * kHalfBytes + at) = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
}

// The first `rows` rows of a Q tile (two swizzled halves of 64 features), in
// place, into two tiles of e4m3 terms: row r of the halves (kHalf bytes apart)
// lies where row r of the terms goes.  By `warps` warps, this one the w-th; 16
// lanes hold a row.  row_scale: 2^-k scale; NaN for a row that is not finite.
// (A last odd row takes the one behind it along.)
template <uint32_t kHalf>
__device__ __forceinline__ void split_q(uint8_t* tile, float* row_scale, int rows, int w, int warps, float scale) {
    const int lane = threadIdx.x & 31, c = lane & 15;
    constexpr int kBatch = 4;  // rows a lane has in flight
    for (int base = w * 2; base < rows; base += 2 * kBatch * warps) {
        uint4 u[kBatch];
        float amax[kBatch];
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
            const int r = base + 2 * warps * t + (lane >> 4);
            u[t] = make_uint4(0u, 0u, 0u, 0u);
            if (base + 2 * warps * t < rows)
                u[t] = *reinterpret_cast<const uint4*>(tile + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            auto mag = [](uint32_t x) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)); };
            const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(mag(u[t].x), mag(u[t].y)), __hmax2_nan(mag(u[t].z), mag(u[t].w)));
            const float f = __bfloat162float(__hmax_nan(m.x, m.y));
            amax[t] = f < INFINITY ? f : INFINITY;  // (NaN: infinity, too)
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (int t = 0; t < kBatch; ++t) amax[t] = fmaxf(amax[t], __shfl_xor_sync(0xffffffffu, amax[t], o));
        // (every lane has read its part of these rows: they may be overwritten)
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
            const int r = base + 2 * warps * t + (lane >> 4);
            if (base + 2 * warps * t >= rows) continue;
            int k = 7 - ((int)(__float_as_uint(amax[t]) >> 23) - 127);  // amax 2^k in [2^7, 2^8)
            k = k > 120 ? 120 : k;
            const float up = __uint_as_float((uint32_t)(127 + k) << 23), down = __uint_as_float((uint32_t)(127 - k) << 23);
            const uint32_t words[4] = {u[t].x, u[t].y, u[t].z, u[t].w};
            uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = make_float2(__uint_as_float(words[i] << 16) * up, __uint_as_float(words[i] & 0xffff0000u) * up);
                const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
                const __nv_fp8x2_storage_t l =
                    __nv_cvt_float2_to_fp8x2(make_float2(y.x - back.x, y.y - back.y), __NV_SATFINITE, __NV_E4M3);
                hi[i >> 1] |= (uint32_t)h << (16 * (i & 1));
                lo[i >> 1] |= (uint32_t)l << (16 * (i & 1));
            }
            uint8_t* to = tile + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to + kHalf) = make_uint2(lo[0], lo[1]);
            if (c == 0) row_scale[r] = amax[t] < INFINITY ? down * scale : __int_as_float(0x7fffffff);
        }
    }
}

// The loading warp: this CTA's pieces one after the other, their descriptors
// published to the other roles, their Q tiles and their blocks' pages (found
// through the page table) loaded by TMA.  S: the kernel's shared memory.  wwait:
// the bounded wait.  Returns false if one ran out; waits for its own loads
// either way.
template <bool kCodes, class S, class Wait>
__device__ __forceinline__ bool load_pieces(S& sm, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                            const CUtensorMap& tm_v, const PagedAttend& a, const Plan& pl,
                                            const Tiling& tl, Wait wwait) {
    const PagedGeom& g = a.g;
    const int lane = threadIdx.x & 31;
    const int no_abort = 0;
    auto arrive1 = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(bar));
    };
    ptx::tma_prefetch_desc(&tm_q);
    ptx::tma_prefetch_desc(&tm_k);
    ptx::tma_prefetch_desc(&tm_v);
    Cursor cur = pl.first;
    const int page_tokens = 1 << g.page_log2;
    const int pb_log2 = page_tokens < kKB ? 7 - g.page_log2 : 0;      // pages of a block
    const int per_block = 1 << pb_log2;
    const int absent = g.pages * g.Hk;                                // reads as zeros
    const int batch_log2 = 5 - pb_log2;  // blocks whose pages 32 lanes look up at once
    int kn = 0, vn = 0, qn = 0, tails = 0;
    bool ok = true, more = pl.u1 > pl.u0;
    for (int si = 0; ok; ++si) {
        const int slot = si % kDescs;
        if (si >= kDescs && !wwait(&sm.d_empty[slot], (si / kDescs - 1) & 1)) {
            ok = false;
            break;
        }
        if (!more) {
            if (lane == 0) sm.desc[slot].done = 1;
            arrive1(&sm.d_full[slot]);
            break;
        }
        const Piece pc = piece_at<kKB>(a.mask, sm.plan, pl, cur, tl);
        const bool pair = pc.n > tl.half;
        const int at0 = pc.q.total - pc.q.n + pc.i0;
        if (lane == 0)
            sm.desc[slot] = Desc{0,          cur.s,        cur.h,        pc.q.q0 + pc.i0, pc.n, at0,
                                 pc.q.total, pc.blocks.ns, pc.blocks.w0, pc.b0,           pc.b1, pair,
                                 pc.c0,      pc.c1,        cur.base};
        arrive1(&sm.d_full[slot]);
        const int n = pc.b1 - pc.b0;
        if (n > 0) {
            for (int t = 0; ok && t < (pair ? 2 : 1); ++t, ++qn) {
                const int qs = qn & 1;
                if (qn >= 2 && !wwait(&sm.q_empty[qs], ((qn >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = ptx::smem_u32(sm.q_landed(qs));
                const uint32_t dst = ptx::smem_u32(sm.q[qs]);
                ptx::mbar_arrive_expect_tx_w(bar, (uint32_t)(tl.half * g.G) * 256u);
                const int row = pc.q.q0 + pc.i0 + t * tl.half;
                ptx::tma_load_4d_w(dst, &tm_q, 0, cur.h * g.G, row, 0, bar);
                ptx::tma_load_4d_w(dst + S::kQHalf, &tm_q, 64, cur.h * g.G, row, 0, bar);
            }
            // keys that some query of the tile sees: [0, see_sink) and [see_lo, see_end)
            const Sight last = sight(a.mask, at0 + pc.n - 1, pc.q.total);
            const int see_lo = sight(a.mask, at0 < 0 ? 0 : at0, pc.q.total).lo;
            // Places in the pool (page x heads + head, or absent) of a batch of
            // blocks, one page per lane; a batch is looked up two batches
            // before it is needed, so nobody waits for the page table.
            const int span = page_tokens < kKB ? page_tokens : kKB;
            auto look_up = [&](int b, uint32_t& needed) -> int {
                const int j = (b << batch_log2) + (lane >> pb_log2);
                const int k0 = pc.blocks.at(pc.b0 + j) * kKB + ((lane & (per_block - 1)) << g.page_log2);
                const bool need = j < n && k0 < last.end && (k0 + span > see_lo || k0 < last.sink);
                needed = __ballot_sync(0xffffffffu, need);
                return need ? a.seqs.table[(size_t)cur.s * a.seqs.max_pages + (k0 >> g.page_log2)] : 0;
            };
            uint32_t n0, n1, n2;
            int b0 = look_up(0, n0), b1 = look_up(1, n1), b2 = look_up(2, n2), b_at = 0;
            // this lane's place of block j, in batch b_at or the next one
            auto place_of = [&](int j) -> int {
                const bool later = (j >> batch_log2) > b_at;
                const int src = ((j << pb_log2) & 31) + (lane & (per_block - 1));
                const int page = __shfl_sync(0xffffffffu, later ? b1 : b0, src);
                if (lane >= per_block || !(((later ? n1 : n0) >> src) & 1u)) return absent;
                if ((unsigned)page < (unsigned)g.pages) return page * g.Hk + cur.h;
                report(a.err, kErrPagedTable);
                return absent;
            };
            auto load_k = [&](int j) -> bool {
                const int s = kn % S::kK;
                const int place = place_of(j);
                if (kn >= S::kK && !wwait(&sm.k_empty[s], (kn / S::kK - 1) & 1)) return false;
                const int slot0 = pc.blocks.at(pc.b0 + j) * kKB & (page_tokens - 1);
                const uint32_t bar = ptx::smem_u32(&sm.k_full[s]);
                ptx::mbar_arrive_expect_tx_w(bar, (uint32_t)S::kKBytes);
                if constexpr (kCodes) {
                    // the scales: 16 bytes per lane and tensor (bulk copies of a
                    // page's scales cost the copy engine as much as its codes:
                    // 236 against 191 us without them at 64 streams of 8256 keys)
                    const int of = ((4 * lane) >> g.page_log2) & (per_block - 1);
                    const int there = __shfl_sync(0xffffffffu, place, of);
                    const size_t row = there == absent ? 0 : ((size_t)there << g.page_log2) + slot0 + 4 * lane - (of << g.page_log2);
                    const uint32_t bytes = there == absent ? 0u : 16u;  // (absent: zeros, as the codes will be)
                    ptx::cp_async16(ptx::smem_u32(sm.ks(kn) + 4 * lane), a.pool.ks + row, bytes);
                    ptx::cp_async16(ptx::smem_u32(sm.vs(kn) + 4 * lane), a.pool.vs + row, bytes);
                    ptx::cp_async_arrive(bar);
                }
                __syncwarp();
                if (lane < per_block) {
                    const uint32_t dst = ptx::smem_u32(sm.k[s]) + (uint32_t)(lane << g.page_log2) * 128u;
                    ptx::tma_load_4d(dst, &tm_k, 0, slot0, place, 0, bar);
                    if (!kCodes) ptx::tma_load_4d(dst + kHalfBytes, &tm_k, 64, slot0, place, 0, bar);
                }
                __syncwarp();
                ++kn;
                return true;
            };
            auto load_v = [&](int j) -> bool {
                const int s = vn % S::kVLoads;
                const int place = place_of(j);
                if (vn >= S::kVLoads && !wwait(sm.v_taken(s), (vn / S::kVLoads - 1) & 1)) return false;
                const int key0 = pc.blocks.at(pc.b0 + j) * kKB;
                const int slot0 = key0 & (page_tokens - 1);
                uint64_t* full = sm.v_landed(s);
                if (S::kClearTail && j == n - 1 && key0 + kKB > pc.q.total) {
                    full = &sm.v_tail;  // a warp of its own clears the tail and hands it on
                    ++tails;
                }
                const uint32_t bar = ptx::smem_u32(full);
                ptx::mbar_arrive_expect_tx_w(bar, kCodes ? kCodeTile : kTileBytes);
                __syncwarp();
                if (lane < per_block) {
                    const uint32_t dst = ptx::smem_u32(sm.v_load(s)) + (uint32_t)(lane << g.page_log2) * 128u;
                    ptx::tma_load_4d(dst, &tm_v, 0, slot0, place, 0, bar);
                    if (!kCodes) ptx::tma_load_4d(dst + kHalfBytes, &tm_v, 64, slot0, place, 0, bar);
                }
                __syncwarp();
                ++vn;
                return true;
            };
            // in the order in which the products give the slots back
            const int lead = pair ? S::kK - 1 : S::kK;
            for (int j = 0; ok && j < lead && j < n; ++j) ok = load_k(j);
            for (int j = 0; ok && j < n; ++j) {
                ok = load_v(j);
                if (ok && j + lead < n) ok = load_k(j + lead);
                if (((j + 1) & ((1 << batch_log2) - 1)) == 0) {
                    b0 = b1, n0 = n1;
                    b1 = b2, n1 = n2;
                    ++b_at;
                    b2 = look_up(b_at + 2, n2);
                }
            }
        }
        more = advance(sm.plan, pl, a.seqs, tl, pc.units, cur);
    }
            // the last loads of each ring have landed before exit
    auto landed = [&](uint64_t* bar, int use) {
        ptx::mbar_wait_bounded(ptx::smem_u32(bar), use & 1, &no_abort, kWaitLimitNs);
    };
    for (int i = kn > S::kK ? kn - S::kK : 0; i < kn; ++i) landed(&sm.k_full[i % S::kK], i / S::kK);
    if (tails) landed(&sm.v_tail, tails - 1);
    for (int i = vn > S::kVLoads ? vn - S::kVLoads : 0; i < vn; ++i)
        landed(sm.v_landed(i % S::kVLoads), i / S::kVLoads);
    for (int i = qn > 2 ? qn - 2 : 0; i < qn; ++i) landed(sm.q_landed(i & 1), i >> 1);
    return ok;
}

}  // namespace paged
}  // namespace arl2
