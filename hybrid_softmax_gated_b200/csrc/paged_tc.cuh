// Parts shared by the tensor-core kernels over the paged cache: the pieces of
// work as their roles see them, the loading warp, and what keeps hidden values
// that are not finite out of the products.
#pragma once

#include "paged.cuh"
#include "ptx_paged.cuh"
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
    int taken;               // values that are not finite were taken out of the products (clean_block)
    // first key of this CTA's block j
    __device__ int key0(int j) const {
        const int i = b0 + j;
        return (i < ns ? i : w0 + i - ns) * kKB;
    }
};

__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Keys that all of a tile's queries see, and that some of them see (the
// queries at positions before 0, which see nothing, left out).  Ends, lower
// ends and sinks all move right with a query's position, and each window
// starts no later than the previous one ends.
struct Seen {
    Sight all, any;
    // nothing of the block at key0 is hidden from anybody
    __device__ __forceinline__ bool open(int key0) const {
        return key0 + kKB <= all.end && (key0 >= all.lo || key0 + kKB <= all.sink);
    }
};
__device__ __forceinline__ Seen seen_by(const PagedMask& m, const Desc& d) {
    const Sight first = sight(m, d.at0 < 0 ? 0 : d.at0, d.total), last = sight(m, d.at0 + d.n - 1, d.total);
    return Seen{Sight{first.end, last.lo, first.sink}, Sight{last.end, first.lo, last.sink}};
}

// What a block of V at key0 holds for keys that not all of the tile's queries
// see, in a tile of 128-byte rows (bf16: two halves of 128 rows): a weight of 0
// hides a finite value only, 0 x NaN is not 0.  Keys that nobody sees (behind
// the last one, too) become zeros.  Of the others what is not finite becomes
// zero: an element of bf16 (returns whether there was one: the queries that see
// it get it back from give_back), a code (its scale is NaN, and so are the
// weights of those that see it).  By one warp.
template <bool kCodes>
__device__ __forceinline__ bool clean_block(uint8_t* tile, int key0, const Seen& seen) {
    constexpr int kHalves = kCodes ? 1 : 2, kStep = 16;  // keys whose loads are in flight together
    constexpr uint32_t kMax = kCodes ? 0x7f7f7f7fu : 0x7f807f80u, kOne = kCodes ? 0x01010101u : 0x00800080u;
    constexpr uint32_t kTop = kCodes ? 0x80808080u : 0x80008000u, kFull = kCodes ? 0xffu : 0xffffu;
    constexpr int kShift = kCodes ? 7 : 15;
    // (a code of ones, an exponent of ones: the sum's carry)
    auto hits = [&](uint32_t w) { return ((w & kMax) + kOne) & kTop; };
    const int lane = threadIdx.x & 31;
    bool found = false;
    for (int r = 0; r < kKB; r += kStep) {
        const int key = key0 + r;
        if (key + kStep <= seen.all.end && (key >= seen.all.lo || key + kStep <= seen.all.sink)) continue;
        uint8_t* const base = tile + r * 128 + lane * 16;  // of the lane's 16 bytes of key r + lane / 8 + 4 i: 512 i on
        auto at = [&](int i) { return reinterpret_cast<uint4*>(base + (i >> 2) * kHalfBytes + (i & 3) * 512); };
        if (key >= seen.any.end || (key >= seen.any.sink && key + kStep <= seen.any.lo)) {
#pragma unroll
            for (int i = 0; i < 4 * kHalves; ++i) *at(i) = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint4 u[4 * kHalves];
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i) u[i] = *at(i);
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i) {
            if constexpr (kCodes) {
                bad |= hits(u[i].x) | hits(u[i].y) | hits(u[i].z) | hits(u[i].w);
            } else {
                auto mag = [](uint32_t x) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)); };
                const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(mag(u[i].x), mag(u[i].y)), __hmax2_nan(mag(u[i].z), mag(u[i].w)));
                bad |= hits(*reinterpret_cast<const uint32_t*>(&m));
            }
        }
        // (rare: so are steps with keys that nobody sees among others)
        const bool some_none = !(key + kStep <= seen.any.end && (key >= seen.any.lo || key + kStep <= seen.any.sink));
        if (bad || some_none) {
#pragma unroll 1
            for (int i = 0; i < 4 * kHalves; ++i) {
                const int k = key + (lane >> 3) + 4 * (i & 3);
                if (!sees(seen.any, k)) {
                    *at(i) = make_uint4(0u, 0u, 0u, 0u);
                } else if (!sees(seen.all, k)) {
                    uint4 x = *at(i);
                    uint32_t was = 0u;
                    auto clear = [&](uint32_t& w) {
                        const uint32_t hit = hits(w);
                        was |= hit;
                        w &= ~((hit >> kShift) * kFull);
                    };
                    clear(x.x), clear(x.y), clear(x.z), clear(x.w);
                    if (was) {
                        *at(i) = x;
                        found = true;
                    }
                }
            }
        }
    }
    ptx::fence_proxy_async_smem();
    return __any_sync(0xffffffffu, found);
}

// What clean_block has taken out goes to the outputs of the rows that see it: it
// is an infinity or NaN, and a weight is positive, so it is added as it is.  Only
// keys at the mask's edges are looked at, at most as many as a block and the tile
// have tokens.  Calls use(values, key) for 16 keys at a time of this CTA's
// blocks, `values` their rows in the pool (16 keys share a page; the end of a page
// that is seen in part is read as well, the slots are there).  bf16 pages.
constexpr int kEdgeKeys = 16;
template <class Use>
__device__ __forceinline__ void for_edge_keys(const PagedAttend& a, const Desc& d, const Seen& seen, Use use) {
    for (int bi = d.b0; bi < d.b1; ++bi) {
        const int key0 = d.key0(bi - d.b0);
        if (seen.open(key0)) continue;
        for (int j = key0; j < key0 + kKB; j += kEdgeKeys) {
            if (j >= seen.any.end || (j >= seen.any.sink && j + kEdgeKeys <= seen.any.lo)) continue;
            const int page = a.seqs.table[(size_t)d.s * a.seqs.max_pages + (j >> a.g.page_log2)];
            if ((unsigned)page < (unsigned)a.g.pages)  // (else reported by the loader)
                use(static_cast<const __nv_bfloat16*>(a.pool.v) + pool_row(a.g, page, d.h, j) * kD, j);
        }
    }
}
__device__ __forceinline__ uint32_t not_finite_bf16(uint32_t w) {  // bit 15, bit 31
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
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

// Where a piece's blocks lie: their pages' places in the pool (page x heads +
// head, or `absent`, which reads as zeros), one page per lane for a batch of
// blocks at a time; a batch is looked up two batches before it is needed, so
// nobody waits for the page table.  The whole warp.
struct Places {
    const PagedAttend* a;
    const Desc* d;
    int n, pb_log2, batch_log2, span, absent;  // blocks; pages of a block, blocks of a batch, keys of a page's share
    Seen seen;
    int at;          // batch of p0
    int p0, p1, raw; // places of batches at and at + 1; what the table says of at + 2
    bool need;

    __device__ __forceinline__ int per_block() const { return 1 << pb_log2; }
    __device__ __forceinline__ int slot0(int j) const { return d->key0(j) & ((1 << a->g.page_log2) - 1); }
    __device__ __forceinline__ void look_up(int batch) {
        const int lane = threadIdx.x & 31, j = (batch << batch_log2) + (lane >> pb_log2);
        const int k0 = d->key0(j) + ((lane & (per_block() - 1)) << a->g.page_log2);
        need = j < n && k0 < seen.any.end && (k0 + span > seen.any.lo || k0 < seen.any.sink);
        raw = need ? a->seqs.table[(size_t)d->s * a->seqs.max_pages + (k0 >> a->g.page_log2)] : 0;
    }
    __device__ __forceinline__ int found() const {
        if (!need) return absent;
        if ((unsigned)raw < (unsigned)a->g.pages) return raw * a->g.Hk + d->h;
        report(a->err, kErrPagedTable);
        return absent;
    }
    __device__ __forceinline__ Places(const PagedAttend& a_, const Desc& d_) : a(&a_), d(&d_) {
        const int page_tokens = 1 << a->g.page_log2;
        n = d->b1 - d->b0;
        pb_log2 = page_tokens < kKB ? 7 - a->g.page_log2 : 0;
        batch_log2 = 5 - pb_log2;
        span = page_tokens < kKB ? page_tokens : kKB;
        absent = a->g.pages * a->g.Hk;
        seen = seen_by(a->mask, d_);
        at = 0;
        look_up(0);
        const bool n0 = need;
        const int r0 = raw;
        look_up(1);
        const bool n1 = need;
        const int r1 = raw;
        look_up(2);
        const bool n2 = need;
        const int r2 = raw;
        need = n0, raw = r0;
        p0 = found();
        need = n1, raw = r1;
        p1 = found();
        need = n2, raw = r2;
    }
    // place of this lane's page of block j, in batch `at` or the next one (lanes
    // past the block's pages: any)
    __device__ __forceinline__ int of(int j) const {
        const int src = ((j << pb_log2) & 31) + ((threadIdx.x & 31) & (per_block() - 1));
        return __shfl_sync(0xffffffffu, (j >> batch_log2) > at ? p1 : p0, src);
    }
    // block j (and all before it) is done with
    __device__ __forceinline__ void done(int j) {
        if (((j + 1) & ((1 << batch_log2) - 1)) == 0) {
            p0 = p1;
            p1 = found();
            ++at;
            look_up(at + 2);
        }
    }
};

// A ring's slot and the parity of its barriers' phase, without divisions.
template <int kSlots>
struct Ring {
    int slot = 0, uses = 0;
    uint32_t lap = 0;
    __device__ __forceinline__ bool waits() const { return uses >= kSlots; }
    __device__ __forceinline__ uint32_t parity() const { return (lap & 1) ^ 1; }  // of the slot's previous lap
    __device__ __forceinline__ void next() {
        ++uses;
        if (++slot == kSlots) {
            slot = 0;
            ++lap;
        }
    }
};

// Cleans the blocks that need it, of all pieces in order, in a warp of its own:
// from the slot's v_edge barrier (the loader's) to its v_full.  get_desc and
// wwait: the kernel's.  Returns false if a wait ran out.
template <bool kCodes, class S, class Get, class Wait>
__device__ __forceinline__ bool clean_pieces(S& sm, const PagedMask& m, Get get_desc, Wait wwait) {
    Ring<S::kVLoads> vr;
    uint32_t odd = 0;  // parities of the slots' v_edge
    for (int si = 0;; ++si) {
        Desc d;
        if (!get_desc(si, d)) return false;
        if (d.done) return true;
        const Seen seen = seen_by(m, d);
        for (int j = 0; j < d.b1 - d.b0; ++j, vr.next()) {
            const int key0 = d.key0(j), s = vr.slot;
            if (seen.open(key0)) continue;
            if (!wwait(&sm.v_edge[s], (odd >> s) & 1)) return false;
            odd ^= 1u << s;
            // (the softmax warps hold the piece's descriptor until its end, and
            // look at it after the products with this block)
            if (clean_block<kCodes>(sm.v_load(s), key0, seen)) sm.desc[si % kDescs].taken = 1;
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_u32(sm.v_landed(s)));
        }
    }
}

template <bool kCodes, class S>
struct Loader {
    S& sm;
    const PagedAttend& a;
    const CUtensorMap &tm_q, &tm_k, &tm_v;
    Ring<S::kK> kr;
    Ring<S::kVLoads> vr;
    int qn = 0;
    uint32_t edges = 0, edge_odd = 0;  // V slots that ever held a block to be cleaned; an odd number of them

    // Q tiles of the piece
    template <class Wait>
    __device__ __forceinline__ bool load_q(const Desc& d, int half, Wait wwait) {
        for (int t = 0; t < (d.pair ? 2 : 1); ++t, ++qn) {
            const int qs = qn & 1;
            if (qn >= 2 && !wwait(&sm.q_empty[qs], ((qn >> 1) - 1) & 1)) return false;
            const uint32_t bar = ptx::smem_u32(sm.q_landed(qs)), dst = ptx::smem_u32(sm.q[qs]);
            ptx::mbar_arrive_expect_tx_w(bar, (uint32_t)(half * a.g.G) * 256u);
            ptx::tma_load_4d_w(dst, &tm_q, 0, d.h * a.g.G, d.row0 + t * half, 0, bar);
            ptx::tma_load_4d_w(dst + S::kQHalf, &tm_q, 64, d.h * a.g.G, d.row0 + t * half, 0, bar);
        }
        return true;
    }
    template <class Wait>
    __device__ __forceinline__ bool load_k(const Places& pl, int j, Wait wwait) {
        const int lane = threadIdx.x & 31, s = kr.slot, place = pl.of(j), slot0 = pl.slot0(j);
        if (kr.waits() && !wwait(&sm.k_empty[s], kr.parity())) return false;
        const uint32_t bar = ptx::smem_u32(&sm.k_full[s]);
        ptx::mbar_arrive_expect_tx_w(bar, (uint32_t)S::kKBytes);
        __syncwarp();
        if (lane < pl.per_block()) {
            const uint32_t dst = ptx::smem_u32(sm.k[s]) + (uint32_t)(lane << a.g.page_log2) * 128u;
            ptx::tma_load_4d(dst, &tm_k, 0, slot0, place, 0, bar);
            if (!kCodes) ptx::tma_load_4d(dst + kHalfBytes, &tm_k, 64, slot0, place, 0, bar);
        }
        __syncwarp();
        if constexpr (kCodes) {
            // the scales: 16 bytes per lane and tensor (bulk copies of a page's
            // scales cost the copy engine as much as its codes: 236 us, against
            // 201 this way, at 64 streams of 8256 keys)
            const int of = ((4 * lane) >> a.g.page_log2) & (pl.per_block() - 1);
            const int there = __shfl_sync(0xffffffffu, place, of);
            const bool is = there != pl.absent;
            const size_t row = is ? ((size_t)there << a.g.page_log2) + slot0 + 4 * lane - (of << a.g.page_log2) : 0;
            const uint32_t to = ptx::smem_u32(sm.ks(kr.uses)) + 16u * lane, bytes = is ? 16u : 0u;  // (absent: zeros, as the codes)
            ptx::cp_async16(to, a.pool.ks + row, bytes);
            ptx::cp_async16(to + kKB * 4u, a.pool.vs + row, bytes);
            ptx::cp_async_arrive(bar);
        }
        kr.next();
        return true;
    }
    template <class Wait>
    __device__ __forceinline__ bool load_v(const Places& pl, int j, Wait wwait) {
        const int lane = threadIdx.x & 31, s = vr.slot, place = pl.of(j), slot0 = pl.slot0(j);
        if (vr.waits() && !wwait(sm.v_taken(s), vr.parity())) return false;
        uint64_t* full = sm.v_landed(s);
        if (S::kClean && !pl.seen.open(pl.d->key0(j))) {
            // another warp cleans the block and hands it on
            full = &sm.v_edge[s];
            edges |= 1u << s;
            edge_odd ^= 1u << s;
        }
        const uint32_t bar = ptx::smem_u32(full);
        ptx::mbar_arrive_expect_tx_w(bar, kCodes ? kCodeTile : kTileBytes);
        __syncwarp();
        if (lane < pl.per_block()) {
            const uint32_t dst = ptx::smem_u32(sm.v_load(s)) + (uint32_t)(lane << a.g.page_log2) * 128u;
            ptx::tma_load_4d(dst, &tm_v, 0, slot0, place, 0, bar);
            if (!kCodes) ptx::tma_load_4d(dst + kHalfBytes, &tm_v, 64, slot0, place, 0, bar);
        }
        __syncwarp();
        vr.next();
        return true;
    }
    // the last loads of each ring have landed (before exit)
    __device__ __forceinline__ void drain() {
        const int no_abort = 0;
        auto landed = [&](uint64_t* bar, int use) {
            ptx::mbar_wait_bounded(ptx::smem_u32(bar), use & 1, &no_abort, kWaitLimitNs);
        };
        for (int i = kr.uses > S::kK ? kr.uses - S::kK : 0; i < kr.uses; ++i) landed(&sm.k_full[i % S::kK], i / S::kK);
        if constexpr (S::kClean)
            for (int i = 0; i < S::kVLoads; ++i)
                if (edges >> i & 1) landed(&sm.v_edge[i], (edge_odd >> i & 1) ^ 1);
        for (int i = vr.uses > S::kVLoads ? vr.uses - S::kVLoads : 0; i < vr.uses; ++i)
            landed(sm.v_landed(i % S::kVLoads), i / S::kVLoads);
        for (int i = qn > 2 ? qn - 2 : 0; i < qn; ++i) landed(sm.q_landed(i & 1), i >> 1);
    }
};

// The loading warp: this CTA's pieces one after the other, their descriptors
// published to the other roles, their Q tiles and their blocks' pages loaded by
// TMA; with_v: V's too (else a warp of its own loads them, load_values).  S: the
// kernel's shared memory.  wwait: the bounded wait.  Returns false if one ran
// out; waits for its own loads either way.
template <bool kCodes, bool with_v, class S, class Wait>
__device__ __forceinline__ bool load_pieces(S& sm, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                            const CUtensorMap& tm_v, const PagedAttend& a, const Plan& pl,
                                            const Tiling& tl, Wait wwait) {
    const int lane = threadIdx.x & 31;
    auto arrive1 = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(bar));
    };
    ptx::tma_prefetch_desc(&tm_q);
    ptx::tma_prefetch_desc(&tm_k);
    if (with_v) ptx::tma_prefetch_desc(&tm_v);
    Loader<kCodes, S> ld{sm, a, tm_q, tm_k, tm_v};
    Cursor cur = pl.first;
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
        const Desc d{0,          cur.s,        cur.h,        pc.q.q0 + pc.i0, pc.n,  pc.q.total - pc.q.n + pc.i0,
                     pc.q.total, pc.blocks.ns, pc.blocks.w0, pc.b0,           pc.b1, pair,
                     pc.c0,      pc.c1,        cur.base,     0};
        if (lane == 0) sm.desc[slot] = d;
        arrive1(&sm.d_full[slot]);
        const int n = pc.b1 - pc.b0;
        if (n > 0) {
            ok = ld.load_q(d, tl.half, wwait);
            Places at(a, d);
            if (with_v) {
                // in the order in which the products give the slots back
                const int lead = pair ? S::kK - 1 : S::kK;
                for (int j = 0; ok && j < lead && j < n; ++j) ok = ld.load_k(at, j, wwait);
                for (int j = 0; ok && j < n; ++j) {
                    ok = ld.load_v(at, j, wwait);
                    if (ok && j + lead < n) ok = ld.load_k(at, j + lead, wwait);
                    at.done(j);
                }
            } else {
                for (int j = 0; ok && j < n; ++j) {
                    ok = ld.load_k(at, j, wwait);
                    at.done(j);
                }
            }
        }
        more = advance(sm.plan, pl, a.seqs, tl, pc.units, cur);
    }
    ld.drain();
    return ok;
}

}  // namespace paged
}  // namespace arl2
