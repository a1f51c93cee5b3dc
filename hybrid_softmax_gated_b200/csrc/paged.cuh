// Device code shared by the kernels that read the paged cache: the batch's
// tables (checked before use), the keys a query tile sees, and the schedule
// that splits the tiles' key blocks evenly over the CTAs.
#pragma once

#include "paged.h"

#include <cuda_fp8.h>

namespace arl2 {
namespace paged {

__device__ __forceinline__ void report(int* err, int bit) { atomicOr(err, bit); }

// New tokens and length of sequence s; n = 0 if its entries are wrong.
struct Seq {
    int q0, n, total;
};
__device__ __forceinline__ Seq seq_at(const PagedSeqs& b, int page_log2, int s, int* err) {
    const int q0 = b.q_off[s], q1 = b.q_off[s + 1], t = b.kv_len[s];
    const bool bad = q0 < 0 || q1 < q0 || q1 > b.tokens || t < 0 || t > (b.max_pages << page_log2);
    if (bad) {
        report(err, kErrPagedTable);
        return Seq{0, 0, 0};
    }
    return Seq{q0, q1 - q0, t};
}

// Page that holds key j of sequence s, or page 0 if the table's entry is
// outside the pool: an address in bounds either way.
__device__ __forceinline__ int page_at(const PagedSeqs& b, const PagedGeom& g, int s, int j, int* err) {
    const int p = b.table[(size_t)s * b.max_pages + (j >> g.page_log2)];
    if ((unsigned)p < (unsigned)g.pages) return p;
    report(err, kErrPagedTable);
    return 0;
}

// Row (page, head, slot) of key j in the pool's [pages][Hk][page] order.
__device__ __forceinline__ size_t pool_row(const PagedGeom& g, int page, int head, int j) {
    return (((size_t)page * g.Hk + head) << g.page_log2) + (j & ((1 << g.page_log2) - 1));
}

// Keys the query at position `at` sees: [0, sink) and [lo, end).
struct Sight {
    int end, lo, sink;
};
__device__ __forceinline__ Sight sight(const PagedMask& m, int at, int total) {
    if (at < 0) return Sight{0, 0, 0};
    // (positions and blocks stay below 2^30 + 1: e below 2^31 + 1)
    const uint32_t e = m.block == 1 ? (uint32_t)at + 1u : ((uint32_t)at / (uint32_t)m.block + 1u) * (uint32_t)m.block;
    Sight s;
    s.end = (int)min(e, (uint32_t)total);
    s.lo = 0;
    s.sink = 0;
    if (m.window) {
        s.lo = e < (uint32_t)m.window ? 0 : (int)(e - (uint32_t)m.window);
        s.sink = m.sinks < s.end ? m.sinks : s.end;
    }
    return s;
}
__device__ __forceinline__ bool sees(const Sight& s, int j) {
    return j < s.end && (j >= s.lo || j < s.sink);
}

// Key blocks of KB keys that the tile of the new tokens [i0, i0 + n) sees:
// blocks [0, ns) and [w0, w1).  Both ends of a query's window move right with
// its position, so the first query gives the lower bound and the last the
// upper one.
struct Blocks {
    int ns, w0, w1;
    __device__ int count() const { return ns + w1 - w0; }
    __device__ int at(int i) const { return i < ns ? i : w0 + i - ns; }
};
template <int KB>
__device__ __forceinline__ Blocks blocks_of(const PagedMask& m, const Seq& q, int i0, int n) {
    const int first = q.total - q.n + i0;
    const Sight hi = sight(m, first + n - 1, q.total);
    const Sight lo = sight(m, first < 0 ? 0 : first, q.total);
    Blocks b;
    b.w1 = (hi.end + KB - 1) / KB;
    b.w0 = lo.lo / KB;
    if (b.w0 > b.w1) b.w0 = b.w1;
    b.ns = (hi.sink + KB - 1) / KB;
    if (b.ns > b.w0) b.ns = b.w0;
    return b;
}

// ---- schedule ---------------------------------------------------------------
// A tile is a run of new tokens of one sequence with the G query heads of one
// key head; it counts some units (its cost) for each block of KB keys that it
// sees and some for itself.  In the order (head, sequence, tile, block), CTA c
// takes the units [c U / P, (c + 1) U / P) of all U, P CTAs taking part; a
// border in a small tile, or in what a tile costs for itself, moves back to the
// tile's start.  A tile cut by a border leaves one partial in each CTA's piece
// of it; the last CTA to arrive merges them, in order.  Nobody waits for anybody.
// Every CTA works this out from the device's tables: no host copy of the
// lengths, no planning launch.
struct PlanSmem {
    int q_off[kPagedMaxSeqs + 1];
    int total[kPagedMaxSeqs];
    long long warp_sum[32];
    int warp_tiles[32];
    long long start_base;          // units of the head before the first tile
    int start_seq, start_tile;
    long long start, end;          // the CTA's first unit and its last + 1, of their heads
};

struct Cursor {
    int h, s, t;       // head, sequence, tile of the sequence
    long long base;    // the tile's first unit
};

struct Plan {
    long long U, u0, u1;  // all units, this CTA's
    int P;                // CTAs that take part
    Cursor first;
};

// Exclusive prefix over the block's threads (32 warps at most); *all gets the sum.
template <typename T>
__device__ __forceinline__ T warp_scan(T x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
template <typename T>
__device__ __forceinline__ T block_prefix(T v, T* warp_sum, T* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const T x = warp_scan(v);
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    const T sums = warp_scan(lane < warps ? warp_sum[lane] : (T)0);
    *all = __shfl_sync(0xffffffffu, sums, 31);
    const T before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : (T)0) + x - v;
}
// a b / c and a / c, in 32 bits where they fit (64-bit divisions cost hundreds of cycles)
__device__ __forceinline__ long long mul_div(long long a, int b, long long c) {
    const unsigned long long p = (unsigned long long)a * (unsigned)b;
    return p >> 32 || c >> 32 ? (long long)(p / (unsigned long long)c) : (long long)((uint32_t)p / (uint32_t)c);
}

__device__ __forceinline__ Seq seq_of(const PlanSmem& ps, int s) {
    return ps.total[s] < 0 ? Seq{0, 0, 0} : Seq{ps.q_off[s], ps.q_off[s + 1] - ps.q_off[s], ps.total[s]};
}

// Tiles of a kernel: tokens of a tile and of one half of it (half = tokens: no
// halves); in units, what a block of keys costs a tile of two halves, one whose
// tokens fit a half and one whose tokens fit a quarter, what a tile costs on
// top (its queries, its outputs), and up to how many it is never cut.
struct Tiling {
    int tokens, half, pair_cost, single_cost, small_cost, tile_cost, whole;
};
__device__ __forceinline__ int weight_of(const Seq& q, int t, const Tiling& tl) {
    const int n = q.n - t * tl.tokens;
    return n > tl.half ? tl.pair_cost : 2 * n > tl.half ? tl.single_cost : tl.small_cost;
}

template <int KB>
__device__ __forceinline__ int units_of(const PagedMask& m, const Seq& q, int t, const Tiling& tl) {
    const int i0 = t * tl.tokens;
    const int c = blocks_of<KB>(m, q, i0, q.n - i0 < tl.tokens ? q.n - i0 : tl.tokens).count();
    return (c > 0 ? c : 1) * weight_of(q, t, tl) + tl.tile_cost;
}

// The whole block.  tiles: kPagedMaxSeqs + 1 integers of shared memory for the
// exclusive prefix of the sequences' tiles, free again afterwards.  grid CTAs; no CTA gets fewer than min_units units while
// others have them (each cut costs a partial and its merge).
// Where a border at unit u of a tile [at, at + units) goes.
__device__ __forceinline__ long long border(long long u, long long at, int units, const Tiling& tl) {
    return units <= tl.whole || u - at <= tl.tile_cost ? at : u;
}

template <int KB>
__device__ Plan make_plan(const PagedGeom& g, const PagedSeqs& b, const PagedMask& m, const Tiling& tl,
                          int min_units, PlanSmem& ps, int* tiles, int* err) {
    const int N = blockDim.x, tid = threadIdx.x;
    // tiles of each sequence
    const int per = (b.S + N - 1) / N;
    const int s0 = min(tid * per, b.S), s1 = min(s0 + per, b.S);
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
        const Seq q = seq_at(b, g.page_log2, s, err);
        ps.q_off[s] = b.q_off[s];
        ps.total[s] = q.n > 0 ? q.total : -1;  // (-1: no rows, or wrong entries)
        tiles[s] = mine;
        mine += (q.n + tl.tokens - 1) / tl.tokens;
    }
    if (tid == 0) ps.q_off[b.S] = b.q_off[b.S];
    int n_tiles;
    const int before = block_prefix(mine, ps.warp_tiles, &n_tiles);
    for (int s = s0; s < s1; ++s) tiles[s] += before;
    if (tid == 0) tiles[b.S] = n_tiles;
    __syncthreads();
    Plan pl{};
    if (n_tiles == 0) return pl;
    // units of this thread's share of the tiles
    const int tper = (n_tiles + N - 1) / N;
    const int f0 = min(tid * tper, n_tiles), f1 = min(f0 + tper, n_tiles);
    int s_first = 0;
    if (f0 < f1) {  // last sequence whose first tile is <= f0 and that has tiles
        int lo = 0, hi = b.S;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tiles[mid] <= f0)
                lo = mid;
            else
                hi = mid;
        }
        s_first = lo;
    }
    long long sum = 0;
    for (int f = f0, s = s_first; f < f1; ++f) {
        while (f >= tiles[s + 1]) ++s;
        sum += units_of<KB>(m, seq_of(ps, s), f - tiles[s], tl);
    }
    long long all;
    const long long pre = block_prefix(sum, ps.warp_sum, &all);
    pl.U = all * g.Hk;
    pl.P = gridDim.x;
    if (pl.U < (long long)pl.P * min_units) pl.P = pl.U < min_units ? 1 : (int)(pl.U / min_units);
    if ((int)blockIdx.x >= pl.P) return pl;
    pl.u0 = mul_div(pl.U, blockIdx.x, pl.P);
    pl.u1 = mul_div(pl.U, blockIdx.x + 1, pl.P);
    // the tiles under both borders
    const int h0 = (int)mul_div(pl.u0, 1, all), h1 = (int)mul_div(pl.u1, 1, all);
    const long long rem0 = pl.u0 - h0 * all, rem1 = pl.u1 - h1 * all;
    const bool has0 = rem0 >= pre && rem0 < pre + sum, has1 = rem1 >= pre && rem1 < pre + sum && rem1 > 0;
    if (has0 || has1) {
        long long at = pre;
        for (int f = f0, s = s_first; f < f1; ++f) {
            while (f >= tiles[s + 1]) ++s;
            const int u = f1 - f0 == 1 ? (int)sum : units_of<KB>(m, seq_of(ps, s), f - tiles[s], tl);
            if (has0 && rem0 >= at && rem0 < at + u) {
                ps.start_base = at;
                ps.start_seq = s;
                ps.start_tile = f - tiles[s];
                ps.start = border(rem0, at, u, tl);
            }
            if (has1 && rem1 >= at && rem1 < at + u) ps.end = border(rem1, at, u, tl);
            at += u;
        }
    }
    __syncthreads();
    pl.first = Cursor{h0, ps.start_seq, ps.start_tile, h0 * all + ps.start_base};
    pl.u0 = h0 * all + ps.start;
    if (rem1 > 0) pl.u1 = h1 * all + ps.end;
    return pl;
}

// The tile under the cursor: its queries, blocks, and the CTA's piece of it.
struct Piece {
    Seq q;
    int i0, n;          // first new token of the tile, tokens
    Blocks blocks;
    int units;          // of the whole tile
    int b0, b1;         // the CTA's blocks of it: indices into blocks (b0 == b1: none)
    int c0, c1;         // CTAs that share it
};
template <int KB>
__device__ __forceinline__ Piece piece_at(const PagedMask& m, const PlanSmem& ps, const Plan& pl, const Cursor& c,
                                          const Tiling& tl) {
    Piece p;
    p.q = seq_of(ps, c.s);
    p.i0 = c.t * tl.tokens;
    p.n = min(tl.tokens, p.q.n - p.i0);
    p.blocks = blocks_of<KB>(m, p.q, p.i0, p.n);
    const int count = p.blocks.count();
    const int w = weight_of(p.q, c.t, tl);
    p.units = (count > 0 ? count : 1) * w + tl.tile_cost;
    const long long a = pl.u0 > c.base ? pl.u0 - c.base : 0;
    const long long z = pl.u1 - c.base < p.units ? pl.u1 - c.base : p.units;
    // (a border inside a block leaves it to the CTA that has its first unit)
    p.b0 = count > 0 && a > 0 ? ((int)a - tl.tile_cost + w - 1) / w : 0;
    p.b1 = count > 0 ? ((int)z - tl.tile_cost + w - 1) / w : 0;
    if (a == 0 && z == p.units) {
        p.c0 = p.c1 = blockIdx.x;
    } else {
        p.c0 = (int)(((c.base + 1) * pl.P - 1) / pl.U);
        if (mul_div(pl.U, p.c0 + 1, pl.P) - c.base <= tl.tile_cost) ++p.c0;  // (that border moved to the tile's start)
        p.c1 = (int)(((c.base + p.units) * pl.P - 1) / pl.U);
    }
    return p;
}
// To the next tile; false when it is not this CTA's.
__device__ __forceinline__ bool advance(const PlanSmem& ps, const Plan& pl, const PagedSeqs& b, const Tiling& tl, int units,
                                        Cursor& c) {
    c.base += units;
    if (c.base >= pl.u1) return false;
    ++c.t;
    if (c.t * tl.tokens >= seq_of(ps, c.s).n) {
        c.t = 0;
        do {
            if (++c.s == b.S) {
                c.s = 0;
                ++c.h;
            }
        } while (seq_of(ps, c.s).n <= 0);
    }
    return true;
}
// Where CTA c keeps its partial of the tile that starts at unit `base`: slot
// 0 if the tile reaches back to or before the CTA's first unit, else 1 (a CTA
// has at most one cut tile at each end).
__device__ __forceinline__ int partial_slot(const Plan& pl, int c, long long base) {
    return 2 * c + (mul_div(pl.U, c, pl.P) >= base ? 0 : 1);
}

template <typename T>
__device__ __forceinline__ float to_float(T x) {
    return static_cast<float>(x);
}
template <>
__device__ __forceinline__ float to_float<__nv_fp8_e4m3>(__nv_fp8_e4m3 x) {
    return static_cast<float>(x);
}
__device__ __forceinline__ void store_as(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

}  // namespace paged
}  // namespace arl2
