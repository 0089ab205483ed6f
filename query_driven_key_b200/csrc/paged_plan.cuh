// paged_plan.cuh -- how the attention of new tokens over the paged cache is
// divided among the thread blocks, and how what the division cut is joined.
//
// Query rows: row r of request b is its new token r / G and query head r % G of
// the KV head's group, so that the G heads that share keys fill a tile
// together.  An item is (request, KV head, tile of R rows); its work, in units,
// is the number of BN-key tiles that any of its rows sees (at least 1, so that
// rows that see nothing are still written) and a fixed cost.  The items' units
// form one sequence, requests first, then heads, then row tiles; block i of P
// takes the i-th of P equal parts of it.  Whatever the mix of lengths, all blocks
// get the same work to within a unit or a short item, which is not cut; an item that a part's border cuts is computed in
// pieces, each piece leaves its (max, sum, O) in the workspace, and the block
// that finishes the last one joins them in order.  Lengths stay on the device: the plan is
// recomputed from q_start and kv_lens by every launch, so that a captured
// launch follows the lengths of each replay.
#pragma once

#include <type_traits>

#include "pages.cuh"
#include "ptx.cuh"

namespace think {

struct PagedArgs {
    const void *q, *k, *v;
    void *out;
    const int32_t *q_start, *kv_lens, *table;
    unsigned *status;
    unsigned *tickets;  // [parts] pieces of the item that a part begins which are done; zero between calls
    float *part;  // [parts][2 pieces][sides] partials
    int64_t q_st, q_sh, o_st, o_sh;
    int64_t k_sp, k_sh, k_sn, v_sp, v_sh, v_sn;
    int64_t table_ld;
    Divisor group, page;  // query heads a KV head, rows a page
    int B, T, Hkv, num_pages, limit, window;
    int rows_cap;  // rows of a partial that may hold data
    int parts;     // blocks of the attention launch
    int sides;     // partials of a piece: 2 where two warpgroups work on it
    float scale_log2;
};

constexpr int kPartLd = kD + 2;  // a partial: O [128 channels][rows_cap], maxima [rows_cap], sums [rows_cap]

struct Request {
    int row0, n, kv;  // first row of q, new tokens, tokens with the new ones
};

// Lengths and offsets from the device arrays, held to the buffers' bounds.
__device__ __forceinline__ Request load_request(const PagedArgs &a, int b)
{
    Request s;
    s.row0 = min(max(a.q_start[b], 0), a.T);
    s.n = min(max(a.q_start[b + 1], s.row0), a.T) - s.row0;
    s.kv = min(max(a.kv_lens[b], 0), a.limit);
    return s;
}

// The keys that some row of row tile qt sees: [lo, hi), and the range of key
// tiles [j0, j1) that holds them (one empty tile if there are none).
struct TileRange {
    int lo, hi, j0, j1;
};
template <int R, int BN>
__device__ __forceinline__ TileRange tile_range(const PagedArgs &a, const Request &s, int qt)
{
    const int rows = s.n * a.group.d;
    const int r0 = qt * R, r1 = min(r0 + R, rows) - 1;
    const int p0 = s.kv - s.n + a.group.quot(r0), p1 = s.kv - s.n + a.group.quot(r1);  // first and last position
    TileRange t;
    t.lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    t.hi = max(p1 + 1, 0);
    if (t.hi <= t.lo) {
        t.lo = t.hi = t.j0 = 0;
        t.j1 = 1;
    } else {
        t.j0 = t.lo / BN;
        t.j1 = (t.hi + BN - 1) / BN;
    }
    return t;
}

// What an item costs beyond its key tiles (its queries, its output, the
// pipeline's start and end), in key tiles: the sequence that is divided counts
// it before the item's first tile.
// Measured for a prompt of 16384 tokens (R = 256): 0 tiles 2231 us, 2: 2089,
// 3: 2040, 4: 2024; the fp32 kernel's items cost less than one of its tiles.
template <int R>
constexpr int kItemCost = R == 256 ? 4 : 1;
// The least units of a part: more parts only make for longer joins (one token over
// 4000 keys with 4 units a part 18.0 us, with 1 19.8).
template <int R>
constexpr int kLeast = R == 256 ? 4 : 1;

template <int R>
__device__ __forceinline__ int row_tiles(const PagedArgs &a, const Request &s)
{
    return (s.n * a.group.d + R - 1) / R;
}

// Units of one KV head of a request: the key tiles and costs of its row tiles, every `step`-th from `first`.
template <int R, int BN>
__device__ __forceinline__ int64_t head_units(const PagedArgs &a, const Request &s, int first, int step)
{
    const int nt = row_tiles<R>(a, s);
    int64_t u = 0;
    for (int qt = first; qt < nt; qt += step) {
        const TileRange t = tile_range<R, BN>(a, s, qt);
        u += kItemCost<R> + t.j1 - t.j0;
    }
    return u;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T x)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T x)  // inclusive
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// A place in the sequence.
struct Place {
    int b, h, qt, off;  // the item, and the units of it that lie before the place
};

// (Divisions of 64 bits take some hundred cycles, and every block starts with
// three: most totals fit 32.)
__device__ __forceinline__ int64_t quot64(int64_t x, int64_t d)  // x, d >= 0, d > 0
{
    return ((x | d) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}

// Scratch of plan(): one block's.
struct PlanSmem {
    int64_t ws[33];
    Place place;
    Request request;  // of the place
};

// Items of up to so many key tiles are not cut: a join takes longer than their
// tiles in one block.  (Tiles of items that the warpgroups share by keys take
// half the time; an fp32 tile takes as long as a join.)  Measured, cut -> whole: 16
// single tokens over 250 to 500 keys 29.0 -> 14.6 us, over 1000 to 2000 39.0 -> 34.2,
// 64 over 500 to 1000 67.0 -> 58.8; a prompt of 400 tokens 26.7 -> 15.4, of 1000 37.2
// -> 24.2.  Where whole items are fewer than the blocks it is not slower either (single
// calls between events, which add about 10 us, 8 heads): one request of 1000 keys
// 29.7 -> 23.6, of 2000 30.8 -> 30.7, 4 of 2000 31.7 both ways.
template <int R>
__device__ __forceinline__ int uncut(int rows)
{
    return R == 256 ? (rows <= 128 ? 16 : 8) : 0;
}

// The sequence of `total` units in at most `parts` parts of at least `least`
// units each (but for a rest).
struct Parts {
    int64_t total, per;
    int n, rem;
    __device__ __forceinline__ Parts(int64_t units, int parts, int least) : total(units)
    {
        n = (int)min((int64_t)parts, (total + least - 1) / least);
        per = n > 0 ? quot64(total, n) : 0;
        rem = (int)(total - per * n);
    }
    // first unit of part i; total for the parts behind the last one
    __device__ __forceinline__ int64_t begin(int i) const { return i >= n ? total : per * i + rem * i / n; }
    // the part that holds unit u < total
    __device__ __forceinline__ int of(int64_t u) const
    {
        int i = min(n - 1, (int)((double)u * n / (double)total));
        while (i > 0 && begin(i) > u) --i;
        while (begin(i + 1) <= u) ++i;
        return i;
    }
};

// The division of the sequence, and (in sm->place) the place of part `part`'s
// first unit; all NT threads call it.  Up to NT / 32 requests: a warp each, a lane a row tile (a
// prompt has hundreds of row tiles); more: a thread each.
template <int R, int BN, int NT>
__device__ __forceinline__ Parts plan(const PagedArgs &a, PlanSmem *sm, int part)
{
    static_assert(NT % 32 == 0 && NT <= 1024, "whole warps");
    constexpr int W = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.B <= W) {
        Request s;
        int64_t uh = 0;  // of one head of the warp's request
        if (warp < a.B) {
            s = load_request(a, warp);
            uh = warp_sum(head_units<R, BN>(a, s, lane, 32));
        }
        if (lane == 0) sm->ws[warp] = uh * a.Hkv;
        __syncthreads();
        int64_t total = 0, before = 0;
        for (int w = 0; w < W; ++w) {
            if (w == warp) before = total;
            total += sm->ws[w];
        }
        const Parts parts(total, a.parts, kLeast<R>);
        int64_t rem = parts.begin(part) - before;
        if (rem >= 0 && rem < uh * a.Hkv) {  // this warp's request holds the place
            Place p;
            p.b = warp;
            p.h = (int)quot64(rem, uh);
            rem -= p.h * uh;
            const int nt = row_tiles<R>(a, s);
            for (int q0 = 0; q0 < nt; q0 += 32) {
                int n = 0;
                if (q0 + lane < nt) {
                    const TileRange t = tile_range<R, BN>(a, s, q0 + lane);
                    n = kItemCost<R> + t.j1 - t.j0;
                }
                const int end = warp_scan(n);
                if (rem >= end - n && rem < end) {
                    p.qt = q0 + lane;
                    p.off = (int)rem - (end - n);
                    sm->place = p;
                    sm->request = s;
                }
                rem -= __shfl_sync(0xffffffffu, end, 31);
                if (rem < 0) break;
            }
        }
        __syncthreads();
        return parts;
    }
    int64_t mine = 0, sum = 0;  // the last request of this thread, all of them
    for (int b = tid; b < a.B; b += NT) {
        mine = head_units<R, BN>(a, load_request(a, b), 0, 1) * a.Hkv;
        sum += mine;
    }
    sum = warp_sum(sum);
    if (lane == 0) sm->ws[warp] = sum;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < W; ++w) total += sm->ws[w];
    __syncthreads();
    const Parts parts(total, a.parts, kLeast<R>);
    const int64_t u = parts.begin(part);
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B && base <= u; b0 += NT) {
        const int b = b0 + tid;
        const int64_t x0 = a.B <= NT ? mine : (b < a.B ? head_units<R, BN>(a, load_request(a, b), 0, 1) * a.Hkv : 0);
        int64_t x = warp_scan(x0);
        if (lane == 31) sm->ws[warp] = x;
        __syncthreads();
        int64_t chunk = 0;
        for (int w = 0; w < W; ++w) {
            if (w == warp) x += chunk;
            chunk += sm->ws[w];
        }
        x += base;
        if (u >= x - x0 && u < x) {  // this thread's request holds the place
            const Request s = load_request(a, b);
            const int64_t uh = quot64(x0, a.Hkv);
            int64_t rem = u - (x - x0);
            Place p;
            p.b = b;
            p.h = (int)quot64(rem, uh);
            rem -= p.h * uh;
            for (p.qt = 0;; ++p.qt) {
                const TileRange t = tile_range<R, BN>(a, s, p.qt);
                if (rem < kItemCost<R> + t.j1 - t.j0) break;
                rem -= kItemCost<R> + t.j1 - t.j0;
            }
            p.off = (int)rem;
            sm->place = p;
            sm->request = s;
        }
        base += chunk;
        __syncthreads();
    }
    return parts;
}

// Walk over the items of a part: the current item's piece [j0, j1) of key
// tiles, and whether the piece is the whole item.
template <int R, int BN>
struct Walk {
    const PagedArgs &a;
    Place p;
    Request s;
    int64_t first;  // the item's first unit
    int64_t left;   // units of the part from the place on
    TileRange t;    // the item
    int j0, j1;     // the piece
    bool whole, head;  // head: the piece begins with the item
    __device__ __forceinline__ Walk(const PagedArgs &args, const PlanSmem &plan, const Parts &parts, int part)
        : a(args), p(plan.place), s(plan.request), first(parts.begin(part)), left(parts.begin(part + 1) - first)
    {
        if (left > 0) {
            first -= p.off;
            set();
        }
    }
    __device__ __forceinline__ void set()
    {
        t = tile_range<R, BN>(a, s, p.qt);
        // the part's borders, in key tiles; an item that is not cut is the part's that holds its end
        const int n = t.j1 - t.j0, whole_to = n <= uncut<R>(s.n * a.group.d - p.qt * R) ? n - 1 : 0;
        const int64_t to = p.off - kItemCost<R> + left;
        j0 = t.j0 + (whole_to > 0 ? 0 : max(0, p.off - kItemCost<R>));
        j1 = to >= n ? t.j1 : t.j0 + (to <= whole_to ? 0 : (int)to);
        head = j0 == t.j0;
        whole = head && j1 == t.j1;
        if (j0 == j1) left = 0;  // the part ends before the item's first tile
    }
    __device__ __forceinline__ bool live() const { return left > 0; }
    __device__ __forceinline__ void assign(const Walk &o)
    {
        p = o.p, s = o.s, first = o.first, left = o.left, t = o.t, j0 = o.j0, j1 = o.j1, whole = o.whole, head = o.head;
    }
    __device__ __forceinline__ void next()
    {
        first += kItemCost<R> + t.j1 - t.j0;
        left -= kItemCost<R> + t.j1 - t.j0 - p.off;
        if (left <= 0) return;
        p.off = 0;
        if (++p.qt == row_tiles<R>(a, s)) {
            p.qt = 0;
            if (++p.h == a.Hkv) {
                p.h = 0;
                do {  // the sequence has `left` more units: a request with rows follows
                    if (++p.b == a.B) {
                        left = 0;
                        return;
                    }
                    s = load_request(a, p.b);
                } while (s.n == 0);
            }
        }
        set();
    }
};

// Partial of piece `piece` (0: continues an item that an earlier part began,
// 1: begins an item that a later part continues) and side (the two halves of a
// block's work on the piece, where it has two).
__device__ __forceinline__ float *part_at(const PagedArgs &a, int part, int piece, int side)
{
    return a.part + ((int64_t)((part * 2 + piece) * a.sides + side)) * a.rows_cap * kPartLd;
}

// N neighbouring channels of an output row.
template <int N>
__device__ __forceinline__ void store_out(float *p, const float (&x)[N])
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = x[i];
    }
}
template <int N>
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, const float (&x)[N])
{
    if constexpr (N == 8) {
        uint4 v;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// 16 bytes, zeros if not `real`.  (A volatile statement: a plain load would be
// moved down to its use.)
__device__ __forceinline__ float4 load_cg(const float *p, bool real)
{
    float4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w)
        : "l"(p), "r"((uint32_t)real)
        : "memory");
    return v;
}

// Join the pieces of an item, in the parts c0 .. c1:
//     m = max m_i,  l = sum l_i 2^(m_i - m),  out = sum O_i 2^(m_i - m) / l.
// A row that sees no key has l = 0 and gets zeros.  First m, l and the factors
// of the partials, with as many lanes a row as the threads allow (a decode step
// has few rows and up to hundreds of partials each), then four rows of eight
// channels a thread (four in the fp32 kernel, which has fewer registers; one with few
// rows, so that more threads share them): rows are the partials' fast dimension, a
// thread's loads are 16 bytes, and 8 to 16 of them are under way at a time.  Bound by
// the bytes that one block has in flight, by the stores (8 channels a row: 16
// bytes; 4 took 5 us more for chunks of 300 tokens), and by its code, which is cold:
// the same loops unrolled further are slower.  131072 keys and one token, 36
// partials of 4 rows: 7 us of 96; chunks of 300 tokens of 6 requests: 16 of 37.
// As a launch of its own after the attention (an earlier form): 52 instead of
// 54 us for 3 fp32 chunks, but 211 instead of 194 for 32 single tokens and 13.8
// instead of 9.0 for one short request.  The
// order of the sums is fixed, so that the result does not depend on timing.
// Called by NT threads with sync() as their barrier.
struct MergeSmem {
    float m[256], inv[256];  // of a row: maximum, 1 / sum
    float4 g[1024];          // of a partial and four rows, where they fit: 2^(m_i - m) / l
};
// The parts c0 .. c1 that hold pieces of an item; whether all others are done.
struct Pieces {
    int c0, c1, last;
};

template <int R, int BN>
__device__ __forceinline__ void find_pieces(Pieces &x, const Parts &parts, const Walk<R, BN> &w)
{
    const int64_t tile0 = w.first + kItemCost<R>;  // the unit of the item's first key tile
    x.c0 = parts.of(tile0);
    x.c1 = parts.of(tile0 + (w.t.j1 - w.t.j0) - 1);
}


template <typename T, int R, bool TWO_SIDES, int NT, typename Sync>
__device__ __forceinline__ void merge_pieces(const PagedArgs &a, MergeSmem &sm, const Pieces &x, const Request &s, const Place &p,
                                             int tid, Sync sync)
{
    static_assert(R <= NT && R <= 256, "a thread a row at least");
    const int c0 = x.c0, c1 = x.c1;
    const int rows = min(R, s.n * a.group.d - p.qt * R), quads = (rows + 3) / 4;
    const bool two_sides = TWO_SIDES && rows <= R / 2;  // the two sides hold the same rows
    const int count = (c1 - c0 + 1) * (two_sides ? 2 : 1);
    // partial i from row r on
    auto at = [&](int i, int r) {
        const int part = c0 + (two_sides ? i >> 1 : i);
        const int side = two_sides ? i & 1 : TWO_SIDES ? r / (R / 2) : 0;
        return part_at(a, part, part == c0 ? 1 : 0, side) + (TWO_SIDES && !two_sides ? r % (R / 2) : r);
    };
    const int64_t ld = a.rows_cap;
    int lanes = 32;  // of a row
    while (rows * lanes > NT) lanes >>= 1;
    const bool kept = count * quads <= 1024 && count <= 8 * lanes;
    {
        const int r = tid / lanes, i0 = tid % lanes;
        float m = -INFINITY, l = 0.f, mi[8];
        for (int ib = i0; ib < count; ib += 8 * lanes) {
            float li[8], mn = m;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = ib + u * lanes;
                mi[u] = -INFINITY, li[u] = 0.f;
                if (i < count && r < rows) mi[u] = __ldcg(at(i, r) + kD * ld), li[u] = __ldcg(at(i, r) + (kD + 1) * ld);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) mn = fmaxf(mn, mi[u]);
            const float ref = mn == -INFINITY ? 0.f : mn;
            l *= exp2f(m - ref);
#pragma unroll
            for (int u = 0; u < 8; ++u) l += li[u] * exp2f(mi[u] - ref);
            m = mn;
        }
        float top = m;
        for (int d = lanes >> 1; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == -INFINITY ? 0.f : top;
        l *= exp2f(m - ref);
        for (int d = lanes >> 1; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const float inv = l > 0.f ? 1.f / l : 0.f;
        if (r < rows) {
            if (i0 == 0) sm.m[r] = ref, sm.inv[r] = inv;
            if (kept) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int i = i0 + u * lanes;
                    if (i < count) reinterpret_cast<float *>(&sm.g[i * quads + r / 4])[r & 3] = exp2f(mi[u] - ref) * inv;
                }
            }
        }
    }
    sync();
    // N channels of four rows, from U partials at a time
    auto channels = [&](auto width, auto partials) {
        constexpr int N = decltype(width)::value, U = decltype(partials)::value;
#pragma unroll 1
        for (int k = tid; k < quads * (kD / N); k += NT) {
            const int c = k / quads * N, q = k % quads;
            float4 o[N];
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int i0 = 0; i0 < count; i0 += U) {
                float4 v[U][N], g[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = min(i0 + u, count - 1);  // (those behind the last are zeros)
                    const float *y = at(i, 4 * q);
#pragma unroll
                    for (int j = 0; j < N; ++j) v[u][j] = load_cg(y + (c + j) * ld, i0 + u < count);
                    if (kept) {
                        g[u] = sm.g[i * quads + q];
                    } else {
                        const float4 mi = __ldcg(reinterpret_cast<const float4 *>(y + kD * ld));
                        const float4 m = *reinterpret_cast<const float4 *>(sm.m + 4 * q), inv = *reinterpret_cast<const float4 *>(sm.inv + 4 * q);
                        g[u] = make_float4(exp2f(mi.x - m.x) * inv.x, exp2f(mi.y - m.y) * inv.y, exp2f(mi.z - m.z) * inv.z,
                                           exp2f(mi.w - m.w) * inv.w);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        o[j].x += v[u][j].x * g[u].x, o[j].y += v[u][j].y * g[u].y, o[j].z += v[u][j].z * g[u].z, o[j].w += v[u][j].w * g[u].w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * q + e, gr = p.qt * R + r;
                if (r >= rows) break;
                const int tok = a.group.quot(gr), g = gr - tok * a.group.d;
                float z[N];
#pragma unroll
                for (int j = 0; j < N; ++j) z[j] = e == 0 ? o[j].x : e == 1 ? o[j].y : e == 2 ? o[j].z : o[j].w;
                store_out(static_cast<T *>(a.out) + (int64_t)(s.row0 + tok) * a.o_st + (int64_t)(p.h * a.group.d + g) * a.o_sh + c, z);
            }
        }
    };
    using std::integral_constant;
    if (quads > 2) channels(integral_constant<int, R == 256 ? 8 : 4>{}, integral_constant<int, 2>{});
    else channels(integral_constant<int, 1>{}, integral_constant<int, 8>{});
}

// A piece's partial has been written by (some of) the calling NT threads: count it, and
// join the item's pieces if it was the last one.  `x` (shared) comes from
// find_pieces.  The counters are in the workspace, one a part (a part begins at
// most one item that another one ends), and are zero again when the item is
// done.
template <typename T, int R, bool TWO_SIDES, int NT, typename Sync>
__device__ __forceinline__ void finish_piece(const PagedArgs &a, MergeSmem &sm, Pieces &x, const Request &s, const Place &p,
                                             int tid, Sync sync)
{
    sync();
    if (tid == 0) {
        x.last = atom_add_acq_rel_gpu(a.tickets + x.c0, 1u) == (unsigned)(x.c1 - x.c0);
        if (x.last) a.tickets[x.c0] = 0u;
    }
    sync();
    if (x.last) merge_pieces<T, R, TWO_SIDES, NT>(a, sm, x, s, p, tid, sync);
    sync();
}

}  // namespace think
