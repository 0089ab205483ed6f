// paged_plan.cuh -- how the attention of new tokens over the paged cache is
// divided among the thread blocks, and the merge of what the division cut.
//
// Query rows: row r of request b is its new token r / G and query head r % G of
// the KV head's group, so that the G heads that share keys fill a tile
// together.  An item is (request, KV head, tile of R rows); its work, in units,
// is the number of BN-key tiles that any of its rows sees (at least 1, so that
// rows that see nothing are still written) and a fixed cost.  The items' units
// form one sequence, requests first, then heads, then row tiles; block i of P
// takes the i-th of P equal parts of it.  Whatever the mix of lengths, all blocks
// get the same work to within a unit; an item that a part's border cuts is computed in
// pieces, each piece leaves its (max, sum, O) in the workspace, and
// merge_kernel joins them in order.  Lengths stay on the device: the plan is
// recomputed from q_start and kv_lens by every launch, so that a captured
// launch follows the lengths of each replay.
#pragma once

#include "pages.cuh"
#include "ptx.cuh"

namespace think {

struct PagedArgs {
    const void *q, *k, *v;
    void *out;
    const int32_t *q_start, *kv_lens, *table;
    unsigned *status;
    float *part;  // [parts][2 pieces][sides][rows_cap][kPartLd]
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

constexpr int kPartLd = kD + 2;  // O[128], max, sum of a row

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
constexpr int kItemCost = 2;

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
        u += kItemCost + t.j1 - t.j0;
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

// Scratch of plan(): one block's.
struct PlanSmem {
    int64_t ws[33];
    Place place;
};

// The total number of units and the place of unit first(total); all NT
// threads call it.  Up to NT / 32 requests: a warp each, a lane a row tile (a
// prompt has hundreds of row tiles); more: a thread each.
template <int R, int BN, int NT, typename First>
__device__ __forceinline__ int64_t plan(const PagedArgs &a, PlanSmem *sm, First first)
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
        int64_t rem = first(total) - before;
        if (rem >= 0 && rem < uh * a.Hkv) {  // this warp's request holds the place
            Place p;
            p.b = warp;
            p.h = (int)(rem / uh);
            rem -= p.h * uh;
            const int nt = row_tiles<R>(a, s);
            for (int q0 = 0; q0 < nt; q0 += 32) {
                int n = 0;
                if (q0 + lane < nt) {
                    const TileRange t = tile_range<R, BN>(a, s, q0 + lane);
                    n = kItemCost + t.j1 - t.j0;
                }
                const int end = warp_scan(n);
                if (rem >= end - n && rem < end) {
                    p.qt = q0 + lane;
                    p.off = (int)rem - (end - n);
                    sm->place = p;
                }
                rem -= __shfl_sync(0xffffffffu, end, 31);
                if (rem < 0) break;
            }
        }
        __syncthreads();
        return total;
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
    const int64_t u = first(total);
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
            const int64_t uh = x0 / a.Hkv;
            int64_t rem = u - (x - x0);
            Place p;
            p.b = b;
            p.h = (int)(rem / uh);
            rem -= p.h * uh;
            for (p.qt = 0;; ++p.qt) {
                const TileRange t = tile_range<R, BN>(a, s, p.qt);
                if (rem < kItemCost + t.j1 - t.j0) break;
                rem -= kItemCost + t.j1 - t.j0;
            }
            p.off = (int)rem;
            sm->place = p;
        }
        base += chunk;
        __syncthreads();
    }
    return total;
}

// First unit of part `part` of the min(parts, total) parts, none of which
// is empty; total for the parts behind the last one.
__device__ __forceinline__ int64_t part_begin(int64_t total, int part, int parts)
{
    const int64_t n = min((int64_t)parts, total);
    return part >= n ? total : total / n * part + total % n * part / n;
}

// Walk over the items of a part: the current item's piece [j0, j1) of key
// tiles, and whether the piece is the whole item.
template <int R, int BN>
struct Walk {
    const PagedArgs &a;
    Place p;
    Request s;
    int64_t left;   // units of the part from the place on
    TileRange t;    // the item
    int j0, j1;     // the piece
    bool whole, head;  // head: the piece begins with the item
    __device__ __forceinline__ Walk(const PagedArgs &args, const Place &place, int64_t units) : a(args), p(place), left(units)
    {
        if (left > 0) {
            s = load_request(a, p.b);
            set();
        }
    }
    __device__ __forceinline__ void set()
    {
        t = tile_range<R, BN>(a, s, p.qt);
        j0 = t.j0 + max(0, p.off - kItemCost);
        j1 = (int)min((int64_t)t.j1, t.j0 + max((int64_t)0, p.off - kItemCost + left));
        head = j0 == t.j0;
        whole = head && j1 == t.j1;
        if (j0 == j1) left = 0;  // the part ends before the item's first tile
    }
    __device__ __forceinline__ bool live() const { return left > 0; }
    __device__ __forceinline__ void assign(const Walk &o)
    {
        p = o.p, s = o.s, left = o.left, t = o.t, j0 = o.j0, j1 = o.j1, whole = o.whole, head = o.head;
    }
    __device__ __forceinline__ void next()
    {
        left -= kItemCost + t.j1 - t.j0 - p.off;
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

template <typename T>
__device__ __forceinline__ void store_out4(T *p, float4 x);
template <>
__device__ __forceinline__ void store_out4<float>(float *p, float4 x)
{
    *reinterpret_cast<float4 *>(p) = x;
}
template <>
__device__ __forceinline__ void store_out4<__nv_bfloat16>(__nv_bfloat16 *p, float4 x)
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

// Join the pieces of the item that the border between parts c - 1 and c cuts,
// if that is the first border inside the item (blockIdx.x = c - 1; the blocks
// of one x share the rows):
//     m = max m_i,  l = sum l_i 2^(m_i - m),  out = sum O_i 2^(m_i - m) / l.
// A row that sees no key has l = 0 and gets zeros.  With fewer rows than warps
// several warps share a row's partials (a decode step has few rows and up to
// hundreds of partials each); the lanes of a warp read 32 (m, l) at once, and
// the loads of the O_i do not wait for one another.  The order of the sums is
// fixed, so that the result does not depend on timing.
constexpr int kMergeThreads = 256;
constexpr int kMergeSlices = 8;

template <typename T, int R, int BN, bool TWO_SIDES>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedArgs a)
{
    constexpr int W = kMergeThreads / 32;
    __shared__ PlanSmem sm;
    __shared__ __align__(16) float s_o[W][kD];
    __shared__ float2 s_ml[W];
    const int c = (int)blockIdx.x + 1;
    const int64_t total = plan<R, BN, kMergeThreads>(a, &sm, [&](int64_t n) { return part_begin(n, c, a.parts); });
    const int64_t u = part_begin(total, c, a.parts);
    grid_dependency_wait();  // every block waits, so that this grid ends after the attention
    if (u >= total) return;
    const Place p = sm.place;
    const int64_t start = u - p.off + kItemCost;  // the item's first key tile in the sequence
    if (u <= start || part_begin(total, c - 1, a.parts) > start) return;
    const Request s = load_request(a, p.b);
    const TileRange t = tile_range<R, BN>(a, s, p.qt);
    // the last part that holds a piece of the item: that of its last key tile
    const int64_t end = start + (t.j1 - t.j0);
    int lo = c, hi = a.parts - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (part_begin(total, mid, a.parts) < end) lo = mid;
        else hi = mid - 1;
    }
    const int rows = min(R, s.n * a.group.d - p.qt * R);
    const bool two_sides = TWO_SIDES && rows <= R / 2;  // the two sides hold the same rows
    const int count = (lo - c + 2) * (two_sides ? 2 : 1);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // rows blockIdx.y, blockIdx.y + kMergeSlices, ..., `share` warps a row
    const int mine = (rows - (int)blockIdx.y + kMergeSlices - 1) / kMergeSlices;
    const int share = mine >= W ? 1 : mine > 4 ? 1 : mine > 2 ? 2 : mine > 1 ? 4 : W;
    for (int k0 = 0; k0 < mine; k0 += W / share) {
        const int k = k0 + warp / share, r = (int)blockIdx.y + k * kMergeSlices;
        const bool real = k < mine;
        const int side0 = TWO_SIDES && !two_sides ? r / (R / 2) : 0;
        const int row = TWO_SIDES && !two_sides ? r % (R / 2) : r;
        auto partial = [&](int i) {
            const int part = c - 1 + (two_sides ? i >> 1 : i);
            return part_at(a, part, part == c - 1 ? 1 : 0, two_sides ? i & 1 : side0) + (int64_t)row * kPartLd;
        };
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (real)
            for (int i0 = warp % share; i0 < count; i0 += 32 * share) {  // partials i0, i0 + share, ...
                const int n = min(32, (count - i0 + share - 1) / share);
                float2 ml = make_float2(-INFINITY, 0.f);
                if (lane < n) ml = __ldcg(reinterpret_cast<const float2 *>(partial(i0 + lane * share) + kD));
                float mn = ml.x;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
                mn = fmaxf(mn, m);
                const float ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m - ref), g = exp2f(ml.x - ref);
                l = l * f + warp_sum(ml.y * g);
                m = mn;
                o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll 8
                for (int i = 0; i < n; ++i) {
                    const float *x = partial(i0 + i * share);
                    const float2 a0 = __ldcg(reinterpret_cast<const float2 *>(x) + 2 * lane);
                    const float2 a1 = __ldcg(reinterpret_cast<const float2 *>(x) + 2 * lane + 1);
                    const float gi = __shfl_sync(0xffffffffu, g, i);
                    o.x += a0.x * gi, o.y += a0.y * gi, o.z += a1.x * gi, o.w += a1.y * gi;
                }
            }
        if (share > 1) {  // the row's first warp adds the others' sums in order
            __syncthreads();
            *reinterpret_cast<float4 *>(&s_o[warp][4 * lane]) = o;
            if (lane == 0) s_ml[warp] = make_float2(m, l);
            __syncthreads();
            if (warp % share) continue;
            for (int w = warp + 1; w < warp + share; ++w) {
                const float2 y = s_ml[w];
                const float4 q = *reinterpret_cast<const float4 *>(&s_o[w][4 * lane]);
                const float mn = fmaxf(m, y.x), ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m - ref), g = exp2f(y.x - ref);
                o.x = o.x * f + q.x * g, o.y = o.y * f + q.y * g, o.z = o.z * f + q.z * g, o.w = o.w * f + q.w * g;
                l = l * f + y.y * g;
                m = mn;
            }
        }
        if (!real) continue;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int gr = p.qt * R + r, tok = a.group.quot(gr), g = gr - tok * a.group.d;
        store_out4(static_cast<T *>(a.out) + (int64_t)(s.row0 + tok) * a.o_st + (int64_t)(p.h * a.group.d + g) * a.o_sh + 4 * lane,
                   make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
}

}  // namespace think
