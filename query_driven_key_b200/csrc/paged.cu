// paged.cu -- host side of the paged cache's entry points declared in
// include/think.h: argument validation, launch planning, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <numeric>

#include "host.cuh"
#include "paged_plan.cuh"
#include "paged_tc.cuh"
#include "paged_tc32.cuh"
#include "pages.cuh"
#include "rope.cuh"
#include "think.h"

namespace think {
namespace {

constexpr size_t kPagedHeader = 256;     // status word + reserved, start of a workspace
constexpr size_t kPagedTickets = 2048;   // then the attention's counters
constexpr int kPageStep = 16;            // page sizes are multiples of 16 rows
constexpr int64_t kExtendRowsPerBlock = 4096;

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Strides of `n` leading dimensions: non-negative multiples of 16 bytes.
inline bool strides16(const int64_t *s, int n, size_t es)
{
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] % (int64_t)(16 / es) != 0) return false;
    return true;
}

// Rows that a call writes: no stride of 0 along a dimension of more than one element
// (several rows would be written to one place, in no order).
inline bool apart(const int64_t *s, std::initializer_list<int64_t> sizes)
{
    for (const int64_t n : sizes)
        if (*s++ == 0 && n > 1) return false;
    return true;
}

// A block table of B rows: its pages and the tokens that a row can hold.
think_status_t check_table(const int32_t *table, int64_t table_ld, int max_blocks, int page_size, int num_pages)
{
    if (page_size < 1 || max_blocks < 1 || num_pages < 1 || table_ld < max_blocks) return THINK_ERR_INVALID_ARG;
    if (page_size % kPageStep != 0) return THINK_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks * page_size > kMaxPosition) return THINK_ERR_UNSUPPORTED;
    if (!table) return THINK_ERR_INVALID_ARG;
    return aligned4(table) ? THINK_OK : THINK_ERR_ALIGNMENT;
}

struct PagedPlan {
    int sides;     // partials of a piece
    int rows_cap;  // rows of a partial, a multiple of 4
    size_t ws_bytes;
};

// A block an SM; bf16: items of 256 query rows in two halves, fp32: of 128.
PagedPlan plan_paged(think_dtype_t dtype, int64_t T, int G)
{
    PagedPlan p;
    p.sides = dtype == THINK_BF16 ? 2 : 1;
    p.rows_cap = (int)std::min<int64_t>(128, ceil_div(T * G, 4) * 4);
    static_assert(kPagedTickets >= kTargetSMs * sizeof(unsigned), "a counter a part");
    p.ws_bytes = kPagedHeader + kPagedTickets + sizeof(float) * (size_t)kTargetSMs * 2 * p.sides * (size_t)p.rows_cap * kPartLd;
    return p;
}

// How far a page and a head are along a cache map's last dimension, which steps by
// what divides both strides.
struct CacheSteps {
    int64_t step, page, head, n;
    CacheSteps(const PagedArgs &a, int64_t sp, int64_t sh)
    {
        step = a.num_pages == 1 ? (a.Hkv == 1 ? kD : sh) : a.Hkv == 1 ? sp : std::gcd(sp, sh);
        page = a.num_pages == 1 ? 0 : sp / step, head = a.Hkv == 1 ? 0 : sh / step;
        n = page > INT32_MAX || head > INT32_MAX ? INT64_MAX : (a.num_pages - 1) * page + (a.Hkv - 1) * head + 1;
    }
    bool ok() const { return n <= INT32_MAX; }
    PtOuter outer() const { return {(int)page, (int)head, (int)n}; }
};

// Map of a cache for loads of `chunk` rows: (64 channels, 8 rows, 2 halves, page_size
// / 8 groups of rows, (page, head)).
bool make_cache_map(CUtensorMap *m, const CacheSteps &x, const void *base, int64_t sn, int page_size, int chunk)
{
    const uint64_t dims[5] = {64, 8, 2, (uint64_t)page_size / 8, (uint64_t)x.n};
    const int64_t strides[4] = {sn, 64, 8 * sn, x.step};
    const uint32_t box[5] = {64, 8, 2, (uint32_t)chunk / 8, 1};
    return make_map(m, THINK_BF16, base, 5, dims, strides, box, true);
}

think_status_t launch_paged_tc(const PagedArgs &a, cudaStream_t st)
{
    // rows of one TMA load: the largest power of two that divides the page, at most half a tile
    const int chunk = std::min(kPtBN / 2, a.page.d & -a.page.d);
    // a tile's 128 query rows, tokens x heads of a group, as one TMA box; not if
    // the group does not divide them, a negative scale turns them on the way, or
    // the strides are none of TMA's
    const int G = a.group.d, Hq = a.Hkv * G;
    const auto fits = [](int64_t stride, int n) { return n == 1 || (stride > 0 && stride < ((int64_t)1 << 39)); };
    const bool tma_q = 128 % G == 0 && a.scale_log2 >= 0.f && fits(a.q_sh, Hq) && fits(a.q_st, a.T);
    CUtensorMap mk, mv, mq;
    const CacheSteps ks(a, a.k_sp, a.k_sh), vs(a, a.v_sp, a.v_sh);
    if (!ks.ok() || !vs.ok()) return THINK_ERR_UNSUPPORTED;
    if (!make_cache_map(&mk, ks, a.k, a.k_sn, a.page.d, chunk) || !make_cache_map(&mv, vs, a.v, a.v_sn, a.page.d, chunk))
        return THINK_ERR_CUDA;
    // (the stride of a dimension of one element is free)
    if (!tma_q) mq = mk;
    else if (!make_map_4d(&mq, THINK_BF16, a.q, kD, Hq, a.T, 1, Hq > 1 ? a.q_sh : kD, a.T > 1 ? a.q_st : kD, kD, 64, G, true, 128 / G))
        return THINK_ERR_CUDA;
    // the most key tiles of an item that a block can have: an item's, or an equal share of all items' and what is not cut
    const int64_t tiles = ceil_div(a.limit, kPtBN), items = a.Hkv * (ceil_div((int64_t)a.T * G, kPtRows) + a.B);
    const bool is_long = std::min(tiles, std::min<int64_t>(items, INT32_MAX) * (tiles + kItemCost<kPtRows>) / kTargetSMs + 17) > kPtFold;
    const auto kern = is_long ? paged_tc_kernel<true> : paged_tc_kernel<false>;
    if (!ensure_smem(reinterpret_cast<const void *>(kern), paged_tc_smem())) return THINK_ERR_CUDA;
    return launch_pdl(kern, dim3(kTargetSMs), dim3(kPtThreads), paged_tc_smem(), st, mk, mv, mq, a, ks.outer(), vs.outer(), chunk, tma_q);
}

think_status_t launch_paged_tc32(const PagedArgs &a, cudaStream_t st)
{
    if (!ensure_smem(reinterpret_cast<const void *>(&paged_tc32_kernel), kP32Smem)) return THINK_ERR_CUDA;
    return launch_pdl(paged_tc32_kernel, dim3(kTargetSMs), dim3(kP32Threads), kP32Smem, st, a);
}

template <typename T, bool NEIGHBOURS, bool ALL, int SLOTS, bool SHARED>
think_status_t launch_rope_s(const RopeArgs &a, int64_t shares, int64_t blocks, cudaStream_t st)
{
    const int groups = kRopeThreads * 16 / (kD * (int)sizeof(T));
    const int64_t rows = ceil_div(a.Hq + 2 * (int64_t)a.Hkv, shares) * a.unit;
    const size_t smem = (size_t)kRopeStages * (size_t)ceil_div(rows, groups) * kRopeThreads * 16;
    auto kern = norm_rope_append_kernel<T, NEIGHBOURS, ALL, SLOTS, SHARED>;
    if (!ensure_smem(reinterpret_cast<const void *>(kern), smem)) return THINK_ERR_CUDA;
    return launch_pdl(kern, dim3((unsigned)blocks, (unsigned)shares), dim3(kRopeThreads), smem, st, a);
}

template <typename T, bool NEIGHBOURS, bool ALL>
think_status_t launch_rope_n(RopeArgs a, cudaStream_t st)
{
    // A group of 16 (bf16) or 32 (fp32) lanes takes up to three head rows of a token, and blocks share the heads so
    // that a block's tokens times (its rows a group, and a half for the factors, which each forms) are fewest: three
    // for many tokens (8192 of 48 bf16 heads: 42.1 us, two 43.7), one for few, which are then spread over the blocks.
    // With few heads and many tokens a step takes as many tokens as fill one place, or two.
    const int groups = kRopeThreads * 16 / (kD * (int)sizeof(T));
    const int64_t heads = a.Hq + 2 * (int64_t)a.Hkv;
    int64_t shares = 1, most = 1, least = INT64_MAX;
    for (int s = 3; s > 0; --s) {
        const int64_t n = ceil_div(heads, s * groups), x = std::max<int64_t>(1, kTargetSMs * kRopeBlocksPerSM / n);
        const int64_t cost = ceil_div(a.T, x) * (2 * ceil_div(ceil_div(heads, n), groups) + 1);
        if (cost < least) least = cost, shares = n, most = x;
    }
    const auto places = [&](int64_t unit) { return ceil_div(heads * unit, groups); };
    a.unit = 1;
    for (int u = 2; u <= kRopeBatch && places(u) <= 2 && u * most <= a.T; u *= 2)
        if (u * places(a.unit) > a.unit * places(u)) a.unit = u;
    const int64_t blocks = std::min(a.T, most);
    if (a.unit > 1) return launch_rope_s<T, NEIGHBOURS, ALL, 2, true>(a, shares, blocks, st);
    if (ceil_div(heads, shares) > 2 * groups) return launch_rope_s<T, NEIGHBOURS, ALL, 3, false>(a, shares, blocks, st);
    return launch_rope_s<T, NEIGHBOURS, ALL, 2, false>(a, shares, blocks, st);
}

template <typename T>
think_status_t launch_rope(bool neighbours, const RopeArgs &a, cudaStream_t st)
{
    if (a.rot == kD) return neighbours ? launch_rope_n<T, true, true>(a, st) : launch_rope_n<T, false, true>(a, st);
    return neighbours ? launch_rope_n<T, true, false>(a, st) : launch_rope_n<T, false, false>(a, st);
}

}  // namespace
}  // namespace think

using namespace think;

extern "C" {

size_t think_extend_pages_workspace_size(void) { return kPagedHeader; }

think_status_t think_extend_pages(const int32_t *new_lens, const int32_t *kv_lens, int B, int page_size, int32_t *block_table,
                                  int64_t table_ld, int max_blocks, const int32_t *free_pages, int n_free,
                                  const int32_t *free_count, int64_t T, int32_t *kv_lens_out, int32_t *free_count_out,
                                  int32_t *q_start, int32_t *positions, int64_t *slots, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    if (B < 0 || T < 0 || n_free < 0) return THINK_ERR_INVALID_ARG;
    if (T > INT32_MAX) return THINK_ERR_UNSUPPORTED;
    if (B == 0) return THINK_OK;
    const think_status_t rc = check_table(block_table, table_ld, max_blocks, page_size, 1);
    if (rc != THINK_OK) return rc;
    if (!new_lens || !kv_lens || !free_count || !kv_lens_out || !free_count_out || !q_start || !workspace ||
        (n_free > 0 && !free_pages) || (T > 0 && (!positions || !slots)))
        return THINK_ERR_INVALID_ARG;
    if (!aligned4(new_lens) || !aligned4(kv_lens) || !aligned4(free_pages) || !aligned4(free_count) ||
        !aligned4(kv_lens_out) || !aligned4(free_count_out) || !aligned4(q_start) || !aligned4(positions) ||
        !aligned8(slots) || !aligned16(workspace))
        return THINK_ERR_ALIGNMENT;
    if (workspace_bytes < think_extend_pages_workspace_size()) return THINK_ERR_WORKSPACE;
    ExtendArgs a;
    a.new_lens = new_lens;
    a.kv_lens = kv_lens;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.kv_lens_out = kv_lens_out;
    a.free_count_out = free_count_out;
    a.table = block_table;
    a.q_start = q_start;
    a.positions = positions;
    a.slots = slots;
    a.status = static_cast<unsigned *>(workspace);
    a.table_ld = table_ld;
    a.T = T;
    a.limit = (int64_t)max_blocks * page_size;
    a.B = B;
    a.page = Divisor(page_size);
    a.n_free = n_free;
    a.in_place = kv_lens_out == kv_lens || free_count_out == free_count;
    // A decode step's few requests and rows: one small block.  Prompts: a block
    // for every 4096 rows (four a thread); at most the eight of a cluster in place.
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (B <= kPagesThreadsFew && T <= 4 * kPagesThreadsFew) {
        return launch_pdl(extend_pages_kernel<kPagesThreadsFew>, dim3(1), dim3(kPagesThreadsFew), 0, st, a);
    }
    int blocks = 1;
    while (blocks < (a.in_place ? 8 : 32) && T > blocks * kExtendRowsPerBlock) blocks *= 2;
    return launch_pdl_cluster(extend_pages_kernel<kPagesThreads>, dim3((unsigned)blocks), dim3(kPagesThreads), 0, st,
                              a.in_place ? blocks : 0, a);
}

think_status_t think_norm_rope_append(const void *q, const int64_t q_strides[2], const void *k, const int64_t k_strides[2],
                                      const void *v, const int64_t v_strides[2], int64_t T, int Hq, int Hkv, int d,
                                      think_dtype_t dtype, const void *q_weight, const void *k_weight, float eps,
                                      const double *inv_freq, int rot, int neighbours, const int32_t *positions,
                                      const int64_t *slots, void *q_out, const int64_t q_out_strides[2], void *k_cache,
                                      const int64_t k_cache_strides[3], void *v_cache, const int64_t v_cache_strides[3],
                                      int num_pages, int page_size, void *stream)
{
    if (T < 0 || Hq < 0 || Hkv < 0 || !dtype_ok(dtype)) return THINK_ERR_INVALID_ARG;
    if (d != kD) return THINK_ERR_UNSUPPORTED;
    if (T == 0 || Hq + Hkv == 0) return THINK_OK;
    if (T > INT32_MAX || Hq > 65535 || Hkv > 65535) return THINK_ERR_UNSUPPORTED;
    if (rot < 0 || rot > kD || page_size < 1 || num_pages < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return THINK_ERR_INVALID_ARG;
    if (rot % 16 != 0 || page_size % kPageStep != 0) return THINK_ERR_UNSUPPORTED;
    if ((Hq > 0 && (!q || !q_strides || !q_out || !q_out_strides)) || (rot > 0 && !inv_freq) || !positions || !slots)
        return THINK_ERR_INVALID_ARG;
    if (Hkv > 0 && (!k || !k_strides || !v || !v_strides || !k_cache || !k_cache_strides || !v_cache || !v_cache_strides))
        return THINK_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(q_weight) || !aligned16(k_weight) || !aligned8(inv_freq) || !aligned4(positions) || !aligned8(slots))
        return THINK_ERR_ALIGNMENT;
    if ((Hq > 0 && (!strides16(q_strides, 2, es) || !strides16(q_out_strides, 2, es))) ||
        (Hkv > 0 && (!strides16(k_strides, 2, es) || !strides16(v_strides, 2, es) || !strides16(k_cache_strides, 3, es) ||
                     !strides16(v_cache_strides, 3, es))))
        return THINK_ERR_ALIGNMENT;
    if ((Hq > 0 && !apart(q_out_strides, {T, Hq})) ||
        (Hkv > 0 && (!apart(k_cache_strides, {num_pages, Hkv, page_size}) || !apart(v_cache_strides, {num_pages, Hkv, page_size}))))
        return THINK_ERR_INVALID_ARG;
    RopeArgs a = {};
    a.q = q, a.k = k, a.v = v, a.wq = q_weight, a.wk = k_weight;
    a.q_out = q_out, a.k_cache = k_cache, a.v_cache = v_cache;
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.slots = slots;
    if (Hq > 0) a.q_st = q_strides[0], a.q_sh = q_strides[1], a.qo_st = q_out_strides[0], a.qo_sh = q_out_strides[1];
    if (Hkv > 0) {
        a.k_st = k_strides[0], a.k_sh = k_strides[1], a.v_st = v_strides[0], a.v_sh = v_strides[1];
        a.kc_sp = k_cache_strides[0], a.kc_sh = k_cache_strides[1], a.kc_sn = k_cache_strides[2];
        a.vc_sp = v_cache_strides[0], a.vc_sh = v_cache_strides[1], a.vc_sn = v_cache_strides[2];
    }
    a.num_slots = (int64_t)num_pages * page_size;
    a.T = T;
    a.Hq = Hq, a.Hkv = Hkv, a.rot = rot, a.page_size = page_size;
    a.eps = eps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == THINK_BF16 ? launch_rope<__nv_bfloat16>(neighbours != 0, a, st) : launch_rope<float>(neighbours != 0, a, st);
}

size_t think_paged_attn_workspace_size(int64_t T, int Hq, int Hkv, int d, think_dtype_t dtype)
{
    if (T < 0 || Hkv <= 0 || Hq < Hkv || Hq % Hkv != 0 || d != kD || !dtype_ok(dtype)) return 0;
    return plan_paged(dtype, T, Hq / Hkv).ws_bytes;
}

think_status_t think_paged_attn(const void *q, const int64_t q_strides[2], const void *k_cache,
                                const int64_t k_cache_strides[3], const void *v_cache, const int64_t v_cache_strides[3],
                                int num_pages, int page_size, const int32_t *block_table, int64_t table_ld, int max_blocks,
                                const int32_t *q_start, const int32_t *kv_lens, int B, int64_t T, int max_new, int Hq,
                                int Hkv, int d, think_dtype_t dtype, float scale, int window, void *out,
                                const int64_t out_strides[2], void *workspace, size_t workspace_bytes, void *stream)
{
    if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || window < 0 || max_new < 0 || !dtype_ok(dtype)) return THINK_ERR_INVALID_ARG;
    if (d != kD) return THINK_ERR_UNSUPPORTED;
    if (B == 0 || T == 0 || Hkv == 0) return THINK_OK;
    if (Hq < Hkv || Hq % Hkv != 0 || !std::isfinite(scale * 1.44269504088896341f)) return THINK_ERR_INVALID_ARG;
    const int G = Hq / Hkv;
    if (Hkv > 65535 || G > 4096 || T > INT32_MAX || T * G > INT32_MAX - 4096) return THINK_ERR_UNSUPPORTED;
    const think_status_t rc = check_table(block_table, table_ld, max_blocks, page_size, num_pages);
    if (rc != THINK_OK) return rc;
    if (!q || !q_strides || !k_cache || !k_cache_strides || !v_cache || !v_cache_strides || !q_start || !kv_lens || !out ||
        !out_strides || !workspace)
        return THINK_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
        !aligned4(q_start) || !aligned4(kv_lens) || !strides16(q_strides, 2, es) || !strides16(out_strides, 2, es) ||
        !strides16(k_cache_strides, 3, es) || !strides16(v_cache_strides, 3, es))
        return THINK_ERR_ALIGNMENT;
    if (!apart(out_strides, {T, Hq})) return THINK_ERR_INVALID_ARG;
    for (const int64_t *c : {k_cache_strides, v_cache_strides})  // TMA: strides (eight rows' too) above 0 and below 2^40 bytes
        for (int i = 0; i < 3; ++i) {
            if (c[i] == 0 && (i == 0 ? num_pages : i == 1 ? Hkv : page_size) > 1) return THINK_ERR_INVALID_ARG;
            if (c[i] >= ((int64_t)1 << (i < 2 ? 40 : 37)) / (int64_t)es) return THINK_ERR_UNSUPPORTED;
        }
    const PagedPlan p = plan_paged(dtype, T, G);
    if (workspace_bytes < p.ws_bytes) return THINK_ERR_WORKSPACE;
    PagedArgs a = {};
    a.q = q, a.k = k_cache, a.v = v_cache, a.out = out;
    a.q_start = q_start, a.kv_lens = kv_lens, a.table = block_table;
    a.status = static_cast<unsigned *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kPagedHeader + kPagedTickets);
    a.tickets = reinterpret_cast<unsigned *>(static_cast<unsigned char *>(workspace) + kPagedHeader);
    a.q_st = q_strides[0], a.q_sh = q_strides[1], a.o_st = out_strides[0], a.o_sh = out_strides[1];
    // the stride of a dimension of one element is free
    a.k_sp = num_pages > 1 ? k_cache_strides[0] : kD, a.k_sh = Hkv > 1 ? k_cache_strides[1] : kD, a.k_sn = k_cache_strides[2];
    a.v_sp = num_pages > 1 ? v_cache_strides[0] : kD, a.v_sh = Hkv > 1 ? v_cache_strides[1] : kD, a.v_sn = v_cache_strides[2];
    a.table_ld = table_ld;
    a.B = B, a.T = (int)T, a.Hkv = Hkv, a.group = Divisor(G), a.page = Divisor(page_size);
    a.num_pages = num_pages, a.limit = max_blocks * page_size;
    a.window = window < kMaxPosition ? window : 0;  // (every key is within such a window)
    a.rows_cap = p.rows_cap, a.parts = kTargetSMs, a.sides = p.sides;
    a.scale_log2 = scale * 1.44269504088896341f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == THINK_BF16 ? launch_paged_tc(a, st) : launch_paged_tc32(a, st);
}

think_status_t think_gather_pages(const void *cache, const int64_t cache_strides[3], int num_pages, int page_size,
                                  const int32_t *block_table, int64_t table_ld, int max_blocks, const int32_t *kv_lens,
                                  int B, int Hkv, int64_t N, int d, think_dtype_t dtype, void *out, void *stream)
{
    if (B < 0 || Hkv < 0 || N < 0 || !dtype_ok(dtype)) return THINK_ERR_INVALID_ARG;
    if (d != kD) return THINK_ERR_UNSUPPORTED;
    if (B == 0 || Hkv == 0 || N == 0) return THINK_OK;
    const int64_t heads = (int64_t)B * Hkv;
    if (heads > 65535 || N > kMaxPosition) return THINK_ERR_UNSUPPORTED;
    const think_status_t rc = check_table(block_table, table_ld, max_blocks, page_size, num_pages);
    if (rc != THINK_OK) return rc;
    if (!cache || !cache_strides || !kv_lens || !out) return THINK_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    if (!aligned16(cache) || !aligned16(out) || !aligned4(kv_lens) || !strides16(cache_strides, 3, es)) return THINK_ERR_ALIGNMENT;
    const int rows = kGatherThreads / (kD / (int)(16 / es)) * kGatherRows;
    const dim3 grid((unsigned)ceil_div(N, rows), (unsigned)heads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == THINK_BF16)
        return launch_pdl(gather_pages_kernel<__nv_bfloat16>, grid, dim3(kGatherThreads), 0, st,
                          static_cast<const __nv_bfloat16 *>(cache), cache_strides[0], cache_strides[1], cache_strides[2],
                          num_pages, Divisor(page_size), block_table, table_ld, max_blocks, kv_lens, Hkv, N,
                          static_cast<__nv_bfloat16 *>(out));
    return launch_pdl(gather_pages_kernel<float>, grid, dim3(kGatherThreads), 0, st, static_cast<const float *>(cache),
                      cache_strides[0], cache_strides[1], cache_strides[2], num_pages, Divisor(page_size), block_table, table_ld,
                      max_blocks, kv_lens, Hkv, N, static_cast<float *>(out));
}

}  // extern "C"
