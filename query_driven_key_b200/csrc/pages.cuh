// pages.cuh -- the paged cache's bookkeeping and the way out of it: block
// tables and slot maps from request lengths, and the gather of a request's
// pages into the contiguous layout that the channel pruning reads.
//
// A pool of num_pages pages of page_size token rows holds the keys (another
// the values) of every request; page block_table[b][j] of the pool holds the
// positions [j * page_size, (j + 1) * page_size) of request b, and the slot of
// a position is page * page_size + its row in the page.
#pragma once

#include "ptx.cuh"

namespace think {

constexpr int kPagesThreads = 1024, kPagesThreadsFew = 256;
constexpr int kMaxPosition = 1 << 30;  // positions and lengths stay below, so that tile arithmetic fits 32 bits

// Quotients by a divisor that a launch fixes, of dividends in [0, 2^31): the
// high word of a product with a reciprocal of 33 bits (Granlund and Montgomery,
// "Division by invariant integers using multiplication").
struct Divisor {
    int d, shift;
    uint32_t mul;
    Divisor() = default;
    explicit Divisor(int divisor) : d(divisor), shift(0)
    {
        while ((1ll << shift) < d) ++shift;
        mul = (uint32_t)((((1ull << shift) - (uint64_t)d) << 32) / (uint64_t)d + 1);
    }
    __device__ __forceinline__ int quot(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
};

struct ExtendArgs {
    const int32_t *new_lens, *free_pages, *free_count;
    const int32_t *kv_lens;
    int32_t *kv_lens_out, *free_count_out, *table, *q_start, *positions;
    int64_t *slots;
    unsigned *status;
    int64_t table_ld, T, limit;  // limit: the tokens that a table row can hold
    Divisor page;
    int B, n_free;
    bool in_place;  // an output is its own input: the blocks form a cluster
};

// Inclusive scan of one value a thread over the block (NT threads); *total receives the block's sum.  `ws` holds 33 words.
template <int NT>
__device__ __forceinline__ int64_t block_scan_i64(int64_t x, int64_t *ws, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t s = lane < NT / 32 ? ws[lane] : 0;
#pragma unroll
        for (int d = 1; d < NT / 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane < NT / 32) ws[lane] = s;
    }
    __syncthreads();
    x += warp ? ws[warp - 1] : 0;
    *total = ws[NT / 32 - 1];
    __syncthreads();
    return x;
}

// Every block scans the requests, NT at a time, and keeps their row range,
// length and place in the free stack in shared memory; then the blocks share
// the new tokens, four neighbouring ones each:
// a binary search finds the first one's request, the others follow it, and
// positions and slots leave as vectors.  A page is fresh exactly where its first
// row is a new token, so that token's thread writes the table entry, and no
// thread reads an entry that another one writes.  kv_lens and free_count may be
// the outputs themselves: the blocks are then one cluster, and every block has
// read a chunk's lengths before block 0 writes them.
// Bound by latency: a few dependent loads, two scans of ten shuffles and the
// stores.  Measured: 256 requests of one token 4.3 us, 33 prompts (40 thousand
// tokens, 0.5 MB) 6.2 us, 11 in place (8 blocks of one cluster instead of 16); an
// empty launch takes 2 to 3.  One token a thread and one block took 5.3 and 13.9.
template <int NT>
__global__ void __launch_bounds__(NT, 1) extend_pages_kernel(const ExtendArgs a)
{
    __shared__ int64_t ws[33];
    __shared__ int s_row[NT + 1];  // first row of the request, held to T
    __shared__ int s_len[NT];      // tokens before
    __shared__ int s_free[NT];     // pages handed out before it; -1: not admitted
    __shared__ int s_used;                    // pages of the admitted requests
    const int tid = threadIdx.x;
    const int rank = (int)blockIdx.x, blocks = (int)gridDim.x;
    if (tid == 0) s_used = 0;
    grid_dependency_wait();
    const int count = min(max(*a.free_count, 0), a.n_free);
    const bool vectors = (((uintptr_t)a.positions | (uintptr_t)a.slots) & 15u) == 0;
    const int T = (int)a.T;
    int64_t rows = 0, pages = 0;  // over the chunks so far
    unsigned bits = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        const bool real = b < a.B;
        const int n = real ? min(max(a.new_lens[b], 0), kMaxPosition) : 0;
        const int len = real ? min(max(a.kv_lens[b], 0), kMaxPosition) : 0;
        int64_t total, taken;
        const int64_t row_end = rows + block_scan_i64<NT>(n, ws, &total);
        // a request whose tokens do not fit its table row or the row arrays takes no page
        const bool fits = (int64_t)len + n <= a.limit && row_end <= a.T;
        const int need = fits ? a.page.quot(len + n + a.page.d - 1) - a.page.quot(len + a.page.d - 1) : 0;
        const int64_t page_end = pages + block_scan_i64<NT>(need, ws, &taken);
        const bool admitted = fits && (need == 0 || page_end <= count);
        s_row[tid] = (int)min(row_end - n, a.T);
        s_len[tid] = len;
        s_free[tid] = admitted ? (int)min(page_end - need, (int64_t)count) : -1;
        if (tid == NT - 1) s_row[NT] = (int)min(row_end, a.T);
        if (real && !admitted && n > 0) bits |= THINK_DEVICE_NO_PAGES;
        // (the admitted requests that want pages are a prefix of those that fit and want some)
        const int used = __reduce_max_sync(0xffffffffu, admitted && need > 0 ? (int)page_end : 0);
        if ((tid & 31) == 0 && used > 0) atomicMax(&s_used, used);
        if (a.in_place) cluster_sync_all();  // every block has read this chunk's lengths
        __syncthreads();
        if (rank == 0 && real) {
            a.kv_lens_out[b] = admitted ? len + n : len;
            a.q_start[b] = s_row[tid];
            if (b == a.B - 1) a.q_start[a.B] = (int32_t)min(row_end, a.T);
        }
        const int lo = s_row[0], hi = s_row[NT];
        for (int64_t g = (lo >> 2) + (int64_t)rank * NT + tid; 4 * g < hi; g += (int64_t)blocks * NT) {
            const int r0 = max(lo, (int)(4 * g)), r1 = min(hi, (int)min(4 * g + 4, (int64_t)T));
            // the last request whose first row is <= r0: it holds r0 (empty requests before it start there too)
            int l = 0, h = NT - 1;
            while (l < h) {
                const int m = (l + h + 1) >> 1;
                if (s_row[m] <= r0) l = m;
                else h = m - 1;
            }
            int pos[4];
            int64_t slot[4];
            int at_l = -1, at_j = -1, page = -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + i;
                pos[i] = 0, slot[i] = -1;
                if (r >= r1) continue;
                while (l < NT - 1 && s_row[l + 1] <= r) ++l;
                const int len0 = s_len[l];
                pos[i] = len0 + (r - s_row[l]);
                if (s_free[l] >= 0) {
                    const int j = a.page.quot(pos[i]);
                    if (l != at_l || j != at_j) {
                        const int before = a.page.quot(len0 + a.page.d - 1);
                        const int64_t at = (int64_t)(b0 + l) * a.table_ld + j;
                        if (j < before) {
                            page = a.table[at];
                        } else {
                            page = a.free_pages[count - 1 - (s_free[l] + (j - before))];
                            if (pos[i] - j * a.page.d == 0) a.table[at] = page;
                        }
                        at_l = l, at_j = j;
                    }
                    if (page >= 0) slot[i] = (int64_t)page * a.page.d + (pos[i] - j * a.page.d);
                    else bits |= THINK_DEVICE_BAD_PAGE;
                }
            }
            if (vectors && r1 - r0 == 4) {
                *reinterpret_cast<int4 *>(a.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                *reinterpret_cast<longlong2 *>(a.slots + r0) = make_longlong2(slot[0], slot[1]);
                *reinterpret_cast<longlong2 *>(a.slots + r0 + 2) = make_longlong2(slot[2], slot[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r0 + i < r1) a.positions[r0 + i] = pos[i], a.slots[r0 + i] = slot[i];
            }
        }
        rows += total;
        pages += taken;
        __syncthreads();  // the shared arrays are rewritten
    }
    // rows behind the last request
    for (int64_t r = min(rows, a.T) + (int64_t)rank * NT + tid; r < a.T; r += (int64_t)blocks * NT) {
        a.positions[r] = 0;
        a.slots[r] = -1;
    }
    if (a.in_place) cluster_sync_all();  // every block has read free_count
    else __syncthreads();
    if (rank == 0 && tid == 0) *a.free_count_out = count - s_used;
    if (bits) atomicOr(a.status, bits);
}

// Pages -> contiguous rows: out[b][h][n][:] = cache[table[b][n / page_size]][h][n % page_size][:]
// for n < kv_lens[b], zero behind it (zero keys add nothing to a channel's
// energy) and for pages outside the pool.  A copy, bound by HBM: one 16-byte
// vector a lane, kGatherRows rows a thread, all loaded before the first store.
// Measured: 131072 tokens of 8 bf16 heads (537 MB) 83.3 us = 6.45 TB/s, the rate
// of a plain copy; 5 requests of up to 1300 tokens (16 MB) 3.8 us.
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 4;

template <typename TIn>
__global__ void __launch_bounds__(kGatherThreads)
    gather_pages_kernel(const TIn *__restrict__ cache, int64_t sp, int64_t sh, int64_t sn, int num_pages, Divisor page_size,
                        const int32_t *__restrict__ table, int64_t table_ld, int max_blocks,
                        const int32_t *__restrict__ kv_lens, int Hkv, int64_t N, TIn *__restrict__ out)
{
    constexpr int VEC = 16 / sizeof(TIn);
    constexpr int LANES = kD / VEC;
    constexpr int STEP = kGatherThreads / LANES;  // rows of one vector step
    grid_dependency_wait();
    const int head = blockIdx.y, b = head / Hkv, h = head % Hkv;
    const int c = (threadIdx.x % LANES) * VEC;
    const int64_t len = min((int64_t)max(kv_lens[b], 0), (int64_t)max_blocks * page_size.d);
    const int64_t n0 = (int64_t)blockIdx.x * (STEP * kGatherRows) + threadIdx.x / LANES;
    uint4 v[kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
        const int64_t n = n0 + i * STEP;
        v[i] = make_uint4(0, 0, 0, 0);
        if (n < len && n < N) {
            const int j = page_size.quot((int)n);
            const int page = table[(int64_t)b * table_ld + j];
            if ((unsigned)page < (unsigned)num_pages)
                v[i] = *reinterpret_cast<const uint4 *>(cache + (int64_t)page * sp + (int64_t)h * sh +
                                                        (int64_t)((int)n - j * page_size.d) * sn + c);
        }
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
        const int64_t n = n0 + i * STEP;
        if (n < N) *reinterpret_cast<uint4 *>(out + ((int64_t)head * N + n) * kD + c) = v[i];
    }
}

}  // namespace think
