// paged_tc.cuh -- attention of new tokens over the paged cache on the
// 5th-generation tensor cores (bf16; the plan: paged_plan.cuh).
//
// Per 128-key tile, for a tile of 128 query rows (rows x keys x channels):
//     S = Q K^T         tcgen05.mma, both operands in shared memory, S in TMEM
//     P = 2^(s S - m)   one thread a row: S to registers, bf16 P back to TMEM
//     O += P V          tcgen05.mma, P from TMEM, V in shared memory as loaded
// with the running reference m and sum l of each row in its thread's registers
// (fp32).  m follows the maximum only when that has grown by more than
// 2^kLazy: until then the weights just exceed 1, which neither fp32 sums nor
// bf16 (8 significant bits at any magnitude) lose by, and O, which a new m
// rescales in TMEM, is touched a few times an item instead of every tile.
//
// P is rounded to bf16 (off by at most 2^-8 of each weight, independently): with the
// output's own rounding the result is 2.0e-3 to 2.4e-3 off (relative, 2-norm, the calls
// measured below), where the output's alone is 1.6e-3.  A second product, with what the
// first one's P leaves, brings 1.6e-3, but takes the tensor core half as long again: a prompt of
// 16384 tokens 1999 -> 2627 us, 13 requests with a window 249 -> 314, 131072 keys 100 ->
// 110, 32 single tokens 191 -> 218.  A bf16 output does not repay that; fp32 callers
// have the fp32 kernel.  Sums, maxima and O are fp32.
//
// Two softmax warpgroups t = 0, 1 work in turn, so that the tensor core runs
// one's products while the other forms its P.  An item of more than 128 query
// rows gives warpgroup t the rows 128 t .. (side by side over the same keys); an
// item of fewer (the single tokens of a decode step above all) gives both the
// same rows and warpgroup t the key tiles 2 i + t, and their (m, l, O) are
// joined at its end.
//
// Keys and values come by TMA, page by page: a load moves `chunk` rows (the
// largest power of two that divides page_size, at most 64), so that no load
// crosses a page, into a ring of 32 KB stages with the 128-byte swizzle.  A tile
// lies there as [8 rows][64-channel half][row][64 channels], so that one load
// brings both halves of a chunk: the cost of many small loads is a load's, not a
// byte's (a load a half took 207 us for the batch of single tokens below).  Chunks that no row of the item sees (and pages outside the pool) are loaded from behind the pool's end, which TMA fills with zeros.
// Value rows behind the request's last token are set to zero in shared memory
// before their product, whatever the page holds there.
//
// Warps: 8 softmax, 2 producers, 2 for the products (a warpgroup each; the first
// owns the TMEM).  TMEM columns: S_t (and P_t in its first half) at 128 t, O_t at
// 256 + 128 t.  Every wait is bounded; one that runs out sets the status bit and
// the block's abort flag, after which every wait returns at once and all warps
// still reach the final barrier, where the TMEM is released.
//
// Bound: single tokens by HBM (each key and value is read once), long chunks by
// the softmax between the two products, which share a TMEM region and hence
// alternate for a warpgroup; the other one's fill the gap.  Measured: 131072
// keys of 8 heads, one token (537 MB) 100 us = 5.4 TB/s; 32 requests of 500 to
// 16000 keys in pages of 16 (978 MB) 190 us = 5.1 TB/s; a prompt of 16384 tokens
// and 32 heads (2.2 TFLOP) 1.99 ms = 1.10 PFLOP/s, at the power cap; 13 requests
// with a window (0.21 TFLOP) 247 us.  One product warp for both warpgroups
// took 2.70 ms for the prompt, 16 softmax warps (two threads a row) 2.19,
// exponentials of a quarter of the keys by a polynomial 2.18; one producer
// warp 233 us for the batch.
#pragma once

#include "paged_plan.cuh"
#include "rope.cuh"
#include "tc05.cuh"

namespace think {

constexpr int kPtRows = 256;
constexpr int kPtBN = 128;
constexpr int kPtThreads = 384;
constexpr int kPtProducer = 8;
constexpr int kPtMma = 9;
constexpr int kPtStages = 5;
constexpr uint32_t kPtTile = 32768u;
constexpr float kPtLazy = 8.f;
constexpr int kPtFold = 256;  // key tiles of a warpgroup after which its O moves on
constexpr int kPtEarly = 96;  // keys of a tile whose P is handed over while the rest's is formed

struct PtBars {
    // A wait tells only a phase's parity, so that who waits on a barrier has to
    // see each of its phases: what both warpgroups' products use (rows split)
    // has barriers of its own, and so has what one of them uses (keys split).
    uint64_t full[3][kPtStages];  // loads: for both, for warpgroup 0, for 1
    uint64_t empty[kPtStages];
    uint64_t q_full[3];  // Q of warpgroup 0, of 1, of a split item
    uint64_t q_free[3];  // its place: of a warpgroup between items of split rows, of both around split items
    uint64_t s_full[2], o_full[2];
    uint64_t p_full[4];  // [t]: the early part of P, [2 + t]: all of it
    uint64_t turn[2];    // warpgroup t's products may go next
    uint64_t done;
    uint32_t tmem;
    uint32_t abort_flag;
};

constexpr size_t paged_tc_smem() { return 1024u + (2u + kPtStages) * (size_t)kPtTile; }

// A warp's bounded wait.  The phase has mostly completed already: one try and
// one vote; the block's abort flag is looked at only while it has not.
__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, unsigned *status,
                                        unsigned code)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag, status, code));
}

// A value that every lane holds, in a form that the compiler knows to be the
// same in all of them: the products' operands then stay in uniform registers
// (otherwise each of the 16 tcgen05.mma of a tile took about 80 cycles to
// issue, more than the 64 that it runs).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The largest of a row's 128 logits.
__device__ __forceinline__ float row_max(const uint32_t (&u)[4][32])
{
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = __uint_as_float(u[i][0]);
#pragma unroll
        for (int c = 1; c < 31; c += 2) m[i] = max3(m[i], __uint_as_float(u[i][c]), __uint_as_float(u[i][c + 1]));
        m[i] = fmaxf(m[i], __uint_as_float(u[i][31]));
    }
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// 16 bytes from global memory, zeros if not `real`.  (A volatile statement: as
// a plain load the compiler moves each one down to its use, and a row tile's 16
// loads then wait one after another, 14000 cycles instead of 2000.)
__device__ __forceinline__ uint4 load16(const void *p, bool real)
{
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)real));
    return v;
}

// One item's shape for the block's roles.
struct PtItem {
    int rows;    // query rows
    bool split;  // the key tiles are shared between the warpgroups, not the rows
    int n;       // key tiles of the piece
};
__device__ __forceinline__ PtItem pt_item(const PagedArgs &a, const Walk<kPtRows, kPtBN> &w)
{
    PtItem x;
    x.rows = min(kPtRows, w.s.n * a.group.d - w.p.qt * kPtRows);
    x.split = x.rows <= 128;
    x.n = w.j1 - w.j0;
    return x;
}

// The loads of a piece in the order in which the products use them: the first
// `ahead` key tiles, then value tile j and key tile j + ahead in turn.
struct PtOrder {
    int ahead, n;
    __device__ __forceinline__ int loads() const { return 2 * n; }
    // load i: its tile, and whether it is a value tile
    __device__ __forceinline__ int tile(int i, bool &value) const
    {
        const int first = min(ahead, n);
        if (i < first) {
            value = false;
            return i;
        }
        i -= first;
        const int pairs = n - first;  // (V_j, K_{j+ahead}) pairs
        if (i < 2 * pairs) {
            value = (i & 1) == 0;
            return value ? i / 2 : i / 2 + first;
        }
        value = true;
        return i - pairs;
    }
    // the places of key tile j and of value tile j among them
    __device__ __forceinline__ int key(int j) const
    {
        const int first = min(ahead, n);
        return j < first ? j : 2 * j - first + 1;
    }
    __device__ __forceinline__ int value(int j) const
    {
        const int first = min(ahead, n), pairs = n - first;
        return j < pairs ? first + 2 * j : first + pairs + j;
    }
};

// Where a (page, head) lies along a cache map's last dimension; `none` is behind its end.
struct PtOuter {
    int page, head, none;
};

// LONG: a block may have so many tiles of one item that its O has to move on (see
// there).  Its code costs the calls that cannot 1 to 2.5% (prompt of 16384
// tokens 1999 -> 2031 us, 131072 keys 100.5 -> 103.0), so that it is a variant.
template <bool LONG>
__global__ void __launch_bounds__(kPtThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_q, const PagedArgs a, const PtOuter outer_k,
                    const PtOuter outer_v, const int chunk, const bool tma_q)
{
    using W = Walk<kPtRows, kPtBN>;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
    __shared__ PlanSmem plan_sm;
    __shared__ PtBars bars;
    __shared__ float2 s_ml[128];  // split items: (m, l) of warpgroup 1
    __shared__ Pieces pieces;
    unsigned char *qs = smem, *ring = smem + 2 * kPtTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t *abort_flag = &bars.abort_flag;
    const uint32_t full0 = smem_addr(bars.full), empty0 = smem_addr(bars.empty), qfull0 = smem_addr(bars.q_full), qfree0 = smem_addr(bars.q_free),
                   sfull0 = smem_addr(bars.s_full), pfull0 = smem_addr(bars.p_full), ofull0 = smem_addr(bars.o_full), turn0 = smem_addr(bars.turn), done = smem_addr(&bars.done);
    if (tid == 0) {
        for (int s = 0; s < 3 * kPtStages; ++s) mbar_init(full0 + 8 * s, 2);
        for (int s = 0; s < kPtStages; ++s) mbar_init(empty0 + 8 * s, 2);
        mbar_init(qfull0 + 16, tma_q ? 1 : 8);
        mbar_init(qfree0 + 16, 8);
        for (int t = 0; t < 2; ++t) {
            mbar_init(qfull0 + 8 * t, tma_q ? 1 : 4);
            mbar_init(qfree0 + 8 * t, 4);
            mbar_init(sfull0 + 8 * t, 1);
            mbar_init(pfull0 + 8 * t, 4);
            mbar_init(pfull0 + 16 + 8 * t, 4);
            mbar_init(ofull0 + 8 * t, 1);
            mbar_init(turn0 + 8 * t, 1);
        }
        mbar_init(done, 2);
        bars.abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_q);
    }
    if (warp == kPtMma) {
        tc05::tmem_alloc(smem_addr(&bars.tmem), 512);
        tc05::tmem_relinquish();
    }
    grid_dependency_wait();
    const int part = blockIdx.x;
    const Parts parts = plan<kPtRows, kPtBN, kPtThreads>(a, &plan_sm, part);
    grid_launch_dependents();
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = bars.tmem;

    // A softmax thread holds a row of 128 logits: 384 x 168 registers at launch
    // = 256 x 216 for the softmax warps + 128 x 72 for the others.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kPtProducer || warp == kPtMma + 2) {
        // --------------------------------------------------------- producers
        // A warp half of a tile's rows, a lane a chunk: a warp's lanes issue their
        // loads one after another, and with 16-row pages a tile has 8.
        const int per_warp = kPtBN / 2 / chunk;
        const int chunk0 = lane + (warp != kPtProducer ? per_warp : 0);
        const uint32_t bytes = (uint32_t)chunk * 256u;
        uint32_t ld = 0;                     // loads issued: stage ld % kPtStages
        uint32_t phases = 0, used = 0;       // of each full barrier its next phase; of each stage the last one's set
        bool ok = true;
        for (W w(a, plan_sm, parts, part); w.live() && ok; w.next()) {
            const PtItem x = pt_item(a, w);
            const PtOrder order{x.split ? 2 : 1, x.n};
            // this lane's rows of load i: the table entry (-1: no key of them is
            // seen; read an iteration ahead, looked at when it is used) and the
            // row in the page
            auto locate = [&](int i, int &entry, int &row, bool &needed, bool &value, int &tile) {
                tile = order.tile(i, value);
                const int key = (w.j0 + tile) * kPtBN + chunk0 * chunk;
                needed = lane < per_warp && key < w.t.hi && key + chunk > w.t.lo;
                const int j = a.page.quot(key);
                row = key - j * a.page.d;
                entry = needed ? a.table[(int64_t)w.p.b * a.table_ld + j] : -1;
            };
            int entry, row, tile;
            bool needed, value;
            locate(0, entry, row, needed, value, tile);
            for (int i = 0; i < order.loads(); ++i, ++ld) {
                const int cur_entry = entry, cur_row = row, cur_tile = tile;
                const bool cur_needed = needed, cur_value = value;
                if (i + 1 < order.loads()) locate(i + 1, entry, row, needed, value, tile);
                const uint32_t s = ld % kPtStages;
                if (ld >= kPtStages)
                    ok = pt_wait(empty0 + 8 * s, ((ld / kPtStages) - 1) & 1, abort_flag, a.status, THINK_DEVICE_TIMEOUT_EMPTY);
                if (!ok) break;
                const uint32_t set = x.split ? 1u + (cur_tile & 1) : 0u, full = full0 + 8 * (set * kPtStages + s);
                phases ^= 1u << (set * kPtStages + s);
                used = (used & ~(3u << (2 * s))) | set << (2 * s);
                if (lane == 0) mbar_arrive_expect_tx(full, kPtTile / 2);
                __syncwarp();
                if (lane < per_warp) {
                    const bool inside = cur_needed && (unsigned)cur_entry < (unsigned)a.num_pages;
                    if (cur_needed && !inside) atomicOr(a.status, THINK_DEVICE_BAD_PAGE);
                    const PtOuter outer = cur_value ? outer_v : outer_k;
                    tma_load_5d(smem_addr(ring + s * kPtTile) + (uint32_t)chunk0 * bytes, cur_value ? &tm_v : &tm_k, 0, 0, 0,
                                inside ? cur_row / 8 : 0, inside ? cur_entry * outer.page + w.p.h * outer.head : outer.none,
                                full);
                }
            }
        }
        if (!ok)  // the loads in flight land before the block ends
            for (uint32_t s = 0; s < min(ld, (uint32_t)kPtStages); ++s) {
                const uint32_t b = (used >> (2 * s) & 3u) * kPtStages + s;
                mbar_wait_bounded(full0 + 8 * b, (phases >> b & 1u) ^ 1u, a.status, THINK_DEVICE_TIMEOUT_FULL);
            }
        __syncwarp();
    } else if (warp == kPtMma || warp == kPtMma + 1) {
        // ------------------------------------------------------ the products
        // One warp a softmax warpgroup t: what it issues waits for one thing
        // after another (keys, values, P), and the other warp's products run
        // meanwhile.  The two take turns, a tile's product with V and the next
        // one's logits at a time: otherwise their products would mix on the
        // tensor core and both warpgroups form their P at the same time, with
        // the tensor core idle.
        constexpr uint32_t idesc_s = tc05::idesc_bf16_f32<128, 128, false>();
        constexpr uint32_t idesc_o = tc05::idesc_bf16_f32_bmn<128, 128>();
        const int t = warp - kPtMma;
        const bool leader = elect_one();
        uint32_t base = 0;              // loads of the items before
        uint32_t items = 0, nfree = 0, nfree2 = 0;
        bool was_split = false;
        uint32_t nq = 0, nqs = 0, np = 0, nt = t ^ 1;  // items begun (rows split, keys split), P tiles taken, turns
        uint32_t phases = 0;               // of each full barrier of the two sets waited on
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t phase, unsigned code) {
            if (ok) ok = pt_wait(bar, phase & 1, abort_flag, a.status, code);
        };
        const uint64_t q_desc = tc05::smem_desc(smem_addr(qs), 16u, 1024u, tc05::kLayoutSwizzle128B);
        const uint64_t k_desc = tc05::smem_desc(smem_addr(ring), 16u, 2048u, tc05::kLayoutSwizzle128B);
        const uint64_t v_desc = tc05::smem_desc(smem_addr(ring), 1024u, 2048u, tc05::kLayoutSwizzle128B);
        const uint32_t s_tmem = uniform(tmem + 128u * t), o_tmem = s_tmem + 256u;
        const uint32_t s_bar = uniform(sfull0 + 8 * t), o_bar = uniform(ofull0 + 8 * t);
        for (W w(a, plan_sm, parts, part); w.live() && ok; w.next()) {
            const PtItem x = pt_item(a, w);
            const PtOrder order{x.split ? 2 : 1, x.n};
            const int j0 = x.split ? t : 0, step = x.split ? 2 : 1;
            // a key or value tile is released by both warps, or twice by the one that uses it
            auto release = [&](uint32_t s) {
                if (leader && ok) {
                    tc05::commit(empty0 + 8 * s);
                    if (x.split) tc05::commit(empty0 + 8 * s);
                }
            };
            // load i of the item has arrived: its stage
            auto take = [&](int i) {
                const uint32_t s = (base + i) % kPtStages, set = x.split ? 1u + t : 0u;
                const uint32_t bit = (x.split ? kPtStages : 0) + s;
                wait(full0 + 8 * (set * kPtStages + s), phases >> bit, THINK_DEVICE_TIMEOUT_FULL);
                phases ^= 1u << bit;
                return s;
            };
            auto logits = [&](uint32_t s) {  // S = Q K^T, K in stage s
                if (!ok) return;
                const uint64_t qd = q_desc + uniform(x.split ? 0u : (uint32_t)t * (kPtTile >> 4));
                const uint64_t kd = k_desc + uniform(s * (kPtTile >> 4));
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t o = (uint32_t)(ks & 3) * 32u;
                        tc05::mma_bf16(s_tmem, qd + (((uint32_t)(ks >> 2) * 16384u + o) >> 4),
                                       kd + (((uint32_t)(ks >> 2) * 1024u + o) >> 4), idesc_s, ks > 0);
                    }
                    tc05::commit(s_bar);
                }
                release(s);
            };
            auto pass = [&]() {
                if (leader) mbar_arrive(turn0 + 8 * (t ^ 1));
            };
            const uint32_t q_bar = qfull0 + (x.split ? 16 : 8 * t);
            if (tma_q) {  // bring Q: each warp its own rows, the first one those of a split item
                if (items > 0) {
                    if (x.split || was_split) wait(qfree0 + 16, nfree2++, THINK_DEVICE_TIMEOUT_EMPTY);
                    else wait(qfree0 + 8 * t, nfree++, THINK_DEVICE_TIMEOUT_EMPTY);
                }
                ++items;
                was_split = x.split;
                if (leader && ok && !(x.split && t)) {
                    const int tok = w.s.row0 + a.group.quot(w.p.qt * kPtRows + (x.split ? 0 : 128 * t));
                    const uint32_t dst = smem_addr(qs) + (x.split ? 0u : t * kPtTile);
                    mbar_arrive_expect_tx(q_bar, kPtTile);
                    tma_load_4d(dst, &tm_q, 0, w.p.h * a.group.d, tok, 0, q_bar);
                    tma_load_4d(dst + 16384u, &tm_q, 64, w.p.h * a.group.d, tok, 0, q_bar);
                }
                __syncwarp();
            }
            wait(q_bar, x.split ? nqs++ : nq++, THINK_DEVICE_TIMEOUT_FULL);
            if (j0 < x.n) {
                const uint32_t s = take(order.key(j0));
                tc05::fence_after_sync();
                logits(s);
            }
            for (int j = j0; j < x.n && ok; j += step) {  // O (+)= P V_j, then the next tile's logits
                const uint32_t s = take(order.value(j));
                if (!ok) break;
                // value rows from the request's end on are zeroed before the product
                const int from = max(0, w.s.kv - (w.j0 + j) * kPtBN);
                if (from < kPtBN) {
                    unsigned char *v = ring + s * kPtTile;
                    for (int c = lane; c < (kPtBN - from) * 16; c += 32) {
                        const int i = from + (c >> 4);
                        *reinterpret_cast<uint4 *>(v + (i >> 3) * 2048 + (c & 8) * 128 + (i & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    tc05::fence_proxy_async_smem();
                    __syncwarp();
                }
                const bool next = j + step < x.n;
                const uint32_t sk = next ? take(order.key(j + step)) : 0;
                const uint64_t vd = v_desc + uniform(s * (kPtTile >> 4));
                const bool more = uniform(j > j0) != 0;
                auto issue = [&](int k0, int k1) {
                    if (!ok) return;
                    tc05::fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int ks = k0; ks < k1; ++ks)
                            tc05::mma_bf16_ts(o_tmem, s_tmem + 8u * ks, vd + 256u * ks, idesc_o, ks > 0 || more);
                    }
                };
                wait(turn0 + 8 * t, nt++, THINK_DEVICE_TIMEOUT_FULL);
                wait(pfull0 + 8 * t, np, THINK_DEVICE_TIMEOUT_FULL);
                issue(0, kPtEarly / 16);
                wait(pfull0 + 16 + 8 * t, np, THINK_DEVICE_TIMEOUT_FULL);
                issue(kPtEarly / 16, kPtBN / 16);
                ++np;
                if (next) logits(sk);
                else if (leader && ok) tc05::commit(o_bar);
                pass();
                release(s);
            }
            if (x.split && t == 1 && (x.n & 1)) {  // the turn of a tile that there is not
                wait(turn0 + 8, nt++, THINK_DEVICE_TIMEOUT_FULL);
                pass();
            }
            base += order.loads();
        }
        // no load, product or arrival may be under way when the block ends
        if (!ok && tma_q && !(was_split && t))
            mbar_wait_bounded(qfull0 + (was_split ? 16 : 8 * t), ((was_split ? nqs : nq) - 1) & 1, a.status, THINK_DEVICE_TIMEOUT_FULL);
        if (leader) {
            tc05::commit(done);
            mbar_wait_bounded(done, 0, a.status, THINK_DEVICE_TIMEOUT_FULL);
        }
        __syncwarp();
    }
    } else {
        // ----------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int t = warp >> 2, wq = warp & 3;
        const int r = 32 * wq + lane;  // this thread's row of the tile
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t s_addr = lane_addr + 128u * t, o_addr = lane_addr + 256u + 128u * t;
        const float sl = fmaxf(fabsf(a.scale_log2), 1.0e-30f);  // a scale of 0 still sends -inf to -inf
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative one turns q
        const uint64_t sl2 = pack2(sl, sl);
        uint32_t ns = 0, no = 0, nsplit = 0;
        bool was_split = false;
        auto wait = [&](uint32_t bar, uint32_t phase) {
            pt_wait(bar, phase & 1, abort_flag, a.status, THINK_DEVICE_TIMEOUT_FULL);
        };
        // Q of an item, where its rows do not make a TMA box (see the products'
        // warps): a warpgroup's own rows, the products of whose last tile
        // have been waited for; in and around split items the rows are shared,
        // so that both warpgroups have to be there
        auto load_q = [&](const W &w) {
            const PtItem x = pt_item(a, w);
            if (x.split || was_split) named_barrier(1, 256);
            was_split = x.split;
            const int first = x.split ? 64 * t : 0, count = x.split ? 64 : 128;
            unsigned char *dst = qs + (x.split ? 0u : (uint32_t)t * kPtTile);
            const int c16 = tid & 15;
            const int i0 = first + ((tid & 127) >> 4);
            uint4 v[16];  // loads first: one latency for all rows
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int local = i0 + 8 * k + (x.split ? 0 : 128 * t);
                const int gr = w.p.qt * kPtRows + local, tok = a.group.quot(gr), g = gr - tok * a.group.d;
                v[k] = load16(static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)(w.s.row0 + tok) * a.q_st +
                                  (int64_t)(w.p.h * a.group.d + g) * a.q_sh + 8 * c16,
                              local < x.rows && 8 * k < count);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int i = i0 + 8 * k;
                v[k].x ^= flip, v[k].y ^= flip, v[k].z ^= flip, v[k].w ^= flip;
                if (8 * k < count)
                    *reinterpret_cast<uint4 *>(dst + (c16 >> 3) * 16384 + i * 128 + (((c16 & 7) ^ (i & 7)) << 4)) = v[k];
            }
            tc05::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull0 + (x.split ? 16 : 8 * t));
        };
        W w(a, plan_sm, parts, part);
        if (w.live() && !tma_q) load_q(w);
        while (w.live()) {
            const PtItem x = pt_item(a, w);
            const int base = w.s.kv - w.s.n;
            const int row = w.p.qt * kPtRows + (x.split ? r : 128 * t + r);
            const bool real = row - w.p.qt * kPtRows < x.rows;
            const bool warp_real = __any_sync(0xffffffffu, real);
            // (a row that is not real takes part as the last one of its request: what it holds is not stored)
            const int tok = a.group.quot(row);
            const int pos = base + (real ? tok : w.s.n - 1);
            if (!w.whole && tid == 0) find_pieces(pieces, parts, w);
            float m = -INFINITY, l = 0.f;
            const int step = x.split ? 2 : 1, j0 = x.split ? t : 0;
            // The tensor core's sums drop what is below their last place, always towards zero: over 200000 keys of one
            // item a sum of values of one sign lost 8e-4 to 1.2e-3.  So every kPtFold tiles O moves on: it is added, rounded
            // to nearest, to what moved on before, in the place of this piece's partial, and starts from zero; at
            // the item's end it comes back (to_end).  2.5e-4 at any length, a sixteenth of the output's half step.
            auto move = [&](bool before, bool to_end) {
                tc05::fence_after_sync();
                float *y = part_at(a, part, w.head ? 1 : 0, t) + r;  // element c of the row at y[c * rows_cap]
                const float m_moved = before && real ? y[kD * a.rows_cap] : -INFINITY;
                const float f = m_moved == -INFINITY ? 0.f : exp2_approx((m_moved - m) * sl);
                if (real && !to_end) y[kD * a.rows_cap] = m;
#pragma unroll 1
                for (int i = 0; i < 16; ++i, y += 8 * a.rows_cap) {
                    uint32_t o[8];
                    tc05::tmem_ld8(o_addr + 8u * i, o);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (f != 0.f) o[c] = __float_as_uint(__uint_as_float(o[c]) + f * y[c * a.rows_cap]);
                        if (real && !to_end) y[c * a.rows_cap] = __uint_as_float(o[c]);
                        if (!to_end) o[c] = 0u;
                    }
                    __syncwarp();
                    tc05::tmem_st8(o_addr + 8u * i, o);
                }
                tc05::tmem_st_wait();
            };
            for (int j = j0; j < x.n; j += step) {
                if (LONG && j >= kPtFold * step && (j & (kPtFold * step - 1)) == j0) {
                    wait(sfull0 + 8 * t, ns);  // (of the tile to come: the products before it are done)
                    if (warp_real) move(j >= 2 * kPtFold * step, false);
                }
                wait(sfull0 + 8 * t, ns++);
                if (warp_real) {
                    tc05::fence_after_sync();
                    uint32_t u[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc05::tmem_ld32_issue(s_addr + 32u * i, u[i]);
                    tc05::tmem_ld32_wait(u[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) tc05::tmem_ld32_keep(u[i]);
                    // the columns that this row sees: [clo, chi)
                    const int at = (w.j0 + j) * kPtBN;
                    const int chi = pos + 1 - at, clo = a.window > 0 ? pos - a.window + 1 - at : 0;
                    if (!__all_sync(0xffffffffu, chi >= kPtBN && clo <= 0)) {
#pragma unroll
                        for (int c = 0; c < kPtBN; ++c)
                            if (c >= chi || c < clo) u[c >> 5][c & 31] = 0xff800000u;  // -inf
                    }
                    // The weights are formed with the reference as it stands,
                    // beside the search for the maximum; where that has grown
                    // too much (a few times an item), they are formed again.
                    if (j == j0) m = row_max(u);
                    uint64_t sum[4];
                    uint64_t nm2;
                    auto weights = [&](int i) {  // P of the keys 32 i .. (its columns of S have been read)
                        uint32_t p[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const uint64_t z =
                                fma2(pack2(__uint_as_float(u[i][2 * c]), __uint_as_float(u[i][2 * c + 1])), sl2, nm2);
                            float p0, p1;
                            unpack2(z, p0, p1);
                            p0 = exp2_approx(p0), p1 = exp2_approx(p1);
                            sum[c & 3] = add2(sum[c & 3], pack2(p0, p1));
                            p[c] = bf16_pair(p0, p1);
                        }
                        tc05::tmem_st16(s_addr + 16u * i, p);
                    };
                    const float mx = row_max(u);
#pragma unroll 1
                    for (;;) {
                        const float nm = m == -INFINITY ? 0.f : -m * sl;
                        nm2 = pack2(nm, nm);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] = 0;
#pragma unroll
                        for (int i = 0; i < kPtEarly / 32; ++i) weights(i);
                        const bool grow = (mx - m) * sl > kPtLazy;  // NaN (both -inf): false
                        if (!__any_sync(0xffffffffu, grow)) break;
                        const float f = grow ? exp2_approx((m - mx) * sl) : 1.f;
                        if (grow) m = mx;
                        l *= f;
                        if (j > j0) {  // the products before this tile's have been waited for with S
#pragma unroll 1
                            for (int i = 0; i < 8; ++i) {
                                uint32_t o[16];
                                tc05::tmem_ld16_issue(o_addr + 16u * i, o);
                                tc05::tmem_ld_wait(o);
#pragma unroll
                                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                                tc05::tmem_st16(o_addr + 16u * i, o);
                            }
                        }
                    }
                    tc05::tmem_st_wait();
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pfull0 + 8 * t);
#pragma unroll
                    for (int i = kPtEarly / 32; i < 4; ++i) weights(i);
                    tc05::tmem_st_wait();
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pfull0 + 16 + 8 * t);
                    float s0, s1;
                    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                    l += s0 + s1;
                } else if (lane == 0) {
                    mbar_arrive(pfull0 + 8 * t);
                    mbar_arrive(pfull0 + 16 + 8 * t);
                }
            }
            const bool any = j0 < x.n;  // this warpgroup had key tiles
            // (A warpgroup without any does not run ahead of the other one: the
            // item's Q comes when both have let the one before go.)
            if (tma_q && x.split) wait(qfull0 + 16, nsplit++);
            const bool join = x.split && w.whole && x.n > 1;
            // the next item's Q, unless it needs the second Q tile while that is
            // used below: its first products then run beside this item's end
            W nx = w;
            nx.next();
            const bool late = (join || !w.whole) && nx.live() && !pt_item(a, nx).split;
            // the next item's Q may come: (with TMA) say so, or bring it
            auto next_q = [&]() {
                if (!nx.live()) return;
                if (!tma_q) {
                    load_q(nx);
                    return;
                }
                tc05::fence_proxy_async_smem();  // the scratch in the second Q tile
                __syncwarp();
                if (lane == 0) mbar_arrive(qfree0 + (x.split || pt_item(a, nx).split ? 16 : 8 * t));
            };
            if (!late) next_q();
            if (any) wait(ofull0 + 8 * t, no++);
            tc05::fence_after_sync();
            if (LONG && x.n > kPtFold * step + j0 && warp_real) move(true, true);
            auto load_o = [&](int i, uint32_t (&o)[32]) {
                if (any) {
                    tc05::tmem_ld32_issue(o_addr + 32u * i, o);
                    tc05::tmem_ld32_wait(o);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0u;
                }
            };
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)(w.s.row0 + tok) * a.o_st +
                                 (int64_t)(w.p.h * a.group.d + row - tok * a.group.d) * a.o_sh;
            auto store_o = [&](int i, const float (&o)[32], float f) {
#pragma unroll
                for (int c = 0; c < 32; c += 8)
                    *reinterpret_cast<uint4 *>(dst + 32 * i + c) =
                        make_uint4(bf16_pair(o[c] * f, o[c + 1] * f),
                                   bf16_pair(o[c + 2] * f, o[c + 3] * f),
                                   bf16_pair(o[c + 4] * f, o[c + 5] * f),
                                   bf16_pair(o[c + 6] * f, o[c + 7] * f));
            };
            if (join) {
                // warpgroup 1 hands its state over in the unused second Q tile,
                // 64 channels at a time, [channel][row]
                float *xch = reinterpret_cast<float *>(qs + kPtTile);
                if (t == 1 && warp_real) s_ml[r] = make_float2(m * sl, l);
                float f0 = 0.f, f1 = 0.f;
                for (int hh = 0; hh < 2; ++hh) {
                    if (t == 1 && warp_real)
#pragma unroll 1
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[32];
                            load_o(2 * hh + i, o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) xch[(32 * i + c) * 128 + r] = __uint_as_float(o[c]);
                        }
                    named_barrier(2, 256);
                    if (t == 0 && warp_real) {
                        if (hh == 0) {
                            const float2 y = s_ml[r];
                            const float mm = fmaxf(m * sl, y.x), ref = mm == -INFINITY ? 0.f : mm;
                            f0 = exp2_approx(m * sl - ref), f1 = exp2_approx(y.x - ref);
                            const float tot = l * f0 + y.y * f1, inv = tot > 0.f ? 1.f / tot : 0.f;
                            f0 *= inv, f1 *= inv;
                        }
#pragma unroll 1
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[32];
                            float y[32];
                            load_o(2 * hh + i, o);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                y[c] = __uint_as_float(o[c]) * f0 + xch[(32 * i + c) * 128 + r] * f1;
                            if (real) store_o(2 * hh + i, y, 1.f);
                        }
                    }
                    named_barrier(2, 256);
                }
            } else if (warp_real && (any || !w.whole)) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                float *pt = part_at(a, part, w.head ? 1 : 0, t) + r;  // element x of the row at pt[x * rows_cap]
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    load_o(i, o);
                    if (!real) continue;
                    if (w.whole) {
                        float y[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) y[c] = __uint_as_float(o[c]);
                        store_o(i, y, inv);
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) pt[(32 * i + c) * a.rows_cap] = __uint_as_float(o[c]);
                    }
                }
                if (real && !w.whole) pt[kD * a.rows_cap] = m * sl, pt[(kD + 1) * a.rows_cap] = l;
            }
            tc05::fence_before_sync();
            if (!w.whole)
                finish_piece<__nv_bfloat16, kPtRows, true, 256>(a, *reinterpret_cast<MergeSmem *>(qs + kPtTile), pieces, w.s, w.p, tid,
                                                           [] { named_barrier(2, 256); });
            if (late) next_q();
            w.assign(nx);
        }
    }

    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kPtMma) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, 512);
    }
}

}  // namespace think
