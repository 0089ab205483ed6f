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
// Two softmax warpgroups t = 0, 1 work in turn, so that the tensor core runs
// one's products while the other forms its P.  An item of more than 128 query
// rows gives warpgroup t the rows 128 t .. (side by side over the same keys); an
// item of fewer (the single tokens of a decode step above all) gives both the
// same rows and warpgroup t the key tiles 2 i + t, and their (m, l, O) are
// joined at its end.
//
// Keys and values come by TMA, page by page: a load moves `chunk` rows (the
// largest power of two that divides page_size, at most 128) of one 64-channel
// half, so that no load crosses a page, into a ring of 32 KB stages with the
// 128-byte swizzle; chunks that no row of the item sees (and pages outside the
// pool) are loaded from behind the pool's end, which TMA fills with zeros.
// Value rows behind the request's last token are set to zero in shared memory
// before their product, whatever the page holds there.
//
// Warps: 8 softmax, 1 producer (a lane a load), 1 for the products (which owns
// the TMEM), 2 idle.  TMEM columns: S_t (and P_t in its first half) at 128 t, O_t at
// 256 + 128 t.  Every wait is bounded; one that runs out sets the status bit and
// the block's abort flag, after which every wait returns at once and all warps
// still reach the final barrier, where the TMEM is released.
#pragma once

#include "paged_plan.cuh"
#include "rope.cuh"
#include "tc05.cuh"

namespace think {

constexpr int kPtRows = 256;
constexpr int kPtBN = 128;
constexpr int kPtThreads = 384;  // 12 warps: the last two only lend their registers
constexpr int kPtProducer = 8;
constexpr int kPtMma = 9;
constexpr int kPtStages = 5;
constexpr uint32_t kPtTile = 32768u;
constexpr float kPtLazy = 8.f;

struct PtBars {
    uint64_t full[kPtStages], empty[kPtStages], q_full[2], s_full[2], p_full[2], o_full[2], done;
    uint32_t tmem;
    uint32_t abort_flag;
};

constexpr size_t paged_tc_smem() { return 1024u + (2u + kPtStages) * (size_t)kPtTile; }

// One item's shape for the block's roles.
struct PtItem {
    int rows;    // query rows
    bool split;  // the key tiles are shared between the warpgroups, not the rows
    int n;       // key tiles of the piece
};
__device__ __forceinline__ PtItem pt_item(const PagedArgs &a, const Walk<kPtRows, kPtBN> &w)
{
    PtItem x;
    x.rows = min(kPtRows, w.s.n * a.G - w.p.qt * kPtRows);
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
};

__global__ void __launch_bounds__(kPtThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedArgs a,
                    const int chunk)
{
    using W = Walk<kPtRows, kPtBN>;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
    __shared__ PlanSmem plan_sm;
    __shared__ PtBars bars;
    __shared__ float2 s_ml[128];  // split items: (m, l) of warpgroup 1
    unsigned char *qs = smem, *ring = smem + 2 * kPtTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t *abort_flag = &bars.abort_flag;
    const uint32_t full0 = smem_addr(bars.full), empty0 = smem_addr(bars.empty), qfull0 = smem_addr(bars.q_full),
                   sfull0 = smem_addr(bars.s_full), pfull0 = smem_addr(bars.p_full), ofull0 = smem_addr(bars.o_full), done = smem_addr(&bars.done);
    if (tid == 0) {
        for (int s = 0; s < kPtStages; ++s) mbar_init(full0 + 8 * s, 1), mbar_init(empty0 + 8 * s, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(qfull0 + 8 * t, 4);
            mbar_init(sfull0 + 8 * t, 1);
            mbar_init(pfull0 + 8 * t, 4);
            mbar_init(ofull0 + 8 * t, 1);
        }
        mbar_init(done, 1);
        bars.abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == kPtMma) {
        tc05::tmem_alloc(smem_addr(&bars.tmem), 512);
        tc05::tmem_relinquish();
    }
    grid_dependency_wait();
    const int part = blockIdx.x;
    const int64_t total =
        plan<kPtRows, kPtBN, kPtThreads>(a, &plan_sm, [&](int64_t n) { return part_begin(n, part, a.parts); });
    grid_launch_dependents();
    const int64_t units = part_begin(total, part + 1, a.parts) - part_begin(total, part, a.parts);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = bars.tmem;
    const Place place = plan_sm.place;

    // A softmax thread holds a row of 128 logits: 384 x 168 registers at launch
    // = 256 x 208 for the softmax warps + 128 x 88 for the others.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kPtProducer) {
        // ---------------------------------------------------------- producer
        const int per_tile = kPtBN / chunk;  // loads of one 64-channel half
        const uint32_t bytes = (uint32_t)chunk * 128u;
        uint32_t ld = 0;                     // loads issued: stage ld % kPtStages
        bool ok = true;
        for (W w(a, place, units); w.live() && ok; w.next()) {
            const PtItem x = pt_item(a, w);
            const PtOrder order{x.split ? 2 : 1, x.n};
            // this lane's rows of load i: the table entry (-1: no key of them is
            // seen; read an iteration ahead, looked at when it is used) and the
            // row in the page
            auto locate = [&](int i, int &entry, int &row, bool &needed, bool &value) {
                const int key = (w.j0 + order.tile(i, value)) * kPtBN + (lane >> 1) * chunk;
                needed = (lane >> 1) < per_tile && key < w.t.hi && key + chunk > w.t.lo;
                const int j = key / a.page_size;
                row = key - j * a.page_size;
                entry = needed ? a.table[(int64_t)w.p.b * a.table_ld + j] : -1;
            };
            int entry, row;
            bool needed, value;
            locate(0, entry, row, needed, value);
            for (int i = 0; i < order.loads(); ++i, ++ld) {
                const int cur_entry = entry, cur_row = row;
                const bool cur_needed = needed, cur_value = value;
                if (i + 1 < order.loads()) locate(i + 1, entry, row, needed, value);
                const uint32_t s = ld % kPtStages, full = full0 + 8 * s;
                if (ld >= kPtStages)
                    ok = tc_wait(empty0 + 8 * s, ((ld / kPtStages) - 1) & 1, abort_flag, a.status, THINK_DEVICE_TIMEOUT_EMPTY);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, kPtTile);
                __syncwarp();
                if ((lane >> 1) < per_tile) {
                    const bool inside = cur_needed && (unsigned)cur_entry < (unsigned)a.num_pages;
                    if (cur_needed && !inside) atomicOr(a.status, THINK_DEVICE_BAD_PAGE);
                    tma_load_4d(smem_addr(ring + s * kPtTile) + (uint32_t)(lane & 1) * 16384u + (uint32_t)(lane >> 1) * bytes,
                                cur_value ? &tm_v : &tm_k, (lane & 1) * 64, inside ? cur_row : 0, w.p.h,
                                inside ? cur_entry : a.num_pages, full);
                }
            }
        }
        if (!ok)  // the loads in flight land before the block ends
            for (uint32_t i = ld > kPtStages ? ld - kPtStages : 0; i < ld; ++i)
                mbar_wait_bounded(full0 + 8 * (i % kPtStages), (i / kPtStages) & 1, a.status, THINK_DEVICE_TIMEOUT_FULL);
        __syncwarp();
    } else if (warp == kPtMma) {
        // ------------------------------------------------------ the products
        constexpr uint32_t idesc_s = tc05::idesc_bf16_f32<128, 128, false>();
        constexpr uint32_t idesc_o = tc05::idesc_bf16_f32_bmn<128, 128>();
        uint32_t ld = 0;              // loads taken
        uint32_t items = 0, np0 = 0, np1 = 0;  // items begun, P tiles taken
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t phase, unsigned code) {
            if (ok) ok = __all_sync(0xffffffffu, tc_wait(bar, phase & 1, abort_flag, a.status, code));
        };
        auto stage = [&](uint32_t i) { return smem_addr(ring + (i % kPtStages) * kPtTile); };
        auto take = [&](uint32_t i) { wait(full0 + 8 * (i % kPtStages), i / kPtStages, THINK_DEVICE_TIMEOUT_FULL); };
        auto release = [&](uint32_t i) {
            if (lane == 0 && ok) tc05::commit(empty0 + 8 * (i % kPtStages));
        };
        auto logits = [&](int t, int qt, uint32_t i) {  // S_t = Q_qt K^T
            if (!ok) return;
            tc05::fence_after_sync();
            if (lane == 0) {
                const uint32_t qa = smem_addr(qs + qt * kPtTile), kb = stage(i);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t o = (uint32_t)(ks >> 2) * 16384u + (uint32_t)(ks & 3) * 32u;
                    tc05::mma_bf16(tmem + 128u * t, tc05::smem_desc(qa + o, 16u, 1024u, tc05::kLayoutSwizzle128B),
                                   tc05::smem_desc(kb + o, 16u, 1024u, tc05::kLayoutSwizzle128B), idesc_s, ks > 0);
                }
                tc05::commit(sfull0 + 8 * t);
            }
        };
        auto values = [&](int t, uint32_t i, bool accumulate) {  // O_t (+)= P_t V
            wait(pfull0 + 8 * t, t ? np1++ : np0++, THINK_DEVICE_TIMEOUT_FULL);
            if (!ok) return;
            tc05::fence_after_sync();
            if (lane == 0) {
                const uint32_t vb = stage(i);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc05::mma_bf16_ts(tmem + 256u + 128u * t, tmem + 128u * t + 8u * ks,
                                      tc05::smem_desc(vb + 2048u * ks, 16384u, 1024u, tc05::kLayoutSwizzle128B), idesc_o,
                                      accumulate || ks > 0);
            }
        };
        // value rows from the request's end on are zeroed before their product
        auto clean = [&](uint32_t i, int jt, int kv) {
            const int from = max(0, kv - jt * kPtBN);
            if (!ok || from >= kPtBN) return;
            unsigned char *v = ring + (i % kPtStages) * kPtTile;
            for (int j = lane; j < (kPtBN - from) * 8; j += 32) {
                *reinterpret_cast<uint4 *>(v + from * 128 + j * 16) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(v + 16384 + from * 128 + j * 16) = make_uint4(0, 0, 0, 0);
            }
            tc05::fence_proxy_async_smem();
            __syncwarp();
        };
        for (W w(a, place, units); w.live() && ok; w.next(), ++items) {
            const PtItem x = pt_item(a, w);
            wait(qfull0, items, THINK_DEVICE_TIMEOUT_FULL);
            if (!x.split) {
                take(ld);
                logits(0, 0, ld);
                wait(qfull0 + 8, items, THINK_DEVICE_TIMEOUT_FULL);
                logits(1, 1, ld);
                release(ld++);
                for (int j = 0; j < x.n && ok; ++j) {
                    const uint32_t vi = ld++, ki = ld;
                    const bool more = j + 1 < x.n;
                    take(vi);
                    clean(vi, w.j0 + j, w.s.kv);
                    values(0, vi, j > 0);
                    if (more) {
                        take(ki);
                        logits(0, 0, ki);
                    } else if (lane == 0 && ok) {
                        tc05::commit(ofull0);
                    }
                    values(1, vi, j > 0);
                    release(vi);
                    if (more) {
                        logits(1, 1, ki);
                        release(ki);
                        ++ld;
                    } else if (lane == 0 && ok) {
                        tc05::commit(ofull0 + 8);
                    }
                }
            } else {
                wait(qfull0 + 8, items, THINK_DEVICE_TIMEOUT_FULL);
                for (int j = 0; j < min(2, x.n); ++j) {
                    take(ld);
                    logits(j, 0, ld);
                    release(ld++);
                }
                for (int j = 0; j < x.n && ok; ++j) {
                    const int t = j & 1;
                    take(ld);
                    clean(ld, w.j0 + j, w.s.kv);
                    values(t, ld, j > 1);
                    release(ld++);
                    if (j + 2 < x.n) {
                        take(ld);
                        logits(t, 0, ld);
                        release(ld++);
                    } else if (lane == 0 && ok) {
                        tc05::commit(ofull0 + 8 * t);
                    }
                }
            }
        }
        // no product and no arrival may be under way when the block ends
        if (lane == 0) {
            tc05::commit(done);
            mbar_wait_bounded(done, 0, a.status, THINK_DEVICE_TIMEOUT_FULL);
        }
        __syncwarp();
    }
    } else {
        // ----------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2, wq = warp & 3;
        const int r = 32 * wq + lane;  // this thread's row of the tile
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t s_addr = lane_addr + 128u * t, o_addr = lane_addr + 256u + 128u * t;
        const float sl = fmaxf(fabsf(a.scale_log2), 1.0e-30f);  // a scale of 0 still sends -inf to -inf
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative one turns q
        const uint64_t sl2 = pack2(sl, sl);
        uint32_t ns = 0, no = 0;
        bool was_split = false;
        auto wait = [&](uint32_t bar, uint32_t phase) {
            tc_wait(bar, phase & 1, abort_flag, a.status, THINK_DEVICE_TIMEOUT_FULL);
            __syncwarp();
        };
        // Q of an item: a warpgroup's own rows, the products of whose last tile
        // have been waited for; in and around split items the rows are shared,
        // so that both warpgroups have to be there
        auto load_q = [&](const W &w) {
            const PtItem x = pt_item(a, w);
            if (x.split || was_split) named_barrier(1, 256);
            was_split = x.split;
            const int first = x.split ? 64 * t : 0, count = x.split ? 64 : 128;
            unsigned char *dst = qs + (x.split ? 0u : (uint32_t)t * kPtTile);
            const int c16 = tid & 15;
            for (int i = first + ((tid & 127) >> 4); i < first + count; i += 8) {
                const int local = x.split ? i : 128 * t + i;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (local < x.rows) {
                    const int gr = w.p.qt * kPtRows + local;
                    v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                              (int64_t)(w.s.row0 + gr / a.G) * a.q_st +
                                                              (int64_t)(w.p.h * a.G + gr % a.G) * a.q_sh + 8 * c16));
                    v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
                }
                *reinterpret_cast<uint4 *>(dst + (c16 >> 3) * 16384 + i * 128 + (((c16 & 7) ^ (i & 7)) << 4)) = v;
            }
            tc05::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull0 + 8 * t);
        };
        W w(a, place, units);
        if (w.live()) load_q(w);
        while (w.live()) {
            const PtItem x = pt_item(a, w);
            const int base = w.s.kv - w.s.n;
            const int row = w.p.qt * kPtRows + (x.split ? r : 128 * t + r);
            const bool real = row - w.p.qt * kPtRows < x.rows;
            const bool warp_real = __any_sync(0xffffffffu, real);
            const int pos = real ? base + row / a.G : -1;
            float m = -INFINITY, l = 0.f;
            const int step = x.split ? 2 : 1, j0 = x.split ? t : 0;
            for (int j = j0; j < x.n; j += step) {
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
                    float mx = __uint_as_float(u[0][0]);
#pragma unroll
                    for (int c = 1; c < kPtBN; ++c) mx = fmaxf(mx, __uint_as_float(u[c >> 5][c & 31]));
                    const bool grow = (mx - m) * sl > kPtLazy;  // NaN (both -inf): false
                    if (__any_sync(0xffffffffu, grow)) {
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
                    const float nm = m == -INFINITY ? 0.f : -m * sl;
                    const uint64_t nm2 = pack2(nm, nm);
                    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t p[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const int k = 32 * i + 2 * c;
                            const uint64_t z = fma2(pack2(__uint_as_float(u[k >> 5][k & 31]),
                                                          __uint_as_float(u[k >> 5][(k & 31) + 1])), sl2, nm2);
                            float z0, z1;
                            unpack2(z, z0, z1);
                            const float p0 = exp2_approx(z0), p1 = exp2_approx(z1);
                            sum[c & 3] = add2(sum[c & 3], pack2(p0, p1));
                            const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
                            p[c] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                        tc05::tmem_st16(s_addr + 16u * i, p);
                    }
                    float s0, s1;
                    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                    l += s0 + s1;
                    tc05::tmem_st_wait();
                    tc05::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull0 + 8 * t);
            }
            const bool any = j0 < x.n;  // this warpgroup had key tiles
            const bool join = x.split && w.whole && x.n > 1;
            // the next item's Q, unless the second Q tile is used below: its
            // first products then run beside this item's end
            W nx = w;
            nx.next();
            if (!join && nx.live()) load_q(nx);
            if (any) wait(ofull0 + 8 * t, no++);
            tc05::fence_after_sync();
            auto load_o = [&](int i, uint32_t (&o)[32]) {
                if (any) {
                    tc05::tmem_ld32_issue(o_addr + 32u * i, o);
                    tc05::tmem_ld32_wait(o);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0u;
                }
            };
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)(w.s.row0 + row / a.G) * a.o_st +
                                 (int64_t)(w.p.h * a.G + row % a.G) * a.o_sh;
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
                float *pt = part_at(a, part, w.head ? 1 : 0, t) + (int64_t)r * kPartLd;
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
                        for (int c = 0; c < 32; c += 2)
                            *reinterpret_cast<float2 *>(pt + 32 * i + c) =
                                make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1]));
                    }
                }
                if (real && !w.whole) *reinterpret_cast<float2 *>(pt + kD) = make_float2(m * sl, l);
            }
            tc05::fence_before_sync();
            if (join && nx.live()) load_q(nx);
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
