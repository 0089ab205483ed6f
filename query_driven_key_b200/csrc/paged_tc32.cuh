// paged_tc32.cuh -- attention of new tokens over the paged cache in fp32 on the
// 5th-generation tensor cores (the plan: paged_plan.cuh).
//
// An fp32 number is the sum of three bf16 ones to its last bit or so: x = x0 +
// x1 + x2, each the rounding of what the ones before it leave (8 significant
// bits each).  A product of two such sums, without the terms below 2^-24 of
// it, is
//     x0 y2 + x2 y0 + x1 y1 + x0 y1 + x1 y0 + x0 y0,
// six bf16 products with fp32 sums, added from the smallest on.  The tensor
// core's sums drop what is below their last place, up to two units a step and
// always towards zero, so that a sum over a long item would lose in
// proportion to its steps (1.6e-4 over 40000 keys of one sign in one block).  A
// tile's O is therefore a sum of its own, of 4 steps with the large terms, and
// the softmax threads add it, rounded to nearest, to the item's O in another part
// of TMEM, beside the next logits' products: 6e-7 over those 40000 keys, 3e-7 over
// 131072 keys of 8 heads shared by all blocks (plain fp32: 2e-7 to 1.5e-6), for
// 4% of the time there and none for short chunks.  Both products
// of the attention are formed that way, at a sixth of the bf16
// rate, which is several times the rate of the FMA pipes:
//     S = Q K^T      128 query rows x 64 keys; the parts of Q, K in shared memory
//     P = 2^(s S - m) and its three parts: one thread a row, to TMEM
//     O_j = P V      the parts of P in TMEM, those of V in shared memory
//     O = f (O + O_j)    f: 2^(old m - new m)
// with the running reference m and sum l as in the bf16 kernel (m follows the
// maximum when that has grown by more than 2^kPtLazy).
//
// Warps: 4 softmax (a thread a query row), 4 that bring keys and 4 values, with
// the queries (one row of 128 channels a warp at a time: loaded into registers a
// tile ahead, split, and stored in the layouts of the products with the
// 128-byte swizzle; rows that no query of the item sees are zeros, whatever
// the page holds), 1 for the products.  Shared memory holds one tile of keys
// and one of values (48 KB each with their parts) beside the queries (96 KB);
// logits have two buffers in TMEM, so that the next tile's run beside this one's
// softmax.  Long items are bound by the products, 72 a tile, about 4100 cycles, whatever
// the rows (131072 keys of 8 heads, one token: 436 us, where HBM would take 166); short
// ones by an item's start and end, a tile's chain from logits to O, which only the
// next tile's logits overlap, and joins (the tensor pipe is active 17% of the chunks' time).  Measured:
// 3 chunks of 90 to 400 tokens over up to 2900 keys, 8 heads (1.5 GFLOP) 52.7 us;
// on the FMA pipes with cp.async 102, and 61 without warps of their own for the
// keys' and the values' parts.
// Every wait is bounded, as in the bf16 kernel.
#pragma once

#include "paged_tc.cuh"

namespace think {

constexpr int kP32Rows = 128;
constexpr int kP32BN = 64;
constexpr int kP32Softmax = 128;  // threads
constexpr int kP32Bring = 256;
constexpr int kP32Threads = kP32Softmax + kP32Bring + 32;
constexpr int kP32Mma = (kP32Softmax + kP32Bring) / 32;
constexpr uint32_t kP32QPart = 32768u;   // one part of Q: [2 channel halves][128 rows][128 B]
constexpr uint32_t kP32KPart = 16384u;   // one part of a tile of K or V: [2][64][128 B]
constexpr size_t kP32Smem = 1024u + 3u * kP32QPart + 6u * kP32KPart;

struct P32Bars {
    uint64_t q_full, q_empty, k_full, k_empty, v_full, p_full, pv_done, s_full[2], done;
    uint32_t tmem;
    uint32_t abort_flag;
};

// Two numbers as a pair of bf16, the largest bf16 number in place of one that would
// round to infinity.
__device__ __forceinline__ uint32_t bf16_pair_finite(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The three parts of two numbers, each as a pair of bf16.  (fp32 numbers beyond the
// largest bf16 one leave a remainder for the second part like others; an
// infinity leaves infinities, and NaN as the third part.)
__device__ __forceinline__ void split3(float a, float b, uint32_t (&w)[3])
{
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        w[p] = p == 0 ? bf16_pair_finite(a, b) : bf16_pair(a, b);
        a -= bf16lo(w[p]);
        b -= bf16hi(w[p]);
    }
}

// The products' terms, smallest first: the parts of the left and of the right factor.
__device__ __forceinline__ int term_left(int i) { return (0x021010 >> (4 * (5 - i))) & 15; }   // 0 2 1 0 1 0
__device__ __forceinline__ int term_right(int i) { return (0x201100 >> (4 * (5 - i))) & 15; }  // 2 0 1 1 0 0

__global__ void __launch_bounds__(kP32Threads, 1) paged_tc32_kernel(const PagedArgs a)
{
    using W = Walk<kP32Rows, kP32BN>;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char *qs = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
    unsigned char *ks = qs + 3 * kP32QPart, *vs = ks + 3 * kP32KPart;
    __shared__ PlanSmem plan_sm;
    __shared__ P32Bars bars;
    __shared__ MergeSmem merge_sm;
    __shared__ Pieces pieces;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t *abort_flag = &bars.abort_flag;
    const uint32_t q_full = smem_addr(&bars.q_full), q_empty = smem_addr(&bars.q_empty), k_full = smem_addr(&bars.k_full),
                   k_empty = smem_addr(&bars.k_empty), v_full = smem_addr(&bars.v_full), p_full = smem_addr(&bars.p_full),
                   pv_done = smem_addr(&bars.pv_done), s_full = smem_addr(bars.s_full), done = smem_addr(&bars.done);
    if (tid == 0) {
        mbar_init(q_full, kP32Bring / 32);
        mbar_init(k_full, kP32Bring / 64);
        mbar_init(v_full, kP32Bring / 64);
        mbar_init(p_full, kP32Softmax / 32);
        mbar_init(q_empty, 1);
        mbar_init(k_empty, 1);
        mbar_init(pv_done, 1);
        mbar_init(s_full, 1);
        mbar_init(s_full + 8, 1);
        mbar_init(done, 1);
        bars.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kP32Mma) {
        tc05::tmem_alloc(smem_addr(&bars.tmem), 512);
        tc05::tmem_relinquish();
    }
    grid_dependency_wait();
    const int part = blockIdx.x;
    const Parts parts = plan<kP32Rows, kP32BN, kP32Threads>(a, &plan_sm, part);
    grid_launch_dependents();
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = bars.tmem;  // S 0 .. 127 (two buffers), a tile's O 128 .. 255, P 256 .. 351 (three parts), the item's O 352 .. 479
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t phase) {  // false from the first wait that runs out on
        if (ok) ok = pt_wait(bar, phase & 1, abort_flag, a.status, THINK_DEVICE_TIMEOUT_FULL);
        return ok;
    };

    // A part's last piece is counted, and its item joined, by the bringing
    // warps too, which have nothing left to bring.
    auto finish_last = [&](const Request &s, const Place &p) {
        constexpr int NT = kP32Softmax + kP32Bring;
        finish_piece<float, kP32Rows, false, NT>(a, merge_sm, pieces, s, p, tid, [] { named_barrier(2, NT); });
    };

    if (warp == kP32Mma) {
        // ------------------------------------------------------ the products
        constexpr uint32_t idesc_s = tc05::idesc_bf16_f32<128, 64, false>();
        constexpr uint32_t idesc_o = tc05::idesc_bf16_f32_bmn<128, 128>();
        const bool leader = elect_one();
        const uint64_t q_desc = tc05::smem_desc(smem_addr(qs), 16u, 1024u, tc05::kLayoutSwizzle128B);
        const uint64_t k_desc = tc05::smem_desc(smem_addr(ks), 16u, 1024u, tc05::kLayoutSwizzle128B);
        const uint64_t v_desc = tc05::smem_desc(smem_addr(vs), kP32KPart / 2, 1024u, tc05::kLayoutSwizzle128B);
        uint32_t items = 0, nk = 0, nv = 0;  // items begun, key tiles and value tiles taken
        for (W w(a, plan_sm, parts, part); w.live() && ok; w.next(), ++items) {
            const int n = w.j1 - w.j0;
            auto logits = [&](int j) {  // S = Q K_j^T
                if (!wait(k_full, nk)) return;
                tc05::fence_after_sync();
                const uint32_t d = uniform(tmem + 64u * (nk & 1)), bar = uniform(s_full + 8 * (nk & 1));
                ++nk;
                if (leader) {
#pragma unroll
                    for (int i = 0; i < 6; ++i)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t oq = (uint32_t)term_left(i) * kP32QPart + (uint32_t)(k >> 2) * (kP32QPart / 2) + (k & 3) * 32u;
                            const uint32_t ok_ = (uint32_t)term_right(i) * kP32KPart + (uint32_t)(k >> 2) * (kP32KPart / 2) + (k & 3) * 32u;
                            tc05::mma_bf16(d, q_desc + (oq >> 4), k_desc + (ok_ >> 4), idesc_s, i > 0 || k > 0);
                        }
                    tc05::commit(bar);
                    tc05::commit(k_empty);
                    if (j + 1 == n) tc05::commit(q_empty);
                }
            };
            wait(q_full, items);
            logits(0);
            for (int j = 0; j < n && ok; ++j) {
                if (j + 1 < n) logits(j + 1);
                wait(v_full, nv);
                if (!wait(p_full, nv)) break;
                ++nv;
                tc05::fence_after_sync();
                if (leader) {  // O = P V_j
#pragma unroll
                    for (int i = 0; i < 6; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc05::mma_bf16_ts(tmem + 128u, tmem + 256u + 32u * term_left(i) + 8u * k,
                                              v_desc + (((uint32_t)term_right(i) * kP32KPart + 2048u * k) >> 4), idesc_o,
                                              i > 0 || k > 0);
                    tc05::commit(pv_done);
                }
            }
        }
        if (leader) {  // no product and no arrival may be under way when the block ends
            tc05::commit(done);
            mbar_wait_bounded(done, 0, a.status, THINK_DEVICE_TIMEOUT_FULL);
        }
        __syncwarp();
    } else if (warp >= kP32Softmax / 32) {
        // ------------------------------------------- keys, values and queries
        // Warps 0 .. 3 bring keys, 4 .. 7 values, each at its own pace; queries
        // all of them.
        const int bw = warp - kP32Softmax / 32;
        const bool keys = bw < kP32Bring / 64;
        const float flip = a.scale_log2 < 0.f ? -1.f : 1.f;  // a negative scale turns q
        // channels 4 lane .. of a row go to 8 bytes of its line in half lane / 16
        auto put = [&](unsigned char *base, uint32_t part_bytes, int row, uint4 v, float sign) {
            uint32_t lo[3], hi[3];
            split3(sign * __uint_as_float(v.x), sign * __uint_as_float(v.y), lo);
            split3(sign * __uint_as_float(v.z), sign * __uint_as_float(v.w), hi);
            unsigned char *p = base + (lane >> 4) * (part_bytes / 2) + row * 128 + ((((lane & 15) >> 1) ^ (row & 7)) << 4) + (lane & 1) * 8;
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(p + i * part_bytes) = make_uint2(lo[i], hi[i]);
        };
        auto hand_over = [&](uint32_t bar) {
            tc05::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        const float *pool = static_cast<const float *>(keys ? a.k : a.v) + 4 * lane;
        const int64_t sp = keys ? a.k_sp : a.v_sp, sh = keys ? a.k_sh : a.v_sh, sn = keys ? a.k_sn : a.v_sn;
        unsigned char *tile = keys ? ks : vs;
        const uint32_t full = keys ? k_full : v_full, empty = keys ? k_empty : pv_done;
        const int r0 = bw & 3;  // this warp's rows r0 + 4 i of a tile: lane i looks row i up
        uint32_t items = 0, g = 0;  // items begun, tiles stored
        bool cut = false;           // the part ends inside an item: this one
        Request cut_s;
        Place cut_p;
        for (W w(a, plan_sm, parts, part); w.live(); w.next(), ++items) {
            cut = !w.whole, cut_s = w.s, cut_p = w.p;
            uint4 x[16];
            auto load = [&](int jt) {
                const int key = jt * kP32BN + r0 + 4 * (lane & 15);
                int page = -1, row = 0;
                if (key >= w.t.lo && key < w.t.hi) {
                    const int j = a.page.quot(key);
                    page = a.table[(int64_t)w.p.b * a.table_ld + j];
                    row = key - j * a.page.d;
                    if ((unsigned)page >= (unsigned)a.num_pages) {
                        page = -1;
                        atomicOr(a.status, THINK_DEVICE_BAD_PAGE);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int p = __shfl_sync(0xffffffffu, page, i), r = __shfl_sync(0xffffffffu, row, i);
                    x[i] = load16(pool + (p >= 0 ? p * sp + w.p.h * sh + r * sn : 0), p >= 0);
                }
            };
            load(w.j0);
            const int rows = min(kP32Rows, w.s.n * a.group.d - w.p.qt * kP32Rows);
            if (items > 0) wait(q_empty, items - 1);
#pragma unroll 1
            for (int q0 = bw; q0 < kP32Rows; q0 += 32) {  // four rows of queries at a time
                uint4 y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = q0 + 8 * i, gr = w.p.qt * kP32Rows + r, tok = a.group.quot(gr);
                    y[i] = load16(static_cast<const float *>(a.q) + 4 * lane +
                                      (r < rows ? (int64_t)(w.s.row0 + tok) * a.q_st +
                                                      (int64_t)(w.p.h * a.group.d + gr - tok * a.group.d) * a.q_sh
                                                : 0),
                                  r < rows);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) put(qs, kP32QPart, q0 + 8 * i, y[i], flip);
            }
            hand_over(q_full);
            for (int jt = w.j0; jt < w.j1; ++jt, ++g) {
                if (g > 0) wait(empty, g - 1);
#pragma unroll
                for (int i = 0; i < 16; ++i) put(tile, kP32KPart, r0 + 4 * i, x[i], 1.f);
                hand_over(full);
                if (jt + 1 < w.j1) load(jt + 1);
            }
        }
        if (cut) finish_last(cut_s, cut_p);
    } else {
        // ----------------------------------------------------------- softmax
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * warp) << 16), o_addr = lane_addr + 128u, p_addr = lane_addr + 256u,
                       sum_addr = lane_addr + 352u;
        const float sl = fmaxf(fabsf(a.scale_log2), 1.0e-30f);  // a scale of 0 still sends -inf to -inf
        uint32_t g = 0;  // tiles of the part
        for (W w(a, plan_sm, parts, part); w.live(); w.next()) {
            const int rows = min(kP32Rows, w.s.n * a.group.d - w.p.qt * kP32Rows);
            const int row = w.p.qt * kP32Rows + tid, tok = a.group.quot(row);
            const bool real = tid < rows;
            const bool warp_real = __any_sync(0xffffffffu, real);
            // (a row that is not real takes part as the last one of its request: what it holds is not stored)
            const int pos = w.s.kv - w.s.n + (real ? tok : w.s.n - 1);
            if (!w.whole && tid == 0) find_pieces(pieces, parts, w);
            float m = -INFINITY, l = 0.f;
            // channels 16 i .. of O: the last tile's, added to those of the tiles before where there are any
            auto item_o = [&](int i, bool more, uint32_t (&o)[16]) {
                tc05::tmem_ld16_issue(o_addr + 16u * i, o);
                if (more) {
                    uint32_t x[16];
                    tc05::tmem_ld16_issue(sum_addr + 16u * i, x);
                    tc05::tmem_ld_wait(x);
                    tc05::tmem_ld_wait(o);
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(x[c]));
                } else {
                    tc05::tmem_ld_wait(o);
                }
            };
            for (int jt = w.j0; jt < w.j1; ++jt, ++g) {
                wait(s_full + 8 * (g & 1), g >> 1);
                if (warp_real) {
                    tc05::fence_after_sync();
                    uint32_t u[2][32];
                    tc05::tmem_ld32_issue(lane_addr + 64u * (g & 1), u[0]);
                    tc05::tmem_ld32_issue(lane_addr + 64u * (g & 1) + 32u, u[1]);
                    tc05::tmem_ld32_wait(u[0]);
                    tc05::tmem_ld32_keep(u[1]);
                    const int at = jt * kP32BN;
                    const int chi = pos + 1 - at, clo = a.window > 0 ? pos - a.window + 1 - at : 0;
                    if (!__all_sync(0xffffffffu, chi >= kP32BN && clo <= 0)) {
#pragma unroll
                        for (int c = 0; c < kP32BN; ++c)
                            if (c >= chi || c < clo) u[c >> 5][c & 31] = 0xff800000u;  // -inf
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mx[i] = __uint_as_float(u[i >> 1][16 * (i & 1)]);
#pragma unroll
                        for (int c = 1; c < 16; ++c) mx[i] = fmaxf(mx[i], __uint_as_float(u[i >> 1][16 * (i & 1) + c]));
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool grow = (top - m) * sl > kPtLazy;  // NaN (both -inf): false
                    const float f = grow ? exp2_approx((m - top) * sl) : 1.f;
                    if (grow) m = top;
                    l *= f;
                    const float nm = m == -INFINITY ? 0.f : -m * sl;
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kP32BN; ++c) {
                        const float p = exp2_approx(fmaf(__uint_as_float(u[c >> 5][c & 31]), sl, nm));
                        s[c & 3] += p;
                        u[c >> 5][c & 31] = __float_as_uint(p);
                    }
                    l += (s[0] + s[1]) + (s[2] + s[3]);
                    if (g > 0) wait(pv_done, g - 1);  // P and O are free
                    tc05::fence_after_sync();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t p[3][16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            uint32_t x[3];
                            split3(__uint_as_float(u[i][2 * c]), __uint_as_float(u[i][2 * c + 1]), x);
                            p[0][c] = x[0], p[1][c] = x[1], p[2][c] = x[2];
                        }
#pragma unroll
                        for (int k = 0; k < 3; ++k) tc05::tmem_st16(p_addr + 32u * k + 16u * i, p[k]);
                    }
                    if (jt > w.j0) {  // the tile before: its O joins the item's, on the new reference
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            uint32_t o[16];
                            item_o(i, jt - 1 > w.j0, o);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                            tc05::tmem_st16(sum_addr + 16u * i, o);
                        }
                    }
                    tc05::tmem_st_wait();
                    tc05::fence_before_sync();
                } else if (g > 0) {
                    wait(pv_done, g - 1);  // (each of its phases)
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            wait(pv_done, g - 1);
            tc05::fence_after_sync();
            if (warp_real) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                float *dst = static_cast<float *>(a.out) + (int64_t)(w.s.row0 + tok) * a.o_st +
                             (int64_t)(w.p.h * a.group.d + row - tok * a.group.d) * a.o_sh;
                float *pt = part_at(a, part, w.head ? 1 : 0, 0) + tid;  // element x of the row at pt[x * rows_cap]
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    uint32_t o[16];
                    item_o(i, w.j1 - w.j0 > 1, o);
                    if (!real) continue;
                    if (w.whole) {
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            *reinterpret_cast<float4 *>(dst + 16 * i + c) =
                                make_float4(__uint_as_float(o[c]) * inv, __uint_as_float(o[c + 1]) * inv,
                                            __uint_as_float(o[c + 2]) * inv, __uint_as_float(o[c + 3]) * inv);
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c) pt[(16 * i + c) * a.rows_cap] = __uint_as_float(o[c]);
                    }
                }
                if (real && !w.whole) pt[kD * a.rows_cap] = m * sl, pt[(kD + 1) * a.rows_cap] = l;
            }
            tc05::fence_before_sync();
            if (!w.whole) {
                W nx = w;
                nx.next();
                if (nx.live())
                    finish_piece<float, kP32Rows, false, kP32Softmax>(a, merge_sm, pieces, w.s, w.p, tid,
                                                                      [] { named_barrier(1, kP32Softmax); });
                else finish_last(w.s, w.p);
            }
        }
    }

    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kP32Mma) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, 512);
    }
}

}  // namespace think
