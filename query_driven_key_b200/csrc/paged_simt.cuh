// paged_simt.cuh -- attention of new tokens over the paged cache in fp32, on
// the CUDA cores (the plan: paged_plan.cuh).
//
// Per item, over its key tiles of BN = 64, with running maxima m and sums l
// (fp32, logarithms to base 2):
//     z = scale * log2(e) * q . k   (masked: -inf),  m' = max(m, max z),
//     p = 2^(z - m'),  l = l 2^(m - m') + sum p,  O = O 2^(m - m') + p V.
// A row whose keys are all masked keeps m = -inf; the reference is then 0, so
// that p = 0 and the row ends as zeros.  Keys and values that no row of the
// item sees are staged as zeros, whatever the page holds there.
//
// Bound by the FMA pipes: both products are 64 x 64 x 128 a tile, in packed
// pairs (fma.rn.f32x2: the logits over even and odd channels, the output over
// neighbouring channels).  Keys and values come with cp.async into one buffer
// each: the next tile's keys while the softmax and the product with V run, its
// values beside the next logits.  Two blocks an SM fill each other's barriers.
// The pages of a tile's rows are looked up a tile ahead, once a row.
#pragma once

#include "paged_plan.cuh"
#include "rope.cuh"

namespace think {

constexpr int kSimtThreads = kMergeThreads;
constexpr int kSimtBN = 64;

template <int R>
constexpr size_t paged_simt_smem()
{
    return sizeof(float) * ((size_t)R * kD + 2 * (size_t)kSimtBN * kD + (size_t)kSimtBN * R);
}

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void cp_async_16_or_0(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// Element 4 c4 of row n of a 128-wide fp32 tile whose 16-byte vectors are
// permuted within 8 rows, so that 8 rows' equal columns lie in 8 bank groups
// (in Q, within 8 threads' rows: a warp reads those of two at once).
__device__ __forceinline__ int swz(int n, int c4) { return n * kD + ((c4 ^ (n & 7)) << 2); }

// Thread (tx, ty) = (tid % 16, tid / 16) holds rows MI ty .. and, of the
// logits, tokens tx + 16 j, of the output channels 4 tx + 64 jj.
template <int R>
__global__ void __launch_bounds__(kSimtThreads, 2) paged_simt_kernel(const PagedArgs a)
{
    constexpr int BN = kSimtBN, MI = R / 16;
    extern __shared__ __align__(16) float smem[];
    float *qs = smem, *ks = qs + R * kD, *vs = ks + BN * kD, *ps = vs + BN * kD;  // ps: [BN][R], see p_at
    __shared__ PlanSmem sm;
    __shared__ Pieces pieces;
    __shared__ int2 s_row[BN];  // of the next tile to fetch: a row's page (-1: zeros) and place in it
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const float *kp = static_cast<const float *>(a.k), *vp = static_cast<const float *>(a.v);
    grid_dependency_wait();
    const int part = blockIdx.x;
    const Parts parts = plan<R, BN, kSimtThreads>(a, &sm, part);
    grid_launch_dependents();
    // the rows' blocks of a token's weights, permuted so that 16 tokens' equal blocks lie in different banks
    auto p_at = [&](int n) { return ps + n * R + (R == 64 ? (ty ^ (n & 15)) * 4 : ty); };
    for (Walk<R, BN> w(a, sm.place, parts, part); w.live(); w.next()) {
        const int rows = min(R, w.s.n * a.group.d - w.p.qt * R);
        auto locate = [&](int jt) {  // a thread a row of the tile
            if (tid < BN) {
                const int key = jt * BN + tid;
                int2 x = make_int2(-1, 0);
                if (key >= w.t.lo && key < w.t.hi) {
                    const int j = a.page.quot(key), page = a.table[(int64_t)w.p.b * a.table_ld + j];
                    if ((unsigned)page < (unsigned)a.num_pages) x = make_int2(page, key - j * a.page.d);
                    else atomicOr(a.status, THINK_DEVICE_BAD_PAGE);
                }
                s_row[tid] = x;
            }
        };
        auto fetch = [&](bool value) {
            const uint32_t base = smem_addr(value ? vs : ks);
            const int64_t sp = value ? a.v_sp : a.k_sp, sn = value ? a.v_sn : a.k_sn, head = w.p.h * (value ? a.v_sh : a.k_sh);
#pragma unroll
            for (int i = 0; i < BN * 32 / kSimtThreads; ++i) {
                const int n = (tid >> 5) + 8 * i, c4 = tid & 31;
                const int2 x = s_row[n];
                cp_async_16_or_0(base + 4u * (value ? n * kD + 4 * c4 : swz(n, c4)),
                                 (value ? vp : kp) + (x.x >= 0 ? x.x * sp + head + x.y * sn + 4 * c4 : 0), x.x >= 0);
            }
            cp_async_commit();
        };
        __syncthreads();  // the previous item's tiles have been read
        if (!w.whole && tid == 0) find_pieces(pieces, parts, w);
        locate(w.j0);
        for (int i = tid; i < R * 32; i += kSimtThreads) {
            const int r = i >> 5, c4 = i & 31;
            const int gr = w.p.qt * R + r, tok = a.group.quot(gr), g = gr - tok * a.group.d;
            cp_async_16_or_0(smem_addr(qs + r * kD + 4 * (c4 ^ (r / MI & 7))),
                             static_cast<const float *>(a.q) +
                                 (r < rows ? (int64_t)(w.s.row0 + tok) * a.q_st + (int64_t)(w.p.h * a.group.d + g) * a.q_sh + 4 * c4 : 0),
                             r < rows);
        }
        __syncthreads();
        fetch(false);  // (with the queries)
        fetch(true);
        int pos[MI];
        float m[MI], l[MI];
        uint64_t o[MI][4];  // channels 4 tx + (0, 1), (2, 3), 64 + 4 tx + (0, 1), (2, 3)
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = MI * ty + i;
            pos[i] = r < rows ? w.s.kv - w.s.n + a.group.quot(w.p.qt * R + r) : -1;
            m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0;
        }
        const int first = w.s.kv - w.s.n + a.group.quot(w.p.qt * R);  // the tile's first position
        const int final = w.s.kv - w.s.n + a.group.quot(w.p.qt * R + rows - 1);
        for (int jt = w.j0; jt < w.j1; ++jt) {
            const bool more = jt + 1 < w.j1;
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // this tile's keys
            __syncthreads();
            if (more) locate(jt + 1);  // (this tile's rows have all been asked for)
            uint64_t z2[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) z2[i][j] = 0;
#pragma unroll 2
            for (int c4 = 0; c4 < 32; ++c4) {
                ulonglong2 kk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const ulonglong2 *>(ks + swz(tx + 16 * j, c4));
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(qs + (MI * ty + i) * kD + 4 * (c4 ^ (ty & 7)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) z2[i][j] = fma2(x.y, kk[j].y, fma2(x.x, kk[j].x, z2[i][j]));
                }
            }
            __syncthreads();  // the keys have been read, the next tile's places are known
            if (more) fetch(false);
            else cp_async_commit();
            const bool full = (jt + 1) * BN <= first + 1 && rows == R && (a.window == 0 || jt * BN > final - a.window);
            float p[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float even, odd;
                    unpack2(z2[i][j], even, odd);
                    const int key = jt * BN + tx + 16 * j;
                    const bool seen = full || (key <= pos[i] && (a.window == 0 || key > pos[i] - a.window));
                    p[i][j] = seen ? (even + odd) * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, p[i][j]);
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float ref = mx == -INFINITY ? 0.f : mx;
                const float f = exp2_approx(m[i] - ref);
                m[i] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) p[i][j] = exp2_approx(p[i][j] - ref), sum += p[i][j];
                l[i] = l[i] * f + sum;  // this thread's tokens; the 16 sums are added at the end
                const uint64_t f2 = pack2(f, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] = mul2(o[i][j], f2);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float *dst = p_at(tx + 16 * j);
                if constexpr (MI == 4) *reinterpret_cast<float4 *>(dst) = make_float4(p[0][j], p[1][j], p[2][j], p[3][j]);
                else dst[0] = p[0][j];
            }
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // this tile's values
            __syncthreads();
#pragma unroll 2
            for (int n = 0; n < BN; ++n) {
                const ulonglong2 y0 = *reinterpret_cast<const ulonglong2 *>(vs + n * kD + 4 * tx);
                const ulonglong2 y1 = *reinterpret_cast<const ulonglong2 *>(vs + n * kD + 64 + 4 * tx);
                float pn[MI];
                if constexpr (MI == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(p_at(n));
                    pn[0] = x.x, pn[1] = x.y, pn[2] = x.z, pn[3] = x.w;
                } else {
                    pn[0] = *p_at(n);
                }
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const uint64_t p2 = pack2(pn[i], pn[i]);
                    o[i][0] = fma2(p2, y0.x, o[i][0]), o[i][1] = fma2(p2, y0.y, o[i][1]);
                    o[i][2] = fma2(p2, y1.x, o[i][2]), o[i][3] = fma2(p2, y1.y, o[i][3]);
                }
            }
            __syncthreads();  // the values and weights have been read
            if (more) fetch(true);
            else cp_async_commit();
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = MI * ty + i;
            float s = l[i];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (r >= rows) continue;
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) unpack2(o[i][j], x[2 * j], x[2 * j + 1]);
            if (w.whole) {
                const float inv = s > 0.f ? 1.f / s : 0.f;
                const int gr = w.p.qt * R + r, tok = a.group.quot(gr), g = gr - tok * a.group.d;
                float *dst = static_cast<float *>(a.out) + (int64_t)(w.s.row0 + tok) * a.o_st +
                             (int64_t)(w.p.h * a.group.d + g) * a.o_sh + 4 * tx;
                *reinterpret_cast<float4 *>(dst) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                *reinterpret_cast<float4 *>(dst + 64) = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
            } else {
                float *dst = part_at(a, part, w.head ? 1 : 0, 0) + r;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dst[(4 * tx + j) * a.rows_cap] = x[j], dst[(64 + 4 * tx + j) * a.rows_cap] = x[4 + j];
                if (tx == 0) dst[kD * a.rows_cap] = m[i], dst[(kD + 1) * a.rows_cap] = s;
            }
        }
        if (!w.whole)
            finish_piece<float, R, false>(a, *reinterpret_cast<MergeSmem *>(vs), pieces, w, tid, [] { __syncthreads(); });
    }
    cp_async_wait_all();
}

}  // namespace think
