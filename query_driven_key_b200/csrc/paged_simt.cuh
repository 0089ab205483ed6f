// paged_simt.cuh -- attention of new tokens over the paged cache in fp32, on
// the CUDA cores (the plan: paged_plan.cuh).
//
// Per item, over its key tiles of BN = 64, with running maxima m and sums l
// (fp32, logarithms to base 2):
//     z = scale * log2(e) * q . k   (masked: -inf),  m' = max(m, max z),
//     p = 2^(z - m'),  l = l 2^(m - m') + sum p,  O = O 2^(m - m') + p V.
// A row whose keys are all masked keeps m = -inf; the reference is then 0, so
// that p = 0 and the row ends as zeros.  Keys and values behind a request's
// last token are never used: their rows are staged as zeros, whatever the page
// holds there.
#pragma once

#include "paged_plan.cuh"

namespace think {

constexpr int kSimtThreads = kMergeThreads;
constexpr int kSimtBN = 64;

template <int R>
constexpr size_t paged_simt_smem()
{
    return sizeof(float) * ((size_t)R * kD + 2 * (size_t)kSimtBN * kD + (size_t)kSimtBN * R);
}

__device__ __forceinline__ float4 load_row4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

// Element 4 c4 of row n of a 128-wide fp32 tile whose 16-byte vectors are
// permuted within 8 rows, so that 8 rows' equal columns lie in 8 bank groups.
__device__ __forceinline__ int swz(int n, int c4) { return n * kD + ((c4 ^ (n & 7)) << 2); }

// Thread (tx, ty) = (tid % 16, tid / 16) holds rows ty + 16 i and, of the
// logits, tokens tx + 16 j, of the output channels 4 tx + 64 jj.
template <int R>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const PagedArgs a)
{
    constexpr int BN = kSimtBN, MI = R / 16;
    extern __shared__ __align__(16) float smem[];
    float *qs = smem, *ks = qs + R * kD, *vs = ks + BN * kD, *ps = vs + BN * kD;  // ps: [BN][R]
    __shared__ PlanSmem sm;
    __shared__ Pieces pieces;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    grid_dependency_wait();
    const int part = blockIdx.x;
    const Parts parts = plan<R, BN, kSimtThreads>(a, &sm, part);
    grid_launch_dependents();
    for (Walk<R, BN> w(a, sm.place, parts, part); w.live(); w.next()) {
        const int rows = min(R, w.s.n * a.group.d - w.p.qt * R);
        __syncthreads();  // the previous item's tiles have been read
        if (!w.whole && tid == 0) find_pieces(pieces, parts, w);
        for (int i = tid; i < R * 32; i += kSimtThreads) {
            const int r = i >> 5, c4 = i & 31;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int gr = w.p.qt * R + r, tok = a.group.quot(gr), g = gr - tok * a.group.d;
                x = load_row4(static_cast<const float *>(a.q) + (int64_t)(w.s.row0 + tok) * a.q_st +
                              (int64_t)(w.p.h * a.group.d + g) * a.q_sh + 4 * c4);
            }
            *reinterpret_cast<float4 *>(qs + r * kD + 4 * c4) = x;
        }
        int pos[MI];
        float m[MI], l[MI], o[MI][8];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = ty + 16 * i;
            pos[i] = r < rows ? w.s.kv - w.s.n + a.group.quot(w.p.qt * R + r) : -1;
            m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[i][j] = 0.f;
        }
        for (int jt = w.j0; jt < w.j1; ++jt) {
            __syncthreads();
            for (int i = tid; i < BN * 32; i += kSimtThreads) {
                const int n = i >> 5, c4 = i & 31, key = jt * BN + n;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (key >= w.t.lo && key < w.t.hi) {
                    const int j = a.page.quot(key);
                    const int page = a.table[(int64_t)w.p.b * a.table_ld + j];
                    if ((unsigned)page < (unsigned)a.num_pages) {
                        const int64_t off = key - (int64_t)j * a.page.d;
                        x = load_row4(static_cast<const float *>(a.k) + page * a.k_sp + w.p.h * a.k_sh + off * a.k_sn + 4 * c4);
                        y = load_row4(static_cast<const float *>(a.v) + page * a.v_sp + w.p.h * a.v_sh + off * a.v_sn + 4 * c4);
                    } else if (c4 == 0) {
                        atomicOr(a.status, THINK_DEVICE_BAD_PAGE);
                    }
                }
                *reinterpret_cast<float4 *>(ks + swz(n, c4)) = x;
                *reinterpret_cast<float4 *>(vs + n * kD + 4 * c4) = y;
            }
            __syncthreads();
            float z[MI][4];
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i][j] = 0.f;
#pragma unroll 4
            for (int c4 = 0; c4 < 32; ++c4) {
                float4 kk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4 *>(ks + swz(tx + 16 * j, c4));
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const float4 x = *reinterpret_cast<const float4 *>(qs + (ty + 16 * i) * kD + 4 * c4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        z[i][j] += x.x * kk[j].x + x.y * kk[j].y + x.z * kk[j].z + x.w * kk[j].w;
                }
            }
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = jt * BN + tx + 16 * j;
                    const bool seen = key <= pos[i] && (a.window == 0 || key > pos[i] - a.window);
                    z[i][j] = seen ? z[i][j] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, z[i][j]);
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float ref = mx == -INFINITY ? 0.f : mx;
                const float f = exp2f(m[i] - ref);
                m[i] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(z[i][j] - ref);
                    sum += p;
                    ps[(tx + 16 * j) * R + ty + 16 * i] = p;
                }
                l[i] = l[i] * f + sum;  // this thread's tokens; the 16 sums are added at the end
#pragma unroll
                for (int j = 0; j < 8; ++j) o[i][j] *= f;
            }
            __syncthreads();
#pragma unroll 4
            for (int n = 0; n < BN; ++n) {
                const float4 y0 = *reinterpret_cast<const float4 *>(vs + n * kD + 4 * tx);
                const float4 y1 = *reinterpret_cast<const float4 *>(vs + n * kD + 64 + 4 * tx);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const float p = ps[n * R + ty + 16 * i];
                    o[i][0] += p * y0.x, o[i][1] += p * y0.y, o[i][2] += p * y0.z, o[i][3] += p * y0.w;
                    o[i][4] += p * y1.x, o[i][5] += p * y1.y, o[i][6] += p * y1.z, o[i][7] += p * y1.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = ty + 16 * i;
            float s = l[i];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (r >= rows) continue;
            if (w.whole) {
                const float inv = s > 0.f ? 1.f / s : 0.f;
                const int gr = w.p.qt * R + r, tok = a.group.quot(gr), g = gr - tok * a.group.d;
                float *dst = static_cast<float *>(a.out) + (int64_t)(w.s.row0 + tok) * a.o_st +
                             (int64_t)(w.p.h * a.group.d + g) * a.o_sh + 4 * tx;
                *reinterpret_cast<float4 *>(dst) = make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
                *reinterpret_cast<float4 *>(dst + 64) = make_float4(o[i][4] * inv, o[i][5] * inv, o[i][6] * inv, o[i][7] * inv);
            } else {
                float *dst = part_at(a, part, w.head ? 1 : 0, 0) + r;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dst[(4 * tx + j) * a.rows_cap] = o[i][j], dst[(64 + 4 * tx + j) * a.rows_cap] = o[i][4 + j];
                if (tx == 0) dst[kD * a.rows_cap] = m[i], dst[(kD + 1) * a.rows_cap] = s;
            }
        }
        if (!w.whole)
            finish_piece<float, R, false>(a, *reinterpret_cast<MergeSmem *>(vs), pieces, w, tid, [] { __syncthreads(); });
    }
}

}  // namespace think
