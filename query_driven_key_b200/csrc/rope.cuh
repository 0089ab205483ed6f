// rope.cuh -- norms of the query and key heads, the rotation by position and
// the write of the new keys and values into the paged cache, in one pass.
//
// Per token t and head row x (128 channels): x^ = x * rsqrt(mean(x^2) + eps) * w
// (queries and keys, where a weight is given), then for each pair (x1, x2) of
// the first `rot` channels, with a = position * inv_freq[i],
//     (x1, x2) -> (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
// pairs (i, i + rot/2) or (2i, 2i + 1).  Values are copied.
//
// Bound by HBM: every head row is read once and written once.  One block a
// token; a lane holds 16 bytes of a head row, so that 16 (bf16) or 32 (fp32)
// lanes hold a row and the norm is a shuffle reduction.  The block's rows are
// loaded into registers first, so that the loads run while its first threads
// turn the position into the token's cosines and sines (shared by its heads).
// The angle is formed and reduced in fp64: at position 131072 an fp32 product
// is off by up to 2^-24 * 131072 = 0.008 rad.  All arithmetic after it is fp32,
// with one rounding at the store.
#pragma once

#include "ptx.cuh"

namespace think {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;  // head rows a lane group holds at once

struct RopeArgs {
    const void *q, *k, *v, *wq, *wk;
    void *q_out, *k_cache, *v_cache;
    const double *inv_freq;
    const int32_t *positions;
    const int64_t *slots;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;
    int64_t kc_sp, kc_sh, kc_sn, vc_sp, vc_sh, vc_sn;
    int64_t num_slots;
    int Hq, Hkv, rot, page_size;
    float eps;
};

template <typename T> struct RopeVec;  // 16 bytes of a row as fp32 channels
template <> struct RopeVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 w, float x[8])
    {
        x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
        x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
    }
    static __device__ __forceinline__ uint32_t two(float lo, float hi)
    {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    static __device__ __forceinline__ uint4 pack(const float x[8])
    {
        return make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
    }
};
template <> struct RopeVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 w, float x[4])
    {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float x[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

template <typename T, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_append_kernel(const RopeArgs a)
{
    constexpr int VEC = RopeVec<T>::N;
    constexpr int LANES = kD / VEC;             // lanes of a head row
    constexpr int GROUPS = kRopeThreads / LANES;  // head rows at once
    __shared__ float2 s_cs[kD / 2];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    const int lane = tid % LANES, grp = tid / LANES;
    const int c = lane * VEC;
    const int rows = a.Hq + 2 * a.Hkv;
    grid_dependency_wait();

    const T *q = static_cast<const T *>(a.q) + t * a.q_st + c;
    const T *k = static_cast<const T *>(a.k) + t * a.k_st + c;
    const T *v = static_cast<const T *>(a.v) + t * a.v_st + c;
    auto load = [&](int r) {
        const T *p = r < a.Hq             ? q + (int64_t)r * a.q_sh
                     : r < a.Hq + a.Hkv ? k + (int64_t)(r - a.Hq) * a.k_sh
                                        : v + (int64_t)(r - a.Hq - a.Hkv) * a.v_sh;
        return *reinterpret_cast<const uint4 *>(p);
    };
    uint4 w[kRopeUnroll];
#pragma unroll
    for (int i = 0; i < kRopeUnroll; ++i)
        if (grp + i * GROUPS < rows) w[i] = load(grp + i * GROUPS);

    if (tid < a.rot / 2) {
        // the angle in turns, reduced to [-1/2, 1/2] in fp64
        const double turns = (double)a.positions[t] * a.inv_freq[tid] * 0.15915494309189533577;
        float sn, cs;
        sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
        s_cs[tid] = make_float2(cs, sn);
    }
    const int64_t slot = a.slots[t];
    const bool kept = slot >= 0 && slot < a.num_slots;
    const int64_t page = kept ? slot / a.page_size : 0, off = kept ? slot % a.page_size : 0;
    T *qo = static_cast<T *>(a.q_out) + t * a.qo_st + c;
    T *kc = static_cast<T *>(a.k_cache) + page * a.kc_sp + off * a.kc_sn + c;
    T *vc = static_cast<T *>(a.v_cache) + page * a.vc_sp + off * a.vc_sn + c;
    __syncthreads();

    // this lane's factors: y[i] = x[i] * cs[i] + partner[i] * sn[i]
    float cs[VEC], sn[VEC];
    const int half = a.rot / 2;
    const bool turned = c < a.rot;
    const int src = NEIGHBOURS ? lane : (c < half ? lane + half / VEC : lane - half / VEC);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        cs[i] = 1.f, sn[i] = 0.f;
        if (turned) {
            const float2 f = s_cs[NEIGHBOURS ? (c + i) / 2 : (c < half ? c + i : c + i - half)];
            cs[i] = f.x;
            sn[i] = (NEIGHBOURS ? (i & 1) == 0 : c < half) ? -f.y : f.y;
        }
    }

    for (int r0 = grp; r0 - grp < rows; r0 += GROUPS * kRopeUnroll) {
#pragma unroll
        for (int i = 0; i < kRopeUnroll; ++i) {
            const int r = r0 + i * GROUPS;
            // whole warps take part in the shuffles: rows past the last one carry zeros
            const bool real = r < rows;
            const bool is_v = r >= a.Hq + a.Hkv;
            if (!__any_sync(0xffffffffu, real)) continue;
            uint4 u = real ? w[i] : make_uint4(0, 0, 0, 0);
            float x[VEC];
            RopeVec<T>::unpack(u, x);
            const T *wt = static_cast<const T *>(r < a.Hq ? a.wq : a.wk);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            if (!is_v && wt) {
                const float inv = rsqrtf(ss * (1.f / kD) + a.eps);
                float wv[VEC];
                RopeVec<T>::unpack(*reinterpret_cast<const uint4 *>(wt + c), wv);
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[j] = x[j] * inv * wv[j];
            }
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float p = NEIGHBOURS ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], src, LANES);
                y[j] = turned ? fmaf(x[j], cs[j], p * sn[j]) : x[j];
            }
            if (!real) continue;
            if (is_v) {
                if (kept) *reinterpret_cast<uint4 *>(vc + (int64_t)(r - a.Hq - a.Hkv) * a.vc_sh) = u;
            } else if (r < a.Hq) {
                *reinterpret_cast<uint4 *>(qo + (int64_t)r * a.qo_sh) = RopeVec<T>::pack(y);
            } else if (kept) {
                *reinterpret_cast<uint4 *>(kc + (int64_t)(r - a.Hq) * a.kc_sh) = RopeVec<T>::pack(y);
            }
        }
#pragma unroll
        for (int i = 0; i < kRopeUnroll; ++i) {
            const int r = r0 + GROUPS * (kRopeUnroll + i);
            if (r < rows) w[i] = load(r);
        }
    }
}

}  // namespace think
