// rope.cuh -- norms of the query and key heads, the rotation by position and
// the write of the new keys and values into the paged cache, in one pass.
//
// Per token t and head row x (128 channels): x^ = x * rsqrt(mean(x^2) + eps) * w
// (queries and keys, where a weight is given), then for each pair (x1, x2) of
// the first `rot` channels, with a = position * inv_freq[i],
//     (x1, x2) -> (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
// pairs (i, i + rot/2) or (2i, 2i + 1).  Values are copied.
//
// Bound by HBM: every head row is read once and written once.  Persistent
// blocks take runs of tokens; the threads copy the head rows of the next tokens
// (up to 16 KB each) to shared memory ahead with cp.async, which holds no
// registers.  16 (bf16) or 32 (fp32) lanes of a warp share a row, and each
// reads back two 8-byte chunks chosen so that it holds both partners of its
// pairs; only the norm is a shuffle reduction.  With the weights folded into a
// token's factors (y = rsqrt(..) * (x * cos w + partner * (-+ sin) w')) a row
// costs a few packed fp32 operations a lane.  Rows of one warp are its own
// copies, so that the steady state has no barrier but the two of a batch of
// tokens, in which the threads turn positions into factors (one thread a pair;
// all heads of a token share them).  The angle is formed and reduced in fp64:
// at position 131072 an fp32 product is off by up to 2^-24 * 131072 = 0.008 rad.
// All arithmetic after it is fp32, with one rounding at the store (the reduced angle's to
// fp32 is off by at most 2^-26 of a turn, 1e-7 rad, as much as a sine's last place).
// Measured: 8192 tokens of 32 + 8 + 8 bf16 heads (201 MB) 42.1 us = 4.8 TB/s;
// 1777 tokens of 12 + 4 + 4 fp32 heads (36 MB) 8.5 us; one token 3.5 us.  Bound by
// the issue of instructions (140 for two rows of a warp, 0.67 of the issue slots)
// beside HBM: what helps is fewer idle lanes.  512 threads of two rows each 43.3
// (48 rows are one and a half a thread group); rows held in registers instead
// of the ring (90 a thread, two blocks an SM) 90; the ring without fixed heads a
// thread 65.
#pragma once

#include "ptx.cuh"

namespace think {

constexpr int kRopeThreads = 256;
constexpr int kRopeStages = 3;       // steps in shared memory (four blocks an SM)
constexpr int kRopeBatch = kRopeThreads / (kD / 2);  // tokens whose factors are formed together
constexpr int kRopeBlocksPerSM = 4;

struct RopeArgs {
    const void *q, *k, *v, *wq, *wk;
    void *q_out, *k_cache, *v_cache;
    const double *inv_freq;
    const int32_t *positions;
    const int64_t *slots;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;
    int64_t kc_sp, kc_sh, kc_sn, vc_sp, vc_sh, vc_sn;
    int64_t num_slots, T;
    int Hq, Hkv, rot, page_size;
    int unit;  // tokens of a step, a power of two up to kRopeBatch
    float eps;
};

__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t swap2(uint64_t a)
{
    float lo, hi;
    unpack2(a, lo, hi);
    return pack2(hi, lo);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// An 8-byte chunk of a row as pairs of fp32 channels.
template <typename T> struct RopeChunk;
template <> struct RopeChunk<__nv_bfloat16> {
    static constexpr int N = 4;  // channels
    static __device__ __forceinline__ void unpack(uint2 w, uint64_t x[2])
    {
        x[0] = pack2(bf16lo(w.x), bf16hi(w.x)), x[1] = pack2(bf16lo(w.y), bf16hi(w.y));
    }
    static __device__ __forceinline__ uint2 pack(const uint64_t x[2])
    {
        float a, b, c, d;
        unpack2(x[0], a, b), unpack2(x[1], c, d);
        return make_uint2(bf16_pair(a, b), bf16_pair(c, d));
    }
};
template <> struct RopeChunk<float> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void unpack(uint2 w, uint64_t x[1])
    {
        x[0] = pack2(__uint_as_float(w.x), __uint_as_float(w.y));
    }
    static __device__ __forceinline__ uint2 pack(const uint64_t x[1])
    {
        float a, b;
        unpack2(x[0], a, b);
        return make_uint2(__float_as_uint(a), __float_as_uint(b));
    }
};

// Rows of a block: blockIdx.y's share of the q, k and v heads (at most SLOTS a thread group),
// of the tokens [T x / X, T (x + 1) / X), x = blockIdx.x of X.  Row slot i of a
// thread is a fixed head, so that its addresses only move with the token.
// SHARED: few heads; a step takes a.unit tokens (else one), whose rows, one after
// another, fill the row slots (8192 tokens of 1 + 1 + 1 bf16 heads 10.9 us, a token a
// step 22.7).
// ALL: every channel is turned (rot == 128); looking whether a lane's are costs 2% (8192
// tokens of 48 heads 42.2 -> 43.2 us).
template <typename T, bool NEIGHBOURS, bool ALL, int SLOTS, bool SHARED>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSM) norm_rope_append_kernel(const RopeArgs a)
{
    constexpr int CH = RopeChunk<T>::N;           // channels of a chunk
    constexpr int VEC = 2 * CH;                   // channels of a lane
    constexpr int LANES = kD / VEC;               // lanes of a head row
    constexpr int GROUPS = kRopeThreads / LANES;  // head rows at once
    constexpr int P = CH / 2;                     // fp32 pairs of a chunk
    extern __shared__ unsigned char ring[];       // [stages][row slots][threads][16 B]
    // per token of the batch, rows of q or k, and lane: what its first chunk's and its second chunk's channels
    // are multiplied by, then what their partners are
    __shared__ float4 s_f[kRopeBatch][2][VEC / 2][LANES];
    __shared__ int64_t s_off[kRopeBatch][4];  // the token's row in q_out, the key and the value pool, -1: none
    const int tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES;
    const int rows = a.Hq + 2 * a.Hkv, half = a.rot / 2;
    const int row0 = (int)((int64_t)rows * blockIdx.y / gridDim.y), row1 = (int)((int64_t)rows * (blockIdx.y + 1) / gridDim.y);
    const int64_t t0 = a.T * blockIdx.x / gridDim.x, t1 = a.T * (blockIdx.x + 1) / gridDim.x;
    const int U = SHARED ? a.unit : 1;
    const uint32_t stage_bytes = (uint32_t)(((row1 - row0) * U + GROUPS - 1) / GROUPS) * (kRopeThreads * 16);
    // This lane's chunks: channels a0 .. and b0 .., each the other's partners
    // (NEIGHBOURS: partners lie beside each other); lanes past the turned
    // channels hold neighbouring chunks of the rest.
    const int turning = NEIGHBOURS ? 0 : half / CH;
    const int a0 = NEIGHBOURS ? lane * VEC : lane < turning ? lane * CH : a.rot + (lane - turning) * VEC;
    const int b0 = !NEIGHBOURS && lane < turning ? a0 + half : a0 + CH;
    const unsigned char *src[SLOTS];  // the next step's vector of this thread
    int64_t step[SLOTS];              // bytes to the step after it
    T *dst[SLOTS];                    // the head's row but for s_off
    int kind[SLOTS];                  // 0 q, 1 k, 2 v, 3 none
    int tok[SLOTS];                   // token of the step
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        const int at = grp + i * GROUPS;
        tok[i] = SHARED ? min(at / (row1 - row0), U) : at >= row1 - row0 ? 1 : 0;
        const int r = row0 + at - tok[i] * (row1 - row0);
        kind[i] = tok[i] == U ? 3 : r < a.Hq ? 0 : r < a.Hq + a.Hkv ? 1 : 2;
        const int h = r - (kind[i] == 0 ? 0 : kind[i] == 1 ? a.Hq : a.Hq + a.Hkv);
        const void *p = kind[i] == 0 ? a.q : kind[i] == 1 ? a.k : a.v;
        const int64_t st = kind[i] == 0 ? a.q_st : kind[i] == 1 ? a.k_st : a.v_st;
        const int64_t sh = kind[i] == 0 ? a.q_sh : kind[i] == 1 ? a.k_sh : a.v_sh;
        step[i] = U * st * (int64_t)sizeof(T);
        src[i] = kind[i] == 3 ? nullptr : static_cast<const unsigned char *>(p) + ((t0 + tok[i]) * st + h * sh + lane * VEC) * (int64_t)sizeof(T);
        dst[i] = kind[i] == 0   ? static_cast<T *>(a.q_out) + h * a.qo_sh
                 : kind[i] == 1 ? static_cast<T *>(a.k_cache) + h * a.kc_sh
                                : static_cast<T *>(a.v_cache) + h * a.vc_sh + lane * VEC;
    }
    grid_dependency_wait();

    int ahead = (int)(t1 - t0);  // tokens not yet fetched
    uint32_t fs = 0;             // stage of the next one
    auto fetch = [&]() {
        if (ahead > 0) {
            const uint32_t to = smem_addr(ring) + fs + tid * 16;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                if (SHARED ? tok[i] < min(ahead, U) : tok[i] == 0) {
                    cp_async_16(to + i * (kRopeThreads * 16), src[i]);
                    src[i] += step[i];
                }
            ahead -= U;
        }
        cp_async_commit();
        fs = fs == (kRopeStages - 1) * stage_bytes ? 0 : fs + stage_bytes;
    };
#pragma unroll
    for (int n = 0; n < kRopeStages - 1; ++n) fetch();

    // where channel ch is held: its lane, and its place among the lane's VEC
    auto held = [&](int ch, int &l, int &at) {
        if (NEIGHBOURS || ch >= a.rot) {
            const int u = NEIGHBOURS ? ch : ch - a.rot;
            l = turning + u / VEC, at = u % VEC;
        } else {
            const int u = ch < half ? ch : ch - half;
            l = u / CH, at = (ch < half ? 0 : CH) + u % CH;
        }
    };
    // the pair whose factors this thread forms, for every batch
    const int pair = tid % (kD / 2);
    const bool turns_it = pair < half;
    const int c1 = NEIGHBOURS || !turns_it ? 2 * pair : pair;
    const int c2 = NEIGHBOURS || !turns_it ? c1 + 1 : c1 + half;
    int l1, p1, l2, p2;
    held(c1, l1, p1);
    held(c2, l2, p2);
    float w1[2], w2[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const T *w = static_cast<const T *>(y ? a.wk : a.wq);
        w1[y] = w ? Elem<T>::to_float(w[c1]) : 1.f, w2[y] = w ? Elem<T>::to_float(w[c2]) : 1.f;
    }
    const double turns_per = turns_it ? a.inv_freq[pair] : 0.0;

    uint32_t stage = 0;
    for (int64_t first = t0; first < t1; first += kRopeBatch) {
        __syncthreads();  // the previous batch's factors have been read
        {
            const int k = tid / (kD / 2);  // kRopeBatch x 64 threads: one a pair of each token
            const int64_t t = first + k;
            if (t < t1) {
                // the angle in turns, reduced to [-1/2, 1/2] in fp64
                const double turns = (double)a.positions[t] * turns_per * 0.15915494309189533577;
                float sn, cs;
                sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    auto put = [&](int l, int at, float f) { reinterpret_cast<float *>(&s_f[k][y][at >> 2][l])[at & 3] = f; };
                    put(l1, p1, cs * w1[y]), put(l1, VEC + p1, -sn * w2[y]);
                    put(l2, p2, cs * w2[y]), put(l2, VEC + p2, sn * w1[y]);
                }
                if (pair == 0) {
                    const int64_t slot = a.slots[t];
                    const bool kept = slot >= 0 && slot < a.num_slots;
                    int64_t page = 0, off = 0;
                    if (kept) {
                        if ((slot >> 32) == 0) page = (uint32_t)slot / (uint32_t)a.page_size;  // the short division
                        else page = slot / a.page_size;
                        off = slot - page * a.page_size;
                    }
                    s_off[k][0] = t * a.qo_st;
                    s_off[k][1] = kept ? page * a.kc_sp + off * a.kc_sn : -1;
                    s_off[k][2] = kept ? page * a.vc_sp + off * a.vc_sn : -1;
                }
            }
        }
        __syncthreads();
        const int n = (int)min((int64_t)kRopeBatch, t1 - first);
        for (int k0 = 0; k0 < n; k0 += U) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRopeStages - 2) : "memory");
            __syncwarp();  // the warp's lanes share its rows
            const unsigned char *held_rows = ring + stage + (uint32_t)grp * (kD * sizeof(T));
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                if (i * GROUPS >= (row1 - row0) * U) break;
                const int k = k0 + (SHARED ? tok[i] : 0);
                if (SHARED && k >= n) continue;
                const unsigned char *row = held_rows + i * (kRopeThreads * 16);
                if (kind[i] >= 2) {  // a value row: as it is
                    if (kind[i] == 2 && s_off[k][2] >= 0)
                        *reinterpret_cast<uint4 *>(dst[i] + s_off[k][2]) = *reinterpret_cast<const uint4 *>(row + lane * 16);
                    continue;
                }
                uint64_t x[P], z[P];
                RopeChunk<T>::unpack(*reinterpret_cast<const uint2 *>(row + a0 * sizeof(T)), x);
                RopeChunk<T>::unpack(*reinterpret_cast<const uint2 *>(row + b0 * sizeof(T)), z);
                float inv = 1.f;
                if (kind[i] ? a.wk : a.wq) {
                    uint64_t s2 = fma2(z[0], z[0], mul2(x[0], x[0]));
#pragma unroll
                    for (int j = 1; j < P; ++j) s2 = fma2(z[j], z[j], fma2(x[j], x[j], s2));
                    float ss, ss1;
                    unpack2(s2, ss, ss1);
                    ss += ss1;
                    // the lanes of this row (another row of the warp may be of another kind)
                    const unsigned mask = LANES == 32 ? 0xffffffffu : 0xffffu << (tid & 16);
#pragma unroll
                    for (int d = LANES / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(mask, ss, d);
                    inv = rsqrtf(ss * (1.f / kD) + a.eps);
                }
                const uint64_t inv2 = pack2(inv, inv);
                float4 f4[VEC / 2];
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) f4[j] = s_f[k][kind[i]][j][lane];
                const uint64_t *f = reinterpret_cast<const uint64_t *>(f4);  // cos w: P + P pairs, sin w': P + P
                if (ALL || a0 < a.rot) {
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const uint64_t px = NEIGHBOURS ? swap2(x[j]) : z[j], pz = NEIGHBOURS ? swap2(z[j]) : x[j];
                        const uint64_t y = fma2(px, f[2 * P + j], mul2(x[j], f[j]));
                        z[j] = mul2(fma2(pz, f[3 * P + j], mul2(z[j], f[P + j])), inv2);
                        x[j] = mul2(y, inv2);
                    }
                } else {  // no partners (an infinity times a sine of 0 would be NaN)
#pragma unroll
                    for (int j = 0; j < P; ++j) x[j] = mul2(mul2(x[j], f[j]), inv2), z[j] = mul2(mul2(z[j], f[P + j]), inv2);
                }
                const int64_t off = s_off[k][kind[i]];
                if (off >= 0) {
                    *reinterpret_cast<uint2 *>(dst[i] + off + a0) = RopeChunk<T>::pack(x);
                    *reinterpret_cast<uint2 *>(dst[i] + off + b0) = RopeChunk<T>::pack(z);
                }
            }
            __syncwarp();  // its rows have been read
            fetch();       // into the stage of the token before
            stage = stage == (kRopeStages - 1) * stage_bytes ? 0 : stage + stage_bytes;
        }
    }
    cp_async_wait_all();
}

}  // namespace think
