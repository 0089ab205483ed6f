// host.cuh -- host helpers shared by the library's source files: environment
// switches, argument checks, launches with programmatic stream serialisation,
// TMA descriptors.  Host code only.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "think.h"

namespace think {
namespace {

constexpr int kTargetSMs = 148;             // B200
constexpr size_t kSmemPerSM = 233472;       // 228 KB
constexpr size_t kSmemPerBlockMax = 232448; // 227 KB opt-in
constexpr size_t kSmemReservedPerBlock = 1024;

inline bool env_flag(const char *name)
{
    const char *v = std::getenv(name);
    return v && v[0] == '1';
}

inline int env_int(const char *name, int dflt, int lo, int hi)
{
    const char *v = std::getenv(name);
    if (!v || !*v) return dflt;
    const int x = std::atoi(v);
    return x < lo ? lo : (x > hi ? hi : x);
}

inline size_t esize(think_dtype_t t) { return t == THINK_BF16 ? 2 : 4; }
inline bool dtype_ok(int t) { return t == THINK_F32 || t == THINK_BF16; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline think_status_t launch_status()
{
    return cudaGetLastError() == cudaSuccess ? THINK_OK : THINK_ERR_CUDA;
}

// Launch with programmatic stream serialisation (the kernel may start while
// the previous kernel of the stream drains; it waits in griddepcontrol.wait
// before its first global access).  THINK_PDL=0 launches plainly.
// With cluster > 0, blocks (x, y) .. (x + cluster - 1, y), x a multiple of
// cluster, form one thread-block cluster.
template <typename... KArgs, typename... Args>
think_status_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                  int cluster, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (env_int("THINK_PDL", 1, 0, 1)) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? THINK_OK : THINK_ERR_CUDA;
}

template <typename... KArgs, typename... Args>
think_status_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                          Args &&...args)
{
    return launch_pdl_cluster(kern, grid, block, smem, st, 0, std::forward<Args>(args)...);
}

// ------------------------------------------------------------ TMA maps --

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Encoded maps are kept in a small per-thread cache keyed by every input of
// the encoding (a decode step re-encodes the same two maps otherwise).
struct MapKey {
    const void *base;
    cuuint64_t dims[5], strides[4];
    uint32_t box[5];
    int dtype, swizzle;
};

bool map_cache_find(const MapKey &k, CUtensorMap *m);
void map_cache_put(const MapKey &k, const CUtensorMap &m);

// Map of `rank` (4 or 5) dimensions, strides in elements for all but the first.
bool make_map(CUtensorMap *m, think_dtype_t dt, const void *base, int rank, const uint64_t *dims, const int64_t *strides,
              const uint32_t *box, bool swizzle128)
{
    MapKey key;
    memset(&key, 0, sizeof(key));
    key.base = base;
    for (int i = 0; i < rank; ++i) key.dims[i] = dims[i], key.box[i] = box[i];
    for (int i = 0; i + 1 < rank; ++i) key.strides[i] = (uint64_t)strides[i];
    key.dtype = (int)dt;
    key.swizzle = swizzle128 ? 1 : 0;
    if (map_cache_find(key, m)) return true;
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t bytes[4];
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = (cuuint64_t)strides[i] * esize(dt);
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(m, dt == THINK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                          (cuuint32_t)rank, const_cast<void *>(base), key.dims, bytes, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return false;
    map_cache_put(key, *m);
    return true;
}

// 4-D map over (x, y, z, w) with element strides sy, sz, sw for y, z, w; box (bx, by, bz, 1).
bool make_map_4d(CUtensorMap *m, think_dtype_t dt, const void *base, uint64_t dx, uint64_t dy,
                 uint64_t dz, uint64_t dw, int64_t sy, int64_t sz, int64_t sw, uint32_t bx,
                 uint32_t by, bool swizzle128 = false, uint32_t bz = 1)
{
    const uint64_t dims[4] = {dx, dy, dz, dw};
    const int64_t strides[3] = {sy, sz, sw};
    const uint32_t box[4] = {bx, by, bz, 1};
    return make_map(m, dt, base, 4, dims, strides, box, swizzle128);
}

constexpr int kMapCacheSize = 16;
struct MapCacheEntry {
    MapKey key;
    CUtensorMap map;
    bool used;
};
thread_local MapCacheEntry g_map_cache[kMapCacheSize];
thread_local int g_map_next = 0;

bool map_cache_find(const MapKey &k, CUtensorMap *m)
{
    for (int i = 0; i < kMapCacheSize; ++i)
        if (g_map_cache[i].used && memcmp(&g_map_cache[i].key, &k, sizeof(MapKey)) == 0) {
            *m = g_map_cache[i].map;
            return true;
        }
    return false;
}

void map_cache_put(const MapKey &k, const CUtensorMap &m)
{
    MapCacheEntry &e = g_map_cache[g_map_next];
    g_map_next = (g_map_next + 1) % kMapCacheSize;
    e.key = k;
    e.map = m;
    e.used = true;
}

// Allow a kernel `bytes` of dynamic shared memory.  The attribute belongs to the
// kernel and the device, whichever thread sets it, so that the sizes are kept for
// the process and only ever raised: a call that needs less must not take away
// what another thread's next launch of the same kernel relies on.
bool ensure_smem(const void *kern, size_t bytes)
{
    static std::mutex mutex;
    static std::map<std::pair<const void *, int>, size_t> allowed;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const std::lock_guard<std::mutex> lock(mutex);
    size_t &have = allowed[{kern, dev}];
    if (have >= bytes) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return false;
    have = bytes;
    return true;
}

// 4-D map of any element type with byte strides; box (bx, by, 1, 1), no swizzle.
bool make_map_raw_4d(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t dx, uint64_t dy,
                     uint64_t dz, uint64_t dw, uint64_t sy_bytes, uint64_t sz_bytes, uint64_t sw_bytes,
                     uint32_t bx, uint32_t by)
{
    MapKey key;
    memset(&key, 0, sizeof(key));
    key.base = base;
    key.dims[0] = dx, key.dims[1] = dy, key.dims[2] = dz, key.dims[3] = dw;
    key.strides[0] = sy_bytes, key.strides[1] = sz_bytes, key.strides[2] = sw_bytes;
    key.box[0] = bx, key.box[1] = by;
    key.dtype = 100 + (int)dt;
    if (map_cache_find(key, m)) return true;
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {dx, dy, dz, dw};
    cuuint64_t strides[3] = {sy_bytes, sz_bytes, sw_bytes};
    cuuint32_t box[4] = {bx, by, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    if (fn(m, dt, 4, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    map_cache_put(key, *m);
    return true;
}

bool strides_ok(const int64_t s[3], size_t es)
{
    const int64_t q = (int64_t)(16 / es);
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] % q != 0) return false;
    return true;
}

}  // namespace
}  // namespace think
