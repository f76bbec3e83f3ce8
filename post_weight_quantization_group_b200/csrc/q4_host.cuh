// q4_host.cuh -- host-side helpers shared by the translation units of the C
// ABI (q4_api.cu, kv_api.cu): device queries, TMA descriptor encoding, kernel
// attributes and launches, the device status word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <utility>

#include "q4.h"

// Device address of the library's status word (see q4dev::kStatusTimeout) on
// the current device, or nullptr if the lookup fails; defined in q4_api.cu.
unsigned* q4_status_word();

namespace {

constexpr int kMaxDevices = 64;

[[maybe_unused]] bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

[[maybe_unused]] int current_device() {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) return -1;
    return d;
}

[[maybe_unused]] int sm_count(int dev) {
    static std::atomic<int> cache[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return 148;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

[[maybe_unused]] int max_smem_optin(int dev) {
    static std::atomic<int> cache[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return 227 * 1024;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        n <= 0)
        n = 227 * 1024;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda
// link dependency).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

[[maybe_unused]] EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D row-major tensor [rows, cols] of `elem` bytes, box [box_rows, box_cols],
// out-of-bounds elements read as zero.
[[maybe_unused]] bool make_tmap_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int elem,
                  uint64_t rows, uint64_t cols, uint32_t box_rows, uint32_t box_cols,
                  CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * static_cast<uint64_t>(elem)};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

[[maybe_unused]] q4_status launch_status(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

// Per-(kernel, device) one-time attribute setup.
template <typename K>
bool set_kernel_attrs(K kernel, int smem_bytes, bool nonportable_cluster) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes);
    if (e != cudaSuccess) return false;
    if (nonportable_cluster) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return false;
    }
    return true;
}

// Launch with an optional cluster shape and, for kernels written for it,
// programmatic stream serialization (the kernel may start before the previous
// kernel of the stream has finished; it waits with griddepcontrol.wait).
template <typename... KArgs, typename... Args>
q4_status launch_ex(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                    int cluster_x, bool pdl, cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster_x > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster_x;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = n ? attr : nullptr;
    cfg.numAttrs = n;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

[[maybe_unused]] bool valid_dtype(int d) { return d == Q4_F16 || d == Q4_BF16 || d == Q4_F32; }

// Workspace layout, the same for every shape, batch and kernel so that one
// buffer can serve any sequence of calls: [one counter per row tile, at most
// 65535 tiles: kWsCounterBytes] [partial slots of the launch's grid].
// Counters are reset by every call that uses them; partial slots never
// overlap counters.
constexpr size_t kWsCounterBytes = static_cast<size_t>(65536) * 4;

}  // namespace
