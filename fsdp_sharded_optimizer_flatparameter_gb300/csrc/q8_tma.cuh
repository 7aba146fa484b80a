// Barriers, tiled copies and tensor maps that the 8-bit kernels share.
#pragma once

#include <cuda.h>

#include <atomic>

#include "q8.cuh"

namespace zs {

constexpr int kMaxDevices = 64;

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
// Counts bytes as landed that a copy never issued would have brought.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, long long limit) {
    if (mbar_try_wait(b, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(b, parity)) {
        if (clock64() - t0 > limit) return false;
    }
    return true;
}

// The same, which looks once with a limit of 0 (try_wait itself may wait).  The waits of the products' warp, which is short
// of issue slots, do without that test (8192 x 22016 x 4096: 511 us with it, 496 without).
__device__ __forceinline__ bool mbar_wait_or_look(uint64_t* b, uint32_t parity, long long limit) {
    if (limit != 0) return mbar_wait(b, parity, limit);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}

// What a wait may take (zs_set_q8_wait_limit changes it), and a wait for what is under way already, which a kernel that
// gave up makes before its shared memory goes: ~2 s at the 2.07 GHz maximum SM clock.
constexpr long long kWaitLimit = 4000000000LL, kDrainLimit = 4000000000LL;

// A whole warp, lane k for barrier k: waits for the last of the `count` events that came to a ring of barriers in turn.
__device__ __forceinline__ void ring_settled(uint64_t* ring, uint32_t stages, uint32_t count) {
    const uint32_t lane = threadIdx.x & 31;
    if (lane < stages && lane < count) mbar_wait(ring + lane, ((count - 1 - lane) / stages) & 1, kDrainLimit);
    __syncwarp();
}

// A map's box at column x and row y; x is a multiple of 128 elements here, so that the copy starts on a
// 16-byte boundary as it must.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            su32(dst)),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(su32(bar))
        : "memory");
}

// The two halves of dependent_launch_prologue with what touches no global memory between them: barriers, the
// tensor memory's allocation (it may wait for the predecessor's CTAs on this SM to release theirs, which never
// wait for this kernel) and the fetch of the maps overlap the predecessor's end.
__device__ __forceinline__ void early_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)map) : "memory");
}

// ------------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// A matrix of rows x cols elements (`pitch` bytes between rows) in boxes of box_rows x box_cols; what lies past its
// rows and columns reads as 0.  A thread that has made no CUDA call of its own yet has no current context,
// which the driver call needs; the runtime binds the device's own on cudaSetDevice.
inline cudaError_t make_map(CUtensorMap* map, const void* p, bool bf16, int64_t rows, int64_t cols, int64_t pitch, int box_rows,
                            int box_cols, CUtensorMapSwizzle swizzle) {
    if (!encode_tiled()) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, unit[2] = {1, 1};
    for (int attempt = 0; attempt < 2; ++attempt) {
        if (encode_tiled()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void*)p, dims, strides,
                           box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            return cudaSuccess;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaSetDevice(dev);
        if (e != cudaSuccess) return e;
    }
    return cudaErrorInvalidValue;
}

// Raises a kernel's dynamic shared-memory limit once per device.
inline cudaError_t ready_once(std::atomic<uint64_t>& ready, const void* kern, int smem) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (ready.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < kMaxDevices) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return e;
}

// Cycles that a wait of the 8-bit kernels may take.
inline std::atomic<long long>& wait_limit() {
    static std::atomic<long long> cycles{kWaitLimit};
    return cycles;
}

// The current device's status word (zs_device_status).
inline cudaError_t error_word(unsigned int** out) {
    static std::atomic<unsigned int*> cached[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*out = cached[dev].load(std::memory_order_acquire))) return cudaSuccess;
    e = device_error_word(out);
    if (e == cudaSuccess && dev < kMaxDevices) cached[dev].store(*out, std::memory_order_release);
    return e;
}

}  // namespace zs
