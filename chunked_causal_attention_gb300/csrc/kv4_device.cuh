// Device helpers of the 4-bit cache: conversions of e2m1 codes and e4m3 scales
// (PTX cvt of sm_100 and later) and small reductions.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kv4.h"

namespace attn {
namespace kv4 {

// Programmatic dependent launch: a kernel launched with it may start while the one
// before it in the stream runs, and waits in grid_wait until that one has ended and its
// writes are visible. Every block of every kernel here waits, so that no kernel ends
// ahead of the one before it, and lets the next one go only then: what a kernel reads
// before its own wait has to be older than the kernel before it.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// Let the next kernel of the stream be launched.
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A launch that may begin before the kernel ahead of it ends. Clusters (cluster > 1 blocks
// each) are launched after it: they wait for whole groups of SMs, and were slower early
// (eviction from 128K slots 32 against 25 us).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at = {};
    if (cluster > 1) {
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = cluster;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
    } else {
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return counted(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// The two e2m1 codes of byte I of w as f16x2 (low code in the low half).
template <int I>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
    uint32_t d;
    if constexpr (I == 0)
        asm("{\n .reg .b8 x, y, z, t;\n mov.b32 {x, y, z, t}, %1;\n cvt.rn.f16x2.e2m1x2 %0, x;\n}\n" : "=r"(d) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n .reg .b8 x, y, z, t;\n mov.b32 {x, y, z, t}, %1;\n cvt.rn.f16x2.e2m1x2 %0, y;\n}\n" : "=r"(d) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n .reg .b8 x, y, z, t;\n mov.b32 {x, y, z, t}, %1;\n cvt.rn.f16x2.e2m1x2 %0, z;\n}\n" : "=r"(d) : "r"(w));
    else
        asm("{\n .reg .b8 x, y, z, t;\n mov.b32 {x, y, z, t}, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(d) : "r"(w));
    return d;
}

// Two e4m3 scales (low byte first) as f16x2.
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t two) {
    uint32_t d;
    asm("{\n .reg .b16 x;\n cvt.u16.u32 x, %1;\n cvt.rn.f16x2.e4m3x2 %0, x;\n}\n" : "=r"(d) : "r"(two));
    return d;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// (lo, hi) -> one byte of two e2m1 codes (lo in the low four bits), to nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t d;
    asm("{\n .reg .b8 x, z;\n mov.b16 {z, x}, 0;\n cvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n mov.b32 %0, {x, z, z, z};\n}\n"
        : "=r"(d)
        : "f"(lo), "f"(hi));
    return d;
}

// One e4m3 value, to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3(float x) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n" : "=h"(d) : "f"(x), "f"(0.f));
    return d & 0xFFu;
}

// lens[b], taken into [0, most] (ATTN_E_BOUNDS if it is not there).
__device__ __forceinline__ int32_t length_of(const int32_t* lens, int32_t b, int32_t most, uint32_t* status) {
    const int32_t n = lens[b];
    if (n < 0 || n > most) set_error(status, ATTN_E_BOUNDS);
    return min(max(n, 0), most);
}

}  // namespace kv4
}  // namespace attn
