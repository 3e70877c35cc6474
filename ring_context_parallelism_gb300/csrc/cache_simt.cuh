// cache_simt.cuh -- what the CUDA-core kernels over a batch of paged sequences share.
#pragma once

#include "cache_batch.cuh"

namespace ra {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 bytes from global to shared memory, zeros where !ok.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Whether new token t (stacked row lo + t) of a sequence sees its key j.
__device__ __forceinline__ bool sees(const CacheBatch& p, const CacheSeq& s, int t, int j) {
    if (j >= s.kv) return false;
    const int jn = j - (s.kv - s.n);
    if (jn < 0) return true;
    if (!p.tree_mask) return jn <= t;
    return jn < p.mask_cols && p.tree_mask[static_cast<long long>(s.lo + t) * p.mask_cols + jn] != 0;
}

}  // namespace ra
