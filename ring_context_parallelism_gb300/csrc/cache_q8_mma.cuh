// cache_q8_mma.cuh -- what the tensor-core kernels over an 8-bit cache share: MMAs of 8-bit
// operands, their tiles in shared memory, and the queries as two 8-bit parts.
#pragma once

#include "cache_q8.cuh"

namespace ra {

// What the kernels take besides the tensor maps of the pages.
struct Q8Params {
    CacheBatch p;
    float scale_log2;
    const __nv_bfloat16* q;
    const unsigned char *ks, *vs;
    __nv_bfloat16* out;
    float* lse;
    JoinJob* jobs;
    float2* stats;
    float* part_o;
    int slot_rows;
    int columns, heads;  // KV heads are walked in `columns` of `heads` each
};

// The CTAs of a call walk the batch's keys in columns of KV heads, side by side: CTA blockIdx = range * columns + column
// walks the range'th part of the batch's work over the column's heads (one, but for more heads than CTAs).  A token's
// heads lie next to each other in a page, a row of 128 bytes each: walked at the same time, they are read from DRAM
// while its pages are open (the decode batch of cache_q8_tc.cu, in units of 16 rows: 128 us one head after the other, 112 side by side).  Ranges of a column are
// numbered one after the other, as the join of cut units goes.
struct Column {
    int index, ranges, range, cta;  // cta: its number in the order of the join
};
__device__ __forceinline__ Column column_of(int columns) {
    const int ranges = gridDim.x / columns, index = blockIdx.x % columns, range = blockIdx.x / columns;
    return {index, ranges, range, index * ranges + range};
}

// The kernel for many rows (cache_q8_wide.cu): nt row tiles of 128 rows to a unit, and the keys of its tiles.
int q8_wide_key_tile(int nt);
cudaError_t launch_q8_wide(int D, int nt, const CUtensorMap& k, const CUtensorMap& v, const Q8Params& a, int ctas,
                           cudaStream_t stream);

// D[tmem] (+)= A[smem] . B[smem]^T  (kind::f8f6f4, one CTA)
__device__ __forceinline__ void mma8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: fp32 results; A e4m3; B e4m3 or e5m2.
constexpr uint32_t idesc8(int N, bool b_e5m2, bool mn_major) {
    return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (mn_major ? (1u << 15) | (1u << 16) : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// Tiles of `pitch` bytes a row, swizzled as the tensor copies write them: 128 bytes (16-byte pieces of row r in place
// p ^ r % 8) or 64 (p ^ r / 2 % 4).  The high word of a descriptor for eight-row groups one after the other.
constexpr uint32_t desc_hi(int pitch) {
    return static_cast<uint32_t>(8 * pitch >> 4) | (1u << 14) | ((pitch == 128 ? 2u : 4u) << 29);
}
__device__ __forceinline__ uint64_t desc8(uint32_t hi, uint32_t lo) { return static_cast<uint64_t>(hi) << 32 | lo; }
template <int PITCH>
__device__ __forceinline__ int piece_at(int row, int piece) {
    return row * PITCH + ((piece ^ (PITCH == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}

// Codes of four queries' two parts: the row's values times f are at most 256; the first part keeps four bits, the second
// what is left.
__device__ __forceinline__ void query_parts4(const float* x, float f, uint32_t& hi, uint32_t& lo) {
    hi = codes4(x, f);
    float y[4];
    values4(hi, y);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(x[j], f, -y[j]);
    lo = codes4(y, 1.f);
}

// The power of two that brings a row whose largest magnitude has these bits to [128, 256), as a scale byte; its inverse
// is 254 - byte.
__device__ __forceinline__ int query_scale_byte(uint32_t largest) { return min(261 - static_cast<int>(largest >> 23), 253); }

// The scales of four keys of a tile per lane (of one page: they start on a multiple of four); zeros without a page.
__device__ __forceinline__ void copy_scales4(unsigned char* dst, const unsigned char* src, bool have) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(have ? 4 : 0) : "memory");
}
// Arrives once the thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace ra
