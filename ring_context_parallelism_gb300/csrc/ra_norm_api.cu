// ra_norm_api.cu -- the C ABI's norm of the heads with the rotation by position: host-side
// validation and dispatch.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/ra.h"
#include "ra_internal.h"

namespace {

template <typename... A>
ra_status fail(ra_status st, const char* fmt, A... a) {
    return static_cast<ra_status>(ra::set_error(st, fmt, a...));
}

ra_status ok() { return static_cast<ra_status>(ra::set_error(RA_OK, "")); }

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kMaxHeads = 1 << 16;

// Sizes, the weights and what the rotation goes by; fills those fields of a.
ra_status check_norm(const void* q_weight, const void* k_weight, const int* positions, const float* inv_freq, int R, int Hq,
                     int Hkv, int D, int rot, const int* sections, int n_axes, int interleaved, float eps, ra_dtype dt,
                     ra::NormRopeArgs* a) {
    if (dt != RA_BF16 && dt != RA_F32) return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dt));
    if (D != 64 && D != 128) return fail(RA_ERR_INVALID_ARG, "D must be 64 or 128 (got %d)", D);
    if (Hq < 1 || Hkv < 1 || Hq > kMaxHeads || Hkv > kMaxHeads)
        return fail(RA_ERR_INVALID_ARG, "Hq and Hkv must be in [1, 2^16]");
    if (R < 0 || R > (1 << 30)) return fail(RA_ERR_INVALID_ARG, "R must be in [0, 2^30]");
    // every (token, step of a warp's heads) has a number that a grid holds
    if (static_cast<long long>(R) * (Hq + Hkv) > INT_MAX) return fail(RA_ERR_INVALID_ARG, "R * (Hq + Hkv) too large");
    if (rot < 0 || rot > D || rot % 8) return fail(RA_ERR_INVALID_ARG, "rot must be a multiple of 8 in [0, D] (got %d)", rot);
    if (!std::isfinite(eps) || eps < 0.f) return fail(RA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!q_weight != !k_weight) return fail(RA_ERR_INVALID_ARG, "one weight without the other");
    if (!aligned(q_weight, 16) || !aligned(k_weight, 16))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (rot) {
        if (n_axes < 1 || n_axes > ra::kMaxAxes || !sections)
            return fail(RA_ERR_INVALID_ARG, "one to %d position axes, with their sections, required", ra::kMaxAxes);
        long long pairs = 0;
        for (int i = 0; i < n_axes; ++i) {
            if (sections[i] < 0) return fail(RA_ERR_INVALID_ARG, "negative section");
            pairs += sections[i];
        }
        if (pairs != rot / 2)
            return fail(RA_ERR_INVALID_ARG, "sections of %lld pairs, %d are rotated", pairs, rot / 2);
        if (R > 0 && (!positions || !inv_freq)) return fail(RA_ERR_INVALID_ARG, "null positions or inv_freq");
        if (!aligned(positions, 4) || !aligned(inv_freq, 4))
            return fail(RA_ERR_INVALID_ARG, "positions and inv_freq must be 4-byte aligned");
    }
    int end = 0;
    for (int i = 0; i < ra::kMaxAxes - 1; ++i) {
        if (rot && i < n_axes) end += sections[i];
        a->section_end[i] = rot && i < n_axes - 1 ? end : INT_MAX;
    }
    a->q_weight = q_weight;
    a->k_weight = k_weight;
    a->positions = positions;
    a->inv_freq = inv_freq;
    a->R = R;
    a->Hq = Hq;
    a->Hkv = Hkv;
    a->D = D;
    a->rot = rot;
    a->eps = eps;
    a->interleaved = interleaved ? 1 : 0;
    a->bf16 = dt == RA_BF16;
    return RA_OK;
}

// A tensor of tokens `stride` elements apart.
ra_status check_rows(const void* p, long long stride, int heads, bool written, const ra::NormRopeArgs& a) {
    if (a.R == 0) return RA_OK;
    const int step = a.bf16 ? 8 : 4;  // elements in 16 bytes
    if (!p) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(p, 16)) return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (stride < 0 || stride % step || stride > (1ll << 31))
        return fail(RA_ERR_INVALID_ARG, "strides must be multiples of 16 bytes, at most 2^31 elements");
    if (written && a.R > 1 && stride < static_cast<long long>(heads) * a.D)
        return fail(RA_ERR_INVALID_ARG, "the tokens of an output overlap");
    return RA_OK;
}

// Results over their own input, token by token, are fine; at other strides, over the other input or the other result they
// would be read after they were written.
ra_status check_in_place(const void* y, long long y_stride, const void* x, long long x_stride, const void* other,
                         const void* other_y, const ra::NormRopeArgs& a) {
    if (a.R == 0) return RA_OK;
    if (y == x && a.R > 1 && y_stride != x_stride)
        return fail(RA_ERR_INVALID_ARG, "a result over its input at another stride");
    if (y == other || y == other_y) return fail(RA_ERR_INVALID_ARG, "a result over the other's memory");
    return RA_OK;
}

}  // namespace

extern "C" {

ra_status ra_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride, const void* q_weight,
                          const void* k_weight, const int* positions, const float* inv_freq, void* q_out,
                          long long q_out_stride, void* k_out, long long k_out_stride, int R, int Hq, int Hkv, int D, int rot,
                          const int* sections, int n_axes, int interleaved, float eps, ra_dtype dt, void* stream) {
    ra::NormRopeArgs a{};
    ra_status st = check_norm(q_weight, k_weight, positions, inv_freq, R, Hq, Hkv, D, rot, sections, n_axes, interleaved, eps,
                              dt, &a);
    if (st == RA_OK) st = check_rows(q, q_stride, Hq, false, a);
    if (st == RA_OK) st = check_rows(k, k_stride, Hkv, false, a);
    if (st == RA_OK) st = check_rows(q_out, q_out_stride, Hq, true, a);
    if (st == RA_OK) st = check_rows(k_out, k_out_stride, Hkv, true, a);
    if (st == RA_OK) st = check_in_place(q_out, q_out_stride, q, q_stride, k, k_out, a);
    if (st == RA_OK) st = check_in_place(k_out, k_out_stride, k, k_stride, q, q_out, a);
    if (st != RA_OK) return st;
    if (R == 0) return ok();
    a.q = q;
    a.k = k;
    a.q_row = q_stride;
    a.k_row = k_stride;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_out_row = q_out_stride;
    a.k_out_row = k_out_stride;
    const cudaError_t e = ra::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "head norm launch: %s", cudaGetErrorString(e));
    return ok();
}

size_t ra_qk_norm_rope_bwd_workspace_size(int D) {
    if (D != 64 && D != 128) return 0;
    return sizeof(float) * D * static_cast<size_t>(ra::norm_rope_bwd_ctas());
}

ra_status ra_qk_norm_rope_bwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* q_weight,
                              const void* k_weight, const int* positions, const float* inv_freq, const void* dq_out,
                              const void* dk_out, void* dq, long long dq_stride, void* dk, long long dk_stride,
                              float* dq_weight, float* dk_weight, int R, int Hq, int Hkv, int D, int rot, const int* sections,
                              int n_axes, int interleaved, float eps, ra_dtype dt, void* workspace, size_t workspace_bytes,
                              void* stream) {
    ra::NormRopeArgs a{};
    ra_status st = check_norm(q_weight, k_weight, positions, inv_freq, R, Hq, Hkv, D, rot, sections, n_axes, interleaved, eps,
                              dt, &a);
    if (st == RA_OK && q_weight) st = check_rows(q, q_stride, Hq, false, a);
    if (st == RA_OK && q_weight) st = check_rows(k, k_stride, Hkv, false, a);
    if (st == RA_OK) st = check_rows(dq_out, 0, Hq, false, a);
    if (st == RA_OK) st = check_rows(dk_out, 0, Hkv, false, a);
    if (st == RA_OK) st = check_rows(dq, dq_stride, Hq, true, a);
    if (st == RA_OK) st = check_rows(dk, dk_stride, Hkv, true, a);
    const long long gq_stride = static_cast<long long>(Hq) * D, gk_stride = static_cast<long long>(Hkv) * D;
    if (st == RA_OK) st = check_in_place(dq, dq_stride, dq_out, gq_stride, dk_out, dk, a);
    if (st == RA_OK) st = check_in_place(dk, dk_stride, dk_out, gk_stride, dq_out, dq, a);
    if (st == RA_OK && q_weight) st = check_in_place(dq, dq_stride, q, q_stride, k, dk, a);
    if (st == RA_OK && q_weight) st = check_in_place(dk, dk_stride, k, k_stride, q, dq, a);
    if (st != RA_OK) return st;
    if (q_weight) {
        if (!dq_weight || !dk_weight) return fail(RA_ERR_INVALID_ARG, "null weight gradient");
        if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))
            return fail(RA_ERR_INVALID_ARG, "weight gradients must be 4-byte aligned");
        const size_t need = ra_qk_norm_rope_bwd_workspace_size(D);
        if (!workspace) return fail(RA_ERR_WORKSPACE, "workspace is NULL");
        if (!aligned(workspace, 256)) return fail(RA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
        if (workspace_bytes < need)
            return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    } else if (R == 0) {
        return ok();
    }
    a.q = q;
    a.k = k;
    a.q_row = q_stride;
    a.k_row = k_stride;
    a.dq_out = dq_out;
    a.dk_out = dk_out;
    a.q_out = dq;
    a.k_out = dk;
    a.q_out_row = dq_stride;
    a.k_out_row = dk_stride;
    const cudaError_t e = ra::launch_norm_rope_bwd(a, static_cast<float*>(workspace), dq_weight, dk_weight,
                                                   static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "head norm gradient launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
