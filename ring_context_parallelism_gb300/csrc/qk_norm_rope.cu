// qk_norm_rope.cu -- the RMS norm of every head of a token's queries and keys and the
// rotation by the token's position, in one pass, and the gradient of both.
//
//   n = x r, r = (mean(x^2) + eps)^(-1/2);  y = n w;  pair i of the rotated dims is turned
//   by angle_i = position[axis of i] * inv_freq[i]:  (a, b) -> (a c - b s, b c + a s).
// Backward, for the upstream gradient dy: g = dy turned back, dx = r (g w - n mean(g w n)),
// dw = the sum over rows and heads of g n.
//
// D / 8 lanes hold a head, eight dims (four pairs) each; a warp takes one token and walks
// some of its heads, so that the angles and weights of its lanes' pairs are found once.
// Everything between the load and the store is fp32; the result is rounded once.
//
// Angles: a far position times a frequency leaves no bits of the fraction of a turn in fp32.
// inv_freq / 2 pi is taken as a 64-bit binary fraction of a turn (a product in fp64, off by
// 2^-53 of itself); a position times it, modulo 2^64, drops whole turns exactly.
//
// Bytes bound it: each value is read once and written once.
#include <cmath>

#include "cache_batch.cuh"

namespace ra {

namespace {

constexpr int kThreads = 128;

template <typename T>
struct Four;  // four consecutive elements as one load
template <>
struct Four<__nv_bfloat16> {
    using V = uint2;
    static __device__ __forceinline__ void get(V v, float* x) {
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    static __device__ __forceinline__ V put(const float* x) { return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); }
};
template <>
struct Four<float> {
    using V = float4;
    static __device__ __forceinline__ void get(V v, float* x) {
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    }
    static __device__ __forceinline__ V put(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};

// The dims of lane `l` of a head: four at e0 and four at e1.  Pairs in halves: (e0 + j, e1 + j); next to each other:
// (e0, e0 + 1), (e0 + 2, e0 + 3) and as much at e1.
struct LaneDims {
    int e0, e1;
    bool turns;
};
__device__ __forceinline__ LaneDims lane_dims(int l, int rot, bool interleaved) {
    const bool turns = 8 * l < rot;
    if (interleaved || !turns) return {8 * l, 8 * l + 4, turns};
    return {4 * l, rot / 2 + 4 * l, true};
}

// cos and sin of the four pairs of a lane at one token.
__device__ __forceinline__ void pair_angles(const NormRopeArgs& a, int l, int row, float* c, float* s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = 4 * l + j;
        int axis = 0;
#pragma unroll
        for (int x = 0; x < kMaxAxes - 1; ++x) axis += i >= a.section_end[x] ? 1 : 0;
        const float f = a.inv_freq[i];
        const double turns = static_cast<double>(f) * 0.15915494309189533577;  // 1 / (2 pi)
        const double part = turns - floor(turns);
        const unsigned long long step = static_cast<unsigned long long>(part * 18446744073709551616.0);
        const long long pos = a.positions[static_cast<long long>(axis) * a.R + row];
        const unsigned long long at = static_cast<unsigned long long>(pos) * step;
        const float half_turns = static_cast<float>(static_cast<int>(at >> 32)) * 4.656612873077393e-10f;  // 2^-31
        sincospif(isfinite(f) ? half_turns : NAN, &s[j], &c[j]);
    }
}

// The lane's eight dims as the firsts and seconds of its pairs, and back.
template <bool INTER>
__device__ __forceinline__ void to_pairs(const float* x0, const float* x1, float* a, float* b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a[j] = INTER ? (j < 2 ? x0[2 * j] : x1[2 * j - 4]) : x0[j];
        b[j] = INTER ? (j < 2 ? x0[2 * j + 1] : x1[2 * j - 3]) : x1[j];
    }
}
template <bool INTER>
__device__ __forceinline__ void from_pairs(const float* a, const float* b, float* x0, float* x1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x0[j] = INTER ? (j & 1 ? b[j / 2] : a[j / 2]) : a[j];
        x1[j] = INTER ? (j & 1 ? b[2 + j / 2] : a[2 + j / 2]) : b[j];
    }
}

template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Weights of a lane's pairs (ones without a norm).
template <typename T, bool INTER, bool NORM>
__device__ __forceinline__ void load_weight(const void* w, const LaneDims& d, float* a, float* b) {
    float x0[4] = {1.f, 1.f, 1.f, 1.f}, x1[4] = {1.f, 1.f, 1.f, 1.f};
    if (NORM) {
        using F = Four<T>;
        F::get(*reinterpret_cast<const typename F::V*>(static_cast<const T*>(w) + d.e0), x0);
        F::get(*reinterpret_cast<const typename F::V*>(static_cast<const T*>(w) + d.e1), x1);
    }
    to_pairs<INTER>(x0, x1, a, b);
}

// A token's heads are walked in steps of the 32 / LANES heads that a warp holds, queries first.  `per` steps make an
// item; a warp takes an item.
template <int D>
struct Steps {
    static constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    int q, all;
    __host__ __device__ __forceinline__ Steps(int Hq, int Hkv)
        : q((Hq + kHeads - 1) / kHeads), all(q + (Hkv + kHeads - 1) / kHeads) {}
};

template <typename T, int D, bool INTER, bool NORM, int DEPTH>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int per, int chunks) {
    using S = Steps<D>;
    using F = Four<T>;
    using V = typename F::V;
    const S steps(a.Hq, a.Hkv);
    const int lane = threadIdx.x & 31, l = lane % S::kLanes, sub = lane / S::kLanes;
    const long long item = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.R) * chunks) return;
    const int row = static_cast<int>(item / chunks), i0 = static_cast<int>(item % chunks) * per, i1 = min(steps.all, i0 + per);
    const LaneDims d = lane_dims(l, a.rot, INTER);
    grid_dependency_wait();
    // the first heads are on their way while the angles are found
    V x0[DEPTH], x1[DEPTH];
    auto head_of = [&](int i, bool& is_q) {
        is_q = i < steps.q;
        const int h = (is_q ? i : i - steps.q) * S::kHeads + sub;
        return i < i1 && h < (is_q ? a.Hq : a.Hkv) ? h : -1;
    };
    auto load = [&](int i, int u) {
        bool is_q;
        const int h = head_of(i, is_q);
        x0[u] = x1[u] = V{};
        if (h >= 0) {
            const T* p = static_cast<const T*>(is_q ? a.q : a.k) + row * (is_q ? a.q_row : a.k_row) + h * D;
            x0[u] = *reinterpret_cast<const V*>(p + d.e0);
            x1[u] = *reinterpret_cast<const V*>(p + d.e1);
        }
    };
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) load(i0 + u, u);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (d.turns) pair_angles(a, l, row, c, s);
    float wqa[4], wqb[4], wka[4], wkb[4];
    load_weight<T, INTER, NORM>(a.q_weight, d, wqa, wqb);
    load_weight<T, INTER, NORM>(a.k_weight, d, wka, wkb);
    for (int base = i0; base < i1; base += DEPTH) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            const int i = base + u;
            if (i >= i1) break;
            bool is_q;
            const int h = head_of(i, is_q);
            float y0[4], y1[4], pa[4], pb[4];
            F::get(x0[u], y0);
            F::get(x1[u], y1);
            load(i + DEPTH, u);
            if (NORM) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = fmaf(y0[j], y0[j], fmaf(y1[j], y1[j], sum));
                const float r = rsqrtf(head_sum<S::kLanes>(sum) * (1.f / D) + a.eps);
                to_pairs<INTER>(y0, y1, pa, pb);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pa[j] *= r * (is_q ? wqa[j] : wka[j]);
                    pb[j] *= r * (is_q ? wqb[j] : wkb[j]);
                }
            } else {
                to_pairs<INTER>(y0, y1, pa, pb);
            }
            float ya[4], yb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ya[j] = fmaf(pa[j], c[j], -pb[j] * s[j]);
                yb[j] = fmaf(pb[j], c[j], pa[j] * s[j]);
            }
            if (!d.turns) {  // as they are, whatever 0 times them would be
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ya[j] = pa[j];
                    yb[j] = pb[j];
                }
            }
            if (h >= 0) {
                T* p = static_cast<T*>(is_q ? a.q_out : a.k_out) + row * (is_q ? a.q_out_row : a.k_out_row) + h * D;
                from_pairs<INTER>(ya, yb, y0, y1);
                *reinterpret_cast<V*>(p + d.e0) = F::put(y0);
                *reinterpret_cast<V*>(p + d.e1) = F::put(y1);
            }
        }
    }
}

// Gradient: warps take items in a fixed stride and keep the sums of their lanes' dw; a CTA's are added up in a fixed
// order and written to its row of `parts` [CTAs][2 D], which the next kernel adds up.
template <typename T, int D, bool INTER, bool NORM, int DEPTH>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, int per, int chunks,
                                                                 float* parts) {
    using S = Steps<D>;
    using F = Four<T>;
    using V = typename F::V;
    constexpr int kWarps = kThreads / 32;
    __shared__ float sums[kWarps][2 * D];
    const S steps(a.Hq, a.Hkv);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % S::kLanes, sub = lane / S::kLanes;
    const LaneDims d = lane_dims(l, a.rot, INTER);
    const long long items = static_cast<long long>(a.R) * chunks;
    grid_dependency_wait();
    float wqa[4], wqb[4], wka[4], wkb[4];
    load_weight<T, INTER, NORM>(a.q_weight, d, wqa, wqb);
    load_weight<T, INTER, NORM>(a.k_weight, d, wka, wkb);
    float dqa[4] = {}, dqb[4] = {}, dka[4] = {}, dkb[4] = {};
    for (long long item = static_cast<long long>(blockIdx.x) * kWarps + warp; item < items;
         item += static_cast<long long>(gridDim.x) * kWarps) {
        const int row = static_cast<int>(item / chunks), i0 = static_cast<int>(item % chunks) * per, i1 = min(steps.all, i0 + per);
        auto head_of = [&](int i, bool& is_q) {
            is_q = i < steps.q;
            const int h = (is_q ? i : i - steps.q) * S::kHeads + sub;
            return i < i1 && h < (is_q ? a.Hq : a.Hkv) ? h : -1;
        };
        V x0[DEPTH], x1[DEPTH], g0[DEPTH], g1[DEPTH];
        auto load = [&](int i, int u) {
            bool is_q;
            const int h = head_of(i, is_q);
            x0[u] = x1[u] = g0[u] = g1[u] = V{};
            if (h >= 0) {
                const T* g = static_cast<const T*>(is_q ? a.dq_out : a.dk_out) +
                             (static_cast<long long>(row) * (is_q ? a.Hq : a.Hkv) + h) * D;
                g0[u] = *reinterpret_cast<const V*>(g + d.e0);
                g1[u] = *reinterpret_cast<const V*>(g + d.e1);
                if (NORM) {
                    const T* p = static_cast<const T*>(is_q ? a.q : a.k) + row * (is_q ? a.q_row : a.k_row) + h * D;
                    x0[u] = *reinterpret_cast<const V*>(p + d.e0);
                    x1[u] = *reinterpret_cast<const V*>(p + d.e1);
                }
            }
        };
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) load(i0 + u, u);
        float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
        if (d.turns) pair_angles(a, l, row, c, s);
        for (int base = i0; base < i1; base += DEPTH) {
#pragma unroll
            for (int u = 0; u < DEPTH; ++u) {
                const int i = base + u;
                if (i >= i1) break;
                bool is_q;
                const int h = head_of(i, is_q);
                float y0[4], y1[4], ya[4], yb[4], ga[4], gb[4];
                F::get(g0[u], y0);
                F::get(g1[u], y1);
                to_pairs<INTER>(y0, y1, ya, yb);
                F::get(x0[u], y0);
                F::get(x1[u], y1);
                load(i + DEPTH, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ga[j] = d.turns ? fmaf(ya[j], c[j], yb[j] * s[j]) : ya[j];
                    gb[j] = d.turns ? fmaf(yb[j], c[j], -ya[j] * s[j]) : yb[j];
                }
                if (NORM) {
                    float xa[4], xb[4], sq = 0.f, dot = 0.f;
                    to_pairs<INTER>(y0, y1, xa, xb);
                    float va[4], vb[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        va[j] = ga[j] * (is_q ? wqa[j] : wka[j]);
                        vb[j] = gb[j] * (is_q ? wqb[j] : wkb[j]);
                        sq = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], sq));
                        dot = fmaf(va[j], xa[j], fmaf(vb[j], xb[j], dot));
                    }
                    const float r = rsqrtf(head_sum<S::kLanes>(sq) * (1.f / D) + a.eps);
                    const float m = head_sum<S::kLanes>(dot) * r * (1.f / D);  // mean(g w n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float na = xa[j] * r, nb = xb[j] * r;
                        const float ta = ga[j] * na, tb = gb[j] * nb;
                        if (is_q) {
                            dqa[j] += ta;
                            dqb[j] += tb;
                        } else {
                            dka[j] += ta;
                            dkb[j] += tb;
                        }
                        ga[j] = r * (va[j] - na * m);
                        gb[j] = r * (vb[j] - nb * m);
                    }
                }
                if (h >= 0) {
                    T* p = static_cast<T*>(is_q ? a.q_out : a.k_out) + row * (is_q ? a.q_out_row : a.k_out_row) + h * D;
                    from_pairs<INTER>(ga, gb, y0, y1);
                    *reinterpret_cast<V*>(p + d.e0) = F::put(y0);
                    *reinterpret_cast<V*>(p + d.e1) = F::put(y1);
                }
            }
        }
    }
    if (!NORM) return;
    // heads of the warp, then the warps
    float z[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        z[0][j] = dqa[j];
        z[1][j] = dqb[j];
        z[2][j] = dka[j];
        z[3][j] = dkb[j];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int o = S::kLanes; o < 32; o <<= 1) z[x][j] += __shfl_xor_sync(0xffffffffu, z[x][j], o);
    }
    if (sub == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float y0[4], y1[4];
            from_pairs<INTER>(z[2 * t], z[2 * t + 1], y0, y1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sums[warp][t * D + d.e0 + j] = y0[j];
                sums[warp][t * D + d.e1 + j] = y1[j];
            }
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += sums[w][x];
        parts[static_cast<long long>(blockIdx.x) * (2 * D) + x] = total;
    }
}

// dw: 32 columns of the parts per CTA, 32 threads each, in a fixed order.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* parts, int n, int D, float* dwq, float* dwk) {
    __shared__ float sums[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    grid_dependency_wait();
    float total = 0.f;
#pragma unroll 4
    for (int i = part; i < n; i += 32) total += parts[static_cast<long long>(i) * (2 * D) + col];
    sums[part][threadIdx.x & 31] = total;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) total += sums[i][threadIdx.x];
    (col < D ? dwq : dwk)[col < D ? col : col - D] = total;
}

// Steps per item: few tokens are spread over warps of one step each, many keep their angles for more heads.
int steps_per_item(long long R, int steps, int warps) {
    const long long per = (R * steps + warps - 1) / warps;
    return static_cast<int>(per < 1 ? 1 : per > steps ? steps : per);
}

constexpr int kWarpsPerSm = 32;

template <typename T, int D, bool INTER, bool NORM>
cudaError_t run_fwd(const NormRopeArgs& a, cudaStream_t stream) {
    const int steps = Steps<D>(a.Hq, a.Hkv).all, per = steps_per_item(a.R, steps, kWarpsPerSm * device_sm_count());
    const int chunks = (steps + per - 1) / per;
    const long long blocks = (static_cast<long long>(a.R) * chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_overlapped(norm_rope_kernel<T, D, INTER, NORM, 4>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream,
                             a, per, chunks);
}

template <typename T, int D, bool INTER, bool NORM>
cudaError_t run_bwd(const NormRopeArgs& a, float* parts, float* dwq, float* dwk, cudaStream_t stream) {
    const int steps = Steps<D>(a.Hq, a.Hkv).all, per = steps_per_item(a.R, steps, kWarpsPerSm * device_sm_count());
    const int chunks = (steps + per - 1) / per, most = norm_rope_bwd_ctas();
    const long long want = (static_cast<long long>(a.R) * chunks + kThreads / 32 - 1) / (kThreads / 32);
    const int ctas = static_cast<int>(want < most ? want : most);
    if (ctas) {
        const cudaError_t e = launch_overlapped(norm_rope_bwd_kernel<T, D, INTER, NORM, 2>, dim3(ctas), kThreads, 0, stream, a,
                                                per, chunks, parts);
        if (e != cudaSuccess) return e;
    }
    if (!NORM) return cudaSuccess;
    return launch_overlapped(norm_weight_grad_kernel, dim3(2 * D / 32), 1024, 0, stream, static_cast<const float*>(parts), ctas,
                             D, dwq, dwk);
}

// Calls f with the types and flags of a call as template arguments.
template <typename F>
cudaError_t with_form(const NormRopeArgs& a, F f) {
    auto flags = [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        if (a.interleaved)
            return a.q_weight ? f.template operator()<T, D, true, true>() : f.template operator()<T, D, true, false>();
        return a.q_weight ? f.template operator()<T, D, false, true>() : f.template operator()<T, D, false, false>();
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (a.bf16) return a.D == 128 ? flags(__nv_bfloat16(), D128()) : flags(__nv_bfloat16(), D64());
    return a.D == 128 ? flags(0.f, D128()) : flags(0.f, D64());
}

struct Fwd {
    const NormRopeArgs& a;
    cudaStream_t stream;
    template <typename T, int D, bool INTER, bool NORM>
    cudaError_t operator()() const {
        return run_fwd<T, D, INTER, NORM>(a, stream);
    }
};
struct Bwd {
    const NormRopeArgs& a;
    float *parts, *dwq, *dwk;
    cudaStream_t stream;
    template <typename T, int D, bool INTER, bool NORM>
    cudaError_t operator()() const {
        return run_bwd<T, D, INTER, NORM>(a, parts, dwq, dwk, stream);
    }
};

}  // namespace

int norm_rope_bwd_ctas() { return 8 * device_sm_count(); }

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) { return with_form(a, Fwd{a, stream}); }

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, float* parts, float* dwq, float* dwk, cudaStream_t stream) {
    return with_form(a, Bwd{a, parts, dwq, dwk, stream});
}

}  // namespace ra
