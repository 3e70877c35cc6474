// qk_norm_rope.cu -- the RMS norm of every head of a token's queries and keys and the
// rotation by the token's position, in one pass, and the gradient of both.
//
//   n = x r, r = (mean(x^2) + eps)^(-1/2);  y = n w;  pair i of the rotated dims is turned
//   by angle_i = position[axis of i] * inv_freq[i]:  (a, b) -> (a c - b s, b c + a s).
// Backward, for the upstream gradient dy: g = dy turned back, dx = r (g w - n mean(g w n)),
// dw = the sum over rows and heads of g n.
//
// D / 8 lanes hold a head, eight dims (four pairs) each.  A warp keeps to the queries or to the
// keys, takes a token (or some of its heads, where tokens are few), finds the angles of its
// lanes' pairs once and walks the heads; it stays for several tokens, with the next heads
// on their way whatever token they belong to.  Everything between the load and the store is
// fp32, two values to an instruction; the result is rounded once.
//
// Angles: a far position times a frequency leaves no bits of the fraction of a turn in fp32.
// inv_freq / 2 pi is taken as a 64-bit binary fraction of a turn, the 24 bits of inv_freq times
// 96 of 1 / 2 pi in integers (fp64 would take a sixth of the prompt's time: it runs at a
// sixty-fourth of fp32's rate); a position times it, modulo 2^64, drops whole turns exactly.
//
// Bytes bound it: each value is read once and written once.  8192 tokens of 32 + 8 heads in bf16: 31.6 us, 5.3
// TB/s (0.79 of the measured copy rate); the gradient 52.6 us, 4.8 TB/s, held back by its latencies (128 registers,
// 16 warps an SM, one step of each on its way; fewer registers spill); 32 tokens of 64 + 8 heads 2.5 us.
// Dims that are not rotated go by themselves, not turned by nothing, where an infinity would reach the lane's other dims
// (0.4 us of these, D = 64 and its gradient 0.9 of 29.8).
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

// f / 2 pi modulo 1 in units of 2^-64; |f| < 2^32.
__device__ __forceinline__ unsigned long long turn_step(float f) {
    const uint32_t u = __float_as_uint(f), e = u >> 23 & 255u, m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
    // 1 / 2 pi = c 2^-96
    constexpr uint32_t c2 = 0x28be60dbu, c1 = 0x9391054au, c0 = 0x7f09d5f4u;
    const unsigned long long p0 = static_cast<unsigned long long>(m) * c0;
    const unsigned long long p1 = static_cast<unsigned long long>(m) * c1 + (p0 >> 32);
    const unsigned long long p2 = static_cast<unsigned long long>(m) * c2 + (p1 >> 32);
    const uint32_t w[4] = {static_cast<uint32_t>(p0), static_cast<uint32_t>(p1), static_cast<uint32_t>(p2),
                           static_cast<uint32_t>(p2 >> 32)};
    // f = m 2^(e - 150): the product 2^(150 + 96 - 64 - e) down, at least 23 places for |f| < 2^32
    const uint32_t down = 182u - (e ? e : 1u), words = down >> 5, bits = down & 31u;
    auto word = [&](uint32_t i) { return i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : i == 3 ? w[3] : 0u; };
    const uint32_t a0 = word(words), a1 = word(words + 1), a2 = word(words + 2);
    const unsigned long long step = static_cast<unsigned long long>(__funnelshift_r(a1, a2, bits)) << 32 | __funnelshift_r(a0, a1, bits);
    return u >> 31 ? 0ull - step : step;
}

// The four pairs of a lane: their steps, and which axis' positions they go by.
struct Turns {
    unsigned long long step[4];
    const int* positions;
    unsigned axis[4];
    bool finite[4];
    __device__ __forceinline__ void start(const NormRopeArgs& a, int l) {
        positions = a.positions;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = 4 * l + j;
            axis[j] = 0;
#pragma unroll
            for (int x = 0; x < kMaxAxes - 1; ++x) axis[j] += i >= a.section_end[x] ? static_cast<unsigned>(a.R) : 0u;
            const float f = a.inv_freq[i];
            step[j] = turn_step(f);
            finite[j] = fabsf(f) < 4294967296.f;
        }
    }
    __device__ __forceinline__ void fetch(int row, int (&pos)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) pos[j] = positions[axis[j] + row];
    }
    __device__ __forceinline__ void angles(const int (&pos)[4], float* c, float* s) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned long long at = static_cast<unsigned long long>(static_cast<long long>(pos[j])) * step[j];
            const float half_turns = static_cast<float>(static_cast<int>(at >> 32)) * 4.656612873077393e-10f;  // 2^-31
            sincospif(finite[j] ? half_turns : NAN, &s[j], &c[j]);
        }
    }
};

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

// Sums over the lanes of a head, of N values at a time.
template <int LANES, int N>
__device__ __forceinline__ void head_sums(float (&x)[N]) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1)
#pragma unroll
        for (int v = 0; v < N; ++v) x[v] += __shfl_xor_sync(0xffffffffu, x[v], d);
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

// A token's heads are walked in steps; `per` steps make an item.  Of a step a lane has two heads, kNext apart: what is
// found of them (two sums over lanes and a root, one after the other) has the other's to wait with.
template <int D>
struct Steps {
    static constexpr int kLanes = D / 8, kNext = 32 / kLanes, kHeads = 2 * kNext;
    static int of(int heads) { return (heads + kHeads - 1) / kHeads; }
};

// The queries' or the keys' side of a call.
struct Side {
    const void *x, *g, *w;
    void* y;
    long long x_row, y_row;
    int heads, per;
};
__device__ __forceinline__ Side side_of(const NormRopeArgs& a, bool is_q, int q_per, int k_per) {
    return is_q ? Side{a.q, a.dq_out, a.q_weight, a.q_out, a.q_row, a.q_out_row, a.Hq, q_per}
                : Side{a.k, a.dk_out, a.k_weight, a.k_out, a.k_row, a.k_out_row, a.Hkv, k_per};
}

// Where a warp is on its side: `left` steps of an item of token `row`, this lane's head of the step `head`.  Items in a
// fixed stride.
struct Cursor {
    unsigned item, stride, items;
    int chunks, per, heads, step_heads, sub;
    int row, left, head;
    __device__ __forceinline__ void start(unsigned first, unsigned stride_, const Side& side, int R, int step_heads_, int sub_) {
        const int steps = (side.heads + step_heads_ - 1) / step_heads_;
        per = side.per;
        chunks = (steps + per - 1) / per;
        item = first;
        stride = stride_;
        items = static_cast<unsigned>(R) * static_cast<unsigned>(chunks);
        heads = side.heads;
        step_heads = step_heads_;
        sub = sub_;
        enter();
    }
    __device__ __forceinline__ bool more() const { return item < items; }
    __device__ __forceinline__ int row_of(unsigned x) const { return static_cast<int>(chunks == 1 ? x : x / chunks); }
    __device__ __forceinline__ void enter() {
        row = row_of(item);
        const int i0 = static_cast<int>(item - static_cast<unsigned>(row) * chunks) * per;
        left = min((heads + step_heads - 1) / step_heads - i0, per);
        head = i0 * step_heads + sub;
    }
    // Whether the next step belongs to another item.
    __device__ __forceinline__ bool next() {
        head += step_heads;
        if (--left) return false;
        item += stride;
        enter();
        return true;
    }
};

// a lane's four pairs times (c, s): firsts a c - b s, seconds b c + a s, where the two products' factors may differ
__device__ __forceinline__ void turn_pairs(const float* a, const float* b, const float* ac, const float* bs, const float* bc,
                                           const float* as, float* ya, float* yb) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        fmul2(ya[j], ya[j + 1], b[j], b[j + 1], bs[j], bs[j + 1]);
        ffma2(ya[j], ya[j + 1], a[j], a[j + 1], ac[j], ac[j + 1], ya[j], ya[j + 1]);
        fmul2(yb[j], yb[j + 1], a[j], a[j + 1], as[j], as[j + 1]);
        ffma2(yb[j], yb[j + 1], b[j], b[j + 1], bc[j], bc[j + 1], yb[j], yb[j + 1]);
    }
}
// the sum of a lane's products a x + b y
__device__ __forceinline__ float dot_pairs(const float* a, const float* x, const float* b, const float* y) {
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        ffma2(t0, t1, a[j], a[j + 1], x[j], x[j + 1], t0, t1);
        ffma2(t0, t1, b[j], b[j + 1], y[j], y[j + 1], t0, t1);
    }
    return t0 + t1;
}
__device__ __forceinline__ void scale_pairs(float* a, float* b, float f) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        fmul2(a[j], a[j + 1], a[j], a[j + 1], f, f);
        fmul2(b[j], b[j + 1], b[j], b[j + 1], f, f);
    }
}

template <typename T, int D, bool INTER, bool NORM, int DEPTH>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int q_ctas, int q_per,
                                                             int k_per) {
    using S = Steps<D>;
    using F = Four<T>;
    using V = typename F::V;
    const int lane = threadIdx.x & 31, l = lane % S::kLanes;
    const LaneDims d = lane_dims(l, a.rot, INTER);
    const bool is_q = static_cast<int>(blockIdx.x) < q_ctas;
    const Side side = side_of(a, is_q, q_per, k_per);
    const int cta = is_q ? blockIdx.x : blockIdx.x - q_ctas, ctas = is_q ? q_ctas : gridDim.x - q_ctas;
    Cursor at;  // the step in work; `ahead`: the next to load
    at.start(cta * (kThreads / 32) + (threadIdx.x >> 5), ctas * (kThreads / 32), side, a.R, S::kHeads, lane / S::kLanes);
    if (!at.more()) return;
    Cursor ahead = at;
    grid_dependency_wait();
    V x0[DEPTH][2], x1[DEPTH][2];
    auto load = [&](int u) {
        const T* p = static_cast<const T*>(side.x) + ahead.row * side.x_row + ahead.head * D;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            x0[u][v] = x1[u][v] = V{};
            if (ahead.more() && ahead.head + v * S::kNext < side.heads) {
                x0[u][v] = *reinterpret_cast<const V*>(p + v * S::kNext * D + d.e0);
                x1[u][v] = *reinterpret_cast<const V*>(p + v * S::kNext * D + d.e1);
            }
        }
        if (ahead.more()) ahead.next();
    };
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) load(u);
    Turns turns;
    int pos[4] = {};
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (d.turns) {
        turns.start(a, l);
        turns.fetch(at.row, pos);
    }
    float wa[4], wb[4];
    load_weight<T, INTER, NORM>(side.w, d, wa, wb);
    float ac[4], bs[4], bc[4], as[4];  // weights times cos and sin
    bool fresh = true;                 // the step is its item's first
    for (;;) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            if (fresh) {
                if (d.turns) {
                    turns.angles(pos, c, s);
                    if (at.item + at.stride < at.items) turns.fetch(at.row_of(at.item + at.stride), pos);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ac[j] = wa[j] * c[j];
                    bs[j] = -wb[j] * s[j];
                    bc[j] = wb[j] * c[j];
                    as[j] = wa[j] * s[j];
                }
            }
            float ya[2][4], yb[2][4], sq[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float y0[4], y1[4], pa[4], pb[4];
                F::get(x0[u][v], y0);
                F::get(x1[u][v], y1);
                to_pairs<INTER>(y0, y1, pa, pb);
                turn_pairs(pa, pb, ac, bs, bc, as, ya[v], yb[v]);
                if (NORM) sq[v] = dot_pairs(pa, pa, pb, pb);
                if (!d.turns) {  // each by itself, whatever 0 times its neighbour would be
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ya[v][j] = pa[j] * ac[j];
                        yb[v][j] = pb[j] * bc[j];
                    }
                }
            }
            load(u);
            if (NORM) {
                head_sums<S::kLanes>(sq);
#pragma unroll
                for (int v = 0; v < 2; ++v) scale_pairs(ya[v], yb[v], rsqrtf(sq[v] * (1.f / D) + a.eps));
            }
            T* p = static_cast<T*>(side.y) + at.row * side.y_row + at.head * D;
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (at.head + v * S::kNext < side.heads) {
                    float y0[4], y1[4];
                    from_pairs<INTER>(ya[v], yb[v], y0, y1);
                    *reinterpret_cast<V*>(p + v * S::kNext * D + d.e0) = F::put(y0);
                    *reinterpret_cast<V*>(p + v * S::kNext * D + d.e1) = F::put(y1);
                }
            fresh = at.next();
            if (!at.more()) return;
        }
    }
}

// Gradient.  A warp keeps the sums of its lanes' dw; a CTA's are added up in a fixed order and written to its row of
// `parts` [CTAs][D], which the next kernel adds up.
template <typename T, int D, bool INTER, bool NORM, int DEPTH>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, int q_ctas, int q_per,
                                                                 int k_per, float* parts) {
    using S = Steps<D>;
    using F = Four<T>;
    using V = typename F::V;
    constexpr int kWarps = kThreads / 32;
    __shared__ float sums[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % S::kLanes, sub = lane / S::kLanes;
    const LaneDims d = lane_dims(l, a.rot, INTER);
    const bool is_q = static_cast<int>(blockIdx.x) < q_ctas;
    const Side side = side_of(a, is_q, q_per, k_per);
    const int cta = is_q ? blockIdx.x : blockIdx.x - q_ctas, ctas = is_q ? q_ctas : gridDim.x - q_ctas;
    Cursor at;  // the step in work; `ahead`: the next to load
    at.start(cta * kWarps + warp, ctas * kWarps, side, a.R, S::kHeads, sub);
    Cursor ahead = at;
    grid_dependency_wait();
    V x0[DEPTH][2], x1[DEPTH][2], g0[DEPTH][2], g1[DEPTH][2];
    auto load = [&](int u) {
        const T* gp = static_cast<const T*>(side.g) + (static_cast<long long>(ahead.row) * side.heads + ahead.head) * D;
        const T* xp = static_cast<const T*>(side.x) + ahead.row * side.x_row + ahead.head * D;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            x0[u][v] = x1[u][v] = g0[u][v] = g1[u][v] = V{};
            if (ahead.more() && ahead.head + v * S::kNext < side.heads) {
                g0[u][v] = *reinterpret_cast<const V*>(gp + v * S::kNext * D + d.e0);
                g1[u][v] = *reinterpret_cast<const V*>(gp + v * S::kNext * D + d.e1);
                if (NORM) {
                    x0[u][v] = *reinterpret_cast<const V*>(xp + v * S::kNext * D + d.e0);
                    x1[u][v] = *reinterpret_cast<const V*>(xp + v * S::kNext * D + d.e1);
                }
            }
        }
        if (ahead.more()) ahead.next();
    };
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) load(u);
    Turns turns;
    int pos[4] = {};
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f}, ns[4];
    if (d.turns) turns.start(a, l);
    if (d.turns && at.more()) turns.fetch(at.row, pos);
    float wa[4], wb[4], da[4] = {}, db[4] = {};
    load_weight<T, INTER, NORM>(side.w, d, wa, wb);
    bool fresh = true;  // the step is its item's first
    while (at.more()) {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) {
            if (!at.more()) break;
            if (fresh) {
                if (d.turns) {
                    turns.angles(pos, c, s);
                    if (at.item + at.stride < at.items) turns.fetch(at.row_of(at.item + at.stride), pos);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) ns[j] = -s[j];
            }
            float ga[2][4], gb[2][4], xa[2][4], xb[2][4], sums2[4];  // of both heads: x^2, g w x
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float y0[4], y1[4], ya[4], yb[4];
                F::get(g0[u][v], y0);
                F::get(g1[u][v], y1);
                to_pairs<INTER>(y0, y1, ya, yb);
                turn_pairs(ya, yb, c, s, c, ns, ga[v], gb[v]);  // back
                if (!d.turns) {  // as they are, whatever 0 times their neighbours would be
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ga[v][j] = ya[j];
                        gb[v][j] = yb[j];
                    }
                }
                if (NORM) {
                    F::get(x0[u][v], y0);
                    F::get(x1[u][v], y1);
                    to_pairs<INTER>(y0, y1, xa[v], xb[v]);
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        fmul2(ya[j], ya[j + 1], ga[v][j], ga[v][j + 1], wa[j], wa[j + 1]);
                        fmul2(yb[j], yb[j + 1], gb[v][j], gb[v][j + 1], wb[j], wb[j + 1]);
                    }
                    sums2[v] = dot_pairs(xa[v], xa[v], xb[v], xb[v]);
                    sums2[2 + v] = dot_pairs(ya, xa[v], yb, xb[v]);
                }
            }
            load(u);
            if (NORM) {
                head_sums<S::kLanes>(sums2);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    // a head past the last adds nothing, also without an eps
                    const float r = at.head + v * S::kNext < side.heads ? rsqrtf(sums2[v] * (1.f / D) + a.eps) : 0.f;
                    scale_pairs(xa[v], xb[v], r);                             // n
                    const float rm = -r * (sums2[2 + v] * r * (1.f / D));     // r mean(g w n)
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        ffma2(da[j], da[j + 1], ga[v][j], ga[v][j + 1], xa[v][j], xa[v][j + 1], da[j], da[j + 1]);
                        ffma2(db[j], db[j + 1], gb[v][j], gb[v][j + 1], xb[v][j], xb[v][j + 1], db[j], db[j + 1]);
                        fmul2(ga[v][j], ga[v][j + 1], ga[v][j], ga[v][j + 1], wa[j] * r, wa[j + 1] * r);
                        fmul2(gb[v][j], gb[v][j + 1], gb[v][j], gb[v][j + 1], wb[j] * r, wb[j + 1] * r);
                        ffma2(ga[v][j], ga[v][j + 1], xa[v][j], xa[v][j + 1], rm, rm, ga[v][j], ga[v][j + 1]);
                        ffma2(gb[v][j], gb[v][j + 1], xb[v][j], xb[v][j + 1], rm, rm, gb[v][j], gb[v][j + 1]);
                    }
                }
            }
            T* p = static_cast<T*>(side.y) + at.row * side.y_row + at.head * D;
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (at.head + v * S::kNext < side.heads) {
                    float y0[4], y1[4];
                    from_pairs<INTER>(ga[v], gb[v], y0, y1);
                    *reinterpret_cast<V*>(p + v * S::kNext * D + d.e0) = F::put(y0);
                    *reinterpret_cast<V*>(p + v * S::kNext * D + d.e1) = F::put(y1);
                }
            fresh = at.next();
        }
    }
    if (!NORM) return;
    // heads of the warp, then the warps
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int o = S::kLanes; o < 32; o <<= 1) {
            da[j] += __shfl_xor_sync(0xffffffffu, da[j], o);
            db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
        }
    if (sub == 0) {
        float y0[4], y1[4];
        from_pairs<INTER>(da, db, y0, y1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sums[warp][d.e0 + j] = y0[j];
            sums[warp][d.e1 + j] = y1[j];
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < D; x += kThreads) {
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += sums[w][x];
        parts[static_cast<long long>(blockIdx.x) * D + x] = total;
    }
}

// dw: 32 columns of the parts per CTA (blockIdx.y: of the queries' or the keys'), 32 threads each, in a fixed order.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* parts, int q_n, int n, int D, float* dwq, float* dwk) {
    __shared__ float sums[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    const int first = blockIdx.y ? q_n : 0, last = blockIdx.y ? n : q_n;
    grid_dependency_wait();
    float total = 0.f;
#pragma unroll 8
    for (int i = first + part; i < last; i += 32) total += parts[static_cast<long long>(i) * D + col];
    sums[part][threadIdx.x & 31] = total;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) total += sums[i][threadIdx.x];
    (blockIdx.y ? dwk : dwq)[col] = total;
}

// Steps of a warp on their way, and CTAs per SM.  Forward, 8192 tokens of 32 + 8 heads, D = 128, three axes: bf16 31.2 us
// with three steps (a lane's loads are 8 bytes) and 4 CTAs, 35.4 with two and 8, 36.5 with one; fp32, one axis, 55.5 with
// one step (16 bytes) and 8 CTAs, 56.5 with 7, 57.5 with 10, 61.8 with two steps.  Gradient, bf16: 52 us with one step and 8 CTAs (two rounds of the
// four that fit) as with 4 or with two steps; D = 64, pairs next to each other: 28.8 with 8 CTAs, 30.7 with 4, 30.1 with two
// steps; held to the registers of 6 CTAs 66 and 40.
template <typename T>
constexpr int kFwdDepth = sizeof(T) == 2 ? 3 : 1;
template <typename T>
constexpr int kFwdCtas = sizeof(T) == 2 ? 4 : 8;
constexpr int kBwdDepth = 1, kBwdCtas = 8;
constexpr int kAngleSteps = 2;               // what a token's angles cost, in steps
constexpr int kItems = 2;                    // of a warp, at least, before a token's heads stay in one item

// How a call is cut up: CTAs of the queries and in all, steps of an item.  Each side gets CTAs by its heads; few tokens
// are spread over warps of one step each, many keep their angles for more heads.
struct Cut {
    int q_ctas, ctas, q_per, k_per;
};
template <int D>
Cut cut_of(const NormRopeArgs& a, int most) {
    constexpr int warps = kThreads / 32;
    const int sq = Steps<D>::of(a.Hq), sk = Steps<D>::of(a.Hkv);
    const int k_share = 1 + static_cast<int>(static_cast<long long>(most - 2) * (sk + kAngleSteps) / (sq + sk + 2 * kAngleSteps));
    auto per_of = [&](int steps, int share) {
        const long long items = static_cast<long long>(kItems) * share * warps, per = (static_cast<long long>(a.R) * steps + items - 1) / items;
        return static_cast<int>(per < 1 ? 1 : per > steps ? steps : per);
    };
    auto ctas_of = [&](int steps, int per, int share) {
        const long long want = (static_cast<long long>(a.R) * ((steps + per - 1) / per) + warps - 1) / warps;
        return static_cast<int>(want < share ? want : share);
    };
    Cut c;
    c.q_per = per_of(sq, most - k_share);
    c.k_per = per_of(sk, k_share);
    c.q_ctas = ctas_of(sq, c.q_per, most - k_share);
    c.ctas = c.q_ctas + ctas_of(sk, c.k_per, k_share);
    return c;
}

template <typename T, int D, bool INTER, bool NORM>
cudaError_t run_fwd(const NormRopeArgs& a, cudaStream_t stream) {
    const Cut c = cut_of<D>(a, kFwdCtas<T> * device_sm_count());
    return launch_overlapped(norm_rope_kernel<T, D, INTER, NORM, kFwdDepth<T>>, dim3(c.ctas), kThreads, 0, stream, a, c.q_ctas, c.q_per,
                             c.k_per);
}

template <typename T, int D, bool INTER, bool NORM>
cudaError_t run_bwd(const NormRopeArgs& a, float* parts, float* dwq, float* dwk, cudaStream_t stream) {
    const Cut c = cut_of<D>(a, norm_rope_bwd_ctas());
    if (c.ctas) {
        const cudaError_t e = launch_overlapped(norm_rope_bwd_kernel<T, D, INTER, NORM, kBwdDepth>, dim3(c.ctas), kThreads, 0,
                                                stream, a, c.q_ctas, c.q_per, c.k_per, parts);
        if (e != cudaSuccess) return e;
    }
    if (!NORM) return cudaSuccess;
    return launch_overlapped(norm_weight_grad_kernel, dim3(D / 32, 2), 1024, 0, stream, static_cast<const float*>(parts), c.q_ctas,
                             c.ctas, D, dwq, dwk);
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

int norm_rope_bwd_ctas() { return kBwdCtas * device_sm_count(); }

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) { return with_form(a, Fwd{a, stream}); }

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, float* parts, float* dwq, float* dwk, cudaStream_t stream) {
    return with_form(a, Bwd{a, parts, dwq, dwk, stream});
}

}  // namespace ra
