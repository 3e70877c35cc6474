// cache_q8_ops.cu -- keys and values into the pages of an 8-bit cache, and back into rows.
//
// D / 8 lanes hold one head of a token, eight dims each; a warp takes a token and walks its
// heads, K and V of a step together.  Written: the largest magnitude of the head's row by
// shuffles, its scale byte, the codes.  Both are bound by the bytes of the rows (16- or
// 32-bit) and of the pages (8-bit): 4 x up to 8192 tokens of 8 heads, D = 128, in bf16 written in 27
// us, 5.4 TB/s (0.81 of the measured copy rate); 4 x up to 16384 tokens read back in 52 us, 5.7 TB/s
// (0.85); 64 single tokens written in 4.7 us (launch, the search for a warp's row, one trip to
// memory, the chain from the largest value to the codes).
#include "cache_q8.cuh"

namespace ra {

static __device__ unsigned g_cache_q8_status[2];

namespace {

constexpr int kThreads = 256;
constexpr int kAppendCtas = 4, kReadCtas = 6;  // per SM: all that fit run at once, on equal parts

// Calls f(stacked row, key's pool row or -1) for the rows of the CTA's range, a warp each, whatever sequence they
// belong to; -1 where the key is before the sequence's first or its page out of range.
template <class F>
__device__ __forceinline__ void for_rows(const CacheBatch& p, const WorkRange& range, F f) {
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5;
    long long a = range.a;  // weight before the sequence
    for (int b = range.b; b < p.n_seqs && a < range.hi; ++b) {
        CacheSeq s = range.s;
        if (b != range.b) load_seq(p, b, s);
        const int t0 = static_cast<int>(max(0ll, range.lo - a));
        const int t1 = static_cast<int>(min(static_cast<long long>(s.n), range.hi - a));
        const int turn = static_cast<int>(a + t0 - range.lo) & (kWarps - 1);
        a += s.n;
        auto row_of = [&](int t) {
            const int j = s.kv - s.n + t;
            return t >= t1 || j < 0 ? -1
                                    : cache_row(p.pages + static_cast<long long>(b) * p.max_pages, p.n_pages, p.page_shift, j,
                                                g_cache_q8_status);
        };
        int t = t0 + ((warp - turn) & (kWarps - 1)), row = row_of(t);
        for (; t < t1; t += kWarps) {
            const int next = row_of(t + kWarps);  // its page is found while this row is worked on
            f(s.lo + t, row);
            row = next;
        }
    }
}

// Eight consecutive elements as they come.
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (auto& x : v) x = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[sizeof(T) / 2 - 1].x, v[sizeof(T) / 2 - 1].y,
                               v[sizeof(T) / 2 - 1].z, v[sizeof(T) / 2 - 1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(sizeof(T) == 2 ? w[j] << 16 : w[2 * j]);
            x[2 * j + 1] = __uint_as_float(sizeof(T) == 2 ? w[j] & 0xffff0000u : w[2 * j + 1]);
        }
    }
};

// Place of the scale byte of head h of a pool row: [page][head][row of the page].
__device__ __forceinline__ long long scale_at(const CacheBatch& p, int row, int h) {
    const int page = row >> p.page_shift;
    return ((static_cast<long long>(page) * p.Hkv + h) << p.page_shift) + (row - (page << p.page_shift));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const CacheBatch p, const T* k_rows, const T* v_rows, Q8Pools pools) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    __shared__ RangeScratch<kThreads> scratch;
    grid_dependency_wait();
    const WorkRange range = find_range<kThreads>(p, kThreads / 32, g_cache_q8_status, RowWeight{}, scratch);
    const int lane = threadIdx.x & 31, sub = lane / kLanes, c = lane % kLanes * 8;
    constexpr int kDepth = 2;  // steps of a lane's heads on their way at once (four: 32 us, with fewer warps an SM)
    for_rows(p, range, [&](int from, int row) {
        if (row < 0) return;
#pragma unroll 1
        for (int h0 = sub; h0 < p.Hkv + sub; h0 += kDepth * kHeads) {
            Eight<T> raw[kDepth][2];
#pragma unroll
            for (int u = 0; u < kDepth; ++u) {
                const int h = h0 + u * kHeads;
                raw[u][0].zero();
                raw[u][1].zero();
                if (h < p.Hkv) {
                    const long long at = (static_cast<long long>(from) * p.Hkv + h) * D + c;
                    raw[u][0].load(k_rows + at);
                    raw[u][1].load(v_rows + at);
                }
            }
#pragma unroll
            for (int u = 0; u < kDepth; ++u) {
                const int h = h0 + u * kHeads;
                if (h - sub >= p.Hkv) break;
                float x[2][8];
                unsigned most[2] = {0, 0};
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    raw[u][t].get(x[t]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) most[t] = max(most[t], __float_as_uint(x[t][j]) & 0x7fffffffu);
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int t = 0; t < 2; ++t) most[t] = max(most[t], __shfl_xor_sync(0xffffffffu, most[t], o));
                if (h >= p.Hkv) continue;
                const long long to = (static_cast<long long>(row) * p.Hkv + h) * D + c;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const unsigned e = scale_byte(most[t]);
                    const float inverse = scale_of(254u - e);
                    *reinterpret_cast<uint2*>((t ? pools.v : pools.k) + to) =
                        make_uint2(codes4(x[t], inverse), codes4(x[t] + 4, inverse));
                    if (c == 0) (t ? pools.vs : pools.ks)[scale_at(p, row, h)] = static_cast<unsigned char>(e);
                }
            }
        }
    });
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheBatch p, Q8Pools pools, T* k_rows, T* v_rows) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    __shared__ RangeScratch<kThreads> scratch;
    grid_dependency_wait();
    const WorkRange range = find_range<kThreads>(p, kThreads / 32, g_cache_q8_status, RowWeight{}, scratch);
    const int lane = threadIdx.x & 31, sub = lane / kLanes, c = lane % kLanes * 8;
    for_rows(p, range, [&](int to, int row) {
#pragma unroll 4
        for (int h = sub; h < p.Hkv; h += kHeads) {
            uint2 codes[2] = {};
            unsigned e[2] = {0, 0};
            if (row >= 0) {
                const long long at = (static_cast<long long>(row) * p.Hkv + h) * D + c, s = scale_at(p, row, h);
                codes[0] = *reinterpret_cast<const uint2*>(pools.k + at);
                codes[1] = *reinterpret_cast<const uint2*>(pools.v + at);
                e[0] = pools.ks[s];
                e[1] = pools.vs[s];
            }
            const long long out = (static_cast<long long>(to) * p.Hkv + h) * D + c;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float x[8];
                values4(codes[t].x, x);
                values4(codes[t].y, x + 4);
                const float scale = scale_of(e[t]);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= scale;
                store8((t ? v_rows : k_rows) + out, x);
            }
        }
    });
}

template <typename T, int D>
cudaError_t run(const CacheBatch& p, const Q8Pools& pools, const void* k_in, const void* v_in, void* k_out, void* v_out,
                cudaStream_t stream) {
    const int most = (k_in ? kAppendCtas : kReadCtas) * device_sm_count(), blocks = (p.R + 7) / 8 < most ? (p.R + 7) / 8 : most;
    if (k_in)
        return launch_overlapped(append_kernel<T, D>, dim3(blocks), kThreads, 0, stream, p, static_cast<const T*>(k_in),
                                 static_cast<const T*>(v_in), pools);
    return launch_overlapped(read_kernel<T, D>, dim3(blocks), kThreads, 0, stream, p, pools, static_cast<T*>(k_out),
                             static_cast<T*>(v_out));
}

cudaError_t run_any(const CacheBatch& p, const Q8Pools& pools, const void* k_in, const void* v_in, void* k_out, void* v_out,
                    int D, int bf16, cudaStream_t stream) {
    if (bf16)
        return D == 128 ? run<__nv_bfloat16, 128>(p, pools, k_in, v_in, k_out, v_out, stream)
                        : run<__nv_bfloat16, 64>(p, pools, k_in, v_in, k_out, v_out, stream);
    return D == 128 ? run<float, 128>(p, pools, k_in, v_in, k_out, v_out, stream)
                    : run<float, 64>(p, pools, k_in, v_in, k_out, v_out, stream);
}

}  // namespace

cudaError_t launch_append_q8(const CacheBatch& p, const void* k_rows, const void* v_rows, const Q8Pools& pools, int D, int bf16,
                             cudaStream_t stream) {
    return run_any(p, pools, k_rows, v_rows, nullptr, nullptr, D, bf16, stream);
}

cudaError_t launch_read_q8(const CacheBatch& p, const Q8Pools& pools, void* k_rows, void* v_rows, int D, int bf16,
                           cudaStream_t stream) {
    return run_any(p, pools, nullptr, nullptr, k_rows, v_rows, D, bf16, stream);
}

unsigned read_clear_status_cache_q8(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_q8_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_q8_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
