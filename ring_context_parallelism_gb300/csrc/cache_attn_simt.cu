// cache_attn_simt.cu -- exact attention over a paged cache on the CUDA cores, the
// join of cut units, and the attention weight gathered per key.
//
// Scores, exponentials and P V are fp32 FMA and exp2f; nothing is rounded to
// fewer bits but a bf16 output.
#include <cmath>

#include "cache_batch.cuh"

namespace ra {

static __device__ unsigned g_cache_simt_status[2];

namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
// Whether new token t (stacked row lo + t) of a sequence sees its key j.
__device__ __forceinline__ bool sees(const CacheBatch& p, const CacheSeq& s, int t, int j) {
    if (j >= s.kv) return false;
    const int jn = j - (s.kv - s.n);
    if (jn < 0) return true;
    if (!p.tree_mask) return jn <= t;
    return jn < p.mask_cols && p.tree_mask[static_cast<long long>(s.lo + t) * p.mask_cols + jn] != 0;
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
constexpr int kThreads = 128;
constexpr int kRT = kTreeSimtRows;  // rows of a unit: 8 threads each
constexpr int kKT = 32;             // keys staged per step
constexpr int kOV = 1;              // weight of a unit beyond its tiles
constexpr int kMinW = 4;            // least weight per CTA

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const CacheBatch p, const T* __restrict__ q,
                                                             const T* __restrict__ k, const T* __restrict__ v,
                                                             T* __restrict__ out, float* __restrict__ lse,
                                                             JoinJob* jobs, float2* stats, float* part_o, int slot_rows,
                                                             float scale_log2) {
    __shared__ __align__(16) float qs[kRT][D];
    __shared__ __align__(16) float ks[kKT][D + 4];  // 4 words of padding: 8 keys x 16 bytes hit all banks
    __shared__ __align__(16) float vs[kKT][D];
    __shared__ float ps[kRT][kKT];
    const int tid = threadIdx.x, r = tid >> 3, sub = tid & 7;
    unsigned* status = g_cache_simt_status;
    const bool tree = p.tree_mask != nullptr;
    __shared__ RangeScratch<kThreads> scratch;
    const WorkRange range =
        find_range<kThreads>(p, kMinW, status, TreeWeight<kKT, kOV>{p.G, p.Hkv, tree, kRT}, scratch);
    if (tid == 0) jobs[blockIdx.x].rows = 0;
    SegmentWalk<kKT, kOV> walk;
    walk.start(p, range, kRT);
    Segment g;
    while (walk.next(p, range, g)) {
        const int fr0 = g.rt * kRT, nrows = min(kRT, g.s.n * p.G - fr0);
        __syncthreads();
        for (int i = tid; i < kRT * (D / 4); i += kThreads) {
            const int rr = i / (D / 4), c = i % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (rr < nrows) {
                const int fr = fr0 + rr;
                x = load4(q + (static_cast<long long>(g.s.lo + fr / p.G) * p.Hq + g.head * p.G + fr % p.G) * D + c);
            }
            *reinterpret_cast<float4*>(&qs[rr][c]) = x;
        }
        const int t = min(fr0 + r, g.s.n * p.G - 1) / p.G;  // this thread's token
        const bool row_ok = r < nrows;
        const int* table = p.pages + static_cast<long long>(g.b) * p.max_pages;
        float m = -INFINITY, l = 0.f, o[D / 8];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j] = 0.f;
        for (int tile = g.t0; tile < g.t1; ++tile) {
            const int k0 = tile * kKT;
            __syncthreads();
            for (int i = tid; i < kKT * (D / 4); i += kThreads) {
                const int kk = i / (D / 4), c = i % (D / 4) * 4;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                if (k0 + kk < g.s.kv) {
                    const int row = cache_row(table, p.n_pages, p.page_shift, k0 + kk, status);
                    if (row >= 0) {
                        const long long at = (static_cast<long long>(row) * p.Hkv + g.head) * D + c;
                        a = load4(k + at);
                        b = load4(v + at);
                    }
                }
                *reinterpret_cast<float4*>(&ks[kk][c]) = a;
                *reinterpret_cast<float4*>(&vs[kk][c]) = b;
            }
            __syncthreads();
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c = 0; c < D; c += 4) {
                const float4 a = *reinterpret_cast<const float4*>(&qs[r][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 b = *reinterpret_cast<const float4*>(&ks[sub + 8 * i][c]);
                    s4[i] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s4[i]))));
                }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s4[i] = row_ok && sees(p, g.s, t, k0 + sub + 8 * i) ? s4[i] * scale_log2 : -INFINITY;
                mx = fmaxf(mx, s4[i]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float m_new = fmaxf(m, mx);
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = exp2f(m - base);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = exp2f(s4[i] - base);
                ps[r][sub + 8 * i] = e;
                sum += e;
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            m = m_new;
            l = l * alpha + sum;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[j] *= alpha;
            __syncwarp();
            for (int kk = 0; kk < kKT; ++kk) {
                const float e = ps[r][kk];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const float4 b = *reinterpret_cast<const float4*>(&vs[kk][4 * (sub + 8 * c)]);
                    o[4 * c] = fmaf(e, b.x, o[4 * c]);
                    o[4 * c + 1] = fmaf(e, b.y, o[4 * c + 1]);
                    o[4 * c + 2] = fmaf(e, b.z, o[4 * c + 2]);
                    o[4 * c + 3] = fmaf(e, b.w, o[4 * c + 3]);
                }
            }
        }
        if (g.whole()) {
            if (row_ok) {
                const int fr = fr0 + r, row = g.s.lo + fr / p.G, h = g.head * p.G + fr % p.G;
                const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    store4(out + (static_cast<long long>(row) * p.Hq + h) * D + 4 * (sub + 8 * c),
                           make_float4(o[4 * c] * inv, o[4 * c + 1] * inv, o[4 * c + 2] * inv, o[4 * c + 3] * inv));
                if (lse && sub == 0)
                    lse[static_cast<long long>(h) * p.R + row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            }
        } else {
            const long long slot = static_cast<long long>(partial_slot(g)) * slot_rows;
            if (row_ok) {
                if (sub == 0) stats[slot + r] = make_float2(m, l);
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    reinterpret_cast<float4*>(part_o + slot * D)[(sub + 8 * c) * slot_rows + r] =
                        make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            }
            if (tid == 0 && g.t0 == 0)
                jobs[blockIdx.x] = JoinJob{fr0, nrows, g.s.lo, g.head, owner_of(range, g.a + kOV + g.tiles - 1), {0, 0, 0}};
        }
    }
}

// ---------------------------------------------------------------------------
// join of the cut units: O = sum w_i O_i / sum w_i l_i, w_i = 2^(m_i - max m), parts in key order
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;
constexpr int kJoinDims = 4;  // head dims of a thread

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const JoinJob* jobs, const float2* stats,
                                                                 const float* part_o, int slot_rows, T* out, float* lse,
                                                                 int R, int Hq, int G) {
    constexpr int V = kJoinDims / 4;
    grid_dependency_wait();
    const int c = blockIdx.x;
    const JoinJob job = jobs[c];
    const int x = blockIdx.y * kJoinThreads + threadIdx.x;  // (16 head dims, row), rows fastest
    if (job.rows == 0 || x >= job.rows * (D / kJoinDims)) return;
    const int r = x % job.rows, d16 = x / job.rows;
    const int parts = job.last - c + 1;
    auto slot = [&](int i) { return static_cast<long long>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_rows; };
    float m = -INFINITY, l = 0.f;
    float4 o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    // the running maximum of the parts so far, as in the walk over keys
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
        const float2 st = stats[slot(i) + r];
        const float4* src = reinterpret_cast<const float4*>(part_o + slot(i) * D) + d16 * V * slot_rows + r;
        float4 y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = src[j * slot_rows];
        const float m_new = fmaxf(m, st.x), base = m_new == -INFINITY ? 0.f : m_new;
        const float keep = exp2f(m - base), w = exp2f(st.x - base);
        m = m_new;
        l = fmaf(l, keep, w * st.y);
#pragma unroll
        for (int j = 0; j < V; ++j)
            o[j] = make_float4(fmaf(o[j].x, keep, w * y[j].x), fmaf(o[j].y, keep, w * y[j].y),
                               fmaf(o[j].z, keep, w * y[j].z), fmaf(o[j].w, keep, w * y[j].w));
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int fr = job.row0 + r, row = job.seq_lo + fr / G, h = job.head * G + fr % G;
    T* dst = out + (static_cast<long long>(row) * Hq + h) * D + kJoinDims * d16;
#pragma unroll
    for (int j = 0; j < V; ++j)
        store4(dst + 4 * j, make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv));
    if (lse && d16 == 0) lse[static_cast<long long>(h) * R + row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------
// gathered weight
// ---------------------------------------------------------------------------
constexpr int kMassKT = 64;   // keys of a tile
constexpr int kMassRT = 16;   // rows staged per step

// A tile of keys weighs its row steps plus one.
struct MassWeight {
    int G, Hkv;
    __device__ __forceinline__ int tile(const CacheSeq& s) const { return (s.n * G + kMassRT - 1) / kMassRT + 1; }
    __device__ __forceinline__ long long operator()(const CacheSeq& s) const {
        return static_cast<long long>((s.kv + kMassKT - 1) / kMassKT) * Hkv * tile(s);
    }
    __device__ __forceinline__ long long locate(const CacheSeq&, long long, int&, int&) const { return 0; }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) mass_simt_kernel(const CacheBatch p, const T* __restrict__ q,
                                                             const T* __restrict__ k, const float* __restrict__ lse,
                                                             const float* mass_in, float* mass_out,
                                                             int mass_cols, float decay, float scale_log2) {
    __shared__ __align__(16) float qs[kMassRT][D];
    __shared__ __align__(16) float ks[kMassKT][D + 4];
    __shared__ float ls[kMassRT], half_sum[kMassKT];
    const int tid = threadIdx.x, key = tid % kMassKT, half = tid / kMassKT;
    unsigned* status = g_cache_simt_status;
    const MassWeight weight{p.G, p.Hkv};
    __shared__ RangeScratch<kThreads> scratch;
    const WorkRange range = find_range<kThreads>(p, 1, status, weight, scratch);
    long long a = range.a;  // weight before the sequence
    for (int b = range.b; b < p.n_seqs && a < range.hi; ++b) {
        CacheSeq s;
        load_seq(p, b, s);
        const int w = weight.tile(s), tiles = (s.kv + kMassKT - 1) / kMassKT;
        const long long count = static_cast<long long>(tiles) * p.Hkv;
        // the tiles whose weight starts inside the range
        long long i = range.lo > a ? (range.lo - a + w - 1) / w : 0;
        const int* table = p.pages + static_cast<long long>(b) * p.max_pages;
        for (; i < count && a + i * w < range.hi; ++i) {
            const int head = static_cast<int>(i / tiles), k0 = static_cast<int>(i % tiles) * kMassKT;
            __syncthreads();
            for (int x = tid; x < kMassKT * (D / 4); x += kThreads) {
                const int kk = x / (D / 4), c = x % (D / 4) * 4;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + kk < s.kv) {
                    const int row = cache_row(table, p.n_pages, p.page_shift, k0 + kk, status);
                    if (row >= 0) y = load4(k + (static_cast<long long>(row) * p.Hkv + head) * D + c);
                }
                *reinterpret_cast<float4*>(&ks[kk][c]) = y;
            }
            float sum = 0.f;
            for (int fr0 = 0; fr0 < s.n * p.G; fr0 += kMassRT) {
                __syncthreads();
                for (int x = tid; x < kMassRT * (D / 4); x += kThreads) {
                    const int fr = fr0 + x / (D / 4), c = x % (D / 4) * 4;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (fr < s.n * p.G)
                        y = load4(q + (static_cast<long long>(s.lo + fr / p.G) * p.Hq + head * p.G + fr % p.G) * D + c);
                    *reinterpret_cast<float4*>(&qs[x / (D / 4)][c]) = y;
                }
                if (tid < kMassRT) {
                    const int fr = fr0 + tid;
                    float x = -INFINITY;
                    if (fr < s.n * p.G)
                        x = lse[static_cast<long long>(head * p.G + fr % p.G) * p.R + s.lo + fr / p.G];
                    ls[tid] = x == -INFINITY ? INFINITY : x * kLog2e;
                }
                __syncthreads();
                float acc[kMassRT / 2];
#pragma unroll
                for (int j = 0; j < kMassRT / 2; ++j) acc[j] = 0.f;
                for (int c = 0; c < D; c += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(&ks[key][c]);
#pragma unroll
                    for (int j = 0; j < kMassRT / 2; ++j) {
                        const float4 x = *reinterpret_cast<const float4*>(&qs[half * (kMassRT / 2) + j][c]);
                        acc[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc[j]))));
                    }
                }
#pragma unroll
                for (int j = 0; j < kMassRT / 2; ++j) {
                    const int rr = half * (kMassRT / 2) + j, fr = fr0 + rr;
                    if (fr < s.n * p.G && sees(p, s, fr / p.G, k0 + key)) sum += exp2f(acc[j] * scale_log2 - ls[rr]);
                }
            }
            __syncthreads();
            if (half == 1) half_sum[key] = sum;
            __syncthreads();
            if (half == 0 && k0 + key < s.kv) {
                const long long at = (static_cast<long long>(b) * p.Hkv + head) * mass_cols + k0 + key;
                const float got = sum + half_sum[key];
                mass_out[at] = mass_in ? fmaf(decay, mass_in[at], got) : got;
            }
        }
        a += count * w;
    }
}

template <typename T, int D>
cudaError_t run_tree(const TreeArgs& a, const TreeWs& w, cudaStream_t stream) {
    char* ws = static_cast<char*>(a.ws);
    tree_simt_kernel<T, D><<<w.ctas, kThreads, 0, stream>>>(
        a.p, static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v),
        static_cast<T*>(a.out), a.lse, reinterpret_cast<JoinJob*>(ws), reinterpret_cast<float2*>(ws + w.stat_off),
        reinterpret_cast<float*>(ws + w.o_off), w.slot_rows,
        static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))));
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_join(const TreeArgs& a, const TreeWs& w, cudaStream_t stream) {
    char* ws = static_cast<char*>(a.ws);
    return launch_overlapped(tree_join_kernel<T, D>, dim3(w.ctas, (w.slot_rows * (D / kJoinDims) + kJoinThreads - 1) / kJoinThreads),
                             kJoinThreads, 0, stream, static_cast<const JoinJob*>(a.ws),
                             reinterpret_cast<const float2*>(ws + w.stat_off),
                             reinterpret_cast<const float*>(ws + w.o_off), w.slot_rows, static_cast<T*>(a.out), a.lse,
                             a.p.R, a.p.Hq, a.p.G);
}

template <typename T, int D>
cudaError_t run_mass(const MassArgs& a, cudaStream_t stream) {
    mass_simt_kernel<T, D><<<tree_simt_ctas(), kThreads, 0, stream>>>(
        a.p, static_cast<const T*>(a.q), static_cast<const T*>(a.k), a.lse, a.in, a.out, a.mass_cols, a.decay,
        static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))));
    return cudaGetLastError();
}

}  // namespace

TreeWs tree_workspace(int R, int G, int D, int ctas, int row_tile) {
    TreeWs w;
    w.ctas = ctas;
    const long long rows = static_cast<long long>(R) * G;
    w.slot_rows = rows < row_tile ? static_cast<int>(rows) : row_tile;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    w.stat_off = up(sizeof(JoinJob) * ctas);
    w.o_off = w.stat_off + up(sizeof(float2) * 2 * ctas * w.slot_rows);
    w.bytes = w.o_off + up(sizeof(float) * 2 * ctas * w.slot_rows * D);
    return w;
}

int tree_simt_ctas() { return 4 * device_sm_count(); }

cudaError_t launch_tree_join(const TreeArgs& a, const TreeWs& w, int bf16, cudaStream_t stream) {
    if (bf16) return a.D == 128 ? run_join<__nv_bfloat16, 128>(a, w, stream) : run_join<__nv_bfloat16, 64>(a, w, stream);
    return a.D == 128 ? run_join<float, 128>(a, w, stream) : run_join<float, 64>(a, w, stream);
}

cudaError_t launch_tree_simt(const TreeArgs& a, int bf16, cudaStream_t stream) {
    const TreeWs w = tree_workspace(a.p.R, a.p.G, a.D, tree_simt_ctas(), kTreeSimtRows);
    cudaError_t e;
    if (bf16)
        e = a.D == 128 ? run_tree<__nv_bfloat16, 128>(a, w, stream) : run_tree<__nv_bfloat16, 64>(a, w, stream);
    else
        e = a.D == 128 ? run_tree<float, 128>(a, w, stream) : run_tree<float, 64>(a, w, stream);
    return e != cudaSuccess ? e : launch_tree_join(a, w, bf16, stream);
}

cudaError_t launch_mass_simt(const MassArgs& a, int bf16, cudaStream_t stream) {
    if (bf16) return a.D == 128 ? run_mass<__nv_bfloat16, 128>(a, stream) : run_mass<__nv_bfloat16, 64>(a, stream);
    return a.D == 128 ? run_mass<float, 128>(a, stream) : run_mass<float, 64>(a, stream);
}

unsigned read_clear_status_cache_simt(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_simt_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_simt_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
