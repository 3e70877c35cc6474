// cache_attn_simt.cu -- attention over a paged cache and the weight gathered per key in
// exact fp32 on the CUDA cores, and the join of cut units (for both precisions).
//
// Scores, exponentials and P V are fp32 FMA (two at a time, fma.rn.f32x2) and exp2f;
// nothing is rounded to fewer bits.  K and V tiles arrive by cp.async one tile ahead of
// their use, their pool rows looked up two ahead.
#include <cmath>
#include <mutex>

#include "cache_batch.cuh"

namespace ra {

static __device__ unsigned g_cache_simt_status[2];

namespace {

constexpr float kLn2 = 0.69314718055994531f;
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

// ---------------------------------------------------------------------------
// attention: 8 threads per row, two rows (r and r + 16) per thread
// ---------------------------------------------------------------------------
constexpr int kThreads = 128;
constexpr int kRT = kTreeSimtRows;  // rows of a unit
constexpr int kKT = 32;             // keys of a tile
constexpr int kOV = 2;              // weight of a unit beyond its tiles
constexpr int kMinW = 6;            // least weight per CTA: fewer parts to join than one tile each would leave

template <int D>
struct TreeShared {
    float q[kRT][D];
    float k[2][kKT][D + 4];  // 4 words of padding: 8 keys x 16 bytes hit all banks
    float v[2][kKT][D];
    float p[kRT][kKT + 4];
    int rows[2][kKT];        // pool rows of a tile's keys, -1: zeros
    RangeScratch<kThreads> scratch;
};

template <int D>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const CacheBatch p, const float* __restrict__ q,
                                                             const float* __restrict__ k, const float* __restrict__ v,
                                                             float* __restrict__ out, float* __restrict__ lse,
                                                             JoinJob* jobs, float2* stats, float* part_o, int slot_rows,
                                                             float scale_log2) {
    extern __shared__ __align__(16) unsigned char raw[];
    TreeShared<D>& sh = *reinterpret_cast<TreeShared<D>*>(raw);
    const int tid = threadIdx.x, r = tid >> 3, sub = tid & 7;
    unsigned* status = g_cache_simt_status;
    const bool tree = p.tree_mask != nullptr;
    const WorkRange range =
        find_range<kThreads>(p, kMinW, status, TreeWeight<kKT, kOV>{p.G, p.Hkv, tree, kRT}, sh.scratch);
    if (tid == 0) jobs[blockIdx.x].rows = 0;
    SegmentWalk<kKT, kOV> walk;
    walk.start(p, range, kRT);
    Segment g;
    while (walk.next(p, range, g)) {
        const int fr0 = g.rt * kRT, nrows = min(kRT, g.s.n * p.G - fr0);
        const bool two = nrows > 16;
        const int* table = p.pages + static_cast<long long>(g.b) * p.max_pages;
        auto pool_row = [&](int tile) {  // of key tid of the tile
            const int j = tile * kKT + tid;
            return tile < g.t1 && j < g.s.kv ? cache_row(table, p.n_pages, p.page_shift, j, status) : -1;
        };
        auto fetch = [&](int tile, int buf) {
#pragma unroll
            for (int i = tid; i < kKT * (D / 4); i += kThreads) {
                const int kk = i / (D / 4), c = i % (D / 4) * 4, row = sh.rows[buf][kk];
                const long long at = row < 0 ? 0 : (static_cast<long long>(row) * p.Hkv + g.head) * D + c;
                copy16(&sh.k[buf][kk][c], k + at, row >= 0);
                copy16(&sh.v[buf][kk][c], v + at, row >= 0);
            }
        };
        __syncthreads();  // the segment before is done with shared memory
        if (tid < kKT) {
            sh.rows[0][tid] = pool_row(g.t0);
            sh.rows[1][tid] = pool_row(g.t0 + 1);
        }
        for (int i = tid; i < kRT * (D / 4); i += kThreads) {
            const int rr = i / (D / 4), c = i % (D / 4) * 4, fr = min(fr0 + rr, g.s.n * p.G - 1);
            copy16(&sh.q[rr][c],
                   q + (static_cast<long long>(g.s.lo + fr / p.G) * p.Hq + g.head * p.G + fr % p.G) * D + c, rr < nrows);
        }
        __syncthreads();
        if (g.t0 < g.t1) fetch(g.t0, 0);
        copies_done();
        __syncthreads();
        const int last = g.s.n * p.G - 1;
        const int tok[2] = {min(fr0 + r, last) / p.G, min(fr0 + r + 16, last) / p.G};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][D / 8];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[x][j] = 0.f;
        for (int tile = g.t0; tile < g.t1; ++tile) {
            const int buf = (tile - g.t0) & 1, k0 = tile * kKT;
            if (tile + 1 < g.t1) fetch(tile + 1, buf ^ 1);
            const int row_ahead = tid < kKT ? pool_row(tile + 2) : -1;
            // scores: (even, odd) head dims in the two lanes of a packed sum
            float s0[2][4], s1[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) s0[x][i] = s1[x][i] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = lds4(&sh.k[buf][sub + 8 * i][c]);
                const float4 a = lds4(&sh.q[r][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ffma2(s0[0][i], s1[0][i], a.x, a.y, b[i].x, b[i].y, s0[0][i], s1[0][i]);
                    ffma2(s0[0][i], s1[0][i], a.z, a.w, b[i].z, b[i].w, s0[0][i], s1[0][i]);
                }
                if (two) {
                    const float4 a1 = lds4(&sh.q[r + 16][c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ffma2(s0[1][i], s1[1][i], a1.x, a1.y, b[i].x, b[i].y, s0[1][i], s1[1][i]);
                        ffma2(s0[1][i], s1[1][i], a1.z, a1.w, b[i].z, b[i].w, s0[1][i], s1[1][i]);
                    }
                }
            }
            const bool masked = k0 + kKT > g.s.kv - g.s.n;  // new tokens in the tile
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x == 1 && !two) break;
                float y[4], mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = (s0[x][i] + s1[x][i]) * scale_log2;
                    if (masked && !sees(p, g.s, tok[x], k0 + sub + 8 * i)) y[i] = -INFINITY;
                    mx = fmaxf(mx, y[i]);
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float m_new = fmaxf(m[x], mx), base = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m[x] - base);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = exp2f(y[i] - base);
                    sh.p[r + 16 * x][sub + 8 * i] = e;
                    sum += e;
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                m[x] = m_new;
                l[x] = l[x] * alpha + sum;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) o[x][j] *= alpha;
            }
            __syncwarp();  // a row's weights are written and read by its eight threads
#pragma unroll 2
            for (int kk = 0; kk < kKT; kk += 4) {
                const float4 e0 = lds4(&sh.p[r][kk]), e1 = two ? lds4(&sh.p[r + 16][kk]) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float w0[4] = {e0.x, e0.y, e0.z, e0.w}, w1[4] = {e1.x, e1.y, e1.z, e1.w};
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        const float4 b = lds4(&sh.v[buf][kk + z][4 * (sub + 8 * c)]);
                        ffma2(o[0][4 * c], o[0][4 * c + 1], w0[z], w0[z], b.x, b.y, o[0][4 * c], o[0][4 * c + 1]);
                        ffma2(o[0][4 * c + 2], o[0][4 * c + 3], w0[z], w0[z], b.z, b.w, o[0][4 * c + 2], o[0][4 * c + 3]);
                        if (two) {
                            ffma2(o[1][4 * c], o[1][4 * c + 1], w1[z], w1[z], b.x, b.y, o[1][4 * c], o[1][4 * c + 1]);
                            ffma2(o[1][4 * c + 2], o[1][4 * c + 3], w1[z], w1[z], b.z, b.w, o[1][4 * c + 2], o[1][4 * c + 3]);
                        }
                    }
            }
            copies_done();
            __syncthreads();  // the next tile is there, and everyone is done with this one's rows
            if (tid < kKT) sh.rows[buf][tid] = row_ahead;
            __syncthreads();
        }
        const bool whole = g.whole();
        const long long slot = static_cast<long long>(partial_slot(g)) * slot_rows;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rr = r + 16 * x;
            if (rr >= nrows) break;
            if (whole) {
                const int fr = fr0 + rr, row = g.s.lo + fr / p.G, h = g.head * p.G + fr % p.G;
                const float inv = l[x] > 0.f ? 1.f / l[x] : 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    store4(out + (static_cast<long long>(row) * p.Hq + h) * D + 4 * (sub + 8 * c),
                           make_float4(o[x][4 * c] * inv, o[x][4 * c + 1] * inv, o[x][4 * c + 2] * inv, o[x][4 * c + 3] * inv));
                if (lse && sub == 0)
                    lse[static_cast<long long>(h) * p.R + row] = l[x] > 0.f ? (m[x] + log2f(l[x])) * kLn2 : -INFINITY;
            } else {
                if (sub == 0) stats[slot + rr] = make_float2(m[x], l[x]);
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    reinterpret_cast<float4*>(part_o + slot * D)[(sub + 8 * c) * slot_rows + rr] =
                        make_float4(o[x][4 * c], o[x][4 * c + 1], o[x][4 * c + 2], o[x][4 * c + 3]);
            }
        }
        if (tid == 0 && !whole && g.t0 == 0)
            jobs[blockIdx.x] = JoinJob{fr0, nrows, g.s.lo, g.head, owner_of(range, g.a + kOV + g.tiles - 1), {0, 0, 0}};
    }
}

// ---------------------------------------------------------------------------
// join of the cut units: O = sum w_i O_i / sum w_i l_i, w_i = 2^(m_i - max m), parts in key order
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;
constexpr int kJoinBatch = 4;  // parts a thread has in flight

// A thread per 16 bytes of O: four head dims of one row of the unit.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const JoinJob* jobs, const float2* stats,
                                                                 const float* part_o, int slot_rows, T* out, float* lse,
                                                                 int R, int Hq, int G) {
    grid_dependency_wait();
    const int c = blockIdx.x;
    const JoinJob job = jobs[c];
    const int x = blockIdx.y * kJoinThreads + threadIdx.x;  // (head dims / 4, row), rows fastest
    if (job.rows == 0 || x >= job.rows * (D / 4)) return;
    const int r = x % job.rows, d4 = x / job.rows;
    const int parts = job.last - c + 1;
    auto slot = [&](int i) { return static_cast<long long>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_rows; };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += kJoinBatch) {
        float2 st[kJoinBatch];
        float4 y[kJoinBatch];
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u)
            if (i0 + u < parts) {
                st[u] = stats[slot(i0 + u) + r];
                y[u] = reinterpret_cast<const float4*>(part_o + slot(i0 + u) * D)[d4 * slot_rows + r];
            }
        float top = m;
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u)
            if (i0 + u < parts) top = fmaxf(top, st[u].x);
        const float base = top == -INFINITY ? 0.f : top, keep = exp2f(m - base);
        m = top;
        l *= keep;
        o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u)
            if (i0 + u < parts) {
                const float w = exp2f(st[u].x - base);
                l = fmaf(w, st[u].y, l);
                o = make_float4(fmaf(w, y[u].x, o.x), fmaf(w, y[u].y, o.y), fmaf(w, y[u].z, o.z), fmaf(w, y[u].w, o.w));
            }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int fr = job.row0 + r, row = job.seq_lo + fr / G, h = job.head * G + fr % G;
    store4(out + (static_cast<long long>(row) * Hq + h) * D + 4 * d4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (lse && d4 == 0) lse[static_cast<long long>(h) * R + row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------
// gathered weight: a thread per key and half of a step's rows
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

template <int D>
struct MassShared {
    float q[kMassRT][D];
    float k[kMassKT][D + 4];
    float nl[kMassRT], half_sum[kMassKT];  // -lse in log2 units
    int rows[kMassKT];
    RangeScratch<kThreads> scratch;
};

template <int D>
__global__ void __launch_bounds__(kThreads) mass_simt_kernel(const CacheBatch p, const float* __restrict__ q,
                                                             const float* __restrict__ k, const float* __restrict__ lse,
                                                             const float* mass_in, float* mass_out,
                                                             int mass_cols, float decay, float scale_log2) {
    __shared__ __align__(16) MassShared<D> sh;
    const int tid = threadIdx.x, key = tid % kMassKT, half = tid / kMassKT;
    unsigned* status = g_cache_simt_status;
    const MassWeight weight{p.G, p.Hkv};
    const WorkRange range = find_range<kThreads>(p, 1, status, weight, sh.scratch);
    long long a = range.a;  // weight before the sequence
    for (int b = range.b; b < p.n_seqs && a < range.hi; ++b) {
        CacheSeq s;
        load_seq(p, b, s);
        const int w = weight.tile(s), tiles = (s.kv + kMassKT - 1) / kMassKT, rows = s.n * p.G;
        const long long count = static_cast<long long>(tiles) * p.Hkv;
        // the tiles whose weight starts inside the range
        long long i = range.lo > a ? quotient(range.lo - a + w - 1, w) : 0;
        const int* table = p.pages + static_cast<long long>(b) * p.max_pages;
        for (; i < count && a + i * w < range.hi; ++i) {
            const int head = static_cast<int>(i / tiles), k0 = static_cast<int>(i % tiles) * kMassKT;
            const long long at = (static_cast<long long>(b) * p.Hkv + head) * mass_cols + k0 + key;
            const bool mine = half == 0 && k0 + key < s.kv;
            const float old = mine && mass_in ? mass_in[at] : 0.f;
            __syncthreads();
            if (tid < kMassKT)
                sh.rows[tid] = rows && k0 + tid < s.kv ? cache_row(table, p.n_pages, p.page_shift, k0 + tid, status) : -1;
            float sum = 0.f;
            for (int fr0 = 0; fr0 < rows; fr0 += kMassRT) {
                __syncthreads();
                if (fr0 == 0) {
#pragma unroll
                    for (int x = tid; x < kMassKT * (D / 4); x += kThreads) {
                        const int kk = x / (D / 4), c = x % (D / 4) * 4, row = sh.rows[kk];
                        copy16(&sh.k[kk][c], k + (row < 0 ? 0 : (static_cast<long long>(row) * p.Hkv + head) * D + c), row >= 0);
                    }
                }
                for (int x = tid; x < kMassRT * (D / 4); x += kThreads) {
                    const int fr = min(fr0 + x / (D / 4), rows - 1), c = x % (D / 4) * 4;
                    copy16(&sh.q[x / (D / 4)][c],
                           q + (static_cast<long long>(s.lo + fr / p.G) * p.Hq + head * p.G + fr % p.G) * D + c, true);
                }
                if (tid < kMassRT) {
                    const int fr = min(fr0 + tid, rows - 1);
                    const float x = lse[static_cast<long long>(head * p.G + fr % p.G) * p.R + s.lo + fr / p.G];
                    sh.nl[tid] = x == -INFINITY ? -INFINITY : -x * kLog2e;
                }
                copies_done();
                __syncthreads();
                float s0[kMassRT / 2], s1[kMassRT / 2];
#pragma unroll
                for (int j = 0; j < kMassRT / 2; ++j) s0[j] = s1[j] = 0.f;
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    const float4 y = lds4(&sh.k[key][c]);
#pragma unroll
                    for (int j = 0; j < kMassRT / 2; ++j) {
                        const float4 x = lds4(&sh.q[half * (kMassRT / 2) + j][c]);
                        ffma2(s0[j], s1[j], x.x, x.y, y.x, y.y, s0[j], s1[j]);
                        ffma2(s0[j], s1[j], x.z, x.w, y.z, y.w, s0[j], s1[j]);
                    }
                }
                const bool masked = k0 + kMassKT > s.kv - s.n;
#pragma unroll
                for (int j = 0; j < kMassRT / 2; ++j) {
                    const int rr = half * (kMassRT / 2) + j, fr = fr0 + rr;
                    if (fr < rows && (!masked || sees(p, s, fr / p.G, k0 + key)))
                        sum += exp2f(fmaf(s0[j] + s1[j], scale_log2, sh.nl[rr]));
                }
            }
            __syncthreads();
            if (half == 1) sh.half_sum[key] = sum;
            __syncthreads();
            if (mine) {
                const float got = sum + sh.half_sum[key];
                mass_out[at] = mass_in ? fmaf(decay, old, got) : got;
            }
        }
        a += count * w;
    }
}

template <int D>
cudaError_t run_tree(const TreeArgs& a, const TreeWs& w, cudaStream_t stream) {
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [&] {
        attr_err = cudaFuncSetAttribute(tree_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(sizeof(TreeShared<D>)));
    });
    if (attr_err != cudaSuccess) return attr_err;
    char* ws = static_cast<char*>(a.ws);
    tree_simt_kernel<D><<<w.ctas, kThreads, sizeof(TreeShared<D>), stream>>>(
        a.p, static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v),
        static_cast<float*>(a.out), a.lse, reinterpret_cast<JoinJob*>(ws), reinterpret_cast<float2*>(ws + w.stat_off),
        reinterpret_cast<float*>(ws + w.o_off), w.slot_rows,
        static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))));
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_join(const TreeArgs& a, const TreeWs& w, cudaStream_t stream) {
    char* ws = static_cast<char*>(a.ws);
    return launch_overlapped(tree_join_kernel<T, D>, dim3(w.ctas, (w.slot_rows * (D / 4) + kJoinThreads - 1) / kJoinThreads),
                             kJoinThreads, 0, stream, static_cast<const JoinJob*>(a.ws),
                             reinterpret_cast<const float2*>(ws + w.stat_off),
                             reinterpret_cast<const float*>(ws + w.o_off), w.slot_rows, static_cast<T*>(a.out), a.lse,
                             a.p.R, a.p.Hq, a.p.G);
}

template <int D>
cudaError_t run_mass(const MassArgs& a, cudaStream_t stream) {
    mass_simt_kernel<D><<<4 * device_sm_count(), kThreads, 0, stream>>>(
        a.p, static_cast<const float*>(a.q), static_cast<const float*>(a.k), a.lse, a.in, a.out, a.mass_cols, a.decay,
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

TreeWs tree_simt_workspace(int R, int G, int D) {
    return tree_workspace(R, G, D, (D == 64 ? 4 : 2) * device_sm_count(), kTreeSimtRows);  // CTAs that fit an SM
}

cudaError_t launch_tree_join(const TreeArgs& a, const TreeWs& w, int bf16, cudaStream_t stream) {
    if (bf16) return a.D == 128 ? run_join<__nv_bfloat16, 128>(a, w, stream) : run_join<__nv_bfloat16, 64>(a, w, stream);
    return a.D == 128 ? run_join<float, 128>(a, w, stream) : run_join<float, 64>(a, w, stream);
}

cudaError_t launch_tree_simt(const TreeArgs& a, cudaStream_t stream) {
    const TreeWs w = tree_simt_workspace(a.p.R, a.p.G, a.D);
    const cudaError_t e = a.D == 128 ? run_tree<128>(a, w, stream) : run_tree<64>(a, w, stream);
    return e != cudaSuccess ? e : launch_tree_join(a, w, 0, stream);
}

cudaError_t launch_mass_simt(const MassArgs& a, cudaStream_t stream) {
    return a.D == 128 ? run_mass<128>(a, stream) : run_mass<64>(a, stream);
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
