// cache_attn_simt.cu -- attention over a paged cache and the weight gathered per key in
// exact fp32 on the CUDA cores, and the join of cut units (for both precisions).
//
// Scores, exponentials and P V are fp32 FMA (two at a time, fma.rn.f32x2) and exp2f;
// nothing is rounded to fewer bits.  K and V tiles arrive by cp.async one tile ahead of
// their use, their pool rows looked up two ahead.
#include <cmath>

#include "cache_simt.cuh"

namespace ra {

static __device__ unsigned g_cache_simt_status[2];

namespace {

// ---------------------------------------------------------------------------
// attention
//
// What bounds a CUDA-core kernel here is the 128 bytes a cycle that shared memory hands
// to registers, so every 16 bytes of K or V that a lane receives meet four rows: a lane
// holds sixteen head dims of four rows' queries and of their O in registers (D / 16
// lanes share a row group) and reads nothing but K and V.  The lanes' partial scores are
// added up so that each of four lanes ends with one row's score, does that row's
// softmax, and hands its weight back to the others.  Units of few rows take several
// keys at a time instead of idle row groups.  Per key and 32 rows (D = 64) that is 39
// cycles of shared memory, against 88 with scores split over the threads (2 x 4 each)
// and 130 with a lane per row.  The states of the warps and key groups are combined at
// the end of a segment as those of cut units are.  4 sequences of up to 8 tokens and 4096
// keys, 16 / 4 heads, D = 64: 26 us (42 with a row per 8 threads).
// ---------------------------------------------------------------------------
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kOV = 2;              // weight of a unit beyond its tiles
constexpr int kMinW = 2;            // least weight per CTA
// Weights are taken against a reference that follows the row's maximum only where a score is past it by kSlack: a
// weight stays below 2^8 and keeps its relative error, and few batches scale O (27.5 -> 25.8 us on the case above).
constexpr float kSlack = 8.f;
constexpr int kBatch = 2;           // keys of a lane whose scores are taken together

template <int D>
struct TreeCfg {
    static constexpr int kLanes = D / 16;           // of a row group
    static constexpr int kGroups = 32 / kLanes;     // of a warp
    static constexpr int kRT = 4 * kGroups;         // rows of a unit
    static constexpr int kKT = 4096 / D;            // keys of a tile
};
template <int D>
struct TreeShared {
    float k[2][TreeCfg<D>::kKT][D];
    float v[2][TreeCfg<D>::kKT][D];
    float m[128], l[128];          // [state][row]
    int rows[2][TreeCfg<D>::kKT];  // pool rows of a tile's keys, -1: zeros
    RangeScratch<kThreads> scratch;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) tree_simt_kernel(const CacheBatch p, const float* q, const float* k,
                                                                const float* v, float* out, float* lse,
                                                                JoinJob* jobs, float2* stats, float* part_o, int slot_rows,
                                                                float scale_log2) {
    using C = TreeCfg<D>;
    constexpr int KT = C::kKT, RT = C::kRT, L = C::kLanes;
    extern __shared__ __align__(16) unsigned char raw[];
    TreeShared<D>& sh = *reinterpret_cast<TreeShared<D>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, dl = lane % L, group = lane / L;
    const bool b0 = lane & 1, b1 = lane & 2;
    unsigned* status = g_cache_simt_status;
    const bool tree = p.tree_mask != nullptr;
    grid_dependency_wait();
    const WorkRange range =
        find_range<kThreads>(p, kMinW, status, TreeWeight<KT, kOV>{p.G, p.Hkv, tree, RT}, sh.scratch);
    if (tid == 0) jobs[blockIdx.x].rows = 0;
    SegmentWalk<KT, kOV> walk;
    walk.start(p, range, RT);
    Segment g;
    while (walk.next(p, range, g)) {
        const int fr0 = g.rt * RT, nrows = min(RT, g.s.n * p.G - fr0);
        // row groups of the unit (a power of two) and keys that the other groups of a warp take next to them
        int rg = 1;
        while (4 * rg < nrows) rg *= 2;
        const int ks = C::kGroups / rg, row0 = (group % rg) * 4, state = warp * ks + group / rg, states = kWarps * ks;
        const int* table = p.pages + static_cast<long long>(g.b) * p.max_pages;
        auto pool_row = [&](int tile) {  // of key tid of the tile
            const int j = tile * KT + tid;
            return tile < g.t1 && j < g.s.kv ? cache_row(table, p.n_pages, p.page_shift, j, status) : -1;
        };
        auto fetch = [&](int tile, int buf) {
#pragma unroll 4
            for (int i = tid; i < KT * (D / 4); i += kThreads) {
                const int kk = i / (D / 4), c = i % (D / 4) * 4, row = sh.rows[buf][kk];
                const long long at = row < 0 ? 0 : (static_cast<long long>(row) * p.Hkv + g.head) * D + c;
                copy16(&sh.k[buf][kk][c], k + at, row >= 0);
                copy16(&sh.v[buf][kk][c], v + at, row >= 0);
            }
        };
        __syncthreads();  // the segment before is done with shared memory
        if (tid < KT) {
            sh.rows[0][tid] = pool_row(g.t0);
            sh.rows[1][tid] = pool_row(g.t0 + 1);
        }
        __syncthreads();
        if (g.t0 < g.t1) fetch(g.t0, 0);
        // this lane's dims of its four rows: 16-byte pieces dl, dl + L, ...
        float qr[4][16], o[4][16], m = -INFINITY, l = 0.f;
        const int last = g.s.n * p.G - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int fr = min(fr0 + row0 + j, last);
            const float* src = q + (static_cast<long long>(g.s.lo + fr / p.G) * p.Hq + g.head * p.G + fr % p.G) * D + 4 * dl;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 x = lds4(src + 4 * L * c);
                qr[j][4 * c] = x.x;
                qr[j][4 * c + 1] = x.y;
                qr[j][4 * c + 2] = x.z;
                qr[j][4 * c + 3] = x.w;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) o[j][c] = 0.f;
        }
        const int own = row0 + (lane & 3), tok = min(fr0 + own, last) / p.G;  // the row whose softmax this lane does
        copies_done();
        __syncthreads();
        for (int tile = g.t0; tile < g.t1; ++tile) {
            const int buf = (tile - g.t0) & 1, k0 = tile * KT;
            if (tile + 1 < g.t1) fetch(tile + 1, buf ^ 1);
            const int row_ahead = tid < KT ? pool_row(tile + 2) : -1;
            const bool masked = k0 + KT > g.s.kv - g.s.n;  // new tokens in the tile
#pragma unroll 1
            for (int kb = state; kb < KT; kb += states * kBatch) {
                float e[kBatch];
                // scores, even and odd dims in the two lanes of a packed sum
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float* key = sh.k[buf][kb + states * i] + 4 * dl;
                    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float4 x = lds4(key + 4 * L * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            ffma2(s0[j], s1[j], qr[j][4 * c], qr[j][4 * c + 1], x.x, x.y, s0[j], s1[j]);
                            ffma2(s0[j], s1[j], qr[j][4 * c + 2], qr[j][4 * c + 3], x.z, x.w, s0[j], s1[j]);
                        }
                    }
                    // each lane of four keeps one row: two halvings
                    const float r0 = s0[0] + s1[0], r1 = s0[1] + s1[1], r2 = s0[2] + s1[2], r3 = s0[3] + s1[3];
                    const float u0 = (b1 ? r2 : r0) + __shfl_xor_sync(0xffffffffu, b1 ? r0 : r2, 2);
                    const float u1 = (b1 ? r3 : r1) + __shfl_xor_sync(0xffffffffu, b1 ? r1 : r3, 2);
                    float x = (b0 ? u1 : u0) + __shfl_xor_sync(0xffffffffu, b0 ? u0 : u1, 1);
                    if (L == 8) x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x *= scale_log2;
                    if (masked && !sees(p, g.s, tok, k0 + kb + states * i)) x = -INFINITY;
                    e[i] = x;
                }
                float mx = m;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) mx = fmaxf(mx, e[i]);
                const float next_m = mx > m + kSlack ? mx : m;
                const float base = next_m == -INFINITY ? 0.f : next_m, alpha = exp2f(m - base);
                const bool scale = __any_sync(0xffffffffu, next_m != m);
                m = next_m;
                l *= alpha;
                float w[kBatch][4];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    e[i] = exp2f(e[i] - base);
                    l += e[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[i][j] = __shfl_sync(0xffffffffu, e[i], (lane & ~3) | j);
                }
                if (scale) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float f = __shfl_sync(0xffffffffu, alpha, (lane & ~3) | j);
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[j][c] *= f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float* val = sh.v[buf][kb + states * i] + 4 * dl;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float4 x = lds4(val + 4 * L * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            ffma2(o[j][4 * c], o[j][4 * c + 1], w[i][j], w[i][j], x.x, x.y, o[j][4 * c], o[j][4 * c + 1]);
                            ffma2(o[j][4 * c + 2], o[j][4 * c + 3], w[i][j], w[i][j], x.z, x.w, o[j][4 * c + 2], o[j][4 * c + 3]);
                        }
                    }
                }
            }
            copies_done();
            __syncthreads();  // the next tile is there, and everyone is done with this one's rows
            if (tid < KT) sh.rows[buf][tid] = row_ahead;
            __syncthreads();
        }
        // the states, O as [state][16-byte piece][row] in the K tiles' place
        const int rows = 4 * rg;
        float4* const so = reinterpret_cast<float4*>(raw);
        static_assert(sizeof(float) * 32 * 64 * kWarps <= sizeof(TreeShared<D>::k), "the states' O fits the K tiles");
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                so[(state * (D / 4) + dl + L * c) * rows + row0 + j] =
                    make_float4(o[j][4 * c], o[j][4 * c + 1], o[j][4 * c + 2], o[j][4 * c + 3]);
        if (dl < 4) {
            sh.m[state * rows + own] = m;
            sh.l[state * rows + own] = l;
        }
        __syncthreads();
        const bool whole = g.whole();
        const long long slot = static_cast<long long>(partial_slot(g)) * slot_rows;
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int rr = x % rows, d4 = x / rows;
            if (rr >= nrows) continue;
            float top = -INFINITY, sum = 0.f;
            for (int w = 0; w < states; ++w) top = fmaxf(top, sh.m[w * rows + rr]);
            const float base = top == -INFINITY ? 0.f : top;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = 0; w < states; ++w) {
                const float f = exp2f(sh.m[w * rows + rr] - base);
                const float4 z = so[w * rows * (D / 4) + x];
                sum = fmaf(f, sh.l[w * rows + rr], sum);
                y = make_float4(fmaf(f, z.x, y.x), fmaf(f, z.y, y.y), fmaf(f, z.z, y.z), fmaf(f, z.w, y.w));
            }
            if (whole) {
                const int fr = fr0 + rr, row = g.s.lo + fr / p.G, h = g.head * p.G + fr % p.G;
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
                store4(out + (static_cast<long long>(row) * p.Hq + h) * D + 4 * d4,
                       make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
                if (lse && d4 == 0)
                    lse[static_cast<long long>(h) * p.R + row] = row_lse(top, sum);
            } else {
                reinterpret_cast<float4*>(part_o + slot * D)[d4 * slot_rows + rr] = y;
                if (d4 == 0) stats[slot + rr] = make_float2(top, sum);
            }
        }
        if (tid == 0 && !whole && g.t0 == 0)
            jobs[blockIdx.x] = JoinJob{fr0, nrows, g.s.lo, g.head, owner_of(range, g.a + kOV + g.tiles - 1), {0, 0, 0}};
    }
}

// ---------------------------------------------------------------------------
// join of the cut units: O = sum w_i O_i / sum w_i l_i, w_i = 2^(m_i - max m), parts in key order
// ---------------------------------------------------------------------------
constexpr int kJoinBatch = 4;  // parts a thread has in flight

// State of a row's four head dims over some of its parts.
struct JoinState {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void scale_to(float top) {
        const float keep = exp2f(m - (top == -INFINITY ? 0.f : top));
        m = top;
        l *= keep;
        o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
    }
    __device__ __forceinline__ void add(float pm, float pl, float4 y) {  // pm <= m
        const float w = exp2f(pm - (m == -INFINITY ? 0.f : m));
        l = fmaf(w, pl, l);
        o = make_float4(fmaf(w, y.x, o.x), fmaf(w, y.y, o.y), fmaf(w, y.z, o.z), fmaf(w, y.w, o.w));
    }
};

// A thread per 16 bytes of O: four head dims of one row of the unit.  LANES threads share one where few long units
// are cut into many parts (one token over 16000 keys, 38 parts: the call takes 24.4 us joined by one thread each,
// 21.8 by eight; 8 sequences of 2000 keys in fp32, 5 parts: 41.5 and 44.2).
template <typename T, int D, int LANES>
__global__ void __launch_bounds__(128) tree_join_kernel(const JoinJob* jobs, const float2* stats, const float* part_o,
                                                        int slot_rows, T* out, float* lse, int R, int Hq, int G) {
    constexpr int kOut = 128 / LANES;
    __shared__ float sm[LANES][kOut], sl[LANES][kOut];
    __shared__ float4 so[LANES][kOut];
    grid_dependency_wait();
    const int c = blockIdx.x;
    const JoinJob job = jobs[c];
    const int outs = job.rows * (D / 4);
    if (static_cast<int>(blockIdx.y) * kOut >= outs) return;
    const int x = blockIdx.y * kOut + threadIdx.x % kOut, pl = threadIdx.x / kOut;  // (head dims / 4, row), rows fastest
    const bool in = x < outs;
    const int r = in ? x % job.rows : 0, d4 = in ? x / job.rows : 0;
    const int parts = in ? job.last - c + 1 : 0;
    auto slot = [&](int i) { return static_cast<long long>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_rows; };
    JoinState s;
    for (int i0 = pl; i0 < parts; i0 += LANES * kJoinBatch) {
        float2 st[kJoinBatch];
        float4 y[kJoinBatch];
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u) {
            const int i = i0 + u * LANES;
            if (i < parts) {
                st[u] = stats[slot(i) + r];
                y[u] = reinterpret_cast<const float4*>(part_o + slot(i) * D)[d4 * slot_rows + r];
            }
        }
        float top = s.m;
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u)
            if (i0 + u * LANES < parts) top = fmaxf(top, st[u].x);
        s.scale_to(top);
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u)
            if (i0 + u * LANES < parts) s.add(st[u].x, st[u].y, y[u]);
    }
    if (LANES > 1) {
        const int at = threadIdx.x % kOut;
        sm[pl][at] = s.m;
        sl[pl][at] = s.l;
        so[pl][at] = s.o;
        __syncthreads();
        if (pl > 0) return;
        float top = s.m;
#pragma unroll
        for (int u = 1; u < LANES; ++u) top = fmaxf(top, sm[u][at]);
        s.scale_to(top);
#pragma unroll
        for (int u = 1; u < LANES; ++u) s.add(sm[u][at], sl[u][at], so[u][at]);
    }
    if (!in) return;
    const float inv = s.l > 0.f ? 1.f / s.l : 0.f;
    const int fr = job.row0 + r, row = job.seq_lo + fr / G, h = job.head * G + fr % G;
    store4(out + (static_cast<long long>(row) * Hq + h) * D + 4 * d4,
           make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv));
    if (lse && d4 == 0) lse[static_cast<long long>(h) * R + row] = row_lse(s.m, s.l);
}

// ---------------------------------------------------------------------------
// gathered weight: a thread per key and half of a step's rows, summed in registers.  2 sequences of 2048 keys and 8
// tokens, 8 / 4 heads, D = 64: 8.2 us, the latencies of one tile per CTA.
// ---------------------------------------------------------------------------
constexpr int kMassKT = 64;   // keys of a tile
constexpr int kMassRT = 16;   // rows staged per step

// A tile of keys weighs its row steps plus one.
struct MassWeight {
    int G, heads;
    __device__ __forceinline__ int tile(const CacheSeq& s) const { return (s.n * G + kMassRT - 1) / kMassRT + 1; }
    __device__ __forceinline__ long long head(const CacheSeq& s) const {
        return static_cast<long long>((s.kv + kMassKT - 1) / kMassKT) * tile(s);
    }
    __device__ __forceinline__ long long locate(const CacheSeq&, long long, long long, int&, int&) const { return 0; }
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
__global__ void __launch_bounds__(kThreads) mass_simt_kernel(const CacheBatch p, const float* q, const float* k, const float* lse,
                                                             const float* mass_in, float* mass_out,
                                                             int mass_cols, float decay, float scale_log2) {
    __shared__ __align__(16) MassShared<D> sh;
    const int tid = threadIdx.x, key = tid % kMassKT, half = tid / kMassKT;
    unsigned* status = g_cache_simt_status;
    const MassWeight weight{p.G, p.Hkv};
    grid_dependency_wait();
    const WorkRange range = find_range<kThreads>(p, 1, status, weight, sh.scratch);
    long long a = range.a;  // weight before the sequence
    for (int b = range.b; b < p.n_seqs && a < range.hi; ++b) {
        CacheSeq s = range.s;
        if (b != range.b) load_seq(p, b, s);
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
    static OncePerDevice once;
    const cudaError_t set = once([] {
        return cudaFuncSetAttribute(tree_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(sizeof(TreeShared<D>)));
    });
    if (set != cudaSuccess) return set;
    char* ws = static_cast<char*>(a.ws);
    return launch_overlapped(
        tree_simt_kernel<D>, dim3(w.ctas), kThreads, sizeof(TreeShared<D>), stream, a.p, static_cast<const float*>(a.q),
        static_cast<const float*>(a.k), static_cast<const float*>(a.v), static_cast<float*>(a.out), a.lse,
        reinterpret_cast<JoinJob*>(ws), reinterpret_cast<float2*>(ws + w.stat_off), reinterpret_cast<float*>(ws + w.o_off),
        w.slot_rows, static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))));
}

template <typename T, int D, int LANES>
cudaError_t run_join_lanes(const TreeArgs& a, const TreeWs& w, cudaStream_t stream) {
    char* ws = static_cast<char*>(a.ws);
    const int outs = 128 / LANES;
    return launch_overlapped(tree_join_kernel<T, D, LANES>, dim3(w.ctas, (w.slot_rows * (D / 4) + outs - 1) / outs), 128, 0,
                             stream, static_cast<const JoinJob*>(a.ws), reinterpret_cast<const float2*>(ws + w.stat_off),
                             reinterpret_cast<const float*>(ws + w.o_off), w.slot_rows, static_cast<T*>(a.out), a.lse,
                             a.p.R, a.p.Hq, a.p.G);
}

template <typename T, int D>
cudaError_t run_join(const TreeArgs& a, const TreeWs& w, cudaStream_t stream) {
    // few rows and many parts (the CTAs over the sequences' KV heads): several threads per output
    const bool many = w.slot_rows <= 32 && w.ctas >= 16ll * a.p.n_seqs * a.p.Hkv;
    return many ? run_join_lanes<T, D, 8>(a, w, stream) : run_join_lanes<T, D, 1>(a, w, stream);
}

template <int D>
cudaError_t run_mass(const MassArgs& a, cudaStream_t stream) {
    return launch_overlapped(
        mass_simt_kernel<D>, dim3(4 * device_sm_count()), kThreads, 0, stream, a.p, static_cast<const float*>(a.q),
        static_cast<const float*>(a.k), a.lse, a.in, a.out, a.mass_cols, a.decay,
        static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))));
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
    return tree_workspace(R, G, D, 2 * device_sm_count(), D == 128 ? TreeCfg<128>::kRT : TreeCfg<64>::kRT);
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
