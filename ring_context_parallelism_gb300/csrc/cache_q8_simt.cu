// cache_q8_simt.cu -- attention over an 8-bit paged cache on the CUDA cores (fp32 queries).
//
// The walk, the split of a unit's rows and keys over the lanes and the joining of their
// states are those of the fp32 attention over 16- and 32-bit pages: a lane holds sixteen
// head dims of four rows' queries and of their O, so that every code it reads from shared
// memory meets four rows.  The codes stay codes until a lane has them in registers (16
// dims are one 16-byte load, not four); a key's scale multiplies its score, a value's
// scale the weight it gets in O, so scaling costs one product per row and key.
//
// 4 sequences of 1 to 8 tokens over 4K keys, 16 / 4 heads, D = 64: 27 us (25 over 32-bit pages), where the FMAs
// alone would take 4: the prelude and the joining of the states, and in between the chain from scores over shuffles to
// weights with 7 warps an SM at work, and the conversion of the codes, which each row group does for itself.
#include <cmath>

#include "cache_q8.cuh"

namespace ra {

static __device__ unsigned g_cache_q8_simt_status[2];

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kOV = 2;              // weight of a unit beyond its tiles
constexpr int kMinW = 2;            // least weight per CTA
constexpr float kSlack = 8.f;       // log2 by which a score may pass the reference of its row's weights
constexpr int kBatch = 2;           // keys of a lane whose scores are taken together

template <int D>
struct Q8Cfg {
    static constexpr int kLanes = D / 16;           // of a row group
    static constexpr int kGroups = 32 / kLanes;     // of a warp
    static constexpr int kRT = 4 * kGroups;         // rows of a unit
    static constexpr int kKT = 4096 / D;            // keys of a tile
};
template <int D>
struct Q8Shared {
    static constexpr int KT = Q8Cfg<D>::kKT;
    union {
        struct {
            unsigned char k[2][KT][D], v[2][KT][D];
            float ks[2][KT], vs[2][KT];  // scales, those of K with the scale of the scores
            int rows[2][KT];             // pool rows of a tile's keys, -1: zeros
        };
        float4 o[32 * 64 * kWarps / 4];  // the states' O
    };
    float m[128], l[128];                // [state][row]
    RangeScratch<kThreads> scratch;
};

__device__ __forceinline__ void load16(const float* p, float* x) {
    load8(p, x);
    load8(p + 8, x + 8);
}
__device__ __forceinline__ void load16(const unsigned char* p, float* x) {
    const uint4 c = *reinterpret_cast<const uint4*>(p);
    values4(c.x, x);
    values4(c.y, x + 4);
    values4(c.z, x + 8);
    values4(c.w, x + 12);
}
__device__ __forceinline__ void copy16_codes(unsigned char* dst, const unsigned char* src, bool ok) {
    copy16(reinterpret_cast<float*>(dst), reinterpret_cast<const float*>(src), ok);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) q8_simt_kernel(const CacheBatch p, const float* q, const Q8Pools pools, float* out,
                                                              float* lse, JoinJob* jobs, float2* stats, float* part_o,
                                                              int slot_rows, float scale_log2) {
    using C = Q8Cfg<D>;
    constexpr int KT = C::kKT, RT = C::kRT, L = C::kLanes;
    __shared__ __align__(16) Q8Shared<D> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, dl = lane % L, group = lane / L;
    const bool b0 = lane & 1, b1 = lane & 2;
    unsigned* status = g_cache_q8_simt_status;
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
        // pool row and scales of key tid of a tile
        auto look_up = [&](int tile, int& row, unsigned& ek, unsigned& ev) {
            const int j = tile * KT + tid;
            row = tile < g.t1 && j < g.s.kv ? cache_row(table, p.n_pages, p.page_shift, j, status) : -1;
            ek = ev = 0;
            if (row >= 0) {
                const int page = row >> p.page_shift;
                const long long at = ((static_cast<long long>(page) * p.Hkv + g.head) << p.page_shift) + (row - (page << p.page_shift));
                ek = pools.ks[at];
                ev = pools.vs[at];
            }
        };
        auto note = [&](int buf, int row, unsigned ek, unsigned ev) {
            sh.rows[buf][tid] = row;
            sh.ks[buf][tid] = scale_of(ek) * scale_log2;
            sh.vs[buf][tid] = scale_of(ev);
        };
        auto fetch = [&](int buf) {
#pragma unroll
            for (int i = tid; i < KT * (D / 16); i += kThreads) {
                const int kk = i / (D / 16), c = i % (D / 16) * 16, row = sh.rows[buf][kk];
                const long long at = row < 0 ? 0 : (static_cast<long long>(row) * p.Hkv + g.head) * D + c;
                copy16_codes(&sh.k[buf][kk][c], pools.k + at, row >= 0);
                copy16_codes(&sh.v[buf][kk][c], pools.v + at, row >= 0);
            }
        };
        __syncthreads();  // the segment before is done with shared memory
        if (tid < KT) {
            int row[2];
            unsigned ek[2], ev[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) look_up(g.t0 + t, row[t], ek[t], ev[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t) note(t, row[t], ek[t], ev[t]);
        }
        __syncthreads();
        if (g.t0 < g.t1) fetch(0);
        // this lane's dims of its four rows: 16 dl .. 16 dl + 15
        float qr[4][16], o[4][16], m = -INFINITY, l = 0.f;
        const int last = g.s.n * p.G - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int fr = min(fr0 + row0 + j, last);
            load16(q + (static_cast<long long>(g.s.lo + fr / p.G) * p.Hq + g.head * p.G + fr % p.G) * D + 16 * dl, qr[j]);
#pragma unroll
            for (int c = 0; c < 16; ++c) o[j][c] = 0.f;
        }
        const int own = row0 + (lane & 3), tok = min(fr0 + own, last) / p.G;  // the row whose softmax this lane does
        copies_done();
        __syncthreads();
        for (int tile = g.t0; tile < g.t1; ++tile) {
            const int buf = (tile - g.t0) & 1, k0 = tile * KT;
            if (tile + 1 < g.t1) fetch(buf ^ 1);
            int row_ahead = -1;
            unsigned ek_ahead = 0, ev_ahead = 0;
            if (tid < KT) look_up(tile + 2, row_ahead, ek_ahead, ev_ahead);
            const bool masked = k0 + KT > g.s.kv - g.s.n;  // new tokens in the tile
#pragma unroll 1
            for (int kb = state; kb < KT; kb += states * kBatch) {
                float e[kBatch];
                // scores, even and odd dims in the two lanes of a packed sum
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int kk = kb + states * i;
                    float key[16];
                    load16(&sh.k[buf][kk][16 * dl], key);
                    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 16; c += 2)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            ffma2(s0[j], s1[j], qr[j][c], qr[j][c + 1], key[c], key[c + 1], s0[j], s1[j]);
                    // each lane of four keeps one row: two halvings
                    const float r0 = s0[0] + s1[0], r1 = s0[1] + s1[1], r2 = s0[2] + s1[2], r3 = s0[3] + s1[3];
                    const float u0 = (b1 ? r2 : r0) + __shfl_xor_sync(0xffffffffu, b1 ? r0 : r2, 2);
                    const float u1 = (b1 ? r3 : r1) + __shfl_xor_sync(0xffffffffu, b1 ? r1 : r3, 2);
                    float x = (b0 ? u1 : u0) + __shfl_xor_sync(0xffffffffu, b0 ? u0 : u1, 1);
                    if (L == 8) x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x *= sh.ks[buf][kk];
                    if (masked && !sees(p, g.s, tok, k0 + kk)) x = -INFINITY;
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
                    const float sv = sh.vs[buf][kb + states * i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[i][j] = __shfl_sync(0xffffffffu, e[i], (lane & ~3) | j) * sv;
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
                    float val[16];
                    load16(&sh.v[buf][kb + states * i][16 * dl], val);
#pragma unroll
                    for (int c = 0; c < 16; c += 2)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            ffma2(o[j][c], o[j][c + 1], w[i][j], w[i][j], val[c], val[c + 1], o[j][c], o[j][c + 1]);
                }
            }
            copies_done();
            __syncthreads();  // the next tile is there, and everyone is done with this one
            if (tid < KT) note(buf, row_ahead, ek_ahead, ev_ahead);
            __syncthreads();
        }
        // the states, O as [state][16-byte piece][row] in the tiles' place
        const int rows = 4 * rg;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sh.o[(state * (D / 4) + 4 * dl + c) * rows + row0 + j] =
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
                const float4 z = sh.o[w * rows * (D / 4) + x];
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

template <int D>
cudaError_t run(const TreeArgs& a, const Q8Pools& pools, const TreeWs& w, cudaStream_t stream) {
    char* ws = static_cast<char*>(a.ws);
    return launch_overlapped(q8_simt_kernel<D>, dim3(w.ctas), kThreads, 0, stream, a.p, static_cast<const float*>(a.q), pools,
                             static_cast<float*>(a.out), a.lse, reinterpret_cast<JoinJob*>(ws),
                             reinterpret_cast<float2*>(ws + w.stat_off), reinterpret_cast<float*>(ws + w.o_off), w.slot_rows,
                             static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))));
}

}  // namespace

TreeWs tree_q8_simt_workspace(int R, int G, int D) {
    return tree_workspace(R, G, D, 2 * device_sm_count(), D == 128 ? Q8Cfg<128>::kRT : Q8Cfg<64>::kRT);
}

cudaError_t launch_tree_q8_simt(const TreeArgs& a, const Q8Pools& pools, cudaStream_t stream) {
    const TreeWs w = tree_q8_simt_workspace(a.p.R, a.p.G, a.D);
    const cudaError_t e = a.D == 128 ? run<128>(a, pools, w, stream) : run<64>(a, pools, w, stream);
    return e != cudaSuccess ? e : launch_tree_join(a, w, 0, stream);
}

unsigned read_clear_status_cache_q8_simt(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_q8_simt_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_q8_simt_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
