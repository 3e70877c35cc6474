// cache_attn_tc.cu -- attention over a paged cache on the tensor cores (bf16).
//
// A unit is NT row tiles of 128 rows (whole tokens: 128 / G tokens of G rows
// each) of one sequence and KV head, walked over KT-key tiles with the online
// softmax: S = Q K^T (tcgen05, fp32 in TMEM), P = 2^(S c - m) (bf16 over S), O +=
// P V (tcgen05, O in TMEM).  m only moves when a tile's maximum passes it by 2^8.
//   NT = 1, KT = 64, two CTAs per SM: few rows, the cache's bytes bound it.  Two S
//     buffers, so that Q K^T of the next tile runs under the softmax of this one.
//     32 sequences of 4K-16K keys, one token each, 64 / 8 heads, D = 128: 204 us, 6.6
//     TB/s (0.97 of the measured copy rate).
//   NT = 2, KT = 128, one CTA per SM: many rows, the tensor pipe bounds it.  Both
//     row tiles read one K/V tile from shared memory and take turns on the pipe: 2580
//     cycles a pair, 2048 of them MMAs.  4 trees of up to 64 tokens over up to 32768
//     keys: 128 us, 1150 TFLOP/s, call after call (the clocks fall under the power cap);
//     118 us in a burst of twenty.
//
// Roles: 4 NT softmax warps (a thread per row), one warp each that streams K and V
// pages into a ring of its own, one that issues the MMAs.  Keys past a sequence's
// length: pages past its list load zeros, the rest of its last page is masked in S and
// zeroed in the V tile (stale memory there may hold NaN, and 0 * NaN is NaN).
#include <cmath>

#include "cache_batch.cuh"

namespace ra {

static __device__ unsigned g_cache_tc_status[2];

namespace {

constexpr float kRescaleLog2 = 8.0f;

template <int D, int NT>
struct Cfg {
    static constexpr int kKT = NT == 1 ? 64 : 128;      // keys per tile
    static constexpr int kChunks = D / 64;
    static constexpr int kSoftmax = 128 * NT;           // softmax threads
    // softmax warps, K producer, V (and Q) producer, issuer; NT = 2 fills its last warpgroup for setmaxnreg
    static constexpr int kThreads = kSoftmax + (NT == 1 ? 96 : 128);
    static constexpr int kQBytes = 128 * D * 2;         // one row tile of Q
    static constexpr int kStageBytes = kKT * D * 2;
    static constexpr int kHead = 1024;                  // barriers and scratch ahead of the tiles
    static constexpr int kBudget = NT == 1 ? 112 * 1024 : 224 * 1024;
    static constexpr int kFit = (kBudget - NT * kQBytes) / kStageBytes;
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr int kV = kStages / 2, kK = kStages - kV;  // stages of the two rings
    static constexpr int kSmem = kHead + NT * kQBytes + kStages * kStageBytes;
    static constexpr int kTmemCols = 256 * NT;
    static constexpr int kOCol = 128;   // O columns of a row tile, behind its S
    static constexpr int kOV = NT == 1 ? 3 : 4;         // weight of a unit beyond its tiles
    static constexpr int kMinW = NT == 1 ? 2 : 3;       // least weight per CTA
};

struct TcParams {
    CacheBatch p;
    int rpt;         // tokens of a row tile
    int q_bytes;     // bytes of Q a row tile's load brings per 64-column chunk
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    JoinJob* jobs;
    float2* stats;
    float* part_o;
    int slot_rows;
};

struct Bars {
    uint64_t full[2][5], empty[2][5];  // stages of the K ring and the V ring
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2];  // by S buffer (NT = 1) or row tile (NT = 2)
    uint64_t p_half[2];             // NT = 2: the first 64 keys of P
    uint64_t o_done[2];             // P V done: as s_full, so that one parity tells its phases apart
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// NT = 2 launches 384 threads with 168 registers each and hands the softmax warpgroups 224 of them (256 x 224 +
// 128 x 56 = 384 x 168): their 128 scores then stay in registers (216 and 72: more spilled, 25-token trees 51.5 us
// against 51.2; with 232 and 40 the other warps spill).  NT = 1 has 64 scores and needs no split.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= 384 * kLaunchRegs, "the split exceeds the launch's registers");
template <int NT>
__device__ __forceinline__ void reg_dec() {
    if (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs) : "memory");
}
template <int NT>
__device__ __forceinline__ void reg_inc() {
    if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, NT == 1 ? 2 : 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcParams a) {
    using C = Cfg<D, NT>;
    constexpr int KT = C::kKT;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars& bar = *reinterpret_cast<Bars*>(smem);
    RangeScratch<C::kThreads>& scratch = *reinterpret_cast<RangeScratch<C::kThreads>*>(smem + 512);
    static_assert(sizeof(Bars) <= 512 && sizeof(RangeScratch<C::kThreads>) <= 512, "head of the shared memory");
    uint8_t* q_smem = smem + C::kHead;
    uint8_t* k_ring = q_smem + NT * C::kQBytes;
    uint8_t* v_ring = k_ring + C::kK * C::kStageBytes;
    const CacheBatch& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* status = g_cache_tc_status;
    const bool tree = p.tree_mask != nullptr;
    const int row_tile = NT * a.rpt * p.G;
    if (smem_u32(smem) & 1023) {  // swizzled tiles start on 1024 bytes
        if (threadIdx.x == 0) cache_report(status, 0x0C000000u);
        return;
    }

    constexpr int kProducerK = C::kSoftmax / 32, kProducerV = kProducerK + 1, kIssuer = kProducerK + 2;
    if (warp == kIssuer) {
        if (lane == 0) {
            for (int s = 0; s < 5; ++s)
                for (int r = 0; r < 2; ++r) {
                    mbar_init(&bar.full[r][s], 1);
                    mbar_init(&bar.empty[r][s], 1);
                }
            mbar_init(&bar.q_full, 1);
            mbar_init(&bar.q_empty, 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(&bar.s_full[t], 1);
                mbar_init(&bar.p_half[t], 128);
                mbar_init(&bar.p_full[t], 128);
                mbar_init(&bar.o_done[t], 1);
            }
            mbar_init(&bar.drain, 1);
            bar.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&bar.tmem, C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kProducerK && lane == 0) tma_prefetch_desc(&tm_k);
    if (warp == kProducerV && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_v);
    }
    grid_dependency_wait();    // nothing above reads or writes global memory
    grid_launch_dependents();  // the join may take its place on the SMs; it waits for this grid's end
    if (threadIdx.x == 0) a.jobs[blockIdx.x].rows = 0;
    tc_fence_before();
    const WorkRange& range = find_range<C::kThreads>(
        p, C::kMinW, status, TreeWeight<KT, C::kOV>{p.G, p.Hkv, tree, row_tile}, scratch);
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    volatile int* abort_flag = &bar.abort;
    SegmentWalk<KT, C::kOV> walk;
    walk.start(p, range, row_tile);
    Segment g;
    int place = 0, n_q_loads = 0;  // of a producer: tiles and row tiles of Q loaded so far

    if (warp == kProducerK || warp == kProducerV) {
        // ---------------------------------------------------------------- pages -> shared memory
        // one warp brings K, one V (and Q): a box costs its warp some hundred cycles to issue
        reg_dec<NT>();
        const bool is_k = warp == kProducerK;
        const CUtensorMap* map = is_k ? &tm_k : &tm_v;
        const int ring = is_k ? 0 : 1, n_stages = is_k ? C::kK : C::kV;
        int segs = 0;
        bool ok = true;
        const int sub_rows = min(1 << p.page_shift, KT);  // rows of a box
        const int groups = KT / sub_rows;                 // pages of a tile (at most 16): lane g finds page g
        const int none = p.n_pages << p.page_shift;       // past the pool: loads zeros
        uint8_t* const dst = is_k ? k_ring : v_ring;
        while (ok && walk.next(p, range, g)) {
            const int T = g.t1 - g.t0;
            if (T == 0) continue;
            const int* table = p.pages + static_cast<long long>(g.b) * p.max_pages;
            const int listed = (g.s.kv + (1 << p.page_shift) - 1) >> p.page_shift;
            // a window of 64 entries of the page list, two per lane, moved on by 32 (a tile has at most 16)
            int win = (g.t0 * KT) >> p.page_shift;
            auto entry = [&](int lp) { return lp < listed ? table[lp] : -1; };
            int e0 = entry(win + lane), e1 = entry(win + 32 + lane);
            if (!is_k) {
                ok = segs == 0 || warp_wait(&bar.q_empty, (segs - 1) & 1, abort_flag, status, 0x01000000u);
                if (!ok) break;
                if (lane == 0) {
                    const int row0 = g.s.lo + g.rt * NT * a.rpt;
                    const int n_q = NT == 2 && g.rt * NT * a.rpt + a.rpt < g.s.n ? 2 : 1;  // row tiles with rows
                    mbar_arrive_expect_tx(&bar.q_full, n_q * C::kChunks * a.q_bytes);
                    for (int t = 0; t < n_q; ++t)
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_4d(&tm_q, &bar.q_full, q_smem + t * C::kQBytes + c * 16384, c * 64, 0, g.head,
                                        row0 + t * a.rpt);
                }
                __syncwarp();
                ++n_q_loads;
            }
            for (int i = 0; i < T; ++i, ++place) {
                const int key0 = (g.t0 + i) * KT, first = key0 >> p.page_shift;
                if (first >= win + 32) {
                    win += 32;
                    e0 = e1;
                    e1 = entry(win + 32 + lane);
                }
                const int key = key0 + lane * sub_rows, lp = key >> p.page_shift, at = lp - win;
                const int pg0 = __shfl_sync(0xffffffffu, e0, at & 31), pg1 = __shfl_sync(0xffffffffu, e1, at & 31);
                const int pg = at < 32 ? pg0 : pg1;
                int row = none;
                if (lane < groups && lp < listed) {
                    if (pg >= 0 && pg < p.n_pages)
                        row = (pg << p.page_shift) + (key - (lp << p.page_shift));
                    else
                        cache_report(status, 0x0E000000u | static_cast<unsigned>(lp & 0xFFFFFF));
                }
                const int stage = place % n_stages;
                if (place >= n_stages) {
                    ok = warp_wait(&bar.empty[ring][stage], (place / n_stages - 1) & 1, abort_flag, status, 0x02000000u | i);
                    if (!ok) break;
                }
                if (elect_one()) mbar_arrive_expect_tx(&bar.full[ring][stage], C::kStageBytes);
                __syncwarp();  // the bytes are expected before any box can land
                load_tile<C::kChunks>(map, &bar.full[ring][stage], dst + stage * C::kStageBytes, KT * 128, groups, sub_rows,
                                      g.head, row);
            }
            if (!ok) break;
            ++segs;
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------------- MMAs
        reg_dec<NT>();
        if (elect_one()) {
            constexpr uint32_t id_qk = idesc_bf16_f32(128, KT, false, false);
            constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
            const uint32_t q_lo = sw128_desc_lo(smem_u32(q_smem), 16);
            const uint32_t k_lo = sw128_desc_lo(smem_u32(k_ring), 16);
            const uint32_t v_lo = sw128_desc_lo(smem_u32(v_ring), KT * 128);
            constexpr uint32_t kStageLo = C::kStageBytes >> 4;
            int segs = 0;
            int tiles[2] = {0, 0};  // of each row tile so far: the second may sit out a segment
            bool ok = true;
            // low descriptor words are formed next to their MMAs: hoisted out of the loop they cost more than they save
            auto qk = [&](int t, uint32_t s_col, int stage) {
                uint32_t ql = q_lo + t * (C::kQBytes >> 4), kl = k_lo + stage * kStageLo, ts = tmem + s_col;
                asm volatile("" : "+r"(ql), "+r"(kl), "+r"(ts));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(ts, sw128_desc(ql + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2),
                           sw128_desc(kl + (kk >> 2) * (KT * 128 >> 4) + (kk & 3) * 2), id_qk, kk > 0 ? 1u : 0u);
            };
            // 64 keys of P V, starting at key 16 * k0
            auto pv = [&](uint32_t o_col, uint32_t p_col, int stage, int k0, bool accumulate) {
                uint32_t vl = v_lo + stage * kStageLo + k0 * (2048 >> 4), to = tmem + o_col, tp = tmem + p_col + k0 * 8;
                asm volatile("" : "+r"(vl), "+r"(to), "+r"(tp));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts(to, tp + kk * 8, sw128_desc(vl + kk * (2048 >> 4)), id_pv, (kk > 0 || accumulate) ? 1u : 0u);
            };
            while (ok && walk.next(p, range, g)) {
                const int T = g.t1 - g.t0;
                if (T == 0) continue;
                const bool two = NT == 2 && g.rt * NT * a.rpt + a.rpt < g.s.n;
                ok = mbar_wait(&bar.q_full, segs & 1, abort_flag, status, 0x03000000u);
                tc_fence_after();
                for (int i = 0; ok && i <= T; ++i) {
                    const int kn = tiles[0] + i, vn = kn - 1;  // K tile, V tile: every segment's tiles count for row tile 0
                    const int ks = kn % C::kK, vs = (vn + C::kV) % C::kV;
                    if (NT == 1) {
                        if (i < T) {
                            const int buf = (tiles[0] + i) & 1;
                            if (!(ok = mbar_wait(&bar.full[0][ks], (kn / C::kK) & 1, abort_flag, status, 0x04000000u | i))) break;
                            tc_fence_after();
                            qk(0, buf * 64, ks);
                            mma_commit(&bar.s_full[buf]);
                            mma_commit(&bar.empty[0][ks]);
                            if (i == T - 1) mma_commit(&bar.q_empty);
                        }
                        if (i > 0) {
                            const int n = tiles[0] + i - 1, buf = n & 1;
                            if (!(ok = mbar_wait(&bar.full[1][vs], (vn / C::kV) & 1, abort_flag, status, 0x05000000u | i))) break;
                            if (!(ok = mbar_wait(&bar.p_full[buf], (n >> 1) & 1, abort_flag, status, 0x06000000u | i))) break;
                            tc_fence_after();
                            pv(C::kOCol, buf * 64, vs, 0, i > 1);
                            mma_commit(&bar.empty[1][vs]);
                            mma_commit(&bar.o_done[buf]);
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (!ok) break;
                            const uint32_t col = 256 * t;
                            if (t == 1 && !two) continue;
                            if (i > 0) {
                                const int n = tiles[t] + i - 1;
                                if (t == 0 && !(ok = mbar_wait(&bar.full[1][vs], (vn / C::kV) & 1, abort_flag, status, 0x05000000u | i))) break;
                                // the first half of P V runs under the exponentials of the second
                                if (!(ok = mbar_wait(&bar.p_half[t], n & 1, abort_flag, status, 0x0B000000u | i))) break;
                                tc_fence_after();
                                pv(col + C::kOCol, col, vs, 0, i > 1);
                                if (!(ok = mbar_wait(&bar.p_full[t], n & 1, abort_flag, status, 0x06000000u | i))) break;
                                tc_fence_after();
                                pv(col + C::kOCol, col, vs, 4, true);
                                mma_commit(&bar.o_done[t]);
                                if (t == 1 || !two) mma_commit(&bar.empty[1][vs]);
                            }
                            if (i < T) {
                                if (t == 0 && !(ok = mbar_wait(&bar.full[0][ks], (kn / C::kK) & 1, abort_flag, status, 0x04000000u | i))) break;
                                tc_fence_after();
                                qk(t, col, ks);
                                mma_commit(&bar.s_full[t]);
                            }
                        }
                        if (!ok) break;
                        if (i < T) mma_commit(&bar.empty[0][ks]);
                        if (i == T - 1) mma_commit(&bar.q_empty);
                    }
                }
                tiles[0] += T;
                if (two) tiles[1] += T;
                ++segs;
            }
            mma_commit(&bar.drain);   // every MMA has completed before TMEM is released
            mbar_wait_landing(&bar.drain, 0);
        }
        __syncwarp();
    } else if (warp > kIssuer) {
        reg_dec<NT>();
    } else {
        // ---------------------------------------------------------------- softmax and results
        reg_inc<NT>();
        const int t = warp >> 2, quad = warp & 3, lane_row = quad * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lane_off + (NT == 2 ? 256 * t : 0);
        const uint32_t t_o = t_s + C::kOCol;
        int v_tiles = 0, tiles = 0;  // of the CTA, of this row tile
        bool ok = true;
        while (ok && walk.next(p, range, g)) {
            const int T = g.t1 - g.t0;
            const int tok0 = (g.rt * NT + t) * a.rpt;                    // first token of this row tile
            const int nrows = min(a.rpt, g.s.n - tok0) * p.G;            // its rows (<= 0: none)
            const bool mine = nrows > 0;
            const bool row_ok = lane_row < nrows;
            const int tok = tok0 + lane_row / p.G;
            const int row = g.s.lo + tok, head = g.head * p.G + lane_row % p.G;
            const int ctx = g.s.kv - g.s.n;                              // keys before the new tokens (may be < 0)
            float m_use = -INFINITY, l_sum = 0.f;
            for (int i = 0; mine && i < T; ++i) {
                const int n = tiles + i;
                const int buf = NT == 1 ? n & 1 : 0;
                const uint32_t phase = NT == 1 ? (n >> 1) & 1 : n & 1;
                const uint32_t ts = t_s + buf * 64;
                ok = warp_wait(&bar.s_full[NT == 1 ? buf : t], phase, abort_flag, status, 0x07000000u | i);
                if (!ok) break;
                tc_fence_after();
                const int k0 = (g.t0 + i) * KT;
                float mx = -INFINITY;
                uint32_t sr[KT];
#pragma unroll
                for (int c = 0; c < KT / 32; ++c) tmem_ld32(ts + c * 32, sr + c * 32);
                tmem_wait_ld();
                if (k0 + KT > ctx) {
                    // keys this row sees: a prefix, and under a tree mask the set new tokens after it
                    const int prefix = (tree ? ctx : min(g.s.kv, ctx + tok + 1)) - k0;
                    uint32_t bits[KT / 32];
#pragma unroll
                    for (int w = 0; w < KT / 32; ++w) {
                        const int r = prefix - 32 * w;
                        bits[w] = r >= 32 ? 0xffffffffu : r <= 0 ? 0u : (1u << r) - 1u;
                    }
                    if (tree && row_ok) {
                        const unsigned char* mrow = p.tree_mask + static_cast<long long>(row) * p.mask_cols;
#pragma unroll
                        for (int w = 0; w < KT / 32; ++w) {
                            const int j0 = k0 + 32 * w - ctx;   // new token of the word's first bit
                            const int lo = max(0, -j0), hi = min(32, min(g.s.n, p.mask_cols) - j0);
                            uint32_t add = 0;
                            for (int j = lo; j < hi; ++j)
                                if (mrow[j0 + j]) add |= 1u << j;
                            bits[w] |= add;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < KT; ++c)
                        if (!((bits[c >> 5] >> (c & 31)) & 1u)) sr[c] = 0xff800000u;
                    if (k0 + KT > g.s.kv) {
                        // the rest of the last page: zero rows in the V tile
                        const int vn = v_tiles + i, vs = vn % C::kV;
                        ok = warp_wait(&bar.full[1][vs], (vn / C::kV) & 1, abort_flag, status, 0x08000000u | i);
                        if (!ok) break;
                        const int r0 = max(0, g.s.kv - k0), vecs = (KT - r0) * 8;
                        for (int x = lane_row; x < vecs * C::kChunks; x += 128)
                            *reinterpret_cast<uint4*>(v_ring + vs * C::kStageBytes + x / vecs * (KT * 128) +
                                                      r0 * 128 + x % vecs * 16) = make_uint4(0, 0, 0, 0);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < KT; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        m4[x] = fmax3(m4[x], __uint_as_float(sr[c + 2 * x]), __uint_as_float(sr[c + 2 * x + 1]));
                mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * a.scale_log2;
                if (!row_ok) mx = -INFINITY;
                float alpha = 1.f;
                bool resc = false;
                if (i == 0) {
                    m_use = mx;
                } else if (mx > m_use + kRescaleLog2) {
                    alpha = m_use == -INFINITY ? 0.f : ex2_approx(m_use - mx);
                    m_use = mx;
                    resc = true;
                }
                const float neg = m_use == -INFINITY ? 0.f : -m_use;
                auto rescale = [&]() {
                    if (!__any_sync(0xffffffffu, resc)) return;
                        // O holds the tiles before this one once their P V is done (NT = 2: done when this S was)
                        if (NT == 1) {
                            ok = warp_wait(&bar.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, status, 0x09000000u | i);
                            if (!ok) return;
                            tc_fence_after();
                        }
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t r[32];
                            tmem_ld32(t_o + c * 32, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
                            tmem_st32(t_o + c * 32, r);
                        }
                };
                if (NT == 2) rescale();  // its first half of P goes out before the exponentials are done
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int c0 = 0; c0 < KT; c0 += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float y0, y1;
                        ffma2(y0, y1, __uint_as_float(sr[c0 + 2 * j]), __uint_as_float(sr[c0 + 2 * j + 1]), a.scale_log2,
                              a.scale_log2, neg, neg);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        if (j & 1)
                            fadd2(s2, s3, p0, p1);
                        else
                            fadd2(s0, s1, p0, p1);
                        pk[j] = pack_bf16x2(p0, p1);  // weights in (0, 2^8]: half a bf16 step each, as the output's own
                    }
                    asm volatile(
                        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(ts + c0 / 2),
                        "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]),
                        "r"(pk[8]), "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]), "r"(pk[14]),
                        "r"(pk[15])
                        : "memory");
                    if (NT == 2 && c0 == 32) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&bar.p_half[t]);
                    }
                }
                l_sum = l_sum * alpha + ((s0 + s1) + (s2 + s3));
                if (NT == 1) rescale();
                if (!ok) break;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bar.p_full[NT == 1 ? buf : t]);
            }
            if (!ok) break;
            // result: the whole unit's rows, or a partial
            if (mine && T > 0) {
                const int n = tiles + T - 1;
                ok = warp_wait(&bar.o_done[NT == 1 ? n & 1 : t], (NT == 1 ? n >> 1 : n) & 1, abort_flag, status, 0x0A000000u);
                if (!ok) break;
                tc_fence_after();
            }
            if (mine && quad * 32 < nrows) {  // warps with rows
                const bool whole = g.whole();
                const float inv = !whole ? 1.f : l_sum > 0.f ? 1.f / l_sum : 0.f;
                const int part_row = t * a.rpt * p.G + lane_row;
                const long long slot = static_cast<long long>(partial_slot(g)) * a.slot_rows;
#pragma unroll 1  // runs once or twice a CTA: less code to fetch (64-token trees 118.0 -> 116.7 us)
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    if (T > 0) {
                        tmem_ld32(t_o + c * 32, r);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0;
                    }
                    const float* o = reinterpret_cast<const float*>(r);
                    if (row_ok && whole) {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + (static_cast<long long>(row) * p.Hq + head) * D + c * 32);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[j] = make_uint4(pack_bf16x2(o[8 * j] * inv, o[8 * j + 1] * inv),
                                                pack_bf16x2(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                                pack_bf16x2(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                                                pack_bf16x2(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
                    } else if (row_ok) {
                        float4* dst = reinterpret_cast<float4*>(a.part_o + slot * D) + c * 8 * a.slot_rows + part_row;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j * a.slot_rows] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (row_ok && whole && a.lse)
                    a.lse[static_cast<long long>(head) * p.R + row] = row_lse(m_use, l_sum);
                if (row_ok && !whole) a.stats[slot + part_row] = make_float2(m_use, l_sum);
            }
            if (threadIdx.x == 0 && !g.whole() && g.t0 == 0) {
                const int first = g.rt * row_tile;
                a.jobs[blockIdx.x] = JoinJob{first, min(row_tile, g.s.n * p.G - first), g.s.lo, g.head,
                                             owner_of(range, g.a + C::kOV + g.tiles - 1), {0, 0, 0}};
            }
            tc_fence_before();
            v_tiles += T;
            if (mine) tiles += T;
        }
        tmem_wait_st();  // a tile that was given up half way
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kIssuer) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    // Given up: the CTA's shared memory stays until the copies in flight have landed.  Only here is it known: a role
    // may give up on a copy after its producer has done all of its work.
    if (*abort_flag && (warp == kProducerK || warp == kProducerV)) {
        const int ring = warp - kProducerK, n_stages = ring == 0 ? C::kK : C::kV;
        for (int n = max(0, place - n_stages); n < place; ++n)
            mbar_wait_landing(&bar.full[ring][n % n_stages], (n / n_stages) & 1);
        if (n_q_loads > 0) mbar_wait_landing(&bar.q_full, (n_q_loads - 1) & 1);
    }
}

template <int D, int NT>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const TcParams& a, int ctas,
                   cudaStream_t stream) {
    using C = Cfg<D, NT>;
    static OncePerDevice once;
    const cudaError_t set = once([] {
        cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        // the register increase draws on the launch's registers: with fewer it would wait for ever
        cudaFuncAttributes fa;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, tree_tc_kernel<D, NT>);
        return e == cudaSuccess && NT == 2 && fa.numRegs < kLaunchRegs ? cudaErrorLaunchOutOfResources : e;
    });
    if (set != cudaSuccess) return set;
    return launch_overlapped(tree_tc_kernel<D, NT>, dim3(ctas), C::kThreads, C::kSmem, stream, q, k, v, a);
}

}  // namespace

bool cache_q_map(CUtensorMap* m, const CacheBatch& p, const void* q, int D, int tokens) {
    const unsigned long long d = D, es = 2, G = p.G, Hkv = p.Hkv;
    const unsigned long long dims[4] = {d, G, Hkv, (unsigned long long)(p.R > 0 ? p.R : 1)};
    const unsigned long long strides[3] = {d * es, d * es * G, d * es * G * Hkv};
    const unsigned box[4] = {64, (unsigned)G, 1, (unsigned)tokens};
    return make_map(m, q, dims, strides, box);
}

bool cache_page_map(CUtensorMap* m, const CacheBatch& p, const void* pages, int D, int rows) {
    const unsigned long long d = D, es = 2, Hkv = p.Hkv;
    const unsigned long long all = static_cast<unsigned long long>(p.n_pages) << p.page_shift;
    const unsigned long long dims[4] = {d, Hkv, all, 1};
    const unsigned long long strides[3] = {d * es, d * es * Hkv, d * es * Hkv * all};
    const unsigned page = 1u << p.page_shift;
    const unsigned box[4] = {64, 1, page < (unsigned)rows ? page : (unsigned)rows, 1};
    return make_map(m, pages, dims, strides, box);
}

// Row tiles of a unit: two where a sequence has more than one row tile of rows on average (8 sequences of 8000
// keys: 144 rows 62.5 us in pairs, 95.5 one by one; 96 rows 58.2 and 55.9).
static int tree_tc_nt(int R, int n_seqs, int G) {
    return static_cast<long long>(R) * G > 128ll * n_seqs ? 2 : 1;
}

TreeWs tree_tc_workspace(int R, int n_seqs, int G, int D) {
    const int nt = tree_tc_nt(R, n_seqs, G);
    return tree_workspace(R, G, D, (nt == 1 ? 2 : 1) * device_sm_count(), nt * (128 / G) * G);
}

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream) {
    const int G = a.p.G, nt = tree_tc_nt(a.p.R, a.p.n_seqs, G);
    const TreeWs w = tree_tc_workspace(a.p.R, a.p.n_seqs, G, a.D);
    char* ws = static_cast<char*>(a.ws);
    TcParams t{};
    t.p = a.p;
    t.rpt = 128 / G;
    t.q_bytes = t.rpt * G * 128;
    t.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
    t.out = static_cast<__nv_bfloat16*>(a.out);
    t.lse = a.lse;
    t.jobs = reinterpret_cast<JoinJob*>(ws);
    t.stats = reinterpret_cast<float2*>(ws + w.stat_off);
    t.part_o = reinterpret_cast<float*>(ws + w.o_off);
    t.slot_rows = w.slot_rows;
    CUtensorMap tq, tk, tv;
    const int kt = nt == 1 ? 64 : 128;
    if (!cache_q_map(&tq, a.p, a.q, a.D, t.rpt) || !cache_page_map(&tk, a.p, a.k, a.D, kt) ||
        !cache_page_map(&tv, a.p, a.v, a.D, kt))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (a.D == 128)
        e = nt == 1 ? launch<128, 1>(tq, tk, tv, t, w.ctas, stream) : launch<128, 2>(tq, tk, tv, t, w.ctas, stream);
    else
        e = nt == 1 ? launch<64, 1>(tq, tk, tv, t, w.ctas, stream) : launch<64, 2>(tq, tk, tv, t, w.ctas, stream);
    return e != cudaSuccess ? e : launch_tree_join(a, w, 1, stream);
}

unsigned read_clear_status_cache_tc(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_tc_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_tc_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
