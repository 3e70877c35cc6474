// cache_q8_tc.cu -- attention over an 8-bit paged cache on the tensor cores, few rows (bf16 queries).
//
// The codes go into the MMAs as they lie in the pages (kind::f8f6f4, e4m3): no value of the
// cache is converted.  What is wider than 8 bits is cut into 8-bit parts instead:
//   queries: a row, brought to a largest value in [128, 256) by a power of two, is the sum
//     of two e4m3 parts (4 + 4 of its 8 bits);
//   weights: rounded to fp16, the sum of three e5m2 parts (3 bits each; what a part leaves goes
//     into the next times 2^3, so that small weights keep as many).
// The parts are columns of one MMA, so a K or V tile is read from shared memory once:
//   S^T = K [Q hi; Q lo]^T   128 keys x 2 RT columns, hi and lo of a row in one lane;
//   O^T += V^T [P1; P2; P3]^T   D x 3 RT columns, added up when a unit is done.
// A TMEM lane, and so a thread, is a key: its scales are one product per thread and row, the
// scores of RT = 8 or 16 rows cost 2 RT columns instead of a 128-row tile that is mostly empty
// (decode has 1 to 16 rows per KV head), and few exponentials are computed for rows that are
// not there.  The price is the maximum over keys, across lanes: a tile only asks whether some
// weight passed its row's reference by 2^5, or what goes into P 2^15 (one barrier that ORs a bit); the
// maxima are taken, and O and the sums scaled, where one did, and in a unit's first tile.
//
// A row has two references: of its scores, for the sum of its weights (kept in fp32), and of its scores plus the exponents
// of the V scales, for what goes into P, so that a key of large weight and small value (or a hidden one of any value) takes
// no bits from the others.  P holds a weight times its V scale over 2^reference times 2^10: at most 2^15 (e5m2 holds
// 57344), off by half a step of the last part, 2^-16 2^-6, or 2^-9 and fp16's 2^-11 of itself, less than a weight rounded to
// bf16: what n keys of little weight add up to is off by n 2^-32 of the row's largest product at most.
//
// The cache's bytes bound it.  32 sequences of 4K-16K keys, one token each, 64 / 8 heads, D = 128: 107
// to 109 us, 6.3 TB/s (0.94 of the measured copy rate), 204 us and more in 16 bits; D = 64: 72, 4.7 TB/s: the softmax
// warps' way through a tile takes as long (each instruction more shows; a third CTA per SM changed nothing).  Short calls
// wait: one token over 1000 keys takes 9.7 us for 2 MB (the prelude, the queries, a tile or two and the join).  The row's
// own reference for P costs 0.1 to 3 us of these (D = 64: 68.8 with one V scale for all rows of a unit).  Units of 32 rows
// took as long for 32 rows per head as the kernel for many rows and longer for 64 (72 us against 63, both before the rows
// had references of their own).
//
// Roles: four softmax warps, a warp each that streams K pages (and the scales of K and V) and
// V pages into a ring of its own, one that issues the MMAs; two CTAs per SM.
#include <cmath>

#include "cache_q8_mma.cuh"

namespace ra {

static __device__ unsigned g_cache_q8_tc_status[2];

namespace {

constexpr float kSlackLog2 = 5.0f;   // a weight is at most 2^5 times its row's reference ...
constexpr float kWeightLog2 = 10.f;  // ... and goes into P, with its value's scale, times 2^10 over O's reference
constexpr float kLeastB = -64.f;     // O's reference is no further below that of the scores: nothing of such products is left
constexpr int KT = 128;              // keys of a tile
constexpr int kOV = 3;               // weight of a unit beyond its tiles (with 2, 8 x 2 tokens over up to 16K keys take 42 us, not 41)
constexpr int kMinW = 1;             // least weight per CTA (one token over 1000 keys: 9.5 us; 9.9 with 2, 10.6 with 3)
constexpr int kThreads = 128 + 96;   // softmax; K producer, V producer, issuer
constexpr int kPitch = 64;           // bytes of a key in P: 3 RT and its padding

// RT: rows of a unit, 16 or 8 (half the scores, exponentials and parts; three parts of 8 rows fill 32 columns of P V).
template <int D, int RT>
struct Cfg {
    static constexpr int kPCols = (3 * RT + 15) / 16 * 16;  // columns of P V, a multiple of 16: the rest are zeros
    static constexpr int kOCol = 4 * RT;                // O columns, behind two S buffers of 2 RT
    static constexpr int kTmemCols = 8 * RT;
    static_assert(kPCols <= kPitch && kOCol + kPCols <= kTmemCols, "P's rows, tensor memory");
    static constexpr int kQBytes = 2 * RT * D;
    static constexpr int kPBytes = KT * kPitch;
    static constexpr int kStageBytes = KT * D;
    static constexpr int kHead = 4096;                  // barriers, scales and statistics ahead of the tiles
    static constexpr int kFit = (113 * 1024 - kHead - kQBytes - 2 * kPBytes) / kStageBytes;
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr int kV = kStages / 2, kK = kStages - kV;
    static constexpr int kSmem = kHead + kQBytes + 2 * kPBytes + kStages * kStageBytes;
    static_assert(kV >= 2, "stages");
};

struct Bars {
    uint64_t full[2][5], empty[2][5];  // stages of the K ring and the V ring
    uint64_t q_full;
    uint64_t s_full[2], p_full[2], o_done[2];  // by S and P buffer
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// What the softmax warps tell one another.
template <int RT>
struct Soft {
    float4 row[RT / 2];    // of two rows: scales of their scores (the inverse of their queries' power of two), minus their references
    alignas(16) int into_p[RT];  // kWeightLog2 less what O's reference is beyond that of the scores, + 127
    alignas(16) float alpha[RT], beta[RT];  // what the rows' sums and O are scaled by
    float warp[4][RT];     // maxima of the scores, and at the end the sums
    float warp_o[4][RT];   // maxima of the scores plus V's exponents
};

template <int RT>
struct Head {
    Bars bar;
    alignas(16) unsigned char scales[5][2][KT];  // of a K stage's keys: K's, V's
    alignas(16) Soft<RT> soft;
};

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    if (N == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[N - 8]),
              "=r"(u[N - 7]), "=r"(u[N - 6]), "=r"(u[N - 5]), "=r"(u[N - 4]), "=r"(u[N - 3]), "=r"(u[N - 2]), "=r"(u[N - 1])
            : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float* r) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    if (N == 16)
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
            "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[N - 8]), "r"(u[N - 7]),
            "r"(u[N - 6]), "r"(u[N - 5]), "r"(u[N - 4]), "r"(u[N - 3]), "r"(u[N - 2]), "r"(u[N - 1])
            : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(u[0]), "r"(u[1]),
                     "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
}

// The 128 softmax threads: whether one of them says so.  Every one comes here the same number of times, also one that
// gave up a wait: the others learn of it here, and all leave together.
__device__ __forceinline__ bool group_any(bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(mine ? 1u : 0u)
        : "memory");
    return any != 0;
}

// v[r] of all lanes put together by op, row lane % RT in each lane: every step halves the rows a lane keeps.
template <int RT, class Op>
__device__ __forceinline__ float over_lanes(float (&v)[RT], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = RT / 2; half > 0; half >>= 1) {
        const bool upper = lane & half;
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const float keep = upper ? v[j + half] : v[j], send = upper ? v[j] : v[j + half];
            v[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, half));
        }
    }
#pragma unroll
    for (int other = RT; other < 32; other <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], other));
    return v[0];
}

// 2^(a + b - 127), as far as a float goes: 0 below, 2^127 above.
__device__ __forceinline__ float power_of_two(int a, int b) {
    return scale_of(static_cast<unsigned>(__viaddmin_s32_relu(a, b, 254)));
}

struct Larger {
    __device__ __forceinline__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
// The largest of row r over the four warps.
template <int RT>
__device__ __forceinline__ float largest_of(const float (&w)[4][RT], int r) {
    return fmaxf(fmaxf(w[0][r], w[1][r]), fmaxf(w[2][r], w[3][r]));
}

// Four weights as the bytes of three e5m2 parts, the second times 2^3 and the third times 2^6.  An e5m2 is the upper byte
// of an fp16: a part is what lies there, cut off; what is left after it is below 2^12 for weights up to 2^15, exact in fp16,
// also times 2^3.  The last is rounded to the nearest (weights are not negative).
__device__ __forceinline__ void weight_parts(uint32_t h0, uint32_t h1, uint32_t (&part)[3]) {
    uint32_t h[2] = {h0, h1};
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        if (t == 2) {
            h[0] += 0x00800080u;
            h[1] += 0x00800080u;
        }
        part[t] = __byte_perm(h[0], h[1], 0x7531);
        if (t < 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(h[i] & 0xff00ff00u));
                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(0x48004800u));  // 8
            }
        }
    }
}

// A row's value in four lanes' registers -> four dims of one of four rows in each: lane l holds v[j] = row j at dim l, and
// gets row l % 4 at dims l - l % 4 ... + 3.
__device__ __forceinline__ float4 four_dims(const float* v, int lane) {
    const bool b0 = lane & 1, b1 = lane & 2;
    const float a = __shfl_xor_sync(0xffffffffu, b0 ? v[0] : v[1], 1), b = __shfl_xor_sync(0xffffffffu, b0 ? v[2] : v[3], 1);
    const float p0 = b0 ? a : v[0], p1 = b0 ? v[1] : a;  // row b0, two dims
    const float q0 = b0 ? b : v[2], q1 = b0 ? v[3] : b;  // row 2 + b0
    const float s0 = __shfl_xor_sync(0xffffffffu, b1 ? p0 : q0, 2), s1 = __shfl_xor_sync(0xffffffffu, b1 ? p1 : q1, 2);
    return b1 ? make_float4(s0, s1, q0, q1) : make_float4(p0, p1, s0, s1);
}

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, 2)
    q8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ Q8Params a) {
    using C = Cfg<D, RT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    using Shared = Head<RT>;
    Shared& head = *reinterpret_cast<Shared*>(smem);
    Bars& bar = head.bar;
    RangeScratch<kThreads>& scratch = *reinterpret_cast<RangeScratch<kThreads>*>(smem + C::kHead - 512);
    static_assert(sizeof(Shared) <= C::kHead - 512 && sizeof(RangeScratch<kThreads>) <= 512, "head of the shared memory");
    uint8_t* q_smem = smem + C::kHead;
    uint8_t* p_smem = q_smem + C::kQBytes;
    uint8_t* k_ring = p_smem + 2 * C::kPBytes;
    uint8_t* v_ring = k_ring + C::kK * C::kStageBytes;
    static_assert(C::kHead % 1024 == 0 && C::kQBytes % 1024 == 0 && C::kPBytes % 1024 == 0 && C::kStageBytes % 1024 == 0,
                  "swizzled tiles start on 1024 bytes");
    const CacheBatch& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* status = g_cache_q8_tc_status;
    const bool tree = p.tree_mask != nullptr;
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) cache_report(status, 0x0C000000u);
        return;
    }

    constexpr int kProducerK = 4, kProducerV = kProducerK + 1, kIssuer = kProducerK + 2;
    if (warp == kIssuer) {
        if (lane == 0) {
            for (int s = 0; s < 5; ++s) {
                mbar_init(&bar.full[0][s], 1 + 32);           // the tile's bytes, and every lane's scales
                mbar_init(&bar.full[1][s], 1);
                mbar_init(&bar.empty[0][s], 1 + 4);           // the MMAs, and every warp that reads the scales
                mbar_init(&bar.empty[1][s], 1);
            }
            mbar_init(&bar.q_full, 128);
            for (int t = 0; t < 2; ++t) {
                mbar_init(&bar.s_full[t], 1);
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
    if (warp == kProducerV && lane == 0) tma_prefetch_desc(&tm_v);
    grid_dependency_wait();    // nothing above reads or writes global memory
    grid_launch_dependents();  // the join may take its place on the SMs; it waits for this grid's end
    const Column col = column_of(a.columns);
    if (threadIdx.x == 0) a.jobs[col.cta].rows = 0;
    tc_fence_before();
    const WorkRange& range = find_range<kThreads>(p, kMinW, status, TreeWeight<KT, kOV>{p.G, a.heads, tree, RT}, scratch,
                                                     col.range, col.ranges);
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    volatile int* abort_flag = &bar.abort;
    SegmentWalk<KT, kOV> walk;
    walk.start(p, range, RT, a.heads, col.index * a.heads);
    Segment g;
    int place = 0;  // tiles a producer has loaded so far

    if (warp == kProducerK || warp == kProducerV) {
        // ---------------------------------------------------------------- pages -> shared memory
        const bool is_k = warp == kProducerK;
        const CUtensorMap* map = is_k ? &tm_k : &tm_v;
        const int ring = is_k ? 0 : 1, n_stages = is_k ? C::kK : C::kV;
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
            auto page_of = [&](int lp) {  // whole warp
                const int at = lp - win;
                const int pg0 = __shfl_sync(0xffffffffu, e0, at & 31), pg1 = __shfl_sync(0xffffffffu, e1, at & 31);
                return lp >= listed ? -1 : at < 32 ? pg0 : pg1;
            };
            for (int i = 0; i < T; ++i, ++place) {
                const int key0 = (g.t0 + i) * KT, first = key0 >> p.page_shift;
                if (first >= win + 32) {
                    win += 32;
                    e0 = e1;
                    e1 = entry(win + 32 + lane);
                }
                const int key = key0 + min(lane, groups - 1) * sub_rows, lp = key >> p.page_shift, pg = page_of(lp);
                int row = none;
                if (lane < groups && lp < listed) {
                    if (pg >= 0 && pg < p.n_pages)
                        row = (pg << p.page_shift) + (key - (lp << p.page_shift));
                    else
                        cache_report(status, 0x0E000000u | static_cast<unsigned>(lp & 0xFFFFFF));
                }
                const int key4 = key0 + 4 * lane, lp4 = key4 >> p.page_shift, pg4 = page_of(lp4);
                const int stage = place % n_stages;
                if (place >= n_stages) {
                    ok = warp_wait(&bar.empty[ring][stage], (place / n_stages - 1) & 1, abort_flag, status, 0x02000000u | i);
                    if (!ok) break;
                }
                if (elect_one()) mbar_arrive_expect_tx(&bar.full[ring][stage], C::kStageBytes);
                __syncwarp();  // the bytes are expected before any box can land
                if (lane < groups)
                    tma_load_4d(map, &bar.full[ring][stage], dst + stage * C::kStageBytes + lane * sub_rows * D, 0, g.head, row, 0);
                if (is_k) {
                    const bool have = pg4 >= 0 && pg4 < p.n_pages;
                    const long long at = have ? ((static_cast<long long>(pg4) * p.Hkv + g.head) << p.page_shift) +
                                                    (key4 - (lp4 << p.page_shift))
                                              : 0;
                    copy_scales4(&head.scales[stage][0][4 * lane], a.ks + at, have);
                    copy_scales4(&head.scales[stage][1][4 * lane], a.vs + at, have);
                    copies_arrive(&bar.full[0][stage]);
                }
            }
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------------- MMAs
        if (elect_one()) {
            constexpr uint32_t id_qk = idesc8(2 * RT, false, false);
            constexpr uint32_t id_pv = idesc8(C::kPCols, true, true);
            constexpr uint32_t hi = desc_hi(D), p_hi = desc_hi(kPitch);
            constexpr uint32_t kStageLo = C::kStageBytes >> 4;
            const uint32_t q_lo = sw128_desc_lo(smem_u32(q_smem), 16);
            const uint32_t k_lo = sw128_desc_lo(smem_u32(k_ring), 16);
            // D = 64: the rows of O^T past 64 repeat the first 64 (a stride of 0) and are not read
            const uint32_t v_lo = sw128_desc_lo(smem_u32(v_ring), 0);
            const uint32_t p_lo = sw128_desc_lo(smem_u32(p_smem), KT * kPitch);
            int segs = 0, tiles = 0;
            bool ok = true;
            while (ok && walk.next(p, range, g)) {
                const int T = g.t1 - g.t0;
                if (T == 0) continue;
                ok = mbar_wait(&bar.q_full, segs & 1, abort_flag, status, 0x03000000u);
                tc_fence_after();
                for (int i = 0; ok && i <= T; ++i) {
                    if (i < T) {
                        const int n = tiles + i, buf = n & 1, ks = n % C::kK;
                        if (!(ok = mbar_wait(&bar.full[0][ks], (n / C::kK) & 1, abort_flag, status, 0x04000000u | i))) break;
                        tc_fence_after();
                        uint32_t kl = k_lo + ks * kStageLo, ts = tmem + buf * 2 * RT;
                        asm volatile("" : "+r"(kl), "+r"(ts));
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            mma8(ts, desc8(hi, kl + kk * 2), desc8(hi, q_lo + kk * 2), id_qk, kk > 0 ? 1u : 0u);
                        mma_commit(&bar.s_full[buf]);
                        mma_commit(&bar.empty[0][ks]);
                    }
                    if (i > 0) {
                        const int n = tiles + i - 1, buf = n & 1, vs = n % C::kV;
                        if (!(ok = mbar_wait(&bar.full[1][vs], (n / C::kV) & 1, abort_flag, status, 0x05000000u | i))) break;
                        if (!(ok = mbar_wait(&bar.p_full[buf], (n >> 1) & 1, abort_flag, status, 0x06000000u | i))) break;
                        tc_fence_after();
                        uint32_t vl = v_lo + vs * kStageLo, pl = p_lo + buf * (C::kPBytes >> 4), to = tmem + C::kOCol;
                        asm volatile("" : "+r"(vl), "+r"(pl), "+r"(to));
#pragma unroll
                        for (int kk = 0; kk < KT / 32; ++kk)
                            mma8(to, desc8(hi, vl + kk * (32 * D >> 4)), desc8(p_hi, pl + kk * (32 * kPitch >> 4)), id_pv,
                                 (kk > 0 || i > 1) ? 1u : 0u);
                        mma_commit(&bar.empty[1][vs]);
                        mma_commit(&bar.o_done[buf]);
                    }
                }
                tiles += T;
                ++segs;
            }
            mma_commit(&bar.drain);  // every MMA has completed before TMEM is released
            mbar_wait_landing(&bar.drain, 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax and results
        const int quad = warp, lane_row = quad * 32 + lane;  // its key of a tile; its dim of O
        const int r_own = lane % RT;                          // row whose statistics the lane keeps
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_o = tmem + lane_off + C::kOCol;
        Soft<RT>& soft = head.soft;
        int tiles = 0;
        bool dead = false;  // gave up a wait
        auto wait = [&](uint64_t* b, uint32_t parity, unsigned where) {
            if (!dead && !warp_wait(b, parity, abort_flag, status, where)) dead = true;
        };
        while (!dead && walk.next(p, range, g)) {
            const int T = g.t1 - g.t0;
            const int fr0 = g.rt * RT, nrows = min(RT, g.s.n * p.G - fr0);  // its rows
            const bool whole = g.whole();
            const int ctx = g.s.kv - g.s.n;                        // keys before the new tokens (may be < 0)
            if (T > 0) {
                // ---- queries of its rows (the last row again past the end) as two e4m3 parts
                constexpr int kLanes = 128 / RT, kEach = D / kLanes;  // threads of a row, dims of a thread
                const int r = lane_row / kLanes, d0 = lane_row % kLanes * kEach;
                const int fr = min(fr0 + r, g.s.n * p.G - 1);
                const __nv_bfloat16* src =
                    a.q + (static_cast<long long>(g.s.lo + fr / p.G) * p.Hq + g.head * p.G + fr % p.G) * D + d0;
                float x[kEach];
                uint32_t most = 0;
#pragma unroll
                for (int c = 0; c < kEach; c += 8) {
                    if (kEach >= 8) {
                        load8(src + c, x + c);
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(src);
                        x[0] = __uint_as_float(w.x << 16);
                        x[1] = __uint_as_float(w.x & 0xffff0000u);
                        x[2] = __uint_as_float(w.y << 16);
                        x[3] = __uint_as_float(w.y & 0xffff0000u);
                    }
                }
#pragma unroll
                for (int c = 0; c < kEach; ++c) most = max(most, __float_as_uint(x[c]) & 0x7fffffffu);
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                const int up = query_scale_byte(most);
                const float f = scale_of(up);
#pragma unroll
                for (int c = 0; c < kEach; c += 4) {
                    uint32_t hi, lo;
                    query_parts4(x + c, f, hi, lo);
                    const int at = (d0 + c) & 15;
                    *reinterpret_cast<uint32_t*>(q_smem + piece_at<D>(r, (d0 + c) >> 4) + at) = hi;
                    *reinterpret_cast<uint32_t*>(q_smem + piece_at<D>(RT + r, (d0 + c) >> 4) + at) = lo;
                }
                // a row with a NaN or an infinity has no scores
                if (d0 == 0) reinterpret_cast<float*>(&soft.row[r / 2])[r & 1] = most >= 0x7f800000u ? NAN : scale_of(254 - up);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(&bar.q_full);
            }
            group_any(false);  // the rows' scales are there; everyone is done with the segment before
            float m_own = -INFINITY;  // reference of row r_own's scores
            float b_own = kLeastB;    // what O's is beyond it
            float l[RT];
#pragma unroll
            for (int j = 0; j < RT; ++j) l[j] = 0.f;
            bool out = false;         // the group leaves
            for (int i = 0; i < T; ++i) {
                const int n = tiles + i, buf = n & 1, ks = n % C::kK;
                const int key = (g.t0 + i) * KT + lane_row;
                wait(&bar.full[0][ks], (n / C::kK) & 1, 0x07000000u | i);
                const unsigned ek = head.scales[ks][0][lane_row];
                unsigned ev = head.scales[ks][1][lane_row];
                __syncwarp();
                if (!dead && lane == 0) mbar_arrive(&bar.empty[0][ks]);
                if (key >= g.s.kv) ev = 0;
                const float sc = scale_of(ek) * a.scale_log2;
                // rows that see the key
                uint32_t bits = 0xffffffffu;
                const bool masked = (g.t0 + i + 1) * KT > ctx;
                if (masked) {
                    const int jn = key - ctx;  // which new token it is
                    if (key >= g.s.kv) {
                        bits = 0;
                    } else if (jn >= 0 && !tree) {
                        const int first = jn * p.G - fr0;
                        bits = first <= 0 ? 0xffffffffu : first >= RT ? 0u : 0xffffffffu << first;
                    } else if (jn >= 0) {
                        bits = 0;
                        if (jn < p.mask_cols) {
                            const int t1 = min(g.s.n - 1, (fr0 + RT - 1) / p.G);
                            const unsigned char* seen = p.tree_mask + static_cast<long long>(g.s.lo) * p.mask_cols + jn;
#pragma unroll 4
                            for (int t = fr0 / p.G; t <= t1; ++t) {
                                const int lo = max(0, t * p.G - fr0), len = min(RT, (t + 1) * p.G - fr0) - lo;
                                if (seen[static_cast<long long>(t) * p.mask_cols]) bits |= ((1u << len) - 1u) << lo;
                            }
                        }
                    }
                }
                const int ev2 = ev ? static_cast<int>(ev) : -0x10000;  // nothing of a key without a scale
                wait(&bar.s_full[buf], (n >> 1) & 1, 0x08000000u | i);
                tc_fence_after();
                float z[RT];
                // scores in log2 units, less the rows' references if `less`
                auto scores = [&](bool less) {
                    if (dead) return;
                    float lo[RT];
                    const uint32_t ts = tmem + lane_off + buf * 2 * RT;
                    tmem_ld<RT>(ts, z);
                    tmem_ld<RT>(ts + RT, lo);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < RT; j += 2) {
                        const float4 row = soft.row[j / 2];
                        fadd2(z[j], z[j + 1], lo[j], lo[j + 1]);
                        fmul2(z[j], z[j + 1], z[j], z[j + 1], row.x, row.y);
                        ffma2(z[j], z[j + 1], z[j], z[j + 1], sc, sc, less ? row.z : 0.f, less ? row.w : 0.f);
                    }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < RT; ++j)
                            if (!(bits >> j & 1u)) z[j] = -INFINITY;
                    }
                };
                // from the scores: the weights, and as fp16 what goes into P, 2^(V's exponent - O's reference + kWeightLog2)
                // times as much
                float w[RT];
                uint32_t h[RT / 2];
                auto weigh = [&]() {
#pragma unroll
                    for (int j = 0; j < RT; j += 4) {
                        const int4 c = *reinterpret_cast<const int4*>(&soft.into_p[j]);
                        const float f[4] = {power_of_two(ev2, c.x), power_of_two(ev2, c.y), power_of_two(ev2, c.z), power_of_two(ev2, c.w)};
#pragma unroll
                        for (int x = 0; x < 4; x += 2) {
                            float y0, y1;
                            w[j + x] = ex2_approx(z[j + x]);
                            w[j + x + 1] = ex2_approx(z[j + x + 1]);
                            fmul2(y0, y1, w[j + x], w[j + x + 1], f[x], f[x + 1]);
                            asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h[(j + x) / 2]) : "f"(y0), "f"(y1));
                        }
                    }
                };
                bool high = i == 0;
                if (i > 0) {
                    scores(true);
                    weigh();
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < RT; j += 2) top = fmax3(top, z[j], z[j + 1]);
                    static_assert(kSlackLog2 + kWeightLog2 == 15.f, "0x7800 is 2^15 in fp16");
                    uint32_t most = h[0];
#pragma unroll
                    for (int j = 1; j < RT / 2; ++j) asm("max.f16x2 %0, %0, %1;" : "+r"(most) : "r"(h[j]));
                    const bool above = top > kSlackLog2 || max(most & 0xffffu, most >> 16) > 0x7800u;
                    high = group_any(dead || above);
                }
                if (high) {
                    // new references: the rows' maxima over the tile's keys
                    if (group_any(dead)) {
                        out = true;
                        break;
                    }
                    scores(false);
                    float v[RT];
#pragma unroll
                    for (int j = 0; j < RT; ++j) v[j] = ev ? z[j] + static_cast<float>(ev) : -INFINITY;
                    const float top = over_lanes(z, Larger()), top_o = over_lanes(v, Larger());
                    if (lane < RT) {
                        soft.warp[quad][lane] = top;
                        soft.warp_o[quad][lane] = top_o;
                    }
                    group_any(false);
                    const float m_new = fmaxf(m_own, largest_of(soft.warp, r_own));
                    // whole numbers, so that O's unit is exact; a NaN (nothing seen so far) is passed over
                    const float b_new = fmaxf(fmaxf(ceilf(largest_of(soft.warp_o, r_own) - m_new), ceilf(b_own - (m_new - m_own))), kLeastB);
                    const float moved = m_own - m_new, alpha = m_own == -INFINITY ? 0.f : ex2_approx(moved);
                    const float beta = m_own == -INFINITY ? 0.f : ex2_approx(moved + (b_own - b_new));
                    m_own = m_new;
                    b_own = b_new;
                    if (quad == 0 && lane < RT) {
                        reinterpret_cast<float*>(&soft.row[lane / 2])[2 + (lane & 1)] = -m_new;  // none so far: +inf, so that the row's first score is above it
                        soft.alpha[lane] = alpha;
                        soft.beta[lane] = beta;
                        soft.into_p[lane] = static_cast<int>(kWeightLog2 - b_new) + 127;
                    }
                    group_any(false);
                    if (i > 0) {
                        wait(&bar.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, 0x09000000u | i);
                        tc_fence_after();
                        float f[RT];
#pragma unroll
                        for (int j = 0; j < RT; j += 4) {
                            *reinterpret_cast<float4*>(f + j) = *reinterpret_cast<const float4*>(&soft.alpha[j]);
#pragma unroll
                            for (int h = j; h < j + 4; ++h) l[h] *= f[h];
                            *reinterpret_cast<float4*>(f + j) = *reinterpret_cast<const float4*>(&soft.beta[j]);
                        }
                        if (!dead) {
#pragma unroll 1
                            for (int t = 0; t < 3; ++t) {
                                float o[RT];
                                tmem_ld<RT>(t_o + t * RT, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < RT; ++j) o[j] *= f[j];
                                tmem_st<RT>(t_o + t * RT, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    scores(true);
                    weigh();
                }
                // weights, their sum, and their parts in the key's row of P
                if (n >= 2) wait(&bar.o_done[buf], ((n - 2) >> 1) & 1, 0x0A000000u | i);
                if (!dead) {
                    uint32_t word[3][RT / 4];
#pragma unroll
                    for (int j = 0; j < RT; j += 4) {
                        uint32_t part[3];
                        fadd2(l[j], l[j + 1], w[j], w[j + 1]);
                        fadd2(l[j + 2], l[j + 3], w[j + 2], w[j + 3]);
                        weight_parts(h[j / 2], h[j / 2 + 1], part);
#pragma unroll
                        for (int t = 0; t < 3; ++t) word[t][j / 4] = part[t];
                    }
                    uint8_t* dst = p_smem + buf * C::kPBytes;
                    if (RT == 16) {
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            *reinterpret_cast<uint4*>(dst + piece_at<kPitch>(lane_row, t)) =
                                make_uint4(word[t][0], word[t][1], word[t][RT / 4 - 2], word[t][RT / 4 - 1]);
                    } else {
                        *reinterpret_cast<uint4*>(dst + piece_at<kPitch>(lane_row, 0)) =
                            make_uint4(word[0][0], word[0][1], word[1][0], word[1][1]);
                        *reinterpret_cast<uint4*>(dst + piece_at<kPitch>(lane_row, 1)) = make_uint4(word[2][0], word[2][1], 0, 0);
                    }
                    if ((g.t0 + i + 1) * KT > g.s.kv) {
                        // the rest of the last page: zero rows in the V tile (0 times a NaN code is NaN)
                        const int vs = n % C::kV;
                        wait(&bar.full[1][vs], (n / C::kV) & 1, 0x0B000000u | i);
                        if (!dead && key >= g.s.kv) {
#pragma unroll
                            for (int c = 0; c < D; c += 16)
                                *reinterpret_cast<uint4*>(v_ring + vs * C::kStageBytes + lane_row * D + c) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_fence_before();
                    mbar_arrive(&bar.p_full[buf]);
                }
            }
            // ---- result: the whole unit's rows, or a partial
            if (out) break;
            const int n = tiles + T - 1;
            if (T > 0) wait(&bar.o_done[n & 1], (n >> 1) & 1, 0x0D000000u);
            const float l_warp = over_lanes(l, [](float x, float y) { return x + y; });
            if (lane < RT) soft.warp[quad][lane] = l_warp;
            if (group_any(dead)) break;
            tc_fence_after();
            const long long slot = static_cast<long long>(partial_slot(g, col.cta)) * a.slot_rows;
            const int d4 = lane_row / 4;
            if (quad * 32 < D) {  // warps with dims of O
                float o[RT];
                if (T > 0) {
                    float o1[RT], o2[RT];
                    tmem_ld<RT>(t_o, o);
                    tmem_ld<RT>(t_o + RT, o1);
                    tmem_ld<RT>(t_o + 2 * RT, o2);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < RT; ++j) o[j] = fmaf(o1[j], 0.125f, fmaf(o2[j], 1.f / 64, o[j]));
                } else {
#pragma unroll
                    for (int j = 0; j < RT; ++j) o[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < RT; j += 4) {
                    float4 v = four_dims(o + j, lane);
                    const int rr = j + (lane & 3);
                    if (rr >= nrows) continue;
                    const float sum = (soft.warp[0][rr] + soft.warp[1][rr]) + (soft.warp[2][rr] + soft.warp[3][rr]);
                    // O's unit in two powers of two: it may lie below what a float holds
                    const int unit = T > 0 ? -soft.into_p[rr] : 0, half = unit / 2;
                    const float up = scale_of(static_cast<unsigned>(127 + half)), up2 = scale_of(static_cast<unsigned>(127 + unit - half));
                    // a row with a NaN keeps it, one that saw no key gets zeros
                    const float f = !whole ? up2 : sum > 0.f ? up2 / sum : sum == 0.f ? 0.f : NAN;
                    v = make_float4(v.x * up * f, v.y * up * f, v.z * up * f, v.w * up * f);
                    const int fr = fr0 + rr;
                    if (whole)
                        store4(a.out + (static_cast<long long>(g.s.lo + fr / p.G) * p.Hq + g.head * p.G + fr % p.G) * D + 4 * d4, v);
                    else
                        reinterpret_cast<float4*>(a.part_o + slot * D)[d4 * a.slot_rows + rr] = v;
                }
            }
            if (quad == 0 && lane < RT && lane < nrows) {
                const float sum = (soft.warp[0][lane] + soft.warp[1][lane]) + (soft.warp[2][lane] + soft.warp[3][lane]);
                const int fr = fr0 + lane;
                if (!whole)
                    a.stats[slot + lane] = make_float2(m_own, sum);
                else if (a.lse)
                    a.lse[static_cast<long long>(g.head * p.G + fr % p.G) * p.R + g.s.lo + fr / p.G] = row_lse(m_own, sum);
            }
            if (threadIdx.x == 0 && !whole && g.t0 == 0) {
                const int first = g.rt * RT;
                a.jobs[col.cta] = JoinJob{first, min(RT, g.s.n * p.G - first), g.s.lo, g.head,
                                             col.index * col.ranges + owner_of(range, g.a + kOV + g.tiles - 1), {0, 0, 0}};
            }
            tc_fence_before();
            tiles += T;
        }
        tmem_wait_st();
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
    }
}

template <int D, int RT>
cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const Q8Params& a, int ctas, cudaStream_t stream) {
    using C = Cfg<D, RT>;
    static OncePerDevice once;
    const cudaError_t set =
        once([] { return cudaFuncSetAttribute(q8_tc_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    if (set != cudaSuccess) return set;
    return launch_overlapped(q8_tc_kernel<D, RT>, dim3(ctas), kThreads, C::kSmem, stream, k, v, a);
}

// How a call is cut up: rows of a unit (8 and 16 here; 128 and 256 in cache_q8_wide.cu), columns of KV heads, and CTAs.  By
// the mean number of rows of a sequence and KV head, all the host knows.  8 rows: 32 sequences of 4K-16K keys take 109 us
// in units of 8 and 115 in units of 16, with D = 64 68 and 85.  16 rows: 8 sequences of up to 16000 keys take 41 us here and 62
// with units of 128 rows; 32 rows: 66 here (in units of 32, with twice the warps) and 62 there.
struct Cut {
    int rt, columns, heads, ctas;
};
Cut cut_of(int R, int n_seqs, int G, int Hkv) {
    const long long rows = static_cast<long long>(R) * G;  // of a KV head, over the batch
    Cut c;
    c.rt = rows <= 8ll * n_seqs ? 8 : rows <= 16ll * n_seqs ? 16 : rows <= 128ll * n_seqs ? 128 : 256;
    const int most = (c.rt == 256 ? 1 : 2) * device_sm_count();
    c.heads = (Hkv + most - 1) / most;
    c.columns = (Hkv + c.heads - 1) / c.heads;
    c.ctas = most / c.columns * c.columns;
    return c;
}

}  // namespace

TreeWs tree_q8_tc_workspace(int R, int n_seqs, int G, int Hkv, int D) {
    const Cut cut = cut_of(R, n_seqs, G, Hkv);
    return tree_workspace(R, G, D, cut.ctas, cut.rt);
}

cudaError_t launch_tree_q8_tc(const TreeArgs& a, const Q8Pools& pools, cudaStream_t stream) {
    const Cut cut = cut_of(a.p.R, a.p.n_seqs, a.p.G, a.p.Hkv);
    const int rt = cut.rt;
    const TreeWs w = tree_q8_tc_workspace(a.p.R, a.p.n_seqs, a.p.G, a.p.Hkv, a.D);
    char* ws = static_cast<char*>(a.ws);
    Q8Params t{};
    t.p = a.p;
    t.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
    t.q = static_cast<const __nv_bfloat16*>(a.q);
    t.ks = pools.ks;
    t.vs = pools.vs;
    t.out = static_cast<__nv_bfloat16*>(a.out);
    t.lse = a.lse;
    t.jobs = reinterpret_cast<JoinJob*>(ws);
    t.stats = reinterpret_cast<float2*>(ws + w.stat_off);
    t.part_o = reinterpret_cast<float*>(ws + w.o_off);
    t.slot_rows = w.slot_rows;
    t.columns = cut.columns;
    t.heads = cut.heads;
    // boxes of a page, at most a tile's rows of one KV head
    const unsigned long long d = a.D, Hkv = a.p.Hkv, all = static_cast<unsigned long long>(a.p.n_pages) << a.p.page_shift;
    const unsigned long long dims[4] = {d, Hkv, all, 1}, strides[3] = {d, d * Hkv, d * Hkv * all};
    const unsigned kt = rt <= 16 ? KT : q8_wide_key_tile(rt / 128), page = 1u << a.p.page_shift;
    const unsigned box[4] = {static_cast<unsigned>(a.D), 1, page < kt ? page : kt, 1};
    CUtensorMap tk, tv;
    if (!make_map_bytes(&tk, pools.k, dims, strides, box) || !make_map_bytes(&tv, pools.v, dims, strides, box))
        return cudaErrorInvalidValue;
    const cudaError_t e = rt > 16 ? launch_q8_wide(a.D, rt / 128, tk, tv, t, w.ctas, stream)
                          : a.D == 128
                              ? rt == 16 ? launch<128, 16>(tk, tv, t, w.ctas, stream) : launch<128, 8>(tk, tv, t, w.ctas, stream)
                              : rt == 16 ? launch<64, 16>(tk, tv, t, w.ctas, stream) : launch<64, 8>(tk, tv, t, w.ctas, stream);
    return e != cudaSuccess ? e : launch_tree_join(a, w, 1, stream);
}

unsigned read_clear_status_cache_q8_tc(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_q8_tc_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_q8_tc_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
