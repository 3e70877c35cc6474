// cache_q8_wide.cu -- attention over an 8-bit paged cache on the tensor cores, many rows (bf16 queries).
//
// Past some sixteen rows a thread per key (cache_q8_tc.cu) does too much per score: it pays for the maximum
// across lanes, for the rows' factors from shared memory and for three parts of every weight.  Here a thread has
// a row, as in the attention over 16-bit pages: NT row tiles of 128 rows, S = Q K^T with the online softmax along
// registers, O += P V with P in tensor memory.
//   S: the K codes as they lie in the pages, queries as two e4m3 parts (two MMAs into one S, at twice the rate of a
//     16-bit one).
//   P V: in fp16.  Two warps turn each V tile's codes into fp16 times the key's scale, relative to the tile's largest
//     scale: one pass over 16 KB per 128 keys, where splitting the weights would cost some five instructions
//     for every score, and P V half as much time again on the tensor pipe (three 8-bit passes against one 16-bit).
//     Codes and scales within 2^4 of one another are exact in fp16.  Where a tile's scales are further apart the codes go
//     in as they are and every weight takes its key's scale along: such tiles look at their scores twice.
//   K's scales multiply the scores, as floats from shared memory that the same two warps write.
// A row has two references: of its scores, for the sum of its weights (fp32), and of its scores plus the exponents of the
// V scales, for what goes into P, so that a key of large weight and small value (or a hidden one of any value) takes no
// bits from the others.  They move when a tile's maximum passes them by 2^8; what goes into P is at most 2^8 2^7 in fp16, off
// by 2^-25 or 2^-11 of itself: what n keys of little weight add up to is off by n 2^-28 of the row's largest product.
//   NT = 1, KT = 64, two CTAs per SM: a unit of at most 128 rows.
//   NT = 2, KT = 128, one CTA per SM: both row tiles read one K and one V tile and take turns on the pipe.
//
// Measured, 16 / 8 or 64 / 8 heads, D = 128, against the attention over 16-bit pages:
//   8 trees of 10 to 25 tokens behind 2K-8K keys (up to 200 rows, NT = 2): 59 us; 50 in 16 bits.
//   4 trees of up to 64 tokens behind 32K keys (512 rows, NT = 2): 155 us, 950 TFLOP/s of the formula's; 117.
//   8 x 4 tokens over up to 16K keys (32 rows, NT = 1): 66 us; 68.  16 tokens (128 rows), up to 8K keys: 46; 46.
// With one V scale for all of a unit, which lost what lay 2^-24 below it, these took 58, 150, 62 and 44.
// Where every tile's V scales are 2^5 and more apart they take 107, 309, 111 and 69.
// NT = 2 is bound by the chain of a row tile, softmax (2000 cycles), P V, the next Q K^T: 4000 cycles per 128 keys of both
// tiles, of which the pipe works 2048; a warp's first scores come 14000 cycles after the launch (the batch's scan, the
// walk, the queries).  NT = 1 by the issue of its MMAs (12 per 64 keys, each 40 to 50 cycles at this width) and by shared
// memory.  Halving the chain's links (S in two halves of 64 keys, 188 us for the 64-token trees), a softmax in one
// pass that is taken again where a maximum moved (184), and 32 rows to a softmax warpgroup (spills, 370) cost more.
//
// Roles: 4 NT softmax warps (a thread per row), one warp that streams K and V pages (and scales), one that issues
// the MMAs, two that convert.
#include <cmath>

#include "cache_q8_mma.cuh"

namespace ra {

static __device__ unsigned g_cache_q8_wide_status[2];

namespace {

constexpr float kRescaleLog2 = 8.0f;
constexpr float kWeightLog2 = 7.0f;  // weights go into P times 2^7 over their reference
constexpr unsigned kSpread = 4;      // log2 by which a tile's V scales may differ to be one scale
constexpr unsigned kFar = 60;        // log2 by which they may lie below the unit's largest so far for P's weights, in fp32, to give the row's sum
constexpr int kMostUp = 240;         // queries are scaled up by at most 2^113, so that a score plus an exponent over it is finite

template <int D, int NT>
struct Cfg {
    static constexpr int kKT = NT == 1 ? 64 : 128;      // keys per tile
    static constexpr int kSoftmax = 128 * NT;           // softmax threads
    static constexpr int kThreads = kSoftmax + 128;     // producer, issuer, two converters
    static constexpr int kQPart = 128 * D;              // one part of a row tile's queries
    static constexpr int kStageBytes = kKT * D;
    static constexpr int kVBytes = kKT * D * 2;         // an fp16 V tile, of two
    static constexpr int kHead = 6144;                  // barriers, scales and scratch ahead of the tiles
    static constexpr int kBudget = NT == 1 ? 113 * 1024 : 227 * 1024;
    static constexpr int kFit = (kBudget - kHead - NT * 2 * kQPart - 2 * kVBytes) / kStageBytes;
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr int kV = kStages / 2, kK = kStages - kV;  // stages of the two rings
    static constexpr int kSmem = kHead + NT * 2 * kQPart + 2 * kVBytes + kStages * kStageBytes;
    static constexpr int kTmemCols = 256 * NT;
    static constexpr int kOCol = 128;                   // O columns of a row tile, behind its S
    // weight of a unit beyond its tiles (NT = 1: with 3, 128 rows of 8 sequences take 45.5 us, not 43.8; NT = 2: with 3 and
    // 6 the 25-token trees take 56.7 and 58.6 us, the 64-token ones 150.5 and 148.2)
    static constexpr int kOV = NT == 1 ? 6 : 4;
    static constexpr int kMinW = NT == 1 ? 2 : 3;       // least weight per CTA
    static_assert(kV >= 2, "stages");
};

struct Bars {
    uint64_t full[2][5], empty[2][5];  // stages of the K ring and the V ring
    uint64_t q_full[2];                // by row tile
    uint64_t s_full[2], p_full[2];     // by S buffer (NT = 1) or row tile (NT = 2)
    uint64_t p_half[2];                // NT = 2: the first 64 keys of P
    uint64_t o_done[2];                // P V done: as s_full, so that one parity tells its phases apart
    uint64_t cv_full[2], cv_empty[2];  // converted tiles
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

struct Head {
    Bars bar;
    // Of a converted tile: the V exponent (+ 127) that it is relative to, for P and for the sum; 0 and infinity where the
    // keys' V scales are far apart, and it is relative to each key's own.
    float2 v_ref[2];
    alignas(16) unsigned char scales[5][2][128];  // of a V stage's keys: K's, V's
    // of a converted tile's keys: K's scales times that of the scores, what the softmax multiplies S with (the same, or ones
    // where V's scales are far apart), and log2 of what V is relative to (+ 127; -inf: no scale)
    alignas(16) float k_scale[2][128], s_scale[2][128], v_exp[2][128];
};

// NT = 2 launches 384 threads with 168 registers each and hands the softmax warpgroups 224 of them (256 x 224 +
// 128 x 56 = 384 x 168), as the attention over 16-bit pages does.
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

// Instruction descriptor, kind::f16 with fp16 A and B (B with its columns contiguous) and fp32 results.
constexpr uint32_t idesc_f16_pv(int N) {
    return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// 16 codes of a key as fp16 times `scale`.
__device__ __forceinline__ void to_f16(const uint4& codes, __half2 scale, uint32_t (&h)[8]) {
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c[j / 2] >> (16 * (j & 1))), __NV_E4M3);
        const __half2 y = __hmul2(__half2(r), scale);
        h[j] = *reinterpret_cast<const uint32_t*>(&y);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, NT == 1 ? 2 : 1)
    q8_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ Q8Params a) {
    using C = Cfg<D, NT>;
    constexpr int KT = C::kKT, RT = 128 * NT;
    extern __shared__ __align__(1024) uint8_t smem[];
    Head& head = *reinterpret_cast<Head*>(smem);
    Bars& bar = head.bar;
    RangeScratch<C::kThreads>& scratch = *reinterpret_cast<RangeScratch<C::kThreads>*>(smem + C::kHead - 512);
    static_assert(sizeof(Head) <= C::kHead - 512 && sizeof(RangeScratch<C::kThreads>) <= 512, "head of the shared memory");
    uint8_t* q_smem = smem + C::kHead;                    // [row tile][part]
    uint8_t* cv_smem = q_smem + NT * 2 * C::kQPart;       // two fp16 V tiles
    uint8_t* k_ring = cv_smem + 2 * C::kVBytes;
    uint8_t* v_ring = k_ring + C::kK * C::kStageBytes;
    static_assert(C::kHead % 1024 == 0 && C::kQPart % 1024 == 0 && C::kVBytes % 1024 == 0 && C::kStageBytes % 1024 == 0,
                  "swizzled tiles start on 1024 bytes");
    const CacheBatch& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* status = g_cache_q8_wide_status;
    const bool tree = p.tree_mask != nullptr;
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) cache_report(status, 0x0C000000u);
        return;
    }

    constexpr int kProducer = C::kSoftmax / 32, kIssuer = kProducer + 1, kConverter = kProducer + 2;
    if (warp == kIssuer) {
        if (lane == 0) {
            for (int s = 0; s < 5; ++s) {
                mbar_init(&bar.full[0][s], 1);
                mbar_init(&bar.full[1][s], 1 + 32);  // the tile's bytes, and every lane's scales
                mbar_init(&bar.empty[0][s], 1);
                mbar_init(&bar.empty[1][s], 2);      // the converters
            }
            for (int t = 0; t < 2; ++t) {
                mbar_init(&bar.q_full[t], 128);
                mbar_init(&bar.s_full[t], 1);
                mbar_init(&bar.p_half[t], 128);
                mbar_init(&bar.p_full[t], 128);
                mbar_init(&bar.o_done[t], 1);
                mbar_init(&bar.cv_full[t], 64);
                mbar_init(&bar.cv_empty[t], 1);
            }
            mbar_init(&bar.drain, 1);
            bar.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&bar.tmem, C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kProducer && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    grid_dependency_wait();    // nothing above reads or writes global memory
    grid_launch_dependents();  // the join may take its place on the SMs; it waits for this grid's end
    const Column col = column_of(a.columns);
    if (threadIdx.x == 0) a.jobs[col.cta].rows = 0;
    tc_fence_before();
    const WorkRange& range = find_range<C::kThreads>(p, C::kMinW, status, TreeWeight<KT, C::kOV>{p.G, a.heads, tree, RT}, scratch,
                                                     col.range, col.ranges);
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    volatile int* abort_flag = &bar.abort;
    SegmentWalk<KT, C::kOV> walk;
    walk.start(p, range, RT, a.heads, col.index * a.heads);
    Segment g;
    int place = 0, v_place = 0;  // K and V tiles the producer has loaded so far

    if (warp == kProducer) {
        // ---------------------------------------------------------------- pages -> shared memory
        reg_dec<NT>();
        bool ok = true;
        const int sub_rows = min(1 << p.page_shift, KT);  // rows of a box
        const int groups = KT / sub_rows;                 // pages of a tile (at most 16): lane g finds page g
        const int none = p.n_pages << p.page_shift;       // past the pool: loads zeros
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
            for (int i = 0; i < T; ++i) {
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
                const int key4 = key0 + 4 * (lane % (KT / 4)), lp4 = key4 >> p.page_shift, pg4 = page_of(lp4);
#pragma unroll
                for (int ring = 0; ring < 2; ++ring) {
                    const int n_stages = ring == 0 ? C::kK : C::kV, n = ring == 0 ? place : v_place, stage = n % n_stages;
                    if (n >= n_stages) {
                        ok = warp_wait(&bar.empty[ring][stage], (n / n_stages - 1) & 1, abort_flag, status, 0x02000000u | i);
                        if (!ok) break;
                    }
                    if (elect_one()) mbar_arrive_expect_tx(&bar.full[ring][stage], C::kStageBytes);
                    __syncwarp();  // the bytes are expected before any box can land
                    if (lane < groups)
                        tma_load_4d(ring == 0 ? &tm_k : &tm_v, &bar.full[ring][stage],
                                    (ring == 0 ? k_ring : v_ring) + stage * C::kStageBytes + lane * sub_rows * D, 0, g.head, row, 0);
                    if (ring == 0) {
                        ++place;
                        continue;
                    }
                    const bool have = pg4 >= 0 && pg4 < p.n_pages;
                    const long long at = have ? ((static_cast<long long>(pg4) * p.Hkv + g.head) << p.page_shift) +
                                                    (key4 - (lp4 << p.page_shift))
                                              : 0;
                    if (lane < KT / 4) {
                        copy_scales4(&head.scales[stage][0][4 * lane], a.ks + at, have);
                        copy_scales4(&head.scales[stage][1][4 * lane], a.vs + at, have);
                    }
                    copies_arrive(&bar.full[1][stage]);
                    ++v_place;
                }
                if (!ok) break;
            }
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------------------- MMAs
        reg_dec<NT>();
        if (elect_one()) {
            constexpr uint32_t id_qk = idesc8(KT, false, false);
            constexpr uint32_t id_pv = idesc_f16_pv(D);
            constexpr uint32_t hi = desc_hi(D);
            constexpr uint32_t kStageLo = C::kStageBytes >> 4;
            const uint32_t q_lo = sw128_desc_lo(smem_u32(q_smem), 16);
            const uint32_t k_lo = sw128_desc_lo(smem_u32(k_ring), 16);
            const uint32_t v_lo = sw128_desc_lo(smem_u32(cv_smem), KT * 128);
            int segs[2] = {0, 0}, tiles[2] = {0, 0};  // of each row tile so far: the second may sit out a segment
            bool ok = true;
            auto qk = [&](int t, uint32_t s_col, int stage) {
                uint32_t ql = q_lo + t * (2 * C::kQPart >> 4), kl = k_lo + stage * kStageLo, ts = tmem + s_col;
                asm volatile("" : "+r"(ql), "+r"(kl), "+r"(ts));
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        mma8(ts, desc8(hi, ql + part * (C::kQPart >> 4) + kk * 2), desc8(hi, kl + kk * 2), id_qk,
                             part + kk > 0 ? 1u : 0u);
            };
            // 64 keys of P V, starting at key 16 * k0
            auto pv = [&](uint32_t o_col, uint32_t p_col, int buf, int k0, bool accumulate) {
                uint32_t vl = v_lo + buf * (C::kVBytes >> 4) + k0 * (2048 >> 4), to = tmem + o_col, tp = tmem + p_col + k0 * 8;
                asm volatile("" : "+r"(vl), "+r"(to), "+r"(tp));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts(to, tp + kk * 8, sw128_desc(vl + kk * (2048 >> 4)), id_pv, (kk > 0 || accumulate) ? 1u : 0u);
            };
            while (ok && walk.next(p, range, g)) {
                const int T = g.t1 - g.t0;
                if (T == 0) continue;
                const bool two = NT == 2 && g.rt * RT + 128 < g.s.n * p.G;
                ok = mbar_wait(&bar.q_full[0], segs[0] & 1, abort_flag, status, 0x03000000u);
                if (two) ok = ok && mbar_wait(&bar.q_full[1], segs[1] & 1, abort_flag, status, 0x03000001u);
                tc_fence_after();
                for (int i = 0; ok && i <= T; ++i) {
                    const int kn = tiles[0] + i, vn = kn - 1;  // K tile, V tile: every segment's tiles count for row tile 0
                    const int ks = kn % C::kK, vb = vn & 1;
                    const uint32_t v_phase = (vn >> 1) & 1;
                    if (NT == 1) {
                        if (i < T) {
                            const int buf = kn & 1;
                            if (!(ok = mbar_wait(&bar.full[0][ks], (kn / C::kK) & 1, abort_flag, status, 0x04000000u | i))) break;
                            tc_fence_after();
                            qk(0, buf * 64, ks);
                            mma_commit(&bar.s_full[buf]);
                            mma_commit(&bar.empty[0][ks]);
                        }
                        if (i > 0) {
                            if (!(ok = mbar_wait(&bar.cv_full[vb], v_phase, abort_flag, status, 0x05000000u | i))) break;
                            if (!(ok = mbar_wait(&bar.p_full[vb], v_phase, abort_flag, status, 0x06000000u | i))) break;
                            tc_fence_after();
                            pv(C::kOCol, vb * 64, vb, 0, i > 1);
                            mma_commit(&bar.cv_empty[vb]);
                            mma_commit(&bar.o_done[vb]);
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (!ok) break;
                            const uint32_t col = 256 * t;
                            if (t == 1 && !two) continue;
                            if (i > 0) {
                                const int n = tiles[t] + i - 1;
                                if (t == 0 && !(ok = mbar_wait(&bar.cv_full[vb], v_phase, abort_flag, status, 0x05000000u | i))) break;
                                // the first half of P V runs under the exponentials of the second
                                if (!(ok = mbar_wait(&bar.p_half[t], n & 1, abort_flag, status, 0x0B000000u | i))) break;
                                tc_fence_after();
                                pv(col + C::kOCol, col, vb, 0, i > 1);
                                if (!(ok = mbar_wait(&bar.p_full[t], n & 1, abort_flag, status, 0x06000000u | i))) break;
                                tc_fence_after();
                                pv(col + C::kOCol, col, vb, 4, true);
                                mma_commit(&bar.o_done[t]);
                                if (t == 1 || !two) mma_commit(&bar.cv_empty[vb]);
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
                    }
                }
                tiles[0] += T;
                ++segs[0];
                if (two) {
                    tiles[1] += T;
                    ++segs[1];
                }
            }
            mma_commit(&bar.drain);  // every MMA has completed before TMEM is released
            mbar_wait_landing(&bar.drain, 0);
        }
        __syncwarp();
    } else if (warp >= kConverter) {
        // ---------------------------------------------------------------- V codes -> fp16, scales -> floats
        reg_dec<NT>();
        const int id = (warp - kConverter) * 32 + lane;
        constexpr int kPieces = D / 16;  // 16 codes each
        int tiles = 0;
        bool ok = true;
        while (ok && walk.next(p, range, g)) {
            const int T = g.t1 - g.t0;
            unsigned so_far = 0;  // largest of the segment's V scale bytes
            for (int i = 0; i < T; ++i) {
                const int n = tiles + i, vs = n % C::kV, buf = n & 1;
                ok = warp_wait(&bar.full[1][vs], (n / C::kV) & 1, abort_flag, status, 0x0D000000u | i);
                if (ok && n >= 2) ok = warp_wait(&bar.cv_empty[buf], ((n >> 1) - 1) & 1, abort_flag, status, 0x0F000000u | i);
                if (!ok) break;
                const int valid = g.s.kv - (g.t0 + i) * KT;  // keys of the tile; what lies behind them becomes zeros
                const unsigned char* sk = head.scales[vs][0];
                const unsigned char* sv = head.scales[vs][1];
                unsigned most = 0, least = 255;
#pragma unroll
                for (int j = lane; j < KT; j += 32)
                    if (j < valid) {
                        most = max(most, static_cast<unsigned>(sv[j]));
                        least = min(least, static_cast<unsigned>(sv[j]));
                    }
                const unsigned largest = __reduce_max_sync(0xffffffffu, most);
                const bool spread = __reduce_min_sync(0xffffffffu, least) + kSpread < largest || largest + kFar < so_far;
                so_far = max(so_far, largest);
                if (id == 0) head.v_ref[buf] = spread ? make_float2(0.f, INFINITY) : make_float2(static_cast<float>(largest), static_cast<float>(largest));
#pragma unroll
                for (int j = id; j < KT; j += 64) {
                    const float ks = j < valid ? scale_of(sk[j]) * a.scale_log2 : 0.f;
                    head.k_scale[buf][j] = ks;
                    head.s_scale[buf][j] = spread ? 1.f : ks;
                    const unsigned e = spread && j < valid ? sv[j] : largest;
                    head.v_exp[buf][j] = e ? static_cast<float>(e) : -INFINITY;
                }
                const uint8_t* src = v_ring + vs * C::kStageBytes;
                uint8_t* dst = cv_smem + buf * C::kVBytes;
#pragma unroll 1
                for (int r = id; r < KT; r += 64) {
                    const unsigned e = r < valid ? sv[r] : 0u;
                    const __half2 scale = __float2half2_rn(e == 0 ? 0.f : spread ? 1.f : scale_of(127u - (largest - e)));
                    // a key's pieces lie in another order than its neighbours': no two of eight lanes meet in a bank
#pragma unroll 4
                    for (int c = 0; c < kPieces; ++c) {
                        uint4 codes = make_uint4(0, 0, 0, 0);
                        if (r < valid) codes = *reinterpret_cast<const uint4*>(src + piece_at<D>(r, c));
                        uint32_t h[8];
                        to_f16(codes, scale, h);
                        uint8_t* half_row = dst + (c / 4) * (KT * 128);  // of 64 columns
                        *reinterpret_cast<uint4*>(half_row + piece_at<128>(r, 2 * (c % 4))) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(half_row + piece_at<128>(r, 2 * (c % 4) + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(&bar.cv_full[buf]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.empty[1][vs]);
            }
            tiles += T;
        }
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
            const int fr0 = g.rt * RT + 128 * t;                         // first row of this row tile
            const int nrows = min(128, g.s.n * p.G - fr0);               // its rows (<= 0: none)
            const bool mine = nrows > 0;
            const bool row_ok = lane_row < nrows;
            const int fr = min(fr0 + lane_row, g.s.n * p.G - 1), tok = fr / p.G;
            const int row = g.s.lo + tok, q_head = g.head * p.G + fr % p.G;
            const int ctx = g.s.kv - g.s.n;                              // keys before the new tokens (may be < 0)
            float factor = 0.f, unfactor = 0.f;                          // of the row's scores; its inverse
            if (mine && T > 0) {
                // the row's queries as two parts (the last row again past the end)
                const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<long long>(row) * p.Hq + q_head) * D);
                uint4 q8[D / 8];  // all of it on its way at once
#pragma unroll
                for (int c = 0; c < D / 8; ++c) q8[c] = src[c];
                uint32_t most = 0;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint32_t w[4] = {q8[c].x, q8[c].y, q8[c].z, q8[c].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) most = max(most, max(w[j] << 16 & 0x7fffffffu, w[j] & 0x7fff0000u));
                }
                const int up = min(query_scale_byte(most), kMostUp);
                const float f = scale_of(up);
                unfactor = f;
                factor = most >= 0x7f800000u ? NAN : scale_of(254 - up);  // a row with a NaN or an infinity has no scores
                uint8_t* dst = q_smem + t * 2 * C::kQPart;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 v = q8[2 * c + j / 2];
                        const uint32_t w0 = j & 1 ? v.z : v.x, w1 = j & 1 ? v.w : v.y;
                        const float x[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                                            __uint_as_float(w1 & 0xffff0000u)};
                        query_parts4(x, f, hi[j], lo[j]);
                    }
                    *reinterpret_cast<uint4*>(dst + piece_at<D>(lane_row, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(dst + C::kQPart + piece_at<D>(lane_row, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(&bar.q_full[t]);
            }
            float m = -INFINITY, l_sum = 0.f;  // reference of the scores, sum of the weights relative to it
            float o_ref = -INFINITY;           // of what goes into P: scores plus V's exponents, less kWeightLog2
            for (int i = 0; mine && i < T; ++i) {
                const int n = tiles + i, vn = v_tiles + i;
                const int buf = NT == 1 ? n & 1 : 0;
                const uint32_t phase = NT == 1 ? (n >> 1) & 1 : n & 1;
                const uint32_t ts = t_s + buf * 64;
                // S first: once it is there the converted tile two before this one is long done, and one parity tells
                ok = warp_wait(&bar.s_full[NT == 1 ? buf : t], phase, abort_flag, status, 0x07000000u | i);
                ok = ok && warp_wait(&bar.cv_full[vn & 1], (vn >> 1) & 1, abort_flag, status, 0x08000000u | i);
                if (!ok) break;
                tc_fence_after();
                const int k0 = (g.t0 + i) * KT;
                const float* ksc = head.s_scale[vn & 1];
                const float2 v_ref = head.v_ref[vn & 1];
                if (__builtin_expect(v_ref.y == INFINITY, 0)) {
                    // the row's sum by itself, and its scores with V's exponents back into S's columns, to be multiplied by
                    // `factor` as S is; 32 at a time: unrolled it costs 4 us of 66 (32 rows a unit) where it is not run
                    const float *ks = head.k_scale[vn & 1], *ve = head.v_exp[vn & 1];
#pragma unroll 1
                    for (int c0 = 0; c0 < KT; c0 += 32) {
                        uint32_t bits = 0xffffffffu;
                        if (k0 + KT > ctx) {  // keys this row sees
                            const int r = (tree ? ctx : min(g.s.kv, ctx + tok + 1)) - k0 - c0;
                            bits = r >= 32 ? 0xffffffffu : r <= 0 ? 0u : (1u << r) - 1u;
                            if (tree) {
                                const unsigned char* mrow = p.tree_mask + static_cast<long long>(row) * p.mask_cols;
                                const int j0 = k0 + c0 - ctx, lo = max(0, -j0), hi = min(32, min(g.s.n, p.mask_cols) - j0);
                                for (int j = lo; j < hi; ++j)
                                    if (mrow[j0 + j]) bits |= 1u << j;
                            }
                        }
                        float x[32], mx = -INFINITY;
                        __syncwarp();
                        tmem_ld32(ts + c0, reinterpret_cast<uint32_t*>(x));
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            x[c] = bits >> c & 1u ? x[c] * ks[c0 + c] * factor : -INFINITY;
                            mx = fmaxf(mx, x[c]);
                        }
                        if (mx > m + kRescaleLog2) {
                            l_sum *= m == -INFINITY ? 0.f : ex2_approx(m - mx);
                            m = mx;
                        }
                        const float neg_m = m == -INFINITY ? 0.f : -m;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            l_sum += ex2_approx(x[c] + neg_m);
                            x[c] = (x[c] + ve[c0 + c]) * unfactor;
                        }
                        __syncwarp();
                        tmem_st32(ts + c0, reinterpret_cast<uint32_t*>(x));
                    }
                    tmem_wait_st();
                }
                float sr[KT];
#pragma unroll
                for (int c = 0; c < KT / 32; ++c) tmem_ld32(ts + c * 32, reinterpret_cast<uint32_t*>(sr) + c * 32);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < KT; c += 4) {
                    const float4 f = lds4(ksc + c);
                    fmul2(sr[c], sr[c + 1], sr[c], sr[c + 1], f.x, f.y);
                    fmul2(sr[c + 2], sr[c + 3], sr[c + 2], sr[c + 3], f.z, f.w);
                }
                if (k0 + KT > ctx) {
                    // keys this row sees: a prefix, and under a tree mask the set new tokens after it
                    const int prefix = (tree ? ctx : min(g.s.kv, ctx + tok + 1)) - k0;
                    uint32_t bits[KT / 32];
#pragma unroll
                    for (int w = 0; w < KT / 32; ++w) {
                        const int r = prefix - 32 * w;
                        bits[w] = r >= 32 ? 0xffffffffu : r <= 0 ? 0u : (1u << r) - 1u;
                    }
                    if (tree) {
                        const unsigned char* mrow = p.tree_mask + static_cast<long long>(row) * p.mask_cols;
#pragma unroll
                        for (int w = 0; w < KT / 32; ++w) {
                            const int j0 = k0 + 32 * w - ctx;  // new token of the word's first bit
                            const int lo = max(0, -j0), hi = min(32, min(g.s.n, p.mask_cols) - j0);
                            uint32_t add = 0;
                            for (int j = lo; j < hi; ++j)
                                if (mrow[j0 + j]) add |= 1u << j;
                            bits[w] |= add;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < KT; ++c)
                        if (!((bits[c >> 5] >> (c & 31)) & 1u)) sr[c] = -INFINITY;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < KT; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x) m4[x] = fmax3(m4[x], sr[c + 2 * x], sr[c + 2 * x + 1]);
                const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * factor;
                if (mx > m + (v_ref.y - v_ref.x + kRescaleLog2)) {  // (not where the sum is there already)
                    l_sum *= m == -INFINITY ? 0.f : ex2_approx(m - mx);
                    m = mx;
                }
                const float top = mx + (v_ref.x - kWeightLog2);
                float alpha = 1.f;
                bool resc = false;
                if (i == 0) {
                    o_ref = top;
                } else if (top > o_ref + kRescaleLog2) {
                    alpha = o_ref == -INFINITY ? 0.f : ex2_approx(o_ref - top);
                    o_ref = top;
                    resc = true;
                }
                const float neg = o_ref == -INFINITY ? 0.f : v_ref.x - o_ref;
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
                        ffma2(y0, y1, sr[c0 + 2 * j], sr[c0 + 2 * j + 1], factor, factor, neg, neg);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        if (j & 1)
                            fadd2(s2, s3, p0, p1);
                        else
                            fadd2(s0, s1, p0, p1);
                        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(pk[j]) : "f"(p0), "f"(p1));  // half an fp16 step each
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
                // P's weights are 2^(V's exponent) of the sum's; a NaN stays one
                const float in_p = (s0 + s1) + (s2 + s3);
                l_sum += in_p == 0.f ? 0.f : in_p * ex2_approx(o_ref - v_ref.y - m);
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
                // O's unit in two powers of two: it may lie below what a float holds
                const float unit = o_ref == -INFINITY ? 0.f : o_ref - m - 127.f, half = floorf(unit * 0.5f);
                const float up = ex2_approx(half), up2 = ex2_approx(unit - half);
                // a row with a NaN keeps it, one that saw no key gets zeros
                const float f = !whole ? up2 : l_sum > 0.f ? up2 / l_sum : l_sum == 0.f ? 0.f : NAN;
                const int part_row = t * 128 + lane_row;
                const long long slot = static_cast<long long>(partial_slot(g, col.cta)) * a.slot_rows;
#pragma unroll 1  // runs once or twice a CTA: less code to fetch
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    if (T > 0) {
                        tmem_ld32(t_o + c * 32, r);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0;
                    }
                    float* o = reinterpret_cast<float*>(r);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = o[j] * up * f;
                    if (row_ok && whole) {
                        __nv_bfloat16* dst = a.out + (static_cast<long long>(row) * p.Hq + q_head) * D + c * 32;
#pragma unroll
                        for (int j = 0; j < 4; ++j) store8(dst + 8 * j, o + 8 * j);
                    } else if (row_ok) {
                        float4* dst = reinterpret_cast<float4*>(a.part_o + slot * D) + c * 8 * a.slot_rows + part_row;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j * a.slot_rows] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (row_ok && whole && a.lse)
                    a.lse[static_cast<long long>(q_head) * p.R + row] = row_lse(m, l_sum);
                if (row_ok && !whole) a.stats[slot + part_row] = make_float2(m, l_sum);
            }
            if (threadIdx.x == 0 && !g.whole() && g.t0 == 0) {
                const int first = g.rt * RT;
                a.jobs[col.cta] = JoinJob{first, min(RT, g.s.n * p.G - first), g.s.lo, g.head,
                                             col.index * col.ranges + owner_of(range, g.a + C::kOV + g.tiles - 1), {0, 0, 0}};
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
    if (*abort_flag && warp == kProducer) {
        for (int n = max(0, place - C::kK); n < place; ++n)
            mbar_wait_landing(&bar.full[0][n % C::kK], (n / C::kK) & 1);
        for (int n = max(0, v_place - C::kV); n < v_place; ++n)
            mbar_wait_landing(&bar.full[1][n % C::kV], (n / C::kV) & 1);
    }
}

template <int D, int NT>
cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const Q8Params& a, int ctas, cudaStream_t stream) {
    using C = Cfg<D, NT>;
    static OncePerDevice once;
    const cudaError_t set = once([] {
        cudaError_t e = cudaFuncSetAttribute(q8_wide_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        // the register increase draws on the launch's registers: with fewer it would wait for ever
        cudaFuncAttributes fa;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, q8_wide_kernel<D, NT>);
        return e == cudaSuccess && NT == 2 && fa.numRegs < kLaunchRegs ? cudaErrorLaunchOutOfResources : e;
    });
    if (set != cudaSuccess) return set;
    return launch_overlapped(q8_wide_kernel<D, NT>, dim3(ctas), C::kThreads, C::kSmem, stream, k, v, a);
}

}  // namespace

int q8_wide_key_tile(int nt) { return nt == 1 ? 64 : 128; }

cudaError_t launch_q8_wide(int D, int nt, const CUtensorMap& k, const CUtensorMap& v, const Q8Params& a, int ctas,
                           cudaStream_t stream) {
    if (D == 128) return nt == 1 ? launch<128, 1>(k, v, a, ctas, stream) : launch<128, 2>(k, v, a, ctas, stream);
    return nt == 1 ? launch<64, 1>(k, v, a, ctas, stream) : launch<64, 2>(k, v, a, ctas, stream);
}

unsigned read_clear_status_cache_q8_wide(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_q8_wide_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_q8_wide_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
