// key_mass_tc.cu -- attention weight gathered per cached key, on the tensor cores (bf16).
//
// The scores are taken transposed, S^T = K Q^T (tcgen05, fp32 in TMEM): a key is a
// TMEM lane, so a thread owns a key and adds up 2^(s c - lse_r) over the rows r
// that see it in its own registers -- no reduction across threads, no atomics,
// one order of summation.
//
// A CTA walks tiles of 128 keys of one (sequence, KV head) in pairs, two warpgroups
// per tile where chunks have more than 32 rows (rows 0-63 and 64-127: four warps per
// scheduler hide the latencies of a thread's chain of loads, exponentials and sums;
// a 64-token window takes 32 us with two, 36 with one); both tiles meet
// the same rows, in chunks of 128 / G tokens
// (N of the MMA is the chunk's rows rounded up to 16: decode costs 16 columns, not
// 128).  Up to two chunks stay in shared memory for the whole run of tiles, more
// are streamed again for every pair.  Under the chain mask the chunks before a
// pair's keys are skipped.
//
// Bounds: with few rows the bytes of K (16 sequences of 4K-16K keys, one token, 64 / 8
// heads: 65 us, 5.6 TB/s with a start of 5 us); with many (64 tokens over 16000 keys, 4
// sequences, 32 / 8 heads: 32 us) shared memory: for two tiles and 128 rows the MMAs read
// their operands for 1024 cycles at 128 bytes a cycle, the weights their rows' lse for
// another 1024, K arrives for 256, of 2300 cycles in all; the exponentials take 1024.
// Without the lse reads the call would take 29.7 us, without exponentials 29.1.
//
// Roles: the weight warps first, then two that stream K pages (64 columns each), one
// for the row chunks and the issuer of the MMAs.
#include <cmath>

#include "cache_batch.cuh"

namespace ra {

static __device__ unsigned g_mass_tc_status[2];

namespace {

constexpr int kKT = kMassTile;      // keys of a tile
constexpr int kParts = 4;      // sums of second halves on their way (they run at most two chunks ahead)
constexpr int kQ = kMassResident;   // row chunks in shared memory
constexpr int kOld = 4;        // tiles ahead that the old mass is fetched
constexpr int kHead = 13312;   // barriers, scratch, lse, second halves, old mass
constexpr float kLog2e = 1.44269504088896341f;

// QR: rows of a chunk.  128, or 32 for batches of few rows (decode, small trees), where the cache's bytes bound
// the kernel: one warpgroup per tile then does, and the room goes to K stages (16 x 16384 keys, one token: 64 us,
// 67 us with chunks of 128 rows).
template <int D, int QR>
struct Cfg {
    static constexpr int kHalves = QR == 128 ? 2 : 1;   // warpgroups per tile of the pair
    static constexpr int kThreads = 256 * kHalves + 128;
    static constexpr int kWarpK = 8 * kHalves, kWarpQ = kWarpK + 1, kWarpMma = kWarpK + 2, kWarpK2 = kWarpK + 3;
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kQBytes = QR * D * 2;
    static constexpr int kFit = (232448 - kHead - kQ * kQBytes) / kTileBytes;
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr int kSmem = kHead + kQ * kQBytes + kStages * kTileBytes;
    static_assert(kSmem <= 232448, "exceeds the 227 KB of shared memory a CTA may use");
};

struct MassParams {
    CacheBatch p;
    int rpt, q_bytes;
    float scale_log2, decay;
    const float* lse;
    const float* in;
    float* out;
    int cols;
};

struct Bars {
    uint64_t k_full[10], k_empty[10];
    uint64_t q_full[kQ], q_empty[kQ];
    uint64_t s_full[2][2], s_empty[2][2];  // [tile of the pair][buffer]
    uint64_t lse_ready[2];                 // by tile of the pair
    uint64_t part_ready[2][kParts];
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

template <int D, int QR>
__global__ void __launch_bounds__(Cfg<D, QR>::kThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ MassParams m) {
    using C = Cfg<D, QR>;
    constexpr int kRing = C::kStages, kThreads = C::kThreads;
    constexpr int kWarpK = C::kWarpK, kWarpQ = C::kWarpQ, kWarpMma = C::kWarpMma, kWarpK2 = C::kWarpK2;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars& bar = *reinterpret_cast<Bars*>(smem);
    RangeScratch<kThreads>& scratch = *reinterpret_cast<RangeScratch<kThreads>*>(smem + 512);
    float* lse_s = reinterpret_cast<float*>(smem + 1024);   // [tile of the pair][run parity][kQ][128]
    float* old_s = reinterpret_cast<float*>(smem + 9216);   // [tile of the pair][kOld][128]
    float* part_s = reinterpret_cast<float*>(smem + 5120);  // [tile of the pair][kParts][128]
    static_assert(sizeof(Bars) <= 512 && sizeof(RangeScratch<kThreads>) <= 512, "head of the shared memory");
    uint8_t* q_smem = smem + kHead;
    uint8_t* ring = q_smem + kQ * C::kQBytes;
    const CacheBatch& p = m.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* status = g_mass_tc_status;
    const bool tree = p.tree_mask != nullptr;
    if (smem_u32(smem) & 1023) {  // swizzled tiles start on 1024 bytes
        if (threadIdx.x == 0) cache_report(status, 0x0C000000u);
        return;
    }
    if (warp == kWarpMma) {
        if (lane == 0) {
            for (int s = 0; s < kRing; ++s) {
                mbar_init(&bar.k_full[s], C::kChunks);  // a warp per 64 columns
                mbar_init(&bar.k_empty[s], 1);
            }
            for (int s = 0; s < kQ; ++s) {
                mbar_init(&bar.q_full[s], 1);
                mbar_init(&bar.q_empty[s], 1);
            }
            for (int t = 0; t < 2; ++t) {
                for (int s = 0; s < 2; ++s) {
                    mbar_init(&bar.s_full[t][s], 1);
                    mbar_init(&bar.s_empty[t][s], 128 * C::kHalves);
                }
                mbar_init(&bar.lse_ready[t], 128 * C::kHalves);
                for (int s = 0; s < kParts; ++s) mbar_init(&bar.part_ready[t][s], 128);
            }
            mbar_init(&bar.drain, 1);
            bar.abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    if (warp == kWarpK && lane == 0) tma_prefetch_desc(&tm_k);
    if (warp == kWarpQ && lane == 0) tma_prefetch_desc(&tm_q);
    grid_dependency_wait();  // nothing above reads or writes global memory
    tc_fence_before();
    const MassTiles weight{p.Hkv, m.rpt, tree};
    const WorkRange& range = find_range<kThreads>(p, 1, status, weight, scratch);
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    volatile int* abort_flag = &bar.abort;
    MassWalk walk;
    walk.b = range.b;
    walk.head = range.head;
    walk.i = range.idx;
    walk.a = range.a;
    if (range.b < p.n_seqs) walk.s = range.s;
    int head, i0, i1;
    auto next_run = [&] {
        return walk.next(p.n_seqs, range.hi, weight, [&](int b, CacheSeq& s) { load_seq(p, b, s); }, head, i0, i1);
    };
    bool ok = true;
    int place = 0;  // of a producer: tiles or row chunks loaded so far

    if (warp == kWarpK || (warp == kWarpK2 && C::kChunks == 2)) {
        // ---------------------------------------------------------------- K pages
        const int sub_rows = min(1 << p.page_shift, kKT);
        const int groups = kKT / sub_rows;  // pages of a tile (at most 16): lane g finds page g
        const int none = p.n_pages << p.page_shift;
        while (ok && next_run()) {
            const CacheSeq s = walk.s;
            if (s.n == 0) continue;
            const int* table = p.pages + static_cast<long long>(walk.b) * p.max_pages;
            const int listed = (s.kv + (1 << p.page_shift) - 1) >> p.page_shift;
            auto entry = [&](int lp) { return lp < listed ? table[lp] : -1; };
            int win = (i0 * kKT) >> p.page_shift;
            int e0 = entry(win + lane), e1 = entry(win + 32 + lane);
            for (int i = i0; i < i1; ++i, ++place) {
                const int stage = place % kRing;
                if (place >= kRing) {
                    ok = warp_wait(&bar.k_empty[stage], (place / kRing - 1) & 1, abort_flag, status, 0x02000000u | i);
                    if (!ok) break;
                }
                const int first = (i * kKT) >> p.page_shift;
                while (first >= win + 32) {
                    win += 32;
                    e0 = e1;
                    e1 = entry(win + 32 + lane);
                }
                const int key = i * kKT + lane * sub_rows, lp = key >> p.page_shift, at = lp - win;
                const int pg0 = __shfl_sync(0xffffffffu, e0, at & 31), pg1 = __shfl_sync(0xffffffffu, e1, at & 31);
                const int pg = at < 32 ? pg0 : pg1;
                int row = none;
                if (lane < groups && lp < listed) {
                    if (pg >= 0 && pg < p.n_pages)
                        row = (pg << p.page_shift) + (key - (lp << p.page_shift));
                    else
                        cache_report(status, 0x0E000000u | static_cast<unsigned>(lp & 0xFFFFFF));
                }
                if (elect_one()) mbar_arrive_expect_tx(&bar.k_full[stage], 16384);
                __syncwarp();  // the bytes are expected before any box can land
                load_tile<1>(&tm_k, &bar.k_full[stage], ring + stage * C::kTileBytes, 16384, groups, sub_rows, head, row,
                             warp == kWarpK ? 0 : 1);
            }
        }
    } else if (warp == kWarpQ) {
        // ---------------------------------------------------------------- row chunks
        if (lane == 0) {
            auto load = [&](const CacheSeq& s, int c) {
                const int stage = place % kQ;
                if (place >= kQ && !mbar_wait(&bar.q_empty[stage], (place / kQ - 1) & 1, abort_flag, status, 0x01000000u))
                    return false;
                mbar_arrive_expect_tx(&bar.q_full[stage], C::kChunks * m.q_bytes);
                for (int x = 0; x < C::kChunks; ++x)
                    tma_load_4d(&tm_q, &bar.q_full[stage], q_smem + stage * C::kQBytes + x * (QR * 128), x * 64, 0, head,
                                s.lo + c * m.rpt);
                ++place;
                return true;
            };
            while (ok && next_run()) {
                const CacheSeq s = walk.s;
                const int nch = weight.chunks(s);
                if (weight.resident(s)) {
                    for (int c = weight.run_chunk(s, i0); ok && c < nch; ++c) ok = load(s, c);
                } else {
                    for (int i = i0; ok && i < i1; i += 2)
                        for (int c = weight.first_chunk(s, i); ok && c < nch; ++c) ok = load(s, c);
                }
            }
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ---------------------------------------------------------------- MMAs
        if (elect_one()) {
            const uint32_t q_lo = sw128_desc_lo(smem_u32(q_smem), 16), k_lo = sw128_desc_lo(smem_u32(ring), 16);
            constexpr uint32_t kTileLo = C::kTileBytes >> 4;
            int kn = 0, qn = 0, task[2] = {0, 0};
            while (ok && next_run()) {
                const CacheSeq s = walk.s;
                const int nch = weight.chunks(s);
                if (nch == 0) continue;
                const bool resident = weight.resident(s);
                const int c0 = weight.run_chunk(s, i0);
                for (int i = i0; ok && i < i1; i += 2) {
                    const int two = i + 1 < i1 ? 2 : 1;
                    int k_ready = 0;
                    for (int c = weight.first_chunk(s, i); ok && c < nch; ++c) {
                        const int q = resident ? qn + c - c0 : qn;
                        ok = mbar_wait(&bar.q_full[q % kQ], (q / kQ) & 1, abort_flag, status, 0x03000000u | c);
                        if (!ok) break;
                        const int cols = min(m.rpt, s.n - c * m.rpt) * p.G;
                        const uint32_t idesc = idesc_bf16_f32(128, (cols + 15) & ~15, false, false);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t == two) break;
                            const int stage = (kn + t) % kRing;
                            if (k_ready == t) {
                                ok = mbar_wait(&bar.k_full[stage], ((kn + t) / kRing) & 1, abort_flag, status, 0x04000000u | i);
                                if (!ok) break;
                                ++k_ready;
                            }
                            const int n = task[t]++, buf = n & 1;
                            if (n >= 2) {
                                ok = mbar_wait(&bar.s_empty[t][buf], ((n >> 1) - 1) & 1, abort_flag, status, 0x05000000u | c);
                                if (!ok) break;
                            }
                            tc_fence_after();
                            uint32_t kl = k_lo + stage * kTileLo, ql = q_lo + (q % kQ) * (C::kQBytes >> 4);
                            uint32_t ts = tmem + t * 256 + buf * 128;
                            asm volatile("" : "+r"(kl), "+r"(ql), "+r"(ts));  // descriptors formed next to their MMAs
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                mma_ss(ts, sw128_desc(kl + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2),
                                       sw128_desc(ql + (kk >> 2) * (QR * 128 >> 4) + (kk & 3) * 2), idesc, kk > 0 ? 1u : 0u);
                            }
                            mma_commit(&bar.s_full[t][buf]);
                            if (c == nch - 1) mma_commit(&bar.k_empty[stage]);
                        }
                        if (!ok) break;
                        if (!resident) mma_commit(&bar.q_empty[qn++ % kQ]);
                    }
                    kn += two;
                }
                if (ok && resident) {
                    for (int c = c0; c < nch; ++c) mma_commit(&bar.q_empty[qn++ % kQ]);
                }
            }
            mma_commit(&bar.drain);
            mbar_wait_landing(&bar.drain, 0);
        }
        __syncwarp();
    } else if (warp < kWarpK) {
        // ---------------------------------------------------------------- weights, a thread per key
        const int t = warp / (4 * C::kHalves), half = (warp >> 2) % C::kHalves, row = threadIdx.x & 127;
        const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 256;
        float* part = part_s + t * kParts * 128;
        int task = 0, lse_turn = 0, part_turn = 0;
        LseSets lse_sets;
        while (ok && next_run()) {
            const CacheSeq s = walk.s;
            const int nch = weight.chunks(s), ctx = s.kv - s.n;
            const bool resident = weight.resident(s);
            const bool wide = C::kHalves == 2 && min(s.n, m.rpt) * p.G > 64;  // the second half has rows
            const long long mass_row = (static_cast<long long>(walk.b) * p.Hkv + head) * m.cols;
            // lse of this thread's row of chunk c
            auto row_lse = [&](int c) {
                const int tok0 = c * m.rpt;
                if (c >= nch || row >= min(m.rpt, s.n - tok0) * p.G) return 0.f;
                return m.lse[static_cast<long long>(head * p.G + row % p.G) * p.R + s.lo + tok0 + row / p.G];
            };
            // The old mass of this thread's key of tile i, fetched into a slot of its own: a register would be waited
            // for where it is handed on from tile to tile.
            float* old = old_s + t * kOld * 128 + row;
            auto fetch_old = [&](int i) {
                const int key = i * kKT + row;
                if (half == 0 && m.in && i < i1 && key < s.kv)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(old + (i >> 1) % kOld * 128)),
                                 "l"(m.in + mass_row + key)
                                 : "memory");
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            float next_lse = row_lse(weight.first_chunk(s, i0));
            for (int u = 0; u < kOld - 1; ++u) fetch_old(i0 + t + 2 * u);
            int held = 0;  // resident: chunks whose lse is in lse_wg
            // a run's first write must not meet the last reads of the run before
            float* lse_wg = lse_s + (t * 2 + lse_sets.take(nch, i0, i1, t)) * kQ * 128;
            for (int i = i0 + t; ok && i < i1; i += 2) {
                fetch_old(i + 2 * (kOld - 1));
                const int k0 = i * kKT, key = k0 + row, jn = key - ctx;
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
                // the pair starts at its first tile's first chunk; the second tile's rows before its own add 0
                for (int c = weight.first_chunk(s, i - t); c < nch; ++c) {
                    const int tok0 = c * m.rpt, cols = min(m.rpt, s.n - tok0) * p.G;
                    const int lse_buf = resident ? c : lse_turn & 1;
                    if (!resident || !((held >> c) & 1)) {
                        if (resident) next_lse = held == 0 ? next_lse : row_lse(c);
                        // -lse in log2 units, so that a row without keys (lse = -inf) adds 2^-inf = 0
                        if (half == 0) lse_wg[lse_buf * 128 + row] = next_lse == -INFINITY ? -INFINITY : -next_lse * kLog2e;
                        if (!resident) next_lse = row_lse(c + 1 < nch ? c + 1 : weight.first_chunk(s, i - t + 2));
                        mbar_arrive(&bar.lse_ready[t]);
                        ok = warp_wait(&bar.lse_ready[t], lse_turn++ & 1, abort_flag, status, 0x06000000u | i);
                        if (!ok) break;
                        held |= 1 << (c & 31);
                    }
                    const float* nl = lse_wg + lse_buf * 128;
                    const int buf = task & 1;
                    ok = warp_wait(&bar.s_full[t][buf], (task >> 1) & 1, abort_flag, status, 0x07000000u | i);
                    if (!ok) break;
                    ++task;
                    tc_fence_after();
                    const bool tail = k0 + kKT > ctx;   // new tokens in the tile
                    auto add_rows = [&](const uint32_t* sr, int c0) {
                        uint32_t bits = 0xffffffffu;
                        if (tail || cols - c0 < 32) {
                            if (cols - c0 < 32) bits = (1u << (cols - c0)) - 1u;
                            if (tail && jn >= 0) {
                                if (!tree) {
                                    const long long hide = (static_cast<long long>(jn) - tok0) * p.G - c0;
                                    bits &= hide <= 0 ? 0xffffffffu : hide >= 32 ? 0u : 0xffffffffu << hide;
                                } else {
                                    uint32_t see = 0;
                                    if (jn < p.mask_cols && jn < s.n)
                                        for (int tk = c0 / p.G; tk * p.G < min(cols, c0 + 32); ++tk)
                                            if (p.tree_mask[static_cast<long long>(s.lo + tok0 + tk) * p.mask_cols + jn]) {
                                                const int lo = max(0, tk * p.G - c0), hi = min(32, (tk + 1) * p.G - c0);
                                                see |= (hi - lo >= 32 ? 0xffffffffu : (1u << (hi - lo)) - 1u) << lo;
                                            }
                                    bits &= see;
                                }
                            }
                            if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    const float y = fmaf(__uint_as_float(sr[j]), m.scale_log2, nl[c0 + j]);
                                    const float e = (bits >> j) & 1u ? ex2_approx(y) : 0.f;
                                    if ((j & 3) == 0) s0 += e;
                                    if ((j & 3) == 1) s1 += e;
                                    if ((j & 3) == 2) s2 += e;
                                    if ((j & 3) == 3) s3 += e;
                                }
                                return;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 n4 = *reinterpret_cast<const float4*>(nl + c0 + j);
                            float y0, y1, y2, y3;
                            ffma2(y0, y1, __uint_as_float(sr[j]), __uint_as_float(sr[j + 1]), m.scale_log2, m.scale_log2,
                                  n4.x, n4.y);
                            ffma2(y2, y3, __uint_as_float(sr[j + 2]), __uint_as_float(sr[j + 3]), m.scale_log2,
                                  m.scale_log2, n4.z, n4.w);
                            fadd2(s0, s1, ex2_approx(y0), ex2_approx(y1));
                            fadd2(s2, s3, ex2_approx(y2), ex2_approx(y3));
                        }
                    };
                    const uint32_t ts = t_s + buf * 128;
#pragma unroll 1
                    for (int c0 = half * 64; c0 < min(cols, half * 64 + 64); c0 += 32) {  // QR = 32: one step
                        uint32_t sr[32];
                        tmem_ld32(ts + c0, sr);
                        tmem_wait_ld();
                        add_rows(sr, c0);
                    }
                    tc_fence_before();
                    mbar_arrive(&bar.s_empty[t][buf]);
                }
                if (!ok) break;
                float sum = (s0 + s1) + (s2 + s3);
                if (wide) {
                    const int slot = part_turn & (kParts - 1);
                    if (half == 1) {
                        part[slot * 128 + row] = sum;
                        mbar_arrive(&bar.part_ready[t][slot]);
                    } else {
                        ok = warp_wait(&bar.part_ready[t][slot], (part_turn / kParts) & 1, abort_flag, status, 0x08000000u | i);
                        if (!ok) break;
                        sum += part[slot * 128 + row];
                    }
                    ++part_turn;
                }
                if (half == 0 && key < s.kv) {
                    float got = sum;
                    if (m.in) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kOld - 1) : "memory");
                        got = fmaf(m.decay, old[(i >> 1) % kOld * 128], sum);
                    }
                    m.out[mass_row + key] = got;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // Given up: the CTA's shared memory stays until the copies in flight have landed.  Only here is it known: a role
    // may give up on a copy after its producer has done all of its work.
    if (*abort_flag) {
        if (warp == kWarpK || warp == kWarpK2)
            for (int n = max(0, place - kRing); n < place; ++n)
                mbar_wait_landing(&bar.k_full[n % kRing], (n / kRing) & 1);
        if (warp == kWarpQ)
            for (int n = max(0, place - kQ); n < place; ++n)
                mbar_wait_landing(&bar.q_full[n % kQ], (n / kQ) & 1);
    }
}

template <int D, int QR>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const MassParams& m, cudaStream_t stream) {
    using C = Cfg<D, QR>;
    static OncePerDevice once;
    const cudaError_t set = once([] {
        return cudaFuncSetAttribute(mass_tc_kernel<D, QR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (set != cudaSuccess) return set;
    return launch_overlapped(mass_tc_kernel<D, QR>, dim3(device_sm_count()), C::kThreads, C::kSmem, stream, q, k, m);
}

}  // namespace

cudaError_t launch_mass_tc(const MassArgs& a, cudaStream_t stream) {
    MassParams m{};
    m.p = a.p;
    const int G = a.p.G;
    // rows of a sequence on average: one chunk of 32, or chunks of 128 (1 x 16000 keys: 32 rows 10.0 us against 11.3,
    // 96 rows 16.1 against 13.2)
    const bool narrow = G <= 32 && static_cast<long long>(a.p.R) * G <= 32ll * a.p.n_seqs;
    m.rpt = (narrow ? 32 : 128) / G;
    m.q_bytes = m.rpt * G * 128;
    m.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
    m.decay = a.decay;
    m.lse = a.lse;
    m.in = a.in;
    m.out = a.out;
    m.cols = a.mass_cols;
    CUtensorMap tq, tk;
    // without rows nothing reads q: its map then describes some memory that exists
    if (!cache_q_map(&tq, a.p, a.p.R > 0 ? a.q : a.k, a.D, m.rpt) || !cache_page_map(&tk, a.p, a.k, a.D, kKT)) return cudaErrorInvalidValue;
    if (narrow) return a.D == 128 ? launch<128, 32>(tq, tk, m, stream) : launch<64, 32>(tq, tk, m, stream);
    return a.D == 128 ? launch<128, 128>(tq, tk, m, stream) : launch<64, 128>(tq, tk, m, stream);
}

unsigned read_clear_status_mass_tc(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_mass_tc_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_mass_tc_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
