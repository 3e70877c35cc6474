// cache_ops.cu -- upkeep of a paged cache: the choice of the keys that stay, moves
// of rows between pages, and the write of new rows.
#include <cooperative_groups.h>

#include "cache_batch.cuh"

namespace cg = cooperative_groups;

namespace ra {

static __device__ unsigned g_cache_ops_status[2];

namespace {

// 16 bytes that are read once; not moved up past grid_dependency_wait().
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 x;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
    return x;
}

// ---------------------------------------------------------------------------
// choice of the keys that stay
//
// The need-th largest mass is found by its bits, eight at a time from the top: a
// histogram of the next eight bits of the keys that share the bits found so far.
// A cluster of CTAs holds one (sequence, KV head), a warp consecutive masses of it, a
// lane an odd number of consecutive ones in registers, as ordered integers (loaded in
// order and turned over shared memory, whose banks an odd stride meets once each;
// longer rows are read again for every step).  The histograms of the CTAs are added up
// over distributed shared memory, 256 consecutive bytes of a CTA per half warp (eight
// CTAs' 64 bytes per warp instead: 21 -> 19 us for 8 rows of 131072 equal masses, which
// take all four steps).  A lane marks what stays of its masses in two bit masks; the
// counts of the lanes, warps and CTAs before it give its place, and a warp's positions
// go through a list in shared memory, so that they are written in order and together.
// What a step costs is latency: the barrier of the cluster, the remote reads, the search
// for the digit (by one warp: sixteen that each search for themselves get in each
// other's way, 24 us where one takes 20).  8 rows of 131072 masses: 16.2 us (19.4 with
// a mass per lane and two ballots for every 32 of them); 128 rows of 6144: 10.7 us (11.3).
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 17;                               // most masses of a lane, odd
constexpr int kSelSlice = kSelThreads * (kSelKeys - 1);    // of a CTA
constexpr int kSelStep = 32 * kSelKeys;                    // of a warp
constexpr int kSelSmem = kSelWarps * kSelStep * (sizeof(float) + sizeof(unsigned short));
constexpr int kBins = 256;
constexpr int kSelMaxCluster = 16;

// Monotone map of a mass to an unsigned integer: larger mass, larger integer; NaN below everything, -0 as 0.
__device__ __forceinline__ unsigned mass_key(float x) {
    if (x != x) return 0u;
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Bits [lo, hi) of a word, both clamped to [0, kSelKeys].
__device__ __forceinline__ unsigned bit_range(int lo, int hi) {
    lo = max(0, min(lo, kSelKeys));
    hi = max(lo, min(hi, kSelKeys));
    return ((1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// ROUNDS = 1: a CTA's slice is in its registers; 0: the slice is read again, a step of every warp at a time.
template <int ROUNDS>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const SelectArgs a) {
    __shared__ __align__(16) unsigned hist[2][kBins];  // of this CTA; two, so that one barrier a step is enough
    __shared__ __align__(16) unsigned total[4][kBins];  // of the cluster, in four parts
    __shared__ unsigned warp_sure[kSelWarps], warp_equal[kSelWarps];
    __shared__ unsigned sh_digit, sh_left, sh_all;
    __shared__ unsigned cta_counts[2];                 // read by the CTAs after this one
    extern __shared__ __align__(16) float sel_smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int size = cluster.num_blocks(), rank = cluster.block_rank();
    const int row = blockIdx.x / size, b = row / a.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dependency_wait();
    int kv = a.kv_lens[b];
    if (kv < 0 || kv > a.mass_cols) {
        if (tid == 0) cache_report(g_cache_ops_status, 0x0F000000u | static_cast<unsigned>(b & 0xFFFFFF));
        kv = 0;
    }
    const int count = min(kv, a.budget);
    const float* mass = a.mass + static_cast<long long>(row) * a.mass_cols;
    int* pos = a.positions + static_cast<long long>(row) * a.budget;
    float* kept = a.kept_mass ? a.kept_mass + static_cast<long long>(row) * a.kept_cols : nullptr;
    if (tid == 0 && rank == 0 && row % a.Hkv == 0) a.counts[b] = count;
    const int at = rank * kSelThreads + tid, stride = size * kSelThreads;
    for (int i = count + at; i < a.budget; i += stride) pos[i] = -1;
    if (kept)
        for (int i = count + at; i < a.kept_cols; i += stride) kept[i] = 0.f;
    if (kv <= a.budget) {  // everything stays
        for (int i = at; i < kv; i += stride) {
            pos[i] = i;
            if (kept) kept[i] = mass[i];
        }
        return;
    }
    // this warp's part [w0, w1): `nu` masses a lane and round, the same for every warp of the cluster
    const int share = (kv + stride - 1) / stride;
    const int nu = ROUNDS == 1 ? share | 1 : kSelKeys, step_keys = 32 * nu;
    const int rounds = ROUNDS ? ROUNDS : (share + kSelKeys - 1) / kSelKeys;
    const long long first = (static_cast<long long>(rank) * kSelWarps + warp) * rounds * step_keys;
    const int w0 = static_cast<int>(min(static_cast<long long>(kv), first));
    const int w1 = static_cast<int>(min(static_cast<long long>(kv), first + static_cast<long long>(rounds) * step_keys));
    // candidates: between the first and the recent ones; the `need` largest stay
    const int lo = a.n_first, hi = kv - a.n_recent;
    unsigned need = static_cast<unsigned>(a.budget - a.n_first - a.n_recent), prefix = 0;
    int low = 0;  // bits below the prefix
    float* const buf = sel_smem + warp * kSelStep;  // a step's masses
    unsigned short* const list = reinterpret_cast<unsigned short*>(sel_smem + kSelWarps * kSelStep) + warp * kSelStep;
    unsigned key[kSelKeys], inside = 0, live = 0;  // this lane's masses, those below w1, the candidates
    auto load = [&](int j0) {
        float x[kSelKeys];
#pragma unroll
        for (int u = 0; u < kSelKeys; ++u) {
            if (u >= nu) break;
            x[u] = j0 + u * 32 + lane < w1 ? mass[j0 + u * 32 + lane] : 0.f;
        }
        __syncwarp();  // the round before is done with the buffer
#pragma unroll
        for (int u = 0; u < kSelKeys; ++u) {
            if (u >= nu) break;
            buf[u * 32 + lane] = x[u];
        }
        __syncwarp();
        const int j = j0 + lane * nu;
#pragma unroll
        for (int u = 0; u < kSelKeys; ++u) {
            if (u >= nu) break;
            key[u] = mass_key(buf[lane * nu + u]);
        }
        const unsigned all = bit_range(0, nu);
        inside = all & bit_range(0, w1 - j);
        live = inside & bit_range(lo - j, hi - j);
    };
    if (tid < kBins) hist[0][tid] = 0;
    if (ROUNDS == 1) load(w0);
    __syncthreads();
    for (int step = 0, shift = 24; need > 0 && step < 4; ++step, shift -= 8) {
        for (int r = 0; r < rounds; ++r) {
            const int j0 = w0 + r * step_keys;
            if (j0 >= w1) break;
            if (ROUNDS != 1) load(j0);
#pragma unroll
            for (int u = 0; u < kSelKeys; ++u) {
                if (u >= nu) break;
                if (((live >> u) & 1u) && (step == 0 || (key[u] >> (shift + 8)) == prefix))
                    atomicAdd(&hist[step & 1][(key[u] >> shift) & 255], 1u);
            }
        }
        cluster.sync();
        {
            // half a warp reads 64 consecutive bins of a CTA; a warp's halves and the two turns add up in registers
            const int quad = (warp >> 2) * 16 + (lane & 15), from = (warp & 3) * 2 + (lane >> 4);
            uint4 n = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < kSelMaxCluster; r += 8) {
                if (r + from >= size) continue;
                const uint4 x = *cluster.map_shared_rank(reinterpret_cast<const uint4*>(hist[step & 1]) + quad, r + from);
                n = make_uint4(n.x + x.x, n.y + x.y, n.z + x.z, n.w + x.w);
            }
            const bool upper = lane & 16;  // each half keeps two of the four bins
            const unsigned u0 = (upper ? n.z : n.x) + __shfl_xor_sync(0xffffffffu, upper ? n.x : n.z, 16);
            const unsigned u1 = (upper ? n.w : n.y) + __shfl_xor_sync(0xffffffffu, upper ? n.y : n.w, 16);
            reinterpret_cast<uint2*>(total[warp & 3])[2 * quad + (lane >> 4)] = make_uint2(u0, u1);
            if (tid < kBins) hist[(step & 1) ^ 1][tid] = 0;  // read by everyone before this step's barrier
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: the bins 255 - 8 l .. 248 - 8 l, from the top; the first lane to reach `need` has the digit
            unsigned n[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                const uint4 t1 = reinterpret_cast<const uint4*>(total[part])[63 - 2 * lane];
                const uint4 t0 = reinterpret_cast<const uint4*>(total[part])[62 - 2 * lane];
                const unsigned t[8] = {t1.w, t1.z, t1.y, t1.x, t0.w, t0.z, t0.y, t0.x};
#pragma unroll
                for (int d = 0; d < 8; ++d) n[d] += t[d];
            }
            unsigned mine = 0;
#pragma unroll
            for (int d = 0; d < 8; ++d) mine += n[d];
            unsigned incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            unsigned left = need - (incl - mine), digit = 0;
            bool found = false, all = false;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                if (!found && n[d] >= left) {
                    found = true;
                    digit = 255 - 8 * lane - d;
                    all = n[d] == left;
                }
                left -= found ? 0 : n[d];
            }
            if (incl >= need && incl - mine < need) {
                sh_digit = digit;
                sh_left = left;
                sh_all = all;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | sh_digit;
        need = sh_left;
        low = shift;
        if (sh_all) break;  // all keys with this prefix stay: its lower bits decide nothing
    }
    // prefix: the top bits of the least mass that stays; `need` of the keys that share them do, the lowest positions
    const unsigned quota = need;
    auto mark = [&](unsigned& sure, unsigned& equal) {
        sure = equal = 0;
#pragma unroll
        for (int u = 0; u < kSelKeys; ++u) {
            if (u >= nu) break;
            const unsigned top = key[u] >> low;
            sure |= static_cast<unsigned>(top > prefix) << u;
            equal |= static_cast<unsigned>(top == prefix) << u;
        }
        sure = (quota > 0 ? sure & live : 0u) | (inside & ~live);
        equal = quota > 0 ? equal & live : 0u;
    };
    unsigned n_sure = 0, n_equal = 0, sure = 0, equal = 0;
    for (int r = 0; r < rounds; ++r) {
        const int j0 = w0 + r * step_keys;
        if (j0 >= w1) break;
        if (ROUNDS != 1) load(j0);
        mark(sure, equal);
        n_sure += __reduce_add_sync(0xffffffffu, __popc(sure));
        n_equal += __reduce_add_sync(0xffffffffu, __popc(equal));
    }
    if (lane == 0) {
        warp_sure[warp] = n_sure;
        warp_equal[warp] = n_equal;
    }
    __syncthreads();
    {
        const unsigned x = lane < kSelWarps ? warp_sure[lane] : 0, y = lane < kSelWarps ? warp_equal[lane] : 0;
        n_sure = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
        n_equal = __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
        if (warp == 0) {
            const unsigned cx = __reduce_add_sync(0xffffffffu, x), cy = __reduce_add_sync(0xffffffffu, y);
            if (lane == 0) {
                cta_counts[0] = cx;
                cta_counts[1] = cy;
            }
        }
    }
    cluster.sync();
    {
        // counts of the CTAs before this one: a lane each
        unsigned x = 0, y = 0;
        if (lane < rank) {
            const unsigned* c = cluster.map_shared_rank(cta_counts, lane);
            x = c[0];
            y = c[1];
        }
        n_sure += __reduce_add_sync(0xffffffffu, x);
        n_equal += __reduce_add_sync(0xffffffffu, y);
    }
    cluster.barrier_arrive();  // done with the other CTAs' counts
    for (int r = 0; r < rounds; ++r) {
        const int j0 = w0 + r * step_keys;
        if (j0 >= w1) break;
        if (ROUNDS != 1) {
            load(j0);
            mark(sure, equal);
        }
        const unsigned mine = __popc(sure) | static_cast<unsigned>(__popc(equal)) << 16;  // sums up to 544 each
        unsigned incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const unsigned before = incl - mine, step_all = __shfl_sync(0xffffffffu, incl, 31);
        const unsigned base = n_sure + min(n_equal, quota);
        const unsigned eq = n_equal + (before >> 16);  // keys equal to the least one before this lane's
        unsigned slot = n_sure + (before & 0xffffu) + min(eq, quota) - base;
        unsigned room = quota - min(eq, quota), out = sure | equal;
        while (out) {
            const unsigned bit = out & (0u - out);
            out ^= bit;
            if (equal & bit) {
                if (room == 0) continue;
                --room;
            }
            list[slot++] = static_cast<unsigned short>(lane * nu + __ffs(bit) - 1);
        }
        __syncwarp();
        n_sure += step_all & 0xffffu;
        n_equal += step_all >> 16;
        const int n = static_cast<int>(n_sure + min(n_equal, quota) - base);
        for (int i = lane; i < n; i += 32) {
            const int x = list[i];
            pos[base + i] = j0 + x;
            if (kept) kept[base + i] = buf[x];
        }
    }
    cluster.barrier_wait();  // the counts are read before their CTA goes
}

// ---------------------------------------------------------------------------
// moves between pages
// ---------------------------------------------------------------------------
// Byte offset of head h of the row of key j in a page list, -1 (and the status) if it is out of range.
__device__ __forceinline__ long long row_offset(const MoveArgs& a, const int* pages, int max_pages, int j, int h) {
    if (j < 0 || (j >> a.page_shift) >= max_pages) {
        cache_report(g_cache_ops_status, 0x0D000000u);
        return -1;
    }
    const int row = cache_row(pages, a.n_pages, a.page_shift, j, g_cache_ops_status);
    return row < 0 ? -1 : (static_cast<long long>(row) * a.Hkv + h) * a.row_bytes;
}

// The sequence's rows to move and the first slot they go to.
__device__ __forceinline__ int move_count(const MoveArgs& a, int b, int& start) {
    start = a.dst_start ? a.dst_start[b] : 0;
    const int n = a.counts[b];
    if (n < 0 || start < 0) {
        cache_report(g_cache_ops_status, 0x0F000000u | static_cast<unsigned>(b & 0xFFFFFF));
        return 0;
    }
    return min(n, a.max_count);
}

constexpr int kMoveThreads = 256;

// Into other pages.  A CTA takes kMoveRows slots of one sequence and head: a thread per slot finds where its row
// lies and goes, then all threads copy, kMoveDepth 16-byte pieces each in flight (one each: 89 us instead of 74 for
// 16 x 4096 kept keys of 8 heads, 5.7 TB/s).  Bound by the bytes of rows of 128 to 512 bytes.
constexpr int kMoveRows = 64;
constexpr int kMoveDepth = 8;

__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const MoveArgs a) {
    __shared__ long long from[kMoveRows], to[kMoveRows];
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x;
    grid_dependency_wait();
    int start;
    const int count = move_count(a, b, start);
    const int* pos = a.positions + (static_cast<long long>(b) * a.pos_heads + (a.pos_heads == 1 ? 0 : h)) * a.max_count;
    const int vecs = a.row_bytes / 16, shift = 31 - __clz(vecs);  // a power of two: 8, 16 or 32
    for (int i0 = blockIdx.y * kMoveRows; i0 < count; i0 += gridDim.y * kMoveRows) {
        __syncthreads();
        if (tid < kMoveRows) {
            long long src = -1, dst = -1;
            if (i0 + tid < count) {
                const long long slot = static_cast<long long>(start) + i0 + tid;
                src = row_offset(a, a.src_pages + static_cast<long long>(b) * a.src_max_pages, a.src_max_pages,
                                 pos[i0 + tid], h);
                dst = row_offset(a, a.dst_pages + static_cast<long long>(b) * a.dst_max_pages, a.dst_max_pages,
                                 slot > 0x7fffffffll ? -1 : static_cast<int>(slot), h);
            }
            from[tid] = dst < 0 ? -1 : src;
            to[tid] = dst;
        }
        __syncthreads();
        // pieces: (tensor, slot, 16 bytes of its row)
        const int pieces = 2 * kMoveRows << shift;
        for (int x0 = tid; x0 < pieces; x0 += kMoveThreads * kMoveDepth) {
            uint4 v[kMoveDepth];
#pragma unroll
            for (int u = 0; u < kMoveDepth; ++u) {
                const int x = x0 + u * kMoveThreads, i = (x >> shift) & (kMoveRows - 1);
                if (x < pieces && from[i] >= 0)
                    v[u] = load_once(static_cast<const char*>(x >> shift >= kMoveRows ? a.v : a.k) + from[i] +
                                     (x & (vecs - 1)) * 16);
            }
#pragma unroll
            for (int u = 0; u < kMoveDepth; ++u) {
                const int x = x0 + u * kMoveThreads, i = (x >> shift) & (kMoveRows - 1);
                if (x < pieces && from[i] >= 0)
                    *reinterpret_cast<uint4*>(static_cast<char*>(x >> shift >= kMoveRows ? a.v : a.k) + to[i] +
                                              (x & (vecs - 1)) * 16) = v[u];
            }
        }
    }
}

// In place: increasing positions at or past their slots.  One CTA walks the slots of one sequence, head and
// tensor in order, a step of rows at a time: all of a step's rows are read before any is written, and a
// later step's rows lie at or past its slots, which are past this step's.  Bound by the latency of a step, one in
// flight: paths of 8 rows in 32 sequences 2.4 us, 16 x 4096 kept keys of 8 heads 341 us (into other pages 86).
__global__ void __launch_bounds__(kMoveThreads) cache_move_inplace_kernel(const MoveArgs a) {
    const int vecs = a.row_bytes / 16, step = kMoveThreads / vecs;
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    char* pool = static_cast<char*>(blockIdx.y ? a.v : a.k);
    grid_dependency_wait();
    int start;
    const int count = move_count(a, b, start);
    const int* pos = a.positions + (static_cast<long long>(b) * a.pos_heads + (a.pos_heads == 1 ? 0 : h)) * a.max_count;
    const int* table = a.src_pages + static_cast<long long>(b) * a.src_max_pages;
    const int c = threadIdx.x % vecs * 16;
    for (int i0 = 0; i0 < count; i0 += step) {
        const int i = i0 + threadIdx.x / vecs;
        long long src = -1, dst = -1;
        if (i < count) {
            const long long slot = static_cast<long long>(start) + i;
            src = row_offset(a, table, a.src_max_pages, pos[i], h);
            dst = row_offset(a, table, a.src_max_pages, slot > 0x7fffffffll ? -1 : static_cast<int>(slot), h);
        }
        const bool go = src >= 0 && dst >= 0 && src != dst;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (go) x = *reinterpret_cast<const uint4*>(pool + src + c);
        __syncthreads();
        if (go) *reinterpret_cast<uint4*>(pool + dst + c) = x;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// new rows into the pages
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendDepth = 4;  // 16-byte pieces of each tensor a lane has in flight

// All heads of a token are contiguous on both sides: one warp copies a token's keys and values, both tensors'
// pieces in flight (4 x 8192 tokens of 8 heads: 33.6 us, 5.8 TB/s; 64 single tokens 3.6 us).
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const CacheBatch p, const char* k_rows,
                                                                      const char* v_rows, char* k, char* v,
                                                                      int token_bytes) {
    __shared__ RangeScratch<kAppendThreads> scratch;
    grid_dependency_wait();
    const WorkRange range =
        find_range<kAppendThreads>(p, kAppendThreads / 32, g_cache_ops_status, RowWeight{}, scratch);
    constexpr int kWarps = kAppendThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long a = range.a;  // weight before the sequence
    for (int b = range.b; b < p.n_seqs && a < range.hi; ++b) {
        CacheSeq s = range.s;
        if (b != range.b) load_seq(p, b, s);
        // the range's rows in turn, a warp each, whatever sequence they belong to
        const int t0 = static_cast<int>(max(0ll, range.lo - a));
        const int t1 = static_cast<int>(min(static_cast<long long>(s.n), range.hi - a));
        const int turn = static_cast<int>(a + t0 - range.lo) & (kWarps - 1);
        a += s.n;
        for (int t = t0 + ((warp - turn) & (kWarps - 1)); t < t1; t += kWarps) {
            const int j = s.kv - s.n + t;
            if (j < 0) continue;
            const int row = cache_row(p.pages + static_cast<long long>(b) * p.max_pages, p.n_pages, p.page_shift, j,
                                      g_cache_ops_status);
            if (row < 0) continue;
            const long long from = (static_cast<long long>(s.lo) + t) * token_bytes;
            const long long to = static_cast<long long>(row) * token_bytes;
            for (int c0 = lane * 16; c0 < token_bytes; c0 += 512 * kAppendDepth) {
                uint4 x[kAppendDepth], y[kAppendDepth];
#pragma unroll
                for (int u = 0; u < kAppendDepth; ++u)
                    if (c0 + 512 * u < token_bytes) {
                        x[u] = load_once(k_rows + from + c0 + 512 * u);
                        y[u] = load_once(v_rows + from + c0 + 512 * u);
                    }
#pragma unroll
                for (int u = 0; u < kAppendDepth; ++u)
                    if (c0 + 512 * u < token_bytes) {
                        *reinterpret_cast<uint4*>(k + to + c0 + 512 * u) = x[u];
                        *reinterpret_cast<uint4*>(v + to + c0 + 512 * u) = y[u];
                    }
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, cudaStream_t stream) {
    // CTAs of a row: at most two per SM in all, of at least 2048 masses each, more where the masses then fit the
    // registers
    const long long rows = static_cast<long long>(a.n_seqs) * a.Hkv;
    int size = 1;
    while (size < kSelMaxCluster && ((rows * size * 2 <= 2ll * device_sm_count() && a.mass_cols / (size * 2) >= 2048) ||
                                     a.mass_cols > static_cast<long long>(size) * kSelSlice))
        size *= 2;
    auto* kernel = a.mass_cols <= static_cast<long long>(size) * kSelSlice ? evict_select_kernel<1> : evict_select_kernel<0>;
    static OncePerDevice once;
    const cudaError_t set = once([] {
        for (auto* f : {evict_select_kernel<0>, evict_select_kernel<1>}) {
            cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);  // of sixteen
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmem);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    });
    if (set != cudaSuccess) return set;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * size));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = kSelSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_overlapped
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_cache_move(const MoveArgs& a, cudaStream_t stream) {
    const int rows = a.n_seqs * a.Hkv;
    if (a.src_pages == a.dst_pages)
        return launch_overlapped(cache_move_inplace_kernel, dim3(rows, 2), kMoveThreads, 0, stream, a);
    const long long blocks = (static_cast<long long>(a.max_count) + kMoveRows - 1) / kMoveRows;
    return launch_overlapped(cache_move_kernel, dim3(rows, static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), kMoveThreads,
                             0, stream, a);
}

cudaError_t launch_cache_append(const CacheBatch& p, const void* k_rows, const void* v_rows, void* k, void* v,
                                int row_bytes, cudaStream_t stream) {
    const int most = 8 * device_sm_count(), blocks = (p.R + 7) / 8 < most ? (p.R + 7) / 8 : most;
    return launch_overlapped(cache_append_kernel, dim3(blocks), kAppendThreads, 0, stream, p, static_cast<const char*>(k_rows),
                             static_cast<const char*>(v_rows), static_cast<char*>(k), static_cast<char*>(v), row_bytes * p.Hkv);
}

unsigned read_clear_status_cache_ops(unsigned* where) {
    unsigned h[2] = {0, 0};
    cudaMemcpyFromSymbol(h, g_cache_ops_status, sizeof h);
    if (h[0]) {
        const unsigned z[2] = {0, 0};
        cudaMemcpyToSymbol(g_cache_ops_status, z, sizeof z);
    }
    if (where) *where = h[1];
    return h[0];
}

}  // namespace ra
