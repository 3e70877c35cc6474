// cache_batch.cuh -- what the kernels over a batch of paged sequences share: the
// checked lengths of a sequence, page translation, and the cut of the batch's
// work into equal parts.
//
// Work of an attention call: units (sequence, KV head, row tile), in that order;
// a row tile is RT consecutive rows of the n_b * G (new token, head of the group)
// rows of one sequence and KV head (token slowest).  A unit walks the KT-key tiles its rows can
// see.  Its weight is its tiles plus OV, what starting and finishing a unit
// costs in tiles.  The weights of the batch, end to end, are cut into as many
// equal ranges as CTAs run; a CTA walks the units its range meets, of the first
// and the last possibly a part.  Every CTA derives its range from row_offsets and
// kv_lens by itself, so the launch needs no sizes but the stacked row count.
#pragma once

#include <atomic>

#include "mass_walk.h"
#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {

__device__ __forceinline__ void cache_report(unsigned* status, unsigned where) {
    atomicCAS(&status[0], 0u, kDevInvalidArg);
    atomicCAS(&status[1], 0u, where);
}

__device__ __forceinline__ bool load_seq(const CacheBatch& p, int b, CacheSeq& s) {
    // plain loads: a non-coherent one could be moved up past grid_dependency_wait()
    const int lo = p.row_offsets[b], hi = p.row_offsets[b + 1], kv = p.kv_lens[b];
    const bool ok = lo >= 0 && hi >= lo && hi <= p.R && (b > 0 || lo == 0) && (b < p.n_seqs - 1 || hi == p.R) &&
                    kv >= 0 && kv <= p.max_keys;
    s.lo = lo;
    s.n = ok ? hi - lo : 0;
    s.kv = ok ? kv : 0;
    return ok;
}

// Set-up of a kernel that each device needs once (its attributes belong to a device's context).
class OncePerDevice {
    std::atomic<unsigned long long> done_{0};

  public:
    template <class F>
    cudaError_t operator()(F set_up) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = set_up();
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Launch that may be scheduled while the kernel before it on the stream drains: the kernel calls
// grid_dependency_wait() before its first access to global memory.  Its pointers carry no __restrict__: that would
// allow non-coherent loads of what the kernel before may still be writing.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(KArgs...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                              const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// One lane of a fully active warp; unlike a test of the lane number it tells the compiler that one thread is
// left, which then issues MMAs without a loop over lanes (30 against 90 cycles each).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Loads a key tile in boxes of `sub_rows` rows and 64 columns (whole warp): lane g holds the pool row of group g.
// A lane issues a box, CHUNKS of them next to each other.  The lanes take turns at some 100 cycles a box (one
// elected lane that issues them all measured 115), so small pages want several warps.
template <int CHUNKS>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int chunk_stride,
                                          int groups, int sub_rows, int head, int row, int first_chunk = 0) {
    const int lane = threadIdx.x & 31, g = lane / CHUNKS, c = first_chunk + lane % CHUNKS;
    const int r = __shfl_sync(0xffffffffu, row, g);
    if (g < groups) tma_load_4d(map, bar, dst + c * chunk_stride + g * sub_rows * 128, c * 64, head, r, 0);
}

// mbar_wait of a whole warp: gives up together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* status,
                                          unsigned where) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, where));
}

// Row of the page pool that holds key j of sequence b, -1 (and the status) if its page is out of range.
__device__ __forceinline__ int cache_row(const int* pages, int n_pages, int page_shift, int j, unsigned* status) {
    const int lp = j >> page_shift;
    const int pg = pages[lp];
    if (pg < 0 || pg >= n_pages) {
        cache_report(status, 0x0E000000u | static_cast<unsigned>(lp & 0xFFFFFF));
        return -1;
    }
    return (pg << page_shift) + (j - (lp << page_shift));
}

// Keys the tokens 0 .. t of a sequence can see together: all of them under a tree mask.
__device__ __forceinline__ int visible_keys(const CacheSeq& s, bool tree, int t) {
    return tree ? s.kv : max(0, s.kv - s.n + t + 1);
}

template <int KT>
__device__ __forceinline__ int unit_tiles(const CacheSeq& s, int G, bool tree, int rt, int RT) {
    const int last = min(s.n * G, (rt + 1) * RT) - 1;
    return (visible_keys(s, tree, last / G) + KT - 1) / KT;
}

// Weight of one KV head of a sequence.
template <int KT, int OV>
__device__ __forceinline__ long long head_weight(const CacheSeq& s, int G, bool tree, int RT) {
    const int nrt = (s.n * G + RT - 1) / RT;
    if (tree || nrt == 1) return static_cast<long long>(nrt) * ((visible_keys(s, tree, s.n - 1) + KT - 1) / KT + OV);
    long long w = 0;
    for (int rt = 0; rt < nrt; ++rt) w += unit_tiles<KT>(s, G, tree, rt, RT) + OV;
    return w;
}

// A CTA's range of the batch's weight and where it starts.
struct WorkRange {
    long long lo, hi;
    long long q;     // weight of a range; the first `rem` ranges hold one more
    int rem;
    int b;           // sequence that holds `lo` (n_seqs: nothing to do)
    CacheSeq s;      // that sequence
    long long a;     // weight before the unit of work the walk starts with: unit `idx` of KV head `head`
    int head, idx;
};

// One segment: the part of a unit that falls into the CTA's range.
struct Segment {
    CacheSeq s;
    int b, head, rt;
    int tiles, t0, t1;      // key tiles of the unit, of the segment
    long long a;            // weight before the unit
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Prelude, called by every thread of the CTA: sums the sequences' weights over the batch and finds the
// CTA's range.  At least `min_w` of weight per CTA, so that short work runs on fewer CTAs.
// weight.head() is the weight of one of a sequence's weight.heads KV heads; weight.locate() says with
// which unit of its sequence a range starts.  What is found is handed on with its sequence and nothing is
// computed twice (2000 cycles of 4200 in the search for the unit alone: one decode over 1000 keys 10.9 ->
// 10.2 us).  The range stays in shared memory, for loops that need all of their registers; others copy it
// (one appended token per sequence 3.55 us with a copy, 3.9 without).
template <int THREADS>
struct RangeScratch {
    long long warp_sum[THREADS / 32];
    WorkRange found;
};
// The CTAs of a grid may walk several batches side by side (columns of KV heads): `which` of the `ranges` is this CTA's.
template <int THREADS, class Weight>
__device__ const WorkRange& find_range(const CacheBatch& p, int min_w, unsigned* status, Weight weight,
                                       RangeScratch<THREADS>& sh, int which, int ranges) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int per = (p.n_seqs + THREADS - 1) / THREADS;
    const int b0 = min(p.n_seqs, tid * per), b1 = min(p.n_seqs, b0 + per);
    long long mine = 0, wh = 0;
    CacheSeq s{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        if (load_seq(p, b, s))
            mine += (wh = weight.head(s)) * weight.heads;
        else if (blockIdx.x == 0)
            cache_report(status, 0x0F000000u | static_cast<unsigned>(b & 0xFFFFFF));
    }
    long long incl = mine;
    if ((tid - lane) * per < p.n_seqs) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
    }
    if (lane == 31) sh.warp_sum[tid >> 5] = incl;
    if (tid == 0) sh.found.b = p.n_seqs;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < (tid >> 5)) before += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    // equal ranges: CTA c starts at c q + min(c, rem)
    const int active = static_cast<int>(min(static_cast<long long>(ranges), max(1ll, quotient(total, min_w))));
    const long long q = quotient(total, active);
    const int rem = static_cast<int>(total - q * active);
    const int c = which;
    const long long lo = c < active ? c * q + min(c, rem) : total;
    const long long hi = c < active ? lo + q + (c < rem ? 1 : 0) : total;
    if (lo < hi && lo >= before && lo < before + mine) {
        for (int b = b0; b < b1; ++b) {
            if (per > 1) {  // else s and wh are those of this sequence
                load_seq(p, b, s);
                wh = weight.head(s);
            }
            const long long w = wh * weight.heads;
            if (lo < before + w) {
                WorkRange r{lo, hi, q, rem, b, s, 0, 0, 0};
                r.a = before + weight.locate(s, wh, lo - before, r.head, r.idx);
                sh.found = r;
                break;
            }
            before += w;
        }
    }
    __syncthreads();
    return sh.found;
}
template <int THREADS, class Weight>
__device__ __forceinline__ const WorkRange& find_range(const CacheBatch& p, int min_w, unsigned* status, Weight weight,
                                                       RangeScratch<THREADS>& sh) {
    return find_range<THREADS>(p, min_w, status, weight, sh, blockIdx.x, gridDim.x);
}

// Rows of new tokens: those of the batch, end to end, are cut into equal ranges over the CTAs.
struct RowWeight {
    static constexpr int heads = 1;
    __device__ __forceinline__ long long head(const CacheSeq& s) const { return s.n; }
    __device__ __forceinline__ long long locate(const CacheSeq&, long long, long long, int&, int&) const { return 0; }
};

template <int KT, int OV>
struct TreeWeight {
    int G, heads;
    bool tree;
    int RT;
    __device__ __forceinline__ long long head(const CacheSeq& s) const {
        return s.n ? head_weight<KT, OV>(s, G, tree, RT) : 0;
    }
    // The row tile that holds weight x of the sequence, and the weight before it.
    __device__ __forceinline__ long long locate(const CacheSeq& s, long long wh, long long x, int& head, int& rt) const {
        head = static_cast<int>(quotient(x, wh));
        long long a = wh * head;
        for (rt = 0;; ++rt) {
            const int w = unit_tiles<KT>(s, G, tree, rt, RT) + OV;
            if (x < a + w) return a;
            a += w;
        }
    }
};

// Walk over the non-empty segments of a range; every role of a CTA runs its own copy.  Of the KV heads it covers
// `heads_`, from head0 on (those past the last have no segments).
template <int KT, int OV>
struct SegmentWalk {
    CacheSeq s;
    int b, head, rt, nrt, RT, heads, head0;
    long long a;
    __device__ __forceinline__ void start(const CacheBatch& p, const WorkRange& r, int row_tile) {
        start(p, r, row_tile, p.Hkv, 0);
    }
    __device__ __forceinline__ void start(const CacheBatch& p, const WorkRange& r, int row_tile, int heads_, int first_head) {
        RT = row_tile;
        heads = heads_;
        head0 = first_head;
        b = r.b;
        head = r.head;
        rt = r.idx;
        a = r.a;
        if (b >= p.n_seqs) return;
        const volatile CacheSeq& first = r.s;  // read once, here: a copy the compiler may repeat cost spills
        s.lo = first.lo;
        s.n = first.n;
        s.kv = first.kv;
        nrt = (s.n * p.G + RT - 1) / RT;
    }
    // Next non-empty segment; false at the end of the range.
    __device__ __forceinline__ bool next(const CacheBatch& p, const WorkRange& r, Segment& g) {
        const bool tree = p.tree_mask != nullptr;
        while (b < p.n_seqs && a < r.hi) {
            const int tiles = unit_tiles<KT>(s, p.G, tree, rt, RT);
            g.s = s;
            g.b = b;
            g.head = head0 + head;
            g.rt = rt;
            g.tiles = tiles;
            g.a = a;
            g.t0 = static_cast<int>(max(0ll, r.lo - a - OV));
            g.t1 = static_cast<int>(max(0ll, min(static_cast<long long>(tiles), r.hi - a - OV)));
            const bool take = (tiles == 0 ? r.lo <= a : g.t1 > g.t0) && g.head < p.Hkv;
            a += tiles + OV;
            if (++rt == nrt) {
                rt = 0;
                if (++head == heads) {
                    head = 0;
                    do {
                        if (++b >= p.n_seqs) break;
                        load_seq(p, b, s);
                    } while (!s.n);
                    nrt = (s.n * p.G + RT - 1) / RT;
                }
            }
            if (take) return true;
        }
        return false;
    }
};

// Partials of a cut unit.  CTA c writes the part that continues a unit cut before
// it to slot 2c, the part that opens a unit cut inside its range to slot 2c + 1,
// and describes that unit's join in job c: the parts are slot 2c + 1 and the slots
// 2c', c < c' <= last.  A slot holds (m, l) of its rows, and O as [D / 4][rows][4]:
// threads that own a row each write, and the join reads, consecutive 16-byte pieces.
struct JoinJob {
    int row0;     // first of the unit's rows (flattened over the group) ...
    int rows;     // ... and their number; 0: nothing to join
    int seq_lo;   // stacked row of the sequence's first new token
    int head;
    int last;     // CTA with the unit's last part
    int pad[3];
};

__device__ __forceinline__ int partial_slot(const Segment& g, int cta) { return 2 * cta + (g.t0 > 0 ? 0 : 1); }
__device__ __forceinline__ int partial_slot(const Segment& g) { return partial_slot(g, static_cast<int>(blockIdx.x)); }

constexpr float kLn2 = 0.69314718055994531f;

// lse of a row from its reference (log2 units) and the sum relative to it: -inf where it saw no key, and NaN where the
// sum is one, as its output is; -inf there would take a row that is not a number out of a merge by lse.
__device__ __forceinline__ float row_lse(float m, float sum) {
    return sum > 0.f ? (m + log2f(sum)) * kLn2 : sum == 0.f ? -INFINITY : NAN;
}

// CTA whose range holds weight position x.
__device__ __forceinline__ int owner_of(const WorkRange& r, long long x) {
    const long long cut = r.rem * (r.q + 1);
    return static_cast<int>(x < cut ? quotient(x, r.q + 1) : r.rem + quotient(x - cut, r.q));
}

}  // namespace ra
