// cache_ops.cu -- upkeep of a paged cache: the choice of the keys that stay, moves
// of rows between pages, and the write of new rows.
#include "cache_batch.cuh"

namespace ra {

static __device__ unsigned g_cache_ops_status[2];

namespace {

// ---------------------------------------------------------------------------
// choice of the keys that stay
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kBins = 256;

// Monotone map of a mass to an unsigned integer: larger mass, larger integer; NaN below everything, -0 as 0.
__device__ __forceinline__ unsigned mass_key(float x) {
    if (x != x) return 0u;
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ unsigned long long block_scan(unsigned long long mine, unsigned long long* warp_sum,
                                                         unsigned long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    unsigned long long before = incl - mine, sum = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        sum += warp_sum[w];
    }
    __syncthreads();
    *total = sum;
    return before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectArgs a) {
    __shared__ unsigned hist[kBins];
    __shared__ unsigned sh_prefix, sh_need;
    __shared__ unsigned long long warp_sum[kSelThreads / 32];
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x;
    int kv = a.kv_lens[b];
    if (kv < 0 || kv > a.mass_cols) {
        if (tid == 0) cache_report(g_cache_ops_status, 0x0F000000u | static_cast<unsigned>(b & 0xFFFFFF));
        kv = 0;
    }
    const int count = min(kv, a.budget);
    const float* mass = a.mass + static_cast<long long>(blockIdx.x) * a.mass_cols;
    int* pos = a.positions + static_cast<long long>(blockIdx.x) * a.budget;
    float* kept = a.kept_mass ? a.kept_mass + static_cast<long long>(blockIdx.x) * a.kept_cols : nullptr;
    if (tid == 0 && h == 0) a.counts[b] = count;
    for (int i = count + tid; i < a.budget; i += kSelThreads) pos[i] = -1;
    if (kept)
        for (int i = count + tid; i < a.kept_cols; i += kSelThreads) kept[i] = 0.f;
    // candidates: the keys [lo, hi) between the first and the recent ones; the `need` largest stay
    const bool all = kv <= a.budget;
    const int lo = all ? 0 : a.n_first, hi = all ? 0 : kv - a.n_recent;
    unsigned prefix = 0, need = all ? 0 : static_cast<unsigned>(a.budget - a.n_first - a.n_recent);
    if (need > 0) {
        // the need-th largest key, eight bits at a time from the top
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                const unsigned x = mass_key(mass[j]);
                if (shift == 24 || (x >> (shift + 8)) == prefix) atomicAdd(&hist[(x >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                unsigned left = need;
                int d = 255;
                for (; d > 0 && hist[d] < left; --d) left -= hist[d];
                sh_prefix = (prefix << 8) | static_cast<unsigned>(d);
                sh_need = left;
            }
            __syncthreads();
            prefix = sh_prefix;
            need = sh_need;
        }
    }
    // prefix: the least key that stays; `need` of those equal to it stay, the lowest positions
    const unsigned quota = need;
    unsigned long long done = 0;  // (kept for sure, equal to the threshold) so far, 32 bits each
    for (int j0 = 0; j0 < kv; j0 += kSelThreads) {
        const int j = j0 + tid;
        bool sure = false, equal = false;
        float x = 0.f;
        if (j < kv) {
            x = mass[j];
            if (all || j < lo || j >= hi) {
                sure = true;
            } else if (quota > 0) {
                const unsigned y = mass_key(x);
                sure = y > prefix;
                equal = y == prefix;
            }
        }
        unsigned long long total;
        const unsigned long long at =
            done + block_scan((sure ? 1ull : 0ull) | (equal ? 1ull << 32 : 0ull), warp_sum, &total);
        const unsigned n_sure = static_cast<unsigned>(at), n_equal = static_cast<unsigned>(at >> 32);
        if (sure || (equal && n_equal < quota)) {
            const unsigned slot = n_sure + min(n_equal, quota);
            pos[slot] = j;
            if (kept) kept[slot] = x;
        }
        done += total;
    }
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

// Into other pages: one thread per 16 bytes of a K row and the same of the V row.
__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const MoveArgs a) {
    const int vecs = a.row_bytes / 16;
    const long long per = static_cast<long long>(a.max_count) * vecs;
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    int start;
    const int count = move_count(a, b, start);
    const int* pos = a.positions + (static_cast<long long>(b) * a.pos_heads + (a.pos_heads == 1 ? 0 : h)) * a.max_count;
    for (long long x = static_cast<long long>(blockIdx.y) * kMoveThreads + threadIdx.x; x < per;
         x += static_cast<long long>(gridDim.y) * kMoveThreads) {
        const int i = static_cast<int>(x / vecs), c = static_cast<int>(x % vecs) * 16;
        if (i >= count) return;
        const long long src = row_offset(a, a.src_pages + static_cast<long long>(b) * a.src_max_pages, a.src_max_pages,
                                         pos[i], h);
        const long long slot = static_cast<long long>(start) + i;
        const long long dst = row_offset(a, a.dst_pages + static_cast<long long>(b) * a.dst_max_pages, a.dst_max_pages,
                                         slot > 0x7fffffffll ? -1 : static_cast<int>(slot), h);
        if (src < 0 || dst < 0) continue;
        *reinterpret_cast<uint4*>(static_cast<char*>(a.k) + dst + c) =
            *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + src + c);
        *reinterpret_cast<uint4*>(static_cast<char*>(a.v) + dst + c) =
            *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + src + c);
    }
}

// In place: increasing positions at or past their slots.  One CTA walks the slots of one sequence, head and
// tensor in order, a step of rows at a time: all of a step's rows are read before any is written, and a
// later step's rows lie at or past its slots, which are past this step's.
__global__ void __launch_bounds__(kMoveThreads) cache_move_inplace_kernel(const MoveArgs a) {
    const int vecs = a.row_bytes / 16, step = kMoveThreads / vecs;
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    char* pool = static_cast<char*>(blockIdx.y ? a.v : a.k);
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

// The rows of the batch, end to end, are cut into equal ranges over the CTAs.
struct RowWeight {
    __device__ __forceinline__ long long operator()(const CacheSeq& s) const { return s.n; }
};

// All heads of a token are contiguous on both sides: one warp copies a token's keys and values.
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const CacheBatch p, const char* k_rows,
                                                                      const char* v_rows, char* k, char* v,
                                                                      int token_bytes) {
    __shared__ RangeScratch<kAppendThreads> scratch;
    const WorkRange range =
        find_range<kAppendThreads>(p, kAppendThreads / 32, g_cache_ops_status, RowWeight{}, scratch);
    const int lane = threadIdx.x & 31;
    long long a = range.base;
    for (int b = range.b; b < p.n_seqs && a < range.hi; ++b) {
        CacheSeq s;
        load_seq(p, b, s);
        const int t0 = static_cast<int>(max(0ll, range.lo - a));
        const int t1 = static_cast<int>(min(static_cast<long long>(s.n), range.hi - a));
        a += s.n;
        for (int t = t0 + (threadIdx.x >> 5); t < t1; t += kAppendThreads / 32) {
            const int j = s.kv - s.n + t;
            if (j < 0) continue;
            const int row = cache_row(p.pages + static_cast<long long>(b) * p.max_pages, p.n_pages, p.page_shift, j,
                                      g_cache_ops_status);
            if (row < 0) continue;
            const long long from = (static_cast<long long>(s.lo) + t) * token_bytes;
            const long long to = static_cast<long long>(row) * token_bytes;
            for (int c = lane * 16; c < token_bytes; c += 512) {
                const uint4 x = *reinterpret_cast<const uint4*>(k_rows + from + c);
                const uint4 y = *reinterpret_cast<const uint4*>(v_rows + from + c);
                *reinterpret_cast<uint4*>(k + to + c) = x;
                *reinterpret_cast<uint4*>(v + to + c) = y;
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, cudaStream_t stream) {
    evict_select_kernel<<<a.n_seqs * a.Hkv, kSelThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_move(const MoveArgs& a, cudaStream_t stream) {
    const int rows = a.n_seqs * a.Hkv;
    if (a.src_pages == a.dst_pages) {
        cache_move_inplace_kernel<<<dim3(rows, 2), kMoveThreads, 0, stream>>>(a);
    } else {
        const long long blocks = (static_cast<long long>(a.max_count) * (a.row_bytes / 16) + kMoveThreads - 1) / kMoveThreads;
        cache_move_kernel<<<dim3(rows, static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), kMoveThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_cache_append(const CacheBatch& p, const void* k_rows, const void* v_rows, void* k, void* v,
                                int row_bytes, cudaStream_t stream) {
    const int most = 8 * device_sm_count(), blocks = (p.R + 7) / 8 < most ? (p.R + 7) / 8 : most;
    cache_append_kernel<<<blocks, kAppendThreads, 0, stream>>>(p, static_cast<const char*>(k_rows),
                                                               static_cast<const char*>(v_rows), static_cast<char*>(k),
                                                               static_cast<char*>(v), row_bytes * p.Hkv);
    return cudaGetLastError();
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
