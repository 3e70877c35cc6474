// ra_cache_api.cu -- the C ABI's operators over a batch of paged sequences: host-side
// validation and dispatch.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/ra.h"
#include "ra_internal.h"

namespace {

std::atomic<bool> g_used{false}, g_q8_used{false};

template <typename... A>
ra_status fail(ra_status st, const char* fmt, A... a) {
    return static_cast<ra_status>(ra::set_error(st, fmt, a...));
}

ra_status ok() { return static_cast<ra_status>(ra::set_error(RA_OK, "")); }

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The launch of an operator; from the first one on ra_device_status reads their status words too.
template <typename F>
ra_status launched(const char* what, F launch, std::atomic<bool>& used = g_used) {
    used.store(true, std::memory_order_release);
    const cudaError_t e = launch();
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return ok();
}

constexpr long long kMaxRow = 0x7fffffffll;
constexpr int kMaxCount = 1 << 30;   // rows a call counts with an int, with room for a step past the last
constexpr int kMaxSeqs = 1 << 24;

ra_status check_pool(const void* k_pages, const void* v_pages, int n_pages, int page_size, int Hkv, int D, ra_dtype dt,
                     bool need_v, int* shift) {
    if (dt != RA_BF16 && dt != RA_F32) return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dt));
    if (D != 64 && D != 128) return fail(RA_ERR_INVALID_ARG, "D must be 64 or 128 (got %d)", D);
    if (Hkv < 1) return fail(RA_ERR_INVALID_ARG, "Hkv must be >= 1");
    if (page_size < 8 || page_size > (1 << 20) || (page_size & (page_size - 1)))
        return fail(RA_ERR_INVALID_ARG, "page_size must be a power of two in [8, 2^20] (got %d)", page_size);
    if (n_pages < 1) return fail(RA_ERR_INVALID_ARG, "n_pages must be >= 1");
    if (static_cast<long long>(n_pages) * page_size > kMaxRow)
        return fail(RA_ERR_INVALID_ARG, "page pool of more than 2^31 - 1 rows");
    if (!k_pages || (need_v && !v_pages)) return fail(RA_ERR_INVALID_ARG, "null page pool");
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    *shift = 0;
    while ((1 << *shift) < page_size) ++*shift;
    return RA_OK;
}

// The same for an 8-bit cache, whose rows outside it have dtype dt.
ra_status check_q8_pools(const void* k_pages, const void* v_pages, const unsigned char* k_scales, const unsigned char* v_scales,
                         int n_pages, int page_size, int Hkv, int D, ra_dtype dt, int* shift) {
    const ra_status st = check_pool(k_pages, v_pages, n_pages, page_size, Hkv, D, dt, true, shift);
    if (st != RA_OK) return st;
    if (!k_scales || !v_scales) return fail(RA_ERR_INVALID_ARG, "null scales");
    if (!aligned(k_scales, 16) || !aligned(v_scales, 16))
        return fail(RA_ERR_INVALID_ARG, "scales must be 16-byte aligned");
    return RA_OK;
}

ra::Q8Pools q8_pools(const void* k, const void* v, const unsigned char* ks, const unsigned char* vs) {
    auto bytes = [](const void* p) { return static_cast<unsigned char*>(const_cast<void*>(p)); };
    return {bytes(k), bytes(v), bytes(ks), bytes(vs)};
}

// Longest length a page list holds (kept clear of int overflow when rounded up to a tile).
int list_keys(int max_pages, int page_size) {
    const long long n = static_cast<long long>(max_pages) * page_size;
    return static_cast<int>(n < kMaxRow - 1024 ? n : kMaxRow - 1024);
}

ra_status check_batch(const int* row_offsets, int n_seqs, int R, const int* pages, int max_pages, const int* kv_lens) {
    if (n_seqs < 1 || R < 0 || max_pages < 1)
        return fail(RA_ERR_INVALID_ARG, "n_seqs >= 1, R >= 0, max_pages >= 1 required");
    if (n_seqs > kMaxSeqs || R > kMaxCount) return fail(RA_ERR_INVALID_ARG, "n_seqs > 2^24 or R > 2^30");
    if (!row_offsets || !pages || !kv_lens) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(row_offsets, 4) || !aligned(pages, 4) || !aligned(kv_lens, 4))
        return fail(RA_ERR_INVALID_ARG, "offsets, page lists and lengths must be 4-byte aligned");
    return RA_OK;
}

ra_status check_heads(int R, int Hq, int Hkv) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv) return fail(RA_ERR_INVALID_ARG, "Hq must be a positive multiple of Hkv");
    if (Hq / Hkv > 128) return fail(RA_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
    if (static_cast<long long>(R) * Hq > kMaxRow - 1024) return fail(RA_ERR_INVALID_ARG, "R * Hq too large");
    return RA_OK;
}

ra_status check_mask(const unsigned char* tree_mask, int mask_cols) {
    if (tree_mask && mask_cols < 1) return fail(RA_ERR_INVALID_ARG, "mask_cols must be >= 1 with a tree mask");
    return RA_OK;
}

ra::CacheBatch batch(const int* row_offsets, int n_seqs, int R, int n_pages, int shift, const int* pages, int max_pages,
                     const int* kv_lens, const unsigned char* tree_mask, int mask_cols, int Hq, int Hkv) {
    ra::CacheBatch p{};
    p.row_offsets = row_offsets;
    p.kv_lens = kv_lens;
    p.pages = pages;
    p.tree_mask = tree_mask;
    p.n_seqs = n_seqs;
    p.R = R;
    p.max_pages = max_pages;
    p.max_keys = list_keys(max_pages, 1 << shift);
    p.page_shift = shift;
    p.n_pages = n_pages;
    p.mask_cols = tree_mask ? mask_cols : 0;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    return p;
}

}  // namespace

bool ra::cache_used() { return g_used.load(std::memory_order_acquire); }
bool ra::cache_q8_used() { return g_q8_used.load(std::memory_order_acquire); }

extern "C" {

size_t ra_tree_attn_workspace_size(int R, int n_seqs, int Hq, int Hkv, int D, ra_dtype dt) {
    if (R < 0 || n_seqs < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 128 || (D != 64 && D != 128) ||
        (dt != RA_BF16 && dt != RA_F32) || n_seqs > kMaxSeqs || static_cast<long long>(R) * Hq > kMaxRow - 1024)
        return 0;
    if (dt == RA_BF16) return ra::tree_tc_workspace(R, n_seqs, Hq / Hkv, D).bytes;
    return ra::tree_simt_workspace(R, Hq / Hkv, D).bytes;
}

ra_status ra_tree_attn_paged(const void* q_rows, const int* row_offsets, int n_seqs, int R, const void* k_pages,
                             const void* v_pages, int n_pages, int page_size, const int* pages, int max_pages,
                             const int* kv_lens, const unsigned char* tree_mask, int mask_cols, void* out, float* lse,
                             int Hq, int Hkv, int D, ra_dtype dt, void* workspace, size_t workspace_bytes,
                             void* stream) {
    int shift;
    ra_status st = check_pool(k_pages, v_pages, n_pages, page_size, Hkv, D, dt, true, &shift);
    if (st == RA_OK) st = check_batch(row_offsets, n_seqs, R, pages, max_pages, kv_lens);
    if (st == RA_OK) st = check_heads(R, Hq, Hkv);
    if (st == RA_OK) st = check_mask(tree_mask, mask_cols);
    if (st != RA_OK) return st;
    if (R == 0) return ok();
    if (!q_rows || !out) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(q_rows, 16) || !aligned(out, 16) || !aligned(lse, 4))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!workspace) return fail(RA_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, 256)) return fail(RA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    const size_t need = ra_tree_attn_workspace_size(R, n_seqs, Hq, Hkv, D, dt);
    if (workspace_bytes < need)
        return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    ra::TreeArgs a{};
    a.p = batch(row_offsets, n_seqs, R, n_pages, shift, pages, max_pages, kv_lens, tree_mask, mask_cols, Hq, Hkv);
    a.q = q_rows;
    a.k = k_pages;
    a.v = v_pages;
    a.out = out;
    a.lse = lse;
    a.D = D;
    a.ws = workspace;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched("tree attention", [&] { return dt == RA_BF16 ? ra::launch_tree_tc(a, s) : ra::launch_tree_simt(a, s); });
}

ra_status ra_key_mass_paged(const void* q_rows, const float* lse, const int* row_offsets, int n_seqs, int R,
                            const void* k_pages, int n_pages, int page_size, const int* pages, int max_pages,
                            const int* kv_lens, const unsigned char* tree_mask, int mask_cols, const float* mass_in,
                            float* mass_out, int mass_cols, float decay, int Hq, int Hkv, int D, ra_dtype dt,
                            void* stream) {
    int shift;
    ra_status st = check_pool(k_pages, nullptr, n_pages, page_size, Hkv, D, dt, false, &shift);
    if (st == RA_OK) st = check_batch(row_offsets, n_seqs, R, pages, max_pages, kv_lens);
    if (st == RA_OK) st = check_heads(R, Hq, Hkv);
    if (st == RA_OK) st = check_mask(tree_mask, mask_cols);
    if (st != RA_OK) return st;
    if (mass_cols < 1) return fail(RA_ERR_INVALID_ARG, "mass_cols must be >= 1");
    if (!std::isfinite(decay)) return fail(RA_ERR_INVALID_ARG, "decay must be finite");
    if (!mass_out || (R > 0 && (!q_rows || !lse))) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(q_rows, 16) || !aligned(lse, 4) || !aligned(mass_in, 4) || !aligned(mass_out, 4))
        return fail(RA_ERR_INVALID_ARG, "misaligned tensor pointer");
    ra::MassArgs a{};
    a.p = batch(row_offsets, n_seqs, R, n_pages, shift, pages, max_pages, kv_lens, tree_mask, mask_cols, Hq, Hkv);
    if (mass_cols < a.p.max_keys) a.p.max_keys = mass_cols;
    a.q = q_rows;
    a.k = k_pages;
    a.lse = lse;
    a.in = mass_in;
    a.out = mass_out;
    a.mass_cols = mass_cols;
    a.D = D;
    a.decay = decay;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched("key mass", [&] { return dt == RA_BF16 ? ra::launch_mass_tc(a, s) : ra::launch_mass_simt(a, s); });
}

ra_status ra_evict_select(const float* mass, int mass_cols, const int* kv_lens, int n_seqs, int Hkv, int budget,
                          int n_first, int n_recent, int* positions, int* counts, float* kept_mass, int kept_cols,
                          void* stream) {
    if (n_seqs < 1 || Hkv < 1 || mass_cols < 1 || budget < 1)
        return fail(RA_ERR_INVALID_ARG, "n_seqs, Hkv, mass_cols, budget must be >= 1");
    if (static_cast<long long>(n_seqs) * Hkv > kMaxRow / 16) return fail(RA_ERR_INVALID_ARG, "n_seqs * Hkv too large");
    if (n_first < 0 || n_recent < 0 || static_cast<long long>(n_first) + n_recent > budget)
        return fail(RA_ERR_INVALID_ARG, "n_first and n_recent must be >= 0 and at most budget together");
    if (mass_cols > kMaxCount || budget > kMaxCount || (kept_mass && kept_cols > kMaxCount))
        return fail(RA_ERR_INVALID_ARG, "mass_cols, budget and kept_cols must be at most 2^30");
    if (kept_mass && kept_cols < budget) return fail(RA_ERR_INVALID_ARG, "kept_cols (%d) < budget (%d)", kept_cols, budget);
    if (!mass || !kv_lens || !positions || !counts) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(mass, 4) || !aligned(kv_lens, 4) || !aligned(positions, 4) || !aligned(counts, 4) ||
        !aligned(kept_mass, 4))
        return fail(RA_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
    if (kept_mass == mass) return fail(RA_ERR_INVALID_ARG, "kept_mass must not be mass");
    ra::SelectArgs a{mass,   mass_cols, kv_lens,   n_seqs, Hkv,       budget,
                     n_first, n_recent,  positions, counts, kept_mass, kept_mass ? kept_cols : 0};
    return launched("eviction choice", [&] { return ra::launch_evict_select(a, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_cache_move_paged(void* k_pages, void* v_pages, int n_pages, int page_size, const int* src_pages,
                              int src_max_pages, const int* dst_pages, int dst_max_pages, const int* positions,
                              int pos_heads, int max_count, const int* counts, const int* dst_start, int n_seqs,
                              int Hkv, int D, ra_dtype dt, void* stream) {
    int shift;
    ra_status st = check_pool(k_pages, v_pages, n_pages, page_size, Hkv, D, dt, true, &shift);
    if (st != RA_OK) return st;
    if (n_seqs < 1 || src_max_pages < 1 || dst_max_pages < 1 || max_count < 0)
        return fail(RA_ERR_INVALID_ARG, "n_seqs, src_max_pages, dst_max_pages >= 1, max_count >= 0 required");
    if (pos_heads != 1 && pos_heads != Hkv) return fail(RA_ERR_INVALID_ARG, "pos_heads must be 1 or Hkv (got %d)", pos_heads);
    if (static_cast<long long>(n_seqs) * Hkv > kMaxRow) return fail(RA_ERR_INVALID_ARG, "n_seqs * Hkv too large");
    if (max_count > kMaxCount) return fail(RA_ERR_INVALID_ARG, "max_count must be at most 2^30");
    if (max_count == 0) return ok();
    if (!src_pages || !dst_pages || !positions || !counts) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (src_pages == dst_pages && src_max_pages != dst_max_pages)
        return fail(RA_ERR_INVALID_ARG, "one page list with two lengths");
    if (!aligned(src_pages, 4) || !aligned(dst_pages, 4) || !aligned(positions, 4) || !aligned(counts, 4) ||
        !aligned(dst_start, 4))
        return fail(RA_ERR_INVALID_ARG, "page lists, positions and counts must be 4-byte aligned");
    ra::MoveArgs a{k_pages,   v_pages,   n_pages,  shift,  src_pages, src_max_pages, dst_pages, dst_max_pages,
                   positions, pos_heads, max_count, counts, dst_start, n_seqs,        Hkv,
                   D * (dt == RA_BF16 ? 2 : 4)};
    return launched("cache move", [&] { return ra::launch_cache_move(a, static_cast<cudaStream_t>(stream)); });
}

ra_status ra_cache_append_paged(const void* k_rows, const void* v_rows, const int* row_offsets, int n_seqs, int R,
                                void* k_pages, void* v_pages, int n_pages, int page_size, const int* pages,
                                int max_pages, const int* kv_lens, int Hkv, int D, ra_dtype dt, void* stream) {
    int shift;
    ra_status st = check_pool(k_pages, v_pages, n_pages, page_size, Hkv, D, dt, true, &shift);
    if (st == RA_OK) st = check_batch(row_offsets, n_seqs, R, pages, max_pages, kv_lens);
    if (st != RA_OK) return st;
    const int row_bytes = D * (dt == RA_BF16 ? 2 : 4);
    if (static_cast<long long>(row_bytes) * Hkv > (1 << 20)) return fail(RA_ERR_INVALID_ARG, "Hkv too large");
    if (R == 0) return ok();
    if (!k_rows || !v_rows) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(k_rows, 16) || !aligned(v_rows, 16))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const ra::CacheBatch p = batch(row_offsets, n_seqs, R, n_pages, shift, pages, max_pages, kv_lens, nullptr, 0, Hkv, Hkv);
    return launched("cache append", [&] {
        return ra::launch_cache_append(p, k_rows, v_rows, k_pages, v_pages, row_bytes, static_cast<cudaStream_t>(stream));
    });
}

ra_status ra_cache_append_paged_q8(const void* k_rows, const void* v_rows, const int* row_offsets, int n_seqs, int R,
                                   void* k_pages, void* v_pages, unsigned char* k_scales, unsigned char* v_scales, int n_pages,
                                   int page_size, const int* pages, int max_pages, const int* kv_lens, int Hkv, int D,
                                   ra_dtype dt, void* stream) {
    int shift;
    ra_status st = check_q8_pools(k_pages, v_pages, k_scales, v_scales, n_pages, page_size, Hkv, D, dt, &shift);
    if (st == RA_OK) st = check_batch(row_offsets, n_seqs, R, pages, max_pages, kv_lens);
    if (st != RA_OK) return st;
    if (Hkv > (1 << 16)) return fail(RA_ERR_INVALID_ARG, "Hkv too large");
    if (R == 0) return ok();
    if (!k_rows || !v_rows) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(k_rows, 16) || !aligned(v_rows, 16))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const ra::CacheBatch p = batch(row_offsets, n_seqs, R, n_pages, shift, pages, max_pages, kv_lens, nullptr, 0, Hkv, Hkv);
    return launched("8-bit cache append", [&] {
        return ra::launch_append_q8(p, k_rows, v_rows, q8_pools(k_pages, v_pages, k_scales, v_scales), D, dt == RA_BF16,
                                    static_cast<cudaStream_t>(stream));
    }, g_q8_used);
}

ra_status ra_cache_read_paged_q8(const int* row_offsets, int n_seqs, int R, const void* k_pages, const void* v_pages,
                                 const unsigned char* k_scales, const unsigned char* v_scales, int n_pages, int page_size,
                                 const int* pages, int max_pages, const int* kv_lens, void* k_rows, void* v_rows, int Hkv,
                                 int D, ra_dtype dt, void* stream) {
    int shift;
    ra_status st = check_q8_pools(k_pages, v_pages, k_scales, v_scales, n_pages, page_size, Hkv, D, dt, &shift);
    if (st == RA_OK) st = check_batch(row_offsets, n_seqs, R, pages, max_pages, kv_lens);
    if (st != RA_OK) return st;
    if (Hkv > (1 << 16)) return fail(RA_ERR_INVALID_ARG, "Hkv too large");
    if (R == 0) return ok();
    if (!k_rows || !v_rows) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(k_rows, 16) || !aligned(v_rows, 16))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const ra::CacheBatch p = batch(row_offsets, n_seqs, R, n_pages, shift, pages, max_pages, kv_lens, nullptr, 0, Hkv, Hkv);
    return launched("8-bit cache read", [&] {
        return ra::launch_read_q8(p, q8_pools(k_pages, v_pages, k_scales, v_scales), k_rows, v_rows, D, dt == RA_BF16,
                                  static_cast<cudaStream_t>(stream));
    }, g_q8_used);
}

size_t ra_tree_attn_q8_workspace_size(int R, int n_seqs, int Hq, int Hkv, int D, ra_dtype dt) {
    if (R < 0 || n_seqs < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 128 || (D != 64 && D != 128) ||
        (dt != RA_BF16 && dt != RA_F32) || n_seqs > kMaxSeqs || static_cast<long long>(R) * Hq > kMaxRow - 1024)
        return 0;
    if (dt == RA_BF16) return ra::tree_q8_tc_workspace(R, n_seqs, Hq / Hkv, Hkv, D).bytes;
    return ra::tree_q8_simt_workspace(R, Hq / Hkv, D).bytes;
}

ra_status ra_tree_attn_paged_q8(const void* q_rows, const int* row_offsets, int n_seqs, int R, const void* k_pages,
                                const void* v_pages, const unsigned char* k_scales, const unsigned char* v_scales, int n_pages,
                                int page_size, const int* pages, int max_pages, const int* kv_lens,
                                const unsigned char* tree_mask, int mask_cols, void* out, float* lse, int Hq, int Hkv, int D,
                                ra_dtype dt, void* workspace, size_t workspace_bytes, void* stream) {
    int shift;
    ra_status st = check_q8_pools(k_pages, v_pages, k_scales, v_scales, n_pages, page_size, Hkv, D, dt, &shift);
    if (st == RA_OK) st = check_batch(row_offsets, n_seqs, R, pages, max_pages, kv_lens);
    if (st == RA_OK) st = check_heads(R, Hq, Hkv);
    if (st == RA_OK) st = check_mask(tree_mask, mask_cols);
    if (st != RA_OK) return st;
    if (R == 0) return ok();
    if (!q_rows || !out) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned(q_rows, 16) || !aligned(out, 16) || !aligned(lse, 4))
        return fail(RA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!workspace) return fail(RA_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, 256)) return fail(RA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    const size_t need = ra_tree_attn_q8_workspace_size(R, n_seqs, Hq, Hkv, D, dt);
    if (workspace_bytes < need)
        return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    ra::TreeArgs a{};
    a.p = batch(row_offsets, n_seqs, R, n_pages, shift, pages, max_pages, kv_lens, tree_mask, mask_cols, Hq, Hkv);
    a.q = q_rows;
    a.out = out;
    a.lse = lse;
    a.D = D;
    a.ws = workspace;
    const ra::Q8Pools pools = q8_pools(k_pages, v_pages, k_scales, v_scales);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched("8-bit cache attention", [&] { return dt == RA_BF16 ? ra::launch_tree_q8_tc(a, pools, s) : ra::launch_tree_q8_simt(a, pools, s); }, g_q8_used);
}

}  // extern "C"
