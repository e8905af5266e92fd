// api_draft.cu -- the extern "C" entry points behind a drafting step (idx.h): verification, compaction of the accepted
// tokens, page rows and page copies. Argument validation, then the launches on the caller's stream.
#include "api_util.h"
#include "kernels.h"
#include "kv.cuh"

namespace {

// One layer's pages end in front of the next one's, or every page holds a part for each layer.
bool layers_apart(int32_t layers, int64_t layer_stride, int64_t num_pages, int64_t page_bytes, int64_t page_stride) {
    if (layers <= 1 || num_pages < 1) return true;
    const __int128 whole = (__int128)(num_pages - 1) * page_stride + page_bytes;
    return layer_stride >= whole || (layer_stride >= page_bytes && (__int128)(layers - 1) * layer_stride + page_bytes <= page_stride);
}

// An array of the caller's, in bytes; NULL or empty arrays overlap nothing.
struct Bytes {
    const void* at;
    __int128 n;
};
Bytes words(const void* p, int64_t rows, int64_t width = 1) { return {p, 4 * ((__int128)rows * width)}; }  // of 4 bytes each
bool overlap(const Bytes& x, const Bytes& y) {
    if (!x.at || !y.at || x.n <= 0 || y.n <= 0) return false;
    const __int128 a = (__int128)reinterpret_cast<uintptr_t>(x.at), b = (__int128)reinterpret_cast<uintptr_t>(y.at);
    return a < b + y.n && b < a + x.n;
}

// what both caches' compaction asks of its lists
int check_compact(const int32_t* path, int32_t max_path, const int32_t* n_path, const int32_t* seq_lens_k,
                  const int32_t* cu_seqlens_q, int32_t B, const int32_t* page_table, int32_t pt_stride, const void* pool,
                  int32_t layers, int64_t layer_stride, int64_t num_pages, int32_t page_size, int64_t page_bytes,
                  int64_t page_stride, int32_t* new_lens) {
    if (max_path < 0 || B < 0 || pt_stride < 0 || layers < 0 || num_pages < 0) return IDX_EINVAL;
    if (page_stride < page_bytes || page_stride % 16 != 0 || layer_stride % 16 != 0 || layer_stride < 0) return IDX_EINVAL;
    if (!layers_apart(layers, layer_stride, num_pages, page_bytes, page_stride)) return IDX_EINVAL;
    if ((num_pages > 0 && layers > 0 && !pool) || !aligned(pool, 16)) return IDX_EINVAL;
    if (layers > 65535 || (int64_t)pt_stride * page_size > INT32_MAX) return IDX_EUNSUPPORTED;
    if (B > 0 && (!n_path || !seq_lens_k || !cu_seqlens_q || (max_path > 0 && !path) || (pt_stride > 0 && !page_table)))
        return IDX_EINVAL;
    if (!aligned(path, 4) || !aligned(n_path, 4) || !aligned(seq_lens_k, 4) || !aligned(cu_seqlens_q, 4) ||
        !aligned(page_table, 4) || !aligned(new_lens, 4))
        return IDX_EINVAL;
    // warps that have tested the lists read them again while another writes the lengths
    const Bytes in[] = {words(path, B, max_path), words(n_path, B), words(seq_lens_k, B), words(cu_seqlens_q, B + 1ll),
                        words(page_table, B, pt_stride)};
    for (const Bytes& x : in)
        if (overlap(x, words(new_lens, B))) return IDX_EINVAL;
    return IDX_OK;
}

}  // namespace

extern "C" {

int idx_draft_verify(const void* target_probs, const void* draft_probs, int32_t ptype, int64_t target_stride,
                     int64_t draft_stride, int64_t T, int32_t V, const int32_t* tokens, const int32_t* parents,
                     const float* coins, const float* last_coins, const int32_t* cu_seqlens_q, int32_t B,
                     int32_t max_q_len, int32_t max_path, int32_t* path, int32_t* n_path, int32_t* out_tokens,
                     int32_t* dev_status, cudaStream_t stream) {
    Range r("idx_draft_verify");
    if (ptype != IDX_BF16 && ptype != IDX_FP16 && ptype != IDX_FP32) return IDX_EINVAL;
    if (T < 0 || B < 0 || max_q_len < 0 || V < 1 || max_path < 1) return IDX_EINVAL;
    if (V > idx::kVerifyMaxVocab || T > INT32_MAX) return IDX_EUNSUPPORTED;
    if (target_stride < 0 || draft_stride < 0) return IDX_EINVAL;
    if (B == 0) return IDX_OK;
    const size_t size = ptype == IDX_FP32 ? 4 : 2;
    if (T > 0 && (!target_probs || !tokens || !parents || !coins)) return IDX_EINVAL;
    if (!last_coins || !cu_seqlens_q || !path || !n_path || !out_tokens) return IDX_EINVAL;
    if (!aligned(target_probs, size) || !aligned(draft_probs, size)) return IDX_EINVAL;
    const void* in[] = {target_probs, draft_probs, tokens, parents, coins, last_coins, cu_seqlens_q};
    const void* out[] = {path, n_path, out_tokens};
    for (int i = 2; i < 7; ++i)
        if (!aligned(in[i], 4)) return IDX_EINVAL;
    for (int i = 0; i < 3; ++i) {
        if (!aligned(out[i], 4)) return IDX_EINVAL;
        for (const void* p : in)
            if (p == out[i]) return IDX_EINVAL;
    }
    // a request's CTAs follow the walk each for itself: what they read stays as it is
    auto rows = [&](const void* p, int64_t stride) {
        return Bytes{p, T > 0 ? ((__int128)(T - 1) * stride + V) * (int)size : 0};
    };
    const Bytes reads[] = {rows(target_probs, target_stride), rows(draft_probs, draft_stride), words(tokens, T), words(parents, T),
                           words(coins, T), words(last_coins, B), words(cu_seqlens_q, B + 1ll)};
    const Bytes writes[] = {words(path, B, max_path), words(n_path, B), words(out_tokens, B, max_path)};
    for (int i = 0; i < 3; ++i) {
        for (const Bytes& x : reads)
            if (overlap(x, writes[i])) return IDX_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(writes[j], writes[i])) return IDX_EINVAL;
    }
    idx::VerifyArgs a{};
    a.target = target_probs; a.draft = draft_probs; a.ptype = ptype; a.target_stride = target_stride;
    a.draft_stride = draft_stride; a.T = T; a.V = V; a.tokens = tokens; a.parents = parents; a.coins = coins;
    a.last = last_coins; a.cu_seqlens_q = cu_seqlens_q; a.B = B; a.max_q_len = max_q_len; a.max_path = max_path;
    a.path = path; a.n_path = n_path; a.out_tokens = out_tokens; a.dev_status = dev_status;
    return cuda_status(idx::launch_draft_verify(a, stream));
}

int idx_kv_compact(const int32_t* path, int32_t max_path, const int32_t* n_path, const int32_t* seq_lens_k,
                   const int32_t* cu_seqlens_q, int32_t B, const int32_t* page_table, int32_t pt_stride, void* pool,
                   int32_t kv_heads, int32_t head_dim, int32_t layers, int64_t layer_stride, int64_t num_pages,
                   int32_t page_size, int64_t page_stride, int32_t* new_lens, int32_t* dev_status,
                   cudaStream_t stream) {
    Range r("idx_kv_compact");
    if (kv_heads < 1) return IDX_EINVAL;
    if ((page_size != 64 && page_size != 128) || (head_dim != 64 && head_dim != 128) || kv_heads > 1024)
        return IDX_EUNSUPPORTED;
    const int st = check_compact(path, max_path, n_path, seq_lens_k, cu_seqlens_q, B, page_table, pt_stride, pool, layers,
                                 layer_stride, num_pages, page_size, kv_heads * idx::kv_head_bytes(page_size, head_dim),
                                 page_stride, new_lens);
    if (st != IDX_OK || B == 0 || layers == 0) return st;
    idx::CompactArgs a{};
    a.path = path; a.max_path = max_path; a.n_path = n_path; a.seq_lens_k = seq_lens_k; a.cu_seqlens_q = cu_seqlens_q;
    a.B = B; a.page_table = page_table; a.pt_stride = pt_stride; a.pool = static_cast<uint8_t*>(pool);
    a.kv_heads = kv_heads; a.head_dim = head_dim; a.layers = layers; a.layer_stride = layer_stride;
    a.num_pages = num_pages; a.page_size = page_size; a.page_stride = page_stride; a.new_lens = new_lens;
    a.dev_status = dev_status;
    return cuda_status(idx::launch_kv_compact(a, stream));
}

int idx_k_compact(const int32_t* path, int32_t max_path, const int32_t* n_path, const int32_t* seq_lens_k,
                  const int32_t* cu_seqlens_q, int32_t B, const int32_t* page_table, int32_t pt_stride, int32_t dtype,
                  void* pool, int32_t layers, int64_t layer_stride, int64_t num_pages, int32_t page_size,
                  int64_t page_stride, int32_t* new_lens, int32_t* dev_status, cudaStream_t stream) {
    Range r("idx_k_compact");
    if (dtype != IDX_MXFP4 && dtype != IDX_FP8) return IDX_EINVAL;
    if (page_size != 64 && page_size != 128) return IDX_EUNSUPPORTED;
    const int st = check_compact(path, max_path, n_path, seq_lens_k, cu_seqlens_q, B, page_table, pt_stride, pool, layers,
                                 layer_stride, num_pages, page_size, (dtype == IDX_FP8 ? 132ll : 68ll) * page_size,
                                 page_stride, new_lens);
    if (st != IDX_OK || B == 0 || layers == 0) return st;
    idx::CompactArgs a{};
    a.path = path; a.max_path = max_path; a.n_path = n_path; a.seq_lens_k = seq_lens_k; a.cu_seqlens_q = cu_seqlens_q;
    a.B = B; a.page_table = page_table; a.pt_stride = pt_stride; a.pool = static_cast<uint8_t*>(pool); a.dtype = dtype;
    a.layers = layers; a.layer_stride = layer_stride; a.num_pages = num_pages; a.page_size = page_size;
    a.page_stride = page_stride; a.new_lens = new_lens; a.dev_status = dev_status;
    return cuda_status(idx::launch_k_compact(a, stream));
}

int idx_pages_update(const int32_t* parent, const int32_t* keep, int32_t n_out, const int32_t* page_table,
                     int32_t pt_stride, const int32_t* lens, int32_t B, int32_t page_size, int32_t* new_table,
                     int32_t new_stride, int32_t* new_lens, const int32_t* shares, int32_t* new_shares,
                     int32_t num_pages, const int32_t* free_pages, int32_t free_cap, const int32_t* free_span,
                     int32_t* new_free, int32_t new_free_cap, int32_t* new_span, int32_t* copies, int32_t* dev_status,
                     cudaStream_t stream) {
    Range r("idx_pages_update");
    if (n_out < 0 || B < 0 || pt_stride < 0 || new_stride < 0 || num_pages < 0 || free_cap < 0 || new_free_cap < 0)
        return IDX_EINVAL;
    if (page_size != 64 && page_size != 128) return IDX_EUNSUPPORTED;
    if (n_out > idx::kPagesMaxRows || B > idx::kPagesMaxRows || num_pages > (1 << 30)) return IDX_EUNSUPPORTED;
    if (new_free_cap < num_pages) return IDX_EINVAL;  // every page may become free
    if (new_free_cap > 0 && !new_free) return IDX_EINVAL;  // without pages too: what is left of the free list goes there
    if (!free_span || !new_span || (free_cap > 0 && !free_pages) || (num_pages > 0 && (!shares || !new_shares)))
        return IDX_EINVAL;
    if (B > 0 && (!lens || (pt_stride > 0 && !page_table))) return IDX_EINVAL;
    if (n_out > 0 && (!parent || !keep || !new_lens || !copies || (new_stride > 0 && !new_table))) return IDX_EINVAL;
    const void* in[] = {parent, keep, page_table, lens, free_pages, free_span, shares};
    const void* out[] = {new_table, new_lens, new_free, new_span, copies, new_shares};
    for (const void* p : in)
        if (!aligned(p, 4)) return IDX_EINVAL;
    for (int i = 0; i < 6; ++i) {
        if (!aligned(out[i], 4)) return IDX_EINVAL;
        for (const void* p : in)
            if (out[i] && out[i] == p && !(out[i] == new_shares && p == shares)) return IDX_EINVAL;
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return IDX_EINVAL;
    }
    // the phases read the lists again that the first one has tested; only new_shares may be shares, and then as a whole
    const Bytes reads[] = {words(parent, n_out), words(keep, n_out), words(page_table, B, pt_stride), words(lens, B),
                           words(free_pages, free_cap), words(free_span, 2), words(shares, new_shares == shares ? 0 : num_pages)};
    const Bytes writes[] = {words(new_table, n_out, new_stride), words(new_lens, n_out), words(new_free, new_free_cap),
                            words(new_span, 2), words(copies, n_out, 2), words(new_shares, num_pages)};
    for (int i = 0; i < 6; ++i) {
        for (const Bytes& x : reads)
            if (overlap(x, writes[i])) return IDX_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(writes[j], writes[i])) return IDX_EINVAL;
    }
    idx::PagesArgs a{};
    a.parent = parent; a.keep = keep; a.n_out = n_out; a.page_table = page_table; a.pt_stride = pt_stride; a.B = B;
    a.lens = lens; a.page_size = page_size; a.new_table = new_table; a.new_stride = new_stride; a.new_lens = new_lens;
    a.shares = shares; a.new_shares = new_shares; a.num_pages = num_pages; a.free_pages = free_pages;
    a.free_cap = free_cap; a.free_span = free_span; a.new_free = new_free; a.new_free_cap = new_free_cap;
    a.new_span = new_span; a.copies = copies; a.dev_status = dev_status;
    return cuda_status(idx::launch_pages_update(a, stream));
}

int idx_pages_copy(const int32_t* copies, int32_t n, void* pool, int32_t layers, int64_t layer_stride,
                   int64_t num_pages, int64_t page_bytes, int64_t page_stride, int32_t* dev_status, cudaStream_t stream) {
    Range r("idx_pages_copy");
    if (n < 0 || layers < 0 || num_pages < 0 || page_bytes < 0 || layer_stride < 0) return IDX_EINVAL;
    if (page_bytes % 16 != 0 || page_stride % 16 != 0 || layer_stride % 16 != 0 || page_stride < page_bytes) return IDX_EINVAL;
    if (!layers_apart(layers, layer_stride, num_pages, page_bytes, page_stride)) return IDX_EINVAL;
    if (n > 65535 || layers > 65535 || page_bytes > (1ll << 40)) return IDX_EUNSUPPORTED;
    if ((n > 0 && !copies) || !aligned(copies, 4) || (num_pages > 0 && layers > 0 && !pool) || !aligned(pool, 16)) return IDX_EINVAL;
    if (n == 0 || layers == 0 || page_bytes == 0) return IDX_OK;
    idx::CopyArgs a{};
    a.copies = copies; a.n = n; a.pool = static_cast<uint8_t*>(pool); a.layers = layers; a.layer_stride = layer_stride;
    a.num_pages = num_pages; a.page_bytes = page_bytes; a.page_stride = page_stride; a.dev_status = dev_status;
    return cuda_status(idx::launch_pages_copy(a, stream));
}

}  // extern "C"
