// api_attn.cu -- the extern "C" entry points of the step metadata, the 8-bit KV store and the paged
// attention (idx.h): argument validation, then the launches on the caller's stream. Nothing
// here allocates, frees or synchronises.
#include <cmath>

#include "api_util.h"
#include "kernels.h"
#include "kv.cuh"

namespace {

constexpr int32_t kMaxKeys = INT32_MAX - 65536;

inline bool valid_ftype(int32_t f) { return f == IDX_BF16 || f == IDX_FP16; }

// pool checks of the 8-bit KV cache
int check_kv_pool(int32_t kv_heads, int32_t head_dim, const void* pool, int64_t num_pages, int32_t page_size,
                  int64_t page_stride) {
    if (kv_heads < 1 || num_pages < 0) return IDX_EINVAL;
    if (page_size != 64 && page_size != 128) return IDX_EUNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return IDX_EUNSUPPORTED;
    if (kv_heads > 1024) return IDX_EUNSUPPORTED;
    if ((num_pages > 0 && !pool) || !aligned(pool, 16)) return IDX_EINVAL;
    if (page_stride < kv_heads * idx::kv_head_bytes(page_size, head_dim) || page_stride % 16 != 0) return IDX_EINVAL;
    return IDX_OK;
}

// rows of 16-byte vectors: a base and two strides in 2-byte elements
inline bool row_strides(const void* p, int64_t row, int64_t head) {
    return p && aligned(p, 16) && row >= 0 && head >= 0 && row % 8 == 0 && head % 8 == 0;
}

// The workspace that a call's split of the key axis would like (tree: rows are nodes of a tree).
int attn_workspace(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t B, int32_t max_q_len,
                   int32_t max_seq_len_k, int32_t n_sel, bool tree, size_t* bytes) {
    if (!bytes || T < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || B < 0 || max_q_len < 0 ||
        max_seq_len_k < 0 || n_sel < 0)
        return IDX_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || kv_heads > 1024 || max_seq_len_k > kMaxKeys || n_sel > kMaxKeys ||
        T > INT32_MAX || T * q_heads > INT32_MAX - 256)
        return IDX_EUNSUPPORTED;
    idx::AttnArgs a{};
    a.T = T; a.q_heads = q_heads; a.kv_heads = kv_heads; a.group = q_heads / kv_heads; a.head_dim = head_dim;
    a.B = B; a.max_q_len = (int32_t)(max_q_len < T ? max_q_len : T); a.max_seq_len_k = max_seq_len_k; a.n_sel = n_sel;
    if (tree && a.max_q_len > idx::kTreeMaxNodes) return IDX_EUNSUPPORTED;
    static const uint64_t some = 0;
    a.tree = tree ? &some : nullptr;  // the plan only asks whether there is one
    const int64_t n = idx::attn_plan(a, 0);
    if (n < 0) return IDX_ECUDA;
    *bytes = (size_t)n;
    return IDX_OK;
}

// Attention over the 8-bit cache; tree_mask: rows are nodes of a tree, and causal is 0.
int attention(const void* q, int32_t ftype, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
              int64_t q_row_stride, int64_t q_head_stride, const void* pool, int64_t num_pages, int32_t page_size,
              int64_t page_stride, const int32_t* page_table, int32_t pt_stride, const int32_t* seq_lens_k,
              const int32_t* cu_seqlens_q, int32_t B, int32_t causal, bool tree, const uint64_t* tree_mask,
              int64_t mask_stride, int32_t mask_words, int32_t max_q_len, int32_t max_seq_len_k,
              const int32_t* sel_idx, int64_t sel_stride, int32_t n_sel, float softmax_scale, void* out,
              int64_t out_row_stride, int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
              int32_t* dev_status, cudaStream_t stream) {
    if (T < 0 || B < 0 || max_q_len < 0 || max_seq_len_k < 0 || pt_stride < 0 || n_sel < 0 || !valid_ftype(ftype))
        return IDX_EINVAL;
    const int st = check_kv_pool(kv_heads, head_dim, pool, num_pages, page_size, page_stride);
    if (st != IDX_OK) return st;
    if (q_heads < 1 || q_heads % kv_heads != 0) return IDX_EINVAL;
    if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return IDX_EINVAL;
    if (max_seq_len_k > (int64_t)pt_stride * page_size) return IDX_EINVAL;
    if (T > 0 && (sel_idx ? sel_stride < n_sel || !aligned(sel_idx, 4) || n_sel < 1 : n_sel != 0)) return IDX_EINVAL;
    if (!aligned(workspace, 256)) return IDX_EINVAL;
    // 32-bit key positions with room for a step behind the end, 32-bit row numbers
    if (max_seq_len_k > kMaxKeys || n_sel > kMaxKeys || T > INT32_MAX || T * q_heads > INT32_MAX - 256)
        return IDX_EUNSUPPORTED;
    const int64_t group = q_heads / kv_heads;
    if (max_q_len > T) max_q_len = (int32_t)T;  // no sequence within cu_seqlens_q[B] <= T has more
    if (tree) {
        if (max_q_len > idx::kTreeMaxNodes) return IDX_EUNSUPPORTED;
        if (mask_words < 0 || mask_stride < mask_words || (int64_t)mask_words * 64 < max_q_len) return IDX_EINVAL;
        // positions of nodes behind a list's entries, 32-bit as they are
        if (n_sel > kMaxKeys - idx::kTreeMaxNodes) return IDX_EUNSUPPORTED;
    }
    // grids: one unit per 16 rows of a sequence, or of a query's group of heads
    if (B * ((max_q_len * group + 15) / 16) > INT32_MAX) return IDX_EUNSUPPORTED;
    if (T == 0 || B == 0 || max_q_len == 0) return IDX_OK;
    if (!row_strides(q, q_row_stride, q_head_stride) || !row_strides(out, out_row_stride, out_head_stride))
        return IDX_EINVAL;
    if ((T > 1 && out_row_stride < head_dim) || (q_heads > 1 && out_head_stride < head_dim)) return IDX_EINVAL;
    if (!seq_lens_k || !cu_seqlens_q || (max_seq_len_k > 0 && !page_table)) return IDX_EINVAL;
    if (tree && (!tree_mask || !aligned(tree_mask, 8))) return IDX_EINVAL;
    if (!aligned(seq_lens_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
        return IDX_EINVAL;
    idx::AttnArgs a{};
    a.q = static_cast<const uint16_t*>(q); a.ftype = ftype; a.T = T; a.q_heads = q_heads; a.kv_heads = kv_heads;
    a.head_dim = head_dim; a.group = (int32_t)group; a.q_row_stride = q_row_stride; a.q_head_stride = q_head_stride;
    a.pool = static_cast<const uint8_t*>(pool); a.num_pages = num_pages; a.page_size = page_size;
    a.page_stride = page_stride; a.page_table = page_table; a.pt_stride = pt_stride; a.seq_lens_k = seq_lens_k;
    a.cu_seqlens_q = cu_seqlens_q; a.B = B; a.causal = causal != 0; a.max_q_len = max_q_len;
    a.max_seq_len_k = max_seq_len_k; a.sel = sel_idx; a.sel_stride = sel_stride; a.n_sel = n_sel;
    a.tree = tree_mask; a.tree_stride = mask_stride; a.tree_words = mask_words;
    a.scale = softmax_scale; a.out = static_cast<uint16_t*>(out); a.out_row_stride = out_row_stride;
    a.out_head_stride = out_head_stride; a.lse = lse; a.dev_status = dev_status;
    if (idx::attn_plan(a, workspace ? (int64_t)workspace_bytes : 0) < 0) return IDX_ECUDA;
    if (a.n_split > 1) {
        a.part_o = static_cast<float*>(workspace);
        a.part_ml = reinterpret_cast<float2*>(a.part_o + (int64_t)a.n_split * T * q_heads * head_dim);
    }
    return cuda_status(idx::launch_attn(a, stream));
}

}  // namespace

extern "C" {

int idx_step_meta(const int32_t* ctx_lens, const int32_t* q_lens, int32_t B, int32_t* page_table, int32_t pt_stride,
                  int32_t page_size, int32_t max_seq_len_k, const int32_t* free_pages, int32_t free_cap,
                  const int32_t* free_span, int64_t num_pages, int32_t* cu_seqlens_q, int32_t* seq_lens_k,
                  int32_t* positions, int64_t* slot_mapping, int64_t T_cap, int32_t* free_next, int32_t* dev_status,
                  cudaStream_t stream) {
    Range r("idx_step_meta");
    if (B < 0 || pt_stride < 0 || max_seq_len_k < 0 || free_cap < 0 || num_pages < 0 || T_cap < 0) return IDX_EINVAL;
    if (page_size != 64 && page_size != 128) return IDX_EUNSUPPORTED;
    if (B > idx::kMetaMaxRequests || T_cap > INT32_MAX) return IDX_EUNSUPPORTED;
    if (max_seq_len_k > (int64_t)pt_stride * page_size) return IDX_EINVAL;
    if (!free_span || !cu_seqlens_q || !free_next || (free_cap > 0 && !free_pages)) return IDX_EINVAL;
    if (B > 0 && (!ctx_lens || !q_lens || !seq_lens_k || (!page_table && pt_stride > 0))) return IDX_EINVAL;
    if (T_cap > 0 && (!positions || !slot_mapping)) return IDX_EINVAL;
    const void* in[] = {ctx_lens, q_lens, free_pages, free_span};
    const void* out[] = {page_table, cu_seqlens_q, seq_lens_k, positions, slot_mapping, free_next};
    for (const void* p : in)
        if (!aligned(p, 4)) return IDX_EINVAL;
    if (!aligned(slot_mapping, 8)) return IDX_EINVAL;
    for (int i = 0; i < 6; ++i) {
        if (!aligned(out[i], 4)) return IDX_EINVAL;
        for (const void* p : in)
            if (out[i] && out[i] == p) return IDX_EINVAL;
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return IDX_EINVAL;
    }
    idx::MetaArgs a{};
    a.ctx_lens = ctx_lens; a.q_lens = q_lens; a.B = B; a.page_table = page_table; a.pt_stride = pt_stride;
    a.page_size = page_size; a.max_seq_len_k = max_seq_len_k; a.free_pages = free_pages; a.free_cap = free_cap;
    a.free_span = free_span; a.num_pages = num_pages; a.cu_seqlens_q = cu_seqlens_q; a.seq_lens_k = seq_lens_k;
    a.positions = positions; a.slot_mapping = slot_mapping; a.T_cap = T_cap; a.free_next = free_next;
    a.dev_status = dev_status;
    return cuda_status(idx::launch_step_meta(a, stream));
}

int idx_kv_layout(int32_t kv_heads, int32_t head_dim, int32_t page_size, idx_kv_layout_t* out) {
    if (!out || kv_heads < 1) return IDX_EINVAL;
    if ((page_size != 64 && page_size != 128) || (head_dim != 64 && head_dim != 128) || kv_heads > 1024)
        return IDX_EUNSUPPORTED;
    out->head_bytes = idx::kv_head_bytes(page_size, head_dim);
    out->page_bytes = out->head_bytes * kv_heads;
    out->scale_offset = 2ll * page_size * head_dim;
    out->scale_block = idx::kKvBlock;
    out->page_size = page_size;
    out->kv_heads = kv_heads;
    out->head_dim = head_dim;
    return IDX_OK;
}

int idx_kv_store(const void* k, const void* v, int32_t ftype, int64_t n_rows, int32_t kv_heads, int32_t head_dim,
                 int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                 const int64_t* slot_mapping, void* pool, int64_t num_pages, int32_t page_size, int64_t page_stride,
                 int32_t* dev_status, cudaStream_t stream) {
    Range r("idx_kv_store");
    if (n_rows < 0 || !valid_ftype(ftype)) return IDX_EINVAL;
    const int st = check_kv_pool(kv_heads, head_dim, pool, num_pages, page_size, page_stride);
    if (st != IDX_OK || n_rows == 0) return st;
    if (n_rows > INT32_MAX) return IDX_EUNSUPPORTED;
    if (!slot_mapping || !aligned(slot_mapping, 8)) return IDX_EINVAL;
    if (!row_strides(k, k_row_stride, k_head_stride) || !row_strides(v, v_row_stride, v_head_stride))
        return IDX_EINVAL;
    idx::KvStoreArgs a{};
    a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v); a.ftype = ftype; a.n_rows = n_rows;
    a.kv_heads = kv_heads; a.head_dim = head_dim; a.k_row_stride = k_row_stride; a.k_head_stride = k_head_stride;
    a.v_row_stride = v_row_stride; a.v_head_stride = v_head_stride; a.slot_mapping = slot_mapping;
    a.pool = static_cast<uint8_t*>(pool); a.num_pages = num_pages; a.page_size = page_size;
    a.page_stride = page_stride; a.dev_status = dev_status;
    return cuda_status(idx::launch_kv_store(a, stream));
}

int idx_attn_workspace_bytes(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t B,
                             int32_t max_q_len, int32_t max_seq_len_k, int32_t n_sel, size_t* bytes) {
    return attn_workspace(T, q_heads, kv_heads, head_dim, B, max_q_len, max_seq_len_k, n_sel, false, bytes);
}

int idx_attn_tree_workspace_bytes(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t B,
                                  int32_t max_q_len, int32_t max_seq_len_k, int32_t n_sel, size_t* bytes) {
    return attn_workspace(T, q_heads, kv_heads, head_dim, B, max_q_len, max_seq_len_k, n_sel, true, bytes);
}

int idx_attn_paged(const void* q, int32_t ftype, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                   int64_t q_row_stride, int64_t q_head_stride, const void* pool, int64_t num_pages,
                   int32_t page_size, int64_t page_stride, const int32_t* page_table, int32_t pt_stride,
                   const int32_t* seq_lens_k, const int32_t* cu_seqlens_q, int32_t B, int32_t causal,
                   int32_t max_q_len, int32_t max_seq_len_k, const int32_t* sel_idx, int64_t sel_stride,
                   int32_t n_sel, float softmax_scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                   float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status, cudaStream_t stream) {
    Range r("idx_attn_paged");
    return attention(q, ftype, T, q_heads, kv_heads, head_dim, q_row_stride, q_head_stride, pool, num_pages, page_size,
                     page_stride, page_table, pt_stride, seq_lens_k, cu_seqlens_q, B, causal, false, nullptr, 0, 0,
                     max_q_len, max_seq_len_k, sel_idx, sel_stride, n_sel, softmax_scale, out, out_row_stride,
                     out_head_stride, lse, workspace, workspace_bytes, dev_status, stream);
}

int idx_attn_tree(const void* q, int32_t ftype, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                  int64_t q_row_stride, int64_t q_head_stride, const void* pool, int64_t num_pages, int32_t page_size,
                  int64_t page_stride, const int32_t* page_table, int32_t pt_stride, const int32_t* seq_lens_k,
                  const int32_t* cu_seqlens_q, int32_t B, const uint64_t* tree_mask, int64_t mask_stride,
                  int32_t mask_words, int32_t max_q_len, int32_t max_seq_len_k, const int32_t* sel_idx,
                  int64_t sel_stride, int32_t n_sel, float softmax_scale, void* out, int64_t out_row_stride,
                  int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                  cudaStream_t stream) {
    Range r("idx_attn_tree");
    return attention(q, ftype, T, q_heads, kv_heads, head_dim, q_row_stride, q_head_stride, pool, num_pages, page_size,
                     page_stride, page_table, pt_stride, seq_lens_k, cu_seqlens_q, B, 0, true, tree_mask, mask_stride,
                     mask_words, max_q_len, max_seq_len_k, sel_idx, sel_stride, n_sel, softmax_scale, out,
                     out_row_stride, out_head_stride, lse, workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"
