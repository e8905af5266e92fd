// kernels.h -- internal argument blocks and launchers behind the C ABI (idx.h).
// The ABI layer validates every argument before it fills one of these.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace idx {

struct KStoreArgs {
    const uint16_t* k;
    int64_t n_rows, k_row_stride;
    const int64_t* slot_mapping;
    const int32_t* positions;
    const float* cos_sin;
    int32_t max_pos, rope, apply_norm, dtype;
    const float* gamma;
    const float* beta;
    float eps;
    uint8_t* pool;
    int64_t num_pages;
    int32_t page_size;
    int64_t page_stride;
    int32_t* dev_status;
};

// Compressed K store: entries pool raw rows (see idx_compress_k_store).
struct CompressArgs {
    const uint16_t* k_raw;
    const uint16_t* gate;
    int64_t n_raw, row_stride;
    const int64_t* boundary;
    const int64_t* first;
    int64_t n_entries;
    int32_t ratio;
    const int64_t* slot_mapping;
    const int32_t* positions;
    const float* cos_sin;
    int32_t max_pos, rope, norm, dtype;
    const float* gamma;
    const float* beta;
    float eps;
    uint8_t* pool;
    int64_t num_pages;
    int32_t page_size;
    int64_t page_stride;
    int32_t* dev_status;
};

struct QQuantArgs {
    const uint16_t* q;
    int64_t T;  // tokens; each has H heads (Hq = H rounded up to 8 in the image)
    int32_t H;
    const int32_t* positions;
    const float* cos_sin;
    int32_t max_pos, rope, dtype;
    const float* w_in;
    float fold;  // fp32(softmax_scale * head_scale)
    uint8_t* q_codes;
    void* q_scales;
    float* w_out;
    int32_t* dev_status;
};

struct ScoreArgs {
    const uint8_t* q_codes;
    const uint8_t* q_scales;  // MXFP4: E8M0 scale atoms [T][512]; FP8: unused
    const float* w;           // [T][H]
    int64_t T;
    int32_t H, dtype;
    const uint8_t* pool;
    int64_t num_pages;
    int32_t page_size;
    int64_t page_stride;
    const int32_t* page_table;
    int32_t pt_stride;
    const int32_t* seq_lens_k;
    const int32_t* cu_seqlens_q;
    int32_t B, causal, max_q_len, max_seq_len_k;
    float* logits;  // select mode: the workspace's logits scratch (see launch_scorer_topk)
    int64_t ld;
    int32_t* dev_status;
    // select mode only (idx_mqa_topk_paged): top-k size, output [T][topk_k], per-sequence
    // arrival counters of the decode kernel (zero before and after a call)
    int32_t topk_k;
    int32_t* out_idx;
    int32_t* counters;
    // launch without programmatic dependent launch: set when the previous kernel on the
    // stream writes this call's metadata (lengths, page table), which the scorer's prologue
    // reads before its grid-dependency wait
    bool no_pdl;
};

struct TopkArgs {
    const float* logits;
    int64_t ld;
    const int32_t* seq_lens_k;
    const int32_t* cu_seqlens_q;
    int32_t B;
    int64_t T;
    int32_t causal, max_len, k;  // max_len: the scorer's max_seq_len_k (<= ld)
    int32_t* out;
    int32_t* dev_status;
};

cudaError_t launch_k_store(const KStoreArgs& a, cudaStream_t st);
cudaError_t launch_q_quant(const QQuantArgs& a, cudaStream_t st);
cudaError_t launch_qk_prep(const KStoreArgs& ka, const QQuantArgs& qa, cudaStream_t st);
cudaError_t launch_compress(const CompressArgs& a, cudaStream_t st);

// Candidate-pool scoring (idx_mqa_topk_cand_paged): per query, its candidate blocks sorted and
// deduplicated into a virtual page table; the decode scorer and top-k then run on one virtual
// sequence per query, and the indices are mapped back to key positions.
struct CandArgs {
    const int32_t* cu_seqlens_q;
    const int32_t* seq_lens_k;
    const int32_t* page_table;
    int32_t pt_stride, B, causal, max_q_len, max_seq_len_k, page_size;
    int64_t T;
    const int32_t* cand;
    int32_t cand_stride, max_cand;
    const int32_t* n_cand;
    // workspace: cu' [T+1], vlen [T], virtual page table and sorted blocks [T][max_cand]
    int32_t* vcu;
    int32_t* vlen;
    int32_t* vpt;
    int32_t* vblk;
    int32_t* dev_status;
};
cudaError_t launch_cand_prep(const CandArgs& a, cudaStream_t st);
cudaError_t launch_cand_map(const int32_t* vblk, int32_t max_cand, int32_t page_size, int64_t T, int32_t k,
                            int32_t* out_idx, cudaStream_t st);
cudaError_t launch_debug_encode(int kind, const float* in, int64_t n, uint8_t* out, cudaStream_t st);
cudaError_t launch_scorer(const ScoreArgs& a, cudaStream_t st);
cudaError_t launch_scorer_decode(const ScoreArgs& a, cudaStream_t st);
cudaError_t launch_scorer_prefill(const ScoreArgs& a, cudaStream_t st);
cudaError_t launch_topk(const TopkArgs& a, cudaStream_t st);

// Fused scorer -> top-k (idx_mqa_topk_paged): bytes of workspace it needs, and the launch.
int64_t scorer_topk_workspace_bytes(int64_t T, int32_t H, int32_t B, int32_t max_q_len, int32_t max_seq_len_k);
cudaError_t launch_scorer_topk(const ScoreArgs& a, void* workspace, cudaStream_t st);
cudaError_t launch_scorer_decode_select(const ScoreArgs& a, cudaStream_t st);
cudaError_t launch_scorer_prefill_select(const ScoreArgs& a, cudaStream_t st);
int prefill_queries_per_block(int32_t H);
int device_sm_count();

// Step metadata (idx_step_meta).
constexpr int32_t kMetaMaxRequests = 16384;  // 8 bytes each in shared memory
struct MetaArgs {
    const int32_t* ctx_lens;
    const int32_t* q_lens;
    int32_t B;
    int32_t* page_table;
    int32_t pt_stride, page_size, max_seq_len_k;
    const int32_t* free_pages;
    int32_t free_cap;
    const int32_t* free_span;
    int64_t num_pages;
    int32_t* cu_seqlens_q;
    int32_t* seq_lens_k;
    int32_t* positions;
    int64_t* slot_mapping;
    int64_t T_cap;
    int32_t* free_next;
    int32_t* dev_status;
};
cudaError_t launch_step_meta(const MetaArgs& a, cudaStream_t st);

// K and V rows into the 8-bit paged KV cache (idx_kv_store); strides in elements.
struct KvStoreArgs {
    const uint16_t* k;
    const uint16_t* v;
    int32_t ftype;
    int64_t n_rows;
    int32_t kv_heads, head_dim;
    int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    const int64_t* slot_mapping;
    uint8_t* pool;
    int64_t num_pages;
    int32_t page_size;
    int64_t page_stride;
    int32_t* dev_status;
};
cudaError_t launch_kv_store(const KvStoreArgs& a, cudaStream_t st);

// Attention over that cache (idx_attn_paged, idx_attn_tree); strides in elements.
constexpr int32_t kTreeMaxNodes = 1024;  // nodes of a sequence: a bit of shared memory each
struct AttnArgs {
    const uint16_t* q;
    int32_t ftype;
    int64_t T;
    int32_t q_heads, kv_heads, head_dim, group;  // group = q_heads / kv_heads
    int64_t q_row_stride, q_head_stride;
    const uint8_t* pool;
    int64_t num_pages;
    int32_t page_size;
    int64_t page_stride;
    const int32_t* page_table;
    int32_t pt_stride;
    const int32_t* seq_lens_k;
    const int32_t* cu_seqlens_q;
    int32_t B, causal, max_q_len, max_seq_len_k;
    const int32_t* sel;
    int64_t sel_stride;
    int32_t n_sel;
    // a tree of drafted tokens: row t sees its sequence's node j where bit j of its mask is set (causal is 0 then)
    const uint64_t* tree;  // [T][tree_stride], or NULL
    int64_t tree_stride;
    int32_t tree_words;
    float scale;
    uint16_t* out;
    int64_t out_row_stride, out_head_stride;
    float* lse;
    int32_t* dev_status;
    // key axis split: split z takes keys (or list entries) z * chunk .. ; with n_split > 1 the
    // kernels write O and (m, l) of each split there and the combine kernel joins them
    int32_t n_split, chunk;
    float* part_o;    // [n_split][T][q_heads][head_dim]
    float2* part_ml;  // [n_split][T][q_heads]
};
// Fills n_split and chunk for at most `bytes` of workspace (0: none); bytes the split wants.
int64_t attn_plan(AttnArgs& a, int64_t bytes);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_tile(const AttnArgs& a, cudaStream_t st);  // many rows per kv head (attn_tc.cu)

// Walk through trees of drafted tokens (idx_draft_verify); strides in elements.
constexpr int32_t kVerifyMaxVocab = 1 << 20;  // a bit per token in shared memory
struct VerifyArgs {
    const void* target;  // [T][V]
    const void* draft;   // [T][V], or NULL
    int32_t ptype;
    int64_t target_stride, draft_stride, T;
    int32_t V;
    const int32_t* tokens;
    const int32_t* parents;
    const float* coins;
    const float* last;
    const int32_t* cu_seqlens_q;
    int32_t B, max_q_len, max_path;
    int32_t* path;
    int32_t* n_path;
    int32_t* out_tokens;
    int32_t* dev_status;
};
cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t st);

// Accepted tokens moved together (idx_kv_compact, idx_k_compact).
struct CompactArgs {
    const int32_t* path;
    int32_t max_path;
    const int32_t* n_path;
    const int32_t* seq_lens_k;
    const int32_t* cu_seqlens_q;
    int32_t B;
    const int32_t* page_table;
    int32_t pt_stride;
    uint8_t* pool;
    int32_t layers;
    int64_t layer_stride, num_pages;
    int32_t page_size;
    int64_t page_stride;
    int32_t kv_heads, head_dim;  // 8-bit KV cache
    int32_t dtype;               // indexer's cache
    int32_t* new_lens;
    int32_t* dev_status;
};
cudaError_t launch_kv_compact(const CompactArgs& a, cudaStream_t st);
cudaError_t launch_k_compact(const CompactArgs& a, cudaStream_t st);

// Next rows of a page table out of the present ones (idx_pages_update), copies of pages (idx_pages_copy).
constexpr int32_t kPagesMaxRows = 16384;  // 12 bytes each in shared memory, beside a bitmap of 16 KB (pages.cu)
struct PagesArgs {
    const int32_t* parent;
    const int32_t* keep;
    int32_t n_out;
    const int32_t* page_table;
    int32_t pt_stride, B;
    const int32_t* lens;
    int32_t page_size;
    int32_t* new_table;
    int32_t new_stride;
    int32_t* new_lens;
    const int32_t* shares;
    int32_t* new_shares;
    int32_t num_pages;
    const int32_t* free_pages;
    int32_t free_cap;
    const int32_t* free_span;
    int32_t* new_free;
    int32_t new_free_cap;
    int32_t* new_span;
    int32_t* copies;
    int32_t* dev_status;
};
cudaError_t launch_pages_update(const PagesArgs& a, cudaStream_t st);
struct CopyArgs {
    const int32_t* copies;
    int32_t n;
    uint8_t* pool;
    int32_t layers;
    int64_t layer_stride, num_pages, page_bytes, page_stride;
    int32_t* dev_status;
};
cudaError_t launch_pages_copy(const CopyArgs& a, cudaStream_t st);

// Behind a kernel that writes lengths or page tables (meta.cu): returns when its output is visible.
cudaError_t launch_done(cudaStream_t st);

// Bounded-wait test hook (idx_debug_wait_timeout).
cudaError_t launch_wait_timeout(int32_t limit_us, int32_t* status, cudaStream_t st);

// Dense tensor-core rate probe (idx_debug_mma_rate): one CTA per SM, `iters` loop iterations.
cudaError_t launch_mma_rate(int32_t dtype, int32_t iters, int32_t* status, cudaStream_t st);
int mma_rate_flops_per_iter(int32_t dtype);

}  // namespace idx
