// Kernel parameter blocks and launchers shared between the kernels and the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace dsa {

struct IndexerParams {
  const float* w;            // [T, H_I]
  float* scores;             // [T, ld]
  int64_t ld;
  const int32_t* q_seq;      // [T]
  const int32_t* q_pos;      // [T]
  const int64_t* kv_offset;  // [B] (contiguous layout)
  const int32_t* kv_len;     // [B]
  const int32_t* page_table; // [B, pages_per_seq] (paged layout, page_size > 0)
  int page_size;             // 0 = contiguous rows from kv_offset
  int pages_per_seq;
  int64_t kv_rows;           // rows of the k_idx buffer
  uint32_t* hist;            // [T, 2048] histogram of the top 11 key bits per row (zeroed), or null
  // plan (workspace)
  int32_t* group_q0;         // [T]
  int32_t* group_cnt;        // [T]
  int32_t* group_seq;        // [T]
  int32_t* group_tiles;      // [T]
  int32_t* item_off;         // [T + 1]
  int32_t* ngroups;          // [1]
  int32_t* q_nvis;           // [T] visible keys per query, -1 = invalid query
  uint32_t* status;
  int G;                     // query tokens per group (N = G * padded H_I)
  int hi;                    // H_I, heads per query token (a multiple of 4, <= 64)
  int nacc;                  // accumulator buffers in TMEM: 4 when N <= 128, else 2
  int max_kv_len;
};

struct TopkParams {
  const float* scores;       // [T, ld]
  const uint32_t* hist;      // [T, 2048] per-row histogram of the top 11 key bits, or null
  int64_t ld;
  int32_t* idx;              // [T, k]
  int k;
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int32_t* kv_len;
  int num_seqs;
  int max_kv_len;
  uint32_t* status;
};

struct MlaParams {
  const uint16_t* q;         // [T, H, 576] bf16
  const uint16_t* kv;        // [rows, 576] bf16
  const int32_t* idx;        // [T, k]
  int k;
  int H;
  float sm_scale_log2;       // sm_scale * log2(e)
  float sm_scale;
  uint16_t* out;             // [T, H, 512] bf16
  float* lse;                // [T, H] or null
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int64_t* kv_offset;  // contiguous layout
  const int32_t* kv_len;
  const int32_t* page_table; // [B, pages_per_seq] (paged layout, page_size > 0)
  int page_size;             // 0 = contiguous rows from kv_offset
  int pages_per_seq;
  int num_seqs;
  int64_t kv_rows;
  int T;
  int splits;                // index-list splits per query (1 = no combine pass)
  float* part_o;             // [T, splits, H, 512] fp32 (splits > 1)
  float* part_lse;           // [T, splits, H]       fp32 (splits > 1)
  uint32_t* status;
};

struct ProjParams {
  float* y;                  // [T, n_all] fp32 projections (workspace)
  uint8_t* q_idx;            // [T, H_I, 128] E4M3
  float* w;                  // [T, H_I]
  uint16_t* q;               // [T, H, 576] bf16
  uint8_t* k_cache;          // [kv_rows, 128] E4M3
  uint16_t* kv_cache;        // [kv_rows, 576] bf16, or null with kv_new
  uint16_t* kv_new;          // [T, 576] bf16: latent rows by token instead of by cache row, or null
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int64_t* kv_offset;  // contiguous layout
  const int32_t* kv_len;
  const int32_t* page_table; // paged layout (page_size > 0)
  int page_size;
  int pages_per_seq;
  int num_seqs;
  int64_t kv_rows;
  int T;
  int n_all;                 // rows of the stacked projection matrix
  int hi;                    // H_I
  int heads;                 // H
  float rope_base;
  uint32_t* status;
};

struct MlaBwdParams {
  const uint16_t* q;         // [T, H, 576] bf16
  const uint16_t* kv;        // [rows, 576] bf16
  const int32_t* idx;        // [T, k]
  int k;
  int H;
  float sm_scale;
  const uint16_t* out;       // [T, H, 512] bf16, the forward's output
  const float* lse;          // [T, H], the forward's log-sum-exp
  const uint16_t* d_out;     // [T, H, 512] bf16
  float* d_q;                // [T, H, 576]
  float* d_kv;               // [rows, 576], accumulated
  const int32_t* q_seq;
  const int64_t* kv_offset;
  const int32_t* kv_len;
  const int32_t* page_table;
  int page_size;
  int pages_per_seq;
  int num_seqs;
  int64_t kv_rows;
  int T;
  uint32_t* status;
};
cudaError_t launch_mla_backward(const MlaBwdParams& p, cudaStream_t stream);

struct QuantParams {
  const uint16_t* kv;        // [T, 576] bf16, the new rows
  uint8_t* kv8;              // [kv_rows, 576] E4M3
  float* scale;              // [ceil(kv_rows / block)]
  int block_log2;            // tokens per scale = 1 << block_log2
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int64_t* kv_offset;  // contiguous layout
  const int32_t* kv_len;
  const int32_t* page_table; // paged layout (page_size > 0)
  int page_size;
  int pages_per_seq;
  int num_seqs;
  int64_t kv_rows;
  int T;
  int32_t* num_runs;         // [1], 0 at the start
  int32_t* runs;             // [T] tokens that begin runs
  uint32_t* status;
};
cudaError_t launch_quantize_append(const QuantParams& p, int sms, cudaStream_t stream);

struct MlaQ8Params {
  const uint16_t* q;         // [T, H, 576] bf16
  const uint8_t* kv8;        // [kv_rows, 576] E4M3
  const float* scale;        // [ceil(kv_rows / block)]
  int block_log2;            // tokens per scale = 1 << block_log2
  const int32_t* idx;        // [T, k], or null: every visible key
  int k;
  int H;
  float sm_scale;
  uint16_t* out;             // [T, H, 512] bf16
  float* lse;                // [T, H] or null
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int64_t* kv_offset;  // contiguous layout
  const int32_t* kv_len;
  const int32_t* page_table; // paged layout (page_size > 0)
  int page_size;
  int pages_per_seq;
  int num_seqs;
  int64_t kv_rows;
  int T;
  uint32_t* status;
  int splits;                // parts of each query's row list (1 = no combine pass)
  int split_tiles;           // 128-row tiles of a part
  int groups;                // head groups
  int items;                 // T * splits * groups
  int32_t* counter;          // items handed out, 0 at the start
  float* part_o;             // [T, splits, H, 512] fp32 (splits > 1)
  float* part_lse;           // [T, splits, H]       fp32 (splits > 1)
};
// Parts that each query's row list is cut into, and the 128-row tiles of a part.
int mla_q8_plan(int T, int H, int64_t most, int64_t mean, int sms, int* split_tiles);
// clear: the status word and the counter (beside one another) are cleared first.
cudaError_t launch_sparse_mla_q8(const MlaQ8Params& p, bool clear, int sms, cudaStream_t stream);

struct PagesParams {
  int num_seqs, num_pages, page_size, pages_per_seq;
  const int32_t* table_in;   // [num_seqs, pages_per_seq]
  const int32_t* len_in;     // [num_seqs]
  const int32_t* ref_in;     // [num_pages]
  int32_t* table_out;        // the same arrays, or others
  int32_t* len_out;
  int32_t* ref_out;
  int n;                     // entries of the lists
  const int32_t* list_a;     // sequences (resize), sources (fork)
  const int32_t* list_b;     // new lengths (resize), destinations (fork)
  uint8_t* buf[DSA_MAX_PAGE_BUFFERS];
  int64_t buf_bytes[DSA_MAX_PAGE_BUFFERS];
  int buf_chunks[DSA_MAX_PAGE_BUFFERS];
  int buf_vec[DSA_MAX_PAGE_BUFFERS];
  int num_bufs;
  int chunks;                // of one page, over all buffers
  // workspace
  uint32_t* status;
  int32_t* num_moves;        // [3]: page copies, dropped and taken table entries
  int32_t* first;            // [num_seqs]
  int32_t* sharers;          // [num_pages]
  int32_t* last_sharer;      // [num_pages]
  int32_t* free_list;        // [num_pages]
  int32_t* map;              // [num_pages]
  int32_t* move_src;         // [num_pages]
  int32_t* move_dst;         // [num_pages]
  int32_t* old_len;          // [n]
  int32_t* last_page;        // [n]
  int32_t* drop_at;          // [n] prefix sums of the entries' dropped pages
  int32_t* drop_pos;         // [n] table place of the k-th dropped page, minus k
  int32_t* take_at;          // [n] the same of the pages taken
  int32_t* take_pos;         // [n]
};

// Counts kernel launches made by the library (dsa_launch_count).
void count_launches(int n);

size_t project_gemm_workspace_bytes();
cudaError_t launch_project(const ProjParams& p, const uint16_t* hidden, const uint16_t* w_all, int d_model,
                           void* gemm_ws, size_t gemm_ws_bytes, cudaStream_t stream, bool* gemm_failed);
size_t indexer_smem_bytes();
size_t mla_smem_bytes();
cudaError_t launch_indexer(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const IndexerParams& p, int hi_pad,
                           int T, int B, int64_t kv_rows, int num_sms, cudaStream_t stream);
cudaError_t launch_topk(const TopkParams& p, int T, cudaStream_t stream);
// Whether the top-k kernel chosen for these rows takes an emitted histogram as
// its first radix pass (the clustered and the uncached streaming kernels).
bool topk_uses_hist(int max_kv_len, int T, int sms);
cudaError_t launch_sparse_mla(const MlaParams& p, const CUtensorMap& tm_q, cudaStream_t stream);

}  // namespace dsa
