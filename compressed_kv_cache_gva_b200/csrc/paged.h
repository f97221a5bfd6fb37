// Arguments and host launchers of the paged serving calls: the page plan
// (pages.cu), the verification of drafted tokens (verify.cu) and the attention of
// new tokens over a paged cache (paged_mma.cu, paged_tc.cu, paged_simt.cu,
// paged_merge.cu).  Called by paged_api.cu after argument validation.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/gva.h"

namespace gva {

struct PlanArgs {
  int B, page, max_pages, num_pages, max_new;
  long long table_stride;
  const int* kept_len;
  const int* n_new;
  const int* held_in;
  int* held_out;
  int* free_pages;
  const int* free_count_in;
  int* free_count_out;
  int* table;
  int* q_start;
  int* seq_len;
  int* n_granted;
  int* slot;
  int* pos;
  int* err_flag;
};
cudaError_t launch_plan_pages(const PlanArgs& a, cudaStream_t st);

struct VerifyArgs {
  int B, vocab, n_rows;
  const int* tokens;
  const int* q_start;
  const void* target;
  const void* draft;                      // or null
  long long target_stride, draft_stride;  // elements between rows
  const float* u_accept;
  const float* u_sample;
  int* out_tokens;
  int* n_accepted;
  const int* seq_len;                     // with kept_len, or null
  int* kept_len;
  int* err_flag;
};
cudaError_t launch_verify(const VerifyArgs& a, bool bf16, int num_sms, cudaStream_t st);

// Attention of new tokens over a paged cache.  Sequence b's new tokens are query
// rows [q_start[b], q_start[b+1]); they are the last of its seq_len[b] cached tokens.
struct PagedArgs {
  int B, H, G, hpr, d_h, d_r;
  int page, max_pages;                    // tokens per page, table columns
  long long table_stride;
  int num_pages, num_slots;
  int n_rows, max_new;                    // query rows of the buffers; most rows of a sequence
  int lo_rows, hi_rows;                   // this kernel takes sequences with lo < rows*hpr <= hi
  int box;                                // rows of a cache box (divides the page and the tile)
  int box_log2;
  const float* q_abs;
  const void* V;
  const void* KR;
  const int* table;
  const int* q_start;
  const int* seq_len;
  void* out;
  float* lse;
  int out_bf16;
  int wide;                               // out and the workspace are 32-byte aligned
  int* status;
  int flag_errors;                        // this kernel reports inconsistent sequences
  int beside;                             // runs beside the kernel before it (see pdl_enter)
  float2* part_ml;
  float* part_o;
  int4* meta;
  int grid;
};

bool paged_mma_supported(const gva_shape_t& sh, int page);
int paged_mma_cols(const gva_shape_t& sh, long long columns);   // 4, 8 or 16; 0: too many
int paged_mma_tile(const gva_shape_t& sh);
// (cap_B: the batch whose prefix array decides how many CTAs fit an SM)
int paged_mma_grid(const gva_shape_t& sh, int cols, int num_sms, long long max_total, int cap_B);
cudaError_t launch_paged_mma(const gva_shape_t& sh, const PagedArgs& a, int cols,
                             const CUtensorMap& tv, const CUtensorMap& tk, cudaStream_t st);

bool paged_tc_supported(const gva_shape_t& sh, int page);
int paged_tc_tile(const gva_shape_t& sh);
int paged_tc_grid(const gva_shape_t& sh, int n_rows, int max_new, int num_sms, long long max_total);
cudaError_t launch_paged_tc(const gva_shape_t& sh, const PagedArgs& a, const CUtensorMap& tv,
                            const CUtensorMap& tk, cudaStream_t st);

bool paged_simt_supported(const gva_shape_t& sh);
int paged_simt_grid(const gva_shape_t& sh, int n_rows, int num_sms, long long max_total, int cap_B);
cudaError_t launch_paged_simt(const gva_shape_t& sh, const PagedArgs& a, cudaStream_t st);

constexpr int kPagedTcRows = 128;         // query rows (token x head) of a tcgen05 block
constexpr int kPagedSimtRows = 16;        // of a CUDA-core block

// Merge of the pieces of sequences (s: the mma kernel's arguments, with max_new the most
// new tokens it takes) and of row blocks of M rows (r: the tcgen05 or CUDA-core
// kernel's), either or both in one launch.
cudaError_t launch_paged_merge(const PagedArgs* s, const PagedArgs* r, int M, cudaStream_t st);

}  // namespace gva
