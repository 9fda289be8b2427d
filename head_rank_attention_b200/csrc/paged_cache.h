// paged_cache.h -- host-side interface of the kernels that fill and read the paged latent
// cache: the page plan of a step, the append of new tokens and the load of cached rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace hra {

// Formats of the cached latent (the RoPE key is bf16 in all of them).
enum CacheFormat : int { kCacheBf16 = 0, kCacheInt8 = 1, kCacheE4m3 = 2 };

struct PlanArgs {  // device pointers; see hra_plan_params in hra.h
  const int32_t* seq_lens;
  const int32_t* new_tokens;
  int32_t* block_table;
  int32_t* free_pages;
  const int64_t* free_range;
  int32_t* seq_lens_out;
  int64_t* free_range_out;
  int32_t* query_start;
  int32_t* slots;
  int32_t* positions;  // or nullptr
  int32_t* status;
  int batch, page_size, max_pages, num_pages, max_tokens;
};

// Refusals a plan writes to status[0].
enum PlanStatus : int {
  kPlanOk = 0,
  kPlanBadLength = 1,    // status[1] = sequence: cached length negative or past the table
  kPlanTableFull = 2,    // status[1] = sequence: the new length needs more than max_pages pages
  kPlanTooManyTokens = 3,  // status[2] = tokens asked for, status[3] = max_tokens
  kPlanNoPages = 4,        // status[2] = pages needed, status[3] = pages free
  kPlanBadPool = 5,        // the free range does not describe this pool
};

struct AppendArgs {  // see hra_append_params
  const void* latent;
  const void* krope_in;
  long long latent_stride, krope_in_stride;  // bf16 elements
  const int32_t* slots;
  const int32_t* positions;
  void* ckv;
  void* krope;
  long long ckv_stride, krope_stride;  // elements of the cache's types
  long long cache_rows;
  float* scale;
  long long scale_stride;
  void* rows_out;  // or nullptr
  long long rows_out_stride;
  double log2_theta;
  int n_tokens, d_c, scale_block;
};

struct LoadArgs {  // see hra_load_params
  const void* ckv;
  const void* krope;
  long long ckv_stride, krope_stride, cache_rows;
  const float* scale;
  long long scale_stride;
  const int32_t* seq_lens;
  const int32_t* block_table;  // or nullptr
  long long seq_stride;
  void* out;
  long long out_stride, out_seq_stride;
  int batch, max_tokens, d_c, scale_block, max_pages, page_size;
};

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream);
cudaError_t launch_cache_append(CacheFormat format, const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_cache_load(CacheFormat format, const LoadArgs& a, cudaStream_t stream);

}  // namespace hra
