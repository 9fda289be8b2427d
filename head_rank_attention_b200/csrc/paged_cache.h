// paged_cache.h -- host-side interface of the kernels that fill and read the paged latent
// cache: the page plan of a step, the append of new tokens and the load of cached rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace hra {

// Formats of the cached latent (the RoPE key is bf16 in all of them).
enum CacheFormat : int { kCacheBf16 = 0, kCacheInt8 = 1, kCacheE4m3 = 2 };

// Division of a row number (below 2^31) by a divisor d of at most 2^20 as a multiplication: with l the bits of
// d - 1 and m = ceil(2^(31 + l) / d), n / d = n * m >> (31 + l), as m d - 2^(31 + l) < 2^l.
struct RowDivisor {
  uint32_t mul = 0;
  int shift = 0;
  RowDivisor() = default;
  explicit RowDivisor(int d) {
    int l = 0;
    while ((1 << l) < d) ++l;
    shift = 31 + l;
    mul = static_cast<uint32_t>(((uint64_t(1) << shift) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
#endif
};

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
  kPlanBadPage = 6,        // status[2] = place in the ring, status[3] = the page there, which is none of the pool
};

struct AppendArgs {  // see hra_append_params
  const void* latent;
  const void* krope_in;
  int latent_stride, krope_in_stride;  // bf16 elements (row strides are below 2^31: an address is one
                                       //   32 x 32 -> 64-bit multiplication)
  const int32_t* slots;
  const int32_t* positions;
  void* ckv;
  void* krope;
  int ckv_stride, krope_stride;  // elements of the cache's types
  long long cache_rows;
  float* scale;
  int scale_stride;
  void* rows_out;  // or nullptr
  int rows_out_stride;
  double log2_theta;
  int n_tokens, d_c, scale_block;
  RowDivisor block_of;  // by scale_block
};

struct LoadArgs {  // see hra_load_params
  const void* ckv;
  const void* krope;
  int ckv_stride, krope_stride;
  long long cache_rows;
  const float* scale;
  int scale_stride;
  const int32_t* seq_lens;
  const int32_t* block_table;  // or nullptr
  long long seq_stride;
  void* out;
  int out_stride;
  long long out_seq_stride;
  int batch, max_tokens, d_c, max_pages, page_size;
  RowDivisor block_of;  // by the rows that share a scale
};

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream);
cudaError_t launch_cache_append(CacheFormat format, const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_cache_load(CacheFormat format, const LoadArgs& a, cudaStream_t stream);

}  // namespace hra
