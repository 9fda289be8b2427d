// api_cache.cu -- the C ABI of the paged cache around the decode (hra.h): argument checks
// and launches of the page plan, the append and the load.  Nothing here allocates device
// memory or waits, except hra_check_plan_status, which synchronizes its stream.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "hra.h"
#include "paged_cache.h"
#include "schedule.cuh"

namespace hra {
void set_last_error(const char* msg);  // api.cu
}  // namespace hra

namespace {

hra_status fail(hra_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  hra::set_last_error(buf);
  return st;
}

hra_status done(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(HRA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  hra::set_last_error("");
  return HRA_OK;
}

// Most tokens of a call: token numbers and a grid's strides past them stay below 2^31.
constexpr int kMaxTokens = 1 << 30;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

hra_status check_pointer(const void* p, unsigned n, const char* name) {
  if (p == nullptr) return fail(HRA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, n)) return fail(HRA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, n);
  return HRA_OK;
}

// What an append and a load say about the cache, in the same terms.
struct CacheView {
  int d_c, d_rope;
  const void *ckv, *krope;
  long long ckv_stride, krope_stride, cache_rows;
  int dtype;
  const float* scale;
  long long scale_stride;
  int scale_block;
};

hra_status check_cache(const CacheView& c) {
  if ((c.d_c != 128 && c.d_c != 256 && c.d_c != 512) || c.d_rope != 64)
    return fail(HRA_ERR_UNSUPPORTED, "widths (d_c=%d, d_rope=%d): d_c must be 128, 256 or 512, d_rope 64", c.d_c, c.d_rope);
  hra_status st;
  if ((st = check_pointer(c.ckv, 16, "ckv")) != HRA_OK) return st;
  if ((st = check_pointer(c.krope, 16, "krope")) != HRA_OK) return st;
  const bool byte = c.dtype == HRA_INT8 || c.dtype == HRA_E4M3;
  if (!byte && c.dtype != HRA_BF16) return fail(HRA_ERR_INVALID_ARG, "cache_dtype=%d (HRA_BF16, HRA_INT8 or HRA_E4M3)", c.dtype);
  if (c.ckv_stride < c.d_c || c.ckv_stride % (byte ? 16 : 8) != 0)
    return fail(HRA_ERR_INVALID_ARG, "ckv_stride=%lld must be >= d_c=%d and a multiple of %d", c.ckv_stride, c.d_c, byte ? 16 : 8);
  if (c.krope_stride < 64 || c.krope_stride % 8 != 0)
    return fail(HRA_ERR_INVALID_ARG, "krope_stride=%lld must be >= 64 and a multiple of 8", c.krope_stride);
  if (c.ckv_stride > INT_MAX || c.krope_stride > INT_MAX || c.scale_stride > INT_MAX)
    return fail(HRA_ERR_UNSUPPORTED, "row strides must be below 2^31");
  if (c.cache_rows < 1 || c.cache_rows > INT_MAX)
    return fail(HRA_ERR_INVALID_ARG, "cache_rows=%lld out of range [1, 2^31-1]", c.cache_rows);
  if (!byte) {
    if (c.scale_block > 1) return fail(HRA_ERR_INVALID_ARG, "scale_block=%d needs an 8-bit cache", c.scale_block);
    return HRA_OK;
  }
  if (c.scale == nullptr || !aligned(c.scale, 4)) return fail(HRA_ERR_INVALID_ARG, "ckv_scale is NULL or not 4-byte aligned");
  if (c.scale_stride < c.d_c / 128)
    return fail(HRA_ERR_INVALID_ARG, "ckv_scale_stride=%lld must be >= d_c / 128", c.scale_stride);
  if (c.scale_block < 0 || c.scale_block > 1024 || (c.scale_block > 1 && c.scale_block % 32 != 0))
    return fail(HRA_ERR_UNSUPPORTED, "scale_block=%d (supported: 0 or 1, or a multiple of 32 up to 1024)", c.scale_block);
  if (c.dtype == HRA_E4M3 && c.scale_block <= 1)
    return fail(HRA_ERR_UNSUPPORTED, "an e4m3 cache needs scale_block (one scale per block of rows)");
  return HRA_OK;
}

hra::CacheFormat format_of(int dtype) {
  return dtype == HRA_BF16 ? hra::kCacheBf16 : dtype == HRA_INT8 ? hra::kCacheInt8 : hra::kCacheE4m3;
}

hra_status run_plan(const hra_plan_params* p, cudaStream_t stream) {
  if (p == nullptr) return fail(HRA_ERR_INVALID_ARG, "params is NULL");
  if (p->batch < 1 || p->batch > hra::kMaxBatch)
    return fail(HRA_ERR_UNSUPPORTED, "batch=%d (supported: 1..%d)", p->batch, hra::kMaxBatch);
  if (p->page_size < 32 || p->page_size % 32 != 0)
    return fail(HRA_ERR_UNSUPPORTED, "page_size=%d must be a positive multiple of 32", p->page_size);
  if (p->max_pages < 1 || p->num_pages < 1 || p->max_tokens < 1)
    return fail(HRA_ERR_INVALID_ARG, "max_pages=%d, num_pages=%d, max_tokens=%d must be >= 1", p->max_pages, p->num_pages,
                p->max_tokens);
  if (p->max_tokens > kMaxTokens) return fail(HRA_ERR_UNSUPPORTED, "max_tokens=%d is above 2^30", p->max_tokens);
  if (static_cast<long long>(p->batch) * p->max_pages > INT_MAX || static_cast<long long>(p->max_pages) * p->page_size > INT_MAX ||
      static_cast<long long>(p->num_pages) * p->page_size > INT_MAX)
    return fail(HRA_ERR_UNSUPPORTED, "batch * max_pages, max_pages * page_size and num_pages * page_size must be below 2^31");
  const struct { const void* ptr; unsigned align; const char* name; } ptrs[] = {
      {p->seq_lens, 4, "seq_lens"}, {p->new_tokens, 4, "new_tokens"}, {p->block_table, 4, "block_table"},
      {p->free_pages, 4, "free_pages"}, {p->free_range, 8, "free_range"}, {p->seq_lens_out, 4, "seq_lens_out"},
      {p->free_range_out, 8, "free_range_out"}, {p->query_start, 4, "query_start"}, {p->slots, 4, "slots"},
      {p->status, 4, "status"}};
  for (const auto& x : ptrs) {
    hra_status st = check_pointer(x.ptr, x.align, x.name);
    if (st != HRA_OK) return st;
  }
  if (!aligned(p->positions, 4)) return fail(HRA_ERR_INVALID_ARG, "positions is not 4-byte aligned");
  hra::PlanArgs a{};
  a.seq_lens = p->seq_lens;
  a.new_tokens = p->new_tokens;
  a.block_table = p->block_table;
  a.free_pages = p->free_pages;
  a.free_range = p->free_range;
  a.seq_lens_out = p->seq_lens_out;
  a.free_range_out = p->free_range_out;
  a.query_start = p->query_start;
  a.slots = p->slots;
  a.positions = p->positions;
  a.status = p->status;
  a.batch = p->batch;
  a.page_size = p->page_size;
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  a.max_tokens = p->max_tokens;
  return done(hra::launch_page_plan(a, stream), "page_plan launch");
}

hra_status read_plan_status(const hra_plan_params* p, cudaStream_t stream) {
  if (p == nullptr || p->status == nullptr) return fail(HRA_ERR_INVALID_ARG, "params or status is NULL");
  int st[4] = {0, 0, 0, 0};
  cudaError_t e = cudaMemcpyAsync(st, p->status, sizeof(st), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return done(e, "plan status read");
  switch (st[0]) {
    case hra::kPlanOk: return done(cudaSuccess, "");
    case hra::kPlanBadLength:
      return fail(HRA_ERR_PLAN, "sequence %d: cached length negative or longer than its block table row", st[1]);
    case hra::kPlanTableFull: return fail(HRA_ERR_PLAN, "sequence %d needs more than max_pages pages", st[1]);
    case hra::kPlanTooManyTokens: return fail(HRA_ERR_PLAN, "%d new tokens, max_tokens=%d", st[2], st[3]);
    case hra::kPlanNoPages: return fail(HRA_ERR_PLAN, "%d pages needed, %d free", st[2], st[3]);
    case hra::kPlanBadPage:
      return fail(HRA_ERR_PLAN, "place %d of the ring of free pages holds %d, which is no page of the pool", st[2], st[3]);
    default: return fail(HRA_ERR_PLAN, "the free range does not describe a ring of num_pages pages (code %d)", st[0]);
  }
}

hra_status run_append(const hra_append_params* p, cudaStream_t stream) {
  if (p == nullptr) return fail(HRA_ERR_INVALID_ARG, "params is NULL");
  if (p->n_tokens < 1) return fail(HRA_ERR_INVALID_ARG, "n_tokens=%d must be >= 1", p->n_tokens);
  if (p->n_tokens > kMaxTokens) return fail(HRA_ERR_UNSUPPORTED, "n_tokens=%d is above 2^30", p->n_tokens);
  const CacheView c = {p->d_c, p->d_rope, p->ckv, p->krope, p->ckv_stride, p->krope_stride, p->cache_rows, p->cache_dtype,
                       p->ckv_scale, p->ckv_scale_stride, p->scale_block};
  hra_status st = check_cache(c);
  if (st != HRA_OK) return st;
  if ((st = check_pointer(p->latent, 16, "latent")) != HRA_OK) return st;
  if ((st = check_pointer(p->krope_in, 16, "krope_in")) != HRA_OK) return st;
  if ((st = check_pointer(p->slots, 4, "slots")) != HRA_OK) return st;
  if ((st = check_pointer(p->positions, 4, "positions")) != HRA_OK) return st;
  if (p->latent_stride < p->d_c || p->latent_stride % 8 != 0)
    return fail(HRA_ERR_INVALID_ARG, "latent_stride=%lld must be >= d_c=%d and a multiple of 8", (long long)p->latent_stride, p->d_c);
  if (p->krope_in_stride < 64 || p->krope_in_stride % 8 != 0)
    return fail(HRA_ERR_INVALID_ARG, "krope_in_stride=%lld must be >= 64 and a multiple of 8", (long long)p->krope_in_stride);
  if (p->latent_stride > INT_MAX || p->krope_in_stride > INT_MAX || (p->rows_out != nullptr && p->rows_out_stride > INT_MAX))
    return fail(HRA_ERR_UNSUPPORTED, "row strides must be below 2^31");
  if (p->rows_out != nullptr) {
    if (!aligned(p->rows_out, 16)) return fail(HRA_ERR_INVALID_ARG, "rows_out is not 16-byte aligned");
    if (p->rows_out_stride < p->d_c + 64 || p->rows_out_stride % 8 != 0)
      return fail(HRA_ERR_INVALID_ARG, "rows_out_stride=%lld must be >= d_c + 64 and a multiple of 8", (long long)p->rows_out_stride);
  }
  if (!(p->rope_theta > 0.f) || !std::isfinite(p->rope_theta)) return fail(HRA_ERR_INVALID_ARG, "rope_theta must be finite and > 0");
  hra::AppendArgs a{};
  a.latent = p->latent;
  a.krope_in = p->krope_in;
  a.latent_stride = static_cast<int>(p->latent_stride);
  a.krope_in_stride = static_cast<int>(p->krope_in_stride);
  a.slots = p->slots;
  a.positions = p->positions;
  a.ckv = p->ckv;
  a.krope = p->krope;
  a.ckv_stride = static_cast<int>(p->ckv_stride);
  a.krope_stride = static_cast<int>(p->krope_stride);
  a.cache_rows = p->cache_rows;
  a.scale = p->ckv_scale;
  a.scale_stride = static_cast<int>(p->ckv_scale_stride);
  a.rows_out = p->rows_out;
  a.rows_out_stride = static_cast<int>(p->rows_out_stride);
  a.log2_theta = std::log2(static_cast<double>(p->rope_theta));
  a.n_tokens = p->n_tokens;
  a.d_c = p->d_c;
  a.scale_block = p->scale_block > 1 ? p->scale_block : 1;
  a.block_of = hra::RowDivisor(a.scale_block);
  return done(hra::launch_cache_append(format_of(p->cache_dtype), a, stream), "cache_append launch");
}

hra_status run_load(const hra_load_params* p, cudaStream_t stream) {
  if (p == nullptr) return fail(HRA_ERR_INVALID_ARG, "params is NULL");
  if (p->batch < 1 || p->batch > hra::kMaxBatch)
    return fail(HRA_ERR_UNSUPPORTED, "batch=%d (supported: 1..%d)", p->batch, hra::kMaxBatch);
  if (p->max_tokens < 1) return fail(HRA_ERR_INVALID_ARG, "max_tokens=%d must be >= 1", p->max_tokens);
  if (p->max_tokens > kMaxTokens) return fail(HRA_ERR_UNSUPPORTED, "max_tokens=%d is above 2^30", p->max_tokens);
  const CacheView c = {p->d_c, p->d_rope, p->ckv, p->krope, p->ckv_stride, p->krope_stride, p->cache_rows, p->cache_dtype,
                       p->ckv_scale, p->ckv_scale_stride, p->scale_block};
  hra_status st = check_cache(c);
  if (st != HRA_OK) return st;
  if ((st = check_pointer(p->seq_lens, 4, "seq_lens")) != HRA_OK) return st;
  if ((st = check_pointer(p->out, 16, "out")) != HRA_OK) return st;
  if (p->block_table != nullptr) {
    if (!aligned(p->block_table, 4)) return fail(HRA_ERR_INVALID_ARG, "block_table is not 4-byte aligned");
    if (p->max_pages < 1) return fail(HRA_ERR_INVALID_ARG, "max_pages=%d must be >= 1", p->max_pages);
    if (p->page_size < 32 || p->page_size % 32 != 0)
      return fail(HRA_ERR_UNSUPPORTED, "page_size=%d must be a positive multiple of 32", p->page_size);
  } else if (p->seq_stride < 0) {
    return fail(HRA_ERR_INVALID_ARG, "seq_stride=%lld must be >= 0", (long long)p->seq_stride);
  }
  if (p->out_stride < p->d_c + 64 || p->out_stride % 8 != 0)
    return fail(HRA_ERR_INVALID_ARG, "out_stride=%lld must be >= d_c + 64 and a multiple of 8", (long long)p->out_stride);
  if (p->out_stride > INT_MAX) return fail(HRA_ERR_UNSUPPORTED, "row strides must be below 2^31");
  if (p->out_seq_stride < 0 || p->out_seq_stride % 8 != 0)
    return fail(HRA_ERR_INVALID_ARG, "out_seq_stride=%lld must be >= 0 and a multiple of 8", (long long)p->out_seq_stride);
  hra::LoadArgs a{};
  a.ckv = p->ckv;
  a.krope = p->krope;
  a.ckv_stride = static_cast<int>(p->ckv_stride);
  a.krope_stride = static_cast<int>(p->krope_stride);
  a.cache_rows = p->cache_rows;
  a.scale = p->ckv_scale;
  a.scale_stride = static_cast<int>(p->ckv_scale_stride);
  a.seq_lens = p->seq_lens;
  a.block_table = p->block_table;
  a.seq_stride = p->seq_stride;
  a.out = p->out;
  a.out_stride = static_cast<int>(p->out_stride);
  a.out_seq_stride = p->out_seq_stride;
  a.batch = p->batch;
  a.max_tokens = p->max_tokens;
  a.d_c = p->d_c;
  a.block_of = hra::RowDivisor(p->scale_block > 1 ? p->scale_block : 1);
  a.max_pages = p->max_pages;
  a.page_size = p->page_size;
  return done(hra::launch_cache_load(format_of(p->cache_dtype), a, stream), "cache_load launch");
}

}  // namespace

extern "C" {

hra_status hra_page_plan(const hra_plan_params* p, void* stream) {
  return run_plan(p, static_cast<cudaStream_t>(stream));
}

hra_status hra_check_plan_status(const hra_plan_params* p, void* stream) {
  return read_plan_status(p, static_cast<cudaStream_t>(stream));
}

hra_status hra_cache_append(const hra_append_params* p, void* stream) {
  return run_append(p, static_cast<cudaStream_t>(stream));
}

hra_status hra_cache_load(const hra_load_params* p, void* stream) {
  return run_load(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
