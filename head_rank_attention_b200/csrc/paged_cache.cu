// paged_cache.cu -- the latent cache around the decode: the page plan of a step, the append
// of new tokens and the load of cached rows.
//
// page plan: from the requests' cached lengths and new tokens, the step's block table
//   entries, the slot (cache row) and position of every new token, and the page pool after
//   the step.  One request per thread; exclusive prefix sums of the tokens, of the pages
//   taken and of the pages given back place everything.  A few kilobytes are read and
//   written: latency bounds it, so it is one launch of one thread-block cluster.
// append: a cache row is the token's latent in the cache's format and its RoPE key turned
//   by the token's position.  With one scale per block of tokens and 128-wide latent head,
//   s = max|x| / top over the block; a block that grows token by token keeps the larger of
//   its old scale and the new tokens', and the rows it already holds are brought to it.
// load: rows c * s and RoPE keys back as bf16, the form prefill reads.
// Both are bound by HBM: 2 (d_c + 64) bytes of bf16 and d_c + 128 of cache per token.
#include <climits>

#include "launch.h"
#include "paged_cache.h"
#include "quant.cuh"
#include "sm100.cuh"

namespace hra {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---------------------------------------------------------------------------- page plan
constexpr int kPlanThreads = 1024;  // one per sequence (kMaxBatch)
constexpr int kPlanCluster = 8;

// Exclusive prefix of v over the block's threads, and the total.
__device__ __forceinline__ unsigned long long block_exclusive(unsigned long long v, unsigned long long* warp_sums,
                                                              unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long u = __shfl_up_sync(kAll, incl, off);
    if (lane >= off) incl += u;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  unsigned long long w = warp_sums[lane];
  unsigned long long ws = w;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long u = __shfl_up_sync(kAll, ws, off);
    if (lane >= off) ws += u;
  }
  *total = __shfl_sync(kAll, ws, 31);
  const unsigned long long before = __shfl_sync(kAll, ws - w, warp);
  __syncthreads();  // warp_sums may be written again
  return before + incl - v;
}

// The sequence that owns item i of an exclusive prefix over B sequences (prefix[B] > i).
__device__ __forceinline__ int owner(const int* prefix, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid + 1] > i) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs a) {
  __shared__ unsigned long long warp_sums[32];
  __shared__ int len_s[kPlanThreads], have_s[kPlanThreads];
  __shared__ int start_s[kPlanThreads + 1], take_s[kPlanThreads + 1], give_s[kPlanThreads + 1];
  __shared__ int bad_s;  // refusal code << 16 | sequence, the smallest
  const int t = threadIdx.x, B = a.batch, P = a.page_size;
  const int rank = blockIdx.x, ranks = gridDim.x;
  grid_dep_launch();
  grid_dep_wait();
  if (t == 0) bad_s = INT_MAX;
  __syncthreads();
  const bool mine = t < B;
  const int len = mine ? a.seq_lens[t] : 0;
  const int asked = mine ? a.new_tokens[t] : 0;
  const long long head = a.free_range[0], tail = a.free_range[1];
  const bool gone = asked < 0;
  const int add = gone ? 0 : asked;
  const long long room = static_cast<long long>(a.max_pages) * P;
  const long long after = gone ? 0 : static_cast<long long>(len) + add;
  if (len < 0 || len > room) atomicMin(&bad_s, kPlanBadLength << 16 | t);
  else if (after > room) atomicMin(&bad_s, kPlanTableFull << 16 | t);
  __syncthreads();
  int bad = bad_s;
  const bool sane = bad == INT_MAX;
  const int have = sane ? static_cast<int>((static_cast<long long>(len) + P - 1) / P) : 0;
  const int need = sane && !gone ? static_cast<int>((after + P - 1) / P) - have : 0;
  const int freed = sane && gone ? have : 0;
  unsigned long long pages_total, tokens_total;
  const unsigned long long pages =
      block_exclusive(static_cast<unsigned long long>(freed) << 32 | static_cast<unsigned>(need), warp_sums, &pages_total);
  const unsigned long long tokens = block_exclusive(add, warp_sums, &tokens_total);
  const int need_total = static_cast<int>(pages_total & 0xFFFFFFFFu), freed_total = static_cast<int>(pages_total >> 32);
  const long long avail = tail - head;
  int wanted = 0, limit = 0;
  if (sane) {
    if (head < 0 || avail < 0 || avail > a.num_pages || avail + freed_total > a.num_pages) {
      bad = kPlanBadPool << 16;
    } else if (tokens_total > static_cast<unsigned long long>(a.max_tokens)) {
      bad = kPlanTooManyTokens << 16;
      wanted = tokens_total > INT_MAX ? INT_MAX : static_cast<int>(tokens_total);
      limit = a.max_tokens;
    } else if (need_total > avail) {
      bad = kPlanNoPages << 16;
      wanted = need_total;
      limit = static_cast<int>(avail);
    }
  }
  const bool ok = bad == INT_MAX;
  // Every block has read the lengths and the free range once all have arrived: the outputs
  // may be the inputs' own buffers.
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
  len_s[t] = len;
  have_s[t] = have;
  start_s[t] = ok ? static_cast<int>(tokens) : 0;
  take_s[t] = static_cast<int>(pages & 0xFFFFFFFFu);
  give_s[t] = static_cast<int>(pages >> 32);
  if (t == 0) {
    start_s[kPlanThreads] = ok ? static_cast<int>(tokens_total) : 0;
    take_s[kPlanThreads] = need_total;
    give_s[kPlanThreads] = freed_total;
  }
  __syncthreads();
  const int n_tokens = start_s[kPlanThreads];
  if (rank == 0) {
    if (mine) {
      a.seq_lens_out[t] = ok ? static_cast<int>(after) : len;
      a.query_start[t] = start_s[t];
    }
    if (t == 0) {
      a.query_start[B] = n_tokens;
      a.free_range_out[0] = ok ? head + need_total : head;
      a.free_range_out[1] = ok ? tail + freed_total : tail;
      a.status[0] = ok ? 0 : bad >> 16;
      a.status[1] = ok ? 0 : bad & 0xFFFF;
      a.status[2] = wanted;
      a.status[3] = limit;
    }
  }
  const int threads = ranks * kPlanThreads, me = rank * kPlanThreads + t;
  const int head0 = static_cast<int>(head >= 0 ? head % a.num_pages : 0);
  const int tail0 = static_cast<int>(tail >= 0 ? tail % a.num_pages : 0);
  if (ok) {
    // pages taken: the ring's next ones, in the order of the sequences
    for (int i = me; i < need_total; i += threads) {
      const int s = owner(take_s, B, i);
      int at = head0 + i;
      if (at >= a.num_pages) at -= a.num_pages;
      a.block_table[static_cast<long long>(s) * a.max_pages + have_s[s] + (i - take_s[s])] = a.free_pages[at];
    }
    // pages given back: behind the ring's tail.  The ring holds every page at most once, so
    // these places are not among the ones read above.
    for (int i = me; i < freed_total; i += threads) {
      const int s = owner(give_s, B, i);
      int at = tail0 + i;
      if (at >= a.num_pages) at -= a.num_pages;
      a.free_pages[at] = a.block_table[static_cast<long long>(s) * a.max_pages + (i - give_s[s])];
    }
  }
  for (int i = me; i < a.max_tokens; i += threads) {
    int slot = -1, pos = -1;
    if (i < n_tokens) {
      const int s = owner(start_s, B, i);
      pos = len_s[s] + (i - start_s[s]);
      const int p = pos / P;
      int page;
      if (p < have_s[s]) {
        page = a.block_table[static_cast<long long>(s) * a.max_pages + p];
      } else {
        int at = head0 + take_s[s] + (p - have_s[s]);
        if (at >= a.num_pages) at -= a.num_pages;
        page = a.free_pages[at];
      }
      // a table entry that is no page of the pool has no slot
      slot = page >= 0 && page < a.num_pages ? page * P + (pos - p * P) : -1;
    }
    a.slots[i] = slot;
    if (a.positions != nullptr) a.positions[i] = pos;
  }
}

// ------------------------------------------------------------------------------- append
constexpr int kAppendThreads = 256;
constexpr int kShortRun = 8;  // rows of a run that one warp holds in registers

__device__ __forceinline__ uint32_t abs_max_bits(uint32_t m, uint32_t bf16x2) {
  const uint32_t lo = (bf16x2 << 16) & 0x7FFFFFFFu, hi = bf16x2 & 0x7FFF0000u;
  return max(m, max(lo, hi));
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Four columns of one row: codes to the cache, values to rows_out.
template <CacheFormat F>
__device__ __forceinline__ uint32_t quantize4(uint2 v, float s, float* values) {
  const float x[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
  uint32_t w = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t c = s > 0.f || s != s ? to_code<F>(code_quotient<F>(x[u], s)) : 0u;
    values[u] = code_value<F>(c) * s;
    w |= c << (8 * u);
  }
  return w;
}

// Rows [0, rows) of a block brought from its old scale to its new one, by `n` threads of
// which this one is `me`; a thread takes four columns of a row at a time.
template <CacheFormat F>
__device__ __forceinline__ void rescale_rows(uint8_t* block, long long stride, int rows, float s_old, float s_new, int me,
                                             int n) {
  for (int e = me; e < rows * 32; e += n) {
    uint32_t* p = reinterpret_cast<uint32_t*>(block + (e >> 5) * stride) + (e & 31);
    const uint32_t w = *p;
    uint32_t r = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) r |= rescale_code<F>((w >> (8 * u)) & 0xFFu, s_old, s_new) << (8 * u);
    *p = r;
  }
}

// grid (windows of W tokens, d_c / 128 latent heads + 1): the last y turns the RoPE keys.
//
// Tokens that follow one another in the call and lie in one scale block are a run; the run
// belongs to the window that holds its first token, whatever windows it reaches into.  A
// warp takes a run of up to kShortRun rows by itself (a decode step's runs are one row);
// the block takes longer ones together.  No run needs another's result, so no block waits
// for another.
template <CacheFormat F>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a, int W) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y, groups = a.d_c / 128;
  const int i0 = blockIdx.x * W, i1 = min(i0 + W, a.n_tokens);
  const int rows = static_cast<int>(a.cache_rows);
  grid_dep_launch();
  grid_dep_wait();
  const __nv_bfloat16* latent = static_cast<const __nv_bfloat16*>(a.latent);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.rows_out);

  if (g == groups) {
    // RoPE keys: lane j turns the pair (j, j + 32) by pos * theta^(-2j/64).  The angle is
    // carried in turns in fp64 (positions pass 2^20); its fraction is exact.
    const double turns = exp2(-2.0 * lane / 64.0 * a.log2_theta) * 0.15915494309189535;
    const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(a.krope_in);
    for (int i = i0 + warp; i < i1; i += kAppendThreads / 32) {
      const int slot = a.slots[i];
      if (slot < 0 || slot >= rows) continue;
      const float x1 = __bfloat162float(in[i * a.krope_in_stride + lane]);
      const float x2 = __bfloat162float(in[i * a.krope_in_stride + 32 + lane]);
      const double x = a.positions[i] * turns;
      float sn, cs;
      sincospif(2.f * static_cast<float>(x - rint(x)), &sn, &cs);
      const __nv_bfloat16 y1 = __float2bfloat16_rn(fmaf(x1, cs, -x2 * sn));
      const __nv_bfloat16 y2 = __float2bfloat16_rn(fmaf(x1, sn, x2 * cs));
      __nv_bfloat16* k = static_cast<__nv_bfloat16*>(a.krope) + slot * a.krope_stride;
      k[lane] = y1;
      k[32 + lane] = y2;
      if (out != nullptr) {
        out[i * a.rows_out_stride + a.d_c + lane] = y1;
        out[i * a.rows_out_stride + a.d_c + 32 + lane] = y2;
      }
    }
    return;
  }

  if constexpr (F == kCacheBf16) {
    for (int i = i0 + warp; i < i1; i += kAppendThreads / 32) {
      const int slot = a.slots[i];
      if (slot < 0 || slot >= rows) continue;
      const uint2 v = *reinterpret_cast<const uint2*>(latent + i * a.latent_stride + 128 * g + 4 * lane);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.ckv) + slot * a.ckv_stride + 128 * g + 4 * lane) = v;
      if (out != nullptr) *reinterpret_cast<uint2*>(out + i * a.rows_out_stride + 128 * g + 4 * lane) = v;
    }
  } else {
    __shared__ int long_first[kAppendThreads], n_long;
    __shared__ uint32_t warp_max[kAppendThreads / 32];
    if (threadIdx.x == 0) n_long = 0;
    __syncthreads();
    uint8_t* ckv = static_cast<uint8_t*>(a.ckv) + 128 * g;
    const int blk_rows = a.scale_block;
    auto block_of = [&](int i) {  // the scale block of token i, or -1
      if (i < 0 || i >= a.n_tokens) return -1;
      const int slot = a.slots[i];
      return slot >= 0 && slot < rows ? slot / blk_rows : -1;
    };
    for (int i = i0 + warp; i < i1; i += kAppendThreads / 32) {
      const int blk = block_of(i);
      if (blk < 0 || block_of(i - 1) == blk) continue;
      const uint32_t same = __ballot_sync(kAll, block_of(i + lane) == blk);
      const int len = same == kAll ? 32 : __ffs(~same) - 1;
      if (len > kShortRun) {
        if (lane == 0) long_first[atomicAdd(&n_long, 1)] = i;
        continue;
      }
      uint2 v[kShortRun];
      uint32_t m = 0;
      int first = blk_rows;
#pragma unroll
      for (int r = 0; r < kShortRun; ++r) {
        if (r >= len) break;
        v[r] = *reinterpret_cast<const uint2*>(latent + (i + r) * a.latent_stride + 128 * g + 4 * lane);
        first = min(first, a.slots[i + r] - blk * blk_rows);
      }
#pragma unroll
      for (int r = 0; r < kShortRun; ++r) {
        if (r >= len) break;
        m = abs_max_bits(abs_max_bits(m, v[r].x), v[r].y);
      }
      m = __reduce_max_sync(kAll, m);
      float* sp = a.scale + blk * a.scale_stride + g;
      const float s_old = first > 0 ? *sp : 0.f;
      float s = block_scale<F>(m);
      if (!(s > s_old) && s == s) s = s_old;  // a scale that is no number stays one
      if (first > 0 && s != s_old)
        rescale_rows<F>(ckv + static_cast<long long>(blk) * blk_rows * a.ckv_stride, a.ckv_stride, first, s_old, s, lane, 32);
      __syncwarp();
      if (lane == 0) *sp = s;
#pragma unroll
      for (int r = 0; r < kShortRun; ++r) {
        if (r >= len) break;
        float val[4];
        const uint32_t w = quantize4<F>(v[r], s, val);
        *reinterpret_cast<uint32_t*>(ckv + a.slots[i + r] * a.ckv_stride + 4 * lane) = w;
        if (out != nullptr)
          *reinterpret_cast<uint2*>(out + (i + r) * a.rows_out_stride + 128 * g + 4 * lane) =
              make_uint2(pack_bf16x2(val[0], val[1]), pack_bf16x2(val[2], val[3]));
      }
    }
    __syncthreads();
    for (int k = 0; k < n_long; ++k) {
      const int i = long_first[k];
      const int blk = block_of(i);
      // the run's end, and its first row in the block
      int len = 0, first = blk_rows;
      for (;;) {
        const int mine = i + len + lane;
        const bool in = block_of(mine) == blk;
        const uint32_t same = __ballot_sync(kAll, in);
        if (in && (same == kAll || lane < __ffs(~same) - 1)) first = min(first, a.slots[mine] - blk * blk_rows);
        if (same != kAll) {
          len += __ffs(~same) - 1;
          break;
        }
        len += 32;
      }
      first = __reduce_min_sync(kAll, first);
      uint32_t m = 0;
      for (int r = warp; r < len; r += kAppendThreads / 32) {
        const uint2 v = *reinterpret_cast<const uint2*>(latent + (i + r) * a.latent_stride + 128 * g + 4 * lane);
        m = abs_max_bits(abs_max_bits(m, v.x), v.y);
      }
      m = __reduce_max_sync(kAll, m);
      if (lane == 0) warp_max[warp] = m;
      float* sp = a.scale + blk * a.scale_stride + g;
      const float s_old = first > 0 ? *sp : 0.f;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kAppendThreads / 32; ++w) m = max(m, warp_max[w]);
      float s = block_scale<F>(m);
      if (!(s > s_old) && s == s) s = s_old;
      if (first > 0 && s != s_old)
        rescale_rows<F>(ckv + static_cast<long long>(blk) * blk_rows * a.ckv_stride, a.ckv_stride, first, s_old, s,
                        threadIdx.x, kAppendThreads);
      if (threadIdx.x == 0) *sp = s;
      for (int r = warp; r < len; r += kAppendThreads / 32) {
        const uint2 v = *reinterpret_cast<const uint2*>(latent + (i + r) * a.latent_stride + 128 * g + 4 * lane);
        float val[4];
        const uint32_t w = quantize4<F>(v, s, val);
        *reinterpret_cast<uint32_t*>(ckv + a.slots[i + r] * a.ckv_stride + 4 * lane) = w;
        if (out != nullptr)
          *reinterpret_cast<uint2*>(out + (i + r) * a.rows_out_stride + 128 * g + 4 * lane) =
              make_uint2(pack_bf16x2(val[0], val[1]), pack_bf16x2(val[2], val[3]));
      }
      __syncthreads();  // warp_max is written again
    }
  }
}

// --------------------------------------------------------------------------------- load
constexpr int kLoadThreads = 256;
constexpr int kLoadTokens = 32;  // per block

// grid (tokens / kLoadTokens, B).
template <CacheFormat F>
__global__ void __launch_bounds__(kLoadThreads) cache_load_kernel(const LoadArgs a) {
  __shared__ int row_s[kLoadTokens];
  grid_dep_launch();
  grid_dep_wait();
  const int b = blockIdx.y, t0 = blockIdx.x * kLoadTokens;
  const int n = min(min(a.seq_lens[b], a.max_tokens) - t0, kLoadTokens);
  if (n <= 0) return;
  if (threadIdx.x < n) {
    const int t = t0 + threadIdx.x;
    long long row = static_cast<long long>(b) * a.seq_stride + t;
    if (a.block_table != nullptr) {
      const int p = t / a.page_size;
      const long long page = p < a.max_pages ? a.block_table[static_cast<long long>(b) * a.max_pages + p] : -1;
      row = page < 0 ? -1 : page * a.page_size + t % a.page_size;
    }
    row_s[threadIdx.x] = row >= 0 && row < a.cache_rows ? static_cast<int>(row) : -1;
  }
  __syncthreads();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + b * a.out_seq_stride + t0 * a.out_stride;
  constexpr int COLS = F == kCacheBf16 ? 8 : 16;  // columns of one 16-byte load
  const int per_row = a.d_c / COLS;
  for (int e = threadIdx.x; e < n * per_row; e += kLoadThreads) {
    const int r = e / per_row, c = (e % per_row) * COLS;
    const int row = row_s[r];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint4* dst = reinterpret_cast<uint4*>(out + r * a.out_stride + c);
    if constexpr (F == kCacheBf16) {
      if (row >= 0) v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.ckv) + row * a.ckv_stride + c);
      *dst = v;
    } else {
      float s = 0.f;
      if (row >= 0) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.ckv) + row * a.ckv_stride + c);
        s = a.scale[row / a.scale_block * a.scale_stride + c / 128];
      }
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t two = w[u >> 1] >> (16 * (u & 1));
        o[u] = pack_bf16x2(code_value<F>(two & 0xFFu) * s, code_value<F>((two >> 8) & 0xFFu) * s);
      }
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
  for (int e = threadIdx.x; e < n * 8; e += kLoadThreads) {
    const int r = e >> 3, c = (e & 7) * 8;
    const int row = row_s[r];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0) v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.krope) + row * a.krope_stride + c);
    *reinterpret_cast<uint4*>(out + r * a.out_stride + a.d_c + c) = v;
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream) {
  return launch_kernel_cluster(page_plan_kernel, dim3(kPlanCluster), dim3(kPlanThreads), 0, stream, true, kPlanCluster, a);
}

cudaError_t launch_cache_append(CacheFormat format, const AppendArgs& a, cudaStream_t stream) {
  const int W = 8;
  const dim3 grid((a.n_tokens + W - 1) / W, a.d_c / 128 + 1);
  auto kern = format == kCacheBf16   ? cache_append_kernel<kCacheBf16>
              : format == kCacheInt8 ? cache_append_kernel<kCacheInt8>
                                     : cache_append_kernel<kCacheE4m3>;
  return launch_kernel(kern, grid, dim3(kAppendThreads), 0, stream, true, a, W);
}

cudaError_t launch_cache_load(CacheFormat format, const LoadArgs& a, cudaStream_t stream) {
  const dim3 grid((a.max_tokens + kLoadTokens - 1) / kLoadTokens, a.batch);
  auto kern = format == kCacheBf16   ? cache_load_kernel<kCacheBf16>
              : format == kCacheInt8 ? cache_load_kernel<kCacheInt8>
                                     : cache_load_kernel<kCacheE4m3>;
  return launch_kernel(kern, grid, dim3(kLoadThreads), 0, stream, true, a);
}

}  // namespace hra
