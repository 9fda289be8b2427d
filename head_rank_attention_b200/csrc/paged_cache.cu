// paged_cache.cu -- the latent cache around the decode: the page plan of a step, the append
// of new tokens and the load of cached rows.
//
// page plan: from the requests' cached lengths and new tokens, the step's block table
//   entries, the slot (cache row) and position of every new token, and the page pool after
//   the step.  One request per thread; exclusive prefix sums of the tokens, of the pages
//   taken and of the pages given back place everything.  A few kilobytes are read and
//   written: latency bounds it, so it is one launch, each block scanning all lengths itself
//   (3.4 us for 64 requests, 6.2 us for 1024 with 65536 tokens).
// append: a cache row is the token's latent in the cache's format and its RoPE key turned
//   by the token's position.  With one scale per block of tokens and 128-wide latent head,
//   s = max|x| / top over the block; a block that grows token by token keeps the larger of
//   its old scale and the new tokens', and the rows it already holds are brought to it.
//   2 (d_c + 64) bytes a token in, d_c + 128 of cache and 2 (d_c + 64) of rows out: 5.6 us for 6.8 k
//   tokens of 512 columns (3.0 us of HBM time), 2.9 us for a step of 64 tokens.  The same 6.8 k tokens
//   as bf16 take 4.0 us, with a scale per row (a run each, a warp's work) 21 us.
// load: rows c * s and RoPE keys back as bf16, the form prefill reads.  HBM bounds it: 53 us for
//   160 k rows of 512 columns, 87 % of the rate of a plain copy.
#include <climits>

#include "launch.h"
#include "paged_cache.h"
#include "quant.cuh"
#include "schedule.cuh"
#include "sm100.cuh"

namespace hra {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// These kernels may start while the one in front drains, and wait for it before they read anything.
// What they write is complete for whatever comes behind: another of them waits likewise, and a
// decode, a prefill or a combination begins with a plain launch (launch.h).

// An element's place, past 32 bits in a long cache.
__device__ __forceinline__ long long wide(int row, int stride) { return static_cast<long long>(row) * stride; }

// ---------------------------------------------------------------------------- page plan
constexpr int kPlanMinThreads = 128;
constexpr int kPlanMaxBlocks = 128;
constexpr int kPlanCluster = 8;

// Every block reads all lengths and scans them (one thread for a sequence), and takes its
// share of the pages and tokens (whose sequence is found in the prefix sums, as a tile's is);
// block 0 writes what there is one of for a sequence.  With CLUSTER the blocks are one cluster and
// meet before those writes: the outputs may then be the inputs' own buffers.
template <bool CLUSTER>
__global__ void __launch_bounds__(kMaxBatch) page_plan_kernel(const PlanArgs a) {
  __shared__ unsigned long long sum_pages[32], sum_tokens[32];
  __shared__ int len_s[kMaxBatch], have_s[kMaxBatch], start_s[kMaxBatch], take_s[kMaxBatch], give_s[kMaxBatch];
  __shared__ int bad_s;         // refusal code << 16 | sequence, the smallest
  __shared__ int ring_s[2];     // the ring's head and tail as places
  __shared__ int alien_s;       // the first page to be taken that is none of the pool
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, B = a.batch, P = a.page_size;
  const int n_warps = blockDim.x >> 5;
  grid_dep_wait();
  if (t == 0) bad_s = alien_s = INT_MAX;
  __syncthreads();
  const bool mine = t < B;
  const int len = mine ? a.seq_lens[t] : 0;
  const int asked = mine ? a.new_tokens[t] : 0;
  const long long head = a.free_range[0], tail = a.free_range[1];
  const bool gone = asked < 0;
  const int add = gone ? 0 : asked;
  const long long room = static_cast<long long>(a.max_pages) * P;
  const long long after = gone ? 0 : static_cast<long long>(len) + add;
  const bool bad_len = len < 0 || len > room, full = !bad_len && after > room;
  if (bad_len || full) atomicMin(&bad_s, (bad_len ? kPlanBadLength : kPlanTableFull) << 16 | t);
  // room is below 2^31, so the pages of a good length are
  const int have = bad_len ? 0 : static_cast<int>((static_cast<long long>(len) + P - 1) / P);
  const int need = bad_len || full || gone ? 0 : static_cast<int>((after + P - 1) / P) - have;
  const int freed = gone ? have : 0;
  // prefix sums of both page counts (batch * max_pages is below 2^31) and of the tokens
  const unsigned long long my_pages = static_cast<unsigned long long>(freed) << 32 | static_cast<unsigned>(need);
  unsigned long long pages = my_pages, tokens = static_cast<unsigned>(add);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long p = __shfl_up_sync(kAll, pages, off), q = __shfl_up_sync(kAll, tokens, off);
    if (lane >= off) {
      pages += p;
      tokens += q;
    }
  }
  if (lane == 31) {
    sum_pages[warp] = pages;
    sum_tokens[warp] = tokens;
  }
  if (t == 32) ring_s[0] = static_cast<int>(head >= 0 ? head % a.num_pages : 0);
  if (t == 64) ring_s[1] = static_cast<int>(tail >= 0 ? tail % a.num_pages : 0);
  __syncthreads();
  const int head0 = ring_s[0], tail0 = ring_s[1];
  auto place = [&](int from, int i) { return from + i < a.num_pages ? from + i : from + i - a.num_pages; };
  // the first pages that may be taken, asked for ahead of the sums that say how many are
  const int page0 = t < a.num_pages ? a.free_pages[place(head0, t)] : 0;
  unsigned long long wp = lane < n_warps ? sum_pages[lane] : 0, wt = lane < n_warps ? sum_tokens[lane] : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long p = __shfl_up_sync(kAll, wp, off), q = __shfl_up_sync(kAll, wt, off);
    if (lane >= off) {
      wp += p;
      wt += q;
    }
  }
  const unsigned long long pages_total = __shfl_sync(kAll, wp, 31), tokens_total = __shfl_sync(kAll, wt, 31);
  const unsigned long long pages_before = __shfl_sync(kAll, wp, max(warp - 1, 0));
  const unsigned long long tokens_before = __shfl_sync(kAll, wt, max(warp - 1, 0));
  pages += (warp > 0 ? pages_before : 0) - my_pages;
  tokens += (warp > 0 ? tokens_before : 0) - static_cast<unsigned>(add);
  const int need_total = static_cast<int>(pages_total & 0xFFFFFFFFu), freed_total = static_cast<int>(pages_total >> 32);
  const long long avail = tail - head;
  int bad = bad_s, wanted = 0, limit = 0;
  if (bad == INT_MAX) {
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
  if (bad == INT_MAX) {  // every block looks at all pages to be taken: the step is refused as a whole
    for (int i = t; i < need_total; i += blockDim.x) {
      const int page = i == t ? page0 : a.free_pages[place(head0, i)];
      if (page < 0 || page >= a.num_pages) atomicMin(&alien_s, i);
    }
  }
  if (mine) {
    len_s[t] = len;
    have_s[t] = have;
    start_s[t] = static_cast<int>(tokens);
    take_s[t] = static_cast<int>(pages & 0xFFFFFFFFu);
    give_s[t] = static_cast<int>(pages >> 32);
  }
  // all lengths and the free range are read once every block (every thread of the one) is here
  if constexpr (CLUSTER) {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
  }
  __syncthreads();
  if (alien_s != INT_MAX) {
    bad = kPlanBadPage << 16;
    wanted = place(head0, alien_s);
    limit = a.free_pages[wanted];
  }
  const bool ok = bad == INT_MAX;
  const int n_tokens = ok ? static_cast<int>(tokens_total) : 0;
  if (blockIdx.x == 0) {
    if (mine) {
      a.seq_lens_out[t] = ok ? static_cast<int>(after) : len;
      a.query_start[t] = ok ? static_cast<int>(tokens) : 0;
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
  const int threads = gridDim.x * blockDim.x, me = blockIdx.x * blockDim.x + t;
  if (ok) {
    // pages taken: the ring's next ones, in the order of the sequences
    for (int i = me; i < need_total; i += threads) {
      const int s = seq_of_tile(take_s, B, i);
      a.block_table[static_cast<long long>(s) * a.max_pages + have_s[s] + (i - take_s[s])] = a.free_pages[place(head0, i)];
    }
    // pages given back: behind the ring's tail.  The ring holds every page at most once, so
    // these places are not among the ones read above.
    for (int i = me; i < freed_total; i += threads) {
      const int s = seq_of_tile(give_s, B, i);
      a.free_pages[place(tail0, i)] = a.block_table[static_cast<long long>(s) * a.max_pages + (i - give_s[s])];
    }
  }
  for (int i = me; i < a.max_tokens; i += threads) {
    int slot = -1, pos = -1;
    if (i < n_tokens) {
      const int s = seq_of_tile(start_s, B, i);
      pos = len_s[s] + (i - start_s[s]);
      const int p = pos / P;
      // a cached page from the table, a new one from the ring
      const int page = p < have_s[s] ? a.block_table[static_cast<long long>(s) * a.max_pages + p]
                                     : a.free_pages[place(head0, take_s[s] + (p - have_s[s]))];
      // a table entry that is no page of the pool has no slot
      slot = page >= 0 && page < a.num_pages ? page * P + (pos - p * P) : -1;
    }
    a.slots[i] = slot;
    if (a.positions != nullptr) a.positions[i] = pos;
  }
}

// ------------------------------------------------------------------------------- append
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kShortRun = 8;   // rows of a run that one warp takes by itself
constexpr int kMaxWindow = 64;
constexpr int kMaxScaleBlock = 1024;

// Largest magnitude of eight bf16, kept as the bits of |x| in pairs (their unsigned 16-bit order is
// that of the values, Inf and NaN on top).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint4 v) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  return __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & kMag, v.y & kMag), __vmaxu2(v.z & kMag, v.w & kMag)));
}
// The larger of a pair's, over the warp, as fp32 bits.
__device__ __forceinline__ uint32_t warp_abs_max(uint32_t m2) {
  return __reduce_max_sync(kAll, max(m2 << 16, m2 & 0xFFFF0000u));
}
// The scale of a block whose rows before `first` are kept: the larger of its old one and the
// new rows'; a scale that is no number stays one.
template <CacheFormat F>
__device__ __forceinline__ float grown_scale(uint32_t amax_bits, float s_old) {
  const float s = block_scale<F>(amax_bits);
  return !(s > s_old) && s == s ? s_old : s;
}

// Rows [0, rows) of a block brought from its old scale to its new one, by `n` threads of
// which this one is `me`; a thread takes four columns of a row at a time.
template <CacheFormat F>
__device__ __forceinline__ void rescale_rows(uint8_t* block, int stride, int rows, float s_old, float s_new, int me,
                                             int n) {
#pragma unroll 1
  for (int e = me; e < rows * 32; e += n) {
    uint32_t* p = reinterpret_cast<uint32_t*>(block + wide(e >> 5, stride)) + (e & 31);
    const uint32_t w = *p;
    uint32_t r = 0;
#pragma unroll 1
    for (int u = 0; u < 4; ++u) r |= rescale_code<F>((w >> (8 * u)) & 0xFFu, s_old, s_new) << (8 * u);
    *p = r;
  }
}

// (x1, x2) turned by pos times a turn's fraction `turn` / 2^64.  The angle's nearest quarter turn is taken
// out in integers; sine and cosine of the rest, |r| <= 1/8 turn, are polynomials in r^2
// interpolated at the Chebyshev nodes (errors 2.4e-9 and 4.8e-11, 9e-8 and 7e-8 in fp32 arithmetic).
__device__ __forceinline__ float2 turned(float x1, float x2, unsigned long long turn, int pos) {
  const int t = static_cast<int>((turn * static_cast<unsigned long long>(static_cast<long long>(pos))) >> 32);
  const int q = static_cast<int>((static_cast<uint32_t>(t) + (1u << 29)) >> 30);
  const float r = static_cast<float>(static_cast<int>(static_cast<uint32_t>(t) - (static_cast<uint32_t>(q) << 30))) * 0x1p-32f;
  const float u = r * r;
  float sn = r * fmaf(fmaf(fmaf(-75.40161f, u, 81.592545f), u, -41.341663f), u, 6.2831855f);
  float cs = fmaf(fmaf(fmaf(fmaf(59.2201688f, u, -85.44284467f), u, 64.93931614f), u, -19.73920865f), u, 1.f);
  if (q & 1) {  // a quarter on: (sin, cos) -> (cos, -sin)
    const float c = cs;
    cs = -sn;
    sn = c;
  }
  if (q & 2) {
    cs = -cs;
    sn = -sn;
  }
  return make_float2(fmaf(x1, cs, -x2 * sn), fmaf(x1, sn, x2 * cs));
}

// grid (windows of W tokens, d_c / 128 latent heads + 1): the last y turns the RoPE keys.
//
// Tokens that follow one another in the call and lie in one scale block are a run; the run
// belongs to the window that holds its first token, whatever windows it reaches into.  A
// warp takes a run of up to kShortRun rows by itself (a decode step's runs are one row);
// the block takes longer ones together, and holds the first 64 rows in registers between
// the maximum and the codes.  A lane has 8 columns, a warp two rows at a time.  No run needs
// another's result, so no block waits for another.
template <CacheFormat F>
__global__ void __launch_bounds__(kAppendThreads, 3) cache_append_kernel(const AppendArgs a, int W) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y, groups = a.d_c / 128;
  const int i0 = blockIdx.x * W, n_win = min(W, a.n_tokens - i0);
  const int rows = static_cast<int>(a.cache_rows);
  grid_dep_wait();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.rows_out);

  if (g == groups) {
    // RoPE keys, two tokens to a warp: lane l of a token's 16 turns the pairs (j, j + 32), j = 2 l
    // and 2 l + 1, by pos * theta^(-2j/64).  The angle is a fraction of a turn in 64-bit fixed point:
    // its products with positions wrap at whole turns by themselves.
    constexpr int T = kMaxWindow / (2 * kAppendWarps);  // tokens of a lane, all loaded before any is used
    __shared__ unsigned long long turn_s[32];
    const int half = lane >> 4, l = lane & 15;
    const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(a.krope_in) + 2 * l;
    int slot[T], pos[T];
    uint32_t x1[T], x2[T];
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const int w = 2 * (warp + kAppendWarps * k) + half, i = i0 + w;
      const bool on = w < n_win;
      slot[k] = on ? a.slots[i] : -1;
      pos[k] = on ? a.positions[i] : 0;
      x1[k] = on ? *reinterpret_cast<const uint32_t*>(in + wide(i, a.krope_in_stride)) : 0u;
      x2[k] = on ? *reinterpret_cast<const uint32_t*>(in + wide(i, a.krope_in_stride) + 32) : 0u;
    }
    if (warp == 0) {
      const double turns = exp2(-2.0 * lane / 64.0 * a.log2_theta) * 0.15915494309189535;
      turn_s[lane] = static_cast<unsigned long long>((turns - floor(turns)) * 0x1p64);
    }
    __syncthreads();
    const unsigned long long turn0 = turn_s[2 * l], turn1 = turn_s[2 * l + 1];
#pragma unroll
    for (int k = 0; k < T; ++k) {
      if (slot[k] < 0 || slot[k] >= rows) continue;
      const float2 r0 = turned(__uint_as_float(x1[k] << 16), __uint_as_float(x2[k] << 16), turn0, pos[k]);
      const float2 r1 = turned(__uint_as_float(x1[k] & 0xFFFF0000u), __uint_as_float(x2[k] & 0xFFFF0000u), turn1, pos[k]);
      const uint32_t y1 = pack_bf16x2(r0.x, r1.x), y2 = pack_bf16x2(r0.y, r1.y);
      __nv_bfloat16* key = static_cast<__nv_bfloat16*>(a.krope) + wide(slot[k], a.krope_stride) + 2 * l;
      *reinterpret_cast<uint32_t*>(key) = y1;
      *reinterpret_cast<uint32_t*>(key + 32) = y2;
      if (out != nullptr) {
        __nv_bfloat16* o = out + wide(i0 + 2 * (warp + kAppendWarps * k) + half, a.rows_out_stride) + a.d_c + 2 * l;
        *reinterpret_cast<uint32_t*>(o) = y1;
        *reinterpret_cast<uint32_t*>(o + 32) = y2;
      }
    }
    return;
  }

  const int half = lane >> 4;  // of the warp's two rows
  const int col = 128 * g + 8 * (lane & 15);
  const __nv_bfloat16* latent = static_cast<const __nv_bfloat16*>(a.latent) + col;
  if (out != nullptr) out += col;
  if constexpr (F == kCacheBf16) {
    for (int w = 2 * warp + half; w < n_win; w += 2 * kAppendWarps) {
      const int i = i0 + w, slot = a.slots[i];
      if (slot < 0 || slot >= rows) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(latent + wide(i, a.latent_stride));
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.ckv) + wide(slot, a.ckv_stride) + col) = v;
      if (out != nullptr) *reinterpret_cast<uint4*>(out + wide(i, a.rows_out_stride)) = v;
    }
  } else {
    // The slots of the window, the token before it and the tokens that a run may reach into:
    // slot_s[k] is token i0 - 1 + k's, -1 where there is none or it is no row of the cache.  Bit k
    // of `starts`: token k's scale block is another than the token's before.
    constexpr int kSee = (1 + kMaxWindow + kMaxScaleBlock + 31) / 32 * 32;
    __shared__ int slot_s[kSee];
    __shared__ uint32_t starts[kSee / 32 + 1];
    __shared__ uint32_t warp_max[kAppendWarps];
    const int blk_rows = a.scale_block;
    const int n_see = 1 + W + blk_rows, words = (n_see + 31) / 32;
    auto slot_of = [&](int k) {
      const int i = i0 - 1 + k;
      const int slot = i >= 0 && i < a.n_tokens ? a.slots[i] : -1;
      return slot < rows ? max(slot, -1) : -1;
    };
    if (threadIdx.x == 0) starts[words] = 1u;  // the end of what is seen
    for (int w = warp; w < words; w += kAppendWarps) {
      const int slot = slot_of(32 * w + lane);
      const int edge = lane == 0 && w > 0 ? slot_of(32 * w - 1) : -1;
      const int blk = slot < 0 ? -1 : a.block_of(slot);
      const int before = __shfl_up_sync(kAll, blk, 1);
      const uint32_t bits = __ballot_sync(kAll, blk != (lane > 0 ? before : edge < 0 ? -1 : a.block_of(edge)));
      slot_s[32 * w + lane] = slot;
      if (lane == 0) starts[w] = bits;
    }
    __syncthreads();
    auto run_length = [&](int k) {  // of the run that starts at k
      int w = (k + 1) >> 5;
      uint32_t bits = starts[w] & (0xFFFFFFFFu << ((k + 1) & 31));
      while (bits == 0) bits = starts[++w];
      return 32 * w + __ffs(bits) - 1 - k;
    };
    uint8_t* ckv = static_cast<uint8_t*>(a.ckv);
    // The window's runs, a lane looking at two tokens.
    int my_len[2] = {0, 0};
    unsigned long long runs = 0, long_runs = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (32 * h >= W) break;
      const int w = 32 * h + lane;
      const bool run = w < n_win && (starts[(1 + w) >> 5] >> ((1 + w) & 31) & 1u) != 0 && slot_s[1 + w] >= 0;
      my_len[h] = run ? run_length(1 + w) : 0;
      runs |= static_cast<unsigned long long>(__ballot_sync(kAll, run)) << (32 * h);
      long_runs |= static_cast<unsigned long long>(__ballot_sync(kAll, my_len[h] > kShortRun)) << (32 * h);
    }
    auto length_of = [&](int k0) { return __shfl_sync(kAll, k0 > 32 ? my_len[1] : my_len[0], (k0 - 1) & 31); };
    runs &= ~long_runs;
    for (int turn = 0; runs != 0; runs &= runs - 1, ++turn) {
      if (turn % kAppendWarps != warp) continue;
      const int k0 = __ffsll(runs);  // the token's place in the list: 1 + its bit
      const int len = length_of(k0);
      const int blk = a.block_of(slot_s[k0]), i = i0 - 1 + k0;
      const __nv_bfloat16* src = latent + wide(i, a.latent_stride);
      float* sp = a.scale + wide(blk, a.scale_stride) + g;
      const float s_was = *sp;  // before the rows: one latency
      uint4 v[kShortRun / 2];
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < kShortRun / 2; ++r) {
        v[r] = make_uint4(0u, 0u, 0u, 0u);
        if (2 * r + half < len) v[r] = *reinterpret_cast<const uint4*>(src + wide(2 * r + half, a.latent_stride));
      }
      int first = lane < len ? slot_s[k0 + lane] - blk * blk_rows : blk_rows;
      first = __reduce_min_sync(kAll, first);  // the run's first row in the block
#pragma unroll
      for (int r = 0; r < kShortRun / 2; ++r) m = abs_max2(m, v[r]);
      m = warp_abs_max(m);
      const float s_old = first > 0 ? s_was : 0.f;
      const float s = grown_scale<F>(m, s_old);
      if (first > 0 && s != s_old)
        rescale_rows<F>(ckv + 128 * g + wide(blk * blk_rows, a.ckv_stride), a.ckv_stride, first, s_old, s, lane, 32);
      __syncwarp();
      if (lane == 0) *sp = s;
      auto put = [&](int at, uint2 c) {
        *reinterpret_cast<uint2*>(ckv + wide(slot_s[k0 + at], a.ckv_stride) + col) = c;
        if (out != nullptr) *reinterpret_cast<uint4*>(out + wide(i + at, a.rows_out_stride)) = dequantize8<F>(c, s);
      };
      if (quantize_fast_scale(s)) {
        const float r_s = 1.f / s;
#pragma unroll
        for (int r = 0; r < kShortRun / 2; ++r)
          if (2 * r + half < len) put(2 * r + half, quantize8_fast<F, kAnyScale>(v[r], s, r_s));
      } else {
#pragma unroll 1
        for (int at = half; at < len; at += 2)
          put(at, quantize8_exact<F>(*reinterpret_cast<const uint4*>(src + wide(at, a.latent_stride)), s));
      }
    }
    constexpr int HOLD = 4;  // row pairs of a long run that a warp keeps: 8 warps hold 64 rows
    for (; long_runs != 0; long_runs &= long_runs - 1) {
      const int k0 = __ffsll(long_runs), blk = a.block_of(slot_s[k0]), i = i0 - 1 + k0;
      const int len = length_of(k0);
      const int at0 = 2 * warp + half;
      const __nv_bfloat16* src = latent + wide(i, a.latent_stride);
      float* sp = a.scale + wide(blk, a.scale_stride) + g;
      const float s_was = *sp;
      uint4 v[HOLD];
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < HOLD; ++r) {
        const int at = at0 + 2 * kAppendWarps * r;
        v[r] = make_uint4(0u, 0u, 0u, 0u);
        if (at < len) v[r] = *reinterpret_cast<const uint4*>(src + wide(at, a.latent_stride));
      }
      int first = blk_rows;
      for (int at = lane; at < len; at += 32) first = min(first, slot_s[k0 + at] - blk * blk_rows);
      first = __reduce_min_sync(kAll, first);
      const float s_old = first > 0 ? s_was : 0.f;
#pragma unroll
      for (int r = 0; r < HOLD; ++r) m = abs_max2(m, v[r]);
      for (int at = at0 + 2 * kAppendWarps * HOLD; at < len; at += 2 * kAppendWarps)
        m = abs_max2(m, *reinterpret_cast<const uint4*>(src + wide(at, a.latent_stride)));
      m = warp_abs_max(m);
      if (lane == 0) warp_max[warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kAppendWarps; ++w) m = max(m, warp_max[w]);
      const float s = grown_scale<F>(m, s_old);
      if (first > 0 && s != s_old)
        rescale_rows<F>(ckv + 128 * g + wide(blk * blk_rows, a.ckv_stride), a.ckv_stride, first, s_old, s, threadIdx.x,
                        kAppendThreads);
      if (threadIdx.x == 0) *sp = s;
      auto put = [&](int at, uint2 c) {
        *reinterpret_cast<uint2*>(ckv + wide(slot_s[k0 + at], a.ckv_stride) + col) = c;
        if (out != nullptr) *reinterpret_cast<uint4*>(out + wide(i + at, a.rows_out_stride)) = dequantize8<F>(c, s);
      };
      float r_s = 0.f;
      const QuantMode mode = quantize_mode<F>(__uint_as_float(m), s, &r_s);
      int rest = at0;  // rows not in registers, and all of them under scales that need fp64
      if (quantize_fast_scale(s)) {
        rest += 2 * kAppendWarps * HOLD;
        auto put_held = [&](auto quantize) {
#pragma unroll
          for (int r = 0; r < HOLD; ++r)
            if (at0 + 2 * kAppendWarps * r < len) put(at0 + 2 * kAppendWarps * r, quantize(v[r]));
        };
        if (mode == kOwnScale) put_held([&](uint4 x) { return quantize8_fast<F, kOwnScale>(x, s, r_s); });
        else if (mode == kExactScale) put_held([&](uint4 x) { return quantize8_fast<F, kExactScale>(x, s, r_s); });
        else put_held([&](uint4 x) { return quantize8_fast<F, kAnyScale>(x, s, r_s); });
      }
#pragma unroll 1
      for (int at = rest; at < len; at += 2 * kAppendWarps)
        put(at, quantize8_exact<F>(*reinterpret_cast<const uint4*>(src + wide(at, a.latent_stride)), s));
      __syncthreads();  // warp_max is written again
    }
  }
}

// --------------------------------------------------------------------------------- load
constexpr int kLoadThreads = 256;
constexpr int kLoadTokens = 32;  // most of a block

// grid (tokens / per_block, B).  A thread has one 16-byte load in flight and its stores: with two
// or four the long loads were slower (56 to 62 us instead of 53 for 160 k rows), reads and writes
// coming in longer turns.
template <CacheFormat F>
__global__ void __launch_bounds__(kLoadThreads) cache_load_kernel(const LoadArgs a, int per_block) {
  __shared__ int row_s[kLoadTokens];
  grid_dep_wait();
  const int b = blockIdx.y, t0 = blockIdx.x * per_block;
  const int n = min(min(a.seq_lens[b], a.max_tokens) - t0, per_block);
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
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + b * a.out_seq_stride + wide(t0, a.out_stride);
  constexpr int COLS = F == kCacheBf16 ? 8 : 16;  // columns of one 16-byte load
  const int per_row = a.d_c / COLS, shift = __ffs(per_row) - 1;
  for (int e = threadIdx.x; e < n * per_row; e += kLoadThreads) {
    const int r = e >> shift, c = (e & (per_row - 1)) * COLS;
    const int row = row_s[r];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    uint4* dst = reinterpret_cast<uint4*>(out + wide(r, a.out_stride) + c);
    if constexpr (F == kCacheBf16) {
      if (row >= 0) v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.ckv) + wide(row, a.ckv_stride) + c);
      *dst = v;
    } else {
      float s = 0.f;
      if (row >= 0) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.ckv) + wide(row, a.ckv_stride) + c);
        s = a.scale[wide(a.block_of(row), a.scale_stride) + c / 128];
      }
      dst[0] = dequantize8<F>(make_uint2(v.x, v.y), s);
      dst[1] = dequantize8<F>(make_uint2(v.z, v.w), s);
    }
  }
  for (int e = threadIdx.x; e < n * 8; e += kLoadThreads) {
    const int r = e >> 3, c = (e & 7) * 8;
    const int row = row_s[r];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0) v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.krope) + wide(row, a.krope_stride) + c);
    *reinterpret_cast<uint4*>(out + wide(r, a.out_stride) + a.d_c + c) = v;
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream) {
  // A thread for a sequence, and a token or so for a thread: a step of 64 requests is one block of
  // 128, and 65536 tokens are spread over 64 SMs.  Blocks that read lengths which another block
  // overwrites must meet, in one cluster of 8: 13.4 us for 1024 requests and 65536 tokens in place, 6.0 in
  // buffers of their own.
  const int threads = (a.batch > kPlanMinThreads ? a.batch + 31 : kPlanMinThreads) / 32 * 32;
  const int blocks = (a.max_tokens + threads - 1) / threads;
  const bool in_place = a.seq_lens == a.seq_lens_out || a.free_range == a.free_range_out;
  if (!in_place || blocks == 1)
    return launch_kernel(page_plan_kernel<false>, dim3(blocks < kPlanMaxBlocks ? blocks : kPlanMaxBlocks), dim3(threads), 0, stream, true, a);
  return launch_kernel_cluster(page_plan_kernel<true>, dim3(kPlanCluster), dim3(threads), 0, stream, true, kPlanCluster, a);
}

cudaError_t launch_cache_append(CacheFormat format, const AppendArgs& a, cudaStream_t stream) {
  // Windows of 8 tokens, a warp each, while a call can be a decode step (at most kMaxBatch
  // runs); longer calls are prompts, whose runs the block takes together: a window of a block's
  // length has one, more or less.
  const int W = a.n_tokens <= kMaxBatch ? 8 : a.scale_block >= kMaxWindow ? kMaxWindow : 32;
  const dim3 grid((a.n_tokens + W - 1) / W, a.d_c / 128 + 1);
  auto kern = format == kCacheBf16   ? cache_append_kernel<kCacheBf16>
              : format == kCacheInt8 ? cache_append_kernel<kCacheInt8>
                                     : cache_append_kernel<kCacheE4m3>;
  return launch_kernel(kern, grid, dim3(kAppendThreads), 0, stream, true, a, W);
}

cudaError_t launch_cache_load(CacheFormat format, const LoadArgs& a, cudaStream_t stream) {
  // Blocks of 32 tokens, or of 16 where that leaves SMs idle (2048 tokens: 0.5 us less, 2.5 in all;
  // long loads gain 2 % from the larger).
  const int per_block = static_cast<long long>((a.max_tokens + kLoadTokens - 1) / kLoadTokens) * a.batch < 2 * 148 ? 16 : kLoadTokens;
  const dim3 grid((a.max_tokens + per_block - 1) / per_block, a.batch);
  auto kern = format == kCacheBf16   ? cache_load_kernel<kCacheBf16>
              : format == kCacheInt8 ? cache_load_kernel<kCacheInt8>
                                     : cache_load_kernel<kCacheE4m3>;
  return launch_kernel(kern, grid, dim3(kLoadThreads), 0, stream, true, a, per_block);
}

}  // namespace hra
