// decode_block_sm100.cu -- split-KV decode over a latent cache held in 8 bits (int8 or e4m3)
// with one scale for each block of rows and 128-wide latent head, on tcgen05/TMEM.
//
// The step is the decode of decode_split_sm100.cu ("Multi-Head Low-Rank Attention",
// 方法步骤详情, step 2): a CTA is one 128-wide branch of one group's tiles, the query is
// fp16, a tile is fp16 in shared memory, and both products are kind::f16 MMAs with fp32
// accumulation.  What a block scale changes is the arithmetic around them.
//
// Scales.  All rows of a 32-row chunk share the scale s = f * 2^e (f in [1, 2)).  The
// converter writes code * 2^(e - E), with E = e kept in [kMinExp, kMaxExp]: the codes themselves,
// but for scales outside that range, whose codes are shifted (a value is resolved to
// 2^(kMinExp - 24)).  The RoPE key is divided by sigma = f * 2^E in fp32 and rounded to fp16 (half a
// step is 2^-11 of it, or 2^-21 sigma where that is more).  The MMA then gives score / sigma for
// the latent and the RoPE part alike, and the softmax multiplies by its chunk's sigma: the scale
// enters the latent's scores without a rounding.  The values need f * 2^E as well: the softmax works
// on x = score + log2(sigma), so that P = 2^(x - M) times the converted tile is the scaled value,
// and the denominator adds P / sigma, one multiplication per chunk.  M is then the largest weight
// times scale, P (fp16) is rounded by 2^-11 of itself or 2^-25 of that largest, and partial states
// keep their meaning: (M, l) with O and l both in units of 2^M.  E is the chunk's own: with one for
// the tile, codes beside a scale 2^25 times theirs vanished, and RoPE keys became subnormal.
//
// Work decomposition: schedule.cuh, with 96-token tiles.  Even and odd tiles of a CTA are two
// streams, each with its own softmax warpgroup, score buffer, O and (M, l): one stream's
// softmax runs while the tensor core works for the other, and nothing passes between
// them until the segment's end, where they are added.  A thread owns one head row of a
// tile, so that no row is split over threads.
//
// TMEM (512 columns): O of the streams [0, 128), [128, 256) | scores [256, 352), [352, 448) |
// q~ latent fp16 [448, 512).  P (fp16 pairs) is written over the first 48 score columns.
// The rope query is in shared memory (the 4 rope MMAs read A from there).
//
// Warp roles (16 warps, 4 warpgroups):
//   0-3, 4-7   softmax of stream 0, 1 (thread = head row = TMEM lane)
//   8-10, 11-13  converters of even and odd tiles (thread = cache row)
//   14         TMA producer: rows and chunk scales, one batch of 10 tiles ahead
//   15         TMEM allocator, issuer of both products: PV(i), QK(i + 2), PV(i + 1), ...
//              in one thread, whose MMAs run in order: QK(i + 2) may overwrite the buffer
//              that PV(i) reads without a wait.
// Every wait is bounded, as in decode_split_sm100.cu.
//
// What bounds it: a 96-token tile takes 1740 to 1910 cycles in a long loop, half of a stream's P.V and
// QK (1310 to the scores), maximum (480), exponentials (1060), P (150) and the way to the next issue
// (340); the tensor core is busy 46 % of the time, shared memory 55 to 70 % (160 KB a tile), and an
// operation on it takes 150 to 200 cycles under that load.  64 x 32 k tokens, int8, h = 128: 592 tiles
// a CTA in 1.107 M cycles, 17 k of them before the first scores, 4 to 6 k at the end of each of
// three segments; 660 us (a mean of 1.68 GHz; 2.0 TB/s of cache, 0.89 PFLOP/s), some 760 under steady
// load, where the board's power cap sets the clock; the row-scaled kernel takes 1096 for the same
// tokens.  128-token tiles or three groups on one O were equal or slower: they must hand M from tile to
// tile.
#include <cstdint>

#include "decode_sm100.h"
#include "launch.h"
#include "schedule.cuh"
#include "sm100.cuh"

namespace hra {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// E's range.  The rope key is multiplied by 1 / sigma 2^-kRopeShift, at most 2^(-kMinExp - kRopeShift)
// = 2^4, and the rope query by 2^kRopeShift: keys and queries below 4000 stay in fp16's range
// whatever the scales.  Below kMinExp codes are shifted down instead (exact until s = 2^-23);
// above kMaxExp, up.
constexpr int kMinExp = -8, kMaxExp = 10, kRopeShift = 4;

struct BlockCfg {
  static constexpr int NT = 96;
  static constexpr int W = 128;
  static constexpr int BOX_BYTES = NT * 128;            // 64 16-bit columns (or 128 codes) of the tile's rows
  // Two rings.  A tile's copy (codes, and the RoPE key, converted in place) is held until its
  // QK has run; its fp16 latent (columns 0-63, 64-127) from the conversion until its P.V has.
  // One ring for both (36 KB a tile, held 7900 cycles from copy to P.V) made 1980 cycles a tile.
  static constexpr int RAW = 4, LAT = 4;
  static constexpr int RAW_BYTES = 2 * BOX_BYTES, LAT_BYTES = 2 * BOX_BYTES;
  static constexpr int PAR = 8;  // chunk parameters outlive the copy: until the tile's softmax
  static constexpr int CHUNKS = NT / 32;
  static constexpr int TMEM_O = 0, TMEM_S = 256, TMEM_Q = 448, TMEM_COLS = 512;
  static constexpr int WARP_CONV = 8, CONV_WARPS = 3, WARP_PRODUCER = 14, WARP_MMA = 15;
  static constexpr int THREADS = 512;
  // setmaxnreg: 256 softmax threads and 256 others share the 128 * 512 registers of the launch
  static constexpr int LAUNCH_REGS = 128;
  static constexpr int SOFTMAX_REGS = 160, OTHER_REGS = 96;
  static constexpr int QR_BYTES = 128 * 128;
  static constexpr int BAR_BYTES = 512;
  static constexpr int ML_BYTES = 2 * 128 * 8;
  static constexpr int PAR_BYTES = PAR * CHUNKS * 32;  // ChunkParams
  static constexpr int MISC_BYTES = BAR_BYTES + ML_BYTES + PAR_BYTES + 4 * (kMaxBatch + 1);
  static constexpr int SMEM_BYTES = 1024 + RAW * RAW_BYTES + LAT * LAT_BYTES + QR_BYTES + MISC_BYTES;
  static_assert((SOFTMAX_REGS + OTHER_REGS) * 256 == LAUNCH_REGS * THREADS, "register split");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(PAR >= RAW + 4, "chunk parameters");
  // A team waits only for its own tiles' copies, and copies may land out of order: were a stage
  // of that ring shared by the teams, one could take the other's pending phase of it for its
  // own.  (P.V's complete in order, so the other ring needs no such care.)
  static_assert(RAW % 2 == 0, "a stage belongs to one converter team");
};

// What a 32-row chunk of a stage needs besides its bytes; written by the producer.
struct __align__(32) ChunkParams {
  float k;          // sigma * softmax scale * log2 e: score / sigma -> log2 units
  float lambda;     // log2 sigma
  float inv_sigma;
  float rope_mul;   // 2^-kRopeShift / sigma
  uint32_t code_mul;  // 2^(e - E), twice in fp16
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit, volatile int* abort,
                                          int* status, int where) {
  const bool ok = mbar_wait(bar, parity, limit, abort, status, where);
  return __all_sync(kAll, ok);
}

// The CTA's segments: the tiles [begin, end) of one sequence after another.
struct Segments {
  const int* prefix;
  int B, t_begin, t_end, s;
  int first, n;  // the current segment's first tile (of all tiles) and number of tiles
  __device__ Segments(const int* prefix_, int B_, int t_begin_, int t_end_, int s_first)
      : prefix(prefix_), B(B_), t_begin(t_begin_), t_end(t_end_), s(s_first - 1), first(0), n(0) {}
  __device__ bool next() {
    for (++s; s < B && prefix[s] < t_end; ++s) {
      first = max(t_begin, prefix[s]);
      n = min(t_end, prefix[s + 1]) - first;
      if (n > 0) return true;
    }
    return false;
  }
};

template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// D[tmem] (+)= A * B with A in tensor or shared memory, without the output lane mask that the
// forms in sm100.cuh pass.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One lane of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

// One step of transposing the 8 x 8 pieces that 8 lanes hold: the pieces whose number has bit S as
// the lane's has not change places with the lane S away.
template <int S>
__device__ __forceinline__ void exchange_rows(float4* v, int lane) {
  const bool upper = (lane & S) != 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j & S) continue;
    float* lo = reinterpret_cast<float*>(&v[j]);
    float* hi = reinterpret_cast<float*>(&v[j | S]);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float got = __shfl_xor_sync(kAll, upper ? lo[x] : hi[x], S);
      if (upper) lo[x] = got; else hi[x] = got;
    }
  }
}

// Four codes (one word) times a power of two -> four fp16, exactly.
template <bool E4M3>
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w, __half2 mul, __half2 bias) {
  __half2 a, b;
  if constexpr (E4M3) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    a = __hmul2(*reinterpret_cast<const __half2*>(&lo), mul);
    b = __hmul2(*reinterpret_cast<const __half2*>(&hi), mul);
  } else {
    // byte v placed as the fp16 1152 + v (see i8x4_to_f16x4); bias = -1152 * mul
    const uint32_t t = w ^ 0x80808080u;
    const uint32_t lo = __byte_perm(t, 0x64646464u, 0x4140);
    const uint32_t hi = __byte_perm(t, 0x64646464u, 0x4342);
    a = __hfma2(*reinterpret_cast<const __half2*>(&lo), mul, bias);
    b = __hfma2(*reinterpret_cast<const __half2*>(&hi), mul, bias);
  }
  return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

template <bool E4M3>
__global__ void __launch_bounds__(BlockCfg::THREADS, 1)
decode_block_kernel(const __grid_constant__ CUtensorMap map_ckv, const __grid_constant__ CUtensorMap map_krope,
                    const DecodeArgs a) {
  using C = BlockCfg;
  constexpr int NT = C::NT, RAW = C::RAW, LAT = C::LAT, CHUNKS = C::CHUNKS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* raws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* lats = raws + RAW * C::RAW_BYTES;
  uint8_t* q_rope = lats + LAT * C::LAT_BYTES;
  uint8_t* misc = q_rope + C::QR_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* qk_done = full + RAW;    // [RAW] the tile's scores are there, its copy has been read
  uint64_t* conv = qk_done + RAW;    // [LAT] the latent (and the copy's rope part) is fp16
  uint64_t* pv_done = conv + LAT;    // [LAT] O has the tile, its latent has been read
  uint64_t* p_ready = pv_done + LAT; // [2] per stream
  uint64_t* q_ready = p_ready + 2;   // the segment's query is in place, the last one's O is read
  uint64_t* ml_bar = q_ready + 1;    // both streams' (M, l) are in shared memory
  uint64_t* drain = ml_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_flag = abort_flag + 1;  // stays 0: exit-path waits ignore the abort flag
  float2* ml = reinterpret_cast<float2*>(misc + C::BAR_BYTES);  // [2 streams][128]
  ChunkParams* params = reinterpret_cast<ChunkParams*>(misc + C::BAR_BYTES + C::ML_BYTES);  // [PAR][CHUNKS]
  int* prefix = reinterpret_cast<int*>(misc + C::BAR_BYTES + C::ML_BYTES + C::PAR_BYTES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int slice = blockIdx.x;  // = branch
  const int G = gridDim.y;
  const int g = blockIdx.y;
  const int B = a.batch;
  const uint64_t limit = a.wait_limit_ns;
  int* status = a.status;

  if (warp == 0) tile_prefix_warp(a.seq_lens, B, NT, prefix);
  if (threadIdx.x == 0) grid_dep_launch();
  if (threadIdx.x == 32) {
    for (int i = 0; i < RAW; ++i) {
      mbar_init(&full[i], 2);  // the copy's bytes, and its chunk parameters
      mbar_init(&qk_done[i], 1);
    }
    for (int i = 0; i < LAT; ++i) {
      mbar_init(&conv[i], C::CONV_WARPS);
      mbar_init(&pv_done[i], 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(&p_ready[b], 4);
    mbar_init(q_ready, 8);
    mbar_init(ml_bar, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::WARP_MMA) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == C::WARP_PRODUCER && lane == 0) {
    tma_prefetch_desc(&map_ckv);
    tma_prefetch_desc(&map_krope);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int T = prefix[B];
  const int t_begin = T > 0 ? group_tile_begin(g, G, T) : 0;
  const int t_end = T > 0 ? group_tile_begin(g + 1, G, T) : 0;
  const int s_first = (t_begin < t_end) ? seq_of_tile(prefix, B, t_begin) : B;

  if (warp >= C::WARP_CONV) {
    regs_dec<C::OTHER_REGS>();
    if (warp == C::WARP_PRODUCER) {
      // ------------------------------------------------------------------ TMA producer
      // Each lane finds the cache row and the scale of one 32-row chunk of a batch of 10
      // tiles, one batch ahead of the tiles lane 0 is issuing.
      constexpr int TPB = 32 / CHUNKS;
      const int ntiles = t_end - t_begin;
      const uint64_t policy = l2_policy_evict_first();
      const int my_tile = lane / CHUNKS, my_chunk = lane % CHUNKS;
      auto chunk_row = [&](int it0) {
        const int t = t_begin + it0 + my_tile;
        if (my_tile >= TPB || t >= t_end) return static_cast<int>(a.cache_rows);
        const int s = seq_of_tile(prefix, B, t);
        return cache_chunk_row(a, s, (t - prefix[s]) * NT + 32 * my_chunk);
      };
      // a chunk past its sequence's end has no scale
      auto chunk_scale = [&](int row) {
        return row < a.cache_rows ? a.ckv_scale[row / a.scale_block * a.scale_stride + slice] : 0.f;
      };
      // The first copies go out before any scale is known, and later rows and scales are looked up
      // half a batch before they are used: no copy waits for a lookup.
      int rows = chunk_row(0), rows_next = chunk_row(TPB);
      float scale = chunk_scale(rows), scale_next = 0.f;
      auto copy = [&](int it, int k) {  // tile it, the batch's k-th
        const int stage = it % RAW;
        int y[CHUNKS];
#pragma unroll
        for (int r = 0; r < CHUNKS; ++r) y[r] = __shfl_sync(kAll, rows, k * CHUNKS + r);
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[stage], C::RAW_BYTES);
          uint8_t* dst = raws + stage * C::RAW_BYTES;
#pragma unroll
          for (int r = 0; r < CHUNKS; ++r) {
            tma_load_2d(dst + r * 4096, &map_ckv, &full[stage], slice * C::W, y[r], policy);
            tma_load_2d(dst + C::BOX_BYTES + r * 4096, &map_krope, &full[stage], 0, y[r], policy);
          }
        }
        __syncwarp();
      };
      const int ahead = min(RAW, ntiles);
      for (int k = 0; k < ahead; ++k) copy(k, k);
      int issued = ahead;
      bool ok = true;
      for (int it0 = 0; ok && it0 < ntiles; it0 += TPB) {
        // this lane's chunk: s = f * 2^e
        const uint32_t bits = __float_as_uint(scale == 0.f ? 0.f : scale);  // -0 is no negative scale
        const int ex = static_cast<int>(bits >> 23) - 127;  // s >= 0
        const bool none = bits < 0x00800000u;                 // zero (or subnormal: taken as zero)
        const bool bad = bits >= 0x7F800000u;                 // Inf, NaN (or negative)
        const int e = none || bad ? -127 : ex;
        const float f = bad ? __uint_as_float(0x7FC00000u) : none ? 1.f : __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
        const int E = min(max(e, kMinExp), kMaxExp);
        const float sigma = f * __uint_as_float(static_cast<uint32_t>(E + 127) << 23);
        ChunkParams cp;
        cp.k = sigma * a.scale_log2;
        cp.lambda = log2f(f) + static_cast<float>(E);
        cp.inv_sigma = 1.f / sigma;
        cp.rope_mul = cp.inv_sigma * (1.f / (1 << kRopeShift));
        const __half m = none || bad ? __float2half_rn(0.f)
                                     : __float2half_rn(__uint_as_float(static_cast<uint32_t>(max(e - E, -30) + 127) << 23));
        const __half2 m2 = __half2half2(m);
        cp.code_mul = *reinterpret_cast<const uint32_t*>(&m2);
        int rows_after = static_cast<int>(a.cache_rows);
        for (int k = 0; k < TPB && it0 + k < ntiles; ++k) {
          const int it = it0 + k;
          if (it >= ahead) {
            if (it >= RAW && !warp_wait(&qk_done[it % RAW], ((it / RAW) + 1) & 1, limit, abort_flag, status, 1)) {
              ok = false;
              break;
            }
            copy(it, k);
            issued = it + 1;
          }
          // the arrive releases the parameters to the waits on full
          if (my_tile == k) params[it % C::PAR * CHUNKS + my_chunk] = cp;
          warp_arrive(&full[it % RAW]);
          if (k == TPB / 2) {
            scale_next = chunk_scale(rows_next);
            rows_after = chunk_row(it0 + 2 * TPB);
          }
        }
        rows = rows_next;
        scale = scale_next;
        rows_next = rows_after;
      }
      for (int k = max(0, issued - RAW); k < issued; ++k) {  // every stage must come back
        if (ok && !warp_wait(&qk_done[k % RAW], (k / RAW) & 1, limit, abort_flag, status, 2)) ok = false;
        if (!ok) {  // aborted: wait (bounded, ignoring the abort flag) for the copy itself
          warp_wait(&full[k % RAW], (k / RAW) & 1, kDrainNs, never_flag, status, 3);
        }
      }
    } else if (warp == C::WARP_MMA) {
      // ------------------------------------------------------------------ MMA issuer
      // The whole warp walks the tiles, so that what an MMA needs is uniform; one lane issues.
      constexpr uint32_t idesc_qk = idesc_f16_f32(128, NT, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, 128, true);
      const uint32_t t0 = __shfl_sync(kAll, tmem, 0);
      const uint64_t k_desc0 = smem_desc_sw128(smem_u32(lats), 16, 1024);
      const uint64_t v_desc0 = smem_desc_sw128(smem_u32(lats), C::BOX_BYTES, 1024);
      const uint64_t kr_desc0 = smem_desc_sw128(smem_u32(raws) + C::BOX_BYTES, 16, 1024);
      const uint64_t qr_desc = smem_desc_sw128(smem_u32(q_rope), 16, 1024);
      // descriptors count 16 bytes
      constexpr uint32_t LAT_STEP = C::LAT_BYTES >> 4, RAW_STEP = C::RAW_BYTES >> 4, BOX_STEP = C::BOX_BYTES >> 4;
      Segments seg(prefix, B, t_begin, t_end, s_first);
      int i = 0, n_seg = 0;  // i: the segment's first tile
      bool ok = true;
      while (ok && seg.next()) {
        if (!warp_wait(q_ready, n_seg & 1, limit, abort_flag, status, 10)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int n = __shfl_sync(kAll, seg.n, 0);
        // P.V of a tile and QK of the one two on (the same buffer) are issued together, and their
        // commits after both: nothing stands between P and the stream's next scores.
        for (int k = 0; k < n + 2; ++k) {
          const int j = i + k, v = j - 2;
          const bool qk = k < n, pv = k >= 2 && k - 2 < n;
          if ((qk && !warp_wait(&conv[j % LAT], (j / LAT) & 1, limit, abort_flag, status, 11)) ||
              (pv && !warp_wait(&p_ready[v & 1], (v >> 1) & 1, limit, abort_flag, status, 13))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t s_tmem = t0 + C::TMEM_S + NT * (j & 1);
            if (pv) {  // O of the stream (+)= P . latent
              const uint64_t v_desc = v_desc0 + v % LAT * LAT_STEP;
              const uint32_t o = t0 + C::TMEM_O + 128 * (j & 1);
#pragma unroll
              for (int x = 0; x < NT / 16; ++x)  // 16 rows of 128 bytes on
                mma_ts(o, s_tmem + 8 * x, v_desc + x * (16 * 128 >> 4), idesc_pv, (k < 4 && x == 0) ? 0u : 1u);
            }
            if (qk) {
              const uint64_t k_desc = k_desc0 + j % LAT * LAT_STEP, kr_desc = kr_desc0 + j % RAW * RAW_STEP;
#pragma unroll
              for (int x = 0; x < C::W / 16; ++x)
                mma_ts(s_tmem, t0 + C::TMEM_Q + x * 8, k_desc + (x >> 2) * BOX_STEP + (x & 3) * 2, idesc_qk, x > 0 ? 1u : 0u);
#pragma unroll
              for (int x = 0; x < 4; ++x) mma_ss(s_tmem, qr_desc + x * 2, kr_desc + x * 2, idesc_qk, 1u);
              umma_commit(&qk_done[j % RAW]);
            }
            if (pv) umma_commit(&pv_done[v % LAT]);
          }
          __syncwarp();
        }
        i += n;
        ++n_seg;
      }
      if (elect_one()) {
        umma_commit(drain);
        mbar_wait(drain, 0, kDrainNs, never_flag, status, 14);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ converters
      // Thread r of a team converts row r of the team's tiles: 128 codes to fp16, 64 bf16 rope
      // values to fp16 in place.  Latents of rows at or past the sequence end become
      // zero, so that 0 * NaN cannot reach O; their scores are masked by the softmax.
      const int team = warp >= C::WARP_CONV + C::CONV_WARPS ? 1 : 0;
      const int r = threadIdx.x - 32 * (C::WARP_CONV + team * C::CONV_WARPS);
      const int sw = r & 7;
      Segments seg(prefix, B, t_begin, t_end, s_first);
      int i = 0;
      bool ok = true;
      while (ok && seg.next()) {
        const int L = a.seq_lens[seg.s];
        for (int k = 0; k < seg.n; ++k, ++i) {
          if ((i & 1) != team) continue;
          const int stage = i % LAT;
          uint8_t* row = raws + i % RAW * C::RAW_BYTES + r * 128;
          uint8_t* lat = lats + stage * C::LAT_BYTES + r * 128;
          const bool valid = r < L - (seg.first + k - prefix[seg.s]) * NT;
          if ((i >= LAT && !warp_wait(&pv_done[stage], ((i / LAT) + 1) & 1, limit, abort_flag, status, 21)) ||
              !warp_wait(&full[i % RAW], (i / RAW) & 1, limit, abort_flag, status, 20)) {
            ok = false;
            break;
          }
          const ChunkParams& cp = params[i % C::PAR * CHUNKS + (r >> 5)];
          const uint32_t mul_bits = cp.code_mul;
          const __half2 mul = *reinterpret_cast<const __half2*>(&mul_bits);
          const __half2 bias = __hmul2(mul, __float2half2_rn(-1152.f));
          const float rope_mul = cp.rope_mul;
          uint4 raw[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) raw[c] = *reinterpret_cast<const uint4*>(row + ((c ^ sw) << 4));
#pragma unroll
          for (int c = 0; c < 8; ++c) {  // codes [16 c, 16 c + 16) -> fp16 chunks 2 c, 2 c + 1 of 16
            uint2 h0 = codes_to_f16<E4M3>(raw[c].x, mul, bias), h1 = codes_to_f16<E4M3>(raw[c].y, mul, bias);
            uint2 h2 = codes_to_f16<E4M3>(raw[c].z, mul, bias), h3 = codes_to_f16<E4M3>(raw[c].w, mul, bias);
            if (!valid) h0 = h1 = h2 = h3 = make_uint2(0u, 0u);
            uint8_t* box = lat + (c >> 2) * C::BOX_BYTES;
            *reinterpret_cast<uint4*>(box + ((((2 * c) & 7) ^ sw) << 4)) = make_uint4(h0.x, h0.y, h1.x, h1.y);
            *reinterpret_cast<uint4*>(box + ((((2 * c + 1) & 7) ^ sw) << 4)) = make_uint4(h2.x, h2.y, h3.x, h3.y);
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) raw[c] = *reinterpret_cast<const uint4*>(row + C::BOX_BYTES + ((c ^ sw) << 4));
          const float2 rm = make_float2(rope_mul, rope_mul);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float2 x = mul2(make_float2(__uint_as_float(w[u] << 16), __uint_as_float(w[u] & 0xFFFF0000u)), rm);
              w[u] = pack_f16x2(x.x, x.y);
            }
            *reinterpret_cast<uint4*>(row + C::BOX_BYTES + ((c ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          warp_arrive(&conv[stage]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    regs_inc<C::SOFTMAX_REGS>();
    // The query comes from the previous kernel: wait for it.  The other roles touch no memory that
    // another kernel of the call writes.
    grid_dep_wait();
    const int b = warp >> 2;          // stream
    const int row = threadIdx.x & 127;  // head row == TMEM lane
    const bool live_warp = 32 * (warp & 3) < a.heads;  // some row of the warp is a head
    const bool live = row < a.heads;
    const uint32_t t_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_cols = t_row + C::TMEM_S + NT * b, o_cols = t_row + C::TMEM_O + 128 * b;
    const int q_stride = a.d_c + 64;
    Segments seg(prefix, B, t_begin, t_end, s_first);
    int it = 0, n_seg = 0;
    bool ok = true;
    while (ok && seg.next()) {
      const int s = seg.s;
      const int L = a.seq_lens[s];
      {  // this row's query: stream 0 stores the latent part, stream 1 the rope part
        const __half* q = a.q_tilde + (static_cast<long long>(s) * a.heads + min(row, a.heads - 1)) * q_stride;
        if (b == 0) {
          const uint4* src = reinterpret_cast<const uint4*>(q + slice * C::W);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const uint4 v = live ? __ldg(src + 8 * c + u) : make_uint4(0u, 0u, 0u, 0u);
              w[4 * u + 0] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
            }
            tmem_st32(t_row + C::TMEM_Q + 32 * c, w);
          }
          tmem_st_wait();
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(q + a.d_c);
          const __half2 up = __float2half2_rn(static_cast<float>(1 << kRopeShift));
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
            for (int u = 0; u < 4; ++u) h[u] = __hmul2(h[u], up);
            *reinterpret_cast<uint4*>(q_rope + row * 128 + ((c ^ (row & 7)) << 4)) = v;
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        warp_arrive(q_ready);
      }
      float M = -INFINITY, l = 0.f;
      bool first = true;
      for (int k = 0; k < seg.n; ++k) {
        const int i = it + k;
        if ((i & 1) != b) continue;
        // The chunk parameters, while the scores are on their way: the converters have seen them when
        // the tile is converted.  The place of tile i + PAR is written after QK(i + RAW), which
        // comes after this stream's softmax of tile i + 2.
        if (!warp_wait(&conv[i % LAT], (i / LAT) & 1, limit, abort_flag, status, 35)) { ok = false; break; }
        float kc[CHUNKS], lam[CHUNKS], inv[CHUNKS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          const float4 p = *reinterpret_cast<const float4*>(&params[i % C::PAR * CHUNKS + c]);
          kc[c] = p.x;
          lam[c] = p.y;
          inv[c] = p.z;
        }
        if (!warp_wait(&qk_done[i % RAW], (i / RAW) & 1, limit, abort_flag, status, 30)) { ok = false; break; }
        tc_fence_after();
        if (!live_warp) {  // rows that are no head: their P and O are never read
          warp_arrive(&p_ready[b]);
          continue;
        }
        uint32_t sr[NT];
        tmem_load<NT>(s_cols, sr);
        tmem_ld_wait();
        const int n_valid = L - (seg.first + k - prefix[s]) * NT;
        if (n_valid < NT) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
            if (u >= n_valid) sr[u] = __float_as_uint(-INFINITY);
        }
        float mt = -INFINITY;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          float m0 = __uint_as_float(sr[32 * c]), m1 = __uint_as_float(sr[32 * c + 1]);
#pragma unroll
          for (int u = 2; u + 4 <= 32; u += 4) {
            m0 = fmax3(m0, __uint_as_float(sr[32 * c + u]), __uint_as_float(sr[32 * c + u + 1]));
            m1 = fmax3(m1, __uint_as_float(sr[32 * c + u + 2]), __uint_as_float(sr[32 * c + u + 3]));
          }
          m0 = fmax3(m0, __uint_as_float(sr[32 * c + 30]), __uint_as_float(sr[32 * c + 31]));
          mt = fmaxf(mt, fmaf(fmaxf(m0, m1), kc[c], lam[c]));
        }
        float factor = 1.f;
        bool rescale = false;
        if (first) {
          M = mt;
        } else if (mt > M + 8.f) {  // lazy rescale: keep the reference unless it grew by 2^8
          factor = ex2_approx(M - mt);
          M = mt;
          rescale = true;
        }
        l *= factor;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          const float2 kv = make_float2(kc[c], kc[c]);
          const float2 off = make_float2(lam[c] - M, lam[c] - M);
          float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const float2 x = fma2(make_float2(__uint_as_float(sr[32 * c + 2 * u]), __uint_as_float(sr[32 * c + 2 * u + 1])), kv, off);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            if (u & 1) s1 = add2(s1, p); else s0 = add2(s0, p);
            sr[16 * c + u] = pack_f16x2(p.x, p.y);
          }
          const float2 st = add2(s0, s1);
          l = fmaf(inv[c], st.x + st.y, l);
        }
        if (__any_sync(kAll, rescale)) {
          // the stream's earlier P.V must have completed before O is rescaled
          if (!warp_wait(&pv_done[(i - 2) % LAT], ((i - 2) / LAT) & 1, limit, abort_flag, status, 31)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(o_cols + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * factor);
            tmem_st16(o_cols + 16 * c, o);
          }
        }
        tmem_store<NT / 2>(s_cols, sr);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&p_ready[b]);
        first = false;
      }
      if (!ok) break;
      it += seg.n;
      // segment end: the streams' states are added; stream b writes O columns [64 b, 64 b + 64).
      // A stream without a tile here may come early: the other one has read the last segment's
      // states once the query of this one is in place.
      if (!warp_wait(q_ready, n_seg & 1, limit, abort_flag, status, 36)) { ok = false; break; }
      ml[b * 128 + row] = make_float2(M, l);
      warp_arrive(ml_bar);
      if (!warp_wait(ml_bar, n_seg & 1, limit, abort_flag, status, 34)) { ok = false; break; }
      // Each stream's last P.V (a stream without a tile in the segment has M = -inf).
      const int last = it - 1;
      for (int c = 0; c < 2 && ok; ++c) {
        const int i = last - c;
        if (c < seg.n) ok = warp_wait(&pv_done[i % LAT], (i / LAT) & 1, limit, abort_flag, status, 32);
      }
      if (!ok) break;
      tc_fence_after();
      if (live_warp) {
        const float2 ml0 = ml[row], ml1 = ml[128 + row];
        const int b0 = last & 1;                         // a stream that had a tile
        const bool both = seg.n > 1;
        const float M_all = both ? fmaxf(ml0.x, ml1.x) : (b0 ? ml1.x : ml0.x);
        const bool use0 = both || b0 == 0, use1 = both || b0 == 1;
        const float w0 = use0 ? ex2_approx(ml0.x - M_all) : 0.f, w1 = use1 ? ex2_approx(ml1.x - M_all) : 0.f;
        const long long slot = static_cast<long long>(g) + s;
        const long long at = (slot * gridDim.x + slice) * 128 + row;
        // Eight lanes exchange their rows' 16-byte pieces, so that a store covers whole 128-byte lines: with
        // a lane for a row, 32 lines to an instruction, a segment's end took 2500 cycles more (now 3600 to
        // 6400 with the waits for the last P.V).
        const int group_row = row - (lane & 7);
        float4* dst = reinterpret_cast<float4*>(a.o_part + (at - (lane & 7)) * 128 + 64 * b) + (lane & 7);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t o0[32], o1[32];
          tmem_ld32(t_row + C::TMEM_O + 64 * b + 32 * c, o0);
          tmem_ld32(t_row + C::TMEM_O + 128 + 64 * b + 32 * c, o1);
          tmem_ld_wait();
          float4 v[8];
#pragma unroll
          for (int u = 0; u < 32; ++u)
            reinterpret_cast<float*>(v)[u] = (use0 ? w0 * __uint_as_float(o0[u]) : 0.f) + (use1 ? w1 * __uint_as_float(o1[u]) : 0.f);
          exchange_rows<1>(v, lane);
          exchange_rows<2>(v, lane);
          exchange_rows<4>(v, lane);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (group_row + u < a.heads) dst[32 * u + 8 * c] = v[u];
        }
        if (b == 0 && live)
          a.ml_part[at] = make_float2(M_all, (use0 ? w0 * ml0.y : 0.f) + (use1 ? w1 * ml1.y : 0.f));
      }
      tc_fence_before();
      ++n_seg;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace

int decode_block_tile_tokens() { return BlockCfg::NT; }

// The softmax warps' setmaxnreg waits for registers that a launch with fewer would not have.  128 is
// the most that 512 threads can have and what the compiler takes; a build with another number is
// refused, not tried.
cudaError_t decode_block_registers(int* have, int* need) {
  *have = 0;
  *need = BlockCfg::LAUNCH_REGS;
  cudaFuncAttributes i8{}, f8{};
  cudaError_t e = cudaFuncGetAttributes(&i8, decode_block_kernel<false>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&f8, decode_block_kernel<true>);
  if (e == cudaSuccess) *have = i8.numRegs < f8.numRegs ? i8.numRegs : f8.numRegs;
  return e;
}

cudaError_t launch_decode_block_kernel(const CUtensorMap& map_ckv, const CUtensorMap& map_krope, const DecodeArgs& a,
                                       int groups, cudaStream_t stream, bool pdl) {
  using C = BlockCfg;
  auto kern = a.cache_int8 == 2 ? decode_block_kernel<true> : decode_block_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(a.d_c / 128, groups), dim3(C::THREADS), C::SMEM_BYTES, stream, pdl, map_ckv,
                       map_krope, a);
}

}  // namespace hra
