// Window attention over the 8-bit cache on the tensor cores, head_dim 128.
//
//   k_window_tc    one persistent CTA an SM: the cached tokens, and the window's own
//   k_join         joins the pieces of units that more than one CTA worked on
//
// The cache is read once and its bytes go to the tensor cores as they are: TMA brings pages
// into shared memory and tcgen05.mma (kind f8f6f4) takes the e4m3 codes, so no thread touches K
// or V. What the products need in more than four significant bits is split into e4m3 parts.
// Both products are turned round, so that the long side of the tile, 128 tokens or 128 dims,
// is the M = 128 of the instruction and the window's rows, few as they are, its N:
//
//   S^T [128 tokens x ROWS] = K [128 x D] (Q_hi + Q_lo (+ Q_lo2))^T      one accumulator
//   O^T [D x 2 or 3 ROWS]   += V^T [D x 128 tokens] P^T, P in three parts, accumulators as below
//
// P = 2^(x - m) with a reference m a row (x in log2 units, V's scale in the exponent as in
// ts_window.cu); a reference follows only when a score exceeds it by 2^8 (one vote a tile), and
// then O is scaled in TMEM. Parts of P: the fp16 rounding of p in three codes, the row's largest p
// between 2^4 and 2^8.
//
//   32 rows  e4m3, each rest scaled by 2^5: an accumulator a part, one instruction (222 clocks a
//            tile against 384 for two types). All 11 bits of p down to 2^-9, values down to 2^-20.
//   64 rows  e4m3; its rest in e5m2 as it is, so that both share an accumulator; and what is left times
//            2^9 in e4m3. All 11 bits down to 2^-8, values down to 2^-19. The columns of TMEM that
//            this saves are second buffers of S, so that the first products run a whole round
//            of turns ahead (with the parts of 32 rows: 390 us for 16 trees of 32 nodes
//            over 8191 tokens, 351 with these).
//
// What the smallest lose, 2^-19 each at most, comes to 2^-7 in the kLook tiles of a turn; after as many
// a row whose largest p is below 2^4 has its reference lowered. So the loss stays below 2^-11 of the
// row's sum however many small ones follow a large one. A reference is set so that the largest p is 2^4
// exactly: where it outweighs the rest, its rounding would not cancel in the quotient (the sums take p
// unrounded: V's scale is in it, and a token whose scale is small may weigh much where its p is lost to
// fp16). With whole numbers as references ragged fp16 chains erred by 2.9e-4 (rms, relative), with these by 2.2e-4.
//
// (Two parts, e4m3 and 2^12 times the rest in e5m2, were faster by a little. Below 2^-10 the second
// alone holds p then, in three bits: behind a large probability many small ones, all alike, err by
// up to 12 % to the same side.)
//
// A softmax thread is a token: it reads its row of S^T from TMEM, the scales of its block and
// its validity are its own, and it writes its row of P. Its work on a tile is a chain of waits
// and short bursts, so four groups of four warps work on different parts of the line: with
// blocks of 32 rows each group takes every fourth tile, with blocks of 64 two groups share a
// tile (32 rows each) and two pairs take turns. Tiles of one turn have their own S, P and O; the
// turns meet at the end of a unit and the result is written. The window's own tokens
// (ts_window_own.cuh) are worked on at a unit's beginning, while Q is split. One warp each loads K (with the blocks' scales) and V, rings of four
// tiles or 64 KB; a lane each of two warps issues the first and the second products. The first
// of them also splits Q, the second looks up what the rows of a tree see.
//
// Every wait on a barrier is bounded; after one ran out no wait waits and nothing more is
// issued, so that the CTA runs to its end (results unspecified, reported by ts_device_error).
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "ts_window.cuh"
#include "ts_window_own.cuh"

namespace tsv {

namespace {

constexpr int kTile = 128;
constexpr int kD = 128;
constexpr int kStages = 4;         // tiles of K, and as many of V, in shared memory
constexpr int kStageBytes = kTile * kD;
constexpr int kMeta = 16;          // tiles whose scales are in shared memory
constexpr int kGroups = 4;         // of softmax threads
constexpr int kGroupThreads = 128;
constexpr int kSoftmaxThreads = kGroups * kGroupThreads;
constexpr int kThreads = kSoftmaxThreads + 128;
constexpr int kCols = 32;          // rows of a block that a softmax thread has scores of
constexpr int kMinTiles = 2;       // least tiles a CTA takes: pieces of 256 tokens or more
constexpr int kParts = 3;          // of a probability
constexpr float kSlack = 8.f;      // how far, in log2, a score may exceed its row's reference
constexpr float kHead = 4.f;       // a reference is set this far below the largest score
constexpr int kLook = 32;          // tiles of a turn after which references may be lowered
constexpr float kDeep = 12.f;      // the most that a reference lies below an earlier one of its row (sums must not overflow)
constexpr int kBarAll = kGroups + 1;  // named barrier of all softmax threads; 1 .. kGroups: a group's

__device__ uint32_t g_window_error;

template <int ROWS, int QP>
struct Layout {
  static constexpr int q_bytes = QP * ROWS * kD;
  static constexpr int p_part = ROWS * kTile;
  static constexpr bool split = ROWS == 2 * kCols;        // two groups share a tile's rows
  static constexpr int turns = split ? kGroups / 2 : kGroups;  // tiles in work at a time
  static constexpr int off_v = kStages * kStageBytes;
  static constexpr int off_q = 2 * kStages * kStageBytes;
  static constexpr int off_p = off_q + q_bytes;
  static constexpr int off_x = off_p + turns * kParts * p_part;
  // TMEM columns: the buffers of S, then the turns' O, a part after the other
  static constexpr int s_bufs = split ? 2 * turns : turns;
  static constexpr int accs = split ? 2 : 3;  // accumulators
  static constexpr int col_o = s_bufs * ROWS, o_cols = accs * ROWS;
  static constexpr int tmem_cols = 512;
  // a tile's scales are overwritten kMeta tiles later, when the first product of the tile kStages
  // before that one is done, and with it the groups' reading of the scores s_bufs before that
  static_assert(kMeta >= s_bufs + kStages, "scales");
  static_assert(col_o + turns * o_cols <= tmem_cols, "TMEM");
};

template <int ROWS>
struct Shared {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], meta_full[kMeta];
  uint64_t s_full[2 * kGroups], s_free[2 * kGroups];  // a buffer's
  uint64_t p_full[kGroups], o_done[kGroups];          // a turn's
  uint64_t q_full, q_empty, o_free, trees_full;
  float q_fac[ROWS];                        // the factors of a unit's rows (split_q)
  float ks[kMeta][8], vs[kMeta][8];         // scales of a tile's pages (vs 0: no such page)
  alignas(16) float neg_m[kGroups][kCols];  // a group's references, negated; read as vectors
  alignas(16) float fac[kGroups][kCols];    // a group's rows' factors
  alignas(16) float delta[kGroups][kCols];  // factors of outputs and sums whose references move
  float peak[kGroups][kCols];               // the rows' largest references so far
  float red[kGroups][4][kCols];
  float w[kGroups + 1][ROWS];  // a row's factors: the turns', and the window's own part
  float2 own[ROWS];            // the own part's references and sums
  int32_t at[ROWS];            // a row's index in [total_rows][heads_q]
  int32_t parents[TS_MAX_WINDOW];
  Sees trees[TS_MAX_WINDOW];
  int32_t live[kGroups];
  uint32_t tmem;
  alignas(16) int32_t stop;
  uint64_t wait_cycles;  // 8 bytes behind stop: wait reads it
};
static_assert(offsetof(Shared<32>, wait_cycles) == offsetof(Shared<32>, stop) + 8 &&
                  offsetof(Shared<64>, wait_cycles) == offsetof(Shared<64>, stop) + 8,
              "wait");

static_assert(offsetof(Shared<32>, neg_m) % 16 == 0 && offsetof(Shared<64>, neg_m) % 16 == 0 &&
                  offsetof(Shared<32>, fac) % 16 == 0 && offsetof(Shared<64>, fac) % 16 == 0 &&
                  offsetof(Shared<32>, delta) % 16 == 0 && offsetof(Shared<64>, delta) % 16 == 0 &&
                  Layout<32, 2>::off_x % 16 == 0 && Layout<64, 3>::off_x % 16 == 0,
              "vector loads");

template <int ROWS, int QP>
constexpr int smem_bytes() { return Layout<ROWS, QP>::off_x + (int)sizeof(Shared<ROWS>) + 1024; }
static_assert(smem_bytes<64, 3>() <= 227 * 1024, "shared memory");

__device__ __forceinline__ bool stopped(const int32_t* stop) { return *reinterpret_cast<const volatile int32_t*>(stop) != 0; }

// Waits for a phase; gives up after the call's budget of SM clock cycles (8 bytes behind stop) and
// sets *stop, or when that is set. Written out for size: it stands in every loop, and the loops
// of the six roles have to stay in the instruction caches. The lanes of a warp need not see the phase at
// the same try: they part here, and callers bring them together (__syncwarp) before anything that takes a
// whole warp.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int32_t* stop) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .u32 f;\n .reg .u64 t0, t1, b;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n"
      " @p bra DONE_%=;\n"
      " mov.u64 t0, %%clock64;\n"
      "AGAIN_%=:\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n"
      " @p bra DONE_%=;\n"
      " ld.volatile.shared.u32 f, [%2];\n"
      " setp.ne.u32 p, f, 0;\n"
      " @p bra DONE_%=;\n"
      " mov.u64 t1, %%clock64;\n"
      " sub.u64 t1, t1, t0;\n"
      " ld.shared.u64 b, [%2 + 8];\n"
      " setp.le.u64 p, t1, b;\n"
      " @p bra AGAIN_%=;\n"
      " st.volatile.shared.u32 [%2], 1;\n"
      "DONE_%=:\n}\n" ::"r"(smem_u32(bar)),
      "r"(parity), "r"(smem_u32(stop))
      : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool bar_or(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred.aligned q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Of the lanes' 16 columns x: lane l gets the reduction of column l % 16 over the lanes. 16 shuffles.
template <int O, typename F>
__device__ __forceinline__ void halve(float* y, int lane, F f) {
  const bool up = lane & O;
#pragma unroll
  for (int i = 0; i < O; ++i) {
    const float keep = up ? y[i + O] : y[i], give = up ? y[i] : y[i + O];
    y[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, O));
  }
  if constexpr (O > 1) halve<O / 2>(y, lane, f);
}
template <typename F>
__device__ __forceinline__ float reduce_columns(float* x, int lane, F f) {
  halve<8>(x, lane, f);
  return f(x[0], __shfl_xor_sync(0xffffffffu, x[0], 16));
}

// Four probabilities (two fp16 pairs) in parts, for three accumulators; or for two: then codes[1] is
// the third part, so that the two of e4m3 lie side by side, and codes[2] the second.
template <int ACCS>
__device__ __forceinline__ void split_p(__half2 a, __half2 b, uint32_t* codes) {
#pragma unroll
  for (int part = 0; part < ACCS; ++part) {
    uint32_t back_a, back_b;
    asm("{\n .reg .b16 u, v;\n cvt.rn.satfinite.e4m3x2.f16x2 u, %3;\n cvt.rn.satfinite.e4m3x2.f16x2 v, %4;\n"
        " mov.b32 %0, {u, v};\n cvt.rn.f16x2.e4m3x2 %1, u;\n cvt.rn.f16x2.e4m3x2 %2, v;\n}\n"
        : "=r"(codes[part]), "=r"(back_a), "=r"(back_b)
        : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
    a = __hsub2(a, *reinterpret_cast<const __half2*>(&back_a));
    b = __hsub2(b, *reinterpret_cast<const __half2*>(&back_b));
    if (ACCS == 2 && part == 0) {  // e5m2: the upper byte of an fp16
      asm("{\n .reg .b16 u, v;\n cvt.rn.satfinite.e5m2x2.f16x2 u, %1;\n cvt.rn.satfinite.e5m2x2.f16x2 v, %2;\n mov.b32 %0, {u, v};\n}\n"
          : "=r"(codes[2])
          : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
      back_a = __byte_perm(codes[2], 0, 0x1404);
      back_b = __byte_perm(codes[2], 0, 0x3424);
      a = __hsub2(a, *reinterpret_cast<const __half2*>(&back_a));
      b = __hsub2(b, *reinterpret_cast<const __half2*>(&back_b));
    }
    const __half2 by = __float2half2_rn(ACCS == 2 ? 512.f : 32.f);
    a = __hmul2(a, by);
    b = __hmul2(b, by);
  }
}

// A value that the compiler knows nothing about: branches on it are not merged into copies of
// the code between them (the loops have to stay in the instruction caches).
__device__ __forceinline__ int apart(int v) {
  asm volatile("" : "+r"(v));
  return v;
}

template <int ROWS, int QP, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_tc(const __grid_constant__ WindowParams p, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<ROWS, QP>;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char* s_q = sm + L::off_q;
  unsigned char* s_p = sm + L::off_p;
  Shared<ROWS>& x = *reinterpret_cast<Shared<ROWS>*>(sm + L::off_x);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kFirst = kSoftmaxThreads / 32;  // the warps behind the softmax groups
  int4 desc = make_int4(-1, 0, 0, 0);
  grid_launch();
  Line<ROWS, kTile> line;
  if (!line_begin<ROWS, kTile, kThreads>(p, kMinTiles, line)) {
    if (tid == 0) p.desc[blockIdx.x] = desc;
    return;
  }
  if (warp == kFirst) tmem_alloc(&x.tmem, L::tmem_cols);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&x.k_full[i], 1);
      mbar_init(&x.k_empty[i], 1);
      mbar_init(&x.v_full[i], 1);
      mbar_init(&x.v_empty[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&x.meta_full[i], 1);
    for (int i = 0; i < L::s_bufs; ++i) {
      mbar_init(&x.s_full[i], 1);
      mbar_init(&x.s_free[i], L::split ? 8 : 4);
    }
    for (int i = 0; i < L::turns; ++i) {
      mbar_init(&x.p_full[i], L::split ? 8 : 4);
      mbar_init(&x.o_done[i], 1);
    }
    mbar_init(&x.q_full, 1);
    mbar_init(&x.q_empty, 1 + kGroups);  // the products, and the groups have read the factors
    mbar_init(&x.o_free, kSoftmaxThreads / 32);
    mbar_init(&x.trees_full, 1);
    x.stop = 0;
    x.wait_cycles = p.wait_cycles;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = x.tmem;
  Segment s{};

  if (warp >= kFirst) {
    if (warp < kFirst + 2) {
      // ---- loads: one warp K and the scales, one V. Page numbers come 32 a round, one a lane,
      // two rounds ahead, and the scales one round ahead (they are scattered reads of DRAM, two
      // of them in a row before a tile's scores can be formed; the same goes for the unit
      // ahead). The lanes that hold a tile's pages bring them.
      const bool is_k = warp == kFirst;
      const CUtensorMap* map = is_k ? &k_map : &v_map;
      unsigned char* ring = sm + (is_k ? 0 : L::off_v);
      uint64_t *full = is_k ? x.k_full : x.v_full, *empty = is_k ? x.k_empty : x.v_empty;
      const int per_tile = kTile >> p.page_shift, per_round = 32 / per_tile;  // pages, tiles
      const int page_bytes = p.c.page_size * kD;
      const int32_t outside = (int32_t)max(p.c.num_pages, (int64_t)1);  // reads as zeros
      // the lane's page of round r of a segment, or -1
      auto page_of = [&](const Segment& g, int r) -> int32_t {
        const int i = g.t0 * per_tile + r * 32 + lane;
        if (i >= g.t1 * per_tile || (int64_t)i << p.page_shift >= g.r.len) return -1;
        const int32_t id = p.c.page_table[g.b * p.c.ld_table + i];
        return id >= 0 && id < p.c.num_pages ? id : -1;
      };
      auto scales_of = [&](const Segment& g, int32_t page, float& ks, float& vs) {
        ks = vs = 0.f;
        if (page < 0 || !is_k) return;
        const int64_t at = (int64_t)page * p.c.heads + g.kvh;
        ks = __ldg(p.c.k_scale + at);
        vs = scale_of_v(__ldg(p.c.v_scale + at), ks);
      };
      Segment ahead;
      bool more = line.next(p, s);
      int32_t page = page_of(s, 0), page1 = page_of(s, 1);
      float ks, vs, next_ks, next_vs;
      scales_of(s, page, ks, vs);
      uint32_t i = 0;
#pragma unroll 1
      while (more) {
        const bool next = line.next(p, ahead);
        const int32_t next0 = next ? page_of(ahead, 0) : -1, next1 = next ? page_of(ahead, 1) : -1;
        const int n = s.t1 - s.t0;
#pragma unroll 1
        for (int r = 0; r * per_round < n; ++r) {
          const int32_t page2 = page_of(s, r + 2);
          float ks1, vs1;
          scales_of(s, page1, ks1, vs1);
          const int end = min(n - r * per_round, per_round);
#pragma unroll 1
          for (int j = 0; j < end; ++j, ++i) {
            const int at = lane - j * per_tile, st = i % kStages;
            wait(&empty[st], (i / kStages & 1) ^ 1, &x.stop);
            if (!__any_sync(0xffffffffu, stopped(&x.stop))) {  // one answer a warp: its lanes meet inside
              if (lane == 0) mbar_arrive_expect_tx(&full[st], kStageBytes);
              __syncwarp();
              if (at >= 0 && at < per_tile)
                tma_load_4d(ring + st * kStageBytes + at * page_bytes, map, 0, 0, s.kvh, page >= 0 ? page : outside, &full[st]);
            }
            if (is_k) {
              if (at >= 0 && at < per_tile) {
                x.ks[i % kMeta][at] = ks;
                x.vs[i % kMeta][at] = vs;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&x.meta_full[i % kMeta]);
            }
          }
          if (r == 0) scales_of(ahead, next0, next_ks, next_vs);
          page = page1;
          page1 = page2;
          ks = ks1;
          vs = vs1;
        }
        s = ahead;
        more = next;
        page = next0;
        page1 = next1;
        ks = next_ks;
        vs = next_vs;
      }
    } else if (warp == kFirst + 2) {
      // ---- Q of a unit, by the warp, and the first products, by a lane. Tiles are counted
      // through the CTA's units; tile i has turn i % turns and buffer i % s_bufs.
      const uint32_t k_lo = desc_lo(smem_u32(sm), 16), q_lo = desc_lo(smem_u32(s_q), 16), hi = desc_hi(8 * kD, kSwizzle128);
      uint32_t i = 0, u = 0;
#pragma unroll 1
      while (line.next(p, s)) {
#pragma unroll 1
        for (int r = lane >> 1; r < s.rows; r += 16)  // on its way while the unit before is worked on
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q_row(p, s, ROWS, r) + (lane & 1) * 128));
        wait(&x.q_empty, (u & 1) ^ 1, &x.stop);
        __syncwarp();
        split_q<ROWS, QP, T>(p, s, p.scale_log2, s_q, x.q_fac);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.q_full);
        const int n = s.t1 - s.t0;
        if (lane == 0) {
#pragma unroll 1
          for (int j = 0; j < n; ++j, ++i) {
            const int w = i % L::s_bufs, st = i % kStages;
            wait(&x.k_full[st], i / kStages & 1, &x.stop);
            if (i >= L::s_bufs) wait(&x.s_free[w], (i / L::s_bufs - 1) & 1, &x.stop);
            if (stopped(&x.stop)) continue;
            tc_fence_after();
            const uint32_t d = tmem + w * ROWS, a = k_lo + st * (kStageBytes / 16);
#pragma unroll
            for (int part = 0; part < QP; ++part)
#pragma unroll
              for (int k = 0; k < kD / 32; ++k)
                mma_f8(d, a + k * 2, hi, q_lo + part * (ROWS * kD / 16) + k * 2, hi, f8_idesc(kTile, ROWS, false, false), part > 0 || k > 0);
            mma_commit(&x.s_full[w]);
            mma_commit(&x.k_empty[st]);
          }
          mma_commit(&x.q_empty);
        }
        __syncwarp();
        ++u;
      }
    } else {
      // ---- what the rows of a tree see, by the warp, and the second products, by a lane
      const uint32_t v_lo = desc_lo(smem_u32(sm) + L::off_v, 16), v_hi = desc_hi(8 * kD, kSwizzle128);
      const uint32_t p_lo = desc_lo(smem_u32(s_p), L::p_part), p_hi = desc_hi(8 * ROWS, ROWS == 64 ? kSwizzle64 : kSwizzle32);
      uint32_t i = 0, u = 0;
#pragma unroll 1
      while (line.next(p, s)) {
        const int n = s.t1 - s.t0;
        if (u > 0) wait(&x.o_free, (u - 1) & 1, &x.stop);  // the unit before is written
        __syncwarp();
        if (p.a.k_new && s.t0 == 0) {
          // the window's rows on their way to L1: 256 bytes each of K and V
#pragma unroll 1
          for (int k = lane; k < s.r.rows * 4; k += 32) {
            const int64_t row = s.r.row0 + (k >> 2);
            const char* at = k & 2 ? static_cast<const char*>(p.a.v_new) + row * p.a.v_row_stride + s.kvh * p.a.v_head_stride
                                   : static_cast<const char*>(p.a.k_new) + row * p.a.k_row_stride + s.kvh * p.a.k_head_stride;
            asm volatile("prefetch.global.L1 [%0];" ::"l"(at + (k & 1) * 128));
          }
          if (p.a.parents) {
#pragma unroll 1
            for (int k = lane; k < s.r.rows; k += 32) x.parents[k] = p.a.parents[s.r.row0 + k];
            __syncwarp();
#pragma unroll 1
            for (int k = lane; k < s.r.rows; k += 32) x.trees[k] = tree_sees(x.parents, k);
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&x.trees_full);
#pragma unroll 1
          for (int j = 0; j < n; ++j, ++i) {
            const int w = i % L::turns, st = i % kStages;
            wait(&x.v_full[st], i / kStages & 1, &x.stop);
            wait(&x.p_full[w], i / L::turns & 1, &x.stop);
            if (stopped(&x.stop)) continue;
            tc_fence_after();
            const uint32_t d = tmem + L::col_o + w * L::o_cols, a = v_lo + st * (kStageBytes / 16), b = p_lo + w * (kParts * L::p_part / 16);
            // the parts of one type: columns side by side in one instruction
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma_f8(d, a + k * (32 * kD / 16), v_hi, b + k * (32 * ROWS / 16), p_hi, f8_idesc(kD, L::accs * ROWS, true, true), j >= L::turns || k > 0);
            if constexpr (L::accs == 2)
#pragma unroll
              for (int k = 0; k < kTile / 32; ++k)
                mma_f8(d, a + k * (32 * kD / 16), v_hi, b + 2 * (L::p_part / 16) + k * (32 * ROWS / 16), p_hi, f8_idesc(kD, ROWS, true, true, true), true);
            mma_commit(&x.o_done[w]);
            mma_commit(&x.v_empty[st]);
          }
        }
        __syncwarp();
        ++u;
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: a thread is a token. A group's turn, and its first row.
    const int group = warp >> 2, token = tid & (kGroupThreads - 1);
    const int turn = L::split ? group >> 1 : group, col0 = L::split ? (group & 1) * kCols : 0;
    const uint32_t quarter = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    const uint32_t my_o = quarter + L::col_o + turn * L::o_cols + col0;
    const int flip = ROWS == 64 ? token >> 1 & 3 : token >> 2 & 1;  // the swizzle of a token's row of P
    unsigned char* my_p = s_p + turn * kParts * L::p_part + token * ROWS;
    uint32_t i0 = 0, u = 0;  // tiles and units of the CTA before this one
    f32x2 l[kCols / 2];
#pragma unroll 1
    while (line.next(p, s)) {
      const int n = s.t1 - s.t0;
      const int rows = min(kCols, s.rows - col0);  // of this group (< 1: none)
      const int j0 = (turn - (int)(i0 % L::turns) + L::turns) % L::turns;  // its first tile
      // the window's own part, while Q is split and the first scores are formed: 16 rows a warp,
      // and a share of the dims
      const bool own = p.a.k_new != nullptr && s.t0 == 0;  // the first piece takes the window in
      float* own_o = p.own_o + (int64_t)blockIdx.x * ROWS * kD;
      if (own) {
        constexpr int kSlices = 16 / (ROWS / 16);  // of the dims
        const int i16 = warp / kSlices * 16, j1 = (warp % kSlices + 1) * (kD / 8 / kSlices), jn = kD / 8 / kSlices;
        if (p.a.parents) wait(&x.trees_full, u & 1, &x.stop);
        __syncwarp();
        if (i16 < s.rows) {
          const Sees* trees = p.a.parents ? x.trees : nullptr;
          const bool odd = own_part<kD, ROWS, T>(p, s, i16, j1 - jn, j1, trees, own_o, kD, x.own);
          if (odd) {
            // this warp's dims, from its own references (they are the same in every slice)
            __syncwarp();
#pragma unroll 1
            for (int i = i16; i < min(s.rows, i16 + 16); ++i)
              own_odd<kD, ROWS, T>(p, s, i, (j1 - jn) * 8, j1 * 8, trees, x.own[i].x, own_o + i * kD);
          }
        }
      }
      wait(&x.q_full, u & 1, &x.stop);
      __syncwarp();
#pragma unroll
      for (int r = 0; r < kCols / 2; ++r) l[r] = 0;
      if (token < kCols) {
        x.neg_m[group][token] = token < rows ? 0.f : kNone;  // no row: its scores ask for nothing
        x.fac[group][token] = x.q_fac[col0 + token];
      }
      if (tid < s.rows) x.at[tid] = (int32_t)s.at(p, ROWS, tid);
      bool fresh = true;  // no token of this unit seen yet: the references are not set
      int look = j0 + kLook * L::turns;  // the tile from which on references may be lowered
      bar_sync(1 + group, kGroupThreads);
      if (token == 0) mbar_arrive(&x.q_empty);
      int j = j0;
#pragma unroll 1
      for (; j < n; j += L::turns) {
        const uint32_t i = i0 + j, slot = i % kMeta, phase = i / L::turns & 1, buf = i % L::s_bufs;
        const uint32_t my_s = quarter + buf * ROWS + col0;
        wait(&x.meta_full[slot], i / kMeta & 1, &x.stop);
        const float ks = x.ks[slot][token >> p.page_shift], vs = x.vs[slot][token >> p.page_shift];
        const bool valid = vs > 0.f && (s.t0 + j) * kTile + token < s.r.len;
        const float lv = __log2f(vs), inv_v = valid ? 1.f / vs : 0.f;
        wait(&x.s_full[buf], i / L::s_bufs & 1, &x.stop);
        __syncwarp();
        tc_fence_after();
        // 16 rows a step (registers); rows behind the block's last are skipped. First whether a
        // score is too far above its reference, then, from TMEM again, P.
        const bool all_valid = __all_sync(0xffffffffu, valid);
        const f32x2 ks2 = pair(ks, ks), lv2 = pair(lv, lv);
        // scores less references of rows c .. c + 15
        auto scores = [&](int c, float* y) {
          tmem_ld16(my_s + c, y);
          tmem_wait_ld();
          tmem_tie16(y);
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(&x.neg_m[group][c + r]);
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&x.fac[group][c + r]);
            const float2 a = unpair(fma2(pair(y[r], y[r + 1]), mul2(ks2, f.x), add2(lv2, m.x)));
            const float2 b = unpair(fma2(pair(y[r + 2], y[r + 3]), mul2(ks2, f.y), add2(lv2, m.y)));
            y[r] = a.x, y[r + 1] = a.y, y[r + 2] = b.x, y[r + 3] = b.y;
          }
          if (!all_valid) {
#pragma unroll
            for (int r = 0; r < 16; ++r) y[r] = valid ? y[r] : -INFINITY;
          }
        };
        float top = -INFINITY;
        const bool looks = j >= look;
        if (!fresh && !looks) {
#pragma unroll 1
          for (int c = 0; c < rows; c += 16) {
            float y[16];
            scores(c, y);
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, y[r]);
          }
        }
        if (bar_or(1 + group, kGroupThreads, fresh || looks || top > kSlack)) {
          // rows whose largest score is that far up get a new reference (and at a look those where
          // it is below 2^kHead): each by its own scores, whatever its neighbours do
#pragma unroll 1
          for (int c = 0; c < rows; c += 16) {
            float y[16];
            scores(c, y);
            const float v = reduce_columns(y, lane, [](float a, float b) { return fmaxf(a, b); });
            if (lane < 16) x.red[group][warp & 3][c + lane] = v;
          }
          const bool any_valid = bar_or(1 + group, kGroupThreads, valid);
          bool moves = false;
          if (token < kCols) {
            float d = -INFINITY;
            if (token < rows) {
#pragma unroll
              for (int k = 0; k < 4; ++k) d = fmaxf(d, x.red[group][k][token]);
            }
            const float old = -x.neg_m[group][token], low = x.peak[group][token] - kDeep;
            float m = old;
            if (d > -INFINITY) {
              if (fresh || d > kSlack) m = old + (d - kHead);
              else if (looks && d < kHead) m = fmaxf(old + (d - kHead), low);
            }
            moves = m != old;
            x.delta[group][token] = ex2(old - m);
            x.neg_m[group][token] = -m;
            x.peak[group][token] = fresh ? (d > -INFINITY ? m : kNone) : fmaxf(low + kDeep, m);
          }
          if (bar_or(1 + group, kGroupThreads, moves) && !fresh) {
#pragma unroll
            for (int r = 0; r < kCols / 2; r += 2) {
              const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&x.delta[group][2 * r]);
              l[r] = mul2(l[r], d.x);
              l[r + 1] = mul2(l[r + 1], d.y);
            }
            wait(&x.o_done[turn], phase ^ 1, &x.stop);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < rows; c += 8) {
              const float4 a = *reinterpret_cast<const float4*>(&x.delta[group][c]), b = *reinterpret_cast<const float4*>(&x.delta[group][c + 4]);
              const float by[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
              bool moved = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) moved |= by[e] != 1.f;
              if (!moved) continue;  // the same for every thread
#pragma unroll 1
              for (int part = 0; part < L::accs; ++part) {
                float o[8];
                tmem_ld8(my_o + part * ROWS + c, o);
                tmem_wait_ld();
                tmem_tie8(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= by[e];
                tmem_st8(my_o + part * ROWS + c, o);
              }
            }
            tmem_wait_st();
          }
          if (any_valid) {
            fresh = false;
            if (looks) look = j + kLook * L::turns;
          }
        }
        // P's place: the product that read it is done (one of an earlier unit was awaited there)
        if (j >= L::turns) wait(&x.o_done[turn], phase ^ 1, &x.stop);
        __syncwarp();
        const f32x2 inv2 = pair(inv_v, inv_v);
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (c >= apart(rows)) continue;
          float y[16];
          scores(c, y);
          uint32_t codes[4][kParts];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = c / 2 + 2 * k;
            const float e0 = ex2(y[4 * k]), e1 = ex2(y[4 * k + 1]), e2 = ex2(y[4 * k + 2]), e3 = ex2(y[4 * k + 3]);
            l[r] = fma2(pair(e0, e1), inv2, l[r]);
            l[r + 1] = fma2(pair(e2, e3), inv2, l[r + 1]);
            split_p<L::accs>(__floats2half2_rn(e0, e1), __floats2half2_rn(e2, e3), codes[k]);
          }
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            *reinterpret_cast<uint4*>(my_p + part * L::p_part + (((col0 + c) / 16) ^ flip) * 16) =
                make_uint4(codes[0][part], codes[1][part], codes[2][part], codes[3][part]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.s_free[buf]);
        if (!valid && col0 == 0) {  // whatever lies behind the last token: 0 times it must be 0
          wait(&x.v_full[i % kStages], i / kStages & 1, &x.stop);
          uint4* v = reinterpret_cast<uint4*>(sm + L::off_v + (i % kStages) * kStageBytes + token * kD);
#pragma unroll
          for (int k = 0; k < kD / 16; ++k) v[k] = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.p_full[turn]);
      }
      // ---- the end of the unit: sums over the tokens, then the turns meet
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        float y[16];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float2 v = unpair(l[c / 2 + r]);
          y[2 * r] = v.x;
          y[2 * r + 1] = v.y;
        }
        const float v = reduce_columns(y, lane, [](float a, float b) { return a + b; });
        if (lane < 16) x.red[group][warp & 3][c + lane] = v;
      }
      if (token == 0) x.live[group] = !fresh;
      if (j > j0) wait(&x.o_done[turn], (i0 + j - L::turns) / L::turns & 1, &x.stop);  // its last product
      if (!own || !p.a.parents) wait(&x.trees_full, u & 1, &x.stop);  // every phase has to be seen
      __syncwarp();
      bar_sync(kBarAll, kSoftmaxThreads);
      tc_fence_after();
      const bool whole = s.whole();
      float* part = p.part + (2 * (int64_t)blockIdx.x + (s.t0 == 0 ? 1 : 0)) * slot_floats(ROWS, kD);
      if (tid < s.rows) {
        const int r = tid, c = r % kCols;
        float m[L::turns], sum[L::turns];
        const float2 ml = own ? x.own[r] : make_float2(kNone, 0.f);
        float to = ml.x;
#pragma unroll
        for (int k = 0; k < L::turns; ++k) {
          const int g = L::split ? 2 * k + r / kCols : k;
          const bool live = x.live[g];
          const float (&v)[4][kCols] = x.red[g];
          sum[k] = live ? (v[0][c] + v[1][c]) + (v[2][c] + v[3][c]) : 0.f;
          m[k] = live ? -x.neg_m[g][c] : kNone;
          to = fmaxf(to, m[k]);
        }
        float by = ex2(ml.x - to), all = by * ml.y;
        x.w[L::turns][r] = by;
#pragma unroll
        for (int k = 0; k < L::turns; ++k) {
          m[k] = ex2(m[k] - to);
          all = fmaf(m[k], sum[k], all);
        }
        by = 1.f;
        if (whole) {
          by = finish_row(p, x.at[r], to, all);
        } else {
          part[ROWS * kD + r] = to;
          part[ROWS * kD + ROWS + r] = all;
        }
        x.w[L::turns][r] *= by;
#pragma unroll
        for (int k = 0; k < L::turns; ++k) x.w[k][r] = m[k] * by;
      }
      bar_sync(kBarAll, kSoftmaxThreads);
      // a group finishes 8 rows at a time; a thread is a dim
      const int d = token;
#pragma unroll 1
      for (int c = group * 8; c < s.rows; c += 8 * kGroups) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = own && c + e < s.rows ? x.w[L::turns][c + e] * own_o[(c + e) * kD + d] : 0.f;
#pragma unroll 1
        for (int k = 0; k < L::turns; ++k) {
          if (!x.live[L::split ? 2 * k : k]) continue;  // both groups of a turn see the same tokens
          float y[L::accs][8];
#pragma unroll
          for (int part_ = 0; part_ < L::accs; ++part_) tmem_ld8(quarter + L::col_o + k * L::o_cols + part_ * ROWS + c, y[part_]);
          tmem_wait_ld();
#pragma unroll
          for (int part_ = 0; part_ < L::accs; ++part_) tmem_tie8(y[part_]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float v = y[0][e];
            if constexpr (L::accs == 2) v = fmaf(y[1][e], 0x1p-9f, v);
            else v = fmaf(fmaf(y[L::accs - 1][e], 0x1p-5f, y[1][e]), 0x1p-5f, v);
            o[e] = fmaf(x.w[k][c + e], v, o[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (c + e >= s.rows) break;
          if (whole) reinterpret_cast<T*>(p.a.out)[(int64_t)x.at[c + e] * kD + d] = T(o[e]);
          else part[(c + e) * kD + d] = o[e];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.o_free);
      bar_sync(kBarAll, kSoftmaxThreads);  // what the groups share has been read
      if (!whole) {
        if (s.t0 == 0) {
          desc.x = s.b;
          desc.y = s.kvh * s.r.blocks + s.block;
          desc.z = s.rows;
        } else {
          desc.w = s.t1 == s.r.tiles ? 1 : 0;
        }
      }
      i0 += n;
      ++u;
    }
    if (tid == 0) p.desc[blockIdx.x] = desc;
  }
  if (stopped(&x.stop)) {
    atomicOr(&g_window_error, 1u);  // by any thread: one may have left its loops before another gave up
    // copies in flight land before the CTA leaves its shared memory
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 26)) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kFirst) {
    tc_fence_after();
    tmem_free(tmem, L::tmem_cols);
  }
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, or null.
EncodeTiled encoder() {
  static const EncodeTiled f = [] {
    void* at = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      at = nullptr;
    return reinterpret_cast<EncodeTiled>(at);
  }();
  return f;
}

// K or V as [pages][heads][tokens of a page][D] bytes; a box is one page of one head.
bool page_map(CUtensorMap* map, const ts_kv_cache& c, void* base, int64_t page_stride, int64_t head_stride, int64_t token_stride) {
  // the stride of an extent of one is never used, but has to be a valid one
  if (c.heads == 1) head_stride = token_stride;
  if (c.num_pages <= 1) page_stride = token_stride;
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)std::max<int64_t>(c.num_pages, 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)token_stride, (cuuint64_t)head_stride, (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)kD, (cuuint32_t)c.page_size, 1, 1}, step[4] = {1, 1, 1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int ROWS, int QP, typename T>
cudaError_t launch(const WindowParams& p, const CUtensorMap& k, const CUtensorMap& v, int sms, cudaStream_t s) {
  constexpr int bytes = smem_bytes<ROWS, QP>();
  cudaError_t e = allow_smem<k_window_tc<ROWS, QP, T>>(bytes);
  if (e != cudaSuccess) return e;
  k_window_tc<ROWS, QP, T><<<sms, kThreads, bytes, s>>>(p, k, v);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((int64_t)p.c.max_pages * p.c.page_size <= kTile) return cudaSuccess;  // units of one tile are never split
  return launch_after(k_join<kD, ROWS, kTile, T>, dim3(sms, ROWS / 4), 128, 0, s, p);
}

}  // namespace

cudaError_t window_read_error(uint32_t* word, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_window_error, sizeof(uint32_t));
  if (e == cudaSuccess && clear && *word) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_window_error, &zero, sizeof(zero));
  }
  return e;
}

cudaError_t launch_window_tc(const WindowParams& params, int rows, int sms, cudaStream_t s) {
  WindowParams p = params;
  p.own_ml = nullptr;  // the window's own part is in the pieces; own_o: a block a CTA
  CUtensorMap k, v;
  const ts_kv_cache& c = p.c;
  if (!encoder()) return cudaErrorNotSupported;
  if (!page_map(&k, c, c.k, c.k_page_stride, c.k_head_stride, c.k_token_stride) ||
      !page_map(&v, c, c.v, c.v_page_stride, c.v_head_stride, c.v_token_stride))
    return cudaErrorInvalidValue;
  const bool bf16 = p.a.dtype == TS_BF16;
  if (rows == 32)
    return bf16 ? launch<32, 2, __nv_bfloat16>(p, k, v, sms, s) : launch<32, 3, __half>(p, k, v, sms, s);
  return bf16 ? launch<64, 2, __nv_bfloat16>(p, k, v, sms, s) : launch<64, 3, __half>(p, k, v, sms, s);
}

}  // namespace tsv
