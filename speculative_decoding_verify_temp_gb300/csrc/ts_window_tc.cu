// Window attention over the 8-bit cache on the tensor cores, head_dim 128.
//
//   k_window_prep  (ts_window_prep.cuh) Q in e4m3 parts, and the window's own part
//   k_window_tc    the cached tokens: one persistent CTA an SM
//   k_join         joins the pieces of units that more than one CTA worked on
//
// The cache is read once and its bytes go to the tensor cores as they are: TMA brings pages
// into shared memory and tcgen05.mma (kind f8f6f4) takes the e4m3 codes, so no thread touches K
// or V. What the products need in more than four significant bits is split into e4m3 parts.
// Both products are turned round, so that the long side of the tile, 128 tokens or 128 dims,
// is the M = 128 of the instruction and the window's rows, few as they are, its N:
//
//   S^T [128 tokens x ROWS] = K [128 x D] (Q_hi + Q_lo (+ Q_lo2))^T      one accumulator
//   O^T [D x 3 ROWS]       += V^T [D x 128 tokens] [P_hi | P_lo | P_lo2]  one accumulator a part
//
// A thread of a softmax group is a token: it reads its row of S^T from TMEM, the scales of its
// block and its validity are its own, and it writes its row of P. P = 2^(x - m) with a
// reference m a row (x in log2 units, V's scale in the exponent as in ts_window.cu); a
// reference follows only when a score exceeds it by 2^8 (one vote a tile), and then O is scaled
// in TMEM. Parts of P: the fp16 rounding of p in three codes, the second and third scaled by
// 2^5 and 2^10, so that all 11 bits are kept down to 2^-20 where the row's largest p is between
// 2^7 and 2^8.
//
// Two softmax groups of four warps take turns at the tiles, each with its own S, O, m and
// sums in TMEM and registers, so that one's arithmetic overlaps the other's products; they
// meet at the end of a unit. One warp loads (a ring of four tiles of 32 KB, 128 KB in flight
// an SM), one lane issues the products.
//
// Every wait on a barrier is bounded; after one ran out no wait waits and nothing more is
// issued, so that the CTA runs to its end (results unspecified, reported by ts_device_error).
#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "ts_window.cuh"
#include "ts_window_prep.cuh"

namespace tsv {

namespace {

constexpr int kTile = 128;
constexpr int kD = 128;
constexpr int kStages = 4;         // tiles of K, and as many of V, in shared memory
constexpr int kStageBytes = kTile * kD;
constexpr int kMeta = 8;           // tiles whose scales are in shared memory
constexpr int kAhead = 2;          // tiles that K and its products run ahead of V and its: a unit's
                                   // scores are ready when its group comes to them
constexpr int kParts = 3;          // of a probability
constexpr int kGroupThreads = 128;
constexpr int kThreads = 3 * kGroupThreads;  // two softmax groups; the third's first two warps load and issue
// registers a thread: 2 * 208 + 88 = 3 * 168, what the block is launched with
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "the groups' registers");
constexpr int kMinTiles = 2;       // least tiles a CTA takes: pieces of 256 tokens or more
constexpr float kHead = 4.f;       // a reference is set this far below the largest score
constexpr uint64_t kWaitCycles = (uint64_t)1 << 32;

__device__ uint32_t g_window_error;

template <int ROWS, int QP>
struct Layout {
  static constexpr int q_bytes = QP * ROWS * kD;
  static constexpr int q_buffers = ROWS == 64 && QP == 3 ? 1 : 2;  // what shared memory has room for
  static constexpr int p_part = ROWS * kTile;
  static constexpr int off_v = kStages * kStageBytes;
  static constexpr int off_q = 2 * kStages * kStageBytes;
  static constexpr int off_p = off_q + q_buffers * q_bytes;
  static constexpr int off_x = off_p + 2 * kParts * p_part;
  static constexpr int group_cols = (1 + kParts) * ROWS;  // TMEM columns of a group: S, O parts
};

template <int ROWS>
struct Shared {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], meta_full[kMeta];
  uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], p_full[2], o_done[2], o_free;
  alignas(16) float q_scale[2][4];         // what Q's codes stand for
  float ks[kMeta][8], vs[kMeta][8];        // scales of a tile's pages (vs 0: no such page)
  alignas(16) float m[2][ROWS];            // read as float4
  alignas(16) float delta[2][ROWS];
  float red[2][4][ROWS];
  float4 w[ROWS];  // a row's factors: the groups' and the window's own part
  int32_t at[2][ROWS];  // a row's index in [total_rows][heads_q], a copy for each group
  int32_t live[2];
  uint32_t tmem;
  int32_t stop;
};

static_assert(offsetof(Shared<32>, m) % 16 == 0 && offsetof(Shared<64>, m) % 16 == 0 && offsetof(Shared<32>, w) % 16 == 0 &&
                  offsetof(Shared<64>, w) % 16 == 0 && Layout<32, 2>::off_x % 16 == 0,
              "vector loads");

template <int ROWS, int QP>
constexpr int smem_bytes() { return Layout<ROWS, QP>::off_x + (int)sizeof(Shared<ROWS>) + 1024; }

__device__ __forceinline__ bool stopped(const int32_t* stop) { return *reinterpret_cast<const volatile int32_t*>(stop) != 0; }

__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int32_t* stop) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (stopped(stop)) return;
    if ((uint64_t)(clock64() - t0) > kWaitCycles) {
      *reinterpret_cast<volatile int32_t*>(stop) = 1;
      atomicOr(&g_window_error, 1u);
      return;
    }
  }
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

// Of the lanes' 32 columns x: lane l gets the reduction of column l over the lanes. 31 shuffles.
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
__device__ __forceinline__ float reduce_columns(const float* x, int lane, F f) {
  float y[16];
  const bool up = lane & 16;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float keep = up ? x[i + 16] : x[i], give = up ? x[i] : x[i + 16];
    y[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, 16));
  }
  halve<8>(y, lane, f);
  return y[0];
}

// The next part of two values: its codes; the values become the rest, times 2^5 (exact).
__device__ __forceinline__ uint16_t next_part(__half2& h) {
  uint16_t codes;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(codes) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
  const uint32_t back = e4m3x2_to_f16x2(codes);
  h = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(32.f));
  return codes;
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
  int4 desc = make_int4(-1, 0, 0, 0);
  grid_launch();
  Line<ROWS, kTile> line;
  if (!line_begin<ROWS, kTile, kThreads>(p, kMinTiles, line)) {
    if (tid == 0) p.desc[blockIdx.x] = desc;
    grid_wait();  // so that this kernel's end is the end of the one before too
    return;
  }
  constexpr uint32_t kTmemCols = 2 * L::group_cols;  // 256 or 512
  if (warp == 9) tmem_alloc(&x.tmem, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&x.k_full[i], 1);
      mbar_init(&x.k_empty[i], 1);
      mbar_init(&x.v_full[i], 1);
      mbar_init(&x.v_empty[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&x.meta_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x.q_full[i], 1);
      mbar_init(&x.q_empty[i], 3);  // the products, and both groups have read the scale
      mbar_init(&x.s_full[i], 1);
      mbar_init(&x.s_free[i], 4);
      mbar_init(&x.p_full[i], 4);
      mbar_init(&x.o_done[i], 1);
    }
    mbar_init(&x.o_free, 8);
    x.stop = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = x.tmem;
  Segment s{};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---- loads: lane i brings page i of a tile. K runs kAhead tiles ahead of V, across
      // units.
      const int pages = kTile >> p.page_shift;
      const int page_bytes = p.c.page_size * kD;
      uint32_t ik = 0, iv = 0, u = 0;
      int32_t page_a = -1, head_a = 0, page_b = -1, head_b = 0;  // of the last two tiles, V not loaded yet
      auto load = [&](uint32_t i, unsigned char* base, const CUtensorMap* map, int32_t page, int32_t head, uint64_t* full, uint64_t* empty) {
        const int st = i % kStages;
        wait(&empty[st], (i / kStages & 1) ^ 1, &x.stop);
        __syncwarp();
        if (stopped(&x.stop)) return;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], kStageBytes);
        __syncwarp();
        // a page outside the tensor reads as zeros
        if (lane < pages)
          tma_load_4d(base + st * kStageBytes + lane * page_bytes, map, 0, 0, head, page >= 0 ? page : (int32_t)p.c.num_pages, &full[st]);
      };
      auto load_v = [&]() {
        const bool two = ik - iv == 2;
        load(iv, sm + L::off_v, &v_map, two ? page_a : page_b, two ? head_a : head_b, x.v_full, x.v_empty);
        ++iv;
      };
      auto load_q = [&]() {
        const int qb = u % L::q_buffers;
        wait(&x.q_empty[qb], (u / L::q_buffers & 1) ^ 1, &x.stop);
        __syncwarp();
        if (lane == 0 && !stopped(&x.stop)) {
          const int64_t blk = block_base(s.r.row0, p.group, ROWS, s.b) + s.block;
          const uint8_t* q = p.q_parts + (blk * p.c.heads + s.kvh) * q_block_bytes(ROWS, QP);
          mbar_arrive_expect_tx(&x.q_full[qb], L::q_bytes + 16);
          bulk_g2s(s_q + qb * L::q_bytes, q, L::q_bytes, &x.q_full[qb]);
          bulk_g2s(x.q_scale[qb], q + L::q_bytes, 16, &x.q_full[qb]);
        }
        __syncwarp();
        ++u;
      };
      bool waited = false;
      while (line.next(p, s)) {
        const int32_t* table = p.c.page_table + s.b * p.c.ld_table;
        auto page_of = [&](int t) -> int32_t {
          const int32_t tok = t * kTile + (lane << p.page_shift);
          if (lane >= pages || t >= s.t1 || tok >= s.r.len) return -1;
          const int32_t id = table[tok >> p.page_shift];
          return id >= 0 && id < p.c.num_pages ? id : -1;
        };
        auto scales_of = [&](int32_t page, float& ks, float& vs) {
          ks = vs = 0.f;
          if (page < 0) return;
          ks = __ldg(p.c.k_scale + (int64_t)page * p.c.heads + s.kvh);
          vs = fmaxf(__ldg(p.c.v_scale + (int64_t)page * p.c.heads + s.kvh), 0x1p-100f);
        };
        int32_t page = page_of(s.t0), page1 = page_of(s.t0 + 1);
        // Q comes from the kernel before; the first tiles of the cache need not wait for it
        bool q_due = true;
        if (waited) {
          // with one buffer, Q waits for the unit before, and that for the rest of its V
          if (L::q_buffers == 1)
            while (iv < ik) load_v();
          load_q();
          q_due = false;
        }
        float ks, vs;
        scales_of(page, ks, vs);
        for (int t = s.t0; t < s.t1; ++t) {
          const int32_t page2 = page_of(t + 2);
          float ks1, vs1;
          scales_of(page1, ks1, vs1);
          if (q_due && ik == kAhead) {
            grid_wait();
            waited = true;
            load_q();
            q_due = false;
          }
          load(ik, sm, &k_map, page, s.kvh, x.k_full, x.k_empty);
          // the slot of tile ik - kMeta: its group has freed S of a later tile since
          if (lane < pages) {
            x.ks[ik % kMeta][lane] = ks;
            x.vs[ik % kMeta][lane] = vs;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.meta_full[ik % kMeta]);
          if (ik - iv == kAhead) load_v();
          page_a = page_b, head_a = head_b;
          page_b = page, head_b = s.kvh;
          ++ik;
          page = page1;
          page1 = page2;
          ks = ks1;
          vs = vs1;
        }
        if (q_due) {
          grid_wait();
          waited = true;
          load_q();
        }
      }
      while (iv < ik) load_v();
    } else if (warp == 9 && lane == 0) {
      // ---- the first products, S of tile after tile. Tiles are counted through the CTA's
      // units; tile i belongs to group i % 2.
      const uint32_t k_lo = desc_lo(smem_u32(sm), 16), q_lo = desc_lo(smem_u32(s_q), 16), hi = desc_hi(8 * kD, kSwizzle128);
      uint32_t i = 0, u = 0;
      while (line.next(p, s)) {
        const int n = s.t1 - s.t0, qb = u % L::q_buffers;
        wait(&x.q_full[qb], u / L::q_buffers & 1, &x.stop);
        for (int j = 0; j < n; ++j, ++i) {
          const int w = i & 1, st = i % kStages;
          wait(&x.k_full[st], i / kStages & 1, &x.stop);
          if (i >= 2) wait(&x.s_free[w], (i / 2 - 1) & 1, &x.stop);
          if (stopped(&x.stop)) continue;
          tc_fence_after();
          const uint32_t d = tmem + w * L::group_cols, a = k_lo + st * (kStageBytes / 16), b = q_lo + qb * (L::q_bytes / 16);
#pragma unroll
          for (int part = 0; part < QP; ++part)
#pragma unroll
            for (int k = 0; k < kD / 32; ++k)
              mma_f8(d, a + k * 2, hi, b + part * (ROWS * kD / 16) + k * 2, hi, f8_idesc(kTile, ROWS, false, false), part > 0 || k > 0);
          mma_commit(&x.s_full[w]);
          mma_commit(&x.k_empty[st]);
          if (j == n - 1) mma_commit(&x.q_empty[qb]);
        }
        ++u;
      }
    } else if (warp == 10 && lane == 0) {
      // ---- the second products, O
      const uint32_t v_lo = desc_lo(smem_u32(sm) + L::off_v, 16), v_hi = desc_hi(8 * kD, kSwizzle128);
      const uint32_t p_lo = desc_lo(smem_u32(s_p), L::p_part), p_hi = desc_hi(8 * ROWS, ROWS == 64 ? kSwizzle64 : kSwizzle32);
      uint32_t i = 0, u = 0;
      while (line.next(p, s)) {
        const int n = s.t1 - s.t0;
        for (int j = 0; j < n; ++j, ++i) {
          const int w = i & 1, st = i % kStages;
          wait(&x.v_full[st], i / kStages & 1, &x.stop);
          if (j == 0 && u > 0) wait(&x.o_free, (u - 1) & 1, &x.stop);
          wait(&x.p_full[w], i / 2 & 1, &x.stop);
          if (stopped(&x.stop)) continue;
          tc_fence_after();
          const uint32_t d = tmem + w * L::group_cols + ROWS, a = v_lo + st * (kStageBytes / 16), b = p_lo + w * (kParts * L::p_part / 16);
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma_f8(d, a + k * (32 * kD / 16), v_hi, b + k * (32 * ROWS / 16), p_hi, f8_idesc(kD, kParts * ROWS, true, true), j >= 2 || k > 0);
          mma_commit(&x.o_done[w]);
          mma_commit(&x.v_empty[st]);
        }
        ++u;
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax: group w takes tiles t0 + w, t0 + w + 2, ...; a thread is a token
    const int w = warp >> 2, token = tid & (kGroupThreads - 1);
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + w * L::group_cols;  // this warp's lanes
    unsigned char* my_p = s_p + w * kParts * L::p_part + token * ROWS;
    const int turn = ROWS == 64 ? token >> 1 & 3 : token >> 2 & 1;  // the swizzle of its row
    uint32_t i0 = 0, u = 0;  // tiles and units of the CTA before this one
    float l[ROWS];
    bool waited = false;
    while (line.next(p, s)) {
      const int n = s.t1 - s.t0, j0 = (w ^ i0) & 1;
      const int last = n - 1 - ((n - 1 - j0) & 1);  // this group's last tile (< j0: none)
      wait(&x.q_full[u % L::q_buffers], u / L::q_buffers & 1, &x.stop);
      const float q_scale = x.q_scale[u % L::q_buffers][0] * p.scale_log2;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) l[r] = 0.f;
      if (token < ROWS) x.m[w][token] = 0.f;
      if (token < ROWS) x.at[w][token] = (int32_t)s.at(p, ROWS, min(token, s.rows - 1));
      bool fresh = true;  // no token of this unit seen yet: the references are not set
      bar_sync(1 + w, kGroupThreads);
      if (token == 0) mbar_arrive(&x.q_empty[u % L::q_buffers]);
      for (int j = j0; j < n; j += 2) {
        const uint32_t i = i0 + j, slot = i % kMeta;
        wait(&x.meta_full[slot], i / kMeta & 1, &x.stop);
        const float ks = x.ks[slot][token >> p.page_shift], vs = x.vs[slot][token >> p.page_shift];
        const bool valid = vs > 0.f && (s.t0 + j) * kTile + token < s.r.len;
        const float f = ks * q_scale, lv = __log2f(vs), inv_v = valid ? 1.f / vs : 0.f;
        wait(&x.s_full[w], i / 2 & 1, &x.stop);
        __syncwarp();
        tc_fence_after();
        float t[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; r += 32) tmem_ld32(mine + r, t + r);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.s_free[w]);
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < ROWS; r += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&x.m[w][r]);
          t[r] = fmaf(t[r], f, lv) - m.x;
          t[r + 1] = fmaf(t[r + 1], f, lv) - m.y;
          t[r + 2] = fmaf(t[r + 2], f, lv) - m.z;
          t[r + 3] = fmaf(t[r + 3], f, lv) - m.w;
        }
        if (!__all_sync(0xffffffffu, valid)) {
#pragma unroll
          for (int r = 0; r < ROWS; ++r) t[r] = valid ? t[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) top = fmaxf(top, t[r]);
        if (bar_or(1 + w, kGroupThreads, fresh || top > kSlack)) {
          // rows whose largest score is that far up get a new reference
#pragma unroll
          for (int h = 0; h < ROWS; h += 32) {
            x.red[w][warp & 3][h + lane] = reduce_columns(t + h, lane, [](float a, float b) { return fmaxf(a, b); });
            __syncwarp();  // one half after the other: fewer registers
          }
          const bool any_valid = bar_or(1 + w, kGroupThreads, valid);
          if (token < ROWS) {
            float d = x.red[w][0][token];
#pragma unroll
            for (int k = 1; k < 4; ++k) d = fmaxf(d, x.red[w][k][token]);
            d = (fresh ? d > -INFINITY : d > kSlack) ? d - kHead : 0.f;
            x.delta[w][token] = d;
            x.m[w][token] += d;
          }
          bar_sync(1 + w, kGroupThreads);
#pragma unroll
          for (int r = 0; r < ROWS; r += 4) {
            const float4 d = *reinterpret_cast<const float4*>(&x.delta[w][r]);
            t[r] -= d.x, t[r + 1] -= d.y, t[r + 2] -= d.z, t[r + 3] -= d.w;
            l[r] *= ex2(-d.x), l[r + 1] *= ex2(-d.y), l[r + 2] *= ex2(-d.z), l[r + 3] *= ex2(-d.w);
            asm volatile("" ::: "memory");  // no loads ahead of their turn: registers
          }
          if (!fresh) {
            wait(&x.o_done[w], (i / 2 - 1) & 1, &x.stop);
            __syncwarp();
            tc_fence_after();
            for (int c0 = 0; c0 < kParts * ROWS; c0 += 8) {
              float o[8];
              tmem_ld8(mine + ROWS + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= ex2(-x.delta[w][(c0 + e) % ROWS]);
              tmem_st8(mine + ROWS + c0, o);
            }
            tmem_wait_st();
          }
          if (any_valid) fresh = false;
        }
        // P's shared memory: the product of this group's tile before is done
        if (j >= 2) wait(&x.o_done[w], (i / 2 - 1) & 1, &x.stop);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < ROWS; r += 16) {
          uint32_t codes[kParts][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              e[q] = ex2(t[r + 4 * k + q]);
              l[r + 4 * k + q] = fmaf(e[q], inv_v, l[r + 4 * k + q]);
            }
            __half2 a = __floats2half2_rn(e[0], e[1]), b = __floats2half2_rn(e[2], e[3]);
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              const uint16_t ca = next_part(a), cb = next_part(b);
              codes[part][k] = (uint32_t)ca | ((uint32_t)cb << 16);
            }
          }
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            *reinterpret_cast<uint4*>(my_p + part * L::p_part + ((r / 16) ^ turn) * 16) =
                make_uint4(codes[part][0], codes[part][1], codes[part][2], codes[part][3]);
        }
        if (!valid) {  // whatever lies behind the last token: 0 times it must be 0
          wait(&x.v_full[i % kStages], i / kStages & 1, &x.stop);
          uint4* v = reinterpret_cast<uint4*>(sm + L::off_v + (i % kStages) * kStageBytes + token * kD);
#pragma unroll
          for (int k = 0; k < kD / 16; ++k) v[k] = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.p_full[w]);
      }
      // ---- the end of the unit: sums over the tokens, then the groups meet. Group w finishes
      // half of the rows; a thread is a dim there.
      const bool whole = s.whole();
      if (!waited) {  // for the window's own part
        grid_wait();
        waited = true;
      }
      constexpr int HALF = ROWS / 2;
      const int d = token, c_lo = w * HALF;
      const bool own_part = whole && p.own_ml != nullptr;
#pragma unroll
      for (int h = 0; h < ROWS; h += 32)
        x.red[w][warp & 3][h + lane] = reduce_columns(l + h, lane, [](float a, float b) { return a + b; });
      float own[HALF];
#pragma unroll
      for (int e = 0; e < HALF; ++e)
        own[e] = own_part && c_lo + e < s.rows ? p.own_o[(int64_t)x.at[w][c_lo + e] * kD + d] : 0.f;
      if (token == 0) x.live[w] = !fresh;
      if (last >= j0) wait(&x.o_done[w], (i0 + last) / 2 & 1, &x.stop);
      __syncwarp();
      bar_sync(3, 2 * kGroupThreads);
      tc_fence_after();
      const int slot = 2 * (int)blockIdx.x + (s.t0 == 0 ? 1 : 0);
      float* part = p.part + (int64_t)slot * slot_floats(ROWS, kD);
      const bool live0 = x.live[0], live1 = x.live[1];
      if (tid < ROWS) {
        const int r = tid;
        float sum[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) sum[g] = (x.red[g][0][r] + x.red[g][1][r]) + (x.red[g][2][r] + x.red[g][3][r]);
        const float m0 = live0 ? x.m[0][r] : kNone, m1 = live1 ? x.m[1][r] : kNone;
        const float to = fmaxf(m0, m1);
        float w0 = live0 ? ex2(m0 - to) : 0.f, w1 = live1 ? ex2(m1 - to) : 0.f, wo = 0.f;
        const float all = w0 * sum[0] + w1 * sum[1];
        if (whole) {
          if (r < s.rows) {
            const float by = finish_row(p, x.at[w][r], to, all, wo);
            w0 *= by;
            w1 *= by;
          }
        } else {
          part[ROWS * kD + r] = to;
          part[ROWS * kD + ROWS + r] = all;
        }
        x.w[r] = make_float4(w0, w1, wo, 0.f);
      }
      bar_sync(3, 2 * kGroupThreads);
      const uint32_t quarter = tmem + ((uint32_t)(warp & 3) << 21);
#pragma unroll
      for (int c0 = 0; c0 < HALF; c0 += 8) {
        if (c_lo + c0 < s.rows) {
          float o[8] = {};
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g ? !live1 : !live0) continue;
            float y[kParts][8];
#pragma unroll
            for (int part_ = 0; part_ < kParts; ++part_)
              tmem_ld8(quarter + g * L::group_cols + (1 + part_) * ROWS + c_lo + c0, y[part_]);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 by = x.w[c_lo + c0 + e];
              o[e] = fmaf(g ? by.y : by.x, fmaf(fmaf(y[2][e], 0x1p-5f, y[1][e]), 0x1p-5f, y[0][e]), o[e]);
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = c_lo + c0 + e;
            if (r < s.rows) {
              if (whole)
                reinterpret_cast<T*>(p.a.out)[(int64_t)x.at[w][r] * kD + d] = T(fmaf(x.w[r].z, own[c0 + e], o[e]));
              else
                part[r * kD + d] = o[e];
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.o_free);
      bar_sync(1 + w, kGroupThreads);  // the group's references and indexes have been read
      if (!whole) {
        if (s.t0 == 0) {
          desc.x = (int)s.b;
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
  if (stopped(&x.stop)) {  // copies in flight land before the CTA leaves its shared memory
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 26)) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, kTmemCols);
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
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)token_stride, (cuuint64_t)head_stride, (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)kD, (cuuint32_t)c.page_size, 1, 1}, step[4] = {1, 1, 1, 1};
  for (int64_t st : {page_stride, head_stride, token_stride})
    if (st <= 0 || st >= (int64_t)1 << 40) return false;
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int ROWS, int QP, typename T>
cudaError_t launch(const WindowParams& p, const CUtensorMap& k, const CUtensorMap& v, int sms, cudaStream_t s) {
  constexpr int bytes = smem_bytes<ROWS, QP>();
  cudaError_t e = cudaFuncSetAttribute(k_window_tc<ROWS, QP, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  if ((e = launch_prep<kD, ROWS, QP, T>(p, s)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k_window_tc<ROWS, QP, T>, p, k, v)) != cudaSuccess) return e;
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

cudaError_t launch_window_tc(const WindowParams& p, int rows, int sms, cudaStream_t s, bool* done) {
  CUtensorMap k, v;
  const ts_kv_cache& c = p.c;
  *done = encoder() != nullptr && c.num_pages > 0 && c.num_pages < INT32_MAX &&
          page_map(&k, c, c.k, c.k_page_stride, c.k_head_stride, c.k_token_stride) &&
          page_map(&v, c, c.v, c.v_page_stride, c.v_head_stride, c.v_token_stride);
  if (!*done) return cudaSuccess;
  const bool bf16 = p.a.dtype == TS_BF16;
  if (rows == 32)
    return bf16 ? launch<32, 2, __nv_bfloat16>(p, k, v, sms, s) : launch<32, 3, __half>(p, k, v, sms, s);
  return bf16 ? launch<64, 2, __nv_bfloat16>(p, k, v, sms, s) : launch<64, 3, __half>(p, k, v, sms, s);
}

}  // namespace tsv
