// Shared by the kernels of window attention (ts_window.cu, ts_window_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ts_verify.h"
#include "ts_common.cuh"
#include "ts_internal.h"
#include "ts_kv.cuh"
#include "ts_tc.cuh"

namespace tsv {

struct WindowParams {
  ts_kv_cache c;
  ts_attn_args a;
  int32_t page_shift;
  int32_t group;
  float scale_log2;
  float* part;      // [2 * CTAs][rows * (D + 2)] pieces: outputs, references, sums
  int4* desc;       // [CTAs] {tail unit's request, its head and row block, rows, 0 | 1: the
                    // CTA's first piece ends its unit}
  int32_t* wide;    // blocks of 64 rows (head_dim 64, where the kernel chooses)
  float* own_o;      // [total_rows * heads_q][D] the window's own part: outputs,
  float2* own_ml;    // [total_rows * heads_q] references and sums
  uint64_t wait_cycles;  // SM clock cycles that a wait may take (ts_window_tc.cu)
};

constexpr float kNone = -3.4028234664e38f;  // the reference before any token: no score is below it

// V's scales are taken as this at least. Sums hold p / scale, p at most 2^15 (head_dim 64) or, where a
// reference was lowered, 2^20 (128): 2^100 times the tokens stays in fp32's range.
constexpr float kLeastScale = 0x1p-80f;
// A NaN, which that would hide, reaches the rows through the scores.
__device__ __forceinline__ float scale_of_v(float vs, float& ks) {
  if (vs != vs) ks = vs;
  return fmaxf(vs, kLeastScale);
}

template <typename T>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) { return f16x2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Bits 15 and 31: the low and the high value are not finite (all exponent bits set).
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w);
template <>
__device__ __forceinline__ uint32_t not_finite<__half>(uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }
template <>
__device__ __forceinline__ uint32_t not_finite<__nv_bfloat16>(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// What the line of tiles needs of a request.
struct Req {
  int64_t row0;
  int32_t rows;    // window rows (0: skipped)
  int32_t len;     // cached tokens
  int32_t blocks;  // row blocks
  int32_t tiles;   // of a unit, >= 1
  __device__ __forceinline__ int64_t weight(int heads) const { return rows ? (int64_t)heads * blocks * tiles : 0; }
  __device__ __forceinline__ uint32_t units(int heads) const { return rows ? (uint32_t)heads * blocks : 0; }
};

// The loads behind a request, apart from what follows from them, so that they can be made early.
struct RawReq {
  int32_t row0, row1, len;
};

__device__ __forceinline__ RawReq raw_request(const WindowParams& p, int64_t b) {
  RawReq r = {0, 0, 0};
  if (b >= p.c.batch) return r;
  if (p.a.qo_indptr) {
    r.row0 = p.a.qo_indptr[b];
    r.row1 = p.a.qo_indptr[b + 1];
  } else {
    const int32_t n = (int32_t)(p.a.total_rows / p.c.batch);
    r.row0 = (int32_t)b * n;
    r.row1 = r.row0 + n;
  }
  r.len = p.c.seq_lens[b];
  return r;
}

template <int ROWS, int TILE>
__device__ __forceinline__ Req request(const WindowParams& p, const RawReq& raw) {
  Req r;
  r.row0 = raw.row0;
  const bool fits = raw.row0 >= 0 && raw.row1 <= p.a.total_rows && raw.row1 > raw.row0 && raw.row1 - raw.row0 <= TS_MAX_WINDOW;
  r.rows = fits ? raw.row1 - raw.row0 : 0;
  r.len = min(max(raw.len, 0), p.c.max_pages << p.page_shift);  // at most 2^30
  r.blocks = (int)((unsigned)(r.rows * p.group + ROWS - 1) / ROWS);
  r.tiles = max((int)((unsigned)(r.len + TILE - 1) / TILE), 1);
  return r;
}

// A CTA's share of the line of all units' tiles: segments, each of one unit.
struct Segment {
  Req r;
  int32_t b, kvh, block, rows;  // rows of this block
  int32_t t0, t1;
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == r.tiles; }
  // window row and head of the block's row i, as an index of [total_rows][heads_q]
  __device__ __forceinline__ int64_t at(const WindowParams& p, int rows_per_block, int i) const {
    const int j = block * rows_per_block + i;
    return (r.row0 + j / p.group) * p.a.heads_q + kvh * p.group + j % p.group;
  }
};

template <int ROWS, int TILE>
struct Line {
  Req r;
  RawReq after;  // the request behind it
  int64_t left;
  int32_t b, kvh, block, tile;
  __device__ __forceinline__ bool next(const WindowParams& p, Segment& s) {
    if (left <= 0) return false;
    if (block >= r.blocks) {
      block = 0;
      ++kvh;
    }
#pragma unroll 1
    while (r.rows == 0 || kvh >= p.c.heads) {
      r = request<ROWS, TILE>(p, after);
      after = raw_request(p, ++b + 1);
      kvh = block = 0;
    }
    s.r = r;
    s.b = b;
    s.kvh = kvh;
    s.block = block;
    s.rows = min(ROWS, r.rows * p.group - block * ROWS);
    s.t0 = tile;
    s.t1 = (int)min((int64_t)r.tiles, tile + left);
    left -= s.t1 - s.t0;
    tile = 0;
    ++block;
    return true;
  }
};

// Where the share of CTA blockIdx.x begins, found by the whole CTA: thread i adds up its own
// run of requests, the sums are scanned, and the thread whose run holds the beginning looks
// it up. Returns false for a CTA without work. least_tiles: a CTA takes this many tiles at least, or as
// many as an average unit has where that is less (14 windows of 8 rows over 4 tokens, head_dim 64:
// 16 us, 39 with four such units a CTA).
template <int ROWS, int TILE, int THREADS>
__device__ __forceinline__ bool line_begin(const WindowParams& p, int least_tiles, Line<ROWS, TILE>& line) {
  static_assert(THREADS % 32 == 0, "whole warps");
  __shared__ int64_t s_scan[THREADS / 32], s_start;
  __shared__ uint32_t s_units[THREADS / 32];  // below 2^28: total_rows * heads_q is below 2^31
  __shared__ int32_t s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t mine = 0;
  uint32_t units = 0;
  const int64_t each = (p.c.batch + THREADS - 1) / THREADS;
  const int64_t b_lo = min(p.c.batch, tid * each), b_hi = min(p.c.batch, b_lo + each);
#pragma unroll 1
  for (int64_t b = b_lo; b < b_hi; ++b) {
    const Req r = request<ROWS, TILE>(p, raw_request(p, b));
    mine += r.weight(p.c.heads);
    units += r.units(p.c.heads);
  }
  units = __reduce_add_sync(0xffffffffu, units);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) {
    s_scan[warp] = upto;
    s_units[warp] = units;
  }
  __syncthreads();
  int64_t all = 0;
  units = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) upto += s_scan[w];
    all += s_scan[w];
    units += s_units[w];
  }
  const int64_t least = all < (int64_t)least_tiles * units ? max(all / max(units, 1u), (int64_t)1) : least_tiles;
  const int64_t share = max((all + gridDim.x - 1) / gridDim.x, least);
  const int64_t begin = min(all, blockIdx.x * share), end = min(all, begin + share);
  if (begin < end && upto - mine <= begin && begin < upto) {  // one thread
    int64_t at = upto - mine;
#pragma unroll 1
    for (int64_t b = b_lo; b < b_hi; ++b) {
      const int64_t w = request<ROWS, TILE>(p, raw_request(p, b)).weight(p.c.heads);
      if (begin < at + w) {
        s_b = (int32_t)b;
        s_start = begin - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  if (begin >= end) return false;
  line.b = s_b;
  line.r = request<ROWS, TILE>(p, raw_request(p, line.b));
  line.after = raw_request(p, line.b + 1);
  const int32_t unit = (int32_t)(s_start / line.r.tiles);
  line.tile = (int32_t)(s_start % line.r.tiles);
  line.kvh = unit / line.r.blocks;
  line.block = unit % line.r.blocks;
  line.left = end - begin;
  return true;
}

// The tiles of the whole line, by the whole CTA.
template <int ROWS, int TILE, int THREADS>
__device__ __forceinline__ int64_t line_length(const WindowParams& p) {
  __shared__ int64_t s_sum[THREADS / 32];
  int64_t mine = 0;
#pragma unroll 1
  for (int64_t b = threadIdx.x; b < p.c.batch; b += THREADS) mine += request<ROWS, TILE>(p, raw_request(p, b)).weight(p.c.heads);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = mine;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) all += s_sum[w];
  return all;
}

// A piece's slot: [rows][D] outputs, then [rows] references, then [rows] sums.
__host__ __device__ constexpr int slot_floats(int rows, int D) { return rows * (D + 2); }

// The first row block of request b among all blocks: blocks of different requests are apart.
__host__ __device__ inline int64_t block_base(int64_t row0, int group, int rows, int64_t b) {
  return row0 * group / rows + b;
}
inline int64_t block_count(const WindowParams& p, int rows) { return p.a.total_rows * p.group / rows + p.c.batch; }

// The final scale of a row (1 / sum) and its lse, from its reference and sum; 0 for a row that
// saw nothing.
__device__ __forceinline__ float finish_row(const WindowParams& p, int64_t at, float top, float sum) {
  if (p.a.lse) p.a.lse[at] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
  return sum != 0.f ? 1.f / sum : 0.f;
}

// The same, joined with the window's own part if there is one in own_ml: its factor comes back
// in own.
__device__ __forceinline__ float finish_row(const WindowParams& p, int64_t at, float top, float sum, float& own) {
  own = 0.f;
  if (!p.own_ml) return finish_row(p, at, top, sum);
  const float2 ml = p.own_ml[at];
  const float to = fmaxf(top, ml.x), by = ex2(top - to);
  own = ex2(ml.x - to);
  const float inv = finish_row(p, at, to, fmaf(sum, by, ml.y * own));
  own *= inv;
  return by * inv;
}

// One warp a row of a unit that spans CTAs: the piece of the CTA where it begins (slot
// 2i + 1), then the first pieces (slots 2j) of the CTAs after it up to the one that ends it.
template <int D, int ROWS, int TILE, typename T>
__device__ __forceinline__ void join_row(const WindowParams& p) {
  const int first = blockIdx.x, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int4 d = p.desc[first];
  if (d.x < 0 || row >= d.z) return;
  int pieces = 1;  // the CTAs after this one up to the first that ends the unit, 32 a look
  for (;; pieces += 32) {
    const int i = first + pieces + lane;
    const unsigned ends = __ballot_sync(0xffffffffu, i >= (int)gridDim.x || p.desc[i].w != 0);
    if (ends) {
      pieces += __ffs(ends);
      break;
    }
  }
  auto piece = [&](int i) { return p.part + (int64_t)(i ? 2 * (first + i) : 2 * first + 1) * slot_floats(ROWS, D); };
  float top = kNone;
  for (int i = lane; i < pieces; i += 32) top = fmaxf(top, piece(i)[ROWS * D + row]);
  top = warp_max(top);
  constexpr int PER = D / 32;
  float acc[PER] = {}, sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < pieces; ++i) {
    const float* x = piece(i);
    const float by = ex2(x[ROWS * D + row] - top);
    sum = fmaf(by, x[ROWS * D + ROWS + row], sum);
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
      const float2 v = *reinterpret_cast<const float2*>(x + row * D + lane * PER + e);
      acc[e] = fmaf(by, v.x, acc[e]);
      acc[e + 1] = fmaf(by, v.y, acc[e + 1]);
    }
  }
  Segment s;
  s.r = request<ROWS, TILE>(p, raw_request(p, d.x));
  s.kvh = d.y / s.r.blocks;
  s.block = d.y % s.r.blocks;
  const int64_t at = s.at(p, ROWS, row);
  float own;
  const float by = finish_row(p, at, top, sum, own);  // every lane writes the same lse
#pragma unroll
  for (int e = 0; e < PER; e += 2) {
    float2 o = make_float2(0.f, 0.f);
    if (p.own_ml) o = *reinterpret_cast<const float2*>(p.own_o + at * D + lane * PER + e);
    *reinterpret_cast<uint32_t*>(static_cast<char*>(p.a.out) + (at * D + lane * PER + e) * 2) =
        pack<T>(fmaf(acc[e], by, o.x * own), fmaf(acc[e + 1], by, o.y * own));
  }
}

template <int D, int ROWS, int TILE, typename T>
__global__ void __launch_bounds__(128) k_join(const __grid_constant__ WindowParams p) {
  grid_wait();
  join_row<D, ROWS, TILE, T>(p);
}

// Lets a kernel have this much dynamic shared memory, once on each device.
template <auto kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches with programmatic stream serialisation: the kernel may start before the one
// before it ends, and waits for it (grid_wait) where it needs its results.
template <typename K>
cudaError_t launch_after(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, const WindowParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace tsv
