// Attention of drafted windows over the 8-bit paged KV cache and over themselves.
//
//   k_window   the (request, KV head, row block) units cut into tiles of 64 tokens; the tiles
//              of the whole call lie in one line that the CTAs share equally
//   k_join     joins the pieces of units that more than one CTA worked on
//
// A unit's rows are the window rows of the query heads that share a KV head. Each of a CTA's
// four warps takes 16 tokens of a tile (they lie in one block, so K and V have one scale each)
// and keeps its own running maximum, sum and output; the warps meet once a unit.
//
// Products run on mma.m16n8k16 with fp16 operands: an e4m3 code is exact in fp16. K codes and
// V codes come from global memory straight into the fragments that the products want: a quad's
// lane c holds 16 dims of its token for K, and of four tokens for V, and the order in which the
// products walk the dims and tokens is chosen to fit. Q rows are scaled by a power of two to
// below 2, where bf16 values are exact in fp16 down to 2^-14 of the row's largest and off by at
// most 2^-25 of it below. Probabilities are rounded to fp16 (2^-11 relative), relative to a
// reference m that is at most 2^8 below the running maximum (no rescaling in between).
//
// V's scale s enters through the exponent: the products take p' = 2^(x + log2 s - m), so the
// output needs no scale, whatever the blocks' scales; the sum takes p' / s.
#include <stdint.h>

#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/ts_verify.h"
#include "ts_common.cuh"
#include "ts_internal.h"
#include "ts_kv.cuh"

namespace tsv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16 * kWarps;
constexpr int window_ctas_per_sm(int) { return 2; }
constexpr int kMinTiles = 4;      // least tiles a CTA takes: pieces of 256 tokens or more
constexpr float kNone = -1e30f;   // the reference before any token
constexpr float kSlack = 8.f;

struct Params {
  ts_kv_cache c;
  ts_attn_args a;
  int32_t page_shift;
  int32_t group;
  float scale_log2;
  float* part;      // [2 * CTAs][rows][D + 2] pieces: output, reference, sum
  int4* desc;       // [CTAs] {tail unit's request, its head and row block, rows, 0 | 1: the
                    // CTA's first piece ends its unit}
};

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
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t half_word);  // one 16-bit value
template <>
__device__ __forceinline__ bool not_finite<__half>(uint32_t w) { return (w & 0x7C00u) == 0x7C00u; }
template <>
__device__ __forceinline__ bool not_finite<__nv_bfloat16>(uint32_t w) { return (w & 0x7F80u) == 0x7F80u; }

// What the line of tiles needs of a request.
struct Req {
  int64_t row0;
  int32_t rows;    // window rows (0: skipped)
  int32_t len;     // cached tokens
  int32_t blocks;  // row blocks
  int32_t ctx;     // tiles of cached tokens
  int32_t tiles;   // all tiles of a unit (>= 1)
  __device__ __forceinline__ int64_t weight(int heads) const {
    return rows ? (int64_t)heads * blocks * tiles : 0;
  }
};

template <int ROWS>
__device__ __forceinline__ Req request(const Params& p, int64_t b) {
  Req r;
  if (p.a.qo_indptr) {
    r.row0 = p.a.qo_indptr[b];
    const int64_t r1 = p.a.qo_indptr[b + 1];
    r.rows = r.row0 >= 0 && r1 <= p.a.total_rows && r1 > r.row0 && r1 - r.row0 <= TS_MAX_WINDOW ? (int)(r1 - r.row0) : 0;
  } else {
    r.rows = (int)(p.a.total_rows / p.c.batch);
    r.row0 = b * r.rows;
  }
  const int64_t cap = (int64_t)p.c.max_pages << p.page_shift;
  r.len = (int32_t)min((int64_t)max(p.c.seq_lens[b], 0), cap);
  r.blocks = (r.rows * p.group + ROWS - 1) / ROWS;
  r.ctx = (int)(((int64_t)r.len + kTile - 1) / kTile);
  r.tiles = r.ctx + (p.a.k_new ? (r.rows + kTile - 1) / kTile : 0);
  r.tiles = max(r.tiles, 1);
  return r;
}

// A piece's slot: [rows][D] outputs, then [rows] references, then [rows] sums.
__host__ __device__ constexpr int slot_floats(int rows, int D) { return rows * (D + 2); }

template <int D, int MT, typename T>
__global__ void __launch_bounds__(kThreads) k_window(const __grid_constant__ Params p) {
  constexpr int ROWS = 16 * MT;
  constexpr int KS = D / 16;        // k16 steps over the dims
  constexpr int NT = D / 8;         // n8 tiles over the dims
  constexpr int VW = D / 32;        // words of a token's V codes a lane holds
  extern __shared__ __align__(16) unsigned char smem[];
  // Q fragments [MT][KS][32 lanes] and the factors of their rows; then, for the join of the
  // warps, [kWarps][ROWS][D + 4] outputs with their references and sums
  uint4* s_q = reinterpret_cast<uint4*>(smem);
  float* s_fac = reinterpret_cast<float*>(s_q + MT * KS * 32);
  float* s_o = s_fac + ROWS;
  float* s_m = s_o + kWarps * ROWS * (D + 4);
  float* s_l = s_m + kWarps * ROWS;
  __shared__ uint64_t s_sees[TS_MAX_WINDOW][2];  // bit j: the row sees window token j
  __shared__ int64_t s_scan[kWarps], s_start;
  __shared__ int32_t s_b;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int64_t cta = blockIdx.x, ctas = gridDim.x;

  // ---- this CTA's share of the line
  int64_t mine = 0;
  const int64_t each = (p.c.batch + kThreads - 1) / kThreads;
  const int64_t b_lo = min(p.c.batch, tid * each), b_hi = min(p.c.batch, b_lo + each);
  for (int64_t b = b_lo; b < b_hi; ++b) mine += request<ROWS>(p, b).weight(p.c.heads);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) s_scan[warp] = upto;
  if (tid == 0) s_b = -1;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_scan[w];
    all += s_scan[w];
  }
  const int64_t share = max((all + ctas - 1) / ctas, (int64_t)kMinTiles);
  const int64_t begin = min(all, cta * share), end = min(all, begin + share);
  int4 desc = make_int4(-1, 0, 0, 0);
  if (begin < end && upto - mine <= begin && begin < upto) {  // one thread
    int64_t at = upto - mine;
    for (int64_t b = b_lo; b < b_hi; ++b) {
      const int64_t w = request<ROWS>(p, b).weight(p.c.heads);
      if (begin < at + w) {
        s_b = (int32_t)b;
        s_start = begin - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  if (begin >= end) {
    if (tid == 0) p.desc[cta] = desc;
    return;
  }
  int64_t b = s_b;
  Req r = request<ROWS>(p, b);
  int32_t unit = (int32_t)(s_start / r.tiles), tile = (int32_t)(s_start % r.tiles);
  int64_t left = end - begin;

  while (left > 0) {
    while (r.rows == 0 || unit >= p.c.heads * r.blocks) {
      r = request<ROWS>(p, ++b);
      unit = 0;
    }
    const int kvh = unit / r.blocks, block = unit % r.blocks;
    const int t0 = tile, t1 = (int)min((int64_t)r.tiles, t0 + left);
    const int rows = min(ROWS, r.rows * p.group - block * ROWS);  // of this block
    const bool window = p.a.k_new != nullptr && t1 > r.ctx;

    // ---- Q: row i of the unit is window row (block*ROWS + i) / group of head kvh*group +
    // the remainder. Each row's factor, then the fragments.
    auto q_row = [&](int i) -> const char* {
      const int j = block * ROWS + i;
      return static_cast<const char*>(p.a.q) + (r.row0 + j / p.group) * p.a.q_row_stride +
             (int64_t)(kvh * p.group + j % p.group) * p.a.q_head_stride;
    };
    __syncthreads();  // the previous unit's reads of shared memory are done
    for (int i = warp; i < ROWS; i += kWarps) {
      float top = 0.f;
      if (i < rows) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(q_row(i));
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const float2 f = unpack<T>(q[lane + 32 * k]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = warp_max(top);
      // 2^e <= top < 2^(e+1); the row is divided by 2^e
      const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 227);
      if (lane == 0) s_fac[i] = __uint_as_float((uint32_t)e << 23);
    }
    __syncthreads();
    for (int i = tid; i < MT * KS * 32; i += kThreads) {
      const int l = i & 31, ks = i / 32 % KS, mt = i / 32 / KS, qc = l & 3, qg = l >> 2;
      // K's lane qc holds dims 64h + 16qc .. + 15; step 4h + k takes dims 4k .. 4k + 3 of them
      const int dim = (ks / 4) * 64 + qc * 16 + (ks % 4) * 4;
      uint32_t w[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = mt * 16 + half * 8 + qg;
        uint2 x = make_uint2(0, 0);
        float inv = 1.f;
        if (row < rows) {
          x = *reinterpret_cast<const uint2*>(q_row(row) + dim * 2);
          inv = __uint_as_float(0x7F000000u - __float_as_uint(s_fac[row]));  // 1 / 2^e
        }
        const float2 u = unpack<T>(x.x), v = unpack<T>(x.y);
        w[half] = f16x2(u.x * inv, u.y * inv);
        w[2 + half] = f16x2(v.x * inv, v.y * inv);
      }
      s_q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (window) {
      // what each window row sees; ancestors lie before a row, so the walks end
      for (int i = tid; i < r.rows; i += kThreads) {
        uint64_t lo = 0, hi = 0;
        if (p.a.parents) {
          int at = i;
          while (at >= 0) {
            if (at < 64) lo |= 1ull << at;
            else hi |= 1ull << (at - 64);
            const int up = p.a.parents[r.row0 + at];
            at = up < at ? up : -1;
          }
        } else {
          lo = i >= 63 ? ~0ull : (2ull << i) - 1;
          hi = i >= 64 ? (2ull << (i - 64)) - 1 : 0;
        }
        s_sees[i][0] = lo;
        s_sees[i][1] = hi;
      }
    }
    __syncthreads();

    float o[MT][NT][4], m[MT][2], l[MT][2], fac[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[mt][h] = kNone;
        l[mt][h] = 0.f;
        fac[mt][h] = s_fac[mt * 16 + h * 8 + g] * p.scale_log2;
      }
    }

    // x: scores of 16 tokens in log2 units plus log2 of V's scale (-inf: not seen). Turns
    // them into p' and moves the reference, the outputs and sums with it where needed.
    auto softmax = [&](float (&x)[MT][2][4], float inv_v) {
      bool move = false;
      float top[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t = fmaxf(fmaxf(x[mt][0][2 * h], x[mt][0][2 * h + 1]), fmaxf(x[mt][1][2 * h], x[mt][1][2 * h + 1]));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          top[mt][h] = t;
          move |= t > m[mt][h] + kSlack;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // only where needed: a row's result must not depend on its neighbours'
            const float to = top[mt][h] > m[mt][h] + kSlack ? top[mt][h] : m[mt][h];
            const float by = ex2(m[mt][h] - to);
            m[mt][h] = to;
            l[mt][h] *= by;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              o[mt][j][2 * h] *= by;
              o[mt][j][2 * h + 1] *= by;
            }
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& y = x[mt][n][2 * h + e];
              y = ex2(y - m[mt][h]);
              sum += y;
            }
          l[mt][h] = fmaf(sum, inv_v, l[mt][h]);
        }
    };

    // ---- cached tokens
    const char* kc = static_cast<const char*>(p.c.k) + kvh * p.c.k_head_stride;
    const char* vc = static_cast<const char*>(p.c.v) + kvh * p.c.v_head_stride;
    const int32_t* table = p.c.page_table + b * p.c.ld_table;
    const int ctx_end = min(t1, r.ctx);
    struct Loaded {
      uint4 k[2][D / 64];
      uint32_t v[4][VW];
      float ks, vs;
    };
    auto page_of = [&](int t) -> int32_t {  // page of this warp's tokens of tile t, or -1
      const int64_t tok = (int64_t)t * kTile + warp * 16;
      if (t >= ctx_end || tok >= r.len) return -1;
      const int32_t id = table[tok >> p.page_shift];
      return id >= 0 && id < p.c.num_pages ? id : -1;
    };
    auto fetch = [&](int t, int32_t page, Loaded& x) {
      const int tok = t * kTile + warp * 16;
      const int slot = tok & (p.c.page_size - 1);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const bool ok = page >= 0 && tok + n * 8 + g < r.len;
        const char* at = kc + page * p.c.k_page_stride + (int64_t)(slot + n * 8 + g) * p.c.k_token_stride + c * 16;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) x.k[n][h] = ok ? ldg_stream(at + h * 64) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tt = 2 * c + (i & 1) + (i >> 1) * 8;
        const bool ok = page >= 0 && tok + tt < r.len;
        const char* at = vc + page * p.c.v_page_stride + (int64_t)(slot + tt) * p.c.v_token_stride + g * (D / 8);
        if constexpr (VW == 4) {
          const uint4 w = ok ? ldg_stream(at) : make_uint4(0, 0, 0, 0);
          x.v[i][0] = w.x, x.v[i][1] = w.y, x.v[i][2] = w.z, x.v[i][3] = w.w;
        } else {
          const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0, 0);
          x.v[i][0] = w.x, x.v[i][1] = w.y;
        }
      }
      x.ks = x.vs = 1.f;
      if (page >= 0) {
        x.ks = __ldg(p.c.k_scale + (int64_t)page * p.c.heads + kvh);
        x.vs = fmaxf(__ldg(p.c.v_scale + (int64_t)page * p.c.heads + kvh), 0x1p-100f);
      }
    };
    Loaded next;
    int32_t page = page_of(t0), page2 = page_of(t0 + 1);
    if (t0 < ctx_end) fetch(t0, page, next);
    for (int t = t0; t < ctx_end; ++t) {
      Loaded now = next;
      const int32_t page_now = page;
      page = page2;
      page2 = page_of(t + 2);
      if (t + 1 < ctx_end) fetch(t + 1, page, next);
      if (page_now < 0) continue;
      const int tok = t * kTile + warp * 16;
      float x[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[mt][n][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t kb[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint4 w4 = now.k[n][ks / 4];
          const uint32_t w = ks % 4 == 0 ? w4.x : ks % 4 == 1 ? w4.y : ks % 4 == 2 ? w4.z : w4.w;
          kb[n][0] = e4m3x2_to_f16x2((uint16_t)w);
          kb[n][1] = e4m3x2_to_f16x2((uint16_t)(w >> 16));
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 q4 = s_q[(mt * KS + ks) * 32 + lane];
          const uint32_t qa[4] = {q4.x, q4.y, q4.z, q4.w};
          mma16816<__half>(x[mt][0], qa, kb[0][0], kb[0][1]);
          mma16816<__half>(x[mt][1], qa, kb[1][0], kb[1][1]);
        }
      }
      const float lv = __log2f(now.vs), inv_v = 1.f / now.vs;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool seen = tok + n * 8 + 2 * c + (e & 1) < r.len;
            x[mt][n][e] = seen ? fmaf(x[mt][n][e], fac[mt][e >> 1] * now.ks, lv) : -INFINITY;
          }
      softmax(x, inv_v);
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        pa[mt][0] = f16x2(x[mt][0][0], x[mt][0][1]);
        pa[mt][1] = f16x2(x[mt][0][2], x[mt][0][3]);
        pa[mt][2] = f16x2(x[mt][1][0], x[mt][1][1]);
        pa[mt][3] = f16x2(x[mt][1][2], x[mt][1][3]);
      }
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // dims 4w + 2half and the next: their bytes of tokens (2c, 2c+1) and (2c+8, 2c+9)
          const uint32_t lo = __byte_perm(now.v[0][w], now.v[1][w], half ? 0x7362 : 0x5140);
          const uint32_t hi = __byte_perm(now.v[2][w], now.v[3][w], half ? 0x7362 : 0x5140);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)(lo >> (16 * e)));
            const uint32_t b1 = e4m3x2_to_f16x2((uint16_t)(hi >> (16 * e)));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816<__half>(o[mt][w * 4 + half * 2 + e], pa[mt], b0, b1);
          }
        }
    }

    // ---- the window's own tokens, in their own type; probabilities in two parts of it
    for (int t = max(t0, r.ctx); window && t < t1; ++t) {
      const int tok = (t - r.ctx) * kTile + warp * 16;
      if (tok >= r.rows) continue;
      const char* kn = static_cast<const char*>(p.a.k_new) + (r.row0 + tok) * p.a.k_row_stride + kvh * p.a.k_head_stride;
      const char* vn = static_cast<const char*>(p.a.v_new) + (r.row0 + tok) * p.a.v_row_stride + kvh * p.a.v_head_stride;
      float x[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[mt][n][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int dim = (ks / 4) * 64 + c * 16 + (ks % 4) * 4;
        uint2 kb[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          kb[n] = make_uint2(0, 0);
          if (tok + n * 8 + g < r.rows)
            kb[n] = *reinterpret_cast<const uint2*>(kn + (n * 8 + g) * p.a.k_row_stride + dim * 2);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t qa[4];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = mt * 16 + half * 8 + g;
            uint2 w = make_uint2(0, 0);
            if (row < rows) w = *reinterpret_cast<const uint2*>(q_row(row) + dim * 2);
            qa[half] = w.x;
            qa[2 + half] = w.y;
          }
          mma16816<T>(x[mt][0], qa, kb[0].x, kb[0].y);
          mma16816<T>(x[mt][1], qa, kb[1].x, kb[1].y);
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = mt * 16 + (e >> 1) * 8 + g, j = tok + n * 8 + 2 * c + (e & 1);
            const bool seen = i < rows && j < r.rows && (s_sees[(block * ROWS + i) / p.group][j >> 6] >> (j & 63) & 1);
            x[mt][n][e] = seen ? x[mt][n][e] * p.scale_log2 : -INFINITY;
          }
      softmax(x, 1.f);
      uint32_t pa[MT][4], pb[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float u = x[mt][n][2 * h], v = x[mt][n][2 * h + 1];
            const uint32_t w = pack<T>(u, v);
            const float2 f = unpack<T>(w);
            pa[mt][n * 2 + h] = w;
            pb[mt][n * 2 + h] = pack<T>(u - f.x, v - f.y);
          }
      // a value that is not finite must reach only the rows that see it: 0 in the product,
      // added row by row below
      bool odd = false;
      auto v_at = [&](int i, int dim) -> uint32_t {
        if (tok + i >= r.rows) return 0;
        return *reinterpret_cast<const uint16_t*>(vn + i * p.a.v_row_stride + dim * 2);
      };
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int dim = g * (D / 8) + j;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = v_at(2 * c + (i & 1) + (i >> 1) * 8, dim);
          if (not_finite<T>(w[i])) {
            odd = true;
            w[i] = 0;
          }
        }
        const uint32_t b0 = w[0] | (w[1] << 16), b1 = w[2] | (w[3] << 16);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816<T>(o[mt][j], pa[mt], b0, b1);
          mma16816<T>(o[mt][j], pb[mt], b0, b1);
        }
      }
      if (__any_sync(0xffffffffu, odd)) {
        for (int i = 0; i < 16; ++i) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // p of (row h*8 + g, token i) lies in lane i % 8 / 2 of the quad
              const int from = (lane & ~3) | ((i & 7) >> 1);
              const float p0 = __shfl_sync(0xffffffffu, i < 8 ? x[mt][0][2 * h] : x[mt][1][2 * h], from);
              const float p1 = __shfl_sync(0xffffffffu, i < 8 ? x[mt][0][2 * h + 1] : x[mt][1][2 * h + 1], from);
              const int row = mt * 16 + h * 8 + g;
              if (row >= rows || tok + i >= r.rows) continue;
              const int j = tok + i;
              if (!(s_sees[(block * ROWS + row) / p.group][j >> 6] >> (j & 63) & 1)) continue;
#pragma unroll
              for (int d = 0; d < NT; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t w = v_at(i, (2 * c + e) * (D / 8) + d);
                  if (not_finite<T>(w)) o[mt][d][2 * h + e] += (i & 1 ? p1 : p0) * unpack<T>(w).x;
                }
            }
        }
      }
    }

    // ---- the warps meet: lane (g, c) holds dims (2c + e) * D/8 + j of rows g and g + 8
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[mt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int row = mt * 16 + h * 8 + g;
        if (c == 0) {
          s_m[warp * ROWS + row] = m[mt][h];
          s_l[warp * ROWS + row] = sum;
        }
        float* at = s_o + (warp * ROWS + row) * (D + 4);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            *reinterpret_cast<float4*>(at + (2 * c + e) * (D / 8) + j) =
                make_float4(o[mt][j][2 * h + e], o[mt][j + 1][2 * h + e], o[mt][j + 2][2 * h + e], o[mt][j + 3][2 * h + e]);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == r.tiles;
    const int slot = (int)(2 * cta) + (t0 == 0 ? 1 : 0);
    float* part = p.part + (int64_t)slot * slot_floats(ROWS, D);
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float top = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * ROWS + row]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float by = ex2(s_m[w * ROWS + row] - top);
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * ROWS + row) * (D + 4) + d);
        sum = fmaf(by, s_l[w * ROWS + row], sum);
        acc.x = fmaf(by, v.x, acc.x), acc.y = fmaf(by, v.y, acc.y);
        acc.z = fmaf(by, v.z, acc.z), acc.w = fmaf(by, v.w, acc.w);
      }
      if (whole) {
        const int j = block * ROWS + row;
        const int64_t at = (r.row0 + j / p.group) * p.a.heads_q + kvh * p.group + j % p.group;
        const float inv = sum != 0.f ? 1.f / sum : 0.f;  // a row that saw nothing: 0
        const uint2 w = make_uint2(pack<T>(acc.x * inv, acc.y * inv), pack<T>(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(static_cast<char*>(p.a.out) + (at * D + d) * 2) = w;
        if (d == 0 && p.a.lse) p.a.lse[at] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(part + row * D + d) = acc;
        if (d == 0) {
          part[ROWS * D + row] = top;
          part[ROWS * D + ROWS + row] = sum;
        }
      }
    }
    if (!whole) {
      if (t0 == 0) {
        desc.x = (int)b;
        desc.y = unit;
        desc.z = rows;
      } else {
        desc.w = t1 == r.tiles ? 1 : 0;
      }
    }
    left -= t1 - t0;
    tile = 0;
    ++unit;
  }
  if (tid == 0) p.desc[cta] = desc;
}

// One warp a row of a unit that spans CTAs: the piece of the CTA where it begins (slot
// 2i + 1), then the first pieces (slots 2j) of the CTAs after it up to the one that ends it.
template <int D, int ROWS, typename T>
__global__ void __launch_bounds__(kThreads) k_join(const __grid_constant__ Params p) {
  const int first = blockIdx.x, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int4 d = p.desc[first];
  if (d.x < 0 || row >= d.z) return;
  int pieces = 1;
  while (first + pieces < (int)gridDim.x && p.desc[first + pieces].w == 0) ++pieces;
  ++pieces;
  auto piece = [&](int i) { return p.part + (int64_t)(i ? 2 * (first + i) : 2 * first + 1) * slot_floats(ROWS, D); };
  float top = kNone;
  for (int i = lane; i < pieces; i += 32) top = fmaxf(top, piece(i)[ROWS * D + row]);
  top = warp_max(top);
  constexpr int PER = D / 32;
  float acc[PER] = {}, sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const float* x = piece(i);
    const float by = ex2(x[ROWS * D + row] - top);
    sum = fmaf(by, x[ROWS * D + ROWS + row], sum);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(by, x[row * D + lane * PER + e], acc[e]);
  }
  const Req r = request<ROWS>(p, d.x);
  const int kvh = d.y / r.blocks, j = d.y % r.blocks * ROWS + row;
  const int64_t at = (r.row0 + j / p.group) * p.a.heads_q + kvh * p.group + j % p.group;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(static_cast<char*>(p.a.out) + (at * D + lane * PER + e) * 2) = pack<T>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.a.lse) p.a.lse[at] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

constexpr int smem_bytes(int D, int rows) {
  return rows / 16 * (D / 16) * 32 * 16 + rows * 4 + kWarps * rows * (D + 4) * 4 + kWarps * rows * 8;
}

template <int D, int MT, typename T>
cudaError_t launch(const Params& p, int sms, cudaStream_t s) {
  constexpr int ROWS = 16 * MT, bytes = smem_bytes(D, ROWS);
  cudaError_t e = cudaFuncSetAttribute(k_window<D, MT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int grid = sms * window_ctas_per_sm(MT);
  k_window<D, MT, T><<<grid, kThreads, bytes, s>>>(p);
  k_join<D, ROWS, T><<<dim3(grid, ROWS / kWarps), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int MT>
cudaError_t launch_mt(const Params& p, int sms, cudaStream_t s) {
  const bool bf16 = p.a.dtype == TS_BF16;
  if (p.c.head_dim == 128)
    return bf16 ? launch<128, MT, __nv_bfloat16>(p, sms, s) : launch<128, MT, __half>(p, sms, s);
  return bf16 ? launch<64, MT, __nv_bfloat16>(p, sms, s) : launch<64, MT, __half>(p, sms, s);
}

}  // namespace

size_t window_workspace(int head_dim, int sms) {
  size_t most = 0;
  for (int mt = 1; mt <= 2; ++mt) {
    const size_t ctas = (size_t)sms * window_ctas_per_sm(mt);
    const size_t n = ctas * sizeof(int4) + 2 * ctas * slot_floats(16 * mt, head_dim) * sizeof(float);
    most = std::max(most, n);
  }
  return (most + 255) & ~(size_t)255;
}

cudaError_t launch_window(const ts_kv_cache& c, const ts_attn_args& a, void* ws, int sms, cudaStream_t s) {
  Params p{};
  p.c = c;
  p.a = a;
  p.page_shift = __builtin_ctz((unsigned)c.page_size);
  p.group = a.heads_q / c.heads;
  p.scale_log2 = a.sm_scale * kLog2e;
  // blocks of 16 rows where the average window has no more, else of 32: the cached codes are
  // converted and read once a block
  const int64_t rows = (a.total_rows * p.group + c.batch - 1) / c.batch;
  const int mt = rows <= 16 ? 1 : 2;
  p.desc = static_cast<int4*>(ws);
  p.part = reinterpret_cast<float*>(p.desc + (size_t)sms * window_ctas_per_sm(mt));
  return mt == 1 ? launch_mt<1>(p, sms, s) : launch_mt<2>(p, sms, s);
}

}  // namespace tsv
