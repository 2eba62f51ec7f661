// What is left of each request behind a shared prefix, in shared attention (ts_shared.cu): the request's
// own cached tokens and the window's own, joined with the prefix's part of each row.
//
//   k_tail       the units (request, KV head, block of 16 or 32 rows), their tiles of 64 tokens in one line
//                that the CTAs share equally
//   k_tail_join  joins the pieces of units that more than one CTA worked on
//
// These are many short units of few rows: time goes into what a unit has to do one after the other (page
// numbers, their loads, Q, the window's own tokens, the end), so little of it is repeated. A lane looks
// up the page and the scales of a tile, for 32 tiles at once; K and V go to shared memory by asynchronous
// copies, two or three tiles ahead, each of the four warps its own 16 tokens of a tile with no barrier between
// warps; rows' addresses are worked out once. Measured, 100 requests of 382 tokens and one row of 4 heads a KV
// head, 8 KV heads of 128: 40 us (78 MB: 1.9 TB/s; window attention's kernel 81, a tile ahead in registers 54);
// 32 requests of 530 tokens and 64 rows: 64 us (81, 98). With 16 rows a block three CTAs an SM (two: 50 us).
//
// Products run on mma.m16n8k16 with fp16 operands, the precision is that of ts_window.cu: codes are exact in
// fp16, Q rows are scaled by a power of two to below 2, probabilities are rounded to fp16 relative to a
// reference that is set 2^h below the largest score and follows when that is 2^15 above it; V's scale
// is in the exponent. The small ones lose at most 2^-25 each; h goes by the tokens N of a warp, log2 N - 14 and 7
// at least, so that this is below 2^-11 of the row's sum (of 2^30 tokens a warp has 2^28).
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ts_tail.h"
#include "ts_window_own.cuh"

namespace tsv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = kTailTile;
constexpr float kSlack = 15.f, kLeastHead = 7.f;

template <int D, int MT>
struct Shape {
  static constexpr int stages = MT == 1 && D == 128 ? 3 : 4;  // tiles on their way or worked on
  static constexpr int rows = 16 * MT, ks = D / 16, nt = D / 8, ld = D + 4;
  static constexpr int stage = kWarps * 16 * D * 2;  // bytes: K, then V, of each warp
  static constexpr int off_ring = MT * ks * 512;     // Q's fragments before
  // the warps' outputs lie in the place of the ring, which is empty then
  static constexpr int ring = stages * stage > kWarps * rows * ld * 4 ? stages * stage : kWarps * rows * ld * 4;
  static constexpr int off_own = off_ring + ring;
  static constexpr int off_x = off_own + rows * ld * 4;
};
template <int MT>
struct Shared {
  int64_t q[16 * MT];    // a row's place in Q, in bytes
  Sees trees[TS_MAX_WINDOW];
  float2 own[16 * MT];   // references and sums of the window's own tokens
  int32_t at[16 * MT];   // a row's index in [total_rows][heads_q]
  float fac[16 * MT];
  float m[kWarps][16 * MT], l[kWarps][16 * MT];
  float w[kWarps + 2][16 * MT];  // a row's factors: the warps', the window's own part, the prefix's
  int32_t parents[TS_MAX_WINDOW];
};
template <int D, int MT>
constexpr int smem_bytes() { return Shape<D, MT>::off_x + (int)sizeof(Shared<MT>); }

template <int D, int MT, typename T>
__global__ void __launch_bounds__(kThreads, tail_ctas(16 * MT)) k_tail(const __grid_constant__ TailParams p) {
  using S = Shape<D, MT>;
  constexpr int kStages = S::stages, ROWS = S::rows, KS = S::ks, NT = S::nt, LD = S::ld, PIECES = D / 16;
  extern __shared__ __align__(16) unsigned char sm[];
  uint4* s_q = reinterpret_cast<uint4*>(sm);
  float* s_o = reinterpret_cast<float*>(sm + S::off_ring);
  float* s_own = reinterpret_cast<float*>(sm + S::off_own);
  Shared<MT>& x = *reinterpret_cast<Shared<MT>*>(sm + S::off_x);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  unsigned char* ring = sm + S::off_ring + warp * (16 * D * 2);
  int4 desc = make_int4(-1, 0, 0, 0);
  grid_launch();
  grid_wait();
  Line<ROWS, kTile, TailParams> line;
  if (!line_at<ROWS, kTile>(p, p.starts[blockIdx.x], line)) {
    if (tid == 0) p.desc[blockIdx.x] = desc;
    return;
  }
  Segment s;
#pragma unroll 1
  while (line.next(p, s)) {
    const char* kc = static_cast<const char*>(p.c.k) + s.kvh * p.c.k_head_stride;
    const char* vc = static_cast<const char*>(p.c.v) + s.kvh * p.c.v_head_stride;
    const int32_t* table = p.c.page_table + s.b * p.c.ld_table + s.r.skip;
    // the lane's tile of a round of 32: its page (or -1) and scales
    int32_t page = -1;
    float ks = 0.f, vs = 0.f;
    auto look_up = [&](int t) {
      const int tok = t * kTile + warp * 16;
      page = -1;
      if (t < s.t1 && tok < s.r.len) {
        const int32_t id = table[tok >> p.page_shift];
        if (id >= 0 && id < p.c.num_pages) page = id;
      }
      ks = vs = 1.f;
      if (page >= 0) {
        ks = __ldg(p.c.k_scale + (int64_t)page * p.c.heads + s.kvh);
        vs = __ldg(p.c.v_scale + (int64_t)page * p.c.heads + s.kvh);
      }
    };
    // the warp's 16 tokens of tile t; each token's 16-byte pieces at their place XOR what keeps the lanes that
    // read V together from one bank
    auto bring = [&](int t, int round) {
      const int32_t id = __shfl_sync(0xffffffffu, page, (t - round) & 31);
      const int tok = t * kTile + warp * 16;
      unsigned char* to = ring + ((t - s.t0) % kStages) * S::stage;
      if (t < s.t1) {
        const char* k0 = kc + max(id, 0) * p.c.k_page_stride + (int64_t)(tok & (p.c.page_size - 1)) * p.c.k_token_stride;
        const char* v0 = vc + max(id, 0) * p.c.v_page_stride + (int64_t)(tok & (p.c.page_size - 1)) * p.c.v_token_stride;
#pragma unroll
        for (int i = 0; i < PIECES / 2; ++i) {
          const int n = i * 32 + lane, token = n / PIECES, piece = n % PIECES;
          const bool there = id >= 0 && tok + token < s.r.len;
          const int at = token * D + (piece ^ (D == 128 ? token & 6 : token >> 1 & 3)) * 16;
          copy16(to + at, there ? k0 + token * p.c.k_token_stride + piece * 16 : k0, there);
          copy16(to + 16 * D + at, there ? v0 + token * p.c.v_token_stride + piece * 16 : v0, there);
        }
      }
      copies_commit();
    };
    __syncthreads();  // the unit before has left shared memory
    look_up(s.t0 + lane);
    if (tid < ROWS) {
      const int j = s.block * ROWS + tid, t = j / p.group, h = s.kvh * p.group + j - t * p.group;
      x.at[tid] = (int)((s.r.row0 + t) * p.a.heads_q + h);
      x.q[tid] = (s.r.row0 + t) * p.a.q_row_stride + (int64_t)h * p.a.q_head_stride;
    }
    const bool whole = s.whole(), front = s.r.skip > 0 && s.t0 == 0;  // the first piece takes the prefix in too
    const bool own = p.a.k_new && s.t0 == 0;  // the first piece takes the window in
    if (own && p.a.parents)
      for (int i = tid; i < s.r.rows; i += kThreads) x.parents[i] = p.a.parents[s.r.row0 + i];
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) bring(s.t0 + k, s.t0);
    __syncthreads();

    // ---- Q: a warp a row, four rows' loads at a time; scaled by 2^-e, 2^e <= the row's largest < 2^(e+1) (both
    // factors stay normal), straight into the fragments that the products want: K's lane c holds dims 16c .. + 15
    // of each 64, step k takes dims 4k .. 4k + 3 of them. A row with a value that is not finite: NaN, and with
    // it its scores.
#pragma unroll 1
    for (int i0 = warp; i0 < ROWS; i0 += 4 * kWarps) {
      uint2 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kWarps;
        w[k] = make_uint2(0, 0);
        if (i < s.rows && lane < D / 4) w[k] = __ldg(reinterpret_cast<const uint2*>(static_cast<const char*>(p.a.q) + x.q[i]) + lane);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kWarps;
        const uint32_t m = __vmaxu2(w[k].x & 0x7FFF7FFFu, w[k].y & 0x7FFF7FFFu);
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xFFFFu));
        const int e = min(max((int)(__float_as_uint(unpack<T>(top).x) >> 23), 1), 253);
        if (lane == 0) x.fac[i] = not_finite<T>(top) ? NAN : __uint_as_float((uint32_t)e << 23);
        const float inv = __uint_as_float(0x7F000000u - ((uint32_t)e << 23));  // 1 / 2^e
        if (lane < D / 4) {
          const int dim = lane * 4, step = dim / 64 * 4 + dim % 16 / 4, to = dim % 64 / 16;
          const float2 u = unpack<T>(w[k].x), v = unpack<T>(w[k].y);
          uint32_t* frag = reinterpret_cast<uint32_t*>(s_q + ((i >> 4) * KS + step) * 32 + (i & 7) * 4 + to) + (i >> 3 & 1);
          frag[0] = f16x2(u.x * inv, u.y * inv);
          frag[2] = f16x2(v.x * inv, v.y * inv);
        }
      }
    }
    if (front && tid < s.rows * (D / 32)) {  // the prefix's part on its way to L1
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p.pre_o + (int64_t)x.at[tid / (D / 32)] * D + tid % (D / 32) * 32));
      if (tid < s.rows) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.pre_ml + x.at[tid]));
    }
    if (own && p.a.parents)
      for (int i = tid; i < s.r.rows; i += kThreads) x.trees[i] = tree_sees(x.parents, i);
    __syncthreads();
    if (own) {  // each warp a share of the dims
      constexpr int kSlices = kWarps / MT;
      const int i16 = warp / kSlices * 16, j0 = warp % kSlices * (NT / kSlices), j1 = j0 + NT / kSlices;
      const Sees* trees = p.a.parents ? x.trees : nullptr;
      if (i16 < s.rows && own_part<D, ROWS, T>(p, s, i16, j0, j1, trees, s_own, LD, x.own)) {
        __syncwarp();
#pragma unroll 1
        for (int i = i16; i < min(s.rows, i16 + 16); ++i) own_odd<D, ROWS, T>(p, s, i, j0 * 8, j1 * 8, trees, x.own[i].x, s_own + i * LD);
      }
    }

    // ---- the cached tokens
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
        fac[mt][h] = x.fac[mt * 16 + h * 8 + g] * p.scale_log2;
      }
    }
#pragma unroll 1
    for (int t = s.t0; t < s.t1; ++t) {
      const int nth = t - s.t0;
      if (nth > 0 && (nth & 31) == 0) {  // the next round's pages; its tiles come when they are known
        copies_wait<0>();
        look_up(t + lane);
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) bring(t + k, t);
      }
      const int round = s.t0 + (nth & ~31);
      copies_wait<kStages - 2>();
      __syncwarp();
      const int32_t id = __shfl_sync(0xffffffffu, page, nth & 31);
      float k_scale = __shfl_sync(0xffffffffu, ks, nth & 31);
      const float v_scale = scale_of_v(__shfl_sync(0xffffffffu, vs, nth & 31), k_scale);
      const unsigned char* from = ring + (nth % kStages) * S::stage;
      const int tok = t * kTile + warp * 16;
      if (id >= 0) {
        float y[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[mt][n][e] = 0.f;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          uint4 kw[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int token = n * 8 + g, piece = half * 4 + c;
            kw[n] = *reinterpret_cast<const uint4*>(from + token * D + (piece ^ (D == 128 ? token & 6 : token >> 1 & 3)) * 16);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t kb[2][2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t w = k == 0 ? kw[n].x : k == 1 ? kw[n].y : k == 2 ? kw[n].z : kw[n].w;
              kb[n][0] = e4m3x2_to_f16x2((uint16_t)w);
              kb[n][1] = e4m3x2_to_f16x2((uint16_t)(w >> 16));
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint4 q4 = s_q[(mt * KS + half * 4 + k) * 32 + lane];
              const uint32_t qa[4] = {q4.x, q4.y, q4.z, q4.w};
              mma16816<__half>(y[mt][0], qa, kb[0][0], kb[0][1]);
              mma16816<__half>(y[mt][1], qa, kb[1][0], kb[1][1]);
            }
          }
        }
        const float lv = __log2f(v_scale), inv_v = 1.f / v_scale;
        bool move = false;
        float top[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float z = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& v = y[mt][n][2 * h + e];
                v = tok + n * 8 + 2 * c + e < s.r.len ? fmaf(v, fac[mt][h] * k_scale, lv) : -INFINITY;
                z = fmaxf(z, v);
              }
            z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 1));
            z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 2));
            top[mt][h] = z;
            move |= z > m[mt][h] + kSlack;
          }
        if (__any_sync(0xffffffffu, move)) {
          const float head = fmaxf((float)(22 - __clz(s.t1 - s.t0)), kLeastHead);  // of 16 tokens a tile
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // only where needed: a row's result must not depend on its neighbours'
              const float to = top[mt][h] > m[mt][h] + kSlack ? top[mt][h] - head : m[mt][h];
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
        uint32_t pa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float e0 = ex2(y[mt][n][2 * h] - m[mt][h]), e1 = ex2(y[mt][n][2 * h + 1] - m[mt][h]);
              sum += e0 + e1;
              pa[mt][2 * n + h] = f16x2(e0, e1);
            }
            l[mt][h] = fmaf(sum, inv_v, l[mt][h]);
          }
        // V: lane (g, c) holds dims g * D/8 .. of tokens 2c, 2c + 1, 2c + 8, 2c + 9
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = 2 * c + (i & 1) + (i >> 1) * 8;
          const unsigned char* row = from + 16 * D + token * D;
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + (g ^ (token & 6)) * 16);
            vw[i][0] = w.x, vw[i][1] = w.y, vw[i][2] = w.z, vw[i][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(row + ((g >> 1) ^ (token >> 1 & 3)) * 16 + (g & 1) * 8);
            vw[i][0] = w.x, vw[i][1] = w.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // dims 4w + 2half and the next: their bytes of tokens (2c, 2c+1) and (2c+8, 2c+9)
            const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], half ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(vw[2][w], vw[3][w], half ? 0x7362 : 0x5140);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)(lo >> (16 * e)));
              const uint32_t b1 = e4m3x2_to_f16x2((uint16_t)(hi >> (16 * e)));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<__half>(o[mt][w * 4 + half * 2 + e], pa[mt], b0, b1);
            }
          }
      }
      __syncwarp();
      if (((nth + kStages - 1) & ~31) == (nth & ~31)) bring(t + kStages - 1, round);
      else copies_commit();  // of the next round: brought there
    }
    copies_wait<0>();

    // ---- the warps meet, in the place of the ring
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[mt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int row = mt * 16 + h * 8 + g;
        if (c == 0) {
          x.m[warp][row] = m[mt][h];
          x.l[warp][row] = sum;
        }
        float* at = s_o + (warp * ROWS + row) * LD;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            *reinterpret_cast<float4*>(at + (2 * c + e) * (D / 8) + j) =
                make_float4(o[mt][j][2 * h + e], o[mt][j + 1][2 * h + e], o[mt][j + 2][2 * h + e], o[mt][j + 3][2 * h + e]);
      }
    __syncthreads();
    float* part = p.part + (int64_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * slot_floats(ROWS, D);
    if (tid < s.rows) {
      const float2 none = make_float2(kNone, 0.f), mine = own ? x.own[tid] : none, pre = front ? p.pre_ml[x.at[tid]] : none;
      float top = fmaxf(mine.x, pre.x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, x.m[w][tid]);
      float f[kWarps + 2] = {}, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = ex2(x.m[w][tid] - top);
        sum = fmaf(f[w], x.l[w][tid], sum);
      }
      f[kWarps] = ex2(mine.x - top);
      f[kWarps + 1] = ex2(pre.x - top);
      sum = fmaf(f[kWarps], mine.y, sum);
      sum = fmaf(f[kWarps + 1], pre.y, sum);
      float by = 1.f;
      if (whole) by = finish_row(p, x.at[tid], top, sum);
      else part[ROWS * D + tid] = top, part[ROWS * D + ROWS + tid] = sum;
#pragma unroll
      for (int w = 0; w < kWarps + 2; ++w) x.w[w][tid] = f[w] * by;
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < s.rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      const int64_t at = x.at[row];
      float4 pre = make_float4(0.f, 0.f, 0.f, 0.f);
      if (front) pre = *reinterpret_cast<const float4*>(p.pre_o + at * D + d);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float by, const float4& v) {
        acc.x = fmaf(by, v.x, acc.x), acc.y = fmaf(by, v.y, acc.y);
        acc.z = fmaf(by, v.z, acc.z), acc.w = fmaf(by, v.w, acc.w);
      };
#pragma unroll
      for (int w = 0; w < kWarps; ++w) add(x.w[w][row], *reinterpret_cast<const float4*>(s_o + (w * ROWS + row) * LD + d));
      if (own) add(x.w[kWarps][row], *reinterpret_cast<const float4*>(s_own + row * LD + d));
      if (front) add(x.w[kWarps + 1][row], pre);  // 0 times NaN is NaN
      if (whole)
        *reinterpret_cast<uint2*>(static_cast<char*>(p.a.out) + (at * D + d) * 2) = make_uint2(pack<T>(acc.x, acc.y), pack<T>(acc.z, acc.w));
      else
        *reinterpret_cast<float4*>(part + row * D + d) = acc;
    }
    if (!whole) {
      if (s.t0 == 0) {
        desc.x = s.b;
        desc.y = s.kvh * s.r.blocks + s.block;
        desc.z = s.rows;
      } else {
        desc.w = s.t1 == s.r.tiles ? 1 : 0;
      }
    }
  }
  if (tid == 0) p.desc[blockIdx.x] = desc;
}

// join_row, of the rows of these units.
template <int D, int MT, typename T>
__global__ void __launch_bounds__(128) k_tail_join(const __grid_constant__ TailParams p) {
  grid_wait();
  join_row<D, 16 * MT, kTile, T>(p);
}

template <int D, int MT, typename T>
cudaError_t launch(const TailParams& p, int sms, cudaStream_t s) {
  constexpr int bytes = smem_bytes<D, MT>();
  static_assert(bytes <= 227 * 1024 / tail_ctas(16 * MT) - 1024, "CTAs an SM");
  cudaError_t e = allow_smem<k_tail<D, MT, T>>(bytes);
  if (e != cudaSuccess) return e;
  const int grid = sms * tail_ctas(16 * MT);
  if ((e = launch_after(k_tail<D, MT, T>, dim3(grid), kThreads, bytes, s, p)) != cudaSuccess) return e;
  if ((int64_t)p.c.max_pages * p.c.page_size <= kTile) return cudaSuccess;  // units of one tile are never split
  return launch_after(k_tail_join<D, MT, T>, dim3(grid, 4 * MT), 128, 0, s, p);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t lay_out(TailParams& p, void* ws, int sms) {
  const size_t ctas = (size_t)sms * tail_ctas(tail_rows(p));
  size_t off = 0;
  auto take = [&](auto*& at, size_t n) {
    at = reinterpret_cast<std::remove_reference_t<decltype(at)>>(static_cast<char*>(ws) + off);
    off += up256(n * sizeof(*at));
  };
  take(p.desc, ctas);
  take(p.part, 2 * ctas * slot_floats(tail_rows(p), p.c.head_dim));
  return off;
}

}  // namespace

// By the average window: blocks of 32 rows read K and V half as often.
int tail_rows(const WindowParams& p) { return (p.a.total_rows * p.group + p.c.batch - 1) / p.c.batch <= 16 ? 16 : 32; }

size_t tail_workspace(int64_t batch, int64_t total_rows, int heads_q, int heads, int head_dim, int sms) {
  TailParams p{};
  p.c.batch = batch;
  p.c.head_dim = head_dim;
  p.a.total_rows = total_rows;
  p.group = heads_q / heads;
  return lay_out(p, nullptr, sms);
}

TailParams tail_params(const ts_kv_cache& c, const ts_attn_args& a, void* ws, int sms) {
  TailParams p{};
  p.c = c;
  p.a = a;
  p.page_shift = __builtin_ctz((unsigned)c.page_size);
  p.group = a.heads_q / c.heads;
  p.scale_log2 = a.sm_scale * kLog2e;
  lay_out(p, ws, sms);
  return p;
}

cudaError_t launch_tail(const TailParams& p, int sms, cudaStream_t s) {
  const bool bf16 = p.a.dtype == TS_BF16, few = tail_rows(p) == 16;
  if (p.c.head_dim == 64) {
    if (few) return bf16 ? launch<64, 1, __nv_bfloat16>(p, sms, s) : launch<64, 1, __half>(p, sms, s);
    return bf16 ? launch<64, 2, __nv_bfloat16>(p, sms, s) : launch<64, 2, __half>(p, sms, s);
  }
  if (few) return bf16 ? launch<128, 1, __nv_bfloat16>(p, sms, s) : launch<128, 1, __half>(p, sms, s);
  return bf16 ? launch<128, 2, __nv_bfloat16>(p, sms, s) : launch<128, 2, __half>(p, sms, s);
}

}  // namespace tsv
