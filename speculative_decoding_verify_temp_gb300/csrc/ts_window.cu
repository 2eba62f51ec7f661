// Attention of drafted windows over the 8-bit paged KV cache and over themselves: the workspace,
// and the kernels for head_dim 64 (128: ts_window_tc.cu).
//
//   k_window_own  the window's own tokens, for every row
//   k_window      the cached tokens: the (request, KV head, row block) units cut into tiles of 64
//                 tokens; the tiles of the whole call lie in one line that the CTAs share equally
//   k_join        joins the pieces of units that more than one CTA worked on
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
// reference m that is set 2^7 below the largest score so far and follows when that is 2^15 above it (no
// rescaling in between): fp16 holds 65504, and at the other end the small ones lose at most
// 2^-25 each, 2^-11 of the row's sum in 2^21 tokens of a warp (with the largest at 1 it was 2^14 tokens).
//
// V's scale s enters through the exponent: the products take p' = 2^(x + log2 s - m), so the
// output needs no scale, whatever the blocks' scales; the sum takes p' / s.
#include <stdint.h>

#include <algorithm>

#include "ts_window.cuh"
#include "ts_window_own.cuh"

namespace tsv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16 * kWarps;
constexpr int kCtasPerSm = 2;
constexpr float kSlack = 15.f;    // how far, in log2, a score may exceed its row's reference
constexpr float kHead = 7.f;      // a reference is set this far below the largest score
constexpr int kMinTiles = 4;      // least tiles a CTA takes: pieces of 256 tokens or more

using Params = WindowParams;

template <int MT, typename T>
__device__ __forceinline__ void attend(const Params& p) {
  constexpr int D = 64, ROWS = 16 * MT;
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

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int64_t cta = blockIdx.x;
  int4 desc = make_int4(-1, 0, 0, 0);
  Line<ROWS, kTile> line;
  if (!line_begin<ROWS, kTile, kThreads>(p, kMinTiles, line)) {
    if (tid == 0) p.desc[cta] = desc;
    grid_wait();  // so that this kernel's end is the end of the one before too
    return;
  }
  bool waited = false;
  Segment sg;
  while (line.next(p, sg)) {
    const Req& r = sg.r;
    const int kvh = sg.kvh, block = sg.block, t0 = sg.t0, t1 = sg.t1, rows = sg.rows;

    // ---- Q: row i of the unit is window row (block*ROWS + i) / group of head kvh*group +
    // the remainder. Each row's factor, then the fragments.
    __syncthreads();  // the previous unit's reads of shared memory are done
    for (int i = warp; i < ROWS; i += kWarps) {
      float top = 0.f;
      uint32_t bad = 0;
      if (i < rows) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(q_row(p, sg, ROWS, i))[lane];
        const float2 f = unpack<T>(w);
        top = fmaxf(fabsf(f.x), fabsf(f.y));
        bad = not_finite<T>(w);
      }
      top = warp_max(top);
      // 2^e <= top < 2^(e+1); the row is divided by 2^e (both factors stay normal: by 2^126 above
      // that). A row with a value that is not finite: NaN, and with it its scores
      const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) s_fac[i] = bad ? NAN : __uint_as_float((uint32_t)e << 23);
    }
    __syncthreads();
    for (int i = tid; i < MT * KS * 32; i += kThreads) {
      const int l = i & 31, ks = i / 32 % KS, mt = i / 32 / KS, qc = l & 3, qg = l >> 2;
      // K's lane qc holds dims 16qc .. + 15; step k takes dims 4k .. 4k + 3 of them
      const int dim = qc * 16 + ks * 4;
      uint32_t w[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = mt * 16 + half * 8 + qg;
        uint2 x = make_uint2(0, 0);
        float inv = 1.f;
        if (row < rows) {
          x = *reinterpret_cast<const uint2*>(q_row(p, sg, ROWS, row) + dim * 2);
          inv = __uint_as_float(0x7F000000u - __float_as_uint(s_fac[row]));  // 1 / 2^e
        }
        const float2 u = unpack<T>(x.x), v = unpack<T>(x.y);
        w[half] = f16x2(u.x * inv, u.y * inv);
        w[2 + half] = f16x2(v.x * inv, v.y * inv);
      }
      s_q[i] = make_uint4(w[0], w[1], w[2], w[3]);
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
            const float to = top[mt][h] > m[mt][h] + kSlack ? top[mt][h] - kHead : m[mt][h];
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
    const int32_t* table = p.c.page_table + sg.b * p.c.ld_table;
    struct Loaded {
      uint4 k[2];
      uint32_t v[4][VW];
      float ks, vs;
    };
    auto page_of = [&](int t) -> int32_t {  // page of this warp's tokens of tile t, or -1
      const int64_t tok = (int64_t)t * kTile + warp * 16;
      if (t >= t1 || tok >= r.len) return -1;
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
        x.k[n] = ok ? ldg_stream(at) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tt = 2 * c + (i & 1) + (i >> 1) * 8;
        const bool ok = page >= 0 && tok + tt < r.len;
        const char* at = vc + page * p.c.v_page_stride + (int64_t)(slot + tt) * p.c.v_token_stride + g * (D / 8);
        const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0, 0);
        x.v[i][0] = w.x, x.v[i][1] = w.y;
      }
      x.ks = x.vs = 1.f;
      if (page >= 0) {
        x.ks = __ldg(p.c.k_scale + (int64_t)page * p.c.heads + kvh);
        x.vs = scale_of_v(__ldg(p.c.v_scale + (int64_t)page * p.c.heads + kvh), x.ks);
      }
    };
    Loaded next;
    int32_t page = page_of(t0), page2 = page_of(t0 + 1);
    if (t0 < t1) fetch(t0, page, next);
    for (int t = t0; t < t1; ++t) {
      Loaded now = next;
      const int32_t page_now = page;
      page = page2;
      page2 = page_of(t + 2);
      if (t + 1 < t1) fetch(t + 1, page, next);
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
          const uint4 w4 = now.k[n];
          const uint32_t w = ks == 0 ? w4.x : ks == 1 ? w4.y : ks == 2 ? w4.z : w4.w;
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
    if (!waited) {  // for the window's own part
      grid_wait();
      waited = true;
    }
    __syncthreads();
    const bool whole = sg.whole();
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
        const int64_t at = sg.at(p, ROWS, row);
        float own;
        const float by = finish_row(p, at, top, sum, own);  // the row's threads write the same lse
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.own_ml) v = *reinterpret_cast<const float4*>(p.own_o + at * D + d);
        const uint2 w = make_uint2(pack<T>(fmaf(acc.x, by, v.x * own), fmaf(acc.y, by, v.y * own)),
                                   pack<T>(fmaf(acc.z, by, v.z * own), fmaf(acc.w, by, v.w * own)));
        *reinterpret_cast<uint2*>(static_cast<char*>(p.a.out) + (at * D + d) * 2) = w;
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
        desc.x = (int)sg.b;
        desc.y = kvh * r.blocks + block;
        desc.z = rows;
      } else {
        desc.w = t1 == r.tiles ? 1 : 0;
      }
    }
  }
  if (tid == 0) p.desc[cta] = desc;
}

template <int MT, typename T>
__global__ void __launch_bounds__(kThreads) k_window(const __grid_constant__ Params p) {
  grid_launch();
  attend<MT, T>(p);
}

// More than 32 rows a window: blocks of 64 rows, for which K and V are converted half as often, where the
// cached tokens are many; blocks of 32 where the ends of units weigh more. Tiles a CTA in blocks of
// 64, us with 64 and with 32 rows: 5: 83 and 56; 8: 69 and 59; 16: 136 and 136; 26: 66 and 58; 41: 97 and
// 100; 66: 143 and 150; 111: 174 and 203; 344: 559 and 686. The lengths are on the device, so the choice is made here.
constexpr int kWideTiles = 36;

template <typename T>
__global__ void __launch_bounds__(kThreads) k_window_rows(const __grid_constant__ Params p) {
  grid_launch();
  const bool wide = line_length<64, kTile, kThreads>(p) >= (int64_t)kWideTiles * gridDim.x;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.wide = wide;
  if (wide) attend<4, T>(p);
  else attend<2, T>(p);
}

template <typename T>
__global__ void __launch_bounds__(128) k_join_rows(const __grid_constant__ Params p) {
  grid_wait();
  if (*p.wide) join_row<64, 64, kTile, T>(p);
  else join_row<64, 32, kTile, T>(p);
}

constexpr int smem_bytes(int D, int rows) {
  return rows / 16 * (D / 16) * 32 * 16 + rows * 4 + kWarps * rows * (D + 4) * 4 + kWarps * rows * 8;
}

// kernel, join: k_window and k_join, or k_window_rows and k_join_rows, for blocks of at most ROWS rows.
template <auto kernel, auto join, int ROWS, typename T>
cudaError_t launch(const Params& p, int sms, cudaStream_t s) {
  constexpr int D = 64, bytes = smem_bytes(D, ROWS);
  cudaError_t e = allow_smem<kernel>(bytes);
  if (e != cudaSuccess) return e;
  const int grid = sms * kCtasPerSm;
  if (p.a.k_new) {
    if ((e = launch_own<D, ROWS, T>(p, s)) != cudaSuccess) return e;
    e = launch_after(kernel, dim3(grid), kThreads, bytes, s, p);
  } else {
    kernel<<<grid, kThreads, bytes, s>>>(p);
    e = cudaGetLastError();
  }
  // units of one tile are never split
  if (e != cudaSuccess || (int64_t)p.c.max_pages * p.c.page_size <= kTile) return e;
  return launch_after(join, dim3(grid, ROWS / 4), 128, 0, s, p);
}

template <typename T>
cudaError_t launch_64(const Params& p, int rows, int sms, cudaStream_t s) {
  switch (rows) {
    case 16: return launch<k_window<1, T>, k_join<64, 16, kTile, T>, 16, T>(p, sms, s);
    case 32: return launch<k_window<2, T>, k_join<64, 32, kTile, T>, 32, T>(p, sms, s);
    default: return launch<k_window_rows<T>, k_join_rows<T>, 64, T>(p, sms, s);
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// The rows of a block: by the average window. head_dim 128, ragged chains of 4 to 20 rows: 162 us
// with 32, 189 with 64; trees of 256 rows: 416 with 32, 330 with 64. head_dim 64, one row of 4
// heads over 37 tokens: 9.7 us with 16, 11.1 with 32; 64 there means at most 64 (k_window_rows).
int block_rows(const WindowParams& p) {
  const int64_t rows = (p.a.total_rows * p.group + p.c.batch - 1) / p.c.batch;
  if (p.c.head_dim == 128) return rows <= 32 ? 32 : 64;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// Lays the workspace out; returns its bytes.
size_t lay_out(WindowParams& p, void* ws, int sms) {
  const int rows = block_rows(p), D = p.c.head_dim;
  const size_t ctas = (size_t)sms * kCtasPerSm;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* at = static_cast<char*>(ws) + off;
    off += up256(bytes);
    return at;
  };
  p.desc = reinterpret_cast<int4*>(take(ctas * sizeof(int4)));
  p.wide = reinterpret_cast<int32_t*>(take(sizeof(int32_t)));
  p.part = reinterpret_cast<float*>(take(2 * ctas * slot_floats(rows, D) * sizeof(float)));
  const size_t n = (size_t)p.a.total_rows * p.a.heads_q;
  // the window's own part: of every row, or (ts_window_tc.cu) of a block a CTA
  p.own_o = reinterpret_cast<float*>(take(std::max(n, (size_t)sms * rows) * D * sizeof(float)));
  p.own_ml = reinterpret_cast<float2*>(take(n * sizeof(float2)));
  return off;
}

}  // namespace

size_t window_workspace(int64_t batch, int64_t total_rows, int heads_q, int heads, int head_dim, int sms) {
  WindowParams p{};
  p.c.batch = batch;
  p.c.heads = heads;
  p.c.head_dim = head_dim;
  p.a.total_rows = total_rows;
  p.a.heads_q = heads_q;
  p.group = heads_q / heads;
  return lay_out(p, nullptr, sms);
}

cudaError_t launch_window(const ts_kv_cache& c, const ts_attn_args& a, void* ws, int sms, uint64_t wait_cycles,
                          cudaStream_t s) {
  Params p{};
  p.c = c;
  p.a = a;
  p.page_shift = __builtin_ctz((unsigned)c.page_size);
  p.group = a.heads_q / c.heads;
  p.scale_log2 = a.sm_scale * kLog2e;
  p.wait_cycles = wait_cycles;
  lay_out(p, ws, sms);
  if (!a.k_new) p.own_ml = nullptr;
  if (c.head_dim == 128) return launch_window_tc(p, block_rows(p), sms, s);
  const int rows = block_rows(p);
  return a.dtype == TS_BF16 ? launch_64<__nv_bfloat16>(p, rows, sms, s) : launch_64<__half>(p, rows, sms, s);
}

}  // namespace tsv
