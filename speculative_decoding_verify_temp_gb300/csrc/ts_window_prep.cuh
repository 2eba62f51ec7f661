// What comes before the cached tokens in window attention: the window's own part, and Q as the
// tensor cores want it.
#pragma once

#include "ts_window.cuh"

namespace tsv {

constexpr int kPrepThreads = 128;

__host__ __device__ constexpr int q_block_bytes(int rows, int parts) { return parts * rows * 128 + 16; }

// One CTA a row block of a KV head.
//
// The window's own tokens: 16 rows a warp, m16n8k16 products of Q, K and V in their own type,
// probabilities in two parts of it (16 and more significant bits). A row's result is left
// unnormalised in own_o with its reference and sum in own_ml.
//
// Q in e4m3 parts (PARTS > 0, D = 128): the block is scaled by a power of two to below 2^8 and
// each value is split into PARTS codes, each the rounded rest of the ones before. Four
// significant bits a part: two parts hold a bf16 value, three an fp16 value, exactly down to
// 2^-9 of the block's largest magnitude, below that to within 2^-18 of it. The codes are
// written as the product wants them in shared memory: rows of 128 bytes, the 16-byte pieces of
// row r at their place XOR r % 8.
template <int D, int ROWS, int PARTS, typename T>
__global__ void __launch_bounds__(kPrepThreads) k_window_prep(const __grid_constant__ WindowParams p) {
  constexpr int KS = D / 16, NT = D / 8, kTile = 64;
  grid_launch();
  __shared__ uint64_t s_sees[TS_MAX_WINDOW][2];  // bit j: the row sees window token j
  __shared__ float s_top[kPrepThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.x % p.c.heads;
  const int64_t blk = blockIdx.x / p.c.heads;
  // the request whose blocks hold blk
  auto base = [&](int64_t b) {
    const int64_t row0 = p.a.qo_indptr ? max(p.a.qo_indptr[b], 0) : b * (p.a.total_rows / p.c.batch);
    return block_base(row0, p.group, ROWS, b);
  };
  int64_t lo = 0, hi = p.c.batch;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (base(mid) <= blk) lo = mid;
    else hi = mid;
  }
  Segment s;
  s.b = lo;
  s.r = request<ROWS, kTile>(p, raw_request(p, lo));
  s.kvh = kvh;
  s.block = (int)(blk - base(lo));
  if (s.r.rows == 0 || s.block < 0 || s.block >= s.r.blocks) return;
  s.rows = min(ROWS, s.r.rows * p.group - s.block * ROWS);
  auto q_row = [&](int i) -> const char* {
    const int j = s.block * ROWS + i;
    return static_cast<const char*>(p.a.q) + (s.r.row0 + j / p.group) * p.a.q_row_stride +
           (int64_t)(kvh * p.group + j % p.group) * p.a.q_head_stride;
  };

  if constexpr (PARTS > 0) {
    static_assert(D == 128, "rows of 128 bytes");
    float top = 0.f;
    for (int i = tid; i < s.rows * (D / 8); i += kPrepThreads) {
      const uint4 w = *reinterpret_cast<const uint4*>(q_row(i / (D / 8)) + i % (D / 8) * 16);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack<T>(x[k]);
        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    top = warp_max(top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) top = fmaxf(top, s_top[w]);
    // 2^e <= top < 2^(e+1); values are multiplied by 2^(7 - e)
    const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 227);
    const float by = __uint_as_float((uint32_t)(254 + 7 - e) << 23);
    uint8_t* out = p.q_parts + (blk * p.c.heads + kvh) * q_block_bytes(ROWS, PARTS);
    if (tid == 0) *reinterpret_cast<float*>(out + PARTS * ROWS * D) = __uint_as_float((uint32_t)(e - 7) << 23);
    for (int i = tid; i < ROWS * (D / 16); i += kPrepThreads) {
      const int row = i / (D / 16), piece = i % (D / 16);
      uint4 w[2] = {};
      if (row < s.rows) {
        const uint4* q = reinterpret_cast<const uint4*>(q_row(row) + piece * 32);
        w[0] = q[0];
        w[1] = q[1];
      }
      float x[16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t y[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack<T>(y[k]);
          x[h * 8 + 2 * k] = f.x * by;
          x[h * 8 + 2 * k + 1] = f.y * by;
        }
      }
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        uint32_t z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[k] = e4m3x4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          const float4 f = e4m3x4_to_f32(z[k]);
          x[4 * k] -= f.x, x[4 * k + 1] -= f.y, x[4 * k + 2] -= f.z, x[4 * k + 3] -= f.w;
        }
        *reinterpret_cast<uint4*>(out + part * ROWS * D + row * D + (piece ^ (row & 7)) * 16) = make_uint4(z[0], z[1], z[2], z[3]);
      }
    }
  }

  if (!p.a.k_new) return;
  // ancestors lie before a row, so the walks end
  for (int i = tid; i < s.r.rows; i += kPrepThreads) {
    uint64_t lo64 = 0, hi64 = 0;
    if (p.a.parents) {
      int at = i;
      while (at >= 0) {
        if (at < 64) lo64 |= 1ull << at;
        else hi64 |= 1ull << (at - 64);
        const int up = p.a.parents[s.r.row0 + at];
        at = up < at ? up : -1;
      }
    } else {
      lo64 = i >= 63 ? ~0ull : (2ull << i) - 1;
      hi64 = i >= 64 ? (2ull << (i - 64)) - 1 : 0;
    }
    s_sees[i][0] = lo64;
    s_sees[i][1] = hi64;
  }
  __syncthreads();

  for (int i0 = warp * 16; i0 < s.rows; i0 += 16 * (kPrepThreads / 32)) {
    float o[NT][4], m[2] = {kNone, kNone}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    // the last window row of these rows: no row sees a token behind its own
    const int last = (s.block * ROWS + min(i0 + 15, s.rows - 1)) / p.group;
    for (int tok = 0; tok <= last; tok += 16) {
      const char* kn = static_cast<const char*>(p.a.k_new) + (s.r.row0 + tok) * p.a.k_row_stride + kvh * p.a.k_head_stride;
      const char* vn = static_cast<const char*>(p.a.v_new) + (s.r.row0 + tok) * p.a.v_row_stride + kvh * p.a.v_head_stride;
      float x[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        // lane c's four dims of step ks: any order serves, as Q's and K's agree
        const int dim = (ks / 4) * 64 + c * 16 + (ks % 4) * 4;
        uint32_t qa[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = i0 + half * 8 + g;
          uint2 w = make_uint2(0, 0);
          if (row < s.rows) w = *reinterpret_cast<const uint2*>(q_row(row) + dim * 2);
          qa[half] = w.x;
          qa[2 + half] = w.y;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint2 kb = make_uint2(0, 0);
          if (tok + n * 8 + g < s.r.rows) kb = *reinterpret_cast<const uint2*>(kn + (n * 8 + g) * p.a.k_row_stride + dim * 2);
          mma16816<T>(x[n], qa, kb.x, kb.y);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = i0 + h * 8 + g;
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = tok + n * 8 + 2 * c + e;
            const bool seen = i < s.rows && j < s.r.rows && (s_sees[(s.block * ROWS + i) / p.group][j >> 6] >> (j & 63) & 1);
            x[n][2 * h + e] = seen ? x[n][2 * h + e] * p.scale_log2 : -INFINITY;
            top = fmaxf(top, x[n][2 * h + e]);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float to = fmaxf(m[h], top), by = ex2(m[h] - to);
        m[h] = to;
        l[h] *= by;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][2 * h] *= by;
          o[j][2 * h + 1] *= by;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[n][2 * h + e] = ex2(x[n][2 * h + e] - to);
            l[h] += x[n][2 * h + e];
          }
      }
      uint32_t pa[4], pb[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float u = x[n][2 * h], v = x[n][2 * h + 1];
          const uint32_t w = pack<T>(u, v);
          const float2 f = unpack<T>(w);
          pa[n * 2 + h] = w;
          pb[n * 2 + h] = pack<T>(u - f.x, v - f.y);
        }
      // a value that is not finite must reach only the rows that see it: 0 in the product,
      // added row by row below
      bool odd = false;
      auto v_at = [&](int i, int dim) -> uint32_t {
        if (tok + i >= s.r.rows) return 0;
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
        mma16816<T>(o[j], pa, b0, b1);
        mma16816<T>(o[j], pb, b0, b1);
      }
      if (__any_sync(0xffffffffu, odd)) {
        for (int i = 0; i < 16; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // p of (row h*8 + g, token i) lies in lane i % 8 / 2 of the quad
            const int from = (lane & ~3) | ((i & 7) >> 1);
            const float p0 = __shfl_sync(0xffffffffu, i < 8 ? x[0][2 * h] : x[1][2 * h], from);
            const float p1 = __shfl_sync(0xffffffffu, i < 8 ? x[0][2 * h + 1] : x[1][2 * h + 1], from);
            const int row = i0 + h * 8 + g, j = tok + i;
            if (row < s.rows && j < s.r.rows && (s_sees[(s.block * ROWS + row) / p.group][j >> 6] >> (j & 63) & 1)) {
#pragma unroll
              for (int d = 0; d < NT; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t w = v_at(i, (2 * c + e) * (D / 8) + d);
                  if (not_finite<T>(w)) o[d][2 * h + e] += (i & 1 ? p1 : p0) * unpack<T>(w).x;
                }
            }
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int row = i0 + h * 8 + g;
      if (row >= s.rows) continue;
      const int64_t at = s.at(p, ROWS, row);
      if (c == 0) p.own_ml[at] = make_float2(m[h], sum);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < NT; j += 4)
          *reinterpret_cast<float4*>(p.own_o + at * D + (2 * c + e) * (D / 8) + j) =
              make_float4(o[j][2 * h + e], o[j + 1][2 * h + e], o[j + 2][2 * h + e], o[j + 3][2 * h + e]);
    }
  }
}

template <int D, int ROWS, int PARTS, typename T>
cudaError_t launch_prep(const WindowParams& p, cudaStream_t s) {
  k_window_prep<D, ROWS, PARTS, T><<<(unsigned)(block_count(p, ROWS) * p.c.heads), kPrepThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tsv
