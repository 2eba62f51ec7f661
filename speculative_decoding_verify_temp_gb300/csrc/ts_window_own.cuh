// The window's own tokens in window attention, and Q as the tensor cores want it.
#pragma once

#include "ts_window.cuh"

namespace tsv {

constexpr int kPrepThreads = 128;

// Which window tokens a window row sees, as bits.
struct Sees {
  uint64_t lo, hi;
  __device__ __forceinline__ bool operator()(int j) const { return (j < 64 ? lo >> j : hi >> (j - 64)) & 1; }
};

// Row i of a chain: tokens 0 .. i.
__device__ __forceinline__ Sees chain_sees(int i) {
  return {i >= 63 ? ~0ull : (2ull << i) - 1, i >= 64 ? (2ull << (i - 64)) - 1 : 0};
}

// Row i of a tree: itself and its ancestors. parents in shared memory; ancestors lie before a
// row, so the walk ends.
__device__ __forceinline__ Sees tree_sees(const int32_t* parents, int i) {
  Sees s = {0, 0};
#pragma unroll 1
  while (i >= 0) {
    if (i < 64) s.lo |= 1ull << i;
    else s.hi |= 1ull << (i - 64);
    const int up = parents[i];
    i = up < i ? up : -1;
  }
  return s;
}

// The address of the block's row i of Q.
__device__ __forceinline__ const char* q_row(const WindowParams& p, const Segment& s, int rows_per_block, int i) {
  const int j = s.block * rows_per_block + i;
  return static_cast<const char*>(p.a.q) + (s.r.row0 + j / p.group) * p.a.q_row_stride +
         (int64_t)(s.kvh * p.group + j % p.group) * p.a.q_head_stride;
}

// The window's own part for 16 rows of a block and dims 8 j0 .. 8 j1 - 1, by one warp:
// unnormalised outputs into o (the block's row i at o + i * ld), references (log2 units) and
// sums into ml. Products are m16n8k16 of Q, K and V in their own type; probabilities go in two
// parts of it (16 and more significant bits). A value of V that is not finite must reach only
// the rows that see it: it counts as 0 here, and where this returns true own_odd adds it row by
// row. The loops stay rolled and the outputs in memory: this runs once a unit, and code that
// has to be fetched costs more than it saves.
template <int D, int ROWS, typename T>
__device__ __forceinline__ bool own_part(const WindowParams& p, const Segment& s, int i0, int j0, int j1, const Sees* trees,
                                         float* o, int ld, float2* ml) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const char* q[2];
  Sees sees[2];
  float m[2] = {kNone, kNone}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = i0 + h * 8 + g;
    q[h] = i < s.rows ? q_row(p, s, ROWS, i) : nullptr;
    const int t = (s.block * ROWS + i) / p.group;
    sees[h] = i >= s.rows ? Sees{0, 0} : trees ? trees[t] : chain_sees(t);
  }
  o += (i0 + g) * ld + 2 * c;
  uint32_t odd = 0, bad[2] = {0, 0};  // values of V, of the rows' q that are not finite
  // the last window row of these rows: no row sees a token behind its own
  const int last = (s.block * ROWS + min(i0 + 15, s.rows - 1)) / p.group;
#pragma unroll 1
  for (int tok = 0; tok <= last; tok += 16) {
    const char* kn = static_cast<const char*>(p.a.k_new) + (s.r.row0 + tok) * p.a.k_row_stride + s.kvh * p.a.k_head_stride;
    const char* vn = static_cast<const char*>(p.a.v_new) + (s.r.row0 + tok) * p.a.v_row_stride + s.kvh * p.a.v_head_stride;
    float x[2][4] = {};
#pragma unroll 2
    for (int ks = 0; ks < D / 32; ++ks) {
      // lane c's eight dims, two steps of four: any order serves, as Q's and K's agree
      const int dim = ks * 32 + c * 8;
      uint4 qw[2], kw[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        qw[h] = q[h] ? __ldg(reinterpret_cast<const uint4*>(q[h] + dim * 2)) : make_uint4(0, 0, 0, 0);
        bad[h] |= not_finite<T>(qw[h].x) | not_finite<T>(qw[h].y) | not_finite<T>(qw[h].z) | not_finite<T>(qw[h].w);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        kw[n] = make_uint4(0, 0, 0, 0);
        if (tok + n * 8 + g < s.r.rows) kw[n] = __ldg(reinterpret_cast<const uint4*>(kn + (n * 8 + g) * p.a.k_row_stride + dim * 2));
      }
      const uint32_t q0[4] = {qw[0].x, qw[1].x, qw[0].y, qw[1].y}, q1[4] = {qw[0].z, qw[1].z, qw[0].w, qw[1].w};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        mma16816<T>(x[n], q0, kw[n].x, kw[n].y);
        mma16816<T>(x[n], q1, kw[n].z, kw[n].w);
      }
    }
    float by[2];
    uint32_t pa[4], pb[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = tok + n * 8 + 2 * c + e;
          x[n][2 * h + e] = j < s.r.rows && sees[h](j) ? x[n][2 * h + e] * p.scale_log2 : -INFINITY;
          top = fmaxf(top, x[n][2 * h + e]);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float to = fmaxf(m[h], top);
      by[h] = ex2(m[h] - to);
      m[h] = to;
      l[h] *= by[h];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float a = ex2(x[n][2 * h] - to), b = ex2(x[n][2 * h + 1] - to);
        l[h] += a + b;
        pa[n * 2 + h] = pack<T>(a, b);
        const float2 f = unpack<T>(pa[n * 2 + h]);
        pb[n * 2 + h] = pack<T>(a - f.x, b - f.y);
      }
    }
#pragma unroll 2
    for (int j = j0; j < j1; ++j) {
      // V: dim 8j + g of tokens 2c, 2c + 1, 2c + 8, 2c + 9
      uint32_t v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t* a = reinterpret_cast<const uint16_t*>(vn + (2 * c + h * 8) * p.a.v_row_stride) + j * 8 + g;
        const uint16_t* b = reinterpret_cast<const uint16_t*>(vn + (2 * c + h * 8 + 1) * p.a.v_row_stride) + j * 8 + g;
        const int t = tok + 2 * c + h * 8;
        v[h] = (t < s.r.rows ? (uint32_t)__ldg(a) : 0u) | (t + 1 < s.r.rows ? (uint32_t)__ldg(b) << 16 : 0u);
        const uint32_t bad = not_finite<T>(v[h]);
        odd |= bad;
        v[h] &= ~((bad >> 15) * 0xFFFFu);
      }
      float* at = o + j * 8;
      float2 u0 = make_float2(0.f, 0.f), u1 = u0;
      if (tok > 0) {
        u0 = *reinterpret_cast<float2*>(at);
        u1 = *reinterpret_cast<float2*>(at + 8 * ld);
      }
      float acc[4] = {u0.x * by[0], u0.y * by[0], u1.x * by[1], u1.y * by[1]};
      mma16816<T>(acc, pa, v[0], v[1]);
      mma16816<T>(acc, pb, v[0], v[1]);
      *reinterpret_cast<float2*>(at) = make_float2(acc[0], acc[1]);
      *reinterpret_cast<float2*>(at + 8 * ld) = make_float2(acc[2], acc[3]);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (bad[h]) l[h] = NAN;  // even where its scores are all -inf: a row sees itself at least
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (c == 0) ml[i0 + h * 8 + g] = make_float2(m[h], l[h]);
  }
  return __any_sync(0xffffffffu, odd);
}

// The values of V that are not finite in dims d0 .. d1 - 1, for the block's row i with reference
// m: each token that the row sees adds p times them to the row's outputs o. One warp.
template <int D, int ROWS, typename T>
__device__ __noinline__ void own_odd(const WindowParams& p, const Segment& s, int i, int d0, int d1, const Sees* trees, float m, float* o) {
  const int lane = threadIdx.x & 31, t = (s.block * ROWS + i) / p.group;
  const Sees sees = trees ? trees[t] : chain_sees(t);
  const T* q = reinterpret_cast<const T*>(q_row(p, s, ROWS, i));
#pragma unroll 1
  for (int j = 0; j <= t; ++j) {
    if (!sees(j)) continue;
    const T* k = reinterpret_cast<const T*>(static_cast<const char*>(p.a.k_new) + (s.r.row0 + j) * p.a.k_row_stride + s.kvh * p.a.k_head_stride);
    const T* v = reinterpret_cast<const T*>(static_cast<const char*>(p.a.v_new) + (s.r.row0 + j) * p.a.v_row_stride + s.kvh * p.a.v_head_stride);
    float x = 0.f;
#pragma unroll 1
    for (int d = lane; d < D; d += 32) x = fmaf((float)q[d], (float)k[d], x);
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const float w = ex2(x * p.scale_log2 - m);
#pragma unroll 1
    for (int d = d0 + lane; d < d1; d += 32) {
      const float y = (float)v[d];
      if (!(fabsf(y) < INFINITY)) o[d] += w * y;
    }
  }
}

// A walk over the block's rows of Q, two rows a step: 16 lanes share a row. Without divisions, and
// the loads of kAhead steps are in flight: a warp walks alone, while others wait for its codes
// (16 trees of 32 nodes over 8191 tokens: 317 us, 331 with a load a step and divisions).
struct QWalk {
  static constexpr int kAhead = 4;
  const char* at;
  int64_t head, row;  // strides: to the next head, and from behind the last head to the next row
  int h, group, left;
  uint4 w[kAhead];
  __device__ __forceinline__ uint4 load() {
    const uint4 x = left > 0 ? __ldg(reinterpret_cast<const uint4*>(at)) : make_uint4(0, 0, 0, 0);
    left -= 2;
    h += 2;
    at += 2 * head;
#pragma unroll 1
    for (; h >= group; h -= group) at += row;
    return x;
  }
  __device__ __forceinline__ QWalk(const WindowParams& p, const Segment& s, int rows_per_block) {
    const int lane = threadIdx.x & 31, j = s.block * rows_per_block + (lane >> 4);
    head = p.a.q_head_stride;
    row = p.a.q_row_stride - p.group * p.a.q_head_stride;
    group = p.group;
    h = j % group;
    left = s.rows - (lane >> 4);
    at = static_cast<const char*>(p.a.q) + (s.r.row0 + j / group) * p.a.q_row_stride + (int64_t)(s.kvh * group + h) * head +
         (lane & 15) * 16;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) w[k] = load();
  }
  __device__ __forceinline__ uint4 next() {
    const uint4 x = w[0];
#pragma unroll
    for (int k = 0; k + 1 < kAhead; ++k) w[k] = w[k + 1];
    w[kAhead - 1] = load();
    return x;
  }
};

// Two fp16 or bf16 magnitudes, the larger bit pattern of eight side by side.
__device__ __forceinline__ uint32_t largest_of_8(const uint4& w) {
  const uint32_t sign = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & sign, w.y & sign), __vmaxu2(w.z & sign, w.w & sign));
  return max(m >> 16, m & 0xFFFFu);
}

// Q in e4m3 parts, by one warp, into shared memory as the product wants it: rows of 128 bytes,
// the 16-byte pieces of row r at their place XOR r % 8. Each row is scaled by a power of two of
// its own, so that its largest magnitude lies in [2^7, 2^8) and no row has to do with another
// (one scale a block cost the small rows their bits, and an infinity all rows theirs), and each value split
// into PARTS codes, each the rounded rest of the ones before. Four significant bits a part down to
// steps of 2^-9: two parts hold a bf16 value exactly down to 2^-9 of the row's largest, three an
// fp16 value down to 2^-6 of it, smaller ones to within 2^-17 of it. Rows behind the block's last
// are zeros up to a multiple of 16. fac: what a row's codes stand for, times `by`; NaN, and with it the
// row's scores, where a value is not finite.
template <int ROWS, int PARTS, typename T>
__device__ __forceinline__ void split_q(const WindowParams& p, const Segment& s, float by, unsigned char* out, float* fac) {
  constexpr int D = 128;
  const int lane = threadIdx.x & 31, piece = lane & 15;
  QWalk q(p, s, ROWS);
#pragma unroll 1
  for (int r = lane >> 4; r < (s.rows + 15 & ~15); r += 2) {
    const uint4 w = q.next();
    const uint32_t y[4] = {w.x, w.y, w.z, w.w};
    // the two rows' largest magnitudes, as bits: a reduction each, which do not wait for each other
    const uint32_t mine = largest_of_8(w);
    const uint32_t even = __reduce_max_sync(0xffffffffu, lane < 16 ? mine : 0u), odd = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : mine);
    const uint32_t top = lane < 16 ? even : odd;
    // the exponent field of the largest as a float; both factors stay normal
    const int e = min(max((int)(__float_as_uint(unpack<T>(top).x) >> 23), 8), 254);
    const float scale = __uint_as_float((uint32_t)(254 + 7 - e) << 23);
    if (piece == 0) fac[r] = not_finite<T>(top) ? NAN : __uint_as_float((uint32_t)(e - 7) << 23) * by;
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack<T>(y[k]);
      x[2 * k] = f.x * scale;
      x[2 * k + 1] = f.y * scale;
    }
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      uint32_t z[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        z[k] = e4m3x4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        const float4 f = e4m3x4_to_f32(z[k]);
        x[4 * k] -= f.x, x[4 * k + 1] -= f.y, x[4 * k + 2] -= f.z, x[4 * k + 3] -= f.w;
      }
      *reinterpret_cast<uint2*>(out + part * ROWS * D + r * D + ((piece >> 1) ^ (r & 7)) * 16 + (piece & 1) * 8) = make_uint2(z[0], z[1]);
    }
  }
}

// The window's own part of every row into own_o and own_ml: one CTA a row block of a KV head,
// a warp 16 rows (head_dim 64).
template <int D, int ROWS, typename T>
__global__ void __launch_bounds__(kPrepThreads) k_window_own(const __grid_constant__ WindowParams p) {
  constexpr int kTile = 64;
  grid_launch();
  constexpr int kLd = D + 4;
  __shared__ float s_o[ROWS * kLd];
  __shared__ float2 s_ml[ROWS];
  __shared__ Sees s_trees[TS_MAX_WINDOW];
  __shared__ int32_t s_parents[TS_MAX_WINDOW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t blk = blockIdx.x / p.c.heads;
  // the request whose blocks hold blk: the last one that begins at or before it, by 32 probes
  // a step
  auto base = [&](int64_t b) {
    const int64_t row0 = p.a.qo_indptr ? max(p.a.qo_indptr[b], 0) : b * (p.a.total_rows / p.c.batch);
    return block_base(row0, p.group, ROWS, b);
  };
  int64_t lo = 0, n = p.c.batch;
  while (n > 1) {
    const int64_t each = (n + 31) / 32;
    const bool at = lane * each < n && base(lo + lane * each) <= blk;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, at) | 1u);
    lo += last * each;
    n = min(each, n - last * each);
  }
  Segment s;
  s.b = lo;
  s.r = request<ROWS, kTile>(p, raw_request(p, lo));
  s.kvh = blockIdx.x % p.c.heads;
  s.block = (int)(blk - base(lo));
  if (s.r.rows == 0 || s.block < 0 || s.block >= s.r.blocks) return;
  s.rows = min(ROWS, s.r.rows * p.group - s.block * ROWS);
  if (p.a.parents) {
    if (tid < s.r.rows) s_parents[tid] = p.a.parents[s.r.row0 + tid];
    __syncthreads();
    if (tid < s.r.rows) s_trees[tid] = tree_sees(s_parents, tid);
    __syncthreads();
  }
  for (int i0 = warp * 16; i0 < s.rows; i0 += 16 * (kPrepThreads / 32)) {
    const Sees* trees = p.a.parents ? s_trees : nullptr;
    const bool odd = own_part<D, ROWS, T>(p, s, i0, 0, D / 8, trees, s_o, kLd, s_ml);
    __syncwarp();
#pragma unroll 1
    for (int i = i0; i < min(s.rows, i0 + 16); ++i) {
      if (odd) own_odd<D, ROWS, T>(p, s, i, 0, D, trees, s_ml[i].x, s_o + i * kLd);
      __syncwarp();
      const int64_t at = s.at(p, ROWS, i);
      if (lane == 0) p.own_ml[at] = s_ml[i];
      for (int d = lane; d < D; d += 32) p.own_o[at * D + d] = s_o[i * kLd + d];
    }
  }
}

template <int D, int ROWS, typename T>
cudaError_t launch_own(const WindowParams& p, cudaStream_t s) {
  k_window_own<D, ROWS, T><<<(unsigned)(block_count(p, ROWS) * p.c.heads), kPrepThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tsv
