// The 8-bit KV cache: quantising rows as they are written and reading them back.
//
//   k_kv_append  one CTA a block (a page of one head of K or V) that the call touches
//   k_kv_read    one CTA for 16 (or 4) consecutive output rows, all heads
//
// A block's scale is a power of two, so that dividing by it is exact: the code is the
// element's own significand rounded to four bits, and rounding the block again to a larger
// scale changes only codes that fall below the normal range (2^-6 of the scale).
#include <stdint.h>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/ts_verify.h"
#include "ts_common.cuh"
#include "ts_internal.h"
#include "ts_kv.cuh"

namespace tsv {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;  // most rows of a CTA

// Eight elements of a row: as they lie in memory, and widened to fp32 (exact). fold: the larger
// magnitudes (a float's, or two 16-bit ones side by side), by their bits; bits: those of the
// largest as a float, or 0x7F800000 and more where one was not finite.
template <typename T>
struct Src;
__device__ __forceinline__ uint32_t fold_pairs(uint32_t m, const uint4& r) {
  const uint32_t sign = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(__vmaxu2(m, r.x & sign), r.y & sign), __vmaxu2(r.z & sign, r.w & sign));
}
template <>
struct Src<float> {
  struct Raw {
    float4 a, b;
  };
  __device__ __forceinline__ static Raw load(const void* p) {
    return {__ldg(static_cast<const float4*>(p)), __ldg(static_cast<const float4*>(p) + 1)};
  }
  __device__ __forceinline__ static void widen(const Raw& r, float* x) {
    x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
    x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
  }
  __device__ __forceinline__ static uint32_t fold(uint32_t m, const Raw& r) {
    float x[8];
    widen(r, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
};
template <>
struct Src<__nv_bfloat16> {
  typedef uint4 Raw;
  __device__ __forceinline__ static Raw load(const void* p) { return __ldg(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ static void widen(const Raw& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static uint32_t fold(uint32_t m, const Raw& r) { return fold_pairs(m, r); }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return max(m >> 16, m & 0xFFFFu) << 16; }
};
template <>
struct Src<__half> {
  typedef uint4 Raw;
  __device__ __forceinline__ static Raw load(const void* p) { return __ldg(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ static void widen(const Raw& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ static uint32_t fold(uint32_t m, const Raw& r) { return fold_pairs(m, r); }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) {  // fp16's infinity widens to fp32's
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(m >> 16, m & 0xFFFFu)))) & 0x7FFFFFFFu;
  }
};

// The least 2^e, e in [-60, 60], with a <= 448 * 2^e = 1.75 * 2^(e + 8); a finite, >= 0.
__device__ __forceinline__ float block_scale(float a) {
  const uint32_t b = __float_as_uint(a);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = a > 0.f ? min(max(e, -60), 60) : -60;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The rows of request b: the first position, how many, and where their numbers come from.
struct Rows {
  int64_t first;  // of a run of rows, or -1: src_index
  int64_t count;
};

__device__ __forceinline__ Rows rows_of(const ts_kv_append_args& a, int64_t batch, int64_t b) {
  if (a.src_index) return {-1, min((int64_t)max(a.src_len[b], 0), a.ld_src)};
  if (!a.qo_indptr) return {b * (a.total_rows / batch), a.total_rows / batch};
  const int64_t r0 = a.qo_indptr[b], r1 = a.qo_indptr[b + 1];
  if (r0 < 0 || r1 < r0 || r1 > a.total_rows) return {0, 0};
  return {r0, r1 - r0};
}

// One CTA: every `step`-th block that request b touches in head h of K or V. N = the eighths of
// a thousand elements of a block: a thread holds N times eight of them in registers between the
// maximum and the codes, with all loads in flight at once. Bound: HBM for prompts (24 k rows of
// 8 heads of 128, 147 MB of traffic); for the few rows after a verify step, the chain of
// dependent loads seq_len -> page -> rows (128 windows: 8 us). The prompts' 24 k rows take 32 us, 4.6
// TB/s (64 when the rows were read twice), and 78 % of the issue slots.
template <typename T, int D, int N>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(ts_kv_cache c, ts_kv_append_args a, int32_t step) {
  constexpr int per_row = D / 8, n = N * kAppendThreads * 8 / D;  // n: page_size
  const int64_t unit = blockIdx.x / step;
  const int h = (int)(unit % c.heads);
  const bool is_v = (unit / c.heads) & 1;
  const int64_t b = unit / (2 * c.heads);
  const int64_t cap = (int64_t)c.max_pages * n;
  const int64_t len = min((int64_t)max(c.seq_lens[b], 0), cap);
  const Rows rows = rows_of(a, c.batch, b);
  const char* src = static_cast<const char*>(is_v ? a.v : a.k) + h * (is_v ? a.v_head_stride : a.k_head_stride);
  const int64_t src_ld = is_v ? a.v_row_stride : a.k_row_stride;
  const int64_t tok_ld = is_v ? c.v_token_stride : c.k_token_stride;
  float* scales = is_v ? c.v_scale : c.k_scale;
  __shared__ int32_t s_max[kAppendThreads / 32];

  for (int64_t p = len / n + blockIdx.x % step;; p += step) {
    const int64_t lo = max(len, p * n), hi = min(min(len + rows.count, (p + 1) * n), cap);
    if (lo >= hi) return;
    const int64_t page = c.page_table[b * c.ld_table + p];
    const bool stored = page >= 0 && page < c.num_pages;
    const int held = (int)(lo - p * n);  // earlier tokens of the block
    const int chunks = stored ? (int)(hi - lo) * per_row : 0;
    // eight elements of row i / per_row of the block's new rows
    typename Src<T>::Raw raw[N];
    uint32_t there = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = k * kAppendThreads + threadIdx.x;
      if (i >= chunks) continue;
      const int64_t j = lo - len + i / per_row;
      const int64_t r = rows.first < 0 ? (int64_t)a.src_index[b * a.ld_src + j] : rows.first + j;
      if (r < 0 || r >= a.total_rows) continue;
      there |= 1u << k;
      raw[k] = Src<T>::load(src + r * src_ld + (int64_t)(i % per_row) * 8 * sizeof(T));
    }
    const float old = stored ? scales[page * c.heads + h] : 0.f;
    // the largest finite magnitude, as bits (-1: no row to store): of all at first (the largest
    // by integers, two at a time: prompts took 34 us with a test of each element), and where that
    // is not finite once more without those that are not
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (there >> k & 1) m = Src<T>::fold(m, raw[k]);
    int32_t top = there ? (int32_t)Src<T>::bits(m) : -1;
    if (top >= 0x7F800000) {
      top = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (!(there >> k & 1)) continue;
        float x[8];
        Src<T>::widen(raw[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int32_t y = __float_as_int(fabsf(x[e]));
          top = y < 0x7F800000 ? max(top, y) : top;
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();  // the previous block's reads of s_max are done
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) top = max(top, s_max[w]);
    if (top < 0) continue;
    char* block = static_cast<char*>(is_v ? c.v : c.k) + page * (is_v ? c.v_page_stride : c.k_page_stride) +
                  h * (is_v ? c.v_head_stride : c.k_head_stride);
    float scale = block_scale(__int_as_float(top));
    if (held) scale = fmaxf(old, scale);
    const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0;  // false: a caller's own scale
    const float inv = 1.f / scale;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (!(there >> k & 1)) continue;
      const int i = k * kAppendThreads + threadIdx.x;
      float x[8];
      Src<T>::widen(raw[k], x);
      if (pow2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], scale);
      }
      uint2 w;
      w.x = e4m3x4(x[0], x[1], x[2], x[3]);
      w.y = e4m3x4(x[4], x[5], x[6], x[7]);
      *reinterpret_cast<uint2*>(block + (held + i / per_row) * tok_ld + (i % per_row) * 8) = w;
    }
    if (held && scale != old) {
      const float ratio = __fdiv_rn(old, scale);
      for (int i = threadIdx.x; i < held * (D / 16); i += kAppendThreads) {
        uint4* at = reinterpret_cast<uint4*>(block + (i / (D / 16)) * tok_ld + (i % (D / 16)) * 16);
        const uint4 v = *at;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 f = e4m3x4_to_f32(w[k]);
          w[k] = e4m3x4(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (threadIdx.x == 0) scales[page * c.heads + h] = scale;
  }
}

template <typename T>
__device__ __forceinline__ void store16(void* p, const float* x);
template <>
__device__ __forceinline__ void store16<float>(void* p, const float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    __stcs(static_cast<float4*>(p) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
template <typename T2, typename F>
__device__ __forceinline__ void store16_half(void* p, const float* x, F two) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const T2 t = two(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(static_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(void* p, const float* x) {
  store16_half<__nv_bfloat162>(p, x, [](float u, float v) { return __floats2bfloat162_rn(u, v); });
}
template <>
__device__ __forceinline__ void store16<__half>(void* p, const float* x) {
  store16_half<__half2>(p, x, [](float u, float v) { return __floats2half2_rn(u, v); });
}

// One CTA: n output rows, whose request and page one thread each looks up; then 16
// codes a thread. Bound: HBM (the writes are two to four times the reads): 67 us for 62 k tokens of 8
// heads of 128 to bf16, 5.7 TB/s.
template <typename T>
__global__ void __launch_bounds__(kReadThreads) k_kv_read(ts_kv_cache c, ts_kv_read_args a, int n) {
  __shared__ int64_t s_page[kReadRows];  // -1: zeros, -2: no row
  __shared__ int32_t s_slot[kReadRows];
  const int64_t r0 = (int64_t)blockIdx.x * n;
  if (threadIdx.x < n) {
    const int64_t r = r0 + threadIdx.x;
    int64_t page = -2;
    int32_t slot = 0;
    if (r < a.total_rows) {
      int64_t lo = 0, hi = c.batch;  // the last b with out_indptr[b] <= r
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.out_indptr[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int64_t first = a.out_indptr[lo], last = a.out_indptr[lo + 1];
      if (first >= 0 && first <= r && r < last && last <= a.total_rows) {
        const int64_t pos = (a.start ? (int64_t)a.start[lo] : 0) + (r - first);
        page = -1;
        if (pos >= 0 && pos < c.seq_lens[lo] && pos < (int64_t)c.max_pages * c.page_size) {
          const int64_t id = c.page_table[lo * c.ld_table + pos / c.page_size];
          if (id >= 0 && id < c.num_pages) page = id;
          slot = (int32_t)(pos % c.page_size);
        }
      }
    }
    s_page[threadIdx.x] = page;
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();
  const int D = c.head_dim, parts = D / 16;
  const int per_row = c.heads * parts, all = n * per_row;
  constexpr int kAtOnce = 4;  // steps whose loads are in flight together
  for (int i0 = threadIdx.x; i0 < all; i0 += kAtOnce * kReadThreads) {
    uint4 kw[kAtOnce], vw[kAtOnce];
    float ks[kAtOnce], vs[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kReadThreads;
      kw[u] = vw[u] = make_uint4(0, 0, 0, 0);
      ks[u] = vs[u] = 0.f;
      if (i >= all) continue;
      const int t = i / per_row, h = i % per_row / parts, part = i % parts;
      const int64_t page = s_page[t];
      if (page < 0) continue;
      kw[u] = ldg_stream(static_cast<const char*>(c.k) + page * c.k_page_stride + h * c.k_head_stride +
                         s_slot[t] * c.k_token_stride + part * 16);
      vw[u] = ldg_stream(static_cast<const char*>(c.v) + page * c.v_page_stride + h * c.v_head_stride +
                         s_slot[t] * c.v_token_stride + part * 16);
      ks[u] = __ldg(c.k_scale + page * c.heads + h);
      vs[u] = __ldg(c.v_scale + page * c.heads + h);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kReadThreads;
      if (i >= all || s_page[i / per_row] == -2) continue;
      const int t = i / per_row, h = i % per_row / parts, part = i % parts;
      const int64_t at = (((r0 + t) * c.heads + h) * D + part * 16) * (int64_t)sizeof(T);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint4 w = which ? vw[u] : kw[u];
        const float s = which ? vs[u] : ks[u];
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
        float x[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 f = e4m3x4_to_f32(words[j]);
          x[4 * j] = f.x * s, x[4 * j + 1] = f.y * s, x[4 * j + 2] = f.z * s, x[4 * j + 3] = f.w * s;
        }
        store16<T>(static_cast<char*>(which ? a.v_out : a.k_out) + at, x);
      }
    }
  }
}

template <typename F>
cudaError_t by_dtype(int32_t dt, F f) {
  if (dt == TS_F32) f(float{});
  else if (dt == TS_BF16) f(__nv_bfloat16{});
  else f(__half{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const ts_kv_cache& c, const ts_kv_append_args& a, cudaStream_t s) {
  const int64_t units = c.batch * c.heads * 2;
  // CTAs a unit: the blocks an average request touches (a unit strides over the rest: 24 k rows in
  // 32 us; 158 with 2 CTAs a unit, when the kernel took 34), at least 2 (a window that crosses a page)
  const int64_t rows = a.src_index ? a.ld_src : (a.total_rows + c.batch - 1) / c.batch;
  const int64_t want = (rows + c.page_size - 1) / c.page_size + 1;
  const int64_t step = std::max<int64_t>(2, std::min(want, ((int64_t)1 << 30) / units));
  const int n = c.page_size * c.head_dim / (kAppendThreads * 8);
  return by_dtype(a.dtype, [&](auto t) {
    auto go = [&](auto kernel) { kernel<<<(unsigned)(units * step), kAppendThreads, 0, s>>>(c, a, (int32_t)step); };
    using T = decltype(t);
    if (c.head_dim == 64) {
      if (n == 1) go(k_kv_append<T, 64, 1>);
      else if (n == 2) go(k_kv_append<T, 64, 2>);
      else if (n == 4) go(k_kv_append<T, 64, 4>);
      else go(k_kv_append<T, 64, 8>);
    } else {
      if (n == 2) go(k_kv_append<T, 128, 2>);
      else if (n == 4) go(k_kv_append<T, 128, 4>);
      else if (n == 8) go(k_kv_append<T, 128, 8>);
      else go(k_kv_append<T, 128, 16>);
    }
  });
}

cudaError_t launch_kv_read(const ts_kv_cache& c, const ts_kv_read_args& a, int sms, cudaStream_t s) {
  // few rows are spread further: 300 rows of 2 heads of 64 in 3.5 us, 4.2 with 16; more CTAs than run at
  // once only repeat the lookup (62 k rows of 8 heads of 128: 67 us with 16 rows, 72 with 8)
  const int n = a.total_rows * c.heads * c.head_dim < (int64_t)sms * kReadThreads * 64 ? 4 : kReadRows;
  const int64_t grid = (a.total_rows + n - 1) / n;
  return by_dtype(a.dtype, [&](auto t) { k_kv_read<decltype(t)><<<(unsigned)grid, kReadThreads, 0, s>>>(c, a, n); });
}

}  // namespace tsv
