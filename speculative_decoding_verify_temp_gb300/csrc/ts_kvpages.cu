// The pages of the 8-bit KV cache among requests: counted holders, continuations that share their
// source's pages, room for new tokens (with a copy of a page that others hold too), release, and
// moving the live pages to the lowest ids.
//
//   k_counts      refcount_out = refcount, where they are not the same array
//   k_fork        tables and lengths of continuations; a holder more for each entry
//   k_free        a holder less for each entry of a released request
//   k_pool_scan   which pages are free, as bits, and how many in each chunk of pages; for reserve
//                 also what each request asks for
//   k_reserve     gives the pages out, writes the tables, copies the pages that are copied
//   k_lists       for compact: the holes, the pages that fill them, and where each goes
//   k_compact     moves them and follows with tables and counts
//
// Nothing depends on the order in which CTAs run: counts are integer sums, and every page number
// follows from prefix sums over the whole pool and the whole batch.
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/ts_verify.h"
#include "ts_common.cuh"
#include "ts_internal.h"
#include "ts_tc.cuh"

namespace tsv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunkUnit = kThreads * 8;  // pages; chunks are multiples of it
constexpr int kMaxChunks = 1024;
constexpr int kColumns = kThreads * 4;    // table entries of a CTA's step

struct Pool {
  ts_kv_cache c;
  const int32_t* count;
  int32_t* count_out;
  int32_t shift;             // log2 of page_size
  int32_t chunks;
  int64_t chunk;             // pages of a chunk
  uint32_t* mask;            // a bit a page: free
  int32_t* chunk_free;
  // reserve and compact
  int32_t* table_out;
  int64_t ld_out;
  const int32_t* new_lens;
  const int32_t* held_lens;  // or null
  int32_t* reserved;
  uint32_t* ask;             // pages a request asks for | kCopies | kKeeps
  int32_t* last;             // its last page, where it copies it (the table may be written in place)
  int32_t* hole;
  int32_t* come;
  int32_t* place;            // of a page that moves: its number among those
  int32_t* live;             // the caller's
  int32_t* moves;
};

constexpr uint32_t kCopies = 1u << 30, kKeeps = 1u << 31, kAsk = kCopies - 1;

__device__ __forceinline__ int32_t length(const ts_kv_cache& c, int shift, int64_t b) {
  return min(max(c.seq_lens[b], 0), c.max_pages << shift);  // at most 2^30
}
// The tokens that the request's pages have room for.
__device__ __forceinline__ int32_t room(const ts_kv_cache& c, const int32_t* held, int shift, int64_t b, int32_t len) {
  return held ? max(len, min(held[b], c.max_pages << shift)) : len;
}
__device__ __forceinline__ int32_t entries(int32_t len, int shift) { return (int)(((unsigned)len + (1u << shift) - 1) >> shift); }
__device__ __forceinline__ bool names(const ts_kv_cache& c, int32_t page) { return page >= 0 && page < c.num_pages; }

__global__ void __launch_bounds__(kThreads) k_counts(const int32_t* in, int32_t* out, int64_t n) {
  grid_launch();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) out[i] = in[i];
}

// Rows of tables, kColumns entries a step. Bound: for small calls the chain sources -> length and
// table -> count; for large ones the reductions on the counts (512 continuations of 940 to 1876 entries: 8.9 us,
// of which the 4 MB of tables are 1).
__global__ void __launch_bounds__(kThreads) k_fork(ts_kv_cache c, ts_kv_fork_args a, int shift, int64_t columns) {
  grid_wait();
  for (int64_t u = blockIdx.x; u < a.n * columns; u += gridDim.x) {
    const int64_t i = u / columns, first = u % columns * kColumns;
    const int64_t b = a.sources[i];
    const bool ok = b >= 0 && b < c.batch;
    const int32_t len = ok ? length(c, shift, b) : 0, used = entries(len, shift);
    if (first == 0 && threadIdx.x == 0) a.lens_out[i] = len;
#pragma unroll
    for (int k = 0; k < kColumns / kThreads; ++k) {
      const int64_t j = first + k * kThreads + threadIdx.x;
      if (j >= c.max_pages) break;
      const int32_t page = j < used ? c.page_table[b * c.ld_table + j] : -1;
      a.table_out[i * a.ld_out + j] = page;
      if (names(c, page)) atomicAdd(a.refcount_out + page, 1);
    }
  }
}

__global__ void __launch_bounds__(kThreads) k_free(ts_kv_cache c, ts_kv_free_args a, int shift, int64_t columns) {
  grid_wait();
  for (int64_t u = blockIdx.x; u < c.batch * columns; u += gridDim.x) {
    const int64_t b = u / columns, first = u % columns * kColumns;
    if (a.release && a.release[b] == 0) continue;
    const int32_t used = entries(room(c, a.held_lens, shift, b, length(c, shift, b)), shift);
#pragma unroll
    for (int k = 0; k < kColumns / kThreads; ++k) {
      const int64_t j = first + k * kThreads + threadIdx.x;
      if (j >= used) break;
      const int32_t page = c.page_table[b * c.ld_table + j];
      if (names(c, page)) atomicSub(a.refcount_out + page, 1);
    }
  }
}

// ---- free pages

// The last page of a request that is to write to it while others hold it too, or -1.
__device__ __forceinline__ int32_t shared_last(const Pool& p, int64_t b, int32_t& len, int32_t& want) {
  const int32_t cap = p.c.max_pages << p.shift;
  len = length(p.c, p.shift, b);
  want = max(len, min(p.new_lens[b], cap));
  if (want == len || (len & ((1 << p.shift) - 1)) == 0) return -1;
  const int32_t page = p.c.page_table[b * p.c.ld_table + (len >> p.shift)];
  return names(p.c, page) && p.count[page] > 1 ? page : -1;
}

// The first p.chunks CTAs: a chunk of pages each. The ones behind, for reserve: kWarps requests each.
__global__ void __launch_bounds__(kThreads) k_pool_scan(const __grid_constant__ Pool p) {
  grid_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x < p.chunks) {
    __shared__ int32_t s_free[kWarps];
    const int64_t lo = blockIdx.x * p.chunk;
    int32_t free = 0;
    for (int64_t base = lo; base < lo + p.chunk; base += kChunkUnit) {
      int32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t i = base + k * kThreads + tid;
        v[k] = i < p.c.num_pages ? p.count[i] : 1;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t i = base + k * kThreads + tid;
        const uint32_t bits = __ballot_sync(0xffffffffu, v[k] <= 0);
        if (lane == 0) {
          p.mask[i >> 5] = bits;
          free += __popc(bits);
        }
        if (p.count_out != p.count && i < p.c.num_pages) p.count_out[i] = v[k];
      }
    }
    if (lane == 0) s_free[warp] = free;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) free += s_free[w];
      p.chunk_free[blockIdx.x] = free;
    }
    return;
  }
  // a request a warp; the last pages of the whole batch pass through shared memory
  __shared__ int32_t s_last[kThreads];
  const int64_t b = (int64_t)(blockIdx.x - p.chunks) * kWarps + warp;
  int32_t len = 0, want = 0, mine = -1;
  if (b < p.c.batch) mine = shared_last(p, b, len, want);
  int32_t sharers = 0;
  bool last = true;
  for (int64_t base = 0; base < p.c.batch; base += kThreads) {
    int32_t x, y;
    __syncthreads();
    s_last[tid] = base + tid < p.c.batch ? shared_last(p, base + tid, x, y) : -1;
    __syncthreads();
    if (mine < 0) continue;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const unsigned same = __ballot_sync(0xffffffffu, s_last[k * 32 + lane] == mine);
      sharers += __popc(same);
      const int64_t top = base + k * 32 + 31 - __clz(same | 1u);
      if (same && top > b) last = false;
    }
  }
  if (b < p.c.batch && lane == 0) {
    uint32_t ask = (uint32_t)max(entries(want, p.shift) - entries(room(p.c, p.held_lens, p.shift, b, len), p.shift), 0);
    if (mine >= 0) {
      const bool keeps = last && sharers >= p.count[mine];
      ask = keeps ? ask | kKeeps : (ask + 1) | kCopies;
    }
    p.ask[b] = ask;
    p.last[b] = mine;
  }
}

// The sum over the CTA; every thread gets it.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += s[w];
  return v;
}

// The free pages before each chunk into s_before [kMaxChunks]; returns those of the pool.
__device__ __forceinline__ int64_t free_before(const Pool& p, int32_t* s_before, int32_t* s_warp) {
  constexpr int kEach = kMaxChunks / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t v[kEach], all = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = tid * kEach + k;
    v[k] = i < p.chunks ? p.chunk_free[i] : 0;
    all += v[k];
  }
  int32_t upto = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int32_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_warp[w];
    total += s_warp[w];
  }
  int32_t before = upto - all;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    s_before[tid * kEach + k] = before;
    before += v[k];
  }
  __syncthreads();
  return total;
}

// A warp: calls give(i, page) for the free pages number first + i, i < n, which there are, in
// parallel over the lanes.
template <typename F>
__device__ __forceinline__ void walk_free(const Pool& p, const int32_t* s_before, int64_t first, int64_t n, F give) {
  const int lane = threadIdx.x & 31;
  // the last chunk with at most `first` free pages before it
  int lo = 0;
#pragma unroll 1
  for (int step = kMaxChunks / 2; step > 0; step >>= 1)
    if (lo + step < p.chunks && s_before[lo + step] <= first) lo += step;
  int64_t rank = s_before[lo];
  const int64_t words = (int64_t)p.chunks * p.chunk / 32;
#pragma unroll 1
  for (int64_t w = lo * (p.chunk / 32); w < words && rank < first + n; w += 64) {  // a chunk is a multiple of 64 words
    const uint2 m = *reinterpret_cast<const uint2*>(p.mask + w + 2 * lane);
    const int mine = __popc(m.x) + __popc(m.y);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    int64_t at = rank + upto - mine;
    uint64_t bits = (uint64_t)m.y << 32 | m.x;
    while (bits && at < first + n) {
      if (at >= first) give(at - first, (int32_t)((w + 2 * lane) * 32 + __ffsll(bits) - 1));
      bits &= bits - 1;
      ++at;
    }
    rank += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// One warp: tokens of one head of a page, 16 bytes a lane. kAtOnce loads are in flight.
__device__ __forceinline__ void copy_block(const char* from, char* to, int64_t token_stride, int D, int tokens) {
  constexpr int kAtOnce = 8;
  const int lane = threadIdx.x & 31, per = D / 16, log_per = per == 4 ? 2 : 3, n = tokens << log_per;
  for (int i0 = lane; i0 < n; i0 += 32 * kAtOnce) {
    uint4 w[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + 32 * k;
      if (i < n) w[k] = ldg_stream(from + (i >> log_per) * token_stride + (i & (per - 1)) * 16);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + 32 * k;
      if (i < n) *reinterpret_cast<uint4*>(to + (i >> log_per) * token_stride + (i & (per - 1)) * 16) = w[k];
    }
  }
}

// The same of head h of K or V (unit = 2 h + is_v), with its scale.
__device__ __forceinline__ void copy_unit(const ts_kv_cache& c, int unit, int64_t from, int64_t to, int tokens) {
  const bool is_v = unit & 1;
  const int h = unit >> 1;
  char* base = static_cast<char*>(is_v ? c.v : c.k) + h * (is_v ? c.v_head_stride : c.k_head_stride);
  const int64_t ld = is_v ? c.v_page_stride : c.k_page_stride;
  float* scale = (is_v ? c.v_scale : c.k_scale) + h;
  if ((threadIdx.x & 31) == 0) scale[to * c.heads] = scale[from * c.heads];
  copy_block(base + from * ld, base + to * ld, is_v ? c.v_token_stride : c.k_token_stride, c.head_dim, tokens);
}

// A request's CTAs: blockIdx.x / parts; each copies its share of the heads, the first also writes the
// table. Every CTA finds out for itself which pages the request gets, which costs less than a kernel in
// between. Bound: the chain demand -> prefix sums -> bits of the pool -> page; for many copies this chain in front of
// each CTA's, and HBM (512 requests, 427 of which copy half of a page of 64 tokens of 8 heads of 128: 15 us, 59 MB, 58 % of
// its rate). The sums before a request are formed by each request anew: batches of thousands feel it (65536: 2 to 5 ms).
__global__ void __launch_bounds__(kThreads) k_reserve(const __grid_constant__ Pool p, int parts) {
  grid_wait();
  __shared__ int32_t s_before[kMaxChunks], s_warp[kWarps], s_copy;
  __shared__ int64_t s_sum[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int64_t b = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const uint32_t word = p.ask[b];
  const int64_t ask = word & kAsk;
  bool copies = word & kCopies;
  if (part && !copies) return;
  const int64_t free = free_before(p, s_before, s_warp);
  int64_t first = 0;
#pragma unroll 4
  for (int64_t i = tid; i < b; i += kThreads) first += p.ask[i] & kAsk;
  first = block_sum(first, s_sum);
  const bool served = first + ask <= free || (ask == 0 && !(word & kKeeps));
  copies = copies && served;
  if (part && !copies) return;
  const int32_t len = length(p.c, p.shift, b), have = entries(room(p.c, p.held_lens, p.shift, b, len), p.shift);
  const int32_t want = max(len, min(p.new_lens[b], p.c.max_pages << p.shift));
  const int32_t need = served ? max(entries(want, p.shift), have) : have;
  const int32_t* row = p.c.page_table + b * p.c.ld_table;
  int32_t* out = p.table_out + b * p.ld_out;
  const int32_t from = p.last[b];
  if (warp == 0 && served && ask > 0)
    walk_free(p, s_before, first, part ? 1 : ask, [&](int64_t i, int32_t page) {
      if (copies && i == 0) s_copy = page;
      else out[have + i - (copies ? 1 : 0)] = page;
      if (part == 0) p.count_out[page] = 1;
    });
  __syncthreads();
  if (part == 0) {
    for (int32_t j = tid; j < p.c.max_pages; j += kThreads) {
      if (j < have && copies && j == len >> p.shift) out[j] = s_copy;
      else if (j < have) out[j] = row[j];
      else if (j >= need) out[j] = -1;
    }
    if (tid == 0) {
      p.reserved[b] = served ? want : len;
      if (copies) atomicSub(p.count_out + from, 1);
    }
  }
  if (!copies) return;
  const int32_t to = s_copy, tokens = len & ((1 << p.shift) - 1);
  for (int unit = part * kWarps + warp; unit < 2 * p.c.heads; unit += parts * kWarps) copy_unit(p.c, unit, from, to, tokens);
}

// ---- compact

// A chunk a CTA: with n live pages, the holes below n and the live pages from n on, both in order.
__global__ void __launch_bounds__(kThreads) k_lists(const __grid_constant__ Pool p) {
  grid_launch();
  grid_wait();
  __shared__ int32_t s_before[kMaxChunks], s_warp[kWarps];
  __shared__ int64_t s_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t pages = p.c.num_pages, n = pages - free_before(p, s_before, s_warp);
  // the holes: free pages below n
  int64_t holes = 0;
  if (n < pages) {
    const int64_t c = n / p.chunk;
    for (int64_t w = c * (p.chunk / 32) + tid; w <= n / 32; w += kThreads) {
      const uint32_t m = p.mask[w];
      holes += __popc(w == n / 32 ? m & ((1u << (n & 31)) - 1) : m);
    }
    holes = block_sum(holes, s_sum) + s_before[c];
  }
  if (blockIdx.x == 0 && tid == 0) {
    *p.live = (int32_t)n;
    *p.moves = (int32_t)holes;
  }
  int64_t rank = s_before[blockIdx.x];
  const int64_t lo = blockIdx.x * p.chunk;
  for (int64_t base = lo; base < lo + p.chunk && base < pages; base += kChunkUnit) {
    const uint32_t byte = reinterpret_cast<const uint8_t*>(p.mask)[base / 8 + tid];
    const int mine = __popc(byte);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int64_t at = rank + upto - mine;  // free pages before this thread's eight
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += s_warp[w];
      rank += s_warp[w];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = base + tid * 8 + k;
      if (byte >> k & 1) {
        if (i < n) p.hole[at] = (int32_t)i;
        ++at;
      } else if (i >= n && i < pages) {
        const int32_t r = (int32_t)(i - at - (n - holes));
        p.come[r] = (int32_t)i;
        p.place[i] = r;
      }
    }
  }
}

// Persistent: tables, counts, then the pages, a unit (K or V of a head of a page) a warp, eight loads of a lane in
// flight. Bound: HBM, each moved byte read and written once (1890 pages of 65 KB: 35.4 us, 7.0 TB/s).
__global__ void __launch_bounds__(kThreads) k_compact(const __grid_constant__ Pool p, int64_t columns) {
  grid_wait();
  const int tid = threadIdx.x;
  const int64_t n = *p.live, moves = *p.moves;
  for (int64_t u = blockIdx.x; u < p.c.batch * columns; u += gridDim.x) {
    const int64_t b = u / columns, first = u % columns * kColumns;
    const int32_t used = entries(room(p.c, p.held_lens, p.shift, b, length(p.c, p.shift, b)), p.shift);
#pragma unroll
    for (int k = 0; k < kColumns / kThreads; ++k) {
      const int64_t j = first + k * kThreads + tid;
      if (j >= p.c.max_pages) break;
      int32_t page = j < used ? p.c.page_table[b * p.c.ld_table + j] : -1;
      if (!names(p.c, page) || (p.mask[page >> 5] >> (page & 31) & 1)) page = -1;
      else if (page >= n) page = p.hole[p.place[page]];
      p.table_out[b * p.ld_out + j] = page;
    }
  }
  for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < moves; i += (int64_t)gridDim.x * kThreads) {
    const int32_t from = p.come[i], to = p.hole[i];
    const int32_t v = p.count[from];
    p.count_out[to] = v;
    p.count_out[from] = 0;
  }
  const int64_t per = 2 * p.c.heads, units = moves * per;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (tid >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
    const int64_t i = u / per;
    copy_unit(p.c, (int)(u % per), p.come[i], p.hole[i], p.c.page_size);
  }
}

// Launches with programmatic stream serialisation: the kernel may start before the one before it
// ends, and waits for it (grid_wait).
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), int64_t grid, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int64_t kCtasPerSm = 8;

// kernel over rows * columns steps, behind k_counts where the counts go to another array.
template <typename A>
cudaError_t count_rows(void (*kernel)(ts_kv_cache, A, int, int64_t), const ts_kv_cache& c, const A& a, int64_t rows, int sms,
                       cudaStream_t s) {
  const int64_t columns = std::max<int64_t>((c.max_pages + kColumns - 1) / kColumns, 1);
  const int64_t grid = std::min(rows * columns, sms * kCtasPerSm);
  const int shift = __builtin_ctz((unsigned)c.page_size);
  if (a.refcount_out == a.refcount || c.num_pages == 0) {
    kernel<<<(unsigned)grid, kThreads, 0, s>>>(c, a, shift, columns);
    return cudaGetLastError();
  }
  k_counts<<<(unsigned)std::min<int64_t>((c.num_pages + kThreads - 1) / kThreads, sms * kCtasPerSm), kThreads, 0, s>>>(a.refcount, a.refcount_out, c.num_pages);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_next(kernel, grid, s, c, a, shift, columns);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t lay_out(Pool& p, int64_t batch, int64_t pages, void* ws) {
  const int64_t units = std::max<int64_t>((pages + kChunkUnit - 1) / kChunkUnit, 1);
  const int64_t each = (units + kMaxChunks - 1) / kMaxChunks;
  p.chunk = each * kChunkUnit;
  p.chunks = (int32_t)((units + each - 1) / each);
  size_t off = 0;
  auto take = [&](auto*& at, size_t n) {
    at = reinterpret_cast<std::remove_reference_t<decltype(at)>>(static_cast<char*>(ws) + off);
    off += up256(n * 4);
  };
  take(p.mask, (size_t)(p.chunk / 32) * p.chunks);
  take(p.chunk_free, kMaxChunks);
  take(p.ask, (size_t)batch);
  take(p.last, (size_t)batch);
  take(p.hole, (size_t)pages);
  take(p.come, (size_t)pages);
  take(p.place, (size_t)pages);
  take(p.moves, 1);
  return off;
}

Pool pool(const ts_kv_cache& c, const int32_t* count, int32_t* count_out, int32_t* table_out, int64_t ld_out, void* ws) {
  Pool p{};
  p.c = c;
  p.count = count;
  p.count_out = count_out;
  p.shift = __builtin_ctz((unsigned)c.page_size);
  p.table_out = table_out;
  p.ld_out = ld_out;
  lay_out(p, c.batch, c.num_pages, ws);
  return p;
}

}  // namespace

size_t pages_workspace(int64_t batch, int64_t num_pages) {
  Pool p{};
  return lay_out(p, batch, num_pages, nullptr);
}

cudaError_t launch_kv_fork(const ts_kv_cache& c, const ts_kv_fork_args& a, int sms, cudaStream_t s) {
  return count_rows(k_fork, c, a, a.n, sms, s);
}

cudaError_t launch_kv_free(const ts_kv_cache& c, const ts_kv_free_args& a, int sms, cudaStream_t s) {
  return count_rows(k_free, c, a, c.batch, sms, s);
}

cudaError_t launch_kv_reserve(const ts_kv_cache& c, const ts_kv_reserve_args& a, void* ws, cudaStream_t s) {
  Pool p = pool(c, a.refcount, a.refcount_out, a.table_out, a.ld_out, ws);
  p.new_lens = a.new_lens;
  p.held_lens = a.held_lens;
  p.reserved = a.reserved;
  k_pool_scan<<<(unsigned)(p.chunks + (c.batch + kWarps - 1) / kWarps), kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int parts = std::max(1, 2 * c.heads / kWarps);
  return launch_next(k_reserve, c.batch * parts, s, p, parts);
}

cudaError_t launch_kv_compact(const ts_kv_cache& c, const ts_kv_compact_args& a, void* ws, int sms, cudaStream_t s) {
  Pool p = pool(c, a.refcount, a.refcount_out, a.table_out, a.ld_out, ws);
  p.live = a.live;
  p.held_lens = a.held_lens;
  k_pool_scan<<<(unsigned)p.chunks, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = launch_next(k_lists, p.chunks, s, p)) != cudaSuccess) return e;
  return launch_next(k_compact, sms * kCtasPerSm, s, p, std::max<int64_t>((c.max_pages + kColumns - 1) / kColumns, 1));
}

}  // namespace tsv
