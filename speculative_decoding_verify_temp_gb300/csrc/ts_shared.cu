// Attention of windows whose requests share a prefix: the prefix is read and multiplied once for all
// rows of a group, the rest of each request by ts_tail.cu, which takes the prefix's part of a
// row in.
//
//   k_plan         the groups: rows, shared tokens (whole pages); what each request has left; how
//                  many CTAs go through the tokens side by side
//   k_prefix       one persistent CTA an SM: the shared tokens of the groups
//   k_prefix_join  joins the pieces of units that more than one CTA worked on, and plans the shares of ts_tail.cu
//
// The rows of a group's windows, all query heads of a KV head, are one matrix, so the products are
// proper matrix products: 128 rows of Q are the M = 128 of tcgen05.mma (kind f16),
//
//   S [128 x 128 tokens] = Q [128 x D] K^T        O [128 x D] += P [128 x 128 tokens] V
//
// with S, P and O in TMEM. K and V codes become fp16 (exact) on their way into shared memory,
// once for the two blocks of 128 rows that a CTA works on; Q is fp16 with a factor a row: a power
// of two that puts the row's largest magnitude into [2^14, 2^15), so that bf16 values are exact down to
// 2^-31 of it. P = 2^(x - m) is rounded to fp16 (2^-11), m a reference of the row that is set 2^h below a
// score and follows when a tile's sum is past fp16's range. V's scale is in the exponent. The small ones lose at
// most 2^-25 each; h goes by the tokens N of the CTA's share of the unit, log2 N - 13 and 4 at least, so that
// this is below 2^-12 of the row's sum however many small ones follow a large one (with h = 4 for all, a
// million of 2^-29 behind one lost 2^-9). At 14 fp16 ends it: 2^-11 in 2^28 tokens. (References that are lowered again
// where only small ones follow need no such end, but took 961 us in the case below.)
//
// Two slots, each 128 rows and 128 threads, a thread a row (no reduction crosses threads): while one
// slot's scores are made into P, the tensor cores work on the other's products. More than 128 rows
// of a block: a slot takes 128 of them, both work on every tile. At most 128: both slots have the
// same rows and take turns at the tiles, and meet at the end. TMA brings the pages, up to three tiles of
// K or V ahead; four warps make their codes fp16 and a lane of another issues the products.
//
// Groups with many rows: CTAs in gangs of up to 8 take the same share of the tokens at the same time, a
// block of rows each, so that a tile comes from DRAM once for a gang.
//
// Measured, 32 windows of 8 rows, 64 query and 8 KV heads of 128, 131071 shared tokens: 832 us, 1321 TFLOP/s,
// 0.68 of the measured bf16 peak. Bound: a slot's softmax takes 2300 clocks a tile (TMEM loads, 32 exponentials a
// clock and SM), the products of both slots 2054, and what is left of either is not hidden behind the other.
//
// Every wait is bounded, as in ts_window_tc.cu: after one ran out no wait waits and no copy is issued, products
// run on whatever is there (a test of each wait's outcome before them cost 8 %), and the CTA runs to its end.
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ts_tail.h"

namespace tsv {

struct PrefixParams {
  ts_kv_cache c;  // batch: the groups; page_table: the requests'
  ts_attn_args a;
  int32_t page_shift;
  int32_t group;
  float scale_log2;
  const int4* groups;  // {first row, rows, shared tokens, first request with a window}
  const int32_t* gang; // CTAs that share tokens
  const Start* starts; // [CTAs]
  float* part;         // [2 * CTAs] pieces of kBlock rows: outputs, references, sums
  int4* desc;          // [CTAs] {tail unit's group, its head, rows, 2 * its block | the CTA's first piece ends its unit}
  float* pre_o;
  float2* pre_ml;
  uint64_t wait_cycles;
};

__device__ __forceinline__ RawReq raw_request(const PrefixParams& p, int64_t g) {
  if (g >= p.c.batch) return {0, 0, 0};
  const int4 x = p.groups[g];
  return {x.x, x.x + x.y, x.z};
}
template <int ROWS, int TILE>
__device__ __forceinline__ Req request(const PrefixParams& p, const RawReq& raw) {
  Req r;
  r.row0 = raw.row0;
  r.rows = raw.len > 0 ? raw.row1 - raw.row0 : 0;
  r.len = raw.len;
  r.blocks = (int)(((unsigned)r.rows * p.group + ROWS - 1) / ROWS);  // here: sets of as many as a gang takes
  r.blocks = (r.blocks + *p.gang - 1) / *p.gang;
  r.tiles = max((int)((unsigned)(r.len + TILE - 1) / TILE), 1);
  return r;
}

namespace {

constexpr int kTile = 128;
constexpr int kRows = 128;   // of a slot
constexpr int kBlock = 2 * kRows;
constexpr int kConvert = 4;  // warps that make codes fp16: half of them K's, half V's
constexpr int kThreads = 256 + kConvert * 32 + 128;
// Registers of a thread: 128 at launch (512 threads), then by role
constexpr int kSoftmaxRegs = 184, kConvertRegs = 80, kIssueRegs = 64;
static_assert(256 * kSoftmaxRegs + kConvert * 32 * kConvertRegs + 128 * kIssueRegs <= kThreads * 128, "registers");
constexpr int kMeta = 8;     // tiles whose scales are in shared memory
// Barriers of K's and V's arrival, in turn: an even number, so that each is K's or V's alone. Who waits for it
// then sees all of its phases; one that saw every second would take the one before last for the last.
constexpr int kArrive = 6;
constexpr float kLeastHead = 4.f, kMostHead = 14.f;  // how far, in log2, a reference is set below the largest score
constexpr float kMostSum = 65504.f;  // of a tile's probabilities, where the reference stays: none is past fp16
constexpr float kMostRef = 65536.f;  // references of at most this size: scores and reference in one operation
constexpr int kMinTiles = 1;
constexpr int kPlanThreads = 1024;

__device__ uint32_t g_prefix_error;

template <int D>
struct Layout {
  static constexpr int k_stages = D == 128 ? 2 : 4;  // tiles of K in fp16
  static constexpr int v_halves = D == 128 ? 3 : 8;  // halves of tiles of V
  static constexpr int units = D == 128 ? 3 : 6;     // tiles of K or V as they come: K, V, K, ...
  static_assert(kArrive % 2 == 0 && kArrive % units == 0, "a unit's barrier is free when its place is");
  static constexpr int atoms = D / 64;               // of 64 values (128 bytes) a row
  static constexpr int atom_bytes = kTile * 128;     // of Q and K; of a half of V half as many
  static constexpr int tile_bytes = atoms * atom_bytes;
  static constexpr int unit_bytes = kTile * D;
  static constexpr int off_k = 2 * tile_bytes;       // Q of both slots before
  static constexpr int off_v = off_k + k_stages * tile_bytes;
  static constexpr int off_raw = off_v + v_halves * tile_bytes / 2;
  static constexpr int off_x = off_raw + units * unit_bytes;
  static constexpr int col_o = 2 * kTile;            // TMEM: S (and P) of both slots, then O
};

static_assert(2 * kRows * 8 <= 2 * Layout<64>::tile_bytes && kRows * 64 * 2 == Layout<64>::tile_bytes && kRows * 128 * 2 == Layout<128>::tile_bytes,
              "Q's place: where the slots meet");

struct Shared {
  uint64_t k_full[4], k_empty[4], v_full[8], v_empty[8], raw_full[kArrive], raw_empty[6], meta_full[kMeta];
  uint64_t s_full[2], p_full[2], o_done[2], q_full, q_empty;
  alignas(16) float4 meta[kMeta][8];  // of 16 tokens: K's scale, log2 of V's, 1 / V's, 2 (0: not there; 1: others of the tile are not)
  uint32_t tmem;
  alignas(16) int32_t stop;
  uint64_t wait_cycles;  // 8 bytes behind stop: wait reads it
};
static_assert(offsetof(Shared, wait_cycles) == offsetof(Shared, stop) + 8, "wait");

template <int D>
constexpr int smem_bytes() { return Layout<D>::off_x + (int)sizeof(Shared) + 1024; }
static_assert(smem_bytes<128>() <= 227 * 1024, "shared memory");

// All threads of four neighbouring warps.
template <int N, bool MORE>
__device__ __forceinline__ void set_regs() {
  if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A CTA's share: its gang's, of which it takes one block of each set.
struct Share {
  Line<kBlock, kTile, PrefixParams> line;
  int gang, rank;
  __device__ __forceinline__ static bool any(const PrefixParams& p) { return p.starts[blockIdx.x].b >= 0; }
  __device__ __forceinline__ explicit Share(const PrefixParams& p) {
    const Start at = p.starts[blockIdx.x];
    gang = at.gang;
    rank = blockIdx.x % gang;
    line_at<kBlock, kTile>(p, at, line);
  }
  __device__ __forceinline__ bool next(const PrefixParams& p, Segment& s) {
    while (line.next(p, s)) {
      s.block = s.block * gang + rank;
      s.rows = min(kBlock, s.r.rows * p.group - s.block * kBlock);
      if (s.rows > 0) return true;
    }
    return false;
  }
};

// ---- the groups

__global__ void __launch_bounds__(kPlanThreads) k_plan(const __grid_constant__ PrefixParams p, ts_kv_cache c, ts_shared_args sh,
                                                       int4* groups, int32_t* first, int32_t* gang, Start* starts, int ctas) {
  grid_launch();
  const ts_attn_args& a = p.a;
  const int page_shift = p.page_shift;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ unsigned long long s_cost[4];  // tiles, as gangs of 1, 2, 4 and 8 go through them
  if (threadIdx.x < 4) s_cost[threadIdx.x] = 0;
  for (int64_t b = threadIdx.x; b < c.batch; b += kPlanThreads) first[b] = 0;
  __syncthreads();
  WindowParams w{};  // windows as window attention reads them
  w.c = c;
  w.a = a;
  w.page_shift = page_shift;
  w.group = 1;
  for (int64_t g = warp; g < sh.groups; g += kPlanThreads / 32) {
    int64_t b0 = sh.group_indptr[g], b1 = sh.group_indptr[g + 1];
    if (b0 < 0 || b1 > c.batch || b1 < b0) b0 = b1 = 0;
    int least = INT32_MAX, lo = INT32_MAX, hi = 0, head = INT32_MAX;
    for (int64_t b = b0 + lane; b < b1; b += 32) {
      const Req r = request<1, 1>(w, raw_request(w, b));
      if (r.rows == 0) continue;
      least = min(least, r.len);
      lo = min(lo, (int)r.row0);
      hi = max(hi, (int)r.row0 + r.rows);
      head = min(head, (int)b);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    head = __reduce_min_sync(0xffffffffu, head);
    const bool some = lo < hi;
    const int s = some ? max(min(least, sh.shared_lens[g]), 0) >> page_shift << page_shift : 0;
    if (lane == 0) groups[g] = some ? make_int4(lo, hi - lo, s, head) : make_int4(0, 0, 0, 0);
    if (lane < 4 && s > 0) {
      const int64_t blocks = ((int64_t)(hi - lo) * (a.heads_q / c.heads) + kBlock - 1) / kBlock;
      atomicAdd(&s_cost[lane], (unsigned long long)((s + kTile - 1) / kTile * ((blocks + (1 << lane) - 1) >> lane << lane)));
    }
    for (int64_t b = b0 + lane; b < b1; b += 32) {
      const Req r = request<1, 1>(w, raw_request(w, b));
      if (r.rows) first[b] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {  // the largest that leaves at most a 32nd of the work to no one
    int k = 3;
    while (k > 0 && (1 << k > ctas || s_cost[k] > s_cost[0] + s_cost[0] / 32)) --k;
    *gang = 1 << k;
  }
  __syncthreads();
  line_starts<kBlock, kTile, kPlanThreads>(p, kMinTiles, ctas, starts, *gang);
}

// ---- the shared tokens

// 16 codes to fp16.
__device__ __forceinline__ void widen(const uint4& w, uint4& lo, uint4& hi) {
  lo.x = e4m3x2_to_f16x2((uint16_t)w.x), lo.y = e4m3x2_to_f16x2((uint16_t)(w.x >> 16));
  lo.z = e4m3x2_to_f16x2((uint16_t)w.y), lo.w = e4m3x2_to_f16x2((uint16_t)(w.y >> 16));
  hi.x = e4m3x2_to_f16x2((uint16_t)w.z), hi.y = e4m3x2_to_f16x2((uint16_t)(w.z >> 16));
  hi.z = e4m3x2_to_f16x2((uint16_t)w.w), hi.w = e4m3x2_to_f16x2((uint16_t)(w.w >> 16));
}

// A warp's 32 rows of Q (rows r0 .. r0 + 31 of `left`; the others zeros) as fp16 into their place: rows of 128
// bytes in atoms of 64 values, the 16-byte pieces of row r at their place XOR r % 8. Returns what a
// unit of the products of the lane's row stands for. The rows come as they are, all at once, by asynchronous
// copies, and are scaled in place, in loops of little code: this runs once a unit, from cold instruction
// caches (steps unrolled sixteen times took 14 us, a load a step 10).
template <int D, typename T>
__device__ __forceinline__ float load_q(const PrefixParams& p, const Segment& s, int r0, int left, unsigned char* to) {
  constexpr int kLanes = D / 8, kEach = 32 / kLanes;  // lanes of a row, rows a step
  const int lane = threadIdx.x & 31, piece = lane % kLanes, sub = lane / kLanes;
  const int j = s.block * kBlock + r0 + min(lane, max(left, 1) - 1), t = j / p.group;  // the lane's row
  const int64_t mine_at = (s.r.row0 + t) * p.a.q_row_stride + (int64_t)(s.kvh * p.group + j - t * p.group) * p.a.q_head_stride;
  unsigned char* const at = to + (piece >> 3) * Layout<D>::atom_bytes + (r0 & (kRows - 1)) * 128;
  auto place = [&](int r) { return at + r * 128 + ((piece & 7) ^ (r & 7)) * 16; };
#pragma unroll 4
  for (int r = sub; r < 32; r += kEach)
    copy16(place(r), static_cast<const char*>(p.a.q) + __shfl_sync(0xffffffffu, mine_at, r) + piece * 16, r < left);
  copies_commit();
  copies_wait<0>();  // a lane scales what it has copied itself
  float mine = 0.f;
#pragma unroll 2
  for (int r = sub; r < 32; r += kEach) {
    uint4* const here = reinterpret_cast<uint4*>(place(r));
    const uint4 w = *here;
    const uint32_t sign = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & sign, w.y & sign), __vmaxu2(w.z & sign, w.w & sign));
    uint32_t top = max(m >> 16, m & 0xFFFFu);  // the largest magnitude of the row, as bits
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // its exponent field as a float; both factors stay normal
    const int e = min(max((int)(__float_as_uint(unpack<T>(top).x) >> 23), 15), 254);
    const float by = __uint_as_float((uint32_t)(268 - e) << 23), back = not_finite<T>(top) ? NAN : __uint_as_float((uint32_t)(e - 14) << 23);
    const float f = __shfl_sync(0xffffffffu, back, lane % kEach * kLanes);  // to the lane whose row it is
    if (lane / kEach == r / kEach) mine = f;
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 v = unpack<T>(x[c]);
      x[c] = f16x2(v.x * by, v.y * by);
    }
    *here = make_uint4(x[0], x[1], x[2], x[3]);
  }
  return mine;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1) k_prefix(const __grid_constant__ PrefixParams p, const __grid_constant__ CUtensorMap k_map,
                                                        const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<D>;
  extern __shared__ unsigned char raw_smem[];
  unsigned char* sm = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  Shared& x = *reinterpret_cast<Shared*>(sm + L::off_x);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kIssue = 8 + kConvert;  // the warp that issues the products
  int4 desc = make_int4(-1, 0, 0, 0);
  grid_wait();
  grid_launch();  // behind the wait: a CTA of the next kernel reads the plan without one
  if (!Share::any(p)) {
    if (tid == 0) p.desc[blockIdx.x] = desc;
    return;
  }
  if (warp == kIssue) tmem_alloc(&x.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < L::k_stages; ++i) {
      mbar_init(&x.k_full[i], kConvert / 2);
      mbar_init(&x.k_empty[i], 1);
    }
    for (int i = 0; i < L::v_halves; ++i) {
      mbar_init(&x.v_full[i], kConvert / 2);
      mbar_init(&x.v_empty[i], 1);
    }
    for (int i = 0; i < kArrive; ++i) mbar_init(&x.raw_full[i], 1);
    for (int i = 0; i < L::units; ++i) mbar_init(&x.raw_empty[i], kConvert / 2);
    for (int i = 0; i < kMeta; ++i) mbar_init(&x.meta_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x.s_full[i], 1);
      mbar_init(&x.p_full[i], 4);
      mbar_init(&x.o_done[i], 1);
    }
    mbar_init(&x.q_full, 8);
    mbar_init(&x.q_empty, 1);
    x.stop = 0;
    x.wait_cycles = p.wait_cycles;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = x.tmem;
  // every role walks the line by itself: what lives through the change of registers is spilled
  if (warp >= kIssue) {
    set_regs<kIssueRegs, false>();
    if (warp == kIssue) {
      Share line(p);
      Segment s;
      // ---- the products. Tiles are counted through the CTA's units; tile i is in stage i % k_stages, its
      // halves of V in those of 2 i and 2 i + 1 % v_halves.
      const uint32_t leader = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = desc_lo(smem_u32(sm), 16), k_lo = desc_lo(smem_u32(sm) + L::off_k, 16);
      const uint32_t v_lo = desc_lo(smem_u32(sm) + L::off_v, L::atom_bytes / 2), hi = desc_hi(1024, kSwizzle128);
      uint32_t i = 0, u = 0, jobs0 = 0, jobs1 = 0;
      auto scores = [&](int slot, uint32_t t, bool last) {  // of tile t; last: of those that read it
        const int st = t % L::k_stages;
        wait(&x.k_full[st], t / L::k_stages & 1, &x.stop);
        __syncwarp();
        tc_fence_after();
        const uint32_t d = tm + slot * kTile, a = q_lo + slot * (L::tile_bytes / 16), b = k_lo + st * (L::tile_bytes / 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (k >> 2) * (L::atom_bytes / 16) + (k & 3) * 2;
          mma_f16(leader, d, a + at, hi, b + at, hi, f16_idesc(kRows, kTile, false), k > 0);
        }
        mma_commit(leader, &x.s_full[slot]);
        if (last) mma_commit(leader, &x.k_empty[st]);
      };
      auto outputs = [&](int slot, uint32_t t, bool fresh, bool last) {
        const uint32_t jobs = slot ? jobs1++ : jobs0++;
        const uint32_t d = tm + L::col_o + slot * D, a = tm + slot * kTile;
        wait(&x.p_full[slot], jobs & 1, &x.stop);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t h = 2 * t + half, st = h % L::v_halves;
          wait(&x.v_full[st], h / L::v_halves & 1, &x.stop);
          __syncwarp();
          tc_fence_after();
          const uint32_t b = v_lo + st * (L::tile_bytes / 32);
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma_f16_ts(leader, d, a + half * (kTile / 4) + k * 8, b + k * (16 * 128 / 16), hi, f16_idesc(kRows, D, true), !fresh || half > 0 || k > 0);
          if (last) mma_commit(leader, &x.v_empty[st]);
        }
        mma_commit(leader, &x.o_done[slot]);
      };
#pragma unroll 1
      while (line.next(p, s)) {
        // the same for every lane, as the compiler is to see
        const int n = __shfl_sync(0xffffffffu, s.t1 - s.t0, 0);
        const bool wide = __shfl_sync(0xffffffffu, s.rows, 0) > kRows;
        wait(&x.q_full, u & 1, &x.stop);
        __syncwarp();
        if (wide) {
          scores(0, i, false);
          scores(1, i, true);
#pragma unroll 1
          for (int j = 0; j < n; ++j, ++i) {
            outputs(0, i, j == 0, false);
            if (j + 1 < n) scores(0, i + 1, false);
            outputs(1, i, j == 0, true);
            if (j + 1 < n) scores(1, i + 1, true);
          }
        } else {  // tiles in turn
          scores(0, i, true);
          if (n > 1) scores(1, i + 1, true);
#pragma unroll 1
          for (int j = 0; j < n; j += 2) {
            outputs(0, i + j, j == 0, true);
            if (j + 2 < n) scores(0, i + j + 2, true);
            if (j + 1 < n) outputs(1, i + j + 1, j == 0, true);
            if (j + 3 < n) scores(1, i + j + 3, true);
          }
          i += n;
        }
        mma_commit(leader, &x.q_empty);
        ++u;
      }
    } else if (warp == kIssue + 1) {
      Share line(p);
      Segment s;
      // ---- loads: lanes hold a tile's pages and bring them, K and V in turn; page numbers come four
      // tiles ahead, scales one.
      struct Tile {
        int32_t page = -1;
        int kvh = 0;
        bool is = false;
      };
      const int per_tile = kTile >> p.page_shift, page_bytes = D << p.page_shift;
      const int32_t outside = (int32_t)max(p.c.num_pages, (int64_t)1);  // reads as zeros
      int j = 0;
      const int32_t* table = nullptr;
      bool more = line.next(p, s);
      if (more) table = p.c.page_table + (int64_t)p.groups[s.b].w * p.c.ld_table;
      auto next_tile = [&]() {
        Tile t;
        if (!more) return t;
        t.is = true;
        t.kvh = s.kvh;
        const int at = (s.t0 + j) * per_tile + lane;
        if (lane < per_tile && at << p.page_shift < s.r.len) {
          const int32_t id = table[at];
          if (id >= 0 && id < p.c.num_pages) t.page = id;
        }
        if (++j == s.t1 - s.t0) {
          j = 0;
          more = line.next(p, s);
          if (more) table = p.c.page_table + (int64_t)p.groups[s.b].w * p.c.ld_table;
        }
        return t;
      };
      float ks, vs;
      auto fetch_scales = [&](const Tile& t) {
        ks = vs = 0.f;
        if (t.page < 0) return;
        const int64_t at = (int64_t)t.page * p.c.heads + t.kvh;
        ks = __ldg(p.c.k_scale + at);
        vs = __ldg(p.c.v_scale + at);
      };
      auto to_l2 = [&](const Tile& t) {
        if (t.page < 0) return;
        tma_prefetch_4d(&k_map, 0, 0, t.kvh, t.page);
        tma_prefetch_4d(&v_map, 0, 0, t.kvh, t.page);
      };
      // shared memory has room for a tile and a half on its way, which at DRAM's latency is a third of its rate:
      // the tiles behind are on their way to L2
      Tile now = next_tile(), then, third, fourth;
      fetch_scales(now);
      uint32_t i = 0;
#pragma unroll 1
      while (now.is) {
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          const uint32_t n = 2 * i + v, st = n % L::units;
          wait(&x.raw_empty[st], (n / L::units & 1) ^ 1, &x.stop);
          if (!__any_sync(0xffffffffu, stopped(&x.stop))) {  // one answer a warp: its lanes meet inside
            if (lane == 0) mbar_arrive_expect_tx(&x.raw_full[n % kArrive], L::unit_bytes);
            __syncwarp();
            if (lane < per_tile)
              tma_load_4d(sm + L::off_raw + st * L::unit_bytes + lane * page_bytes, v ? &v_map : &k_map, 0, 0, now.kvh,
                          now.page >= 0 ? now.page : outside, &x.raw_full[n % kArrive]);
          }
        }
        // the scales' place was last read kMeta tiles ago: the products of later tiles have been issued since
        const bool all = __all_sync(0xffffffffu, lane >= per_tile || now.page >= 0);
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
        if (now.page >= 0) {
          g.x = ks;
          vs = scale_of_v(vs, g.x);
          g.y = __log2f(vs), g.z = 1.f / vs, g.w = all ? 2.f : 1.f;
        }
        if (lane < per_tile)
          for (int k = 0; k < 8 / per_tile; ++k) x.meta[i % kMeta][lane * (8 / per_tile) + k] = g;
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.meta_full[i % kMeta]);
        if (i == 0) {  // behind the first loads
          then = next_tile();
          third = next_tile();
          fourth = next_tile();
          to_l2(then);
          to_l2(third);
        }
        to_l2(fourth);
        now = then;
        then = third;
        third = fourth;
        fourth = next_tile();
        fetch_scales(now);
        ++i;
      }
    }
  } else if (warp >= 8) {
    set_regs<kConvertRegs, false>();
    Share line(p);
    Segment s;
    // ---- codes to fp16, 16 a step of a thread; half of the warps K, half V, so that neither waits for the other
    constexpr int kPer = D / 16, kStep = kConvert / 2 * 32 / kPer;  // pieces of a token, tokens a step
    const bool is_v = warp >= 8 + kConvert / 2;
    const int ct = tid - 256 - (is_v ? kConvert / 2 * 32 : 0), piece = ct % kPer, tok = ct / kPer, atom = piece >> 2;
    // the second atom's lanes store their halves the other way round: no two at one bank
    const int chunk = (piece & 3) * 2 + (atom & 1);
    const int swizzled = (chunk ^ (tok & 7)) * 16;  // steps are multiples of 8 tokens
    // 64 tokens of a unit into an array of rows of 128 bytes; all loads are in flight at once
    auto widen_half = [&](const unsigned char* from, unsigned char* to, int atom_bytes) {
      constexpr int N = kTile / 2 / kStep;
      const unsigned char* a = from + tok * D + piece * 16;
      unsigned char* b = to + atom * atom_bytes + tok * 128;
      uint4 w[N];
#pragma unroll
      for (int e = 0; e < N; ++e) w[e] = *reinterpret_cast<const uint4*>(a + e * kStep * D);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        uint4 lo, hi;
        widen(w[e], lo, hi);
        *reinterpret_cast<uint4*>(b + e * kStep * 128 + swizzled) = atom & 1 ? hi : lo;
        *reinterpret_cast<uint4*>(b + e * kStep * 128 + (swizzled ^ 16)) = atom & 1 ? lo : hi;
      }
    };
    uint32_t i = 0;
#pragma unroll 1
    while (line.next(p, s)) {
#pragma unroll 1
      for (int j = s.t0; j < s.t1; ++j, ++i) {
        const uint32_t n = 2 * i + (is_v ? 1 : 0), st = n % L::units;
        const unsigned char* raw = sm + L::off_raw + st * L::unit_bytes;
        wait(&x.raw_full[n % kArrive], n / kArrive & 1, &x.stop);
        if (!is_v) {
          const uint32_t k = i % L::k_stages;
          wait(&x.k_empty[k], (i / L::k_stages & 1) ^ 1, &x.stop);
          __syncwarp();
#pragma unroll 1
          for (int half = 0; half < 2; ++half)
            widen_half(raw + half * (L::unit_bytes / 2), sm + L::off_k + k * L::tile_bytes + half * (L::atom_bytes / 2), L::atom_bytes);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.k_full[k]);
        } else {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint32_t h = 2 * i + half, v = h % L::v_halves;
            wait(&x.v_empty[v], (h / L::v_halves & 1) ^ 1, &x.stop);
            __syncwarp();
            widen_half(raw + half * (L::unit_bytes / 2), sm + L::off_v + v * (L::tile_bytes / 2), L::atom_bytes / 2);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.v_full[v]);
          }
        }
        if (lane == 0) mbar_arrive(&x.raw_empty[st]);
      }
    }
  } else {
    set_regs<kSoftmaxRegs, true>();
    Share line(p);
    Segment s;
    // ---- softmax: a thread is a row of its slot
    const int slot = warp >> 2, r = tid & (kRows - 1);
    const uint32_t quarter = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's lanes
    const uint32_t my_s = quarter + slot * kTile, my_o = quarter + L::col_o + slot * D;
    uint32_t i0 = 0, u = 0, jobs = 0;
#pragma unroll 1
    while (line.next(p, s)) {
      const int n = s.t1 - s.t0;
      const bool wide = s.rows > kRows;
      const int row = wide ? slot * kRows + r : r;  // of the block
      const int step = wide ? 1 : 2, j0 = wide ? 0 : slot;
      const bool mine = row < s.rows;
      const bool active = (wide ? slot * kRows : 0) + (warp & 3) * 32 < s.rows;  // any row of the warp
      const int64_t at = mine ? s.at(p, kBlock, row) : 0;
      wait(&x.q_empty, (u & 1) ^ 1, &x.stop);
      __syncwarp();
      const int r0 = row - lane;  // the warp's first row
      const float fac = load_q<D, T>(p, s, r0, s.rows - r0, sm + slot * L::tile_bytes) * p.scale_log2;
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.q_full);
      float m = fac == fac ? kNone : 0.f, l = 0.f;  // a row whose q is not finite asks for nothing
      const uint32_t before = jobs;
#pragma unroll 1
      for (int j = j0; j < n; j += step, ++jobs) {
        const uint32_t i = i0 + j;
        wait(&x.meta_full[i % kMeta], i / kMeta & 1, &x.stop);
        wait(&x.s_full[slot], jobs & 1, &x.stop);
        __syncwarp();
        tc_fence_after();
        const float4* meta = x.meta[i % kMeta];
        if (active) {
          // The tile's probabilities with the reference as it is, kept in registers; their sum tells whether one
          // was too far above it. Before the unit's first tile, its second, fifth, 17th and so on a row looks at its
          // largest score and moves its reference up to it, so that rows hardly ever have to in between, where each
          // holds up its neighbours (document of 131071 tokens: 1121 us without, 876 if none ever moved). What a row
          // does is its own affair: its result does not depend on its neighbours.
          uint32_t w[kTile / 2];
          float part = 0.f;  // the tile's probabilities, each over its scale of V
          const uint32_t nth = jobs - before;
          const bool partial = !__all_sync(0xffffffffu, meta[0].w == 2.f);  // pages that are not there
          bool look = partial || ((nth & (nth - 1)) == 0 && (nth & 0x55555555u) == nth), may = look, stored = false;
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            if (look) {
              float top = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < kTile; c += 16) {
                const float4 g = meta[c / 16];
                if (g.w == 0.f) continue;  // the same for every thread
                float y[16], z[4];
                tmem_ld16(my_s + c, y);
                tmem_wait_ld();
                tmem_tie16(y);
                const float a = fac * g.x;
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e & 3] = e < 4 ? fmaf(y[e], a, g.y) : fmaxf(z[e & 3], fmaf(y[e], a, g.y));
                top = fmaxf(top, fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
              }
              const float head = fminf(fmaxf((float)(26 - __clz(n)), kLeastHead), kMostHead);  // of 128 n tokens
              const float to = may && top > m + (head + 1.f) ? top - head : m, by = ex2(m - to);
              const bool moves = to != m;
              m = to;
              if (__any_sync(0xffffffffu, moves) && nth > 0) {
                l *= by;
                wait(&x.o_done[slot], (jobs - 1) & 1, &x.stop);
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  float o[16];
                  tmem_ld16(my_o + c, o);
                  tmem_wait_ld();
                  tmem_tie16(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] *= by;
                  tmem_st16(my_o + c, reinterpret_cast<const uint32_t*>(o));
                }
              }
            }
            const bool far = !(fabsf(m) <= kMostRef);
            part = 0.f;
            if (partial || __any_sync(0xffffffffu, far && pass > 0)) {
              // Scores are rounded before a far reference is subtracted: the difference stays small, however large
              // both are. The sums' order is that of the other way.
#pragma unroll 1
              for (int c = 0; c < kTile; c += 16) {
                const float4 g = meta[c / 16];
                float y[16];
                tmem_ld16(my_s + c, y);
                tmem_wait_ld();
                tmem_tie16(y);
                const bool there = g.w != 0.f;
                const float a = fac * g.x, b = far ? g.y : g.y - m, less = far ? m : 0.f;
                f32x2 sum[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float e0 = there ? ex2(fmaf(y[2 * e], a, b) - less) : 0.f;
                  const float e1 = there ? ex2(fmaf(y[2 * e + 1], a, b) - less) : 0.f;
                  sum[e & 1] = add2(sum[e & 1], pair(e0, e1));
                  w[e] = f16x2(e0, e1);
                }
                tmem_st8(my_s + c / 2, reinterpret_cast<const float*>(w));  // P over the scores that have been read
                const float2 both = unpair(add2(sum[0], sum[1]));
                if (there) part = fmaf(both.x + both.y, g.z, part);
              }
              stored = true;
              break;
            }
            float all = 0.f, y[2][16];
            tmem_ld16(my_s, y[0]);
#pragma unroll
            for (int c = 0; c < kTile / 16; ++c) {
              const float4 g = meta[c];
              const f32x2 a = pair(fac * g.x, fac * g.x), b = pair(g.y - m, g.y - m);
              tmem_wait_ld();
              tmem_tie16(y[c & 1]);
              if (c + 1 < kTile / 16) tmem_ld16(my_s + (c + 1) * 16, y[(c + 1) & 1]);
              const float* v = y[c & 1];
              f32x2 sum[2] = {0, 0};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 z = unpair(fma2(pair(v[2 * e], v[2 * e + 1]), a, b));
                const float e0 = ex2(z.x), e1 = ex2(z.y);
                sum[e & 1] = add2(sum[e & 1], pair(e0, e1));
                w[8 * c + e] = f16x2(e0, e1);
              }
              const float2 both = unpair(add2(sum[0], sum[1]));
              all += both.x + both.y;
              part = fmaf(both.x + both.y, g.z, part);
            }
            may = all > kMostSum || far;
            look = true;
            if (!__any_sync(0xffffffffu, may)) break;
          }
          if (!stored) {
#pragma unroll
            for (int c = 0; c < kTile / 2; c += 16) tmem_st16(my_s + c, w + c);
          }
          l += part;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.p_full[slot]);
      }
      // ---- the end of the unit
      const bool live = jobs != before;
      if (live) wait(&x.o_done[slot], (jobs - 1) & 1, &x.stop);
      __syncwarp();
      tc_fence_after();
      const bool whole = s.whole();
      float* part = p.part + (2 * (int64_t)blockIdx.x + (s.t0 == 0 ? 1 : 0)) * slot_floats(kBlock, D);
      float by = 1.f;
      if (!wide) {  // the slots meet, when the last scores of both are formed and Q has been read
        bar_sync(1, 256);
        float2* ml = reinterpret_cast<float2*>(sm);
        ml[slot * kRows + r] = make_float2(m, l);
        bar_sync(1, 256);
        const float2 other = ml[(slot ^ 1) * kRows + r];
        const float top = fmaxf(m, other.x);
        by = live ? ex2(m - top) : 0.f;
        l = fmaf(l, by, other.y * ex2(other.x - top));
        m = top;
        bar_sync(1, 256);
      }
      if (mine && (wide || slot == 0)) {
        if (whole) p.pre_ml[at] = make_float2(m, l);
        else part[kBlock * D + row] = m, part[kBlock * D + kBlock + row] = l;
      }
      // Outputs pass through the place of Q, half of the columns at a time, so that rows are written in runs. A
      // row's 16-byte pieces lie where its Q lies, at their place XOR the row: a warp that is done loads the next
      // unit's Q over its own rows' alone, while its neighbours still write. Where the slots meet, each hands the
      // other one half and adds that up.
      constexpr int kHalf = D / 2, kPieces = kHalf / 4;
      const int target = mine && (wide || row < s.rows) ? (whole ? (int)at : row) : -1;
      float* const base = whole ? p.pre_o : part;
      static_assert(kPieces <= 8 * L::atoms, "a row's pieces where its Q is");
      auto piece_of = [&](int region, int rr, int piece) {
        return reinterpret_cast<float4*>(sm + region * L::tile_bytes + (piece >> 3) * L::atom_bytes + rr * 128) + ((piece ^ rr) & 7);
      };
      auto pour = [&](int half, int region, bool add) {
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 16) {
          float o[16];
          if (live) {
            tmem_ld16(my_o + half * kHalf + c, o);
            tmem_wait_ld();
            tmem_tie16(o);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float4* at4 = piece_of(region, r, c / 4 + e);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (add) y = *at4;
            if (live) y = make_float4(fmaf(o[4 * e], by, y.x), fmaf(o[4 * e + 1], by, y.y), fmaf(o[4 * e + 2], by, y.z), fmaf(o[4 * e + 3], by, y.w));
            *at4 = y;
          }
        }
      };
      auto write = [&](int half, int region) {
        __syncwarp();
#pragma unroll 4
        for (int k = lane; k < 32 * kPieces; k += 32) {
          const int rr = k / kPieces, piece = k % kPieces, to = __shfl_sync(0xffffffffu, target, rr);
          if (to >= 0) *reinterpret_cast<float4*>(base + (int64_t)to * D + half * kHalf + piece * 4) = *piece_of(region, r - lane + rr, piece);
        }
        __syncwarp();
      };
      if (!wide) {
        pour(slot ^ 1, slot ^ 1, false);
        bar_sync(1, 256);
      }
#pragma unroll 1
      for (int half = wide ? 0 : slot; half < (wide ? 2 : slot + 1); ++half) {
        pour(half, slot, !wide);
        write(half, slot);
      }
      if (!wide) bar_sync(1, 256);  // before the next unit's Q
      tc_fence_before();
      if (!whole) {
        if (s.t0 == 0) {
          desc.x = s.b;
          desc.y = s.kvh;
          desc.z = s.rows;
          desc.w |= s.block << 1;
        } else {
          desc.w |= s.t1 == s.r.tiles ? 1 : 0;
        }
      }
      i0 += n;
      ++u;
    }
    if (tid == 0) p.desc[blockIdx.x] = desc;
  }
  if (stopped(&x.stop)) {
    atomicOr(&g_prefix_error, 1u);
    // products in flight are done before the CTA leaves its memory
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 26)) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssue) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// The rows of a unit that spans CTAs, as join_row, into their prefix part: a warp takes every
// kJoinY * kJoinWarps-th.
constexpr int kJoinWarps = 8, kJoinY = 16;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_prefix_join(const __grid_constant__ PrefixParams p, const __grid_constant__ TailParams tail,
                                                                 int tail_ctas, int rows, Start* starts) {
  grid_launch();
  if (blockIdx.y == kJoinY) {  // one CTA, the last to find room: the shares of the kernel behind this one
    if (blockIdx.x == 0) {
      if (rows == 16) line_starts<16, kTailTile, kJoinWarps * 32>(tail, kTailLeast, tail_ctas, starts);
      else line_starts<32, kTailTile, kJoinWarps * 32>(tail, kTailLeast, tail_ctas, starts);
    }
    grid_wait();
    return;
  }
  grid_wait();
  const int first = blockIdx.x, lane = threadIdx.x & 31;
  const int4 d = p.desc[first];
  if (d.x < 0) return;
  const int gang = *p.gang;  // the pieces' CTAs are this far apart
  int pieces = 1;
  for (;; pieces += 32) {
    const int i = first + (pieces + lane) * gang;
    const unsigned ends = __ballot_sync(0xffffffffu, i >= (int)gridDim.x || (p.desc[i].w & 1));
    if (ends) {
      pieces += __ffs(ends);
      break;
    }
  }
  Segment s;
  s.r = request<kBlock, kTile>(p, raw_request(p, d.x));
  s.kvh = d.y;
  s.block = d.w >> 1;
  auto piece = [&](int i) { return p.part + (int64_t)(i ? 2 * (first + i * gang) : 2 * first + 1) * slot_floats(kBlock, D); };
  for (int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); row < d.z; row += kJoinY * kJoinWarps) {
    float top = kNone;
    for (int i = lane; i < pieces; i += 32) top = fmaxf(top, piece(i)[kBlock * D + row]);
    top = warp_max(top);
    constexpr int PER = D / 32;
    float2 acc[PER / 2];
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) acc[e] = make_float2(0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const float* y = piece(i);
      const float by = ex2(y[kBlock * D + row] - top);
      sum = fmaf(by, y[kBlock * D + kBlock + row], sum);
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) add_scaled(acc[e], by, *reinterpret_cast<const float2*>(y + row * D + lane * PER + 2 * e));
    }
    const int64_t at = s.at(p, kBlock, row);
    if (lane == 0) p.pre_ml[at] = make_float2(top, sum);
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) *reinterpret_cast<float2*>(p.pre_o + at * D + lane * PER + 2 * e) = acc[e];
  }
}

template <int D, typename T>
cudaError_t launch(const PrefixParams& p, const CUtensorMap& k, const CUtensorMap& v, const TailParams& tail, Start* starts, int sms,
                   cudaStream_t s) {
  constexpr int bytes = smem_bytes<D>();
  cudaError_t e = allow_smem<k_prefix<D, T>>(bytes);
  if (e != cudaSuccess) return e;
  if ((e = launch_after(k_prefix<D, T>, dim3(sms), kThreads, bytes, s, p, k, v)) != cudaSuccess) return e;
  return launch_after(k_prefix_join<D>, dim3(sms, kJoinY + 1), kJoinWarps * 32, 0, s, p, tail, sms * tail_ctas(tail_rows(tail)), tail_rows(tail), starts);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Scratch {
  int4* groups;
  int32_t* gang;
  int32_t* first;
  Start *starts, *tails;
  float* pre_o;
  float2* pre_ml;
  int4* desc;
  float* part;
  char* tail;  // the workspace of what is left
};

size_t lay_out(Scratch& x, int64_t batch, int64_t groups, int64_t total_rows, int heads_q, int heads, int D, int sms, void* ws) {
  size_t off = 0;
  auto take = [&](auto*& at, size_t n) {
    at = reinterpret_cast<std::remove_reference_t<decltype(at)>>(static_cast<char*>(ws) + off);
    off += up256(n * sizeof(*at));
  };
  const size_t rows = (size_t)total_rows * heads_q;
  take(x.groups, (size_t)groups);
  take(x.gang, 1);
  take(x.first, (size_t)batch);
  take(x.starts, (size_t)sms);
  take(x.tails, (size_t)sms * tail_ctas(16));
  take(x.pre_o, rows * D);
  take(x.pre_ml, rows);
  take(x.desc, (size_t)sms);
  take(x.part, (size_t)2 * sms * slot_floats(kBlock, D));
  take(x.tail, tail_workspace(batch, total_rows, heads_q, heads, D, sms));
  return off;
}

}  // namespace

size_t shared_workspace(int64_t batch, int64_t groups, int64_t total_rows, int heads_q, int heads, int head_dim, int sms) {
  Scratch x;
  return lay_out(x, batch, groups, total_rows, heads_q, heads, head_dim, sms, nullptr);
}

cudaError_t shared_read_error(uint32_t* word, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_prefix_error, sizeof(uint32_t));
  if (e == cudaSuccess && clear && *word) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_prefix_error, &zero, sizeof(zero));
  }
  return e;
}

cudaError_t launch_shared(const ts_shared_args& sh, void* ws, int sms, uint64_t wait_cycles, cudaStream_t s) {
  const ts_attn_args& a = *sh.attn;
  const ts_kv_cache& c = *a.cache;
  Scratch x;
  lay_out(x, c.batch, sh.groups, a.total_rows, a.heads_q, c.heads, c.head_dim, sms, ws);
  PrefixParams p{};
  p.c = c;
  p.c.batch = sh.groups;
  p.a = a;
  p.page_shift = __builtin_ctz((unsigned)c.page_size);
  p.group = a.heads_q / c.heads;
  p.scale_log2 = a.sm_scale * kLog2e;
  p.groups = x.groups;
  p.gang = x.gang;
  p.part = x.part;
  p.desc = x.desc;
  p.pre_o = x.pre_o;
  p.pre_ml = x.pre_ml;
  p.wait_cycles = wait_cycles;
  p.starts = x.starts;
  TailParams tail = tail_params(c, a, x.tail, sms);
  tail.first = x.first;
  tail.pre_o = x.pre_o;
  tail.pre_ml = x.pre_ml;
  tail.starts = x.tails;
  CUtensorMap k, v;  // before anything is launched: a call that fails leaves nothing on the stream
  if (!page_map(&k, c, c.k, c.k_page_stride, c.k_head_stride, c.k_token_stride, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !page_map(&v, c, c.v, c.v_page_stride, c.v_head_stride, c.v_token_stride, CU_TENSOR_MAP_SWIZZLE_NONE))
    return encoder_found() ? cudaErrorInvalidValue : cudaErrorNotSupported;
  k_plan<<<1, kPlanThreads, 0, s>>>(p, c, sh, x.groups, x.first, x.gang, x.starts, sms);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.dtype == TS_BF16)
    e = c.head_dim == 128 ? launch<128, __nv_bfloat16>(p, k, v, tail, x.tails, sms, s) : launch<64, __nv_bfloat16>(p, k, v, tail, x.tails, sms, s);
  else
    e = c.head_dim == 128 ? launch<128, __half>(p, k, v, tail, x.tails, sms, s) : launch<64, __half>(p, k, v, tail, x.tails, sms, s);
  return e != cudaSuccess ? e : launch_tail(tail, sms, s);
}

}  // namespace tsv
