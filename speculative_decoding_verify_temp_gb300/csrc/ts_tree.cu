// Verification of drafted trees against the target's probabilities with given coins.
//
// One cluster a request. Every CTA of it repeats the walk (a few hundred bytes, one round of
// loads for the nodes and one for their probabilities): the tests of all nodes are formed at
// once, since a node's test does not depend on the path, only on its earlier siblings; the
// path then follows each node's first child that passes. The row of the path's end is split
// over the CTAs, whose warps sum contiguous runs of it; the sums meet through distributed
// shared memory and the CTA that owns the crossing reads its run again (from L2).
//
// Sums are pairs of fp32 numbers (a value and the rounding errors carried along, Knuth's
// TwoSum), good to about 2^-46: the double-precision units have about a sixtieth of the fp32
// rate and several times its latency, and with them the scans and the search took longer than
// the row's reading (33 us for 64 trees of vocabulary 128256, 18 now; 256 trees of 151936: 43 us,
// 3.6 TB/s). Only a node's test is formed in double, a few operations a node.
#include <stdint.h>

#include <cooperative_groups.h>

#include "../../include/ts_verify.h"
#include "ts_common.cuh"
#include "ts_internal.h"

namespace tsv {

namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kTreeMaxCluster = 8;
constexpr int kTreeCtasPerSm = 4;
constexpr int kMarkBits = 2048;  // filter of the vectors that hold a removed token

// A sum: h + l, |l| at most half a step of h.
struct alignas(8) Sum {
  float h, l;
};

__device__ __forceinline__ Sum operator+(Sum a, Sum b) {
  const float s = __fadd_rn(a.h, b.h), z = __fsub_rn(s, a.h);
  const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.h, __fsub_rn(s, z)), __fsub_rn(b.h, z)), __fadd_rn(a.l, b.l));
  const float h = __fadd_rn(s, e);
  return {h, __fsub_rn(e, __fsub_rn(h, s))};
}
__device__ __forceinline__ Sum operator*(float u, Sum a) {
  const float p = __fmul_rn(u, a.h), e = __fmaf_rn(u, a.h, -p);
  return Sum{p, 0.f} + Sum{__fmaf_rn(u, a.l, e), 0.f};
}
__device__ __forceinline__ bool operator>(Sum a, Sum b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }

__device__ __forceinline__ Sum shuffle(Sum v, int from) {
  return {__shfl_sync(0xffffffffu, v.h, from), __shfl_sync(0xffffffffu, v.l, from)};
}

__device__ __forceinline__ Sum warp_sum(Sum v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = v + Sum{__shfl_xor_sync(0xffffffffu, v.h, o), __shfl_xor_sync(0xffffffffu, v.l, o)};
  return v;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ Sum warp_scan(Sum v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum t = {__shfl_up_sync(0xffffffffu, v.h, o), __shfl_up_sync(0xffffffffu, v.l, o)};
    if (lane >= o) v = t + v;
  }
  return v;
}

struct TreeShared {
  int32_t parent[TS_MAX_WINDOW], token[TS_MAX_WINDOW], next[TS_MAX_WINDOW], path[TS_MAX_WINDOW + 1];
  double px[TS_MAX_WINDOW];
  int32_t removed[TS_MAX_WINDOW];
  int32_t n_removed, kept, limited;
  uint32_t mark[kMarkBits / 32];
  Sum sums[kTreeMaxCluster * kTreeWarps];  // every warp's sum over the cluster
  Sum mine[kTreeWarps];
  Sum part[kTreeWarps];
  int32_t found;
};

// s + e += x, the error of s kept in e (Knuth's TwoSum).
__device__ __forceinline__ void two_add(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

template <bool VEC>
__global__ void __launch_bounds__(kTreeThreads, kTreeCtasPerSm) k_tree(ts_tree_args a) {
  __shared__ TreeShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int64_t b = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t R = a.D + 1;
  int64_t row0;
  int n;
  if (a.qo_indptr) {
    row0 = a.qo_indptr[b];
    const int64_t r1 = a.qo_indptr[b + 1];
    n = row0 >= 0 && r1 <= a.total_rows && r1 > row0 && r1 - row0 <= TS_MAX_WINDOW ? (int)(r1 - row0) : 0;
  } else {
    n = (int)(a.total_rows / a.batch);
    row0 = b * n;
  }
  if (n == 0) {  // the same for the whole cluster
    if (rank == 0)
      for (int i = tid; i < R; i += kTreeThreads) {
        if (i == 0) a.accept_length[b] = 0;
        a.accepted_tokens[b * R + i] = -1;
        if (a.accept_index) a.accept_index[b * R + i] = -1;
        if (a.logprobs) a.logprobs[b * R + i] = 0.f;
      }
    return;
  }

  // 1. the nodes, each with its own probability under its parent
  float coin = 0.f;
  if (tid < n) {
    const int32_t p = a.parents[row0 + tid], x = a.tokens[row0 + tid];
    coin = a.uniforms[row0 + tid];
    const bool node = tid > 0 && p >= 0 && p < tid;
    const bool real = node && x >= 0 && (int64_t)x < a.vocab;
    sh.parent[tid] = node ? p : -1;
    sh.token[tid] = x;
    sh.next[tid] = -1;
    sh.px[tid] = real ? (double)a.target_probs[(row0 + p) * a.ld + x] : 0.0;
  }
  if (tid < kMarkBits / 32) sh.mark[tid] = 0;
  const float u_last = a.uniforms[row0];
  __syncthreads();

  // 2. its test, if its earlier siblings were all rejected; a token that one of them holds
  // has no mass left
  const int my_parent = tid < n ? sh.parent[tid] : -1;
  bool again = false;
  uint64_t before = 0;  // its earlier siblings (bit j - 1: node j)
  if (my_parent >= 0) {
#pragma unroll 8
    for (int j = 1; j < tid; ++j) {
      const bool sibling = sh.parent[j] == my_parent;
      before |= (uint64_t)sibling << (j - 1);
      again |= sibling && sh.token[j] == sh.token[tid];
    }
  }
  __syncthreads();
  if (again) sh.px[tid] = 0.0;
  __syncthreads();
  bool test = false;
  if (my_parent >= 0) {
    double gone = 0.0;
    for (; before; before &= before - 1) gone += sh.px[__ffsll(before)];
    test = __dmul_rn((double)coin, 1.0 - gone) < sh.px[tid];
  }
  // the first sibling that passes: the lowest row wins
  if (test) {
    int32_t* slot = &sh.next[sh.parent[tid]];
    int32_t cur = atomicCAS(slot, -1, tid);
    while (cur >= 0 && cur > tid) cur = atomicCAS(slot, cur, tid);
  }
  __syncthreads();

  // 3. the path, and the tokens rejected at its end
  if (tid == 0) {
    int node = 0, k = 0;
    sh.path[0] = 0;
    while (k < a.D && sh.next[node] >= 0) {
      node = sh.next[node];
      sh.path[++k] = node;
    }
    sh.kept = k + 1;
    sh.limited = k == a.D;
    sh.n_removed = 0;
    sh.found = -1;
  }
  __syncthreads();
  const int kept = sh.kept, end = sh.path[kept - 1];
  if (!sh.limited && tid < n && sh.parent[tid] == end && tid > 0) {
    const int32_t x = sh.token[tid];
    if (x >= 0 && (int64_t)x < a.vocab) {
      sh.removed[atomicAdd(&sh.n_removed, 1)] = x;
      const uint32_t v = (uint32_t)x / 4 % kMarkBits;
      atomicOr(&sh.mark[v / 32], 1u << (v % 32));
    }
  }
  __syncthreads();

  // 4. the masses of the warps' runs (in vectors of four tokens)
  const float* row = a.target_probs + (row0 + end) * a.ld;
  const int64_t vecs = (a.vocab + 3) / 4;
  const int64_t runs = (int64_t)ranks * kTreeWarps;
  const int64_t per = (vecs + runs - 1) / runs;
  auto load = [&](int64_t v, float* x) {
    const int64_t i = v * 4;
    if (VEC && i + 4 <= a.vocab) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(row + i));
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < a.vocab ? __ldg(row + i + e) : 0.f;
    }
  };
  int n_removed = sh.n_removed;
  auto drop = [&](int64_t v, float* x) {
    if (n_removed == 0) return;
    const uint32_t m = (uint32_t)(v % kMarkBits);
    if (!(sh.mark[m / 32] >> (m % 32) & 1u)) return;
    for (int k = 0; k < n_removed; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((int64_t)sh.removed[k] == v * 4 + e) x[e] = 0.f;
  };
  const Sum none = {0.f, 0.f};
  Sum total = none, w0 = none, w1 = none, upto = none;
  for (int round = 0; round < 2; ++round) {
    const int64_t lo = min(vecs, (rank * (int64_t)kTreeWarps + warp) * per), hi = min(vecs, lo + per);
    float s[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
    int64_t v = lo + lane;
    for (; v + 96 < hi; v += 128) {
      float x[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) load(v + 32 * k, x[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        drop(v + 32 * k, x[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) two_add(s[i], e[i], x[k][i]);
      }
    }
    for (; v < hi; v += 32) {
      float x[4];
      load(v, x);
      drop(v, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) two_add(s[i], e[i], x[i]);
    }
    const Sum mass = warp_sum((Sum{s[0], e[0]} + Sum{s[1], e[1]}) + (Sum{s[2], e[2]} + Sum{s[3], e[3]}));
    if (lane == 0) sh.mine[warp] = mass;
    cluster.sync();
    if (tid < runs) sh.sums[tid] = *cluster.map_shared_rank(&sh.mine[tid % kTreeWarps], tid / kTreeWarps);
    cluster.sync();  // all have read: the sums may be written again, or the CTA may leave
    // lane l of every warp: runs 2l and 2l + 1
    w0 = 2 * lane < runs ? sh.sums[2 * lane] : none;
    w1 = 2 * lane + 1 < runs ? sh.sums[2 * lane + 1] : none;
    upto = warp_scan(w0 + w1, lane);
    total = shuffle(upto, 31);
    if (total.h > 0.f || n_removed == 0) break;
    n_removed = 0;  // nothing is left without the rejected children: draw from p itself
  }

  // 5. the run that holds the crossing (without one, by rounding or a coin of 1: the last
  // run that has mass)
  const Sum want = u_last * total;
  const Sum before0 = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
  const Sum below0 = lane ? before0 : none, below1 = below0 + w0;
  const unsigned cross0 = __ballot_sync(0xffffffffu, w0.h > 0.f && below1 > want);
  const unsigned cross1 = __ballot_sync(0xffffffffu, w1.h > 0.f && upto > want);
  const unsigned mass0 = __ballot_sync(0xffffffffu, w0.h > 0.f), mass1 = __ballot_sync(0xffffffffu, w1.h > 0.f);
  int run = 0;
  if (cross0 | cross1) {
    const int l = __ffs(cross0 | cross1) - 1;
    run = 2 * l + (cross0 >> l & 1u ? 0 : 1);
  } else if (mass0 | mass1) {
    const int l = 31 - __clz(mass0 | mass1);
    run = 2 * l + (mass1 >> l & 1u ? 1 : 0);
  }
  const Sum below = shuffle(run & 1 ? below1 : below0, run >> 1);
  if (run / kTreeWarps != rank) return;

  // 6. the crossing within the run: a contiguous piece a thread
  const int64_t lo = min(vecs, run * per), hi = min(vecs, lo + per);
  const int64_t piece = (hi - lo + kTreeThreads - 1) / kTreeThreads;
  const int64_t plo = min(hi, lo + tid * piece), phi = min(hi, plo + piece);
  Sum mass = none;
  for (int64_t v = plo; v < phi; ++v) {
    float x[4];
    load(v, x);
    drop(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) two_add(mass.h, mass.l, x[i]);
  }
  mass = none + mass;
  const Sum in_warp = warp_scan(mass, lane);
  if (lane == 31) sh.part[warp] = in_warp;
  __syncthreads();
  Sum base = below;  // the mass before this thread's piece
  for (int w = 0; w < warp; ++w) base = base + sh.part[w];
  const Sum lanes = {__shfl_up_sync(0xffffffffu, in_warp.h, 1), __shfl_up_sync(0xffffffffu, in_warp.l, 1)};
  if (lane) base = base + lanes;
  const bool cross = mass.h > 0.f && base + mass > want;
  // the first piece that crosses; else the last one with mass
  const int first = __syncthreads_or(cross);
  if (first ? cross : mass.h > 0.f) {
    if (first) atomicMin(reinterpret_cast<uint32_t*>(&sh.found), (uint32_t)tid);
    else atomicMax(&sh.found, tid);
  }
  __syncthreads();
  if (sh.found < 0 ? tid == 0 : tid == sh.found) {
    int64_t token = a.vocab - 1;
    Sum acc = base;
    bool done = sh.found < 0;
    for (int64_t v = plo; v < phi && !done; ++v) {
      float x[4];
      load(v, x);
      drop(v, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = acc + Sum{x[i], 0.f};
        if (!done && x[i] > 0.f) {
          token = v * 4 + i;
          done = acc > want;
        }
      }
    }
    const int j = kept - 1;
    a.accepted_tokens[b * R + j] = (int32_t)token;
    if (a.logprobs) a.logprobs[b * R + j] = logf(row[token]);
  }
  // the rest of the outputs, by the same CTA
  for (int j = tid; j < R; j += kTreeThreads) {
    if (j == 0) a.accept_length[b] = kept;
    if (j != kept - 1) a.accepted_tokens[b * R + j] = j < kept - 1 ? sh.token[sh.path[j + 1]] : -1;
    if (a.accept_index) a.accept_index[b * R + j] = j < kept ? (int32_t)(row0 + sh.path[j]) : -1;
    if (a.logprobs && j != kept - 1)
      a.logprobs[b * R + j] = j < kept - 1 ? logf((float)sh.px[sh.path[j + 1]]) : 0.f;
  }
}

}  // namespace

cudaError_t launch_tree(const ts_tree_args& a, int sms, cudaStream_t s) {
  // CTAs a request: as many as run at once (256 trees of vocabulary 151936: 43 us with 2, 46
  // with 4 CTAs each; 64 of 128256: 18 us with 8, 27 with 2), runs of 16 vectors a lane or more
  int ranks = 1;
  while (ranks < kTreeMaxCluster && a.batch * ranks * 2 <= (int64_t)sms * kTreeCtasPerSm &&
         a.vocab > (int64_t)ranks * kTreeThreads * 4 * 4)
    ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.batch * ranks));
  cfg.blockDim = dim3(kTreeThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const bool vec = reinterpret_cast<uintptr_t>(a.target_probs) % 16 == 0 && a.ld % 4 == 0;
  return vec ? cudaLaunchKernelEx(&cfg, k_tree<true>, a) : cudaLaunchKernelEx(&cfg, k_tree<false>, a);
}

}  // namespace tsv
