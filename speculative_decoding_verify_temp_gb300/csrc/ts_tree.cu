// Verification of drafted trees against the target's probabilities with given coins.
//
// One cluster a request. Every CTA of it repeats the walk (a few hundred bytes, one round of
// loads for the nodes and one for their probabilities): the tests of all nodes are formed at
// once, since a node's test does not depend on the path, only on its earlier siblings; the
// path then follows each node's first child that passes. The row of the path's end is split
// over the CTAs, whose warps sum contiguous runs of it; the sums meet through distributed
// shared memory and the CTA that owns the crossing reads its run again (from L2).
//
// Sums: a lane adds its elements in fp32 with the rounding errors carried along (TwoSum), to
// about 2^-48 of its sum, and everything above a lane is double. Doubles throughout would be
// bound by the double-precision units, a sixty-fourth of the fp32 rate.
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
constexpr int kMarkBits = 2048;  // filter of the vectors that hold a removed token

struct TreeShared {
  int32_t parent[TS_MAX_WINDOW], token[TS_MAX_WINDOW], next[TS_MAX_WINDOW], path[TS_MAX_WINDOW + 1];
  double px[TS_MAX_WINDOW];
  int32_t removed[TS_MAX_WINDOW];
  int32_t n_removed, kept, limited;
  uint32_t mark[kMarkBits / 32];
  double sums[kTreeMaxCluster * kTreeWarps];  // every warp's sum over the cluster
  double mine[kTreeWarps];
  double part[kTreeWarps];
  int32_t found;
};

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ double warp_scan_f64(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// s + e += x, the error of s kept in e (Knuth's TwoSum).
__device__ __forceinline__ void two_add(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

template <bool VEC>
__global__ void __launch_bounds__(kTreeThreads) k_tree(ts_tree_args a) {
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
  const double u_last = (double)a.uniforms[row0];
  __syncthreads();

  // 2. its test, if its earlier siblings were all rejected; a token that one of them holds
  // has no mass left
  const int my_parent = tid < n ? sh.parent[tid] : -1;
  bool again = false;
  if (my_parent >= 0)
    for (int j = 1; j < tid; ++j) again |= sh.parent[j] == my_parent && sh.token[j] == sh.token[tid];
  __syncthreads();
  if (again) sh.px[tid] = 0.0;
  __syncthreads();
  bool test = false;
  if (my_parent >= 0) {
    double gone = 0.0;
    for (int j = 1; j < tid; ++j)
      if (sh.parent[j] == my_parent) gone += sh.px[j];
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
  double total = 0.0, w0 = 0.0, w1 = 0.0, upto = 0.0;
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
    double mass = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) mass += (double)s[i] + (double)e[i];
    mass = warp_sum_f64(mass);
    if (lane == 0) sh.mine[warp] = mass;
    cluster.sync();
    if (tid < runs) sh.sums[tid] = *cluster.map_shared_rank(&sh.mine[tid % kTreeWarps], tid / kTreeWarps);
    cluster.sync();  // all have read: the sums may be written again, or the CTA may leave
    // lane l of every warp: runs 2l and 2l + 1
    w0 = 2 * lane < runs ? sh.sums[2 * lane] : 0.0;
    w1 = 2 * lane + 1 < runs ? sh.sums[2 * lane + 1] : 0.0;
    upto = warp_scan_f64(w0 + w1, lane);
    total = __shfl_sync(0xffffffffu, upto, 31);
    if (total > 0.0 || n_removed == 0) break;
    n_removed = 0;  // nothing is left without the rejected children: draw from p itself
  }

  // 5. the run that holds the crossing (without one, by rounding or a coin of 1: the last
  // run that has mass)
  const double want = __dmul_rn(u_last, total);
  const double before1 = upto - w1, before0 = before1 - w0;
  const unsigned cross0 = __ballot_sync(0xffffffffu, w0 > 0.0 && before0 + w0 > want);
  const unsigned cross1 = __ballot_sync(0xffffffffu, w1 > 0.0 && upto > want);
  const unsigned mass0 = __ballot_sync(0xffffffffu, w0 > 0.0), mass1 = __ballot_sync(0xffffffffu, w1 > 0.0);
  int run = 0;
  if (cross0 | cross1) {
    const int l = __ffs(cross0 | cross1) - 1;
    run = 2 * l + (cross0 >> l & 1u ? 0 : 1);
  } else if (mass0 | mass1) {
    const int l = 31 - __clz(mass0 | mass1);
    run = 2 * l + (mass1 >> l & 1u ? 1 : 0);
  }
  const double below = __shfl_sync(0xffffffffu, run & 1 ? before1 : before0, run >> 1);
  if (run / kTreeWarps != rank) return;

  // 6. the crossing within the run: a contiguous piece a thread
  const int64_t lo = min(vecs, run * per), hi = min(vecs, lo + per);
  const int64_t piece = (hi - lo + kTreeThreads - 1) / kTreeThreads;
  const int64_t plo = min(hi, lo + tid * piece), phi = min(hi, plo + piece);
  double mass = 0.0;
  for (int64_t v = plo; v < phi; ++v) {
    float x[4];
    load(v, x);
    drop(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) mass += (double)x[i];
  }
  const double in_warp = warp_scan_f64(mass, lane);
  if (lane == 31) sh.part[warp] = in_warp;
  __syncthreads();
  double base = below;
#pragma unroll
  for (int w = 0; w < kTreeWarps; ++w) base += w < warp ? sh.part[w] : 0.0;
  base += in_warp - mass;
  const bool cross = mass > 0.0 && base + mass > want;
  // the first piece that crosses; else the last one with mass
  const int first = __syncthreads_or(cross);
  if (first ? cross : mass > 0.0) {
    if (first) atomicMin(reinterpret_cast<uint32_t*>(&sh.found), (uint32_t)tid);
    else atomicMax(&sh.found, tid);
  }
  __syncthreads();
  if (sh.found < 0 ? tid == 0 : tid == sh.found) {
    int64_t token = a.vocab - 1;
    double acc = base;
    bool done = sh.found < 0;
    for (int64_t v = plo; v < phi && !done; ++v) {
      float x[4];
      load(v, x);
      drop(v, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc += (double)x[i];
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
  // CTAs a request: enough to fill the GPU a few times over, runs of 16 vectors a lane or more
  int ranks = 1;
  while (ranks < kTreeMaxCluster && a.batch * ranks < (int64_t)sms * 4 &&
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
