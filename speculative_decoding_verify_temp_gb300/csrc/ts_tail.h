// What is left of the requests behind a shared prefix: shared by ts_shared.cu and ts_tail.cu.
#pragma once

#include "ts_window.cuh"

namespace tsv {

struct TailParams : WindowParams {
  const int32_t* first;  // [batch] tokens in front that are not attended to here (whole pages)
  const float* pre_o;    // [total_rows * heads_q][D] their part of the rows: outputs,
  const float2* pre_ml;  // references and sums (of the rows of requests with first > 0)
  const Start* starts;   // [CTAs] their shares
};

constexpr int kTailTile = 64, kTailLeast = 2;  // tokens of a tile; least tiles a CTA takes
constexpr int tail_ctas(int rows) { return rows == 16 ? 3 : 2; }  // CTAs an SM: registers, and shared memory

int tail_rows(const WindowParams& p);  // of a block
size_t tail_workspace(int64_t batch, int64_t total_rows, int heads_q, int heads, int head_dim, int sms);
TailParams tail_params(const ts_kv_cache& c, const ts_attn_args& a, void* ws, int sms);  // without the prefix's
cudaError_t launch_tail(const TailParams& p, int sms, cudaStream_t s);

struct RawTail : RawReq {
  int32_t first;
};
__device__ __forceinline__ RawTail raw_request(const TailParams& p, int64_t b) {
  RawTail r;
  static_cast<RawReq&>(r) = raw_request(static_cast<const WindowParams&>(p), b);
  r.first = b < p.c.batch ? __ldcg(p.first + b) : 0;  // the kernel that plans ahead may run while the one that wrote it ends
  return r;
}
template <int ROWS, int TILE>
__device__ __forceinline__ Req request(const TailParams& p, const RawTail& raw) {
  Req r = request<ROWS, TILE>(static_cast<const WindowParams&>(p), static_cast<const RawReq&>(raw));
  r.skip = raw.first >> p.page_shift;
  r.len -= raw.first;  // which is not above it
  r.tiles = max((int)((unsigned)(r.len + TILE - 1) / TILE), 1);
  return r;
}

}  // namespace tsv
