// tg_paged.cuh -- device helpers shared by the kernels that read the paged
// key/value cache.
#pragma once

#include "tg_device.cuh"
#include "tg_internal.h"

namespace tg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Logits (log2 units) at or below this count as masked: the weight is zero
// even where a row has no other key. Gate biases are held above -1e38, so
// that a bias of -inf (or of the type's lowest value) times a zero gain is
// zero and not NaN; times any gain above 1e-8 it lands below this bound.
constexpr float kMaskedLogit = -1e30f;
constexpr float kLowestBias = -1e38f;
// Only keys with a bias below this one can be removed by it (gains up to
// 1e10): the kernels look at a block's logits one by one when it holds some.
constexpr float kRemovableBias = -1e20f;

__device__ __forceinline__ float key_bias(float b) { return b < kLowestBias ? kLowestBias : b; }

// One tile of query rows of a request. A row is a (token, query head of the
// KV head's group) pair: row r is token r / group, head r % group.
struct PagedTile {
  int req;       // request, or -1: no such tile
  int64_t tok0;  // first token of the request in q
  int64_t n;     // its new tokens
  int64_t past;  // cached rows before them (below 0 when kv_len < n)
  int64_t row0;  // first row of the tile
};

// New tokens of request b, their first row in q, and the cached rows before
// them; offsets or lengths that run out of range are cut (and reported).
__device__ __forceinline__ void request_span(const PagedAttnArgs& a, int b, int64_t& lo, int64_t& n,
                                             int64_t& past) {
  lo = __ldg(a.cu_q + b);
  int64_t hi = __ldg(a.cu_q + b + 1);
  int64_t len = __ldg(a.kv_len + b);
  if (lo < 0 || hi < lo || hi > a.rows || len > a.max_kv) {
    report_error(a.err, kErrIndexRange);
    lo = lo < 0 ? 0 : lo;
    hi = hi > a.rows ? a.rows : hi;
    hi = hi < lo ? lo : hi;
    len = len > a.max_kv ? a.max_kv : len;
  }
  n = hi - lo;
  past = len - n;
}

// The idx-th tile of `rows_per_tile` rows, counted through the requests in
// order. One full warp; every lane returns the same tile.
__device__ __forceinline__ PagedTile find_tile(const PagedAttnArgs& a, int rows_per_tile, int64_t idx) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int group = a.hq / a.kv.hkv;
  int64_t before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int64_t lo = 0, n = 0, past = 0;
    if (b0 + lane < a.batch) request_span(a, b0 + lane, lo, n, past);
    const int64_t cnt = (n * group + rows_per_tile - 1) / rows_per_tile;
    int64_t sum = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += up;
    }
    const int64_t all = __shfl_sync(0xFFFFFFFFu, sum, 31);
    if (idx < before + all) {
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, idx < before + sum);
      const int src = __ffs(static_cast<int>(hit)) - 1;
      PagedTile t;
      t.req = b0 + src;
      t.tok0 = __shfl_sync(0xFFFFFFFFu, lo, src);
      t.n = __shfl_sync(0xFFFFFFFFu, n, src);
      t.past = __shfl_sync(0xFFFFFFFFu, past, src);
      const int64_t first = before + __shfl_sync(0xFFFFFFFFu, sum - cnt, src);
      t.row0 = (idx - first) * rows_per_tile;
      return t;
    }
    before += all;
  }
  PagedTile none;
  none.req = -1;
  none.tok0 = none.n = none.past = none.row0 = 0;
  return none;
}

// Page that holds row j of request b, or -1 (reported) when it is out of range.
__device__ __forceinline__ int64_t page_of(const PagedAttnArgs& a, int b, int64_t j) {
  const int64_t blk = j / a.kv.page_size;
  if (blk < a.kv.table_stride) {
    const int64_t page = __ldg(a.kv.table + static_cast<int64_t>(b) * a.kv.table_stride + blk);
    if (page >= 0 && page < a.kv.n_pages) return page;
  }
  report_error(a.err, kErrIndexRange);
  return -1;
}

}  // namespace tg
