// tg_paged.cuh -- device helpers shared by the kernels that read the paged
// key/value cache.
#pragma once

#include "tg_device.cuh"
#include "tg_internal.h"

namespace tg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A key is removed by its gate bias: where the bias is below kRemovableBias and
// the logit (log2 units) at or below kMaskedLogit, the weight is zero even if a
// row has no other key. (The kernels look at a block's logits one by one when it
// holds such a bias. A logit that the product alone takes so far down is one
// like any other.) Gate biases are held above -1e38, so that a bias of -inf (or
// of the type's lowest value) times a zero gain is zero and not NaN; times any
// gain above 1e-8 it lands below the bound.
constexpr float kMaskedLogit = -1e30f;
constexpr float kLowestBias = -1e38f;
constexpr float kRemovableBias = -1e20f;

__device__ __forceinline__ float key_bias(float b) { return b < kLowestBias ? kLowestBias : b; }

// Weight of a partial state (maximum m, sum l) under the maximum `top` of all.
// A state without keys (l = 0) has none; one whose logits are all NaN has m =
// -inf and l = NaN, and passes that on.
__device__ __forceinline__ float state_weight(float m, float l, float top) {
  return l == 0.f ? 0.f : ex2_approx(m - (top == -INFINITY ? 0.f : top));
}

// One tile of query rows of a request. A row is a (token, query head of the
// KV head's group) pair: row r is token r / group, head r % group. Rows and
// keys are 32-bit (the call has fewer than 2^31 rows x heads).
struct PagedTile {
  int req;    // request, or -1: no such tile
  int tok0;   // first token of the request in q
  int n;      // its new tokens
  int past;   // cached rows before them (below 0 when kv_len < n)
  int row0;   // first row of the tile
};

// New tokens of request b, their first row in q, and the cached rows before
// them; offsets or lengths that run out of range are cut (and reported).
__device__ __forceinline__ void request_span(const PagedAttnArgs& a, int b, int& lo, int& n, int& past) {
  lo = __ldg(a.cu_q + b);
  int hi = __ldg(a.cu_q + b + 1);
  int len = __ldg(a.kv_len + b);
  const int rows = static_cast<int>(a.rows);
  const int max_kv = static_cast<int>(a.max_kv < 0x7FFFFFFF ? a.max_kv : 0x7FFFFFFF);
  if (lo < 0 || hi < lo || hi > rows || len > max_kv) {
    report_error(a.err, kErrIndexRange);
    lo = lo < 0 ? 0 : lo;
    hi = hi > rows ? rows : hi;
    hi = hi < lo ? lo : hi;
    len = len > max_kv ? max_kv : len;
  }
  len = len < 0 ? 0 : len;  // no keys at all: as many rows as there are see nothing
  n = hi - lo;
  past = len - n;
}

// Narrows the requests [skip, skip + left) down to 32 or fewer among which is
// the last one that begins at or before `idx`; `begin(b)` ascends. 32 probes a
// step; one full warp.
template <typename F>
__device__ __forceinline__ void narrow_requests(F&& begin, int64_t idx, int& skip, int& left) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  while (left > 32) {
    const int step = (left + 31) / 32;
    const int behind =
        __popc(__ballot_sync(0xFFFFFFFFu, begin(skip + min((lane + 1) * step, left)) <= idx));
    const int gone = min(behind * step, left);
    skip += gone;
    left = min(step, left - gone);
  }
}

// The tile of `kTile` rows in slot `idx` of a.tiles, if its request fills the
// slot. Requests are searched by their first slots, which follow from cu_q alone
// (a count of the tiles before a slot reads every request: 2000 requests of one
// token 966 us, so 560). One full warp; every lane returns the same tile.
template <int kTile>
__device__ __forceinline__ PagedTile find_tile(const PagedAttnArgs& a, int idx) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int group = a.hq / a.kv.hkv;
  const int rows = static_cast<int>(a.rows);
  const bool sparse = a.rows < a.batch;
  auto slot = [&](int b, int cu) {
    return paged_first_slot(min(max(cu, 0), rows), b, sparse, group, kTile);
  };
  int skip = 0, left = a.batch;
  narrow_requests([&](int b) { return slot(b, __ldg(a.cu_q + b)); }, idx, skip, left);
  const int b = skip + lane;
  int lo = 0, n = 0, past = 0;
  if (lane < left) request_span(a, b, lo, n, past);
  const int64_t first = slot(b, lo);
  const int src = __popc(__ballot_sync(0xFFFFFFFFu, lane < left && first <= idx)) - 1;
  PagedTile t{-1, 0, 0, 0, 0};
  if (src >= 0) {
    t.tok0 = __shfl_sync(0xFFFFFFFFu, lo, src);
    t.n = __shfl_sync(0xFFFFFFFFu, n, src);
    t.past = __shfl_sync(0xFFFFFFFFu, past, src);
    const int64_t row0 = (idx - __shfl_sync(0xFFFFFFFFu, first, src)) * kTile;
    if (row0 < t.n * group) {
      t.req = skip + src;
      t.row0 = static_cast<int>(row0);
    }
  }
  // offsets and lengths out of range are reported wherever they are
  if (a.batch > 32)
    for (int64_t c = static_cast<int64_t>(idx) * 32 + lane; c < a.batch; c += a.tiles * 32)
      request_span(a, static_cast<int>(c), lo, n, past);
  return t;
}

// Page that holds row j of request b, or -1 (reported) when it is out of range.
__device__ __forceinline__ int64_t page_of(const PagedAttnArgs& a, int b, int j) {
  const int blk = j >> a.kv.page_shift;
  if (blk < a.kv.table_stride) {
    const int64_t page = __ldg(a.kv.table + static_cast<int64_t>(b) * a.kv.table_stride + blk);
    if (page >= 0 && page < a.kv.n_pages) return page;
  }
  report_error(a.err, kErrIndexRange);
  return -1;
}

// Row of j in its page.
__device__ __forceinline__ int row_in_page(const PagedAttnArgs& a, int j) {
  return j & (a.kv.page_size - 1);
}

}  // namespace tg
