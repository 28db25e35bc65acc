// k_paged_tc.cu -- tg_paged_attn for chunks of new tokens, bf16, on the
// 5th-generation tensor cores (tcgen05, sm_100a).
//
// A row is a (token, query head of the KV head's group) pair, token-major. One
// CTA takes up to 256 rows of a request and KV head over one split of its keys,
// in 128-key tiles that TMA gathers from the pages (a box per page piece and 64
// columns, 128-byte swizzle). Two softmax warpgroups (A, B) take turns with the
// tensor core, as in the contiguous kernel (k_attn_tc.cu):
//   over 128 rows   A holds rows 0 .. 127, B rows 128 .. 255; both read every tile
//   up to 128 rows  both hold the same rows; A takes the even tiles, B the odd
//                   ones, and the two states merge at the end, so that short
//                   chunks (drafted tokens) keep the tensor core and the loads as
//                   busy
// Warps: 0 fetches the keys and 3 the values (lanes walk the page table two tiles
// ahead), 1 issues the MMAs, 2 allocates TMEM, prepares the keys' gate biases and
// cleans value rows that must not reach a row, 4-7 softmax A, 8-11 softmax B (one
// thread a row).
//
// Per tile and warpgroup: S = Q K^T into 128 TMEM columns, P (bf16) written over
// S, O += P V with P read from TMEM and V as it lies in the page (keys as K, dh
// as the contiguous MN dimension): no transposed copy. The order PV(j), QK(j + 1)
// per warpgroup means that S(j + 1) is seen only after PV(j) has finished, so O
// may be rescaled and P overwritten without another wait.
//
// P is rounded to bf16 (2^-8 of each weight), the type of the values that the
// tensor core multiplies it with: an fp32 or two-part P would take the 128 TMEM
// columns of S and as much of the tensor core again. Logits, maxima, sums (of
// the weights before that rounding) and O up to the last rounding are fp32.
//
// Gate bias: one more 16-wide K-step adds g b with g = gain sqrt(dh) tau, each
// of g and b in three bf16 parts and the six products down to 2^-24 kept. Keys
// whose bias is below -1e20 get b = 0 there and are decided one by one in fp32.
//
// Value rows: a weight of zero does not hide an infinity or a NaN from the
// matrix product. Rows behind the request's end are cleared in shared memory
// (they were never written); infinities and NaN of keys that only some rows see
// (the chunk's own tokens, keys removed by their bias) are cleared, noted, and
// added at the end to the rows that do see them.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tg_device.cuh"
#include "tg_internal.h"
#include "tg_paged.cuh"

namespace tg {
namespace {

constexpr int kBlk = 128;          // rows of a warpgroup = keys of a tile
constexpr int kThreads = 384;
constexpr int kSub = 128 * 128;    // [128 rows x 64 bf16], 128-byte swizzle
constexpr float kRescale = 8.0f;   // log2 units
// From this maximum on (log2 units) a logit is rounded before the maximum is
// taken off it: see the loop of the exponentials.
constexpr float kFarMax = 4194304.0f;  // 2^22

template <int kDh>
struct Lay {
  static constexpr int kSubs = kDh / 64;
  static constexpr int kTile = kSubs * kSub;         // [128 x kDh] bf16
  // the gate-bias K-steps: one tile whose four 16-column groups are the two
  // stages of the keys and the rows of A and of B
  static constexpr int kOffAug = 0;
  static constexpr int kOffQ = kSub;                 // A, B
  // two stages of K and of V at head_dim 128 (32 KB each), four at 64
  static constexpr int kStages = kDh == 128 ? 2 : 4;
  static constexpr int kOffK = kOffQ + 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffBias = kOffV + kStages * kTile;  // 4 x 128 fp32
  static constexpr int kOffMask = kOffBias + 4 * 512;
  static constexpr int kOffBar = kOffMask + 64;
  static constexpr size_t kSmem = 1024 + kOffBar + 512;
  static_assert(kSmem <= 232448, "shared memory per CTA");
  // B's output rows wait for the merge in the (by then idle) K tiles
  static_assert(128 * kDh * 4 <= kStages * kTile, "merge buffer");
};

constexpr uint32_t idesc_bmn(int m, int n) { return idesc_bf16_f32(m, n) | (1u << 16); }

// MN-major operand, 128-byte swizzle: 128-byte rows of 64 MN elements, one K
// index each, 8-row groups 1024 bytes apart, 64-element MN blocks `lbo` apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 2^x for a pair on the FMA pipe, x <= 8: x = j + f with j = round(x) (adding
// 1.5 * 2^23 leaves it in the low mantissa bits), a degree-4 polynomial for
// 2^f, |f| <= 1/2, fitted here with p(0) = 1 (largest relative error 2.9e-6, a
// thousandth of what rounding the weight to bf16 takes; of degree 3 1.0e-4),
// and j added to the exponent field. Below -127 that gives exactly 0, so a
// masked logit (-inf) has no weight; a polynomial with p(0) < 1
// (exp2_poly3_x2) would leave the exponent's range there. A NaN has no weight
// either: its row is marked where the maximum is formed.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
  x.x = fmaxf(x.x, -127.0f);
  x.y = fmaxf(x.y, -127.0f);
  const float2 kShift = make_float2(12582912.0f, 12582912.0f);
  const float2 t = fadd2(x, kShift);
  const float2 f = fadd2(x, fadd2(make_float2(-t.x, -t.y), kShift));
  float2 p = ffma2(f, make_float2(0.009585382f, 0.009585382f), make_float2(0.055906627f, 0.055906627f));
  p = ffma2(p, f, make_float2(0.24024038f, 0.24024038f));
  p = ffma2(p, f, make_float2(0.6931242f, 0.6931242f));
  p = ffma2(p, f, make_float2(1.0f, 1.0f));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}

// x in three bf16 parts (each the rest of the one before)
__device__ __forceinline__ void split3(float x, float& p0, float& p1, float& p2) {
  p0 = __bfloat162float(__float2bfloat16_rn(x));
  p1 = __bfloat162float(__float2bfloat16_rn(x - p0));
  p2 = x - p0 - p1;
}
// Row r of 16-column group `col` of a 128-byte-swizzled tile.
__device__ __forceinline__ void store_aug(uint8_t* tile, int r, int col, uint32_t a, uint32_t b, uint32_t c) {
  const int u = 2 * col, sw = r & 7;
  *reinterpret_cast<uint4*>(tile + r * 128 + ((u ^ sw) << 4)) = make_uint4(a, b, c, 0u);
  *reinterpret_cast<uint4*>(tile + r * 128 + (((u + 1) ^ sw) << 4)) = make_uint4(0u, 0u, 0u, 0u);
}

// Clears the infinities and NaN among 8 bf16 values.
__device__ __forceinline__ bool clear_nonfinite(uint4& u) {
  bool any = false;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7F80u) == 0x7F80u) {
      w[i] &= 0xFFFF0000u;
      any = true;
    }
    if ((w[i] & 0x7F800000u) == 0x7F800000u) {
      w[i] &= 0x0000FFFFu;
      any = true;
    }
  }
  return any;
}

template <int kDh, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ PagedAttnArgs a) {
  using L = Lay<kDh>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  float* s_bias = reinterpret_cast<float*>(smem + L::kOffBias);        // [4][128]
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + L::kOffMask);  // [4][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  constexpr int kSt = L::kStages;
  uint64_t* k_full = bars + 0;
  uint64_t* k_empty = bars + 4;
  uint64_t* v_full = bars + 8;    // the bytes are there
  uint64_t* go = bars + 12;       // and cleaned; the next tile's keys and biases are there, too
  uint64_t* v_empty = bars + 16;
  uint64_t* b_full = bars + 20;   // [4] biases and mask of a tile
  uint64_t* p_full = bars + 24;   // [A, B]
  uint64_t* s_full = bars + 28;   // [A, B]
  uint64_t* o_full = bars + 30;   // [A, B]
  uint64_t* q_full = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 33);
  __shared__ PagedTile s_tile;
  __shared__ int s_found;
  __shared__ float2 s_ml[kBlk];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_idx = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.tiles));
  const int rest = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.tiles));
  const int g = rest % a.kv.hkv, split = rest / a.kv.hkv;
  const int group = a.hq / a.kv.hkv;

  pdl_trigger();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 256);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&go[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&b_full[i], 1);
      mbar_init(&p_full[i], 4);  // the warps of a warpgroup
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    s_found = 0;
  }
  pdl_wait();
  if (warp == 0) {
    const PagedTile t = find_tile<2 * kBlk>(a, tile_idx);
    if (lane == 0) s_tile = t;
  }
  __syncthreads();
  const PagedTile tile = s_tile;
  if (tile.req < 0) return;
  const int n_rows = min(2 * kBlk, tile.n * group - tile.row0);
  const bool dual = n_rows <= kBlk;
  const int row0 = tile.row0, past = tile.past;
  // keys that the first and the last row of the tile see, and this CTA's keys
  const int min_limit = past + row0 / group + 1;
  const int max_limit = past + (row0 + n_rows - 1) / group + 1;
  const int64_t lo64 = split == 0 ? 0 : a.chunk0 + (split - 1) * a.chunk;
  const int64_t hi64 = min(static_cast<int64_t>(max_limit), lo64 + (split == 0 ? a.chunk0 : a.chunk));
  const int nt = hi64 > lo64 ? static_cast<int>((hi64 - lo64 + kBlk - 1) / kBlk) : 0;
  const int lo = static_cast<int>(lo64), hi = static_cast<int>(hi64);
  // output row of row r of the tile: (token, head)
  auto out_row = [&](int r) -> int64_t {
    const int rr = row0 + r;
    return static_cast<int64_t>(tile.tok0 + rr / group) * a.hq + g * group + rr % group;
  };
  if (nt == 0) {  // nothing to see
    for (int r = threadIdx.x; r < n_rows; r += kThreads) {
      const int64_t at = out_row(r);
      if (a.splits > 1) {
        *reinterpret_cast<float2*>(a.part_ml + (split * a.rows * a.hq + at) * 2) =
            make_float2(-INFINITY, 0.f);
      } else {
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * kDh);
        for (int i = 0; i < kDh / 8; ++i) out[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr) a.lse[(at % a.hq) * a.rows + at / a.hq] = -INFINITY;
      }
    }
    return;
  }
  if (warp == 2) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // tiles of the two warpgroups
  const int n_h[2] = {dual ? (nt + 1) / 2 : nt, dual ? nt / 2 : nt};

  if (warp < 4) {
    // A tile's boxes (page pieces x 64 columns), one a lane.
    const int box = min(a.kv.page_size, kBlk);  // rows of a box
    const int n_box = kBlk / box;               // a power of two
    const int my_box = lane & (n_box - 1), my_sub = lane / n_box;
    auto page_at = [&](int t) -> int {  // -1: nothing to fetch; n_pages: reads zeros
      const int j = lo + t * kBlk + my_box * box;
      if (t >= nt || j >= hi || my_sub >= L::kSubs) return -1;
      const int64_t p = page_of(a, tile.req, j);
      return p < 0 ? static_cast<int>(a.kv.n_pages) : static_cast<int>(p);
    };
    auto fetch = [&](const CUtensorMap* tm, uint64_t* full, uint8_t* dst, int t, int pg) {
      const unsigned live = __popc(__ballot_sync(0xFFFFFFFFu, pg >= 0));
      if (lane == 0) mbar_arrive_expect_tx(full, live * static_cast<unsigned>(box * 128));
      __syncwarp();
      if (pg >= 0)
        tma_load_4d(tm, full, dst + my_sub * kSub + my_box * box * 128, my_sub * 64, g,
                    row_in_page(a, lo + t * kBlk + my_box * box), pg);
    };
    if (warp == 0) {
      // ------------------------------------------------------------ keys
      int pg = page_at(0), pg1 = page_at(1);
      for (int t = 0; t < nt; ++t) {
        const int s = t % kSt;
        const int pg2 = page_at(t + 2);
        if (!mbar_wait_warp(&k_empty[s], ((t / kSt) & 1) ^ 1, a.err)) break;
        fetch(&tmK, &k_full[s], smem + L::kOffK + s * L::kTile, t, pg);
        pg = pg1;
        pg1 = pg2;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA
      // One warp for A and B. (A warp for each measured 633 us where this takes
      // 520: the two then want the tensor core, and the MUFU units, at the same
      // time.) The whole warp runs this, on values it knows to be the same in every
      // lane (a vote, a reduction), so that descriptors are formed and held in
      // uniform registers.
      const bool both = __any_sync(0xFFFFFFFFu, dual);
      const int last_a = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(n_h[0])));
      const int last_b = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(n_h[1])));
      const uint32_t base = smem_addr(smem);
      const uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, tmem);
      auto qk = [&](int h, int t) {
        constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
        const uint64_t qd = sdesc_kmajor_sw128(base + L::kOffQ + (h && !both ? L::kTile : 0));
        const uint64_t kd = sdesc_kmajor_sw128(base + L::kOffK + (t % kSt) * L::kTile);
        const uint32_t d = tm + static_cast<uint32_t>(h * 128);
#pragma unroll
        for (int kk = 0; kk < kDh / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kSub + (kk & 3) * 32) >> 4;
          umma_f16_ss_warp(d, qd + off, kd + off, idesc, kk > 0 ? 1u : 0u);
        }
        if (kBias)
          umma_f16_ss_warp(d, sdesc_kmajor_sw128(base + L::kOffAug + (h && !both ? 96 : 64)),
                           sdesc_kmajor_sw128(base + L::kOffAug + (t & 1) * 32), idesc, 1u);
        umma_commit_warp(&s_full[h]);
        if (h == 1 || both) umma_commit_warp(&k_empty[t % kSt]);
      };
      auto pv = [&](int h, int t, bool first) {
        constexpr uint32_t idesc = idesc_bmn(128, kDh);
        const uint64_t vd = sdesc_mn(base + L::kOffV + (t % kSt) * L::kTile, kSub);
        const uint32_t p_tm = tm + static_cast<uint32_t>(h * 128);
        const uint32_t d = tm + 256u + static_cast<uint32_t>(h * 128);
#pragma unroll
        for (int ks = 0; ks < kBlk / 16; ++ks)
          umma_f16_ts_warp(d, p_tm + static_cast<uint32_t>(ks * 8), vd + ((ks * 2048) >> 4), idesc,
                           (!first || ks > 0) ? 1u : 0u);
      };
      auto k_there = [&](int t) -> bool {
        return mbar_wait_warp(&k_full[t % kSt], (t / kSt) & 1, a.err) &&
               (!kBias || mbar_wait_warp(&b_full[t & 3], (t >> 2) & 1, a.err));
      };
      bool ok = mbar_wait_warp(q_full, 0, a.err) && k_there(0);
      if (ok) {
        tc_fence_after();
        qk(0, 0);
        if (last_b > 0) {
          if (both) ok = k_there(1);
          tc_fence_after();
          if (ok) qk(1, both ? 1 : 0);
        }
      }
      // warpgroup h's step j
      auto step = [&](auto hc, int j) -> bool {
        constexpr int h = decltype(hc)::value;
        const int n = h == 0 ? last_a : last_b;
        const int t = both ? 2 * j + h : j;
        if ((h == 0 || both) && !mbar_wait_warp(&go[t % kSt], (t / kSt) & 1, a.err)) return false;
        const bool more = j + 1 < n;
        if (!mbar_wait_warp(&p_full[h], j & 1, a.err)) return false;
        tc_fence_after();
        pv(h, t, j == 0);
        if (more) qk(h, both ? t + 2 : j + 1);
        else umma_commit_warp(&o_full[h]);
        if (h == 1 || both) umma_commit_warp(&v_empty[t % kSt]);
        return true;
      };
      for (int j = 0; j < last_a && ok; ++j) {
        ok = step(std::integral_constant<int, 0>(), j);
        if (ok && j < last_b) ok = step(std::integral_constant<int, 1>(), j);
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ values
      int pg = page_at(0), pg1 = page_at(1);
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        const int s = t % kSt;
        const int pg2 = page_at(t + 2);
        if (!mbar_wait_warp(&v_empty[s], ((t / kSt) & 1) ^ 1, a.err)) break;
        fetch(&tmV, &v_full[s], smem + L::kOffV + s * L::kTile, t, pg);
        pg = pg1;
        pg1 = pg2;
      }
    } else {
      // ------------------------------------------------------------ gate biases, cleaning
      // Keys lane, lane + 32, ... of a tile (rows of their K-step that store
      // without bank conflicts). Lane l holds the page of keys 16 (l & 7) on; pages
      // two tiles ahead, biases one.
      auto bias_pages = [&](int t) -> int {
        const int j = lo + t * kBlk + (lane & 7) * 16;
        return kBias && t < nt && j < hi ? static_cast<int>(page_of(a, tile.req, j)) : -1;
      };
      float b[4];
      auto load_bias = [&](int t, int pages) {
        const int j = lo + t * kBlk + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t p = __shfl_sync(0xFFFFFFFFu, pages, (lane >> 4) + 2 * i);
          b[i] = p >= 0 && j + 32 * i < hi
                     ? __ldg(a.kv.bias + p * a.kv.bias_page_stride + row_in_page(a, j + 32 * i))
                     : 0.f;
        }
      };
      int pg = -1;
      if (kBias) {
        load_bias(0, bias_pages(0));
        pg = bias_pages(1);
      }
      // Step i: the biases of tile i, then the values of the tile that it follows in
      // its warpgroup; with the keys of tile i that is all that P V of the one
      // and Q K of the other need, and the MMAs wait for it once.
      const int dt = dual ? 2 : 1;
#pragma unroll 1
      for (int i = 0; i < nt + dt; ++i) {
        if (kBias && i < nt) {
          // QK(i - 2) has read its K-step; so the softmax of tile i - 4 is over
          if (i >= 2 && !mbar_wait_warp(&k_empty[(i - 2) % kSt], ((i - 2) / kSt) & 1, a.err)) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool rem = b[e] < kRemovableBias;
            const unsigned bits = __ballot_sync(0xFFFFFFFFu, rem);
            if (lane == 0) s_mask[(i & 3) * 4 + e] = bits;
            s_bias[(i & 3) * 128 + lane + 32 * e] = key_bias(b[e]);
            float b0, b1, b2;
            split3(rem ? 0.f : b[e], b0, b1, b2);
            // against (g0, g0, g1, g0, g2, g1)
            store_aug(smem + L::kOffAug, lane + 32 * e, i & 1, pack_bf16x2(b0, b1), pack_bf16x2(b0, b2),
                      pack_bf16x2(b0, b1));
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_full[i & 3]);
          load_bias(i + 1, pg);
          pg = bias_pages(i + 2);
        }
        const int t = i - dt;
        if (t < 0) continue;
        const int s = t % kSt, key0 = lo + t * kBlk;
        uint4 part = make_uint4(0u, 0u, 0u, 0u);  // keys that their bias may remove
        if (kBias) part = *reinterpret_cast<const uint4*>(s_mask + (t & 3) * 4);
        if (!mbar_wait_warp(&v_full[s], (t / kSt) & 1, a.err)) break;
        if ((part.x | part.y | part.z | part.w) != 0u || key0 + kBlk > min_limit) {
          uint8_t* v = smem + L::kOffV + s * L::kTile;
          constexpr int kUnits = kDh / 8;  // 16-byte units of a row
          // units of a lane that are read at once (221 tokens of one request, 10/2 x
          // 128: one at a time, over the whole tile, 22.1 us, so 17.7)
          constexpr int kBatch = 8;
          const bool any_part = (part.x | part.y | part.z | part.w) != 0u;
          const int first = any_part ? 0 : max(min_limit - key0, 0);  // (the rows before it are whole)
          bool found = false;
#pragma unroll 1
          for (int e0 = first * kUnits + lane; e0 < kBlk * kUnits; e0 += 32 * kBatch) {
            uint4 x[kBatch];
            unsigned live = 0;
            auto unit = [&](int i) -> uint4* {
              const int r = (e0 + 32 * i) / kUnits, u = (e0 + 32 * i) % kUnits;
              return reinterpret_cast<uint4*>(v + (u >> 3) * kSub + r * 128 + (((u & 7) ^ (r & 7)) << 4));
            };
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int r = (e0 + 32 * i) / kUnits;
              x[i] = make_uint4(0u, 0u, 0u, 0u);
              if (r >= kBlk) continue;
              if (key0 + r >= hi) {
                *unit(i) = x[i];
                continue;
              }
              const unsigned word = r < 32 ? part.x : r < 64 ? part.y : r < 96 ? part.z : part.w;
              if (key0 + r < min_limit && !((word >> (r & 31)) & 1u)) continue;
              live |= 1u << i;
              x[i] = *unit(i);
            }
            // 0 x + 0 is NaN where x is infinite or NaN, else 0
            const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
            __nv_bfloat162 sum = zero;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
              for (int w = 0; w < 4; ++w)
                sum = __hfma2(reinterpret_cast<const __nv_bfloat162*>(&x[i])[w], zero, sum);
            if (*reinterpret_cast<const unsigned*>(&sum) != 0u) {
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                if (((live >> i) & 1u) && clear_nonfinite(x[i])) {
                  found = true;
                  *unit(i) = x[i];
                }
            }
          }
          if (found) s_found = 1;
          fence_async_smem();
          __syncwarp();
        }
        if (i < nt && !mbar_wait_warp(&k_full[i % kSt], (i / kSt) & 1, a.err)) break;
        if (lane == 0) mbar_arrive(&go[s]);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int h = (warp - 4) >> 2;            // warpgroup A or B
    const int r = (threadIdx.x - 128) & 127;  // row of the warpgroup = TMEM lane
    const int rt = (dual ? 0 : h * kBlk) + r; // row of the tile
    const int w_row = rt - lane;              // the warp's first row
    const bool row_ok = rt < n_rows;
    // the row's place: token x heads + head (rows x heads of the call: 32 bits)
    const int head = g * group + (row0 + rt) % group;
    const int tok = tile.tok0 + (row0 + rt) / group;
    const int at = tok * a.hq + head;
    const float tau = a.tau && row_ok ? __ldg(a.tau + head) : 1.0f;
    const float gain = kBias && row_ok ? __ldg(a.gain + head) : 0.0f;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + static_cast<uint32_t>(h * 128);
    const uint32_t o_tm = tmem + lane_off + 256u + static_cast<uint32_t>(h * 128);
    const float scale2 = kLog2e / (sqrtf(static_cast<float>(kDh)) * tau);
    // rows without a query see everything (their output goes nowhere)
    const int limit = row_ok ? past + (row0 + rt) / group + 1 : 0x7FFFFFFF;
    if (!dual || h == 0) {  // this warp's rows of Q: 16 bytes a lane, whole rows side by side
      uint8_t* qd = smem + L::kOffQ + (dual ? 0 : h * L::kTile);
      constexpr int kUnits = kDh / 8, kStep = 32 / kUnits;  // 16-byte units of a row
      const int u = lane % kUnits;
      const int64_t mine = static_cast<int64_t>(tok) * a.q_stride + head * kDh;
      uint4 x[kUnits];
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int src = i * kStep + lane / kUnits;
        const int64_t off = __shfl_sync(0xFFFFFFFFu, mine, src);
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (w_row + src < n_rows)
          x[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + off + u * 8);
      }
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int qr = (r - lane) + i * kStep + lane / kUnits;
        *reinterpret_cast<uint4*>(qd + (u >> 3) * kSub + qr * 128 + (((u & 7) ^ (qr & 7)) << 4)) = x[i];
      }
      if (kBias) {
        float g0, g1, g2;
        split3(gain * sqrtf(static_cast<float>(kDh)) * tau, g0, g1, g2);
        store_aug(smem + L::kOffAug, r, 2 + (dual ? 0 : h), pack_bf16x2(g0, g0), pack_bf16x2(g1, g0),
                  pack_bf16x2(g2, g1));
      }
      fence_async_smem();
    }
    mbar_arrive(q_full);
    float m = -INFINITY, l = 0.f;
    bool far = false;  // some row of the warp has its maximum at 2^22 or beyond
    bool ok = true;
    for (int j = 0; j < n_h[h] && ok; ++j) {
      const int t = dual ? 2 * j + h : j;
      const int key0 = lo + t * kBlk;
      if (!mbar_wait_warp(&s_full[h], j & 1, a.err)) { ok = false; break; }
      tc_fence_after();
      // Tiles that hold keys some row of the warp must not see, or keys that
      // their bias may remove (then decided in fp32): their logits are put
      // right in TMEM first, 32 at a time, so that the loop's own code, which
      // is all that most tiles run, stays small enough for the instruction
      // cache (with the masks inlined in it: 740 us, so 625, for 2048 tokens
      // after 30720).
      uint4 rem = make_uint4(0u, 0u, 0u, 0u);
      if (kBias) {
        if (!mbar_wait_warp(&b_full[t & 3], (t >> 2) & 1, a.err)) { ok = false; break; }
        rem = *reinterpret_cast<const uint4*>(s_mask + (t & 3) * 4);
      }
      if (__any_sync(0xFFFFFFFFu, key0 + kBlk > limit) || (rem.x | rem.y | rem.z | rem.w) != 0u) {
        const float* bs = s_bias + (t & 3) * 128;
        const float gs = gain * sqrtf(static_cast<float>(kDh)) * tau;
        const float floor_x = kMaskedLogit / scale2;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t word = c == 0 ? rem.x : c == 1 ? rem.y : c == 2 ? rem.z : rem.w;
          const int seen = limit - key0 - c * 32;  // of these 32 keys
          if (word == 0u && !__any_sync(0xFFFFFFFFu, seen < 32)) continue;
          float z[32];
          tmem_ld32_wait(s_tm + static_cast<uint32_t>(c * 32), z);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (kBias && ((word >> i) & 1u)) {
              z[i] = fmaf(gs, bs[c * 32 + i], z[i]);
              if (z[i] <= floor_x) z[i] = -INFINITY;
            }
            if (i >= seen) z[i] = -INFINITY;
          }
          tmem_st32_wait(s_tm + static_cast<uint32_t>(c * 32), z);
        }
      }
      // P = 2^(S scale2 - m), 32 keys at a time, in packed pairs, three of the 16 pairs
      // on the FMA pipe (the MUFU unit is this loop's bottleneck; 2048 tokens after
      // 30720: none 551 us, two 531, these three 516, four 541); 32 keys' P covers 16
      // columns of logits that have been read. The running maximum m is moved (to a
      // whole number, so that every rescaling is by an exact power of two) only when 32
      // logits pass it by more than 2^8, after their exponentials: no pass over the row
      // comes before them (2048 tokens after 30720, no bias: 482 us with one, 470
      // without). What the row has gathered, the P of this tile included, is rescaled
      // then, and the 32 exponentials are formed again.
      float2 sp[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                      make_float2(0.f, 0.f)};
      // The product S scale2 is exact in the FMA, but the maximum comes from the rounded
      // product, half a unit in its last place away: from 2^22 on that is a quarter and
      // more (512 where a gate bias of -1e10 holds every key: the largest weight would be
      // 2^512 or 0). There (`far`) the logits are rounded like their maximum, before the
      // loop, whose factor is then 1. (2048 tokens after 30720: 515 us with this, 511
      // without; 541 with the far logits' exponentials formed anew behind the loop, 594
      // with the rounding inside it.)
      float base = m == -INFINITY ? 0.f : m;
      uint32_t y0[32];
      auto round_logits = [&](uint32_t (&u)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * scale2);
      };
      auto weights = [&](uint32_t (&u)[32], int c, float factor) {
        float mx4[4];  // NaN stays
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx4[k] =
              fmax3f_nan(__uint_as_float(u[k]), __uint_as_float(u[4 + k]), __uint_as_float(u[8 + k]));
#pragma unroll
        for (int i = 12; i < 28; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx4[k] = fmax3f_nan(mx4[k], __uint_as_float(u[i + k]), __uint_as_float(u[i + 4 + k]));
        const float last4 = fmax3f_nan(
            mx4[3],
            fmax3f_nan(__uint_as_float(u[28]), __uint_as_float(u[29]), __uint_as_float(u[30])),
            __uint_as_float(u[31]));
        const float mx = max_nan(fmax3f_nan(mx4[0], mx4[1], mx4[2]), last4) * factor;
        uint32_t pk[16];
        float2 cs[4];
        // with the maximum as it stands; once more when these logits move it
#pragma unroll 1
        for (bool again = false;; again = true) {
          const float2 nm2 = make_float2(-base, -base), sc2 = make_float2(factor, factor);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y =
                ffma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), sc2, nm2);
            float2 e;
            if (i > 3 && (i & 3) == 3) {
              e = exp2_fma(y);
            } else {
              e.x = ex2_approx(y.x);
              e.y = ex2_approx(y.y);
            }
            cs[i & 3] = i < 4 ? e : fadd2(cs[i & 3], e);
            pk[i] = pack_bf16x2(e.x, e.y);
          }
          if (again) break;
          const bool grow = mx > m + kRescale || (m == -INFINITY && mx > -INFINITY);
          if (!__any_sync(0xFFFFFFFFu, grow)) break;
          float alpha = 1.0f;
          if (grow) {
            const float m_new = ceilf(mx);
            alpha = ex2_approx(m - m_new);  // 0 on the first keys
            m = base = m_new;
          }
          far = __any_sync(0xFFFFFFFFu, fabsf(base) >= kFarMax);
          if (far && factor != 1.0f) {
            round_logits(u);
            factor = 1.0f;
          }
          l *= alpha;
#pragma unroll
          for (int k = 0; k < 4; ++k) sp[k] = fmul2(sp[k], make_float2(alpha, alpha));
          tmem_wait_st();
#pragma unroll 1
          for (int e = 0; e < c; ++e) {
            uint32_t old[16];
            tmem_ld16(s_tm + static_cast<uint32_t>(16 * e), old);
            tmem_wait_ld_dep16(old);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              old[i] = pack_bf16x2(__uint_as_float(old[i] << 16) * alpha,
                                   __uint_as_float(old[i] & 0xFFFF0000u) * alpha);
            tmem_st16(s_tm + static_cast<uint32_t>(16 * e), old);
          }
          if (j > 0) {
#pragma unroll 1
            for (int e = 0; e < kDh / 32; ++e) {
              float o[32];
              const uint32_t ta = o_tm + static_cast<uint32_t>(e * 32);
              tmem_ld32_wait(ta, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32_wait(ta, o);
            }
          }
        }
        // a row with a logit that is NaN or +infinity: so are its sum and its outputs
        // (the exponentials on the FMA pipe do not carry a NaN)
        if (!(mx < INFINITY)) l = __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int k = 0; k < 4; ++k) sp[k] = fadd2(sp[k], cs[k]);
        tmem_st16(s_tm + static_cast<uint32_t>(16 * c), pk);
      };
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        tmem_ld32(s_tm + static_cast<uint32_t>(32 * c), y0);
        tmem_wait_ld_dep(y0);
        if (far) round_logits(y0);
        weights(y0, c, far ? 1.0f : scale2);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[h]);
      const float2 s2 = fadd2(fadd2(sp[0], sp[1]), fadd2(sp[2], sp[3]));
      l += s2.x + s2.y;
    }
    // -------------------------------------------------------------- output
    // With `dual`, B's rows wait in the idle K tiles for A's threads.
    const bool active = !dual || h == 0;
    ok = ok && (n_h[h] == 0 || mbar_wait_warp(&o_full[h], 0, a.err));
    if (dual && h == 1) ok = ok && mbar_wait_warp(&o_full[0], 0, a.err);  // all MMAs have read K
    // the last tile's values are cleaned: s_found is final
    ok = ok && mbar_wait_warp(&go[(nt - 1) % kSt], ((nt - 1) / kSt) & 1, a.err);
    tc_fence_after();
    float4* xo = reinterpret_cast<float4*>(smem + L::kOffK) + r;  // [kDh / 4][128 rows]
    float wa = 1.0f, wb = 0.f;
    if (dual) {
      if (h == 1) {
        s_ml[r] = make_float2(m, ok ? l : 0.f);
        if (ok && n_h[1] > 0) {
#pragma unroll 1
          for (int c = 0; c < kDh / 32; ++c) {
            float o[32];
            tmem_ld32_wait(o_tm + static_cast<uint32_t>(c * 32), o);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              xo[(c * 8 + v) * 128] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
        }
      }
      named_bar_sync(1, 256);
      if (h == 0) {
        const float2 b = s_ml[r];
        const float top = fmaxf(m, b.x);
        wa = state_weight(m, l, top);
        wb = state_weight(b.x, b.y, top);
        m = top;
        l = l * wa + b.y * wb;
      }
    }
    if (active && ok && w_row < n_rows) {
      const bool part = a.splits > 1;
      const bool any = l != 0.f;  // a row that sees nothing is zero
      const float inv = part ? 1.0f : any ? 1.0f / l : 0.f;
      const int64_t part0 = split * a.rows * a.hq;
      if (row_ok) {
        if (part)
          *reinterpret_cast<float2*>(a.part_ml + (part0 + at) * 2) = make_float2(m, l);
        else if (a.lse != nullptr)
          a.lse[head * a.rows + tok] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
      // each warp's 32 rows x 32 columns through its part of the idle Q tile
      uint8_t* stage = smem + L::kOffQ + h * L::kTile + (warp & 3) * 4096;
      const int found = *const_cast<volatile int*>(&s_found);
#pragma unroll 1
      for (int c = 0; c < kDh / 32; ++c) {
        float o[32];
        tmem_ld32_wait(o_tm + static_cast<uint32_t>(c * 32), o);
        if (dual) {
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const float4 b = wb != 0.f ? xo[(c * 8 + v) * 128] : make_float4(0.f, 0.f, 0.f, 0.f);
            o[4 * v] = o[4 * v] * wa + b.x * wb;
            o[4 * v + 1] = o[4 * v + 1] * wa + b.y * wb;
            o[4 * v + 2] = o[4 * v + 2] * wa + b.z * wb;
            o[4 * v + 3] = o[4 * v + 3] * wa + b.w * wb;
          }
        }
        if (found && row_ok) {
          for (int jj = lo; jj < min(hi, limit); ++jj) {
            const int64_t p = page_of(a, tile.req, jj);
            if (p < 0) continue;
            const int in = row_in_page(a, jj);
            const float b = kBias ? key_bias(__ldg(a.kv.bias + p * a.kv.bias_page_stride + in)) : 0.f;
            const bool rem = b < kRemovableBias;
            if ((jj < min_limit && !rem) || (rem && gain * kLog2e * b <= kMaskedLogit)) continue;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.kv.v) + p * a.kv.v_page_stride +
                                     (static_cast<int64_t>(in) * a.kv.hkv + g) * kDh + c * 32;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float f = __bfloat162float(v[i]);
              if (!isfinite(f)) o[i] += f;
            }
          }
        }
#pragma unroll
        for (int v = 0; v < 8; ++v)
          *reinterpret_cast<float4*>(stage + lane * 128 + ((v ^ (lane & 7)) << 4)) =
              make_float4(o[4 * v] * inv, o[4 * v + 1] * inv, o[4 * v + 2] * inv, o[4 * v + 3] * inv);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3), u = lane & 7;
          const float4 f = *reinterpret_cast<const float4*>(stage + rr * 128 + ((u ^ (rr & 7)) << 4));
          const int64_t to = __shfl_sync(0xFFFFFFFFu, at, rr);
          if (w_row + rr < n_rows) {
            if (part)
              *reinterpret_cast<float4*>(a.part_o + (part0 + to) * kDh + c * 32 + u * 4) = f;
            else
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to * kDh + c * 32 + u * 4) =
                  make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// Splits of the keys, from the sizes that the host knows (requests may be
// shorter). Times in microseconds, as measured per CTA: a 128-key tile of two
// warpgroups (of one, where it waits for memory), the fixed cost of a CTA, the
// merge with its partial rows.
void plan(PagedAttnArgs* a) {
  const int64_t sms = num_sms();
  const int group = a->hq / a->kv.hkv;
  const int64_t jobs = a->tiles * a->kv.hkv;
  const int64_t nt = (a->max_kv + kBlk - 1) / kBlk;
  const int64_t mean_rows = a->rows * group / (a->tiles > 0 ? a->tiles : 1);
  const double tile_us = (mean_rows <= kBlk ? 1.6 : 2.2) * (a->kv.dh == 128 ? 1.0 : 0.7), cta_us = 12.0;
  const double part_us = double(a->rows) * a->hq * a->kv.dh * 8.0 / 5.0e6;  // one split's, out and in
  const int most = paged_max_splits(a->rows, a->hq, a->kv.dh);
  double best = 1e300;
  for (int s = 1; s <= most && s <= nt; ++s) {
    const int64_t c = (nt + s - 1) / s;
    const double piece = c * tile_us + cta_us;
    // whole waves of pieces; of several requests, whose lengths differ, about a
    // fifth of them are empty (8 requests' drafts, 18 jobs over up to 71 tiles: 8 to
    // 10 splits 21 us, 6 or 12 25, 16 29)
    const double filled = a->batch == 1 ? 1.0 : 0.8;
    const double us = std::ceil(filled * jobs * s / sms) * piece + (s > 1 ? 4.0 + s * part_us : 0.0);
    if (us < best - 1e-9) {
      best = us;
      a->splits = static_cast<int>((nt + c - 1) / c);
      a->chunk0 = a->chunk = c * kBlk;
    }
  }
  // One request that leaves SMs idle: those take the last tiles of all the
  // others, k each.
  if (a->batch == 1 && jobs < sms && most >= 2) {
    const int64_t k = (jobs + sms - jobs - 1) / (sms - jobs);
    const double y = (nt * tile_us + cta_us * (1 - k)) / ((k + 1) * tile_us);
    const int64_t tail = static_cast<int64_t>(y);
    if (tail >= 1 && tail < nt) {
      const double us = std::max((nt - tail) * tile_us + cta_us, k * (tail * tile_us + cta_us)) + 4.0 +
                        2 * part_us;
      if (us < best) {
        a->splits = 2;
        a->chunk0 = (nt - tail) * kBlk;
        a->chunk = tail * kBlk;
      }
    }
  }
}

template <int kDh, bool kBias>
cudaError_t run(const PagedAttnArgs& a, cudaStream_t st) {
  using L = Lay<kDh>;
  CUtensorMap tk, tv;
  const int box = a.kv.page_size < kBlk ? a.kv.page_size : kBlk;
  if (!make_tmap_pages_bf16(&tk, a.kv.k, kDh, a.kv.hkv, a.kv.page_size, a.kv.n_pages,
                            a.kv.k_page_stride, box) ||
      !make_tmap_pages_bf16(&tv, a.kv.v, kDh, a.kv.hkv, a.kv.page_size, a.kv.n_pages,
                            a.kv.v_page_stride, box))
    return cudaErrorInvalidValue;
  auto kern = paged_attn_tc<kDh, kBias>;
  TG_CUDA_TRY(set_smem_attr_once(reinterpret_cast<const void*>(kern), static_cast<int>(L::kSmem)));
  const int64_t grid = a.tiles * a.splits * a.kv.hkv;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), L::kSmem, st, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_tc(PagedAttnArgs a, void* ws, cudaStream_t st) {
  a.tiles = paged_row_tiles(a.rows, a.batch, a.hq, a.kv.hkv, 2 * kBlk);
  plan(&a);
  paged_partials(&a, ws);
  const bool bias = a.gain != nullptr && a.kv.bias != nullptr;
  cudaError_t e;
  if (a.kv.dh == 128) e = bias ? run<128, true>(a, st) : run<128, false>(a, st);
  else e = bias ? run<64, true>(a, st) : run<64, false>(a, st);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_paged_merge(a, true, st);
}

}  // namespace tg
