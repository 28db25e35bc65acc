// k_paged_decode.cu -- tg_paged_attn for requests with few new rows (decoding,
// short drafts), bf16: every cached key and value is read once for at most 16
// query rows, so the call is bound by HBM.
//
// A row is a (token, query head of the KV head's group) pair. One CTA takes a
// tile of up to 16 rows of a request and KV head over one split of its keys:
//   warp 4     reads the page table, fetches 64-key blocks of K and V by TMA
//              (one box per page piece and 64 columns, 128-byte swizzle) into a
//              ring, and the keys' gate biases beside them, one block ahead.
//   warps 0-3  16 keys of the block each: S = Q K^T and O += P V as
//              mma.sync m16n8k16 (Q and O in registers, P stays in registers:
//              the accumulators of S are the A operand of P V), with a running
//              maximum and sum of their own, rescaled only when a maximum grows
//              by more than 2^8.
// At the end the four warps' states merge in shared memory. With one split the
// CTA writes the output; otherwise it writes its unnormalised rows and their
// (maximum, sum), and paged_merge adds up the splits in their order.
//
// Weights P are rounded to bf16 (2^-8 of each), as the tensor core multiplies
// them with bf16 values at full rate; P in two bf16 parts would double the
// second product. Logits, maxima, sums (of the weights before that rounding)
// and outputs up to the last rounding are fp32.
//
// Why mma.sync: 16 rows use an eighth of a tcgen05 tile (M = 128), whose
// softmax would run one thread per row; here all 128 threads hold logits, and
// the tensor work is a fifth of the time that the keys take to arrive.
#include <algorithm>
#include <atomic>

#include "tg_device.cuh"
#include "tg_internal.h"
#include "tg_paged.cuh"

namespace tg {
namespace {

constexpr int kRows = 16;
constexpr int kKeys = 64;    // keys of a ring stage, 16 for each consumer warp
constexpr int kThreads = 160;
constexpr int kRing = 96 * 1024;  // two CTAs on an SM
constexpr float kRescale = 8.0f;  // log2 units
constexpr int kMaxCluster = 16;

template <int kDh>
struct Cfg {
  static constexpr int kSubs = kDh / 64;
  static constexpr int kSub = kKeys * 128;                // [64 keys x 64 columns] bf16
  static constexpr int kStageBytes = 2 * kSubs * kSub;    // K, then V
  static constexpr int kStages = kRing / kStageBytes;
  static constexpr size_t kSmem = 1024 + kRing + 1024;    // (bias and barriers are static)
  static_assert(5 * kRows * kDh * 4 <= kRing, "the warps' outputs reuse the ring");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Clears the halves of a bf16 pair whose key no row sees; where only some
// rows see it (bit of `partial`), clears an infinity or NaN too and notes it.
__device__ __forceinline__ uint32_t clean_pair(uint32_t v, uint32_t dead, uint32_t partial, int bit,
                                               bool& found) {
  if ((dead >> bit) & 1u) v &= 0xFFFF0000u;
  if ((dead >> (bit + 1)) & 1u) v &= 0x0000FFFFu;
  if (((partial >> bit) & 1u) && (v & 0x7F80u) == 0x7F80u) {
    v &= 0xFFFF0000u;
    found = true;
  }
  if (((partial >> (bit + 1)) & 1u) && (v & 0x7F800000u) == 0x7F800000u) {
    v &= 0x0000FFFFu;
    found = true;
  }
  return v;
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// kCluster: the splits of a tile are the CTAs of a cluster and merge through
// distributed shared memory.
template <int kDh, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<kDh>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ float s_bias[C::kStages][kKeys];
  __shared__ float s_m[4][kRows], s_l[4][kRows];
  __shared__ PagedTile s_tile;
  __shared__ int s_found;
  __shared__ float2 s_out_ml[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // heads innermost (a page's heads are read at the same time), or the splits
  // where they have to be neighbours
  const unsigned inner = static_cast<unsigned>(kCluster ? a.splits : a.kv.hkv);
  const int b_in = static_cast<int>(blockIdx.x % inner), b_out = static_cast<int>(blockIdx.x / inner);
  const int g = kCluster ? b_out % a.kv.hkv : b_in;
  const int split = kCluster ? b_in : b_out % a.splits;
  const int tile_idx = b_out / (kCluster ? a.kv.hkv : a.splits);
  const int group = a.hq / a.kv.hkv;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 2);  // the fetch (and its bytes), the biases
      mbar_init(&empty[s], 4);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    s_found = 0;
  }
  pdl_wait();
  if (warp == 0) {
    const PagedTile t = find_tile<kRows>(a, tile_idx);
    if (lane == 0) s_tile = t;
  }
  __syncthreads();
  const PagedTile tile = s_tile;
  if (tile.req < 0) return;
  const int n_rows = min(kRows, tile.n * group - tile.row0);
  // keys that the first and the last row of the tile see
  const int min_limit = tile.past + tile.row0 / group + 1;
  const int max_limit = tile.past + (tile.row0 + n_rows - 1) / group + 1;
  const int64_t lo64 = split * a.chunk;
  const int hi = static_cast<int>(min(static_cast<int64_t>(max_limit), lo64 + a.chunk));
  const int blocks = hi > lo64 ? static_cast<int>((hi - lo64 + kKeys - 1) / kKeys) : 0;
  const int lo = static_cast<int>(lo64);  // (not used when behind every key)

  float o[kDh / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int row[2] = {tile.row0 + (lane >> 2), tile.row0 + (lane >> 2) + 8};
  float gain2[2];

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int page = a.kv.page_size;
    const int box = min(page, kKeys);          // rows of a box
    const int n_box = kKeys / box;             // boxes of a block (a power of two)
    const int n_load = n_box * 2 * C::kSubs;   // loads of a block: box, K or V, columns
    const int my_box = lane & (n_box - 1), my_part = lane / n_box;
    // The split's pages, 32 boxes (a group) a load: lane l holds box 32 grp + l
    // (n_pages, read as zeros, where the table is out of range; -1 behind the
    // keys). Two groups are held, so that no fetch waits for the table.
    auto load_group = [&](int grp) -> int {
      const int64_t j64 = lo64 + (static_cast<int64_t>(grp) * 32 + lane) * box;
      if (j64 >= hi) return -1;
      const int j = static_cast<int>(j64);
      const int64_t p = page_of(a, tile.req, j);
      return p < 0 ? static_cast<int>(a.kv.n_pages) : static_cast<int>(p);
    };
    int grp0 = 0, cur = load_group(0), nxt = load_group(1);
    auto page_at = [&](int i, int b) -> int {
      const int idx = i * n_box + b;
      const int p0 = __shfl_sync(0xFFFFFFFFu, cur, idx & 31), p1 = __shfl_sync(0xFFFFFFFFu, nxt, idx & 31);
      return (idx >> 5) == grp0 ? p0 : p1;
    };
    auto bias_at = [&](int i, int key) -> float {
      const int64_t p = page_at(i, key / box);
      if (a.kv.bias == nullptr || p < 0 || p >= a.kv.n_pages) return 0.f;
      const int j = lo + i * kKeys + key;
      return key_bias(__ldg(a.kv.bias + p * a.kv.bias_page_stride + row_in_page(a, j)));
    };
    auto fetch = [&](int i, int s) {
      const int pg = page_at(i, my_box);
      const bool go = pg >= 0 && lane < n_load;
      const int n_live = __popc(__ballot_sync(0xFFFFFFFFu, go));
      if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(n_live * box * 128));
      __syncwarp();
      if (go) {
        const int sub = my_part % C::kSubs, is_v = my_part / C::kSubs;
        const int j = lo + i * kKeys + my_box * box;
        tma_load_4d(is_v ? &tmV : &tmK, &full[s],
                    ring + s * C::kStageBytes + (is_v * C::kSubs + sub) * C::kSub + my_box * box * 128,
                    sub * 64, g, row_in_page(a, j), pg);
      }
    };
    // the ring's first fill at once; then, a block at a time, its biases (read
    // two blocks ahead) and the next fill of its stage
    for (int i = 0; i < C::kStages && i < blocks; ++i) fetch(i, i);
    float b0 = bias_at(0, lane), b1 = bias_at(0, lane + 32);
    float c0 = bias_at(1, lane), c1 = bias_at(1, lane + 32);
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < blocks; ++i) {
      if (((i + 2) * n_box) >> 5 > grp0) {
        ++grp0;
        cur = nxt;
        nxt = load_group(grp0 + 1);
      }
      const float d0 = bias_at(i + 2, lane), d1 = bias_at(i + 2, lane + 32);
      s_bias[s][lane] = b0;
      s_bias[s][lane + 32] = b1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      if (i + C::kStages < blocks) {
        if (!mbar_wait_warp(&empty[s], ph, a.err)) break;
        fetch(i + C::kStages, s);
      }
      b0 = c0;
      b1 = c1;
      c0 = d0;
      c1 = d1;
      if (++s == C::kStages) {
        s = 0;
        ph ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------ consumers
    uint32_t q[kDh / 16][4];
    float scale[2];
    int limit[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool on = (lane >> 2) + 8 * i < n_rows;
      const int h = g * group + row[i] % group;
      scale[i] = kLog2e / (sqrtf(static_cast<float>(kDh)) * (a.tau && on ? __ldg(a.tau + h) : 1.0f));
      gain2[i] = a.gain && a.kv.bias && on ? __ldg(a.gain + h) * kLog2e : 0.0f;
      limit[i] = on ? tile.past + row[i] / group + 1 : 0;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                              static_cast<int64_t>(tile.tok0 + row[i] / group) * a.q_stride +
                                                              h * kDh) + (lane & 3);
#pragma unroll
      for (int kk = 0; kk < kDh / 16; ++kk) {
        q[kk][i] = on ? __ldg(src + kk * 8) : 0u;
        q[kk][i + 2] = on ? __ldg(src + kk * 8 + 4) : 0u;
      }
    }
#pragma unroll
    for (int t = 0; t < kDh / 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    const int key0 = warp * 16;  // this warp's keys of a block
    const int mi = lane >> 3, r8 = lane & 7;
    // ldmatrix rows: K: matrices (keys 0-7 | 8-15) x (columns 0-7 | 8-15);
    // V: the same with the halves of the keys innermost
    const uint32_t k_row = static_cast<uint32_t>((key0 + (mi >> 1) * 8 + r8) * 128);
    const uint32_t v_row = static_cast<uint32_t>((key0 + (mi & 1) * 8 + r8) * 128);
    bool found = false;
    for (int i = 0; i < blocks; ++i) {
      const int s = i % C::kStages;
      if (!mbar_wait_warp(&full[s], (i / C::kStages) & 1, a.err)) break;
      const uint32_t kb = smem_addr(ring + s * C::kStageBytes), vb = kb + C::kSubs * C::kSub;
      float sc[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < kDh / 16; ++kk) {
        uint32_t b[4];
        ldsm4(kb + (kk >> 2) * C::kSub + k_row + ((((kk & 3) * 2 + (mi & 1)) ^ r8) << 4), b);
        mma16816(sc[0], q[kk], b[0], b[1]);
        mma16816(sc[1], q[kk], b[2], b[3]);
      }
      // logits in log2 units
      const int j0 = lo + i * kKeys + key0;
      uint32_t dead = 0, partial = 0;
      if (a.kv.bias != nullptr) {
        const float mine = s_bias[s][key0 + (lane & 15)];
        partial = __ballot_sync(0xFFFFFFFFu, mine < kRemovableBias) & 0xFFFFu;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 b = *reinterpret_cast<const float2*>(&s_bias[s][key0 + t * 8 + (lane & 3) * 2]);
          sc[t][0] = fmaf(gain2[0], b.x, sc[t][0] * scale[0]);
          sc[t][1] = fmaf(gain2[0], b.y, sc[t][1] * scale[0]);
          sc[t][2] = fmaf(gain2[1], b.x, sc[t][2] * scale[1]);
          sc[t][3] = fmaf(gain2[1], b.y, sc[t][3] * scale[1]);
        }
        if (partial != 0) {  // keys that their bias may remove
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (((partial >> (t * 8 + (lane & 3) * 2 + (e & 1))) & 1u) && sc[t][e] <= kMaskedLogit)
                sc[t][e] = -INFINITY;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][e] *= scale[e >> 1];
      }
      const bool edge = partial != 0 || j0 + 16 > min_limit;
      if (edge) {
        const int past_min = min_limit - j0, past_max = min(max_limit, hi) - j0;
        if (past_min < 16) partial |= past_min <= 0 ? 0xFFFFu : (0xFFFFu << past_min) & 0xFFFFu;
        if (past_max < 16) dead = past_max <= 0 ? 0xFFFFu : (0xFFFFu << past_max) & 0xFFFFu;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + t * 8 + (lane & 3) * 2 + (e & 1);
            if (j >= limit[e >> 1] || j >= hi) sc[t][e] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
        mx[r] = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
      if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] + kRescale || mx[1] > m[1] + kRescale)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 2));
          const float m_new = fmaxf(m[r], mx[r]);
          const float corr = m_new == -INFINITY ? 1.0f : ex2_approx(m[r] - m_new);
          m[r] = m_new;
          l[r] *= corr;
#pragma unroll
          for (int t = 0; t < kDh / 8; ++t) {
            o[t][2 * r] *= corr;
            o[t][2 * r + 1] *= corr;
          }
        }
      }
      const float m_use[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[t][e] = ex2_approx(sc[t][e] - m_use[e >> 1]);
          l[e >> 1] += sc[t][e];
        }
      const uint32_t p[4] = {pack_bf16x2(sc[0][0], sc[0][1]), pack_bf16x2(sc[0][2], sc[0][3]),
                             pack_bf16x2(sc[1][0], sc[1][1]), pack_bf16x2(sc[1][2], sc[1][3])};
#pragma unroll
      for (int t = 0; t < kDh / 16; ++t) {
        uint32_t b[4];
        ldsm4_t(vb + (t >> 2) * C::kSub + v_row + ((((t & 3) * 2 + (mi >> 1)) ^ r8) << 4), b);
        if (edge) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            b[e] = clean_pair(b[e], dead, partial & ~dead, (lane & 3) * 2 + (e & 1) * 8, found);
        }
        mma16816(o[2 * t], p, b[0], b[1]);
        mma16816(o[2 * t + 1], p, b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    if (found) s_found = 1;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
      if ((lane & 3) == 0) {
        s_m[warp][(lane >> 2) + 8 * r] = m[r];
        s_l[warp][(lane >> 2) + 8 * r] = l[r];
      }
    }
  }
  __syncthreads();  // the ring is read, the warps' maxima and sums are there
  float* acc = reinterpret_cast<float*>(ring);  // [4 warps][16 rows][kDh]
  if (warp < 4) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int rr = (lane >> 2) + 8 * r;
      const float top = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
      const float w = state_weight(s_m[warp][rr], s_l[warp][rr], top);
#pragma unroll
      for (int t = 0; t < kDh / 8; ++t)
        *reinterpret_cast<float2*>(acc + (warp * kRows + rr) * kDh + t * 8 + (lane & 3) * 2) =
            make_float2(o[t][2 * r] * w, o[t][2 * r + 1] * w);
    }
  }
  __syncthreads();
  if (s_found) {
    // Infinite or NaN values of keys that only some rows see were left out:
    // each goes to the rows that see it.
    for (int j = lo; j < hi; ++j) {
      const int64_t page = page_of(a, tile.req, j);
      if (page < 0) continue;
      const float b = a.kv.bias ? key_bias(__ldg(a.kv.bias + page * a.kv.bias_page_stride + row_in_page(a, j))) : 0.f;
      if (j < min_limit && !(b < kRemovableBias)) continue;
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.kv.v) + page * a.kv.v_page_stride +
                               (static_cast<int64_t>(row_in_page(a, j)) * a.kv.hkv + g) * kDh;
      for (int d = threadIdx.x; d < kDh; d += kThreads) {
        const float f = __bfloat162float(v[d]);
        if (isfinite(f)) continue;
        for (int r = 0; r < n_rows; ++r) {
          const int rr = tile.row0 + r;
          const float gn = a.gain ? __ldg(a.gain + g * group + rr % group) * kLog2e : 0.f;
          if (j < tile.past + rr / group + 1 && !(gn * b <= kMaskedLogit)) acc[r * kDh + d] += f;
        }
      }
    }
    __syncthreads();
  }
  // 16 rows x kDh columns, four columns a thread
  for (int e = threadIdx.x; e < kRows * (kDh / 4); e += kThreads) {
    const int r = e / (kDh / 4), c = (e % (kDh / 4)) * 4;
    if (r >= n_rows) break;
    const float top = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      sum += s_l[w][r] * state_weight(s_m[w][r], s_l[w][r], top);
      const float4 f = *reinterpret_cast<const float4*>(acc + (w * kRows + r) * kDh + c);
      v = make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w);
    }
    const int rr = tile.row0 + r;
    const int64_t t = tile.tok0 + rr / group;
    const int h = g * group + rr % group;
    if (kCluster) {
      if (c == 0) s_out_ml[r] = make_float2(top, sum);
      *reinterpret_cast<float4*>(acc + 4 * kRows * kDh + r * kDh + c) = v;
    } else if (a.splits > 1) {
      const int64_t at = (split * a.rows + t) * a.hq + h;
      if (c == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(top, sum);
      if (blocks > 0) *reinterpret_cast<float4*>(a.part_o + at * kDh + c) = v;
    } else {
      const bool any = sum != 0.f;  // a row that sees nothing is zero
      const float inv = any ? 1.0f / sum : 0.f;
      if (c == 0 && a.lse != nullptr)
        a.lse[h * a.rows + t] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (t * a.hq + h) * kDh + c) =
          make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    }
  }
  if constexpr (kCluster) {
    cluster_sync();
    // row r is merged by CTA r % splits: the parts' states, in their order
    for (int e = threadIdx.x; e < kRows * (kDh / 4); e += kThreads) {
      const int r = e / (kDh / 4), c = (e % (kDh / 4)) * 4;
      if (r >= n_rows) break;
      if (r % a.splits != split) continue;
      const uint32_t ml_at = smem_addr(&s_out_ml[r]), o_at = smem_addr(acc + 4 * kRows * kDh + r * kDh + c);
      float2 ml[kMaxCluster];
      float4 o4[kMaxCluster];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        ml[q] = make_float2(-INFINITY, 0.f);
        o4[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q < a.splits) {
          ml[q] = ld_cluster2(mapa_shared(ml_at, static_cast<uint32_t>(q)));
          o4[q] = ld_cluster(mapa_shared(o_at, static_cast<uint32_t>(q)));
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) top = fmaxf(top, ml[q].x);
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        const float w = state_weight(ml[q].x, ml[q].y, top);
        sum = fmaf(ml[q].y, w, sum);
        v = make_float4(fmaf(o4[q].x, w, v.x), fmaf(o4[q].y, w, v.y), fmaf(o4[q].z, w, v.z),
                        fmaf(o4[q].w, w, v.w));
      }
      const int rr = tile.row0 + r;
      const int64_t t = tile.tok0 + rr / group;
      const int h = g * group + rr % group;
      const bool any = sum != 0.f;
      const float inv = any ? 1.0f / sum : 0.f;
      if (c == 0 && a.lse != nullptr)
        a.lse[h * a.rows + t] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (t * a.hq + h) * kDh + c) =
          make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    }
    cluster_sync();  // the others have read this CTA's state
  }
}

// ---------------------------------------------------------------- merge
// kWarps warps per (row, head): the splits' unnormalised outputs with weights
// 2^(m_s - max m); warp w adds up splits w, w + kWarps, ... in order, and the
// warps' sums are added in order. A split without keys for the row has sum 0
// and its output is not read. One warp a row where there are few splits; with
// many of them (few rows then) eight, so that they arrive together.
template <typename T, int kDh, int kWarps>
__global__ void __launch_bounds__(256) paged_merge(const __grid_constant__ PagedAttnArgs a) {
  __shared__ float s_acc[kWarps > 1 ? kWarps : 1][kDh];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5);
  const int sub = warp % kWarps;  // this warp's share of the splits
  const int idx = static_cast<int>(blockIdx.x) * (8 / kWarps) + warp / kWarps;
  const int t = idx / a.hq, h = idx % a.hq;
  // Rows behind the last request are left alone. All that is needed is read at
  // once: the request bounds, the states, and the first rows (of splits without
  // keys, too: what memory holds there is not used).
  if (t >= a.rows) return;
  const int row_lo = __ldg(a.cu_q), row_hi = __ldg(a.cu_q + a.batch);
  constexpr int kN = kDh / 32;
  const int64_t step = a.rows * a.hq;
  const float* src = a.part_o + static_cast<int64_t>(idx) * kDh + lane * kN;
  float v[8][kN];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = s0 + i * kWarps;
      const float* p = src + static_cast<int64_t>(s) * step * kDh;
      if constexpr (kN == 4) {
        const float4 f = s < a.splits ? __ldcg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[i][0] = f.x;
        v[i][1] = f.y;
        v[i][2] = f.z;
        v[i][3] = f.w;
      } else {
        const float2 f = s < a.splits ? __ldcg(reinterpret_cast<const float2*>(p)) : make_float2(0.f, 0.f);
        v[i][0] = f.x;
        v[i][1] = f.y;
      }
    }
  };
  load(sub);
  float m0 = -INFINITY, l0 = 0.f, m1 = -INFINITY, l1 = 0.f;
  if (lane < a.splits) {
    const float2 f = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (lane * step + idx) * 2));
    m0 = f.x;
    l0 = f.y;
  }
  if (lane + 32 < a.splits) {
    const float2 f = __ldcg(reinterpret_cast<const float2*>(a.part_ml + ((lane + 32) * step + idx) * 2));
    m1 = f.x;
    l1 = f.y;
  }
  if (t < row_lo || t >= row_hi) return;
  float top = fmaxf(m0, m1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float w0 = state_weight(m0, l0, top), w1 = state_weight(m1, l1, top);
  float sum = l0 * w0 + l1 * w1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  float acc[kN] = {};
  const unsigned live0 = __ballot_sync(0xFFFFFFFFu, l0 != 0.f);
  const unsigned live1 = __ballot_sync(0xFFFFFFFFu, l1 != 0.f);
  for (int s0 = sub; s0 < a.splits; s0 += 8 * kWarps) {
    if (s0 != sub) load(s0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = s0 + i * kWarps;
      const float w = __shfl_sync(0xFFFFFFFFu, s < 32 ? w0 : w1, s & 31);
      if (s < a.splits && (((s < 32 ? live0 : live1) >> (s & 31)) & 1u)) {
#pragma unroll
        for (int e = 0; e < kN; ++e) acc[e] = fmaf(v[i][e], w, acc[e]);
      }
    }
  }
  if constexpr (kWarps > 1) {  // (the whole block has one row: no warp left above)
#pragma unroll
    for (int e = 0; e < kN; ++e) s_acc[sub][lane * kN + e] = acc[e];
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int e = 0; e < kN; ++e)
      for (int w = 1; w < kWarps; ++w) acc[e] += s_acc[w][lane * kN + e];
  }
  const bool any = sum != 0.f;
  const float inv = any ? 1.0f / sum : 0.f;
  if (lane == 0 && a.lse != nullptr)
    a.lse[h * a.rows + t] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
  T* out = static_cast<T*>(a.out) + static_cast<int64_t>(idx) * kDh + lane * kN;
#pragma unroll
  for (int e = 0; e < kN; e += 2) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(out + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

template <typename T, int kDh>
cudaError_t merge(const PagedAttnArgs& a, cudaStream_t st) {
  const int64_t n = a.rows * a.hq;
  // (4096 keys in 33 splits, 16 rows: 13.1 us with one warp, 4.7 with eight)
  if (a.splits <= 2 || (a.splits <= 8 && n > 16 * num_sms()))
    return launch_pdl(paged_merge<T, kDh, 1>, dim3(static_cast<unsigned>((n + 7) / 8)), dim3(256), 0, st, a);
  return launch_pdl(paged_merge<T, kDh, 8>, dim3(static_cast<unsigned>(n)), dim3(256), 0, st, a);
}

template <int kDh>
cudaError_t run(const PagedAttnArgs& a, int64_t tiles, bool cluster, cudaStream_t st) {
  using C = Cfg<kDh>;
  CUtensorMap tk, tv;
  const int box = a.kv.page_size < kKeys ? a.kv.page_size : kKeys;
  if (!make_tmap_pages_bf16(&tk, a.kv.k, kDh, a.kv.hkv, a.kv.page_size, a.kv.n_pages,
                            a.kv.k_page_stride, box) ||
      !make_tmap_pages_bf16(&tv, a.kv.v, kDh, a.kv.hkv, a.kv.page_size, a.kv.n_pages,
                            a.kv.v_page_stride, box))
    return cudaErrorInvalidValue;
  const int64_t grid = tiles * a.splits * a.kv.hkv;
  auto launch = [&](auto kern, int cluster) -> cudaError_t {
    TG_CUDA_TRY(set_smem_attr_once(reinterpret_cast<const void*>(kern), static_cast<int>(C::kSmem)));
    if (cluster > 8) {  // once for each device
      static std::atomic<uint64_t> allowed{0};
      int dev = 0;
      TG_CUDA_TRY(cudaGetDevice(&dev));
      const uint64_t bit = uint64_t(1) << (dev & 63);
      if (!(allowed.load() & bit)) {
        TG_CUDA_TRY(cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
        allowed.fetch_or(bit);
      }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, a);
  };
  return cluster ? launch(paged_decode<kDh, true>, a.splits) : launch(paged_decode<kDh, false>, 1);
}

}  // namespace

cudaError_t launch_paged_merge(const PagedAttnArgs& a, bool bf16, cudaStream_t st) {
  if (bf16) return a.kv.dh == 128 ? merge<__nv_bfloat16, 128>(a, st) : merge<__nv_bfloat16, 64>(a, st);
  return a.kv.dh == 128 ? merge<float, 128>(a, st) : merge<float, 64>(a, st);
}

cudaError_t launch_paged_decode(PagedAttnArgs a, void* ws, cudaStream_t st) {
  const int64_t tiles = a.tiles = paged_row_tiles(a.rows, a.batch, a.hq, a.kv.hkv, kRows);
  const int64_t jobs = tiles * a.kv.hkv;
  // Few jobs over keys that 16 splits of 128 hold: a cluster for each, which
  // merges its splits itself (one token, 8 KV heads: 1000 keys 8.8 us, 2000
  // keys 9.2; merged by a second kernel 11.0 and 10.0. Over 4096 keys, 16
  // splits no longer draw on enough SMs: 15.4 against 13.5).
  int cluster = kMaxCluster;
  while (cluster > 1 && jobs * cluster > 2 * num_sms()) cluster /= 2;
  const int64_t piece = (a.max_kv + cluster - 1) / cluster;
  if (cluster > 1 && piece <= 128) {
    while (cluster > 1 && (cluster / 2) * 128 >= a.max_kv) cluster /= 2;
    a.splits = cluster;
    a.chunk = ((a.max_kv + cluster - 1) / cluster + kKeys - 1) / kKeys * kKeys;
    a.chunk0 = a.chunk;
    return a.kv.dh == 128 ? run<128>(a, tiles, cluster > 1, st) : run<64>(a, tiles, cluster > 1, st);
  }
  // Splits for every SM's two CTAs, of 128 keys at least. Few jobs, whose pieces
  // are short: one wave of them (2 requests of 1000 to 9000 keys, 16 jobs: 16
  // splits 23 us, 37 27; 4 requests of 2000, 32 jobs: 9 splits 18, 18 22). More:
  // two, since the pieces of short requests leave their SMs idle (30 requests of
  // 1000 to 9000 keys, 60 jobs: 9 splits 51, 4 65). Long ones in pieces of 4096 keys,
  // so that the last CTAs to finish have little left (64 requests of 500 to 32768
  // keys: pieces of 1024 keys 754 us, 2048 666, 4096 643, 8192 649).
  const int most = paged_max_splits(a.rows, a.hq, a.kv.dh);
  const int64_t waves = a.batch == 1 || 8 * jobs <= 2 * num_sms() ? 1 : 2;
  const int64_t want = std::max<int64_t>(1, waves * 2 * num_sms() / jobs);
  int64_t chunk = std::max<int64_t>(128, (a.max_kv + want - 1) / want);
  if (chunk > 4096) chunk = 4096;
  chunk = std::max<int64_t>(chunk, (a.max_kv + most - 1) / most);
  a.chunk = (chunk + kKeys - 1) / kKeys * kKeys;
  a.chunk0 = a.chunk;
  a.splits = static_cast<int>((a.max_kv + a.chunk - 1) / a.chunk);
  paged_partials(&a, ws);
  const cudaError_t e = a.kv.dh == 128 ? run<128>(a, tiles, false, st) : run<64>(a, tiles, false, st);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_paged_merge(a, true, st);
}

}  // namespace tg
