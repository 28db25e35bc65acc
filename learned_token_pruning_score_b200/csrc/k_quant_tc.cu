// k_quant_tc.cu -- the 8-bit projection product on the 5th-generation tensor
// cores (sm_100a), tg_linear_quantized:
//
//   y[i, j] = (sum_k xq[i, k] wq[j, k]) xs[i] ws[j] (+ residual[i, j])
//
// tcgen05.mma kind::i8 (signed 8-bit operands, 32-bit integer accumulators in
// TMEM): the sum is exact, so the order of its terms, and how it is split,
// never changes a result. Both operands are K-major with 128-byte rows of 128
// integers, swizzled, as TMA lays them down; columns past k and rows past m
// or n are read as zeros.
//
// Two kernels, chosen by the rows of x:
//   wide    persistent CTA pairs, 256 x 256 tiles (cta_group::2), for the
//           chunks of a prefill: bound by the tensor pipe.
//   narrow  up to 128 rows of x a tile: the weights are the M operand (128
//           output channels a CTA), the rows of x the N operand, and a cluster
//           of up to 8 CTAs splits k, so that a decoding batch's weights stream
//           through every SM; the partial sums meet through distributed shared
//           memory. Bound by HBM (each weight read once).
#include <atomic>
#include <type_traits>

#include "tg_device.cuh"
#include "tg_internal.h"

namespace tg {
namespace {

// Instruction descriptor of tcgen05.mma kind::i8: signed 8-bit A and B (both
// K-major), 32-bit integer accumulator, shape M x N.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int m, int n) {
  return (2u << 4)                                   // accumulator format: s32
         | (1u << 7)                                 // A format: s8
         | (1u << 10)                                // B format: s8
         | (static_cast<uint32_t>(n >> 3) << 17)     // N / 8
         | (static_cast<uint32_t>(m >> 4) << 24);    // M / 16
}

__device__ __forceinline__ void umma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_i8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

constexpr int kBK = 128;       // integers (bytes) of k per stage: one swizzled row
constexpr int kThreads = 256;

struct Params {
  int64_t m;
  int n, k;
  const float* xs;
  const float* ws;
  const void* residual;
  void* y;
  int tiles_m, tiles_n;
  int stages;  // narrow
  int cols;    // narrow: columns of the N operand (rows of x of a tile, padded to 16)
  unsigned int* err;
};

// ------------------------------------------------------------------ wide
// Structure and barriers are those of the bf16 GEMM's CTA pairs (k_gemm_tc.cu):
//   warp 0 (both) TMA into a 6-stage ring of 32 KB (128 rows of x and 128 of w
//   a CTA), warp 1 (rank 0) issues four MMAs of 256 x 256 x 32 a stage into one
//   of two TMEM accumulators, warps 4-7 (both) scale and store the other one.
struct Wide {
  static constexpr int kHalfBytes = 128 * kBK;
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kStages = 6;
  static constexpr int kTmemCols = 512;
  static constexpr int kOffOut = kStages * kStageBytes;  // two 4 KB buffers an epilogue warp
  static constexpr int kOffBar = kOffOut + 4 * 2 * 4096;
  static constexpr size_t kSmem = 1024 + kOffBar + 256;
};

// The residual of a piece of 32 rows x 128 bytes, 4 rows an instruction.
template <typename T>
__device__ __forceinline__ void load_residual(const Params& p, int64_t row0, int col, uint4 (&t)[8]) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int64_t c0 = col + (lane & 7) * (16 / static_cast<int>(sizeof(T)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + 4 * i + (lane >> 3);
    t[i] = make_uint4(0, 0, 0, 0);
    if (r < p.m && c0 < p.n)
      t[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.residual) + r * p.n + c0);
  }
}

// One warp's 32 rows x 128 bytes of outputs (64 bf16 or 32 fp32 columns from
// column `col` on): the accumulators, scaled, plus the residual, into `buf`
// (rows of 128 bytes, 16-byte unit u of row r at u ^ (r & 7), the layout of
// the output map's boxes) and from there by TMA. A thread's own row is a
// piece of 128 bytes far from its neighbour's: stored and read directly it
// costs a sector per thread and instruction, which made the epilogue the
// longer side of a tile at k = 2048 (8192 x 12288: 180 us).
// `ahead` holds the piece's residual and receives the one of the next piece
// (columns from next_col of the rows from next_row), which is on its way
// while this one is scaled (8192 x 2048 x 272 onto a residual: read where it
// is added 44 us, a piece ahead 41, asked into L2 a tile ahead as well 37; two
// pieces ahead 36, with twice the code).
template <typename T>
__device__ __forceinline__ void scale_store(const Params& p, const CUtensorMap* tmY, int64_t row0,
                                            int col, float xs, uint32_t t_col, uint8_t* buf,
                                            uint4 (&ahead)[8], int64_t next_row, int next_col) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // outputs of a 16-byte unit
  constexpr int kCols = 8 * kVec;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const bool res = p.residual != nullptr;
  if (res) {
    if (lane == 0) bulk_wait_read_but_one();  // the store that last used buf has read it
    __syncwarp();
    const int u = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      *reinterpret_cast<uint4*>(buf + r * 128 + ((u ^ (r & 7)) << 4)) = ahead[i];
    }
    load_residual<T>(p, next_row, next_col, ahead);
  } else if (lane == 0) {
    bulk_wait_read_but_one();
  }
  __syncwarp();
  uint8_t* mine = buf + lane * 128;
#pragma unroll
  for (int h = 0; h < kCols / 32; ++h) {
    uint32_t acc[32];
    tmem_ld32(t_col + h * 32, acc);
    tmem_wait_ld_dep(acc);
    const int hc = col + h * 32;
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 w = hc < p.n ? __ldg(reinterpret_cast<const float4*>(p.ws + hc + j))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
      v[j] = static_cast<float>(static_cast<int>(acc[j])) * xs * w.x;
      v[j + 1] = static_cast<float>(static_cast<int>(acc[j + 1])) * xs * w.y;
      v[j + 2] = static_cast<float>(static_cast<int>(acc[j + 2])) * xs * w.z;
      v[j + 3] = static_cast<float>(static_cast<int>(acc[j + 3])) * xs * w.w;
    }
#pragma unroll
    for (int q = 0; q < 32 / kVec; ++q) {
      uint4* at = reinterpret_cast<uint4*>(mine + (((h * 32 / kVec + q) ^ (lane & 7)) << 4));
      if constexpr (sizeof(T) == 4) {
        if (res) {
          const uint4 r = *at;
          v[4 * q] += __uint_as_float(r.x);
          v[4 * q + 1] += __uint_as_float(r.y);
          v[4 * q + 2] += __uint_as_float(r.z);
          v[4 * q + 3] += __uint_as_float(r.w);
        }
        *at = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                         __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
      } else {
        if (res) {
          const uint4 r = *at;
          const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(e[i]);
            v[8 * q + 2 * i] += f.x;
            v[8 * q + 2 * i + 1] += f.y;
          }
        }
        *at = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                         pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                         pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
      }
    }
  }
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {  // rows past m and columns past n are not written
    if (row0 < p.m && col < p.n) tma_store_2d(tmY, buf, col, static_cast<int>(row0));
    bulk_commit();
  }
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_i8_wide(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Params p) {
  using C = Wide;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t* tiles = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 8);  // rank 0: 4 epilogue warps x 2 CTAs
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, C::kTmemCols);
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  const int num_tiles = p.tiles_m * p.tiles_n;
  const int num_kb = (p.k + kBK - 1) / kBK;
  const int pair = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);

  if (warp == 0 && lane == 0) {
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = pair; tile < num_tiles && ok; tile += n_pairs) {
      const int mb = tile / p.tiles_n, nb = tile % p.tiles_n;
      const int x_row = mb * 256 + static_cast<int>(rank) * 128;
      const int w_row = nb * 256 + static_cast<int>(rank) * 128;
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!mbar_wait(&empty[s], ph ^ 1u, p.err)) { ok = false; break; }
        uint8_t* dst = tiles + size_t(s) * C::kStageBytes;
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStageBytes);
        const uint32_t bar = mapa_shared(smem_addr(&full[s]), 0);
        tma_load_2d_pair(&tmX, bar, dst, kb * kBK, x_row);
        tma_load_2d_pair(&tmW, bar, dst + C::kHalfBytes, kb * kBK, w_row);
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
    }
    // Every stage this CTA filled is released (by a commit that writes into
    // this CTA's shared memory) before the CTA may exit.
    for (int i = 0; i < C::kStages && ok; ++i) {
      if (!mbar_wait(&empty[s], ph ^ 1u, p.err)) break;
      if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr uint32_t idesc = idesc_s8_s32(256, 256);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    int it = 0;
    for (int tile = pair; tile < num_tiles && ok; tile += n_pairs, ++it) {
      const int a = it & 1;
      if (!mbar_wait(&acc_empty[a], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, p.err)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(a * 256);
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!mbar_wait(&full[s], ph, p.err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t x_addr = smem_addr(tiles + size_t(s) * C::kStageBytes);
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)
          umma_i8_ss_pair(d_tmem, sdesc_kmajor_sw128(x_addr + kk * 32),
                          sdesc_kmajor_sw128(x_addr + C::kHalfBytes + kk * 32), idesc,
                          (kb | kk) != 0 ? 1u : 0u);
        const uint32_t e = smem_addr(&empty[s]);
        umma_commit_pair(e);
        umma_commit_pair(mapa_shared(e, 1));
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      if (ok) {
        const uint32_t f = smem_addr(&acc_full[a]);
        umma_commit_pair(f);
        umma_commit_pair(mapa_shared(f, 1));
      }
    }
    // Both accumulators released by both CTAs' epilogues before exit.
    for (int i = 0; i < 2 && ok; ++i, ++it)
      if (!mbar_wait(&acc_empty[it & 1], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, p.err)) break;
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    uint8_t* out = tiles + C::kOffOut + quarter * 8192;
    constexpr int kStep = 128 / static_cast<int>(sizeof(T));
    int flip = 0;
    int it = 0;
    auto first_row = [&](int tile) {
      return static_cast<int64_t>(tile / p.tiles_n) * 256 + rank * 128 + quarter * 32;
    };
    // A piece ahead leaves too few bytes on their way from DRAM: the next tile's
    // residual is asked into L2 a tile ahead, each lane's row of it.
    auto prefetch = [&](int tile) {
      const int64_t r = first_row(tile) + lane;
      const int col = tile % p.tiles_n * 256;
      if (r >= p.m) return;
      const T* at = static_cast<const T*>(p.residual) + r * p.n + col;
#pragma unroll
      for (int c = 0; c < 256; c += kStep)
        if (col + c < p.n) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c));
    };
    if (p.residual != nullptr) prefetch(pair);
    uint4 ahead[8];
    if (p.residual != nullptr) load_residual<T>(p, first_row(pair), pair % p.tiles_n * 256, ahead);
    for (int tile = pair; tile < num_tiles; tile += n_pairs, ++it) {
      const int nb = tile % p.tiles_n;
      const int a = it & 1;
      if (!mbar_wait_warp(&acc_full[a], static_cast<uint32_t>(it >> 1) & 1u, p.err)) break;
      tc_fence_after();
      const int64_t row0 = first_row(tile);
      // (behind the last tile: rows past m, of which nothing is read)
      const int64_t next_row = tile + n_pairs < num_tiles ? first_row(tile + n_pairs) : p.m;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(a * 256);
      const float xs = row0 + lane < p.m ? __ldg(p.xs + row0 + lane) : 0.f;
      if (p.residual != nullptr && tile + n_pairs < num_tiles) prefetch(tile + n_pairs);
#pragma unroll 1
      for (int c = 0; c < 256; c += kStep) {
        const bool last = c + kStep == 256;
        scale_store<T>(p, &tmY, row0, nb * 256 + c, xs, t_row + c, out + (flip ? 4096 : 0), ahead,
                       last ? next_row : row0,
                       last ? (tile + n_pairs) % p.tiles_n * 256 : nb * 256 + c + kStep);
        flip ^= 1;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_addr(&acc_empty[a]), 0));
    }
    if (lane == 0) bulk_wait_read_all();  // the buffers are read before the CTA may exit
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  __syncwarp();
  if (warp == 2) tmem_dealloc_pair(tmem_base, C::kTmemCols);
}

// ------------------------------------------------------------------ narrow
// One CTA: 128 output channels (M, TMEM lanes) x `cols` rows of x (N, TMEM
// columns) over its share of k. A cluster (z) shares the tile; each CTA lays
// its 32-bit sums out in shared memory, [column][lane], and adds up and
// stores every cluster-size-th group of columns.
struct Narrow {
  static constexpr int kWBytes = 128 * kBK;
  // two CTAs on an SM, of one call or of one and the next
  static constexpr int kRing = 96 * 1024;
  static constexpr int kMaxCols = 128;
  static constexpr int kMaxStages = 5;
  static constexpr size_t kSmem = 1024 + kRing + 256;
};
static_assert(Narrow::kMaxCols * 128 * 4 <= Narrow::kRing, "the sums reuse the ring");

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_i8_narrow(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ Params p) {
  using C = Narrow;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t* tiles = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + C::kRing);
  uint64_t* empty = full + C::kMaxStages;
  uint64_t* acc_full = empty + C::kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  __shared__ int s_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(gridDim.z), part = static_cast<int>(blockIdx.z);
  const int w_row = static_cast<int>(blockIdx.x) * 128;
  const int64_t x_row = static_cast<int64_t>(blockIdx.y) * C::kMaxCols;
  const int stage_bytes = C::kWBytes + p.cols * kBK;
  const int num_kb = (p.k + kBK - 1) / kBK;
  const int kb_lo = part * num_kb / split, kb_hi = (part + 1) * num_kb / split;
  uint32_t tmem_cols = 32;
  while (static_cast<int>(tmem_cols) < p.cols) tmem_cols *= 2;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    s_bad = 0;
  }
  if (warp == 2) tmem_alloc(tmem_slot, tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  // What the end needs besides the sums is read now: the scales of this lane's
  // four channels, and for the warp's first two columns (part 8 + warp, then
  // split 8 on) the row's scale and the residual.
  const int cols = static_cast<int>(min(static_cast<int64_t>(p.cols), p.m - x_row));
  const int ch = w_row + lane * 4;
  const int c_first = part * 8 + warp, c_step = split * 8;
  const bool ch_ok = ch < p.n;
  using Quad = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;  // four outputs
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  float xs[2];
  Quad res[2];
  auto column = [&](int c, float& x, Quad& r) {
    x = 0.f;
    r = Quad{};
    if (ch_ok && c < cols) {
      x = __ldg(p.xs + x_row + c);
      if (p.residual != nullptr)
        r = *reinterpret_cast<const Quad*>(static_cast<const T*>(p.residual) + (x_row + c) * p.n + ch);
    }
  };
  if (ch_ok) w = __ldg(reinterpret_cast<const float4*>(p.ws + ch));
  column(c_first, xs[0], res[0]);
  column(c_first + c_step, xs[1], res[1]);
  if (warp == 0 && lane == 0) {
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      if (!mbar_wait(&empty[s], ph ^ 1u, p.err)) break;
      uint8_t* dst = tiles + s * stage_bytes;
      mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(stage_bytes));
      tma_load_2d(&tmW, &full[s], dst, kb * kBK, w_row);
      tma_load_2d(&tmX, &full[s], dst + C::kWBytes, kb * kBK, static_cast<int>(x_row));
      if (++s == p.stages) { s = 0; ph ^= 1u; }
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_s8_s32(128, p.cols);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      if (!mbar_wait(&full[s], ph, p.err)) { ok = false; break; }
      tc_fence_after();
      const uint32_t w_addr = smem_addr(tiles + s * stage_bytes);
#pragma unroll
      for (int kk = 0; kk < kBK / 32; ++kk)
        umma_i8_ss(tmem, sdesc_kmajor_sw128(w_addr + kk * 32),
                   sdesc_kmajor_sw128(w_addr + C::kWBytes + kk * 32), idesc,
                   (kb > kb_lo || kk > 0) ? 1u : 0u);
      umma_commit(&empty[s]);
      if (++s == p.stages) { s = 0; ph ^= 1u; }
    }
    if (ok) umma_commit(acc_full);
    else s_bad = 1;  // the sums are not complete: this part's columns are not stored
  }
  // The ring is free once the last MMA has read it: the sums go there.
  int* sums = reinterpret_cast<int*>(tiles);
  __syncwarp();
  if (warp >= 4) {
    if (mbar_wait_warp(acc_full, 0, p.err)) {
      tc_fence_after();
      const int quarter = warp & 3;
      for (int c = 0; c < p.cols; c += 16) {
        uint32_t acc[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c), acc);
        tmem_wait_ld_dep16(acc);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sums[(c + i) * 128 + quarter * 32 + lane] = static_cast<int>(acc[i]);
      }
    } else {
      s_bad = 1;
    }
  }
  tc_fence_before();
  if (split > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (s_bad == 0 && ch_ok) {
    // one warp per column: lane's four channels, the parts' sums in their order
#pragma unroll 1
    for (int c = c_first, k = 0; c < cols; c += c_step, ++k) {
      if (k >= 2) column(c, xs[0], res[0]);
      const float x = k == 1 ? xs[1] : xs[0];
      const Quad r = k == 1 ? res[1] : res[0];
      const uint32_t at = smem_addr(sums + c * 128 + lane * 4);
      int4 a = make_int4(0, 0, 0, 0);
      if (split > 1) {
        int4 b[8];  // all on their way before the first is added
#pragma unroll
        for (int q = 0; q < 8; ++q)
          b[q] = q < split ? ld_cluster_int4(mapa_shared(at, static_cast<uint32_t>(q)))
                           : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          a.x += b[q].x;
          a.y += b[q].y;
          a.z += b[q].z;
          a.w += b[q].w;
        }
      } else {
        a = *reinterpret_cast<const int4*>(sums + c * 128 + lane * 4);
      }
      float4 v = make_float4(static_cast<float>(a.x) * x * w.x, static_cast<float>(a.y) * x * w.y,
                             static_cast<float>(a.z) * x * w.z, static_cast<float>(a.w) * x * w.w);
      T* y = static_cast<T*>(p.y) + (x_row + c) * p.n + ch;
      const bool add = p.residual != nullptr;
      if constexpr (sizeof(T) == 4) {
        if (add)
          v = make_float4(v.x + __uint_as_float(r.x), v.y + __uint_as_float(r.y),
                          v.z + __uint_as_float(r.z), v.w + __uint_as_float(r.w));
        *reinterpret_cast<float4*>(y) = v;
      } else {
        if (add) {
          const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
          const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
          v = make_float4(v.x + lo.x, v.y + lo.y, v.z + hi.x, v.w + hi.y);
        }
        *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      }
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync();  // the other parts have read this CTA's sums
  else __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, tmem_cols);
}

template <typename T>
cudaError_t run_wide(const QuantGemmArgs& g, cudaStream_t st) {
  CUtensorMap tx, tw, ty;
  if (!make_tmap_2d_u8(&tx, g.x, g.m, g.k, 128) || !make_tmap_2d_u8(&tw, g.w, g.n, g.k, 128) ||
      !make_tmap_2d_out(&ty, g.y, g.m, g.n, g.bf16, 32))
    return cudaErrorInvalidValue;
  Params p{};
  p.m = g.m;
  p.n = g.n;
  p.k = g.k;
  p.xs = g.xs;
  p.ws = g.ws;
  p.residual = g.residual;
  p.y = g.y;
  p.tiles_m = static_cast<int>((g.m + 255) / 256);
  p.tiles_n = (g.n + 255) / 256;
  p.err = device_error_word();
  auto kern = gemm_i8_wide<T>;
  TG_CUDA_TRY(set_smem_attr_once(reinterpret_cast<const void*>(kern), static_cast<int>(Wide::kSmem)));
  // Persistent grid: as many pairs as can be resident at once (the SMs of a
  // pair must share a TPC, so this can be below num_sms() / 2).
  constexpr int kMaxDevices = 64;
  static std::atomic<int> resident[kMaxDevices];
  int dev = 0;
  cudaGetDevice(&dev);
  int max_pairs = (dev >= 0 && dev < kMaxDevices) ? resident[dev].load() : 0;
  if (max_pairs <= 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms() & ~1), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Wide::kSmem;
    cfg.stream = st;
    if (cudaOccupancyMaxActiveClusters(&max_pairs, kern, &cfg) != cudaSuccess || max_pairs <= 0) {
      cudaGetLastError();
      max_pairs = num_sms() / 2;
    }
    if (dev >= 0 && dev < kMaxDevices) resident[dev].store(max_pairs);
  }
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const unsigned pairs = static_cast<unsigned>(tiles < max_pairs ? tiles : max_pairs);
  return launch_pdl(kern, dim3(2 * pairs), dim3(kThreads), Wide::kSmem, st, tx, tw, ty, p);
}

template <typename T>
cudaError_t run_narrow(const QuantGemmArgs& g, cudaStream_t st) {
  using C = Narrow;
  Params p{};
  p.m = g.m;
  p.n = g.n;
  p.k = g.k;
  p.xs = g.xs;
  p.ws = g.ws;
  p.residual = g.residual;
  p.y = g.y;
  p.cols = g.m >= C::kMaxCols ? C::kMaxCols : static_cast<int>((g.m + 15) / 16 * 16);
  p.err = device_error_word();
  CUtensorMap tx, tw;
  if (!make_tmap_2d_u8(&tx, g.x, g.m, g.k, p.cols) || !make_tmap_2d_u8(&tw, g.w, g.n, g.k, 128))
    return cudaErrorInvalidValue;
  const int tiles_n = (g.n + 127) / 128;
  const int tiles_m = static_cast<int>((g.m + C::kMaxCols - 1) / C::kMaxCols);
  // k is split while one CTA an SM holds the parts. Into four as soon as there
  // are four blocks of k (64 x 2048 x 608: 1 part 6.1 us, 2 parts 7.3, 4 parts
  // 5.8; 128 x 2048 x 4096: 16.4, 14.6, 9.3); into eight where SMs stay idle or
  // the parts are long (64 x 1024 x 1024: 4 parts 5.7, 8 parts 5.2; 128 x 2048 x
  // 2048, 128 CTAs: 8.2 and 8.9; 64 x 2048 x 6144: 8.5 and 7.9). Two parts add up
  // half a tile each, which only a long k repays (512 x 2048: k = 2048 12.3 us,
  // 2 parts 13.6; 6144 21.6 and 18.8).
  const int num_kb = (g.k + kBK - 1) / kBK;
  const int tiles = tiles_n * tiles_m;
  int split = 1;
  if (tiles * 8 <= num_sms() && num_kb >= (tiles * 16 <= num_sms() ? 8 : 32)) split = 8;
  else if (tiles * 4 <= num_sms() && num_kb >= 4) split = 4;
  else if (tiles * 2 <= num_sms() && num_kb >= 28) split = 2;
  p.stages = C::kRing / (C::kWBytes + p.cols * kBK);
  if (p.stages > C::kMaxStages) p.stages = C::kMaxStages;
  auto kern = gemm_i8_narrow<T>;
  TG_CUDA_TRY(set_smem_attr_once(reinterpret_cast<const void*>(kern), static_cast<int>(C::kSmem)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles_n), static_cast<unsigned>(tiles_m),
                     static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(split);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tx, tw, p);
}

}  // namespace

cudaError_t launch_quant_gemm_wide(const QuantGemmArgs& g, cudaStream_t st) {
  return g.bf16 ? run_wide<__nv_bfloat16>(g, st) : run_wide<float>(g, st);
}

cudaError_t launch_quant_gemm_narrow(const QuantGemmArgs& g, cudaStream_t st) {
  return g.bf16 ? run_narrow<__nv_bfloat16>(g, st) : run_narrow<float>(g, st);
}

}  // namespace tg
