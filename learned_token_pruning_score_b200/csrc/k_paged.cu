// k_paged.cu -- the paged key/value cache of a serving process: appending new
// rows to it (tg_paged_append) and the CUDA-core attention over it
// (tg_paged_attn, fp32).
//
// The cache is a pool of pages of page_size rows; request b's row j sits in
// page table[b][j / page_size], row j % page_size. Layers above the gate hold
// the kept tokens' rows with their gate bias logsigmoid(s_j), layers at or
// below it every row; generated rows have bias 0 (Tencent Cloud article
// "TokenGate：端到端可训练的 Token 剪枝机制，让大模型 Prefill 提速 11.3 倍", sections
// "TokenGate 提前筛选 Token" and "TokenGate 的工程验证仍有限": generated tokens are
// never pruned, and the bias fixed at prefill acts as an additive mask).
//
// Lengths, chunk offsets, positions and page numbers are device data: they are
// checked where they are used, and a row or page out of range is skipped and
// reported in the device error word.
#include <algorithm>

#include "tg_device.cuh"
#include "tg_internal.h"
#include "tg_paged.cuh"

namespace tg {
namespace {

// a 16-byte vector as pairs of fp32
__device__ __forceinline__ void unpack2(const uint4& u, float2 (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack2(const uint4& u, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 repack2(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                    pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ uint4 repack2(const float2 (&f)[2]) {
  return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                    __float_as_uint(f[1].y));
}

// ---------------------------------------------------------------- append
// y = x / sqrt(mean(x^2) + eps) * w per head (when a weight is given), then
// the rotate-half rotation by pos * theta_i; q to q_out, k and v to their
// pages, bias = logsigmoid(s). Bound by HBM: every row in once, out once.
// One head is held by dh / 2 / kVec lanes (8 lanes of bf16 at dh 128), each
// with one 16-byte vector of the first half and the matching one of the
// second, so that rotation pairs meet in one thread and the norm needs three
// shuffles. A CTA takes `tok` tokens: their angles (fp64, from the host's
// theta_i, so that no thread evaluates a power) go to shared memory first.
// CTAs run through groups of `tok` tokens: while one group is worked on, the next
// one's vectors are on their way to shared memory (cp.async; each thread reads
// back what it fetched itself) and its angles are formed, and a ninth warp finds
// the pages of the one after that. (Loads into registers instead, a group a CTA:
// 113 us for 32768 tokens; so 101.)
constexpr int kAppThreads = 256, kAppTok = 4;

// 16 bytes global -> shared
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

template <typename T, int kDh>
struct AppSmem {
  uint4 ring[2][kAppTok][2][kAppThreads];  // halves of a head's row, by thread
  // by quads of a thread's frequencies (app_at): lanes read side by side
  float cos[2][kAppTok][kDh / 2], sin[2][kAppTok][kDh / 2];
  float norm[2][2][kDh / 2];               // weights of q and k (read as they are aligned), halves
  int64_t page[3][kAppTok];                // page of the token's row, or -1 (skip)
  int64_t pos[3][kAppTok];
  int row[3][kAppTok];
};
// Place of frequency f, of which a thread has kVec in a row.
template <int kDh, int kVec>
__device__ __forceinline__ int app_at(int f) {
  constexpr int kLanes = kDh / 2 / kVec;
  const int sub = f / kVec, e = f % kVec;
  return (e >> 2) * (kLanes * 4) + sub * 4 + (e & 3);
}

template <typename T, int kDh>
__global__ void __launch_bounds__(kAppThreads + 32, 3)
    paged_append(const __grid_constant__ PagedAppendArgs a, int tok) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  AppSmem<T, kDh>& sm = *reinterpret_cast<AppSmem<T, kDh>*>(smem_raw);
  pdl_trigger();
  pdl_wait();
  constexpr int kHalf = kDh / 2;
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kPairs = kVec / 2;
  constexpr int kLanes = kHalf / kVec;           // lanes of one head
  constexpr int kHeads = kAppThreads / kLanes;   // heads of one pass
  const int tid = threadIdx.x, lane = tid & 31;
  const bool finder = tid >= kAppThreads;        // the ninth warp
  const int64_t groups = (a.rows + tok - 1) / tok;
  // rows from cu_q[batch] on belong to no request: neither read nor written
  const int64_t total = min(a.rows, static_cast<int64_t>(__ldg(a.cu_q + a.batch)));
  const int sub = tid % kLanes, d0 = sub * kVec;
  const int heads = a.hq + 2 * a.kv.hkv;
  // head h0's row of token 0: q, k and v in turn
  auto source = [&](int h0, int64_t& stride) -> const T* {
    if (h0 < a.hq) {
      stride = a.q_stride;
      return static_cast<const T*>(a.q) + h0 * kDh + d0;
    }
    h0 -= a.hq;
    if (h0 < a.kv.hkv) {
      stride = a.k_stride;
      return static_cast<const T*>(a.k) + h0 * kDh + d0;
    }
    stride = a.v_stride;
    return static_cast<const T*>(a.v) + (h0 - a.kv.hkv) * kDh + d0;
  };
  int64_t stride0 = 0;
  const T* src0 = !finder && tid / kLanes < heads ? source(tid / kLanes, stride0) : nullptr;
  auto fetch = [&](int64_t group, int st) {
#pragma unroll
    for (int i = 0; i < kAppTok; ++i) {
      const int64_t t = group * tok + i;
      if (i < tok && t < total && src0 != nullptr) {
        cp_async16(&sm.ring[st][i][0][tid], src0 + t * stride0);
        cp_async16(&sm.ring[st][i][1][tid], src0 + t * stride0 + kHalf);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // pages, rows, positions and gate biases of a group; lane i has token i
  auto find = [&](int64_t group, int st) {
    const int64_t t = group * tok + lane;
    const bool on = lane < tok && t < total;
    int64_t pos = on && a.rotate && a.pos != nullptr ? __ldg(a.pos + t) : 0;
    const float s_t = on && a.s != nullptr && a.kv.bias != nullptr ? __ldg(a.s + t) : 0.f;
    // Its request: the number of requests that end at or before it (cu_q ascends).
    // The first token's is searched (a count over all of 2000 requests: 60 us, so
    // 10); the others are counted from there.
    int skip = 0, left = a.batch;
    narrow_requests([&](int b) { return __ldg(a.cu_q + b); }, group * tok, skip, left);
    int req = skip;
    int64_t lo = __ldg(a.cu_q + skip), hi = -1, len = 0;
    for (int b0 = skip; b0 < a.batch; b0 += 32) {
      const bool there = b0 + lane < a.batch;
      const int end = there ? __ldg(a.cu_q + b0 + lane + 1) : 0x7FFFFFFF;
      const int l = there ? __ldg(a.kv_len + b0 + lane) : 0;
#pragma unroll
      for (int i = 0; i < kAppTok; ++i) {
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, !there || end > group * tok + i));
        const int first = 32 - n;  // (the ones before it have ended)
        const int e = __shfl_sync(0xFFFFFFFFu, end, first & 31);
        const int before = __shfl_sync(0xFFFFFFFFu, end, (first + 31) & 31);
        const int el = __shfl_sync(0xFFFFFFFFu, l, first & 31);
        if (lane == i && hi < 0) {
          req += first;
          if (first > 0) lo = before;
          if (first < 32) {
            hi = e;
            len = el;
          }
        }
      }
      if (__all_sync(0xFFFFFFFFu, lane >= tok || hi >= 0)) break;
    }
    int64_t page = -1;
    int row = 0;
    if (on) {
      bool bad = req >= a.batch;  // (offsets that do not ascend)
      if (!bad) {
        const int64_t dst = len - (hi - lo) + (t - lo);
        const int64_t blk = dst >> a.kv.page_shift;
        if (a.pos == nullptr) pos = dst;  // the row's index in its request
        bad = lo > t || dst < 0 || blk >= a.kv.table_stride;
        if (!bad) {
          page = __ldg(a.kv.table + static_cast<int64_t>(req) * a.kv.table_stride + blk);
          row = static_cast<int>(dst) & (a.kv.page_size - 1);
          bad = page < 0 || page >= a.kv.n_pages;
        }
      }
      if (bad) {
        page = -1;
        report_error(a.err, kErrIndexRange);
      }
      if (page >= 0 && a.kv.bias != nullptr)
        a.kv.bias[page * a.kv.bias_page_stride + row] = a.s ? logsigmoid_f(s_t) : 0.0f;
    }
    if (lane < kAppTok) {
      sm.page[st][lane] = page;
      sm.pos[st][lane] = pos;
      sm.row[st][lane] = row;
    }
  };
  auto angles = [&](int st, int meta) {
    if (!a.rotate) return;
    for (int e = tid; e < tok * kHalf; e += kAppThreads) {
      const int i = e / kHalf, f = e % kHalf;
      const float2 cs = rope_cos_sin_theta(sm.pos[meta][i], a.theta[f]);
      sm.cos[st][i][app_at<kDh, kVec>(f)] = cs.x;
      sm.sin[st][i][app_at<kDh, kVec>(f)] = cs.y;
    }
  };
  // this thread's kVec entries of such a table
  auto entries = [&](const float* table, float2 (&out)[kPairs]) {
#pragma unroll
    for (int q = 0; q < kVec / 4; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(table + q * (kLanes * 4) + sub * 4);
      out[2 * q] = make_float2(v.x, v.y);
      out[2 * q + 1] = make_float2(v.z, v.w);
    }
  };
  const bool norm_any = a.q_norm != nullptr || a.k_norm != nullptr;
  auto work = [&](int64_t group, int st, int meta) {
    // every lane of a warp reaches the shuffles
    for (int pass = 0; pass < heads; pass += kHeads) {
      const int h0 = pass + tid / kLanes;
      const int kind = h0 < a.hq ? 0 : (h0 < a.hq + a.kv.hkv ? 1 : 2);
      const int h = kind == 0 ? h0 : (kind == 1 ? h0 - a.hq : h0 - a.hq - a.kv.hkv);
      const bool norm = kind == 0 ? a.q_norm != nullptr : (kind == 1 && a.k_norm != nullptr);
      int64_t stride = stride0;
      const T* src = pass == 0 ? src0 : h0 < heads ? source(h0, stride) : nullptr;
#pragma unroll 1
      for (int i = 0; i < tok; ++i) {
        const int64_t t = group * tok + i;
        if (t >= total) break;
        uint4 ulo = make_uint4(0, 0, 0, 0), uhi = ulo;
        if (pass == 0) {
          ulo = sm.ring[st][i][0][tid];
          uhi = sm.ring[st][i][1][tid];
        } else if (src != nullptr) {
          ulo = *reinterpret_cast<const uint4*>(src + t * stride);
          uhi = *reinterpret_cast<const uint4*>(src + t * stride + kHalf);
        }
        if (norm_any || a.rotate) {
          float2 lo[kPairs], hi[kPairs];
          unpack2(ulo, lo);
          unpack2(uhi, hi);
          if (norm_any) {
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) s2 = ffma2(lo[e], lo[e], ffma2(hi[e], hi[e], s2));
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            if (norm) {
              const float r = rsqrtf(ss * (1.0f / kDh) + a.eps);
              const float2 r2 = make_float2(r, r);
              float2 wl[kPairs], wh[kPairs];
              entries(sm.norm[kind][0], wl);
              entries(sm.norm[kind][1], wh);
#pragma unroll
              for (int e = 0; e < kPairs; ++e) {
                lo[e] = fmul2(fmul2(lo[e], r2), wl[e]);
                hi[e] = fmul2(fmul2(hi[e], r2), wh[e]);
              }
            }
          }
          if (kind < 2) {
            if (a.rotate) {
              float2 cs[kPairs], sn[kPairs];
              entries(sm.cos[st][i], cs);
              entries(sm.sin[st][i], sn);
#pragma unroll
              for (int e = 0; e < kPairs; ++e) {
                const float2 c = cs[e], s = sn[e], x = lo[e], y = hi[e];
                lo[e] = ffma2(x, c, fmul2(y, make_float2(-s.x, -s.y)));
                hi[e] = ffma2(y, c, fmul2(x, s));
              }
            }
            ulo = repack2(lo);
            uhi = repack2(hi);
          }
        }
        if (h0 >= heads) continue;
        T* dst;
        if (kind == 0) {
          dst = static_cast<T*>(a.q_out) + (t * a.hq + h) * kDh;
        } else {
          const int64_t page = sm.page[meta][i];
          if (page < 0) continue;
          dst = static_cast<T*>(kind == 1 ? a.kv.k : a.kv.v) +
                page * (kind == 1 ? a.kv.k_page_stride : a.kv.v_page_stride) +
                (static_cast<int64_t>(sm.row[meta][i]) * a.kv.hkv + h) * kDh;
        }
        *reinterpret_cast<uint4*>(dst + d0) = ulo;
        *reinterpret_cast<uint4*>(dst + kHalf + d0) = uhi;
      }
    }
  };

  int64_t group = blockIdx.x;
  if (finder) {
    find(group, 0);
  } else {
    fetch(group, 0);
    if (tid < kDh) {
      const int half = tid / kHalf, at = app_at<kDh, kVec>(tid % kHalf);
      if (a.q_norm != nullptr) sm.norm[0][half][at] = __ldg(a.q_norm + tid);
      if (a.k_norm != nullptr) sm.norm[1][half][at] = __ldg(a.k_norm + tid);
    }
  }
  __syncthreads();
  if (!finder) angles(0, 0);
  else if (group + gridDim.x < groups) find(group + gridDim.x, 1);
  __syncthreads();
  for (int st = 0, meta = 0; group < groups; group += gridDim.x, st ^= 1, meta = meta == 2 ? 0 : meta + 1) {
    const int64_t next = group + gridDim.x;
    const int meta1 = meta == 2 ? 0 : meta + 1;
    if (finder) {
      if (next + gridDim.x < groups) find(next + gridDim.x, meta == 0 ? 2 : meta - 1);
    } else {
      if (next < groups) {
        fetch(next, st ^ 1);
        angles(st ^ 1, meta1);
      } else {
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      work(group, st, meta);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- attention, CUDA cores
// One CTA per (32 rows of a request and KV head, KV head, split of the keys); a
// row is a (token, query head of the group) pair, token-major, so that the keys
// are read once for the whole group. Keys go through shared memory 32 at a time,
// the next 32 on their way (cp.async) while these are worked on; thread (ty, tx)
// holds rows 2 ty, 2 ty + 1 and keys tx + 8 i in the logits, columns 4 tx + 32 c
// in the outputs, and the running maximum and sum of its two rows (equal in the
// eight lanes of a row). All in fp32: the fp32 block's parity needs
// full-precision products, which no tensor-core type gives. Its calls are small,
// so the keys are split until the SMs are filled (three requests of up to 130
// tokens over up to 530 keys: 65 us unsplit and unbuffered, 25 so).
constexpr int kSimtRows = 32, kSimtKeys = 32, kSimtThreads = 128;

template <int kDh>
struct SimtSmem {
  float q[kSimtRows][kDh + 4];
  float k[2][kSimtKeys][kDh + 4];
  float v[2][kSimtKeys][kDh];
  float p[kSimtRows][kSimtKeys + 1];
  float bias[2][kSimtKeys];
};

// 16 bytes global -> shared, zeros where `there` is false
__device__ __forceinline__ void cp_async16_if(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

template <int kDh>
__global__ void __launch_bounds__(kSimtThreads)
    paged_attn_simt(const __grid_constant__ PagedAttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<kDh>& sm = *reinterpret_cast<SimtSmem<kDh>*>(smem_raw);
  __shared__ PagedTile s_tile;
  pdl_trigger();
  pdl_wait();
  constexpr int kCols = kDh / 32;  // float4 columns of a thread's outputs
  constexpr int kUnits = kDh / 4;  // 16-byte units of a row
  const int group = a.hq / a.kv.hkv;
  const int g = blockIdx.y, split = blockIdx.z;
  if (threadIdx.x < 32) {
    const PagedTile t = find_tile<kSimtRows>(a, static_cast<int>(blockIdx.x));
    if (threadIdx.x == 0) s_tile = t;
  }
  __syncthreads();
  const PagedTile tile = s_tile;
  if (tile.req < 0) return;
  const int tid = threadIdx.x, tx = tid & 7, ty = tid >> 3;
  const int n_rows = min(kSimtRows, tile.n * group - tile.row0);
  const int64_t lo64 = split * a.chunk;
  const int max_limit = tile.past + (tile.row0 + n_rows - 1) / group + 1;  // the last row's limit
  const int kv_end = static_cast<int>(min(static_cast<int64_t>(max_limit), lo64 + a.chunk));
  const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(0x7FFFFFFF)));
  auto load = [&](int kv0, int st) {
#pragma unroll
    for (int i = 0; i < kSimtKeys * kUnits / kSimtThreads; ++i) {
      const int e = tid + i * kSimtThreads;
      const int r = e / kUnits, c = (e % kUnits) * 4;
      const int j = kv0 + r;
      const int64_t page = j < kv_end ? page_of(a, tile.req, j) : -1;
      const int in = row_in_page(a, j);
      const int64_t off = (static_cast<int64_t>(in) * a.kv.hkv + g) * kDh + c;
      const bool there = page >= 0;
      const float* kp = static_cast<const float*>(a.kv.k);
      const float* vp = static_cast<const float*>(a.kv.v);
      cp_async16_if(&sm.k[st][r][c], there ? kp + page * a.kv.k_page_stride + off : kp, there);
      cp_async16_if(&sm.v[st][r][c], there ? vp + page * a.kv.v_page_stride + off : vp, there);
      if (c == 0)
        sm.bias[st][r] =
            there && a.kv.bias ? key_bias(__ldg(a.kv.bias + page * a.kv.bias_page_stride + in)) : 0.f;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (lo < kv_end) load(lo, 0);
  for (int e = tid; e < kSimtRows * kUnits; e += kSimtThreads) {
    const int r = e / kUnits, c = (e % kUnits) * 4;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n_rows) {
      const int rr = tile.row0 + r;
      u = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                           static_cast<int64_t>(tile.tok0 + rr / group) * a.q_stride +
                                           (g * group + rr % group) * kDh + c);
    }
    *reinterpret_cast<float4*>(&sm.q[r][c]) = u;
  }
  float scale[2], gain[2];
  int limit[2];  // keys that the row sees
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * ty + i;
    const bool on = r < n_rows;
    const int rr = tile.row0 + r;
    const int h = g * group + rr % group;
    scale[i] = kLog2e / (sqrtf(static_cast<float>(kDh)) * (a.tau && on ? __ldg(a.tau + h) : 1.0f));
    gain[i] = a.gain && a.kv.bias && on ? __ldg(a.gain + h) * kLog2e : 0.0f;
    limit[i] = on ? tile.past + rr / group + 1 : 0;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float4 o[2][kCols];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);

  int st = 0;
  for (int kv0 = lo; kv0 < kv_end; kv0 += kSimtKeys, st ^= 1) {
    if (kv0 + kSimtKeys < kv_end) load(kv0 + kSimtKeys, st ^ 1);
    else asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // this stage's keys are there for every thread
    float s[2][4] = {};
#pragma unroll 4
    for (int d = 0; d < kDh; d += 4) {
      const float4 q0 = *reinterpret_cast<const float4*>(&sm.q[2 * ty][d]);
      const float4 q1 = *reinterpret_cast<const float4*>(&sm.q[2 * ty + 1][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&sm.k[st][tx + 8 * i][d]);
        s[0][i] += q0.x * kk.x + q0.y * kk.y + q0.z * kk.z + q0.w * kk.w;
        s[1][i] += q1.x * kk.x + q1.y * kk.y + q1.z * kk.z + q1.w * kk.w;
      }
    }
    bool all = true;  // every key of the stage is seen by both rows
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
      bool seen[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = kv0 + tx + 8 * i;
        const float b = sm.bias[st][tx + 8 * i];
        const float z = s[r][i] * scale[r] + gain[r] * b;
        seen[i] = j < limit[r] && j < kv_end && !(b < kRemovableBias && z <= kMaskedLogit);
        all = all && seen[i];
        s[r][i] = seen[i] ? z : -INFINITY;
        mx = fmaxf(mx, s[r][i]);
      }
#pragma unroll
      for (int w = 4; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
      const float m_new = fmaxf(m[r], mx);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: all weights 0
      const float corr = exp2f(m[r] - m_use);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = exp2f(s[r][i] - m_use);
        sm.p[2 * ty + r][tx + 8 * i] = seen[i] ? w : -1.0f;
        sum += w;
      }
#pragma unroll
      for (int w = 4; w > 0; w >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
      l[r] = l[r] * corr + sum;
      m[r] = m_new;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        o[r][c].x *= corr;
        o[r][c].y *= corr;
        o[r][c].z *= corr;
        o[r][c].w *= corr;
      }
    }
    // (also: a row's weights are written and read by one warp)
    all = __all_sync(0xFFFFFFFFu, all);
    __syncwarp();
    auto add = [&](float4& acc, float p, const float4& vv) {
      acc.x = fmaf(p, vv.x, acc.x);
      acc.y = fmaf(p, vv.y, acc.y);
      acc.z = fmaf(p, vv.z, acc.z);
      acc.w = fmaf(p, vv.w, acc.w);
    };
    if (all) {
#pragma unroll 4
      for (int j = 0; j < kSimtKeys; ++j) {
        const float p0 = sm.p[2 * ty][j], p1 = sm.p[2 * ty + 1][j];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float4 vv = *reinterpret_cast<const float4*>(&sm.v[st][j][4 * tx + 32 * c]);
          add(o[0][c], p0, vv);
          add(o[1][c], p1, vv);
        }
      }
    } else {
      // keys that a row does not see (weight -1) are skipped, not weighted with
      // zero: their values may be infinite or NaN
#pragma unroll 1
      for (int j = 0; j < kSimtKeys; ++j) {
        const float p0 = sm.p[2 * ty][j], p1 = sm.p[2 * ty + 1][j];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float4 vv = *reinterpret_cast<const float4*>(&sm.v[st][j][4 * tx + 32 * c]);
          if (!(p0 < 0.f)) add(o[0][c], p0, vv);
          if (!(p1 < 0.f)) add(o[1][c], p1, vv);
        }
      }
    }
    __syncthreads();  // the stage is read: the next load but one may fill it
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (2 * ty + r >= n_rows) continue;
    const int rr = tile.row0 + 2 * ty + r;
    const int64_t t = tile.tok0 + rr / group;
    const int h = g * group + rr % group;
    const bool part = a.splits > 1;
    const bool any = l[r] != 0.f;  // a row that sees nothing is zero
    const float inv = part ? 1.0f : any ? 1.0f / l[r] : 0.f;
    const int64_t at = (part ? split * a.rows * a.hq : 0) + t * a.hq + h;
    if (tx == 0) {
      if (part) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m[r], l[r]);
      else if (a.lse != nullptr) a.lse[h * a.rows + t] = any ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
    }
    float* out = (part ? a.part_o : static_cast<float*>(a.out)) + at * kDh;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      *reinterpret_cast<float4*>(out + 4 * tx + 32 * c) =
          make_float4(o[r][c].x * inv, o[r][c].y * inv, o[r][c].z * inv, o[r][c].w * inv);
  }
}

template <typename T, int kDh>
cudaError_t run_append(const PagedAppendArgs& a, cudaStream_t st) {
  // one token a group until every SM has several CTAs
  int tok = 1;
  while (tok < kAppTok && a.rows / (2 * tok) >= 3 * num_sms()) tok *= 2;
  const int64_t groups = (a.rows + tok - 1) / tok;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(groups, 3 * num_sms()));
  auto kern = paged_append<T, kDh>;
  constexpr int kBytes = static_cast<int>(sizeof(AppSmem<T, kDh>));
  TG_CUDA_TRY(set_smem_attr_once(reinterpret_cast<const void*>(kern), kBytes));
  TG_CUDA_TRY(launch_pdl(kern, dim3(grid), dim3(kAppThreads + 32), kBytes, st, a, tok));
  return cudaGetLastError();
}

template <int kDh>
cudaError_t run_simt(const PagedAttnArgs& a, cudaStream_t st) {
  constexpr int kBytes = static_cast<int>(sizeof(SimtSmem<kDh>));
  auto kern = paged_attn_simt<kDh>;
  TG_CUDA_TRY(set_smem_attr_once(reinterpret_cast<const void*>(kern), kBytes));
  return launch_pdl(kern,
                    dim3(static_cast<unsigned>(a.tiles), static_cast<unsigned>(a.kv.hkv),
                         static_cast<unsigned>(a.splits)),
                    dim3(kSimtThreads), kBytes, st, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool bf16, cudaStream_t st) {
  if (a.rows <= 0 || a.batch <= 0) return cudaSuccess;
  if (bf16)
    return a.kv.dh == 128 ? run_append<__nv_bfloat16, 128>(a, st) : run_append<__nv_bfloat16, 64>(a, st);
  return a.kv.dh == 128 ? run_append<float, 128>(a, st) : run_append<float, 64>(a, st);
}

cudaError_t launch_paged_attn_simt(PagedAttnArgs a, void* ws, cudaStream_t st) {
  a.tiles = paged_row_tiles(a.rows, a.batch, a.hq, a.kv.hkv, kSimtRows);
  // splits of 64 keys at least, until every SM has three CTAs
  const int64_t jobs = a.tiles * a.kv.hkv;
  const int64_t most = std::min<int64_t>(paged_max_splits(a.rows, a.hq, a.kv.dh), 3 * num_sms() / jobs);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, a.max_kv / 64));
  a.chunk = ((a.max_kv + want - 1) / want + kSimtKeys - 1) / kSimtKeys * kSimtKeys;
  a.chunk0 = a.chunk;
  a.splits = static_cast<int>((a.max_kv + a.chunk - 1) / a.chunk);
  paged_partials(&a, ws);
  const cudaError_t e = a.kv.dh == 128 ? run_simt<128>(a, st) : run_simt<64>(a, st);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_paged_merge(a, false, st);
}

}  // namespace tg
