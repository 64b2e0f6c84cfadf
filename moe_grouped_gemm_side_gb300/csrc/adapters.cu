// Low-rank adapters of many requests beside a projection that they share:
//   Y[t] = base[t] + scale_e (X[t] A_e^T) B_e^T,  e the adapter of token t,
// on tokens that the slot map has sorted by adapter.
//
// A cluster takes a tile of rows, which have one adapter.  Its blocks share the
// contraction over K, exchange the [rows, r] sums through distributed shared
// memory, and share the columns of Y: one launch and no scratch, every weight read
// once a tile, and a single token's weights still spread over a cluster's SMs.
// The sums stay fp32; for the second product they go into two bf16 numbers each,
// which together hold 16 of their bits.
//
// Tiles of 16 rows for steps of single tokens: bound by the chain of a tile's loads,
// its two exchanges and its stores, 5 us for one token (7168 to 4096, rank 16), 13 us for
// 96 of 40 adapters of rank 32, whose 32 MB would take 4.7 us; a block's rows of B and
// of base are fetched before the exchanges (one token 5.7 us without).  Prompts: below.
#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "ops_internal.h"

namespace mg {
namespace adapters {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kCluster = 8;      // of a cluster, at most
constexpr int kRows = 16;                  // of a tile: the rows of one MMA

// D [16, 8] += A [16, 16] B [16, 8], bf16 into fp32.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two steps of 16 along k from 16-byte pieces: lane q = lane % 4 of a row holds k =
// 8q .. 8q + 7 of 32, words 0 and 1 as the first step's k = (2q, 2q + 1) and (2q
// + 8, 2q + 9), words 2 and 3 as the second's.  Both operands in the same order,
// so the sum is over the same products.
__device__ __forceinline__ void mma_pair(float (&d)[4], const uint4& a, const uint4& a8, const uint4& b) {
  mma_16x8x16(d, a.x, a8.x, a.y, a8.y, b.x, b.y);
  mma_16x8x16(d, a.z, a8.z, a.w, a8.w, b.z, b.w);
}
__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p, bool there) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there) v = __ldg(reinterpret_cast<const uint4*>(p));
  return v;
}
// The same where this place of the load counts: the compiler moves the others.
__device__ __forceinline__ uint4 ld16_now(const __nv_bfloat16* p, bool there) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there) asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld16_plain(const __nv_bfloat16* p) {        // Y may be what is read
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Two fp32 as the nearest bf16, past the largest the largest.  What is left of a finite
// number is then a bf16, and of an infinity that infinity, never infinity minus infinity.
__device__ __forceinline__ uint32_t pack_finite(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight fp32 as the nearest bf16 and the nearest bf16 of what is left.
__device__ __forceinline__ void split8(const float (&f)[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_finite(f[2 * i], f[2 * i + 1]);
    l[i] = pack(f[2 * i] - lo_of(h[i]), f[2 * i + 1] - hi_of(h[i]));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// Rows of tokens without an adapter, where Y is not base itself: a warp a token.
__device__ void copy_rows(const AdaptersArgs& a, int64_t warp, int64_t warps) {
  const int lane = threadIdx.x & 31;
  for (int64_t t = warp; t < a.T; t += warps) {
    const int32_t r = __ldg(a.rows + t);
    if (r >= 0 && r < a.rows_total) continue;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.base) + t * a.ldb);
    uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) + t * a.ldy);
    for (int32_t c = lane; c < a.N / 8; c += 32) to[c] = from[c];
  }
}

// The j-th of the tiles that hold a token (-1: there are fewer), found by the whole block
// from the tiles' first rows, which hold one where any does (with all 16 rows read,
// 1200 tokens of 10 among 200 adapters in a map of 862 tiles 21.4 us instead of 15.3).
__device__ int32_t tile_at(const AdaptersArgs& a, int32_t tiles, int32_t j) {
  constexpr int kEach = 4;                   // tiles a thread and round
  __shared__ int32_t counts[kEach][kWarps], found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t seen = 0;
  for (int32_t from = 0; from < tiles && seen <= j; from += kEach * kThreads) {
    bool held[kEach];
    uint32_t votes[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int32_t tile = from + i * kThreads + (int32_t)threadIdx.x;
      held[i] = tile < tiles && __ldg(a.src + (int64_t)tile * kRows) >= 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      votes[i] = __ballot_sync(0xffffffffu, held[i]);
      if (lane == 0) counts[i][warp] = __popc(votes[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      int32_t before = seen;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? counts[i][w] : 0;
        seen += counts[i][w];
      }
      if (held[i] && before + __popc(votes[i] & ((1u << lane) - 1)) == j) found = from + i * kThreads + (int32_t)threadIdx.x;
    }
    __syncthreads();
  }
  return seen > j ? found : -1;
}

// kR: eights of the rank, rounded up to a power of two.  A cluster takes every
// `clusters`-th of the tiles, or (`scan`) of those that hold a token.
template <int kR, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) adapters_kernel(const AdaptersArgs a, int32_t tiles, int32_t clusters,
                                                                     bool scan) {
  constexpr int kStride = 8 * kR + 4;        // floats a row of sums
  __shared__ alignas(16) float part[kWarps / 2][kRows][kStride];
  __shared__ alignas(16) float mine[kRows][kStride];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int32_t C = (int32_t)cluster_size(), rank = (int32_t)cluster_ctarank();
  if ((int32_t)(blockIdx.x / C) >= clusters) {
    copy_rows(a, (int64_t)(blockIdx.x - clusters * C) * kWarps + warp, (int64_t)(gridDim.x - clusters * C) * kWarps);
    return;
  }
  // a tile's tokens (-1: none) and their adapter, the same in every block of the
  // cluster
  auto token = [&](int64_t r) -> int32_t {
    if (r >= a.rows_total) return -1;
    const int32_t t = __ldg(a.src + r);
    if (t >= a.T) {
      set_status(a.status, MG_ERR_DEVICE_ARG);
      return -1;
    }
    return t;
  };
  for (int32_t nth = (int32_t)(blockIdx.x / C); nth < tiles; nth += clusters) {
    const int32_t tile = scan ? tile_at(a, tiles, nth) : nth;
    if (tile < 0) break;
    const int64_t row0 = (int64_t)tile * kRows;
    const int32_t t0 = token(row0 + g), t8 = token(row0 + g + 8);
    const uint32_t low = __ballot_sync(0xffffffffu, t0 >= 0), high = __ballot_sync(0xffffffffu, t8 >= 0);
    if ((low | high) == 0) continue;
    const int32_t t_first = __shfl_sync(0xffffffffu, low != 0 ? t0 : t8, __ffs(low != 0 ? low : high) - 1);
    const int32_t e = __ldg(a.idx + t_first);
    if (e < 0 || e >= a.E) {
      set_status(a.status, MG_ERR_DEVICE_ARG);
      continue;
    }
    // rows up to the last that holds a token; the others' sums are not needed, and no
    // row sees another's
    const int32_t rows = high != 0 ? 16 - (__clz(high) >> 2) : 8 - (__clz(low) >> 2);
    const int32_t r = a.r, K = a.K, N = a.N;
    const __nv_bfloat16* X = static_cast<const __nv_bfloat16*>(a.X);
    const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.A) + (int64_t)e * r * K;
    const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(a.B) + (int64_t)e * N * r;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.base);
    const int32_t per = C * kWarps, first = rank * kWarps + warp;
    // ---- sums over this warp's part of K: units of 64, dealt over the cluster's warps
    float acc[kR][4];
#pragma unroll
    for (int n = 0; n < kR; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    {
      const __nv_bfloat16* x0 = X + (int64_t)max(t0, 0) * a.ldx;
      const __nv_bfloat16* x8 = X + (int64_t)max(t8, 0) * a.ldx;
      for (int32_t u = first; u * 64 < K; u += per) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int32_t k = u * 64 + h * 32 + q * 8;
          const bool in = k < K;
          const uint4 va = ld16(x0 + k, in && t0 >= 0), v8 = ld16(x8 + k, in && t8 >= 0);
          uint4 w[kR];
#pragma unroll
          for (int n = 0; n < kR; ++n) w[n] = ld16(A + (int64_t)(n * 8 + g) * K + k, in && n * 8 < r);
#pragma unroll
          for (int n = 0; n < kR; ++n) mma_pair(acc[n], va, v8, w[n]);
        }
      }
    }
    // columns of Y: 32 at a time, dealt over the cluster's warps.  Column j of MMA i is
    // column 8 (j / 2) + 2 i + j % 2 of the 32: a lane then ends up with eight
    // neighbours.  The rows of B and the base of the next 32 are on their way while the
    // sums, or the 32 before, are worked on.
    constexpr int kK2 = (kR + 3) / 4;          // 32s of the rank
    uint4 wb[4][kK2], old[2];
    auto fetch = [&](int32_t u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t n = u * 32 + (g >> 1) * 8 + 2 * i + (g & 1);
#pragma unroll
        for (int c = 0; c < kK2; ++c) wb[i][c] = ld16_now(B + (int64_t)n * r + c * 32 + q * 8, n < N && c * 32 + q * 8 < r);
      }
      const int32_t col = u * 32 + q * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t t = i == 0 ? t0 : t8;
        old[i] = make_uint4(0, 0, 0, 0);
        if (col < N && t >= 0) old[i] = ld16_plain(base + (int64_t)t * a.ldb + col);
      }
    };
    fetch(first);
    // ---- over the block's warps: the upper four into the lower four, those in order
    auto slot = [&](int w, int n, int i) -> float2* {
      return reinterpret_cast<float2*>(&part[w][g + 8 * i][n * 8 + 2 * q]);
    };
    if (warp >= kWarps / 2) {
#pragma unroll
      for (int n = 0; n < kR; ++n) {
        if (g < rows) *slot(warp - kWarps / 2, n, 0) = make_float2(acc[n][0], acc[n][1]);
        if (g + 8 < rows) *slot(warp - kWarps / 2, n, 1) = make_float2(acc[n][2], acc[n][3]);
      }
    }
    __syncthreads();
    if (warp < kWarps / 2) {
#pragma unroll
      for (int n = 0; n < kR; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (g + 8 * i >= rows) continue;
          float2* p = slot(warp, n, i);
          const float2 v = *p;
          *p = make_float2(v.x + acc[n][2 * i], v.y + acc[n][2 * i + 1]);
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < rows * 8 * kR; i += kThreads) {
      const int row = i / (8 * kR), c = i % (8 * kR);
      float s = part[0][row][c];
#pragma unroll
      for (int w = 1; w < kWarps / 2; ++w) s += part[w][row][c];
      mine[row][c] = s;
    }
    // ---- over the cluster's blocks, in their order; times the adapter's scale
    __syncwarp();
    cluster_arrive();
    const float scale = a.scale != nullptr ? __ldg(a.scale + e) : 1.0f;
    cluster_wait();
    for (int i = tid; i < rows * 2 * kR; i += kThreads) {
      const int row = i / (2 * kR), c = i % (2 * kR) * 4;
      const uint32_t at = smem_u32(&mine[row][c]);
      float4 v[kCluster];
#pragma unroll
      for (int b = 0; b < kCluster; ++b) {
        v[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (b < C) v[b] = ld_cluster_f32x4(mapa_shared(at, (uint32_t)b));
      }
      float4 s = v[0];
#pragma unroll
      for (int b = 1; b < kCluster; ++b) s = make_float4(s.x + v[b].x, s.y + v[b].y, s.z + v[b].z, s.w + v[b].w);
      *reinterpret_cast<float4*>(&part[0][row][c]) = make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
    }
    __syncwarp();
    cluster_arrive();                          // this block reads no other's memory any more
    __syncthreads();
    // ---- columns of Y
    uint4 hh[kK2], hl[kK2], h8h[kK2], h8l[kK2];
#pragma unroll
    for (int c = 0; c < kK2; ++c) {
      float f[8], f8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = c * 32 + q * 8 + i;
        const bool in = k < 8 * kR;
        f[i] = in ? part[0][g][k] : 0.0f;
        f8[i] = in ? part[0][g + 8][k] : 0.0f;
      }
      split8(f, hh[c], hl[c]);
      split8(f8, h8h[c], h8l[c]);
    }
    __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(a.Y);
    for (int32_t u = first; u * 32 < N; u += per) {
      float d[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < kK2; ++c) {
          mma_pair(d[i], hh[c], h8h[c], wb[i][c]);
          mma_pair(d[i], hl[c], h8l[c], wb[i][c]);
        }
      }
      const uint4 was[2] = {old[0], old[1]};
      if ((u + per) * 32 < N) fetch(u + per);
      const int32_t col = u * 32 + q * 8;
      if (col >= N) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t t = i == 0 ? t0 : t8;
        if (t < 0) continue;
        const uint4 v = was[i];
        uint4 o;
        o.x = pack(lo_of(v.x) + d[0][2 * i], hi_of(v.x) + d[0][2 * i + 1]);
        o.y = pack(lo_of(v.y) + d[1][2 * i], hi_of(v.y) + d[1][2 * i + 1]);
        o.z = pack(lo_of(v.z) + d[2][2 * i], hi_of(v.z) + d[2][2 * i + 1]);
        o.w = pack(lo_of(v.w) + d[3][2 * i], hi_of(v.w) + d[3][2 * i + 1]);
        *reinterpret_cast<uint4*>(Y + (int64_t)t * a.ldy + col) = o;
      }
    }
    __syncwarp();
    cluster_wait();                            // the others have read this block's sums
    __syncthreads();
  }
}

template <int kR, int kBlocks>
cudaError_t launch_with(const AdaptersArgs& a, int32_t tiles, int32_t clusters, int32_t C, cudaStream_t s) {
  const int64_t want = a.base == a.Y ? 0 : ((int64_t)a.T + kWarps - 1) / kWarps;
  const int64_t copies = want < 2 * 152 ? want : 2 * 152;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((clusters + (copies + C - 1) / C) * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, adapters_kernel<kR, kBlocks>, a, tiles, clusters, clusters < tiles);
}
// kMost: blocks an SM that the registers allow with hardly a spill.
template <int kR, int kMost>
cudaError_t launch_as(const AdaptersArgs& a, cudaStream_t s) {
  const int32_t tiles = (int32_t)((a.rows_total + kRows - 1) / kRows);
  // Tiles that hold tokens: `most` of a full map, which has room for a last tile of
  // every adapter (215 tokens of 2 among 200 adapters in a map of 800 tiles, 4096 to
  // 7168 at rank 64: a cluster a tile 23.4 us, for `most` of them 16.3); with a half
  // and a quarter of the adapters in a step's use `many` and `some`, in prompts' an
  // eighth.
  const int64_t full = a.T / kRows, used = a.T < a.E ? a.T : a.E, most = full + used;
  const bool step = a.align_q == kRows;
  const int64_t many = full + (used + 1) / (step ? 2 : 8), some = full + (used + 3) / (step ? 4 : 8);
  const int64_t slots = (int64_t)kMost * num_sms_current_device();
  const int32_t clusters = most < tiles - tiles / 4 ? (int32_t)most : tiles;
  // Blocks a tile: as many as all run at once (us with 8, 4, 2 and 1: one token 5.0,
  // 6.4, 8.6, 13.7; 240 tokens of 50 adapters of rank 64, 4096 to 4096, 20.1, 16.2, 21.3,
  // 30; 4000 tokens of 10 of rank 32, 2048 to 2048, 42, 27, 24.5, 18.9).
  const int32_t C = full * 2 > slots ? 1 : many * 8 <= slots ? 8 : some * 4 <= slots ? 4 : 2;
  // With a block less an SM the loads of a tile go out earlier (one token 0.3 us).
  if (kMost > 1 && most * C <= slots / kMost * (kMost - 1))
    return launch_with<kR, (kMost > 1 ? kMost - 1 : 1)>(a, tiles, clusters, C, s);
  return launch_with<kR, kMost>(a, tiles, clusters, C, s);
}

// ---------------------------------------------------------------------------
// Prompts: tiles of 128 rows on the tensor cores' own memory.  The two products
// are tcgen05 MMAs of 128 rows, X (gathered by the slot map, four rows a TMA load)
// against A_e and the sums against B_e, into TMEM.  A cluster of C blocks shares a
// tile as above: each contracts a run of K, sums a C-th of the rows over the
// cluster and hands them to all its blocks as two bf16 each, in the second MMA's
// layout, and makes every C-th tile of 128 columns.
//
// Warps 0-7 copy rows of tokens without an adapter while the first product runs,
// then reduce, load B and run the epilogue; warp 8 issues the MMAs, warp 9 the TMA
// loads.  Measured on 8192 tokens of 16 adapters, rank 64, 7168 to 4096, at each step
// of its building: cp.async by all warps for the first product 74 us (a slot of the
// ring came round too late), every row by gather loads 79, boxes of 16 rows 67, sums
// pushed to the cluster and base fetched a tile ahead 53; tiles of 16 rows as above
// then 235, today 101.  It reads and writes 259 MB at least, 38 us; what is left are the two handovers
// within a cluster, in which its tensor cores and its copies rest.
constexpr int kTile = 128, kBigWarps = 8, kBigThreads = 32 * (kBigWarps + 2), kWorkers = 32 * kBigWarps;
constexpr int kMaxBigStages = 6;
constexpr int kBaseBytes = kTile * kTile * 2;
constexpr uint32_t kTmemColumns = 256;     // the sums, then two column tiles in turn
// Blocks that take part of an SM's TMEM and wait for their cluster must find it
// free: no more than two of them may be resident, so each takes at least this
// much of the 228 KB of shared memory (the GEMMs take all of it).
constexpr int kLeastSmem = 80 * 1024;
// Limit of the drains on the way out, from their start, however short the waits' own
// limit is: what is in flight would otherwise land in memory that the block has given back.
constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;

struct BigShape {
  int32_t tiles, stages, total;            // stages of the ring; bytes of shared memory
  int64_t wait_ns;
};
struct BigShared {
  uint64_t full[kMaxBigStages], empty[kMaxBigStages], sums, b_full[2], d_full[2], d_free[2], drain;
  uint32_t tmem;
  int32_t abort_flag;
};

// 16 bytes to shared memory, zeros with size 0 (nothing is read then)
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, int32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
// An arrival on `bar` once this thread's copies so far are there.  The thread that
// then issues MMAs on them orders those behind the copies (fence_proxy_async_smem);
// in a copier that fence would wait for its later copies too.
__device__ __forceinline__ void arrive_when_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// 64 columns from x on of rows r[0..3], 128 bytes each, one after another at dst
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            const int32_t (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
      : "memory");
}
__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }
__device__ __forceinline__ void st_cluster8(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// 16 rows by 32 columns of TMEM in the layout of an MMA's result: lane 4 g + q holds
// columns 8 i + 2 q and the next of row g in v[4 i] and v[4 i + 1], of row g + 8 in
// the two after.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__global__ void __launch_bounds__(kBigThreads, 2)
    adapters_big_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x16,
                        const __grid_constant__ CUtensorMap tm_a, const AdaptersArgs a, const BigShape h) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  BigShared& sh = *reinterpret_cast<BigShared*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t C = (int32_t)cluster_size(), rank = (int32_t)cluster_ctarank(), tile = (int32_t)(blockIdx.x / C);
  const int64_t row0 = (int64_t)tile * kTile;
  auto token = [&](int64_t row) -> int32_t {
    if (row >= a.rows_total) return -1;
    const int32_t t = __ldg(a.src + row);
    if (t >= a.T) {
      set_status(a.status, MG_ERR_DEVICE_ARG);
      return -1;
    }
    return t;
  };
  auto copy = [&]() {
    if (warp < kBigWarps && a.base != a.Y)
      copy_rows(a, (int64_t)blockIdx.x * kBigWarps + warp, (int64_t)gridDim.x * kBigWarps);
  };
  // the tile's first token, in every warp: four rows a lane
  int32_t t_lane = -1;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const int32_t t = token(row0 + 4 * lane + i);
    t_lane = t < 0 ? t_lane : t;
  }
  const uint32_t holders = __ballot_sync(0xffffffffu, t_lane >= 0);
  const int32_t t_first = holders == 0 ? -1 : __shfl_sync(0xffffffffu, t_lane, __ffs(holders) - 1);
  const int32_t e = t_first < 0 ? -1 : __ldg(a.idx + t_first);
  if (e < 0 || e >= a.E) {                 // the whole cluster
    if (t_first >= 0) set_status(a.status, MG_ERR_DEVICE_ARG);
    copy();
    return;
  }
  const uint64_t deadline = globaltimer_ns() + (uint64_t)h.wait_ns;
  const int32_t r = a.r, K = a.K, N = a.N, rN = (r + 15) & ~15, kb = (rN + 63) >> 6, S = h.stages;
  const int32_t R = kTile / C;             // rows that this block sums over the cluster
  const int32_t stage_bytes = (kTile + rN) * 128, b_bytes = kb * kTile * 128;
  // the ring; after the first product, in its place: this block's sums (and in theirs
  // a column tile of base), both bf16 parts of all rows, and two column tiles' rows of B
  const int32_t stride = r + 4;            // floats: 16-byte pieces of eight rows on different banks
  const uint32_t part = smem_u32(smem + 1024), parts = part + max((kTile * stride * 4 + 1023) & ~1023, kBaseBytes);
  const uint32_t b_buf = parts + 2 * kb * kTile * 128;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.sums, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.b_full[s], kWorkers);
      mbar_init(&sh.d_full[s], 1);
      mbar_init(&sh.d_free[s], kWorkers);
    }
    mbar_init(&sh.drain, 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kBigWarps) tmem_alloc(&sh.tmem, kTmemColumns);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int32_t* abort_flag = &sh.abort_flag;

  const int32_t nk = (K + 63) >> 6, k0 = (int32_t)((int64_t)nk * rank / C), n = (int32_t)((int64_t)nk * (rank + 1) / C) - k0;
  const int32_t tiles_n = (N + kTile - 1) / kTile, nt = rank < tiles_n ? (tiles_n - rank + C - 1) / C : 0;

  if (warp == kBigWarps + 1) {
    // ---- loads of the first product, in groups of 16 rows, a lane four of them: one box
    // where the group's tokens are neighbours, as those of a prompt are, else four rows
    // a load, each of which costs the copy engine as much as a box.  Rows without a
    // token hold anything: their sums are not stored, and no row sees another's.
    int32_t rows[4];
    bool near = true, held = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[i] = token(row0 + 4 * lane + i);
    const int32_t first = __shfl_sync(0xffffffffu, rows[0], lane & ~3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      near &= rows[i] < 0 || rows[i] == first + 4 * (lane & 3) + i;
      held |= rows[i] >= 0;
      rows[i] = max(rows[i], 0);
    }
    const uint32_t nears = __ballot_sync(0xffffffffu, near && first >= 0) >> (lane & ~3);
    const uint32_t helds = __ballot_sync(0xffffffffu, held) >> (lane & ~3);
    near = (nears & 15u) == 15u;
    const bool some = (helds & 15u) != 0;
    const uint32_t groups = __popc(__ballot_sync(0xffffffffu, some)) / 4;
    const uint32_t bytes = (uint32_t)rN * 128 + groups * 16 * 128;
    int32_t it = 0;
    for (; it < n; ++it) {
      const int32_t s = it % S;
      const bool ok = it < S || wait_bounded(&sh.empty[s], ((it / S) & 1) ^ 1, deadline, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* dst = smem + 1024 + s * stage_bytes;
      const int32_t k = (k0 + it) * 64;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.full[s], bytes);
        tma_load_2d(dst + kTile * 128, &tm_a, &sh.full[s], k, e * r);
      }
      __syncwarp();
      if (some && near) {
        if ((lane & 3) == 0) tma_load_2d(dst + lane * 512, &tm_x16, &sh.full[s], k, first);
      } else if (some) {
        tma_gather4(smem_u32(dst) + lane * 512, &tm_x, &sh.full[s], k, rows);
      }
    }
    // what was asked for has landed before this block's memory goes
    const uint64_t dl = globaltimer_ns() + kDrainNs;
    for (int32_t i = max(it - S, 0); i < it; ++i) wait_drain(&sh.full[i % S], (i / S) & 1, dl);
  } else if (warp == kBigWarps) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(kTile, (uint32_t)rN, 0, 0);
      for (int32_t it = 0; it < n; ++it) {
        const int32_t s = it % S;
        if (!wait_bounded(&sh.full[s], (it / S) & 1, deadline, abort_flag, a.status)) break;
        tc_fence_after();
        const uint32_t x = part + s * stage_bytes;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_f16(tmem, desc_kmajor_sw128(x + ks * 32), desc_kmajor_sw128(x + kTile * 128 + ks * 32), idesc, it + ks > 0);
        mma_commit(&sh.empty[s]);
      }
      mma_commit(&sh.sums);
    }
  } else {
    copy();
  }
  __syncwarp();

  // Rows of B for the i-th column tile, 2048 pieces at most.  Column 8 i + 2 q + b of 32
  // is column 8 q + 2 i + b of Y, so that a lane of the epilogue ends up with eight
  // neighbours.
  const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(a.B) + (int64_t)e * N * r;
  const int32_t pieces = rN >> 3, b_rows = kWorkers / pieces;      // rows of a round of the workers
  const int32_t b_row0 = tid / pieces, b_piece = tid - b_row0 * pieces;
  auto copy_b = [&](int32_t i) {
    if (i < nt) {
      const int32_t n0 = (rank + i * C) * kTile;
      const uint32_t to = b_buf + (i & 1) * b_bytes + (b_piece >> 3) * (kTile * 128);
      if (b_row0 < b_rows) {
        for (int32_t row = b_row0; row < kTile; row += b_rows) {
          const int32_t col = n0 + (row & ~31) + ((row >> 1) & 3) * 8 + ((row >> 3) & 3) * 2 + (row & 1);
          const bool there = col < N && b_piece * 8 < r;
          cp_async_or_zero(to + swizzled(row, b_piece & 7), there ? B + (int64_t)col * r + b_piece * 8 : B, there ? 16 : 0);
        }
      }
      arrive_when_copied(&sh.b_full[i & 1]);
    }
  };

  // ---- this block's sums to shared memory, where the cluster reads them
  const int quad = warp & 3, half = warp >> 2;
  if (warp < kBigWarps) {
    wait_bounded(&sh.sums, 0, deadline, abort_flag, a.status);
    __syncwarp();
    tc_fence_after();
    const int row = quad * 32 + lane;
    for (int32_t c = half * 16; c < rN; c += 32) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = n > 0 ? make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]) : make_uint4(0, 0, 0, 0);
        if (c + 4 * q < r) st_shared16(part + (row * stride + c + 4 * q) * 4, w);
      }
    }
    tc_fence_before();
    // the first two tiles' rows of B; the ring's last reader is done
    copy_b(0);
    copy_b(1);
  }
  __syncwarp();
  cluster_sync();
  // ---- the cluster's sums of this block's rows, in the blocks' order, times the
  // scale, as two bf16 each, to every block
  if (warp < kBigWarps) {
    const float scale = a.scale != nullptr ? __ldg(a.scale + e) : 1.0f;
    const int32_t fours = rN >> 2;
    for (int32_t i = tid; i < R * fours; i += kWorkers) {
      const int32_t row = rank * R + i / fours, c = (i % fours) * 4;
      const uint32_t at = part + (row * stride + c) * 4;
      float4 w[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        w[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (b < C && c < r) w[b] = ld_cluster_f32x4(mapa_shared(at, (uint32_t)b));
      }
      float4 v = w[0];
#pragma unroll
      for (int b = 1; b < 8; ++b) {
        v.x += w[b].x;
        v.y += w[b].y;
        v.z += w[b].z;
        v.w += w[b].w;
      }
      v.x *= scale;
      v.y *= scale;
      v.z *= scale;
      v.w *= scale;
      const uint32_t h0 = pack_finite(v.x, v.y), h1 = pack_finite(v.z, v.w);
      const uint32_t l0 = pack(v.x - lo_of(h0), v.y - hi_of(h0)), l1 = pack(v.z - lo_of(h1), v.w - hi_of(h1));
      const uint32_t to = parts + (c >> 6) * (kTile * 128) + swizzled(row, (c >> 3) & 7) + (c & 4) * 2;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (b < C) {
          const uint32_t there = mapa_shared(to, (uint32_t)b);
          st_cluster8(there, h0, h1);
          st_cluster8(there + kb * kTile * 128, l0, l1);
        }
      }
    }
    // before the MMAs of every block that reads them
    asm volatile("fence.proxy.async;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();                          // no block touches another's memory from here on

  if (warp < kBigWarps) {
    // ---- columns: lane 4 g + q has eight neighbours, 8 q on, of rows g, g + 8, g + 16
    // and g + 24 of the warp's 32: four lanes 64 bytes of a row
    const int g = lane >> 2, q = lane & 3;
    const int32_t t_own = token(row0 + quad * 32 + lane);
    const __nv_bfloat16* base[4];
    int64_t y_at[4];
    bool live[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int32_t t = __shfl_sync(0xffffffffu, t_own, g + 8 * m);
      live[m] = t >= 0;
      base[m] = static_cast<const __nv_bfloat16*>(a.base) + (int64_t)max(t, 0) * a.ldb;
      y_at[m] = (int64_t)max(t, 0) * a.ldy;
    }
    __nv_bfloat16* Y = static_cast<__nv_bfloat16*>(a.Y);
    constexpr int kWidth = kTile / 2;      // columns of a warp
    // base of the i-th tile's c-th 32 columns: a thread's own words, a tile ahead
    const uint32_t mine = part + tid * 16;
    auto fetch = [&](int32_t i, int c) {
      const int32_t col = (rank + i * C) * kTile + half * kWidth + q * 8 + 32 * c;
      if (i < nt && col < N) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (live[m]) cp_async_or_zero(mine + (c * 4 + m) * (kWorkers * 16), base[m] + col, 16);
      }
      cp_async_commit();
    };
    fetch(0, 0);
    fetch(0, 1);
    for (int32_t i = 0; i < nt; ++i) {
      const int32_t col0 = (rank + i * C) * kTile + half * kWidth + q * 8;
      const bool ok = wait_bounded(&sh.d_full[i & 1], (i >> 1) & 1, deadline, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      copy_b(i + 2);                       // this tile's rows of B are done with
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[2][16];
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + (i & 1) * kTile + half * kWidth + 32 * c;
        tmem_ld_16x32(from, v[0]);
        tmem_ld_16x32(from + (16u << 16), v[1]);
        cp_async_wait<1>();                // this half of the base
        tmem_ld_wait();
        tmem_regs_ready(v[0]);
        tmem_regs_ready(v[1]);
        if (c == 1) {
          tc_fence_before();
          mbar_arrive(&sh.d_free[i & 1]);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t(&f)[16] = v[m >> 1];
          const int s = (m & 1) * 2;
          const uint4 o = lds16(mine + (c * 4 + m) * (kWorkers * 16));
          auto sum = [&](uint32_t old, int k) {
            return pack(lo_of(old) + __uint_as_float(f[4 * k + s]), hi_of(old) + __uint_as_float(f[4 * k + s + 1]));
          };
          const uint4 out = make_uint4(sum(o.x, 0), sum(o.y, 1), sum(o.z, 2), sum(o.w, 3));
          if (live[m] && col0 + 32 * c < N) *reinterpret_cast<uint4*>(Y + y_at[m] + col0 + 32 * c) = out;
        }
        fetch(i + 1, c);                   // where those words were
      }
    }
    cp_async_wait_all();
  } else if (tid == kWorkers) {
    const uint32_t idesc = idesc_bf16(kTile, kTile, 0, 0);
    asm volatile("fence.proxy.async;" ::: "memory");
    for (int32_t i = 0; i < nt; ++i) {
      if (!wait_bounded(&sh.b_full[i & 1], (i >> 1) & 1, deadline, abort_flag, a.status)) break;
      if (i >= 2 && !wait_bounded(&sh.d_free[i & 1], ((i >> 1) & 1) ^ 1, deadline, abort_flag, a.status)) break;
      fence_proxy_async_smem();
      tc_fence_after();
      const uint32_t b = b_buf + (i & 1) * b_bytes;
      for (int which = 0; which < 2; ++which) {
        for (int32_t ks = 0; ks < rN >> 4; ++ks) {
          const uint32_t off = (ks >> 2) * (kTile * 128) + (ks & 3) * 32;
          mma_f16(tmem + (i & 1) * kTile, desc_kmajor_sw128(parts + which * kb * (kTile * 128) + off),
                  desc_kmajor_sw128(b + off), idesc, which + ks > 0);
        }
      }
      mma_commit(&sh.d_full[i & 1]);
    }
    // nothing of this block is in flight when its memory goes
    mma_commit(&sh.drain);
    wait_drain(&sh.drain, 0, globaltimer_ns() + kDrainNs);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kBigWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColumns);
  }
}

cudaError_t launch_big(const AdaptersArgs& a, cudaStream_t s) {
  BigShape h;
  h.tiles = (int32_t)((a.rows_total + kTile - 1) / kTile);
  const int32_t rN = (a.r + 15) & ~15, kb = (rN + 63) / 64;
  // Two blocks an SM up to rank 64, one above; as many blocks a tile as all run at once,
  // were an eighth of the adapters in use (a map has room for a last tile of all):
  // 8192 tokens, 7168 to 4096 at rank 64, 64 us with 8, 53 with 4, 62 with 2.  (With one
  // block an SM in return for base two or three tiles ahead, 2048 tokens, 4096 to 4096
  // at rank 16: 32 us instead of 22, the clusters no longer all at once.)
  const int32_t slots = (kb == 1 ? 2 : 1) * num_sms_current_device();
  const int32_t some = a.T / kTile + ((a.T < a.E ? a.T : a.E) + 7) / 8;
  const int32_t C = some * 8 <= slots ? 8 : some * 4 <= slots ? 4 : 2;
  const int32_t stage = (kTile + rN) * 128;
  const int32_t sums = (kTile * (a.r + 4) * 4 + 1023) / 1024 * 1024;
  const int32_t after = (sums > kBaseBytes ? sums : kBaseBytes) + 4 * kb * kTile * 128;
  const int32_t room = ((kb == 1 ? 111 : 218) * 1024 - 2048) / stage;
  h.stages = room < kMaxBigStages ? room : kMaxBigStages;
  h.total = 2048 + (h.stages * stage > after ? h.stages * stage : after);
  if (h.total < kLeastSmem) h.total = kLeastSmem;
  h.wait_ns = mg_get_wait_limit_ns();
  CUtensorMap tm_x, tm_x16, tm_a;
  if (encode_bf16_rows(&tm_x, a.X, a.K, a.T, a.ldx * 2, 64, 1) != MG_OK ||
      encode_bf16_rows(&tm_x16, a.X, a.K, a.T, a.ldx * 2, 64, 16) != MG_OK ||
      encode_bf16_rows(&tm_a, a.A, a.K, (int64_t)a.E * a.r, (int64_t)a.K * 2, 64, (uint32_t)rN) != MG_OK)
    return cudaErrorUnknown;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !done[dev].load()) {
    err = cudaFuncSetAttribute(adapters_big_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (err != cudaSuccess) return err;
    // left to itself the SM gives one block's worth
    err = cudaFuncSetAttribute(adapters_big_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (err != cudaSuccess) return err;
    if (dev < 64) done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(h.tiles * C));
  cfg.blockDim = dim3(kBigThreads);
  cfg.dynamicSmemBytes = (size_t)h.total;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, adapters_big_kernel, tm_x, tm_x16, tm_a, a, h);
}

}  // namespace adapters

cudaError_t launch_adapters(const AdaptersArgs& a, cudaStream_t s) {
  using namespace adapters;
  // Few rows are faster in tiles of 16 (us in tiles of 16 and of 128, one adapter, 4096 to
  // 4096: rank 128, 500 rows 17.8 and 21.9, 700 rows 26 and 22.6; 64, 1000 rows 17.4 and
  // 19.3, 1400 rows 24.8 and 19.8; 32, 2000 rows 19.7 and 21.4, 3000 rows 25 and 23.6; 16,
  // 2000 rows 19 and 20.6, 4000 rows 31 and 25; 8, 3000 rows 21.6 and 22.8, 4000 rows 31
  // and 25.  2048 to 2048 the two meet later: 64, 1400 rows 16.4 and 15.2, 2000 rows 17
  // and 18; 16, 3000 rows 14.4 and 17, 4000 rows 19 and 18.8).
  const bool many = a.T >= 3000 || (int64_t)a.T * a.r >= 80000;
  if (a.align_q % kTile == 0 && many && (int64_t)a.E * a.r < (int64_t(1) << 31))
    return launch_big(a, s);
  if (a.r <= 8) return launch_as<1, 3>(a, s);
  if (a.r <= 16) return launch_as<2, 3>(a, s);
  if (a.r <= 32) return launch_as<4, 3>(a, s);
  if (a.r <= 64) return launch_as<8, 2>(a, s);
  return launch_as<16, 1>(a, s);
}

}  // namespace mg
