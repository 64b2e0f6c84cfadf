// The residual's addition with a root-mean-square norm, as bf16 and as E4M3
// with UE8M0 scales, and its gradients:
//   s = x + r,  y = s * rstd * w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   dx = rstd (g - xh mean(g xh)) + dr,  dw = sum over rows of dy xh,
// with xh = s * rstd and g = dy * w.  One pass over a row each: it stays in
// registers between its statistics and its outputs.  Bound by memory traffic;
// fp32 throughout, two columns to an instruction.
#include <atomic>

#include "blockq.cuh"
#include "common.cuh"
#include "ops_internal.h"

namespace mg {
namespace norm {

constexpr int kThreads = 512;              // of a block, at most, where rows are copied ahead
constexpr int kBwdThreads = 1024;          // of one of the backward pass with a vector a thread

// Eight columns as four pairs, from bf16 or fp32 words.
template <bool kF32>
__device__ __forceinline__ void pairs_of(const uint4& a, const uint4& b, uint64_t (&x)[4]) {
  if (kF32) {
    x[0] = pack2(__uint_as_float(a.x), __uint_as_float(a.y));
    x[1] = pack2(__uint_as_float(a.z), __uint_as_float(a.w));
    x[2] = pack2(__uint_as_float(b.x), __uint_as_float(b.y));
    x[3] = pack2(__uint_as_float(b.z), __uint_as_float(b.w));
  } else {
    bf16x8_to_f32x2(a, x);
  }
}
template <bool kF32>
__device__ __forceinline__ const char* row_at(const void* base, int64_t at) {
  return static_cast<const char*>(base) + at * (kF32 ? 4 : 2);
}
template <bool kF32>
__device__ __forceinline__ char* row_at(void* base, int64_t at) {
  return static_cast<char*>(base) + at * (kF32 ? 4 : 2);
}

// The eight columns of a thread's vector v.  bf16 alone: eight neighbours, one
// 16-byte word.  Where fp32 takes part, four at c0 and four at c1: a warp's
// 16-byte accesses of fp32 are neighbours then, as its 8-byte ones of bf16 are
// (with eight neighbours of fp32 a lane each access leaves every second 16 bytes
// of its sectors to the next one: twice the requests to L2).
template <bool kSplit>
struct Cols {
  int32_t c0, c1;
  __device__ __forceinline__ Cols(int32_t tpr, int32_t i, int v) {
    if (kSplit) {
      const int32_t lanes = min(tpr, 32), l = i & (lanes - 1);
      c0 = (v * tpr + i - l) * 8 + l * 4;
      c1 = c0 + lanes * 4;
    } else {
      c0 = (v * tpr + i) * 8;
      c1 = c0 + 4;
    }
  }
};

template <bool kF32, bool kSplit>
__device__ __forceinline__ void load8(const char* row, const Cols<kSplit>& c, int32_t K, uint64_t (&x)[4]) {
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (kF32) {
    if (c.c0 < K) a = __ldcs(reinterpret_cast<const uint4*>(row + 4 * c.c0));
    if (c.c1 < K) b = __ldcs(reinterpret_cast<const uint4*>(row + 4 * c.c1));
  } else if (kSplit) {
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (c.c0 < K) lo = __ldcs(reinterpret_cast<const uint2*>(row + 2 * c.c0));
    if (c.c1 < K) hi = __ldcs(reinterpret_cast<const uint2*>(row + 2 * c.c1));
    a = make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    if (c.c0 < K) a = __ldcs(reinterpret_cast<const uint4*>(row + 2 * c.c0));
  }
  pairs_of<kF32>(a, b, x);
}
template <bool kF32, bool kSplit>
__device__ __forceinline__ void store8(char* row, const Cols<kSplit>& c, int32_t K, const uint64_t (&x)[4]) {
  if (kF32) {
    const float2 p = unpack2(x[0]), q = unpack2(x[1]), r = unpack2(x[2]), s = unpack2(x[3]);
    if (c.c0 < K) *reinterpret_cast<float4*>(row + 4 * c.c0) = make_float4(p.x, p.y, q.x, q.y);
    if (c.c1 < K) *reinterpret_cast<float4*>(row + 4 * c.c1) = make_float4(r.x, r.y, s.x, s.y);
  } else {
    const uint4 v = f32x2_to_bf16x8(x);
    if (kSplit) {
      if (c.c0 < K) *reinterpret_cast<uint2*>(row + 2 * c.c0) = make_uint2(v.x, v.y);
      if (c.c1 < K) *reinterpret_cast<uint2*>(row + 2 * c.c1) = make_uint2(v.z, v.w);
    } else {
      if (c.c0 < K) *reinterpret_cast<uint4*>(row + 2 * c.c0) = v;
    }
  }
}
// Eight columns of the weight, zeros behind its end.
template <bool kSplit>
__device__ __forceinline__ void load_w(const void* w, bool f32, const Cols<kSplit>& c, int32_t K, uint64_t (&x)[4]) {
  if (f32)
    load8<true, kSplit>(static_cast<const char*>(w), c, K, x);
  else
    load8<false, kSplit>(static_cast<const char*>(w), c, K, x);
}

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const char* src) {
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// The oldest of `stages` - 1 rows on their way has arrived.
__device__ __forceinline__ void wait_oldest(int stages) {
  if (stages == 3)
    cp_async_wait<1>();
  else
    cp_async_wait<0>();
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// The ring of rows on their way: 16-byte words, 32 lanes side by side, a warp's
// words of a stage (kWords of them) one after another.  A thread reads only what
// it copied itself, so no barrier is needed.
template <int kWords>
struct Ring {
  uint32_t first, at, stage_bytes, end;    // of this thread
  __device__ __forceinline__ Ring(const void* smem, int stages) {
    stage_bytes = blockDim.x * kWords * 16;
    first = smem_u32(smem) + (threadIdx.x >> 5) * (kWords * 512) + (threadIdx.x & 31) * 16;
    at = first;
    end = first + stages * stage_bytes;
  }
  __device__ __forceinline__ void next() {
    at += stage_bytes;
    if (at == end) at = first;
  }
};
// Eight columns to the words at `at`, and from there as pairs.
template <bool kF32, bool kSplit>
__device__ __forceinline__ void copy8(uint32_t at, const char* row, const Cols<kSplit>& c, int32_t K) {
  if (kF32) {
    if (c.c0 < K) cp_async<16>(at, row + 4 * c.c0);
    if (c.c1 < K) cp_async<16>(at + 512, row + 4 * c.c1);
  } else if (kSplit) {
    if (c.c0 < K) cp_async<8>(at, row + 2 * c.c0);
    if (c.c1 < K) cp_async<8>(at + 8, row + 2 * c.c1);
  } else {
    if (c.c0 < K) cp_async<16>(at, row + 2 * c.c0);
  }
}
template <bool kF32, bool kSplit>
__device__ __forceinline__ void read8(uint32_t at, uint64_t (&x)[4]) {
  const uint4 a = lds16(at), b = kF32 ? lds16(at + 512) : a;
  pairs_of<kF32>(a, b, x);
}
template <bool kF32, bool kSplit>
__device__ __forceinline__ void read8(uint32_t at, const Cols<kSplit>& c, int32_t K, uint64_t (&x)[4]) {
  read8<kF32, kSplit>(at, x);
  if (kSplit && c.c1 >= K) x[2] = x[3] = 0;          // never copied
}

// Sum over the tpr threads of a row, the same in all of them: by shuffles in a
// warp, across warps through shared memory in a fixed order.  Two buffers in
// turn, so that one barrier of the row's threads is enough.
__device__ __forceinline__ float row_sum(float v, int32_t tpr, int team, float* part, int& buf) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr == 16) return v;
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if (tpr == 32) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = team * (tpr >> 5);
  float* p = part + buf * 32;
  if (lane == 0) p[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(tpr) : "memory");
  v = lane < (tpr >> 5) ? p[first + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  buf ^= 1;
  return v;
}

// The largest magnitude of two pairs and m; NaN does not count.
__device__ __forceinline__ float amax4(uint64_t a, uint64_t b, float m) {
  const float2 p = unpack2(a), q = unpack2(b);
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(p.x), "f"(p.y));
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(q.x), "f"(q.y));
  return m;
}
// A magnitude as a number of nine bits that grows with it and gives the scale: the
// sum of ue8m0_of_amax and 1; 0 for a magnitude of 0.
__device__ __forceinline__ uint32_t scale_key(float amax) {
  return amax == 0.0f ? 0u : (__float_as_uint(amax) + 0x9fffffu) >> 23;
}
__device__ __forceinline__ int32_t ue8m0_of_key(uint32_t key) { return key == 0 ? 127 : max((int32_t)key - 9, 1); }
__device__ __forceinline__ uint32_t e4m3x4_encode(uint64_t a, uint64_t b, uint64_t inv) {
  const float2 p = unpack2(mul2(a, inv)), q = unpack2(mul2(b, inv));
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(p.x), "f"(p.y), "f"(q.x), "f"(q.y));
  return r;
}

// Codes and scales of a thread's vectors of row t.  Blocks of 128 columns: 16 lanes of
// eight neighbours, or 32 lanes of four (half a warp of both fours with 128 columns a
// row).  The maxima go through the lanes two at a time, as keys.
template <bool kSplit, int kVec>
__device__ __forceinline__ void quantise(const NormArgs& a, int64_t t, bool there, int32_t tpr, int32_t i,
                                         const uint64_t (&y)[kVec][4]) {
  constexpr int kB = kSplit ? 2 : 1, kKeys = kVec * kB;
  const bool two = kSplit && tpr >= 32;      // two blocks a vector
  uint32_t key[kKeys + 1];
  key[kKeys] = 0;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const float m0 = amax4(y[v][0], y[v][1], 0.0f);
    if (two) {
      key[v * kB] = scale_key(m0);
      key[v * kB + kB - 1] = scale_key(amax4(y[v][2], y[v][3], 0.0f));
    } else {
      key[v * kB] = key[v * kB + kB - 1] = scale_key(amax4(y[v][2], y[v][3], m0));
    }
  }
#pragma unroll
  for (int k = 0; k < kKeys; k += 2) {
    uint32_t m = key[k] | key[k + 1] << 16;
    if (two) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 16));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    key[k] = m & 0xffffu;
    key[k + 1] = m >> 16;
  }
  if (!there) return;
  const Cols<kSplit> c(tpr, i, 0);
  uint8_t* row = a.Q + t * a.K;
  // a block's first columns write its scale
  const int64_t next = a.sq_rows > 0 ? a.sq_rows : 1;
  uint8_t* sq = a.SQ + (c.c0 >> 7) * next + t * (a.sq_rows > 0 ? 1 : a.K >> 7);
  const bool first = (c.c0 & 127) == 0;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int32_t c0 = c.c0 + v * tpr * 8, c1 = c.c1 + v * tpr * 8;
    const int32_t e0 = ue8m0_of_key(key[v * kB]), e1 = ue8m0_of_key(key[v * kB + kB - 1]);
    const uint64_t k0 = pack2(ue8m0_inverse(e0), ue8m0_inverse(e0)), k1 = pack2(ue8m0_inverse(e1), ue8m0_inverse(e1));
    const uint32_t lo = e4m3x4_encode(y[v][0], y[v][1], k0), hi = e4m3x4_encode(y[v][2], y[v][3], kSplit ? k1 : k0);
    if (kSplit) {
      if (c0 < a.K) *reinterpret_cast<uint32_t*>(row + c0) = lo;
      if (c1 < a.K) *reinterpret_cast<uint32_t*>(row + c1) = hi;
    } else if (c0 < a.K) {
      *reinterpret_cast<uint2*>(row + c0) = make_uint2(lo, hi);
    }
    if (first && c0 < a.K) sq[0] = (uint8_t)e0;
    if (two && first && c1 < a.K) sq[next] = (uint8_t)e1;
    sq += (tpr >> 4) * next;
  }
}

// Rows of up to 16384 columns (14336 where X and the residual are fp32; two rows of wider
// ones do not fit): blocks walk over rows, tpr threads a row, which are copied stages - 1
// ahead, before a row's sum or (`late`) between that and its outputs.  Bound by memory, and by how reads and writes meet there: the copies
// on their way want to be 32 to 64 KB an SM (launch rule below).  16384 rows of 7168
// with a residual to bf16 and E4M3 160 us, 6.6 TB/s; 8191 of 2048 with an fp32 stream
// 32 us, 6.3; 61 rows 3.6 us, a row's latency.  Without a residual to E4M3 alone
// instructions bind, with two vectors a thread 178 a warp's 256 columns: 97 us for 16384
// rows of 7168 (to bf16 138 and 73 us; with row addresses made anew 161 and 77), 83 us,
// 4.2 TB/s, with four vectors, which share a row's own.
template <bool kXF, bool kSF, int kVec>
__global__ void __launch_bounds__(kThreads, kVec <= 2 ? 2 : 1) norm_kernel(const NormArgs a, int32_t tpr, int32_t stages,
                                                                           bool late) {
  constexpr bool kSplit = kXF || kSF;
  constexpr int kWX = kXF ? 2 : 1, kW = kWX + (kSF ? 2 : 1);       // words of a vector
  using C = Cols<kSplit>;
  extern __shared__ uint4 smem[];
  __shared__ float part[64];
  const int teams = blockDim.x / tpr, team = threadIdx.x / tpr, i = threadIdx.x - team * tpr;
  const int32_t K = a.K;
  // rows as unsigned numbers: a step or three past the last one does not wrap
  const uint32_t T = (uint32_t)a.T, step = gridDim.x * (uint32_t)teams, t_first = blockIdx.x * (uint32_t)teams + team;
  const bool res = a.R != nullptr;
  Ring<kVec * kW> in(smem, stages), out(smem, stages);
  // places behind a row's end are read as they are now
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const C c(tpr, i, v);
    if (c.c1 < K) continue;
    for (uint32_t at = in.first; at != in.end; at += in.stage_bytes)
#pragma unroll
      for (int w = 0; w < kW; ++w)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + (v * kW + w) * 512), "r"(0) : "memory");
  }
  uint32_t ta = t_first;
  const char* xa = row_at<kXF>(a.X, (int64_t)ta * a.ldx);
  const char* ra = row_at<kSF>(a.R, (int64_t)ta * a.ldr);
  const int64_t x_step = (int64_t)step * a.ldx * (kXF ? 4 : 2), r_step = (int64_t)step * a.ldr * (kSF ? 4 : 2);
  auto ahead = [&]() {
    if (ta < T) {
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const C c(tpr, i, v);
        copy8<kXF>(in.at + v * (kW * 512), xa, c, K);
        if (res) copy8<kSF>(in.at + (v * kW + kWX) * 512, ra, c, K);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ta += step;
    xa += x_step;
    ra += r_step;
    in.next();
  };
  for (int n = 1; n < stages; ++n) ahead();
  uint64_t w[kVec][4];
#pragma unroll
  for (int v = 0; v < kVec; ++v) load_w(a.w, a.w_f32, C(tpr, i, v), K, w[v]);
  const float inv = 1.0f / (float)K;
  int buf = 0;
  for (uint32_t t = t_first; t - team < T; t += step) {      // the same for all rows of the block
    const bool there = t < T;
    wait_oldest(stages);
    uint64_t s[kVec][4];
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      read8<kXF, kSplit>(out.at + v * (kW * 512), s[v]);
      if (res) {
        uint64_t r[4];
        read8<kSF, kSplit>(out.at + (v * kW + kWX) * 512, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[v][j] = add2(s[v][j], r[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(s[v][j], s[v][j], ss);
    }
    // into the stage that was read a row ago
    if (!late) ahead();
    out.next();
    const float2 q = unpack2(ss);
    const float mean = row_sum(q.x + q.y, tpr, team, part, buf) * inv;
    const float rstd = __frsqrt_rn(mean + a.eps);
    if (a.rstd != nullptr && there && i == 0) a.rstd[t] = rstd;
    const uint64_t k = pack2(rstd, rstd);
    if (late) ahead();
    if (a.H != nullptr && there) {
      char* h = row_at<kSF>(a.H, (int64_t)t * a.ldh);
#pragma unroll
      for (int v = 0; v < kVec; ++v) store8<kSF>(h, C(tpr, i, v), K, s[v]);
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[v][j] = mul2(mul2(s[v][j], k), w[v][j]);
    if (a.Y != nullptr && there) {
      char* y = row_at<false>(a.Y, (int64_t)t * a.ldy);
#pragma unroll
      for (int v = 0; v < kVec; ++v) store8<false>(y, C(tpr, i, v), K, s[v]);
    }
    if (a.Q != nullptr) quantise<kSplit, kVec>(a, t, there, tpr, i, s);
  }
  cp_async_wait<0>();
}

// Wider rows: a block each, straight from memory, nothing ahead (4000 rows of 16384 in
// fp32 with a residual 197 us, 4.7 TB/s; of 12288 through the ring 111, 6.2).
constexpr int kWide = 4, kWideThreads = 1024;
template <bool kXF, bool kSF>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const NormArgs a) {
  constexpr bool kSplit = kXF || kSF;
  using C = Cols<kSplit>;
  __shared__ float part[64];
  const int tpr = kWideThreads, i = threadIdx.x;
  const int64_t t = blockIdx.x;
  uint64_t s[kWide][4];
  uint64_t ss = 0;
#pragma unroll
  for (int v = 0; v < kWide; ++v) {
    const C c(tpr, i, v);
    load8<kXF>(row_at<kXF>(a.X, t * a.ldx), c, a.K, s[v]);
    if (a.R != nullptr) {
      uint64_t r[4];
      load8<kSF>(row_at<kSF>(a.R, t * a.ldr), c, a.K, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[v][j] = add2(s[v][j], r[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) ss = fma2(s[v][j], s[v][j], ss);
  }
  const float2 q = unpack2(ss);
  int buf = 0;
  const float mean = row_sum(q.x + q.y, tpr, 0, part, buf) * (1.0f / (float)a.K);
  const float rstd = __frsqrt_rn(mean + a.eps);
  if (a.rstd != nullptr && i == 0) a.rstd[t] = rstd;
  const uint64_t k = pack2(rstd, rstd);
#pragma unroll
  for (int v = 0; v < kWide; ++v) {
    const C c(tpr, i, v);
    if (a.H != nullptr) store8<kSF>(row_at<kSF>(a.H, t * a.ldh), c, a.K, s[v]);
    uint64_t w[4];
    load_w(a.w, a.w_f32, c, a.K, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[v][j] = mul2(mul2(s[v][j], k), w[j]);
    if (a.Y != nullptr) store8<false>(row_at<false>(a.Y, t * a.ldy), c, a.K, s[v]);
  }
  if (a.Q != nullptr) quantise<kSplit, kWide>(a, t, true, tpr, i, s);
}

// The row's own terms, with x = H and k = rstd: dw += (dy x) k, and the sum of (dy x)
// w, whose k and 1/K the row multiplies once: dx = (dy w) k + x c + dr with
// c = -k^2 (k sum / K).
__device__ __forceinline__ float bwd_factor(float sum, float k, float inv) { return -(sum * k * inv) * k * k; }

// Gradients of rows of up to 16384 columns, copied ahead in the same way: 14336 with dY
// in fp32, 10752 with H and dX in fp32, 9216 with all three.  Each
// thread has the same columns of every row and keeps their part of dw; a block's
// parts go to `work`, one row of K a block, and a second kernel adds those up in
// the blocks' order.  A row's words are read from shared memory twice, for its
// sum and for its result, which leaves the registers to dw and w (64 of them with a
// vector a thread: addresses kept from row to row spill, 95 us instead of 76).  Bound
// by memory: 8191 rows of 7168 76 us, 6.2 TB/s, 28000 of 2048 with an fp32 stream 120
// us, 6.7.
template <bool kGF, bool kSF, int kVec>
__global__ void __launch_bounds__(kVec == 1 ? kBwdThreads : kThreads) norm_bwd_kernel(const NormBwdArgs a, int32_t tpr,
                                                                                      int32_t stages) {
  constexpr bool kSplit = kGF || kSF;
  constexpr int kWG = kGF ? 2 : 1, kWS = kSF ? 2 : 1, kW = kWG + 2 * kWS;
  using C = Cols<kSplit>;
  extern __shared__ uint4 smem[];
  __shared__ float part[64];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int teams = blockDim.x / tpr, team = threadIdx.x / tpr, i = threadIdx.x - team * tpr;
  const int32_t K = a.K;
  const int64_t step = (int64_t)gridDim.x * teams;
  const bool res = a.dR != nullptr;
  Ring<kVec * kW> in(smem, stages), out(smem, stages);
  int64_t ta = (int64_t)blockIdx.x * teams + team;
  auto ahead = [&]() {
    if (ta < a.T) {
      const char* g = row_at<kGF>(a.dY, ta * a.ldd);
      const char* h = row_at<kSF>(a.H, ta * a.ldh);
      const char* r = row_at<kSF>(a.dR, ta * a.ldr);
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const C c(tpr, i, v);
        copy8<kGF>(in.at + v * (kW * 512), g, c, K);
        copy8<kSF>(in.at + (v * kW + kWG) * 512, h, c, K);
        if (res) copy8<kSF>(in.at + (v * kW + kWG + kWS) * 512, r, c, K);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ta += step;
    in.next();
  };
  for (int n = 1; n < stages; ++n) ahead();
  uint64_t dw[kVec][4], w[kVec][4];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[v][j] = 0;
    load_w(a.w, a.w_f32, C(tpr, i, v), K, w[v]);
  }
  const float inv = 1.0f / (float)K;
  int buf = 0;
  float rstd = (int64_t)blockIdx.x * teams + team < a.T ? a.rstd[(int64_t)blockIdx.x * teams + team] : 0.0f;
  for (int64_t t0 = (int64_t)blockIdx.x * teams; t0 < a.T; t0 += step) {
    const int64_t t = t0 + team;
    const bool there = t < a.T;
    const float k = rstd;
    const uint64_t k2 = pack2(k, k);
    if (t + step < a.T) rstd = a.rstd[t + step];
    wait_oldest(stages);
    ahead();                               // into the stage that was read a row ago
    uint64_t dot = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const C c(tpr, i, v);
      if (there && c.c0 < K) {
        uint64_t g[4], x[4];
        read8<kGF>(out.at + v * (kW * 512), c, K, g);
        read8<kSF>(out.at + (v * kW + kWG) * 512, c, K, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t gx = mul2(g[j], x[j]);
          dw[v][j] = fma2(gx, k2, dw[v][j]);
          dot = fma2(gx, w[v][j], dot);
        }
      }
    }
    const float2 q = unpack2(dot);
    const float f = bwd_factor(row_sum(q.x + q.y, tpr, team, part, buf), k, inv);
    const uint64_t f2 = pack2(f, f);
    char* dx = row_at<kSF>(a.dX, t * a.ldx);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const C c(tpr, i, v);
      if (there && c.c0 < K) {
        uint64_t g[4], x[4], r[4] = {0, 0, 0, 0};
        read8<kGF>(out.at + v * (kW * 512), c, K, g);
        read8<kSF>(out.at + (v * kW + kWG) * 512, c, K, x);
        if (res) read8<kSF>(out.at + (v * kW + kWG + kWS) * 512, c, K, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = fma2(x[j], f2, fma2(mul2(g[j], w[v][j]), k2, r[j]));
        store8<kSF>(dx, c, K, r);
      }
    }
    out.next();
  }
  cp_async_wait<0>();
  if (a.dw == nullptr) return;
  if (teams > 1) {                         // the block's rows at once, one after another
    char* cols = reinterpret_cast<char*>(smem);
    const int32_t wide = kVec * tpr * 8;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const C c(tpr, i, v);
      ulonglong2* p0 = reinterpret_cast<ulonglong2*>(cols + ((team - 1) * wide + c.c0) * 4);
      ulonglong2* p1 = reinterpret_cast<ulonglong2*>(cols + ((team - 1) * wide + c.c1) * 4);
      if (team > 0) {
        *p0 = make_ulonglong2(dw[v][0], dw[v][1]);
        *p1 = make_ulonglong2(dw[v][2], dw[v][3]);
      }
    }
    __syncthreads();
    if (team > 0) return;
    for (int o = 1; o < teams; ++o)
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const C c(tpr, i, v);
        const char* p = row_at<true>(static_cast<const void*>(cols), (o - 1) * wide);
        uint64_t x[4];
        pairs_of<true>(*reinterpret_cast<const uint4*>(p + 4 * c.c0), *reinterpret_cast<const uint4*>(p + 4 * c.c1), x);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[v][j] = add2(dw[v][j], x[j]);
      }
  }
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    store8<true>(row_at<true>(static_cast<void*>(a.work), (int64_t)blockIdx.x * K), C(tpr, i, v), K, dw[v]);
}

// Wider rows, straight from memory: dY, H and w read twice, this block's part of dw once
// a row, and nothing ahead (4000 rows of 10240 with all in fp32 181 us, 3.6 TB/s; of 9216
// through the ring 90, 6.6).
template <bool kGF, bool kSF>
__global__ void __launch_bounds__(kWideThreads) norm_bwd_wide_kernel(const NormBwdArgs a) {
  constexpr bool kSplit = kGF || kSF;
  using C = Cols<kSplit>;
  __shared__ float part[64];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tpr = kWideThreads, i = threadIdx.x;
  const int32_t K = a.K;
  // this block's part of dw: no register is free for it
  char* mine = row_at<true>(static_cast<void*>(a.work), (int64_t)blockIdx.x * K);
  int buf = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float k = a.rstd[t];
    const uint64_t k2 = pack2(k, k);
    const char* dy = row_at<kGF>(a.dY, t * a.ldd);
    const char* h = row_at<kSF>(a.H, t * a.ldh);
    uint64_t dot = 0;
#pragma unroll
    for (int v = 0; v < kWide; ++v) {
      const C c(tpr, i, v);
      uint64_t g[4], x[4], w[4], d[4] = {0, 0, 0, 0};
      load8<kGF>(dy, c, K, g);
      load8<kSF>(h, c, K, x);
      load_w(a.w, a.w_f32, c, K, w);
      if (a.dw != nullptr && t != blockIdx.x) load8<true>(static_cast<const char*>(mine), c, K, d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t gx = mul2(g[j], x[j]);
        d[j] = fma2(gx, k2, d[j]);
        dot = fma2(gx, w[j], dot);
      }
      if (a.dw != nullptr) store8<true>(mine, c, K, d);
    }
    const float2 q = unpack2(dot);
    const float f = bwd_factor(row_sum(q.x + q.y, tpr, 0, part, buf), k, 1.0f / (float)K);
    const uint64_t f2 = pack2(f, f);
#pragma unroll
    for (int v = 0; v < kWide; ++v) {
      const C c(tpr, i, v);
      uint64_t g[4], x[4], w[4], r[4] = {0, 0, 0, 0};
      load8<kGF>(dy, c, K, g);
      load8<kSF>(h, c, K, x);
      load_w(a.w, a.w_f32, c, K, w);
      if (a.dR != nullptr) load8<kSF>(row_at<kSF>(a.dR, t * a.ldr), c, K, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = fma2(x[j], f2, fma2(mul2(g[j], w[j]), k2, r[j]));
      store8<kSF>(row_at<kSF>(a.dX, t * a.ldx), c, K, r);
    }
  }
}

// Few rows in one launch: the first `dw_blocks` take 64 columns of dw each, which needs
// no other result (H and dY are read twice for it), the others a row a team.  Not
// where dX is written over what they read.  Bound by a row's latency and the column
// blocks' chain of loads, eight rows a warp at once: 259 rows of 2176, fp32, 5.2 to 6.1
// us box to box (in two launches 7.8).
template <bool kF32>
__device__ __forceinline__ float2 two_of(const void* base, int64_t at) {
  if (kF32) return *reinterpret_cast<const float2*>(row_at<true>(base, at));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(row_at<false>(base, at));
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool kGF, bool kSF>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_few_kernel(const NormBwdArgs a, int32_t tpr, int32_t dw_blocks) {
  constexpr bool kSplit = kGF || kSF;
  __shared__ float part[64];
  __shared__ float2 cols[kBwdThreads / 32][32];
  const int32_t K = a.K;
  if ((int32_t)blockIdx.x < dw_blocks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int32_t c = (int32_t)blockIdx.x * 64 + 2 * lane;
    float2 sum = make_float2(0.0f, 0.0f);
    if (c < K) {
#pragma unroll 8
      for (int32_t t = warp; t < a.T; t += warps) {
        const float k = a.rstd[t];
        const float2 g = two_of<kGF>(a.dY, t * a.ldd + c), x = two_of<kSF>(a.H, t * a.ldh + c);
        sum.x = fmaf(g.x * x.x, k, sum.x);
        sum.y = fmaf(g.y * x.y, k, sum.y);
      }
    }
    cols[warp][lane] = sum;
    __syncthreads();
    if (warp > 0 || c >= K) return;
    for (int w = 1; w < warps; ++w) {
      sum.x += cols[w][lane].x;
      sum.y += cols[w][lane].y;
    }
    a.dw[c] = sum.x;
    a.dw[c + 1] = sum.y;
    return;
  }
  const int teams = blockDim.x / tpr, team = threadIdx.x / tpr, i = threadIdx.x - team * tpr;
  const int64_t t = (int64_t)((int32_t)blockIdx.x - dw_blocks) * teams + team;
  const bool there = t < a.T;
  const Cols<kSplit> c(tpr, i, 0);
  uint64_t g[4] = {}, x[4] = {}, r[4] = {}, w[4] = {};
  float k = 0.0f;
  if (there) {
    load8<kGF>(row_at<kGF>(a.dY, t * a.ldd), c, K, g);
    load8<kSF>(row_at<kSF>(a.H, t * a.ldh), c, K, x);
    if (a.dR != nullptr) load8<kSF>(row_at<kSF>(a.dR, t * a.ldr), c, K, r);
    load_w(a.w, a.w_f32, c, K, w);
    k = a.rstd[t];
  }
  uint64_t dot = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) dot = fma2(mul2(g[j], x[j]), w[j], dot);
  const float2 q = unpack2(dot);
  int buf = 0;
  const float f = bwd_factor(row_sum(q.x + q.y, tpr, team, part, buf), k, 1.0f / (float)K);
  if (!there) return;
  const uint64_t k2 = pack2(k, k), f2 = pack2(f, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = fma2(x[j], f2, fma2(mul2(g[j], w[j]), k2, r[j]));
  store8<kSF>(row_at<kSF>(a.dX, t * a.ldx), c, K, r);
}

// dw from the blocks' parts, which are in L2 still: a block takes 32 columns, a warp of
// it every 16th part, all in a fixed order.  Its launch overlaps the kernel before;
// about 3 us, a chain of ten loads.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) norm_dw_kernel(const float* work, int32_t parts, int32_t K, float* dw) {
  __shared__ float sh[kSumWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t c = (int32_t)blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (c < K) {
#pragma unroll 10
    for (int32_t p = warp; p < parts; p += kSumWarps) sum += work[(int64_t)p * K + c];
  }
  sh[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < K) {
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) sum += sh[w][lane];
    dw[c] = sum;
  }
}

}  // namespace norm

namespace {
constexpr int kPipedK = 16384;
constexpr int kRoom = 224 * 1024;          // shared memory of an SM that the rings take
constexpr int kSms = 152;                  // so that the scratch needs no device to be asked for
constexpr int kFewRows = 384;

struct Shape {
  int vec, tpr, teams;                     // vectors of eight columns a thread, threads a row, rows a block
  int threads() const { return teams * tpr; }
  // of a ring, with `words` of 16 bytes a vector
  int64_t bytes(int words, int stages) const { return (int64_t)threads() * vec * words * 16 * stages; }
};

// As few vectors a thread as a block's threads allow, from `least` on (of the forward
// pass: 8191 rows of 2048 with an fp32 stream 32 us on one vector each, 34 on two; of
// the backward pass: 28000 of 2048 120 and 148); half a warp to 128 columns.  Rows
// share a block once there is a row for each of `blocks`.
Shape shape_of(int64_t T, int32_t K, int threads, int64_t blocks, int least = 1) {
  const int n = K / 8;
  int vec = 1, tpr = 16;
  if (n > 16) {
    while (vec < least && n >= 32 * (vec + 1)) ++vec;
    while ((n + vec - 1) / vec > (vec == 1 ? threads : norm::kThreads)) ++vec;
    tpr = ((n + vec - 1) / vec + 31) / 32 * 32;
  }
  const int64_t want = (T + blocks - 1) / blocks;
  int teams = (vec == 1 ? threads : norm::kThreads) / tpr;
  if (tpr > 32 && teams > 15) teams = 15;  // a barrier each, beside the block's
  if (want < teams) teams = want > 0 ? (int)want : 1;
  return {vec, tpr, tpr == 16 ? (teams + 1) / 2 * 2 : teams};      // whole warps
}

template <auto kKernel>
cudaError_t allow_ring() {
  static std::atomic<bool> done[64];       // of this kernel, by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev].load()) {
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    if (e == cudaSuccess && dev < 64) done[dev].store(true);
  }
  return e;
}

template <bool kXF, bool kSF, int kVec>
cudaError_t norm_ring(const NormArgs& a, const Shape& h, int64_t grid, int stages, bool late, cudaStream_t s) {
  constexpr auto kernel = norm::norm_kernel<kXF, kSF, kVec>;
  const cudaError_t e = allow_ring<kernel>();
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)grid, (unsigned)h.threads(), (size_t)h.bytes((kXF ? 2 : 1) + (kSF ? 2 : 1), stages), s>>>(
      a, h.tpr, stages, late);
  return cudaGetLastError();
}

template <bool kXF, bool kSF>
cudaError_t norm_as(const NormArgs& a, cudaStream_t s) {
  constexpr int words = (kXF ? 2 : 1) + (kSF ? 2 : 1);
  const int sms = num_sms_current_device();
  Shape h = {};
  int per = 0;                             // blocks an SM; none where a ring of two rows does not fit
  if (a.K <= kPipedK) {
    // Where a column costs more instructions than bytes, its row's own are shared by
    // more vectors a thread (us with 1, 2 and 4 of them, rows of bf16: 20000 of 2048
    // without a residual to bf16 33, 29, 31, to E4M3 41, 34, 29, to both 44, 37, 37;
    // 4000 to E4M3 11.3, 9.8, 10.3; with a residual to it and E4M3 49, 46, 48, to all
    // three 58, 64, 64; of fp32 without one to bf16 42, 38, 39, 1000 of them 5.2, 5.4, 6.4).
    const bool codes = a.Q != nullptr && a.Y == nullptr, alone = a.R == nullptr;
    int least = a.T >= 8 * sms && (alone || (codes && words == 2)) ? 2 : 1;
    if (alone && codes && !kXF && (int64_t)a.T * a.K >= (int64_t)8 * sms * 16384) least = 4;
    h = shape_of(a.T, a.K, norm::kThreads, 2 * (int64_t)sms, least);
    per = h.vec <= 2 && 2 * h.bytes(words, 2) <= kRoom ? 2 : h.bytes(words, 2) <= kRoom ? 1 : 0;
  }
  if (per == 0) {
    norm::norm_wide_kernel<kXF, kSF><<<(unsigned)a.T, norm::kWideThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  // Bytes that one row ahead in every block of an SM reads: with less than 32 KB two
  // rows are copied ahead (16384 rows of 7168 without a residual 73 us, one ahead
  // 80).  Where those and a row's results are more than 96 KB the copies wait for a
  // row's sum (us late and not: 16384 rows of 7168 to bf16 and E4M3 160 and 181, 20000
  // of 2048 fp32 to all three 93 and 104, with an fp32 stream alone 83 and 92; with
  // less, 20000 of 2048 in bf16 60 and 52, 8191 with an fp32 stream 34 and 32), but not
  // without a residual (8000 of 7168 fp32 to bf16 and E4M3, 98 KB, 67 and 65).
  const int64_t read = (kXF ? 4 : 2) + (a.R != nullptr ? (kSF ? 4 : 2) : 0);
  const int64_t write = (a.H != nullptr ? (kSF ? 4 : 2) : 0) + (a.Y != nullptr ? 2 : 0) + (a.Q != nullptr ? 1 : 0);
  const int64_t columns = (int64_t)a.K * h.teams * per, flight = read * columns;
  const int stages = flight < 32 * 1024 && per * h.bytes(words, 3) <= kRoom ? 3 : 2;
  const bool late = a.R != nullptr && flight + write * columns > 96 * 1024;
  const int64_t need = ((int64_t)a.T + h.teams - 1) / h.teams, most = (int64_t)per * sms;
  const int64_t grid = need < most ? need : most;
  if (h.vec == 1) return norm_ring<kXF, kSF, 1>(a, h, grid, stages, late, s);
  if (h.vec == 2) return norm_ring<kXF, kSF, 2>(a, h, grid, stages, late, s);
  if (h.vec == 3) return norm_ring<kXF, kSF, 3>(a, h, grid, stages, late, s);
  return norm_ring<kXF, kSF, 4>(a, h, grid, stages, late, s);
}

// The backward pass: one block an SM.
Shape bwd_shape(int64_t T, int32_t K) { return shape_of(T, K, norm::kBwdThreads, kSms); }
int64_t bwd_blocks(int64_t T, int32_t K) {
  const int teams = K > kPipedK ? 1 : bwd_shape(T, K).teams;
  const int64_t n = (T + teams - 1) / teams;
  return n < kSms ? n : kSms;
}

template <bool kGF, bool kSF, int kVec>
cudaError_t norm_bwd_ring(const NormBwdArgs& a, const Shape& h, unsigned grid, int stages, int64_t bytes,
                          cudaStream_t s) {
  constexpr auto kernel = norm::norm_bwd_kernel<kGF, kSF, kVec>;
  const cudaError_t e = allow_ring<kernel>();
  if (e != cudaSuccess) return e;
  kernel<<<grid, (unsigned)h.threads(), (size_t)bytes, s>>>(a, h.tpr, stages);
  return cudaGetLastError();
}

// Three rows in the ring where they fit (8191 rows of 7168 77 us, with two 83).
template <bool kGF, bool kSF>
cudaError_t norm_bwd_rows(const NormBwdArgs& a, unsigned grid, cudaStream_t s) {
  constexpr int words = (kGF ? 2 : 1) + 2 * (kSF ? 2 : 1);
  const Shape h = a.K > kPipedK ? Shape{} : bwd_shape(a.T, a.K);
  const int stages = h.bytes(words, 3) <= kRoom ? 3 : 2;
  const int64_t bytes = h.bytes(words, stages);
  if (h.vec == 0 || bytes > kRoom) {
    norm::norm_bwd_wide_kernel<kGF, kSF><<<grid, norm::kWideThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (h.vec == 1) return norm_bwd_ring<kGF, kSF, 1>(a, h, grid, stages, bytes, s);
  if constexpr (words < 5) {               // four vectors of five words do not fit
    if (h.vec == 4) return norm_bwd_ring<kGF, kSF, 4>(a, h, grid, stages, bytes, s);
  }
  return norm_bwd_ring<kGF, kSF, 3>(a, h, grid, stages, bytes, s);
}

template <bool kGF, bool kSF>
cudaError_t norm_bwd_as(const NormBwdArgs& a, cudaStream_t s) {
  // Few rows in one launch (us in one and two: 64 rows of 2048 2.6 and 4.6, 250 of 7168
  // 9.0 and 11.8, 500 of them 14.1 and 14.1; fp32, 256 of 2048 4.1 and 7.5, 512 of them
  // 11.4 and 9.3).
  if (a.dw != nullptr && a.T > 0 && a.T <= kFewRows && a.K <= 8 * norm::kBwdThreads && a.dX != a.dY && a.dX != a.H) {
    const int32_t tpr = a.K <= 128 ? 16 : (a.K / 8 + 31) / 32 * 32, teams = tpr < 256 ? 256 / tpr : 1, dw_blocks = (a.K + 63) / 64;
    norm::norm_bwd_few_kernel<kGF, kSF>
        <<<(unsigned)(dw_blocks + (a.T + teams - 1) / teams), (unsigned)(teams * tpr), 0, s>>>(a, tpr, dw_blocks);
    return cudaGetLastError();
  }
  const unsigned grid = (unsigned)bwd_blocks(a.T, a.K);
  if (grid > 0) {
    const cudaError_t e = norm_bwd_rows<kGF, kSF>(a, grid, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dw == nullptr) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((a.K + 31) / 32));
  cfg.blockDim = dim3(32 * norm::kSumWarps);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm::norm_dw_kernel, static_cast<const float*>(a.work), (int32_t)grid, a.K, a.dw);
}
}  // namespace

int64_t norm_work_bytes(int64_t T, int32_t K) { return bwd_blocks(T, K) * K * (int64_t)sizeof(float); }

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  if (a.x_f32) return a.s_f32 ? norm_as<true, true>(a, s) : norm_as<true, false>(a, s);
  return a.s_f32 ? norm_as<false, true>(a, s) : norm_as<false, false>(a, s);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
  if (a.g_f32) return a.s_f32 ? norm_bwd_as<true, true>(a, s) : norm_bwd_as<true, false>(a, s);
  return a.s_f32 ? norm_bwd_as<false, true>(a, s) : norm_bwd_as<false, false>(a, s);
}

}  // namespace mg
