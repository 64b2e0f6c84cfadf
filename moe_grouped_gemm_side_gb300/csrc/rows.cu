// Token rows on their way into and out of the grouped GEMMs: dispatch into the
// contiguous or masked layout (as bf16, or E4M3 with UE8M0 scales), combine
// and its gradients, and SwiGLU with its rows kept in 8 bits for the backward
// pass.  All of these are bound by memory traffic: each reads its inputs once
// and writes its outputs once, eight columns to a thread, and computes in
// fp32, two columns to an instruction.
#include <atomic>

#include "blockq.cuh"
#include "common.cuh"
#include "ops_internal.h"

namespace mg {
namespace rows {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPass = kThreads * 8;        // columns of one pass of a block
constexpr int kMaxSpan = 4 * kPass;        // columns of a token a dispatch block stages

// Row of choice j of token t; -1 where there is none.  A coherent load:
// dispatch_kernel may be resident while the slot map is still being written, and
// the non-coherent path is for data that nothing writes meanwhile.
__device__ __forceinline__ int32_t load_row(const int32_t* rows, int64_t t, int32_t k, int j, int64_t rows_total,
                                            int32_t* status) {
  if (j >= k) return -1;
  const int32_t r = rows[t * k + j];
  if (r >= rows_total) {
    set_status(status, MG_ERR_DEVICE_ARG);
    return -1;
  }
  return r;
}

// shared -> global, asynchronous; 16-byte aligned, whole 16-byte units
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
}

// 16 bytes read once, or zeros: predicated rather than branched around, so that
// a thread's loads of several rows leave together.
__device__ __forceinline__ uint4 load_or_zero(const void* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@p ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)there));
  return v;
}

// Block (t, y): columns [y * span, (y + 1) * span) of token t are read once,
// converted into shared memory, and written to each of the token's rows by a
// bulk copy: a token is quantised once however many rows it gets, and the
// writes, most of the traffic, take one instruction a row.  Bound by those
// writes: 65536 bf16 rows of 2048 from 8-bit tokens 42 us (the copy rate), 32768
// of 7168 copied as bf16 79 us (5.9 TB/s), as E4M3 50 us (4.7 TB/s; 44 without
// the scale bytes, each an L2 write of its own, because the rows of one token
// are never neighbours).
template <bool kSrcQ, bool kDstQ, bool kCkpt>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs a, int32_t span) {
  static_assert(!(kSrcQ && kCkpt), "a checkpoint is taken of bf16 tokens");
  constexpr bool kNeedQ = kDstQ || kCkpt, kNeedH = !kDstQ;
  __shared__ alignas(128) uint8_t buf_h[kNeedH ? 2 * kMaxSpan : 16];
  __shared__ alignas(128) uint8_t buf_q[kNeedQ ? kMaxSpan : 16];
  __shared__ uint8_t sc[kMaxSpan / 128];
  __shared__ int32_t sh[kMaxTopK];
  const int64_t t = blockIdx.x;
  const int32_t c0 = (int32_t)blockIdx.y * span, n = min(span, a.K - c0), KB = a.K >> 7;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t pass = (int32_t)blockDim.x * 8;
  // launched while the kernel before it may still run: its results first, by
  // coherent loads
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint4 h[4];
  uint2 q[4];
  uint32_t s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t c = tid * 8 + i * pass;
    h[i] = make_uint4(0, 0, 0, 0);
    q[i] = make_uint2(0, 0);
    s[i] = 127;
    if (c < n) {
      if (kSrcQ) {
        q[i] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.X) + t * a.ldx + c0 + c));
        s[i] = a.SX[t * KB + ((c0 + c) >> 7)];
      } else {
        h[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.X) + t * a.ldx + c0 + c));
      }
    }
  }
  if (tid < a.k) sh[tid] = load_row(a.rows, t, a.k, tid, a.rows_total, a.status);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t c = tid * 8 + i * pass;
    if (i * pass >= n) break;
    uint64_t x[4];
    if (kSrcQ) {
      if (!kDstQ) {
        e4m3x8_decode(q[i], ue8m0_value(s[i]), x);
        h[i] = f32x2_to_bf16x8(x);
      }
    } else if (kNeedQ) {
      s[i] = (uint32_t)ue8m0_of_amax(block_amax_bf16(h[i]));
      bf16x8_to_f32x2(h[i], x);
      q[i] = e4m3x8_encode(x, ue8m0_inverse((int32_t)s[i]));
    }
    if (c < n) {
      if (kNeedH) *reinterpret_cast<uint4*>(buf_h + 2 * c) = h[i];
      if (kNeedQ) {
        *reinterpret_cast<uint2*>(buf_q + c) = q[i];
        if ((tid & 15) == 0) sc[c >> 7] = (uint8_t)s[i];
      }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {
    const int32_t r = lane < a.k ? sh[lane] : -1;
    if (r >= 0) {
      const int64_t at = (int64_t)r * a.K + c0;
      if (kDstQ)
        bulk_store(static_cast<uint8_t*>(a.A) + at, buf_q, (uint32_t)n);
      else
        bulk_store(static_cast<__nv_bfloat16*>(a.A) + at, buf_h, 2u * (uint32_t)n);
    }
    if (kCkpt && lane == 0) bulk_store(a.CX + t * a.K + c0, buf_q, (uint32_t)n);
    bulk_commit_group();
  }
  if (kCkpt && tid < (n >> 7)) a.SCX[t * KB + (c0 >> 7) + tid] = sc[tid];
  if (kDstQ) {
    for (int j = warp; j < a.k; j += (int)(blockDim.x >> 5)) {
      const int32_t r = sh[j];
      if (r < 0) continue;
      const uint32_t G = (uint32_t)a.group_rows, z = (uint32_t)r / G;
      uint8_t* dst = a.SFA + ((int64_t)z * KB + (c0 >> 7)) * G + ((uint32_t)r - z * G);
      for (int32_t b = lane; b < (n >> 7); b += 32) dst[(int64_t)b * G] = sc[b];
    }
  }
  if (warp == 0) bulk_wait_read_all();       // the block's shared memory may go
}

// Choice j of token tok of a block's kTok, at its place among the block's.
// kTok > 1 only where kN choices are all of a token's.
template <int kN, int kTok, typename Args>
__device__ __forceinline__ void load_choices(const Args& a, int64_t t0, int tid, int32_t* sh, float* sw) {
  const int tok = kTok > 1 ? tid / kN : 0, j = kTok > 1 ? tid % kN : tid;
  if (tid < (kTok > 1 ? kN * kTok : kMaxTopK)) {
    const int64_t t = t0 + tok;
    const int32_t r = kTok == 1 || t < a.T ? load_row(a.rows, t, a.k, j, a.rows_total, a.status) : -1;
    sh[tid] = r;
    sw[tid] = r < 0 ? 0.0f : a.w != nullptr ? __ldg(a.w + t * a.k + j) : 1.0f;
  }
}

// Block (b, y): out[t] = sum_j w_tj D[row(t, j)] over a span of columns, for
// kTok tokens t, in the order of the choices, in fp32, rounded once.  kN rows of
// each token are loaded together.  Bound by reading the rows: 32768 of 7168
// 83 us, 6.3 TB/s.
template <bool kF32, int kN, int kTok>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
  __shared__ int32_t sh[kMaxTopK];
  __shared__ float sw[kMaxTopK];
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int tid = threadIdx.x;
  load_choices<kN, kTok>(a, t0, tid, sh, sw);
  __syncthreads();
  const int32_t c = (int32_t)((blockIdx.y * blockDim.x + tid) * 8);
  if (c >= a.K) return;
  const __nv_bfloat16* D = static_cast<const __nv_bfloat16*>(a.D) + c;
  uint64_t acc[kTok][4] = {};
  for (int j0 = 0; j0 < (kTok > 1 ? 1 : a.k); j0 += kN) {
    uint4 v[kN * kTok];
#pragma unroll
    for (int i = 0; i < kN * kTok; ++i) {
      const int32_t r = sh[j0 + i];
      v[i] = load_or_zero(D + (int64_t)r * a.K, r >= 0);
    }
#pragma unroll
    for (int i = 0; i < kN * kTok; ++i) {
      const float w = sw[j0 + i];
      const uint64_t w2 = pack2(w, w);
      uint64_t x[4];
      bf16x8_to_f32x2(v[i], x);
#pragma unroll
      for (int p = 0; p < 4; ++p) acc[i / kN][p] = fma2(x[p], w2, acc[i / kN][p]);
    }
  }
#pragma unroll
  for (int tok = 0; tok < kTok; ++tok) {
    const int64_t t = t0 + tok;
    if (kTok > 1 && t >= a.T) return;
    if (kF32) {
      float* o = static_cast<float*>(a.out) + t * a.ldo + c;
      const float2 p0 = unpack2(acc[tok][0]), p1 = unpack2(acc[tok][1]);
      const float2 p2 = unpack2(acc[tok][2]), p3 = unpack2(acc[tok][3]);
      *reinterpret_cast<float4*>(o) = make_float4(p0.x, p0.y, p1.x, p1.y);
      *reinterpret_cast<float4*>(o + 4) = make_float4(p2.x, p2.y, p3.x, p3.y);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + t * a.ldo + c) = f32x2_to_bf16x8(acc[tok]);
    }
  }
}

// kN sums over a warp at once: afterwards every lane holds the total of value
// lane / (32 / kN) in v[0].
template <int kN>
__device__ __forceinline__ void warp_sums(float (&v)[kN], int lane) {
  constexpr int kBit = 32 / kN;
#pragma unroll
  for (int n = kN / 2; n >= 1; n >>= 1) {
    const bool hi = (lane & (kBit * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = hi ? v[i + n] : v[i], send = hi ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, kBit * n);
    }
  }
#pragma unroll
  for (int n = kBit / 2; n >= 1; n >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], n);
}

template <bool kF32>
__device__ __forceinline__ void load8(const void* p, int64_t at, uint64_t (&x)[4]) {
  if (kF32) {
    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
    x[0] = pack2(u.x, u.y);
    x[1] = pack2(u.z, u.w);
    x[2] = pack2(v.x, v.y);
    x[3] = pack2(v.z, v.w);
  } else {
    bf16x8_to_f32x2(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at), x);
  }
}

// Block b: dD[row] = w dout[t] and dw = <dout[t], D[row]> for the rows of kTok
// tokens t, kN rows of each in flight together; their dot products are reduced at
// once.  Bound by memory: 65536 rows of 2048 93 us, 6.1 TB/s.
template <bool kF32, int kN, int kTok>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const CombineBwdArgs a) {
  constexpr int kSlots = kN * kTok;
  __shared__ int32_t sh[kMaxTopK];
  __shared__ float sw[kMaxTopK];
  __shared__ float part[kTok > 1 ? 1 : kMaxTopK / kN][kWarps][kSlots];
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  load_choices<kN, kTok>(a, t0, tid, sh, sw);
  __syncthreads();
  const __nv_bfloat16* D = static_cast<const __nv_bfloat16*>(a.D);
  __nv_bfloat16* dD = static_cast<__nv_bfloat16*>(a.dD);
  const bool dots = a.dw != nullptr;
  for (int j0 = 0; j0 < (kTok > 1 ? 1 : a.k); j0 += kN) {
    float dot[kSlots] = {};
    for (int32_t c = tid * 8; c < a.K; c += (int32_t)blockDim.x * 8) {
      uint4 v[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int32_t r = sh[j0 + i];
        v[i] = load_or_zero(D + (int64_t)r * a.K + c, dots && r >= 0);
      }
#pragma unroll
      for (int tok = 0; tok < kTok; ++tok) {
        if (kTok > 1 && t0 + tok >= a.T) break;
        uint64_t g[4];
        load8<kF32>(a.dout, (t0 + tok) * a.ldd + c, g);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const int i = tok * kN + j;
          const int32_t r = sh[j0 + i];
          if (r < 0) continue;
          const float w = sw[j0 + i];
          const uint64_t w2 = pack2(w, w);
          uint64_t x[4], o[4];
          bf16x8_to_f32x2(v[i], x);
          uint64_t d = mul2(g[0], x[0]);
#pragma unroll
          for (int p = 1; p < 4; ++p) d = fma2(g[p], x[p], d);
          const float2 f = unpack2(d);
          dot[i] += f.x + f.y;
#pragma unroll
          for (int p = 0; p < 4; ++p) o[p] = mul2(g[p], w2);
          __stcs(reinterpret_cast<uint4*>(dD + (int64_t)r * a.K + c), f32x2_to_bf16x8(o));
        }
      }
    }
    if (dots) {
      warp_sums<kSlots>(dot, lane);
      if ((lane & (32 / kSlots - 1)) == 0) part[j0 / kN][warp][lane / (32 / kSlots)] = dot[0];
    }
  }
  if (!dots) return;
  __syncthreads();
  const int tok = kTok > 1 ? tid / kN : 0, j = kTok > 1 ? tid % kN : tid;
  if (j < a.k && tok < kTok && (kTok == 1 || t0 + tok < a.T)) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
      if (i < (int)(blockDim.x >> 5)) s += part[tid / kSlots][i][tid % kSlots];
    a.dw[(t0 + tok) * a.k + j] = s;
  }
}

// 1 / (1 + e^-g) of two values from the hardware's exponential and reciprocal,
// results below 2^-126 flushed to 0: the sum under the reciprocal is at least 1,
// so only a sigmoid below 2^-126 is lost (the stated limit of SiLU), and the
// flushing forms cost two instructions where the others scale their operands.
__device__ __forceinline__ uint64_t fast_sigmoid2(uint64_t g) {
  float2 x = unpack2(mul2(g, pack2(-1.4426950408889634f, -1.4426950408889634f)));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.y));
  x = unpack2(add2(pack2(x.x, x.y), pack2(1.0f, 1.0f)));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.y));
  return pack2(x.x, x.y);
}

// Rows that a team of threads walks: `step` teams, the n-th row of team i is
// n step + (i + n turn) mod step.  Rows without a choice come in runs (padding,
// unfilled buffers) whose distance often divides the number of teams: in plain
// strides some teams would meet nothing but choices and others none (buffers of
// 16 to 1024 rows, a tenth to two fifths filled: the busiest team has up to 8
// times its share of rows, with this turn up to 3; backward of 1505 rows in 24
// buffers of 304 15 us instead of 23, of 203 in 64 of 128 7.0 instead of 12.2).
struct Walk {
  uint32_t base, pos;                        // n step; (i + n turn) mod step, the row's place after it
  __device__ __forceinline__ static uint32_t turn(uint32_t step) { return step * 125 / 128 | 1; }
  __device__ __forceinline__ static uint32_t wrap(uint32_t p, uint32_t step) { return p >= step ? p - step : p; }
  __device__ __forceinline__ uint32_t row() const { return base + pos; }
  __device__ __forceinline__ Walk next(uint32_t step) const {
    return Walk{base + step, wrap(pos + turn(step), step)};
  }
};

// The first row from `w` on for which entry(row) >= 0; `at` is its entry, -1
// when there is none.  A warp looks up 32 rows at once.
template <typename F>
__device__ __forceinline__ void next_row(Walk& w, uint32_t step, uint32_t R, int lane, const F& entry, int32_t& at) {
  at = -1;
  if (w.base >= R) return;
  const uint32_t mine = (uint32_t)lane * Walk::turn(step) % step, all = 32u * Walk::turn(step) % step;
  for (; w.base < R; w.base += 32 * step) {
    const uint32_t pos = Walk::wrap(w.pos + mine, step);
    const int32_t e = entry(w.base + lane * step + pos);
    const uint32_t live = __ballot_sync(0xffffffffu, e >= 0);
    if (live != 0) {
      const int i = __ffs(live) - 1;
      at = __shfl_sync(0xffffffffu, e, i);
      w.pos = __shfl_sync(0xffffffffu, pos, i);
      w.base += i * step;
      return;
    }
    w.pos = Walk::wrap(w.pos + all, step);
  }
}

// `tpr` threads per row: feature f of a row sits at gate column 256 (f / 128) +
// f % 128, its up column 128 further.  A thread's next row is on its way
// while it computes the current one; a block takes whole rows, so that a row's
// bytes are read and written together (pieces of more rows at once, copied
// further ahead through shared memory, took 174 to 192 us).  Bound by memory:
// 65536 rows of N = 4096 165 us, 6.5 TB/s; to E4M3 154 us, 6.1 TB/s (the second
// scale's shuffles, and two thirds of the instruction slots taken).
template <bool kYQ>
__global__ void __launch_bounds__(kThreads, 4) swiglu_save_kernel(const SwigluSaveArgs a, int32_t tpr) {
  const int32_t blocks = a.N >> 8, I = a.N >> 1;
  const int tid = threadIdx.x, lane16 = tid & 15;
  const int32_t rows_per_block = (int32_t)blockDim.x / tpr;
  const uint32_t step = gridDim.x * (uint32_t)rows_per_block, R = (uint32_t)a.rows_total;
  const __nv_bfloat16* H = static_cast<const __nv_bfloat16*>(a.H);
  const int32_t off = tid / tpr, first = (tid - off * tpr) * 8;
  for (int32_t f0 = 0; f0 < I; f0 += tpr * 8) {
    const int32_t f = f0 + first, j = f >> 7;
    const bool col = f < I;
    const int64_t c = (int64_t)j * 256 + (f & 127);
    uint4 g = make_uint4(0, 0, 0, 0), u = g;
    auto live = [&](uint32_t r) { return r < R && col && (a.src == nullptr || __ldg(a.src + r) >= 0); };
    auto fetch = [&](uint32_t r, uint4& g, uint4& u) {
      const __nv_bfloat16* h = H + (int64_t)r * a.N + c;
      g = __ldcs(reinterpret_cast<const uint4*>(h));
      u = __ldcs(reinterpret_cast<const uint4*>(h + 128));
    };
    Walk w{0, blockIdx.x * (uint32_t)rows_per_block + off}, w1 = w.next(step);
    bool in = live(w.row()), in1 = live(w1.row());
    if (in) fetch(w.row(), g, u);
    for (; w.base < R; w = w1, w1 = w1.next(step)) {
      const int64_t r = w.row();
      uint4 g1 = make_uint4(0, 0, 0, 0), u1 = g1;
      if (in1) fetch(w1.row(), g1, u1);
      const bool in2 = live(w1.next(step).row());
      if (!__any_sync(0xffffffffu, in)) {      // rows that hold no choice
        in = in1;
        in1 = in2;
        g = g1;
        u = u1;
        continue;
      }
      // gate maximum in the low half, up maximum in the high half
      const uint32_t mg = bf16x8_amax2(g), mu = bf16x8_amax2(u);
      const uint32_t m = block_max2(bf16x2_max(__byte_perm(mg, mu, 0x5410), __byte_perm(mg, mu, 0x7632)));
      const int32_t sg = ue8m0_of_amax(bf16_lo(m)), su = ue8m0_of_amax(bf16_hi(m));
      uint64_t xg[4], xu[4], y[4];
      bf16x8_to_f32x2(g, xg);
      bf16x8_to_f32x2(u, xu);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(xg[i], fast_sigmoid2(xg[i])), xu[i]);
      const int32_t sy = kYQ ? ue8m0_of_amax(block_amax(y)) : 127;
      if (in) {
        uint8_t* hc = a.HC + r * a.N + c;
        __stcs(reinterpret_cast<uint2*>(hc), e4m3x8_encode(xg, ue8m0_inverse(sg)));
        __stcs(reinterpret_cast<uint2*>(hc + 128), e4m3x8_encode(xu, ue8m0_inverse(su)));
        if (lane16 == 0)
          *reinterpret_cast<uint16_t*>(a.SHC + r * 2 * blocks + 2 * j) = (uint16_t)(sg | (su << 8));
        if (kYQ) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + r * I + f) = e4m3x8_encode(y, ue8m0_inverse(sy));
          if (lane16 == 0) {
            const uint32_t G = (uint32_t)a.group_rows, z = (uint32_t)r / G;
            a.SFY[((int64_t)z * blocks + j) * G + ((uint32_t)r - z * G)] = (uint8_t)sy;
          }
        } else {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) + r * I + f) = f32x2_to_bf16x8(y);
        }
      }
      in = in1;
      in1 = in2;
      g = g1;
      u = u1;
    }
  }
}

template <int kBytes>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

constexpr int kBwdStages = 4;
struct BwdSlots {               // one thread's operands of one piece, per stage
  uint4 d[kBwdStages][kThreads];
  uint2 g[kBwdStages][kThreads];
  uint2 u[kBwdStages][kThreads];
  float w[kBwdStages][kThreads];
  int2 row[kBwdStages][kThreads];   // the row and its entry of w and dw (-1: no more rows)
};

// A piece is eight features of a row, tpr threads share a row.  Every thread
// copies its own pieces into its own shared-memory slots kBwdStages - 1
// pieces ahead (a thread waits for its own copies only, so no barrier is
// needed), which keeps enough bytes in flight without the registers.  The
// routing weight's gradient is a sum over the row's threads, in a fixed order:
// within warps by shuffles, across them through shared memory (two buffers, so
// that one barrier of the row's threads per row is enough).
__global__ void __launch_bounds__(kThreads, 4) swiglu_bwd_kernel(const SwigluBwdArgs a, int32_t tpr) {
  __shared__ BwdSlots sl;
  __shared__ float part[2][kWarps];
  const int32_t I = a.N >> 1, span = tpr * 8;      // features between a thread's pieces
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t rows_per_block = kThreads / tpr, off = tid / tpr, first = (tid & (tpr - 1)) * 8;
  const int32_t col = (first >> 7) * 256 + (first & 127);         // gate column of the first piece
  const uint32_t step = gridDim.x * (uint32_t)rows_per_block, R = (uint32_t)a.rows_total;
  const bool weights = a.w != nullptr || a.dw != nullptr;
  // entry of w and dw of row r (0 without a map), -1 for rows to skip
  auto entry = [&](uint32_t r) -> int32_t {
    if (r >= R) return -1;
    if (a.src == nullptr) return 0;
    const int32_t at = __ldg(a.src + r);
    if (weights && at >= a.n) {
      set_status(a.status, MG_ERR_DEVICE_ARG);
      return -1;
    }
    return at;
  };
  // ---- the cursor that runs ahead: its row, the entry of that and of the next
  int32_t cf = first, cs = 0, cat;
  Walk cw{0, blockIdx.x * (uint32_t)rows_per_block + off};
  next_row(cw, step, R, lane, entry, cat);
  int32_t cat1 = entry(cw.next(step).row());
  const uint8_t* chc = a.HC + (int64_t)cw.row() * a.N + col;
  const __nv_bfloat16* cd = static_cast<const __nv_bfloat16*>(a.dY) + (int64_t)cw.row() * I + first;
  const int32_t pieces = (I + span - 1) / span;    // of a row; a thread's last may lie past it
  int32_t cp = pieces;
  auto ahead = [&]() {
    sl.row[cs][tid] = make_int2((int32_t)cw.row(), cat);
    if (cat >= 0) {
      if (cf < I) {
        cp_async<8>(&sl.g[cs][tid], chc);
        cp_async<8>(&sl.u[cs][tid], chc + 128);
        cp_async<16>(&sl.d[cs][tid], cd);
        if (a.w != nullptr) cp_async<4>(&sl.w[cs][tid], a.w + cat);
      }
      cf += span;
      chc += 2 * span;
      cd += span;
      if (--cp == 0) {
        cp = pieces;
        cf = first;
        cw = cw.next(step);
        cat = cat1;
        if (cat < 0) next_row(cw, step, R, lane, entry, cat);   // past rows without a choice
        cat1 = entry(cw.next(step).row());
        chc = a.HC + (int64_t)cw.row() * a.N + col;
        cd = static_cast<const __nv_bfloat16*>(a.dY) + (int64_t)cw.row() * I + first;
      }
    }
    cp_async_commit();
    cs = (cs + 1) & (kBwdStages - 1);
  };
#pragma unroll
  for (int i = 0; i < kBwdStages - 1; ++i) ahead();

  const uint16_t* scales = reinterpret_cast<const uint16_t*>(a.SHC) + (first >> 7);   // (gate, up) pairs
  const uint64_t one = pack2(1.0f, 1.0f), minus = pack2(-1.0f, -1.0f);
  int32_t st = 0, buf = 0;
  int2 row = sl.row[0][tid];
  uint32_t sc = row.y >= 0 && first < I ? __ldg(scales + (int64_t)row.x * (a.N >> 8)) : 0u;
  while (row.y >= 0) {
    const int32_t at = row.y;
    uint64_t dot = 0;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.dH) + (int64_t)row.x * a.N + col;
    __nv_bfloat16* yo = static_cast<__nv_bfloat16*>(a.Y) + (int64_t)row.x * I + first;
    const uint16_t* srow = scales + (int64_t)row.x * (a.N >> 8);
    for (int32_t f = first, p = pieces; p > 0; --p, f += span) {
      cp_async_wait<kBwdStages - 2>();
      const int32_t nst = (st + 1) & (kBwdStages - 1);
      srow += span >> 7;
      uint32_t sc1 = 0;
      if (p > 1) {
        if (f + span < I) sc1 = __ldg(srow);
      } else {
        row = sl.row[nst][tid];
        if (row.y >= 0 && first < I) sc1 = __ldg(scales + (int64_t)row.x * (a.N >> 8));
      }
      if (f < I) {
        const float w = a.w != nullptr ? sl.w[st][tid] : 1.0f;
        const uint64_t w2 = pack2(w, w);
        uint64_t g[4], u[4], d[4], dg[4], du[4], y[4];
        const float2 scale = ue8m0x2_value(sc);
        e4m3x8_decode(sl.g[st][tid], scale.x, g);
        e4m3x8_decode(sl.u[st][tid], scale.y, u);
        bf16x8_to_f32x2(sl.d[st][tid], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t s = fast_sigmoid2(g[i]);
          const uint64_t silu = mul2(g[i], s), yy = mul2(silu, u[i]);
          dot = fma2(d[i], yy, dot);
          const uint64_t wd = mul2(w2, d[i]);
          // sigma (1 + g (1 - sigma))
          const uint64_t slope = mul2(s, fma2(g[i], fma2(s, minus, one), one));
          dg[i] = mul2(mul2(wd, u[i]), slope);
          du[i] = mul2(wd, silu);
          y[i] = mul2(w2, yy);
        }
        __stcs(reinterpret_cast<uint4*>(o), f32x2_to_bf16x8(dg));
        __stcs(reinterpret_cast<uint4*>(o + 128), f32x2_to_bf16x8(du));
        if (a.Y != nullptr) __stcs(reinterpret_cast<uint4*>(yo), f32x2_to_bf16x8(y));
      }
      ahead();
      o += 2 * span;
      yo += span;
      st = nst;
      sc = sc1;
    }
    if (a.dw != nullptr) {
      const float2 q = unpack2(dot);
      float sum = q.x + q.y;
#pragma unroll
      for (int i = 16; i >= 1; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
      if (tpr == 32) {
        if (lane == 0) a.dw[at] = sum;
      } else {
        if (lane == 0) part[buf][warp] = sum;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + off), "r"(tpr) : "memory");
        if (first == 0) {
          float s = 0.0f;
          for (int i = 0; i < tpr / 32; ++i) s += part[buf][warp + i];
          a.dw[at] = s;
        }
        buf ^= 1;
      }
    }
  }
  cp_async_wait<0>();
}

}  // namespace rows

namespace {
int sms() { return num_sms_current_device(); }

// Columns of a token per dispatch block: whole tokens when there are enough
// of them for two blocks an SM, else pieces of at least 512 columns.
int32_t dispatch_span(int32_t T, int32_t K) {
  const int64_t want = 2 * (int64_t)sms();
  int64_t pieces = (want + T - 1) / T;
  const int64_t most = (K + 511) / 512, least = (K + rows::kMaxSpan - 1) / rows::kMaxSpan;
  pieces = pieces > most ? most : pieces;
  pieces = pieces < least ? least : pieces;
  return (int32_t)(((K + pieces - 1) / pieces + 127) / 128 * 128);
}

// Blocks of 256 threads, or of one per sixteen columns where there are more
// than four blocks an SM and thus threads to spare: 16384 tokens of 1024 to
// four E4M3 rows each 28 us instead of 40, 1000 of 640 7.0 instead of 7.8; with
// few blocks more warps hide more of a block's latency, 300 of 1024 6.7 us
// against 7.3.
int32_t dispatch_threads(int64_t blocks, int32_t span) {
  const int32_t n = (span / 16 + 31) / 32 * 32;
  return blocks > 4 * (int64_t)sms() && n < rows::kThreads ? n : rows::kThreads;
}

// Threads of a block that walks rows of K columns, eight to a thread and pass.
// Up to two passes: whole warps, every thread in as many passes as the others
// (the gradients of 65536 combined rows of 256 15 us instead of 70 with 256
// threads, of 2176 101 instead of 110).  Further passes: 256, the last pass short
// (32768 rows of 5120 130 us, with three equal passes 134).
int32_t row_threads(int32_t K) {
  const int32_t passes = (K + rows::kPass - 1) / rows::kPass, n = (K / 8 + passes - 1) / passes;
  return passes > 2 ? rows::kThreads : (n + 31) / 32 * 32;
}

template <bool kSrcQ, bool kDstQ, bool kCkpt>
cudaError_t dispatch_as(const DispatchArgs& a, cudaStream_t s) {
  const int32_t span = dispatch_span(a.T, a.K);
  // set up while the slot map is still being written, where that is what runs
  // before it (a kernel that does not allow it is waited for as ever)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)a.T, (unsigned)((a.K + span - 1) / span));
  cfg.blockDim = dim3((unsigned)dispatch_threads((int64_t)cfg.gridDim.x * cfg.gridDim.y, span));
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows::dispatch_kernel<kSrcQ, kDstQ, kCkpt>, a, span);
}
}  // namespace

cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t s) {
  if (a.src_e4m3) return a.dst_e4m3 ? dispatch_as<true, true, false>(a, s) : dispatch_as<true, false, false>(a, s);
  if (a.CX != nullptr) return a.dst_e4m3 ? dispatch_as<false, true, true>(a, s) : dispatch_as<false, false, true>(a, s);
  return a.dst_e4m3 ? dispatch_as<false, true, false>(a, s) : dispatch_as<false, false, false>(a, s);
}

template <int kN, int kTok>
cudaError_t combine_as(const CombineArgs& a, cudaStream_t s) {
  const int32_t threads = row_threads(a.K);
  const dim3 grid((unsigned)((a.T + kTok - 1) / kTok), (unsigned)((a.K / 8 + threads - 1) / threads));
  if (a.f32)
    rows::combine_kernel<true, kN, kTok><<<grid, threads, 0, s>>>(a);
  else
    rows::combine_kernel<false, kN, kTok><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int kN, int kTok>
cudaError_t combine_bwd_as(const CombineBwdArgs& a, cudaStream_t s) {
  const int32_t threads = row_threads(a.K);
  const unsigned grid = (unsigned)((a.T + kTok - 1) / kTok);
  if (a.f32)
    rows::combine_bwd_kernel<true, kN, kTok><<<grid, threads, 0, s>>>(a);
  else
    rows::combine_bwd_kernel<false, kN, kTok><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

// Rows that a thread of combine loads together: four, of one token, or, where
// tokens have one or two, of four or two tokens (16384 tokens of two rows of 2048
// 34 us, a token to a block 42; of one row of 256 4.1 and 10.2).  Eight rows
// of one token are no faster (32768 rows of 7168 83 us either way).
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) {
  if (a.k == 1) return combine_as<1, 4>(a, s);
  if (a.k == 2) return combine_as<2, 2>(a, s);
  return combine_as<4, 1>(a, s);
}

// The backward pass the same, but with few tokens a block to each (61 tokens
// of two rows of 7168 4.3 us, two tokens to a block 5.4); two tokens of one row
// together, whose dout takes registers too (8000 tokens of one row of 5120 47 us,
// four together 59); and with eight rows together where tokens have more than
// four, so that dout is read once (40960 rows of 5120 149 us, as four and one
// 155).
cudaError_t launch_combine_bwd(const CombineBwdArgs& a, cudaStream_t s) {
  const bool many = a.T > 2 * sms();
  if (many && a.k == 1) return combine_bwd_as<1, 2>(a, s);
  if (many && a.k == 2) return combine_bwd_as<2, 2>(a, s);
  if (a.k <= 4) return combine_bwd_as<4, 1>(a, s);
  return combine_bwd_as<8, 1>(a, s);
}

namespace {
// Blocks of a row kernel of `threads` threads, tpr to a row: all that fit the
// GPU at once, or as many as there are rows for.
template <typename K>
unsigned row_grid(K* kernel, std::atomic<int>& cached, int threads, int64_t rows_total, int tpr) {
  int per = cached.load();
  if (per == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess || per < 1) {
      (void)cudaGetLastError();
      per = 1;
    }
    cached.store(per);
  }
  const int64_t each = threads / tpr, need = (rows_total + each - 1) / each, most = (int64_t)sms() * per;
  return (unsigned)(need < most ? need : most);
}
}  // namespace

cudaError_t launch_swiglu_save(const SwigluSaveArgs& a, cudaStream_t s) {
  using namespace rows;
  // whole warps to a row, every thread in as many passes over it as the others
  // (36000 rows of N = 2816 on 192 threads each 71.6 us, on 256 77.6)
  const int32_t I = a.N >> 1, passes = (I + kPass - 1) / kPass, n = (I / 8 + passes - 1) / passes;
  const int tpr = (n + 31) / 32 * 32, threads = kThreads / tpr * tpr;
  static std::atomic<int> per_sm[2][kWarps + 1];
  if (a.y_e4m3) {
    const unsigned grid = row_grid(swiglu_save_kernel<true>, per_sm[1][threads / 32], threads, a.rows_total, tpr);
    swiglu_save_kernel<true><<<grid, threads, 0, s>>>(a, tpr);
  } else {
    const unsigned grid = row_grid(swiglu_save_kernel<false>, per_sm[0][threads / 32], threads, a.rows_total, tpr);
    swiglu_save_kernel<false><<<grid, threads, 0, s>>>(a, tpr);
  }
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s) {
  using namespace rows;
  // A power of two of threads per row, at most 256.  With many rows, the most
  // that leave a thread four pieces of a row: fewer reductions, barriers and
  // idle threads a row than with more threads, a row's bytes closer together
  // than with fewer.  131072 rows of N = 1536 175 us on 32 threads each, 208 on
  // 64; 65536 of 4096 228 on 32, 219 on 64, 243 on 128; 18720 of 14336 229 on 64,
  // 216 on 128.  Few rows are spread over more threads each, until the GPU has
  // 12 to 24 warps an SM: 518 rows of 4096 6.2 us on 256 threads each, 7.9 on 32;
  // 2400 of 1536 6.0 on 32, 7.3 on 128.
  const int32_t I = a.N >> 1;
  int least = 32, tpr = 32;
  while (least < kThreads && least * 64 <= I) least <<= 1;
  while (tpr < kThreads && tpr * 8 < I) tpr <<= 1;
  // rows that hold a choice: of no more than the weights' choices, where given
  const int64_t live = (a.w != nullptr || a.dw != nullptr) && a.n < a.rows_total ? a.n : a.rows_total;
  while (tpr > least && live * (tpr / 64) >= (int64_t)sms() * 12) tpr >>= 1;
  static std::atomic<int> per_sm;
  swiglu_bwd_kernel<<<row_grid(swiglu_bwd_kernel, per_sm, kThreads, a.rows_total, tpr), kThreads, 0, s>>>(a, tpr);
  return cudaGetLastError();
}

}  // namespace mg
