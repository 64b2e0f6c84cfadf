// Token rows on their way into and out of the grouped GEMMs: dispatch into the
// contiguous or masked layout (as bf16, or E4M3 with UE8M0 scales), combine
// and its gradients, and SwiGLU with its rows kept in 8 bits for the backward
// pass.  All of these are bound by memory traffic: each reads its inputs once
// and writes its outputs once, in 16-byte (8-byte for codes) pieces, eight
// columns to a thread, and computes in fp32.
#include "blockq.cuh"
#include "common.cuh"
#include "ops_internal.h"

namespace mg {
namespace rows {

constexpr int kThreads = 256;
constexpr int kSpan = kThreads * 8;        // columns of one pass of a block

// Rows of token t's k choices into shared memory; -1 where there is none.
__device__ __forceinline__ void load_rows(const int32_t* rows, int64_t t, int32_t k, int64_t rows_total,
                                          int32_t* sh, int32_t* status) {
  if ((int)threadIdx.x < k) {
    int32_t r = __ldg(rows + t * k + threadIdx.x);
    if (r >= rows_total) {
      set_status(status, MG_ERR_DEVICE_ARG);
      r = -1;
    }
    sh[threadIdx.x] = r;
  }
  __syncthreads();
}

// Block (t, y): columns [y * kSpan, (y + 1) * kSpan) of token t, read once and
// written to each of its k rows.
template <bool kSrcQ, bool kDstQ>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs a) {
  __shared__ int32_t sh[kMaxTopK];
  const int64_t t = blockIdx.x;
  load_rows(a.rows, t, a.k, a.rows_total, sh, a.status);
  const int32_t c = (int32_t)(blockIdx.y * kSpan + threadIdx.x * 8);
  const int32_t kb = c >> 7, KB = a.K >> 7;
  const bool in = c < a.K;
  float x[8] = {};
  uint2 q = make_uint2(0, 0);
  uint4 h = make_uint4(0, 0, 0, 0);
  int32_t sc = 127;
  if (in) {
    if (kSrcQ) {
      q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.X) + t * a.ldx + c);
      sc = __ldg(a.SX + t * KB + kb);
    } else {
      h = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.X) + t * a.ldx + c);
    }
  }
  if (!kSrcQ && (kDstQ || a.CX != nullptr)) {
    bf16x8_to_f32(h, x);
    sc = ue8m0_of_amax(block_amax(x));
    q = e4m3x8_encode(x, ue8m0_inverse(sc));
    if (in && a.CX != nullptr) {
      *reinterpret_cast<uint2*>(a.CX + t * a.K + c) = q;
      if ((c & 127) == 0) a.SCX[t * KB + kb] = (uint8_t)sc;
    }
  }
  if (kSrcQ && !kDstQ) {
    e4m3x8_decode(q, ue8m0_value((uint32_t)sc), x);
    h = f32_to_bf16x8(x);
  }
  if (!in) return;
  for (int j = 0; j < a.k; ++j) {
    const int64_t r = sh[j];
    if (r < 0) continue;
    if (kDstQ) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.A) + r * a.K + c) = q;
      if ((c & 127) == 0) {
        const int64_t z = r / a.group_rows;
        a.SFA[(z * KB + kb) * a.group_rows + (r - z * a.group_rows)] = (uint8_t)sc;
      }
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.A) + r * a.K + c) = h;
    }
  }
}

template <bool kF32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if (kF32) {
    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  } else {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at), x);
  }
}

// Block (t, y): out[t] = sum_j w_tj D[row(t, j)] over a span of columns, in
// the order of the choices, in fp32, rounded once.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
  __shared__ int32_t sh[kMaxTopK];
  __shared__ float sw[kMaxTopK];
  const int64_t t = blockIdx.x;
  if ((int)threadIdx.x < a.k) sw[threadIdx.x] = a.w != nullptr ? __ldg(a.w + t * a.k + threadIdx.x) : 1.0f;
  load_rows(a.rows, t, a.k, a.rows_total, sh, a.status);
  const int32_t c = (int32_t)(blockIdx.y * kSpan + threadIdx.x * 8);
  if (c >= a.K) return;
  const __nv_bfloat16* D = static_cast<const __nv_bfloat16*>(a.D);
  float acc[8] = {};
  for (int j = 0; j < a.k; ++j) {
    const int64_t r = sh[j];
    if (r < 0) continue;
    float x[8];
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(D + r * a.K + c), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(sw[j], x[i], acc[i]);
  }
  if (kF32) {
    float* o = static_cast<float*>(a.out) + t * a.ldo + c;
    *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + t * a.ldo + c) = f32_to_bf16x8(acc);
  }
}

// Sum over the block, the same for every run (fixed order); thread 0 has it.
__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x == 0)
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += sh[i];
  return s;
}

// Block t: dD[row] = w dout[t] and dw = <dout[t], D[row]> for the token's rows.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const CombineBwdArgs a) {
  __shared__ int32_t sh[kMaxTopK];
  __shared__ float part[kThreads / 32];
  const int64_t t = blockIdx.x;
  load_rows(a.rows, t, a.k, a.rows_total, sh, a.status);
  const __nv_bfloat16* D = static_cast<const __nv_bfloat16*>(a.D);
  __nv_bfloat16* dD = static_cast<__nv_bfloat16*>(a.dD);
  for (int j = 0; j < a.k; ++j) {
    const int64_t r = sh[j];
    float dot = 0.0f;
    if (r >= 0) {
      const float w = a.w != nullptr ? __ldg(a.w + t * a.k + j) : 1.0f;
      for (int32_t c = threadIdx.x * 8; c < a.K; c += kSpan) {
        float g[8], x[8];
        load8<kF32>(a.dout, t * a.ldd + c, g);
        if (a.D != nullptr) {
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(D + r * a.K + c), x);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(g[i], x[i], dot);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= w;
        *reinterpret_cast<uint4*>(dD + r * a.K + c) = f32_to_bf16x8(g);
      }
    }
    if (a.dw != nullptr) {
      dot = block_sum(dot, part);
      if (threadIdx.x == 0) a.dw[t * a.k + j] = dot;
    }
  }
}

// g / (1 + e^-g) and 1 / (1 + e^-g) with the fast exponential and division,
// as the SwiGLU epilogue of the GEMMs computes them.
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
__device__ __forceinline__ float fast_silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

// 16 lanes per (row, feature block j): gate columns 256j .. 256j+127 and up
// columns 256j+128 .. 256j+255 of H, eight of each to a lane.
template <bool kYQ>
__global__ void __launch_bounds__(kThreads) swiglu_save_kernel(const SwigluSaveArgs a) {
  const int32_t blocks = a.N >> 8, I = a.N >> 1;
  const int64_t items = a.rows_total * blocks;
  const int lane16 = threadIdx.x & 15;
  const __nv_bfloat16* H = static_cast<const __nv_bfloat16*>(a.H);
  const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
  // the two halves of a warp stay together: both shuffle, each for itself
  for (int64_t w = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 5) * 2; w < items; w += step) {
    const int64_t it = w + ((threadIdx.x >> 4) & 1);
    const int64_t r = it / blocks;
    const int32_t j = (int32_t)(it - r * blocks);
    const bool in = it < items && (a.src == nullptr || __ldg(a.src + r) >= 0);
    float g[8] = {}, u[8] = {}, y[8];
    if (in) {
      const __nv_bfloat16* h = H + r * a.N + j * 256 + lane16 * 8;
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(h), g);
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(h + 128), u);
    }
    const int32_t sg = ue8m0_of_amax(block_amax(g)), su = ue8m0_of_amax(block_amax(u));
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fast_silu(g[i]) * u[i];
    const int32_t sy = kYQ ? ue8m0_of_amax(block_amax(y)) : 127;
    if (!in) continue;
    uint8_t* hc = a.HC + r * a.N + j * 256 + lane16 * 8;
    *reinterpret_cast<uint2*>(hc) = e4m3x8_encode(g, ue8m0_inverse(sg));
    *reinterpret_cast<uint2*>(hc + 128) = e4m3x8_encode(u, ue8m0_inverse(su));
    if (lane16 == 0) {
      a.SHC[r * 2 * blocks + 2 * j] = (uint8_t)sg;
      a.SHC[r * 2 * blocks + 2 * j + 1] = (uint8_t)su;
    }
    const int64_t at = r * I + j * 128 + lane16 * 8;
    if (kYQ) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + at) = e4m3x8_encode(y, ue8m0_inverse(sy));
      if (lane16 == 0) {
        const int64_t z = r / a.group_rows;
        a.SFY[(z * blocks + j) * a.group_rows + (r - z * a.group_rows)] = (uint8_t)sy;
      }
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) + at) = f32_to_bf16x8(y);
    }
  }
}

// One block per row (rows in a grid stride).
__global__ void __launch_bounds__(kThreads) swiglu_bwd_kernel(const SwigluBwdArgs a) {
  __shared__ float part[kThreads / 32];
  const int32_t blocks = a.N >> 8, I = a.N >> 1;
  const __nv_bfloat16* dY = static_cast<const __nv_bfloat16*>(a.dY);
  for (int64_t r = blockIdx.x; r < a.rows_total; r += gridDim.x) {
    int64_t at = -1;
    if (a.src != nullptr) {
      at = __ldg(a.src + r);
      if (at < 0) continue;
      if ((a.w != nullptr || a.dw != nullptr) && at >= a.n) {
        if (threadIdx.x == 0) set_status(a.status, MG_ERR_DEVICE_ARG);
        continue;
      }
    }
    const float w = a.w != nullptr ? __ldg(a.w + at) : 1.0f;
    float dot = 0.0f;
    for (int32_t f = threadIdx.x * 8; f < I; f += blockDim.x * 8) {
      const int32_t j = f >> 7, c = j * 256 + (f & 127);
      float g[8], u[8], d[8], dg[8], y[8];
      e4m3x8_decode(*reinterpret_cast<const uint2*>(a.HC + r * a.N + c),
                    ue8m0_value(__ldg(a.SHC + r * 2 * blocks + 2 * j)), g);
      e4m3x8_decode(*reinterpret_cast<const uint2*>(a.HC + r * a.N + c + 128),
                    ue8m0_value(__ldg(a.SHC + r * 2 * blocks + 2 * j + 1)), u);
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(dY + r * I + f), d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = fast_sigmoid(g[i]), silu = g[i] * s;
        const float v = silu * u[i];
        dot = fmaf(d[i], v, dot);
        const float wd = w * d[i];
        dg[i] = wd * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
        d[i] = wd * silu;
        y[i] = w * v;
      }
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.dH) + r * a.N + c;
      *reinterpret_cast<uint4*>(o) = f32_to_bf16x8(dg);
      *reinterpret_cast<uint4*>(o + 128) = f32_to_bf16x8(d);
      if (a.Y != nullptr)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) + r * I + f) = f32_to_bf16x8(y);
    }
    if (a.dw != nullptr) {
      dot = block_sum(dot, part);
      if (threadIdx.x == 0) a.dw[at] = dot;
    }
  }
}

}  // namespace rows

cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t s) {
  using namespace rows;
  const dim3 grid((unsigned)a.T, (unsigned)((a.K + kSpan - 1) / kSpan));
  if (a.src_e4m3 && a.dst_e4m3)
    dispatch_kernel<true, true><<<grid, kThreads, 0, s>>>(a);
  else if (a.src_e4m3)
    dispatch_kernel<true, false><<<grid, kThreads, 0, s>>>(a);
  else if (a.dst_e4m3)
    dispatch_kernel<false, true><<<grid, kThreads, 0, s>>>(a);
  else
    dispatch_kernel<false, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) {
  using namespace rows;
  const dim3 grid((unsigned)a.T, (unsigned)((a.K + kSpan - 1) / kSpan));
  if (a.f32)
    combine_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    combine_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_combine_bwd(const CombineBwdArgs& a, cudaStream_t s) {
  using namespace rows;
  if (a.f32)
    combine_bwd_kernel<true><<<(unsigned)a.T, kThreads, 0, s>>>(a);
  else
    combine_bwd_kernel<false><<<(unsigned)a.T, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_save(const SwigluSaveArgs& a, cudaStream_t s) {
  using namespace rows;
  const int64_t need = (a.rows_total * (a.N >> 8) + kThreads / 16 - 1) / (kThreads / 16);
  const int64_t most = (int64_t)num_sms_current_device() * 8;
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (a.y_e4m3)
    swiglu_save_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    swiglu_save_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s) {
  using namespace rows;
  const int64_t most = (int64_t)num_sms_current_device() * 8;
  swiglu_bwd_kernel<<<(unsigned)(a.rows_total < most ? a.rows_total : most), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mg
