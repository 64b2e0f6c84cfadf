// Routing of tokens to experts and its gradient, and the slot map that turns
// the chosen experts into rows of the grouped GEMMs' layouts.
#include <cfloat>

#include "common.cuh"
#include "ops_internal.h"
#include "sched.cuh"

namespace mg {
namespace route {

constexpr int kWarps = 8;
constexpr uint32_t kAll = 0xffffffffu;

// Order-preserving image of a float in the unsigned integers.  0 is left for
// "never chosen": the smallest image of a number above -inf is 0x00800000.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// One token's logits, expert lane * V + v in x[v]; -inf where there is none.
// NaN counts as -inf and is reported; +inf as the largest finite value.
template <int V, typename L>
__device__ __forceinline__ void load_row(const L* row, int32_t E, int lane, float (&x)[V], int32_t* status) {
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int32_t e = lane * V + v;
    float f = e < E ? load_logit(row + e) : -INFINITY;
    if (f != f) {
      nan = true;
      f = -INFINITY;
    }
    x[v] = fminf(f, FLT_MAX);
  }
  if (nan) set_status(status, MG_ERR_DEVICE_ARG);
}

// Softmax over a token's logits (experts at -inf score 0; a row of nothing
// else scores 0 everywhere), with the running pieces the backward pass needs.
template <int V>
__device__ __forceinline__ void softmax_row(const float (&x)[V], float (&s)[V], float& top, float& sum) {
  top = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = fmaxf(top, x[v]);
  top = warp_max(top);
  const float m = top == -INFINITY ? 0.0f : top;
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = expf(x[v] - m);
    sum += s[v];
  }
  sum = fmaxf(warp_sum(sum), FLT_MIN);
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = s[v] / sum;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// One warp per token.  Lane l holds experts l*V .. l*V+V-1, so the lowest
// lane that holds the largest key, and its lowest position, is the lowest
// expert index among equal keys.
template <int V, typename L>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  __shared__ float group_keys[kWarps][V * 32 + 4 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L* logits = static_cast<const L*>(a.logits);
  const int32_t gs = a.E / a.groups;
  int lpg = 32;                                  // lanes per group in the group step
  while (lpg * a.groups > 32) lpg >>= 1;
  int32_t group_of[V];
#pragma unroll
  for (int v = 0; v < V; ++v) group_of[v] = min((lane * V + v) / gs, 31);
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
    float x[V], s[V];
    load_row<V, L>(logits + t * a.ld, a.E, lane, x, a.status);
    if (a.softmax) {
      float top, sum;
      softmax_row<V>(x, s, top, sum);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = sigmoid(x[v]);
    }
    float key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int32_t e = lane * V + v;
      float b = s[v];
      if (a.bias != nullptr && e < a.E) b += __ldg(a.bias + e);
      key[v] = (x[v] == -INFINITY || b != b) ? -INFINITY : b + 0.0f;   // + 0: -0 and 0 are equal keys
    }
    uint32_t kept = kAll;
    if (a.groups > 1) {
      float* gk = group_keys[warp];
      __syncwarp();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int32_t e = lane * V + v;
        gk[e + 4 * (e >> 5)] = key[v];
      }
      __syncwarp();
      const int g = lane / lpg, sub = lane - g * lpg;
      float m1 = -INFINITY, m2 = -INFINITY;
      if (g < a.groups) {
        for (int32_t i = sub; i < gs; i += lpg) {
          const int32_t e = g * gs + i;
          const float f = gk[e + 4 * (e >> 5)];
          m2 = fmaxf(m2, fminf(m1, f));
          m1 = fmaxf(m1, f);
        }
      }
      for (int o = lpg >> 1; o >= 1; o >>= 1) {
        const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
        m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
        m1 = fmaxf(m1, o1);
      }
      const float sc = (a.group_top == 2 && m2 != -INFINITY) ? m1 + m2 : m1;
      int rank = 0;
      for (int h = 0; h < a.groups; ++h) {
        const float o = __shfl_sync(kAll, sc, h * lpg);
        rank += (o > sc) || (o == sc && h < g);
      }
      const uint32_t in = __ballot_sync(kAll, g < a.groups && rank < a.top_groups);
      kept = 0;
      for (int h = 0; h < a.groups; ++h) kept |= ((in >> (h * lpg)) & 1u) << h;
    }
    uint32_t o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // (positions past E hold -inf)
      o[v] = ((kept >> group_of[v]) & 1u) && key[v] != -INFINITY ? ordered(key[v]) : 0u;
    }
    int32_t my_idx = -1;
    float my_s = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      uint32_t m = o[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = max(m, o[v]);
      const uint32_t M = __reduce_max_sync(kAll, m);
      if (M == 0) break;
      const int win = __ffs(__ballot_sync(kAll, m == M)) - 1;
      int at = 0;
      float sv = 0.0f;
      if (lane == win) {
        bool open = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (open && o[v] == M) {
            open = false;
            at = v;
            sv = s[v];
            o[v] = 0;
          }
        }
      }
      at = __shfl_sync(kAll, at, win);
      sv = __shfl_sync(kAll, sv, win);
      if (lane == j) {
        my_idx = win * V + at;
        my_s = sv;
      }
    }
    if (a.renorm) my_s /= fmaxf(warp_sum(my_s), FLT_MIN);
    if (lane < a.k) {
      a.idx[t * a.k + lane] = my_idx;
      a.w[t * a.k + lane] = my_s * a.scale;
    }
  }
}

// One warp per token.  Softmax weights without renormalisation reach every
// logit of the token; otherwise only the chosen ones have a gradient (a
// renormalised softmax is the softmax over the chosen logits), so only those
// are read and the rest of the row is written as zeros.
template <int V, typename L>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const RouteBwdArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L* logits = static_cast<const L*>(a.logits);
  L* dlogits = static_cast<L*>(a.dlogits);
  const bool full = a.softmax && !a.renorm;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
    int32_t i = -1;
    float up = 0.0f, xs = -INFINITY;
    if (lane < a.k) {
      i = a.idx[t * a.k + lane];
      if (i < -1 || i >= a.E) {
        set_status(a.status, MG_ERR_DEVICE_ARG);
        i = -1;
      }
      if (i >= 0) {
        up = a.scale * a.dw[t * a.k + lane];
        xs = load_logit(logits + t * a.ld + i);
        if (xs != xs) xs = -INFINITY;
        xs = fminf(xs, FLT_MAX);
      }
    }
    float s[V];
    float d;        // gradient at this lane's choice (all but `full`: of the logit itself)
    float dot = 0.0f;
    if (full) {
      float x[V], top, sum;
      load_row<V, L>(logits + t * a.ld, a.E, lane, x, a.status);
      softmax_row<V>(x, s, top, sum);
      const float ss = expf(xs - (top == -INFINITY ? 0.0f : top)) / sum;
      dot = warp_sum(up * ss);
      d = up;
    } else if (a.softmax) {
      const float top = warp_max(xs);
      const float e = expf(xs - (top == -INFINITY ? 0.0f : top));
      const float p = e / fmaxf(warp_sum(e), FLT_MIN);
      d = p * (up - warp_sum(p * up));
    } else {
      const float ss = sigmoid(xs), one = sigmoid(-xs);
      float p = ss;
      float g = up;
      if (a.renorm) {
        p = ss / fmaxf(warp_sum(ss), FLT_MIN);
        g = up - warp_sum(p * up);
      }
      d = p * g * one;
      if (i < 0) d = 0.0f;
    }
    float add[V];
#pragma unroll
    for (int v = 0; v < V; ++v) add[v] = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int32_t ij = __shfl_sync(kAll, i, j);
      const float dj = __shfl_sync(kAll, d, j);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane * V + v == ij) add[v] += dj;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int32_t e = lane * V + v;
      if (e < a.E) store_logit(dlogits + t * a.ldd + e, full ? s[v] * (add[v] - dot) : add[v]);
    }
  }
}

template <int V>
cudaError_t launch_route_v(const RouteArgs& a, int blocks, cudaStream_t s) {
  if (a.f32)
    route_kernel<V, float><<<blocks, kWarps * 32, 0, s>>>(a);
  else
    route_kernel<V, __nv_bfloat16><<<blocks, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}
template <int V>
cudaError_t launch_bwd_v(const RouteBwdArgs& a, int blocks, cudaStream_t s) {
  if (a.f32)
    route_bwd_kernel<V, float><<<blocks, kWarps * 32, 0, s>>>(a);
  else
    route_bwd_kernel<V, __nv_bfloat16><<<blocks, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}
int route_blocks(int64_t T) {
  const int64_t need = (T + kWarps - 1) / kWarps, most = (int64_t)num_sms_current_device() * 8;
  return (int)(need < most ? need : most);
}

}  // namespace route

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  using namespace route;
  const int b = route_blocks(a.T);
  if (a.E <= 32) return launch_route_v<1>(a, b, s);
  if (a.E <= 64) return launch_route_v<2>(a, b, s);
  if (a.E <= 128) return launch_route_v<4>(a, b, s);
  if (a.E <= 256) return launch_route_v<8>(a, b, s);
  if (a.E <= 512) return launch_route_v<16>(a, b, s);
  return launch_route_v<32>(a, b, s);
}

cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t s) {
  using namespace route;
  const int b = route_blocks(a.T);
  if (a.E <= 32) return launch_bwd_v<1>(a, b, s);
  if (a.E <= 64) return launch_bwd_v<2>(a, b, s);
  if (a.E <= 128) return launch_bwd_v<4>(a, b, s);
  if (a.E <= 256) return launch_bwd_v<8>(a, b, s);
  if (a.E <= 512) return launch_bwd_v<16>(a, b, s);
  return launch_bwd_v<32>(a, b, s);
}

// ------------------------------------------------------------------ slot map
namespace slots {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kSlotChunk / kThreads;      // choices a thread holds
constexpr uint32_t kAll = 0xffffffffu;
static_assert(kSlotChunk % kThreads == 0 && kSlotChunk <= 65535, "a chunk's ranks fit 16 bits");

__device__ __forceinline__ int32_t checked_expert(const SlotArgs& a, int64_t i, int64_t n) {
  if (i >= n) return -1;
  const int32_t e = __ldg(a.idx + i);
  if (e < -1 || e >= a.E) {
    set_status(a.status, MG_ERR_DEVICE_ARG);
    return -1;
  }
  return e;
}

// Choices per expert of one chunk (integer additions: any order gives the
// same counts).
__global__ void __launch_bounds__(kThreads) count_kernel(const SlotArgs a) {
  extern __shared__ int32_t hist[];
  for (int32_t e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * kSlotChunk;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t at = c0 + i * kThreads + threadIdx.x;
    const int32_t e = at < a.n ? __ldg(a.idx + at) : -1;
    if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int32_t e = threadIdx.x; e < a.E; e += kThreads) a.work[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// Rank of every choice among its expert's choices, in flat order, and the row
// it gets.  A warp owns 32 * kPer consecutive choices; equal experts inside a
// group of 32 find each other with a match, so ranks come out in order
// without atomics.  Every block sums the chunk histograms itself (of the
// chunks before it, and of all), and lays the experts out from the totals.
__global__ void __launch_bounds__(kThreads) place_kernel(const SlotArgs a) {
  extern __shared__ int32_t sh[];
  int32_t* total = sh;               // choices of expert e
  int32_t* before = total + a.E;     // of them, in earlier chunks
  int32_t* base = before + a.E;      // first row, -1 when the expert is dropped
  uint16_t* wh = reinterpret_cast<uint16_t*>(base + a.E);   // [kWarps][E]
  __shared__ int64_t scan[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t E = a.E;
  for (int32_t e = threadIdx.x; e < E; e += kThreads) total[e] = before[e] = 0;
  for (int32_t i = threadIdx.x; i < kWarps * E; i += kThreads) wh[i] = 0;
  __syncthreads();

  const int64_t c0 = (int64_t)blockIdx.x * kSlotChunk + (int64_t)warp * 32 * kPer;
  int32_t ex[kPer];
  uint32_t same[kPer];
  uint16_t* mine = wh + warp * E;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    ex[i] = checked_expert(a, c0 + i * 32 + lane, a.n);
    same[i] = __match_any_sync(kAll, ex[i]);
    if (ex[i] >= 0 && lane == __ffs(same[i]) - 1) mine[ex[i]] += (uint16_t)__popc(same[i]);
    __syncwarp();
  }
  if (gridDim.x > 1) {
    for (int64_t i = threadIdx.x; i < (int64_t)gridDim.x * E; i += kThreads) {
      const int32_t b = (int32_t)(i / E), e = (int32_t)(i - (int64_t)b * E);
      const int32_t c = __ldg(a.work + i);
      atomicAdd(&total[e], c);
      if (b < (int32_t)blockIdx.x) atomicAdd(&before[e], c);
    }
  }
  __syncthreads();
  // exclusive prefix over the warps of this chunk
  for (int32_t e = threadIdx.x; e < E; e += kThreads) {
    int32_t run = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int32_t c = wh[w * E + e];
      wh[w * E + e] = (uint16_t)run;
      run += c;
    }
    if (gridDim.x == 1) total[e] = run;
  }
  __syncthreads();
  // layout: base rows, counts, -1 in the rows that no choice fills
  int64_t carry = 0;
  bool full = false;
  for (int32_t b = 0; b < E; b += kThreads) {
    const int32_t e = b + threadIdx.x;
    const int64_t c = e < E ? total[e] : 0;
    int64_t start, room, padded;
    if (a.masked) {
      start = (int64_t)e * a.M_max;
      room = min(c, (int64_t)a.M_max);
      padded = a.M_max;
      full |= c > a.M_max;
    } else {
      padded = cdiv64(c, a.align_q) * a.align_q;
      int64_t v = padded;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) scan[warp] = v;
      __syncthreads();
      if (warp == 0) {
        int64_t u = scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t q = __shfl_up_sync(kAll, u, o);
          if (lane >= o) u += q;
        }
        scan[lane] = u;
      }
      __syncthreads();
      start = carry + (warp > 0 ? scan[warp - 1] : 0) + v - padded;
      carry += scan[kWarps - 1];
      __syncthreads();
      room = start + c > a.rows_total ? -1 : c;         // as the GEMMs: an expert that does not fit is skipped
      full |= start + padded > a.rows_total;
    }
    if (e < E) {
      base[e] = room < 0 ? -1 : (int32_t)start;
      if (blockIdx.x == 0) a.counts[e] = (int32_t)(a.masked ? room : c);
    }
  }
  if (blockIdx.x == 0 && full) set_status(a.status, MG_ERR_CAPACITY);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t at = c0 + i * 32 + lane;
    const int32_t e = ex[i];
    int32_t row = -1;
    if (e >= 0) {
      const int32_t in = mine[e] + __popc(same[i] & ((1u << lane) - 1u));
      const int32_t r = before[e] + in;
      if (base[e] >= 0 && (!a.masked || r < a.M_max)) row = base[e] + r;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same[i]) - 1) mine[e] += (uint16_t)__popc(same[i]);
    __syncwarp();
    if (at < a.n) {
      a.rows[at] = row;
      if (row >= 0 && a.src != nullptr) a.src[row] = (int32_t)at;
    }
  }
  if (a.src == nullptr) return;
  const int64_t gw = (int64_t)blockIdx.x * kWarps + warp, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t e = gw; e < E; e += nw) {
    int64_t from, to;
    if (a.masked) {
      from = e * a.M_max + min(total[e], a.M_max);
      to = (e + 1) * a.M_max;
    } else {
      if (base[e] < 0) continue;                         // cleared with the tail below
      from = (int64_t)base[e] + total[e];
      to = min((int64_t)base[e] + cdiv64(total[e], a.align_q) * a.align_q, a.rows_total);
    }
    for (int64_t r = from + lane; r < to; r += 32) a.src[r] = -1;
  }
  if (!a.masked) {
    // segments start in expert order, so the rows past the last expert that
    // fits hold nothing (an expert behind a dropped one starts past the end)
    int64_t end = 0;
    for (int32_t e = E - 1; e >= 0; --e) {
      if (base[e] >= 0) {
        end = (int64_t)base[e] + cdiv64(total[e], a.align_q) * a.align_q;
        break;
      }
    }
    for (int64_t r = end + (int64_t)blockIdx.x * kThreads + threadIdx.x; r < a.rows_total;
         r += (int64_t)gridDim.x * kThreads)
      a.src[r] = -1;
  }
}

}  // namespace slots

namespace {
template <typename K>
cudaError_t allow_smem(K* kernel, bool (&done)[64], int bytes) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 64 && done[dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess && dev < 64) done[dev] = true;
  return err;
}
}  // namespace

cudaError_t launch_slots(const SlotArgs& a, cudaStream_t s) {
  using namespace slots;
  static bool done[64] = {};
  constexpr int per_expert = 3 * (int)sizeof(int32_t) + kWarps * (int)sizeof(uint16_t);
  const cudaError_t err = allow_smem(place_kernel, done, per_expert * kMaxExperts);
  if (err != cudaSuccess) return err;
  const int blocks = a.n <= kSlotChunk ? 1 : (int)((a.n + kSlotChunk - 1) / kSlotChunk);
  if (blocks > 1) {
    count_kernel<<<blocks, kThreads, a.E * sizeof(int32_t), s>>>(a);
    const cudaError_t e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return e1;
  }
  place_kernel<<<blocks, kThreads, per_expert * a.E, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mg
