// Routing of tokens to experts and its gradient, and the slot map that turns
// the chosen experts into rows of the grouped GEMMs' layouts.
#include <atomic>
#include <cfloat>
#include <type_traits>

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
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// Two bf16 logits to packed keys: the ordered bits of the logit above, 0xffff -
// expert below.  Adding +0 makes -0 and 0 one key and every NaN the positive
// one, so -inf and its like order below kFirstKey and NaN at kNanKey or above.
constexpr uint32_t kFirstKey = 0x00800000u, kNanKey = 0xff810000u;
__device__ __forceinline__ void packed_keys(uint32_t w, uint32_t e, uint32_t& k0, uint32_t& k1) {
  uint32_t c;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(w), "r"(0u));
  const uint32_t s = c & 0x80008000u, m = s - (s >> 15);     // 0x7fff in negative halves
  const uint32_t p = c ^ (m | 0x80008000u);
  k0 = __byte_perm(0xffffu - e, p, 0x5410);
  k1 = __byte_perm(0xfffeu - e, p, 0x7610);
}

// over the warp, or each kLanes lanes of it
template <int kLanes = 32>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = kLanes / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int kLanes = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// V consecutive values of a lane as words of up to 16 bytes.
template <int V, typename L>
struct Vec {
  static constexpr int kBytes = V * (int)sizeof(L);
  static constexpr int kWord = kBytes % 16 == 0 ? 16 : kBytes % 8 == 0 ? 8 : kBytes % 4 == 0 ? 4 : 2;
  union {
    L v[V];
    uint16_t h[kBytes / 2];
    uint32_t w[kBytes < 4 ? 1 : kBytes / 4];
    uint2 d[kBytes < 8 ? 1 : kBytes / 8];
    uint4 q[kBytes < 16 ? 1 : kBytes / 16];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const L* p) {
#pragma unroll
    for (int i = 0; i < kBytes / kWord; ++i) {
      if constexpr (kWord == 16) q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
      if constexpr (kWord == 8) d[i] = __ldg(reinterpret_cast<const uint2*>(p) + i);
      if constexpr (kWord == 4) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
      if constexpr (kWord == 2) h[i] = __ldg(reinterpret_cast<const uint16_t*>(p) + i);
    }
  }
  __device__ __forceinline__ void store(L* p) const {
#pragma unroll
    for (int i = 0; i < kBytes / kWord; ++i) {
      if constexpr (kWord == 16) reinterpret_cast<uint4*>(p)[i] = q[i];
      if constexpr (kWord == 8) reinterpret_cast<uint2*>(p)[i] = d[i];
      if constexpr (kWord == 4) reinterpret_cast<uint32_t*>(p)[i] = w[i];
      if constexpr (kWord == 2) reinterpret_cast<uint16_t*>(p)[i] = h[i];
    }
  }
};

// One token's logits, expert lane * V + v in x[v]; -inf where there is none.
// NaN counts as -inf and is reported; +inf as the largest fp32 value.  With
// `vec`, every lane holds V experts or none, at a whole word.
template <int V, typename L>
__device__ __forceinline__ void load_row(const L* row, int32_t E, bool vec, int lane, float (&x)[V],
                                         int32_t* status) {
  if (vec) {
    Vec<V, L> in;
    if ((lane + 1) * V <= E) in.load(row + lane * V);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = (lane + 1) * V <= E ? to_f32(in.v[v]) : -INFINITY;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = lane * V + v < E ? to_f32(row[lane * V + v]) : -INFINITY;
  }
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    nan |= x[v] != x[v];
    x[v] = x[v] != x[v] ? -INFINITY : fminf(x[v], FLT_MAX);
  }
  if (nan) set_status(status, MG_ERR_DEVICE_ARG);
}

// Exponential, sigmoid and quotient from the hardware's base-2 exponential (off
// by two units in the last place at most) and reciprocal (by one); results below
// 2^-126 flushed.  2^t with t the rounded x log2 e alone would be off by |x| / 2
// units of 2^-24 and more; the exact rest x - t ln 2 is put back to first order
// (it is below 2^-16, so the next order is below 2^-33): relative error 5 units,
// whatever x.  For x <= 88, or -inf, or NaN (0); below -128 the result is 0 anyway.
__device__ __forceinline__ float fast_exp(float x) {
  x = fmaxf(x, -128.0f);
  const float t = x * 1.4426950408889634f;
  const float rest = fmaf(-t, -1.9046543e-9f, fmaf(-t, 0.69314718f, x));    // ln 2 in two parts
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return fmaf(e, rest, e);
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 8 units: 5 of the exponential, the sum's rounding and the reciprocal.  From x =
// -88 down the score is below 2^-126, flushed.
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp(fminf(-x, 88.0f))); }

// Maximum of a token's logits (0 for a row at -inf throughout, whose scores
// are then all 0) and the sum of exp(x - maximum), at least 2^-126.
template <int V>
__device__ __forceinline__ void softmax_parts(const float (&x)[V], float (&e)[V], float& top, float& sum) {
  float m = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
  m = warp_max(m);
  top = m == -INFINITY ? 0.0f : m;
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = fast_exp(x[v] - top);
    sum += e[v];
  }
  sum = fmaxf(warp_sum(sum), FLT_MIN);
}

template <typename K>
__device__ __forceinline__ void order(K& a, K& b) {
  const K hi = a > b ? a : b, lo = a > b ? b : a;
  a = hi;
  b = lo;
}
// Descending by a sorting network of 1, 5 or 19 exchanges.
template <int V, typename K>
__device__ __forceinline__ void sort_desc(K (&o)[V]) {
  static_assert(V <= 8, "longer lists go through top_listed");
  if constexpr (V == 2) order(o[0], o[1]);
  if constexpr (V >= 4) {
#pragma unroll
    for (int b = 0; b < V; b += 4) {
      order(o[b], o[b + 1]);
      order(o[b + 2], o[b + 3]);
      order(o[b], o[b + 2]);
      order(o[b + 1], o[b + 3]);
      order(o[b + 1], o[b + 2]);
    }
  }
  if constexpr (V == 8) {
    order(o[0], o[4]);
    order(o[1], o[5]);
    order(o[2], o[6]);
    order(o[3], o[7]);
    order(o[2], o[4]);
    order(o[3], o[5]);
    order(o[1], o[2]);
    order(o[3], o[4]);
    order(o[5], o[6]);
  }
}

// The k largest keys of the warp as top_keys gives them, for long lists: a
// lane's V keys wait in shared memory (`sm`, 32 V words), and each round the
// first V lanes look for the winning lane's key and for its next largest
// together, some 40 instructions a round whatever V is.  (Eight two-word keys a
// lane are better sorted: 32768 x 256 with groups and bias 41 us against 39, but
// 48 tokens 3.9 us against 4.2.)
template <int V, typename K>
__device__ __forceinline__ void top_listed(const uint32_t (&o)[V], uint32_t* sm, int k, int to, int lane, K& mine) {
  __syncwarp();
  uint32_t head = o[0];
#pragma unroll
  for (int v = 1; v < V; ++v) head = max(head, o[v]);
#pragma unroll
  for (int v = 0; v < V; v += 4)
    *reinterpret_cast<uint4*>(sm + lane * V + v) = make_uint4(o[v], o[v + 1], o[v + 2], o[v + 3]);
  __syncwarp();
  for (int j = 0; j < k; ++j) {
    const uint32_t M = __reduce_max_sync(kAll, head);
    if (M == 0) break;
    const int win = __ffs(__ballot_sync(kAll, head == M)) - 1;    // the lowest lane: the lowest experts
    uint32_t key = lane < V ? sm[win * V + lane] : 0u;
    const int at = __ffs(__ballot_sync(kAll, key == M)) - 1;
    if (lane == at) {
      key = 0;
      sm[win * V + lane] = 0;
    }
    const uint32_t next = __reduce_max_sync(kAll, key);
    head = lane == win ? next : head;
    const K won = sizeof(K) == 4 ? (K)M : (((K)M << 16 << 16) | (0xffffffffu - (uint32_t)(win * V + at)));
    mine = lane == to + j ? won : mine;
    __syncwarp();
  }
}

__device__ __forceinline__ uint32_t head_word(uint32_t k) { return k; }
__device__ __forceinline__ uint32_t head_word(uint64_t k) { return (uint32_t)(k >> 32); }

// The k largest keys of the warp, in descending order: lane to + j gets the
// j-th (0 when there are fewer; with an odd k the lane after them may get one
// too), other lanes keep `mine`.  A key's upper part orders it, its lower part
// falls with the expert's index, so keys are distinct and ties go to the
// lowest expert.  K = uint32_t: the whole key in one word; uint64_t: the
// leading words are compared first, and among lanes whose leading word ties
// the lowest lane holds the lowest expert.  The keys of a lane come sorted, so
// that each round only drops the head of one lane's list.
template <int V, typename K>
__device__ __forceinline__ void top_sorted(K (&o)[V], int k, int to, int lane, K& mine) {
  // two rounds at a time: a round past k lands in a lane past the k choices
#pragma unroll 2
  for (int j = 0; j < ((k + 1) & ~1); ++j) {
    const uint32_t head = head_word(o[0]), M = __reduce_max_sync(kAll, head);
    K won;
    bool drop;
    if (sizeof(K) == 4) {
      won = (K)M;
      drop = head == M;
    } else {
      const int win = __ffs(__ballot_sync(kAll, head == M)) - 1;
      won = ((K)M << 16 << 16) | __shfl_sync(kAll, (uint32_t)o[0], win);
      drop = lane == win;
    }
    // (selects, not branches: one lane of the warp drops a key each round)
#pragma unroll
    for (int v = 0; v + 1 < V; ++v) o[v] = drop ? o[v + 1] : o[v];
    o[V - 1] = drop ? (K)0 : o[V - 1];
    mine = lane == to + j ? won : mine;
  }
}

// A warp takes `tpw` tokens (1, 2 or 4) one after another: all lanes score
// and choose for each, and each token's choices end up in a segment of 32 /
// tpw lanes, which finish the weights of all tokens together.  Without a bias
// the keys order as the logits do, so only the chosen experts are scored (and
// all of a softmax's exponentials are needed for its sum alone, when it is not
// renormalised); bf16 logits then fit a key and an index into one word.
// kFast: nothing but the chosen experts is scored and the logits' bits are the
// keys, in a kernel of its own (45 registers; as a branch of the general one, of
// 64, 9.4 us instead of 8.8 in the first case below, both before scores took
// their present form).
// Instructions bound this kernel, not its few bytes: 32768 tokens, softmax top-8
// of 128 bf16 logits 8.9 us (206 instructions a token, 88 of them the eight
// rounds; half are compares and selects at half rate), sigmoid top-8 of 256 in
// groups with a bias 42 us (960); 48 such tokens 4.0 us, one warp's chain.
template <int V, typename L, bool kBias, bool kFast>
__global__ void __launch_bounds__(kWarps * 32, V <= 4 ? 4 : V == 8 ? 3 : V <= 16 ? 2 : 1) route_kernel(const RouteArgs a) {
  constexpr bool kPacked = !kBias && sizeof(L) == 2;
  static_assert(!kFast || (kPacked && V >= 2 && V <= 8), "keys from the logits' bits");
  using K = typename std::conditional<kPacked, uint32_t, uint64_t>::type;
  // a lane's keys are sorted in registers, or listed in shared memory when they
  // are too many for that
  constexpr bool kLong = V > 8;
  __shared__ alignas(16) float group_keys[kWarps][V * 32 + 4 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L* logits = static_cast<const L*>(a.logits);
  float bias[kBias ? V : 1];
  if (kBias) {
#pragma unroll
    for (int v = 0; v < V; ++v) bias[kBias ? v : 0] = lane * V + v < a.E ? __ldg(a.bias + lane * V + v) : 0.0f;
  }
  const bool all_exp = a.softmax && (kBias || !a.renorm);
  const bool here = (lane + 1) * V <= a.E;
  const int seg = 32 / a.tpw;
  const int mine_i = lane / seg, mine_j = lane & (seg - 1);
  const int64_t step = (int64_t)gridDim.x * kWarps * a.tpw;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * a.tpw; t0 < a.T; t0 += step) {
    K mine = 0;
    float top = 0.0f, inv = 1.0f;                // of the token whose choices this lane finishes
    if constexpr (kFast) {
      // keys from the bits, no arithmetic on the logits; four tokens' loads
      // leave together
      Vec<V, L> in[4];
      const L* row = logits + t0 * a.ld + lane * V;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (here && i < a.tpw && t0 + i < a.T) {
          in[i].load(row);
        } else {
#pragma unroll
          for (int v = 0; v < V / 2; ++v) in[i].w[v] = 0xff80ff80u;
        }
        row += a.ld;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= a.tpw) break;
        uint32_t o[V];
#pragma unroll
        for (int v = 0; v < V; v += 2) packed_keys(in[i].w[v / 2], (uint32_t)(lane * V + v), o[v], o[v + 1]);
        sort_desc<V>(o);
        if (o[0] >= kNanKey) {
          set_status(a.status, MG_ERR_DEVICE_ARG);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] = o[v] >= kNanKey ? 0u : o[v];
          sort_desc<V>(o);
        }
        top_sorted<V, uint32_t>(o, a.k, i * seg, lane, mine);
      }
      mine = mine >= kFirstKey ? mine : (K)0;
    }
    for (int i = 0; i < a.tpw && t0 + i < a.T && !kFast; ++i) {
      const L* row = logits + (t0 + i) * a.ld;
      float x[V], key[V];
      load_row<V, L>(row, a.E, a.vec, lane, x, a.status);
      float inv_i = 1.0f;
      if (all_exp) {
        float top_i, sum_i;
        softmax_parts<V>(x, key, top_i, sum_i);
        inv_i = fast_rcp(sum_i);
        if (mine_i == i) {
          top = top_i;
          inv = inv_i;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (kBias) {
          const float b = (a.softmax ? key[v] * inv_i : sigmoid(x[v])) + bias[kBias ? v : 0];
          key[v] = (x[v] == -INFINITY || b != b) ? -INFINITY : b + 0.0f;   // + 0: -0 and 0 are equal keys
        } else {
          key[v] = x[v] + 0.0f;
        }
      }
      if (a.groups > 1) {
        // m1, m2: the two largest keys of the lane's group, g = the group
        float m1 = -INFINITY, m2 = -INFINITY;
        int g, lpg;                                // lanes per group
        if (a.lanes_per_group > 0) {
          // a group is a power of two of whole lanes
          lpg = a.lanes_per_group;
          g = lane / lpg;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            m2 = fmaxf(m2, fminf(m1, key[v]));
            m1 = fmaxf(m1, key[v]);
          }
        } else {
          float* gk = group_keys[warp];
          __syncwarp();
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int32_t e = lane * V + v;
            gk[e + 4 * (e >> 5)] = key[v];
          }
          __syncwarp();
          lpg = 32;
          while (lpg * a.groups > 32) lpg >>= 1;
          g = lane / lpg;
          const int32_t gs = a.group_size;
          if (g < a.groups) {
            for (int32_t j = lane - g * lpg; j < gs; j += lpg) {
              const int32_t e = g * gs + j;
              const float f = gk[e + 4 * (e >> 5)];
              m2 = fmaxf(m2, fminf(m1, f));
              m1 = fmaxf(m1, f);
            }
          }
        }
        for (int o = lpg >> 1; o >= 1; o >>= 1) {
          const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
          m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
          m1 = fmaxf(m1, o1);
        }
        float sc = m1;
        if (a.group_top == 2) {
          // sums of scores; without a bias the keys are logits (a softmax's
          // common denominator changes no comparison)
          if (kBias) {
            sc = m2 != -INFINITY ? m1 + m2 : m1;
          } else {
            const float shift = a.softmax ? warp_max(m1) : 0.0f;
            const float s1 = a.softmax ? fast_exp(m1 - shift) : sigmoid(m1);
            const float s2 = a.softmax ? fast_exp(m2 - shift) : sigmoid(m2);
            sc = m1 != -INFINITY ? s1 + s2 : m1;
          }
        }
        int rank = 0;
        for (int h = 0; h < a.groups; ++h) {
          const float o = __shfl_sync(kAll, sc, h * lpg);
          rank += (o > sc) || (o == sc && h < g);
        }
        const bool stays = g < a.groups && rank < a.top_groups;
        if (a.lanes_per_group > 0) {
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = stays ? key[v] : -INFINITY;
        } else {
          // (positions past E hold -inf, whichever group they are taken for)
          const uint32_t in = __ballot_sync(kAll, stays);
          const int32_t gs = a.group_size;
          if (gs >= V) {
            // a lane's experts are of one group, or of two: `cut` come before the second
            const int32_t g0 = min((int32_t)__umulhi(lane * V, a.group_inverse), a.groups - 1);   // lane * V / gs
            const int32_t cut = (g0 + 1) * gs - lane * V;
            const bool in0 = (in >> (g0 * lpg)) & 1u, in1 = (in >> (min(g0 + 1, a.groups - 1) * lpg)) & 1u;
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = (v < cut ? in0 : in1) ? key[v] : -INFINITY;
          } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
              const int32_t of = min((lane * V + v) / gs, a.groups - 1);
              key[v] = ((in >> (of * lpg)) & 1u) ? key[v] : -INFINITY;
            }
          }
        }
      }
      uint32_t o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t e = (uint32_t)(lane * V + v);
        const bool in = key[v] != -INFINITY;
        if (kPacked)
          o[v] = in ? (key[v] == FLT_MAX ? 0xff800000u : ordered(key[v]) & 0xffff0000u) | (0xffffu - e) : 0u;
        else
          o[v] = in ? ordered(key[v]) : 0u;
      }
      if constexpr (kLong) {
        top_listed<V, K>(o, reinterpret_cast<uint32_t*>(group_keys[warp]), a.k, i * seg, lane, mine);
      } else {
        K key2[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
          key2[v] = kPacked || o[v] == 0 ? (K)o[v] : (((K)o[v] << 16 << 16) | (0xffffffffu - (uint32_t)(lane * V + v)));
        sort_desc<V>(key2);
        top_sorted<V, K>(key2, a.k, i * seg, lane, mine);
      }
    }
    const int64_t t = t0 + mine_i;
    const bool got = mine != 0 && mine_j < a.k;
    int32_t idx = -1;
    float xs = -INFINITY, s = 0.0f;
    if (got) {
      if (kPacked) {
        idx = 0xffff - (int32_t)((uint32_t)mine & 0xffffu);
        xs = fminf(unordered(((uint32_t)mine & 0xffff0000u) | ((uint32_t)mine >> 31 ? 0u : 0xffffu)), FLT_MAX);
      } else {
        idx = (int32_t)(0xffffffffu - (uint32_t)mine);
        xs = kBias ? fminf(to_f32(logits[t * a.ld + idx]), FLT_MAX) : unordered((uint32_t)((uint64_t)mine >> 32));
      }
    }
    if (a.softmax) {
      // the first choice is the largest logit when there is no bias
      if (!all_exp) top = __shfl_sync(kAll, xs, lane & ~(seg - 1));
      if (got) s = fast_exp(xs - top) * inv;
    } else if (got) {
      s = sigmoid(xs);
    }
    if (a.renorm) {
      float total = s;
      for (int o = seg >> 1; o >= 1; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
      s *= fast_rcp(fmaxf(total, FLT_MIN));
    }
    if (mine_j < a.k && t < a.T) {
      a.idx[t * a.k + mine_j] = idx;
      a.w[t * a.k + mine_j] = s * a.scale;
    }
  }
}

template <int V, typename L>
__device__ __forceinline__ void store_row(L* out, int32_t E, bool vec, int lane, const float (&x)[V]) {
  if (vec) {
    Vec<V, L> o;
#pragma unroll
    for (int v = 0; v < V; ++v) from_f32(x[v], o.v[v]);
    if ((lane + 1) * V <= E) o.store(out + lane * V);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane * V + v < E) from_f32(x[v], out[lane * V + v]);
  }
}

// Softmax weights without renormalisation reach every logit of the token
// (kFull): one warp per token.  Otherwise only the chosen ones have a gradient
// (a renormalised softmax is the softmax over the chosen logits), so only those
// are read, of kTok tokens at once, and the rest of the rows is written as zeros.  A row is written whole first, and the chosen elements over it.  8191
// x 160 bf16, softmax without renormalisation: 5.0 us, 2 of them the launch.
template <int V, typename L, bool kFull, int kTok>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const RouteBwdArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L* logits = static_cast<const L*>(a.logits);
  L* dlogits = static_cast<L*>(a.dlogits);
  constexpr int kSeg = 32 / kTok;            // lanes of a token's choices
  const int sub = lane / kSeg, j = lane & (kSeg - 1);
  const int64_t step = (int64_t)gridDim.x * kWarps * kTok;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTok; t0 < a.T; t0 += step) {
    const int64_t t = t0 + sub;
    const L* row = logits + t * a.ld;
    int32_t i = -1;
    float up = 0.0f, xs = -INFINITY;
    if (j < a.k && t < a.T) {
      i = a.idx[t * a.k + j];
      if (i < -1 || i >= a.E) {
        set_status(a.status, MG_ERR_DEVICE_ARG);
        i = -1;
      }
      if (i >= 0) {
        up = a.scale * a.dw[t * a.k + j];
        xs = to_f32(row[i]);
        xs = xs != xs ? -INFINITY : fminf(xs, FLT_MAX);
      }
    }
    // lanes with the same expert of the same token
    const uint32_t same = __match_any_sync(kAll, i < 0 ? -1 : sub * a.E + i);
    const bool twice = __any_sync(kAll, i >= 0 && __popc(same) > 1);
    float d;                // the choice's own gradient
    if (kFull) {
      float x[V], base[V], top, sum;          // base: the row without the choices' own terms
      load_row<V, L>(row, a.E, a.vec, lane, x, a.status);
      softmax_parts<V>(x, base, top, sum);
      const float inv = fast_rcp(sum), ss = fast_exp(xs - top) * inv;
      const float dot = warp_sum(up * ss);
#pragma unroll
      for (int v = 0; v < V; ++v) base[v] *= -dot * inv;
      store_row<V, L>(dlogits + t * a.ldd, a.E, a.vec, lane, base);
      d = ss * (up - dot);
      // an expert that is chosen twice collects both
      if (twice) {
        float all = 0.0f;
        for (int c = 0; c < a.k; ++c) {
          const float u = __shfl_sync(kAll, up, c);
          if ((same >> c) & 1u) all += u;
        }
        d = ss * (all - dot);
      }
    } else {
      if (a.softmax) {
        float top = warp_max<kSeg>(xs);
        top = top == -INFINITY ? 0.0f : top;
        const float e = fast_exp(xs - top);
        const float p = e * fast_rcp(fmaxf(warp_sum<kSeg>(e), FLT_MIN));
        d = p * (up - warp_sum<kSeg>(p * up));
      } else {
        const float ss = sigmoid(xs), rest = sigmoid(-xs);
        float p = ss, g = up;
        if (a.renorm) {
          p = ss * fast_rcp(fmaxf(warp_sum<kSeg>(ss), FLT_MIN));
          g = up - warp_sum<kSeg>(p * up);
        }
        d = p * g * rest;
      }
      if (twice) {
        float all = 0.0f;
        for (int c = 0; c < a.k; ++c) {
          const int from = sub * kSeg + c;
          const float u = __shfl_sync(kAll, d, from);
          if ((same >> from) & 1u) all += u;
        }
        d = all;
      }
      const float zero[V] = {};
#pragma unroll
      for (int q = 0; q < kTok; ++q)
        if (t0 + q < a.T) store_row<V, L>(dlogits + (t0 + q) * a.ldd, a.E, a.vec, lane, zero);
    }
    __syncwarp();           // the rows before the elements over them
    if (i >= 0) from_f32(d, dlogits[t * a.ldd + i]);
  }
}

// Whole words of V values per lane, for rows `ld` apart.
template <int V, typename L>
bool whole_words(const void* p, int64_t ld, int32_t E) {
  constexpr int word = Vec<V, L>::kWord;
  return E % V == 0 && (ld * (int64_t)sizeof(L)) % word == 0 && reinterpret_cast<uintptr_t>(p) % word == 0;
}

// Tokens per warp: as many as their choices' lanes allow, while every SM still
// has 32 warps.
int32_t tokens_per_warp(int64_t T, int32_t k) {
  int32_t n = 1;
  while (2 * n * k <= 32 && n < 4 && T >= (int64_t)num_sms_current_device() * 32 * 2 * n) n *= 2;
  return n;
}

template <int V, typename L>
cudaError_t launch_route_as(RouteArgs a, int blocks, cudaStream_t s) {
  a.vec = whole_words<V, L>(a.logits, a.ld, a.E);
  const int32_t gs = a.E / a.groups, lpg = gs / V;
  a.group_size = gs;
  a.group_inverse = 0xffffffffu / (uint32_t)gs + 1;   // used for gs >= 2 and quotients of numbers below 2^10
  a.lanes_per_group = gs % V == 0 && (lpg & (lpg - 1)) == 0 ? lpg : 0;
  a.tpw = tokens_per_warp(a.T, a.k);
  // bf16 logits in whole words, neither a bias nor groups, and no softmax over
  // all experts: the kernel that works on the logits' bits
  constexpr bool kHasFast = sizeof(L) == 2 && V >= 2 && V <= 8;
  if (a.bias != nullptr)
    route_kernel<V, L, true, false><<<blocks, kWarps * 32, 0, s>>>(a);
  else if (kHasFast && a.vec && a.groups == 1 && !(a.softmax && !a.renorm))
    route_kernel<V, L, false, kHasFast><<<blocks, kWarps * 32, 0, s>>>(a);
  else
    route_kernel<V, L, false, false><<<blocks, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}
template <int V>
cudaError_t launch_route_v(const RouteArgs& a, int blocks, cudaStream_t s) {
  return a.f32 ? launch_route_as<V, float>(a, blocks, s) : launch_route_as<V, __nv_bfloat16>(a, blocks, s);
}
template <int V, typename L>
cudaError_t launch_bwd_as(RouteBwdArgs a, int blocks, cudaStream_t s) {
  a.vec = whole_words<V, L>(a.logits, a.ld, a.E) && whole_words<V, L>(a.dlogits, a.ldd, a.E);
  // four tokens to a warp: 65536 tokens, top-8 of 256, bf16 13 us, one to a warp
  // 24; from 384 on their rows' zeros are most of the work (top-4 of 384, fp32
  // 36 us, 34 with one)
  constexpr int kTok = V <= 8 ? 4 : 1;
  if (a.softmax && !a.renorm)
    route_bwd_kernel<V, L, true, 1><<<blocks, kWarps * 32, 0, s>>>(a);
  else if (tokens_per_warp(a.T, a.k) == 4)
    route_bwd_kernel<V, L, false, kTok><<<blocks, kWarps * 32, 0, s>>>(a);
  else
    route_bwd_kernel<V, L, false, 1><<<blocks, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}
template <int V>
cudaError_t launch_bwd_v(const RouteBwdArgs& a, int blocks, cudaStream_t s) {
  return a.f32 ? launch_bwd_as<V, float>(a, blocks, s) : launch_bwd_as<V, __nv_bfloat16>(a, blocks, s);
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
  if (a.E <= 384) return launch_route_v<12>(a, b, s);
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
  if (a.E <= 384) return launch_bwd_v<12>(a, b, s);
  if (a.E <= 512) return launch_bwd_v<16>(a, b, s);
  return launch_bwd_v<32>(a, b, s);
}

// ------------------------------------------------------------------ slot map
namespace slots {

constexpr int kPer = 4;                          // choices a thread holds
constexpr uint32_t kAll = 0xffffffffu;
static_assert(kSlotChunk <= 65535 && kMaxExperts <= 65535, "a rank and an expert fit 16 bits each");

// Words of a warp's 16-bit counters, one per expert.
__host__ __device__ constexpr int32_t row_words(int32_t E) { return (E + 1) / 2; }
__host__ __device__ constexpr int place_smem(int32_t E, int threads) {
  return 5 * (int)sizeof(int32_t) * E + (threads / 32 * row_words(E) + threads * kPer) * (int)sizeof(uint32_t);
}

// Lanes that hold the same expert as this one: one vote per bit of the index.
__device__ __forceinline__ uint32_t same_expert(int32_t e, int bits) {
  uint32_t same = __ballot_sync(kAll, e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool set = ((e >> b) & 1) != 0;
    const uint32_t v = __ballot_sync(kAll, set);
    same &= set ? v : ~v;
  }
  return same;
}

// Choices per expert of one chunk (integer additions: any order gives the
// same counts).
__global__ void __launch_bounds__(kSlotChunk / kPer) count_kernel(const SlotArgs a) {
  constexpr int kT = kSlotChunk / kPer;
  extern __shared__ int32_t hist[];
  // the place kernel may start: it waits for this grid's results itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t c0 = (int64_t)blockIdx.x * kSlotChunk;
  int32_t ex[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t at = c0 + i * kT + threadIdx.x;
    ex[i] = at < a.n ? __ldg(a.idx + at) : -1;
  }
  for (int32_t e = threadIdx.x; e < a.E; e += kT) hist[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (ex[i] >= 0 && ex[i] < a.E) atomicAdd(&hist[ex[i]], 1);
  __syncthreads();
  for (int32_t e = threadIdx.x; e < a.E; e += kT) a.work[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// Rank of every choice among its expert's choices, in flat order, and the row
// it gets.  A block of kT threads holds a part of 4 kT consecutive choices, a
// warp 128 of them; equal experts inside a group of 32 find each other by
// votes, so ranks come out in order without atomics.  The parts before a
// block's within its chunk of 4096 choices are counted by the block itself;
// the chunks before it by count_kernel, unless there is one chunk only
// (kOne), whose other parts the block counts too.  Every block lays the experts
// out from the totals.  Small blocks finish sooner (an SM that holds a whole
// chunk spends its time issuing), large ones read the chunks' counts less
// often: with the counts, 32768 choices over 64 experts 6.2 us, 61 x 4 over 16
// 3.7 us, 131072 over 256 11.9 us in large blocks and 14.1 in small ones.  The
// blocks' reads of the counts grow with the square of the choices: 2^22 over 256
// 0.37 ms, 1 GB from L2; 2^24 4.9 ms.
template <int kT, bool kOne>
__global__ void __launch_bounds__(kT) place_kernel(const SlotArgs a) {
  constexpr int kW = kT / 32, kPart = kT * kPer, kParts = kSlotChunk / kPart;
  extern __shared__ int32_t sh[];
  // the dispatch that reads the map may be set up meanwhile (it waits for it)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int32_t* chunk = sh;               // choices of expert e in this part
  int32_t* total = chunk + a.E;      // in all
  int32_t* before = total + a.E;     // of those, in front of this part
  int32_t* base = before + a.E;      // first row, -1 when the expert is dropped
  int32_t* first = base + a.E;       // position of expert e's first choice in `sorted`
  uint32_t* words = reinterpret_cast<uint32_t*>(first + a.E);
  uint16_t* wh = reinterpret_cast<uint16_t*>(words);        // [kW][ws]
  uint32_t* sorted = words + kW * row_words(a.E);           // the part's choices by expert
  __shared__ int64_t scan[32];
  __shared__ int32_t scan1[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t E = a.E, ws = 2 * row_words(E);
  // blocks past the choices only clear rows; of one chunk they count the choices
  // as its last part's block does
  const uint32_t block = kOne ? min(blockIdx.x, (uint32_t)kParts - 1) : blockIdx.x;
  const bool extra = block != blockIdx.x || (int64_t)block * kPart >= a.n;
  const int32_t part = (int32_t)(block % kParts), my_chunk = (int32_t)(block / kParts);
  const int64_t p0 = (int64_t)block * kPart, c0 = p0 + warp * 32 * kPer;
  int32_t ex[kPer], other[kParts > 1 ? (kParts - 1) * kPer : 1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t at = c0 + i * 32 + lane;
    ex[i] = at < a.n ? __ldg(a.idx + at) : -1;
  }
#pragma unroll
  for (int i = 0; i < (kParts - 1) * kPer; ++i) {
    // the other parts in order, this one left out
    const int p = i / kPer + (i / kPer >= part ? 1 : 0);
    const int64_t at = (int64_t)my_chunk * kSlotChunk + p * kPart + (i % kPer) * kT + tid;
    other[i] = (kOne || p < part) && at < a.n ? __ldg(a.idx + at) : -1;
  }
  for (int32_t e = tid; e < E; e += kT) total[e] = before[e] = 0;
  for (int32_t i = lane; i < ws / 2; i += 32) words[warp * (ws / 2) + i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (ex[i] < -1 || ex[i] >= E) {
      set_status(a.status, MG_ERR_DEVICE_ARG);
      ex[i] = -1;
    }
  }
  const int bits = 32 - __clz(E - 1);
  uint32_t same[kPer];
  uint16_t* mine = wh + warp * ws;
#pragma unroll
  for (int i = 0; i < kPer; ++i) same[i] = same_expert(ex[i], bits);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (ex[i] >= 0 && lane == __ffs(same[i]) - 1) mine[ex[i]] += (uint16_t)__popc(same[i]);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < (kParts - 1) * kPer; ++i) {
    if (other[i] >= 0 && other[i] < E) {
      if (kOne) atomicAdd(&total[other[i]], 1);
      if (i / kPer < part) atomicAdd(&before[other[i]], 1);
    }
  }
  if (!kOne) {
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the chunk counts
    // a thread adds up one expert's counts, or every kT / E-th of them
    const int32_t chunks = (int32_t)((a.n + kSlotChunk - 1) / kSlotChunk), per = E < kT ? kT / E : 1;
    for (int32_t i = tid; i < per * E; i += kT) {
      const int32_t sub = i / E, e = i - sub * E;
      int32_t t = 0, bf = 0;
#pragma unroll 16
      for (int32_t c = sub; c < chunks; c += per) {
        const int32_t v = __ldcg(a.work + (int64_t)c * E + e);
        t += v;
        bf += c < my_chunk ? v : 0;
      }
      atomicAdd(&total[e], t);
      if (bf != 0) atomicAdd(&before[e], bf);
    }
  }
  __syncthreads();
  // exclusive prefix over the warps of this part
  for (int32_t e = tid; e < E; e += kT) {
    int32_t run = 0;
#pragma unroll
    for (int w0 = 0; w0 < kW; w0 += 8) {
      uint16_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = wh[(w0 + w) * ws + e];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        wh[(w0 + w) * ws + e] = (uint16_t)run;
        run += c[w];
      }
    }
    chunk[e] = run;
    if (kOne) total[e] += run;
  }
  __syncthreads();
  // layout: base rows, counts, and where the experts' choices lie in `sorted`
  const uint32_t q = a.masked ? 1u : (uint32_t)a.align_q;
  int64_t carry = 0;
  int32_t carry1 = 0;
  bool full = false;
  for (int32_t b = 0; b < E; b += kT) {
    const int32_t e = b + tid;
    const bool busy = b + warp * 32 < E;          // warps past the experts only wait
    int64_t c = 0, padded = 0, v = 0;
    int32_t own = 0, v1 = 0;
    if (busy) {
      c = e < E ? total[e] : 0;
      padded = (int64_t)cdiv_u32((uint32_t)c, q) * q;
      own = e < E ? chunk[e] : 0;
      v = padded;
      v1 = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kAll, v, o);
        const int32_t u1 = __shfl_up_sync(kAll, v1, o);
        if (lane >= o) v += u, v1 += u1;
      }
    }
    if (lane == 31) scan[warp] = v, scan1[warp] = v1;
    __syncthreads();
    int64_t below = carry;
    int32_t below1 = carry1;
    const int32_t used = min(kW, (E - b + 31) / 32);
    for (int w = 0; w < used; ++w) {
      if (w < warp) below += scan[w], below1 += scan1[w];
      carry += scan[w];
      carry1 += scan1[w];
    }
    if (b + kT < E) __syncthreads();
    if (e < E) {
      int64_t start = below + v - padded;
      bool fits = true;
      if (a.masked) {
        start = (int64_t)e * a.M_max;
        full |= c > a.M_max;
      } else {
        fits = start + c <= a.rows_total;           // as the GEMMs: an expert that does not fit is skipped
        full |= start + padded > a.rows_total;
      }
      base[e] = fits ? (int32_t)start : -1;
      first[e] = below1 + v1 - own;
      if (blockIdx.x == 0) a.counts[e] = (int32_t)(a.masked ? min(c, (int64_t)a.M_max) : c);
    }
  }
  if (blockIdx.x == 0 && full) set_status(a.status, MG_ERR_CAPACITY);
  __syncthreads();
  // row of the in-th of the part's choices of expert e
  auto row_of = [&](int32_t e, int32_t in) {
    const int32_t r = before[e] + in, b = base[e];
    return b >= 0 && (!a.masked || r < a.M_max) ? b + r : -1;
  };
  if (!extra) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = c0 + i * 32 + lane;
      const int32_t e = ex[i];
      int32_t row = -1;
      if (e >= 0) {
        const int32_t in = mine[e] + __popc(same[i] & ((1u << lane) - 1u));
        row = row_of(e, in);
        sorted[first[e] + in] = ((uint32_t)e << 16) | (uint32_t)((warp * kPer + i) * 32 + lane);
      }
      __syncwarp();
      if (e >= 0 && lane == __ffs(same[i]) - 1) mine[e] += (uint16_t)__popc(same[i]);
      __syncwarp();
      if (at < a.n) a.rows[at] = row;
    }
  }
  if (a.src == nullptr) return;
  __syncthreads();
  // the choice of every row, expert by expert: consecutive rows together
  for (int32_t p = tid; p < carry1 && !extra; p += kT) {
    const uint32_t w = sorted[p];
    const int32_t e = (int32_t)(w >> 16), row = row_of(e, p - first[e]);
    if (row >= 0) a.src[row] = (int32_t)(p0 + (w & 0xffffu));
  }
  // -1 in the rows that no choice fills (rows are below 2^31, their ends
  // below 2^32)
  const uint32_t R = (uint32_t)a.rows_total;
  // a warp's experts, 32 at a time: a lane works out where one's rows end; `share`
  // warps to an expert where there are more warps than experts
  const int32_t warps = (int32_t)gridDim.x * kW, w0 = (int32_t)blockIdx.x * kW + warp;
  const int32_t share = max(1, warps / E), sub = share > 1 ? w0 / E : 0;
  for (int32_t e0 = sub < share ? w0 - sub * E : E; e0 < E; e0 += 32 * warps) {
    const int32_t e = e0 + lane * warps;
    uint32_t from = 0, to = 0;
    if (e < E) {
      const uint32_t c = (uint32_t)total[e];
      if (a.masked) {
        from = (uint32_t)e * (uint32_t)a.M_max + min(c, (uint32_t)a.M_max);
        to = (uint32_t)(e + 1) * (uint32_t)a.M_max;
      } else if (base[e] >= 0) {                         // (a dropped one's: with the tail below)
        to = min((uint32_t)base[e] + cdiv_u32(c, q) * q, R);
        from = (uint32_t)base[e] + c;
      }
    }
    const int32_t n = min(32, (E - e0 + warps - 1) / warps);
    for (int i = 0; i < n; ++i) {
      const uint32_t end = __shfl_sync(kAll, to, i);
      for (uint32_t r = __shfl_sync(kAll, from, i) + 32 * sub + lane; r < end; r += 32 * share) a.src[r] = -1;
    }
  }
  if (!a.masked) {
    // segments start in expert order, so the rows past the last expert that
    // fits hold nothing (an expert behind a dropped one starts past the end)
    uint32_t end = 0;
    for (int32_t e = E - 1; e >= 0; --e) {
      if (base[e] >= 0) {
        end = (uint32_t)base[e] + cdiv_u32((uint32_t)total[e], q) * q;
        break;
      }
    }
    for (int64_t r = (int64_t)end + (int64_t)blockIdx.x * kT + tid; r < R; r += (int64_t)gridDim.x * kT) a.src[r] = -1;
  }
}

template <int kT, bool kOne>
cudaError_t launch_place(const SlotArgs& a, cudaStream_t s) {
  static std::atomic<bool> done[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !done[dev]) {
    err = cudaFuncSetAttribute(place_kernel<kT, kOne>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               place_smem(kMaxExperts, kT));
    if (err != cudaSuccess) return err;
    if (dev < 64) done[dev] = true;
  }
  // blocks of choices, or as many more as leave each 1024 rows of `src` to clear:
  // 244 choices into 256 buffers of 256 4.2 us, by the choices' one block 10.3 (with
  // 8192 rows to a block 4.8); into 16 buffers 3.7 and 4.0
  constexpr int kClearRows = 1024;
  const int64_t own = a.n > 0 ? (a.n + kT * kPer - 1) / (kT * kPer) : 1;
  const int64_t clear = a.src != nullptr ? (a.rows_total + kClearRows - 1) / kClearRows : 0;
  const int64_t most = num_sms_current_device(), wanted = clear < most ? clear : most;
  const int64_t blocks = own > wanted ? own : wanted;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kT);
  cfg.dynamicSmemBytes = (size_t)place_smem(a.E, kT);
  cfg.stream = s;
  if (!kOne) {
    // launched while the counts are still being taken: it waits for them
    // where it needs them, and writes nothing before
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, place_kernel<kT, kOne>, a);
}

}  // namespace slots

cudaError_t launch_slots(const SlotArgs& a, cudaStream_t s) {
  using namespace slots;
  if (a.n <= kSlotChunk) return launch_place<256, true>(a, s);
  count_kernel<<<(unsigned)((a.n + kSlotChunk - 1) / kSlotChunk), kSlotChunk / kPer, a.E * sizeof(int32_t), s>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  return a.n <= 16 * kSlotChunk ? launch_place<256, false>(a, s) : launch_place<1024, false>(a, s);
}

}  // namespace mg
