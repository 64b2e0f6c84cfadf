// The router's balance loss over packed sequences, with its counts per expert,
// and the gradient of the logits.  For each sequence, with c_e the choices of
// expert e, C their sum, n the tokens with a logit above -inf and p a token's
// scores as shares of their sum:
//   gain_e = coef E c_e / (C n),   loss = sum_e gain_e sum_t p_te,
//   dx_e = dloss p_e (gain_e - sum_j gain_j p_j)   (a sigmoid's also times 1 - s_e).
#include <atomic>
#include <type_traits>

#include "blockq.cuh"
#include "cluster.cuh"
#include "ops_internal.h"
#include "scores.cuh"

namespace mg {
namespace balance {

using namespace route;

// Warps of a block of the forward pass, one row of [E] sums each in shared memory
// (36 KB at most); 32 warps for each of 152 SMs for long inputs, so that few parts are
// left to add.  Up to 256 experts (64 registers) they all run at once; above (118 to
// 128 registers) 16 an SM do, and the blocks go in two rounds.
constexpr int warps_of(int32_t E) { return E <= 256 ? 32 : E <= 512 ? 16 : 8; }
// Tokens of a block: the same for all, never less than a token a warp.
int32_t run_of(int64_t T, int64_t blocks, int64_t warps) {
  const int64_t n = (T + blocks - 1) / blocks;
  return (int32_t)(n < warps ? warps : (n + warps - 1) / warps * warps);
}
struct Runs {
  int32_t tokens, count;
  bool split;                              // a block a sequence of the run
};
// A block takes its run's sequences one after another, 3 to 6 us each, or only one of
// them, where there are no more blocks for that and a run hardly grows for it (1066 tokens
// of 160 experts in 64 sequences 8.3 us instead of 19.3, 8191 in 8 8.4 and 9.8;
// 131072 of 128 in 64, whose runs would grow by 600 tokens, 31 instead of 25.5).
Runs runs_of(int64_t T, int32_t E, int64_t S) {
  const int64_t warps = warps_of(E), blocks = 152 * 32 / warps;
  const int32_t whole = run_of(T, blocks, warps), part = S < blocks ? run_of(T, blocks - S + 1, warps) : whole;
  const bool split = S > 1 && S < blocks && part <= whole + 2 * warps;
  const int32_t n = split ? part : whole;
  return {n, (int32_t)((T + n - 1) / n), split};
}

// First and end token of sequence s: 0 and T without bounds.
__device__ __forceinline__ int32_t bound(const int32_t* seqs, int32_t s, int32_t T) {
  if (seqs == nullptr) return s == 0 ? 0 : T;
  return min(max(__ldg(seqs + s), 0), T);
}
// The last sequence that starts at or before token t (-1: none), found by a warp: 32
// bounds a step.
__device__ __forceinline__ int32_t sequence_at(const int32_t* seqs, int32_t S, int32_t T, int32_t t, int lane) {
  int32_t lo = -1, hi = S;                   // bound(lo) <= t < bound(hi), with the ends as sentinels
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) >> 5;
    const int64_t at = lo + (int64_t)(lane + 1) * step;
    const bool below = at < hi && bound(seqs, (int32_t)at, T) <= t;
    lo += __popc(__ballot_sync(kAll, below)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}
// The last sequence whose first part is number p or one before.
__device__ __forceinline__ int32_t sequence_of(const int32_t* seqs, int32_t S, int32_t T, int32_t p, int32_t chunk, int lane) {
  int32_t lo = 0, hi = S;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) >> 5;
    const int64_t at = lo + (int64_t)(lane + 1) * step;
    const bool below = at < hi && bound(seqs, (int32_t)at, T) / chunk + at <= p;
    lo += __popc(__ballot_sync(kAll, below)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A token's experts spread over kLanes lanes, in words of four that the lanes take
// in turns; several tokens a warp where few experts leave room.
template <int V, int kLanes, typename L>
struct Row {
  static constexpr bool kF32 = sizeof(L) == 4;
  uint32_t w[kF32 ? V : V / 2];
  // expert of value v of lane l
  static __device__ __forceinline__ int expert(int l, int v) { return ((v >> 2) * kLanes + l) * 4 + (v & 3); }
  __device__ __forceinline__ Row() {}
  // none: the bits that lanes without experts hold, and the others before their
  // first load
  __device__ __forceinline__ explicit Row(uint32_t none) {
#pragma unroll
    for (int i = 0; i < (kF32 ? V : V / 2); ++i) w[i] = none;
  }
  static constexpr int kPiece = 4 * (int)sizeof(L);      // bytes of a word of four experts
  static constexpr int kStage = 32 * V * (int)sizeof(L); // of a warp's rows in shared memory
  // Rows of whole words (`vec`) go through shared memory, each lane copying ahead
  // what it reads itself; `slot` is this lane's place in a stage.
  static __device__ __forceinline__ void copy(uint32_t slot, const L* row, int32_t E, int l) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const int at = expert(l, 4 * i);
      if (at >= E) continue;
      if constexpr (kF32)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + i * 32 * kPiece), "l"(row + at) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot + i * 32 * kPiece), "l"(row + at) : "memory");
    }
  }
  __device__ __forceinline__ void read(uint32_t slot, int32_t E, int l) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      if (expert(l, 4 * i) >= E) continue;
      if constexpr (kF32)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(slot + i * 32 * kPiece)
                     : "memory");
      else
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[2 * i]), "=r"(w[2 * i + 1]) : "r"(slot + i * 32 * kPiece) : "memory");
    }
  }
  // Other rows straight from memory.  Coherent loads: the gradient may be written over
  // what it is made from.
  __device__ __forceinline__ void fetch(const L* row, int32_t E, int l) {
    if constexpr (kF32) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (expert(l, v) < E) w[v] = reinterpret_cast<const uint32_t*>(row)[expert(l, v)];
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const int at = expert(l, v);
        if (at < E) w[v / 2] = h[at] | (at + 1 < E ? (uint32_t)h[at + 1] << 16 : w[v / 2] & 0xffff0000u);
      }
    }
  }
  // as pairs
  __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (kF32)
        x[v] = __uint_as_float(w[v]);
      else
        x[v] = __uint_as_float(v & 1 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (kF32)
        w[v] = __float_as_uint(x[v]);
      else if (v % 2 == 0)
        w[v / 2] = f32x2_to_bf16x2(pack2(x[v], x[v + 1]));
    }
  }
  __device__ __forceinline__ void store(L* row, int32_t E, bool vec, int l) const {
    if (vec) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const int at = expert(l, 4 * i);
        if (at >= E) continue;
        if constexpr (kF32)
          *reinterpret_cast<uint4*>(row + at) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        else
          *reinterpret_cast<uint2*>(row + at) = make_uint2(w[2 * i], w[2 * i + 1]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (expert(l, v) >= E) continue;
        if constexpr (kF32)
          reinterpret_cast<uint32_t*>(row)[expert(l, v)] = w[v];
        else
          reinterpret_cast<uint16_t*>(row)[expert(l, v)] = (uint16_t)(w[v / 2] >> (16 * (v & 1)));
      }
    }
  }
};
// Rows on their way and in use.
template <int V, typename L>
constexpr int kStagesOf = V * (int)sizeof(L) <= 48 ? 3 : 2;
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// -inf in each value of a word.
template <typename L>
__device__ __forceinline__ constexpr uint32_t no_expert() {
  return sizeof(L) == 4 ? 0xff800000u : 0xff80ff80u;
}

// fast_exp of two numbers, in the same steps: for numbers from -1e38 to 88 (below
// -126 ln 2 the result is 0).
__device__ __forceinline__ uint64_t fast_exp2(uint64_t x) {
  const uint64_t l2e = pack2(1.4426950408889634f, 1.4426950408889634f);
  const uint64_t hi = pack2(-0.69314718f, -0.69314718f), lo = pack2(1.9046543e-9f, 1.9046543e-9f);
  const uint64_t t = mul2(x, l2e), rest = fma2(t, lo, fma2(t, hi, x));
  const float2 f = unpack2(t);
  float p, q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(f.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(f.y));
  const uint64_t e = pack2(p, q);
  return fma2(e, rest, e);
}

// Scores of a token's experts in pairs, and with kRest the sigmoids' 1 - s =
// exp(-x) s, which is 0 where s is below 2^-126; 1 over the scores' sum (at least
// 2^-126).  NaN counts as -inf and is reported, +inf as the largest fp32 value: one
// comparison a logit finds them, with the sigmoid also what exp(-x) leaves fp32 for.
// some: this lane has a logit above -inf.
template <int V, int kLanes, bool kRest>
__device__ __forceinline__ float scores(float (&x)[V], bool softmax, uint64_t (&s)[V / 2], uint64_t (&rest)[V / 2],
                                        bool& some, int32_t* status) {
  bool odd = false;
#pragma unroll
  for (int v = 0; v < V; ++v) odd |= softmax ? !(x[v] <= FLT_MAX) : !(fabsf(x[v]) <= 87.0f);
  some = !odd;
  if (odd) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (x[v] != x[v]) {
        set_status(status, MG_ERR_DEVICE_ARG);
        x[v] = -INFINITY;
      }
      some |= x[v] != -INFINITY;
      x[v] = softmax ? fminf(x[v], FLT_MAX) : fmaxf(fminf(x[v], 128.0f), -88.0f);
    }
  }
  uint64_t sum = 0;
  if (softmax) {
    float top = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, x[v]);
    some = top != -INFINITY;
    top = warp_max<kLanes>(top);
    top = top == -INFINITY ? 0.0f : top;
    const uint64_t down = pack2(-top, -top);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 d = unpack2(add2(pack2(x[2 * i], x[2 * i + 1]), down));
      s[i] = fast_exp2(pack2(fmaxf(d.x, -128.0f), fmaxf(d.y, -128.0f)));
      sum = add2(sum, s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint64_t e = fast_exp2(pack2(-x[2 * i], -x[2 * i + 1]));
      const float2 d = unpack2(add2(e, pack2(1.0f, 1.0f)));
      s[i] = pack2(fast_rcp(d.x), fast_rcp(d.y));
      if (kRest) rest[i] = mul2(e, s[i]);
      sum = add2(sum, s[i]);
    }
  }
  const float2 q = unpack2(sum);
  return fast_rcp(fmaxf(warp_sum<kLanes>(q.x + q.y), FLT_MIN));
}

// Parts of the forward pass: one for every (block, sequence) that meet, at index
// block + sequence, which no other pair of them has; [E] sums of shares, [E]
// counts, tokens, choices.
__host__ __device__ inline int64_t part_words(int32_t E) { return 2 * (int64_t)E + 2; }

// A block takes a run of tokens with the sequences in it one after another, or
// (`split`) a part alone: of a run, the tokens of one sequence.  A warp takes every
// kWarps-th handful of them, the next one's logits on their way; at every sequence's
// end the warps' sums are added in a fixed order and written.  65536 tokens of 256
// experts in 24 sequences, sigmoids of fp32, 20.5 us with the kernel below (68.9 MB,
// 3.4 TB/s): two thirds of the issue slots while it runs (an exponential and a
// reciprocal a logit), its start, and the sums at its end.  8191 of 160 8.5 us, 4 of
// them the kernel below; with rows straight from memory instead of the ring 8.6, and
// 65536 of 160 20 us instead of 16.6.
template <int V, int kLanes, typename L, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) balance_kernel(const BalanceArgs a, int32_t chunk, bool split) {
  constexpr int kTok = 32 / kLanes;          // tokens a warp at once
  using R = Row<V, kLanes, L>;
  constexpr int kStages = kStagesOf<V, L>;
  extern __shared__ uint4 raw[];             // rows, then [kWarps, E] sums, [E + 2] counts, tokens and choices
  float* sh = reinterpret_cast<float*>(raw) + kWarps * kStages * R::kStage / 4;
  int32_t* hist = reinterpret_cast<int32_t*>(sh + kWarps * a.E);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & (kLanes - 1);
  const uint32_t ring = smem_u32(raw) + warp * (kStages * R::kStage) + lane * R::kPiece;
  const int32_t E = a.E;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const L* logits = static_cast<const L*>(a.logits);
  const int64_t step = kWarps * kTok * a.ld;
  const int32_t own = warp * kTok + lane / kLanes;
  R next(no_expert<L>());
  // the part's number is its run's plus its sequence's, and grows with the sequence
  int32_t s = split ? sequence_of(a.seqs, a.S, a.T, (int32_t)blockIdx.x, chunk, lane)
                    : max(sequence_at(a.seqs, a.S, a.T, (int32_t)blockIdx.x * chunk, lane), 0);
  const int32_t run = (int32_t)blockIdx.x - (split ? s : 0), last = split ? s + 1 : a.S;
  const int64_t t0 = (int64_t)run * chunk;
  if (t0 >= a.T) return;                     // more numbers than parts
  const int32_t t1 = (int32_t)min((int64_t)a.T, t0 + chunk);
  for (; s < last; ++s) {
    const int32_t b = max(bound(a.seqs, s, a.T), (int32_t)t0), e = min(bound(a.seqs, s + 1, a.T), t1);
    if (b >= t1) break;
    if (b >= e) continue;
    int32_t t = b + own, ahead_t = t, ahead_s = 0;
    const L* row = logits + (int64_t)t * a.ld;
    auto ahead = [&]() {
      if (a.vec && ahead_t < e) R::copy(ring + ahead_s * R::kStage, row, E, l);
      asm volatile("cp.async.commit_group;" ::: "memory");
      ahead_t += kWarps * kTok;
      row += step;
      ahead_s = ahead_s + 1 == kStages ? 0 : ahead_s + 1;
    };
#pragma unroll
    for (int i = 1; i < kStages; ++i) ahead();
    for (int i = tid; i < E + 2; i += kWarps * 32) hist[i] = 0;
    __syncthreads();
    int32_t live = 0, chosen = 0;
    const int64_t n = (int64_t)(e - b) * a.k;
    const int32_t* idx = a.idx + (int64_t)b * a.k;
#pragma unroll 4
    for (int64_t i = tid; i < n; i += kWarps * 32) {
      const int32_t c = __ldg(idx + i);
      if (c < -1 || c >= E) {
        set_status(a.status, MG_ERR_DEVICE_ARG);
      } else if (c >= 0) {
        atomicAdd(hist + c, 1);
        ++chosen;
      }
    }
    uint64_t sum[V / 2] = {};
    int at = 0;
    for (int32_t u = b + warp * kTok; u < e; u += kWarps * kTok) {      // the same for all lanes
      float x[V];
      uint64_t v[V / 2];
      const bool there = t < e;
      if (a.vec) {
        cp_async_wait<kStages - 2>();
        if (there) next.read(ring + at * R::kStage, E, l);
        ahead();                             // into the stage that was read a round ago
        at = at + 1 == kStages ? 0 : at + 1;
      } else if (there) {
        next.fetch(logits + (int64_t)t * a.ld, E, l);
      }
      next.get(x);
      t += kWarps * kTok;
      bool some;
      const float inv = scores<V, kLanes, false>(x, a.softmax, v, v, some, a.status);
      const uint32_t alive = __ballot_sync(kAll, some && there) >> (lane & ~(kLanes - 1));
      if constexpr (kLanes < 32)
        live += (alive & ((1u << kLanes) - 1)) != 0;
      else
        live += alive != 0;
      const float share = there ? inv : 0.0f;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) sum[i] = fma2(v[i], pack2(share, share), sum[i]);
    }
    cp_async_wait<0>();
    // over the warp's tokens at once
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) sum[i] = add2(sum[i], __shfl_xor_sync(kAll, sum[i], o));
    }
    live = l == 0 ? live : 0;
    live = __reduce_add_sync(kAll, live);
    chosen = __reduce_add_sync(kAll, chosen);
    if (lane == 0) {
      atomicAdd(hist + E, live);
      atomicAdd(hist + E + 1, chosen);
    }
    if (lane < kLanes) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 q = unpack2(sum[i]);
        const int at = next.expert(l, 2 * i);
        if (at < E) sh[warp * E + at] = q.x;
        if (at + 1 < E) sh[warp * E + at + 1] = q.y;
      }
    }
    __syncthreads();
    float* part = static_cast<float*>(a.work) + ((int64_t)run + s) * part_words(E);
    for (int i = tid; i < E + 2; i += kWarps * 32) {
      reinterpret_cast<int32_t*>(part)[E + i] = hist[i];
      if (i >= E) continue;
      float all = sh[i];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all += sh[w * E + i];
      part[i] = all;
    }
    __syncthreads();
  }
}

// A cluster a sequence, its experts dealt over the blocks: the parts in their
// order, then gains, and the blocks' shares of the loss in theirs.  Bound by its chain
// of loads and the exchange at its end, 4 us for one sequence of 128 parts; its launch
// overlaps the kernel before.
constexpr int kSumBlocks = 8, kSumThreads = 512;      // of a cluster, at most
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(const BalanceArgs a, int32_t chunk) {
  __shared__ float sums[kSumThreads];
  __shared__ int32_t counts[kSumThreads];
  __shared__ float red[kSumThreads / 32], losses[kSumBlocks];
  __shared__ int32_t tokens[kSumThreads / 32], choices[kSumThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive_relaxed();                  // this block runs: the others may write to it
  const int32_t C = cluster_size(), s = (int32_t)blockIdx.x / C, rank = (int32_t)cluster_ctarank(), E = a.E;
  const int32_t per = (E + C - 1) / C, e0 = rank * per, mine = max(min(per, E - e0), 0);
  const int32_t groups = kSumThreads / per;
  int32_t b = 0, e = a.T;
  if (a.seqs != nullptr) {
    b = a.seqs[s];
    e = a.seqs[s + 1];
    if (b < 0 || e < b || e > a.T) {
      if (tid == 0 && rank == 0) set_status(a.status, MG_ERR_DEVICE_ARG);
      b = e = 0;
    }
  }
  const int32_t p0 = b / chunk, p1 = e > b ? (e - 1) / chunk + 1 : p0;
  const int64_t words = part_words(E);
  const float* parts = static_cast<const float*>(a.work) + (int64_t)s * words;      // part p of this sequence
  // behind nothing that is written, and while the kernel before runs: with release, or
  // just before the blocks' loss, 0.1 to 0.3 us of 8.5
  __syncwarp();
  cluster_wait();
  // the bounds were there before the kernel that writes the parts
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int32_t tok = 0, cho = 0;
  for (int32_t p = p0 + tid; p < p1; p += kSumThreads) {
    const int32_t* q = reinterpret_cast<const int32_t*>(parts + p * words) + 2 * E;
    tok += q[0];
    cho += q[1];
  }
  const int32_t g = tid / per, i = tid - g * per;
  float sum = 0.0f;
  int32_t n = 0;
  if (i < mine && g < groups) {
    const float* q = parts + e0 + i;
#pragma unroll 8
    for (int32_t p = p0 + g; p < p1; p += groups) {
      sum += q[p * words];
      n += reinterpret_cast<const int32_t*>(q)[p * words + E];
    }
  }
  sums[tid] = sum;
  counts[tid] = n;
  tok = __reduce_add_sync(kAll, tok);
  cho = __reduce_add_sync(kAll, cho);
  if (lane == 0) {
    tokens[warp] = tok;
    choices[warp] = cho;
  }
  __syncthreads();
  float loss = 0.0f;
  if (tid < mine) {
#pragma unroll 8
    for (int32_t h = 1; h < groups; ++h) {
      sum += sums[h * per + tid];
      n += counts[h * per + tid];
    }
    tok = cho = 0;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) {
      tok += tokens[w];
      cho += choices[w];
    }
    const float over = (float)cho * (float)tok;
    const float gain = over > 0.0f ? __fdiv_rn(a.coef * (float)E, over) * (float)n : 0.0f;
    a.counts[(int64_t)s * E + e0 + tid] = n;
    a.gain[(int64_t)s * E + e0 + tid] = gain;
    loss = gain * sum;
  }
  loss = warp_sum(loss);
  if (lane == 0) red[warp] = loss;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kSumThreads / 32; ++w) loss += red[w];
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(losses + rank), 0)), "f"(loss) : "memory");
  }
  __syncwarp();
  cluster_sync();
  if (rank == 0 && tid == 0) {
    loss = losses[0];
    for (int r = 1; r < C; ++r) loss += losses[r];
    a.loss[s] = loss;
  }
}

// A warp takes a run of tokens, the next one's rows on their way, and keeps the
// gains of the sequence it is in.  65536 tokens of 256 experts on top of another
// gradient, fp32, 36.5 us (200 MB, 5.5 TB/s): memory, and a warp's chain a token; 8191 of
// 160 in bf16 5.0 us.
constexpr int kBwdWarps = 8;
template <int V, int kLanes, typename L>
__global__ void __launch_bounds__(kBwdWarps * 32) balance_bwd_kernel(const BalanceBwdArgs a, int32_t run) {
  constexpr int kTok = 32 / kLanes;          // tokens a warp at once
  const int lane = threadIdx.x & 31, l = lane & (kLanes - 1);
  const int64_t w = (int64_t)blockIdx.x * kBwdWarps + (threadIdx.x >> 5);
  const int32_t E = a.E, u0 = (int32_t)min(w * run, (int64_t)a.T);
  const int32_t u1 = (int32_t)min((w + 1) * run, (int64_t)a.T);
  if (u0 >= u1) return;
  int32_t t = u0 + lane / kLanes;
  using R = Row<V, kLanes, L>;
  constexpr int kStages = kStagesOf<V, L>;
  extern __shared__ uint4 raw[];             // each warp's rows of the logits, and of `add`
  const int two = a.add != nullptr ? 2 : 1;
  const uint32_t ring = smem_u32(raw) + (threadIdx.x >> 5) * (kStages * two * R::kStage) + lane * R::kPiece;
  const L* row = static_cast<const L*>(a.logits) + (int64_t)t * a.ld;
  const L* other = static_cast<const L*>(a.add) + (int64_t)t * a.lda;
  L* out = static_cast<L*>(a.dlogits) + (int64_t)t * a.ldd;
  R next(no_expert<L>()), add(0u);
  int32_t ahead_t = t, ahead_s = 0, at = 0;
  auto ahead = [&]() {
    if (a.vec && ahead_t < u1) {
      R::copy(ring + ahead_s * two * R::kStage, row, E, l);
      if (two == 2) R::copy(ring + (ahead_s * 2 + 1) * R::kStage, other, E, l);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead_t += kTok;
    row += kTok * a.ld;
    other += kTok * a.lda;
    ahead_s = ahead_s + 1 == kStages ? 0 : ahead_s + 1;
  };
#pragma unroll
  for (int i = 1; i < kStages; ++i) ahead();
  // the warp's first token's sequence, then each token's own: -1 before the first, S
  // behind the last; and its end
  int32_t s = sequence_at(a.seqs, a.S, a.T, u0, lane), end = bound(a.seqs, s + 1 < a.S ? s + 1 : a.S, a.T);
  uint64_t gain[V / 2] = {};
  bool fresh = true;
  for (int32_t u = u0; u < u1; u += kTok) {        // the same for all lanes
    while (t >= end && s < a.S && t < u1) {
      ++s;
      end = s < a.S ? bound(a.seqs, s + 1, a.T) : a.T;
      fresh = true;
    }
    const bool there = t < u1 && s >= 0 && s < a.S;
    if (fresh && there) {
      const float d = __ldg(a.dloss + s);
      const float* g = a.gain + (int64_t)s * E;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const int at = next.expert(l, 2 * i);
        gain[i] = pack2(at < E ? d * __ldg(g + at) : 0.0f, at + 1 < E ? d * __ldg(g + at + 1) : 0.0f);
      }
      fresh = false;
    }
    float x[V], y[V];
    if (a.vec) {
      cp_async_wait<kStages - 2>();
      if (t < u1) {
        next.read(ring + at * two * R::kStage, E, l);
        if (two == 2) add.read(ring + (at * 2 + 1) * R::kStage, E, l);
      }
      ahead();                               // into the stage that was read a round ago
      at = at + 1 == kStages ? 0 : at + 1;
    } else if (t < u1) {
      next.fetch(static_cast<const L*>(a.logits) + (int64_t)t * a.ld, E, l);
      if (two == 2) add.fetch(static_cast<const L*>(a.add) + (int64_t)t * a.lda, E, l);
    }
    next.get(x);
    add.get(y);
    t += kTok;
    uint64_t v[V / 2], rest[V / 2], dot = 0;
    bool some;
    const float inv = scores<V, kLanes, true>(x, a.softmax, v, rest, some, there ? a.status : nullptr);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dot = fma2(v[i], gain[i], dot);
    const float2 q = unpack2(dot);
    const float along = -warp_sum<kLanes>(q.x + q.y) * inv;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      uint64_t p = mul2(v[i], pack2(inv, inv));
      if (!a.softmax) p = mul2(p, rest[i]);
      const float2 r = unpack2(fma2(p, add2(gain[i], pack2(along, along)), pack2(y[2 * i], y[2 * i + 1])));
      x[2 * i] = r.x;
      x[2 * i + 1] = r.y;
    }
    if (there) {
      Row<V, kLanes, L> row_out;
      row_out.set(x);
      row_out.store(out, E, a.vec, l);
    }
    out += kTok * a.ldd;
  }
  cp_async_wait<0>();
}

// All of an SM's shared memory, once a device.
template <auto kKernel>
cudaError_t allow_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev].load()) {
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess && dev < 64) done[dev].store(true);
  }
  return e;
}

// Rows of whole words of four experts.
template <typename L>
bool fours(const void* p, int64_t ld, int32_t E) {
  return p == nullptr || (E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(L)) == 0);
}

template <int V, int kLanes, typename L>
cudaError_t launch_as(BalanceArgs a, cudaStream_t s) {
  constexpr int kWarps = warps_of(V * kLanes);
  a.vec = fours<L>(a.logits, a.ld, a.E);
  const Runs runs = runs_of(a.T, a.E, a.S);
  constexpr auto kernel = balance_kernel<V, kLanes, L, kWarps>;
  const size_t smem = kWarps * kStagesOf<V, L> * Row<V, kLanes, L>::kStage + ((size_t)kWarps * a.E + a.E + 2) * 4;
  if (runs.count > 0) {
    const cudaError_t ready = allow_smem<kernel>();
    if (ready != cudaSuccess) return ready;
    const int64_t grid = runs.split ? (int64_t)runs.count + a.S - 1 : runs.count;
    kernel<<<(unsigned)grid, kWarps * 32, smem, s>>>(a, runs.tokens, runs.split);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  // fewer parts a sequence, fewer blocks (24 sequences of 65536 tokens 20.7, 20.6 and
  // 20.7 us with 8, 4 and 2, 3 of them 20.6, 21.3 and 22.4, 64 of 1066 11.2, 8.3 and
  // 7.9, 2000 of 65536 194, 126 and 95)
  const int C = a.S <= 4 ? kSumBlocks : a.S < 128 ? 4 : 2;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(a.S * C));
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = runs.count > 0 ? 2 : 1;              // the bounds are read early, behind no kernel but the one above
  return cudaLaunchKernelEx(&cfg, balance_sum_kernel, a, runs.tokens);
}

template <int V, int kLanes, typename L>
cudaError_t launch_bwd_as(BalanceBwdArgs a, cudaStream_t s) {
  a.vec = fours<L>(a.logits, a.ld, a.E) && fours<L>(a.dlogits, a.ldd, a.E) && fours<L>(a.add, a.lda, a.E);
  constexpr int kTok = 32 / kLanes;
  // Runs for 32 warps an SM.  Fewer run at once from 33 experts on, by the registers: 24 up
  // to 128 and in fp32 from 193 to 256, 16 up to 384 (bf16 512), 8 above, so that the blocks
  // go in 1.3 to 4 rounds.
  const int64_t warps = (int64_t)num_sms_current_device() * 32, each = warps * kTok;
  const int32_t run = (int32_t)((a.T + each - 1) / each) * kTok;
  const int64_t need = ((int64_t)a.T + run - 1) / run;
  constexpr auto kernel = balance_bwd_kernel<V, kLanes, L>;
  const cudaError_t ready = allow_smem<kernel>();
  if (ready != cudaSuccess) return ready;
  const size_t smem = kBwdWarps * kStagesOf<V, L> * (a.add != nullptr ? 2 : 1) * Row<V, kLanes, L>::kStage;
  kernel<<<(unsigned)((need + kBwdWarps - 1) / kBwdWarps), kBwdWarps * 32, smem, s>>>(a, run);
  return cudaGetLastError();
}

template <int V, int kLanes, typename L, typename A>
cudaError_t on(const A& a, cudaStream_t s) {
  if constexpr (std::is_same<A, BalanceArgs>::value)
    return launch_as<V, kLanes, L>(a, s);
  else
    return launch_bwd_as<V, kLanes, L>(a, s);
}
template <int V, int kLanes, typename A>
cudaError_t by_type(const A& a, cudaStream_t s) {
  return a.f32 ? on<V, kLanes, float>(a, s) : on<V, kLanes, __nv_bfloat16>(a, s);
}

// Experts a lane and lanes a token: two tokens a warp up to 192 experts, four up to
// 64; up to 256 in bf16, whose rows leave the registers for it (gradient of 65536 x
// 256 20 us, with a token a warp 24; in fp32 43 and 37).
template <typename A>
cudaError_t by_experts(const A& a, cudaStream_t s) {
  if (a.E <= 32) return by_type<4, 8>(a, s);
  if (a.E <= 64) return by_type<8, 8>(a, s);
  if (a.E <= 128) return by_type<8, 16>(a, s);
  if (a.E <= 192) return by_type<12, 16>(a, s);
  if (a.E <= 256 && !a.f32) return on<16, 16, __nv_bfloat16>(a, s);
  if (a.E <= 256) return by_type<8, 32>(a, s);
  if (a.E <= 384) return by_type<12, 32>(a, s);
  if (a.E <= 512) return by_type<16, 32>(a, s);
  return by_type<32, 32>(a, s);
}

}  // namespace balance

int64_t balance_work_bytes(int64_t T, int32_t E, int64_t S) {
  return (balance::runs_of(T, E, S).count + S) * balance::part_words(E) * 4;
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) { return balance::by_experts(a, s); }
cudaError_t launch_balance_bwd(const BalanceBwdArgs& a, cudaStream_t s) { return balance::by_experts(a, s); }

}  // namespace mg
