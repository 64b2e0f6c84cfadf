// C ABI of the operators around the grouped GEMMs (declared in
// include/moegemm.h): argument checks and launches.
#include <cmath>
#include <cstdint>

#include "moegemm.h"
#include "ops_internal.h"

using namespace mg;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
mg_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MG_OK : MG_ERR_CUDA; }
constexpr int64_t kInt32End = int64_t(1) << 31;

// Sizes shared by the calls on [T, k] choices; T = 0 is valid.
mg_status check_choices(int32_t T, int32_t k) {
  if (T < 0 || k <= 0) return MG_ERR_INVALID_ARG;
  if (k > kMaxTopK || (int64_t)T * k >= kInt32End) return MG_ERR_UNSUPPORTED;
  return MG_OK;
}

mg_status check_route(mg_elem lt, const void* logits, int64_t ld, int32_t T, int32_t E, int32_t k,
                      mg_route_score score) {
  if (lt != MG_ELEM_BF16 && lt != MG_ELEM_F32) return MG_ERR_INVALID_ARG;
  if (score != MG_ROUTE_SOFTMAX && score != MG_ROUTE_SIGMOID) return MG_ERR_INVALID_ARG;
  const mg_status st = check_choices(T, k);
  if (st != MG_OK) return st;
  if (E <= 0 || k > E || ld < E) return MG_ERR_INVALID_ARG;
  if (E > kMaxExperts) return MG_ERR_UNSUPPORTED;
  if (T > 0 && logits == nullptr) return MG_ERR_INVALID_ARG;
  if (!aligned(logits, lt == MG_ELEM_F32 ? 4 : 2)) return MG_ERR_INVALID_ARG;
  return MG_OK;
}

mg_status check_slots(SlotArgs& a, const int32_t* d_idx, int32_t T, int32_t k, int32_t E, int32_t* d_rows,
                      int32_t* d_counts, int32_t* d_src, void* d_work, int64_t work_bytes, int32_t* d_status) {
  const mg_status st = check_choices(T, k);
  if (st != MG_OK) return st;
  if (E <= 0 || d_counts == nullptr || (T > 0 && (d_idx == nullptr || d_rows == nullptr)))
    return MG_ERR_INVALID_ARG;
  if (E > kMaxExperts || (int64_t)T * k > kMaxSlots) return MG_ERR_UNSUPPORTED;
  if (!aligned(d_idx, 4) || !aligned(d_rows, 4) || !aligned(d_counts, 16) || !aligned(d_src, 4) ||
      !aligned(d_work, 4))
    return MG_ERR_INVALID_ARG;
  a.n = (int64_t)T * k;
  const int64_t need = moe_slots_work_bytes(a.n, E);
  if (need > 0 && (d_work == nullptr || work_bytes < need)) return MG_ERR_INVALID_ARG;
  a.idx = d_idx;
  a.E = E;
  a.rows = d_rows;
  a.counts = d_counts;
  a.src = d_src;
  a.work = static_cast<int32_t*>(d_work);
  a.status = d_status;
  return MG_OK;
}

// The map's blocks read choices and counts that others do not write yet, and
// write without waiting for them: no two buffers may share a byte.
mg_status check_disjoint(const SlotArgs& a) {
  const struct {
    const void* p;
    int64_t bytes;
  } b[] = {{a.idx, 4 * a.n},
           {a.rows, 4 * a.n},
           {a.counts, 4 * (int64_t)a.E},
           {a.src, 4 * a.rows_total},
           {a.work, moe_slots_work_bytes(a.n, a.E)}};
  constexpr int n = sizeof(b) / sizeof(b[0]);
  for (int i = 0; i < n; ++i) {
    for (int j = i + 1; j < n; ++j) {
      if (b[i].p == nullptr || b[j].p == nullptr || b[i].bytes == 0 || b[j].bytes == 0) continue;
      const uintptr_t p = reinterpret_cast<uintptr_t>(b[i].p), q = reinterpret_cast<uintptr_t>(b[j].p);
      if (p < q + (uintptr_t)b[j].bytes && q < p + (uintptr_t)b[i].bytes) return MG_ERR_INVALID_ARG;
    }
  }
  return MG_OK;
}

// Row buffers of the GEMM layouts: rows_total rows in groups of group_rows.
mg_status check_rows(int64_t rows_total, int64_t group_rows) {
  if (rows_total <= 0 || rows_total >= kInt32End || group_rows <= 0 || group_rows > rows_total ||
      rows_total % group_rows != 0)
    return MG_ERR_INVALID_ARG;
  return MG_OK;
}

// Arguments of a call from their words, one after another.
struct Record {
  const mg_word* at;
  bool fits = true;                 // every integer so far is one of its argument's type
  int64_t i64() { return (at++)->i; }
  int32_t i32() {
    const int64_t v = i64();
    fits = fits && v == (int32_t)v;
    return (int32_t)v;
  }
  float f32() { return (float)(at++)->d; }
  void* ptr() { return (at++)->p; }
  template <typename K>
  K kind() {
    return static_cast<K>(i32());
  }
};

// Row types of the norm.
bool row_elem(mg_elem t) { return t == MG_ELEM_BF16 || t == MG_ELEM_F32; }

mg_status check_norm(int32_t T, int32_t K, float eps) {
  if (T < 0 || K <= 0 || !(eps > 0.0f) || !std::isfinite(eps)) return MG_ERR_INVALID_ARG;
  if (K % 8 != 0 || K > kMaxNormK) return MG_ERR_UNSUPPORTED;
  return MG_OK;
}

// Rows of K elements, ld apart, read in whole 16-byte words; null: not there.
mg_status check_row_stride(const void* p, int64_t ld, int32_t K) {
  if (p == nullptr) return MG_OK;
  if (ld < K || !aligned(p, 16)) return MG_ERR_INVALID_ARG;
  return ld % 8 != 0 ? MG_ERR_UNSUPPORTED : MG_OK;
}

// Rows of `bytes` bytes, `apart` of them from one to the next.
struct Rows {
  const void* p;
  int64_t rows, apart, bytes;
};
Rows rows_of(const void* p, int64_t rows, int64_t ld, int64_t columns, int size) {
  return {p, rows, ld < int64_t(1) << 56 ? ld * size : INT64_MAX, columns * size};
}

// Whether two buffers share a byte in their rows; what lies between the rows (another
// buffer's columns, say) does not count.
bool share_bytes(const Rows& a, const Rows& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0 || a.bytes == 0 || b.bytes == 0) return false;
  using wide = __int128;                   // rows times their stride may pass 64 bits
  const wide p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
  const wide p_end = p + (wide)(a.rows - 1) * a.apart + a.bytes, q_end = q + (wide)(b.rows - 1) * b.apart + b.bytes;
  if (p_end <= q || q_end <= p) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.apart == b.apart) {
    // row i of b begins `at` bytes, less than a stride, behind row i + k of a
    wide k = (q - p) / a.apart, at = (q - p) % a.apart;
    if (at < 0) {
      at += a.apart;
      --k;
    }
    const auto meet = [&](wide d) { return d > -(wide)b.rows && d < a.rows; };       // some row i, and i + d of a
    return (at < a.bytes && meet(k)) || (at + b.bytes > a.apart && meet(k + 1));
  }
  // strides of their own: the rows of b that reach into a's range, one after another
  wide i = q < p ? (p - q) / b.apart : 0;
  for (; i < b.rows && q + i * b.apart < p_end; ++i) {
    const wide from = q + i * b.apart, to = from + b.bytes;
    for (wide j = from < p ? 0 : (from - p) / a.apart; j < a.rows && p + j * a.apart < to; ++j)
      if (p + j * a.apart + a.bytes > from) return true;
  }
  return false;
}

Rows flat(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Outputs over bytes of an input.  Row buffers may be written in place: a row's reader
// writes it.
template <int kOut, int kIn>
bool overwrites(const Rows (&out)[kOut], const Rows (&in)[kIn]) {
  for (const Rows& o : out)
    for (const Rows& i : in)
      if (share_bytes(o, i)) return true;
  return false;
}
template <int kOut, int kIn>
bool overwrites_rows(const Rows (&out)[kOut], const Rows (&in)[kIn]) {
  for (const Rows& o : out) {
    for (const Rows& i : in) {
      const bool in_place = o.p == i.p && o.bytes == i.bytes && (o.apart == i.apart || o.rows == 1);
      if (!in_place && share_bytes(o, i)) return true;
    }
  }
  return false;
}

// S packed sequences of T tokens with a result of E values each.  A warp's walk steps
// past T by less than 4096.
mg_status check_sequences(const int32_t* seqs, int32_t S, int32_t E, int32_t T) {
  if (S <= 0 || (seqs == nullptr && S != 1) || !aligned(seqs, 4)) return MG_ERR_INVALID_ARG;
  return (int64_t)S * E >= kInt32End || S > (1 << 27) || T > kInt32End - 4096 ? MG_ERR_UNSUPPORTED : MG_OK;
}

}  // namespace

extern "C" {

mg_status moe_route(mg_elem lt, const void* d_logits, int64_t ld, const float* d_bias, int32_t T, int32_t E,
                    int32_t k, mg_route_score score, int32_t groups, int32_t top_groups, int32_t group_top,
                    int32_t renorm, float scale, int32_t* d_idx, float* d_w, int32_t* d_status, void* stream) {
  const mg_status st = check_route(lt, d_logits, ld, T, E, k, score);
  if (st != MG_OK) return st;
  if (groups <= 0 || top_groups <= 0 || top_groups > groups || E % groups != 0) return MG_ERR_INVALID_ARG;
  if (group_top != 1 && group_top != 2) return MG_ERR_INVALID_ARG;
  if (groups > kMaxGroups) return MG_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return MG_ERR_INVALID_ARG;
  if (T == 0) return MG_OK;
  if (d_idx == nullptr || d_w == nullptr) return MG_ERR_INVALID_ARG;
  if (!aligned(d_bias, 4) || !aligned(d_idx, 4) || !aligned(d_w, 4)) return MG_ERR_INVALID_ARG;
  RouteArgs a;
  a.logits = d_logits;
  a.ld = ld;
  a.bias = d_bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.groups = groups;
  a.top_groups = top_groups;
  a.group_top = group_top;
  a.f32 = lt == MG_ELEM_F32;
  a.softmax = score == MG_ROUTE_SOFTMAX;
  a.renorm = renorm != 0;
  a.scale = scale;
  a.idx = d_idx;
  a.w = d_w;
  a.status = d_status;
  return from_cuda(launch_route(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_route_backward(mg_elem lt, const void* d_logits, int64_t ld, const int32_t* d_idx,
                             const float* d_dw, int32_t T, int32_t E, int32_t k, mg_route_score score,
                             int32_t renorm, float scale, void* d_dlogits, int64_t ldd, int32_t* d_status,
                             void* stream) {
  const mg_status st = check_route(lt, d_logits, ld, T, E, k, score);
  if (st != MG_OK) return st;
  if (ldd < E || !std::isfinite(scale)) return MG_ERR_INVALID_ARG;
  if (T == 0) return MG_OK;
  if (d_idx == nullptr || d_dw == nullptr || d_dlogits == nullptr) return MG_ERR_INVALID_ARG;
  if (!aligned(d_idx, 4) || !aligned(d_dw, 4) || !aligned(d_dlogits, lt == MG_ELEM_F32 ? 4 : 2))
    return MG_ERR_INVALID_ARG;
  RouteBwdArgs a;
  a.logits = d_logits;
  a.ld = ld;
  a.idx = d_idx;
  a.dw = d_dw;
  a.T = T;
  a.E = E;
  a.k = k;
  a.f32 = lt == MG_ELEM_F32;
  a.softmax = score == MG_ROUTE_SOFTMAX;
  a.renorm = renorm != 0;
  a.scale = scale;
  a.dlogits = d_dlogits;
  a.ldd = ldd;
  a.status = d_status;
  return from_cuda(launch_route_bwd(a, static_cast<cudaStream_t>(stream)));
}

int64_t moe_slots_work_bytes(int64_t n, int32_t E) {
  if (n <= kSlotChunk || E <= 0) return 0;
  return (n + kSlotChunk - 1) / kSlotChunk * E * (int64_t)sizeof(int32_t);
}

mg_status moe_slots_contiguous(const int32_t* d_idx, int32_t T, int32_t k, int32_t E, int32_t align_q,
                               int64_t rows_cap, int32_t* d_rows, int32_t* d_counts, int32_t* d_src,
                               void* d_work, int64_t work_bytes, int32_t* d_status, void* stream) {
  SlotArgs a;
  const mg_status st = check_slots(a, d_idx, T, k, E, d_rows, d_counts, d_src, d_work, work_bytes, d_status);
  if (st != MG_OK) return st;
  if (align_q <= 0 || rows_cap <= 0 || rows_cap >= kInt32End) return MG_ERR_INVALID_ARG;
  a.masked = false;
  a.align_q = align_q;
  a.rows_total = rows_cap;
  if (check_disjoint(a) != MG_OK) return MG_ERR_INVALID_ARG;
  return from_cuda(launch_slots(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_slots_masked(const int32_t* d_idx, int32_t T, int32_t k, int32_t E, int32_t M_max, int32_t* d_rows,
                           int32_t* d_counts, int32_t* d_src, void* d_work, int64_t work_bytes,
                           int32_t* d_status, void* stream) {
  SlotArgs a;
  const mg_status st = check_slots(a, d_idx, T, k, E, d_rows, d_counts, d_src, d_work, work_bytes, d_status);
  if (st != MG_OK) return st;
  if (M_max <= 0 || (int64_t)E * M_max >= kInt32End) return MG_ERR_INVALID_ARG;
  a.masked = true;
  a.M_max = M_max;
  a.rows_total = (int64_t)E * M_max;
  if (check_disjoint(a) != MG_OK) return MG_ERR_INVALID_ARG;
  return from_cuda(launch_slots(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_dispatch(mg_elem xt, const void* d_X, int64_t ldx, const uint8_t* d_SX, const int32_t* d_rows,
                       int32_t T, int32_t k, int32_t K, mg_elem at, void* d_A, uint8_t* d_SFA,
                       int64_t rows_total, int64_t group_rows, uint8_t* d_CX, uint8_t* d_SCX,
                       int32_t* d_status, void* stream) {
  if ((xt != MG_ELEM_BF16 && xt != MG_ELEM_E4M3) || (at != MG_ELEM_BF16 && at != MG_ELEM_E4M3))
    return MG_ERR_INVALID_ARG;
  mg_status st = check_choices(T, k);
  if (st != MG_OK) return st;
  st = check_rows(rows_total, group_rows);
  if (st != MG_OK) return st;
  const bool xq = xt == MG_ELEM_E4M3, aq = at == MG_ELEM_E4M3, ckpt = d_CX != nullptr;
  if (K <= 0 || ldx < K || (d_CX != nullptr) != (d_SCX != nullptr)) return MG_ERR_INVALID_ARG;
  if (ckpt && xq) return MG_ERR_INVALID_ARG;             // the source is a checkpoint already
  if (K % (xq || aq || ckpt ? 128 : 8) != 0 || ldx % (xq ? 16 : 8) != 0) return MG_ERR_UNSUPPORTED;
  if ((int64_t)K > (int64_t(1) << 24)) return MG_ERR_UNSUPPORTED;
  if (T == 0) return MG_OK;
  if (d_X == nullptr || d_rows == nullptr || d_A == nullptr || (xq && d_SX == nullptr) || (aq && d_SFA == nullptr))
    return MG_ERR_INVALID_ARG;
  if (!aligned(d_X, 16) || !aligned(d_A, 16) || !aligned(d_CX, 16) || !aligned(d_rows, 4)) return MG_ERR_INVALID_ARG;
  DispatchArgs a;
  a.X = d_X;
  a.ldx = ldx;
  a.SX = d_SX;
  a.rows = d_rows;
  a.T = T;
  a.k = k;
  a.K = K;
  a.src_e4m3 = xq;
  a.dst_e4m3 = aq;
  a.A = d_A;
  a.SFA = d_SFA;
  a.rows_total = rows_total;
  a.group_rows = group_rows;
  a.CX = d_CX;
  a.SCX = d_SCX;
  a.status = d_status;
  return from_cuda(launch_dispatch(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_combine(const void* d_D, const int32_t* d_rows, const float* d_w, int32_t T, int32_t k, int32_t K,
                      int64_t rows_total, mg_elem ot, void* d_out, int64_t ldo, int32_t* d_status, void* stream) {
  if (ot != MG_ELEM_BF16 && ot != MG_ELEM_F32) return MG_ERR_INVALID_ARG;
  mg_status st = check_choices(T, k);
  if (st != MG_OK) return st;
  st = check_rows(rows_total, rows_total);
  if (st != MG_OK) return st;
  if (K <= 0 || ldo < K) return MG_ERR_INVALID_ARG;
  if (K % 8 != 0 || ldo % 8 != 0 || (int64_t)K > (int64_t(1) << 24)) return MG_ERR_UNSUPPORTED;
  if (T == 0) return MG_OK;
  if (d_D == nullptr || d_rows == nullptr || d_out == nullptr) return MG_ERR_INVALID_ARG;
  if (!aligned(d_D, 16) || !aligned(d_out, 16) || !aligned(d_rows, 4) || !aligned(d_w, 4)) return MG_ERR_INVALID_ARG;
  CombineArgs a;
  a.D = d_D;
  a.rows = d_rows;
  a.w = d_w;
  a.T = T;
  a.k = k;
  a.K = K;
  a.rows_total = rows_total;
  a.f32 = ot == MG_ELEM_F32;
  a.out = d_out;
  a.ldo = ldo;
  a.status = d_status;
  return from_cuda(launch_combine(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_combine_backward(mg_elem gt, const void* d_dout, int64_t ldd, const void* d_D, const int32_t* d_rows,
                               const float* d_w, int32_t T, int32_t k, int32_t K, int64_t rows_total, void* d_dD,
                               float* d_dw, int32_t* d_status, void* stream) {
  if (gt != MG_ELEM_BF16 && gt != MG_ELEM_F32) return MG_ERR_INVALID_ARG;
  mg_status st = check_choices(T, k);
  if (st != MG_OK) return st;
  st = check_rows(rows_total, rows_total);
  if (st != MG_OK) return st;
  if (K <= 0 || ldd < K || (d_D != nullptr) != (d_dw != nullptr)) return MG_ERR_INVALID_ARG;
  if (K % 8 != 0 || ldd % 8 != 0 || (int64_t)K > (int64_t(1) << 24)) return MG_ERR_UNSUPPORTED;
  if (T == 0) return MG_OK;
  if (d_dout == nullptr || d_rows == nullptr || d_dD == nullptr) return MG_ERR_INVALID_ARG;
  if (!aligned(d_dout, 16) || !aligned(d_D, 16) || !aligned(d_dD, 16) || !aligned(d_rows, 4) || !aligned(d_w, 4) ||
      !aligned(d_dw, 4))
    return MG_ERR_INVALID_ARG;
  CombineBwdArgs a;
  a.dout = d_dout;
  a.ldd = ldd;
  a.f32 = gt == MG_ELEM_F32;
  a.D = d_D;
  a.rows = d_rows;
  a.w = d_w;
  a.T = T;
  a.k = k;
  a.K = K;
  a.rows_total = rows_total;
  a.dD = d_dD;
  a.dw = d_dw;
  a.status = d_status;
  return from_cuda(launch_combine_bwd(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_swiglu_save(const void* d_H, int64_t rows_total, int64_t group_rows, int32_t N, const int32_t* d_src,
                          mg_swiglu_out out, void* d_Y, uint8_t* d_SFY, uint8_t* d_HC, uint8_t* d_SHC,
                          void* stream) {
  if (out != MG_SWIGLU_BF16 && out != MG_SWIGLU_FP8_E4M3_UE8M0) return MG_ERR_INVALID_ARG;
  const mg_status st = check_rows(rows_total, group_rows);
  if (st != MG_OK) return st;
  if (N <= 0) return MG_ERR_INVALID_ARG;
  if (N % 256 != 0 || N > (1 << 24)) return MG_ERR_UNSUPPORTED;
  const bool q = out == MG_SWIGLU_FP8_E4M3_UE8M0;
  if (d_H == nullptr || d_Y == nullptr || d_HC == nullptr || d_SHC == nullptr || (q && d_SFY == nullptr))
    return MG_ERR_INVALID_ARG;
  if (!aligned(d_H, 16) || !aligned(d_Y, 16) || !aligned(d_HC, 16) || !aligned(d_SHC, 2) || !aligned(d_src, 4))
    return MG_ERR_INVALID_ARG;
  SwigluSaveArgs a;
  a.H = d_H;
  a.rows_total = rows_total;
  a.group_rows = group_rows;
  a.N = N;
  a.src = d_src;
  a.y_e4m3 = q;
  a.Y = d_Y;
  a.SFY = d_SFY;
  a.HC = d_HC;
  a.SHC = d_SHC;
  return from_cuda(launch_swiglu_save(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_swiglu_backward(const void* d_dY, const uint8_t* d_HC, const uint8_t* d_SHC, int64_t rows_total,
                              int32_t N, const int32_t* d_src, const float* d_w, int64_t n, void* d_dH, void* d_Y,
                              float* d_dw, int32_t* d_status, void* stream) {
  const mg_status st = check_rows(rows_total, rows_total);
  if (st != MG_OK) return st;
  if (N <= 0 || n < 0) return MG_ERR_INVALID_ARG;
  if (N % 256 != 0 || N > (1 << 24)) return MG_ERR_UNSUPPORTED;
  if (d_dY == nullptr || d_HC == nullptr || d_SHC == nullptr || d_dH == nullptr) return MG_ERR_INVALID_ARG;
  if ((d_w != nullptr || d_dw != nullptr) && d_src == nullptr) return MG_ERR_INVALID_ARG;
  if (!aligned(d_dY, 16) || !aligned(d_HC, 16) || !aligned(d_SHC, 2) || !aligned(d_dH, 16) || !aligned(d_Y, 16) ||
      !aligned(d_src, 4) || !aligned(d_w, 4) || !aligned(d_dw, 4))
    return MG_ERR_INVALID_ARG;
  SwigluBwdArgs a;
  a.dY = d_dY;
  a.HC = d_HC;
  a.SHC = d_SHC;
  a.rows_total = rows_total;
  a.N = N;
  a.src = d_src;
  a.w = d_w;
  a.n = n;
  a.dH = d_dH;
  a.Y = d_Y;
  a.dw = d_dw;
  a.status = d_status;
  return from_cuda(launch_swiglu_bwd(a, static_cast<cudaStream_t>(stream)));
}

int64_t moe_norm_work_bytes(int32_t T, int32_t K) { return T <= 0 || K <= 0 ? 0 : norm_work_bytes(T, K); }

mg_status moe_norm(mg_elem xt, const void* d_X, int64_t ldx, mg_elem st, const void* d_R, int64_t ldr, mg_elem wt,
                   const void* d_w, float eps, int32_t T, int32_t K, void* d_H, int64_t ldh, void* d_Y, int64_t ldy,
                   uint8_t* d_Q, uint8_t* d_SQ, int64_t sq_rows, float* d_rstd, void* stream) {
  if (!row_elem(xt) || !row_elem(st) || !row_elem(wt)) return MG_ERR_INVALID_ARG;
  const bool quant = d_Q != nullptr;
  if ((d_Q != nullptr) != (d_SQ != nullptr) || (d_H != nullptr && d_R == nullptr)) return MG_ERR_INVALID_ARG;
  mg_status rs = check_norm(T, K, eps);
  if (rs != MG_OK) return rs;
  if (quant && K % 128 != 0) return MG_ERR_UNSUPPORTED;
  if (sq_rows < 0 || (quant && sq_rows > 0 && sq_rows < T)) return MG_ERR_INVALID_ARG;
  if (T == 0) return MG_OK;
  if (d_X == nullptr || d_w == nullptr || (d_H == nullptr && d_Y == nullptr && !quant && d_rstd == nullptr))
    return MG_ERR_INVALID_ARG;
  rs = check_row_stride(d_X, ldx, K);
  if (rs == MG_OK) rs = check_row_stride(d_R, ldr, K);
  if (rs == MG_OK) rs = check_row_stride(d_H, ldh, K);
  if (rs == MG_OK) rs = check_row_stride(d_Y, ldy, K);
  if (rs != MG_OK) return rs;
  if (!aligned(d_w, 16) || !aligned(d_Q, 16) || !aligned(d_rstd, 4)) return MG_ERR_INVALID_ARG;
  const int xb = xt == MG_ELEM_F32 ? 4 : 2, sb = st == MG_ELEM_F32 ? 4 : 2, wb = wt == MG_ELEM_F32 ? 4 : 2;
  const Rows in[] = {rows_of(d_X, T, ldx, K, xb), rows_of(d_R, T, ldr, K, sb)}, weight[] = {flat(d_w, (int64_t)K * wb)};
  const Rows out[] = {rows_of(d_H, T, ldh, K, sb), rows_of(d_Y, T, ldy, K, 2), rows_of(d_Q, T, K, K, 1)};
  const Rows root[] = {flat(d_rstd, (int64_t)T * 4)};
  if (overwrites_rows(out, in) || overwrites(out, weight) || overwrites(root, in) || overwrites(root, weight))
    return MG_ERR_INVALID_ARG;
  NormArgs a;
  a.X = d_X;
  a.ldx = ldx;
  a.x_f32 = xt == MG_ELEM_F32;
  a.R = d_R;
  a.ldr = ldr;
  a.s_f32 = st == MG_ELEM_F32;
  a.w = d_w;
  a.w_f32 = wt == MG_ELEM_F32;
  a.eps = eps;
  a.T = T;
  a.K = K;
  a.H = d_H;
  a.ldh = ldh;
  a.Y = d_Y;
  a.ldy = ldy;
  a.Q = d_Q;
  a.SQ = d_SQ;
  a.sq_rows = sq_rows;
  a.rstd = d_rstd;
  return from_cuda(launch_norm(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_norm_backward(mg_elem gt, const void* d_dY, int64_t ldd, mg_elem st, const void* d_H, int64_t ldh,
                            mg_elem wt, const void* d_w, const float* d_rstd, const void* d_dR, int64_t ldr, int32_t T,
                            int32_t K, void* d_dX, int64_t ldx, float* d_dw, void* d_work, int64_t work_bytes,
                            void* stream) {
  if (!row_elem(gt) || !row_elem(st) || !row_elem(wt)) return MG_ERR_INVALID_ARG;
  mg_status rs = check_norm(T, K, 1.0f);
  if (rs != MG_OK) return rs;
  if (!aligned(d_dw, 4)) return MG_ERR_INVALID_ARG;
  if (T > 0) {
    if (d_dY == nullptr || d_H == nullptr || d_w == nullptr || d_rstd == nullptr || d_dX == nullptr)
      return MG_ERR_INVALID_ARG;
    rs = check_row_stride(d_dY, ldd, K);
    if (rs == MG_OK) rs = check_row_stride(d_H, ldh, K);
    if (rs == MG_OK) rs = check_row_stride(d_dR, ldr, K);
    if (rs == MG_OK) rs = check_row_stride(d_dX, ldx, K);
    if (rs != MG_OK) return rs;
    if (!aligned(d_w, 16) || !aligned(d_rstd, 4) || !aligned(d_work, 16)) return MG_ERR_INVALID_ARG;
    if (d_dw != nullptr && (d_work == nullptr || work_bytes < norm_work_bytes(T, K))) return MG_ERR_INVALID_ARG;
    const int gb = gt == MG_ELEM_F32 ? 4 : 2, sb = st == MG_ELEM_F32 ? 4 : 2, wb = wt == MG_ELEM_F32 ? 4 : 2;
    const int64_t parts = d_dw != nullptr ? norm_work_bytes(T, K) : 0;
    const Rows in[] = {rows_of(d_dY, T, ldd, K, gb), rows_of(d_H, T, ldh, K, sb), rows_of(d_dR, T, ldr, K, sb)};
    const Rows fixed[] = {flat(d_w, (int64_t)K * wb), flat(d_rstd, (int64_t)T * 4)};
    const Rows out[] = {rows_of(d_dX, T, ldx, K, sb)}, sums[] = {flat(d_dw, (int64_t)K * 4), flat(d_work, parts)};
    if (overwrites_rows(out, in) || overwrites(out, fixed) || overwrites(sums, in) || overwrites(sums, fixed))
      return MG_ERR_INVALID_ARG;
  }
  NormBwdArgs a;
  a.dY = d_dY;
  a.ldd = ldd;
  a.g_f32 = gt == MG_ELEM_F32;
  a.H = d_H;
  a.ldh = ldh;
  a.s_f32 = st == MG_ELEM_F32;
  a.w = d_w;
  a.w_f32 = wt == MG_ELEM_F32;
  a.rstd = d_rstd;
  a.dR = d_dR;
  a.ldr = ldr;
  a.T = T;
  a.K = K;
  a.dX = d_dX;
  a.ldx = ldx;
  a.dw = d_dw;
  a.work = static_cast<float*>(d_work);
  return from_cuda(launch_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

int64_t moe_balance_work_bytes(int32_t T, int32_t E, int32_t S) {
  return T < 0 || E <= 0 || S <= 0 ? 0 : balance_work_bytes(T, E, S);
}

mg_status moe_balance(mg_elem lt, const void* d_logits, int64_t ld, const int32_t* d_idx, int32_t T, int32_t E,
                      int32_t k, mg_route_score score, const int32_t* d_seqs, int32_t S, float coef, int32_t* d_counts,
                      float* d_gain, float* d_loss, void* d_work, int64_t work_bytes, int32_t* d_status,
                      void* stream) {
  mg_status st = check_route(lt, d_logits, ld, T, E, k, score);
  if (st != MG_OK) return st;
  st = check_sequences(d_seqs, S, E, T);
  if (st != MG_OK) return st;
  if (!std::isfinite(coef) || (T > 0 && d_idx == nullptr) || d_counts == nullptr || d_gain == nullptr ||
      d_loss == nullptr)
    return MG_ERR_INVALID_ARG;
  if (!aligned(d_idx, 4) || !aligned(d_counts, 4) || !aligned(d_gain, 4) || !aligned(d_loss, 4) || !aligned(d_work, 4))
    return MG_ERR_INVALID_ARG;
  if (d_work == nullptr || work_bytes < balance_work_bytes(T, E, S)) return MG_ERR_INVALID_ARG;
  BalanceArgs a;
  a.logits = d_logits;
  a.ld = ld;
  a.idx = d_idx;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.f32 = lt == MG_ELEM_F32;
  a.softmax = score == MG_ROUTE_SOFTMAX;
  a.seqs = d_seqs;
  a.coef = coef;
  a.counts = d_counts;
  a.gain = d_gain;
  a.loss = d_loss;
  a.work = d_work;
  a.status = d_status;
  return from_cuda(launch_balance(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_balance_backward(mg_elem lt, const void* d_logits, int64_t ld, const float* d_gain,
                               const float* d_dloss, int32_t T, int32_t E, mg_route_score score,
                               const int32_t* d_seqs, int32_t S, const void* d_add, int64_t lda, void* d_dlogits,
                               int64_t ldd, int32_t* d_status, void* stream) {
  mg_status st = check_route(lt, d_logits, ld, T, E, 1, score);
  if (st != MG_OK) return st;
  st = check_sequences(d_seqs, S, E, T);
  if (st != MG_OK) return st;
  if (ldd < E || (d_add != nullptr && lda < E)) return MG_ERR_INVALID_ARG;
  if (T == 0) return MG_OK;
  if (d_gain == nullptr || d_dloss == nullptr || d_dlogits == nullptr) return MG_ERR_INVALID_ARG;
  const int bytes = lt == MG_ELEM_F32 ? 4 : 2;
  if (!aligned(d_gain, 4) || !aligned(d_dloss, 4) || !aligned(d_dlogits, bytes) || !aligned(d_add, bytes))
    return MG_ERR_INVALID_ARG;
  BalanceBwdArgs a;
  a.logits = d_logits;
  a.ld = ld;
  a.gain = d_gain;
  a.dloss = d_dloss;
  a.T = T;
  a.E = E;
  a.S = S;
  a.f32 = lt == MG_ELEM_F32;
  a.softmax = score == MG_ROUTE_SOFTMAX;
  a.seqs = d_seqs;
  a.add = d_add;
  a.lda = lda;
  a.dlogits = d_dlogits;
  a.ldd = ldd;
  a.status = d_status;
  return from_cuda(launch_balance_bwd(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_adapters(const void* d_X, int64_t ldx, const void* d_A, const void* d_B, const float* d_scale,
                       const int32_t* d_idx, const int32_t* d_rows, const int32_t* d_src, int32_t T, int32_t E,
                       int32_t r, int32_t K, int32_t N, int64_t rows_total, int32_t align_q, const void* d_base,
                       int64_t ldb, void* d_Y, int64_t ldy, int32_t* d_status, void* stream) {
  if (T < 0 || E <= 0 || r <= 0 || K <= 0 || N <= 0 || align_q <= 0) return MG_ERR_INVALID_ARG;
  mg_status st = check_rows(rows_total, rows_total);
  if (st != MG_OK) return st;
  if (r % 8 != 0 || r > kMaxRank || K % 8 != 0 || N % 8 != 0 || align_q % 16 != 0) return MG_ERR_UNSUPPORTED;
  if (K > (1 << 24) || N > (1 << 24)) return MG_ERR_UNSUPPORTED;
  if (T == 0) return MG_OK;
  if (d_X == nullptr || d_A == nullptr || d_B == nullptr || d_idx == nullptr || d_rows == nullptr ||
      d_src == nullptr || d_Y == nullptr)
    return MG_ERR_INVALID_ARG;
  st = check_row_stride(d_X, ldx, K);
  if (st == MG_OK) st = check_row_stride(d_Y, ldy, N);
  if (st == MG_OK) st = check_row_stride(d_base, ldb, N);
  if (st != MG_OK) return st;
  if (!aligned(d_A, 16) || !aligned(d_B, 16) || !aligned(d_scale, 4) || !aligned(d_idx, 4) || !aligned(d_rows, 4) ||
      !aligned(d_src, 4) || (d_base == d_Y && ldb != ldy))
    return MG_ERR_INVALID_ARG;
  // blocks read rows of X and base that others' rows of Y would be written over
  const Rows out = rows_of(d_Y, T, ldy, N, 2);
  if (share_bytes(rows_of(d_X, T, ldx, K, 2), out) || (d_base != d_Y && share_bytes(rows_of(d_base, T, ldb, N, 2), out)))
    return MG_ERR_INVALID_ARG;
  AdaptersArgs a;
  a.X = d_X;
  a.ldx = ldx;
  a.A = d_A;
  a.B = d_B;
  a.scale = d_scale;
  a.idx = d_idx;
  a.rows = d_rows;
  a.src = d_src;
  a.T = T;
  a.E = E;
  a.r = r;
  a.K = K;
  a.N = N;
  a.rows_total = rows_total;
  a.align_q = align_q;
  a.base = d_base != nullptr ? d_base : d_Y;
  a.ldb = d_base != nullptr ? ldb : ldy;
  a.Y = d_Y;
  a.ldy = ldy;
  a.status = d_status;
  return from_cuda(launch_adapters(a, static_cast<cudaStream_t>(stream)));
}

mg_status moe_call(mg_call which, const mg_word* words) {
  if (words == nullptr) return MG_ERR_INVALID_ARG;
  Record r{words};
  auto run = [&](auto fn, auto... args) { return r.fits ? fn(args...) : MG_ERR_INVALID_ARG; };
  switch (which) {
    case MG_CALL_NORM: {
      const auto xt = r.kind<mg_elem>();
      const void* X = r.ptr();
      const int64_t ldx = r.i64();
      const auto st = r.kind<mg_elem>();
      const void* R = r.ptr();
      const int64_t ldr = r.i64();
      const auto wt = r.kind<mg_elem>();
      const void* w = r.ptr();
      const float eps = r.f32();
      const int32_t T = r.i32(), K = r.i32();
      void* H = r.ptr();
      const int64_t ldh = r.i64();
      void* Y = r.ptr();
      const int64_t ldy = r.i64();
      auto* Q = static_cast<uint8_t*>(r.ptr());
      auto* SQ = static_cast<uint8_t*>(r.ptr());
      const int64_t sq_rows = r.i64();
      auto* rstd = static_cast<float*>(r.ptr());
      void* stream = r.ptr();
      return run(moe_norm, xt, X, ldx, st, R, ldr, wt, w, eps, T, K, H, ldh, Y, ldy, Q, SQ, sq_rows, rstd, stream);
    }
    case MG_CALL_NORM_BACKWARD: {
      const auto gt = r.kind<mg_elem>();
      const void* dY = r.ptr();
      const int64_t ldd = r.i64();
      const auto st = r.kind<mg_elem>();
      const void* H = r.ptr();
      const int64_t ldh = r.i64();
      const auto wt = r.kind<mg_elem>();
      const void* w = r.ptr();
      auto* rstd = static_cast<const float*>(r.ptr());
      const void* dR = r.ptr();
      const int64_t ldr = r.i64();
      const int32_t T = r.i32(), K = r.i32();
      void* dX = r.ptr();
      const int64_t ldx = r.i64();
      auto* dw = static_cast<float*>(r.ptr());
      void* work = r.ptr();
      const int64_t work_bytes = r.i64();
      void* stream = r.ptr();
      return run(moe_norm_backward, gt, dY, ldd, st, H, ldh, wt, w, rstd, dR, ldr, T, K, dX, ldx, dw, work, work_bytes,
                 stream);
    }
    case MG_CALL_BALANCE: {
      const auto lt = r.kind<mg_elem>();
      const void* logits = r.ptr();
      const int64_t ld = r.i64();
      auto* idx = static_cast<const int32_t*>(r.ptr());
      const int32_t T = r.i32(), E = r.i32(), k = r.i32();
      const auto score = r.kind<mg_route_score>();
      auto* seqs = static_cast<const int32_t*>(r.ptr());
      const int32_t S = r.i32();
      const float coef = r.f32();
      auto* counts = static_cast<int32_t*>(r.ptr());
      auto* gain = static_cast<float*>(r.ptr());
      auto* loss = static_cast<float*>(r.ptr());
      void* work = r.ptr();
      const int64_t work_bytes = r.i64();
      auto* status = static_cast<int32_t*>(r.ptr());
      void* stream = r.ptr();
      return run(moe_balance, lt, logits, ld, idx, T, E, k, score, seqs, S, coef, counts, gain, loss, work, work_bytes,
                 status, stream);
    }
    case MG_CALL_BALANCE_BACKWARD: {
      const auto lt = r.kind<mg_elem>();
      const void* logits = r.ptr();
      const int64_t ld = r.i64();
      auto* gain = static_cast<const float*>(r.ptr());
      auto* dloss = static_cast<const float*>(r.ptr());
      const int32_t T = r.i32(), E = r.i32();
      const auto score = r.kind<mg_route_score>();
      auto* seqs = static_cast<const int32_t*>(r.ptr());
      const int32_t S = r.i32();
      const void* add = r.ptr();
      const int64_t lda = r.i64();
      void* dlogits = r.ptr();
      const int64_t ldd = r.i64();
      auto* status = static_cast<int32_t*>(r.ptr());
      void* stream = r.ptr();
      return run(moe_balance_backward, lt, logits, ld, gain, dloss, T, E, score, seqs, S, add, lda, dlogits, ldd,
                 status, stream);
    }
    case MG_CALL_ADAPTERS: {
      const void* X = r.ptr();
      const int64_t ldx = r.i64();
      const void* A = r.ptr();
      const void* B = r.ptr();
      auto* scale = static_cast<const float*>(r.ptr());
      auto* idx = static_cast<const int32_t*>(r.ptr());
      auto* rows = static_cast<const int32_t*>(r.ptr());
      auto* src = static_cast<const int32_t*>(r.ptr());
      const int32_t T = r.i32(), E = r.i32(), rank = r.i32(), K = r.i32(), N = r.i32();
      const int64_t rows_total = r.i64();
      const int32_t align_q = r.i32();
      const void* base = r.ptr();
      const int64_t ldb = r.i64();
      void* Y = r.ptr();
      const int64_t ldy = r.i64();
      auto* status = static_cast<int32_t*>(r.ptr());
      void* stream = r.ptr();
      return run(moe_adapters, X, ldx, A, B, scale, idx, rows, src, T, E, rank, K, N, rows_total, align_q, base, ldb, Y,
                 ldy, status, stream);
    }
  }
  return MG_ERR_INVALID_ARG;
}

}  // extern "C"
