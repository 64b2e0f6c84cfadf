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

}  // extern "C"
