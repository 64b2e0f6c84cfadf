// Internal host-side interface of the operators around the grouped GEMMs:
// routing, slot map, dispatch, combine, and the 8-bit SwiGLU checkpoint.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mg_internal.h"
#include "moegemm.h"

namespace mg {

constexpr int kMaxTopK = 32;        // one lane per choice
constexpr int kMaxGroups = 32;
constexpr int kSlotChunk = 4096;    // choices of the slot map counted together
constexpr int64_t kMaxSlots = int64_t(1) << 26;   // every block reads every chunk's counts

struct RouteArgs {
  const void* logits = nullptr;
  int64_t ld = 0;
  const float* bias = nullptr;
  int32_t T = 0, E = 0, k = 0, groups = 1, top_groups = 1, group_top = 1;
  bool f32 = false, softmax = false, renorm = false;
  bool vec = false;                 // rows readable in whole words (set at the launch)
  int32_t tpw = 1;                  // tokens per warp (set at the launch)
  int32_t lanes_per_group = 0;      // 0: groups do not fall on lanes (set at the launch)
  int32_t group_size = 0;           // experts per group (set at the launch)
  uint32_t group_inverse = 0;       // 2^32 / group_size, rounded up (set at the launch)
  float scale = 1.0f;
  int32_t* idx = nullptr;
  float* w = nullptr;
  int32_t* status = nullptr;
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);

struct RouteBwdArgs {
  const void* logits = nullptr;
  int64_t ld = 0;
  const int32_t* idx = nullptr;
  const float* dw = nullptr;
  int32_t T = 0, E = 0, k = 0;
  bool f32 = false, softmax = false, renorm = false;
  bool vec = false;
  float scale = 1.0f;
  void* dlogits = nullptr;
  int64_t ldd = 0;
  int32_t* status = nullptr;
};
cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t s);

struct SlotArgs {
  const int32_t* idx = nullptr;
  int64_t n = 0;                    // T * k choices
  int32_t E = 0;
  bool masked = false;
  int32_t align_q = 1, M_max = 0;
  int64_t rows_total = 0;
  int32_t* rows = nullptr;
  int32_t* counts = nullptr;
  int32_t* src = nullptr;
  int32_t* work = nullptr;          // [chunks, E], more than one chunk only
  int32_t* status = nullptr;
};
cudaError_t launch_slots(const SlotArgs& a, cudaStream_t s);

struct DispatchArgs {
  const void* X = nullptr;
  int64_t ldx = 0;
  const uint8_t* SX = nullptr;      // E4M3 source: [T, K/128]
  const int32_t* rows = nullptr;
  int32_t T = 0, k = 0, K = 0;
  bool src_e4m3 = false, dst_e4m3 = false;
  void* A = nullptr;
  uint8_t* SFA = nullptr;           // [rows_total/group_rows, K/128, group_rows]
  int64_t rows_total = 0, group_rows = 0;
  uint8_t* CX = nullptr;            // checkpoint of a bf16 source: [T, K], [T, K/128]
  uint8_t* SCX = nullptr;
  int32_t* status = nullptr;
};
cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t s);

struct CombineArgs {
  const void* D = nullptr;
  const int32_t* rows = nullptr;
  const float* w = nullptr;
  int32_t T = 0, k = 0, K = 0;
  int64_t rows_total = 0;
  bool f32 = false;                 // out
  void* out = nullptr;
  int64_t ldo = 0;
  int32_t* status = nullptr;
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s);

struct CombineBwdArgs {
  const void* dout = nullptr;
  int64_t ldd = 0;
  bool f32 = false;                 // dout
  const void* D = nullptr;          // with dw, or both null
  const int32_t* rows = nullptr;
  const float* w = nullptr;
  int32_t T = 0, k = 0, K = 0;
  int64_t rows_total = 0;
  void* dD = nullptr;
  float* dw = nullptr;
  int32_t* status = nullptr;
};
cudaError_t launch_combine_bwd(const CombineBwdArgs& a, cudaStream_t s);

struct SwigluSaveArgs {
  const void* H = nullptr;
  int64_t rows_total = 0, group_rows = 0;
  int32_t N = 0;
  const int32_t* src = nullptr;
  bool y_e4m3 = false;
  void* Y = nullptr;
  uint8_t* SFY = nullptr;
  uint8_t* HC = nullptr;
  uint8_t* SHC = nullptr;
};
cudaError_t launch_swiglu_save(const SwigluSaveArgs& a, cudaStream_t s);

struct SwigluBwdArgs {
  const void* dY = nullptr;
  const uint8_t* HC = nullptr;
  const uint8_t* SHC = nullptr;
  int64_t rows_total = 0;
  int32_t N = 0;
  const int32_t* src = nullptr;
  const float* w = nullptr;
  int64_t n = 0;                    // entries of w and dw
  void* dH = nullptr;
  void* Y = nullptr;
  float* dw = nullptr;
  int32_t* status = nullptr;
};
cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s);

}  // namespace mg
