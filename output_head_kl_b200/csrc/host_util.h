// Host helpers shared by the C entry points (defined in api.cu): status codes and messages,
// alignment checks, the current device, TMA descriptors, tuning variables and kernel timing.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/kdkl.h"

namespace kdkl {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;

// Records the message that kdkl_last_error() returns on this host thread and returns `st`.
kdkl_status fail(kdkl_status st, const char* fmt, ...);
kdkl_status ok();
kdkl_status cuda_fail(cudaError_t e, const char* what);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Device {
  int id = 0;
  int sms = 0;
  int cc_major = 0;
};

// The current device; fails when there is none or it is not an sm_100 one.
kdkl_status current_device(Device& dv);

// 2-D tensor maps of a row-major matrix: `inner` contiguous elements per row, `outer` rows,
// row pitch in elements; bf16 and 8-bit elements.
bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch_elems,
              uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);
bool make_map_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch_elems,
                 uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);

// A tuning knob: the environment variable `name` as a non-negative integer, or dflt.
int env_window(const char* name, int dflt);

// Per-kernel timing (kdkl_timing_enable): `launch` is bracketed by two events while it is on.
enum TimedKind {
  kTPrepass = 0, kTFwd, kTMerge, kTGrad, kTDh, kTDw, kTTopK, kTTopKMerge, kTFusedFwd, kTGPass,
  kTNorm, kTNormGrad, kTLinear, kTActGrad, kTLinearDx, kTLinearDw, kTKinds
};
bool timing_on();
void timing_add(int kind, cudaEvent_t a, cudaEvent_t b);

template <class F>
cudaError_t timed(int kind, cudaStream_t s, F&& launch) {
  if (!timing_on()) return launch();
  cudaEvent_t a = nullptr, b = nullptr;
  if (cudaEventCreate(&a) != cudaSuccess || cudaEventCreate(&b) != cudaSuccess) return cudaGetLastError();
  cudaEventRecord(a, s);
  const cudaError_t e = launch();
  cudaEventRecord(b, s);
  timing_add(kind, a, b);
  return e;
}

}  // namespace kdkl
