// Microscaled 4-bit values (include/mx4.h): the held layout, shared by the kernels that write it
// (mx4_quantize.hip) and the products that read it (mx4_matmul.hip).
#pragma once

#include "tensor_list.h"

namespace muon {

constexpr int kMxBlock = 32;                     // values that share a scale
constexpr int kMxPanel = 16;                     // rows of a panel
constexpr int kMxStep = 128;                     // columns of a step: 64 bytes of codes, 4 scales
constexpr int kMxTileBytes = kMxPanel * kMxStep / 2;                  // codes of a panel's step
constexpr int kMxTileScales = kMxPanel * kMxStep / kMxBlock;          // its scales
constexpr int64_t kMxMaxSide = (int64_t(1) << 31) - 256;
constexpr int64_t kMxMaxElems = int64_t(1) << 40;

inline bool mx_sides_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMxMaxSide && cols <= kMxMaxSide &&
         (rows == 0 || cols <= kMxMaxElems / rows);
}
inline int64_t mx_panels(int64_t rows) { return (rows + kMxPanel - 1) / kMxPanel; }
inline int64_t mx_steps(int64_t cols) { return (cols + kMxStep - 1) / kMxStep; }

inline Range mx_range(const void* p, size_t bytes, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + bytes, written};
}

inline int mx_launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return fail(MUON_ERR_HIP, "launch of the %s kernel failed: %s", what, hipGetErrorString(e));
  return MUON_OK;
}

// 2^(b - 127) of a scale byte below 255 (byte 0 is a subnormal).
__device__ __forceinline__ float mx_scale(int b) {
  return __uint_as_float(b == 0 ? 0x00400000u : uint32_t(b) << 23);
}

}  // namespace muon
