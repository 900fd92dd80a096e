// Shared by the kernels that make one pass over a list of tensors (adamw.hip, grad_norm.hip):
// vector access to bf16 and fp32 buffers, the lookup of a block's tensor, and the host's part
// of a C entry point.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "muon.h"
#include "muon_internal.h"

namespace muon {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int64_t kMaxTensorElems = int64_t(1) << 35;

// Two floats -> two bfloat16 in one dword (lo = first), round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <bool NT, typename T>
__device__ __forceinline__ T load_at(const T* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void store_at(T* p, T x) {
  if (NT) __builtin_nontemporal_store(x, p);
  else *p = x;
}

// N (4 or 8) consecutive elements of a bf16 (DT 0) or fp32 (DT 1) buffer, aligned to N elements or
// 16 bytes: accesses of 16 bytes (of 8 for 4 bf16). NT: nontemporal.
template <int DT, bool NT, int N>
__device__ __forceinline__ void load_vec(const void* base, int64_t i, float (&x)[N]) {
  static_assert(N == 4 || N == 8, "elements of an access or two");
  if (DT == 0) {
    typedef uint32_t W __attribute__((ext_vector_type(N / 2)));
    const W w = load_at<NT>(reinterpret_cast<const W*>(static_cast<const uint16_t*>(base) + i));
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
#pragma unroll
    for (int a = 0; a < N / 4; ++a) {
      const f32x4 w = load_at<NT>(q + a);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * a + k] = w[k];
    }
  }
}

template <int DT, bool NT, int N>
__device__ __forceinline__ void store_vec(void* base, int64_t i, const float (&x)[N]) {
  static_assert(N == 4 || N == 8, "elements of an access or two");
  if (DT == 0) {
    typedef uint32_t W __attribute__((ext_vector_type(N / 2)));
    W w;
#pragma unroll
    for (int k = 0; k < N / 2; ++k) w[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
    store_at<NT>(reinterpret_cast<W*>(static_cast<uint16_t*>(base) + i), w);
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(base) + i);
#pragma unroll
    for (int a = 0; a < N / 4; ++a)
      store_at<NT>(q + a, f32x4{x[4 * a], x[4 * a + 1], x[4 * a + 2], x[4 * a + 3]});
  }
}

template <int DT>
__device__ __forceinline__ float load_one(const void* base, int64_t i) {
  if (DT == 0) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(base)[i]) << 16);
  return static_cast<const float*>(base)[i];
}

template <int DT>
__device__ __forceinline__ void store_one(void* base, int64_t i, float x) {
  if (DT == 0) static_cast<uint16_t*>(base)[i] = uint16_t(pack_bf16x2(x, 0.f) & 0xffffu);
  else static_cast<float*>(base)[i] = x;
}

// The tensor of block b: the last of first(0) .. first(count - 1) (ascending, first(0) = 0) that is
// at most b, for count <= 512. Up to 64 entries: a load by every lane and a ballot; more: the same
// over every eighth entry, then over the eight from there.
template <typename F>
__device__ __forceinline__ int find_tensor(F&& first, int count, int b) {
  const int lane = threadIdx.x & 63;
  int base = 0, step = count <= 64 ? 1 : 8;
  int f = lane * step < count ? first(lane * step) : 0x7fffffff;
  if (step == 8) {
    base = 8 * (__popcll(__ballot(f <= b)) - 1);
    f = lane < 8 && base + lane < count ? first(base + lane) : 0x7fffffff;
  }
  return __builtin_amdgcn_readfirstlane(base + __popcll(__ballot(f <= b)) - 1);
}

inline size_t dtype_bytes(muon_dtype d) { return d == MUON_DT_BF16 ? 2 : 4; }
inline bool dtype_known(muon_dtype d) { return d == MUON_DT_BF16 || d == MUON_DT_F32; }
inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Runs the body of a C entry point: no C++ exception (of a container that cannot grow) leaves.
template <typename F>
int c_entry(F&& body) {
  clear_error();
  try {
    return body();
  } catch (...) {
    return fail(MUON_ERR_UNSUPPORTED, "out of host memory");
  }
}

}  // namespace muon
