// Newton-Schulz orthogonalisation of a stack of small matrices: host side and kernels of the C ABI
// in include/orthogonalize.h.
//
// With the short side s as rows, every round multiplies X from the left by a polynomial of its own
// Gram matrix, so that X_r = P_r X_0 and A_r = P_r A_0 P_r, all of them s x s and, as polynomials of
// A_0, symmetric and commuting:
//   Q = a I + b A + c A A,   P <- Q P,   A <- Q A Q
// The stack is read twice and written once, the second time mostly from the caches; rounds on X itself would
// read and write it ten times. One launch, a block a matrix, or three where there are few matrices or they are
// large: the Gram matrices (partial sums over pieces of the long side), the rounds on them, and P X.
//
// What A_0 costs in precision: an error E in A_0 moves a singular value's square by E, and the
// rounds lift the small ones (by up to a^2 each), so that the result is off by about E / 2 sigma^2 for
// ||X_0||_F = 1. With fp32 sums a spectrum of sigma^2 = 1e-5, a square matrix's, would be off by
// several 1e-3 in its smallest directions; in double it is not.
//
// What rounds on A cost: an eigenvalue of A_0 that should be 0 comes out as +-E, and every round multiplies it by
// up to the square of what it multiplies X by. Past 0.1 below zero it runs off to minus infinity, where rounds on X
// itself keep it at 0 or at the noise of X; and P, in fp32 where it meets X, has grown as much. So rounds are done in
// passes (rounds_of_pass): P is applied, and the Gram matrix of the result formed anew, before the rounds of a pass
// could have lifted anything by more than 2^15.
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <vector>

#include "orthogonalize.h"
#include "tensor_list.h"

namespace muon {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxShort = 128;
constexpr int64_t kMaxLong = int64_t(1) << 24;
constexpr int64_t kMaxCount = int64_t(1) << 24;
constexpr int kMaxRounds = 64;
constexpr int kBlocks = 256;                     // blocks that go through a batch's rounds at 128

struct StackArgs {
  const void* in;
  void* out;
  int64_t in_outer, in_inner, in_ld;             // ld: the stride of the side that is not contiguous
  int64_t out_outer, out_inner, out_ld;
  int64_t first;                                 // the batch's first matrix
  int inner, s, l;
  int count;                                     // of the batch
  int splits, span;                              // pieces of the long side, and a piece's length
  bool exact;                                    // bf16: sums of products in double throughout
  double* gram;                                  // count x splits x SP x SP
  uint16_t* p;                                   // count x 3 x SP x SP: P in parts
  int* expo;                                     // count x 2: of two, for X and for the result
  double* scratch;                               // SP = 128: P, a held matrix for each of kBlocks
};

struct Rounds {
  int n;
  float eps;
  bool as_is;                                    // a later pass: X is not divided by its norm
  float abc[3 * kMaxRounds];
};

// ---- loads and stores ------------------------------------------------------------------------

// N consecutive values from element i of a row, of which `left` (any number) are there; 0 beyond.
template <int DT, int N>
__device__ __forceinline__ void load_n(const void* base, int64_t i, int left, float (&x)[N]) {
  if (left >= N) {
    if constexpr (N == 1) {
      x[0] = load_one<DT>(base, i);
    } else if constexpr (DT == 0) {
      typedef uint32_t W __attribute__((ext_vector_type(N / 2), aligned(2)));
      const W w = *reinterpret_cast<const W*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        uint32_t v;
        if constexpr (N == 2) v = w[0]; else v = w[k];
        x[2 * k] = __uint_as_float(v << 16);
        x[2 * k + 1] = __uint_as_float(v & 0xffff0000u);
      }
    } else {
      constexpr int V = N < 4 ? N : 4;
      typedef float W __attribute__((ext_vector_type(V), aligned(4)));
      const W* const p = reinterpret_cast<const W*>(static_cast<const float*>(base) + i);
#pragma unroll
      for (int a = 0; a < N / V; ++a) {
        const W w = p[a];
#pragma unroll
        for (int k = 0; k < V; ++k) x[V * a + k] = w[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = k < left ? load_one<DT>(base, i + k) : 0.f;
  }
}

// The same N values as they lie in memory, all of them there: nothing is done to them before they are used, so
// that many such loads are on their way at once (load_n's branches make each wait for the one before).
template <int DT, int N>
struct Raw {
  static constexpr int W = N * (DT ? 4 : 2) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(W), aligned(DT ? 4 : 2)));
  Words w;
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    w = *reinterpret_cast<const Words*>(static_cast<const char*>(base) + i * (DT ? 4 : 2));
  }
  __device__ __forceinline__ uint32_t word(int k) const {
    if constexpr (W == 1) return w[0]; else return w[k];
  }
  __device__ __forceinline__ float operator[](int k) const {
    if (DT) return __uint_as_float(word(k));
    return __uint_as_float(k & 1 ? word(k / 2) & 0xffff0000u : word(k / 2) << 16);
  }
  // elements k of this and of a next one, packed (bf16)
  __device__ __forceinline__ uint32_t pair(const Raw& next, int k) const {
    return __builtin_amdgcn_perm(next.word(k / 2), word(k / 2), k & 1 ? 0x07060302u : 0x05040100u);
  }
};
template <>
struct Raw<0, 1> {
  uint16_t w;
  __device__ __forceinline__ void load(const void* base, int64_t i) { w = static_cast<const uint16_t*>(base)[i]; }
  __device__ __forceinline__ float operator[](int) const { return __uint_as_float(uint32_t(w) << 16); }
  __device__ __forceinline__ uint32_t pair(const Raw& next, int) const { return uint32_t(next.w) << 16 | w; }
};

template <int DT>
__device__ __forceinline__ void store_4(void* base, int64_t i, int left, f32x4 v) {
  if (left >= 4) {
    if (DT == 0) {
      typedef uint32_t W __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<W*>(static_cast<uint16_t*>(base) + i) =
          W{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
      typedef float W __attribute__((ext_vector_type(4), aligned(4)));
      *reinterpret_cast<W*>(static_cast<float*>(base) + i) = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) store_one<DT>(base, i + k, v[k]);
  }
}

__device__ __forceinline__ int64_t matrix_at(int64_t m, int inner, int64_t so, int64_t si) {
  const int64_t o = m / inner;
  return o * so + (m - o * inner) * si;
}

// ---- fp32 values as bf16 ones ---------------------------------------------------------------------
//
// x = x_1 + x_2 + x_3 with bf16 parts of 8 bits each, 24 together, so that a product of fp32 matrices is
// six of bf16 on the matrix cores (x_1 y_1, x_1 y_2, x_2 y_1, x_2 y_2, x_1 y_3, x_3 y_1; what is left out
// is 2^-24 of |x| |y|), 2.7 times as fast as their fp32 instructions.

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Two values' parts, packed.
template <int PARTS>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&w)[PARTS]) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    w[p] = pack_bf16x2(a, b);
    if (p + 1 < PARTS) {
      a -= __uint_as_float(w[p] << 16);
      b -= __uint_as_float(w[p] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                 0, 0, 0);
}

// c += a b of operands in parts, the smallest terms first.
template <int PA, int PB>
__device__ __forceinline__ f32x4 mma_parts(const u32x4 (&a)[PA], const u32x4 (&b)[PB], f32x4 c) {
  if constexpr (PA == 3) c = mma(a[2], b[0], c);
  if constexpr (PB == 3) c = mma(a[0], b[2], c);
  if constexpr (PA >= 2 && PB >= 2) c = mma(a[1], b[1], c);
  if constexpr (PA >= 2) c = mma(a[1], b[0], c);
  if constexpr (PB >= 2) c = mma(a[0], b[1], c);
  return mma(a[0], b[0], c);
}

// ---- products in double ------------------------------------------------------------------------
//
// The matrix cores' 4x4x4 instruction, four products of 4 x 4 at a time, does 75 TFLOP/s in double and the
// 16x16x4 one 38. A block of 16 x 16 is four of them: lane l has short index r = l % 16 of either
// operand at step k = l / 16, and instruction t multiplies rows 4 b .. 4 b + 3 of the left one by
// columns 4 ((b + t) % 4) .. of the right one, which comes 4 t lanes over. Sum t of lane l is then row
// 4 (r / 4) + l / 16, column 4 ((r / 4 + t) % 4) + r % 4.

template <int CTRL>
__device__ __forceinline__ double row_rotate(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  return __builtin_bit_cast(
      double, u32x2{uint32_t(__builtin_amdgcn_update_dpp(0, int(w[0]), CTRL, 0xf, 0xf, true)),
                    uint32_t(__builtin_amdgcn_update_dpp(0, int(w[1]), CTRL, 0xf, 0xf, true))});
}

// x of the lanes 0, 4, 8 and 12 further on in each 16.
struct Turns {
  double v[4];
  Turns() = default;
  __device__ __forceinline__ explicit Turns(double x)
      : v{x, row_rotate<0x12C>(x), row_rotate<0x128>(x), row_rotate<0x124>(x)} {}
};

__device__ __forceinline__ void mma_block(double a, const Turns& b, f64x4& acc) {
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[t] = __builtin_amdgcn_mfma_f64_4x4x4f64(a, b.v[t], acc[t], 0, 0, 0);
}
__device__ __forceinline__ int block_row(int r, int q) { return 4 * (r / 4) + q; }
__device__ __forceinline__ int block_col(int r, int t) { return (r + 4 * t) % 16; }

// ---- the Gram matrix -------------------------------------------------------------------------
//
// fp32: a wave takes 16 long positions at a time: lane l holds, for each 16 short indexes (a block), the
// values of short index r = l % 16 of it at positions 4 (l / 16) + 0..3, operands of four steps in double for
// every pair of blocks. bf16: 32 positions, eight a lane, are one operand of the bf16 instruction, whose
// products are exact; its sums of 32 are fp32 and are added in double (in double throughout, EXACT, 64 x 768
// takes a compute unit 13 us more). Their trace says whether fp32 held them (fits_fp32); where it does not,
// they are formed again in double, the lane's eight values operands of eight steps.
// Rows contiguous along the long side give a lane's values by one load; contiguous along the short side
// (TALL) a load gives the values of all NB blocks at one position, if block b has the short indexes
// NB r + b. The next positions' values are on their way while these are multiplied.

// Sums of the block's positions begin .. end - 1 into sum[SP * SP], where element (i, j) is there if
// gram_held(i, j), else its mirror image is.
template <bool TALL, int SP>
__device__ __forceinline__ bool gram_held(int i, int j) {
  constexpr int NB = SP / 16;
  return TALL ? i % NB <= j % NB : i / 16 <= j / 16;
}

// LDS doubles that gram_part needs.
template <int SP, int WAVES>
struct GramShape {
  static constexpr int NB = SP / 16, BLOCKS = NB * (NB + 1) / 2;
  static constexpr int LDS = (WAVES / 2) * BLOCKS * 256 > SP * SP ? (WAVES / 2) * BLOCKS * 256 : SP * SP;
};

template <int DT, int NB>
struct GramValues {
  float x[NB][4];
};
template <int NB>
struct GramValues<0, NB> {
  u32x4 x[NB];
};

// Value e of a lane's values of block b.
template <int DT, int NB>
__device__ __forceinline__ double gram_value(const GramValues<DT, NB>& v, int b, int e) {
  if constexpr (DT) return v.x[b][e];
  else return __uint_as_float(e & 1 ? v.x[b][e / 2] & 0xffff0000u : v.x[b][e / 2] << 16);
}

// Whether sums in fp32 over n positions hold what they stand for, by their trace: no diagonal sum of 32 and so
// no other can have passed fp32's range (2^128), and products lost below it, n 2^-126 of an element at most, are
// 2^-30 of the trace. A trace that is not finite, or of zeros, is formed again too.
__device__ __forceinline__ bool fits_fp32(double trace, int n) {
  return trace >= n * 0x1p-96 && trace <= 0x1p120;
}

// The sum of x over a wave, in each lane.
__device__ __forceinline__ double wave_sum(double x) {
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// A lane's loads of a step, as they lie in memory.
template <int DT, bool TALL, int NB>
struct GramRaw {
  static constexpr int V = DT ? 4 : 8;
  Raw<DT, TALL ? NB : V> x[TALL ? V : NB];
};

// The loads of a block's positions begin .. end - 1. Where a lane's loads of a step are whole or not there at all
// (the first `fast` steps) they are made as whole ones, of a place that is there; the others value by value.
template <int DT, bool TALL, int SP>
struct GramLoads {
  static constexpr int NB = SP / 16, STEP = DT ? 16 : 32, V = STEP / 4;
  const char* base;
  int64_t ld;
  int s, begin, end, r, q;
  int steps, fast;
  __device__ __forceinline__ GramLoads(const StackArgs& g, const char* base, int begin, int end, int lane)
      : base(base), ld(g.in_ld), s(g.s), begin(begin), end(end), r(lane & 15), q(lane >> 4) {
    steps = (end - begin + STEP - 1) / STEP;
    fast = TALL && s % NB != 0 ? 0 : TALL || (end - begin) % V == 0 ? steps : (end - begin) / STEP;
  }
  __device__ __forceinline__ void load(int step, GramValues<DT, NB>& to) const {
    const int k = begin + STEP * step + V * q;
    if constexpr (TALL) {
      float v[V][NB];
#pragma unroll
      for (int e = 0; e < V; ++e)
        load_n<DT, NB>(base, int64_t(k + e) * ld + NB * r, k + e < end ? s - NB * r : 0, v[e]);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (DT) to.x[b][e] = v[e][b];
          else to.x[b][e] = pack_bf16x2(v[2 * e][b], v[2 * e + 1][b]);
        }
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float v[V];
        load_n<DT, V>(base, int64_t(16 * b + r) * ld + k, 16 * b + r < s ? end - k : 0, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (DT) to.x[b][e] = v[e];
          else to.x[b][e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        }
      }
    }
  }
  __device__ __forceinline__ void fetch(int step, GramRaw<DT, TALL, NB>& to) const {
    const int k = begin + STEP * step + V * q;
    if constexpr (TALL) {
      const int at = NB * r < s ? NB * r : 0;
#pragma unroll
      for (int e = 0; e < V; ++e) to.x[e].load(base, int64_t(min(k + e, end - 1)) * ld + at);
    } else {
      const int at = min(k, end - V);
#pragma unroll
      for (int b = 0; b < NB; ++b) to.x[b].load(base, int64_t(min(16 * b + r, s - 1)) * ld + at);
    }
  }
  __device__ __forceinline__ void take(int step, const GramRaw<DT, TALL, NB>& from, GramValues<DT, NB>& to) const {
    const int k = begin + STEP * step + V * q;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TALL && DT) {
          to.x[b][e] = NB * r < s && k + e < end ? from.x[e][b] : 0.f;
        } else if constexpr (TALL) {
          const uint32_t w = from.x[2 * e].pair(from.x[2 * e + 1], b);
          to.x[b][e] = NB * r < s && k + 2 * e < end ? (k + 2 * e + 1 < end ? w : w & 0xffffu) : 0;
        } else if constexpr (DT) {
          to.x[b][e] = 16 * b + r < s && k < end ? from.x[b][e] : 0.f;
        } else {
          to.x[b][e] = 16 * b + r < s && k < end ? from.x[b].word(e) : 0;
        }
      }
  }
  // add(values) for steps first, first + by, ..
  template <typename F>
  __device__ __forceinline__ void each(int first, int by, F&& add) const {
    GramRaw<DT, TALL, NB> raw, next;
    GramValues<DT, NB> x;
    int step = first;
    if (step < fast) fetch(step, raw);
    for (; step < fast; step += by) {
      fetch(min(step + by, fast - 1), next);
      take(step, raw, x);
      add(x);
      raw = next;
    }
    for (; step < steps; step += by) {
      load(step, x);
      add(x);
    }
  }
};

template <int DT, bool TALL, int SP, int WAVES, bool EXACT>
__device__ __forceinline__ void gram_part(const StackArgs& g, const char* base, int begin, int end, int wave,
                                          int lane, double* lds) {
  using S = GramShape<SP, WAVES>;
  constexpr int NB = SP / 16;
  const int r = lane & 15, q = lane >> 4;
  f64x4 acc[S::BLOCKS];                          // blocks i <= j, row by row
#pragma unroll
  for (int u = 0; u < S::BLOCKS; ++u) acc[u] = f64x4{0, 0, 0, 0};
  GramLoads<DT, TALL, SP>(g, base, begin, end, lane).each(wave, WAVES, [&](const GramValues<DT, NB>& x) {
    if constexpr (!EXACT) {
#pragma unroll
      for (int i = 0, u = 0; i < NB; ++i)
#pragma unroll
        for (int j = i; j < NB; ++j, ++u) {
          const f32x4 c = mma(x.x[i], x.x[j], f32x4{0, 0, 0, 0});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[u][e] += double(c[e]);
        }
    } else {
#pragma unroll
      for (int e = 0; e < (DT ? 4 : 8); ++e)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const Turns d(gram_value(x, j, e));
#pragma unroll
          for (int i = 0; i <= j; ++i)
            mma_block(gram_value(x, i, e), d, acc[i * NB - i * (i - 1) / 2 + j - i]);
        }
    }
  });
  // the waves' sums, the upper half's to the lower half until one wave has them all
#pragma unroll
  for (int n = WAVES; n > 1; n = (n + 1) / 2) {
    const int half = (n + 1) / 2;
    f64x4* const pass = reinterpret_cast<f64x4*>(lds) + lane;
    if (wave >= half && wave < n)
#pragma unroll
      for (int u = 0; u < S::BLOCKS; ++u) pass[((wave - half) * S::BLOCKS + u) * 64] = acc[u];
    __syncthreads();
    if (wave < n - half)
#pragma unroll
      for (int u = 0; u < S::BLOCKS; ++u) acc[u] += pass[(wave * S::BLOCKS + u) * 64];
    __syncthreads();
  }
  if (wave == 0) {
#pragma unroll
    for (int i = 0, u = 0; i < NB; ++i)
#pragma unroll
      for (int j = i; j < NB; ++j, ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int a = EXACT ? block_row(r, q) : 4 * q + e, c = EXACT ? block_col(r, e) : r;
          lds[TALL ? (NB * a + i) * SP + NB * c + j : (16 * i + a) * SP + 16 * j + c] = acc[u][e];
        }
  }
  __syncthreads();
}

// The Gram matrix of the block's positions begin .. end - 1 into lds, by fp32 sums where they hold it.
template <int DT, bool TALL, int SP, int WAVES>
__device__ __forceinline__ void gram_of(const StackArgs& g, const char* base, int begin, int end, int wave,
                                        int lane, double* lds) {
  if constexpr (DT == 0) {
    if (!g.exact) {
      gram_part<DT, TALL, SP, WAVES, false>(g, base, begin, end, wave, lane, lds);
      double trace = 0;                          // the same in every wave
      for (int i = lane; i < SP; i += 64) trace += lds[i * SP + i];
      if (__builtin_amdgcn_readfirstlane(fits_fp32(wave_sum(trace), end - begin))) return;
      __syncthreads();                           // everyone has read it
    }
  }
  gram_part<DT, TALL, SP, WAVES, true>(g, base, begin, end, wave, lane, lds);
}

// At 128 the 36 blocks are 288 registers, so that they are shared out: wave W of four goes through all positions (the
// loads of the other waves come from the L1 cache) with the blocks of columns W and W + 4, rows c, c + 1, .. (mod 8).
// Straight into `out`; returns the wave's part of the trace. fp32 300 x 128 x 1024: 155 us (all blocks in every wave, with spills: 237), which the matrix
// cores bound at 72; bf16 58 (87).
template <int DT, bool TALL, bool EXACT, int W>
__device__ __forceinline__ double gram_shared(const StackArgs& g, const char* base, int begin, int end, int lane,
                                              double* out) {
  constexpr int SP = 128, NB = 8;
  f64x4 acc[9];
#pragma unroll
  for (int u = 0; u < 9; ++u) acc[u] = f64x4{0, 0, 0, 0};
  GramLoads<DT, TALL, SP>(g, base, begin, end, lane).each(0, 1, [&](const GramValues<DT, NB>& x) {
#pragma unroll
    for (int u = 0; u < 9; ++u) {
      if constexpr (!EXACT) {
        const int j = u < 5 ? W : W + 4, i = (j + u % 5) % NB;
        const f32x4 c = mma(x.x[i], x.x[j], f32x4{0, 0, 0, 0});
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][e] += double(c[e]);
      }
    }
    if constexpr (EXACT) {
#pragma unroll
      for (int e = 0; e < (DT ? 4 : 8); ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = W + 4 * h;
          const Turns d(gram_value(x, j, e));
#pragma unroll
          for (int o = 0; o < 5 - h; ++o) mma_block(gram_value(x, (j + o) % NB, e), d, acc[5 * h + o]);
        }
    }
  });
  const int r = lane & 15, q = lane >> 4;
  double trace = 0;
#pragma unroll
  for (int u = 0; u < 9; ++u) {
    const int j = u < 5 ? W : W + 4, i = (j + u % 5) % NB;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int a = EXACT ? block_row(r, q) : 4 * q + e, c = EXACT ? block_col(r, e) : r;
      const int row = TALL ? NB * a + i : 16 * i + a, col = TALL ? NB * c + j : 16 * j + c;
      out[row * SP + col] = acc[u][e];
      if (i != j) out[col * SP + row] = acc[u][e];
      else if (a == c) trace += acc[u][e];
    }
  }
  return EXACT ? 0.0 : wave_sum(trace);
}

template <int DT, bool TALL, bool EXACT>
__device__ __forceinline__ double gram_shared(const StackArgs& g, const char* base, int begin, int end, int wave,
                                              int lane, double* out) {
  if (wave == 0) return gram_shared<DT, TALL, EXACT, 0>(g, base, begin, end, lane, out);
  if (wave == 1) return gram_shared<DT, TALL, EXACT, 1>(g, base, begin, end, lane, out);
  if (wave == 2) return gram_shared<DT, TALL, EXACT, 2>(g, base, begin, end, lane, out);
  return gram_shared<DT, TALL, EXACT, 3>(g, base, begin, end, lane, out);
}

// A part of a matrix's long side (grid: count * splits) into its own whole matrix.
template <int DT, bool TALL, int SP>
__global__ __launch_bounds__(256, SP == 128 ? 2 : 1) void gram_kernel(const StackArgs g) {
  const int t = threadIdx.x;
  const int m = blockIdx.x / g.splits, z = blockIdx.x - m * g.splits;
  const char* const base = static_cast<const char*>(g.in) +
                           matrix_at(g.first + m, g.inner, g.in_outer, g.in_inner) * (DT ? 4 : 2);
  const int begin = z * g.span;
  const int end = min(g.l, begin + g.span);
  double* const out = g.gram + int64_t(blockIdx.x) * (SP * SP);
  if constexpr (SP == 128) {
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    if constexpr (DT == 0) {
      __shared__ double traces[4];
      if (!g.exact) {
        const double trace = gram_shared<DT, TALL, false>(g, base, begin, end, wave, t & 63, out);
        if ((t & 63) == 0) traces[wave] = trace;
        __syncthreads();                         // (and what the waves stored is ordered before the second form)
        const double trace_all = traces[0] + traces[1] + traces[2] + traces[3];
        if (__builtin_amdgcn_readfirstlane(fits_fp32(trace_all, end - begin))) return;
      }
    }
    gram_shared<DT, TALL, true>(g, base, begin, end, wave, t & 63, out);
  } else {
    __shared__ double sum[GramShape<SP, 4>::LDS];
    gram_of<DT, TALL, SP, 4>(g, base, begin, end, __builtin_amdgcn_readfirstlane(t >> 6), t & 63, sum);
    for (int at = t; at < SP * SP; at += 256) {
      const int i = at / SP, j = at % SP;
      out[at] = gram_held<TALL, SP>(i, j) ? sum[at] : sum[j * SP + i];
    }
  }
}

// ---- the rounds ------------------------------------------------------------------------------

// What comes of the norm. The result is P X / norm. Where X's norm and `norm` are in the middle of fp32's
// range the division goes to P; else X is taken at 2^-ex of itself, P and the result near 1, and
// the result gets the power of two that is left.
struct Norm {
  double scale, p_scale;
  int x_expo, out_expo;
  __device__ __forceinline__ Norm(double trace, const Rounds& R) {
    x_expo = out_expo = 0;
    if (R.as_is) {
      scale = 1.0;
      p_scale = isfinite(trace) ? 1.0 : __longlong_as_double(0x7ff8000000000000ll);
      return;
    }
    const double plain = sqrt(trace), norm = plain + double(R.eps);
    scale = 1.0 / norm;
    const bool fine = isfinite(norm) && norm > 0;
    p_scale = fine ? scale : __longlong_as_double(0x7ff8000000000000ll);
    if (!fine) return;
    int ex, en;
    frexp(plain, &ex);
    const double mant = frexp(norm, &en);
    if (plain == 0) ex = en;
    if (abs(ex) <= 60 && abs(en) <= 60) return;
    p_scale = 1.0 / mant;
    x_expo = -ex;
    out_expo = ex - en;
  }
};

// A block a matrix, in double. Every matrix here is symmetric: of its blocks of 16 x 16 one of each pair
// across the diagonal is computed and held, 10 of 16 for SP = 64 and 36 of 64 for 128, 17 doubles a row. Column
// c has rows c, c + 1, .. (mod NB), NB / 2 + 1 of them for c < NB / 2, one fewer for the others, so that the right
// operand is read and turned once for all of them; over four SIMDs a SIMD's share at SP = 64 is 3 blocks. A
// column is one wave's, at 32, where there are waves to spare, two waves' (H = 2: bf16 1500 x 31 x 800 162 -> 143
// us; at 64 3% slower, as both waves read and turn the right operand).
// A and Q lie in LDS, P too up to SP = 64; at 128 P is in the block's own scratch, in L2. T = Q A takes the
// place of A.
template <int SP, int H>
struct RoundShape {
  static constexpr int NB = SP / 16, BLOCKS = NB * (NB + 1) / 2;
  static constexpr int MOST = NB == 1 ? 1 : NB / 2 + 1;                // blocks of a column
  static constexpr int OWN = (MOST + H - 1) / H;                       // and of a wave
  static constexpr int WAVES = NB * H;
  static constexpr int PITCH = 17, BLOCK = 16 * PITCH, HELD = BLOCKS * BLOCK;  // doubles
  static constexpr bool FAR = SP > 64;
  static constexpr int LDS = (FAR ? 2 : 3) * HELD;
};

template <int SP, int H>
struct RoundBlocks {
  using S = RoundShape<SP, H>;
  static constexpr int NB = S::NB, OWN = S::OWN;
  int c, first;                                  // this wave's column, and its first row there less c
  int own;                                       // blocks: OWN, one fewer or none
  bool full;                                     // OWN
  int r, q;
  __device__ __forceinline__ RoundBlocks(int wave, int lane) : r(lane & 15), q(lane >> 4) {
    c = wave % NB;
    const int h = wave / NB, all = S::MOST - (NB > 1 && c >= NB / 2 ? 1 : 0), lower = (all + H - 1) / H;
    first = h == 0 ? 0 : lower;
    own = h == 0 ? lower : h < H ? all - lower : 0;
    full = own == OWN;
  }
  __device__ __forceinline__ int row_of(int o) const { return (c + first + o) % NB; }
  // f(o, e, row, column) for the elements that this thread holds of a product
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    int lane_r = r;
    asm volatile("" : "+v"(lane_r));             // (else every place's address stays in a register: spills at 128)
#pragma unroll
    for (int o = 0; o < OWN; ++o)
      if (o + 1 < OWN || full)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(o, e, 16 * row_of(o) + block_row(lane_r, q), 16 * c + block_col(lane_r, e));
  }
  // f(o, e, place) for the same elements, in a held matrix: block (c + d, c) is number d NB + c
  template <typename F>
  __device__ __forceinline__ void held(F&& f) const {
    int lane_r = r;
    asm volatile("" : "+v"(lane_r));
#pragma unroll
    for (int o = 0; o < OWN; ++o)
      if (o + 1 < OWN || full)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(o, e, ((first + o) * NB + c) * S::BLOCK + block_row(lane_r, q) * S::PITCH + block_col(lane_r, e));
  }
};

// The operands of N steps from step 4 k + t0: lane l's of step 4 k + t is element (16 k + 4 t + l / 16,
// 16 j + l % 16) of a held matrix, d = k - j (mod NB): in block (k, j), or turned in block (j, k).
template <int SP, int H, int N>
__device__ __forceinline__ void read_steps(const double* M, int d, int k, int t0, int j, int r, int q,
                                           double (&v)[N]) {
  using S = RoundShape<SP, H>;
  constexpr int NB = S::NB;
  const bool turned = 2 * d > NB || (2 * d == NB && j >= NB / 2);
  const int at = (turned ? k : j) * S::BLOCK + (turned ? r * S::PITCH + q : q * S::PITCH + r);
  const double* const from = M + uint32_t(at);
  const int block = (turned ? NB - d : d) * NB * S::BLOCK, step = turned ? 4 : 4 * S::PITCH;
#pragma unroll
  for (int t = 0; t < N; ++t) v[t] = from[block + step * (t0 + t)];
}

// acc = X Y, OWN of this wave's blocks. The next N steps' operands are read while these are multiplied. The
// matrix cores' double products share the vector units, so that every other vector instruction here costs
// their time. Wave c goes through the blocks of k from c: a block's number and turn are then constants, and reads
// take no address of their own (at 128, rolled up and with addresses: 290 us a matrix for 211; all of it in code
// twice, for waves of OWN and of fewer blocks, would not fit the instruction cache there, so that the last block
// is a branch).
template <int SP, int H, int OWN>
__device__ __forceinline__ void round_product(const RoundBlocks<SP, H>& B, const double* X, const double* Y,
                                              f64x4* acc) {
  constexpr int NB = SP / 16, N = SP == 128 ? 2 : 4, GROUPS = 4 * NB / N;
  struct Operands {
    double a[OWN][N], b[N];
  } v[2];
  int r = B.r, q = B.q;
  if (SP == 128) asm volatile("" : "+v"(r), "+v"(q));  // (else the addresses of all products stay in registers)
  auto read = [&](int n, Operands& to) {
    const int d = n * N / 4, k = (B.c + d) % NB, t0 = n * N % 4;
    read_steps<SP, H>(Y, d, k, t0, B.c, r, q, to.b);
#pragma unroll
    for (int o = 0; o < OWN; ++o)
      read_steps<SP, H>(X, (d + 2 * NB - (H > 1 ? B.first : 0) - o) % NB, k, t0, B.row_of(o), r, q, to.a[o]);
  };
  auto add = [&](const Operands& from) {
    Turns d[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
      d[t] = Turns(from.b[t]);
#pragma unroll
      for (int o = 0; o < OWN - (SP == 128); ++o) mma_block(from.a[o][t], d[t], acc[o]);
    }
    if (SP == 128 && B.full)
#pragma unroll
      for (int t = 0; t < N; ++t) mma_block(from.a[OWN - 1][t], d[t], acc[OWN - 1]);
  };
#pragma unroll
  for (int o = 0; o < OWN; ++o) acc[o] = f64x4{0, 0, 0, 0};
  read(0, v[0]);
#pragma unroll
  for (int n = 0; n < GROUPS; ++n) {
    if (n + 1 < GROUPS) read(n + 1, v[(n + 1) & 1]);
    add(v[n & 1]);
  }
}

// The rounds on c, this wave's blocks of the Gram matrix; p receives its blocks of P. lds: LDS doubles;
// scratch: HELD doubles at SP = 128; trace_of: SP doubles of LDS. Waves beyond WAVES only wait.
template <int SP, int H>
__device__ __forceinline__ Norm rounds_part(const Rounds& R, const RoundBlocks<SP, H>& B, int lane, double* lds,
                                            double* scratch, double* trace_of,
                                            f64x4 (&c)[RoundShape<SP, H>::OWN], f64x4 (&p)[RoundShape<SP, H>::OWN]) {
  using S = RoundShape<SP, H>;
  constexpr int OWN = S::OWN;
  double* const Q = lds;
  double* const A = lds + S::HELD;
  double* const P = S::FAR ? scratch : lds + 2 * S::HELD;
  const bool works = B.own > 0;
  auto product = [&](const double* X, const double* Y, f64x4 (&acc)[OWN]) {
    if (SP == 128 || B.full) round_product<SP, H, OWN>(B, X, Y, acc);
    else round_product<SP, H, (OWN > 1 ? OWN - 1 : 1)>(B, X, Y, acc);
  };
  if (works)
    B.each([&](int o, int e, int row, int col) {
      if (row == col) trace_of[row] = c[o][e];
    });
  __syncthreads();
  double trace = 0;                              // the same in every wave
  for (int i = lane; i < SP; i += 64) trace += trace_of[i];
  const Norm norm(wave_sum(trace), R);
  if (works) {
    B.held([&](int o, int e, int at) {
      c[o][e] = c[o][e] * norm.scale * norm.scale;
      A[at] = c[o][e];
    });
    B.each([&](int o, int e, int row, int col) { p[o][e] = row == col ? 1.0 : 0.0; });
  }
  __syncthreads();
  for (int n = 0; n < R.n; ++n) {
    const double a = R.abc[3 * n], b = R.abc[3 * n + 1], cc = R.abc[3 * n + 2];
    const bool last = n + 1 == R.n;
    if (works) {
      f64x4 sq[OWN];
      product(A, A, sq);
      B.each([&](int o, int e, int row, int col) {
        sq[o][e] = (row == col ? a : 0.0) + b * c[o][e] + cc * sq[o][e];
      });
      B.held([&](int o, int e, int at) {
        Q[at] = sq[o][e];
        if (n == 0) p[o][e] = sq[o][e];
      });
    }
    __syncthreads();
    if (works) {
      if (n > 0) product(Q, P, p);
      if (!last) product(Q, A, c);
    }
    if (last) break;
    __syncthreads();                             // A and P are read
    if (works)
      B.held([&](int o, int e, int at) {
        A[at] = c[o][e];
        P[at] = p[o][e];
      });
    __syncthreads();
    if (works) product(Q, A, c);
    __syncthreads();                             // and T
    if (works) B.held([&](int o, int e, int at) { A[at] = c[o][e]; });
    __syncthreads();
  }
  return norm;
}

// P in three bf16 parts, element (i, j) of part k at (k SP + i) pitch + j.
template <int SP, int H>
__device__ __forceinline__ void put_parts(const RoundBlocks<SP, H>& B, const Norm& norm,
                                          const f64x4 (&p)[RoundShape<SP, H>::OWN], uint16_t* out, int pitch) {
  B.each([&](int o, int e, int row, int col) {
    float v = float(p[o][e] * norm.p_scale);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t w = pack_bf16x2(v, 0.f);
      uint16_t* const to = out + k * SP * pitch;
      to[uint32_t(row * pitch + col)] = uint16_t(w);
      if (B.first + o > 0) to[uint32_t(col * pitch + row)] = uint16_t(w);
      v -= __uint_as_float(w << 16);
    }
  });
}

// Of the rounds alone: H, and threads of a block.
constexpr int halves(int sp) { return sp == 32 ? 2 : 1; }
constexpr int round_threads(int sp) { return sp / 16 * halves(sp) * 64; }

template <int SP>
__global__ __launch_bounds__(round_threads(SP), 1) void rounds_kernel(const StackArgs g, const Rounds R) {
  constexpr int H = halves(SP);
  using S = RoundShape<SP, H>;
  __shared__ double lds[S::LDS];
  __shared__ double trace_of[SP];
  const int t = threadIdx.x, lane = t & 63;
  const RoundBlocks<SP, H> B(__builtin_amdgcn_readfirstlane(t >> 6), lane);
  for (int m = blockIdx.x; m < g.count; m += gridDim.x) {
    const double* const part = g.gram + int64_t(m) * g.splits * (SP * SP);
    f64x4 c[S::OWN], p[S::OWN];
    if (B.own > 0) {
      B.each([&](int o, int e, int row, int col) { c[o][e] = part[row * SP + col]; });
      for (int z = 1; z < g.splits; ++z)         // (all elements of a part are on their way at once)
        B.each([&](int o, int e, int row, int col) { c[o][e] += part[z * (SP * SP) + row * SP + col]; });
    }
    const Norm norm = rounds_part<SP, H>(R, B, lane, lds, g.scratch + int64_t(blockIdx.x) * S::HELD, trace_of,
                                      c, p);
    if (t == 0) {
      g.expo[2 * m] = norm.x_expo;
      g.expo[2 * m + 1] = norm.out_expo;
    }
    if (B.own > 0) put_parts<SP, H>(B, norm, p, g.p + int64_t(m) * 3 * SP * SP, SP);
    __syncthreads();
  }
}

// ---- the result ------------------------------------------------------------------------------
//
// P X by bf16 parts, P in three, fp32 values in three and bf16 ones as they are. A wave takes 64 long
// positions: lane l has short indexes
// 8 (l / 16) + 0..7 of each 32 at its positions, P's operands come from LDS. The
// operands' order is chosen so that four values of a register quad lie side by side in the result: along the
// long side (X is the left operand, and lane l has positions 4 t(l) + 0..3 of the 64, t the 4 x 4 transpose
// of l % 16: four lanes then store 64 bytes in a row), or along the short one (TALL, P is
// the left operand, and a lane's eight short indexes one load).

template <int SP>
struct ResultShape {
  static constexpr int PITCH = SP + 8;           // of a part of P in LDS
};

// Positions begin .. end - 1, those of wave 0 first. p: P's parts in LDS, as put_parts writes them.
template <int DT, bool TALL, int SP, int WAVES>
__device__ __forceinline__ void result_part(const StackArgs& g, const char* in, char* out, const uint16_t* p,
                                            int expo, int expo_out, int begin, int end, int wave, int lane) {
  constexpr int NB = SP / 16, KS = SP < 32 ? 1 : SP / 32, PARTS = DT ? 3 : 1, PITCH = ResultShape<SP>::PITCH;
  const int r = lane & 15, q = lane >> 4;
  const int turned = r / 4 + r % 4 * 4;
  const bool whole = !TALL || g.s % 8 == 0;      // a lane's loads: whole or not there at all
  for (int j0 = begin + 64 * wave; j0 < end; j0 += 64 * WAVES) {
    f32x4 acc[NB][4] = {};
#pragma unroll 1
    for (int k = 0; k < KS; ++k) {
      const int row = 32 * k + 8 * q;
      float v[8][4];
      if (whole && (TALL || j0 + 64 <= end || end % 4 == 0)) {
        if constexpr (!TALL) {
          const int j = j0 + 4 * turned;
          Raw<DT, 4> w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e].load(in, int64_t(min(row + e, g.s - 1)) * g.in_ld + min(j, end - 4));
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int b = 0; b < 4; ++b) v[e][b] = row + e < g.s && j < end ? w[e][b] : 0.f;
        } else {
          Raw<DT, 8> w[4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            w[b].load(in, int64_t(min(j0 + 16 * b + r, end - 1)) * g.in_ld + (row < g.s ? row : 0));
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e][b] = row < g.s && j0 + 16 * b + r < end ? w[b][e] : 0.f;
        }
      } else if constexpr (!TALL) {
        const int j = j0 + 4 * turned;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          load_n<DT, 4>(in, int64_t(row + e) * g.in_ld + j, row + e < g.s ? end - j : 0, v[e]);
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j = j0 + 16 * b + r;
          float w[8];
          load_n<DT, 8>(in, int64_t(j) * g.in_ld + row, j < end ? g.s - row : 0, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e][b] = w[e];
        }
      }
      if (expo)
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int b = 0; b < 4; ++b) v[e][b] = ldexpf(v[e][b], expo);
      u32x4 x[4][PARTS];                         // of position block b: the lane's 8 short indexes
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[PARTS];
          split2(v[2 * e][b], v[2 * e + 1][b], w);
#pragma unroll
          for (int a = 0; a < PARTS; ++a) x[b][a][e] = w[a];
        }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        u32x4 o[3];
#pragma unroll
        for (int a = 0; a < 3; ++a) {
          o[a] = *reinterpret_cast<const u32x4*>(p + (a * SP + 16 * i + r) * PITCH +
                                                 (SP < 32 ? 8 * (q & 1) : 32 * k + 8 * q));
          if (SP < 32 && q > 1) o[a] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[i][b] = TALL ? mma_parts(o, x[b], acc[i][b]) : mma_parts(x[b], o, acc[i][b]);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (expo_out)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][b][e] = ldexpf(acc[i][b][e], expo_out);
      if constexpr (TALL) {
        const int row = 16 * i + 4 * q;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j = j0 + 16 * b + r;
          if (j < end) store_4<DT>(out, int64_t(j) * g.out_ld + row, g.s - row, acc[i][b]);
        }
      } else {
        const int row = 16 * i + r;
        if (row < g.s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = j0 + 16 * e + 4 * q;
            store_4<DT>(out, int64_t(row) * g.out_ld + at, end - at,
                        f32x4{acc[i][0][e], acc[i][1][e], acc[i][2][e], acc[i][3][e]});
          }
      }
    }
  }
}

template <int DT, bool TALL, int SP>
__global__ __launch_bounds__(256, SP == 128 ? 1 : 2) void result_kernel(const StackArgs g, int chunks, int chunk) {
  constexpr int PITCH = ResultShape<SP>::PITCH;
  __shared__ uint4 smem[3 * SP * PITCH / 8];
  uint16_t* const lds = reinterpret_cast<uint16_t*>(smem);
  const int t = threadIdx.x;
  const int m = blockIdx.x / chunks, z = blockIdx.x - m * chunks;
  const char* const in = static_cast<const char*>(g.in) +
                         matrix_at(g.first + m, g.inner, g.in_outer, g.in_inner) * (DT ? 4 : 2);
  char* const out = static_cast<char*>(g.out) +
                    matrix_at(g.first + m, g.inner, g.out_outer, g.out_inner) * (DT ? 4 : 2);
  const uint16_t* const p = g.p + int64_t(m) * 3 * SP * SP;
  for (int at = t * 8; at < 3 * SP * SP; at += 2048)
    *reinterpret_cast<u32x4*>(lds + at / SP * PITCH + at % SP) = *reinterpret_cast<const u32x4*>(p + at);
  __syncthreads();
  result_part<DT, TALL, SP, 4>(g, in, out, lds, g.expo[2 * m], g.expo[2 * m + 1], z * chunk,
                               min(g.l, (z + 1) * chunk), t >> 6, t & 63);
}

// ---- all of it in one launch -------------------------------------------------------------------
//
// Where there are enough matrices, or their long sides are short: a block a matrix, which it reads a second
// time from the caches. fp32 1200 x 64 x 1600: 492 us (2.0 TB/s), in three launches 679; bf16 288 and 418; bf16
// 144 x 64 x 768: 55 and 68 us; fp32 1 x 16 x 768: 15 and 17. Four waves, so that two matrices share a
// compute unit, or eight where there is one at most: 1200 x 64 x 1600 493 and 546 us, 144 x 64 x 768 57 and 55.
// Of those 55 us the rounds take 37 (7.3 each, 1.8 a product of 64^3, which the matrix cores bound at 1.3).

template <int DT, bool TALL, int SP, int WAVES>
__global__ __launch_bounds__(WAVES * 64, WAVES == 4 ? 2 : 1) void whole_kernel(const StackArgs g,
                                                                              const Rounds R) {
  constexpr int H = halves(SP);
  using S = RoundShape<SP, H>;
  constexpr int SUMS = GramShape<SP, WAVES>::LDS;
  static_assert(3 * SP * ResultShape<SP>::PITCH * 2 <= S::LDS * 8 && S::WAVES <= WAVES, "P's parts fit");
  __shared__ double lds[SUMS > S::LDS ? SUMS : S::LDS];  // sums, then the rounds' matrices, then P's parts
  __shared__ double trace_of[SP];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const RoundBlocks<SP, H> B(wave, lane);
  const int m = blockIdx.x;
  const char* const in = static_cast<const char*>(g.in) +
                         matrix_at(g.first + m, g.inner, g.in_outer, g.in_inner) * (DT ? 4 : 2);
  char* const out = static_cast<char*>(g.out) +
                    matrix_at(g.first + m, g.inner, g.out_outer, g.out_inner) * (DT ? 4 : 2);
  gram_of<DT, TALL, SP, WAVES>(g, in, 0, g.l, wave, lane, lds);
  f64x4 c[S::OWN], p[S::OWN];
  if (B.own > 0)
    B.each([&](int o, int e, int row, int col) {
      c[o][e] = gram_held<TALL, SP>(row, col) ? lds[row * SP + col] : lds[col * SP + row];
    });
  const Norm norm = rounds_part<SP, H>(R, B, lane, lds, nullptr, trace_of, c, p);
  __syncthreads();
  uint16_t* const parts = reinterpret_cast<uint16_t*>(lds);
  if (B.own > 0) put_parts<SP, H>(B, norm, p, parts, ResultShape<SP>::PITCH);
  __syncthreads();
  result_part<DT, TALL, SP, WAVES>(g, in, out, parts, norm.x_expo, norm.out_expo, 0, g.l, wave, lane);
}

// Up to 16 short indexes a matrix is one block of the 16x16x4 instruction, whose results lie as its
// operands have to: register e of lane l is row 4 e + l / 16, column l % 16, and the operand of step e,
// of a symmetric matrix, is that same element. The rounds then take no LDS and no barrier, and every wave
// does them for itself, which two waves a SIMD pay for: 1 x 16 x 768 14.4 us, of which 17 products of four
// instructions, at the 38 TFLOP/s of this form, are about half.
template <int DT, bool TALL>
__global__ __launch_bounds__(512) void narrow_kernel(const StackArgs g, const Rounds R) {
  constexpr int SP = 16, WAVES = 8, PITCH = ResultShape<SP>::PITCH;
  __shared__ f64x4 sums[WAVES][64];
  __shared__ uint4 smem[3 * SP * PITCH / 8];
  uint16_t* const parts = reinterpret_cast<uint16_t*>(smem);
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int m = blockIdx.x;
  const char* const in = static_cast<const char*>(g.in) +
                         matrix_at(g.first + m, g.inner, g.in_outer, g.in_inner) * (DT ? 4 : 2);
  char* const out = static_cast<char*>(g.out) +
                    matrix_at(g.first + m, g.inner, g.out_outer, g.out_inner) * (DT ? 4 : 2);
  constexpr int AHEAD = 8;                       // loads of a wave that are out at a time
  f64x4 acc[2] = {};
  for (int k0 = 16 * wave; k0 < g.l; k0 += 16 * WAVES * AHEAD) {
    float x[AHEAD][4];
    if (TALL || g.l % 4 == 0) {
      Raw<DT, TALL ? 1 : 4> w[AHEAD][TALL ? 4 : 1];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int k = k0 + 16 * WAVES * u + 4 * q;
        if constexpr (TALL) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[u][e].load(in, int64_t(min(k + e, g.l - 1)) * g.in_ld + min(r, g.s - 1));
        } else {
          w[u][0].load(in, int64_t(min(r, g.s - 1)) * g.in_ld + min(k, g.l - 4));
        }
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = k0 + 16 * WAVES * u + 4 * q + e;
          float v;
          if constexpr (TALL) v = w[u][e][0]; else v = w[u][0][e];
          x[u][e] = r < g.s && k < g.l ? v : 0.f;
        }
    } else {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int k = k0 + 16 * WAVES * u + 4 * q;
        load_n<DT, 4>(in, int64_t(r) * g.in_ld + k, r < g.s ? g.l - k : 0, x[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[e & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[u][e], x[u][e], acc[e & 1], 0, 0, 0);
  }
  sums[wave][lane] = acc[0] + acc[1];
  __syncthreads();
  f64x4 A = sums[0][lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) A += sums[w][lane];
  double trace = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) trace += 4 * e + q == r ? A[e] : 0.0;
  const Norm norm(wave_sum(trace), R);
  f64x4 P;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    A[e] = A[e] * norm.scale * norm.scale;
    P[e] = 4 * e + q == r ? 1.0 : 0.0;
  }
  auto product = [](const f64x4& X, const f64x4& Y) {
    f64x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
    s0 = __builtin_amdgcn_mfma_f64_16x16x4f64(X[0], Y[0], s0, 0, 0, 0);
    s1 = __builtin_amdgcn_mfma_f64_16x16x4f64(X[1], Y[1], s1, 0, 0, 0);
    s0 = __builtin_amdgcn_mfma_f64_16x16x4f64(X[2], Y[2], s0, 0, 0, 0);
    s1 = __builtin_amdgcn_mfma_f64_16x16x4f64(X[3], Y[3], s1, 0, 0, 0);
    return s0 + s1;
  };
  for (int n = 0; n < R.n; ++n) {
    const double a = R.abc[3 * n], b = R.abc[3 * n + 1], c = R.abc[3 * n + 2];
    const f64x4 C = product(A, A);
    f64x4 Q;
#pragma unroll
    for (int e = 0; e < 4; ++e) Q[e] = (4 * e + q == r ? a : 0.0) + b * A[e] + c * C[e];
    P = n == 0 ? Q : product(Q, P);
    if (n + 1 == R.n) break;
    A = product(Q, product(Q, A));
  }
  if (wave == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = float(P[e] * norm.p_scale);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t w = pack_bf16x2(v, 0.f);
        parts[(k * SP + 4 * e + q) * PITCH + r] = uint16_t(w);
        v -= __uint_as_float(w << 16);
      }
    }
  }
  __syncthreads();
  result_part<DT, TALL, SP, WAVES>(g, in, out, parts, norm.x_expo, norm.out_expo, 0, g.l, wave, lane);
}

// ---- host ------------------------------------------------------------------------------------

struct Sizes {
  int s, l, sp;
  int64_t count, batch;
  bool whole;                                    // in one launch
  int splits, span;
  size_t gram, p, expo, scratch;                 // bytes of a batch
  size_t total() const { return gram + p + expo + scratch; }
};

bool limits_ok(int64_t outer, int64_t inner, int64_t rows, int64_t cols) {
  return outer >= 0 && inner >= 0 && rows >= 0 && cols >= 0 && std::min(rows, cols) <= kMaxShort &&
         std::max(rows, cols) <= kMaxLong && outer <= kMaxCount && inner <= kMaxCount &&
         outer * inner <= kMaxCount;
}

Sizes sizes_of(int64_t count, int64_t rows, int64_t cols) {
  Sizes z;
  z.s = int(std::min(rows, cols));
  z.l = int(std::max(rows, cols));
  z.sp = z.s <= 16 ? 16 : z.s <= 32 ? 32 : z.s <= 64 ? 64 : 128;
  z.count = count;
  z.whole = z.sp < 128 && (count >= 64 || z.l <= 1024);
  if (z.whole) {                                 // in the kernel's own memory
    z.batch = std::min<int64_t>(count, int64_t(1) << 20);
    z.splits = 1;
    z.span = z.l;
    z.gram = z.p = z.expo = z.scratch = 0;
    return z;
  }
  // pieces of the long side where there are few matrices, of at least 256 positions
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(1024 / count, z.l / 256));
  z.span = int(((z.l + want - 1) / want + 63) / 64 * 64);
  z.splits = (z.l + z.span - 1) / z.span;
  const size_t elems = size_t(z.sp) * z.sp;
  // a batch's partial Gram matrices take up to 256 MB
  z.batch = std::min<int64_t>(count, std::max<int64_t>(1, (int64_t(256) << 20) / int64_t(elems * 8 * z.splits)));
  z.batch = std::min(z.batch, std::max<int64_t>(1, (int64_t(1) << 32) / z.l));   // and a launch's blocks
  auto pad = [](size_t b) { return (b + 255) & ~size_t(255); };
  z.gram = pad(size_t(z.batch) * z.splits * elems * 8);
  z.p = pad(size_t(z.batch) * elems * 6);
  z.expo = pad(size_t(z.batch) * 8);
  z.scratch = z.sp == 128 ? size_t(std::min<int64_t>(z.batch, kBlocks)) * RoundShape<128, 1>::HELD * 8 : 0;
  return z;
}

// A batch of z.count matrices. What decides about a sum's order goes by the stack, not by the batch.
template <int DT, bool TALL, int SP>
void launch_all(const StackArgs& g, const Rounds& R, const Sizes& z, hipStream_t s) {
  if constexpr (SP == 16) {
    if (z.whole) {
      hipLaunchKernelGGL((narrow_kernel<DT, TALL>), dim3((unsigned)g.count), dim3(512), 0, s, g, R);
      return;
    }
  } else if constexpr (SP <= 64) {
    if (z.whole) {
      if (z.count > kBlocks)
        hipLaunchKernelGGL((whole_kernel<DT, TALL, SP, 4>), dim3((unsigned)g.count), dim3(256), 0, s, g, R);
      else
        hipLaunchKernelGGL((whole_kernel<DT, TALL, SP, 8>), dim3((unsigned)g.count), dim3(512), 0, s, g, R);
      return;
    }
  }
  hipLaunchKernelGGL((gram_kernel<DT, TALL, SP>), dim3((unsigned)(g.count * g.splits)), dim3(256), 0, s, g);
  const int blocks = SP == 128 ? std::min(g.count, kBlocks) : g.count;
  hipLaunchKernelGGL((rounds_kernel<SP>), dim3((unsigned)blocks), dim3(round_threads(SP)), 0, s, g, R);
  const int chunk = int64_t(g.count) * g.l >= int64_t(1) << 20 ? 1024 : 256;
  const int chunks = (g.l + chunk - 1) / chunk;
  hipLaunchKernelGGL((result_kernel<DT, TALL, SP>), dim3((unsigned)(g.count * chunks)), dim3(256), 0, s, g,
                     chunks, chunk);
}

typedef void (*Launch)(const StackArgs&, const Rounds&, const Sizes&, hipStream_t);
template <int DT, bool TALL>
Launch launch_for(int sp) {
  return sp == 16 ? launch_all<DT, TALL, 16> : sp == 32 ? launch_all<DT, TALL, 32>
       : sp == 64 ? launch_all<DT, TALL, 64> : launch_all<DT, TALL, 128>;
}

// What a round can multiply a direction of X by: the largest |q| over [0, top], q(x) = a + b x + c x^2, top the
// largest eigenvalue that A can have; and that one after it, the largest x q(x)^2.
double round_gain(const float* abc, double* top) {
  const double a = abc[0], b = abc[1], c = abc[2], t = *top;
  auto q = [&](double x) { return std::fabs(a + b * x + c * x * x); };
  double gain = std::max(q(0), q(t)), next = t * q(t) * q(t);
  if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < t) gain = std::max(gain, q(-b / (2 * c)));
  // where (x q^2)' = q (a + 3 b x + 5 c x^2) is 0
  const double d = 9 * b * b - 20 * a * c;
  for (int sign = -1; sign <= 1; sign += 2) {
    const double x = c != 0 ? (d >= 0 ? (-3 * b + sign * std::sqrt(d)) / (10 * c) : 0) : b != 0 ? -a / (3 * b) : 0;
    if (x > 0 && x < t) next = std::max(next, x * q(x) * q(x));
  }
  *top = next;
  return gain;
}

// The rounds from `first` on that one pass does: as many as lift nothing by more than 2^15, one at least. By
// then an error of 1e-15 of an eigenvalue of A (double) is 1e-6 and P's rounding to fp32 1e-3 in directions in which X
// has nothing, as with rounds on X in fp32, where the noise of the first is lifted alike (a 64 x 768 matrix of
// rank 8, default coefficients, off by, in norm: 8 rounds 4e-4 here and there, 12 rounds 4e-2 and 5e-2).
// *lift: by how much these do. Eight rounds of the default coefficients are one pass, any number of (1.5, -0.5, 0)
// up to 25.
constexpr double kMostLift = 0x1p15;
// Up to here bf16 stacks are summed by the bf16 instructions, whose errors of 2e-9 of an eigenvalue (64 x 768; up to 1e-8
// for short sums) this lifts to 3e-3; beyond, in double. Five rounds of the default coefficients lift by 485.
constexpr double kMostLiftBf16 = 0x1p9;

int rounds_of_pass(const muon_config* cfg, int first, double* top, double* lift) {
  double run = 1;                                // what the rounds up to here lift most, from whichever on
  *lift = 1;
  int n = first;
  for (; n < cfg->ns_steps; ++n) {
    double after = *top;
    run = std::max(run, 1.0) * round_gain(cfg->schedule ? cfg->schedule + 3 * n : &cfg->a, &after);
    if (n > first && !(run <= kMostLift)) break;
    *lift = std::max(*lift, run);
    *top = after;
  }
  return n - first;
}

// The elements from the first to behind the last of a strided stack; false if it does not fit.
bool extent(const muon_stack& k, const int64_t* stride, int64_t* elems) {
  const int64_t side[4] = {k.outer, k.inner, k.rows, k.cols};
  int64_t e = 1;
  for (int d = 0; d < 4; ++d) {
    if (side[d] <= 1) continue;
    if (stride[d] < 0 || stride[d] > (int64_t(1) << 40) / (side[d] - 1)) return false;
    e += (side[d] - 1) * stride[d];
    if (e > int64_t(1) << 40) return false;
  }
  *elems = e;
  return true;
}

// Whether no two elements share a place: sides by stride, each past the extent of those before it.
bool distinct(const muon_stack& k, const int64_t* stride) {
  const int64_t side[4] = {k.outer, k.inner, k.rows, k.cols};
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + 4, [&](int a, int b) { return stride[a] < stride[b]; });
  int64_t e = 1;
  for (int d : order) {
    if (side[d] <= 1) continue;
    if (stride[d] < e) return false;
    e += (side[d] - 1) * stride[d];
  }
  return true;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_orthogonalize_workspace_size(int64_t outer, int64_t inner, int64_t rows, int64_t cols) {
  if (!limits_ok(outer, inner, rows, cols)) return SIZE_MAX;
  if (outer == 0 || inner == 0 || rows == 0 || cols == 0) return 0;
  return sizes_of(outer * inner, rows, cols).total();
}

int muon_orthogonalize_passes(const muon_config* cfg) {
  return c_entry([&]() -> int {
    if (int st = check_config(cfg)) return st;
    int passes = 0;
    double top = 1, lift;
    for (int first = 0; passes == 0 || first < cfg->ns_steps; ++passes)
      first += rounds_of_pass(cfg, first, &top, &lift);
    return passes;
  });
}

int muon_orthogonalize(const muon_stack* stack, const muon_config* cfg, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  return c_entry([&]() -> int {
    if (!stack) return fail(MUON_ERR_INVALID_ARG, "stack is NULL");
    if (int st = check_config(cfg)) return st;
    const muon_stack& k = *stack;
    if (!dtype_known(k.dtype)) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (k.outer < 0 || k.inner < 0 || k.rows < 0 || k.cols < 0)
      return fail(MUON_ERR_INVALID_ARG, "negative size");
    if (!limits_ok(k.outer, k.inner, k.rows, k.cols))
      return fail(MUON_ERR_UNSUPPORTED, "the shorter side is at most %d, the longer 2^24, and the stack "
                  "2^24 matrices", kMaxShort);
    if (k.outer == 0 || k.inner == 0 || k.rows == 0 || k.cols == 0) return MUON_OK;
    const size_t e = dtype_bytes(k.dtype);
    for (const void* p : {k.in, static_cast<const void*>(k.out)})
      if (!p || (reinterpret_cast<uintptr_t>(p) & (e - 1)))
        return fail(MUON_ERR_INVALID_ARG, "in and out must be non-NULL and aligned to their elements");
    int64_t in_elems, out_elems;
    if (!extent(k, k.in_stride, &in_elems) || !extent(k, k.out_stride, &out_elems))
      return fail(MUON_ERR_INVALID_ARG, "strides must be >= 0 and the stack within 2^40 elements");
    // which side is contiguous: the same one in both
    auto unit = [&](const int64_t* s, int d) { return s[d] == 1 || (d == 2 ? k.rows : k.cols) == 1; };
    const bool by_cols = unit(k.in_stride, 3) && unit(k.out_stride, 3);
    const bool by_rows = unit(k.in_stride, 2) && unit(k.out_stride, 2);
    if (!by_cols && !by_rows)
      return fail(MUON_ERR_INVALID_ARG, "rows or columns must be contiguous, the same in in and out");
    if (!distinct(k, k.out_stride))
      return fail(MUON_ERR_INVALID_ARG, "two elements of out share a place");
    const Sizes z = sizes_of(k.outer * k.inner, k.rows, k.cols);
    if (z.total() > 0 &&
        (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < z.total()))
      return fail(MUON_ERR_WORKSPACE, "a workspace of %zu bytes, 256-byte aligned, is needed", z.total());
    auto range = [](const void* p, size_t bytes, bool written) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      return Range{lo, lo + bytes, written};
    };
    std::vector<Range> rs = {range(k.out, size_t(out_elems) * e, true)};
    if (z.total() > 0) rs.push_back(range(workspace, z.total(), true));
    if (k.in != k.out || !std::equal(k.in_stride, k.in_stride + 4, k.out_stride))
      rs.push_back(range(k.in, size_t(in_elems) * e, false));
    if (int st = check_overlaps(rs)) return st;

    double top = 1, lift;
    int rounds = rounds_of_pass(cfg, 0, &top, &lift);
    if (k.dtype == MUON_DT_BF16 && rounds < cfg->ns_steps)
      return fail(MUON_ERR_UNSUPPORTED, "these rounds take more than one pass, which bf16 stacks cannot (between "
                  "passes values are held in the result's dtype): convert to fp32");

    const bool long_is_cols = k.cols >= k.rows;
    StackArgs g;
    g.out = k.out;
    g.out_outer = k.out_stride[0];
    g.out_inner = k.out_stride[1];
    g.inner = int(k.inner);
    g.s = z.s;
    g.l = z.l;
    g.splits = z.splits;
    g.span = z.span;
    g.exact = lift > kMostLiftBf16;
    char* at = static_cast<char*>(workspace);
    g.gram = reinterpret_cast<double*>(at);
    g.p = reinterpret_cast<uint16_t*>(at += z.gram);
    g.expo = reinterpret_cast<int*>(at += z.p);
    g.scratch = reinterpret_cast<double*>(at += z.expo);
    Rounds R;
    R.eps = cfg->eps;
    // a pass reads the stack, or what the one before has left in out
    for (int first = 0;;) {
      const int64_t* const in_stride = first ? k.out_stride : k.in_stride;
      // the contiguous side is the long one, or the short one (TALL)
      const bool cols_lie = unit(in_stride, 3) && unit(k.out_stride, 3);
      const bool rows_lie = unit(in_stride, 2) && unit(k.out_stride, 2);
      const bool tall = long_is_cols ? !cols_lie : !rows_lie;
      const int other = long_is_cols != tall ? 2 : 3;  // the side whose stride is free
      g.in = first ? k.out : k.in;
      g.in_outer = in_stride[0];
      g.in_inner = in_stride[1];
      g.in_ld = in_stride[other];
      g.out_ld = k.out_stride[other];
      R.n = rounds;
      R.as_is = first > 0;
      for (int n = 0; n < rounds; ++n)
        for (int c = 0; c < 3; ++c)
          R.abc[3 * n + c] = cfg->schedule ? cfg->schedule[3 * (first + n) + c] : (&cfg->a)[c];
      const Launch run = k.dtype == MUON_DT_F32
          ? (tall ? launch_for<1, true>(z.sp) : launch_for<1, false>(z.sp))
          : (tall ? launch_for<0, true>(z.sp) : launch_for<0, false>(z.sp));
      for (int64_t m = 0; m < z.count; m += z.batch) {
        g.first = m;
        g.count = int(std::min(z.batch, z.count - m));
        run(g, R, z, stream);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
          return fail(MUON_ERR_HIP, "launch of an orthogonalisation kernel failed: %s", hipGetErrorString(err));
      }
      first += rounds;
      if (first >= cfg->ns_steps) return MUON_OK;
      rounds = rounds_of_pass(cfg, first, &top, &lift);
    }
  });
}

}  // extern "C"
