// Newton-Schulz orthogonalisation of a stack of small matrices: host side and kernels of the C ABI
// in include/orthogonalize.h.
//
// With the short side s as rows, every round multiplies X from the left by a polynomial of its own
// Gram matrix, so that X_r = P_r X_0 and A_r = P_r A_0 P_r, all of them s x s and, as polynomials of
// A_0, symmetric and commuting:
//   Q = a I + b A + c A A,   P <- Q P,   A <- Q A Q
// Three launches: the Gram matrices (partial sums over pieces of the long side), the rounds on them
// (a block a matrix), and P X. The stack is read twice and written once; rounds on X itself would
// read and write it ten times.
//
// What A_0 costs in precision: an error E in A_0 moves a singular value's square by E, and the
// rounds lift the small ones (by up to a^2 each), so that the result is off by about E / 2 sigma^2 for
// ||X_0||_F = 1. With fp32 sums a spectrum of sigma^2 = 1e-5, a square matrix's, would be off by
// several 1e-3 in its smallest directions; in double it is not.
#include <algorithm>
#include <cmath>
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
  double* gram;                                  // count x splits x SP x SP
  float* p;                                      // count x SP x SP
  int* expo;                                     // count
  double* scratch;                               // SP = 128: kBlocks x 3 x SP x SP
};

struct Rounds {
  int n;
  float eps;
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

// ---- the Gram matrix -------------------------------------------------------------------------
//
// A wave takes 16 long positions at a time: lane l holds, for each 16 short indexes (a block), the
// values of short index r = l % 16 of it at positions 4 (l / 16) + 0..3, which are operands of four
// v_mfma_f64_16x16x4 for every pair of blocks. Rows contiguous along the long side give them by one load
// of four; contiguous along the short side (TALL) a load gives the values of all NB blocks at one
// position, if block b has the short indexes NB r + b.
template <int DT, bool TALL, int SP>
__global__ __launch_bounds__(256, 1) void gram_kernel(const StackArgs g) {
  constexpr int NB = SP / 16;
  __shared__ double sum[SP * SP];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, r = lane & 15, q = lane >> 4;
  const int m = blockIdx.x / g.splits, z = blockIdx.x - m * g.splits;
  const char* const base = static_cast<const char*>(g.in) +
                           matrix_at(g.first + m, g.inner, g.in_outer, g.in_inner) * (DT ? 4 : 2);
  const int begin = z * g.span, end = min(g.l, begin + g.span);

  f64x4 acc[NB][NB];                             // b1 <= b2
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f64x4{0, 0, 0, 0};
  for (int k0 = begin + 16 * wave; k0 < end; k0 += 64) {
    float x[NB][4];
    const int k = k0 + 4 * q;
    if constexpr (TALL) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[NB];
        load_n<DT, NB>(base, int64_t(k + e) * g.in_ld + NB * r, k + e < end ? g.s - NB * r : 0, v);
#pragma unroll
        for (int b = 0; b < NB; ++b) x[b][e] = v[b];
      }
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        load_n<DT, 4>(base, int64_t(16 * b + r) * g.in_ld + k, 16 * b + r < g.s ? end - k : 0, x[b]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double d[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) d[b] = x[b][e];
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = i; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(d[i], d[j], acc[i][j], 0, 0, 0);
    }
  }
  // the four waves' sums in their order; register e of lane l is row 4 e + l / 16, column l % 16
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = i; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = 4 * e + q;
            double* const to = &sum[TALL ? (NB * a + i) * SP + NB * r + j : (16 * i + a) * SP + 16 * j + r];
            *to = w ? *to + acc[i][j][e] : acc[i][j][e];
          }
    }
    __syncthreads();
  }
  double* const out = g.gram + int64_t(blockIdx.x) * (SP * SP);
  for (int at = t; at < SP * SP; at += 256) {
    const int i = at / SP, j = at % SP;
    const bool held = TALL ? i % NB <= j % NB : i / 16 <= j / 16;
    out[at] = held ? sum[at] : sum[j * SP + i];
  }
}

// ---- the rounds ------------------------------------------------------------------------------

template <int SP>
struct RoundShape {
  static constexpr int BM = SP <= 32 ? 1 : 2, BN = SP <= 64 ? 1 : 2;   // blocks of 16 x 16 a wave
  static constexpr int WAVES = SP / 16 / BM * (SP / 16 / BN);
  static constexpr int PITCH = SP == 16 ? 16 : SP + 16;                // banks: rows apart by 128 bytes
};

// acc = X Y of symmetric X and Y (element (i, j) at i * pitch + j).
template <int SP, int PX, int PY>
__device__ __forceinline__ void product(const double* X, const double* Y, int row0, int col0, int r, int q,
                                        f64x4 (&acc)[RoundShape<SP>::BM][RoundShape<SP>::BN]) {
  constexpr int BM = RoundShape<SP>::BM, BN = RoundShape<SP>::BN;
#pragma unroll
  for (int i = 0; i < BM; ++i)
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[i][j] = f64x4{0, 0, 0, 0};
#pragma unroll 4
  for (int k = 0; k < SP; k += 4) {
    double a[BM], b[BN];
#pragma unroll
    for (int i = 0; i < BM; ++i) a[i] = X[(k + q) * PX + row0 + 16 * i + r];
#pragma unroll
    for (int j = 0; j < BN; ++j) b[j] = Y[(k + q) * PY + col0 + 16 * j + r];
#pragma unroll
    for (int i = 0; i < BM; ++i)
#pragma unroll
      for (int j = 0; j < BN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[i], b[j], acc[i][j], 0, 0, 0);
  }
}

// A, Q and P lie in LDS up to SP = 64. At 128 (a matrix is 128 KB) LDS has Q, or A for its square, and
// A, QA and P go through the block's own scratch, in L2.
template <int SP>
__global__ __launch_bounds__(RoundShape<SP>::WAVES * 64, 1) void rounds_kernel(const StackArgs g,
                                                                              const Rounds R) {
  using S = RoundShape<SP>;
  constexpr bool FAR = SP > 64;
  constexpr int P1 = S::PITCH, P2 = FAR ? SP : S::PITCH, THREADS = S::WAVES * 64;
  __shared__ double lds[(FAR ? 1 : 3) * SP * P1];
  __shared__ double trace_of[1];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, r = lane & 15, q = lane >> 4;
  constexpr int ACROSS = SP / 16 / S::BN;        // waves side by side
  const int row0 = wave / ACROSS * 16 * S::BM, col0 = wave % ACROSS * 16 * S::BN;
  double* const Q = lds;
  double* const A = FAR ? g.scratch + int64_t(blockIdx.x) * 3 * SP * SP : lds + SP * P1;
  double* const P = A + SP * P2;
  double* const T = FAR ? P + SP * P2 : A;       // QA

  auto each = [&](auto&& f) {                    // the elements that this thread holds of a product
#pragma unroll
    for (int i = 0; i < S::BM; ++i)
#pragma unroll
      for (int j = 0; j < S::BN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) f(i, j, e, row0 + 16 * i + 4 * e + q, col0 + 16 * j + r);
  };

  for (int m = blockIdx.x; m < g.count; m += gridDim.x) {
    const double* const part = g.gram + int64_t(m) * g.splits * (SP * SP);
    f64x4 c[S::BM][S::BN], p[S::BM][S::BN], own[S::BM][S::BN];
    auto gram_at = [&](int row, int col) {
      double v = part[row * SP + col];
      for (int z = 1; z < g.splits; ++z) v += part[int64_t(z) * SP * SP + row * SP + col];
      return v;
    };
    each([&](int i, int j, int e, int row, int col) {
      own[i][j][e] = gram_at(row, col);
      p[i][j][e] = row == col ? 1.0 : 0.0;
      A[row * P2 + col] = own[i][j][e];
    });
    __syncthreads();
    if (t < 64) {
      double v = 0;
      for (int i = lane; i < SP; i += 64) v += A[i * P2 + i];
      for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
      if (t == 0) trace_of[0] = v;
    }
    __syncthreads();
    const double norm = sqrt(trace_of[0]) + double(R.eps), scale = 1.0 / norm;
    each([&](int i, int j, int e, int row, int col) {
      own[i][j][e] = own[i][j][e] * scale * scale;
      A[row * P2 + col] = own[i][j][e];
      if (FAR) Q[row * P1 + col] = own[i][j][e];
    });
    __syncthreads();
    for (int n = 0; n < R.n; ++n) {
      const double a = R.abc[3 * n], b = R.abc[3 * n + 1], cc = R.abc[3 * n + 2];
      const bool last = n + 1 == R.n;
      if (FAR) product<SP, P1, P1>(Q, Q, row0, col0, r, q, c);         // Q holds A here
      else product<SP, P2, P2>(A, A, row0, col0, r, q, c);
      __syncthreads();
      each([&](int i, int j, int e, int row, int col) {
        const double v = (row == col ? a : 0.0) + b * own[i][j][e] + cc * c[i][j][e];
        Q[row * P1 + col] = v;
        if (n == 0) p[i][j][e] = v;
      });
      __syncthreads();
      if (n > 0) product<SP, P1, P2>(Q, P, row0, col0, r, q, p);
      if (last) break;
      product<SP, P1, P2>(Q, A, row0, col0, r, q, c);
      __syncthreads();
      each([&](int i, int j, int e, int row, int col) {
        T[row * P2 + col] = c[i][j][e];
        P[row * P2 + col] = p[i][j][e];
      });
      __syncthreads();
      product<SP, P1, P2>(Q, T, row0, col0, r, q, own);
      __syncthreads();
      each([&](int i, int j, int e, int row, int col) {
        A[row * P2 + col] = own[i][j][e];
        if (FAR) Q[row * P1 + col] = own[i][j][e];
      });
      __syncthreads();
    }
    // P / norm as a matrix near 1 and a power of two for X, so that neither leaves fp32's range
    int expo = 0;
    const bool fine = isfinite(norm);
    const double f = fine ? 1.0 / frexp(norm, &expo) : __longlong_as_double(0x7ff8000000000000ll);
    each([&](int i, int j, int e, int row, int col) {
      g.p[int64_t(m) * SP * SP + row * SP + col] = float(p[i][j][e] * f);
    });
    if (t == 0) g.expo[m] = fine ? -expo : 0;
    __syncthreads();
  }
}

// ---- the result ------------------------------------------------------------------------------
//
// A wave takes 64 long positions: their values stay in registers, P comes from LDS, one operand for four
// v_mfma_f32_16x16x4. The operands' order is chosen so that four values of a register quad lie side by
// side in the result: along the long side (X is the left operand, and block b of positions is
// 4 r + b), or along the short one (TALL, P is the left operand).
template <int DT, bool TALL, int SP>
__global__ __launch_bounds__(256) void result_kernel(const StackArgs g, int chunks, int chunk) {
  constexpr int NB = SP / 16, PITCH = TALL ? SP + 4 : SP + 16;
  __shared__ float P[SP * PITCH];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, r = lane & 15, q = lane >> 4;
  const int m = blockIdx.x / chunks, z = blockIdx.x - m * chunks;
  const char* const in = static_cast<const char*>(g.in) +
                         matrix_at(g.first + m, g.inner, g.in_outer, g.in_inner) * (DT ? 4 : 2);
  char* const out = static_cast<char*>(g.out) +
                    matrix_at(g.first + m, g.inner, g.out_outer, g.out_inner) * (DT ? 4 : 2);
  const float* const p = g.p + int64_t(m) * SP * SP;
  for (int at = t; at < SP * SP; at += 256) P[at / SP * PITCH + at % SP] = p[at];
  const int expo = g.expo[m];
  __syncthreads();
  const int end = min(g.l, (z + 1) * chunk);
  for (int j0 = z * chunk + 64 * wave; j0 < end; j0 += 256) {
    if constexpr (!TALL) {
      float x[SP / 4][4];
      const int j = j0 + 4 * r;
#pragma unroll
      for (int k = 0; k < SP / 4; ++k) {
        load_n<DT, 4>(in, int64_t(4 * k + q) * g.in_ld + j, 4 * k + q < g.s ? end - j : 0, x[k]);
#pragma unroll
        for (int b = 0; b < 4; ++b) x[k][b] = ldexpf(x[k][b], expo);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        f32x4 acc[4] = {};
#pragma unroll
        for (int k = 0; k < SP / 4; ++k) {
          const float w = P[(4 * k + q) * PITCH + 16 * i + r];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[k][b], w, acc[b], 0, 0, 0);
        }
        const int row = 16 * i + r;
        if (row < g.s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = j0 + 16 * q + 4 * e;
            store_4<DT>(out, int64_t(row) * g.out_ld + at, end - at,
                        f32x4{acc[0][e], acc[1][e], acc[2][e], acc[3][e]});
          }
      }
    } else {
      float x[4][NB][4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int j = j0 + 16 * b + r;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          load_n<DT, 4>(in, int64_t(j) * g.in_ld + 16 * k + 4 * q, j < end ? g.s - 16 * k - 4 * q : 0,
                        x[b][k]);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[b][k][e] = ldexpf(x[b][k][e], expo);
        }
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        f32x4 acc[4] = {};
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = P[(16 * k + 4 * q + e) * PITCH + 16 * i + r];
#pragma unroll
            for (int b = 0; b < 4; ++b)
              acc[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, x[b][k][e], acc[b], 0, 0, 0);
          }
        const int row = 16 * i + 4 * q;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j = j0 + 16 * b + r;
          if (j < end) store_4<DT>(out, int64_t(j) * g.out_ld + row, g.s - row, acc[b]);
        }
      }
    }
  }
}

// ---- host ------------------------------------------------------------------------------------

struct Sizes {
  int s, l, sp;
  int64_t count, batch;
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
  z.p = pad(size_t(z.batch) * elems * 4);
  z.expo = pad(size_t(z.batch) * 4);
  z.scratch = z.sp == 128 ? size_t(std::min<int64_t>(z.batch, kBlocks)) * 3 * elems * 8 : 0;
  return z;
}

template <int SP>
void launch_rounds(const StackArgs& g, const Rounds& R, hipStream_t s) {
  const int blocks = SP == 128 ? std::min(g.count, kBlocks) : g.count;
  hipLaunchKernelGGL(rounds_kernel<SP>, dim3((unsigned)blocks), dim3(RoundShape<SP>::WAVES * 64), 0, s, g, R);
}

template <int DT, bool TALL, int SP>
void launch_all(const StackArgs& g, const Rounds& R, hipStream_t s) {
  hipLaunchKernelGGL((gram_kernel<DT, TALL, SP>), dim3((unsigned)(g.count * g.splits)), dim3(256), 0, s, g);
  launch_rounds<SP>(g, R, s);
  const int chunk = int64_t(g.count) * g.l >= int64_t(1) << 20 ? 1024 : 256;
  const int chunks = (g.l + chunk - 1) / chunk;
  hipLaunchKernelGGL((result_kernel<DT, TALL, SP>), dim3((unsigned)(g.count * chunks)), dim3(256), 0, s, g,
                     chunks, chunk);
}

typedef void (*Launch)(const StackArgs&, const Rounds&, hipStream_t);
template <int DT, bool TALL>
Launch launch_for(int sp) {
  return sp == 16 ? launch_all<DT, TALL, 16> : sp == 32 ? launch_all<DT, TALL, 32>
       : sp == 64 ? launch_all<DT, TALL, 64> : launch_all<DT, TALL, 128>;
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
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < z.total())
      return fail(MUON_ERR_WORKSPACE, "a workspace of %zu bytes, 256-byte aligned, is needed", z.total());
    auto range = [](const void* p, size_t bytes, bool written) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      return Range{lo, lo + bytes, written};
    };
    std::vector<Range> rs = {range(k.out, size_t(out_elems) * e, true), range(workspace, z.total(), true)};
    if (k.in != k.out || !std::equal(k.in_stride, k.in_stride + 4, k.out_stride))
      rs.push_back(range(k.in, size_t(in_elems) * e, false));
    if (int st = check_overlaps(rs)) return st;

    // the contiguous side is the long one, or the short one (TALL)
    const bool long_is_cols = k.cols >= k.rows;
    const bool tall = long_is_cols ? !by_cols : !by_rows;
    const int other = long_is_cols != tall ? 2 : 3;    // the side whose stride is free
    StackArgs g;
    g.in = k.in;
    g.out = k.out;
    g.in_outer = k.in_stride[0];
    g.in_inner = k.in_stride[1];
    g.in_ld = k.in_stride[other];
    g.out_outer = k.out_stride[0];
    g.out_inner = k.out_stride[1];
    g.out_ld = k.out_stride[other];
    g.inner = int(k.inner);
    g.s = z.s;
    g.l = z.l;
    g.splits = z.splits;
    g.span = z.span;
    char* at = static_cast<char*>(workspace);
    g.gram = reinterpret_cast<double*>(at);
    g.p = reinterpret_cast<float*>(at += z.gram);
    g.expo = reinterpret_cast<int*>(at += z.p);
    g.scratch = reinterpret_cast<double*>(at += z.expo);
    Rounds R;
    R.n = cfg->ns_steps;
    R.eps = cfg->eps;
    for (int n = 0; n < R.n; ++n)
      for (int c = 0; c < 3; ++c) R.abc[3 * n + c] = cfg->schedule ? cfg->schedule[3 * n + c] : (&cfg->a)[c];
    const Launch run = k.dtype == MUON_DT_F32
        ? (tall ? launch_for<1, true>(z.sp) : launch_for<1, false>(z.sp))
        : (tall ? launch_for<0, true>(z.sp) : launch_for<0, false>(z.sp));
    for (int64_t first = 0; first < z.count; first += z.batch) {
      g.first = first;
      g.count = int(std::min(z.batch, z.count - first));
      run(g, R, stream);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess)
        return fail(MUON_ERR_HIP, "launch of an orthogonalisation kernel failed: %s", hipGetErrorString(err));
    }
    return MUON_OK;
  });
}

}  // extern "C"
