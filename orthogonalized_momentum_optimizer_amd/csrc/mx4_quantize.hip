// Microscaled 4-bit quantisation of matrices, as they lie and transposed, and the way back: the
// host side and kernels of the C ABI in include/mx4.h.
//
// One read of a source serves both results. Bytes per value: 2 or 4 read, 17/32 written for each
// result; back 17/32 read, 2 or 4 written.
#include <algorithm>
#include <climits>
#include <vector>

#include "mx4.h"
#include "mx4_common.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxItems = 60;                    // matrices per launch, by value

struct Item {
  const void* x;
  int64_t ld;
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* codes_t;
  uint8_t* scales_t;
  int rows, cols;
  int first;                                     // its first block in its launch
  int tiles_n;                                   // tiles across its columns
};

struct QuantLaunch {
  int count;
  uint32_t key;
  Item item[kMaxItems];
};
static_assert(sizeof(QuantLaunch) <= 4096, "kernel arguments");

// ---- blocks ----------------------------------------------------------------------------------

// The smallest byte b with top <= 6 * 2^(b - 127), from the bits of top >= 0: top = 2^(E - 127) f
// has b = E - 2, or E - 1 if f > 3/2. 255 where top is not finite.
__device__ __forceinline__ int block_byte(uint32_t top) {
  const int b = int((top + 0x3fffffu) >> 23) - 2;
  return top >= 0x7f800000u ? 255 : max(b, 0);
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  return max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xf, 0xf, false)));
}

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0xEB26D985u;
  x = (x ^ (x >> 15)) * 0x4A08C6EDu;
  return x ^ (x >> 16);
}

// What the conversions leave to be done where the scale is 255 (codes 0) or 2^126 (where code 6 would
// stand for 2^128: code 5).
__device__ __forceinline__ uint32_t at_the_top(uint32_t c, int byte) {
  if (byte == 255) return 0;
  if (byte == 253) c -= (c >> 2) & (c >> 1) & ~c & 0x11111111u;
  return c;
}

// 8 values, a dword of codes, by the hardware's scaled conversions of a pair: to nearest even, or
// stochastically by a 32-bit number, of which the first value takes all 32 bits as a fraction of a
// step and the second the lower 31. For halves of their own the pair is converted twice. (Measured over
// all ties, random values and numbers, every scale and subnormals: bit by bit what mx4.h defines,
// but the stochastic conversion of bf16 pairs, which cuts fractions below a quarter of the first
// step; so those go as fp32. The stochastic ones also leave the other bytes of their result
// undefined in the compiler's hands, so each has a register of its own.)
struct Pair32 {
  f32x2 v;
  template <int K>
  __device__ __forceinline__ uint32_t nearest(uint32_t old, float s) const {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, v[0], v[1], s, K);
  }
  __device__ __forceinline__ f32x2 values() const { return v; }
};
struct Pair16 {
  uint32_t w;
  template <int K>
  __device__ __forceinline__ uint32_t nearest(uint32_t old, float s) const {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, w), s, K);
  }
  __device__ __forceinline__ f32x2 values() const {
    return f32x2{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
  }
};

// A register whose every bit the next conversions write.
__device__ __forceinline__ uint32_t unset() {
  uint32_t w;
  asm("" : "=v"(w));
  return w;
}

// The lowest bytes of four registers.
__device__ __forceinline__ uint32_t low_bytes(const uint32_t (&b)[4]) {
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u), lo, 0x05040100u);
}

// pair(k), k = 0..3; j: the column of the first value over 2.
template <bool STOCH, typename F>
__device__ __forceinline__ uint32_t encode8(F&& pair, int byte, uint32_t j, uint32_t row_key) {
  const float s = mx_scale(min(byte, 253));
  uint32_t c;
  if (!STOCH) {
    c = unset();
    c = pair(0).template nearest<0>(c, s);
    c = pair(1).template nearest<1>(c, s);
    c = pair(2).template nearest<2>(c, s);
    c = pair(3).template nearest<3>(c, s);
  } else {
    uint32_t first[4], second[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t h = mix32((j + k) ^ row_key);
      const f32x2 v = pair(k).values();
      first[k] = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, v, h << 16 | 0x8000u, s, 0);
      second[k] =
          __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, v, (h & 0xffff0000u) >> 1 | 0x4000u, s, 0);
    }
    c = (low_bytes(first) & 0x0f0f0f0fu) | (low_bytes(second) & 0xf0f0f0f0u);
  }
  return at_the_top(c, byte);
}

// ---- loads -----------------------------------------------------------------------------------

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));   // rows of odd length start anywhere
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

// 8 consecutive values as they are held: 4 dwords of bf16 or 8 of fp32.
template <int DT>
struct Eight {
  u32x4 w[DT ? 2 : 1];

  // from column `col` of a row of `cols`; 0 beyond it
  __device__ __forceinline__ void load(const char* row, int col, int cols) {
    if (col + 8 <= cols) {
      if (DT == 0) {
        w[0] = *reinterpret_cast<const u32x4_a2*>(row + int64_t(col) * 2);
      } else {
        const u32x4_a4* p = reinterpret_cast<const u32x4_a4*>(row + int64_t(col) * 4);
        w[0] = p[0];
        w[DT ? 1 : 0] = p[DT ? 1 : 0];
      }
      return;
    }
    clear();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (col + e >= cols) continue;
      if (DT == 0)
        w[0][e / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[col + e]) << 16 * (e & 1);
      else
        w[DT ? e / 4 : 0][e % 4] = reinterpret_cast<const uint32_t*>(row)[col + e];
    }
  }
  __device__ __forceinline__ void clear() {
    w[0] = u32x4{0, 0, 0, 0};
    if (DT) w[DT ? 1 : 0] = u32x4{0, 0, 0, 0};
  }
  // the bits of the largest magnitude, as fp32's
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if (DT == 0) {
      uint32_t hi = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m = max(m, w[0][k] << 16 & 0x7fff0000u);
        hi = max(hi, w[0][k] & 0x7fff0000u);
      }
      return max(m, hi);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, max(w[0][k] & 0x7fffffffu, w[DT ? 1 : 0][k] & 0x7fffffffu));
    return m;
  }
  __device__ __forceinline__ auto pair(int k) const {
    if constexpr (DT == 0)
      return Pair16{w[0][k]};
    else
      return Pair32{f32x2{__uint_as_float(w[k / 2][2 * (k % 2)]),
                          __uint_as_float(w[k / 2][2 * (k % 2) + 1])}};
  }
};

// ---- the kernel ------------------------------------------------------------------------------
//
// A block takes a tile of TR rows x 128 columns, a step of the result as it lies: 16 lanes have a row,
// 8 values each, and a pass of the block's 256 threads is one panel's step, whose codes leave as one
// contiguous kilobyte. For the transposed result the tile (128 rows, a step of that one) goes through
// LDS: a thread then takes two neighbouring columns of 32 rows, four threads in a row their 128 rows,
// and 16 bytes of codes leave for each column. A row's 64-byte quarters are exchanged by the block of
// rows (XOR with row / 32), so that the 64 lanes of a read, 16 column pairs by four blocks of rows,
// fall on 64 different banks. Tiles are taken whole so that one read serves both results: two passes
// would read 2 or 4 bytes a value again, more than all that is written.
//
// bf16 16384 x 6400 in both layouts: 67 to 82 us, 4.0 TB/s of the 321 MB that move (a copy of 1 GB: 4.8 to
// 5.0); stochastically 104 to 114: the random bits and the step around each value are instructions that
// the same traffic does not cover. fp32 1013 x 1601, 104 blocks, stochastically: 12.6.
template <int DT, bool ROWS, bool COLS, bool STOCH>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const QuantLaunch L) {
  constexpr int E = DT ? 4 : 2;
  constexpr int TR = COLS ? 128 : 64, PASSES = TR / 16;
  constexpr int PITCH = 128 * E;                 // bytes of a tile's row in LDS
  __shared__ uint4 smem[COLS ? 128 * PITCH / 16 : 1];
  char* const lds = reinterpret_cast<char*>(smem);

  const int b = blockIdx.x, t = threadIdx.x;
  const int q = find_tensor([&](int i) { return L.item[i].first; }, L.count, b);
  const Item& I = L.item[q];
  const int rows = I.rows, cols = I.cols;
  const int tile = b - I.first, tr = tile / I.tiles_n, tc = tile - tr * I.tiles_n;
  const int row0 = tr * TR, col0 = tc * 128;
  const int lane8 = t % 16 * 8;

  Eight<DT> x[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int row = row0 + p * 16 + t / 16;
    if (row < rows)
      x[p].load(static_cast<const char*>(I.x) + int64_t(row) * I.ld * E, col0 + lane8, cols);
    else
      x[p].clear();
  }
  if constexpr (COLS) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * 16 + t / 16;
      char* const to = lds + r * PITCH + ((lane8 * E) ^ (r / 32 * (PITCH / 4)));
      reinterpret_cast<u32x4*>(to)[0] = x[p].w[0];
      if (DT) reinterpret_cast<u32x4*>(to)[1] = x[p].w[DT ? 1 : 0];
    }
  }
  if constexpr (ROWS) {
    const int panels = (rows + 15) / 16, steps = I.tiles_n;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int panel = row0 / 16 + p;
      if (panel >= panels) break;
      const uint32_t top = quad_max<0x4E>(quad_max<0xB1>(x[p].top()));
      const int byte = block_byte(top);
      const int row = row0 + p * 16 + t / 16;
      const uint32_t c = encode8<STOCH>([&](int k) { return x[p].pair(k); }, byte,
                                        uint32_t(col0 + lane8) / 2, STOCH ? mix32(row ^ L.key) : 0);
      const int64_t at = int64_t(panel) * steps + tc;
      reinterpret_cast<uint32_t*>(I.codes + at * kMxTileBytes)[t] = c;
      if (t % 4 == 0) I.scales[at * kMxTileScales + t / 4] = uint8_t(byte);
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int rb = t % 4, cp = t / 4;            // rows 32 rb.., columns 2 cp and 2 cp + 1
    const char* const from = lds + rb * 32 * PITCH + ((cp * 2 * E) ^ (rb * (PITCH / 4)));
    const int panels = (cols + 15) / 16, steps = (rows + 127) / 128;
    const int panel = col0 / 16 + cp / 8;
    if (panel >= panels) return;
    const int64_t at = int64_t(panel) * steps + tr;
    uint32_t w0[32], w1[DT ? 32 : 1];
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      if (DT == 0) {
        w0[r] = *reinterpret_cast<const uint32_t*>(from + r * PITCH);
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(from + r * PITCH);
        w0[r] = w[0];
        w1[DT ? r : 0] = w[1];
      }
    }
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      top[0] = max(top[0], DT ? w0[r] & 0x7fffffffu : w0[r] << 16 & 0x7fff0000u);
      top[1] = max(top[1], DT ? w1[DT ? r : 0] & 0x7fffffffu : w0[r] & 0x7fff0000u);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = col0 + 2 * cp + h;
      const int byte = block_byte(top[h]);
      const uint32_t row_key = STOCH ? mix32(uint32_t(col) ^ L.key) : 0;
      u32x4 c;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        c[k] = encode8<STOCH>(
            [&](int e) {
              const int r = 8 * k + 2 * e;
              if constexpr (DT == 0)
                return Pair16{h ? (w0[r] >> 16) | (w0[r + 1] & 0xffff0000u)
                                : (w0[r] & 0xffffu) | (w0[r + 1] << 16)};
              else
                return Pair32{h ? f32x2{__uint_as_float(w1[r]), __uint_as_float(w1[r + 1])}
                                : f32x2{__uint_as_float(w0[r]), __uint_as_float(w0[r + 1])}};
            },
            byte, uint32_t(row0 + 32 * rb + 8 * k) / 2, row_key);
      const int pr = col % 16;
      *reinterpret_cast<u32x4*>(I.codes_t + at * kMxTileBytes + pr * 64 + rb * 16) = c;
      I.scales_t[at * kMxTileScales + pr * 4 + rb] = uint8_t(byte);
    }
  }
}

// ---- the way back ----------------------------------------------------------------------------

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// A thread takes a dword of codes, 8 values; a block four panel's steps, in the order of the codes.
// bf16 16384 x 6400: 48 to 51 us, 5.3 TB/s, the rate of writes.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint32_t* codes,
                                                                const uint8_t* scales, int rows,
                                                                int cols, int steps, int64_t tiles,
                                                                void* out) {
  for (int p = 0; p < 4; ++p) {
    const int64_t at = int64_t(blockIdx.x) * 4 + p;
    if (at >= tiles) return;
    const int panel = int(at / steps), step = int(at - int64_t(panel) * steps);
    const int row = panel * 16 + threadIdx.x / 16, col = step * 128 + threadIdx.x % 16 * 8;
    if (row >= rows || col >= cols) continue;
    const uint32_t c = codes[at * (kMxTileBytes / 4) + threadIdx.x];
    const int byte = scales[at * kMxTileScales + threadIdx.x / 4];
    const float s = byte == 255 ? __uint_as_float(0x7f800000u) : mx_scale(byte);
    f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    const int64_t to = int64_t(row) * cols + col;
    if (col + 8 <= cols) {
      if (DT == 0) {
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(v[k][0], v[k][1]);
        *reinterpret_cast<u32x4_a2*>(static_cast<uint16_t*>(out) + to) = w;
      } else {
        f32x4_a4* const p4 = reinterpret_cast<f32x4_a4*>(static_cast<float*>(out) + to);
        p4[0] = f32x4{v[0][0], v[0][1], v[1][0], v[1][1]};
        p4[1] = f32x4{v[2][0], v[2][1], v[3][0], v[3][1]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < cols) store_one<DT>(out, to + e, v[e / 2][e % 2]);
    }
  }
}

// ---- host ------------------------------------------------------------------------------------

uint32_t key_of(uint64_t z) {
  z = (z ^ (z >> 32)) * 0xE9F8AC216EBC06F5ull;
  z = (z ^ (z >> 32)) * 0xE9F8AC216EBC06F5ull;
  return uint32_t(z ^ (z >> 32));
}

typedef void (*Quantize)(const QuantLaunch);
template <int DT, bool STOCH>
Quantize kernel_for(bool r, bool c) {
  if (r && c) return mx_quantize_kernel<DT, true, true, STOCH>;
  return r ? mx_quantize_kernel<DT, true, false, STOCH> : mx_quantize_kernel<DT, false, true, STOCH>;
}
Quantize kernel_for(int dt, bool stoch, bool r, bool c) {
  if (dt) return stoch ? kernel_for<1, true>(r, c) : kernel_for<1, false>(r, c);
  return stoch ? kernel_for<0, true>(r, c) : kernel_for<0, false>(r, c);
}

// What one launch can hold: kind 0 to 5 of a source, by dtype and the results asked for.
int kind_of(const muon_mx_source& s) {
  return 3 * int(s.dtype == MUON_DT_F32) + (s.codes ? (s.codes_t ? 2 : 0) : 1);
}

constexpr int64_t kMostTiles = int64_t(1) << 23; // per launch: under 2^32 threads
int tile_rows(const muon_mx_source& s) { return s.codes_t ? 128 : 64; }
int64_t tiles_of(const muon_mx_source& s) {
  return (s.rows + tile_rows(s) - 1) / tile_rows(s) * mx_steps(s.cols);
}

int check_source(const muon_mx_source& s, int64_t i, std::vector<Range>& rs) {
  const long long at = (long long)i;
  if (!dtype_known(s.dtype)) return fail(MUON_ERR_INVALID_ARG, "source %lld: unknown dtype", at);
  if (s.rows < 0 || s.cols < 0)
    return fail(MUON_ERR_INVALID_ARG, "source %lld: negative size", at);
  if (!mx_sides_ok(s.rows, s.cols))
    return fail(MUON_ERR_UNSUPPORTED, "source %lld: sides up to 2^31 - 256 and 2^40 values", at);
  if (!s.codes != !s.scales || !s.codes_t != !s.scales_t)
    return fail(MUON_ERR_INVALID_ARG, "source %lld: codes without scales, or scales without codes", at);
  if (s.rows == 0 || s.cols == 0) return MUON_OK;
  if (tiles_of(s) > kMostTiles)
    return fail(MUON_ERR_UNSUPPORTED, "source %lld: more than 2^23 tiles of %d x 128", at, tile_rows(s));
  if (!s.codes && !s.codes_t)
    return fail(MUON_ERR_INVALID_ARG, "source %lld: no result to write", at);
  const size_t e = dtype_bytes(s.dtype);
  if (!s.x || (reinterpret_cast<uintptr_t>(s.x) & (e - 1)))
    return fail(MUON_ERR_INVALID_ARG, "source %lld: x must be non-NULL and aligned to its elements", at);
  if (s.rows > 1 && (s.row_stride < s.cols || s.row_stride > kMxMaxElems))
    return fail(MUON_ERR_INVALID_ARG, "source %lld: row_stride must be at least cols", at);
  for (const void* p : {s.codes, s.scales, s.codes_t, s.scales_t})
    if (!is_aligned16(p))
      return fail(MUON_ERR_INVALID_ARG, "source %lld: codes and scales must be 16-byte aligned", at);
  const int64_t ld = s.rows > 1 ? s.row_stride : s.cols;
  rs.push_back(mx_range(s.x, size_t((s.rows - 1) * ld + s.cols) * e, false));
  if (s.codes) {
    rs.push_back(mx_range(s.codes, muon_mx_codes_size(s.rows, s.cols), true));
    rs.push_back(mx_range(s.scales, muon_mx_scales_size(s.rows, s.cols), true));
  }
  if (s.codes_t) {
    rs.push_back(mx_range(s.codes_t, muon_mx_codes_size(s.cols, s.rows), true));
    rs.push_back(mx_range(s.scales_t, muon_mx_scales_size(s.cols, s.rows), true));
  }
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_mx_codes_size(int64_t rows, int64_t cols) {
  if (!mx_sides_ok(rows, cols)) return SIZE_MAX;
  return size_t(mx_panels(rows)) * size_t(mx_steps(cols)) * kMxTileBytes;
}

size_t muon_mx_scales_size(int64_t rows, int64_t cols) {
  if (!mx_sides_ok(rows, cols)) return SIZE_MAX;
  return size_t(mx_panels(rows)) * size_t(mx_steps(cols)) * kMxTileScales;
}

int muon_mx_quantize(const muon_mx_source* sources, int64_t n, int stochastic, uint64_t seed,
                     hipStream_t stream) {
  return c_entry([&]() -> int {
    if (n < 0 || (n > 0 && !sources)) return fail(MUON_ERR_INVALID_ARG, "sources is NULL or n < 0");
    if (stochastic != 0 && stochastic != 1)
      return fail(MUON_ERR_INVALID_ARG, "stochastic must be 0 or 1");
    std::vector<Range> rs;
    rs.reserve(size_t(n) * 5);
    for (int64_t i = 0; i < n; ++i)
      if (int st = check_source(sources[i], i, rs)) return st;
    if (int st = check_overlaps(rs)) return st;
    QuantLaunch L;
    L.key = key_of(seed);
    for (int kind = 0; kind < 6; ++kind) {
      const int dt = kind / 3;
      const bool rows = kind % 3 != 1, cols = kind % 3 != 0;
      L.count = 0;
      int64_t blocks = 0;
      auto flush = [&]() -> int {
        if (L.count == 0) return MUON_OK;
        hipLaunchKernelGGL(kernel_for(dt, stochastic, rows, cols), dim3((unsigned)blocks),
                           dim3(kThreads), 0, stream, L);
        L.count = 0;
        blocks = 0;
        return mx_launched("4-bit quantisation");
      };
      for (int64_t i = 0; i < n; ++i) {
        const muon_mx_source& s = sources[i];
        if (kind_of(s) != kind || s.rows == 0 || s.cols == 0) continue;
        const int64_t tiles = tiles_of(s);
        if (L.count == kMaxItems || blocks + tiles > kMostTiles)
          if (int st = flush()) return st;
        L.item[L.count++] = {s.x, s.rows > 1 ? s.row_stride : s.cols,
                             static_cast<uint8_t*>(s.codes), static_cast<uint8_t*>(s.scales),
                             static_cast<uint8_t*>(s.codes_t), static_cast<uint8_t*>(s.scales_t),
                             (int)s.rows, (int)s.cols, (int)blocks, (int)mx_steps(s.cols)};
        blocks += tiles;
      }
      if (int st = flush()) return st;
    }
    return MUON_OK;
  });
}

int muon_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols,
                       void* out, muon_dtype dtype, hipStream_t stream) {
  return c_entry([&]() -> int {
    if (!dtype_known(dtype)) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (rows < 0 || cols < 0) return fail(MUON_ERR_INVALID_ARG, "negative size");
    if (!mx_sides_ok(rows, cols))
      return fail(MUON_ERR_UNSUPPORTED, "sides up to 2^31 - 256 and 2^40 values");
    if (rows == 0 || cols == 0) return MUON_OK;
    const int64_t steps = mx_steps(cols), tiles = mx_panels(rows) * steps;
    const int64_t blocks = (tiles + 3) / 4;
    if (blocks > kMostTiles)
      return fail(MUON_ERR_UNSUPPORTED, "more than 2^25 tiles of 16 x 128");
    const size_t e = dtype_bytes(dtype);
    if (!codes || !scales || !is_aligned16(codes) || !is_aligned16(scales))
      return fail(MUON_ERR_INVALID_ARG, "codes and scales must be non-NULL and 16-byte aligned");
    if (!out || (reinterpret_cast<uintptr_t>(out) & (e - 1)))
      return fail(MUON_ERR_INVALID_ARG, "out must be non-NULL and aligned to its elements");
    std::vector<Range> rs = {mx_range(codes, muon_mx_codes_size(rows, cols), false),
                             mx_range(scales, muon_mx_scales_size(rows, cols), false),
                             mx_range(out, size_t(rows) * size_t(cols) * e, true)};
    if (int st = check_overlaps(rs)) return st;
    auto kernel = dtype == MUON_DT_F32 ? mx_dequantize_kernel<1> : mx_dequantize_kernel<0>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream,
                       static_cast<const uint32_t*>(codes), static_cast<const uint8_t*>(scales),
                       (int)rows, (int)cols, (int)steps, tiles, out);
    return mx_launched("4-bit dequantisation");
  });
}

}  // extern "C"
