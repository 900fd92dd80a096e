// The product of two matrices held in microscaled 4-bit values, out = A B^T (include/mx4.h), on the
// scaled matrix instructions: kernels and host side.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 rows x 64 values of either operand, one block of 32 values
// a lane (lane l: row l % 32, block l / 32), and that block's scale byte beside it, so that codes and
// scales go from memory into the instruction as they are held. Products are exact and sums are
// fp32. (With data-like operands and nothing else the matrix cores give 6.2 to 6.6 PFLOP/s by these and
// 3.7 by the 16x16x128 form.)
#include <algorithm>
#include <cmath>
#include <vector>

#include "mfma_common.h"
#include "mx4.h"
#include "mx4_common.h"

namespace muon {
namespace {

using mfma::ds_read_b128_at;
using mfma::f32x16;
using mfma::static_for;
using mfma::vm_wait;
using mfma::xcd_remap;
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct MmArgs {
  const uint8_t* a;
  const uint8_t* sa;
  const uint8_t* b;
  const uint8_t* sb;
  void* out;
  int64_t split_stride;                          // elements between the parts of a split product
  int m, n, steps;
  int panels_a, panels_b;
  int tiles_m, tiles_n, total;                   // total: tiles times splits
  int split_steps;                               // steps of a part
};

template <int OFF>
__device__ __forceinline__ uint32_t ds_read_b32_at(uint32_t addr) {
  uint32_t r;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "n"(OFF));
  return r;
}

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// 16 bytes of a row of out from element `at` on, of whose values `left` (any number) are there; OUT 0:
// bf16, 1: fp32.
template <int OUT>
__device__ __forceinline__ void store16(void* out, int64_t at, int left, u32x4 v) {
  constexpr int N = OUT == 0 ? 8 : 4;
  typedef u32x4 W __attribute__((aligned(2)));
  if (left >= N) {
    *reinterpret_cast<W*>(static_cast<char*>(out) + at * (16 / N)) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (e >= left) continue;
    if (OUT == 0) static_cast<uint16_t*>(out)[at + e] = uint16_t(v[e / 2] >> 16 * (e & 1));
    else static_cast<uint32_t*>(out)[at + e] = v[e % 4];
  }
}

// 4 values likewise.
template <int OUT>
__device__ __forceinline__ void store4(void* out, int64_t at, int left, f32x4 v) {
  if (left >= 4) {
    if (OUT == 0) {
      typedef u32x2 W __attribute__((aligned(2)));
      *reinterpret_cast<W*>(static_cast<uint16_t*>(out) + at) =
          u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
      *reinterpret_cast<f32x4_a4*>(static_cast<float*>(out) + at) = v;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) store_one<OUT>(out, at + e, v[e]);
}

// ---- tiles -----------------------------------------------------------------------------------
//
// Four waves (2 x 2) take a tile of 64 WM x 64 WN, each WM x WN blocks of 32 x 32. A step of 128
// columns is a stage of a ring of S in LDS: the tile's rows of 64 bytes of codes and 4 bytes of
// scales, loaded directly (16 rows, a contiguous kilobyte, an instruction). Chunk c of row r lies at
// c ^ (r / 4 % 4), so that a fragment's 64 lanes read all banks alike. In a stage the two slices of
// 64 columns are read in turn: while the matrix cores work on the first, the second's fragments
// arrive; then a barrier for the next stage; while they work on the second, the loads of the stage
// S ahead go out (into the buffer just read) and the next stage's first fragments arrive. Conditions
// on the stage are the compiler's (whole stages, the last ones), or it moves products past the reads
// (455 for 368 us below). Results leave through LDS as whole rows (368 for 325 us).
//
// bf16 out: 8192^3 245 us, 4.5 PFLOP/s; 16384 x 6400 x 6400 325 to 347, 3.9 to 4.1; 16384 x 6400 x 1600 103.
// The matrix cores alone would take 165 us for 8192^3 (6.6 PFLOP/s, with data-like operands, where power
// bounds them), without the loads it takes 222, without the stores 241. Tried: a stage's loads in two
// halves, one a slice (2 to 5% slower).
template <int WM, int WN, int S, int OUT>
__device__ __forceinline__ void mx_tile(const MmArgs& g) {
  constexpr int TM = 64 * WM, TN = 64 * WN;
  constexpr int PANELS = (TM + TN) / 16, PER = PANELS / 4;             // per stage, per wave
  constexpr int SLOADS = (TM + TN) / 64, SPER = (SLOADS + 3) / 4;      // of scales
  constexpr int LOADS = PER + SPER;
  constexpr int CODES = (TM + TN) * 64, STAGE = CODES + (TM + TN) * 4;
  __shared__ uint4 smem[S * STAGE / 16];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wr = wave >> 1, wc = wave & 1;

  // ---- the tile: an XCD has a contiguous range of them, in strips of four tiles' columns ----
  const int item = xcd_remap(blockIdx.x, g.total);
  const int tiles = g.tiles_m * g.tiles_n;
  const int z = item / tiles, tile = item - z * tiles;
  const int strip = tile / (4 * g.tiles_m), in = tile - strip * 4 * g.tiles_m;
  const int width = min(4, g.tiles_n - 4 * strip);
  const int tm = in / width, tn = 4 * strip + in - tm * width;
  const int row0 = tm * TM, col0 = tn * TN;
  const int k0 = z * g.split_steps, KT = min(g.steps - k0, g.split_steps);

  // ---- loads ----
  const char* src[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = wave * PER + i;
    const bool left = p < TM / 16;
    const int panel = left ? min(row0 / 16 + p, g.panels_a - 1)
                           : min(col0 / 16 + p - TM / 16, g.panels_b - 1);
    src[i] = reinterpret_cast<const char*>(left ? g.a : g.b) +
             (int64_t(panel) * g.steps + k0) * kMxTileBytes;
  }
  const char* ssrc[SPER];
  int sdst[SPER];
#pragma unroll
  for (int i = 0; i < SPER; ++i) {
    const int q = (wave * SPER + i) % SLOADS;    // (waves beyond the last load some again)
    const bool left = q < TM / 64;
    const int p = 4 * (left ? q : q - TM / 64) + lane / 16;
    const int panel = left ? min(row0 / 16 + p, g.panels_a - 1) : min(col0 / 16 + p, g.panels_b - 1);
    ssrc[i] = reinterpret_cast<const char*>(left ? g.sa : g.sb) +
              (int64_t(panel) * g.steps + k0) * kMxTileScales + lane % 16 * 4;
    sdst[i] = CODES + q * 256;
  }
  const uint32_t lane_at = lane / 4 * 64 + ((lane % 4) ^ (lane / 16)) * 16;
  char* const lds = reinterpret_cast<char*>(smem);
  auto load = [&](int kt, int buf, int op) {
    char* const st = lds + buf * STAGE;
    if (op < PER)
      __builtin_amdgcn_global_load_lds(src[op] + int64_t(kt) * kMxTileBytes + lane_at,
                                       MUON_LDS_PTR(st + (wave * PER + op) * 1024), 16, 0, 0);
    else
      __builtin_amdgcn_global_load_lds(ssrc[op - PER] + int64_t(kt) * kMxTileScales,
                                       MUON_LDS_PTR(st + sdst[op - PER]), 4, 0, 0);
  };

  // ---- fragments ----
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(MUON_LDS_PTR(smem)));
  const int r = lane & 31, h = lane >> 5, sw = (r >> 2) & 3;
  const uint32_t arow = (wr * 32 * WM + r) * 64, brow = (TM + wc * 32 * WN + r) * 64;
  const uint32_t ch0 = (h ^ sw) * 16, ch1 = ((2 + h) ^ sw) * 16;
  const uint32_t asc = CODES + (wr * 32 * WM + r) * 4, bsc = CODES + (TM + wc * 32 * WN + r) * 4;
  struct Frags {
    u32x4 a[WM], b[WN];
  } f0, f1;
  uint32_t na[WM], nb[WN], sa[WM], sb[WN];       // scales of the next stage and of this one
  f32x16 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = f32x16{};

  auto read = [&](uint32_t base, uint32_t ch, Frags& f, auto op_t) {
    constexpr int op = decltype(op_t)::value;
    if constexpr (op < WM) f.a[op] = ds_read_b128_at<2048 * op>(base + arow + ch);
    else f.b[op - WM] = ds_read_b128_at<2048 * (op - WM)>(base + brow + ch);
  };
  auto read_scale = [&](uint32_t base, auto op_t) {
    constexpr int op = decltype(op_t)::value;
    if constexpr (op < WM) na[op] = ds_read_b32_at<128 * op>(base + asc);
    else nb[op - WM] = ds_read_b32_at<128 * (op - WM)>(base + bsc);
  };
  // Waits for every LDS read; the results pass through empty assembly after the wait, so that no use
  // of them moves above it.
  auto arrived = [&](Frags& f) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < WM; ++i) asm volatile("" : "+v"(f.a[i]));
#pragma unroll
    for (int j = 0; j < WN; ++j) asm volatile("" : "+v"(f.b[j]));
  };
  auto scales_arrived = [&]() {                  // byte 2 s of a lane's scales is slice s's
#pragma unroll
    for (int i = 0; i < WM; ++i) {
      asm volatile("" : "+v"(na[i]));
      sa[i] = na[i] >> (8 * h);
    }
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      asm volatile("" : "+v"(nb[j]));
      sb[j] = nb[j] >> (8 * h);
    }
  };
  auto mma = [&](const Frags& f, auto m_t, auto slice_t) {
    constexpr int m = decltype(m_t)::value, i = m / WN, j = m % WN, op = 2 * decltype(slice_t)::value;
    const i32x8 x = {int(f.b[j][0]), int(f.b[j][1]), int(f.b[j][2]), int(f.b[j][3]), 0, 0, 0, 0};
    const i32x8 y = {int(f.a[i][0]), int(f.a[i][1]), int(f.a[i][2]), int(f.a[i][3]), 0, 0, 0, 0};
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc[i][j], 4, 4, op, int(sb[j]),
                                                               op, int(sa[i]));
  };
  // This wave's loads of a stage are there (`later` stages went out after it), then everyone's.
  auto stage_ready = [&](int later) {
    static_for<S>([&](auto N) {
      if (later == decltype(N)::value) vm_wait<decltype(N)::value * LOADS>();
    });
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  constexpr int READS = WM + WN, MMAS = WM * WN;
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  if (KT > 0) {
    for (int st = 0; st < min(S, KT); ++st)
#pragma unroll
      for (int op = 0; op < LOADS; ++op) load(st, st, op);
    stage_ready(min(S, KT) - 1);
    static_for<READS>([&](auto O) { read_scale(lds0, O); });
    static_for<READS>([&](auto O) { read(lds0, ch0, f0, O); });
    arrived(f0);
    scales_arrived();
  }
  // One stage. Whether there is one to refill the buffer with, and a next one, is known at compile
  // time: a branch between two products lets the compiler move products past the reads between them.
  int buf = 0;
  auto iteration = [&](int kt, auto refill_t, auto more_t) {
    constexpr bool refill = decltype(refill_t)::value, more = decltype(more_t)::value;
    const uint32_t cur = lds0 + buf * STAGE;
    const int nbuf = buf + 1 == S ? 0 : buf + 1;
    const uint32_t nxt = lds0 + nbuf * STAGE;
    __builtin_amdgcn_sched_barrier(0);
    static_for<MMAS>([&](auto M) {
      constexpr int m = decltype(M)::value;
      mma(f0, M, I0{});
      __builtin_amdgcn_sched_barrier(0);
      static_for<READS>([&](auto O) {
        if constexpr (decltype(O)::value * MMAS / READS / 2 == m) read(cur, ch1, f1, O);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    arrived(f1);
    if constexpr (refill) stage_ready(S - 2);
    else if constexpr (more) stage_ready(min(S - 2, KT - 2 - kt));
    __builtin_amdgcn_sched_barrier(0);
    static_for<MMAS>([&](auto M) {
      constexpr int m = decltype(M)::value;
      mma(f1, M, I1{});
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (refill)
        static_for<LOADS>([&](auto O) {
          if constexpr (decltype(O)::value * MMAS / LOADS == m) load(kt + S, buf, decltype(O)::value);
        });
      if constexpr (more)
        static_for<READS>([&](auto O) {
          if constexpr (decltype(O)::value * MMAS / READS / 2 == m) {
            read(nxt, ch0, f0, O);
            read_scale(nxt, O);
          }
        });
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (more) {
      arrived(f0);
      scales_arrived();
    }
    buf = nbuf;
  };
  using Yes = std::true_type;
  using No = std::false_type;
  int kt = 0;
  for (; kt < KT - S; ++kt) iteration(kt, Yes{}, Yes{});
  for (; kt < KT - 1; ++kt) iteration(kt, No{}, Yes{});
  if (KT > 0) iteration(KT - 1, No{}, No{});

  // ---- out: register quad q of lane l is row l % 32, columns 8 q + 4 (l / 32) .. + 3 of a block ----
  // 32 rows at a time go through a part of LDS of the wave's own (rows 16 bytes further apart than
  // they are long, so that the quads fall on all banks) and leave as whole rows, 16 bytes a lane.
  constexpr int E = OUT == 0 ? 2 : 4, COLS = 32 * WN, PITCH = COLS * E + 16;
  constexpr int LANES = COLS * E / 16, ROWS = 64 / LANES;      // lanes of a row, rows of a store
  static_assert(4 * 32 * PITCH <= S * STAGE, "the waves' parts fit the ring");
  __builtin_amdgcn_s_barrier();                  // everyone is done with the ring
  asm volatile("" ::: "memory");
  char* const part = lds + wave * (32 * PITCH);
  char* const out = static_cast<char*>(g.out) + z * g.split_stride * 4;
  const int col = col0 + wc * COLS + lane % LANES * (16 / E);
#pragma unroll
  for (int i = 0; i < WM; ++i) {
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        char* const to = part + r * PITCH + (32 * j + 8 * q + 4 * h) * E;
        const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if constexpr (OUT == 0)
          *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
          *reinterpret_cast<f32x4*>(to) = v;
      }
    asm volatile("" ::: "memory");               // a wave's LDS accesses complete in their order
    const int row0i = row0 + wr * 32 * WM + 32 * i;
#pragma unroll
    for (int k = 0; k < 32 / ROWS; ++k) {
      const int rr = k * ROWS + lane / LANES, row = row0i + rr;
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + rr * PITCH + lane % LANES * 16);
      if (row < g.m) store16<OUT>(out, int64_t(row) * g.n + col, g.n - col, v);
    }
    asm volatile("" ::: "memory");
  }
}

template <int WM, int WN, int S, int OUT>
__global__ __launch_bounds__(256, WM * WN == 16 ? 1 : 2) void mx_matmul_kernel(const MmArgs g) {
  mx_tile<WM, WN, S, OUT>(g);
}

// ---- few rows ----------------------------------------------------------------------------------
//
// Where one side has few rows the other operand (X) is read once and nothing else takes time: a
// block takes one panel of it, its waves the steps in turn, straight from memory into the 16x16x128
// instruction (a panel's step is a contiguous kilobyte, 16 bytes a lane), with one or two panels Y
// of the short side, which stay in the caches. The waves' sums are added in LDS in their order. LEFT:
// X is A. The operands' order puts four consecutive columns of out into a lane. One row x 6400 x 1600:
// 4.0 us in the kernel, 4.6 with the call, of which a launch is 3.6; 16 x 12800 x 6400 13.3 us, 3.3 TB/s.
template <int PANELS, int WAVES, bool LEFT, int OUT>
__device__ __forceinline__ void mx_few_tile(const MmArgs& g) {
  __shared__ f32x4 sums[PANELS][WAVES][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int panels_y = LEFT ? g.panels_b : g.panels_a;
  const uint8_t* const y = LEFT ? g.b : g.a;
  const uint8_t* const sy = LEFT ? g.sb : g.sa;
  // lane l: row l % 16, block l / 16
  const int at = lane % 16 * 64 + lane / 16 * 16, sat = lane % 16 * 4 + lane / 16;
  auto code = [&](const uint8_t* p, int64_t tile) {
    return *reinterpret_cast<const u32x4*>(p + tile * kMxTileBytes + at);
  };
  auto wide = [](u32x4 v) { return i32x8{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0}; };
  constexpr int AHEAD = 4;                       // steps whose loads are out at a time
  const int panel = blockIdx.x;
  const uint8_t* const x = (LEFT ? g.a : g.b) + int64_t(panel) * g.steps * kMxTileBytes;
  const uint8_t* const sx = (LEFT ? g.sa : g.sb) + int64_t(panel) * g.steps * kMxTileScales;
  f32x4 acc[PANELS] = {};
  for (int k = wave; k < g.steps; k += WAVES * AHEAD) {
    u32x4 cx[AHEAD], cy[AHEAD][PANELS];
    int bx[AHEAD], by[AHEAD][PANELS];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int ku = min(k + u * WAVES, g.steps - 1);
      cx[u] = code(x, ku);
      bx[u] = sx[int64_t(ku) * kMxTileScales + sat];
#pragma unroll
      for (int p = 0; p < PANELS; ++p) {
        const int64_t tile = int64_t(min(p, panels_y - 1)) * g.steps + ku;
        cy[u][p] = code(y, tile);
        by[u][p] = sy[tile * kMxTileScales + sat];
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      // (a step beyond the last is the last again with codes of 0: it adds 0, or a NaN that is there)
      if (k + u * WAVES >= g.steps) cx[u] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < PANELS; ++p)
        acc[p] = LEFT ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(cy[u][p]), wide(cx[u]), acc[p],
                                                                        4, 4, 0, by[u][p], 0, bx[u])
                      : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(cx[u]), wide(cy[u][p]), acc[p],
                                                                        4, 4, 0, bx[u], 0, by[u][p]);
    }
  }
#pragma unroll
  for (int p = 0; p < PANELS; ++p) sums[p][wave][lane] = acc[p];
  __syncthreads();
  // register e of lane l: row l % 16 of the second operand's panel, row 4 (l / 16) + e of the first's
  for (int p = wave; p < PANELS; p += WAVES) {
    f32x4 v = sums[p][0][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[p][w][lane];
    const int row = 16 * (LEFT ? panel : p) + lane % 16, col = 16 * (LEFT ? p : panel) + lane / 16 * 4;
    if (row < g.m) store4<OUT>(g.out, int64_t(row) * g.n + col, g.n - col, v);
  }
}

template <int PANELS, int WAVES, bool LEFT, int OUT>
__global__ __launch_bounds__(WAVES * 64) void mx_few_kernel(const MmArgs g) {
  mx_few_tile<PANELS, WAVES, LEFT, OUT>(g);
}

// The parts of a split product, added in their order.
template <int OUT>
__global__ __launch_bounds__(256) void mx_sum_kernel(const float* part, int64_t count, int parts,
                                                     void* out) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  if (i + 4 <= count) {
    f32x4 s = *reinterpret_cast<const f32x4_a4*>(part + i);
    for (int z = 1; z < parts; ++z) s += *reinterpret_cast<const f32x4_a4*>(part + z * count + i);
    store4<OUT>(out, i, 4, s);
  } else {
    for (int64_t e = i; e < count; ++e) {
      float s = part[e];
      for (int z = 1; z < parts; ++z) s += part[z * count + e];
      store_one<OUT>(out, e, s);
    }
  }
}

// ---- host ------------------------------------------------------------------------------------

// How a product is done: `few` panels of the short side (few rows), or tiles of 64 wm x 64 wn in
// `splits` parts of the steps.
struct Choice {
  int few;
  bool left;                                     // few: the long side is A's
  int wm, wn, splits;
};

// Few rows: up to 32, a long side of up to 16384 (8192 where there are more than 16 rows) and sums of up to
// 16384 (8192). Few rows and tiles, us: 1 x 6400 x 1600 5.1 and 8.3, 16 x 6400 x 6400 7.9 and 11.8,
// 1 x 12800 x 6400 13.2 and 14.8, 32 x 6400 x 6400 10.4 and 13.8; beyond, 1 x 50257 x 1600 11.0 and 10.2,
// 32 x 50257 x 1600 16.4 and 10.7, 32 x 12800 x 6400 18.5 and 14.3, 48 x 6400 x 6400 15.9 and 11.7.

// The tiles by estimated time, in us, from products measured on 256 compute units: a round of tiles
// takes `stage` for each step and `fixed` (first loads, results); tiles of 256 x 256 have a compute
// unit for themselves, the others two a unit. A split product's parts are written and read again (4 TB/s
// and a launch).
struct TileCost {
  int wm, wn, slots;
  double stage, fixed;
};
constexpr TileCost kTiles[] = {{4, 4, 256, 0.86, 6.0}, {2, 4, 512, 0.99, 1.6}, {4, 2, 512, 0.99, 1.6},
                               {2, 2, 512, 0.53, 1.75}};

Choice choose(int64_t m, int64_t n, int64_t steps) {
  Choice c{0, false, 4, 4, 1};
  const int64_t few = mx_panels(std::min(m, n));
  if (few <= 2 && few * mx_panels(std::max(m, n)) <= 1024 && few * steps <= 128) {
    c.left = m > n;
    c.few = int(few);
    return c;
  }
  double best = 1e300;
  for (const TileCost& t : kTiles) {
    const int64_t count = ((m + 64 * t.wm - 1) / (64 * t.wm)) * ((n + 64 * t.wn - 1) / (64 * t.wn));
    for (int64_t z = 1; z == 1 || (z <= 64 && 2 * z <= steps && count * z <= 2 * t.slots); ++z) {
      const double rounds = double(count * z) / t.slots;
      const double each = double((steps + z - 1) / z) * t.stage + t.fixed;
      double time = (rounds > 4 ? rounds + 0.5 : std::ceil(rounds)) * each;
      if (z > 1) time += 3 + double(m) * double(n) * 8e-6 * double(z) / 4;
      if (time < best) {
        best = time;
        c.wm = t.wm;
        c.wn = t.wn;
        c.splits = int(z);
      }
    }
  }
  return c;
}

bool limits_ok(int64_t m, int64_t n, int64_t k) {
  return mx_sides_ok(m, k) && mx_sides_ok(n, k) && mx_sides_ok(m, n) &&
         ((m + 127) / 128) * ((n + 127) / 128) <= (int64_t(1) << 23);
}

int parts_of(const Choice& c, int64_t steps) {
  const int64_t each = (steps + c.splits - 1) / c.splits;      // (few rows: one part)
  return steps == 0 ? 1 : int((steps + each - 1) / each);
}

template <int OUT, int PANELS, bool LEFT>
void launch_few(const MmArgs& g, hipStream_t s) {
  const unsigned blocks = unsigned(LEFT ? g.panels_a : g.panels_b);
  if (g.steps <= 16)
    hipLaunchKernelGGL((mx_few_kernel<PANELS, 4, LEFT, OUT>), dim3(blocks), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((mx_few_kernel<PANELS, 8, LEFT, OUT>), dim3(blocks), dim3(512), 0, s, g);
}

template <int OUT>
void launch(const Choice& c, const MmArgs& g, hipStream_t s) {
  if (c.few == 1) return c.left ? launch_few<OUT, 1, true>(g, s) : launch_few<OUT, 1, false>(g, s);
  if (c.few == 2) return c.left ? launch_few<OUT, 2, true>(g, s) : launch_few<OUT, 2, false>(g, s);
  const dim3 grid((unsigned)g.total), block(256);
  if (c.wm == 4 && c.wn == 4) hipLaunchKernelGGL((mx_matmul_kernel<4, 4, 4, OUT>), grid, block, 0, s, g);
  else if (c.wm == 4) hipLaunchKernelGGL((mx_matmul_kernel<4, 2, 3, OUT>), grid, block, 0, s, g);
  else if (c.wn == 4) hipLaunchKernelGGL((mx_matmul_kernel<2, 4, 3, OUT>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((mx_matmul_kernel<2, 2, 4, OUT>), grid, block, 0, s, g);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_mx_matmul_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (!limits_ok(m, n, k)) return SIZE_MAX;
  if (m == 0 || n == 0 || k == 0) return 0;
  const int parts = parts_of(choose(m, n, mx_steps(k)), mx_steps(k));
  return parts > 1 ? size_t(parts) * size_t(m) * size_t(n) * 4 : 0;
}

int muon_mx_matmul(const void* a_codes, const void* a_scales, const void* b_codes,
                   const void* b_scales, int64_t m, int64_t n, int64_t k, void* out,
                   muon_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return c_entry([&]() -> int {
    if (!dtype_known(dtype)) return fail(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (m < 0 || n < 0 || k < 0) return fail(MUON_ERR_INVALID_ARG, "negative size");
    if (!limits_ok(m, n, k))
      return fail(MUON_ERR_UNSUPPORTED, "sides up to 2^31 - 256, 2^40 values a matrix and 2^23 tiles "
                  "of 128 x 128 in out");
    if (m == 0 || n == 0) return MUON_OK;
    if (!out || (reinterpret_cast<uintptr_t>(out) & (dtype_bytes(dtype) - 1)))
      return fail(MUON_ERR_INVALID_ARG, "out must be non-NULL and aligned to its elements");
    if (k > 0)
      for (const void* p : {a_codes, a_scales, b_codes, b_scales})
        if (!p || !is_aligned16(p))
          return fail(MUON_ERR_INVALID_ARG, "codes and scales must be non-NULL and 16-byte aligned");
    const size_t need = muon_mx_matmul_workspace_size(m, n, k);
    if (need > 0 && (!workspace || !is_aligned16(workspace) || workspace_bytes < need))
      return fail(MUON_ERR_WORKSPACE, "a workspace of %zu bytes, 16-byte aligned, is needed", need);
    std::vector<Range> rs = {mx_range(out, size_t(m) * size_t(n) * dtype_bytes(dtype), true),
                             mx_range(workspace, need, true)};
    if (k > 0) {
      rs.push_back(mx_range(a_codes, muon_mx_codes_size(m, k), false));
      rs.push_back(mx_range(a_scales, muon_mx_scales_size(m, k), false));
      rs.push_back(mx_range(b_codes, muon_mx_codes_size(n, k), false));
      rs.push_back(mx_range(b_scales, muon_mx_scales_size(n, k), false));
    }
    if (int st = check_overlaps(rs)) return st;

    const int64_t steps = mx_steps(k);
    const Choice c = choose(m, n, steps);
    const int parts = parts_of(c, steps);
    MmArgs g;
    g.a = static_cast<const uint8_t*>(a_codes);
    g.sa = static_cast<const uint8_t*>(a_scales);
    g.b = static_cast<const uint8_t*>(b_codes);
    g.sb = static_cast<const uint8_t*>(b_scales);
    g.out = parts > 1 ? workspace : out;
    g.split_stride = m * n;
    g.m = (int)m;
    g.n = (int)n;
    g.steps = (int)steps;
    g.panels_a = (int)mx_panels(m);
    g.panels_b = (int)mx_panels(n);
    g.tiles_m = (int)((m + 64 * c.wm - 1) / (64 * c.wm));
    g.tiles_n = (int)((n + 64 * c.wn - 1) / (64 * c.wn));
    g.total = g.tiles_m * g.tiles_n * parts;
    g.split_steps = (int)((steps + c.splits - 1) / c.splits);
    if (parts > 1 || dtype == MUON_DT_F32) launch<1>(c, g, stream);
    else launch<0>(c, g, stream);
    if (int st = mx_launched("4-bit product")) return st;
    if (parts > 1) {
      const int64_t blocks = (m * n + 1023) / 1024;
      if (dtype == MUON_DT_F32)
        hipLaunchKernelGGL(mx_sum_kernel<1>, dim3((unsigned)blocks), dim3(256), 0, stream,
                           static_cast<const float*>(workspace), m * n, parts, out);
      else
        hipLaunchKernelGGL(mx_sum_kernel<0>, dim3((unsigned)blocks), dim3(256), 0, stream,
                           static_cast<const float*>(workspace), m * n, parts, out);
      return mx_launched("4-bit product's sum");
    }
    return MUON_OK;
  });
}

}  // extern "C"
