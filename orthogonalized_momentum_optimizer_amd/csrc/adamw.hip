// AdamW over many tensors at once, with fp32 or 8-bit states: host side and kernels of the C
// ABI in include/adamw.h.
//
// One pass over HBM either way: every buffer is read once and written once. Bytes per element:
//   fp32 states   g + 2p + 16:    22 for bf16 p and g, 28 for fp32; 28 for bf16 with a master
//   8-bit states  g + 2p + 4:     10 for bf16 p and g, 16 for fp32; 16 for bf16 with a master
#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "adamw.h"
#include "tensor_list.h"

namespace muon {
namespace {

// Both kernels are bound by HBM, and how fast it goes depends on how they ask for it. Measured on
// GPT-2-124M's tables (154 M elements, bf16, fp32 states, 3.40 GB), one choice changed at a time:
//   8 elements per thread, cached                                    632 us   5.4 TB/s
//   4 elements per thread, so that each access of a wave is one
//     contiguous run of whole lines (1 KB of an fp32 stream)         622 us
//   blocks of one wave                                               598 us
//   at most 16 waves per compute unit and not 32                     574 us   5.9 TB/s
//   nontemporal loads and stores                                     506 us   6.7 TB/s
// (a copy of 4 GB reaches 4.9 to 5.4 TB/s). Fewer bytes in flight keep the streams' rows together;
// with 13 waves the time is up again (539 us). Nontemporal accesses pay only together, and only
// where they are whole lines: with 8 elements per thread they cost 10%.
constexpr int kThreadsF32 = 64;
constexpr int kVec = 4;
constexpr int kChunkF32 = kThreadsF32 * kVec;
// Shared memory that such a block asks for and does not use: 16 blocks fit a compute unit, not 32.
constexpr int kHoldF32 = 10000;
// 8-bit states: GPT-2-124M's tables 274 us cached and with 16 neighbouring elements per lane, 242
// with whole lines and nontemporal accesses (6.4 TB/s); blocks of 64, 128 and 512 threads 0 to 4%
// slower. Here 5 blocks per compute unit measured 1% better than the 6 that fit.
constexpr int kThreads = 256;
constexpr int kChunk = 4096;                     // elements per block
constexpr int kHold = 30000;
constexpr int kOwn = kChunk / kThreads;          // elements per thread

constexpr int kMaxItems = 480;                   // tensors per launch: their gradients' addresses
                                                 // travel by value, the rest is in the table
constexpr int64_t kPiece = int64_t(1) << 31;     // elements of a tensor in one item, fp32 states
constexpr int64_t kMaxBlocks = int64_t(1) << 23; // per launch: under 2^32 threads
static_assert(kPiece / kChunkF32 <= kMaxBlocks && kMaxTensorElems / kChunk <= kMaxBlocks,
              "an item fits a launch");

// Parameter modes: a bf16 parameter, an fp32 one, a bf16 one with an fp32 master copy.
enum { kBf16 = 0, kF32 = 1, kMaster = 2 };

// One tensor, or piece of one, in the plan's device table: what does not change from step to step.
struct Item {
  void* p;
  float* w;                                      // master
  void* m;
  void* v;
  uint8_t* ms;                                   // scales of the 8-bit states
  uint8_t* vs;
  int64_t numel;
  float wd_mul;
  int first;                                     // its first block in its launch
};
static_assert(sizeof(Item) == 64, "one line of the scalar cache");

struct Step {
  float lr, beta1, beta2, eps, weight_decay;
  float inv_bc1;                                 // 1 / (1 - beta1^t)
  float inv_sqrt_bc2;                            // 1 / sqrt(1 - beta2^t)
  const float* grad_scale;
  int skip_nonfinite;
  int stochastic;
  uint32_t key;
};

struct AdamwLaunch {
  const Item* item;
  const int* first;                              // the items' first blocks, packed
  int count;
  Step s;
  const void* g[kMaxItems];
};
static_assert(sizeof(AdamwLaunch) <= 4096, "kernel arguments");

// The table, which no kernel writes while steps run, through the scalar cache: its lines stay
// there, where vector loads of it would queue with the streams of the tensors.
template <typename T>
using Constant = const __attribute__((address_space(4))) T*;

// The tensor of block b, by one or two vector loads. (A bisection by scalar loads instead: 154 M
// elements in 1 to 480 equal tensors, bf16, fp32 states 547 to 563 us and 544 to 564 so, 1% either
// way at any count, the tables' five 522 and 524; 8-bit states 259 to 269 us and 253 to 260.)
__device__ __forceinline__ int lookup(const AdamwLaunch& L, int b) {
  return find_tensor([&](int i) { return L.first[i]; }, L.count, b);
}

// Blocks go from the last tensor to the first: a gradient norm, which goes the other way, has left
// the last gradients in the memory-side cache (GPT-2-124M, 8-bit, with its norm: 346 us forwards, 336
// backwards).
__device__ __forceinline__ int block_of_launch() { return gridDim.x - 1 - blockIdx.x; }

__device__ __forceinline__ Item item_of(const AdamwLaunch& L, int q) {
  const Constant<Item> t = (Constant<Item>)(uintptr_t)L.item + q;
  return {t->p, t->w, t->m, t->v, t->ms, t->vs, t->numel, t->wd_mul, t->first};
}

// The gradient scale; false when the step is to be skipped.
__device__ __forceinline__ bool read_scale(const Step& S, float& scale) {
  scale = 1.f;
  if (!S.grad_scale) return true;
  scale = *S.grad_scale;
  return !(S.skip_nonfinite && !(fabsf(scale) <= 3.402823466e38f));
}

// p <- p - lr (u + lam p) from the new m and sqrt(v). The reciprocal is the hardware's, off by at
// most one unit in the last place: its argument is 0 or at least 2^-75 (the root of the smallest
// fp32), so that no subnormal enters it. A division takes ten instructions more.
__device__ __forceinline__ float updated(const Step& S, float lam, float p, float m, float r) {
  const float u = (m * S.inv_bc1) * __builtin_amdgcn_rcpf(fmaf(r, S.inv_sqrt_bc2, S.eps));
  return fmaf(-S.lr, fmaf(lam, p, u), p);
}

// ---- fp32 states -----------------------------------------------------------------------------

__device__ __forceinline__ void step_f32(const Step& S, float scale, float lam, float& p, float g,
                                         float& m, float& v) {
  g *= scale;
  m = fmaf(S.beta1, m, (1.f - S.beta1) * g);
  v = fmaf(S.beta2, v, (1.f - S.beta2) * (g * g));
  p = updated(S, lam, p, m, sqrtf(v));
}

template <int PM, int GD>
__global__ __launch_bounds__(kThreadsF32) void adamw_f32_kernel(const AdamwLaunch L) {
  constexpr int PD = PM == kBf16 ? 0 : 1;        // what p is read from
  const int b = block_of_launch();
  const int q = lookup(L, b);
  const void* const G = L.g[q];
  float scale;
  if (!G || !read_scale(L.s, scale)) return;
  const Item I = item_of(L, q);
  const float lam = L.s.weight_decay * I.wd_mul;
  const int64_t n = I.numel;
  const int64_t base = int64_t(b - I.first) * kChunkF32;
  void* const P = PM == kMaster ? I.w : I.p;
  float* const M = static_cast<float*>(I.m);
  float* const V = static_cast<float*>(I.v);

  if (base + kChunkF32 <= n) {
    const int64_t i = base + int64_t(threadIdx.x) * kVec;
    float p[kVec], g[kVec], m[kVec], v[kVec];
    load_vec<PD, true>(P, i, p);
    load_vec<GD, true>(G, i, g);
    load_vec<1, true>(M, i, m);
    load_vec<1, true>(V, i, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) step_f32(L.s, scale, lam, p[e], g[e], m[e], v[e]);
    store_vec<PD, true>(P, i, p);
    if (PM == kMaster) store_vec<0, true>(I.p, i, p);
    store_vec<1, true>(M, i, m);
    store_vec<1, true>(V, i, v);
    return;
  }
  // the last chunk of a tensor, element by element
  for (int64_t i = base + threadIdx.x; i < n; i += kThreadsF32) {
    float p = load_one<PD>(P, i), m = M[i], v = V[i];
    step_f32(L.s, scale, lam, p, load_one<GD>(G, i), m, v);
    store_one<PD>(P, i, p);
    if (PM == kMaster) store_one<0>(I.p, i, p);
    M[i] = m;
    V[i] = v;
  }
}

// ---- 8-bit states ----------------------------------------------------------------------------
//
// A block of 256 elements lies over LANES lanes, each of which has pieces of PIECE elements of it,
// LANES * PIECE apart. Every access of a wave is then made of whole 128-byte lines, and the
// largest |x| of a block is found among few lanes:
//   all streams bf16 or codes   16 lanes x 2 pieces of 8 (bf16 256 bytes, codes 128 in a run)
//   one of them fp32            32 lanes x 2 pieces of 4 (fp32 512, bf16 256, codes 128)
// A wave has 64 * kOwn consecutive elements, four blocks.

template <int CTRL>
__device__ __forceinline__ float row_rotate(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}

// The largest of x over the lanes of a block, in every lane.
template <int LANES>
__device__ __forceinline__ float block_max(float x) {
  x = fmaxf(x, row_rotate<0x128>(x));            // over the row of 16 lanes
  x = fmaxf(x, row_rotate<0x124>(x));
  x = fmaxf(x, row_rotate<0x122>(x));
  x = fmaxf(x, row_rotate<0x121>(x));
  if (LANES == 32)                               // and the row beside it
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(x), 0x401f)));
  return x;
}

// The smallest scale byte b with top <= T * 2^(b - 127): top = 2^(E - 127) * f has b = E - 8,
// or E - 7 if f is over T's significand 1 + 0x629146 / 2^23.
__device__ __forceinline__ int scale_byte(float top) {
  const int e = int((__float_as_uint(top) + (0x7fffffu - 0x629146u)) >> 23) - 8;
  return max(e, 0);
}
__device__ __forceinline__ float scale_of(int b) {            // 2^(b - 127)
  return __uint_as_float(b == 0 ? 0x00400000u : uint32_t(b) << 23);
}

constexpr float kRootTop = 240.f * 0x1p56f;
constexpr float kMeanTop = 240.f * 0x1p120f;     // of m: the largest code that is finite there
constexpr int kMeanTopByte = 120 + 127;          // its scale, the largest there is

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0xEB26D985u;
  x = (x ^ (x >> 15)) * 0x4A08C6EDu;
  return x ^ (x >> 16);
}

// A register whose every bit the next conversions write.
__device__ __forceinline__ int unset() {
  int w;
  asm("" : "=v"(w));
  return w;
}

template <int PIECE>                             // a piece's codes
using Codes = uint32_t __attribute__((ext_vector_type(PIECE / 4)));

// A piece's codes <-> floats, by the hardware's scaled conversions: exact one way, to nearest even or
// stochastically the other (up with the probability of what is cut off: the upper 20 of the 32
// random bits are added below the format's last place). Measured over all codes and scales and
// over random values, subnormals of the format included: bit by bit what adamw.h defines.
template <int PIECE>
__device__ __forceinline__ void decode(const Codes<PIECE> c, float scale, float* x) {
#pragma unroll
  for (int k = 0; k < PIECE / 4; ++k) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[k], scale, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[k], scale, true);
    x[4 * k] = a[0];
    x[4 * k + 1] = a[1];
    x[4 * k + 2] = b[0];
    x[4 * k + 3] = b[1];
  }
}
template <int PIECE>
__device__ __forceinline__ Codes<PIECE> encode(const float* x, float scale) {
  Codes<PIECE> c;
#pragma unroll
  for (int k = 0; k < PIECE / 4; ++k) {
    i16x2 w = __builtin_bit_cast(i16x2, unset());
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[4 * k], x[4 * k + 1], scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[4 * k + 2], x[4 * k + 3], scale, true);
    c[k] = __builtin_bit_cast(uint32_t, w);
  }
  return c;
}
// Elements 2j and 2j + 1 take the halves of h(j ^ key): 16 random bits, then half of one.
template <int PIECE>
__device__ __forceinline__ Codes<PIECE> encode_stochastic(const float* x, float scale, uint32_t pair,
                                                         uint32_t key) {
  Codes<PIECE> c;
#pragma unroll
  for (int k = 0; k < PIECE / 4; ++k) {
    const uint32_t h0 = mix32((pair + 2 * k) ^ key), h1 = mix32((pair + 2 * k + 1) ^ key);
    int w = unset();
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[4 * k], h0 << 16 | 0x8000u, scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[4 * k + 1], (h0 & 0xffff0000u) | 0x8000u, scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[4 * k + 2], h1 << 16 | 0x8000u, scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[4 * k + 3], (h1 & 0xffff0000u) | 0x8000u, scale, 3);
    c[k] = uint32_t(w);
  }
  return c;
}

// sqrt(v) rounded to nearest, for v = 0 and 2^-101 <= v < 2^128: one step of Newton's method from
// the reciprocal root, whose residual v - s^2 is exact there. Compared with the compiler's sqrt
// over every significand at even and odd exponents: equal. (Its own sequence, which also takes
// the rest of the range, is twice as long; with it, a full division and conversions in steps the
// kernel was bound by instructions: 294 us for the tables.)
__device__ __forceinline__ float root(float v) {
  const float q = __builtin_amdgcn_rsqf(v + 0x1p-126f);       // v itself, but for 0
  const float s = v * q;
  return fmaf(fmaf(-s, s, v) * 0.5f, q, s);
}

// The new m and v, each operation rounded to fp32 (the stored codes are then a function of the
// inputs alone, whatever a compiler fuses).
__device__ __forceinline__ void moments(const Step& S, float g, float& m, float& v) {
#pragma clang fp contract(off)
  const float a = S.beta1 * m, b = (1.f - S.beta1) * g;
  m = a + b;
  const float c = S.beta2 * v, gg = g * g;
  const float d = (1.f - S.beta2) * gg;
  v = c + d;
}

// The chunk from element `base` on; FULL: it ends inside the tensor.
template <int PM, int GD, bool FULL>
__device__ __forceinline__ void step_8bit(const Item& I, const void* grad, const Step& S,
                                          float scale, int64_t base) {
  constexpr int PD = PM == kBf16 ? 0 : 1;
  constexpr bool NARROW = PM == kBf16 && GD == 0;
  constexpr int LANES = NARROW ? 16 : 32, PIECE = NARROW ? 8 : 4;
  constexpr int PER = MUON_ADAMW_BLOCK / (LANES * PIECE);    // pieces of a lane in a block
  constexpr int PIECES = kOwn / PIECE, BLOCKS = PIECES / PER;
  const float lam = S.weight_decay * I.wd_mul;
  // the chunk's own addresses, and elements and blocks counted from there in 32 bits
  char* const P = static_cast<char*>(PM == kMaster ? I.w : I.p) + base * (PD ? 4 : 2);
  uint16_t* const H = static_cast<uint16_t*>(I.p) + base;    // the parameter beside a master
  const char* const G = static_cast<const char*>(grad) + base * (GD ? 4 : 2);
  uint8_t* const M = static_cast<uint8_t*>(I.m) + base;
  uint8_t* const V = static_cast<uint8_t*>(I.v) + base;
  uint8_t* const MS = I.ms + base / MUON_ADAMW_BLOCK;
  uint8_t* const VS = I.vs + base / MUON_ADAMW_BLOCK;
  const uint32_t left = FULL ? kChunk : uint32_t(I.numel - base);
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t first = threadIdx.x / 64 * (64 * kOwn) + lane / LANES * MUON_ADAMW_BLOCK;
  auto block = [&](int k) { return first / MUON_ADAMW_BLOCK + k * (64 / LANES); };
  auto element = [&](int x) {                    // the first of piece x
    return first + x / PER * (64 / LANES * MUON_ADAMW_BLOCK) + x % PER * (LANES * PIECE) +
           lane % LANES * PIECE;
  };
  auto inside = [&](int x) {                     // of the piece's elements
    return FULL ? PIECE : int(min(left - min(left, element(x)), uint32_t(PIECE)));
  };

  float p[PIECES][PIECE], g[PIECES][PIECE], m[kOwn], r[kOwn];
  Codes<PIECE> mc[PIECES], rc[PIECES];
  int mb[BLOCKS], rb[BLOCKS];
#pragma unroll
  for (int k = 0; k < BLOCKS; ++k) {
    mb[k] = rb[k] = 0;
    if (FULL || block(k) * MUON_ADAMW_BLOCK < left) {
      mb[k] = MS[block(k)];
      rb[k] = VS[block(k)];
    }
  }
#pragma unroll
  for (int x = 0; x < PIECES; ++x) {
    const uint32_t i = element(x);
    const int cnt = inside(x);
    if (cnt == PIECE) {
      load_vec<PD, true>(P, i, p[x]);
      load_vec<GD, true>(G, i, g[x]);
      mc[x] = load_at<true>(reinterpret_cast<const Codes<PIECE>*>(M + i));
      rc[x] = load_at<true>(reinterpret_cast<const Codes<PIECE>*>(V + i));
    } else {
      mc[x] = rc[x] = Codes<PIECE>(0);
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        p[x][e] = g[x][e] = 0.f;
        if (e < cnt) {
          p[x][e] = load_one<PD>(P, i + e);
          g[x][e] = load_one<GD>(G, i + e);
          mc[x][e >> 2] |= uint32_t(M[i + e]) << (8 * (e & 3));
          rc[x][e >> 2] |= uint32_t(V[i + e]) << (8 * (e & 3));
        }
      }
    }
  }

  float mtop[BLOCKS], vtop[BLOCKS];
  uint32_t vlow = ~0u;                           // the smallest v over 0, less one unit
#pragma unroll
  for (int k = 0; k < BLOCKS; ++k) mtop[k] = vtop[k] = 0.f;
#pragma unroll
  for (int x = 0; x < PIECES; ++x) {
    const int k = x / PER;
    float* const mx = m + x * PIECE;
    float* const rx = r + x * PIECE;
    decode<PIECE>(mc[x], scale_of(mb[k]), mx);
    decode<PIECE>(rc[x], scale_of(rb[k]), rx);
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      float v = rx[e] * rx[e];
      moments(S, g[x][e] * scale, mx[e], v);
      asm("" : "+v"(mx[e]));                     // kept, not computed again behind the branch
      rx[e] = v;
      mtop[k] = fmaxf(mtop[k], fabsf(mx[e]));
      vtop[k] = fmaxf(vtop[k], v);
      vlow = min(vlow, __float_as_uint(v) - 1u);
    }
  }
  // rare, and the whole wave's: a v that root() does not take
  bool wide = vlow < 0x0d000000u - 1u;
#pragma unroll
  for (int k = 0; k < BLOCKS; ++k) wide = wide || vtop[k] > 3.402823466e38f;
  float rtop[BLOCKS];                            // of the block: its largest v's root
#pragma unroll
  for (int k = 0; k < BLOCKS; ++k) rtop[k] = block_max<LANES>(vtop[k]);
  if (__any(wide)) {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) r[e] = sqrtf(r[e]);
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)             // the scale of an infinite v: the largest finite one's
      rtop[k] = sqrtf(fminf(rtop[k], 3.402823466e38f));
  } else {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) r[e] = root(r[e]);
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) rtop[k] = root(rtop[k]);
  }

#pragma unroll
  for (int k = 0; k < BLOCKS; ++k) {
    mb[k] = scale_byte(block_max<LANES>(mtop[k]));
    rb[k] = scale_byte(rtop[k]);
    const float rs = scale_of(rb[k]);
    // up to the largest code whose square is finite: 240 2^56, at the largest scale. (What rounds
    // to the next one, 2^64, would make v infinite in the next step and from then on.)
    const float low = rs * 0x1p-9f, high = fminf(rs * 448.f, kRootTop);
#pragma unroll
    for (int x = k * PER; x < (k + 1) * PER; ++x) {
      const uint32_t i = element(x);
      const int cnt = inside(x);
      float* const mx = m + x * PIECE;
      float* const rx = r + x * PIECE;
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        p[x][e] = updated(S, lam, p[x][e], mx[e], rx[e]);
        // NaN and 0 as they are
        rx[e] = rx[e] > 0.f ? __builtin_amdgcn_fmed3f(rx[e], low, high) : rx[e];
      }
      if (mb[k] == kMeanTopByte) {               // rare: 2^128, the next code, would read as infinite
#pragma unroll
        for (int e = 0; e < PIECE; ++e)
          if (fabsf(mx[e]) <= 3.402823466e38f) mx[e] = copysignf(fminf(fabsf(mx[e]), kMeanTop), mx[e]);
      }
      mc[x] = encode<PIECE>(mx, scale_of(mb[k]));
      if (S.stochastic) {
        // a chunk's pairs do not cross a multiple of 2^32
        const uint32_t pair = uint32_t(uint64_t(base) >> 1) + i / 2;
        rc[x] = encode_stochastic<PIECE>(rx, rs, pair,
                                         S.key ^ uint32_t(uint64_t(base) >> 33) * 0xEB26D985u);
      } else {
        rc[x] = encode<PIECE>(rx, rs);
      }
      if (cnt == PIECE) {
        store_vec<PD, true>(P, i, p[x]);
        if (PM == kMaster) store_vec<0, true>(H, i, p[x]);
        store_at<true>(reinterpret_cast<Codes<PIECE>*>(M + i), mc[x]);
        store_at<true>(reinterpret_cast<Codes<PIECE>*>(V + i), rc[x]);
      } else {
#pragma unroll
        for (int e = 0; e < PIECE; ++e)
          if (e < cnt) {
            store_one<PD>(P, i + e, p[x][e]);
            if (PM == kMaster) store_one<0>(H, i + e, p[x][e]);
            M[i + e] = uint8_t(mc[x][e >> 2] >> (8 * (e & 3)));
            V[i + e] = uint8_t(rc[x][e >> 2] >> (8 * (e & 3)));
          }
      }
    }
    if (lane % LANES == 0 && (FULL || block(k) * MUON_ADAMW_BLOCK < left)) {
      MS[block(k)] = uint8_t(mb[k]);
      VS[block(k)] = uint8_t(rb[k]);
    }
  }
}

template <int PM, int GD>
__global__ __launch_bounds__(kThreads) void adamw_8bit_kernel(const AdamwLaunch L) {
  const int b = block_of_launch();
  const int q = lookup(L, b);
  const void* const G = L.g[q];
  float scale;
  if (!G || !read_scale(L.s, scale)) return;
  const Item I = item_of(L, q);
  const int64_t base = int64_t(b - I.first) * kChunk;
  if (base + kChunk <= I.numel) step_8bit<PM, GD, true>(I, G, L.s, scale, base);
  else step_8bit<PM, GD, false>(I, G, L.s, scale, base);
}

// ---- the table -------------------------------------------------------------------------------

constexpr int kUpload = 48;                      // items per launch (by value: no pinned memory)
struct Upload {
  Item item[kUpload];
  Item* to;
  int* first;
  int count;
};

__global__ __launch_bounds__(64) void adamw_upload_kernel(const Upload U) {
  const int t = threadIdx.x;
  if (t >= U.count) return;
  U.to[t] = U.item[t];
  U.first[t] = U.item[t].first;
}

// ---- host ------------------------------------------------------------------------------------

struct Launch {
  int pm, gd;                                    // its kernel
  int lo, count;                                 // its items
  int64_t blocks;
};

}  // namespace
}  // namespace muon

struct muon_adamw_plan {
  std::vector<muon_adamw_tensor> tensors;
  std::vector<muon::Range> ranges;               // the plan's buffers, ascending
  std::vector<muon::Item> items;                 // those with elements, by kernel
  std::vector<int> index;                        // the tensor of each item
  std::vector<size_t> grad_offset;               // bytes, of the item's piece in its gradient
  std::vector<muon::Launch> launches;
  muon_adamw_state state = MUON_ADAMW_F32;
  muon::Item* table = nullptr;                   // device: items, then their first blocks
};

namespace muon {
namespace {

typedef void (*AdamwKernel)(AdamwLaunch);

AdamwKernel kernel_of(muon_adamw_state st, int pm, int gd) {
  static const AdamwKernel f32[3][2] = {
      {adamw_f32_kernel<kBf16, 0>, adamw_f32_kernel<kBf16, 1>},
      {adamw_f32_kernel<kF32, 0>, adamw_f32_kernel<kF32, 1>},
      {adamw_f32_kernel<kMaster, 0>, adamw_f32_kernel<kMaster, 1>}};
  static const AdamwKernel e8[3][2] = {
      {adamw_8bit_kernel<kBf16, 0>, adamw_8bit_kernel<kBf16, 1>},
      {adamw_8bit_kernel<kF32, 0>, adamw_8bit_kernel<kF32, 1>},
      {adamw_8bit_kernel<kMaster, 0>, adamw_8bit_kernel<kMaster, 1>}};
  return (st == MUON_ADAMW_F32 ? f32 : e8)[pm][gd];
}

int check_tensor(const muon_adamw_tensor& T, int64_t i, muon_adamw_state state,
                 std::vector<Range>& rs) {
  if (T.numel < 0 || T.numel > kMaxTensorElems)
    return fail(T.numel < 0 ? MUON_ERR_INVALID_ARG : MUON_ERR_UNSUPPORTED,
                "tensor %lld: numel %lld outside [0, 2^35]", (long long)i, (long long)T.numel);
  if (!dtype_known(T.param_dtype) || !dtype_known(T.grad_dtype))
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: unknown dtype (%d, %d)", (long long)i,
                (int)T.param_dtype, (int)T.grad_dtype);
  if (!std::isfinite(T.wd_mul))
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: wd_mul must be finite", (long long)i);
  if (T.numel == 0) return MUON_OK;
  const bool e8 = state == MUON_ADAMW_8BIT;
  if (!T.param || !T.exp_avg || !T.exp_avg_sq)
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: param, exp_avg and exp_avg_sq must be non-NULL",
                (long long)i);
  if (e8 && (!T.exp_avg_scale || !T.exp_avg_sq_scale))
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: 8-bit states need both scale buffers",
                (long long)i);
  if (T.master && T.param_dtype != MUON_DT_BF16)
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: a master copy is for bf16 parameters",
                (long long)i);
  if (!is_aligned16(T.param) || !is_aligned16(T.master) || !is_aligned16(T.exp_avg) ||
      !is_aligned16(T.exp_avg_sq))
    return fail(MUON_ERR_INVALID_ARG, "tensor %lld: buffers must be 16-byte aligned", (long long)i);
  auto add = [&](const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    rs.push_back({lo, lo + bytes, true});
  };
  const size_t n = (size_t)T.numel, blocks = (n + MUON_ADAMW_BLOCK - 1) / MUON_ADAMW_BLOCK;
  add(T.param, n * dtype_bytes(T.param_dtype));
  if (T.master) add(T.master, n * 4);
  add(T.exp_avg, e8 ? n : n * 4);
  add(T.exp_avg_sq, e8 ? n : n * 4);
  if (e8) {
    add(T.exp_avg_scale, blocks);
    add(T.exp_avg_sq_scale, blocks);
  }
  return MUON_OK;
}

int check_config(const muon_adamw_config* cfg) {
  if (!cfg) return fail(MUON_ERR_INVALID_ARG, "cfg is NULL");
  if (!std::isfinite(cfg->lr) || !std::isfinite(cfg->eps) || !std::isfinite(cfg->weight_decay))
    return fail(MUON_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite");
  if (cfg->eps < 0.f) return fail(MUON_ERR_INVALID_ARG, "eps must be >= 0");
  if (!(cfg->beta1 >= 0.f && cfg->beta1 < 1.f) || !(cfg->beta2 >= 0.f && cfg->beta2 < 1.f))
    return fail(MUON_ERR_INVALID_ARG, "beta1 and beta2 must lie in [0, 1)");
  if (cfg->step < 1) return fail(MUON_ERR_INVALID_ARG, "step = %lld < 1", (long long)cfg->step);
  if ((cfg->skip_nonfinite & ~1) || (cfg->stochastic & ~1))
    return fail(MUON_ERR_INVALID_ARG, "skip_nonfinite and stochastic must be 0 or 1");
  if (cfg->skip_nonfinite && !cfg->grad_scale)
    return fail(MUON_ERR_INVALID_ARG, "skip_nonfinite needs grad_scale");
  if (reinterpret_cast<uintptr_t>(cfg->grad_scale) & 3)
    return fail(MUON_ERR_INVALID_ARG, "grad_scale must be 4-byte aligned");
  return MUON_OK;
}

// Whether ranges meet one of the plan's buffers. The gap that the last one lay in is kept:
// gradients of one allocation take one search.
class Buffers {
 public:
  explicit Buffers(const std::vector<Range>& rs) : rs_(rs) {}
  bool meet(uintptr_t lo, uintptr_t hi) {
    if (lo >= gap_lo_ && hi <= gap_hi_) return false;
    const auto it = std::upper_bound(rs_.begin(), rs_.end(), lo,
                                     [](uintptr_t x, const Range& r) { return x < r.hi; });
    gap_lo_ = it == rs_.begin() ? 0 : (it - 1)->hi;
    gap_hi_ = it == rs_.end() ? ~uintptr_t(0) : it->lo;
    return hi > gap_hi_ || lo < gap_lo_;
  }

 private:
  const std::vector<Range>& rs_;
  uintptr_t gap_lo_ = 1, gap_hi_ = 0;
};

int check_step(const muon_adamw_plan* plan, const void* const* grads, int64_t n,
               const muon_adamw_config* cfg) {
  if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
  if (n != (int64_t)plan->tensors.size())
    return fail(MUON_ERR_INVALID_ARG, "n = %lld but the plan has %zu tensors", (long long)n,
                plan->tensors.size());
  if (int st = check_config(cfg)) return st;
  if (n > 0 && !grads) return fail(MUON_ERR_INVALID_ARG, "grads is NULL");
  Buffers buffers(plan->ranges);
  bool any = false;
  for (int64_t i = 0; i < n; ++i) {
    const muon_adamw_tensor& T = plan->tensors[i];
    if (!std::isfinite(cfg->weight_decay * T.wd_mul))
      return fail(MUON_ERR_INVALID_ARG, "tensor %lld: weight_decay * wd_mul overflows",
                  (long long)i);
    if (T.numel == 0 || !grads[i]) continue;
    any = true;
    if (!is_aligned16(grads[i]))
      return fail(MUON_ERR_INVALID_ARG, "gradient %lld must be 16-byte aligned", (long long)i);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i]);
    if (buffers.meet(lo, lo + (size_t)T.numel * dtype_bytes(T.grad_dtype)))
      return fail(MUON_ERR_INVALID_ARG, "gradient %lld overlaps a buffer of the plan",
                  (long long)i);
  }
  if (cfg->grad_scale) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(cfg->grad_scale);
    if (buffers.meet(lo, lo + sizeof(float)))
      return fail(MUON_ERR_INVALID_ARG, "grad_scale overlaps a buffer of the plan");
  }
  if (any && !plan->table)
    return fail(MUON_ERR_WORKSPACE, "muon_adamw_plan_upload has not been called on the plan");
  return MUON_OK;
}

uint32_t key_of(uint64_t seed, int64_t step) {
  uint64_t z = seed + (uint64_t)step * 0x1493FA689CA113ADull;
  for (int k = 0; k < 2; ++k) z = (z ^ (z >> 32)) * 0xE9F8AC216EBC06F5ull;
  return uint32_t(z ^ (z >> 32));
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

void muon_adamw_config_default(muon_adamw_config* cfg) {
  if (!cfg) return;
  *cfg = muon_adamw_config{};
  cfg->lr = 1e-3f;
  cfg->beta1 = 0.9f;
  cfg->beta2 = 0.999f;
  cfg->eps = 1e-8f;
  cfg->weight_decay = 0.01f;
  cfg->step = 1;
  cfg->stochastic = 1;
}

int muon_adamw_plan_create(muon_adamw_plan** out, const muon_adamw_tensor* tensors, int64_t n,
                           muon_adamw_state state) {
  return c_entry([&]() -> int {
    if (!out) return fail(MUON_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (n < 0) return fail(MUON_ERR_INVALID_ARG, "n = %lld < 0", (long long)n);
    if (n > (int64_t(1) << 24))
      return fail(MUON_ERR_UNSUPPORTED, "n = %lld: at most 2^24 tensors", (long long)n);
    if (n > 0 && !tensors) return fail(MUON_ERR_INVALID_ARG, "tensors is NULL");
    if (state != MUON_ADAMW_F32 && state != MUON_ADAMW_8BIT)
      return fail(MUON_ERR_INVALID_ARG, "unknown state %d", (int)state);
    muon_adamw_plan made;
    made.state = state;
    std::vector<int> of[3][2];
    for (int64_t i = 0; i < n; ++i) {
      const muon_adamw_tensor& T = tensors[i];
      if (int st = check_tensor(T, i, state, made.ranges)) return st;
      if (T.numel == 0) continue;
      const int pm = T.master ? kMaster : T.param_dtype == MUON_DT_F32 ? kF32 : kBf16;
      of[pm][T.grad_dtype == MUON_DT_F32].push_back((int)i);
    }
    if (int st = check_overlaps(made.ranges)) return st;   // sorts them
    made.tensors.assign(tensors, tensors + n);
    // (the 8-bit kernel needs an element's index in its tensor, and fits a whole one in a launch)
    const int64_t chunk = state == MUON_ADAMW_8BIT ? kChunk : kChunkF32;
    const int64_t piece = state == MUON_ADAMW_8BIT ? kMaxTensorElems : kPiece;
    for (int pm = 0; pm < 3; ++pm)
      for (int gd = 0; gd < 2; ++gd) {
        Launch l = {pm, gd, (int)made.items.size(), 0, 0};
        for (int i : of[pm][gd]) {
          const muon_adamw_tensor& T = tensors[i];
          const int64_t pb = dtype_bytes(T.param_dtype), sb = state == MUON_ADAMW_8BIT ? 1 : 4;
          for (int64_t off = 0; off < T.numel; off += piece) {
            const int64_t len = std::min(piece, T.numel - off);
            const int64_t nb = (len + chunk - 1) / chunk;
            if (l.count == kMaxItems || l.blocks + nb > kMaxBlocks) {
              made.launches.push_back(l);
              l = {pm, gd, (int)made.items.size(), 0, 0};
            }
            made.items.push_back({static_cast<char*>(T.param) + off * pb,
                                  T.master ? T.master + off : nullptr,
                                  static_cast<char*>(T.exp_avg) + off * sb,
                                  static_cast<char*>(T.exp_avg_sq) + off * sb, T.exp_avg_scale,
                                  T.exp_avg_sq_scale, len, T.wd_mul, (int)l.blocks});
            made.index.push_back(i);
            made.grad_offset.push_back((size_t)off * dtype_bytes(T.grad_dtype));
            ++l.count;
            l.blocks += nb;
          }
        }
        if (l.count) made.launches.push_back(l);
      }
    *out = new muon_adamw_plan(std::move(made));
    return MUON_OK;
  });
}

size_t muon_adamw_plan_table_size(const muon_adamw_plan* plan) {
  return plan ? plan->items.size() * (sizeof(Item) + sizeof(int)) : 0;
}

int muon_adamw_plan_upload(muon_adamw_plan* plan, void* table, size_t table_bytes,
                           hipStream_t stream) {
  return c_entry([&]() -> int {
    if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    const size_t need = muon_adamw_plan_table_size(plan);
    if (need == 0) return MUON_OK;
    if (!table || !is_aligned16(table) || table_bytes < need)
      return fail(MUON_ERR_WORKSPACE, "a table of %zu bytes, 16-byte aligned, is needed", need);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(table);
    if (Buffers(plan->ranges).meet(lo, lo + need))
      return fail(MUON_ERR_INVALID_ARG, "the table overlaps a buffer of the plan");
    const size_t n = plan->items.size();
    Item* const to = static_cast<Item*>(table);
    Upload U;
    for (size_t at = 0; at < n; at += kUpload) {
      U.count = (int)std::min<size_t>(kUpload, n - at);
      std::copy_n(plan->items.begin() + at, U.count, U.item);
      U.to = to + at;
      U.first = reinterpret_cast<int*>(to + n) + at;
      hipLaunchKernelGGL(adamw_upload_kernel, dim3(1), dim3(64), 0, stream, U);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess)
        return fail(MUON_ERR_HIP, "launch of the AdamW table's upload failed: %s",
                    hipGetErrorString(e));
    }
    plan->table = to;
    return MUON_OK;
  });
}

void muon_adamw_plan_destroy(muon_adamw_plan* plan) { delete plan; }

int muon_adamw_check(const muon_adamw_plan* plan, const void* const* grads, int64_t n,
                     const muon_adamw_config* cfg) {
  return c_entry([&]() -> int { return check_step(plan, grads, n, cfg); });
}

int muon_adamw_step(const muon_adamw_plan* plan, const void* const* grads, int64_t n,
                    const muon_adamw_config* cfg, hipStream_t stream) {
  return c_entry([&]() -> int {
    if (int st = check_step(plan, grads, n, cfg)) return st;
    AdamwLaunch L;
    L.s.lr = cfg->lr;
    L.s.beta1 = cfg->beta1;
    L.s.beta2 = cfg->beta2;
    L.s.eps = cfg->eps;
    L.s.weight_decay = cfg->weight_decay;
    const double t = (double)cfg->step;
    L.s.inv_bc1 = (float)(1.0 / (1.0 - std::pow((double)cfg->beta1, t)));
    L.s.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow((double)cfg->beta2, t)));
    L.s.grad_scale = cfg->grad_scale;
    L.s.skip_nonfinite = cfg->skip_nonfinite;
    L.s.stochastic = cfg->stochastic;
    L.s.key = key_of(cfg->seed, cfg->step);
    for (const Launch& l : plan->launches) {
      bool any = false;
      for (int c = 0; c < l.count; ++c) {
        const void* const g = grads[plan->index[l.lo + c]];
        L.g[c] = g ? static_cast<const char*>(g) + plan->grad_offset[l.lo + c] : nullptr;
        any = any || g;
      }
      if (!any) continue;
      L.item = plan->table + l.lo;
      L.first = reinterpret_cast<const int*>(plan->table + plan->items.size()) + l.lo;
      L.count = l.count;
      const bool f32 = plan->state == MUON_ADAMW_F32;
      hipLaunchKernelGGL(kernel_of(plan->state, l.pm, l.gd), dim3((unsigned)l.blocks),
                         dim3(f32 ? kThreadsF32 : kThreads), f32 ? kHoldF32 : kHold, stream, L);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess)
        return fail(MUON_ERR_HIP, "launch of the AdamW kernel failed: %s", hipGetErrorString(e));
    }
    return MUON_OK;
  });
}

}  // extern "C"
