// The global gradient norm and its clipping scale over many tensors: host side and kernels of
// the C ABI in include/grad_norm.h.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  scale = min(1, max_norm / norm)
//
// Each tensor is cut into parts of equal length; a block sums one part's squares in double
// (fp32's squares overflow at 1.8e19 and lose their bits below 1e-19) and writes one partial
// sum. A second launch joins the partial sums in a fixed order.
//
// Bound by HBM: each gradient is read once, and the conversion to double and the fused
// multiply-add of an element are far below what a compute unit does meanwhile. Reads past the
// memory-side cache are faster (GPT-2-1.5B, fp32, 6.2 GB: 1.04 ms cached, 0.92 ms = 6.7 TB/s
// nontemporal), but the step that uses the scale reads the gradients again, from the last to the
// first. So the last 256 MB, which that cache holds, are read through it, and the rest past it:
// GPT-2-124M's bf16 gradients (249 MB) take 51 us and not 46, and the step behind them 31 us less.
#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "grad_norm.h"
#include "tensor_list.h"

struct muon_grad_plan {
  std::vector<int64_t> numel;
  std::vector<muon_dtype> dtype;
  std::vector<int> part0;       // first part of each tensor; [n] = all parts
  int64_t part_elems = 0;
  int keep_part = 0;            // parts from here on are left in the memory-side cache
};

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                       // loads of a thread in flight
constexpr int64_t kMinPart = 32768;              // 16384: 9% slower, GPT-2-124M
constexpr int64_t kMaxPart = int64_t(1) << 30;
constexpr int64_t kMaxParts = 16384;             // beyond one per tensor
constexpr int64_t kCacheBytes = int64_t(1) << 28;  // the memory-side cache: 256 MB
constexpr int kFinishThreads = 1024;
constexpr int kNormItems = 240;                  // tensors per launch (by value)

struct NormItem {
  uint64_t g;                                    // address; bit 0: fp32
  int first;                                     // its first block = its first part
  uint32_t tail;                                 // elements of its last part
};

struct NormLaunch {
  NormItem item[kNormItems];
  double* partial;                               // of the launch's first part
  int* tensor_part;                              // out: first part of each tensor
  int part0;
  int count, blocks;
  int keep_part;
  int part_elems;
};
static_assert(sizeof(NormLaunch) <= 4096, "kernel arguments");

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_down(x, o, 64);
  return x;
}

// The block's sum, in thread 0; the order of additions is fixed.
template <int THREADS>
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double s[THREADS / 64];
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) x += s[w];
  }
  return x;
}

// Sum of squares of n elements at g (16-byte aligned), this thread's share. Each access of a wave
// is one contiguous kilobyte. NT: nontemporal.
template <int GD, bool NT>
__device__ __forceinline__ double squares(const void* g, int n) {
  constexpr int N = GD == 0 ? 8 : 4;             // elements of a 16-byte access
  double acc = 0.0;
  int i = threadIdx.x * N;
  for (; i + (kUnroll - 1) * kThreads * N + N <= n; i += kUnroll * kThreads * N) {
    float x[kUnroll][N];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load_vec<GD, NT>(g, i + u * kThreads * N, x[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) acc = fma(double(x[u][e]), double(x[u][e]), acc);
  }
  for (; i + N <= n; i += kThreads * N) {
    float x[N];
    load_vec<GD, NT>(g, i, x);
#pragma unroll
    for (int e = 0; e < N; ++e) acc = fma(double(x[e]), double(x[e]), acc);
  }
  for (; i < n; ++i) {                           // the thread whose vector the end cuts
    const double x = load_one<GD>(g, i);
    acc = fma(x, x, acc);
  }
  return acc;
}

__global__ __launch_bounds__(kThreads) void grad_norm_parts_kernel(const NormLaunch L) {
  const int b = blockIdx.x;
  const int q = find_tensor([&](int i) { return L.item[i].first; }, L.count, b);
  const NormItem I = L.item[q];
  const int k = b - I.first;
  const bool last = b + 1 == (q + 1 < L.count ? L.item[q + 1].first : L.blocks);
  const int n = last ? int(I.tail) : L.part_elems;
  const int64_t lo = int64_t(k) * L.part_elems;
  double acc = 0.0;
  if (I.g > 1) {
    const float* const f = reinterpret_cast<const float*>(I.g - 1) + lo;
    const uint16_t* const h = reinterpret_cast<const uint16_t*>(I.g) + lo;
    if (L.part0 + b >= L.keep_part) acc = I.g & 1 ? squares<1, false>(f, n) : squares<0, false>(h, n);
    else acc = I.g & 1 ? squares<1, true>(f, n) : squares<0, true>(h, n);
  }
  const double sum = block_sum<kThreads>(acc);
  if (threadIdx.x == 0) {
    L.partial[b] = sum;
    if (k == 0) L.tensor_part[q] = L.part0 + b;
  }
}

// Block 0: the norm and the scale. Blocks beyond it: a tensor's norm for each wave.
__global__ __launch_bounds__(kFinishThreads) void grad_norm_finish_kernel(
    const double* __restrict__ partial, const int* __restrict__ tensor_part, int tensors,
    int parts, float max_norm, float* out, float* norms) {
  if (blockIdx.x == 0) {
    double acc = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < parts; i += kFinishThreads) acc += partial[i];
    const double sum = block_sum<kFinishThreads>(acc);
    if (threadIdx.x == 0) {
      const double norm = sqrt(sum);
      const bool finite = norm <= 1.7976931348623157e308;   // false for NaN too
      out[0] = float(norm);
      out[1] = !finite ? __uint_as_float(0x7fc00000u)
                       : norm > double(max_norm) ? float(double(max_norm) / norm) : 1.f;
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const int t = (blockIdx.x - 1) * (kFinishThreads / 64) + (threadIdx.x >> 6);
  if (t >= tensors) return;
  const int lo = tensor_part[t], hi = t + 1 < tensors ? tensor_part[t + 1] : parts;
  double x = 0.0;
  for (int i = lo + lane; i < hi; i += 64) x += partial[i];
  x = wave_sum(x);
  if (lane == 0) norms[t] = float(sqrt(x));
}

constexpr int kScaleChunk = kThreads * 16;

constexpr int kScaleItems = 160;                 // tensors per launch (by value)

struct ScaleItem {
  uint64_t g;                                    // address; bit 0: fp32
  int64_t numel;
  int first;
};

struct ScaleLaunch {
  ScaleItem item[kScaleItems];
  const float* scale;
  int count;
};
static_assert(sizeof(ScaleLaunch) <= 4096, "kernel arguments");

// Nontemporal whole-line accesses: GPT-2-1.5B's fp32 gradients 1.95 ms (6.4 TB/s), 2.22 cached.
template <int GD>
__device__ __forceinline__ void scale_chunk(void* G, int64_t base, int64_t n, float s) {
  constexpr int N = GD == 0 ? 8 : 4, U = kScaleChunk / (kThreads * N);
  if (base + kScaleChunk <= n) {
    float x[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) load_vec<GD, true>(G, base + (u * kThreads + threadIdx.x) * N, x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < N; ++e) x[u][e] *= s;
      store_vec<GD, true>(G, base + (u * kThreads + threadIdx.x) * N, x[u]);
    }
    return;
  }
  for (int64_t i = base + threadIdx.x; i < n; i += kThreads)
    store_one<GD>(G, i, load_one<GD>(G, i) * s);
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const ScaleLaunch L) {
  const float s = *L.scale;
  if (s == 1.f) return;
  const int b = blockIdx.x;
  const ScaleItem I = L.item[find_tensor([&](int i) { return L.item[i].first; }, L.count, b)];
  const int64_t base = int64_t(b - I.first) * kScaleChunk;
  if (I.g & 1) scale_chunk<1>(reinterpret_cast<void*>(I.g - 1), base, I.numel, s);
  else scale_chunk<0>(reinterpret_cast<void*>(I.g), base, I.numel, s);
}

int check_grads(const muon_grad_plan* plan, const void* const* grads, int64_t n) {
  if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
  if (n != (int64_t)plan->numel.size())
    return fail(MUON_ERR_INVALID_ARG, "n = %lld but the plan has %zu gradients", (long long)n,
                plan->numel.size());
  if (n > 0 && !grads) return fail(MUON_ERR_INVALID_ARG, "grads is NULL");
  for (int64_t i = 0; i < n; ++i)
    if (!is_aligned16(grads[i]) && plan->numel[i] > 0)
      return fail(MUON_ERR_INVALID_ARG, "gradient %lld must be 16-byte aligned", (long long)i);
  return MUON_OK;
}

Range range_of(const void* p, size_t bytes, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + bytes, written};
}

Range grad_range(const muon_grad_plan* plan, const void* const* grads, int64_t i, bool written) {
  return range_of(grads[i], grads[i] ? plan->numel[i] * dtype_bytes(plan->dtype[i]) : 0, written);
}

size_t partial_bytes(const muon_grad_plan* plan) {
  return ((size_t)plan->part0.back() * sizeof(double) + 15) & ~size_t(15);
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return fail(MUON_ERR_HIP, "launch of the %s kernel failed: %s", what, hipGetErrorString(e));
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_grad_plan_create(muon_grad_plan** out, const int64_t* numel, const muon_dtype* dtype,
                          int64_t n) {
  return c_entry([&]() -> int {
    if (!out) return fail(MUON_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (n < 0) return fail(MUON_ERR_INVALID_ARG, "n = %lld < 0", (long long)n);
    if (n > 0 && (!numel || !dtype))
      return fail(MUON_ERR_INVALID_ARG, "numel and dtype must be non-NULL");
    if (n > (int64_t(1) << 24))
      return fail(MUON_ERR_UNSUPPORTED, "n = %lld: at most 2^24 gradients", (long long)n);
    double total = 0;
    for (int64_t i = 0; i < n; ++i) {
      if (numel[i] < 0 || numel[i] > kMaxTensorElems)
        return fail(numel[i] < 0 ? MUON_ERR_INVALID_ARG : MUON_ERR_UNSUPPORTED,
                    "gradient %lld: numel %lld outside [0, 2^35]", (long long)i,
                    (long long)numel[i]);
      if (!dtype_known(dtype[i]))
        return fail(MUON_ERR_INVALID_ARG, "gradient %lld: unknown dtype %d", (long long)i,
                    (int)dtype[i]);
      total += (double)numel[i];
    }
    muon_grad_plan made;
    made.numel.assign(numel, numel + n);
    made.dtype.assign(dtype, dtype + n);
    made.part_elems = kMinPart;
    while (made.part_elems < kMaxPart && total / (double)made.part_elems > (double)kMaxParts)
      made.part_elems *= 2;
    int64_t parts = 0;
    for (int64_t i = 0; i < n; ++i) {
      made.part0.push_back((int)parts);
      parts += std::max<int64_t>(1, (numel[i] + made.part_elems - 1) / made.part_elems);
    }
    made.part0.push_back((int)parts);
    // the last gradients' parts that fit the memory-side cache
    int64_t bytes = 0;
    made.keep_part = (int)parts;
    for (int64_t i = n - 1; i >= 0 && bytes < kCacheBytes; --i) {
      const int64_t size = (int64_t)dtype_bytes(dtype[i]), part = made.part_elems * size;
      const int64_t fit = std::min(numel[i] * size, kCacheBytes - bytes) / part + 1;
      made.keep_part = std::max(made.part0[i], made.part0[i + 1] - (int)fit);
      bytes += numel[i] * size;
    }
    *out = new muon_grad_plan(std::move(made));
    return MUON_OK;
  });
}

void muon_grad_plan_destroy(muon_grad_plan* plan) { delete plan; }

size_t muon_grad_plan_workspace_size(const muon_grad_plan* plan) {
  if (!plan || plan->numel.empty()) return 0;
  return partial_bytes(plan) + plan->numel.size() * sizeof(int);
}

int muon_grad_norm(const muon_grad_plan* plan, const void* const* grads, int64_t n,
                   float max_norm, float* out, float* norms, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
  return c_entry([&]() -> int {
    if (int st = check_grads(plan, grads, n)) return st;
    if (!(max_norm >= 0.f))
      return fail(MUON_ERR_INVALID_ARG, "max_norm must be >= 0 (infinity: no clipping)");
    if (!out) return fail(MUON_ERR_INVALID_ARG, "out is NULL");
    if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(norms)) & 3)
      return fail(MUON_ERR_INVALID_ARG, "out and norms must be 4-byte aligned");
    const size_t need = muon_grad_plan_workspace_size(plan);
    if (need > 0 && (!workspace || !is_aligned16(workspace) || workspace_bytes < need))
      return fail(MUON_ERR_WORKSPACE, "a workspace of %zu bytes, 16-byte aligned, is needed", need);
    // three written buffers against each other and the gradients (which may overlap one another)
    const Range w[3] = {range_of(out, 2 * sizeof(float), true),
                        range_of(norms, norms ? n * sizeof(float) : 0, true),
                        range_of(workspace, need, true)};
    auto meet = [](const Range& a, const Range& b) {
      return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi;
    };
    bool clash = meet(w[0], w[1]) || meet(w[0], w[2]) || meet(w[1], w[2]);
    for (int64_t i = 0; i < n && !clash; ++i) {
      const Range g = grad_range(plan, grads, i, false);
      clash = meet(g, w[0]) || meet(g, w[1]) || meet(g, w[2]);
    }
    if (clash)
      return fail(MUON_ERR_INVALID_ARG, "out, norms and the workspace must not overlap one "
                  "another or a gradient");

    double* const partial = static_cast<double*>(workspace);
    int* const tensor_part =
        n > 0 ? reinterpret_cast<int*>(static_cast<char*>(workspace) + partial_bytes(plan)) : nullptr;
    NormLaunch L;
    L.part_elems = (int)plan->part_elems;
    L.keep_part = plan->keep_part;
    for (int64_t at = 0; at < n; at += kNormItems) {
      L.count = (int)std::min<int64_t>(kNormItems, n - at);
      L.part0 = plan->part0[at];
      L.blocks = plan->part0[at + L.count] - L.part0;
      L.partial = partial + L.part0;
      L.tensor_part = tensor_part + at;
      for (int c = 0; c < L.count; ++c) {
        const int64_t i = at + c;
        const int first = plan->part0[i] - L.part0;
        const int parts = plan->part0[i + 1] - plan->part0[i];
        L.item[c] = {reinterpret_cast<uint64_t>(grads[i]) | uint64_t(plan->dtype[i] == MUON_DT_F32),
                     first, uint32_t(plan->numel[i] - (parts - 1) * plan->part_elems)};
      }
      hipLaunchKernelGGL(grad_norm_parts_kernel, dim3((unsigned)L.blocks), dim3(kThreads), 0,
                         stream, L);
      if (int st = launched("gradient norm")) return st;
    }
    const int waves = kFinishThreads / 64;
    const unsigned blocks = norms ? unsigned(1 + (n + waves - 1) / waves) : 1u;
    hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(blocks), dim3(kFinishThreads), 0, stream,
                       partial, tensor_part, (int)n, plan->part0.back(), max_norm, out, norms);
    return launched("gradient norm");
  });
}

int muon_grad_scale(const muon_grad_plan* plan, void* const* grads, int64_t n,
                    const float* scale, hipStream_t stream) {
  return c_entry([&]() -> int {
    if (int st = check_grads(plan, grads, n)) return st;
    if (!scale || (reinterpret_cast<uintptr_t>(scale) & 3))
      return fail(MUON_ERR_INVALID_ARG, "scale must be non-NULL and 4-byte aligned");
    std::vector<Range> rs;
    rs.reserve(n + 1);
    for (int64_t i = 0; i < n; ++i)
      if (grads[i] && plan->numel[i] > 0) rs.push_back(grad_range(plan, grads, i, true));
    rs.push_back(range_of(scale, sizeof(float), false));
    if (int st = check_overlaps(rs)) return st;
    constexpr int64_t kMaxBlocks = kMaxTensorElems / kScaleChunk;   // per launch
    ScaleLaunch L;
    L.scale = scale;
    L.count = 0;
    int64_t blocks = 0;
    auto flush = [&]() -> int {
      if (L.count == 0) return MUON_OK;
      hipLaunchKernelGGL(grad_scale_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, L);
      L.count = 0;
      blocks = 0;
      return launched("gradient scale");
    };
    for (int64_t i = 0; i < n; ++i) {
      const int64_t nb = (plan->numel[i] + kScaleChunk - 1) / kScaleChunk;
      if (!grads[i] || nb == 0) continue;
      if (L.count == kScaleItems || blocks + nb > kMaxBlocks)
        if (int st = flush()) return st;
      L.item[L.count++] = {reinterpret_cast<uint64_t>(grads[i]) |
                               uint64_t(plan->dtype[i] == MUON_DT_F32),
                           plan->numel[i], (int)blocks};
      blocks += nb;
    }
    if (int st = flush()) return st;
    return MUON_OK;
  });
}

}  // extern "C"
