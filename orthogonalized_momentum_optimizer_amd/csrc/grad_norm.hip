// The global gradient norm and its clipping scale over many tensors: host side and kernels of
// the C ABI in include/grad_norm.h.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  scale = min(1, max_norm / norm)
//
// Each tensor is cut into parts of equal length; a block sums one part's squares in double
// (fp32's squares overflow at 1.8e19 and lose their bits below 1e-19) and writes one partial
// sum. A second launch of one block joins the partial sums in a fixed order.
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
  std::vector<int> of[2];       // tensors of each dtype, in order
};

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;
constexpr int kMaxItems = 64;                    // tensors per launch
constexpr int64_t kMinPart = 16384;
constexpr int64_t kMaxParts = 16384;             // beyond one per tensor
constexpr int kFinishThreads = 1024;

struct NormLaunch {
  const void* g[kMaxItems];
  int64_t numel[kMaxItems];
  int first[kMaxItems];                          // first block of each tensor in this launch
  int part0[kMaxItems];                          // its first part
  int id[kMaxItems];
  double* partial;
  int* tensor_part;                              // out: first part of each tensor
  int64_t part_elems;
};

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

template <int GD>
__global__ __launch_bounds__(kThreads) void grad_norm_parts_kernel(const NormLaunch L) {
  const int b = blockIdx.x;
  const int q = find_tensor(L.first, b);
  const void* const G = L.g[q];
  const int k = b - L.first[q];
  const int64_t lo = int64_t(k) * L.part_elems;
  const int64_t hi = min(lo + L.part_elems, L.numel[q]);
  double acc = 0.0;
  if (G) {
    int64_t i = lo + int64_t(threadIdx.x) * kVec;
    for (; i + kVec <= hi; i += kThreads * kVec) {
      float x[kVec];
      load_vec<GD>(G, i, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc = fma(double(x[e]), double(x[e]), acc);
    }
    for (; i < hi; ++i) {                        // the thread whose vector the end cuts
      const double x = load_one<GD>(G, i);
      acc = fma(x, x, acc);
    }
  }
  const double sum = block_sum<kThreads>(acc);
  if (threadIdx.x == 0) {
    L.partial[L.part0[q] + k] = sum;
    if (k == 0) L.tensor_part[L.id[q]] = L.part0[q];
  }
}

__global__ __launch_bounds__(kFinishThreads) void grad_norm_finish_kernel(
    const double* __restrict__ partial, const int* __restrict__ tensor_part, int tensors,
    int parts, float max_norm, float* out, float* norms) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kFinishThreads) acc += partial[i];
  const double sum = block_sum<kFinishThreads>(acc);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum);
    const bool finite = norm <= 1.7976931348623157e308;   // false for NaN too
    out[0] = float(norm);
    out[1] = !finite ? __uint_as_float(0x7fc00000u)
                     : norm > double(max_norm) ? float(double(max_norm) / norm) : 1.f;
  }
  if (!norms) return;
  const int lane = threadIdx.x & 63;
  for (int t = threadIdx.x >> 6; t < tensors; t += kFinishThreads / 64) {
    const int lo = tensor_part[t], hi = t + 1 < tensors ? tensor_part[t + 1] : parts;
    double x = 0.0;
    for (int i = lo + lane; i < hi; i += 64) x += partial[i];
    x = wave_sum(x);
    if (lane == 0) norms[t] = float(sqrt(x));
  }
}

constexpr int kScaleChunk = kThreads * kVec * 2;

struct ScaleLaunch {
  void* g[kMaxItems];
  int64_t numel[kMaxItems];
  int first[kMaxItems];
  const float* scale;
};

template <int GD>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const ScaleLaunch L) {
  const float s = *L.scale;
  if (s == 1.f) return;
  const int b = blockIdx.x;
  const int q = find_tensor(L.first, b);
  void* const G = L.g[q];
  const int64_t n = L.numel[q];
  const int64_t base = int64_t(b - L.first[q]) * kScaleChunk;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t i = base + int64_t(u * kThreads + threadIdx.x) * kVec;
    if (i + kVec <= n) {
      float x[kVec];
      load_vec<GD>(G, i, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] *= s;
      store_vec<GD>(G, i, x);
    } else {
      for (int64_t j = i; j < n; ++j) store_one<GD>(G, j, load_one<GD>(G, j) * s);
    }
  }
}

int check_grads(const muon_grad_plan* plan, const void* const* grads, int64_t n,
                bool written, std::vector<Range>& rs) {
  if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
  if (n != (int64_t)plan->numel.size())
    return fail(MUON_ERR_INVALID_ARG, "n = %lld but the plan has %zu gradients", (long long)n,
                plan->numel.size());
  if (n > 0 && !grads) return fail(MUON_ERR_INVALID_ARG, "grads is NULL");
  for (int64_t i = 0; i < n; ++i) {
    if (!grads[i] || plan->numel[i] == 0) continue;
    if (!is_aligned16(grads[i]))
      return fail(MUON_ERR_INVALID_ARG, "gradient %lld must be 16-byte aligned", (long long)i);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i]);
    rs.push_back({lo, lo + (size_t)plan->numel[i] * dtype_bytes(plan->dtype[i]), written});
  }
  return MUON_OK;
}

void add_range(std::vector<Range>& rs, const void* p, size_t bytes, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  rs.push_back({lo, lo + bytes, written});
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
    while (total / (double)made.part_elems > (double)kMaxParts) made.part_elems *= 2;
    int64_t parts = 0;
    for (int64_t i = 0; i < n; ++i) {
      made.part0.push_back((int)parts);
      parts += std::max<int64_t>(1, (numel[i] + made.part_elems - 1) / made.part_elems);
      made.of[dtype[i] == MUON_DT_F32].push_back((int)i);
    }
    made.part0.push_back((int)parts);
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
    std::vector<Range> rs;
    if (int st = check_grads(plan, grads, n, false, rs)) return st;
    if (!(max_norm >= 0.f))
      return fail(MUON_ERR_INVALID_ARG, "max_norm must be >= 0 (infinity: no clipping)");
    if (!out) return fail(MUON_ERR_INVALID_ARG, "out is NULL");
    const size_t need = muon_grad_plan_workspace_size(plan);
    if (need > 0 && (!workspace || !is_aligned16(workspace) || workspace_bytes < need))
      return fail(MUON_ERR_WORKSPACE, "a workspace of %zu bytes, 16-byte aligned, is needed", need);
    add_range(rs, out, 2 * sizeof(float), true);
    if (norms && n > 0) add_range(rs, norms, n * sizeof(float), true);
    if (need > 0) add_range(rs, workspace, need, true);
    if (int st = check_overlaps(rs)) return st;

    NormLaunch L;
    L.partial = static_cast<double*>(workspace);
    L.tensor_part = n > 0 ? reinterpret_cast<int*>(static_cast<char*>(workspace) + partial_bytes(plan))
                          : nullptr;
    L.part_elems = plan->part_elems;
    for (int dt = 0; dt < 2; ++dt) {
      const std::vector<int>& of = plan->of[dt];
      for (size_t at = 0; at < of.size(); at += kMaxItems) {
        const int count = (int)std::min<size_t>(kMaxItems, of.size() - at);
        int blocks = 0;
        for (int c = 0; c < kMaxItems; ++c) {
          L.first[c] = INT_MAX;
          if (c >= count) continue;
          const int i = of[at + c];
          L.g[c] = grads[i];
          L.numel[c] = plan->numel[i];
          L.first[c] = blocks;
          L.part0[c] = plan->part0[i];
          L.id[c] = i;
          blocks += plan->part0[i + 1] - plan->part0[i];
        }
        hipLaunchKernelGGL(dt ? grad_norm_parts_kernel<1> : grad_norm_parts_kernel<0>,
                           dim3((unsigned)blocks), dim3(kThreads), 0, stream, L);
        if (int st = launched("gradient norm")) return st;
      }
    }
    hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(1), dim3(kFinishThreads), 0, stream,
                       L.partial, L.tensor_part, (int)n, plan->part0.back(), max_norm, out, norms);
    return launched("gradient norm");
  });
}

int muon_grad_scale(const muon_grad_plan* plan, void* const* grads, int64_t n,
                    const float* scale, hipStream_t stream) {
  return c_entry([&]() -> int {
    std::vector<Range> rs;
    if (int st = check_grads(plan, grads, n, true, rs)) return st;
    if (!scale) return fail(MUON_ERR_INVALID_ARG, "scale is NULL");
    add_range(rs, scale, sizeof(float), false);
    if (int st = check_overlaps(rs)) return st;
    constexpr int64_t kMaxBlocks = kMaxTensorElems / kScaleChunk;   // per launch
    ScaleLaunch L;
    L.scale = scale;
    for (int dt = 0; dt < 2; ++dt) {
      int count = 0;
      int64_t blocks = 0;
      auto flush = [&]() -> int {
        if (count == 0) return MUON_OK;
        for (int c = count; c < kMaxItems; ++c) L.first[c] = INT_MAX;
        hipLaunchKernelGGL(dt ? grad_scale_kernel<1> : grad_scale_kernel<0>,
                           dim3((unsigned)blocks), dim3(kThreads), 0, stream, L);
        count = 0;
        blocks = 0;
        return launched("gradient scale");
      };
      for (int i : plan->of[dt]) {
        if (!grads[i]) continue;
        const int64_t nb = (plan->numel[i] + kScaleChunk - 1) / kScaleChunk;
        if (nb == 0) continue;
        if (count == kMaxItems || blocks + nb > kMaxBlocks)
          if (int st = flush()) return st;
        L.g[count] = grads[i];
        L.numel[count] = plan->numel[i];
        L.first[count++] = (int)blocks;
        blocks += nb;
      }
      if (int st = flush()) return st;
    }
    return MUON_OK;
  });
}

}  // extern "C"
