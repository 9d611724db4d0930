// gradclip.hip -- the 2-norm over many gradients, and their scaling by
// min(1, max_norm / (norm + eps)) (gfx950).
//
// The tensors travel by value in the kernel's arguments (TAB of them per
// launch), so a call uploads nothing and waits for nothing.  Squares are
// summed in 64 bits: the square of a float is exact there and cannot
// overflow.  Each workgroup of the norm writes one partial sum; the workgroups
// of the scaling add all of them in one fixed order, so results do not depend
// on timing.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "internal.h"

namespace snk {
namespace {

constexpr int TAB = 112;          // tensors per launch (the arguments stay under 4 KB)
constexpr int32_t UNIT = 8192;    // elements a workgroup takes at a time
constexpr int32_t MAX_BLOCKS = 1024;

struct grad_tab {
  const void* g[TAB];
  void* o[TAB];
  int64_t n[TAB];         // elements * 2 + (1 if bf16)
  uint32_t first[TAB + 1];  // units before tensor i
  int32_t count;
};

// Sum over the block of one double per thread, in a fixed order (all threads).
__device__ __forceinline__ double block_sum(double x, double* lds) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m, SNK_WAVE);
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / SNK_WAVE] = x;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// The tensor that unit u belongs to: the last i with first[i] <= u.
__device__ __forceinline__ int tensor_of(const grad_tab& tab, uint32_t u) {
  int lo = 0, hi = tab.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tab.first[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ double unit_squares(const T* __restrict__ g, int64_t n) {
  double s = 0;
  for (int64_t i = threadIdx.x; i < n; i += 256) {
    const double v = elem<T>::to_f(g[i]);
    s = fma(v, v, s);
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void unit_scale(const T* g, T* o, int64_t n, double c) {
  for (int64_t i = threadIdx.x; i < n; i += 256)
    o[i] = elem<T>::from_f((float)(elem<T>::to_f(g[i]) * c));
}

__global__ __launch_bounds__(256) void k_grad_squares(grad_tab tab, double* __restrict__ part) {
  __shared__ double lds[4];
  double s = 0;
  for (uint32_t u = blockIdx.x; u < tab.first[tab.count]; u += gridDim.x) {
    const int i = tensor_of(tab, u);
    const int64_t at = (int64_t)(u - tab.first[i]) * UNIT;
    const int64_t n = min((tab.n[i] >> 1) - at, (int64_t)UNIT);
    if (tab.n[i] & 1) s += unit_squares((const bf16*)tab.g[i] + at, n);
    else s += unit_squares((const float*)tab.g[i] + at, n);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of(const double* __restrict__ part, int32_t n_part,
                                          double* lds) {
  double s = 0;
  for (int32_t i = threadIdx.x; i < n_part; i += 256) s += part[i];
  return sqrt(block_sum(s, lds));
}

__global__ __launch_bounds__(256) void k_grad_norm(const double* __restrict__ part,
                                                   int32_t n_part, float* __restrict__ out) {
  __shared__ double lds[4];
  const double norm = norm_of(part, n_part, lds);
  if (threadIdx.x == 0) *out = (float)norm;
}

__global__ __launch_bounds__(256) void k_grad_scale(grad_tab tab, const double* __restrict__ part,
                                                    int32_t n_part, double max_norm, double eps,
                                                    float* __restrict__ out) {
  __shared__ double lds[4];
  const double norm = norm_of(part, n_part, lds);
  if (out && blockIdx.x == 0 && threadIdx.x == 0) *out = (float)norm;
  // In 64 bits: beside gradients of 1e37 the factor is below fp32's normal range.
  const double q = max_norm / (norm + eps);
  const double c = q >= 1.0 ? 1.0 : q;  // NaN stays NaN
  for (uint32_t u = blockIdx.x; u < tab.first[tab.count]; u += gridDim.x) {
    const int i = tensor_of(tab, u);
    if (c == 1.0 && tab.o[i] == tab.g[i]) continue;  // in place: nothing changes
    const int64_t at = (int64_t)(u - tab.first[i]) * UNIT;
    const int64_t n = min((tab.n[i] >> 1) - at, (int64_t)UNIT);
    if (tab.n[i] & 1) unit_scale((const bf16*)tab.g[i] + at, (bf16*)tab.o[i] + at, n, c);
    else unit_scale((const float*)tab.g[i] + at, (float*)tab.o[i] + at, n, c);
  }
}

snack_status check_grads(const snack_grad* g, int32_t count) {
  if (count < 0) return SNACK_E_COUNT;
  if (count > 0 && !g) return SNACK_E_NULL;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].dtype != SNACK_F32 && g[i].dtype != SNACK_BF16) return SNACK_E_DTYPE;
    if (g[i].n < 0) return SNACK_E_SHAPE;
    if (g[i].n > (int64_t)1 << 40) return SNACK_E_OVERFLOW;
    if (g[i].n > 0 && !g[i].grad) return SNACK_E_NULL;
  }
  return SNACK_OK;
}

inline int32_t launches_of(int32_t count) { return (int32_t)cdiv(std::max(count, 1), TAB); }
inline int32_t blocks_of(int32_t count, uint32_t units) {
  const int32_t most = std::min(MAX_BLOCKS, std::max(32, 4096 / launches_of(count)));
  return (int32_t)std::min<uint32_t>((uint32_t)most, std::max(units, 1u));
}

// The tensors [at, at + TAB) of the list.
grad_tab tab_of(const snack_grad* g, int32_t count, int32_t at) {
  grad_tab tab;
  tab.count = std::min(TAB, count - at);
  uint32_t units = 0;
  for (int32_t i = 0; i < tab.count; ++i) {
    const snack_grad& e = g[at + i];
    tab.g[i] = e.grad;
    tab.o[i] = e.out ? e.out : const_cast<void*>(e.grad);
    tab.n[i] = e.n * 2 + (e.dtype == SNACK_BF16);
    tab.first[i] = units;
    units += (uint32_t)cdiv(e.n, UNIT);
  }
  tab.first[tab.count] = units;
  return tab;
}

// Partial sums of squares of the whole list; how many there are.
int32_t launch_squares(const snack_grad* g, int32_t count, double* part, hipStream_t s) {
  int32_t n_part = 0;
  for (int32_t at = 0; at < count; at += TAB) {
    const grad_tab tab = tab_of(g, count, at);
    if (tab.first[tab.count] == 0) continue;
    const int32_t blocks = blocks_of(count, tab.first[tab.count]);
    hipLaunchKernelGGL(k_grad_squares, dim3(blocks), dim3(256), 0, s, tab, part + n_part);
    n_part += blocks;
  }
  return n_part;
}

size_t ws_of(int32_t count) { return (size_t)launches_of(count) * MAX_BLOCKS * sizeof(double); }

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_grad_workspace(int32_t count, size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  if (count < 0) return SNACK_E_COUNT;
  *bytes = ws_of(count);
  return SNACK_OK;
}

snack_status snack_grad_norm(const snack_grad* grads, int32_t count, float* norm, void* ws,
                             size_t ws_bytes, void* stream) {
  if (snack_status st = check_grads(grads, count)) return st;
  if (!norm || !ws) return SNACK_E_NULL;
  if (ws_bytes < ws_of(count)) return SNACK_E_WORKSPACE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int32_t n_part = launch_squares(grads, count, (double*)ws, s);
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, s, (const double*)ws, n_part, norm);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

snack_status snack_grad_clip(const snack_grad* grads, int32_t count, float max_norm, float eps,
                             float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (snack_status st = check_grads(grads, count)) return st;
  if (std::isnan(max_norm) || std::isnan(eps)) return SNACK_E_NAN;
  if (max_norm < 0 || eps < 0) return SNACK_E_SHAPE;
  if (!ws) return SNACK_E_NULL;
  if (ws_bytes < ws_of(count)) return SNACK_E_WORKSPACE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int32_t n_part = launch_squares(grads, count, (double*)ws, s);
  if (n_part == 0 && norm)  // nothing to scale: the norm is 0
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, s, (const double*)ws, 0, norm);
  for (int32_t at = 0; at < count; at += TAB) {
    const grad_tab tab = tab_of(grads, count, at);
    if (tab.first[tab.count] == 0) continue;
    hipLaunchKernelGGL(k_grad_scale, dim3(blocks_of(count, tab.first[tab.count])), dim3(256), 0, s,
                       tab, (const double*)ws, n_part, (double)max_norm, (double)eps, norm);
    norm = nullptr;  // the first launch writes it
  }
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
