// gradclip.hip -- the 2-norm over many gradients, and their scaling by
// min(1, max_norm / (norm + eps)) (gfx950).
//
// The tensors travel by value in the kernel's arguments (TAB of them per
// launch; tensors that follow each other in memory count as one), so a call
// uploads nothing and waits for nothing.  Squares are summed in 64 bits: the
// square of a float is exact there and cannot overflow.  Each workgroup of the
// norm writes one partial sum; the workgroups of the scaling add all of them in
// one fixed order, so results do not depend on timing.
//
// Bound by memory: the gradients are read twice and written once, 16 bytes a
// lane.  48 bf16 gradients of 274 MB: norm 47 us (5.8 TB/s), scaling 91 us (6.0
// TB/s); 600 views of one 37 MB bucket: 11 and 18 us; 48 fp32 gradients of 1 MB:
// 4.3 and 5.5 us, launch and three trips to memory each.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "common.h"
#include "internal.h"

namespace snk {
namespace {

constexpr int TAB = 112;          // tensors per launch (the arguments stay under 4 KB)
constexpr int32_t MAX_BLOCKS = 4096;

// Lists of more than BIG_BYTES leave no room for their outputs in the 256 MB
// cache before memory: those are stored past the caches, since the lines that
// plain stores leave there have to be written back while the next call reads,
// and workgroups take larger units.  Lists of bf16 gradients out of place, small
// units with plain stores against this: 160 MB in 48 tensors 111 and 96 us, 274 MB
// 181 and 147 us, 800 MB 501 and 431 us, in 400 tensors 569 and 581 us; 1 MB of fp32
// in 48: 9.8 and 11.5 us.  Not taken: out of place it pays from 37 MB on (33.5 and
// 28.9 us; 96 MB 68 and 56 us).
constexpr int64_t BIG_BYTES = 128ll << 20;
constexpr int32_t unit_of(bool big) { return big ? 16384 : 4096; }  // elements

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

// A workgroup's share of the units, in order, with the tensor of each: the
// first one is found by all lanes at once, the next ones by walking on.
struct walk_t { uint32_t u, end; int i; };

__device__ __forceinline__ walk_t walk_of(const grad_tab& tab) {
  const uint64_t units = tab.first[tab.count];
  walk_t w;
  w.u = (uint32_t)(units * blockIdx.x / gridDim.x);
  w.end = (uint32_t)(units * (blockIdx.x + 1) / gridDim.x);
  int n = 0;  // tensors that begin at or before unit u
#pragma unroll
  for (int q = 0; q < (TAB + 63) / 64; ++q) {
    const int i = q * 64 + lane_id();
    n += __popcll(__ballot(i < tab.count && tab.first[min(i, TAB)] <= w.u));
  }
  w.i = n - 1;
  return w;
}

// Pieces of 16 bytes, at any alignment.
template <typename T> constexpr int EL = 16 / sizeof(T);
template <typename T, bool BIG> constexpr int PIECES = unit_of(BIG) / 256 / EL<T>;  // of a thread

template <typename T>
__device__ __forceinline__ vec<T, EL<T>> load16(const T* p) {
  vec<T, EL<T>> v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

template <bool BIG, typename T>
__device__ __forceinline__ double unit_squares(const T* __restrict__ g, int64_t n) {
  constexpr int E = EL<T>;
  double s[2] = {0, 0};
  auto add = [&](const vec<T, E>& v) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const double x = elem<T>::to_f(v.v[e]);
      s[e & 1] = fma(x, x, s[e & 1]);
    }
  };
  if (n == unit_of(BIG)) {
    vec<T, E> v[PIECES<T, BIG>];
#pragma unroll
    for (int q = 0; q < PIECES<T, BIG>; ++q) v[q] = load16(g + (q * 256 + threadIdx.x) * E);
#pragma unroll
    for (int q = 0; q < PIECES<T, BIG>; ++q) add(v[q]);
  } else {
    const int32_t whole = (int32_t)n / E;
#pragma unroll 4
    for (int32_t q = threadIdx.x; q < whole; q += 256) add(load16(g + q * E));
    const int32_t i = whole * E + (int32_t)threadIdx.x;
    if (i < n) {
      const double x = elem<T>::to_f(g[i]);
      s[0] = fma(x, x, s[0]);
    }
  }
  return s[0] + s[1];
}

// A rounding of g * c to float and, for bf16, one more.
template <bool BIG, typename T>
__device__ __forceinline__ void unit_scale(const T* g, T* o, int64_t n, double c) {
  constexpr int E = EL<T>;
  auto put = [&](int32_t at, vec<T, E> v) {
#pragma unroll
    for (int e = 0; e < E; ++e) v.v[e] = elem<T>::from_f((float)(elem<T>::to_f(v.v[e]) * c));
    if constexpr (BIG) {
      typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
      __builtin_nontemporal_store(__builtin_bit_cast(u4, v), reinterpret_cast<u4*>(o + at));
    } else {
      __builtin_memcpy(o + at, &v, 16);
    }
  };
  if (n == unit_of(BIG)) {
    vec<T, E> v[PIECES<T, BIG>];
#pragma unroll
    for (int q = 0; q < PIECES<T, BIG>; ++q) v[q] = load16(g + (q * 256 + threadIdx.x) * E);
#pragma unroll
    for (int q = 0; q < PIECES<T, BIG>; ++q) put((q * 256 + threadIdx.x) * E, v[q]);
  } else {
    const int32_t whole = (int32_t)n / E;
#pragma unroll 4
    for (int32_t q = threadIdx.x; q < whole; q += 256) put(q * E, load16(g + q * E));
    const int32_t i = whole * E + (int32_t)threadIdx.x;
    if (i < n) o[i] = elem<T>::from_f((float)(elem<T>::to_f(g[i]) * c));
  }
}

template <bool BIG>
__global__ __launch_bounds__(256) void k_grad_squares(grad_tab tab, double* __restrict__ part) {
  __shared__ double lds[4];
  double s = 0;
  for (walk_t w = walk_of(tab); w.u < w.end; ++w.u) {
    while (tab.first[w.i + 1] <= w.u) ++w.i;
    const int64_t at = (int64_t)(w.u - tab.first[w.i]) * unit_of(BIG);
    const int64_t n = min((tab.n[w.i] >> 1) - at, (int64_t)unit_of(BIG));
    if (tab.n[w.i] & 1) s += unit_squares<BIG>((const bf16*)tab.g[w.i] + at, n);
    else s += unit_squares<BIG>((const float*)tab.g[w.i] + at, n);
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

// The table holds the tensors from the last to the first, and a tensor's units
// are taken from its end: what the norm read last is still in the caches.
template <bool BIG>
__global__ __launch_bounds__(256) void k_grad_scale(grad_tab tab, const double* __restrict__ part,
                                                    int32_t n_part, double max_norm, double eps,
                                                    float* __restrict__ out) {
  __shared__ double lds[4];
  walk_t w = walk_of(tab);
  const double norm = norm_of(part, n_part, lds);
  if (out && blockIdx.x == 0 && threadIdx.x == 0) *out = (float)norm;
  // In 64 bits: beside gradients of 1e37 the factor is below fp32's normal range.
  const double q = max_norm / (norm + eps);
  const double c = q >= 1.0 ? 1.0 : q;  // NaN stays NaN
  for (; w.u < w.end; ++w.u) {
    while (tab.first[w.i + 1] <= w.u) ++w.i;
    if (c == 1.0 && tab.o[w.i] == tab.g[w.i]) continue;  // in place: nothing changes
    const int64_t at = (int64_t)(tab.first[w.i + 1] - 1 - w.u) * unit_of(BIG);
    const int64_t n = min((tab.n[w.i] >> 1) - at, (int64_t)unit_of(BIG));
    if (tab.n[w.i] & 1) unit_scale<BIG>((const bf16*)tab.g[w.i] + at, (bf16*)tab.o[w.i] + at, n, c);
    else unit_scale<BIG>((const float*)tab.g[w.i] + at, (float*)tab.o[w.i] + at, n, c);
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

// Workgroups read and write the list in any order, so what one of them writes
// must belong to no other entry: outputs must not share memory with each other,
// nor with a gradient that is not scaled in place.
snack_status check_shared(const snack_grad* g, int32_t count) {
  struct span { uintptr_t at, end; };
  if (count == 0) return SNACK_OK;
  const std::unique_ptr<span[]> to(new (std::nothrow) span[count]);
  if (!to) return SNACK_E_WORKSPACE;
  auto span_of = [](const snack_grad& e, const void* p) {
    return span{(uintptr_t)p, (uintptr_t)p + e.n * (e.dtype == SNACK_BF16 ? 2 : 4)};
  };
  auto before = [](const span& a, const span& b) { return a.at < b.at; };
  int32_t n = 0;
  for (int32_t i = 0; i < count; ++i)
    if (g[i].n > 0) to[n++] = span_of(g[i], g[i].out ? g[i].out : g[i].grad);
  span *const first = to.get(), *const last = first + n;
  if (!std::is_sorted(first, last, before)) std::sort(first, last, before);
  for (int32_t i = 1; i < n; ++i)
    if (to[i].at < to[i - 1].end) return SNACK_E_SHAPE;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].n == 0 || !g[i].out || g[i].out == g[i].grad) continue;
    const span r = span_of(g[i], g[i].grad);
    if (r.at >= last[-1].end || r.end <= first->at) continue;
    const span* next = std::lower_bound(first, last, r, before);  // the first that begins in r or after it
    if ((next != last && next->at < r.end) || (next != first && next[-1].end > r.at))
      return SNACK_E_SHAPE;
  }
  return SNACK_OK;
}

inline bool is_big(const snack_grad* g, int32_t count) {
  int64_t bytes = 0;
  for (int32_t i = 0; i < count && bytes <= BIG_BYTES; ++i)
    bytes += g[i].n * (g[i].dtype == SNACK_BF16 ? 2 : 4);
  return bytes > BIG_BYTES;
}

inline int32_t launches_of(int32_t count) { return (int32_t)cdiv(std::max(count, 1), TAB); }
// Small units: 8 workgroups on every CU at most (600 views of one 37 MB bucket:
// 29 us, 31 us with 11).
inline int32_t blocks_of(int32_t count, bool big, uint32_t units) {
  const int32_t most =
      std::min(big ? MAX_BLOCKS : MAX_BLOCKS / 2, std::max(64, 16384 / launches_of(count)));
  return (int32_t)std::min<uint32_t>((uint32_t)most, std::max(units, 1u));
}

// Fills the table from entry `at` on, forwards or backwards (step 1 or -1), and
// returns the entry after the last one taken.  Empty tensors are left out;
// tensors that follow each other in memory, as views of one bucket do, become
// one.
int32_t fill_tab(const snack_grad* g, int32_t count, int32_t at, int32_t step, bool big,
                 grad_tab& tab) {
  tab.count = 0;
  for (; at >= 0 && at < count; at += step) {
    const snack_grad& e = g[at];
    if (e.n == 0) continue;
    const int64_t size = e.dtype == SNACK_BF16 ? 2 : 4;
    const char *src = (const char*)e.grad, *dst = e.out ? (const char*)e.out : src;
    if (tab.count > 0) {
      const int i = tab.count - 1;
      const int64_t n = tab.n[i] >> 1;
      const char *ps = (const char*)tab.g[i], *pd = (const char*)tab.o[i];
      const bool after = step > 0 ? src == ps + n * size && dst == pd + n * size
                                  : src + e.n * size == ps && dst + e.n * size == pd;
      if (after && (tab.n[i] & 1) == (e.dtype == SNACK_BF16)) {
        tab.n[i] += e.n * 2;
        if (step < 0) tab.g[i] = e.grad, tab.o[i] = const_cast<char*>(dst);
        continue;
      }
      if (tab.count == TAB) break;
    }
    tab.g[tab.count] = e.grad;
    tab.o[tab.count] = const_cast<char*>(dst);
    tab.n[tab.count++] = e.n * 2 + (e.dtype == SNACK_BF16);
  }
  uint32_t units = 0;
  for (int32_t i = 0; i < tab.count; ++i) {
    tab.first[i] = units;
    units += (uint32_t)cdiv(tab.n[i] >> 1, unit_of(big));
  }
  tab.first[tab.count] = units;
  return at;
}

// Partial sums of squares of the whole list; how many there are.
int32_t launch_squares(const snack_grad* g, int32_t count, bool big, double* part, hipStream_t s) {
  int32_t n_part = 0;
  grad_tab tab;
  for (int32_t at = 0; at < count;) {
    at = fill_tab(g, count, at, 1, big, tab);
    if (tab.count == 0) break;
    const int32_t blocks = blocks_of(count, big, tab.first[tab.count]);
    hipLaunchKernelGGL(big ? k_grad_squares<true> : k_grad_squares<false>, dim3(blocks), dim3(256),
                       0, s, tab, part + n_part);
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
  const bool big = is_big(grads, count);
  const int32_t n_part = launch_squares(grads, count, big, (double*)ws, s);
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
  if (snack_status st = check_shared(grads, count)) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool big = is_big(grads, count);
  const int32_t n_part = launch_squares(grads, count, big, (double*)ws, s);
  if (n_part == 0 && norm)  // nothing to scale: the norm is 0
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, s, (const double*)ws, 0, norm);
  grad_tab tab;
  for (int32_t at = count - 1; at >= 0;) {
    at = fill_tab(grads, count, at, -1, big, tab);
    if (tab.count == 0) break;
    hipLaunchKernelGGL(big ? k_grad_scale<true> : k_grad_scale<false>,
                       dim3(blocks_of(count, big, tab.first[tab.count])), dim3(256), 0, s, tab,
                       (const double*)ws, n_part, (double)max_norm, (double)eps, norm);
    norm = nullptr;  // the first launch writes it
  }
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
