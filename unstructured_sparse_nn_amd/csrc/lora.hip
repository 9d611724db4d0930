// lora.hip -- low-rank adapters of many requests beside a shared projection
// (gfx950).  With a = ids[i] the adapter of token i, r its rank, s its scale:
//   t[i, j]  = sum_k A[a, j, k] X[i, k]                       (reduce)
//   Y[i, m]  = base[i, m] + s sum_{j < r} t[i, j] B[a, j, m]  (expand)
// and, with u[i, j] = sum_m B[a, j, m] dY[i, m] (reduce),
//   dX[i, k] = base[i, k] + s sum_{j < r} u[i, j] A[a, j, k]  (expand)
//   dA[l, j, k] = s sum_{i : ids[i] = l} u[i, j] X[i, k]      (grad)
//   dB[l, j, m] = s sum_{i : ids[i] = l} t[i, j] dY[i, m]     (grad)
// Both factors are stored by rank (L x R x K and L x R x M), so three kernels
// serve both directions.
#include <algorithm>
#include <cstring>

#include "common.h"
#include "internal.h"

namespace snk {
namespace {

struct lora_dev {  // what every kernel needs of the adapters
  int32_t L, R;
  const float* scale;   // [L] or NULL
  const int32_t* rank;  // [L] or NULL
};

__device__ __forceinline__ int32_t rank_of(const lora_dev& d, int32_t l) {
  return d.rank ? min(max(d.rank[l], 0), d.R) : d.R;
}
__device__ __forceinline__ float scale_of(const lora_dev& d, int32_t l) {
  return d.scale ? d.scale[l] : 1.f;
}

// One wave per (token, rank): t[i, j] = sum_k F[a, j, k] X[i, k].
template <typename T>
__global__ __launch_bounds__(256) void k_lora_reduce(lora_dev d, const int32_t* __restrict__ ids,
                                                     const T* __restrict__ F, int32_t K,
                                                     const T* __restrict__ X, int64_t ldx,
                                                     int32_t Tn, float* __restrict__ t) {
  const int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) / SNK_WAVE;
  if (w >= (int64_t)Tn * d.R) return;
  const int32_t i = (int32_t)(w / d.R), j = (int32_t)(w % d.R);
  const int32_t a = ids[i];
  float acc = 0.f;
  if (a >= 0 && a < d.L && j < rank_of(d, a)) {
    const T* f = F + ((int64_t)a * d.R + j) * K;
    const T* x = X + (int64_t)i * ldx;
    for (int32_t k = lane_id(); k < K; k += SNK_WAVE)
      acc = fmaf(elem<T>::to_f(f[k]), elem<T>::to_f(x[k]), acc);
  }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m, SNK_WAVE);
  if (lane_id() == 0) t[(int64_t)i * d.R + j] = acc;
}

// One thread per output: Y[i, m] = base[i, m] + s sum_j t[i, j] F[a, j, m].
// A token whose id lies past the last adapter gets NaN.
template <typename T>
__global__ __launch_bounds__(256) void k_lora_expand(lora_dev d, const int32_t* __restrict__ ids,
                                                     const T* __restrict__ F, int32_t M,
                                                     const float* __restrict__ t, const T* base,
                                                     int64_t ldb, T* Y, int64_t ldy) {
  const int32_t m = blockIdx.y * 256 + threadIdx.x;
  const int64_t i = blockIdx.x;
  if (m >= M) return;
  const int32_t a = ids[i];
  float acc = 0.f;
  if (a >= d.L) {
    acc = __builtin_nanf("");
  } else if (a >= 0) {
    const int32_t r = rank_of(d, a);
    for (int32_t j = 0; j < r; ++j)
      acc = fmaf(t[i * d.R + j], elem<T>::to_f(F[((int64_t)a * d.R + j) * M + m]), acc);
    acc *= scale_of(d, a);
  }
  if (base) acc += elem<T>::to_f(base[i * ldb + m]);
  Y[i * ldy + m] = elem<T>::from_f(acc);
}

// One thread per gradient element of one adapter, over all tokens.
template <typename T>
__global__ __launch_bounds__(256) void k_lora_grad(lora_dev d, const int32_t* __restrict__ ids,
                                                   int32_t Tn, const float* __restrict__ t,
                                                   const T* __restrict__ X, int64_t ldx, int32_t K,
                                                   T* __restrict__ dF) {
  const int32_t k = blockIdx.y * 256 + threadIdx.x;
  const int32_t l = blockIdx.x / d.R, j = blockIdx.x % d.R;
  if (k >= K) return;
  float acc = 0.f;
  if (j < rank_of(d, l))
    for (int64_t i = 0; i < Tn; ++i)
      if (ids[i] == l) acc = fmaf(t[i * d.R + j], elem<T>::to_f(X[i * ldx + k]), acc);
  dF[((int64_t)l * d.R + j) * K + k] = elem<T>::from_f(acc * scale_of(d, l));
}

constexpr int32_t MAX_RANK = 256;
constexpr int32_t MAX_ADAPTERS = 8192;

snack_status check_lora(const snack_lora* p, snack_dtype dt, int32_t T) {
  if (!p) return SNACK_E_NULL;
  if (dt != SNACK_F32 && dt != SNACK_BF16) return SNACK_E_DTYPE;
  if (p->M < 1 || p->K < 1 || p->L < 1 || p->L > MAX_ADAPTERS || p->R < 1 || p->R > MAX_RANK ||
      T < 0)
    return SNACK_E_SHAPE;
  return SNACK_OK;
}

struct bwd_ws {
  size_t u, t, total;
};

bwd_ws bwd_layout(const snack_lora* p, int32_t T) {
  bwd_ws w{};
  const size_t b = align_up(4 * (size_t)T * p->R, 256);
  w.u = 0;
  w.t = b;
  w.total = 2 * b;
  return w;
}

template <typename T>
void reduce(const lora_dev& d, const int32_t* ids, const void* F, int32_t K, const void* X,
            int64_t ldx, int32_t Tn, float* t, hipStream_t s) {
  hipLaunchKernelGGL(k_lora_reduce<T>, dim3((unsigned)cdiv((int64_t)Tn * d.R, 4)), dim3(256), 0, s,
                     d, ids, (const T*)F, K, (const T*)X, ldx, Tn, t);
}

template <typename T>
void expand(const lora_dev& d, const int32_t* ids, const void* F, int32_t M, const float* t,
            const void* base, int64_t ldb, void* Y, int64_t ldy, int32_t Tn, hipStream_t s) {
  hipLaunchKernelGGL(k_lora_expand<T>, dim3(Tn, (unsigned)cdiv(M, 256)), dim3(256), 0, s, d, ids,
                     (const T*)F, M, t, (const T*)base, ldb, (T*)Y, ldy);
}

template <typename T>
void grad(const lora_dev& d, const int32_t* ids, int32_t Tn, const float* t, const void* X,
          int64_t ldx, int32_t K, void* dF, hipStream_t s) {
  hipLaunchKernelGGL(k_lora_grad<T>, dim3(d.L * d.R, (unsigned)cdiv(K, 256)), dim3(256), 0, s, d,
                     ids, Tn, t, (const T*)X, ldx, K, (T*)dF);
}

template <typename T>
void run_bwd(const snack_lora* p, const lora_dev& d, const int32_t* ids, const float* t,
             int32_t Tn, const void* X, int64_t ldx, const void* dY, int64_t lddy,
             const void* base, int64_t ldb, void* dX, int64_t lddx, void* dA, void* dB, char* ws,
             hipStream_t s) {
  const bwd_ws w = bwd_layout(p, Tn);
  float* u = (float*)(ws + w.u);
  if (Tn > 0 && (dX || dA)) reduce<T>(d, ids, p->B, p->M, dY, lddy, Tn, u, s);
  if (Tn > 0 && dB && !t) {
    reduce<T>(d, ids, p->A, p->K, X, ldx, Tn, (float*)(ws + w.t), s);
    t = (const float*)(ws + w.t);
  }
  if (Tn > 0 && dX) expand<T>(d, ids, p->A, p->K, u, base, ldb, dX, lddx, Tn, s);
  if (dA) grad<T>(d, ids, Tn, u, X, ldx, p->K, dA, s);
  if (dB) grad<T>(d, ids, Tn, t, dY, lddy, p->M, dB, s);
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_lora_workspace(const snack_lora* lora, snack_dtype dtype, int32_t T,
                                  int32_t backward, size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  if (snack_status st = check_lora(lora, dtype, T)) return st;
  *bytes = backward ? bwd_layout(lora, T).total : align_up(4 * (size_t)T * lora->R, 256);
  return SNACK_OK;
}

snack_status snack_lora_fwd(const snack_lora* lora, snack_dtype dtype, const int32_t* ids,
                            int32_t T, const void* X, int64_t ldx, const void* base, int64_t ldb,
                            void* Y, int64_t ldy, float* t, void* ws, size_t ws_bytes,
                            void* stream) {
  if (snack_status st = check_lora(lora, dtype, T)) return st;
  if (ldx < lora->K || ldy < lora->M || (base && ldb < lora->M)) return SNACK_E_SHAPE;
  if (T == 0) return SNACK_OK;
  if (!lora->A || !lora->B || !ids || !X || !Y || !ws) return SNACK_E_NULL;
  if (Y == X || (Y == base && ldy != ldb)) return SNACK_E_SHAPE;
  size_t need;
  snack_lora_workspace(lora, dtype, T, 0, &need);
  if (ws_bytes < need) return SNACK_E_WORKSPACE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const lora_dev d{lora->L, lora->R, lora->scale, lora->rank};
  if (!t) t = (float*)ws;
  if (dtype == SNACK_BF16) {
    reduce<bf16>(d, ids, lora->A, lora->K, X, ldx, T, t, s);
    expand<bf16>(d, ids, lora->B, lora->M, t, base, ldb, Y, ldy, T, s);
  } else {
    reduce<float>(d, ids, lora->A, lora->K, X, ldx, T, t, s);
    expand<float>(d, ids, lora->B, lora->M, t, base, ldb, Y, ldy, T, s);
  }
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

snack_status snack_lora_bwd(const snack_lora* lora, snack_dtype dtype, const int32_t* ids,
                            const float* t, int32_t T, const void* X, int64_t ldx, const void* dY,
                            int64_t lddy, const void* base, int64_t ldb, void* dX, int64_t lddx,
                            void* dA, void* dB, void* ws, size_t ws_bytes, void* stream) {
  if (snack_status st = check_lora(lora, dtype, T)) return st;
  if (ldx < lora->K || lddy < lora->M || (dX && lddx < lora->K) || (base && ldb < lora->K))
    return SNACK_E_SHAPE;
  if (T > 0) {
    if (!lora->A || !lora->B || !ids || !X || !dY || !ws) return SNACK_E_NULL;
    if (dX && (dX == X || dX == dY || (dX == base && lddx != ldb))) return SNACK_E_SHAPE;
    size_t need;
    snack_lora_workspace(lora, dtype, T, 1, &need);
    if (ws_bytes < need) return SNACK_E_WORKSPACE;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const lora_dev d{lora->L, lora->R, lora->scale, lora->rank};
  if (dtype == SNACK_BF16)
    run_bwd<bf16>(lora, d, ids, t, T, X, ldx, dY, lddy, base, ldb, dX, lddx, dA, dB, (char*)ws, s);
  else
    run_bwd<float>(lora, d, ids, t, T, X, ldx, dY, lddy, base, ldb, dX, lddx, dA, dB, (char*)ws, s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
