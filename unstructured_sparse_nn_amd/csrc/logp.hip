// logp.hip -- log-probabilities of target tokens from logits, and the logits'
// gradient (gfx950).  With m_i = max_v x[i, v] and l_i = log sum_v exp(x[i, v] - m_i):
//   logp[i]  = (x[i, t_i] - m_i) - l_i
//   dx[i, v] = g_i ([v = t_i] - exp((x[i, v] - m_i) - l_i))
// m and l are kept apart (norm): in their sum l would lose the digits that m has
// before it (logits near 10^4 would leave three of a probability).
//
// Both are bound by memory.  The forward reads the logits once: every thread
// keeps a running maximum and sum, whose sum is scaled where the maximum grows;
// long rows of few are cut among workgroups, whose pairs k_logp_join adds.  The
// backward reads and writes them once, and does not read rows whose gradient is 0.
// Figures here are of replays of a graph of calls.  8,192 rows of 32,000 bf16: 95 us
// (5.5 TB/s; 92 us in calls one after another), backward 190 us (5.5 TB/s); 4,099 of
// 50,001, 30% without a target, backward 134 us (5.2 TB/s); 5 of 128,000: 6.4 us.
#include "common.h"
#include "internal.h"
#include "pieces.h"
#include "spans.h"

namespace snk {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }

// A maximum and the sum of exp(x - maximum).  The maximum starts at the lowest
// float, not at -infinity: a logit of -infinity then adds exp(-infinity), and one
// of the lowest float counts.  NaN and +infinity leave NaN in the sum.
struct soft_t { float m, s; };
constexpr float LOWEST = -3.4028234663852886e38f;

__device__ __forceinline__ soft_t join(soft_t a, soft_t b) {
  const float m = fmaxf(a.m, b.m);
  return {m, a.s * exp_of(a.m - m) + b.s * exp_of(b.m - m)};
}
// Of each N lanes.
template <int N>
__device__ __forceinline__ soft_t lanes_join(soft_t a) {
#pragma unroll
  for (int d = N / 2; d; d >>= 1)
    a = join(a, soft_t{__shfl_xor(a.m, d), __shfl_xor(a.s, d)});
  return a;
}

template <typename T, int U>
__device__ __forceinline__ void add_pieces(soft_t& a, const frag<T> (&f)[U]) {
  constexpr int E = EL<T>;
  float m = a.m;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, at(f[u], e));
  float s = a.s * exp_of(a.m - m), s1 = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      s += exp_of(at(f[u], e) - m);
      s1 += exp_of(at(f[u], e + 1) - m);
    }
  a = {m, s + s1};
}

// n elements at x for N threads, of which this one is number t.
template <int N, typename T>
__device__ __forceinline__ soft_t soft_of(const T* x, int32_t n, int32_t t) {
  constexpr int E = EL<T>, U = 4;
  soft_t a{LOWEST, 0.f};
  const int32_t whole = n / E;
  int32_t q = t;
  for (; q + (U - 1) * N < whole; q += U * N) {
    frag<T> f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) f[u] = load_frag(x + (int64_t)(q + u * N) * E);
    add_pieces<T, U>(a, f);
  }
  for (; q < whole; q += N) {
    const frag<T> f[1] = {load_frag(x + (int64_t)q * E)};
    add_pieces<T, 1>(a, f);
  }
  const int32_t i = whole * E + t;
  if (i < n) a = join(a, soft_t{fmaxf(elem<T>::to_f(x[i]), LOWEST),
                                exp_of(elem<T>::to_f(x[i]) - fmaxf(elem<T>::to_f(x[i]), LOWEST))});
  return a;
}

__device__ __forceinline__ void put_logp(soft_t a, float x, int32_t t, int64_t i,
                                         float* __restrict__ logp, float2* __restrict__ norm) {
  const float l = logf(a.s);
  // a row of -infinity only: nothing can be drawn
  const float lp = a.s == 0.f ? -__builtin_inff() : (x - a.m) - l;
  logp[i] = t == -1 ? 0.f : t == -2 ? __builtin_nanf("") : lp;
  norm[i] = make_float2(a.m, l);
}

// N threads for part c of row i; with one part a row it ends there.  Workgroups
// have 256 threads at least.
template <typename T, int N>
__global__ __launch_bounds__(N < 256 ? 256 : N) void k_logp(
    const T* __restrict__ x, int64_t ldx, int64_t Tn, int32_t V, ids_t ids, int32_t parts,
    int32_t each, float* __restrict__ logp, float2* __restrict__ norm, float2* __restrict__ part) {
  constexpr int ROWS = N < 256 ? 256 / N : 1;  // of a workgroup
  int64_t i = blockIdx.x / parts * (int64_t)ROWS + threadIdx.x / N;
  const bool mine = i < Tn;
  if (!mine) i = Tn - 1;  // the wave's other rows need its lanes
  const int32_t c = blockIdx.x % parts, t = threadIdx.x % N;
  const T* row = x + i * ldx;
  int32_t target = 0;
  float xt = 0.f;
  if (parts == 1 && t == 0) {
    target = ids.get(i, V);
    if (target >= 0) xt = elem<T>::to_f(row[target]);
  }
  soft_t a = lanes_join<(N < 64 ? N : 64)>(
      soft_of<N>(row + (int64_t)c * each, min(each, V - c * each), t));
  if constexpr (N > 64) {
    constexpr int W = N / 64;
    __shared__ soft_t lds[W];
    if (t % 64 == 0) lds[t / 64] = a;
    __syncthreads();
    if (t >= 64) return;
    a = lanes_join<64>(t < W ? lds[t] : soft_t{LOWEST, 0.f});
  }
  if (t != 0 || !mine) return;
  if (parts == 1) put_logp(a, xt, target, i, logp, norm);
  else part[blockIdx.x] = make_float2(a.m, a.s);
}

// A wave for each row.
template <typename T>
__global__ __launch_bounds__(64) void k_logp_join(const T* __restrict__ x, int64_t ldx, int32_t V,
                                                  ids_t ids, int32_t parts,
                                                  const float2* __restrict__ part,
                                                  float* __restrict__ logp,
                                                  float2* __restrict__ norm) {
  const int64_t i = blockIdx.x;
  const int32_t t = ids.get(i, V);
  const float xt = t >= 0 ? elem<T>::to_f(x[i * ldx + t]) : 0.f;
  soft_t a{LOWEST, 0.f};
  for (int32_t c = lane_id(); c < parts; c += 64) {
    const float2 p = part[i * parts + c];
    a = join(a, soft_t{p.x, p.y});
  }
  a = lanes_join<64>(a);
  if (lane_id() == 0) put_logp(a, xt, t, i, logp, norm);
}

// One piece of a row's gradient: lane's piece c, f its logits.
template <typename T>
__device__ __forceinline__ frag<T> grad_piece(const frag<T>& f, cut_t c, int32_t t, float g,
                                              float2 n) {
  constexpr int E = EL<T>;
  // or a row of -infinity only, but for NaN
  const bool zero = g == 0.f || (n.y == -__builtin_inff() && g == g);
  float v[E];
  floats_of(f, v);
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = exp_of((v[e] - n.x) - n.y);
  if ((uint32_t)(t - c.at) < (uint32_t)E) {  // one piece of the row
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] -= c.at + e == t ? 1.f : 0.f;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = zero ? 0.f : -g * v[e];
  return to_frag(v);
}
__device__ __forceinline__ float grad_of(int32_t t, const float* dlogp, int64_t i) {
  return t == -1 ? 0.f : t == -2 ? __builtin_nanf("") : dlogp[i];
}

// Workgroup (c, i): 256 U pieces of row i.  BIG: gradients that leave no room in the
// 256 MB cache before memory are stored past the caches, for the lines that plain
// stores leave there have to be written back while the next kernel reads (8,192 rows
// of 32,000: 203 us, 195 us past them).
constexpr int64_t BIG_BYTES = 128ll << 20;
template <typename T, bool BIG>
__global__ __launch_bounds__(256) void k_logp_grad(const T* x, int64_t ldx, int32_t V, ids_t ids,
                                                   const float* __restrict__ dlogp,
                                                   const float2* __restrict__ norm, T* dx,
                                                   int64_t lddx, uint32_t blocks) {
  constexpr int U = 4;
  const int64_t i = blockIdx.x / blocks;
  const int32_t first = (int32_t)(blockIdx.x % blocks) * (256 * U) + (int32_t)threadIdx.x;
  const int32_t per = (V + EL<T> - 1) / EL<T>, t = ids.get(i, V);
  const float g = grad_of(t, dlogp, i);
  const float2 n = norm[i];
  x += i * ldx;
  dx += i * lddx;
  frag<T> f[U] = {};
  if (g != 0.f) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      f[u] = load_cut(x, cut_of<T>(min(first + u * 256, per - 1), V), V);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (first + u * 256 >= per) break;
    const cut_t c = cut_of<T>(first + u * 256, V);
    const frag<T> o = grad_piece(f[u], c, t, g, n);
    if (BIG && c.from == 0) {  // rows of more than one piece
      typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
      __builtin_nontemporal_store(__builtin_bit_cast(u4, o), reinterpret_cast<u4*>(dx + c.at));
    } else {
      store_cut(dx, c, V, o);
    }
  }
}

// Short rows: a thread for each piece of all of them.
template <typename T>
__global__ __launch_bounds__(256) void k_logp_grad_short(const T* x, int64_t ldx, int64_t Tn,
                                                         int32_t V, ids_t ids,
                                                         const float* __restrict__ dlogp,
                                                         const float2* __restrict__ norm, T* dx,
                                                         int64_t lddx, uint32_t per) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  const int64_t i = at / per;
  if (i >= Tn) return;
  const cut_t c = cut_of<T>((int32_t)(at % per), V);
  const int32_t t = ids.get(i, V);
  const float g = grad_of(t, dlogp, i);
  frag<T> f{};
  if (g != 0.f) f = load_cut(x + i * ldx, c, V);
  store_cut(dx + i * lddx, c, V, grad_piece(f, c, t, g, norm[i]));
}

struct parts_t { int32_t parts, each; };

// Rows up to this many pieces are short: one wave reads them in four loads.
constexpr int32_t SHORT = 256;

// A workgroup takes 3 us and 1 us more for every 22,000 of its row's logits (their
// exponentials, four a cycle): rows of more than CUT are cut where there are few,
// although adding the parts is a launch more (5 rows of 128,000: 9.1 us whole, 6.1 us
// in parts; one of 32,000: 5.0 and 6.0 us; 100 of 128,000: 10.7 and 11.2 us).
constexpr int32_t CUT = 49152;
parts_t parts_of(snack_dtype dt, int64_t Tn, int32_t V) {
  const int32_t e = dt == SNACK_BF16 ? 8 : 4;
  int64_t parts = 1;
  if (V > CUT && Tn <= 64)
    parts = std::min<int64_t>(cdiv(512, std::max<int64_t>(Tn, 1)), V / 8192);
  const int64_t each = cdiv(cdiv(V, parts), 256 * e) * 256 * e;
  return {(int32_t)std::max<int64_t>(1, cdiv(V, each)), (int32_t)std::min<int64_t>(each, INT32_MAX)};
}

snack_status check_logp(snack_dtype dt, int32_t id_bytes, int64_t Tn, int32_t V, int64_t ld) {
  if (dt != SNACK_F32 && dt != SNACK_BF16) return SNACK_E_DTYPE;
  if (id_bytes != 4 && id_bytes != 8) return SNACK_E_DTYPE;
  if (Tn < 0 || V < 1 || ld < V) return SNACK_E_SHAPE;
  if (V > (1 << 30)) return SNACK_E_OVERFLOW;
  const int64_t e = dt == SNACK_BF16 ? 8 : 4;
  // workgroups of 256 threads: 2^24 in a launch
  if (Tn >= (1 << 24) / cdiv(V, 1024 * e)) return SNACK_E_OVERFLOW;
  return SNACK_OK;
}

template <typename T>
void run_fwd(const T* x, int64_t ldx, int64_t Tn, int32_t V, ids_t ids, float* logp, float2* norm,
             float2* part, parts_t p, hipStream_t s) {
  const int64_t pieces = cdiv(V, EL<T>);
  // Up to four pieces a thread (a wave for each of 16,384 rows of 300 logits: 9.3 us,
  // 16 lanes 5.5 us), and 16 waves where rows are few (one row of 32,000 logits: 5.2 us
  // with 4 waves, 5.0 us with 16; 64 rows 5.8 and 5.4 us; 900 rows 13.3 and 15.3 us).
  const int N = pieces <= SHORT / 4 ? 16 : pieces <= SHORT ? 64 : p.parts == 1 && Tn <= 128 ? 1024 : 256;
  auto kernel = N == 16 ? k_logp<T, 16> : N == 64 ? k_logp<T, 64> : N == 256 ? k_logp<T, 256>
                                                                            : k_logp<T, 1024>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(N < 256 ? cdiv(Tn * N, 256) : Tn * p.parts)),
                     dim3(std::max(N, 256)), 0, s, x, ldx, Tn, V, ids, p.parts, p.each, logp, norm,
                     part);
  if (p.parts > 1)
    hipLaunchKernelGGL(k_logp_join<T>, dim3((unsigned)Tn), dim3(64), 0, s, x, ldx, V, ids, p.parts,
                       part, logp, norm);
}

template <typename T>
void run_bwd(const T* x, int64_t ldx, int64_t Tn, int32_t V, ids_t ids, const float* dlogp,
             const float2* norm, T* dx, int64_t lddx, hipStream_t s) {
  const int64_t pieces = cdiv(V, EL<T>), blocks = cdiv(pieces, 1024);
  if (pieces <= 2 * SHORT && Tn * pieces <= MAX_PIECES) {
    hipLaunchKernelGGL(k_logp_grad_short<T>, dim3((unsigned)cdiv(Tn * pieces, 256)), dim3(256), 0, s,
                       x, ldx, Tn, V, ids, dlogp, norm, dx, lddx, (uint32_t)pieces);
  } else {
    const bool big = pieces > 1 && Tn * pieces * 16 > BIG_BYTES;
    auto kernel = big ? k_logp_grad<T, true> : k_logp_grad<T, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(Tn * blocks)), dim3(256), 0, s, x, ldx, V, ids,
                       dlogp, norm, dx, lddx, (uint32_t)blocks);
  }
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_logp_workspace(snack_dtype dtype, int64_t T, int32_t V, size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  if (snack_status st = check_logp(dtype, 4, T, V, V)) return st;
  const parts_t p = parts_of(dtype, T, V);
  *bytes = p.parts > 1 ? (size_t)T * p.parts * sizeof(float2) : 0;
  return SNACK_OK;
}

snack_status snack_logp_fwd(snack_dtype dtype, const void* X, int64_t ldx, int64_t T, int32_t V,
                            const void* targets, int32_t id_bytes, float* logp, float* norm,
                            void* ws, size_t ws_bytes, void* stream) {
  if (snack_status st = check_logp(dtype, id_bytes, T, V, ldx)) return st;
  if (T == 0) return SNACK_OK;
  if (!X || !targets || !logp || !norm) return SNACK_E_NULL;
  const parts_t p = parts_of(dtype, T, V);
  const size_t need = p.parts > 1 ? (size_t)T * p.parts * sizeof(float2) : 0;
  if (need > 0 && !ws) return SNACK_E_NULL;
  if (ws_bytes < need) return SNACK_E_WORKSPACE;
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4;
  const span_t out[] = {{logp, 4 * (__int128)T}, {norm, 8 * (__int128)T},
                        {ws, (__int128)need}};
  const span_t in[] = {{X, V * e, ldx * e, T}, {targets, (__int128)id_bytes * T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const ids_t ids{targets, id_bytes == 8};
  if (dtype == SNACK_BF16)
    run_fwd<bf16>((const bf16*)X, ldx, T, V, ids, logp, (float2*)norm, (float2*)ws, p, s);
  else
    run_fwd<float>((const float*)X, ldx, T, V, ids, logp, (float2*)norm, (float2*)ws, p, s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

snack_status snack_logp_bwd(snack_dtype dtype, const float* dlogp, const void* X, int64_t ldx,
                            int64_t T, int32_t V, const void* targets, int32_t id_bytes,
                            const float* norm, void* dX, int64_t lddx, void* stream) {
  if (snack_status st = check_logp(dtype, id_bytes, T, V, ldx)) return st;
  if (lddx < V) return SNACK_E_SHAPE;
  if (T == 0) return SNACK_OK;
  if (!dlogp || !X || !targets || !norm || !dX) return SNACK_E_NULL;
  if (dX == X && lddx != ldx && T > 1) return SNACK_E_SHAPE;
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4;
  const span_t out[] = {{dX, V * e, lddx * e, T}};
  const span_t in[] = {{dX == X ? nullptr : X, V * e, ldx * e, T},
                       {targets, (__int128)id_bytes * T}, {dlogp, 4 * (__int128)T},
                       {norm, 8 * (__int128)T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const ids_t ids{targets, id_bytes == 8};
  if (dtype == SNACK_BF16)
    run_bwd<bf16>((const bf16*)X, ldx, T, V, ids, dlogp, (const float2*)norm, (bf16*)dX, lddx, s);
  else
    run_bwd<float>((const float*)X, ldx, T, V, ids, dlogp, (const float2*)norm, (float*)dX, lddx,
                   s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
