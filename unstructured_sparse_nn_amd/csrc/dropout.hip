// dropout.hip -- dropout whose mask is never stored (gfx950).
//
// Element i of a call is dropped by 16 bits of a counter-based stream: field
// i mod 4 of output number i / 4 of a SplitMix64 generator (Steele, Lea &
// Flood, OOPSLA 2014) seeded with output number `step` of one seeded with
// `seed`, the same stream of streams that the restructuring draws from.  With
// n = round(p 2^16), fields below n drop; what stays is scaled by
// 2^16 / (2^16 - n), so that the scale is right for the probability that the
// fields really have.  Any thread can find any element's bits, so the backward
// pass is the same pass over the gradient.
//
// Bound by memory: x (and the residual) once, y once.  An output of the
// generator is two 64-bit products and serves four elements; with 32 bits an
// element it would serve two.  8,192 rows of 4,096 bf16 on a residual: 36.5 us
// (5.5 TB/s); into one output again and again 28.6 us, and 32.3 us where x has gaps
// between its rows (20.0 and 21.9 us without a residual).
#include "common.h"
#include "internal.h"
#include "pieces.h"
#include "prune_common.h"
#include "spans.h"

namespace snk {
namespace {

struct drop_arg {
  const void* x;
  const void* res;
  void* y;
  int64_t ldx, ldr, ldy;
  int64_t rows, cols;  // flat: one row,
  int64_t from;        // of which a launch takes the elements from here on
  uint64_t seed, step;
  const uint64_t* more;  // added to step, or NULL
  uint32_t level;        // of 2^16
  float scale;
};

// One piece: elements i0 to i0 + EL.
template <typename T>
__device__ __forceinline__ frag<T> drop_piece(const drop_arg& a, uint64_t stream, uint64_t i0,
                                              bool aligned, const frag<T>& x, const frag<T>& res,
                                              bool with_res) {
  constexpr int E = EL<T>, W = E / 4;
  uint64_t z[W];
  const uint64_t state = stream + ((i0 >> 2) + 1) * SM64_GAMMA;
#pragma unroll
  for (int w = 0; w < W; ++w) z[w] = sm64_mix(state + w * SM64_GAMMA);
  if (!aligned && (i0 & 3)) {
    const uint32_t sh = 16 * (uint32_t)(i0 & 3);
    const uint64_t next = sm64_mix(state + W * SM64_GAMMA);
#pragma unroll
    for (int w = 0; w < W; ++w) z[w] = (z[w] >> sh) | ((w + 1 < W ? z[w + 1] : next) << (64 - sh));
  }
  float v[E], r[E];
  floats_of(x, v);
  floats_of(res, r);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t u = (uint32_t)(z[e / 4] >> (16 * (e % 4))) & 0xFFFFu;
    const float kept = with_res ? fmaf(v[e], a.scale, r[e]) : v[e] * a.scale;
    v[e] = u < a.level ? (with_res ? r[e] : 0.f) : kept;
  }
  return to_frag(v);
}

__device__ __forceinline__ uint64_t stream_of(const drop_arg& a) {
  const uint64_t step = a.step + (a.more ? *a.more : 0);
  return sm64_mix(a.seed + (step + 1) * SM64_GAMMA);
}

// Rows without gaps are one row: U pieces a thread, loaded before any is used.
template <typename T, bool RES>
__global__ __launch_bounds__(256) void k_dropout_flat(drop_arg a) {
  constexpr int E = EL<T>, U = 2;
  const uint64_t stream = stream_of(a);
  const int64_t n = a.cols, block = a.from + (int64_t)blockIdx.x * (256 * U * E);
  const int64_t first = block + threadIdx.x * E;
  const T *x = (const T*)a.x + first, *res = (const T*)a.res + first;
  T* y = (T*)a.y + first;
  frag<T> f[U], r[U] = {};
  if (block + 256 * U * E <= n) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f[u] = load_frag(x + u * 256 * E);
      if (RES) r[u] = load_frag(res + u * 256 * E);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      store_frag(y + u * 256 * E,
                 drop_piece<T>(a, stream, (uint64_t)first + u * 256 * E, true, f[u], r[u], RES), E);
    return;
  }
#pragma unroll 1
  for (int u = 0; u < U; ++u) {
    const int64_t left = n - first - u * 256 * E;
    if (left <= 0) return;
    const int32_t have = (int32_t)min(left, (int64_t)E);
    const cut_t c{0, 0};
    f[0] = load_cut(x + u * 256 * E, c, have);
    if (RES) r[0] = load_cut(res + u * 256 * E, c, have);
    store_cut(y + u * 256 * E, c, have,
              drop_piece<T>(a, stream, (uint64_t)first + u * 256 * E, true, f[0], r[0], RES));
  }
}

template <typename T, bool RES>
__global__ __launch_bounds__(256) void k_dropout_rows(drop_arg a, uint32_t per) {
  const uint32_t g = blockIdx.x * 256u + threadIdx.x;
  const int64_t row = g / per;
  if (row >= a.rows) return;
  const int32_t n = (int32_t)a.cols;
  const cut_t c = cut_of<T>((int32_t)(g % per), n);
  const frag<T> f = load_cut((const T*)a.x + row * a.ldx, c, n);
  frag<T> r{};
  if (RES) r = load_cut((const T*)a.res + row * a.ldr, c, n);
  const uint64_t i0 = (uint64_t)row * (uint64_t)n + (uint64_t)c.at;
  store_cut((T*)a.y + row * a.ldy, c, n, drop_piece<T>(a, stream_of(a), i0, false, f, r, RES));
}

// Elements of a launch, which holds fewer than 2^32 threads.
constexpr int64_t LAUNCH = 1ll << 32;

template <typename T>
snack_status run(const drop_arg& a, hipStream_t s) {
  const bool flat = a.rows == 1 || (a.ldx == a.cols && a.ldy == a.cols &&
                                    (!a.res || a.ldr == a.cols));
  if (flat) {
    drop_arg f = a;
    f.cols = a.rows * a.cols;
    f.rows = 1;
    auto kernel = a.res ? k_dropout_flat<T, true> : k_dropout_flat<T, false>;
    for (f.from = 0; f.from < f.cols; f.from += LAUNCH) {
      const int64_t n = std::min(f.cols - f.from, LAUNCH);
      hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(n, 512 * EL<T>)), dim3(256), 0, s, f);
    }
  } else {
    const int64_t per = cdiv(a.cols, EL<T>);
    if (a.cols > INT32_MAX || per * a.rows > MAX_PIECES) return SNACK_E_OVERFLOW;
    auto kernel = a.res ? k_dropout_rows<T, true> : k_dropout_rows<T, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(per * a.rows, 256)), dim3(256), 0, s, a,
                       (uint32_t)per);
  }
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" snack_status snack_dropout(snack_dtype dtype, const void* X, int64_t ldx,
                                      const void* residual, int64_t ldr, void* Y, int64_t ldy,
                                      int64_t rows, int64_t cols, double p, uint64_t seed,
                                      uint64_t step, const uint64_t* step_dev, void* stream) {
  if (dtype != SNACK_F32 && dtype != SNACK_BF16) return SNACK_E_DTYPE;
  if (p != p) return SNACK_E_NAN;
  if (rows < 0 || cols < 0 || p < 0 || p > 1) return SNACK_E_SHAPE;
  if (ldx < cols || ldy < cols || (residual && ldr < cols)) return SNACK_E_SHAPE;
  if (rows == 0 || cols == 0) return SNACK_OK;
  if (rows > ((int64_t)1 << 36) / cols) return SNACK_E_OVERFLOW;
  if (!X || !Y) return SNACK_E_NULL;
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4;
  // element i of an output is written by the thread that has read element i
  const bool on_x = Y == X && (ldy == ldx || rows == 1),
             on_r = Y == residual && (ldy == ldr || rows == 1);
  const span_t out[] = {{Y, cols * e, ldy * e, rows}};
  const span_t in[] = {{on_x ? nullptr : X, cols * e, ldx * e, rows},
                       {on_r ? nullptr : residual, cols * e, ldr * e, rows},
                       {step_dev, 8}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  const uint32_t level = (uint32_t)(p * 65536.0 + 0.5);
  const drop_arg a{X, residual, Y, ldx, ldr, ldy, rows, cols, 0, seed, step, step_dev, level,
                   level < 65536 ? (float)(65536.0 / (65536 - level)) : 0.f};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == SNACK_BF16 ? run<bf16>(a, s) : run<float>(a, s);
}
