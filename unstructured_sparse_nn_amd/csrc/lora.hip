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
//
// A few tokens take k_lora_few, a workgroup's worth of dot products each.
// More tokens are cut into tiles of up to 32 of one adapter, which feed the
// matrix cores: reduce and expand of a tile in one kernel (k_lora_apply), the
// gradients in a second one (k_lora_grad), for dA needs all of u first.  That
// one reads x and dy: dy for the second time, x too where t was not kept.  Up
// to 8,192 tokens the workgroups find their tiles' tokens themselves; beyond,
// k_lora_route sorts them first.  The ranks are few, so all of it is bound by
// memory: x, base and y once each, beside factors that stay in the caches.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.h"
#include "internal.h"

namespace snk {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int32_t TILE = 32;  // tokens of a tile at most
constexpr int32_t MAX_RANK = 256;
constexpr int32_t MAX_ADAPTERS = 8192;
constexpr int32_t MAX_FEATURES = 1 << 23;  // columns stay far inside 32 bits
// A launch holds fewer than 2^32 threads along x: 2^23 workgroups of 512.
// k_lora_apply has one for each tile of 32 tokens, two in a backward, and up to
// one tile more for each adapter.
constexpr int32_t max_tokens(bool backward) {
  return backward ? (1 << 27) - (1 << 19) : (1 << 28) - (1 << 20);
}

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

// The wave's number in its workgroup, known to be the same for all lanes.
__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
}

// ------------------------------------------------------------- 16-byte pieces
// Rows start at any element, so pieces are loaded and stored without an
// alignment claim; the hardware takes a 16-byte access at any address.
template <typename T> constexpr int EL = 16 / sizeof(T);
template <typename T> struct __attribute__((aligned(16))) frag { uint32_t w[4]; };

__device__ __forceinline__ float at(const frag<bf16>& f, int e) {
  return __uint_as_float(e & 1 ? f.w[e / 2] & 0xFFFF0000u : f.w[e / 2] << 16);
}
__device__ __forceinline__ float at(const frag<float>& f, int e) { return __uint_as_float(f.w[e]); }

template <typename T>
__device__ __forceinline__ frag<T> load_frag(const T* p) {
  frag<T> f;
  __builtin_memcpy(&f, p, 16);
  return f;
}
__device__ __forceinline__ uint32_t pick(bool first, uint32_t a, uint32_t b) { return first ? a : b; }

// f moved down by sh elements, zeros behind.
__device__ __forceinline__ frag<bf16> move_down(const frag<bf16>& f, int32_t sh) {
  const uint32_t a0 = pick(sh & 1, __builtin_amdgcn_alignbit(f.w[1], f.w[0], 16), f.w[0]),
                 a1 = pick(sh & 1, __builtin_amdgcn_alignbit(f.w[2], f.w[1], 16), f.w[1]),
                 a2 = pick(sh & 1, __builtin_amdgcn_alignbit(f.w[3], f.w[2], 16), f.w[2]),
                 a3 = pick(sh & 1, f.w[3] >> 16, f.w[3]);
  const uint32_t b0 = pick(sh & 2, a1, a0), b1 = pick(sh & 2, a2, a1), b2 = pick(sh & 2, a3, a2),
                 b3 = pick(sh & 2, 0, a3);
  const bool none = sh >= 8;
  return frag<bf16>{{pick(none, 0, pick(sh & 4, b2, b0)), pick(none, 0, pick(sh & 4, b3, b1)),
                     pick(none || (sh & 4), 0, b2), pick(none || (sh & 4), 0, b3)}};
}
__device__ __forceinline__ frag<float> move_down(const frag<float>& f, int32_t sh) {
  const uint32_t b0 = pick(sh & 1, f.w[1], f.w[0]), b1 = pick(sh & 1, f.w[2], f.w[1]),
                 b2 = pick(sh & 1, f.w[3], f.w[2]), b3 = pick(sh & 1, 0, f.w[3]);
  const bool none = sh >= 4;
  return frag<float>{{pick(none, 0, pick(sh & 2, b2, b0)), pick(none, 0, pick(sh & 2, b3, b1)),
                      pick(none || (sh & 2), 0, b2), pick(none || (sh & 2), 0, b3)}};
}
// The piece at p of a row of EL elements or more, of which n are left there (n
// may be <= 0), zeros after them.  One load: a piece that ends early is taken
// from the row's last EL elements.
template <typename T>
__device__ __forceinline__ frag<T> load_end(const T* p, int32_t n) {
  const int32_t sh = max(EL<T> - n, 0);
  return move_down(load_frag(p - sh), sh);
}
// The same for a row of `row` elements, which may be fewer.
template <typename T>
__device__ __forceinline__ frag<T> load_frag(const T* p, int32_t n, int64_t row) {
  if (row >= EL<T>) return load_end(p, n);
  frag<T> f{};
#pragma unroll 1
  for (int e = (int)row - 1; e >= 0; --e) {  // the row is shorter than a piece: p is its start
    uint32_t v = 0;
    if (e < n) __builtin_memcpy(&v, p + e, sizeof(T));
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e * (int)sizeof(T) / 4 == q) f.w[q] |= v << (8 * (e * sizeof(T) % 4));
  }
  return f;
}
template <typename T>
__device__ __forceinline__ void store_frag(T* p, const frag<T>& f, int32_t n) {
  if (n >= EL<T>) {
    __builtin_memcpy(p, &f, 16);
  } else {
#pragma unroll
    for (int e = 0; e < EL<T> - 1; ++e)
      if (e < n) {
        const uint32_t v = f.w[e * sizeof(T) / 4] >> (8 * (e * sizeof(T) % 4));
        __builtin_memcpy(p + e, &v, sizeof(T));
      }
  }
}
// Pieces of E elements, loaded and stored likewise.
template <typename T, int E> struct piece { uint32_t w[E * sizeof(T) / 4]; };
template <typename T, int E>
__device__ __forceinline__ uint32_t bits_at(const piece<T, E>& f, int e) {
  return sizeof(T) == 4 ? f.w[e] : f.w[e / 2] >> (16 * (e & 1));
}
template <typename T, int E>
__device__ __forceinline__ float at(const piece<T, E>& f, int e) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(f.w[e]);
  else return __uint_as_float(e & 1 ? f.w[e / 2] & 0xFFFF0000u : f.w[e / 2] << 16);
}
template <typename T, int E>  // the first n elements at p, zeros after them
__device__ __forceinline__ piece<T, E> load_piece(const T* p, int32_t n) {
  piece<T, E> f{};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    uint32_t v = 0;
    if (e < n) __builtin_memcpy(&v, p + e, sizeof(T));
    f.w[e * sizeof(T) / 4] |= v << (8 * (e * sizeof(T) % 4));
  }
  return f;
}
template <typename T, int E>  // elements from `from` up to `to`
__device__ __forceinline__ void store_piece(T* p, const piece<T, E>& f, int32_t from, int32_t to) {
  if (from <= 0 && to >= E) {
    __builtin_memcpy(p, &f, sizeof(f));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e >= from && e < to) {
        const uint32_t v = bits_at(f, e);
        __builtin_memcpy(p + e, &v, sizeof(T));
      }
  }
}

// f, or zeros.
template <typename T>
__device__ __forceinline__ frag<T> keep_if(bool keep, const frag<T>& f) {
  frag<T> o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o.w[q] = keep ? f.w[q] : 0u;
  return o;
}

__device__ __forceinline__ f4 mma(const frag<bf16>& a, const frag<bf16>& b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                 __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// The four elements of a float piece are four steps of the 16x16x4 product:
// the order of the contraction is free as long as both sides share it.
__device__ __forceinline__ f4 mma(const frag<float>& a, const frag<float>& b, f4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(at(a, e), at(b, e), c, 0, 0, 0);
  return c;
}

// Two floats as bf16, rounded to nearest even, in one dword.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
}
__device__ __forceinline__ frag<bf16> to_frag(const float (&v)[8]) {
  return frag<bf16>{{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                     bf16_pair(v[6], v[7])}};
}
__device__ __forceinline__ frag<float> to_frag(const float (&v)[4]) {
  return frag<float>{{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3])}};
}

template <int E>
__device__ __forceinline__ void round_to(const float (&v)[E], piece<bf16, E>& o) {
#pragma unroll
  for (int e = 0; e < E; e += 2) o.w[e / 2] = bf16_pair(v[e], v[e + 1]);
}
template <int E>
__device__ __forceinline__ void round_to(const float (&v)[E], piece<float, E>& o) {
#pragma unroll
  for (int e = 0; e < E; ++e) o.w[e] = __float_as_uint(v[e]);
}

// v as two bf16 parts, hi + lo: off by at most 2^-16 of v, a 256th of the
// rounding of what comes of it (bf16's half step, 2^-8), for two products of
// the matrix cores where fp32's 24 bits would take three.  hi is at most the
// largest bf16, which larger floats would round past.  Infinities and NaN are
// hi alone.
__device__ __forceinline__ void split_frag(const float (&v)[8], frag<bf16>& hi, frag<bf16>& lo) {
  hi = to_frag(v);
  float peak = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) peak = fmaxf(peak, fabsf(v[e]));
  if (peak >= __uint_as_float(0x7F7F8000u)) {  // rounds past the largest bf16, or infinite
    const float most = __uint_as_float(0x7F7F0000u);
    float top[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      top[e] = fabsf(v[e]) < __builtin_inff() ? fminf(fmaxf(v[e], -most), most) : v[e];
    hi = to_frag(top);
  }
  float rest[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float h = at(hi, e);
    rest[e] = fabsf(h) < __builtin_inff() ? v[e] - h : 0.f;
  }
  lo = to_frag(rest);
}

// An infinity times hi is right, but times lo it is a NaN where lo is zero or
// of the other sign: the products with lo take zeros for infinities.  Whether a
// wave's operands hold one at all, their sums tell (the matrix cores have time:
// a forward of 8,192 tokens at 4096x4096 takes 45.2 us, 48.5 us with magnitudes
// compared), or, in the gradients, their largest magnitude.
template <int E>
__device__ __forceinline__ bool any_infinite(const frag<bf16> (&v)[E]) {  // or a huge sum, or NaN
  const frag<bf16> one{{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};
  f4 sum[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e & 1] = mma(one, v[e], sum[e & 1]);
  return __any(!(fabsf(sum[0][0] + sum[1][0]) < __builtin_inff()));
}
struct peak_t {
  typedef uint16_t u2 __attribute__((ext_vector_type(2)));
  u2 m = {0, 0};
  __device__ __forceinline__ void add(uint32_t w) {
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u2, w & 0x7FFF7FFFu));
  }
  __device__ __forceinline__ bool infinite() const {  // for the whole wave; NaN counts too
    return __any(m[0] >= 0x7F80u || m[1] >= 0x7F80u);
  }
};
__device__ __forceinline__ uint32_t without_infinities(uint32_t w) {
  if ((w & 0x7FFFu) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7FFF0000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}
template <int E>
__device__ __forceinline__ void drop_infinities(frag<bf16> (&v)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[e].w[k] = without_infinities(v[e].w[k]);
}

// --------------------------------------------------------------- a few tokens
// A workgroup has one token and nb blocks of 64 pieces of columns at a time.
// Its sixteen waves share the ranks of t (each workgroup of the token computes
// all of t again: the factor comes from the caches).  Then 16 / nb waves share
// the ranks of a block's expansion, whose parts meet in LDS.  What the
// expansion reads first is loaded before t, so one trip to memory covers both.
// K and M hold a piece at least.  One token of rank 16, 4096 to 4096: 6.1 us, all
// of it launch and trips to memory one after the other (ids, factor, factor);
// 37 tokens of ranks 8 to 32, 4096 to 11008: 10.5 us for 23 MB, 2.2 TB/s.
constexpr int FEW_WAVES = 16;

template <typename T>
__device__ __forceinline__ float dot_frag(const frag<T>& a, const frag<T>& b, float acc) {
  vec<T, EL<T>> x, y;
  __builtin_memcpy(&x, &a, 16);
  __builtin_memcpy(&y, &b, 16);
  return dot_acc<T, EL<T>>(x, y, acc);
}

// out[q * FEW_WAVES] = sum_k F[q * FEW_WAVES, k] x[k] for RW rows, by one wave.
template <typename T, int RW>
__device__ __forceinline__ void few_dots(const T* x, const T* __restrict__ F, int32_t K, float* out) {
  constexpr int E = EL<T>, U = RW == 1 ? 8 : 8 / RW;
  const int l = lane_id();
  const int64_t next = (int64_t)FEW_WAVES * K;
  float acc[RW] = {};
  int32_t k = l * E;
  for (; k + (U - 1) * 64 * E + E <= K; k += U * 64 * E) {
    frag<T> xv[U], fv[U][RW];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xv[u] = load_frag(x + k + u * 64 * E);
#pragma unroll
      for (int q = 0; q < RW; ++q) fv[u][q] = load_frag(F + q * next + k + u * 64 * E);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < RW; ++q) acc[q] = dot_frag(xv[u], fv[u][q], acc[q]);
  }
  for (; k + E <= K; k += 64 * E) {
    const frag<T> xv = load_frag(x + k);
#pragma unroll
    for (int q = 0; q < RW; ++q) acc[q] = dot_frag(xv, load_frag(F + q * next + k), acc[q]);
  }
  if (k < K) {
    const frag<T> xv = load_end(x + k, K - k);
#pragma unroll
    for (int q = 0; q < RW; ++q) acc[q] = dot_frag(xv, load_end(F + q * next + k, K - k), acc[q]);
  }
#pragma unroll
  for (int q = 0; q < RW; ++q) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) acc[q] += __shfl_xor(acc[q], m, 64);
    if (l == 0) out[q * FEW_WAVES] = acc[q];
  }
}

template <typename T>
__global__ __launch_bounds__(FEW_WAVES * 64) void k_lora_few(
    lora_dev d, const int32_t* __restrict__ ids, int32_t Tn, int32_t split, int32_t log_nb,
    const T* __restrict__ A, int32_t K, const T* X, int64_t ldx, const T* __restrict__ B, int32_t M,
    const T* base, int64_t ldb, T* Y, int64_t ldy, float* t) {
  constexpr int E = EL<T>, C = 64 * E, AHEAD = 2;
  __shared__ float ts[MAX_RANK];
  __shared__ float red[FEW_WAVES][C];
  // From 8 tokens on a token's workgroups share a die, whose L2 then holds
  // the token's factor once.
  int32_t i = blockIdx.x / split, share = blockIdx.x % split;
  if (Tn >= NUM_XCD) {
    const int32_t at = blockIdx.x / NUM_XCD;
    i = at / split * NUM_XCD + blockIdx.x % NUM_XCD;
    share = at % split;
  }
  if (i >= Tn) return;
  const int32_t a = ids[i];
  const int w = wave_id(), l = lane_id();
  const int32_t r = a >= 0 && a < d.L ? rank_of(d, a) : 0;
  const float s = a >= d.L ? __builtin_nanf("") : r > 0 ? scale_of(d, a) : 1.f;
  const int64_t row0 = r > 0 ? (int64_t)a * d.R : 0;
  const int32_t nb = 1 << log_nb;
  const int32_t groups = FEW_WAVES >> log_nb, j0 = w >> log_nb;  // of the expansion's ranks
  int32_t col0 = share * nb * C;                       // the workgroup's first column
  // A piece that would end past M is the row's last one; what lies before the
  // lane's column is not stored.
  auto column = [&]() { return min(col0 + (w & (nb - 1)) * C + l * E, M - E); };
  frag<T> ahead[AHEAD], base0{};
  auto load_ahead = [&]() {
    const int32_t col = column();
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
      if (j0 + q * groups < r) ahead[q] = load_frag(B + (row0 + j0 + q * groups) * M + col);
    if (base && w < nb) base0 = load_frag(base + i * ldb + col);
  };
  load_ahead();
  const T* x = X + i * ldx;
  for (int32_t j = w; j < r;) {
    const T* F = A + (row0 + j) * K;
    if (j + 3 * FEW_WAVES < r) {
      few_dots<T, 4>(x, F, K, ts + j);
      j += 4 * FEW_WAVES;
    } else if (j + FEW_WAVES < r) {
      few_dots<T, 2>(x, F, K, ts + j);
      j += 2 * FEW_WAVES;
    } else {
      few_dots<T, 1>(x, F, K, ts + j);
      j += FEW_WAVES;
    }
  }
  __syncthreads();
  if (t && share == 0 && (int32_t)threadIdx.x < d.R)
    t[(int64_t)i * d.R + threadIdx.x] = (int32_t)threadIdx.x < r ? ts[threadIdx.x] : 0.f;
  while (true) {
    const int32_t col = column();
    float y[E] = {};
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
      if (j0 + q * groups < r) {
        const float tv = ts[j0 + q * groups];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = fmaf(tv, at(ahead[q], e), y[e]);
      }
#pragma unroll 4
    for (int32_t j = j0 + AHEAD * groups; j < r; j += groups) {
      const frag<T> bv = load_frag(B + (row0 + j) * M + col);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = fmaf(ts[j], at(bv, e), y[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) red[w][l * E + e] = y[e];
    __syncthreads();
    if (w < nb) {
      float v[E] = {};
      for (int32_t q = 0; q < groups; ++q)
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += red[q * nb + w][l * E + e];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] *= s;
        if (base) v[e] += at(base0, e);
      }
      piece<T, E> o;
      round_to(v, o);
      store_piece(Y + i * ldy + col, o, col0 + w * C + l * E - col, M - col);
    }
    col0 += split * nb * C;
    if (col0 >= M) break;
    load_ahead();
    __syncthreads();
  }
}

// ------------------------------------------------------- tokens in adapter order
// A tile is a run of up to `size` (16 or 32) tokens of one adapter in that
// order, which gives tile i the places from i * size on; group L holds the
// tokens without an adapter.  A slot is a run of tiles
// of one adapter whose gradient is summed in one go; the slots of an adapter
// that has several leave partial sums at `part`, part + 1, ...; an adapter
// without tokens has one slot of no tiles.
struct tile_t { int32_t l, begin, n, pad; };
struct slot_t { int32_t l, tile, n, part; };  // part < 0: the adapter's only slot
struct join_t { int32_t slots, part; };

struct route_t {
  const int32_t* ids;
  int32_t Tn;
  int32_t size;            // tokens of a tile at most
  int32_t slot_tiles;      // tiles of a slot
  const int32_t* order;    // NULL: one adapter, tokens in their own order
  const tile_t* tile;
  const slot_t* slot;
  const join_t* join;      // [L]
  const int32_t* count;    // tiles, slots
};

__device__ __forceinline__ int32_t tiles_of(const route_t& p) {
  return p.order ? p.count[0] : (p.Tn + p.size - 1) / p.size;
}
__device__ __forceinline__ tile_t tile_at(const route_t& p, int32_t i) {
  if (p.order) return p.tile[i];
  return tile_t{0, i * p.size, min(p.size, p.Tn - i * p.size), 0};
}
__device__ __forceinline__ slot_t slot_at(const route_t& p, int32_t i) {
  if (p.order) return i < p.count[1] ? p.slot[i] : slot_t{0, 0, -1, 0};
  const int32_t tiles = (p.Tn + p.size - 1) / p.size;
  return slot_t{0, i * p.slot_tiles, min(p.slot_tiles, tiles - i * p.slot_tiles),
                tiles > p.slot_tiles ? i : -1};
}
__device__ __forceinline__ int32_t row_at(const route_t& p, int32_t i) {
  return p.order ? p.order[i] : i;
}

// Exclusive prefixes over a block of 1024 of four values per thread; total
// receives the sums.  Contains barriers.
struct four_t { int32_t v[4]; };
__device__ __forceinline__ four_t scan_four(four_t x, four_t* lds, four_t& total) {
  const int w = wave_id();
  four_t inc, out;
#pragma unroll
  for (int q = 0; q < 4; ++q) inc.v[q] = wave_incl_scan_i32(x.v[q]);
  __syncthreads();
  if (lane_id() == 63) lds[w] = inc;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) total.v[q] = 0, out.v[q] = inc.v[q] - x.v[q];
#pragma unroll 2
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int32_t t = lds[i].v[q];
      if (i < w) out.v[q] += t;
      total.v[q] += t;
    }
  return out;
}

// Stable counting sort of the tokens by adapter, then the tables of tiles and
// slots, in one workgroup: wave w < nw walks its own run of tokens, once to
// count and once to place, where lanes that hold the same adapter find each
// other by one ballot per bit.  A walk loads RUN x 64 ids before it uses the
// first.  Bound by the second walk, a chain of LDS updates: 54 us for 65,536
// tokens of 16 adapters (73 us with the first walk like it).
__global__ __launch_bounds__(1024) void k_lora_route(const int32_t* __restrict__ ids, int32_t Tn,
                                                     int32_t L, int32_t nw, int32_t size,
                                                     int32_t slot_tiles,
                                                     int32_t* __restrict__ order,
                                                     tile_t* __restrict__ tile,
                                                     slot_t* __restrict__ slot,
                                                     join_t* __restrict__ join,
                                                     int32_t* __restrict__ count) {
  extern __shared__ int32_t cnt[];  // [nw][G], then first token and first tile of the groups
  __shared__ four_t lds[16];
  constexpr int RUN = 8;
  const int32_t G = L + 1;
  const int w = wave_id(), l = lane_id();
  int32_t *first = cnt + nw * G, *first_tile = first + G + 1;
  for (int32_t i = threadIdx.x; i < nw * G; i += 1024) cnt[i] = 0;
  __syncthreads();
  const int32_t run = ((Tn + nw - 1) / nw + 63) / 64 * 64;
  const int64_t i0 = (int64_t)w * run, i1 = min(i0 + run, (int64_t)Tn);
  const int bits = 32 - __builtin_clz(L);
  auto walk = [&](bool place) {
    if (w >= nw) return;
    int32_t* mine = cnt + w * G;
    for (int64_t b0 = i0; b0 < i1; b0 += 64 * RUN) {
      int32_t id[RUN];
#pragma unroll
      for (int q = 0; q < RUN; ++q) id[q] = ids[min(b0 + q * 64 + l, i1 - 1)];
#pragma unroll
      for (int q = 0; q < RUN; ++q) {
        const int64_t b = b0 + q * 64;
        if (b >= i1) break;
        const bool in = b + l < i1;
        const int32_t g = id[q] >= 0 && id[q] < L ? id[q] : L;
        if (!place) {  // whole numbers: the order of the additions does not matter
          const int32_t same = __builtin_amdgcn_readfirstlane(g);
          if (__all(in && g == same)) {
            if (l == 0) atomicAdd(&mine[same], 64);
          } else if (in) {
            atomicAdd(&mine[g], 1);
          }
          continue;
        }
        uint64_t peers = __ballot(in);
        for (int k = 0; k < bits; ++k) {
          const uint64_t m = __ballot((g >> k) & 1);
          peers &= ((g >> k) & 1) ? m : ~m;
        }
        const int before = __popcll(peers & lanemask_lt());
        int32_t at = 0;
        if (in) at = mine[g] + before;
        if (in) order[at] = (int32_t)(b + l);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in && before == 0) mine[g] = at + __popcll(peers);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
  };
  walk(false);
  __syncthreads();
  four_t sum{};  // tokens, tiles, slots and partial sums of the groups so far
  for (int32_t g0 = 0; g0 < G; g0 += 1024) {
    const int32_t g = g0 + threadIdx.x;
    int32_t n = 0;
    if (g < G)
      for (int32_t q = 0; q < nw; ++q) n += cnt[q * G + g];
    const int32_t nt = (n + size - 1) / size;
    const int32_t ns = g < L ? max(1, (nt + slot_tiles - 1) / slot_tiles) : 0;
    four_t total;
    four_t b = scan_four(four_t{{n, nt, ns, ns > 1 ? ns : 0}}, lds, total);
#pragma unroll
    for (int q = 0; q < 4; ++q) b.v[q] += sum.v[q], sum.v[q] += total.v[q];
    if (g < G) {
      first[g] = b.v[0];
      first_tile[g] = b.v[1];
      for (int32_t k = 0; k < ns; ++k)
        slot[b.v[2] + k] = slot_t{g, b.v[1] + k * slot_tiles,
                                  min(slot_tiles, nt - k * slot_tiles), ns > 1 ? b.v[3] + k : -1};
      if (g < L) join[g] = join_t{ns, b.v[3]};
      int32_t at = b.v[1] * size;
      for (int32_t q = 0; q < nw; ++q) {
        const int32_t c = cnt[q * G + g];
        cnt[q * G + g] = at;
        at += c;
      }
    }
  }
  if (threadIdx.x == 0) {
    count[0] = sum.v[1];
    count[1] = sum.v[2];
    first[G] = Tn;
  }
  __syncthreads();
  walk(true);
  for (int32_t i = threadIdx.x; i < sum.v[1]; i += 1024) {
    int32_t lo = 0, hi = G;  // the last group whose first tile is <= i
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) / 2;
      if (first_tile[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int32_t at = first[lo] + (i - first_tile[lo]) * size;
    tile[i] = tile_t{lo, i * size, min(size, first[lo + 1] - at), 0};
  }
}

// ------------------------------------------------------------- tiles of tokens
// One workgroup takes a tile through both products.  t of the tile: every wave
// sums its own range of k for all tokens and ranks, and the waves' sums meet
// in LDS.  Then every wave expands t over its own columns.  t never leaves the
// chip, and one launch's x streams while another workgroup's y does.  Forward
// of 8,192 tokens of rank 16 at 4096x4096: 45.2 us for 202 MB, 4.5 TB/s (a copy
// of 1 GiB: 4.8 TB/s).  With the inputs in the memory-side cache 36.2 us, and
// 40.6 us as a reduction and an expansion in two launches.
constexpr int WAVES = 8;
enum { ROW_NONE = 0, ROW_HAS = 1, ROW_BAD = 2 };

template <typename T>
struct reduce_arg {  // t[i, j] = sum_k F[a, j, k] X[i, k]
  const T* F;
  const T* X;
  int64_t ldx;
  int32_t K;
  const float* given;  // t, if it is there already, as `parts` sums to be added
  int32_t parts;
  float* t;            // nullable: where t goes
  void* pack;          // nullable: where t goes as the gradient's operand
};
template <typename T>
struct expand_arg {  // Y[i, m] = base[i, m] + s sum_j t[i, j] F[a, j, m]
  const T* F;
  int32_t M;
  const T* base;
  int64_t ldb;
  T* Y;
  int64_t ldy;
};

struct tile_lds {
  int32_t row[TILE];
  int8_t kind[TILE];
};

// Which tile and role a workgroup has.  From 64 tiles on each die takes a run
// of tiles, so that an adapter's factors fill few L2s.
__device__ __forceinline__ bool place_of(int32_t tiles, int32_t roles, int32_t& ti, int32_t& role) {
  ti = blockIdx.x / roles;
  role = blockIdx.x % roles;
  if (tiles >= 64) {
    const int32_t each = (tiles + NUM_XCD - 1) / NUM_XCD, at = blockIdx.x / NUM_XCD / roles;
    role = blockIdx.x / NUM_XCD % roles;
    ti = at < each ? blockIdx.x % NUM_XCD * each + at : tiles;
  }
  return ti < tiles;
}

// Up to SELF_TOKENS tokens and SELF_GROUPS - 1 adapters, every workgroup finds
// the tokens of its tile itself: it counts the groups in LDS (whole numbers:
// the order of the additions does not matter), finds its tile's group and
// collects that group's tokens.  Against k_lora_route before (rank 16, bf16, 4096
// to 4096; 2 to 500 adapters measured at 300 to 8,192 tokens), of 12 adapters: a
// forward of 1,024 tokens 19.1 us and 23.3 us, of 4,099 37.6 and 43.0, of 8,192
// 71.5 and 76.7; a backward of 4,099 76.9 and 79.4 us, of 6,001 81.1 and 80.3, of
// 8,192 125.6 and 129.2.  SELF_BYTES: LDS that it takes.
constexpr int32_t SELF_TOKENS = 8192, SELF_GROUPS = 1024;
constexpr size_t SELF_BYTES = 4 * (SELF_GROUPS + WAVES + 4 + WAVES);

struct tables_t {  // what the gradients need of it; all NULL: nothing
  int32_t* order;  // tile i's tokens from i * size on
  tile_t* tile;
  slot_t* slot;
  join_t* join;
  int32_t* count;
};

__device__ __forceinline__ bool self_route(const lora_dev& d, const route_t& p, const tables_t& out,
                                           int32_t roles, char* lds, tile_lds& tk, int32_t& ti,
                                           int32_t& role, tile_t& tl) {
  constexpr int Q = SELF_TOKENS / (WAVES * 64);
  int32_t* cnt = reinterpret_cast<int32_t*>(lds);
  int32_t *scan = cnt + SELF_GROUPS, *found = scan + WAVES, *matches = found + 4;
  const int32_t G = d.L + 1;
  const int w = wave_id(), l = lane_id(), t = threadIdx.x;
  const int32_t chunks = (p.Tn + WAVES * 64 - 1) / (WAVES * 64), i0 = w * chunks * 64 + l;
  int32_t id[Q];  // then the token's group, -1 past the last token
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (q < chunks) id[q] = p.ids[min(i0 + q * 64, p.Tn - 1)];
  for (int32_t g = t; g < G; g += WAVES * 64) cnt[g] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (q >= chunks) break;
    id[q] = i0 + q * 64 >= p.Tn ? -1 : id[q] >= 0 && id[q] < d.L ? id[q] : d.L;
    const int32_t same = __builtin_amdgcn_readfirstlane(id[q]);
    if (__all(id[q] == same)) {
      if (l == 0 && same >= 0) atomicAdd(&cnt[same], 64);
    } else if (id[q] >= 0) {
      atomicAdd(&cnt[id[q]], 1);
    }
  }
  __syncthreads();
  int32_t n[2], nt[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    n[h] = 2 * t + h < G ? cnt[2 * t + h] : 0;
    nt[h] = (n[h] + p.size - 1) / p.size;
  }
  int32_t tiles;
  const int32_t before = block_excl_scan_i32<WAVES * 64>(nt[0] + nt[1], scan, &tiles);
  if (!place_of(tiles, roles, ti, role)) return false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int32_t k = ti - before - h * nt[0];
    if (k >= 0 && k < nt[h]) found[0] = 2 * t + h, found[1] = k, found[2] = n[h];
  }
  if (out.order && ti == 0 && role == 0) {
    int32_t ns[2], at = before, slots, parts;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      ns[h] = 2 * t + h < d.L ? max(1, (nt[h] + p.slot_tiles - 1) / p.slot_tiles) : 0;
    const int32_t np[2] = {ns[0] > 1 ? ns[0] : 0, ns[1] > 1 ? ns[1] : 0};
    int32_t bs = block_excl_scan_i32<WAVES * 64>(ns[0] + ns[1], scan, &slots);
    int32_t bp = block_excl_scan_i32<WAVES * 64>(np[0] + np[1], scan, &parts);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * t + h < d.L) out.join[2 * t + h] = join_t{ns[h], bp};
      for (int32_t k = 0; k < ns[h]; ++k)
        out.slot[bs + k] = slot_t{2 * t + h, at + k * p.slot_tiles,
                                  min(p.slot_tiles, nt[h] - k * p.slot_tiles),
                                  ns[h] > 1 ? bp + k : -1};
      bs += ns[h];
      bp += np[h];
      at += nt[h];
    }
    if (t == 0) out.count[0] = tiles, out.count[1] = slots;
  }
  __syncthreads();
  const int32_t g = found[0], k = found[1];
  tl = tile_t{g, ti * p.size, min(p.size, found[2] - k * p.size), 0};
  int32_t m = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (q >= chunks) break;
    m += __popcll(__ballot(id[q] == g));
  }
  if (l == 0) matches[w] = m;
  __syncthreads();
  int32_t at = -k * p.size;
  for (int q = 0; q < w; ++q) at += matches[q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (q >= chunks) break;
    const uint64_t mine = __ballot(id[q] == g);
    const int32_t to = at + __popcll(mine & lanemask_lt());
    if (id[q] == g && to >= 0 && to < p.size) tk.row[to] = i0 + q * 64;
    at += __popcll(mine);
  }
  __syncthreads();
  if (out.order && role == 0) {
    if (t < p.size) out.order[ti * p.size + t] = tk.row[min(t, tl.n - 1)];
    if (t == 0) out.tile[ti] = tl;
  }
  return true;
}

// ts[token][rank < r] = t, 0 for tokens without the adapter; ld: ts's stride.
// Of `parts` equal ranges of k, only range `part` is summed.
// A wave brings 128 bytes of each row at a time: eight lanes a row, so that a
// load touches 8 lines (16 rows of 64 bytes, as the products take them, would
// cost a look-up in the cache for every lane: 52.2 us instead of 45.7 us for
// 8,192 tokens of rank 16, and 165 us instead of 109 us for 6,001 tokens of
// ranks 16 to 64).  LDS of its own turns them into operands; row i's piece s lies at slot s ^ (i & 7), which spreads both the
// writes and the reads over all banks.
template <typename T, int RT, int NR>
__device__ __forceinline__ void reduce_tile(const lora_dev& d, const reduce_arg<T>& q,
                                            const tile_t& tl, int32_t r, const tile_lds& tk,
                                            char* lds, float* ts, int32_t ld, int32_t part,
                                            int32_t parts) {
  constexpr int E = EL<T>, KS = 8 * E;       // contraction of a step
  constexpr int NI = 2 * (RT + NR);          // loads of a step
  constexpr int D = NI <= 4 ? 4 : NI == 8 ? 1 : 2;  // steps whose loads are under way
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int row8 = l >> 3, slot = l & 7;
  frag<T>* mine = reinterpret_cast<frag<T>*>(lds) + w * (NI * 64);
  frag<T>* put = mine + row8 * 8 + (slot ^ row8);
  const frag<T>* get = mine + c * 8;
  const int32_t steps = (q.K + KS - 1) / KS;
  const int64_t at0 = (int64_t)part * WAVES + w, of = (int64_t)parts * WAVES;
  const int32_t s0 = (int32_t)(steps * at0 / of), s1 = (int32_t)(steps * (at0 + 1) / of);
  const int32_t full = min(s1, q.K / KS);
  for (int32_t rb = 0; rb < r; rb += 16 * NR) {
    const T* src[NI];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i)
      src[i] = q.X + (int64_t)tk.row[i * 8 + row8] * q.ldx + slot * E + s0 * KS;
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i)  // rows past the rank: results not used
      src[2 * RT + i] =
          q.F + ((int64_t)tl.l * d.R + min(rb + i * 8 + row8, r - 1)) * q.K + slot * E + s0 * KS;
    f4 acc[RT][NR];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
    auto turn = [&](const frag<T> (&v)[NI]) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < NI; ++i) put[i * 64] = v[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        frag<T> xv[RT], fv[NR];
        const int at = (h * 4 + g) ^ (c & 7);
#pragma unroll
        for (int i = 0; i < RT; ++i) xv[i] = get[i * 128 + at];
#pragma unroll
        for (int j = 0; j < NR; ++j) fv[j] = get[(RT + j) * 128 + at];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < NR; ++j) acc[i][j] = mma(xv[i], fv[j], acc[i][j]);
      }
    };
    frag<T> v[D][NI];
    auto load = [&](int u) {  // the next step
#pragma unroll
      for (int i = 0; i < NI; ++i) v[u][i] = load_frag(src[i]), src[i] += KS;
    };
    int32_t s = s0;
    if (s + D <= full) {
#pragma unroll
      for (int u = 0; u < D; ++u) load(u);
      for (; s + 2 * D <= full; s += D)
#pragma unroll
        for (int u = 0; u < D; ++u) {
          turn(v[u]);
          load(u);
        }
#pragma unroll
      for (int u = 0; u < D; ++u) turn(v[u]);
      s += D;
    }
    for (; s < full; ++s) {
      load(0);
      turn(v[0]);
    }
    if (full < s1) {  // the step that ends past K
      const int32_t left = q.K - full * KS - slot * E;
#pragma unroll
      for (int i = 0; i < NI; ++i) v[0][i] = load_frag(src[i], left, q.K);
      turn(v[0]);
    }
    float* red = reinterpret_cast<float*>(lds);  // over the operands of all waves
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      if (rb + j * 16 >= r) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[w * RT * 256 + (i * 16 + 4 * g + e) * 16 + c] = acc[i][j][e];
      __syncthreads();
      if (threadIdx.x < RT * 256) {
        const int32_t tok = threadIdx.x / 16, rank = threadIdx.x % 16;
        float v = 0.f;
#pragma unroll
        for (int m = 0; m < WAVES; ++m) v += red[m * RT * 256 + threadIdx.x];
        ts[tok * ld + rb + j * 16 + rank] = tk.kind[tok] == ROW_HAS ? v : 0.f;
      }
    }
    if (rb + 16 * NR < r) __syncthreads();
  }
}

// NR: rank tiles at a time, 1 where no adapter has more.
template <typename T, int RT, int NR>
__device__ __forceinline__ void reduce_ranks(const lora_dev& d, const reduce_arg<T>& q,
                                             const tile_t& tl, int32_t r, const tile_lds& tk,
                                             char* lds, float* ts, int32_t ld, int32_t part,
                                             int32_t parts) {
  if (NR == 1 || r <= 16) reduce_tile<T, RT, 1>(d, q, tl, r, tk, lds, ts, ld, part, parts);
  else if (NR == 2 || r <= 32) reduce_tile<T, RT, 2>(d, q, tl, r, tk, lds, ts, ld, part, parts);
  else reduce_tile<T, RT, NR == 4 ? 4 : 1>(d, q, tl, r, tk, lds, ts, ld, part, parts);
}

// The scaled t of a tile as the operand of the products over tokens:
//   bf16  pack[tile][rank tile][hi, lo][lane] pieces of 8 tokens
//   fp32  pack[tile][token][ranks up to a multiple of 16]
// zero for tokens and ranks that are not there.
template <typename T>
__device__ __forceinline__ void write_pack(void* pack, int32_t ti, int32_t NT, int32_t n, int32_t r,
                                           float s, const float* ts, int32_t ld) {
  if constexpr (sizeof(T) == 2) {
    frag<bf16>* o = reinterpret_cast<frag<bf16>*>(pack) + (int64_t)ti * NT * 2 * 64;
    for (int32_t k = threadIdx.x; k < NT * 64; k += WAVES * 64) {
      const int32_t l = k & 63, j = (k >> 6) * 16 + (l & 15);
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int32_t tok = 8 * (l >> 4) + q;
        v[q] = j < r && tok < n ? s * ts[tok * ld + j] : 0.f;
      }
      frag<bf16> hi, lo;
      split_frag(v, hi, lo);
      o[(k >> 6) * 2 * 64 + l] = hi;
      o[(k >> 6) * 2 * 64 + 64 + l] = lo;
    }
  } else {
    float* o = reinterpret_cast<float*>(pack) + (int64_t)ti * TILE * NT * 16;
    for (int32_t k = threadIdx.x; k < TILE * NT * 16; k += WAVES * 64) {
      const int32_t tok = k / (NT * 16), j = k % (NT * 16);
      o[k] = j < r && tok < n ? s * ts[tok * ld + j] : 0.f;
    }
  }
}

// A wave takes 16 E columns at a time, E side by side of a lane.  The factor's
// rows lie along m, so (bf16) a lane's pieces of 8 rows are transposed in
// registers into E operands of 8 ranks each.  bf16 takes t in two parts (hi +
// lo, whose products sum to fp32's accuracy): up to 16 ranks both parts share
// one product (contraction 0-15 hi, 16-31 lo), above them each part has its
// own, 32 ranks a step; they lie in LDS (op).  With E = 4 the factor's rows of
// the next step or block are under way while one is summed; E = 8 (one step a
// block) has no registers for that, but accesses twice as wide.
// E = 8 needs a rank.
// WIDE: M >= 16 E, and a last block that would end past M begins earlier; what
// the block before it has is not stored again.
template <typename T, int RT, bool ONE, int E, bool WIDE>
__device__ __forceinline__ void expand_tile(const expand_arg<T>& q, const T* __restrict__ F,
                                            const tile_t& tl, int32_t r, float s,
                                            const tile_lds& tk, const float* ts, int32_t ld,
                                            const frag<bf16>* op, int32_t role, int32_t split) {
  constexpr int CW = 16 * E;
  constexpr bool H = sizeof(T) == 2, AHEAD = E == 4;
  constexpr int NROW = H ? 8 : 4;             // the factor's rows of a lane in a step
  constexpr int JS = H && !ONE ? 32 : 16;     // ranks of a step
  constexpr int RG = AHEAD ? RT : 1;          // groups of 16 tokens summed at a time
  static_assert(AHEAD || (H && ONE && WIDE), "wide pieces: one step a block");
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int32_t blocks = (q.M + CW - 1) / CW;
  const bool even = r % JS == 0;
  bool whole = tl.n == RT * 16;  // every row of the tile has the adapter
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) whole = whole && tk.kind[i * 16 + 4 * g + k] == ROW_HAS;
  whole = __all(whole);

  auto column = [&](int32_t b) { return (WIDE ? min(b * CW, q.M - CW) : b * CW) + c * E; };
  auto load = [&](const T* p, int32_t col) {
    piece<T, E> f;
    if constexpr (WIDE) __builtin_memcpy(&f, p + col, sizeof(f));
    else f = load_piece<T, E>(p + min(col, q.M - 1), q.M - col);
    return f;
  };
  auto row_of_tile = [&](int32_t tok) {
    int32_t row = tk.row[tok];
    asm volatile("" : "+v"(row));  // addresses kept over the loops cost too many registers
    return (int64_t)row;
  };
  piece<T, E> rows[NROW];
  auto load_rows = [&](int32_t b, int32_t j0) {
    int32_t j = j0 + (H ? 8 * (ONE ? g & 1 : g) : g);
    asm volatile("" : "+v"(j));  // as above
    const int32_t col = column(b);
#pragma unroll
    for (int k = 0; k < NROW; ++k)
      rows[k] = load(F + (int64_t)min(j + (H ? k : 4 * k), r - 1) * q.M, col);
  };
  const int32_t next = split * WAVES, b0 = role * WAVES + w;
  if (AHEAD && r > 0 && b0 < blocks) load_rows(b0, 0);
  for (int32_t b = b0; b < blocks; b += next) {
    const int32_t col = column(b);
    piece<T, E> bv[RT][4];
    auto load_base = [&](int i) {
      if (q.base)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          bv[i][k] = load(q.base + row_of_tile(i * 16 + 4 * g + k) * q.ldb, col);
    };
    auto put = [&](int i, f4 (&acc)[E]) {
      if (!whole)  // rows without an adapter get base alone, wrong ids NaN
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int8_t has = tk.kind[i * 16 + 4 * g + k];
          const float v = has == ROW_BAD ? __builtin_nanf("") : 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e][k] = has == ROW_HAS ? acc[e][k] : v;
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t tok = i * 16 + 4 * g + k;
        if (tok >= tl.n) continue;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[e] = acc[e][k];
          if (q.base) v[e] += at(bv[i][k], e);
        }
        piece<T, E> o;
        round_to(v, o);
        store_piece(q.Y + row_of_tile(tok) * q.ldy + col, o, b * CW - col, WIDE ? E : q.M - col);
      }
    };
    f4 acc[RG][E];
#pragma unroll
    for (int i = 0; i < RG; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[i][e] = f4{0.f, 0.f, 0.f, 0.f};
    if (!AHEAD) load_rows(b, 0);
    load_base(0);
    if constexpr (AHEAD && RT > 1) load_base(1);
    // one step at most where ONE, exactly one for E = 8
    for (int32_t j0 = 0; j0 < (!AHEAD ? 1 : ONE ? min(r, 1) : r); j0 += JS) {
      auto load_next = [&]() {
        const bool more = !ONE && j0 + JS < r;
        if (more || b + next < blocks) load_rows(more ? b : b + next, more ? j0 + JS : 0);
      };
      if constexpr (H) {
        frag<bf16> cols[E];
        if (!even)  // rows past the rank count as zeros
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const bool keep = j0 + 8 * (ONE ? g & 1 : g) + k < r;
#pragma unroll
            for (int x = 0; x < E / 2; ++x) rows[k].w[x] = pick(keep, rows[k].w[x], 0u);
          }
#pragma unroll
        for (int x = 0; x < E / 2; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = rows[2 * k].w[x], a1 = rows[2 * k + 1].w[x];
            cols[2 * x].w[k] = __builtin_amdgcn_perm(a1, a0, 0x05040100u);
            cols[2 * x + 1].w[k] = __builtin_amdgcn_perm(a1, a0, 0x07060302u);
          }
        const bool infinite = any_infinite(cols);
        if (ONE && infinite && g >= 2) drop_infinities(cols);  // these lanes' ranks are lo
        if constexpr (!AHEAD) {
          if constexpr (RT > 1) load_base(1);  // the rows' registers are free now
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const frag<bf16> t1 = op[i * 64 + l];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[0][e] = mma(t1, cols[e], f4{0.f, 0.f, 0.f, 0.f});
            put(i, acc[0]);
          }
        } else {
          load_next();
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const frag<bf16> hi = ONE ? op[i * 64 + l] : op[((j0 / 32 * 2 + i) * 2) * 64 + l];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] = mma(hi, cols[e], acc[i][e]);
          }
          if constexpr (!ONE) {
            if (infinite) drop_infinities(cols);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const frag<bf16> lo = op[((j0 / 32 * 2 + i) * 2 + 1) * 64 + l];
#pragma unroll
              for (int e = 0; e < E; ++e) acc[i][e] = mma(lo, cols[e], acc[i][e]);
            }
          }
        }
      } else {
        piece<T, E> cols[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool keep = even || j0 + g + 4 * k < r;
#pragma unroll
          for (int x = 0; x < E; ++x) cols[k].w[x] = pick(keep, rows[k].w[x], 0u);
        }
        load_next();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int32_t j = j0 + g + 4 * k;
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float tv = j < r ? s * ts[(i * 16 + c) * ld + j] : 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
              acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(tv, at(cols[k], e), acc[i][e], 0, 0, 0);
          }
        }
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < RT; ++i) put(i, acc[i]);
    }
  }
}

// Width of a lane's piece in the expansion.
template <typename T>
__device__ __host__ constexpr int expand_width(bool one, int32_t M) {
  return sizeof(T) == 2 && one && M >= 128 ? 8 : 4;
}

template <typename T, int RT, bool ONE>
__device__ __forceinline__ void expand_any(const expand_arg<T>& q, const T* __restrict__ F,
                                           const tile_t& tl, int32_t r, float s,
                                           const tile_lds& tk, const float* ts, int32_t ld,
                                           const frag<bf16>* op, int32_t role, int32_t split) {
  if constexpr (sizeof(T) == 2 && ONE)
    if (r > 0 && expand_width<T>(ONE, q.M) == 8)
      return expand_tile<T, RT, ONE, 8, true>(q, F, tl, r, s, tk, ts, ld, op, role, split);
  if (q.M >= 64) expand_tile<T, RT, ONE, 4, true>(q, F, tl, r, s, tk, ts, ld, op, role, split);
  else expand_tile<T, RT, ONE, 4, false>(q, F, tl, r, s, tk, ts, ld, op, role, split);
}

// grid: 8 * (tiles of a die) * roles.  Roles 0 to split - 1 of a tile compute t
// of problem a and a share of the columns each, role 0 writes what is wanted
// of t; role `split`, if launched, does the same for problem b, which has no
// expansion.  cut: there is no expansion, and the roles of a and of b compute
// and write a share of the sum over k each.  self: no tables are there yet, see
// self_route.  REDUCE and EXPAND do one half each, for more than 16 ranks: 64
// ranks at a time want 243 registers in the sums, the expansion 121 and twice
// the waves (6,001 tokens of ranks 16 to 64, backward: 59 and 40 us; 120 us as
// one kernel).  BOTH in fp32 keeps 4 of its 132 registers in scratch memory.
enum { BOTH, REDUCE, EXPAND };

template <typename T, int NR, int MODE>
__global__ __launch_bounds__(WAVES * 64, MODE == REDUCE && NR == 4 ? 2 : 4) void k_lora_apply(
    lora_dev d, route_t p, tables_t out, bool self, reduce_arg<T> a, reduce_arg<T> b,
    expand_arg<T> e, int32_t split, int32_t roles, bool cut, uint32_t* __restrict__ mask) {
  extern __shared__ char lds[];
  __shared__ tile_lds tk;
  const int32_t NT = (d.R + 15) / 16, ld = NT * 16 + 1;
  int32_t ti, role;
  tile_t tl;
  if (self) {
    if (!self_route(d, p, out, roles, lds, tk, ti, role, tl)) return;
  } else {
    if (!place_of(tiles_of(p), roles, ti, role)) return;
    tl = tile_at(p, ti);
  }
  const int32_t r = tl.l < d.L ? rank_of(d, tl.l) : 0;
  const float s = r > 0 ? scale_of(d, tl.l) : 0.f;
  if (threadIdx.x < 64) {
    const int32_t tok = threadIdx.x & (TILE - 1), in = min(tok, tl.n - 1);
    const int32_t row = self ? tk.row[in] : row_at(p, tl.begin + in);
    const int32_t id = (self || p.order) && tl.l < d.L ? tl.l : p.ids[row];
    const int8_t kind = tok >= tl.n ? ROW_NONE : id >= d.L ? ROW_BAD : id >= 0 ? ROW_HAS : ROW_NONE;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // rows are read before they are set
    __builtin_amdgcn_wave_barrier();
    tk.row[tok] = row;
    tk.kind[tok] = kind;
    const uint64_t has = __ballot(kind == ROW_HAS);
    if (mask && role == 0 && threadIdx.x == 0) mask[ti] = (uint32_t)has;
  }
  __syncthreads();
  float* ts = reinterpret_cast<float*>(lds);
  char* room = lds + (TILE * ld + 3) / 4 * 16;  // the waves' operands, their sums, the scaled t
  const bool is_a = role < split;
  const reduce_arg<T>& q = is_a ? a : b;
  const int32_t part = cut ? is_a ? role : role - split : 0;
  const int32_t parts = cut ? is_a ? split : roles - split : 1;
  if (q.given) {
    const int64_t next = (int64_t)p.Tn * d.R;
    for (int32_t k = threadIdx.x; k < tl.n * d.R; k += WAVES * 64) {
      const int32_t tok = k / d.R, j = k % d.R;
      const float* from = q.given + (int64_t)tk.row[tok] * d.R + j;
      float v = 0.f;
#pragma unroll 4
      for (int32_t i = 0; i < q.parts; ++i) v += from[i * next];
      ts[tok * ld + j] = tk.kind[tok] == ROW_HAS ? v : 0.f;
    }
  } else if constexpr (MODE != EXPAND) {
    if (tl.n <= 16) reduce_ranks<T, 1, NR>(d, q, tl, r, tk, room, ts, ld, part, parts);
    else reduce_ranks<T, 2, NR>(d, q, tl, r, tk, room, ts, ld, part, parts);
  }
  __syncthreads();
  if (cut || role == 0 || role == split) {
    if (q.t) {
      float* to = q.t + (int64_t)part * p.Tn * d.R;
      for (int32_t k = threadIdx.x; k < tl.n * d.R; k += WAVES * 64) {
        const int32_t tok = k / d.R, j = k % d.R;
        to[(int64_t)tk.row[tok] * d.R + j] = j < r ? ts[tok * ld + j] : 0.f;
      }
    }
    if (q.pack && tl.l < d.L) write_pack<T>(q.pack, ti, NT, tl.n, r, s, ts, ld);
  }
  if constexpr (MODE == REDUCE) return;
  if (role >= split || !e.Y) return;
  frag<bf16>* op = reinterpret_cast<frag<bf16>*>(room);
  if constexpr (sizeof(T) == 2 && NR == 1) {
    if (threadIdx.x < TILE * 4) {
      const int32_t l = threadIdx.x & 63, tok = threadIdx.x / 64 * 16 + (l & 15), j0 = (l >> 4 & 1) * 8;
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = j0 + x < r ? s * ts[tok * ld + j0 + x] : 0.f;
      frag<bf16> hi, lo;
      split_frag(v, hi, lo);
#pragma unroll
      for (int k = 0; k < 4; ++k) op[threadIdx.x].w[k] = pick(l < 32, hi.w[k], lo.w[k]);
    }
    __syncthreads();
  }
  if constexpr (sizeof(T) == 2 && NR > 1) {
    const int32_t rts = tl.n <= 16 ? 1 : 2;
    for (int32_t k = threadIdx.x; k < (r + 31) / 32 * 128; k += WAVES * 64) {
      const int32_t l = k & 63, i = (k >> 6) & 1, j0 = k / 128 * 32 + 8 * (l >> 4);
      const int32_t tok = i * 16 + (l & 15);
      if (i >= rts) continue;
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = j0 + x < r ? s * ts[tok * ld + j0 + x] : 0.f;
      frag<bf16> hi, lo;
      split_frag(v, hi, lo);
      op[(k >> 6) * 128 + l] = hi;
      op[(k >> 6) * 128 + 64 + l] = lo;
    }
    __syncthreads();
  }
  const T* F = e.F + (r > 0 ? (int64_t)tl.l * d.R * e.M : 0);
  if (tl.n <= 16) expand_any<T, 1, NR == 1>(e, F, tl, r, s, tk, ts, ld, op, role, split);
  else expand_any<T, 2, NR == 1>(e, F, tl, r, s, tk, ts, ld, op, role, split);
}

// --------------------------------------------------------------------- grad
template <typename T>
struct grad_arg {
  const T* X;
  int64_t ldx;
  int32_t K;
  const void* pack;
  T* dF;
  float* part;  // [partial slots][R][K]
};

// dF = sum over the slot's tokens.  A wave has 16 pieces of columns and every
// tw-th tile of its slot; the tokens are the contraction, so (bf16) the lane's
// pieces of 8 tokens are transposed in registers into operands, two columns at
// a time.  The rows of the next tile are on their way while one is summed.
// tw > 1: the waves of a workgroup share the columns and their sums meet in
// LDS.  tw = 1: each wave has its own columns.  grid: column blocks (of X, then
// of dY) x slots x rank blocks of 16 * NR.  Bound by the reading of X and dY,
// 256 bytes of a row at a time: 31 us for the 134 MB of 8,192 tokens at
// 4096x4096 (4.3 TB/s), 50 us for the 181 MB of 6,001 tokens of 24 adapters.
// NR is 2 at most: 64 ranks at a time spill registers.  NR = 1 in bf16 keeps 5
// of its 133 in scratch memory, for four waves a SIMD.
constexpr int grad_waves(int NR) { return NR == 1 ? 8 : 4; }

template <typename T, int NR, bool FULL>
__device__ __forceinline__ void grad_sum(const route_t& p, const grad_arg<T>& q, const slot_t& sl,
                                         int32_t NT, int32_t nt, int32_t rt0, int32_t col, int32_t h,
                                         int32_t tw, const uint32_t* __restrict__ mask,
                                         f4 (&acc)[NR][EL<T>]) {
  const int l = lane_id(), c = l & 15, g = l >> 4;
  const int32_t left = q.K - col;
  const T* X = q.X + col;
  // has: which of the tile's tokens count.
  auto fetch = [&](int32_t ti, frag<T> (&rows)[8], uint32_t& has) {
    const int32_t n = tile_at(p, ti).n;
    has = mask[ti];
    int32_t row[8];
    if (p.order) {
      // The tile's tokens come as scalars (`order` goes on for a tile past the
      // last place): loads of theirs among the rows' would have to be waited for
      // together with them.
      int32_t all[TILE];
      __builtin_memcpy(all, p.order + ti * p.size, sizeof(all));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t a = pick(g & 1, all[8 + k], all[k]), b = pick(g & 1, all[24 + k], all[16 + k]);
        row[k] = pick(g & 2, b, a);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) row[k] = ti * p.size + 8 * g + k;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t at = 8 * g + k < n ? row[k] : 0;
      if constexpr (FULL) rows[k] = load_frag(X + at * q.ldx);
      else rows[k] = load_frag(X + at * q.ldx, left, q.K);
    }
  };
  // The tile's operands of t (bf16: hi and lo pieces; fp32: one rank of the
  // lane's 8 tokens).
  constexpr int PN = 8;  // dwords of a rank tile
  auto fetch_pack = [&](int32_t ti, uint32_t (&t)[NR][PN]) {
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      if (rt0 + j >= nt) break;
      if constexpr (sizeof(T) == 2) {
        const frag<bf16>* o =
            reinterpret_cast<const frag<bf16>*>(q.pack) + ((int64_t)ti * NT + rt0 + j) * 128 + l;
        __builtin_memcpy(t[j], o, 16);
        __builtin_memcpy(t[j] + 4, o + 64, 16);
      } else {
        const uint32_t* o = reinterpret_cast<const uint32_t*>(q.pack) +
                            (((int64_t)ti * TILE + 8 * g) * NT + rt0 + j) * 16 + c;
#pragma unroll
        for (int k = 0; k < 8; ++k) t[j][k] = o[k * NT * 16];
      }
    }
  };
  auto use = [&](uint32_t has, frag<T> (&rows)[8], const uint32_t (&t)[NR][PN]) {
    if (has != ~0u)
#pragma unroll
      for (int k = 0; k < 8; ++k) rows[k] = keep_if((has >> (8 * g + k)) & 1, rows[k]);
    if constexpr (sizeof(T) == 2) {
      peak_t peak;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) peak.add(rows[k].w[x]);
      const bool infinite = peak.infinite();
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        frag<bf16> a, b;  // columns e and e + 1
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = rows[2 * k].w[e / 2], y = rows[2 * k + 1].w[e / 2];
          a.w[k] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          b.w[k] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          if (rt0 + j >= nt) break;
          const frag<bf16> hi{{t[j][0], t[j][1], t[j][2], t[j][3]}};
          acc[j][e] = mma(hi, a, acc[j][e]);
          acc[j][e + 1] = mma(hi, b, acc[j][e + 1]);
        }
        if (infinite)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a.w[k] = without_infinities(a.w[k]);
            b.w[k] = without_infinities(b.w[k]);
          }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          if (rt0 + j >= nt) break;
          const frag<bf16> lo{{t[j][4], t[j][5], t[j][6], t[j][7]}};
          acc[j][e] = mma(lo, a, acc[j][e]);
          acc[j][e + 1] = mma(lo, b, acc[j][e + 1]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          if (rt0 + j >= nt) break;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[j][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(t[j][k]),
                                                             at(rows[k], e), acc[j][e], 0, 0, 0);
        }
    }
  };
  if (h >= sl.n || rt0 >= nt) return;
  frag<T> now[8];
  uint32_t t[NR][PN], has_now;
  if constexpr (!FULL) {  // the last columns: no registers for a second tile's rows
    for (; h < sl.n; h += tw) {
      fetch_pack(sl.tile + h, t);
      fetch(sl.tile + h, now, has_now);
      use(has_now, now, t);
    }
    return;
  }
  frag<T> next[8];
  uint32_t has_next;
  fetch(sl.tile + h, now, has_now);
  for (; h + tw < sl.n; h += tw) {
    fetch_pack(sl.tile + h, t);  // before the next rows: waiting for it does not wait for them
    fetch(sl.tile + h + tw, next, has_next);
    use(has_now, now, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) now[k] = next[k];
    has_now = has_next;
  }
  fetch_pack(sl.tile + h, t);
  use(has_now, now, t);
}

template <typename T, int NR>
__global__ __launch_bounds__(grad_waves(NR) * 64, NR == 1 ? 4 : 2) void k_lora_grad(
    lora_dev d, route_t p, grad_arg<T> q0, grad_arg<T> q1, int32_t blocks0, int32_t blocks,
    int32_t tw, const uint32_t* __restrict__ mask) {
  constexpr int E = EL<T>, CW = 16 * E, GW = grad_waves(NR);
  extern __shared__ char lds[];
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int32_t b = tw == 1 ? (int32_t)blockIdx.x * GW + w : (int32_t)blockIdx.x;
  if (b >= blocks) return;
  const bool first = b < blocks0;
  const grad_arg<T>& q = first ? q0 : q1;
  const slot_t sl = slot_at(p, blockIdx.y);
  if (sl.n < 0) return;
  const int32_t c0 = (b - (first ? 0 : blocks0)) * CW, col = c0 + c * E;
  const int32_t r = rank_of(d, sl.l);
  const int32_t NT = (d.R + 15) / 16, rt0 = blockIdx.z * NR, nt = (r + 15) / 16;
  f4 acc[NR][E];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[j][e] = f4{0.f, 0.f, 0.f, 0.f};
  const int32_t h = tw == 1 ? 0 : w;
  if (c0 + CW <= q.K) grad_sum<T, NR, true>(p, q, sl, NT, nt, rt0, col, h, tw, mask, acc);
  else grad_sum<T, NR, false>(p, q, sl, NT, nt, rt0, col, h, tw, mask, acc);
  auto put = [&](int32_t rank, int32_t m, float (&v)[E]) {
    if (rank >= d.R || m >= q.K) return;
    // The products gave a rank that the adapter lacks zeros times the rows: NaN
    // where those are infinite or NaN.
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = rank < r ? v[e] : 0.f;
    if (sl.part < 0) {
      store_frag(q.dF + ((int64_t)sl.l * d.R + rank) * q.K + m, to_frag(v), q.K - m);
    } else {
      float* o = q.part + ((int64_t)sl.part * d.R + rank) * q.K + m;
#pragma unroll
      for (int e = 0; e < E; e += 4)
        store_frag(o + e, to_frag({v[e], v[e + 1], v[e + 2], v[e + 3]}), q.K - m - e);
    }
  };
  if (tw == 1) {
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = acc[j][e][k];
        put((rt0 + j) * 16 + 4 * g + k, col, v);
      }
    return;
  }
  float* red = reinterpret_cast<float*>(lds);  // [GW][16][CW]
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    if (rt0 + j >= NT) break;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) red[(w * 16 + 4 * g + k) * CW + c * E + e] = acc[j][e][k];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int32_t at = threadIdx.x / 16 * CW + threadIdx.x % 16 * E;
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] = 0.f;
#pragma unroll
        for (int m = 0; m < GW; ++m) v[e] += red[m * 16 * CW + at + e];
      }
      put((rt0 + j) * 16 + (int32_t)threadIdx.x / 16, c0 + threadIdx.x % 16 * E, v);
    }
  }
}

// The gradients of adapters with several slots: the sum of their partial sums,
// in slot order.  grid: adapters x shares of the elements
// of dA (blocks0 of them), then of dB.
template <typename T>
__global__ __launch_bounds__(256) void k_lora_join(lora_dev d, route_t p, int32_t slots,
                                                   grad_arg<T> q0, grad_arg<T> q1,
                                                   int32_t blocks0) {
  const int32_t l = blockIdx.x;
  const join_t jn = p.order ? p.join[l] : join_t{slots, 0};
  if (jn.slots == 1) return;
  const bool first = (int32_t)blockIdx.y < blocks0;
  const grad_arg<T>& q = first ? q0 : q1;
  const int32_t at = (int32_t)blockIdx.y - (first ? 0 : blocks0);
  const int32_t of = first ? blocks0 : (int32_t)gridDim.y - blocks0;
  const int64_t size = (int64_t)d.R * q.K;
  const float* part = q.part + jn.part * size;
  T* out = q.dF + l * size;
  for (int64_t m = ((int64_t)at * 256 + threadIdx.x) * 4; m < size; m += (int64_t)of * 1024) {
    const int32_t n = (int32_t)min(size - m, (int64_t)4);
    float v[4] = {};
#pragma unroll 8
    for (int32_t s = 0; s < jn.slots; ++s) {
      const frag<float> f = load_frag(part + s * size + m, n, size);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += __uint_as_float(f.w[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) out[m + e] = elem<T>::from_f(v[e]);
  }
}

// --------------------------------------------------------------------- host
snack_status check_lora(const snack_lora* p, snack_dtype dt, int32_t T, bool backward) {
  if (!p) return SNACK_E_NULL;
  if (dt != SNACK_F32 && dt != SNACK_BF16) return SNACK_E_DTYPE;
  if (p->M < 1 || p->K < 1 || p->L < 1 || p->L > MAX_ADAPTERS || p->R < 1 || p->R > MAX_RANK ||
      T < 0)
    return SNACK_E_SHAPE;
  if (T > max_tokens(backward) || p->M > MAX_FEATURES || p->K > MAX_FEATURES) return SNACK_E_OVERFLOW;
  return SNACK_OK;
}

// Memory of a call: n rows of `row` bytes, ld bytes apart (wide: sizes and
// strides are the caller's).
struct span_t {
  __int128 p, row, ld, n;
  span_t(const void* at, __int128 bytes, __int128 stride = 0, __int128 rows = 1)
      : p((uintptr_t)at), row(bytes), ld(stride), n(at && bytes > 0 ? rows : 0) {
    if (n > 1 && ld == row) row *= n, n = 1;
  }
  __int128 end() const { return p + (n - 1) * ld + row; }
  // Whether a row meets the bytes from lo up to hi.
  bool meets(__int128 lo, __int128 hi) const {
    // the first row that ends past lo
    const __int128 i = lo < p + row ? 0 : n == 1 ? 1 : (lo - row - p) / ld + 1;
    return i < n && p + i * ld < hi;
  }
};

// Whether a byte belongs to both.  Rows may lie between the other's rows.
bool overlap(const span_t& a, const span_t& b) {
  if (a.n == 0 || b.n == 0 || a.end() <= b.p || b.end() <= a.p) return false;
  if (a.n > b.n) return overlap(b, a);
  if (a.n > 1 && a.ld == b.ld) {  // row i of b begins `at` bytes after row i + q of a
    const __int128 d = b.p - a.p, q = d >= 0 ? d / a.ld : -((a.ld - 1 - d) / a.ld), at = d - q * a.ld;
    auto both = [&](__int128 k) { return std::max<__int128>(0, -k) < std::min(b.n, a.n - k); };
    return (at < a.row && both(q)) || (at + b.row > a.ld && both(q + 1));
  }
  for (__int128 i = 0; i < a.n; ++i)
    if (b.meets(a.p + i * a.ld, a.p + i * a.ld + a.row)) return true;
  return false;
}

// Whether an output lies over an input or over another output.
template <size_t O, size_t I>
bool any_overlap(const span_t (&out)[O], const span_t (&in)[I]) {
  for (size_t o = 0; o < O; ++o) {
    for (const span_t& i : in)
      if (overlap(out[o], i)) return true;
    for (size_t q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return true;
  }
  return false;
}

// Tokens up to which k_lora_few is taken.
constexpr int32_t FEW_TOKENS = 64;

struct plan_t {
  int32_t size;   // tokens of a tile at most
  int32_t whole;  // tiles if all tokens had one adapter
  int32_t tiles, slots, slot_tiles, part_slots, blocksA, blocksB, NT;
  int32_t tw;     // waves that share a slot's tokens: 1 or all of a workgroup
  bool self;      // the workgroups find their tokens themselves
  bool two;       // t in a launch of its own, K and M cut into ksK and ksM parts
  int32_t ksK, ksM;
  size_t order, tile, slot, join, count, t, u, pack_t, pack_u, mask, partA, partB, total;
};

// Tiles to be expected: about half the adapters have one that is not full.
int64_t tiles_guess(int32_t L, int32_t T, int32_t size) {
  return cdiv(T, size) + (L > 1 ? std::min(L, T) / 2 : 0);
}

plan_t plan_of(const snack_lora* p, snack_dtype dt, int32_t T, bool backward) {
  plan_t w{};
  const int32_t e = dt == SNACK_BF16 ? 8 : 4;
  w.NT = (int32_t)cdiv(p->R, 16);
  w.size = TILE;
  // Forward, too few tiles for every CU to have a workgroup: smaller ones, as
  // long as those are under way together (300 tokens of one adapter of rank 16,
  // 4096 to 4096: 8.8 us, 11.3 us with tiles of 32).
  if (tiles_guess(p->L, T, TILE) * std::min<int64_t>(8, cdiv(backward ? p->K : p->M, 512)) <
          256 &&
      (w.NT < 3 || tiles_guess(p->L, T, 16) <= 256))
    w.size = 16;
  w.whole = (int32_t)cdiv(T, w.size);
  w.tiles = p->L == 1 ? w.whole : (int32_t)std::min<int64_t>(T, (int64_t)T / w.size + p->L + 1);
  w.blocksA = (int32_t)cdiv(p->K, 16 * e);
  w.blocksB = (int32_t)cdiv(p->M, 16 * e);
  // The waves of a workgroup share a slot where all workgroups are under way
  // together, for tokens may all have one adapter (164 fp32 tokens that do, of 7,
  // 2344 to 2525: 63 us with one wave a slot, 28 us shared), and where adapters
  // have tiles enough for all waves.  Elsewhere one wave sums it alone (300
  // tokens of 16 adapters of rank 64, 4096 to 4096: 8 us, 35 us shared).  Not
  // looked at here: fewer tiles than adapters leave most waves of a shared slot
  // idle (a backward of 100 bf16 tokens of 64 adapters of rank 16, 4096 to 4096:
  // 79 us, 24 us with one wave a slot).
  const int32_t gw = grad_waves(w.NT), users = std::max(1, std::min(p->L, w.whole));
  const int64_t blocks = w.blocksA + w.blocksB, alone = blocks * users * cdiv(w.NT, 2);
  const int32_t per = w.whole / users;  // tiles of an adapter
  w.tw = w.whole > 1 && (alone <= 1024 || (alone < 4096 && per >= 2 * gw)) ? gw : 1;
  const int64_t runs = std::max<int64_t>(1, cdiv(4096 / gw, blocks));
  const int32_t even = (int32_t)cdiv(w.whole, runs);  // tiles of a slot, all slots alike
  // About one tile for each wave (four, where there is one adapter alone): one
  // slot for each adapter, which needs no joining (1,000 tokens of 8 adapters, 768
  // to 2304, fp32: 28.2 us with it, 23.1 us without; 1,024 of 4, lopsided: 26.8 us
  // and 28.2 us).
  if (w.tw > 1 && (p->L == 1 ? w.whole <= 4 * gw : w.whole <= 8 * gw && per <= gw))
    w.slot_tiles = std::max(w.whole, 1);
  else if (w.tw > 1) w.slot_tiles = std::max(gw, even) * (p->L == 1 ? 1 : 2);
  else w.slot_tiles = (int32_t)std::max<int64_t>(16, cdiv(w.whole, 32));
  w.slots = p->L == 1 ? (int32_t)cdiv(w.whole, w.slot_tiles)
                      : w.whole / w.slot_tiles + p->L;
  // an adapter with several slots has more than slot_tiles tiles, so its
  // slots are at most three times its share of the tokens
  w.part_slots = p->L == 1 ? w.slots
                           : (int32_t)std::min<int64_t>(w.slots, 3 * cdiv(w.whole, w.slot_tiles));
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o = align_up(o + b, 256);
    return at;
  };
  w.self = p->L > 1 && T <= SELF_TOKENS && p->L < SELF_GROUPS;
  const int64_t tiles = tiles_guess(p->L, T, w.size);
  // More than 16 ranks: two launches, as the expansion then needs fewer
  // registers than the sums.  Up to 16: two where the rows that t is summed
  // over are long and the tiles few, so that several workgroups of a tile would
  // each sum t anew (fp32, 1,024 tokens, 4096 to 4096: 28.9 us in one launch,
  // 18.5 us in two; bf16 at 4096: 16.1 us either way).
  const int64_t row = (int64_t)(backward ? p->M : p->K) * (16 / e);
  w.two = p->R > 16 || (row >= 12288 && tiles < (backward ? 300 : 160));
  // Two workgroups on every CU (one, where 64 ranks at a time leave registers
  // for one), one step for each wave at least.
  auto cut = [&](int32_t F) {
    return (int32_t)std::max<int64_t>(
        1, std::min<int64_t>((w.NT >= 3 ? 256 : 512) / std::max<int64_t>(tiles * (backward ? 2 : 1), 1),
                             F / (8 * e * WAVES)));
  };
  w.ksK = cut(p->K);
  w.ksM = cut(p->M);
  if (p->L > 1 && (backward || !w.self || w.two)) {
    w.order = take(4 * ((size_t)w.tiles * w.size + TILE));
    w.tile = take(sizeof(tile_t) * (size_t)w.tiles);
    w.slot = take(sizeof(slot_t) * (size_t)w.slots);
    w.join = take(sizeof(join_t) * (size_t)p->L);
    w.count = take(8);
  }
  if (w.two) {
    w.t = take(4 * (size_t)T * p->R * w.ksK);
    if (backward) w.u = take(4 * (size_t)T * p->R * w.ksM);
  }
  if (backward) {
    const size_t pk = 4 * (size_t)w.tiles * TILE * w.NT * 16;
    w.pack_t = take(pk);
    w.pack_u = take(pk);
    w.mask = take(4 * (size_t)w.tiles);
    w.partA = take(4 * (size_t)w.part_slots * p->R * p->K);
    w.partB = take(4 * (size_t)w.part_slots * p->R * p->M);
  }
  w.total = std::max<size_t>(o, 256);
  return w;
}

// The tokens' order, or (self) where k_lora_apply will put it.
route_t launch_route(const snack_lora* p, const plan_t& w, const int32_t* ids, int32_t T, char* ws,
                     bool backward, hipStream_t s) {
  route_t r{ids, T, w.size, w.slot_tiles, nullptr, nullptr, nullptr, nullptr, nullptr};
  if (p->L == 1) return r;
  if (w.self && !backward && !w.two) return r;
  r.order = (const int32_t*)(ws + w.order);
  r.tile = (const tile_t*)(ws + w.tile);
  r.slot = (const slot_t*)(ws + w.slot);
  r.join = (const join_t*)(ws + w.join);
  r.count = (const int32_t*)(ws + w.count);
  if (w.self) return r;
  const int32_t G = p->L + 1, nw = std::max(1, std::min(16, 15360 / G));
  hipLaunchKernelGGL(k_lora_route, dim3(1), dim3(1024), 4 * ((size_t)(nw + 2) * G + 2), s, ids, T,
                     p->L, nw, w.size, w.slot_tiles, (int32_t*)r.order, (tile_t*)r.tile, (slot_t*)r.slot,
                     (join_t*)r.join, (int32_t*)r.count);
  return r;
}

template <typename T>
void launch_apply(const lora_dev& d, const route_t& r, const plan_t& w, bool self, int32_t split,
                  int32_t roles, bool cut, const reduce_arg<T>& a, const reduce_arg<T>& b,
                  const expand_arg<T>& e, uint32_t* mask, hipStream_t s) {
  const size_t ts = 4 * ((size_t)(TILE * (w.NT * 16 + 1) + 3) / 4 * 4);
  const int32_t nr = w.NT >= 3 ? 4 : w.NT;
  const bool sums = cut || w.NT == 1;  // whether sums over k are made here
  const size_t red = std::max<size_t>(sums ? (size_t)WAVES * (2 + nr) * 2048 : SELF_BYTES,
                                      (size_t)cdiv(d.R, 32) * 4096);
  const tables_t out{const_cast<int32_t*>(r.order), const_cast<tile_t*>(r.tile),
                     const_cast<slot_t*>(r.slot), const_cast<join_t*>(r.join),
                     const_cast<int32_t*>(r.count)};
  const dim3 grid((unsigned)(NUM_XCD * cdiv(w.tiles, NUM_XCD) * roles));
  auto kernel = w.NT == 1 ? k_lora_apply<T, 1, BOTH>
                : !cut    ? k_lora_apply<T, 2, EXPAND>
                : nr == 2 ? k_lora_apply<T, 2, REDUCE>
                          : k_lora_apply<T, 4, REDUCE>;
  hipLaunchKernelGGL(kernel, grid, dim3(WAVES * 64), ts + red, s, d, r, out, self, a, b, e, split,
                     roles, cut, mask);
}

// Problem a (ksA parts) with the expansion e, and problem b (ksB parts), each
// if wanted; ta, tb: room for the parts.
template <typename T>
void run_apply(const lora_dev& d, const route_t& r, const plan_t& w, bool with_a, reduce_arg<T> a,
               int32_t ksA, float* ta, bool with_b, reduce_arg<T> b, int32_t ksB, float* tb,
               const expand_arg<T>& e, uint32_t* mask, hipStream_t s) {
  bool self = w.self;
  if (w.two) {
    reduce_arg<T> a1 = a, b1 = b;
    a1.t = ta, a1.pack = nullptr, b1.t = tb, b1.pack = nullptr;
    const int32_t na = with_a ? ksA : 0, nb = with_b && !b.given ? ksB : 0;
    if (na + nb > 0) {
      launch_apply<T>(d, r, w, self, na, na + nb, true, a1, b1, {}, nullptr, s);
      self = false;
    }
    if (with_a) a.given = ta, a.parts = ksA;
    if (nb > 0) b.given = tb, b.parts = ksB;
  }
  // Workgroups of a tile: enough to have two on every CU, each with columns
  // for all its waves.
  int32_t split = with_a ? 1 : 0;
  if (with_a && e.Y)
    split = (int32_t)std::max<int64_t>(
        1, std::min<int64_t>(512 / std::max<int64_t>(tiles_guess(d.L, r.Tn, w.size), 1),
                             cdiv(e.M, 16 * expand_width<T>(w.NT == 1, e.M) * WAVES)));
  launch_apply<T>(d, r, w, self, split, split + (with_b ? 1 : 0), false, a, b, e, mask, s);
}

template <typename T>
void run_fwd(const snack_lora* p, const lora_dev& d, const int32_t* ids, int32_t Tn, const void* X,
             int64_t ldx, const void* base, int64_t ldb, void* Y, int64_t ldy, float* t, char* ws,
             snack_dtype dt, hipStream_t s) {
  if (Tn <= FEW_TOKENS && p->K >= EL<T> && p->M >= EL<T>) {
    const int32_t blocks = (int32_t)cdiv(p->M, 64 * EL<T>);
    // About one workgroup on every CU at most (37 tokens, 4096 to 11008, ranks 8
    // to 32: 10.9 us; 20 us with two), and two ranks at least for each wave.
    const int32_t most = std::max(1, 256 / Tn);
    int32_t log_nb = 0;
    while (log_nb < 4 && (1 << log_nb) < blocks &&
           ((most << log_nb) < blocks || (2 * FEW_WAVES >> log_nb) > p->R))
      ++log_nb;
    const int32_t split = (int32_t)std::min<int64_t>(cdiv(blocks, 1 << log_nb), most);
    const int32_t rows = Tn < NUM_XCD ? Tn : (int32_t)(cdiv(Tn, NUM_XCD) * NUM_XCD);
    hipLaunchKernelGGL(k_lora_few<T>, dim3((unsigned)(rows * split)), dim3(FEW_WAVES * 64), 0, s, d,
                       ids, Tn, split, log_nb, (const T*)p->A, p->K, (const T*)X, ldx, (const T*)p->B, p->M,
                       (const T*)base, ldb, (T*)Y, ldy, t);
    return;
  }
  const plan_t w = plan_of(p, dt, Tn, false);
  const route_t r = launch_route(p, w, ids, Tn, ws, false, s);
  const reduce_arg<T> a{(const T*)p->A, (const T*)X, ldx, p->K, nullptr, 0, t, nullptr};
  const expand_arg<T> e{(const T*)p->B, p->M, (const T*)base, ldb, (T*)Y, ldy};
  run_apply<T>(d, r, w, true, a, w.ksK, (float*)(ws + w.t), false, a, 0, nullptr, e, nullptr, s);
}

template <typename T>
void run_bwd(const snack_lora* p, const lora_dev& d, const int32_t* ids, const float* t,
             int32_t Tn, const void* X, int64_t ldx, const void* dY, int64_t lddy,
             const void* base, int64_t ldb, void* dX, int64_t lddx, void* dA, void* dB, char* ws,
             snack_dtype dt, hipStream_t s) {
  const plan_t w = plan_of(p, dt, Tn, true);
  route_t r{};
  uint32_t* mask = (uint32_t*)(ws + w.mask);
  if (Tn > 0 && (dX || dA || dB)) {
    r = launch_route(p, w, ids, Tn, ws, true, s);
    const reduce_arg<T> u{(const T*)p->B, (const T*)dY, lddy, p->M, nullptr, 0, nullptr,
                          dA ? ws + w.pack_u : nullptr};
    const reduce_arg<T> v{(const T*)p->A, (const T*)X, ldx, p->K, t, 1, nullptr, ws + w.pack_t};
    const expand_arg<T> e{(const T*)p->A, p->K, (const T*)base, ldb, (T*)dX, lddx};
    run_apply<T>(d, r, w, dX || dA, u, w.ksM, (float*)(ws + w.u), dB != nullptr, v, w.ksK,
                 (float*)(ws + w.t), e, mask, s);
  }
  if (!dA && !dB) return;
  grad_arg<T> qa{(const T*)X, ldx, p->K, ws + w.pack_u, (T*)dA, (float*)(ws + w.partA)};
  grad_arg<T> qb{(const T*)dY, lddy, p->M, ws + w.pack_t, (T*)dB, (float*)(ws + w.partB)};
  const int32_t na = dA ? w.blocksA : 0, nb = dB ? w.blocksB : 0;
  if (Tn > 0) {
    const int32_t nr = std::min(w.NT, 2), gw = grad_waves(nr);
    const dim3 grid((unsigned)(w.tw == 1 ? cdiv(na + nb, gw) : na + nb), w.slots,
                    (unsigned)cdiv(w.NT, nr));
    const size_t lds = w.tw == 1 ? 0 : 4 * (size_t)gw * 16 * 16 * EL<T>;
    auto kernel = nr == 1 ? k_lora_grad<T, 1> : k_lora_grad<T, 2>;
    hipLaunchKernelGGL(kernel, grid, dim3(gw * 64), lds, s, d, r, qa, qb, na, na + nb, w.tw, mask);
  }
  const int32_t slots = Tn > 0 ? w.slots : 0;
  if (Tn > 0 && w.whole <= w.slot_tiles) return;  // one slot for each
  // workgroups for about 2,048 of them to be under way, the adapters' alike
  auto shares = [&](int32_t F) {
    return (int32_t)std::min<int64_t>(cdiv((int64_t)p->R * F, 1024), cdiv(2048, p->L));
  };
  const int32_t ja = dA ? shares(p->K) : 0, jb = dB ? shares(p->M) : 0;
  hipLaunchKernelGGL(k_lora_join<T>, dim3((unsigned)p->L, ja + jb), dim3(256), 0, s, d, r, slots, qa,
                     qb, ja);
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_lora_workspace(const snack_lora* lora, snack_dtype dtype, int32_t T,
                                  int32_t backward, size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  if (snack_status st = check_lora(lora, dtype, T, backward != 0)) return st;
  *bytes = plan_of(lora, dtype, T, backward != 0).total;
  return SNACK_OK;
}

snack_status snack_lora_fwd(const snack_lora* lora, snack_dtype dtype, const int32_t* ids,
                            int32_t T, const void* X, int64_t ldx, const void* base, int64_t ldb,
                            void* Y, int64_t ldy, float* t, void* ws, size_t ws_bytes,
                            void* stream) {
  if (snack_status st = check_lora(lora, dtype, T, false)) return st;
  if (ldx < lora->K || ldy < lora->M || (base && ldb < lora->M)) return SNACK_E_SHAPE;
  if (T == 0) return SNACK_OK;
  if (!lora->A || !lora->B || !ids || !X || !Y || !ws) return SNACK_E_NULL;
  if (Y == X || (Y == base && ldy != ldb)) return SNACK_E_SHAPE;
  if (ws_bytes < plan_of(lora, dtype, T, false).total) return SNACK_E_WORKSPACE;
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4, M = lora->M, K = lora->K, L = lora->L, R = lora->R;
  const span_t out[] = {{Y, M * e, ldy * e, T}, {t, 4 * T * R}};
  const span_t in[] = {{X, K * e, ldx * e, T}, {Y == base ? nullptr : base, M * e, ldb * e, T},
                       {lora->A, L * R * K * e}, {lora->B, L * R * M * e},
                       {lora->scale, 4 * L}, {lora->rank, 4 * L}, {ids, 4 * (__int128)T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const lora_dev d{lora->L, lora->R, lora->scale, lora->rank};
  if (dtype == SNACK_BF16)
    run_fwd<bf16>(lora, d, ids, T, X, ldx, base, ldb, Y, ldy, t, (char*)ws, dtype, s);
  else
    run_fwd<float>(lora, d, ids, T, X, ldx, base, ldb, Y, ldy, t, (char*)ws, dtype, s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

snack_status snack_lora_bwd(const snack_lora* lora, snack_dtype dtype, const int32_t* ids,
                            const float* t, int32_t T, const void* X, int64_t ldx, const void* dY,
                            int64_t lddy, const void* base, int64_t ldb, void* dX, int64_t lddx,
                            void* dA, void* dB, void* ws, size_t ws_bytes, void* stream) {
  if (snack_status st = check_lora(lora, dtype, T, true)) return st;
  if (ldx < lora->K || lddy < lora->M || (dX && lddx < lora->K) || (base && ldb < lora->K))
    return SNACK_E_SHAPE;
  if (T > 0) {
    if (!lora->A || !lora->B || !ids || !X || !dY || !ws) return SNACK_E_NULL;
    if (dX && (dX == X || dX == dY || (dX == base && lddx != ldb))) return SNACK_E_SHAPE;
    if (ws_bytes < plan_of(lora, dtype, T, true).total) return SNACK_E_WORKSPACE;
  }
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4, M = lora->M, K = lora->K, L = lora->L, R = lora->R;
  const span_t out[] = {{dX, K * e, lddx * e, T}, {dA, L * R * K * e}, {dB, L * R * M * e}};
  const span_t in[] = {{X, K * e, ldx * e, T}, {dY, M * e, lddy * e, T},
                       {dX == base ? nullptr : base, K * e, ldb * e, T},
                       {lora->A, L * R * K * e}, {lora->B, L * R * M * e},
                       {lora->scale, 4 * L}, {lora->rank, 4 * L}, {ids, 4 * (__int128)T},
                       {t, 4 * T * R}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const lora_dev d{lora->L, lora->R, lora->scale, lora->rank};
  if (dtype == SNACK_BF16)
    run_bwd<bf16>(lora, d, ids, t, T, X, ldx, dY, lddy, base, ldb, dX, lddx, dA, dB, (char*)ws,
                  dtype, s);
  else
    run_bwd<float>(lora, d, ids, t, T, X, ldx, dY, lddy, base, ldb, dX, lddx, dA, dB, (char*)ws,
                   dtype, s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
