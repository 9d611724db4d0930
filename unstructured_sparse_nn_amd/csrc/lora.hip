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
// More tokens are brought into the order of their adapters (k_lora_route) and
// cut into tiles of TILE tokens of one adapter, which feed the matrix cores.
#include <algorithm>
#include <cstring>

#include "common.h"
#include "internal.h"

namespace snk {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int32_t TILE = 64;  // tokens of a tile
constexpr int32_t MAX_RANK = 256;
constexpr int32_t MAX_ADAPTERS = 8192;
constexpr int32_t MAX_FEATURES = 1 << 23;  // column blocks are a grid's y

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

// ------------------------------------------------------------- 16-byte pieces
// Rows start at any element, so pieces are loaded and stored without an
// alignment claim; the hardware takes a 16-byte access at any address.
template <typename T> constexpr int EL = 16 / sizeof(T);
template <typename T> struct __attribute__((aligned(16))) frag { T v[EL<T>]; };

template <typename T>
__device__ __forceinline__ frag<T> load_frag(const T* p) {
  frag<T> f;
  __builtin_memcpy(&f, p, 16);
  return f;
}
// The first n elements at p (n may be <= 0 or past a piece), zeros after them.
template <typename T>
__device__ __forceinline__ frag<T> load_frag(const T* p, int32_t n) {
  if (n >= EL<T>) return load_frag(p);
  frag<T> f{};
  for (int e = 0; e < EL<T> - 1; ++e)
    if (e < n) f.v[e] = p[e];
  return f;
}
template <typename T>
__device__ __forceinline__ void store_frag(T* p, const frag<T>& f, int32_t n) {
  if (n >= EL<T>) {
    __builtin_memcpy(p, &f, 16);
  } else {
    for (int e = 0; e < EL<T> - 1; ++e)
      if (e < n) p[e] = f.v[e];
  }
}

__device__ __forceinline__ f4 mma(const frag<bf16>& a, const frag<bf16>& b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                 __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// The four elements of a float piece are four steps of the 16x16x4 product:
// the order of the contraction is free as long as both sides share it.
__device__ __forceinline__ f4 mma(const frag<float>& a, const frag<float>& b, f4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
  return c;
}

// v as two bf16 parts, hi + lo: off by at most 2^-16 of v.
__device__ __forceinline__ void split_bf16(float v, bf16& hi, bf16& lo) {
  hi = f32_to_bf16(v);
  const float h = bf16_to_f32(hi);
  lo = fabsf(h) < __builtin_inff() ? f32_to_bf16(v - h) : (bf16)0;  // infinities, NaN: hi alone
}

// out[c] = column c of the 8 x 8 matrix whose row q is rows[q].
__device__ __forceinline__ void transpose8(const frag<bf16> (&rows)[8], frag<bf16> (&out)[8]) {
  uint32_t in[8][4], o[8][4];
  __builtin_memcpy(in, rows, sizeof(in));
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      o[2 * d][p] = __builtin_amdgcn_perm(in[2 * p + 1][d], in[2 * p][d], 0x05040100u);
      o[2 * d + 1][p] = __builtin_amdgcn_perm(in[2 * p + 1][d], in[2 * p][d], 0x07060302u);
    }
  __builtin_memcpy(out, o, sizeof(o));
}

// --------------------------------------------------------------- a few tokens
// One token per blockIdx.y; its eight waves split the ranks.
// PARTS & 1: t[i, j] = sum_k F0[a, j, k] X[i, k], kept in LDS (and stored to t
// if given).  PARTS & 2: Y[i, :] from t over 64 pieces of columns per
// workgroup.  With both parts one launch does the whole token, every workgroup
// of it computing t again.
constexpr int FEW_WAVES = 8;

template <typename T>
__device__ __forceinline__ float dot_frag(const frag<T>& a, const frag<T>& b, float acc) {
  vec<T, EL<T>> x, y;
  __builtin_memcpy(&x, &a, 16);
  __builtin_memcpy(&y, &b, 16);
  return dot_acc<T, EL<T>>(x, y, acc);
}

template <typename T, int PARTS>
__global__ __launch_bounds__(FEW_WAVES * 64) void k_lora_few(
    lora_dev d, const int32_t* __restrict__ ids, const T* __restrict__ A, int32_t K, const T* X,
    int64_t ldx, const T* __restrict__ B, int32_t M, const T* base, int64_t ldb, T* Y, int64_t ldy,
    float* t) {
  constexpr int E = EL<T>;
  __shared__ float ts[MAX_RANK];
  __shared__ float red[FEW_WAVES][64 * E];
  const int64_t i = blockIdx.y;
  const int32_t a = ids[i];
  const int w = threadIdx.x / 64, l = lane_id();
  const int32_t r = a >= 0 && a < d.L ? rank_of(d, a) : 0;
  const int32_t col = blockIdx.x * 64 * E + l * E;
  constexpr int RW = 4;  // ranks of a wave at a time
  if (PARTS & 1) {
    const int32_t j_of = PARTS == 1 ? blockIdx.x * FEW_WAVES * RW : 0;
    const int32_t j_end = PARTS == 1 ? min(j_of + FEW_WAVES * RW, d.R) : r;
    const T* x = X + i * ldx;
    for (int32_t j0 = j_of + w; j0 < j_end; j0 += FEW_WAVES * RW) {
      float acc[RW] = {};
      const T* f[RW];
#pragma unroll
      for (int q = 0; q < RW; ++q)
        f[q] = A + ((int64_t)max(a, 0) * d.R + min(j0 + q * FEW_WAVES, max(r - 1, 0))) * K;
      if (j0 < r) {
        int32_t k = l * E;
#pragma unroll 4
        for (; k + E <= K; k += 64 * E) {
          const frag<T> xv = load_frag(x + k);
#pragma unroll
          for (int q = 0; q < RW; ++q) acc[q] = dot_frag(xv, load_frag(f[q] + k), acc[q]);
        }
        if (k < K) {
          const frag<T> xv = load_frag(x + k, K - k);
#pragma unroll
          for (int q = 0; q < RW; ++q) acc[q] = dot_frag(xv, load_frag(f[q] + k, K - k), acc[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < RW; ++q) {
        const int32_t j = j0 + q * FEW_WAVES;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) acc[q] += __shfl_xor(acc[q], m, 64);
        if (l == 0 && j < (PARTS == 1 ? d.R : r)) {
          const float v = j < r ? acc[q] : 0.f;
          if (PARTS & 2) ts[j] = v;
          else t[i * d.R + j] = v;
        }
      }
    }
    if (!(PARTS & 2)) return;
  } else {
    for (int32_t j = threadIdx.x; j < r; j += FEW_WAVES * 64) ts[j] = t[i * d.R + j];
  }
  __syncthreads();
  if (PARTS == 3 && t && blockIdx.x == 0)
    for (int32_t j = threadIdx.x; j < d.R; j += FEW_WAVES * 64) t[i * d.R + j] = j < r ? ts[j] : 0.f;
  float y[E] = {};
  if (col < M) {
#pragma unroll 4
    for (int32_t j = w; j < r; j += FEW_WAVES) {
      const frag<T> bv = load_frag(B + ((int64_t)a * d.R + j) * M + col, M - col);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = fmaf(ts[j], elem<T>::to_f(bv.v[e]), y[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) red[w][l * E + e] = y[e];
  __syncthreads();
  const float s = a >= d.L ? __builtin_nanf("") : r > 0 ? scale_of(d, a) : 1.f;
  for (int32_t c = threadIdx.x; c < 64 * E; c += FEW_WAVES * 64) {
    const int32_t m = blockIdx.x * 64 * E + c;
    if (m >= M) break;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < FEW_WAVES; ++q) v += red[q][c];
    v *= s;
    if (base) v += elem<T>::to_f(base[i * ldb + m]);
    Y[i * ldy + m] = elem<T>::from_f(v);
  }
}

// ------------------------------------------------------- tokens in adapter order
// A tile is a run of up to TILE tokens of one adapter in that order; group L
// holds the tokens without an adapter.  A slot is a run of tiles of one
// adapter whose gradient one workgroup sums; the slots of an adapter that has
// several leave partial sums at `part`, part + 1, ...
struct tile_t { int32_t l, begin, n, pad; };
struct slot_t { int32_t l, tile, n, part; };  // part < 0: the adapter's only slot
struct join_t { int32_t slots, part; };

struct route_t {
  const int32_t* ids;
  int32_t Tn;
  int32_t slot_tiles;      // tiles of a slot
  const int32_t* order;    // NULL: one adapter, tokens in their own order
  const tile_t* tile;
  const slot_t* slot;
  const join_t* join;      // [L]
  const int32_t* count;    // tiles, slots
};

__device__ __forceinline__ tile_t tile_at(const route_t& p, int32_t i) {
  if (p.order) return i < p.count[0] ? p.tile[i] : tile_t{0, 0, 0, 0};
  return tile_t{0, i * TILE, min(TILE, p.Tn - i * TILE), 0};
}
__device__ __forceinline__ slot_t slot_at(const route_t& p, int32_t i) {
  if (p.order) return i < p.count[1] ? p.slot[i] : slot_t{0, 0, 0, 0};
  const int32_t tiles = (p.Tn + TILE - 1) / TILE;
  return slot_t{0, i * p.slot_tiles, min(p.slot_tiles, tiles - i * p.slot_tiles),
                tiles > p.slot_tiles ? i : -1};
}
__device__ __forceinline__ int32_t row_at(const route_t& p, int32_t i) {
  return p.order ? p.order[i] : i;
}
// Whether token `row` of a tile of adapter l has that adapter (tokens in their
// own order may have none).
__device__ __forceinline__ bool has_adapter(const route_t& p, int32_t L, int32_t l, int32_t row) {
  return p.order ? l < L : p.ids[row] == 0;
}

// Stable counting sort of the tokens by adapter, then the tables of tiles and
// slots, in one workgroup: wave w < nw walks its own run of tokens, once to
// count and once to place; lanes that hold the same adapter find each other by
// one ballot per bit.
__global__ __launch_bounds__(1024) void k_lora_route(const int32_t* __restrict__ ids, int32_t Tn,
                                                     int32_t L, int32_t nw, int32_t slot_tiles,
                                                     int32_t* __restrict__ order,
                                                     tile_t* __restrict__ tile,
                                                     slot_t* __restrict__ slot,
                                                     join_t* __restrict__ join,
                                                     int32_t* __restrict__ count) {
  extern __shared__ int32_t cnt[];  // [nw][L + 1]
  __shared__ int32_t lds[16];
  const int32_t G = L + 1;
  const int w = threadIdx.x / 64, l = lane_id();
  for (int32_t i = threadIdx.x; i < nw * G; i += 1024) cnt[i] = 0;
  __syncthreads();
  const int32_t run = ((Tn + nw - 1) / nw + 63) / 64 * 64;
  const int64_t i0 = (int64_t)w * run, i1 = min(i0 + run, (int64_t)Tn);
  const int bits = 32 - __builtin_clz(L);
  auto walk = [&](bool place) {
    if (w >= nw) return;
    int32_t* mine = cnt + w * G;
    for (int64_t b = i0; b < i1; b += 64) {
      const bool in = b + l < i1;
      const int32_t id = in ? ids[b + l] : 0;
      const int32_t g = id >= 0 && id < L ? id : L;
      uint64_t peers = __ballot(in);
      for (int k = 0; k < bits; ++k) {
        const uint64_t m = __ballot((g >> k) & 1);
        peers &= ((g >> k) & 1) ? m : ~m;
      }
      const int before = __popcll(peers & lanemask_lt());
      int32_t at = 0;
      if (in) at = mine[g] + before;
      if (place && in) order[at] = (int32_t)(b + l);
      __builtin_amdgcn_wave_barrier();
      if (in && before == 0) mine[g] = at + __popcll(peers);
      __builtin_amdgcn_wave_barrier();
    }
  };
  walk(false);
  __syncthreads();
  int32_t tok = 0, til = 0, slo = 0, par = 0;  // totals of the groups so far
  for (int32_t g0 = 0; g0 < G; g0 += 1024) {
    const int32_t g = g0 + threadIdx.x;
    int32_t n = 0;
    if (g < G)
      for (int32_t q = 0; q < nw; ++q) n += cnt[q * G + g];
    const int32_t nt = (n + TILE - 1) / TILE;
    const int32_t ns = g < L ? (nt + slot_tiles - 1) / slot_tiles : 0;
    const int32_t np = ns > 1 ? ns : 0;
    int32_t total;
    int32_t b = block_excl_scan_i32<1024>(n, lds, &total) + tok;
    tok += total;
    const int32_t bt = block_excl_scan_i32<1024>(nt, lds, &total) + til;
    til += total;
    const int32_t bs = block_excl_scan_i32<1024>(ns, lds, &total) + slo;
    slo += total;
    const int32_t bp = block_excl_scan_i32<1024>(np, lds, &total) + par;
    par += total;
    if (g < G) {
      for (int32_t k = 0; k < nt; ++k)
        tile[bt + k] = tile_t{g, b + k * TILE, min(TILE, n - k * TILE), 0};
      for (int32_t k = 0; k < ns; ++k)
        slot[bs + k] = slot_t{g, bt + k * slot_tiles, min(slot_tiles, nt - k * slot_tiles),
                              ns > 1 ? bp + k : -1};
      if (g < L) join[g] = join_t{ns, bp};
      for (int32_t q = 0; q < nw; ++q) {
        const int32_t c = cnt[q * G + g];
        cnt[q * G + g] = b;
        b += c;
      }
    }
  }
  if (threadIdx.x == 0) {
    count[0] = til;
    count[1] = slo;
  }
  __syncthreads();
  walk(true);
}

// ------------------------------------------------------------------- reduce
// out[ks][i][j] = the part of sum_k F[a, j, k] X[i, k] that this workgroup's
// range of k gives; the ks parts are summed where they are read.  A wave takes
// its own range of k and all tokens and ranks of the tile: both operands of
// the 16x16 products are rows that lie contiguous along the contraction, so
// each lane loads its operand from memory as it is.
template <typename T>
struct reduce_arg {
  const T* F;
  const T* X;
  int64_t ldx;
  int32_t K;
  int32_t ks;   // parts
  float* out;   // [ks][Tn][R]
};

constexpr int RED_WAVES = 8;

template <typename T, int RT, int NR>
__device__ __forceinline__ void reduce_tile(const lora_dev& d, const route_t& p,
                                            const reduce_arg<T>& q, const tile_t& tl, int32_t r,
                                            int32_t rb, float (*red)[TILE * 16]) {
  constexpr int KS = 4 * EL<T>;  // contraction of a step
  const int w = threadIdx.x / 64, l = lane_id(), c = l & 15, g = l >> 4;
  const T* x[RT];
  const T* f[NR];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    x[i] = q.X + (int64_t)row_at(p, tl.begin + min(i * 16 + c, tl.n - 1)) * q.ldx + g * EL<T>;
#pragma unroll
  for (int j = 0; j < NR; ++j)  // rows past the rank: results not used
    f[j] = q.F + ((int64_t)tl.l * d.R + min(rb + j * 16 + c, r - 1)) * q.K + g * EL<T>;
  f4 acc[RT][NR];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NR; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  const int64_t steps = (q.K + KS - 1) / KS, n = (int64_t)q.ks * RED_WAVES;
  const int64_t at = (int64_t)blockIdx.y * RED_WAVES + w;
  const int32_t s0 = (int32_t)(steps * at / n), s1 = (int32_t)(steps * (at + 1) / n);
  const int32_t full = min(s1, q.K / KS);
#pragma unroll 4
  for (int32_t s = s0; s < full; ++s) {
    frag<T> xv[RT], fv[NR];
#pragma unroll
    for (int i = 0; i < RT; ++i) xv[i] = load_frag(x[i] + (int64_t)s * KS);
#pragma unroll
    for (int j = 0; j < NR; ++j) fv[j] = load_frag(f[j] + (int64_t)s * KS);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[i][j] = mma(xv[i], fv[j], acc[i][j]);
  }
  if (full < s1) {  // the step that ends past K
    const int32_t left = q.K - full * KS - g * EL<T>;
    frag<T> xv[RT], fv[NR];
#pragma unroll
    for (int i = 0; i < RT; ++i) xv[i] = load_frag(x[i] + (int64_t)full * KS, left);
#pragma unroll
    for (int j = 0; j < NR; ++j) fv[j] = load_frag(f[j] + (int64_t)full * KS, left);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[i][j] = mma(xv[i], fv[j], acc[i][j]);
  }
  float* out = q.out + (int64_t)blockIdx.y * p.Tn * d.R;
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    if (rb + j * 16 >= d.R) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[w][(i * 16 + 4 * g + e) * 16 + c] = acc[i][j][e];
    __syncthreads();
    for (int32_t k = threadIdx.x; k < RT * 256; k += RED_WAVES * 64) {
      const int32_t tok = k / 16, rank = rb + j * 16 + k % 16;
      if (tok >= tl.n || rank >= d.R) continue;
      float v = 0.f;
#pragma unroll
      for (int m = 0; m < RED_WAVES; ++m) v += red[m][k];
      const int32_t row = row_at(p, tl.begin + tok);
      out[(int64_t)row * d.R + rank] = rank < r && has_adapter(p, d.L, tl.l, row) ? v : 0.f;
    }
  }
}

// grid: tiles x parts x (problems * rank blocks of 16 * NR)
template <typename T, int NR>
__global__ __launch_bounds__(RED_WAVES * 64) void k_lora_reduce(lora_dev d, route_t p,
                                                                reduce_arg<T> q0,
                                                                reduce_arg<T> q1,
                                                                int32_t rank_blocks) {
  __shared__ float red[RED_WAVES][TILE * 16];
  const reduce_arg<T> q = (int32_t)blockIdx.z < rank_blocks ? q0 : q1;
  const int32_t rb = (int32_t)blockIdx.z % rank_blocks * 16 * NR;
  if ((int32_t)blockIdx.y >= q.ks) return;
  const tile_t tl = tile_at(p, blockIdx.x);
  if (tl.n <= 0) return;
  const int32_t r = tl.l < d.L ? rank_of(d, tl.l) : 0;
  if (rb >= r) {  // nothing of this adapter's here: zeros
    float* out = q.out + (int64_t)blockIdx.y * p.Tn * d.R;
    const int32_t n = min(16 * NR, d.R - rb);
    for (int32_t k = threadIdx.x; k < tl.n * n; k += RED_WAVES * 64)
      out[(int64_t)row_at(p, tl.begin + k / n) * d.R + rb + k % n] = 0.f;
    return;
  }
  if (tl.n <= 16) reduce_tile<T, 1, NR>(d, p, q, tl, r, rb, red);
  else reduce_tile<T, 4, NR>(d, p, q, tl, r, rb, red);
}

// ------------------------------------------------------------------- expand
// Y[i, m] = base[i, m] + s sum_j t[i, j] F[a, j, m] for a tile and 4 waves'
// columns.  t is staged in LDS as the products' operand: for bf16 in two parts
// (hi + lo, whose products sum to fp32's accuracy), for fp32 as it is.  The
// factor's rows lie along m, so a lane's pieces of 8 rows are transposed in
// registers into 8 operands of 8 ranks each; the results leave each lane with
// EL columns side by side, one 16-byte piece of base in and one of Y out.
constexpr int EXP_WAVES = 4;
enum { ROW_NONE = 0, ROW_HAS = 1, ROW_BAD = 2 };

template <typename T> struct expand_lds;
template <> struct expand_lds<bf16> {
  static size_t bytes(int32_t R) { return (size_t)cdiv(R, 32) * 4 * 2 * 64 * 16; }
};
template <> struct expand_lds<float> {
  static size_t bytes(int32_t R) { return (size_t)TILE * (cdiv(R, 4) * 4 + 1) * 4; }
};

// t of token `row` at rank j, all parts summed.
__device__ __forceinline__ float t_sum(const float* __restrict__ t, int64_t at, int64_t part,
                                       int32_t ks) {
  float v = t[at];
  for (int32_t k = 1; k < ks; ++k) v += t[at + k * part];
  return v;
}

template <typename T, int RT>
__device__ __forceinline__ void expand_acc(const T* __restrict__ F, int32_t M, int32_t r,
                                           int32_t R, int32_t col, const char* op,
                                           f4 (&acc)[RT][EL<T>]) {
  const int l = lane_id(), c = l & 15, g = l >> 4;
  if constexpr (sizeof(T) == 2) {
    const frag<bf16>* o = reinterpret_cast<const frag<bf16>*>(op);
    for (int32_t rs = 0; rs * 32 < r; ++rs) {
      frag<T> rows[8], cols[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int32_t j = rs * 32 + 8 * g + q;
        rows[q] = load_frag(F + (int64_t)j * M + col, j < r ? M - col : 0);
      }
      transpose8(rows, cols);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const frag<T> hi = o[((rs * 4 + i) * 2 + 0) * 64 + l], lo = o[((rs * 4 + i) * 2 + 1) * 64 + l];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = mma(lo, cols[e], mma(hi, cols[e], acc[i][e]));
      }
    }
  } else {
    const float* ts = reinterpret_cast<const float*>(op);
    const int32_t ld = (R + 3) / 4 * 4 + 1;
#pragma unroll 4
    for (int32_t q = 0; q < r; q += 4) {
      const int32_t j = q + g;
      const frag<T> row = load_frag(F + (int64_t)j * M + col, j < r ? M - col : 0);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float tv = ts[(i * 16 + c) * ld + j];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(tv, row.v[e], acc[i][e], 0, 0, 0);
      }
    }
  }
}

template <typename T, int RT>
__device__ __forceinline__ void expand_tile(const lora_dev& d, const T* F, int32_t M, int32_t r,
                                            const tile_t& tl, const char* op, const int32_t* rows,
                                            const int8_t* kind, const T* base, int64_t ldb, T* Y,
                                            int64_t ldy) {
  constexpr int E = EL<T>;
  const int l = lane_id(), c = l & 15, g = l >> 4;
  const int32_t col = (blockIdx.y * EXP_WAVES + threadIdx.x / 64) * 16 * E + c * E;
  f4 acc[RT][E];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[i][e] = f4{0.f, 0.f, 0.f, 0.f};
  if (r > 0) expand_acc<T, RT>(F + (int64_t)tl.l * d.R * M, M, r, d.R, col, op, acc);
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t tok = i * 16 + 4 * g + k;
      if (tok >= tl.n || col >= M) continue;
      const int64_t row = rows[tok];
      const int8_t has = kind[tok];
      frag<T> bv{}, out;
      if (base) bv = load_frag(base + row * ldb + col, M - col);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float v = has == ROW_HAS ? acc[i][e][k] : has == ROW_NONE ? 0.f : __builtin_nanf("");
        if (base) v += elem<T>::to_f(bv.v[e]);
        out.v[e] = elem<T>::from_f(v);
      }
      store_frag(Y + row * ldy + col, out, M - col);
    }
}

// grid: tiles x columns of EXP_WAVES waves.  t: ks parts; t_out (nullable)
// receives their sum.
template <typename T>
__global__ __launch_bounds__(EXP_WAVES * 64, 2) void k_lora_expand(
    lora_dev d, route_t p, const T* __restrict__ F, int32_t M, const float* __restrict__ t,
    int32_t ks, float* __restrict__ t_out, const T* base, int64_t ldb, T* Y, int64_t ldy) {
  extern __shared__ char op[];
  __shared__ int32_t rows[TILE];
  __shared__ int8_t kind[TILE];
  const tile_t tl = tile_at(p, blockIdx.x);
  if (tl.n <= 0) return;
  const int32_t r = tl.l < d.L ? rank_of(d, tl.l) : 0;
  if (threadIdx.x < TILE) {
    const int32_t tok = threadIdx.x;
    const int32_t row = row_at(p, tl.begin + min(tok, tl.n - 1));
    rows[tok] = row;
    kind[tok] = tok >= tl.n ? ROW_NONE
                : has_adapter(p, d.L, tl.l, row) ? ROW_HAS
                : p.ids[row] >= d.L ? ROW_BAD : ROW_NONE;
  }
  __syncthreads();
  const int64_t part = (int64_t)p.Tn * d.R;
  const float s = r > 0 ? scale_of(d, tl.l) : 0.f;
  if constexpr (sizeof(T) == 2) {
    frag<bf16>* o = reinterpret_cast<frag<bf16>*>(op);
    const int32_t steps = (r + 31) / 32;
    for (int32_t k = threadIdx.x; k < steps * 4 * 64; k += EXP_WAVES * 64) {
      const int32_t l = k & 63, i = (k >> 6) & 3, rs = k >> 8;
      const int32_t tok = i * 16 + (l & 15), j0 = rs * 32 + 8 * (l >> 4);
      frag<bf16> hi{}, lo{};
      if (tok < tl.n && kind[tok] == ROW_HAS)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (j0 + e >= r) break;
          split_bf16(s * t_sum(t, (int64_t)rows[tok] * d.R + j0 + e, part, ks), hi.v[e], lo.v[e]);
        }
      o[((rs * 4 + i) * 2 + 0) * 64 + l] = hi;
      o[((rs * 4 + i) * 2 + 1) * 64 + l] = lo;
    }
  } else {
    float* ts = reinterpret_cast<float*>(op);
    const int32_t ld = (d.R + 3) / 4 * 4 + 1, n = (r + 3) / 4 * 4;
    for (int32_t k = threadIdx.x; k < n * TILE; k += EXP_WAVES * 64) {
      const int32_t tok = k / n, j = k % n;
      ts[tok * ld + j] = j < r && tok < tl.n && kind[tok] == ROW_HAS
                             ? s * t_sum(t, (int64_t)rows[tok] * d.R + j, part, ks) : 0.f;
    }
  }
  if (t_out && blockIdx.y == 0)
    for (int32_t k = threadIdx.x; k < tl.n * d.R; k += EXP_WAVES * 64) {
      const int64_t at = (int64_t)rows[k / d.R] * d.R + k % d.R;
      t_out[at] = t_sum(t, at, part, ks);
    }
  __syncthreads();
  if (tl.n <= 16) expand_tile<T, 1>(d, F, M, r, tl, op, rows, kind, base, ldb, Y, ldy);
  else expand_tile<T, 4>(d, F, M, r, tl, op, rows, kind, base, ldb, Y, ldy);
}

// --------------------------------------------------------------------- grad
// The scaled t (or u) of a tile as the operand of the products over tokens:
//   bf16  pack[tile][half][rank tile][hi, lo][lane] pieces of 8 tokens
//   fp32  pack[tile][token][ranks up to a multiple of 16]
// zero for tokens and ranks that are not there.  full[tile][half]: whether all
// 32 tokens of the half count.
template <typename T>
__global__ __launch_bounds__(256) void k_lora_pack(lora_dev d, route_t p,
                                                   const float* __restrict__ t0, int32_t ks0,
                                                   void* __restrict__ pack0,
                                                   const float* __restrict__ t1, int32_t ks1,
                                                   void* __restrict__ pack1,
                                                   int32_t* __restrict__ full) {
  __shared__ int32_t rows[TILE];  // -1: does not count
  const tile_t tl = tile_at(p, blockIdx.x);
  if (tl.n <= 0 || tl.l >= d.L) return;
  const bool first = blockIdx.y == 0;
  const float* t = first ? t0 : t1;
  const int32_t ks = first ? ks0 : ks1;
  if (!t) return;
  const int32_t r = rank_of(d, tl.l), NT = (d.R + 15) / 16;
  const float s = scale_of(d, tl.l);
  if (threadIdx.x < TILE) {
    const int32_t tok = threadIdx.x;
    int32_t row = -1;
    if (tok < tl.n) {
      row = row_at(p, tl.begin + tok);
      if (!has_adapter(p, d.L, tl.l, row)) row = -1;
    }
    rows[tok] = row;
    const uint64_t ok = __ballot(row >= 0);
    if ((tok & 31) == 0)
      full[blockIdx.x * 2 + tok / 32] = (uint32_t)(ok >> tok) == 0xFFFFFFFFu;
  }
  __syncthreads();
  const int64_t part = (int64_t)p.Tn * d.R;
  if constexpr (sizeof(T) == 2) {
    frag<bf16>* o = reinterpret_cast<frag<bf16>*>(first ? pack0 : pack1) +
                    (int64_t)blockIdx.x * 2 * NT * 2 * 64;
    for (int32_t k = threadIdx.x; k < 2 * NT * 64; k += 256) {
      const int32_t l = k & 63, x = k >> 6, j = x % NT * 16 + (l & 15), h = x / NT;
      frag<bf16> hi{}, lo{};
      if (j < r)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int32_t row = rows[h * 32 + 8 * (l >> 4) + q];
          if (row >= 0)
            split_bf16(s * t_sum(t, (int64_t)row * d.R + j, part, ks), hi.v[q], lo.v[q]);
        }
      o[(x * 2 + 0) * 64 + l] = hi;
      o[(x * 2 + 1) * 64 + l] = lo;
    }
  } else {
    float* o = reinterpret_cast<float*>(first ? pack0 : pack1) +
               (int64_t)blockIdx.x * TILE * NT * 16;
    for (int32_t k = threadIdx.x; k < TILE * NT * 16; k += 256) {
      const int32_t tok = k / (NT * 16), j = k % (NT * 16), row = rows[tok];
      o[k] = row >= 0 && j < r ? s * t_sum(t, (int64_t)row * d.R + j, part, ks) : 0.f;
    }
  }
}

template <typename T>
struct grad_arg {
  const T* X;
  int64_t ldx;
  int32_t K;
  const void* pack;
  T* dF;
  float* part;  // [partial slots][R][K]
};

constexpr int GRAD_WAVES = 4;

// grid: column blocks (of X, then of dY) x slots x rank blocks of 16 * NR.
// A wave takes every fourth half tile of the slot: 32 tokens, 16 pieces of
// columns; the tokens are the contraction, so (bf16) the lane's pieces of 8
// tokens are transposed in registers into operands.  The waves' sums meet in
// LDS.
template <typename T, int NR>
__global__ __launch_bounds__(GRAD_WAVES * 64, 2) void k_lora_grad(lora_dev d, route_t p,
                                                                  grad_arg<T> q0, grad_arg<T> q1,
                                                                  int32_t blocks0,
                                                                  const int32_t* __restrict__ full) {
  constexpr int E = EL<T>, CW = 16 * E;
  __shared__ float red[GRAD_WAVES][16 * CW];
  const bool first = (int32_t)blockIdx.x < blocks0;
  const grad_arg<T> q = first ? q0 : q1;
  const slot_t sl = slot_at(p, blockIdx.y);
  if (sl.n <= 0) return;
  const int w = threadIdx.x / 64, l = lane_id(), c = l & 15, g = l >> 4;
  const int32_t c0 = ((int32_t)blockIdx.x - (first ? 0 : blocks0)) * CW, col = c0 + c * E;
  const int32_t NT = (d.R + 15) / 16, rt0 = blockIdx.z * NR;
  f4 acc[NR][E];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[j][e] = f4{0.f, 0.f, 0.f, 0.f};
  for (int32_t h = w; h < sl.n * 2; h += GRAD_WAVES) {
    const int32_t ti = sl.tile + h / 2, half = h & 1;
    const tile_t tl = tile_at(p, ti);
    if (half * 32 >= tl.n) continue;
    const bool whole = full[ti * 2 + half] != 0;
    frag<T> rows[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int32_t tok = half * 32 + 8 * g + k;
      const int32_t row = row_at(p, tl.begin + min(tok, tl.n - 1));
      int32_t n = q.K - col;
      if (!whole && (tok >= tl.n || !has_adapter(p, d.L, sl.l, row))) n = 0;
      rows[k] = load_frag(q.X + (int64_t)row * q.ldx + col, n);
    }
    if constexpr (sizeof(T) == 2) {
      frag<T> cols[8];
      transpose8(rows, cols);
      const frag<bf16>* o = reinterpret_cast<const frag<bf16>*>(q.pack) +
                            ((int64_t)(ti * 2 + half) * NT) * 2 * 64 + l;
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        if (rt0 + j >= NT) break;
        const frag<T> hi = o[((rt0 + j) * 2 + 0) * 64], lo = o[((rt0 + j) * 2 + 1) * 64];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j][e] = mma(lo, cols[e], mma(hi, cols[e], acc[j][e]));
      }
    } else {
      const float* o = reinterpret_cast<const float*>(q.pack) +
                       ((int64_t)ti * TILE + half * 32 + 8 * g) * NT * 16 + c;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          if (rt0 + j >= NT) break;
          const float u = o[(k * NT + rt0 + j) * 16];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[j][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(u, rows[k].v[e], acc[j][e], 0, 0, 0);
        }
    }
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    if (rt0 + j >= NT) break;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) red[w][(4 * g + k) * CW + c * E + e] = acc[j][e][k];
    __syncthreads();
    const int32_t rank = (rt0 + j) * 16 + (int32_t)threadIdx.x / 16;
    const int32_t at = threadIdx.x / 16 * CW + threadIdx.x % 16 * E, m = c0 + threadIdx.x % 16 * E;
    if (rank < d.R && m < q.K) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[e] = (red[0][at + e] + red[1][at + e]) + (red[2][at + e] + red[3][at + e]);
      if (sl.part < 0) {
        frag<T> out;
#pragma unroll
        for (int e = 0; e < E; ++e) out.v[e] = elem<T>::from_f(v[e]);
        store_frag(q.dF + ((int64_t)sl.l * d.R + rank) * q.K + m, out, q.K - m);
      } else {
        float* o = q.part + ((int64_t)sl.part * d.R + rank) * q.K + m;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (m + e < q.K) o[e] = v[e];
      }
    }
  }
}

// The gradients of adapters without a slot (zeros) or with several (the sum of
// their partial sums, in slot order).  grid: (adapter, rank) x column blocks.
template <typename T>
__global__ __launch_bounds__(256) void k_lora_join(lora_dev d, route_t p, int32_t slots,
                                                   grad_arg<T> q0, grad_arg<T> q1,
                                                   int32_t blocks0) {
  const bool first = (int32_t)blockIdx.y < blocks0;
  const grad_arg<T> q = first ? q0 : q1;
  const int32_t l = blockIdx.x / d.R, j = blockIdx.x % d.R;
  const int32_t m = (((int32_t)blockIdx.y - (first ? 0 : blocks0)) * 256 + threadIdx.x) * 4;
  const join_t jn = p.order ? p.join[l] : join_t{slots, 0};
  if (m >= q.K || jn.slots == 1) return;
  const int32_t n = min(4, q.K - m);
  float v[4] = {};
  const float* o = q.part + ((int64_t)jn.part * d.R + j) * q.K + m;
  for (int32_t s = 0; s < jn.slots; ++s, o += (int64_t)d.R * q.K)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) v[e] += o[e];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) q.dF[((int64_t)l * d.R + j) * q.K + m + e] = elem<T>::from_f(v[e]);
}

// --------------------------------------------------------------------- host
snack_status check_lora(const snack_lora* p, snack_dtype dt, int32_t T) {
  if (!p) return SNACK_E_NULL;
  if (dt != SNACK_F32 && dt != SNACK_BF16) return SNACK_E_DTYPE;
  if (p->M < 1 || p->K < 1 || p->L < 1 || p->L > MAX_ADAPTERS || p->R < 1 || p->R > MAX_RANK ||
      T < 0)
    return SNACK_E_SHAPE;
  if (T > INT32_MAX - TILE || p->M > MAX_FEATURES || p->K > MAX_FEATURES) return SNACK_E_OVERFLOW;
  return SNACK_OK;
}

// Tokens up to which k_lora_few is taken.
constexpr int32_t FEW_TOKENS = 64;

struct plan_t {
  int32_t tiles, slots, slot_tiles, part_slots, blocksA, blocksB, NT;
  int32_t ksK, ksM;  // parts of the reductions over K and over M
  size_t order, tile, slot, join, count, t, u, pack_t, pack_u, full, partA, partB, total;
};

int32_t parts_of(int32_t tiles, int32_t K, int32_t step) {
  const int64_t want = cdiv(256, std::max(tiles, 1)), most = std::max<int64_t>(1, K / (RED_WAVES * 2 * step));
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>({want, most, 8}));
}

plan_t plan_of(const snack_lora* p, snack_dtype dt, int32_t T, bool backward) {
  plan_t w{};
  const int32_t e = dt == SNACK_BF16 ? 8 : 4;
  const int32_t whole = (int32_t)cdiv(T, TILE);
  w.tiles = p->L == 1 ? whole : (int32_t)std::min<int64_t>(T, (int64_t)T / TILE + p->L + 1);
  w.ksK = parts_of(whole, p->K, 4 * e);
  w.ksM = parts_of(whole, p->M, 4 * e);
  w.NT = (int32_t)cdiv(p->R, 16);
  w.blocksA = (int32_t)cdiv(p->K, 16 * e);
  w.blocksB = (int32_t)cdiv(p->M, 16 * e);
  // slots: enough workgroups to fill the GPU, each of at least 4 tiles
  const int64_t runs = std::max<int64_t>(1, cdiv(512, w.blocksA + w.blocksB));
  w.slot_tiles = (int32_t)std::max<int64_t>(4, cdiv(whole, runs));
  w.slots = p->L == 1 ? (int32_t)cdiv(whole, w.slot_tiles)
                      : (int32_t)std::min<int64_t>(w.tiles, whole / w.slot_tiles + p->L);
  // an adapter with several slots has more than slot_tiles tiles, so its
  // slots are at most three times its share of the tokens
  w.part_slots = p->L == 1 ? w.slots
                           : (int32_t)std::min<int64_t>(w.slots, 3 * cdiv(whole, w.slot_tiles));
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o = align_up(o + b, 256);
    return at;
  };
  if (p->L > 1) {
    w.order = take(4 * (size_t)T);
    w.tile = take(sizeof(tile_t) * (size_t)w.tiles);
    w.slot = take(sizeof(slot_t) * (size_t)w.slots);
    w.join = take(sizeof(join_t) * (size_t)p->L);
    w.count = take(8);
  }
  const size_t tr = 4 * (size_t)T * p->R;
  w.t = take(tr * w.ksK);
  if (backward) {
    w.u = take(tr * w.ksM);
    const size_t pk = 4 * (size_t)w.tiles * TILE * w.NT * 16;
    w.pack_t = take(pk);
    w.pack_u = take(pk);
    w.full = take(8 * (size_t)w.tiles);
    w.partA = take(4 * (size_t)w.part_slots * p->R * p->K);
    w.partB = take(4 * (size_t)w.part_slots * p->R * p->M);
  }
  w.total = std::max<size_t>(o, 256);
  return w;
}

route_t launch_route(const snack_lora* p, const plan_t& w, const int32_t* ids, int32_t T, char* ws,
                     hipStream_t s) {
  route_t r{ids, T, w.slot_tiles, nullptr, nullptr, nullptr, nullptr, nullptr};
  if (p->L == 1) return r;
  r.order = (const int32_t*)(ws + w.order);
  r.tile = (const tile_t*)(ws + w.tile);
  r.slot = (const slot_t*)(ws + w.slot);
  r.join = (const join_t*)(ws + w.join);
  r.count = (const int32_t*)(ws + w.count);
  const int32_t nw = std::max(1, std::min(16, 15360 / (p->L + 1)));
  hipLaunchKernelGGL(k_lora_route, dim3(1), dim3(1024), 4 * (size_t)nw * (p->L + 1), s, ids, T,
                     p->L, nw, w.slot_tiles, (int32_t*)r.order, (tile_t*)r.tile, (slot_t*)r.slot,
                     (join_t*)r.join, (int32_t*)r.count);
  return r;
}

template <typename T>
void launch_reduce(const lora_dev& d, const route_t& r, const plan_t& w, const reduce_arg<T>& q0,
                   const reduce_arg<T>& q1, int32_t problems, hipStream_t s) {
  const int32_t nr = w.NT >= 3 ? 4 : w.NT, rbs = (int32_t)cdiv(w.NT, nr);
  const dim3 grid(w.tiles, problems > 1 ? std::max(q0.ks, q1.ks) : q0.ks, rbs * problems);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(RED_WAVES * 64), 0, s, d, r, q0, q1, rbs);
  };
  if (nr == 1) go(k_lora_reduce<T, 1>);
  else if (nr == 2) go(k_lora_reduce<T, 2>);
  else go(k_lora_reduce<T, 4>);
}

template <typename T>
void launch_expand(const lora_dev& d, const route_t& r, const plan_t& w, const void* F, int32_t M,
                   const float* t, int32_t ks, float* t_out, const void* base, int64_t ldb,
                   void* Y, int64_t ldy, hipStream_t s) {
  const dim3 grid(w.tiles, (unsigned)cdiv(M, EXP_WAVES * 16 * EL<T>));
  hipLaunchKernelGGL(k_lora_expand<T>, grid, dim3(EXP_WAVES * 64), expand_lds<T>::bytes(d.R), s, d,
                     r, (const T*)F, M, t, ks, t_out, (const T*)base, ldb, (T*)Y, ldy);
}

template <typename T>
void run_fwd(const snack_lora* p, const lora_dev& d, const int32_t* ids, int32_t Tn, const void* X,
             int64_t ldx, const void* base, int64_t ldb, void* Y, int64_t ldy, float* t, char* ws,
             snack_dtype dt, hipStream_t s) {
  if (Tn <= FEW_TOKENS) {
    const dim3 grid((unsigned)cdiv(p->M, 64 * EL<T>), Tn);
    hipLaunchKernelGGL((k_lora_few<T, 3>), grid, dim3(FEW_WAVES * 64), 0, s, d, ids, (const T*)p->A,
                       p->K, (const T*)X, ldx, (const T*)p->B, p->M, (const T*)base, ldb, (T*)Y,
                       ldy, t);
    return;
  }
  const plan_t w = plan_of(p, dt, Tn, false);
  const route_t r = launch_route(p, w, ids, Tn, ws, s);
  float* parts = (float*)(ws + w.t);
  const reduce_arg<T> q{(const T*)p->A, (const T*)X, ldx, p->K, w.ksK, parts};
  launch_reduce<T>(d, r, w, q, q, 1, s);
  launch_expand<T>(d, r, w, p->B, p->M, parts, w.ksK, t, base, ldb, Y, ldy, s);
}

template <typename T>
void run_bwd(const snack_lora* p, const lora_dev& d, const int32_t* ids, const float* t,
             int32_t Tn, const void* X, int64_t ldx, const void* dY, int64_t lddy,
             const void* base, int64_t ldb, void* dX, int64_t lddx, void* dA, void* dB, char* ws,
             snack_dtype dt, hipStream_t s) {
  const plan_t w = plan_of(p, dt, Tn, true);
  route_t r{};
  float *tp = (float*)(ws + w.t), *up = (float*)(ws + w.u);
  if (Tn > 0) {
    r = launch_route(p, w, ids, Tn, ws, s);
    const reduce_arg<T> qt{(const T*)p->A, (const T*)X, ldx, p->K, w.ksK, tp};
    const reduce_arg<T> qu{(const T*)p->B, (const T*)dY, lddy, p->M, w.ksM, up};
    const bool need_u = dX || dA, need_t = dB && !t;
    if (need_u && need_t) launch_reduce<T>(d, r, w, qu, qt, 2, s);
    else if (need_u) launch_reduce<T>(d, r, w, qu, qu, 1, s);
    else if (need_t) launch_reduce<T>(d, r, w, qt, qt, 1, s);
    if (dX) launch_expand<T>(d, r, w, p->A, p->K, up, w.ksM, nullptr, base, ldb, dX, lddx, s);
  }
  if (!dA && !dB) return;
  int32_t* full = (int32_t*)(ws + w.full);
  grad_arg<T> qa{(const T*)X, ldx, p->K, ws + w.pack_u, (T*)dA, (float*)(ws + w.partA)};
  grad_arg<T> qb{(const T*)dY, lddy, p->M, ws + w.pack_t, (T*)dB, (float*)(ws + w.partB)};
  const int32_t na = dA ? w.blocksA : 0, nb = dB ? w.blocksB : 0;
  if (Tn > 0) {
    const float* t_src = dB ? (t ? t : tp) : nullptr;
    hipLaunchKernelGGL(k_lora_pack<T>, dim3(w.tiles, 2), dim3(256), 0, s, d, r,
                       dA ? (const float*)up : nullptr, w.ksM, (void*)(ws + w.pack_u), t_src,
                       t ? 1 : w.ksK, (void*)(ws + w.pack_t), full);
    const int32_t nr = w.NT >= 3 ? 4 : w.NT;
    const dim3 grid(na + nb, w.slots, (unsigned)cdiv(w.NT, nr));
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(GRAD_WAVES * 64), 0, s, d, r, qa, qb, na, full);
    };
    if (nr == 1) go(k_lora_grad<T, 1>);
    else if (nr == 2) go(k_lora_grad<T, 2>);
    else go(k_lora_grad<T, 4>);
  }
  const int32_t slots = Tn > 0 ? w.slots : 0;
  if (p->L == 1 && slots == 1) return;
  const int32_t ja = dA ? (int32_t)cdiv(p->K, 1024) : 0, jb = dB ? (int32_t)cdiv(p->M, 1024) : 0;
  hipLaunchKernelGGL(k_lora_join<T>, dim3((unsigned)(p->L * p->R), ja + jb), dim3(256), 0, s, d, r,
                     slots, qa, qb, ja);
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_lora_workspace(const snack_lora* lora, snack_dtype dtype, int32_t T,
                                  int32_t backward, size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  if (snack_status st = check_lora(lora, dtype, T)) return st;
  *bytes = plan_of(lora, dtype, T, backward != 0).total;
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
  if (ws_bytes < plan_of(lora, dtype, T, false).total) return SNACK_E_WORKSPACE;
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
  if (snack_status st = check_lora(lora, dtype, T)) return st;
  if (ldx < lora->K || lddy < lora->M || (dX && lddx < lora->K) || (base && ldb < lora->K))
    return SNACK_E_SHAPE;
  if (T > 0) {
    if (!lora->A || !lora->B || !ids || !X || !dY || !ws) return SNACK_E_NULL;
    if (dX && (dX == X || dX == dY || (dX == base && lddx != ldb))) return SNACK_E_SHAPE;
    if (ws_bytes < plan_of(lora, dtype, T, true).total) return SNACK_E_WORKSPACE;
  }
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
