// embed.hip -- rows of a table looked up by token, and the table's gradient
// (gfx950).
//   Y[i, :]  = scale W[ids[i], :]
//   dW[v, :] = base[v, :] + scale sum_{i : ids[i] = v} dY[i, :]
//
// The lookup is a copy of rows.  The gradient sorts the tokens by their number
// first (k_embed_sort) and then sums each table row's tokens in the sorted order
// (k_embed_sum), so no float is added by an atomic and the same inputs give the
// same bits.  A text's most frequent token has many times the mean: rows of
// more than RUN tokens are summed in pieces of the sorted order, RUN places
// each, which k_embed_join adds.  Rows without a token, most of a table, are
// written beside the sums.  Bound by memory where the table is large: dY once,
// every row of dW once; elsewhere by the three launches and their trips to memory.
// Figures here are of replays of a graph of calls, kernels' of a trace.  37 rows of
// 4,096 looked up: 2.7 us.  8,192 tokens of a text, 50,000 rows of 768 bf16: 28.5 us
// (sort 6.7, sums 16.3: the 89 MB of it all at 5.5 TB/s, join 4.0); 20,001 tokens,
// 32,001 rows of 1,000 fp32 with base: 91 us (8.9, 72: 336 MB at 4.7 TB/s, 7.2).
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "pieces.h"
#include "spans.h"

namespace snk {
namespace {

constexpr int64_t MAX_TOKENS = 1 << 28;
constexpr int32_t MAX_ROWS = 1 << 30;
constexpr int32_t MAX_FEATURES = 1 << 23;

// ------------------------------------------------------------------- lookup
template <typename T>
__global__ __launch_bounds__(256) void k_embed(ids_t ids, int64_t Tn, const T* __restrict__ W,
                                               int32_t V, int32_t D, int64_t ldw, float scale,
                                               T* __restrict__ Y, int64_t ldy, uint32_t per) {
  const uint32_t g = blockIdx.x * 256u + threadIdx.x;
  const int64_t i = g / per;
  if (i >= Tn) return;
  const cut_t c = cut_of<T>((int32_t)(g % per), D);
  const int32_t v = ids.get(i, V);
  frag<T> f{};
  if (v >= 0) f = load_cut(W + (int64_t)v * ldw, c, D);
  if (v >= 0 ? scale != 1.f : v == -2) {  // no token: zeros under every scale
    float x[EL<T>];
    floats_of(f, x);
#pragma unroll
    for (int e = 0; e < EL<T>; ++e) x[e] = v == -2 ? __builtin_nanf("") : x[e] * scale;
    f = to_frag(x);
  }
  store_cut(Y + i * ldy, c, D, f);
}

// --------------------------------------------------------------------- sort
// Sorted places of a piece: a row's chain of trips to memory, against the partial
// sums of longer rows (8,192 tokens, 50,000 rows of 768: 29.2 us with 16, 38.1 us with
// 32; 32,768 tokens, rows of 640: 50.9, 67.9 and, with 8, 56.0 us).
constexpr int32_t RUN = 16;
constexpr int32_t MAX_RANGE = 512;  // table rows of a sorting workgroup

// A place of the sorted order: its table row, and the places [begin, end) of that
// row.  Places past the last token have begin -1.
struct __attribute__((aligned(16))) place_t { int32_t row, begin, end, zero; };

struct sum_arg {
  const void* dY;
  int64_t lddy;
  int32_t V, D;
  float scale;
  const void* base;
  int64_t ldb;
  void* dW;
  int64_t lddw;
  const place_t* order;
  const int32_t* tokens;  // of each place, and RUN more
  const uint8_t* used;    // whether a table row has tokens
  float* part;            // two slots of per * EL floats for each RUN places
  uint32_t per;
};

template <typename T>
__device__ __forceinline__ frag<T> load_base(const sum_arg& a, int32_t v, cut_t c) {
  if (!a.base) return frag<T>{};
  return load_cut((const T*)a.base + (int64_t)v * a.ldb, c, a.D);
}
template <typename T>
__device__ __forceinline__ void store_row(const sum_arg& a, int32_t v, cut_t c, const frag<T>& f) {
  store_cut((T*)a.dW + (int64_t)v * a.lddw, c, a.D, f);
}
// base and acc times the scale.
template <typename T>
__device__ __forceinline__ frag<T> with_base(const sum_arg& a, const frag<T>& base,
                                             const float (&acc)[EL<T>]) {
  float b[EL<T>];
  floats_of(base, b);
#pragma unroll
  for (int e = 0; e < EL<T>; ++e) b[e] = fmaf(acc[e], a.scale, b[e]);
  return to_frag(b);
}

// Each workgroup owns `range` rows of the table and reads all token numbers:
// those below its rows give the place where its own begin, so the workgroups
// need nothing of each other.  What each costs is a few instructions for every
// number, all workgroups together T V / range of them.  Its W waves take every
// W-th block of 64 tokens, count theirs by row and list them, and place them when
// all are counted: a row's tokens are in the order of waves, blocks and lanes.
// (With consecutive shares, the waves of all workgroups read addresses that are a
// multiple of 4 KB apart, one channel of the L2.)  Waves with more than LIST tokens
// read the numbers again instead.
constexpr int LIST = 512;

template <int W, typename I>
__global__ __launch_bounds__(W * 64) void k_embed_sort(const I* __restrict__ ids, int32_t Tn,
                                                       int32_t V, int32_t range, int32_t bits,
                                                       place_t* __restrict__ order,
                                                       int32_t* __restrict__ tokens,
                                                       uint8_t* __restrict__ used) {
  typedef typename std::make_unsigned<I>::type UI;
  extern __shared__ int32_t lds[];
  int32_t *count = lds, *begin_of = count + W * range, *end_of = begin_of + range,
          *below_of = end_of + range, *scan = below_of + W, *list = scan + W;
  uint16_t* list_row = reinterpret_cast<uint16_t*>(list + W * LIST);
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), lane = lane_id();
  const int32_t lo = blockIdx.x * range, hi = min(lo + range, V);
  constexpr int U = 4, STEP = W * 64;
  int32_t *mine = count + w * range, *my_token = list + w * LIST;
  uint16_t* my_row = list_row + w * LIST;
  I v[U];
  auto load = [&](int64_t at) {
    if (at + U * STEP <= Tn) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = ids[at + u * STEP + threadIdx.x];
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = at + u * STEP + threadIdx.x;
        v[u] = i < Tn ? ids[i] : (I)-1;
      }
    }
  };
  // Whether v is one of this workgroup's rows, and which; as an unsigned number a
  // negative one is past every table.
  auto row_of = [&](I v, int32_t* row) {
    const UI d = (UI)v - (UI)lo;
    *row = (int32_t)d;
    return d < (UI)(hi - lo);
  };
  load(0);
  for (int32_t q = threadIdx.x; q < W * range; q += STEP) count[q] = 0;
  __syncthreads();
  int32_t below = 0, hits = 0;
  for (int64_t at = 0; at < Tn;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      below += (int32_t)__popcll(__ballot((UI)v[u] < (UI)lo));
      int32_t row;
      const bool in = row_of(v[u], &row);
      const uint64_t mask = __ballot(in);
      if (mask) {
        const int32_t to = hits + (int32_t)__popcll(mask & lanemask_lt());
        if (in) atomicAdd(&mine[row], 1);
        if (in && to < LIST) {
          my_token[to] = (int32_t)at + u * STEP + (int32_t)threadIdx.x;
          my_row[to] = (uint16_t)row;
        }
        hits += (int32_t)__popcll(mask);
      }
    }
    at += U * STEP;
    if (at < Tn) load(at);
  }
  if (lane == 0) below_of[w] = below;
  __syncthreads();
  int32_t all_below = 0, total = 0, own = 0;
#pragma unroll
  for (int q = 0; q < W; ++q) all_below += below_of[q];
  const int32_t r = threadIdx.x;
  if (r < range) {
#pragma unroll
    for (int q = 0; q < W; ++q) own += count[q * range + r];
    if (lo + r < V) used[lo + r] = own > 0;
  }
  int32_t place = all_below + block_excl_scan_i32<STEP>(own, scan, &total);
  if (hi == V)  // places that no token takes
    for (int64_t k = (int64_t)all_below + total + threadIdx.x; k < Tn; k += STEP)
      order[k] = place_t{-1, -1, -1, 0};
  if (total == 0) return;
  if (r < range) {
    begin_of[r] = place;
    end_of[r] = place + own;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      const int32_t n = count[q * range + r];
      count[q * range + r] = place;
      place += n;
    }
  }
  __syncthreads();
  auto put = [&](bool in, int32_t row, int32_t token) {
    // lanes of the same row: all, where one token fills a text, or bit by bit
    uint64_t same = __ballot(in);
    const int32_t one = __shfl(row, __ffsll((unsigned long long)same) - 1);
    if (__ballot(in && row != one)) {
      for (int32_t k = 0; k < bits; ++k) {
        const bool bit = (row >> k) & 1;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
      }
    }
    int32_t to = 0;
    const int32_t before = (int32_t)__popcll(same & lanemask_lt());
    if (in && before == 0) to = atomicAdd(&mine[row], (int32_t)__popcll(same));
    to = __shfl(to, same ? __ffsll((unsigned long long)same) - 1 : 0) + before;
    if (in) {
      tokens[to] = token;
      order[to] = place_t{row + lo, begin_of[row], end_of[row], 0};
    }
  };
  if (hits <= LIST) {
    for (int32_t h = 0; h < hits; h += 64) {
      const bool in = h + lane < hits;
      put(in, in ? my_row[h + lane] : 0, in ? my_token[h + lane] : 0);
    }
  } else {
    load(0);
    for (int64_t at = 0; at < Tn; at += U * STEP) {
      int32_t row[U];
      bool in[U];
#pragma unroll
      for (int u = 0; u < U; ++u) in[u] = row_of(v[u], &row[u]);
      if (at + U * STEP < Tn) load(at + U * STEP);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (__ballot(in[u]))
          put(in[u], in[u] ? row[u] : 0, (int32_t)at + u * STEP + (int32_t)threadIdx.x);
    }
  }
}

// ---------------------------------------------------------------------- sums
// The tokens of RUN places.
struct run_t { int32_t token[RUN]; };
__device__ __forceinline__ run_t load_run(const sum_arg& a, int64_t k) {
  run_t r;
  __builtin_memcpy(r.token, a.tokens + k, sizeof(r.token));
  return r;
}

// The sum of the first n <= RUN of them, at cut c, four loads at a time (8,192 tokens
// of 50,000 rows of 768, the whole gradient, all three in one run: 28.0 us; eight at a
// time 29.3 us, all 16 35.4 us, for the registers leave fewer waves to wait beside each
// other).
template <typename T>
__device__ __forceinline__ void sum_run(const sum_arg& a, const run_t& r, int32_t n, cut_t c,
                                        float (&acc)[EL<T>]) {
  constexpr int U = RUN / 4;
  const T* dY = (const T*)a.dY;
#pragma unroll
  for (int h = 0; h < RUN; h += U) {
    if (h >= n) break;
    frag<T> f[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      f[u] = load_cut(dY + (int64_t)(h + u < n ? r.token[h + u] : r.token[0]) * a.lddy, c, a.D);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[EL<T>];
      floats_of(f[u], v);
#pragma unroll
      for (int e = 0; e < EL<T>; ++e) acc[e] += h + u < n ? v[e] : 0.f;
    }
  }
}

// Workgroups up to `sums` take the places at which a table row begins; up to
// `pieces` the pieces of rows of more than RUN tokens: of each RUN places those of
// such a row that began before (slot 0) and of one that begins there (slot 1; it
// goes on past them, so there is one at most); the others the rows without a token,
// whose stores fill the sums' trips to memory.
template <typename T>
__global__ __launch_bounds__(256) void k_embed_sum(sum_arg a, int32_t Tn, uint32_t sums,
                                                   uint32_t pieces) {
  constexpr int E = EL<T>;
  float acc[E] = {};
  if (blockIdx.x < sums) {
    const uint32_t g = blockIdx.x * 256u + threadIdx.x;
    const int32_t k = (int32_t)(g / a.per);
    if (k >= Tn) return;
    const place_t p = a.order[k];
    const run_t r = load_run(a, k);
    if (p.begin != k || p.end - k > RUN) return;
    const cut_t c = cut_of<T>((int32_t)(g % a.per), a.D);
    const frag<T> base = load_base<T>(a, p.row, c);
    sum_run<T>(a, r, p.end - k, c, acc);
    store_row(a, p.row, c, with_base(a, base, acc));
    return;
  }
  if (blockIdx.x < pieces) {
    const uint32_t g = (blockIdx.x - sums) * 256u + threadIdx.x;
    const uint32_t slot = g / a.per, q = g % a.per;
    const int64_t from = (int64_t)(slot / 2) * RUN;
    if (from >= Tn) return;
    const int64_t last = min(from + RUN, (int64_t)Tn) - 1;
    const place_t p = a.order[slot & 1 ? last : from];
    if (p.begin < 0 || p.end - p.begin <= RUN || (p.begin < from) == (slot & 1)) return;
    const int64_t k = max((int64_t)p.begin, from);
    sum_run<T>(a, load_run(a, k), (int32_t)(min((int64_t)p.end, from + RUN) - k),
               cut_of<T>((int32_t)q, a.D), acc);
    float* part = a.part + ((int64_t)slot * a.per + q) * E;
#pragma unroll
    for (int e = 0; e < E; ++e) part[e] = acc[e];
    return;
  }
  const uint32_t g = (blockIdx.x - pieces) * 256u + threadIdx.x;
  const int32_t v = (int32_t)(g / a.per);
  if (v >= a.V || a.used[v]) return;
  const cut_t c = cut_of<T>((int32_t)(g % a.per), a.D);
  store_row(a, v, c, load_base<T>(a, v, c));
}

// Rows of more than RUN tokens: workgroup (tiles, slab) takes those that begin in
// JOIN pieces of the order, SLAB pieces of their columns; groups of SLAB lanes add
// consecutive shares of a row's slots.
constexpr int32_t JOIN = 4;
constexpr int JOIN_THREADS = 256, SLAB = 16;

template <typename T>
__global__ __launch_bounds__(JOIN_THREADS) void k_embed_join(sum_arg a, int32_t Tn,
                                                             uint32_t slabs) {
  constexpr int E = EL<T>, GROUPS = JOIN_THREADS / SLAB, WAVES = JOIN_THREADS / 64;
  __shared__ float lds[WAVES][SLAB * E + 1];
  const int lane = lane_id(), group = threadIdx.x / SLAB, col = threadIdx.x % SLAB;
  const int32_t tiles = (int32_t)(blockIdx.x / slabs) * JOIN;
  const int64_t from = ((int64_t)tiles + lane) * RUN;
  place_t at{0, 0, 0, 0};
  if (lane < JOIN && from < Tn) at = a.order[min(from + RUN, (int64_t)Tn) - 1];
  const uint32_t q = blockIdx.x % slabs * SLAB + col;
  for (uint64_t todo = __ballot(at.end - at.begin > RUN && at.begin >= from); todo;
       todo &= todo - 1) {
    const int l = __ffsll((unsigned long long)todo) - 1;
    const int32_t tile = tiles + l, row = __shfl(at.row, l);
    // slots: this piece's second, the others' first
    const int32_t n = (__shfl(at.end, l) - 1) / RUN - tile + 1;
    const cut_t c = cut_of<T>((int32_t)min(q, a.per - 1), a.D);
    frag<T> base{};
    float acc[E] = {};
    if (q < a.per) {
      if (group == 0) base = load_base<T>(a, row, c);
      const int32_t j1 = (int32_t)((int64_t)n * (group + 1) / GROUPS);
#pragma unroll 8
      for (int32_t j = (int32_t)((int64_t)n * group / GROUPS); j < j1; ++j) {
        const int64_t slot = 2ll * (tile + j) + (j == 0);
        const float* p = a.part + (slot * a.per + q) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += p[e];
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
      for (int d = SLAB; d < 64; d <<= 1) acc[e] += __shfl_xor(acc[e], d);
      if (lane < SLAB) lds[threadIdx.x / 64][col * E + e] = acc[e];
    }
    __syncthreads();
    if (group == 0 && q < a.per) {
#pragma unroll
      for (int k = 1; k < WAVES; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += lds[k][col * E + e];
      store_row(a, row, c, with_base(a, base, acc));
    }
    __syncthreads();
  }
}

struct plan_t {
  int64_t per, tiles;  // pieces of a row; of the order, if a row can have more than RUN tokens
  int32_t range, waves;
  size_t order, tokens, used, part, total;
};

plan_t plan_of(snack_dtype dt, int64_t Tn, int32_t V, int32_t D) {
  plan_t p{};
  p.per = cdiv(D, dt == SNACK_BF16 ? 8 : 4);
  p.tiles = Tn > RUN ? cdiv(Tn, RUN) : 0;
  // a sorting workgroup on a CU, with 32 rows at least
  p.range = (int32_t)std::min<int64_t>(MAX_RANGE, std::max<int64_t>(32, cdiv(V, 256)));
  // 16 waves of them once there are two blocks of numbers for each (1,024 tokens, 50,000
  // rows of 768: 22.3 us with 4 waves, 23.7 us with 16)
  p.waves = Tn <= 2048 && p.range <= 256 ? 4 : 16;
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o = align_up(o + b, 256);
    return at;
  };
  p.order = take(sizeof(place_t) * (size_t)Tn);
  p.tokens = take(4 * ((size_t)Tn + RUN));
  p.used = take((size_t)V);
  p.part = take((size_t)p.tiles * 2 * p.per * (dt == SNACK_BF16 ? 32 : 16));
  p.total = std::max<size_t>(o, 256);
  return p;
}

int64_t joins_of(int64_t Tn, int64_t per) {
  return Tn > RUN ? cdiv(cdiv(Tn, RUN), JOIN) * cdiv(per, SLAB) : 0;
}

snack_status check_embed(snack_dtype dt, int32_t id_bytes, int64_t Tn, int32_t V, int32_t D) {
  if (dt != SNACK_F32 && dt != SNACK_BF16) return SNACK_E_DTYPE;
  if (id_bytes != 4 && id_bytes != 8) return SNACK_E_DTYPE;
  if (Tn < 0 || V < 0 || D < 0) return SNACK_E_SHAPE;
  // what a launch of each kernel holds
  const int64_t per = cdiv(D, dt == SNACK_BF16 ? 8 : 4);
  if (Tn > MAX_TOKENS || V > MAX_ROWS || D > MAX_FEATURES) return SNACK_E_OVERFLOW;
  if (per > 0 && V + Tn + Tn / (RUN / 2) + 4 > MAX_PIECES / per) return SNACK_E_OVERFLOW;
  return SNACK_OK;
}

template <int W, typename I>
void launch_sort(const void* ids, int32_t Tn, const plan_t& p, const sum_arg& a, hipStream_t s) {
  int32_t bits = 0;
  while ((1 << bits) < p.range) ++bits;
  hipLaunchKernelGGL((k_embed_sort<W, I>), dim3((unsigned)cdiv(a.V, p.range)), dim3(W * 64),
                     4 * ((size_t)(W + 2) * p.range + 2 * W + W * LIST) + 2 * W * LIST, s, (const I*)ids, Tn,
                     a.V, p.range, bits, const_cast<place_t*>(a.order),
                     const_cast<int32_t*>(a.tokens), const_cast<uint8_t*>(a.used));
}

template <typename T>
void run_bwd(ids_t ids, int32_t Tn, const plan_t& p, const sum_arg& a, hipStream_t s) {
  auto sort = p.waves == 4 ? (ids.wide ? launch_sort<4, int64_t> : launch_sort<4, int32_t>)
                           : (ids.wide ? launch_sort<16, int64_t> : launch_sort<16, int32_t>);
  sort(ids.p, Tn, p, a, s);
  const int64_t sums = cdiv(Tn * p.per, 256), pieces = sums + cdiv(2 * p.tiles * p.per, 256),
                blocks = pieces + (a.base != a.dW ? cdiv(a.V * p.per, 256) : 0);
  if (blocks > 0)
    hipLaunchKernelGGL(k_embed_sum<T>, dim3((unsigned)blocks), dim3(256), 0, s, a, Tn,
                       (uint32_t)sums, (uint32_t)pieces);
  if (p.tiles > 0)
    hipLaunchKernelGGL(k_embed_join<T>, dim3((unsigned)joins_of(Tn, p.per)), dim3(JOIN_THREADS), 0,
                       s, a, Tn, (uint32_t)cdiv(p.per, SLAB));
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_embed_fwd(snack_dtype dtype, const void* ids, int32_t id_bytes, int64_t T,
                             const void* W, int64_t ldw, int32_t V, int32_t D, float scale,
                             void* Y, int64_t ldy, void* stream) {
  if (snack_status st = check_embed(dtype, id_bytes, T, V, D)) return st;
  if (ldw < D || ldy < D) return SNACK_E_SHAPE;
  if (T == 0 || D == 0) return SNACK_OK;
  if (!ids || !Y || (V > 0 && !W)) return SNACK_E_NULL;
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4;
  const span_t out[] = {{Y, D * e, ldy * e, T}};
  const span_t in[] = {{V > 0 ? W : nullptr, D * e, ldw * e, V}, {ids, (__int128)id_bytes * T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const ids_t of{ids, id_bytes == 8};
  const uint32_t per = (uint32_t)cdiv(D, dtype == SNACK_BF16 ? 8 : 4);
  const dim3 grid((unsigned)cdiv(T * per, 256));
  if (dtype == SNACK_BF16)
    hipLaunchKernelGGL(k_embed<bf16>, grid, dim3(256), 0, s, of, T, (const bf16*)W, V, D, ldw,
                       scale, (bf16*)Y, ldy, per);
  else
    hipLaunchKernelGGL(k_embed<float>, grid, dim3(256), 0, s, of, T, (const float*)W, V, D, ldw,
                       scale, (float*)Y, ldy, per);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

snack_status snack_embed_workspace(snack_dtype dtype, int64_t T, int32_t V, int32_t D,
                                   size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  if (snack_status st = check_embed(dtype, 4, T, V, D)) return st;
  *bytes = plan_of(dtype, T, V, D).total;
  return SNACK_OK;
}

snack_status snack_embed_bwd(snack_dtype dtype, const void* ids, int32_t id_bytes, int64_t T,
                             const void* dY, int64_t lddy, int32_t V, int32_t D, float scale,
                             const void* base, int64_t ldb, void* dW, int64_t lddw, void* ws,
                             size_t ws_bytes, void* stream) {
  if (snack_status st = check_embed(dtype, id_bytes, T, V, D)) return st;
  if (lddy < D || lddw < D || (base && ldb < D)) return SNACK_E_SHAPE;
  if (V == 0 || D == 0) return SNACK_OK;
  if (!dW || !ws || (T > 0 && (!ids || !dY))) return SNACK_E_NULL;
  const plan_t p = plan_of(dtype, T, V, D);
  if (ws_bytes < p.total) return SNACK_E_WORKSPACE;
  if (dW == base && lddw != ldb) return SNACK_E_SHAPE;
  const __int128 e = dtype == SNACK_BF16 ? 2 : 4;
  const span_t out[] = {{dW, D * e, lddw * e, V}, {ws, (__int128)p.total}};
  const span_t in[] = {{T > 0 ? dY : nullptr, D * e, lddy * e, T},
                       {dW == base ? nullptr : base, D * e, ldb * e, V},
                       {T > 0 ? ids : nullptr, (__int128)id_bytes * T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* b = (char*)ws;
  const sum_arg a{dY, lddy, V, D, scale, base, ldb, dW, lddw, (const place_t*)(b + p.order),
                  (const int32_t*)(b + p.tokens), (const uint8_t*)(b + p.used),
                  (float*)(b + p.part), (uint32_t)p.per};
  const ids_t of{ids, id_bytes == 8};
  if (dtype == SNACK_BF16) run_bwd<bf16>(of, (int32_t)T, p, a, s);
  else run_bwd<float>(of, (int32_t)T, p, a, s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
