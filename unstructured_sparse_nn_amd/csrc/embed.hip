// embed.hip -- rows of a table looked up by token, and the table's gradient
// (gfx950).
//   Y[i, :]  = scale W[ids[i], :]
//   dW[v, :] = base[v, :] + scale sum_{i : ids[i] = v} dY[i, :]
//
// The lookup is a copy of rows.  The gradient sorts the tokens by their number
// first (k_embed_sort, which also writes the rows that no token has: most of a
// table) and then sums each table row's tokens in the sorted order
// (k_embed_sum), so no float is added by an atomic and the same inputs give the
// same bits.  A text's most frequent token has many times the mean: rows of
// more than RUN tokens are summed in pieces of the sorted order, RUN places
// each, which k_embed_join adds.  Bound by memory: dY once, every row of dW
// once.
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
  if (scale != 1.f || v == -2) {
    float x[EL<T>];
    floats_of(f, x);
#pragma unroll
    for (int e = 0; e < EL<T>; ++e) x[e] = v == -2 ? __builtin_nanf("") : x[e] * scale;
    f = to_frag(x);
  }
  store_cut(Y + i * ldy, c, D, f);
}

// --------------------------------------------------------------------- sort
constexpr int32_t RUN = 32;         // sorted places of a piece
constexpr int SORT_WAVES = 16;
constexpr int32_t MAX_RANGE = 512;  // table rows of a sorting workgroup

// A place of the sorted order: its token and table row, and the places [begin,
// end) of that row.
struct __attribute__((aligned(16))) place_t { int32_t token, row, begin, end; };

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
  const int32_t* all;  // places that the order has
  float* part;         // two slots of per * EL floats for each RUN places
  uint32_t per;
};

// acc times the scale, and base, into row v.
template <typename T>
__device__ __forceinline__ void put_row(const sum_arg& a, int32_t v, cut_t c,
                                        float (&acc)[EL<T>]) {
  float b[EL<T>] = {};
  if (a.base) floats_of(load_cut((const T*)a.base + (int64_t)v * a.ldb, c, a.D), b);
#pragma unroll
  for (int e = 0; e < EL<T>; ++e) acc[e] = fmaf(acc[e], a.scale, b[e]);
  store_cut((T*)a.dW + (int64_t)v * a.lddw, c, a.D, to_frag(acc));
}

// Each workgroup owns `range` rows of the table and reads all token numbers:
// those below its rows give the place where its own begin, so the workgroups
// need nothing of each other.  Its waves take every 16th block of 64 tokens,
// count theirs by row, and walk them again to place them: a row's tokens are in
// the order of waves, blocks and lanes.  (With consecutive shares, the waves of
// all workgroups read addresses that are a multiple of 4 KB apart, one channel of
// the L2: 9.7 us for 8,192 tokens instead of 6.)  Between the two walks it writes
// the rows that have no token.
template <typename T>
__global__ __launch_bounds__(SORT_WAVES * 64) void k_embed_sort(sum_arg a, ids_t ids, int32_t Tn,
                                                                int32_t range) {
  extern __shared__ int32_t lds[];
  int32_t *count = lds, *begin_of = count + SORT_WAVES * range, *end_of = begin_of + range,
          *below_of = end_of + range, *scan = below_of + SORT_WAVES;
  const int w = threadIdx.x / 64, lane = lane_id();
  const int32_t lo = blockIdx.x * range, hi = min(lo + range, a.V);
  for (int32_t q = threadIdx.x; q < SORT_WAVES * range; q += SORT_WAVES * 64) count[q] = 0;
  __syncthreads();
  constexpr int U = 4, STEP = SORT_WAVES * 64;
  int32_t* mine = count + w * range;
  int32_t below = 0;
  auto load = [&](int64_t from, int32_t (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = ids.get(min(from + u * STEP, (int64_t)Tn - 1), a.V);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (from + u * STEP >= Tn) v[u] = -1;
  };
  for (int64_t at = 0; at < Tn; at += U * STEP) {
    int32_t v[U];
    load(at + threadIdx.x, v);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      below += __popcll(__ballot(v[u] >= 0 && v[u] < lo));
      if (v[u] >= lo && v[u] < hi) atomicAdd(&mine[v[u] - lo], 1);
    }
  }
  if (lane == 0) below_of[w] = below;
  __syncthreads();
  int32_t all_below = 0, total = 0, own = 0;
#pragma unroll
  for (int q = 0; q < SORT_WAVES; ++q) all_below += below_of[q];
  const int32_t r = threadIdx.x;
  if (r < range) {
#pragma unroll
    for (int q = 0; q < SORT_WAVES; ++q) own += count[q * range + r];
  }
  int32_t place = all_below + block_excl_scan_i32<SORT_WAVES * 64>(own, scan, &total);
  if (r < range) {
    begin_of[r] = place;
    end_of[r] = place + own;
#pragma unroll
    for (int q = 0; q < SORT_WAVES; ++q) {
      const int32_t n = count[q * range + r];
      count[q * range + r] = place;
      place += n;
    }
  }
  if (threadIdx.x == 0 && hi == a.V) *const_cast<int32_t*>(a.all) = all_below + total;
  __syncthreads();
  if (a.base != a.dW) {  // in place nothing is added to them
    const uint32_t n = (uint32_t)(hi - lo) * a.per;
    for (uint32_t g = threadIdx.x; g < n; g += SORT_WAVES * 64) {
      const int32_t row = (int32_t)(g / a.per);
      if (begin_of[row] != end_of[row]) continue;
      float acc[EL<T>] = {};
      put_row<T>(a, lo + row, cut_of<T>((int32_t)(g % a.per), a.D), acc);
    }
  }
  if (total == 0) return;
  place_t* order = const_cast<place_t*>(a.order);
  for (int64_t at = 0; at < Tn; at += U * STEP) {
    int32_t v[U];
    load(at + threadIdx.x, v);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = v[u] >= lo && v[u] < hi;
      // lanes of one row at a time
      for (uint64_t todo = __ballot(in); todo;) {
        const int leader = __ffsll((unsigned long long)todo) - 1;
        const int32_t row = __shfl(v[u], leader);
        const uint64_t same = __ballot(in && v[u] == row);
        int32_t to = 0;
        if (lane == leader) to = atomicAdd(&mine[row - lo], __popcll(same));
        to = __shfl(to, leader) + __popcll(same & lanemask_lt());
        if (in && v[u] == row)
          order[to] = place_t{(int32_t)(at + u * STEP) + (int32_t)threadIdx.x, row,
                              begin_of[row - lo], end_of[row - lo]};
        todo &= ~same;
      }
    }
  }
}

// ---------------------------------------------------------------------- sums
// acc += the tokens of places [k, end), at cut c.
template <typename T>
__device__ __forceinline__ void add_tokens(const sum_arg& a, int32_t k, int32_t end, cut_t c,
                                           float (&acc)[EL<T>]) {
  constexpr int U = 4;
  const T* dY = (const T*)a.dY;
  for (; k < end; k += U) {
    frag<T> f[U];
    int32_t tok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) tok[u] = a.order[min(k + u, end - 1)].token;
#pragma unroll
    for (int u = 0; u < U; ++u) f[u] = load_cut(dY + (int64_t)tok[u] * a.lddy, c, a.D);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[EL<T>];
      floats_of(f[u], v);
#pragma unroll
      for (int e = 0; e < EL<T>; ++e) acc[e] += k + u < end ? v[e] : 0.f;
    }
  }
}

// The first `blocks` workgroups take the places at which a table row begins, the
// others the pieces of rows of more than RUN tokens: of each RUN places those of
// such a row that began before (slot 0) and of one that begins there (slot 1);
// it goes on past them, so there is one at most.
template <typename T>
__global__ __launch_bounds__(256) void k_embed_sum(sum_arg a, uint32_t blocks) {
  constexpr int E = EL<T>;
  float acc[E] = {};
  const int32_t all = *a.all;
  if (blockIdx.x < blocks) {
    const uint32_t g = blockIdx.x * 256u + threadIdx.x;
    const int32_t k = (int32_t)(g / a.per);
    if (k >= all) return;
    const place_t p = a.order[k];
    if (p.begin != k || p.end - k > RUN) return;
    const cut_t c = cut_of<T>((int32_t)(g % a.per), a.D);
    add_tokens<T>(a, k, p.end, c, acc);
    put_row<T>(a, p.row, c, acc);
    return;
  }
  const uint32_t g = (blockIdx.x - blocks) * 256u + threadIdx.x;
  const uint32_t slot = g / a.per, q = g % a.per;
  const int64_t from = (int64_t)(slot / 2) * RUN;
  if (from >= all) return;
  const int32_t to = (int32_t)min(from + RUN, (int64_t)all);
  const place_t p = a.order[slot & 1 ? to - 1 : from];
  if (p.end - p.begin <= RUN || (p.begin < from) == (slot & 1)) return;
  add_tokens<T>(a, max(p.begin, (int32_t)from), min(p.end, to), cut_of<T>((int32_t)q, a.D), acc);
  float* part = a.part + ((int64_t)slot * a.per + q) * E;
#pragma unroll
  for (int e = 0; e < E; ++e) part[e] = acc[e];
}

// Rows of more than RUN tokens: one that begins among the RUN places of this
// workgroup, 64 pieces of it; the waves add consecutive shares of its slots.
template <typename T>
__global__ __launch_bounds__(256) void k_embed_join(sum_arg a) {
  constexpr int E = EL<T>;
  __shared__ float lds[4][64][E + 1];
  const int32_t tile = blockIdx.x, from = tile * RUN, all = *a.all;
  if (from >= all) return;
  const place_t at = a.order[min(from + RUN, all) - 1];
  if (at.end - at.begin <= RUN || at.begin < from) return;
  const int32_t n = (at.end - 1) / RUN - tile + 1;  // slots: this tile's second, the others' first
  const int w = threadIdx.x / 64, lane = lane_id();
  const uint32_t q = blockIdx.y * 64 + lane;
  float acc[E] = {};
  if (q < a.per) {
    const int32_t j1 = (int32_t)((int64_t)n * (w + 1) / 4);
#pragma unroll 4
    for (int32_t j = (int32_t)((int64_t)n * w / 4); j < j1; ++j) {
      const int64_t slot = 2ll * (tile + j) + (j == 0);
      const float* p = a.part + (slot * a.per + q) * E;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += p[e];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) lds[w][lane][e] = acc[e];
  __syncthreads();
  if (w != 0 || q >= a.per) return;
#pragma unroll
  for (int e = 0; e < E; ++e)
    acc[e] = ((lds[0][lane][e] + lds[1][lane][e]) + lds[2][lane][e]) + lds[3][lane][e];
  put_row<T>(a, at.row, cut_of<T>((int32_t)q, a.D), acc);
}

struct plan_t {
  int64_t per, tiles;  // tiles: 0 if no row can have more than RUN tokens
  int32_t range;
  size_t all, order, part, total;
};

plan_t plan_of(snack_dtype dt, int64_t Tn, int32_t V, int32_t D) {
  plan_t p{};
  p.per = cdiv(D, dt == SNACK_BF16 ? 8 : 4);
  p.tiles = Tn > RUN ? cdiv(Tn, RUN) : 0;
  // two sorting workgroups on a CU, with 32 rows at least: every one reads all
  // token numbers
  p.range = (int32_t)std::min<int64_t>(MAX_RANGE, std::max<int64_t>(32, cdiv(V, 512)));
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o = align_up(o + b, 256);
    return at;
  };
  p.all = take(4);
  p.order = take(sizeof(place_t) * (size_t)Tn);
  p.part = take((size_t)p.tiles * 2 * p.per * (dt == SNACK_BF16 ? 32 : 16));
  p.total = std::max<size_t>(o, 256);
  return p;
}

snack_status check_embed(snack_dtype dt, int32_t id_bytes, int64_t Tn, int32_t V, int32_t D) {
  if (dt != SNACK_F32 && dt != SNACK_BF16) return SNACK_E_DTYPE;
  if (id_bytes != 4 && id_bytes != 8) return SNACK_E_DTYPE;
  if (Tn < 0 || V < 0 || D < 0) return SNACK_E_SHAPE;
  // what a launch of each kernel holds
  const int64_t per = cdiv(D, dt == SNACK_BF16 ? 8 : 4);
  if (Tn > MAX_TOKENS || V > MAX_ROWS || D > MAX_FEATURES) return SNACK_E_OVERFLOW;
  if (per > 0 && (Tn + Tn / (RUN / 2) + 2 > MAX_PIECES / per || V > MAX_PIECES / per))
    return SNACK_E_OVERFLOW;
  return SNACK_OK;
}

template <typename T>
void run_bwd(ids_t ids, int32_t Tn, const plan_t& p, const sum_arg& a, hipStream_t s) {
  hipLaunchKernelGGL(k_embed_sort<T>, dim3((unsigned)cdiv(a.V, p.range)), dim3(SORT_WAVES * 64),
                     4 * ((SORT_WAVES + 2) * (size_t)p.range + 2 * SORT_WAVES), s, a, ids, Tn,
                     p.range);
  if (Tn == 0) return;
  const int64_t blocks = cdiv(Tn * p.per, 256), more = cdiv(2 * p.tiles * p.per, 256);
  hipLaunchKernelGGL(k_embed_sum<T>, dim3((unsigned)(blocks + more)), dim3(256), 0, s, a,
                     (uint32_t)blocks);
  if (p.tiles > 0)
    hipLaunchKernelGGL(k_embed_join<T>, dim3((unsigned)p.tiles, (unsigned)cdiv(p.per, 64)),
                       dim3(256), 0, s, a);
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
                  (const int32_t*)(b + p.all), (float*)(b + p.part), (uint32_t)p.per};
  const ids_t of{ids, id_bytes == 8};
  if (dtype == SNACK_BF16) run_bwd<bf16>(of, (int32_t)T, p, a, s);
  else run_bwd<float>(of, (int32_t)T, p, a, s);
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // extern "C"
