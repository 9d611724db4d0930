// seqloss.hip -- losses of answers by the log-probabilities of their tokens,
// with the gradient of each (gfx950).
//
// Preference (pairs of sequences 2p, the preferred one, and 2p + 1):
//   d_j = sum over the counted tokens of sequence j of (logp - ref)
//   h   = d_2p - d_2p+1,  z = beta h,  loss = mean over the pairs of f
//   f   = -(1 - eps) log sigmoid(z) - eps log sigmoid(-z)   sigmoid
//         max(0, 1 - z)                                     hinge
//         (h - 1 / (2 beta))^2                              squared
// Policy, with r = exp(logp - old) and k = ref - logp at each token:
//   f = -min(r A, clamp(r, 1 - low, 1 + high) A) + kl (exp(k) - k - 1)
//   loss = sum of f over all tokens / their number, or the mean over the
//          sequences of their tokens' mean
//
// The sequences are cut into items of at most 2^log_p tokens, a wave's work each,
// so that one long answer among short ones is many waves'.  A preference's
// gradients need the sums of its sequences first:
//   k_pref_sums    the sums of every item
//   k_pref_finish  the items of a sequence follow each other: their sums, each
//                  pair's loss and what the gradients of its tokens are
//   k_pref_grads   the gradients, and the loss
// A policy's need only how many tokens count, which is known where there is no
// mask, and is cheap to find where it is short:
//   k_policy_counts  the counts of every item (a mask of a large batch)
//   k_policy         gradients, and the sums of every workgroup's items
//   k_policy_finish  the loss and the statistics
// Small batches take one workgroup and one launch (k_seq_small), whose waves keep
// their tokens in registers.  Sums are 64-bit in a fixed order; whether a ratio is
// past its border is decided on logarithms in 64 bits.  A token's terms are fp32.
// Bound by launches, trips to memory and, on one CU, instructions where the batch
// is small: 1,500 tokens in 16 sequences 6.1 us, a policy's 12,345 in 64 7.9 us (replays
// of a graph of calls; kernels of a trace).  Large batches are two to five floats a
// token read and one written, but come to half of memory's rate at most: 4 million
// tokens in 4,096 sequences 24.5 us (sums 12.0, finish 5.0, gradients 7.9; 2.1 TB/s), a
// policy's 2 million in 1,024 22.5 us (counts 4.4, gradients 15.0, finish 4.0; the
// tokens' terms are 6 us of instructions).
#include <cmath>

#include "common.h"
#include "internal.h"
#include "spans.h"

namespace snk {
namespace {

// ---------------------------------------------------------------- sequences
struct batch_t {
  const int32_t* starts;  // [S + 1], or NULL: `each` tokens in every sequence
  const uint8_t* mask;    // [T], or NULL: every token counts
  int32_t S, T, each;
  int32_t log_p, items;
};

// Places that do not fit are cut to [0, T], so a call with wrong ones stays
// inside its arrays.
__device__ __forceinline__ int32_t start_of(const batch_t& q, int32_t i) {
  return q.starts ? min(max(q.starts[i], 0), q.T) : i * q.each;
}

// Sequence i's items are those from first_item(i) up to first_item(i + 1): with
// starts a_i, from a_i / P + i up to a_(i+1) / P + i + 1, at least as many as it
// needs (the last may be empty), without a sum over the sequences before it.
__device__ __forceinline__ int32_t first_item(const batch_t& q, int32_t i, int32_t start) {
  return (start >> q.log_p) + i;
}

struct item_t {
  int32_t seq, from, end;  // its sequence, and that one's tokens
  int32_t a, b;            // its tokens
};

// Item x of the sequence that begins at a; items before the first sequence's or
// past the last one's have no tokens.
__device__ __forceinline__ item_t item_at(const batch_t& q, int32_t x, int32_t seq, int32_t a,
                                          int32_t next) {
  const int32_t b = max(next, a), x0 = first_item(q, seq, a);
  int64_t from = b;
  if (x >= x0) from = a + ((int64_t)(x - x0) << q.log_p);
  return {seq, a, b, (int32_t)min(from, (int64_t)b),
          (int32_t)min(from + (1 << q.log_p), (int64_t)b)};
}

// The sequence of item x is the last one whose first item is not past x: a
// search that cuts the sequences into 63 with every trip to memory; the last trip
// brings the sequence's own start and the next one's too.
__device__ __forceinline__ item_t item_of(const batch_t& q, int32_t x) {
  int32_t lo = 0, n = q.S;
  for (;;) {
    const int32_t step = (n + 62) / 63;
    const int64_t at = (int64_t)lane_id() * step;
    const int32_t i = lo + (int32_t)min(at, (int64_t)n), start = start_of(q, i);
    // none where x comes before the first sequence's items (and a count is unsigned)
    const int32_t found = (int32_t)__popcll(__ballot(at < n && first_item(q, i, start) <= x));
    const int32_t last = max(found - 1, 0);
    lo += last * step;
    if (step == 1) return item_at(q, x, lo, __shfl(start, last), __shfl(start, last + 1));
    n = min(step, n - last * step);
  }
}

// The items of sequence i.
struct range_t { int32_t a, b; };
__device__ __forceinline__ range_t items_of(const batch_t& q, int32_t i) {
  const int32_t a = start_of(q, i), b = max(start_of(q, i + 1), a);
  return {first_item(q, i, a), min(first_item(q, i + 1, b), q.items)};
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// The sums of an item, a sequence or the batch.  Preference: f is d's sum.  cut
// and n are whole.
struct sums_t { double f, kl, cut, n; };
__device__ __forceinline__ sums_t operator+(const sums_t& a, const sums_t& b) {
  return {a.f + b.f, a.kl + b.kl, a.cut + b.cut, a.n + b.n};
}
__device__ __forceinline__ sums_t wave_sum(const sums_t& s) {
  return {wave_sum(s.f), wave_sum(s.kl), wave_sum(s.cut), wave_sum(s.n)};
}

// ---------------------------------------------------------------- preference
struct pref_t {
  static constexpr bool POLICY = false;
  const float *logps, *ref;
  double beta, eps, share;  // share: of a pair in the loss
  int32_t form, average;

  template <int U> struct in_t { float lp[U], ref[U]; };
  template <int U, typename P>
  __device__ __forceinline__ void load(const P& at, int32_t, in_t<U>& v) const {
    at.get(logps, v.lp);
    if (ref) {
      at.get(ref, v.ref);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v.ref[u] = 0.f;
    }
  }
  __device__ __forceinline__ double per(const sums_t& s) const {
    return average ? 1.0 / fmax(s.n, 1.0) : 1.0;
  }
  // A pair's loss, and its derivative by h.
  __device__ __forceinline__ double pair(double h, double* dh) const {
    const double z = beta * h;
    if (form == SNACK_PREF_HINGE) {
      *dh = z < 1.0 ? -beta : z >= 1.0 ? 0.0 : z;  // NaN stays NaN
      return z < 1.0 ? 1.0 - z : z >= 1.0 ? 0.0 : z;
    }
    if (form == SNACK_PREF_SQUARED) {
      const double u = h - 0.5 / beta;
      *dh = 2.0 * u;
      return u * u;
    }
    const double t = exp(-fabs(z)), soft = log1p(t);  // log(1 + exp(z)) = soft + max(z, 0)
    const double up = 1.0 / (1.0 + t), down = t * up;
    const double sig = z >= 0 ? up : down, not_sig = z >= 0 ? down : up;
    *dh = beta * (eps * sig - (1.0 - eps) * not_sig);
    const double a = (1.0 - eps) * (soft + fmax(-z, 0.0)), b = eps * (soft + fmax(z, 0.0));
    return eps == 0.0 ? a : eps == 1.0 ? b : a + b;  // no product of 0 and infinity
  }
};

// -------------------------------------------------------------------- policy
struct policy_t {
  static constexpr bool POLICY = true;
  const float *logps, *old, *ref, *adv;
  double log_low, log_high;  // of 1 - low and 1 + high
  float low, high, kl;
  int32_t by_token, sequence_mean;

  struct token_t { float f, df, kl; bool cut; };
  template <int U> struct in_t { float lp[U], old[U], ref[U], adv[U]; };
  template <int U, typename P>
  __device__ __forceinline__ void load(const P& at, int32_t seq, in_t<U>& v) const {
    at.get(logps, v.lp);
    if (old) at.get(old, v.old);
    if (ref) at.get(ref, v.ref);
    if (by_token) at.get(adv, v.adv);
    const float a = by_token ? 0.f : adv[seq];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (!by_token) v.adv[u] = a;
  }

  // exp(k) - 1 - k without its cancellation near 0, and exp(k) - 1.
  __device__ __forceinline__ static float above(float k, float* em1) {
    float s;
    if (fabsf(k) < 1.f) {
      // k^2 (1/2! + k/3! + ... + k^9/11!): the rest is below 2^-25 of it
      s = 1.f / 39916800.f;
      s = fmaf(s, k, 1.f / 3628800.f);
      s = fmaf(s, k, 1.f / 362880.f);
      s = fmaf(s, k, 1.f / 40320.f);
      s = fmaf(s, k, 1.f / 5040.f);
      s = fmaf(s, k, 1.f / 720.f);
      s = fmaf(s, k, 1.f / 120.f);
      s = fmaf(s, k, 1.f / 24.f);
      s = fmaf(s, k, 1.f / 6.f);
      s = fmaf(s, k, 0.5f);
      s *= k * k;
      *em1 = k + s;
    } else {
      *em1 = expm1f(k);
      s = *em1 - fminf(k, 3.4028234663852886e38f);  // infinite at k = infinity
    }
    return s;
  }

  template <int U>
  __device__ __forceinline__ token_t token(const in_t<U>& v, int u) const {
    const float a = v.adv[u];
    // without old 0, but for NaN
    const double lp = v.lp[u], move = old ? lp - (double)v.old[u] : lp == lp ? 0.0 : lp;
    // an advantage of 0 has nothing of a ratio past every float
    const float r = expf((float)move), ra = a == 0.f && r == r ? 0.f : r * a;
    token_t o;
    o.cut = (a > 0.f && move > log_high) || (a < 0.f && move < log_low);
    o.f = o.cut ? -(a > 0.f ? high : low) * a : -ra;
    o.df = o.cut ? 0.f : -ra;
    o.kl = 0.f;
    if (ref) {
      float em1;
      o.kl = above((float)((double)v.ref[u] - lp), &em1);
      if (kl != 0.f) {  // otherwise for the statistics alone, however large it is
        o.f = fmaf(kl, o.kl, o.f);
        o.df = fmaf(-kl, em1, o.df);
      }
    }
    return o;
  }
  // What a sequence's gradients are multiplied by, beside the loss's own.
  __device__ __forceinline__ double weight(const batch_t& q, double seq_n, double all_n) const {
    return 1.0 / (sequence_mean ? (double)q.S * fmax(seq_n, 1.0) : fmax(all_n, 1.0));
  }
};

struct out_t {
  const float* dloss;  // device, or NULL: 1
  float* loss;         // or NULL
  float* more;         // rewards [S] or stats [2], or NULL
  float* grad;         // [T], or NULL
};
__device__ __forceinline__ double upstream(const out_t& out) {
  return out.dloss ? (double)*out.dloss : 1.0;
}

// A lane's U tokens of an item: runs of four (one, where U is less), which are
// loaded and stored 16 bytes at once at any alignment: where every array is read
// four bytes a lane, the addresses cost as much as the sums (2,048 pairs, 4 million
// tokens: 32.7 us, 26.2 us so).  A run that would pass the end is taken from the last four
// tokens; `in` says which of them are this lane's own, `counts` which the mask has.
// (Items of 1,024 tokens instead of 512: 24.1 us for that batch, but 19.2 instead of
// 18.6 us for 2 million tokens in 4,000 sequences, 12.0 instead of 11.4 us for 100,000 in
// 1,000, and a policy's 2 million 23.1 instead of 21.4 us.)
template <int U> struct places_t {
  static constexpr int W = U >= 4 ? 4 : 1, G = U / W;
  int32_t n;  // the item's tokens
  int32_t at[G];
  uint32_t in[G], counts[G];

  // Whether the wave has tokens in its run g: most items end early, and what is not
  // there costs no instructions (the same batch 26.3 us without this).
  __device__ __forceinline__ bool some(int g) const { return g * 64 * W < n; }

  __device__ __forceinline__ void find(const batch_t& q, int32_t a, int32_t b) {
    n = __builtin_amdgcn_readfirstlane(b - a);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      in[g] = counts[g] = 0;
      if (!some(g)) continue;
      const int32_t start = a + (g * 64 + lane_id()) * W;
      if (W == 1) {
        at[g] = start < b ? start : a;
        in[g] = start < b;
        counts[g] = in[g];
        if (q.mask) counts[g] &= q.mask[at[g]] != 0;
      } else if (b - a >= W) {
        at[g] = min(start, b - W);
        in[g] = start < b ? 15u & (15u << (start - at[g])) : 0u;
        counts[g] = in[g];
        if (q.mask) {
          uint32_t m;
          __builtin_memcpy(&m, q.mask + at[g], 4);
          // a bit of each byte that is not 0, and the four of them side by side
          m = ((((m & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | m) & 0x80808080u) >> 7;
          counts[g] &= (m * 0x01020408u) >> 24;
        }
      } else {  // fewer than four: the first lane's
        at[g] = a;
        in[g] = g == 0 && lane_id() == 0 ? (1u << (b - a)) - 1u : 0u;
        counts[g] = in[g];
        if (q.mask)
          for (int32_t e = 0; e < b - a; ++e)
            if (!q.mask[a + e]) counts[g] &= ~(1u << e);
      }
    }
  }
  __device__ __forceinline__ bool has(int u) const { return counts[u / W] >> (u % W) & 1; }
  // v, or 0 where the mask has a token not.
  __device__ __forceinline__ void put(float* grad, const float (&v)[U]) const {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!some(g)) continue;
      float o[W];
#pragma unroll
      for (int e = 0; e < W; ++e) o[e] = has(g * W + e) ? v[g * W + e] : 0.f;
      if (in[g] == (1u << W) - 1u) {
        __builtin_memcpy(grad + at[g], o, sizeof(o));
      } else if (in[g]) {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (in[g] >> e & 1) grad[at[g] + e] = o[e];
      }
    }
  }
  // Elements of a token array.
  __device__ __forceinline__ void get(const float* p, float (&v)[U]) const {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!some(g)) continue;
      if (W == 1 || n >= W) {
        __builtin_memcpy(&v[g * W], p + at[g], 4 * W);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) v[g * W + e] = p[at[g] + min(e, n - 1)];
      }
    }
  }
};

template <typename L, int U> struct tokens_t {
  places_t<U> at;
  typename L::template in_t<U> v;

  __device__ __forceinline__ void load(const batch_t& q, const L& loss, const item_t& it) {
    at.find(q, it.a, it.b);
    loss.template load<U>(at, it.seq, v);
  }
  // Adds them to this lane's f and kl and to the wave's counts; g: what their
  // gradients are but for the weight.
  __device__ __forceinline__ void add(const L& loss, sums_t& s, float (&g)[U]) const {
    int32_t n = 0, cut = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!at.some(u / places_t<U>::W)) continue;
      const bool has = at.has(u);
      n += (int32_t)__popcll(__ballot(has));
      if constexpr (L::POLICY) {
        const auto o = loss.template token<U>(v, u);
        cut += (int32_t)__popcll(__ballot(has && o.cut));
        s.f += (double)(has ? o.f : 0.f);
        s.kl += (double)(has ? o.kl : 0.f);
        g[u] = o.df;
      } else {
        s.f += has ? (double)v.lp[u] - (double)v.ref[u] : 0.0;
      }
    }
    s.n += n;
    s.cut += cut;
  }
};
template <typename L>
__device__ __forceinline__ void wave_totals(sums_t& s) {
  s.f = wave_sum(s.f);
  if (L::POLICY) s.kl = wave_sum(s.kl);
}

// Tokens of no sequence: their gradient is 0.
__device__ __forceinline__ void write_outside(const batch_t& q, float* grad, int64_t first,
                                              int64_t step) {
  const int32_t a = q.S > 0 ? start_of(q, 0) : q.T;
  const int32_t b = q.S > 0 ? max(start_of(q, q.S), start_of(q, q.S - 1)) : q.T;
  for (int64_t i = first; i < a; i += step) grad[i] = 0.f;
  for (int64_t i = b + first; i < q.T; i += step) grad[i] = 0.f;
}

// A pair's part of the loss; rewards and the two coefficients.
__device__ __forceinline__ double finish_pair(const pref_t& loss, const sums_t& x,
                                              const sums_t& y, int32_t p, const out_t& out,
                                              double* coef) {
  const double px = loss.per(x), py = loss.per(y), dx = x.f * px, dy = y.f * py;
  double dh;
  const double f = loss.pair(dx - dy, &dh);
  if (out.more) {
    out.more[2 * p] = (float)(loss.beta * dx);
    out.more[2 * p + 1] = (float)(loss.beta * dy);
  }
  dh *= upstream(out) * loss.share;
  coef[2 * p] = dh * px;
  coef[2 * p + 1] = -dh * py;
  return f * loss.share;
}
__device__ __forceinline__ void finish_stats(const sums_t& all, const out_t& out) {
  const double n = fmax(all.n, 1.0);
  if (out.more) out.more[0] = (float)(all.kl / n), out.more[1] = (float)(all.cut / n);
}

// ------------------------------------------------------- one workgroup, one launch
constexpr int SMALL_WAVES = 16;
constexpr int32_t SMALL_LOG_P = 7, SMALL_SEQS = 127;
// Items of a wave at most.  A policy's tokens are ten times the instructions, and
// its other path is two launches, not three: 5,000 tokens in 4 sequences 7.1 us
// there, 10.0 us in one workgroup; a preference's in 16 10.0 and 8.8 us.
template <typename L> constexpr int SMALL_EACH = L::POLICY ? 2 : 4;

// The starts of all sequences, two a lane.
struct starts_t {
  int32_t lo, hi;
  __device__ __forceinline__ int32_t at(int32_t i) const {
    const int32_t a = __shfl(lo, i & 63), b = __shfl(hi, i & 63);
    return i < 64 ? a : b;
  }
};

template <typename L>
__global__ __launch_bounds__(SMALL_WAVES * 64) void k_seq_small(batch_t q, L loss, out_t out) {
  constexpr int K = SMALL_EACH<L>, U = 1 << (SMALL_LOG_P - 6);
  __shared__ sums_t sums[K * SMALL_WAVES];
  __shared__ double coef[SMALL_SEQS + 1];
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), lane = lane_id();
  starts_t st{0, 0};
  if (q.S > 0) st = {start_of(q, min(lane, q.S)), start_of(q, min(64 + lane, q.S))};
  const int32_t first_lo = first_item(q, lane, st.lo), first_hi = first_item(q, 64 + lane, st.hi);
  item_t it[K];
  tokens_t<L, U> t[K];
  float g[K][U];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int32_t x = k * SMALL_WAVES + w;
    it[k] = {};
    if (x >= q.items) continue;
    const int32_t found = (int32_t)__popcll(__ballot(lane < q.S && first_lo <= x)) +
                          (int32_t)__popcll(__ballot(64 + lane < q.S && first_hi <= x));
    const int32_t seq = max(found - 1, 0);
    it[k] = item_at(q, x, seq, st.at(seq), st.at(seq + 1));
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (it[k].a < it[k].b) t[k].load(q, loss, it[k]);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int32_t x = k * SMALL_WAVES + w;
    if (x >= q.items) continue;
    sums_t s{0, 0, 0, 0};
    if (it[k].a < it[k].b) {
      t[k].add(loss, s, g[k]);
      wave_totals<L>(s);
    }
    if (lane == 0) sums[x] = s;
  }
  __syncthreads();
  if (w == 0) {
    double f = 0;
    auto total = [&](int32_t i) {  // of sequence i < S
      const int32_t a = st.at(i), b = max(st.at(i + 1), a);
      const int32_t x1 = min(first_item(q, i + 1, b), q.items);
      sums_t s{0, 0, 0, 0};
#pragma unroll 4
      for (int32_t x = first_item(q, i, a); x < x1; ++x) s = s + sums[x];
      return s;
    };
    if constexpr (!L::POLICY) {
      const int32_t pairs = q.S / 2, p = min(lane, max(pairs - 1, 0));
      if (pairs > 0) {
        const sums_t x = total(2 * p), y = total(2 * p + 1);
        if (lane < pairs) f = finish_pair(loss, x, y, p, out, coef);
      }
      f = wave_sum(f);
    } else {
      sums_t all{0, 0, 0, 0};
      for (int32_t x = lane; x < q.items; x += 64) all = all + sums[x];
      all = wave_sum(all);
      const double up = upstream(out);
      for (int32_t i0 = 0; i0 < q.S; i0 += 64) {
        const int32_t i = min(i0 + lane, q.S - 1);
        const sums_t s = total(i);
        if (i0 + lane < q.S) {
          const double weight = loss.weight(q, s.n, all.n);
          f += s.f * weight;
          coef[i] = weight * up;
        }
      }
      f = wave_sum(f);
      if (lane == 0) finish_stats(all, out);
    }
    if (lane == 0 && out.loss) *out.loss = (float)f;
  }
  if (!out.grad) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (it[k].a >= it[k].b) continue;
    const double c = coef[it[k].seq];
#pragma unroll
    for (int u = 0; u < U; ++u) g[k][u] = (float)(L::POLICY ? (double)g[k][u] * c : c);
    t[k].at.put(out.grad, g[k]);
  }
  write_outside(q, out.grad, threadIdx.x, SMALL_WAVES * 64);
}

// ------------------------------------------------------------- several launches
constexpr int32_t LOG_P = 9;
__device__ __forceinline__ int32_t wave_of_block() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
}

template <int W>
__device__ __forceinline__ sums_t block_sum(sums_t s, sums_t* lds) {
  s = wave_sum(s);
  if (lane_id() == 0) lds[threadIdx.x / 64] = s;
  __syncthreads();
  s = lds[0];
#pragma unroll
  for (int w = 1; w < W; ++w) s = s + lds[w];
  return s;
}

// What k_pref_grads needs of an item.
struct __attribute__((aligned(16))) slot_t { int32_t seq, a, b, zero; };

__global__ __launch_bounds__(256) void k_pref_sums(batch_t q, pref_t loss,
                                                   sums_t* __restrict__ sums,
                                                   slot_t* __restrict__ table) {
  const int32_t x = blockIdx.x * 4 + wave_of_block();
  if (x >= q.items) return;
  const item_t it = item_of(q, x);
  sums_t s{0, 0, 0, 0};
  if (it.a < it.b) {
    constexpr int U = 1 << (LOG_P - 6);
    tokens_t<pref_t, U> t;
    float g[U];
    t.load(q, loss, it);
    t.add(loss, s, g);
    wave_totals<pref_t>(s);
  }
  if (lane_id() == 0) sums[x] = s, table[x] = slot_t{it.seq, it.a, it.b, 0};
}

__device__ __forceinline__ sums_t range_sums(const sums_t* __restrict__ sums, range_t r) {
  sums_t s{0, 0, 0, 0};
  for (int32_t x = r.a + lane_id(); x < r.b; x += 64) s = s + sums[x];
  return wave_sum(s);
}

// A wave for each pair.  coef: of each sequence's gradients; terms: of the loss.
__global__ __launch_bounds__(256) void k_pref_finish(batch_t q, pref_t loss,
                                                     const sums_t* __restrict__ sums, out_t out,
                                                     double* __restrict__ coef,
                                                     double* __restrict__ terms) {
  const int32_t p = blockIdx.x * 4 + wave_of_block();
  if (p >= q.S / 2) return;
  const sums_t x = range_sums(sums, items_of(q, 2 * p)),
               y = range_sums(sums, items_of(q, 2 * p + 1));
  if (lane_id() == 0) terms[p] = finish_pair(loss, x, y, p, out, coef);
}

// The first workgroup adds the loss's terms, if it is wanted; the others write
// gradients.
__global__ __launch_bounds__(256) void k_pref_grads(batch_t q, const slot_t* __restrict__ table,
                                                    const double* __restrict__ coef,
                                                    const double* __restrict__ terms,
                                                    float* __restrict__ loss,
                                                    float* __restrict__ grad) {
  constexpr int U = 1 << (LOG_P - 6);
  __shared__ sums_t lds[4];
  const int32_t with_loss = loss ? 1 : 0;
  if ((int32_t)blockIdx.x < with_loss) {
    sums_t s{0, 0, 0, 0};
#pragma unroll 4
    for (int32_t i = threadIdx.x; i < q.S / 2; i += 256) s.f += terms[i];
    s = block_sum<4>(s, lds);
    if (threadIdx.x == 0) *loss = (float)s.f;
    return;
  }
  const int32_t b = blockIdx.x - with_loss;
  const int32_t x = b * 4 + wave_of_block();
  if (x < q.items) {
    const slot_t it = table[x];
    if (it.a < it.b) {
      const float c = (float)coef[it.seq];
      places_t<U> at;
      at.find(q, it.a, it.b);
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = c;
      at.put(grad, v);
    }
  }
  write_outside(q, grad, (int64_t)b * 256 + threadIdx.x,
                ((int64_t)gridDim.x - with_loss) * 256);
}

// ---- policy
// Tokens of [a, b) whose byte is set, by `threads` threads, 16 bytes at a time.
__device__ __forceinline__ int32_t count_bytes(const uint8_t* mask, int32_t a, int32_t b,
                                               int32_t thread, int32_t threads) {
  int32_t n = 0;
  const int32_t whole = (b - a) / 16;
  for (int32_t i = thread; i < whole; i += threads) {
    uint32_t v[4];
    __builtin_memcpy(v, mask + a + (int64_t)i * 16, 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t low = v[k] & 0x7F7F7F7Fu;  // the top bit of a byte that is not 0
      n += __builtin_popcount(((low + 0x7F7F7F7Fu) | v[k]) & 0x80808080u);
    }
  }
  const int32_t i = a + whole * 16 + thread;
  if (i < b) n += mask[i] != 0;
  return n;
}
__device__ __forceinline__ int32_t wave_sum(int32_t x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

__global__ __launch_bounds__(256) void k_policy_counts(batch_t q, int32_t* __restrict__ counts,
                                                       int32_t* __restrict__ totals) {
  __shared__ int32_t lds[4];
  const int32_t w = wave_of_block(), x = blockIdx.x * 4 + w;
  int32_t n = 0;
  if (x < q.items) {
    const item_t it = item_of(q, x);
    if (it.a < it.b) n = wave_sum(count_bytes(q.mask, it.a, it.b, lane_id(), 64));
    if (lane_id() == 0) counts[x] = n;
  }
  if (lane_id() == 0) lds[w] = n;
  __syncthreads();
  if (threadIdx.x == 0) totals[blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

// counts (nullable): what k_policy_counts has left; without them the workgroup
// counts what it needs.  sums: of the workgroup's items, f with its weight.
template <int LOG>
__global__ __launch_bounds__(256) void k_policy(batch_t q, policy_t loss, out_t out,
                                                const int32_t* __restrict__ counts,
                                                const int32_t* __restrict__ totals,
                                                int32_t n_totals, sums_t* __restrict__ sums) {
  constexpr int U = 1 << (LOG - 6);
  __shared__ sums_t lds[4];
  __shared__ int32_t ones[4];
  const int32_t w = wave_of_block(), lane = lane_id(), x = blockIdx.x * 4 + w;
  const bool mine = x < q.items;
  item_t it{};
  if (mine) it = item_of(q, x);
  tokens_t<policy_t, U> t;
  if (it.a < it.b) t.load(q, loss, it);
  double n = 0;  // tokens that the loss's mean is over: of the batch, or of the sequence
  if (!loss.sequence_mean) {
    int32_t part = 0;
    if (!q.mask) {
      n = (double)max(start_of(q, q.S) - start_of(q, 0), 0);
    } else {
      if (totals) {
#pragma unroll 4
        for (int32_t i = threadIdx.x; i < n_totals; i += 256) part += totals[i];
      } else {
        const int32_t a = start_of(q, 0);
        part = count_bytes(q.mask, a, max(start_of(q, q.S), a), threadIdx.x, 256);
      }
      part = wave_sum(part);
      if (lane == 0) ones[w] = part;
      __syncthreads();
      n = (double)(ones[0] + ones[1] + ones[2] + ones[3]);
    }
  } else if (it.a < it.b) {
    if (!q.mask) {
      n = (double)(it.end - it.from);
    } else {
      int32_t part = 0;
      if (counts) {
        const int32_t x1 = min(first_item(q, it.seq + 1, it.end), q.items);
        for (int32_t i = first_item(q, it.seq, it.from) + lane; i < x1; i += 64) part += counts[i];
      } else {
        part = count_bytes(q.mask, it.from, it.end, lane, 64);
      }
      n = (double)wave_sum(part);
    }
  }
  const double weight = loss.weight(q, n, n), c = weight * upstream(out);
  sums_t s{0, 0, 0, 0};
  if (it.a < it.b) {
    float g[U];
    t.add(loss, s, g);
    wave_totals<policy_t>(s);
    s.f *= weight;
    if (out.grad) {
#pragma unroll
      for (int u = 0; u < U; ++u) g[u] = (float)((double)g[u] * c);
      t.at.put(out.grad, g);
    }
  }
  if (lane == 0) lds[w] = s;
  __syncthreads();
  if (threadIdx.x == 0) sums[blockIdx.x] = ((lds[0] + lds[1]) + lds[2]) + lds[3];
  if (out.grad)
    write_outside(q, out.grad, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

template <int W>
__global__ __launch_bounds__(W * 64) void k_policy_finish(const sums_t* __restrict__ sums,
                                                          int32_t n, out_t out) {
  __shared__ sums_t lds[W];
  sums_t s{0, 0, 0, 0};
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < n; i += W * 64) s = s + sums[i];
  s = block_sum<W>(s, lds);
  if (threadIdx.x != 0) return;
  finish_stats(s, out);
  if (out.loss) *out.loss = (float)s.f;
}

// ---------------------------------------------------------------------- host
constexpr int32_t MAX_SEQS = 1 << 24;

// A policy's items are small (128 tokens) where there are few: a wave's tokens are
// then two a lane, and more waves share them (12,345 tokens in 64 sequences 7.7 us,
// 10.0 us with items of 512).
constexpr int32_t MEDIUM_ITEMS = 2048;
// Masks up to this many bytes are counted by every workgroup that needs them, which
// saves a launch (60,000 tokens: a mean over 500 sequences 7.4 us, 10.2 us with it;
// over all tokens 9.9 and 10.1 us).
constexpr int32_t COUNT_TOKENS = 65536;

struct plan_t {
  bool small;
  int32_t log_p, items, blocks;
  size_t sums, coef, terms, table, counts, totals, total;
};

plan_t plan_of(int32_t S, int32_t Tn, bool policy) {
  plan_t p{};
  auto items = [&](int32_t log_p) { return S == 0 ? 0 : S + (Tn >> log_p); };
  p.small = S <= SMALL_SEQS && items(SMALL_LOG_P) <= SMALL_WAVES * (policy ? SMALL_EACH<policy_t> : SMALL_EACH<pref_t>);
  p.log_p = p.small || (policy && items(SMALL_LOG_P) <= MEDIUM_ITEMS) ? SMALL_LOG_P : LOG_P;
  p.items = items(p.log_p);
  p.blocks = (int32_t)cdiv(p.items, 4);
  if (p.small) return p;
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o = align_up(o + b, 256);
    return at;
  };
  p.sums = take((size_t)(policy ? p.blocks : p.items) * sizeof(sums_t));
  if (policy) {
    p.counts = take((size_t)p.items * 4);
    p.totals = take((size_t)p.blocks * 4);
  } else {
    p.table = take((size_t)p.items * sizeof(slot_t));
    p.coef = take((size_t)S * sizeof(double));
    p.terms = take((size_t)S / 2 * sizeof(double));
  }
  p.total = o;
  return p;
}

snack_status check_batch(const snack_seqs* q) {
  if (!q) return SNACK_E_NULL;
  if (q->S < 0 || q->T < 0) return SNACK_E_SHAPE;
  if (q->S > MAX_SEQS || q->T > (1 << 30)) return SNACK_E_OVERFLOW;
  if (!q->starts && (q->S == 0 ? q->T != 0 : q->T % q->S != 0)) return SNACK_E_SHAPE;
  return SNACK_OK;
}

template <typename L>
snack_status run(const snack_seqs* b, const plan_t& p, const L& loss, const out_t& out, void* ws,
                 size_t ws_bytes, hipStream_t s) {
  if (p.total > 0 && !ws) return SNACK_E_NULL;
  if (ws_bytes < p.total) return SNACK_E_WORKSPACE;
  const batch_t q{b->starts, b->mask, b->S, b->T, b->S > 0 ? b->T / b->S : 0, p.log_p, p.items};
  char* w = (char*)ws;
  sums_t* sums = (sums_t*)(w + p.sums);
  if (p.small) {
    hipLaunchKernelGGL(k_seq_small<L>, dim3(1), dim3(SMALL_WAVES * 64), 0, s, q, loss, out);
  } else if constexpr (L::POLICY) {
    int32_t *counts = nullptr, *totals = nullptr;
    if (q.mask && q.T > COUNT_TOKENS) {
      counts = (int32_t*)(w + p.counts), totals = (int32_t*)(w + p.totals);
      hipLaunchKernelGGL(k_policy_counts, dim3(p.blocks), dim3(256), 0, s, q, counts, totals);
    }
    auto kernel = p.log_p == LOG_P ? k_policy<LOG_P> : k_policy<SMALL_LOG_P>;
    hipLaunchKernelGGL(kernel, dim3(p.blocks), dim3(256), 0, s, q, loss, out, counts, totals,
                       p.blocks, sums);
    if (out.loss || out.more)
      hipLaunchKernelGGL(p.blocks <= 512 ? k_policy_finish<2> : k_policy_finish<16>, dim3(1),
                         dim3(p.blocks <= 512 ? 128 : 1024), 0, s, sums, p.blocks, out);
  } else {
    slot_t* table = (slot_t*)(w + p.table);
    double *coef = (double*)(w + p.coef), *terms = (double*)(w + p.terms);
    hipLaunchKernelGGL(k_pref_sums, dim3(p.blocks), dim3(256), 0, s, q, loss, sums, table);
    hipLaunchKernelGGL(k_pref_finish, dim3((unsigned)cdiv(b->S / 2, 4)), dim3(256), 0, s, q, loss,
                       sums, out, coef, terms);
    const int32_t blocks = (out.loss ? 1 : 0) + (out.grad ? p.blocks : 0);
    if (blocks > 0)
      hipLaunchKernelGGL(k_pref_grads, dim3(blocks), dim3(256), 0, s, q, table, coef, terms,
                         out.loss, out.grad);
  }
  SNK_CHECK_LAUNCH();
  return SNACK_OK;
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

snack_status snack_seqs_workspace(int32_t S, int32_t T, size_t* bytes) {
  if (!bytes) return SNACK_E_NULL;
  const int32_t some = 0;
  const snack_seqs q{S, T, &some, nullptr};
  if (snack_status st = check_batch(&q)) return st;
  *bytes = std::max(plan_of(S, T, false).total, plan_of(S, T, true).total);
  return SNACK_OK;
}

snack_status snack_preference(const snack_seqs* batch, const snack_pref* pref, const float* logps,
                              const float* ref, const float* dloss, float* loss, float* rewards,
                              float* dlogps, void* ws, size_t ws_bytes, void* stream) {
  if (!pref) return SNACK_E_NULL;
  if (snack_status st = check_batch(batch)) return st;
  if (std::isnan(pref->beta) || std::isnan(pref->smoothing)) return SNACK_E_NAN;
  if (batch->S % 2 != 0 || !(pref->beta > 0) || std::isinf(pref->beta) || pref->smoothing < 0 ||
      pref->smoothing > 1 || pref->form < SNACK_PREF_SIGMOID || pref->form > SNACK_PREF_SQUARED ||
      (pref->smoothing > 0 && pref->form != SNACK_PREF_SIGMOID))
    return SNACK_E_SHAPE;
  if (batch->T > 0 && !logps) return SNACK_E_NULL;
  const __int128 t = 4 * (__int128)batch->T, n = batch->S;
  const plan_t p = plan_of(batch->S, batch->T, false);
  const span_t out[] = {{loss, 4}, {rewards, 4 * n}, {dlogps, t}, {ws, (__int128)p.total}};
  const span_t in[] = {{logps, t}, {ref, t}, {dloss, 4}, {batch->starts, 4 * (n + 1)},
                       {batch->mask, batch->T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  const pref_t l{logps, ref, pref->beta, pref->smoothing, 2.0 / std::max(batch->S, 2), pref->form,
                 pref->average};
  return run(batch, p, l, out_t{dloss, loss, rewards, dlogps}, ws, ws_bytes,
             reinterpret_cast<hipStream_t>(stream));
}

snack_status snack_policy_loss(const snack_seqs* batch, const snack_policy* policy,
                               const float* logps, const float* old, const float* ref,
                               const float* advantages, const float* dloss, float* loss,
                               float* stats, float* dlogps, void* ws, size_t ws_bytes,
                               void* stream) {
  if (!policy) return SNACK_E_NULL;
  if (snack_status st = check_batch(batch)) return st;
  if (std::isnan(policy->low) || std::isnan(policy->high) || std::isnan(policy->kl))
    return SNACK_E_NAN;
  if (policy->low < 0 || policy->low > 1 || policy->high < 0 || policy->kl < 0)
    return SNACK_E_SHAPE;
  const int64_t na = policy->by_token ? batch->T : batch->S;
  if ((batch->T > 0 && !logps) || (na > 0 && !advantages)) return SNACK_E_NULL;
  const __int128 t = 4 * (__int128)batch->T, n = batch->S;
  const plan_t p = plan_of(batch->S, batch->T, true);
  const span_t out[] = {{loss, 4}, {stats, 8}, {dlogps, t}, {ws, (__int128)p.total}};
  const span_t in[] = {{logps, t}, {old, t}, {ref, t}, {advantages, 4 * (__int128)na}, {dloss, 4},
                       {batch->starts, 4 * (n + 1)}, {batch->mask, batch->T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  const policy_t l{logps, old, ref, advantages, std::log1p(-policy->low), std::log1p(policy->high),
                   (float)(1.0 - policy->low), (float)(1.0 + policy->high), (float)policy->kl,
                   policy->by_token, policy->sequence_mean};
  return run(batch, p, l, out_t{dloss, loss, stats, dlogps}, ws, ws_bytes,
             reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
