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
// Both need a sum over each sequence (or over all of them) before any token's
// gradient: k_seq_sums leaves sums of slices of the sequences, k_seq_grads adds
// them up again in each workgroup that needs them and writes the gradients and
// the loss.  Batches of a few thousand tokens take one workgroup and one launch
// (k_seq_small), for two launches cost more than what they would share.  Sums
// are 64-bit in a fixed order; whether a ratio is past its border is decided
// on logarithms in 64 bits.  A token's terms are fp32.  Bound by memory where the
// batch is large: two to five floats a token, read twice (the second time from
// the caches up to 256 MB), and one written.
#include <cmath>

#include "common.h"
#include "internal.h"
#include "spans.h"

namespace snk {
namespace {

// ---------------------------------------------------------------- sequences
struct batch_t {
  const int32_t* starts;  // [S + 1], or NULL: T / S tokens each
  const uint8_t* mask;    // [T], or NULL: every token counts
  int32_t S, T, each;
};
struct span2 { int32_t a, b; };

// Places that do not fit are cut to [0, T], so a call with wrong ones stays
// inside its arrays.
__device__ __forceinline__ span2 seq_of(const batch_t& q, int32_t i) {
  if (!q.starts) return {i * q.each, (i + 1) * q.each};
  const int32_t a = min(max(q.starts[i], 0), q.T);
  return {a, min(max(q.starts[i + 1], a), q.T)};
}
// Slice c of C.
__device__ __forceinline__ span2 slice_of(span2 s, int32_t c, int32_t C) {
  const int64_t n = s.b - s.a;
  return {s.a + (int32_t)(n * c / C), s.a + (int32_t)(n * (c + 1) / C)};
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// The sums of a sequence or a part of it.  Preference: f is d's sum.
struct sums_t { double f, kl, cut; int64_t n; };
__device__ __forceinline__ sums_t operator+(const sums_t& a, const sums_t& b) {
  return {a.f + b.f, a.kl + b.kl, a.cut + b.cut, a.n + b.n};
}
__device__ __forceinline__ sums_t wave_sum(const sums_t& a) {
  sums_t o = a;
#pragma unroll
  for (int d = 32; d; d >>= 1)
    o = o + sums_t{__shfl_xor(o.f, d), __shfl_xor(o.kl, d), __shfl_xor(o.cut, d),
                   (int64_t)__shfl_xor((long long)o.n, d)};
  return o;
}

// ---------------------------------------------------------------- preference
struct pref_t {
  const float *logps, *ref;
  double beta, eps;
  int32_t form, average;

  __device__ __forceinline__ void add(sums_t& s, int32_t i, int32_t) const {
    s.f += ref ? (double)logps[i] - (double)ref[i] : (double)logps[i];
    s.n += 1;
  }
  __device__ __forceinline__ double per(const sums_t& s) const {
    return average ? 1.0 / (double)max(s.n, (int64_t)1) : 1.0;
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
    const double up = 1.0 / (1.0 + t), down = t / (1.0 + t);
    const double sig = z >= 0 ? up : down, not_sig = z >= 0 ? down : up;
    *dh = beta * (eps * sig - (1.0 - eps) * not_sig);
    const double a = (1.0 - eps) * (soft + fmax(-z, 0.0)), b = eps * (soft + fmax(z, 0.0));
    return eps > 0.0 ? a + b : a;  // eps 0: no product of 0 and infinity
  }
};

// -------------------------------------------------------------------- policy
struct policy_t {
  const float *logps, *old, *ref, *adv;
  double log_low, log_high;  // of 1 - low and 1 + high
  float low, high, kl;
  int32_t by_token, by_sequence_mean;

  struct token_t { float f, df, kl; bool cut; };

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
      s = *em1 - k;
    }
    return s;
  }

  __device__ __forceinline__ token_t token(int32_t i, int32_t seq) const {
    const float lp = logps[i], a = adv[by_token ? i : seq];
    const double move = old ? (double)lp - (double)old[i] : (double)lp - (double)lp;
    const float r = expf((float)move);
    token_t o;
    o.cut = (a > 0.f && move > log_high) || (a < 0.f && move < log_low);
    o.f = o.cut ? -(a > 0.f ? high : low) * a : -r * a;
    o.df = o.cut ? 0.f : -r * a;
    o.kl = 0.f;
    if (ref) {
      float em1;
      o.kl = above((float)((double)ref[i] - (double)lp), &em1);
      o.f = fmaf(kl, o.kl, o.f);
      o.df = fmaf(-kl, em1, o.df);
    }
    return o;
  }
  __device__ __forceinline__ void add(sums_t& s, int32_t i, int32_t seq) const {
    const token_t o = token(i, seq);
    s.f += o.f;
    s.kl += o.kl;
    s.cut += o.cut;
    s.n += 1;
  }
};

// Threads first, first + step, ... of [s.a, s.b).
template <typename L>
__device__ __forceinline__ sums_t sum_slice(const batch_t& q, const L& loss, span2 s, int32_t seq,
                                            int32_t first, int32_t step) {
  sums_t o{0, 0, 0, 0};
#pragma unroll 4
  for (int64_t i = (int64_t)s.a + first; i < s.b; i += step)
    if (!q.mask || q.mask[i]) loss.add(o, (int32_t)i, seq);
  return o;
}

struct out_t {
  const float* dloss;  // device, or NULL: 1
  float* loss;         // or NULL
  float* more;         // rewards [S] or stats [2], or NULL
  float* grad;         // [T], or NULL
};

// What a token's gradient takes from sums: preference, the coefficient of a
// whole sequence; policy, the weight of its tokens.
struct totals_t { int64_t n; };

__device__ __forceinline__ double weight_of(const policy_t& l, const batch_t& q, const sums_t& seq,
                                            const totals_t& all) {
  return l.by_sequence_mean ? 1.0 / ((double)q.S * (double)max(seq.n, (int64_t)1))
                            : 1.0 / (double)max(all.n, (int64_t)1);
}

template <typename L>
__device__ __forceinline__ void write_slice(const batch_t& q, const L& loss, span2 s, int32_t seq,
                                            double c, float* grad, int32_t first, int32_t step) {
#pragma unroll 4
  for (int64_t i = (int64_t)s.a + first; i < s.b; i += step) {
    float g = 0.f;
    if (!q.mask || q.mask[i]) {
      if constexpr (std::is_same<L, pref_t>::value) g = (float)c;
      else g = (float)((double)loss.token((int32_t)i, seq).df * c);
    }
    grad[i] = g;
  }
}

// Tokens of no sequence: their gradient is 0.
__device__ __forceinline__ void write_outside(const batch_t& q, float* grad, int64_t first,
                                              int64_t step) {
  if (!q.starts || q.S == 0) {
    const int64_t from = (int64_t)q.S * q.each;
    for (int64_t i = from + first; i < q.T; i += step) grad[i] = 0.f;
    return;
  }
  const int32_t a = seq_of(q, 0).a, b = seq_of(q, q.S - 1).b;
  for (int64_t i = first; i < a; i += step) grad[i] = 0.f;
  for (int64_t i = (int64_t)b + first; i < q.T; i += step) grad[i] = 0.f;
}

// -------------------------------------------------------- one workgroup, one launch
constexpr int SMALL_WAVES = 16;
constexpr int32_t SMALL_SEQS = 256, SMALL_TOKENS = 8192;

template <typename L>
__global__ __launch_bounds__(SMALL_WAVES * 64) void k_seq_small(batch_t q, L loss, out_t out) {
  __shared__ sums_t sums[SMALL_SEQS];
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), lane = lane_id();
  for (int32_t i = w; i < q.S; i += SMALL_WAVES) {
    const sums_t s = wave_sum(sum_slice(q, loss, seq_of(q, i), i, lane, 64));
    if (lane == 0) sums[i] = s;
  }
  __syncthreads();
  const double up = out.dloss ? (double)*out.dloss : 1.0;
  if constexpr (std::is_same<L, pref_t>::value) {
    const double share = 1.0 / (double)max(q.S / 2, 1);
    if (w == 0) {
      double f = 0;
      for (int32_t p = lane; p < q.S / 2; p += 64) {
        const sums_t &a = sums[2 * p], &b = sums[2 * p + 1];
        const double da = a.f * loss.per(a), db = b.f * loss.per(b);
        double dh;
        f += loss.pair(da - db, &dh);
        if (out.more) {
          out.more[2 * p] = (float)(loss.beta * da);
          out.more[2 * p + 1] = (float)(loss.beta * db);
        }
      }
      f = wave_sum(f);
      if (lane == 0 && out.loss) *out.loss = (float)(f * share);
    }
    if (!out.grad) return;
    for (int32_t i = w; i < q.S; i += SMALL_WAVES) {
      const sums_t &a = sums[i & ~1], &b = sums[i | 1];
      double dh;
      loss.pair(a.f * loss.per(a) - b.f * loss.per(b), &dh);
      const double c = (i & 1 ? -dh : dh) * loss.per(sums[i]) * share * up;
      write_slice(q, loss, seq_of(q, i), i, c, out.grad, lane, 64);
    }
  } else {
    sums_t s{0, 0, 0, 0};
    totals_t all{0};
    for (int32_t i = lane; i < q.S; i += 64) s = s + sums[i];
    s = wave_sum(s);
    all.n = s.n;
    if (w == 0) {
      double f = 0;
      for (int32_t i = lane; i < q.S; i += 64)
        f += sums[i].f * weight_of(loss, q, sums[i], all);
      f = wave_sum(f);
      const double n = (double)max(s.n, (int64_t)1);
      if (lane == 0) {
        if (out.loss) *out.loss = (float)f;
        if (out.more) out.more[0] = (float)(s.kl / n), out.more[1] = (float)(s.cut / n);
      }
    }
    if (!out.grad) return;
    for (int32_t i = w; i < q.S; i += SMALL_WAVES)
      write_slice(q, loss, seq_of(q, i), i, weight_of(loss, q, sums[i], all) * up, out.grad, lane,
                  64);
  }
  write_outside(q, out.grad, threadIdx.x, SMALL_WAVES * 64);
}

// ------------------------------------------------------------------ two launches
// Item x is slice x % C of sequence x / C; ws has its sums.
template <typename L>
__global__ __launch_bounds__(256) void k_seq_sums(batch_t q, L loss, int32_t C,
                                                  sums_t* __restrict__ ws) {
  __shared__ sums_t lds[4];
  for (int64_t x = blockIdx.x; x < (int64_t)q.S * C; x += gridDim.x) {
    const int32_t i = (int32_t)(x / C);
    const sums_t s = wave_sum(sum_slice(q, loss, slice_of(seq_of(q, i), (int32_t)(x % C), C), i,
                                        threadIdx.x, 256));
    if (lane_id() == 0) lds[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) ws[x] = ((lds[0] + lds[1]) + lds[2]) + lds[3];
    __syncthreads();
  }
}

__device__ __forceinline__ sums_t seq_sums(const sums_t* __restrict__ ws, int32_t i, int32_t C) {
  sums_t s{0, 0, 0, 0};
  for (int32_t c = 0; c < C; ++c) s = s + ws[(int64_t)i * C + c];
  return s;
}
// One value a thread, added in a fixed order; all threads get it.
__device__ __forceinline__ sums_t block_sum(sums_t s, sums_t* lds) {
  s = wave_sum(s);
  if (lane_id() == 0) lds[threadIdx.x / 64] = s;
  __syncthreads();
  s = ((lds[0] + lds[1]) + lds[2]) + lds[3];
  __syncthreads();
  return s;
}

// The last workgroup writes the loss and the sums' means, the others gradients.
template <typename L>
__global__ __launch_bounds__(256) void k_seq_grads(batch_t q, L loss, int32_t C,
                                                   const sums_t* __restrict__ ws, out_t out) {
  __shared__ sums_t lds[4];
  const double up = out.dloss ? (double)*out.dloss : 1.0;
  const bool last = blockIdx.x + 1 == gridDim.x;
  const int32_t t = threadIdx.x, grads = (int32_t)gridDim.x - 1;
  const int64_t items = (int64_t)q.S * C;
  if constexpr (std::is_same<L, pref_t>::value) {
    const double share = 1.0 / (double)max(q.S / 2, 1);
    if (last) {
      sums_t f{0, 0, 0, 0};
      for (int32_t p = t; p < q.S / 2; p += 256) {
        const sums_t a = seq_sums(ws, 2 * p, C), b = seq_sums(ws, 2 * p + 1, C);
        const double da = a.f * loss.per(a), db = b.f * loss.per(b);
        double dh;
        f.f += loss.pair(da - db, &dh);
        if (out.more) {
          out.more[2 * p] = (float)(loss.beta * da);
          out.more[2 * p + 1] = (float)(loss.beta * db);
        }
      }
      f = block_sum(f, lds);
      if (t == 0 && out.loss) *out.loss = (float)(f.f * share);
      return;
    }
    for (int64_t x = blockIdx.x; x < items; x += grads) {
      const int32_t i = (int32_t)(x / C);
      const sums_t a = seq_sums(ws, i & ~1, C), b = seq_sums(ws, i | 1, C);
      double dh;
      loss.pair(a.f * loss.per(a) - b.f * loss.per(b), &dh);
      const double c = (i & 1 ? -dh * loss.per(b) : dh * loss.per(a)) * share * up;
      write_slice(q, loss, slice_of(seq_of(q, i), (int32_t)(x % C), C), i, c, out.grad, t, 256);
    }
  } else {
    totals_t all{0};
    if (last || !loss.by_sequence_mean) {
      sums_t s{0, 0, 0, 0};
      if (last) for (int64_t x = t; x < items; x += 256) s = s + ws[x];
      else for (int64_t x = t; x < items; x += 256) s.n += ws[x].n;
      s = block_sum(s, lds);
      all.n = s.n;
      if (last) {
        sums_t f{0, 0, 0, 0};
        for (int32_t i = t; i < q.S; i += 256) {
          const sums_t o = seq_sums(ws, i, C);
          f.f += o.f * weight_of(loss, q, o, all);
        }
        f = block_sum(f, lds);
        const double n = (double)max(s.n, (int64_t)1);
        if (t == 0) {
          if (out.loss) *out.loss = (float)f.f;
          if (out.more) out.more[0] = (float)(s.kl / n), out.more[1] = (float)(s.cut / n);
        }
        return;
      }
    }
    for (int64_t x = blockIdx.x; x < items; x += grads) {
      const int32_t i = (int32_t)(x / C);
      sums_t own{0, 0, 0, 0};
      if (loss.by_sequence_mean) own = seq_sums(ws, i, C);
      write_slice(q, loss, slice_of(seq_of(q, i), (int32_t)(x % C), C), i,
                  weight_of(loss, q, own, all) * up, out.grad, t, 256);
    }
  }
  write_outside(q, out.grad, (int64_t)blockIdx.x * 256 + t, (int64_t)grads * 256);
}

// ---------------------------------------------------------------------- host
constexpr int32_t MAX_SEQS = 1 << 24;

struct plan_t { bool small; int32_t C, blocks; size_t total; };

plan_t plan_of(int32_t S, int32_t Tn) {
  plan_t p{};
  p.small = S <= SMALL_SEQS && Tn <= SMALL_TOKENS;
  // slices: workgroups for every CU to have four, 1,024 tokens each at least
  p.C = (int32_t)std::max<int64_t>(
      1, std::min<int64_t>(1024 / std::max(S, 1), cdiv(Tn, 1024ll * std::max(S, 1))));
  p.blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>((int64_t)S * p.C, 2048));
  p.total = p.small ? 0 : (size_t)S * p.C * sizeof(sums_t);
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
snack_status run(const snack_seqs* b, const L& loss, const out_t& out, void* ws, size_t ws_bytes,
                 hipStream_t s) {
  const plan_t p = plan_of(b->S, b->T);
  if (p.total > 0 && !ws) return SNACK_E_NULL;
  if (ws_bytes < p.total) return SNACK_E_WORKSPACE;
  const batch_t q{b->starts, b->mask, b->S, b->T, b->S > 0 ? b->T / b->S : 0};
  if (p.small) {
    hipLaunchKernelGGL(k_seq_small<L>, dim3(1), dim3(SMALL_WAVES * 64), 0, s, q, loss, out);
  } else {
    hipLaunchKernelGGL(k_seq_sums<L>, dim3(p.blocks), dim3(256), 0, s, q, loss, p.C, (sums_t*)ws);
    hipLaunchKernelGGL(k_seq_grads<L>, dim3(out.grad ? p.blocks + 1 : 1), dim3(256), 0, s, q, loss,
                       p.C, (const sums_t*)ws, out);
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
  *bytes = plan_of(S, T).total;
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
  const plan_t p = plan_of(batch->S, batch->T);
  const span_t out[] = {{loss, 4}, {rewards, 4 * n}, {dlogps, t}, {ws, (__int128)p.total}};
  const span_t in[] = {{logps, t}, {ref, t}, {dloss, 4}, {batch->starts, 4 * (n + 1)},
                       {batch->mask, batch->T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  const pref_t l{logps, ref, pref->beta, pref->smoothing, pref->form, pref->average};
  return run(batch, l, out_t{dloss, loss, rewards, dlogps}, ws, ws_bytes,
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
  const plan_t p = plan_of(batch->S, batch->T);
  const span_t out[] = {{loss, 4}, {stats, 8}, {dlogps, t}, {ws, (__int128)p.total}};
  const span_t in[] = {{logps, t}, {old, t}, {ref, t}, {advantages, 4 * (__int128)na}, {dloss, 4},
                       {batch->starts, 4 * (n + 1)}, {batch->mask, batch->T}};
  if (any_overlap(out, in)) return SNACK_E_SHAPE;
  const policy_t l{logps, old, ref, advantages, std::log1p(-policy->low), std::log1p(policy->high),
                   (float)(1.0 - policy->low), (float)(1.0 + policy->high), (float)policy->kl,
                   policy->by_token, policy->sequence_mean};
  return run(batch, l, out_t{dloss, loss, stats, dlogps}, ws, ws_bytes,
             reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
