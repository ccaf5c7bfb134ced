// The clipped policy loss with a KL term.  For a row's token with
// logp = log softmax(x / tau)[token], r = exp(logp - old), d = ref - logp:
//     l = -min(r A, clamp(r, 1 - lo, 1 + hi) A) + kl (exp(d) - d - 1)
//     dl/dlogp = -[r A <= clamp(r) A] r A + kl (1 - exp(d))
//     dx[v] = dl/dlogp / tau ([v = token] - q[v])
// A row with weight 0 or a token outside the vocabulary adds nothing.
//
// The token's logit and the row's few numbers are scalar loads, the loss is formed
// by one lane.  8192 x 65536 bf16 with gradient, a tenth of the rows masked: 379 us
// (5.4 TB/s); 32 x 65536 forward 9 us; the gradient alone, 2048 x 100003 fp32 to
// bf16, 192 us (6.0 TB/s).  The log-probabilities alone take the same walk.
#include "vocab_loss.h"

namespace moe {
namespace {

using vocab::exp2_of;
using vocab::Logits;

struct Policy {
  struct Args {
    const int* tok;
    const float* old_logp;
    const float* adv;  // nullptr: log-probabilities only
    const float* ref;  // nullptr: no KL term
    float* logp;
    float least, most;  // the ratio's bounds
    double kl;          // the KL term's weight
  };
  template <int NT>
  struct Shared {
    int tok;
    float x, k;
  };
  static constexpr bool kLateFactor = true;
  static int grad_pieces(const Args&) { return 2; }

  template <typename S>
  static __device__ __forceinline__ void init(S&, int) {}
  static __device__ __forceinline__ bool live(const Args& k, int64_t row, int V) {
    return static_cast<unsigned>(vocab::scalar_of(k.tok + row)) < static_cast<unsigned>(V);
  }
  struct Ahead {};
  static __device__ __forceinline__ Ahead ahead(const Args&, int64_t, int) { return {}; }
  template <typename TX>
  struct Few {
    int tok;
    float x;
  };
  template <typename TX>
  static __device__ __forceinline__ Few<TX> begin(const Logits&, const Args& k, int64_t row, const TX* x, int, Ahead) {
    const int tok = vocab::scalar_of(k.tok + row);
    return {tok, vocab::scalar_logit(x, tok)};
  }
  template <typename TX, typename S>
  static __device__ __forceinline__ void share(const Logits&, const Args&, int64_t, const TX*, bool,
                                               const vocab::Owner&, int lane, const Few<TX>& few, S& sh) {
    if (lane != 0) return;
    sh.tok = few.tok;
    sh.x = few.x;
  }

  // The differences of log-probabilities in fp64 (their absolute error is the
  // ratio's relative one).  Near 0 the exponentials are formed in fp32 with the
  // exponent's rounding error carried; elsewhere, and beside a huge advantage or KL
  // weight, the row's few numbers are fp64, which holds products that fp32 holds only
  // after the row's weight.  (fp64 in every row: 65536 x 256 forward 41 us, 39 so.)
  template <typename S>
  static __device__ __forceinline__ void finish(const Logits& p, const Args& k, int64_t row, float gw, float m,
                                                float sum, int lane, S& sh, bool outputs) {
    if (lane != 0) return;
    const double logp = (static_cast<double>(sh.x) - static_cast<double>(m)) * p.inv_tau - vocab::ln_of(sum);
    if (outputs) {
      k.logp[row] = static_cast<float>(logp);
      p.stats[2 * row] = m;
      p.stats[2 * row + 1] = sum;
    }
    if (k.adv == nullptr) return;
    const float a = vocab::scalar_of(k.adv + row);
    const double move = logp - static_cast<double>(vocab::scalar_of(k.old_logp + row));
    const double d = k.ref != nullptr ? static_cast<double>(vocab::scalar_of(k.ref + row)) - logp : 0.0;
    float l, slope;
    if (fabs(move) < kNear && fabs(d) < kNear && fabsf(a) < kSmall && k.kl < kSmall) {
      const float r = exp_of(static_cast<float>(move));
      const float free = r * a, cut = fminf(fmaxf(r, k.least), k.most) * a;
      l = free > cut ? -cut : -free;
      slope = free > cut ? 0.0f : -free;
      if (k.ref != nullptr) {
        const float df = static_cast<float>(d), g = gap_of(df);
        const float kl = static_cast<float>(k.kl);
        l += kl * g;
        slope -= kl * (fabsf(df) < 0.5f ? df + g : exp_of(df) - 1.0f);
      }
      sh.k = within(-slope * p.inv_tau_f * gw);
    } else {
      // an advantage of 0 counts 0 beside any ratio
      const double r = wide_exp_of(move), free = a == 0.0f && r == INFINITY ? 0.0 : r * a;
      const double cut = fmin(fmax(r, static_cast<double>(k.least)), static_cast<double>(k.most)) * a;
      double wide = free > cut ? -cut : -free, s = free > cut ? 0.0 : -free;
      if (k.ref != nullptr) {
        const double e = wide_exp_of(d);
        const bool small = fabs(d) < 0.5;
        const double g = small ? gap_of(static_cast<float>(d)) : e < INFINITY ? e - d - 1.0 : e;
        wide += k.kl * g;
        s -= k.kl * (small ? d + g : e - 1.0);
      }
      l = static_cast<float>(wide);
      s = s > 1e200 ? 1e200 : s < -1e200 ? -1e200 : s;
      sh.k = within(-s * p.inv_tau * static_cast<double>(gw));
    }
    if (outputs) p.row_loss[row] = l;
  }
  static constexpr double kNear = 40.0;  // e^40 1e20 is an fp32 number
  static constexpr float kSmall = 1e20f;
  // held to fp32's range, so that entries of probability 0 keep a gradient of 0 (NaN stays)
  template <typename F>
  static __device__ __forceinline__ float within(F v) {
    return v > FLT_MAX ? FLT_MAX : v < -FLT_MAX ? -FLT_MAX : static_cast<float>(v);
  }
  // |v| up to kNear
  static __device__ __forceinline__ float exp_of(float v) {
    const float t = v * 1.44269504f, lo = __builtin_fmaf(v, 1.44269504f, -t) + v * 1.92596299e-8f;
    const float e = exp2_of(t);
    return __builtin_fmaf(e, lo * 0.693147181f, e);
  }
  // any v, to 3 2^-24: a power of 2 and the fraction's exponential
  static __device__ __forceinline__ double wide_exp_of(double v) {
    v = v > 800.0 ? 800.0 : v < -800.0 ? -800.0 : v;  // infinity and 0 there already; NaN stays
    const double t = v * 1.4426950408889634, n = rint(t);
    const float e = exp2_of(static_cast<float>(t - n));
    return ldexp(static_cast<double>(e), n == n ? static_cast<int>(n) : 0);
  }
  // exp(d) - d - 1; near 0, where that would cancel, as its series to d^10
  static __device__ __forceinline__ float gap_of(float d) {
    if (!(fabsf(d) < 0.5f)) return exp_of(d) - d - 1.0f;
    float s = 1.0f / 3628800;
    constexpr float kInv[] = {1.0f / 362880, 1.0f / 40320, 1.0f / 5040, 1.0f / 720,
                              1.0f / 120,    1.0f / 24,    1.0f / 6,    0.5f};
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(s, d, kInv[i]);
    return s * d * d;
  }

  template <typename S>
  static __device__ __forceinline__ float factor(const Logits&, float, const S& sh) {
    return sh.k;
  }

  template <typename TX, typename S>
  static __device__ __forceinline__ void entries(const Logits& p, const Args& k, int64_t row, const TX* x,
                                                 const vocab::Owner& owner, int, int, int lane, S& sh) {
    share<TX>(p, k, row, x, true, owner, lane, begin<TX>(p, k, row, x, lane, {}), sh);
  }
  // the token
  template <typename S>
  static __device__ __forceinline__ int mine(const vocab::Owner&, const S& sh, int, bool any) {
    return any ? sh.tok : -1;
  }
  template <int E, typename S>
  static __device__ __forceinline__ void correct(S&, int tok, int, int piece, float kr, int, float (&f)[E]) {
    const int i = tok - piece * E;
    if (i < 0 || i >= E) return;
#pragma unroll
    for (int l = 0; l < E; ++l) f[l] = l == i ? f[l] - kr : f[l];
  }
  template <typename S>
  static __device__ __forceinline__ float correct_one(S&, int tok, int at, float kr, int, float f) {
    return tok == at ? f - kr : f;
  }
  template <typename S>
  static __device__ __forceinline__ void done(S&, int) {}

  static __device__ __forceinline__ void none(const Logits& p, const Args& k, int64_t row) {
    p.stats[2 * row] = p.stats[2 * row + 1] = k.logp[row] = 0.0f;
    if (k.adv != nullptr) p.row_loss[row] = 0.0f;
  }
};

}  // namespace

hipError_t launch_policy_loss(int64_t rows, int V, const void* x, int x_dtype, const int32_t* tok,
                              const float* old_logp, const float* adv, const float* ref, double lo, double hi,
                              double kl, double tau, const float* weight, const float* grad, float* loss,
                              float* row_loss, float* logp, float* stats, void* dx, int dx_dtype, hipStream_t s) {
  if (rows > 0) {
    Logits p = vocab::logits_of(rows, V, tau, weight, grad);
    p.x = x;
    p.dx = dx;
    p.stats = stats;
    p.row_loss = row_loss;
    const Policy::Args k{tok, old_logp, adv, ref, logp, static_cast<float>(1.0 - lo),
                         static_cast<float>(1.0 + hi), kl};
    const hipError_t e = vocab::loss_dtypes<Policy>(p, k, x_dtype, dx_dtype, s);
    if (e != hipSuccess || loss == nullptr) return e;
  }
  if (loss == nullptr) return hipSuccess;
  return launch_loss_sum(rows, row_loss, weight, rows > 0 ? static_cast<float>(1.0 / static_cast<double>(rows)) : 0.0f,
                         loss, s);
}

hipError_t launch_policy_loss_bwd(int64_t rows, int V, const void* x, int x_dtype, const float* stats,
                                  const int32_t* tok, const float* old_logp, const float* adv, const float* ref,
                                  double lo, double hi, double kl, double tau, const float* weight, const float* grad,
                                  void* dx, int dx_dtype, hipStream_t s) {
  Logits p = vocab::logits_of(rows, V, tau, weight, grad);
  p.x = x;
  p.dx = dx;
  p.stats = const_cast<float*>(stats);  // read only
  const Policy::Args k{tok, old_logp, adv, ref, nullptr, static_cast<float>(1.0 - lo),
                       static_cast<float>(1.0 + hi), kl};
  return vocab::grad_dtypes<Policy>(p, k, x_dtype, dx_dtype, s);
}

}  // namespace moe
