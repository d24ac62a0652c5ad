// Token log probabilities, the preference loss over paired sequences, the
// clipped policy loss with a KL term, and the gradient of their logits.
//
//   lse_t = log sum_j exp(x[t, j]),  logp_t = x[t, y_t] - lse_t
//   dx[t, j] = c_t * ([j = y_t] - exp(x[t, j] - lse_t))
//
// Both losses depend on the logits only through logp, so every gradient is
// the same rank-one correction of a softmax with a coefficient c_t for each
// token. A token whose target lies outside [0, V) is masked: its row is never
// read, its logp is 0 and its gradient row is zeros.
//
// The softmax's statistics of a row are its largest logit m and the sum s of
// exp(x - m): exp(x - m) / s keeps the precision that
// exp(x - lse) would lose to the rounding of a large lse.
//
// A likely target leaves little to the others: with t their sum, 1 - p is
// t / s and logp is -log(1 + t), and both keep t's precision only if t is
// summed without the target's own term. So it is summed so everywhere, and
// the gradient at the target, c (1 - p), comes from logp as -c expm1(logp).
//
// Kernels:
//   logp_kernel       one pass over a row (or one piece of it): running max and sum
//   join_kernel       the pieces of a row joined, four lanes per row
//   pref_kernel       sequence sums, the loss and each token's coefficient
//   policy_kernel     each token's loss and coefficient, and their sum
//   policy_row_kernel a row from its statistics to its gradient (policy loss)
//   sum_kernel        the sum of the tokens' losses
//   target_kernel     the gradient's entries at likely targets from the statistics
//   logit_grad_kernel the gradient's rows from the statistics and coefficients
//   policy_grad_kernel  the same from the pieces of few long rows, and the policy loss

#include <cmath>
#include <type_traits>

#include "lora_softmax.hpp"

namespace lora {

// exp(d) by the base-2 instruction. log2(e) is carried as a float32 and its
// rest: the float32 alone is off by 1.3e-8 of every exponent, to the same side
// in all terms of a sum (1.6e-7 of them for d from -16 to -8, 5e-9 with the
// rest). One product more, which costs the preference step of 8192 x 128256
// bfloat16 2 us of 794 and the policy step nothing.
__device__ __forceinline__ float exp_of(float d) {
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0c0p-26f;
  return __builtin_amdgcn_exp2f(fmaf(d, kLog2e, d * kRest));
}

// Running maximum m and sum s of exp(x - m). With nothing seen (or only
// -inf) m is -inf and s is 0; +inf and NaN give a NaN sum, as the formula
// does, and values of the type's lowest magnitude are ordinary values.
//
// s is float64 and takes the sum of a batch at a time, which is added up as a
// tree: a hundred thousand terms one after the other in float32 lose what is
// small among them. The target's term is left out of it (see above).
struct MaxSum {
  float m;
  double s;
};

template <int N>
__device__ __forceinline__ float sum_exp(const float* f, float z) {
  if constexpr (N == 1)
    return exp_of(f[0] - z);
  else
    return sum_exp<N / 2>(f, z) + sum_exp<N - N / 2>(f + N / 2, z);
}

template <int N>
__device__ __forceinline__ void add_values(MaxSum& r, const float* f) {
  float m = r.m;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, f[i]);
  const float z = at_max(m);
  r = {m, r.s * exp_of(r.m - z) + sum_exp<N>(f, z)};
}

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  const float z = at_max(m);
  return {m, a.s * exp_of(a.m - z) + b.s * exp_of(b.m - z)};
}

// The wave's maximum first, then every lane's sum brought to it once.
__device__ __forceinline__ MaxSum wave_join(MaxSum v) {
  float m = v.m;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  return {m, wave_sum(v.s * exp_of(v.m - at_max(m)))};
}

// A whole row from its target's logit x and the others: the statistics, and
// logp in float64, rounded once: a loss is a small difference of many, and a
// float32 logarithm of 10 is off by 5e-7.
struct RowStats {
  float x, m, e;  // the target's logit, the largest one, exp(x - m)
  double t;       // the others' sum
  __device__ __forceinline__ float sum() const { return static_cast<float>(t + e); }
  __device__ __forceinline__ float logp() const {
    // t + e is at least 1; with a target that is the largest e - 1 is 0 and t keeps its own precision
    return static_cast<float>(((double)x - m) - log1p(t + ((double)e - 1.0)));
  }
};
__device__ __forceinline__ RowStats with_target(MaxSum others, float x) {
  const float m = fmaxf(others.m, x);
  const float z = at_max(m);
  return {x, m, exp_of(x - z), others.s * exp_of(others.m - z)};
}

// One read of the row or piece, four 16-byte loads per lane in flight, each
// used once (non-temporal: by the default policy 8% slower): 8192 rows of
// 128256 bfloat16, 1.39 GB of them unmasked, in 217 us (6.4 TB/s, where a
// plain read reaches 6.7).
template <class E>
__global__ __launch_bounds__(256) void logp_kernel(const E* __restrict__ x, int64_t stride,
                                                   const int32_t* __restrict__ targets, int V, int splits, int piece,
                                                   float* __restrict__ logp, float2* __restrict__ stats,
                                                   MaxSum* __restrict__ part, float* __restrict__ hits) {
  constexpr int N = Vec<E>::N, U = 4;
  __shared__ MaxSum waves[4];
  const int64_t row = blockIdx.x / (unsigned)splits;
  const int sp = (int)(blockIdx.x % (unsigned)splits);
  const int tid = threadIdx.x;
  const int y = targets[row];
  if (y < 0 || y >= V) {
    if (splits == 1 && tid == 0) {
      logp[row] = 0.0f;
      stats[row] = make_float2(0.0f, 1.0f);
    }
    return;
  }
  const E* src = x + row * stride;
  const int lo = sp * piece;
  const int n = V - lo < piece ? V - lo : piece;
  const E* p = src + lo;
  const int vecs = n / N;
  const int hit = y >= lo && y - lo < n ? y - lo : -1;
  const LeftOut<E> target(hit, vecs);
  MaxSum r{-INFINITY, 0.0};
  int i = tid;
  for (; i + (U - 1) * 256 < vecs; i += U * 256) {
    float f[U * N];
    typename Vec<E>::type w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = vload_nt(p + (int64_t)(i + u * 256) * N);
    target.template from<U>(w, i, 256);
#pragma unroll
    for (int u = 0; u < U; ++u) Vec<E>::unpack(w[u], f + u * N);
    add_values<U * N>(r, f);
  }
  // at most U - 1 more, all loaded before the first is used
  typename Vec<E>::type w[U - 1];
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (i + u * 256 < vecs) w[u] = vload_nt(p + (int64_t)(i + u * 256) * N);
#pragma unroll
  for (int u = 0; u < U - 1; ++u) {
    if (i + u * 256 < vecs) {
      float f[N];
      target.template from<1>(w + u, i + u * 256, 1);
      Vec<E>::unpack(w[u], f);
      add_values<N>(r, f);
    }
  }
  if (tid < n - vecs * N && vecs * N + tid != hit) {
    const float f = Vec<E>::value(p[vecs * N + tid]);
    add_values<1>(r, &f);
  }
  MaxSum all = wave_join(r);
  if ((tid & 63) == 0) waves[tid >> 6] = all;
  __syncthreads();
  if (tid != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) all = join(all, waves[w]);
  if (splits > 1) {
    part[row * splits + sp] = all;
    // kept beside the pieces: the logits may be overwritten while they are joined
    if (hit >= 0) hits[row] = Vec<E>::value(src[y]);
  } else {
    const RowStats v = with_target(all, Vec<E>::value(src[y]));
    logp[row] = v.logp();
    stats[row] = make_float2(v.m, v.sum());
  }
}

// What remains of the softmax once logp_kernel has written `splits` pieces of
// each row: four lanes join a row's.
struct RowPieces {
  const int32_t* targets;
  int64_t V;
  int splits;
  const MaxSum* part;
  const float* hits;  // the rows' target logits
  float2* stats;
};

struct Joined {
  bool live;  // the row is there and not masked
  float m, sum, logp;
};

// Row `row` for lane `sub` of its four (all of them get the result).
__device__ __forceinline__ Joined join_row(const RowPieces& a, int64_t row, int64_t T, int sub) {
  constexpr int U = 8;
  const int y = row < T ? a.targets[row] : -1;
  const bool live = y >= 0 && y < a.V;
  const float hit = live ? a.hits[row] : 0.0f;
  MaxSum r{-INFINITY, 0.0};
  for (int sp = sub; sp < a.splits; sp += 4 * U) {
    MaxSum v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = live && sp + 4 * u < a.splits ? a.part[row * a.splits + sp + 4 * u] : MaxSum{-INFINITY, 0.0};
    float m = r.m;
#pragma unroll
    for (int u = 0; u < U; ++u) m = fmaxf(m, v[u].m);
    const float z = at_max(m);
    double s = r.s * exp_of(r.m - z);
#pragma unroll
    for (int u = 0; u < U; ++u) s += v[u].s * exp_of(v[u].m - z);
    r = {m, s};
  }
  r = join(r, MaxSum{__shfl_xor(r.m, 1, 64), __shfl_xor(r.s, 1, 64)});
  r = join(r, MaxSum{__shfl_xor(r.m, 2, 64), __shfl_xor(r.s, 2, 64)});
  if (!live) return {false, 0.0f, 1.0f, 0.0f};
  const RowStats v = with_target(r, hit);
  return {true, v.m, v.sum(), v.logp()};
}

__device__ __forceinline__ void put_joined(const RowPieces& a, int64_t row, int64_t T, const Joined& v, float* logp) {
  if (row >= T) return;
  logp[row] = v.logp;
  a.stats[row] = make_float2(v.m, v.sum);
}

__global__ __launch_bounds__(256) void join_kernel(RowPieces a, int64_t T, float* __restrict__ logp) {
  const int64_t row = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 2);
  const Joined v = join_row(a, row, T, threadIdx.x & 3);
  if ((threadIdx.x & 3) == 0) put_joined(a, row, T, v, logp);
}

// The same for up to kJoinRows rows in a workgroup of 1024 that goes on with
// their log probabilities, which it finds in `lds`.
constexpr int kJoinRows = 256;
__device__ __forceinline__ void join_rows(const RowPieces& a, int64_t T, float* logp, float* lds) {
  const int row = threadIdx.x >> 2;
  const Joined v = join_row(a, row, T, threadIdx.x & 3);
  if ((threadIdx.x & 3) == 0) {
    put_joined(a, row, T, v, logp);
    lds[row] = v.logp;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// losses on the log probabilities (one workgroup: a few values per token)
// ---------------------------------------------------------------------------

// z = beta * ((S_c - ref_c) - (S_r - ref_r)); loss = mean of
// -(1 - eps) log sigmoid(z) - eps log sigmoid(-z), whose derivative by z is
// eps - sigmoid(-z). Sequence sums and z are float64: z is a small
// difference of long sums. 64 pairs at a time: each wave sums sequences (or,
// with fewer than 8 pairs, a part of one), 64 lanes take a pair each, and the
// waves give their tokens the coefficients beta * dz / pairs and minus that.
// With JOIN the log probabilities are joined from their rows' pieces first.
// A chain of dependent loads and sums bounds it: 5.7 us for 8 pairs of 8192
// tokens, 6.3 for one pair of 96 with its join.
template <bool JOIN>
__global__ __launch_bounds__(1024) void pref_kernel(RowPieces pieces, float* logp_out, int64_t T,
                                                    const int32_t* __restrict__ offsets, int64_t pairs,
                                                    const float* __restrict__ ref, float beta, float eps,
                                                    float* __restrict__ loss, float* __restrict__ seq_logp,
                                                    float* __restrict__ coef) {
  constexpr int kBatch = 64;
  __shared__ double lds[16];
  __shared__ double sums[2 * kBatch];  // of sequences, or of the parts of each
  __shared__ float slope[kBatch];
  __shared__ float joined[JOIN ? kJoinRows : 1];
  if constexpr (JOIN) join_rows(pieces, T, logp_out, joined);
  auto logp = [&](int64_t t) { return JOIN ? joined[t] : logp_out[t]; };
  const int lane = threadIdx.x & 63;
  const int last = (int)T;  // below 2^25
  auto offset = [&](int64_t i) {
    const int o = offsets[i];
    return o < 0 ? 0 : (o > last ? last : o);
  };
  if (coef != nullptr) {
    // tokens before the first sequence and after the last
    const int a = offset(0), b = offset(2 * pairs);
    for (int t = threadIdx.x; t < a; t += 1024) coef[t] = 0.0f;
    for (int t = b + threadIdx.x; t < last; t += 1024) coef[t] = 0.0f;
  }
  // 2^split parts of a sequence, a wave for each
  const int split = pairs >= 8 ? 0 : pairs >= 4 ? 1 : pairs >= 2 ? 2 : 3;
  double total = 0.0;
  for (int64_t p0 = 0; p0 < pairs; p0 += kBatch) {
    const int batch = pairs - p0 < kBatch ? (int)(pairs - p0) : kBatch, units = 2 * batch << split;
    // read before the sums, used after them
    const int p = threadIdx.x;
    float r[2] = {};
    if (p < batch) {
      r[0] = ref[2 * (p0 + p)];
      r[1] = ref[2 * (p0 + p) + 1];
    }
    int lo = 0, hi = 0;  // the tokens of a unit
    auto range = [&](int u) {
      const int64_t s = 2 * p0 + (u >> split);
      const int a = offset(s), n = offset(s + 1) - a;
      const int step = n > 0 ? (n + (1 << split) - 1) >> split : 0;
      lo = a + (u & ((1 << split) - 1)) * step;
      hi = lo + step < a + n ? lo + step : a + n;
    };
    for (int u = wave_id(); u < units; u += 16) {
      range(u);
      double v = 0.0;
#pragma unroll 8
      for (int t = lo + lane; t < hi; t += 64) v += logp(t);
      v = wave_sum(v);
      if (lane == 0) sums[u] = v;
    }
    __syncthreads();
    if (p < batch) {
      double s[2] = {};
      for (int u = 0; u < 1 << split; ++u) {
        s[0] += sums[(2 * p << split) + u];
        s[1] += sums[(2 * p + 1 << split) + u];
      }
      const double z = (double)beta * ((s[0] - r[0]) - (s[1] - r[1]));
      const double e = exp(-fabs(z));
      const double down = (z >= 0.0 ? e : 1.0) / (1.0 + e);  // sigmoid(-z)
      slope[p] = static_cast<float>(((double)eps - down) * (double)beta / (double)pairs);
      const double l = log1p(e);
      // a weight of zero drops its term, also where that is infinite
      if (eps != 1.0f) total += (1.0 - (double)eps) * (l + fmax(-z, 0.0));
      if (eps != 0.0f) total += (double)eps * (l + fmax(z, 0.0));
      if (seq_logp != nullptr) {
        seq_logp[2 * (p0 + p)] = static_cast<float>(s[0]);
        seq_logp[2 * (p0 + p) + 1] = static_cast<float>(s[1]);
      }
    }
    __syncthreads();
    if (coef == nullptr) continue;
    for (int u = wave_id(); u < units; u += 16) {
      if (units > 16) range(u);
      const int s = u >> split;
      const float d = s & 1 ? -slope[s >> 1] : slope[s >> 1];
      for (int t = lo + lane; t < hi; t += 64) coef[t] = d;
    }
  }
  total = block_sum(total, lds);
  if (threadIdx.x == 0) *loss = static_cast<float>(total / (double)pairs);
}

struct PolicyArgs {
  const int32_t* targets;
  const float *old_logp, *ref_logp, *advantages, *weights;
  float clip_low, clip_high, kl;
};

// exp(k) - k - 1 with e = expm1(k): e - k loses it to the rounding of e near
// 0, where it is k^2 / 2. Its series ends within 2^-28 of it at 1/2.
__device__ __forceinline__ float exp_beyond_linear(float k, float e) {
  float s = 1.0f / 362880.0f;
  s = fmaf(s, k, 1.0f / 40320.0f);
  s = fmaf(s, k, 1.0f / 5040.0f);
  s = fmaf(s, k, 1.0f / 720.0f);
  s = fmaf(s, k, 1.0f / 120.0f);
  s = fmaf(s, k, 1.0f / 24.0f);
  s = fmaf(s, k, 1.0f / 6.0f);
  s = fmaf(s, k, 0.5f);
  return fabsf(k) < 0.5f ? s * (k * k) : e - k;
}

// One token of the policy loss: its weighted loss and d loss / d logp. The
// derivative is a difference of two terms that may nearly cancel, so every
// kernel has to round them alike: no products fused with sums here.
__device__ __forceinline__ float2 policy_token(const PolicyArgs& a, int64_t t, float lp) {
#pragma clang fp contract(off)
  const float ratio = expf(lp - a.old_logp[t]);
  const float held = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high);
  const float adv = a.advantages[t], w = a.weights[t];
  const bool clipped = ratio * adv > held * adv;  // the clipped surrogate is the smaller one
  float l = -(clipped ? held * adv : ratio * adv);
  float d = clipped ? 0.0f : -ratio * adv;
  if (a.ref_logp != nullptr) {
    const float k = a.ref_logp[t] - lp;
    const float e = expm1f(k);
    l += a.kl * exp_beyond_linear(k, e);
    d -= a.kl * e;
  }
  return make_float2(w * l, w * d);
}

__global__ __launch_bounds__(1024) void policy_kernel(const float* __restrict__ logp, int64_t T, int64_t V,
                                                      PolicyArgs a, float* __restrict__ loss,
                                                      float* __restrict__ coef) {
  __shared__ double lds[16];
  double sum = 0.0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const int y = a.targets[t];
    float2 v = make_float2(0.0f, 0.0f);
    if (y >= 0 && y < V) v = policy_token(a, t, logp[t]);
    sum += v.x;
    if (coef != nullptr) coef[t] = v.y;
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) *loss = static_cast<float>(sum);
}

// ---------------------------------------------------------------------------
// policy step: a token's coefficient needs nothing but its own row, so one
// workgroup takes a row from its statistics to its gradient. The row's last
// H vectors per lane stay in registers between the two passes; the others are
// read again, the most recently read first. 8192 x 128256 bfloat16 takes 638
// us: 1.39 GB of unmasked rows leave the L2 once and half of them a second
// time, 2.1 GB are written, and the vector units are three quarters busy.
// ---------------------------------------------------------------------------
template <class E, int WAVES, int H>
__global__ __launch_bounds__(64 * WAVES, 8) void policy_row_kernel(const E* x, int64_t stride, int V, PolicyArgs a,
                                                                   float scale, float* __restrict__ logp,
                                                                   float* __restrict__ terms, E* dx,
                                                                   int64_t dx_stride) {
  constexpr int N = Vec<E>::N, U = 4, THREADS = 64 * WAVES;
  __shared__ MaxSum waves[WAVES];
  __shared__ float shared_coef, shared_own;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int y = a.targets[row];
  const int vecs = V / N;
  const int rest = vecs * N + tid;  // the row's last elements, one per lane
  // dx may be x: no restrict on it, and a vector is stored by the lane that loaded it
  const E* p = x + row * stride;
  E* q = dx + row * dx_stride;
  if (y < 0 || y >= V) {
    const typename Vec<E>::type zero = {0u, 0u, 0u, 0u};
    for (int i = tid; i < vecs; i += THREADS) vstore_nt(q + (int64_t)i * N, zero);
    if (rest < V) q[rest] = Vec<E>::round(0.0f);
    if (tid == 0) logp[row] = terms[row] = 0.0f;
    return;
  }
  const int body = vecs > H * THREADS ? vecs - H * THREADS : 0;
  const LeftOut<E> target(y, vecs);
  MaxSum r{-INFINITY, 0.0};
  int i = tid;
  for (; i + (U - 1) * THREADS < body; i += U * THREADS) {
    float f[U * N];
    typename Vec<E>::type w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = vload(p + (int64_t)(i + u * THREADS) * N);
    target.template from<U>(w, i, THREADS);
#pragma unroll
    for (int u = 0; u < U; ++u) Vec<E>::unpack(w[u], f + u * N);
    add_values<U * N>(r, f);
  }
  for (; i < body; i += THREADS) {
    float f[N];
    typename Vec<E>::type w = vload(p + (int64_t)i * N);
    target.template from<1>(&w, i, 1);
    Vec<E>::unpack(w, f);
    add_values<N>(r, f);
  }
  typename Vec<E>::type held[H];
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (body + tid + h * THREADS < vecs) held[h] = vload_nt(p + (int64_t)(body + tid + h * THREADS) * N);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (body + tid + h * THREADS < vecs) {
      float f[N];
      typename Vec<E>::type w = held[h];
      target.template from<1>(&w, body + tid + h * THREADS, 1);
      Vec<E>::unpack(w, f);
      add_values<N>(r, f);
    }
  }
  float last = 0.0f;
  if (rest < V) {
    last = Vec<E>::value(p[rest]);
    if (rest != y) add_values<1>(r, &last);
  }
  const MaxSum part = wave_join(r);
  if ((tid & 63) == 0) waves[tid >> 6] = part;
  __syncthreads();
  MaxSum others = waves[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) others = join(others, waves[w]);
  const RowStats all = with_target(others, Vec<E>::value(p[y]));
  if (tid == 0) {
    const float lp = all.logp();
    const float2 v = policy_token(a, row, lp);
    logp[row] = lp;
    terms[row] = v.x;
    shared_coef = v.y * scale;
    shared_own = -(v.y * scale) * expm1f(lp);
  }
  __syncthreads();
  // the second pass unpacks the held vectors anew: their float32 values would take twice the registers
#pragma unroll
  for (int h = 0; h < H; ++h) asm volatile("" : "+v"(held[h]));
  const float own = shared_own, cs = -shared_coef / all.sum(), m = at_max(all.m);
  auto grad = [&](typename Vec<E>::type w, int j) {
    float f[N];
    Vec<E>::unpack(w, f);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = cs * exp_of(f[e] - m);
    if (static_cast<unsigned>(y - j) < N) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (j + e == y) f[e] = own;
    }
    vstore_nt(q + j, Vec<E>::pack(f));
  };
  if (rest < V) q[rest] = Vec<E>::round(rest == y ? own : cs * exp_of(last - m));
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (body + tid + h * THREADS < vecs) grad(held[h], (body + tid + h * THREADS) * N);
  // the lane's vectors of the body, last first
  i = tid < body ? tid + (body - 1 - tid) / THREADS * THREADS : -1;
  for (; i - (U - 1) * THREADS >= 0; i -= U * THREADS) {
    typename Vec<E>::type w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = vload_nt(p + (int64_t)(i - u * THREADS) * N);
#pragma unroll
    for (int u = 0; u < U; ++u) grad(w[u], (i - u * THREADS) * N);
  }
  for (; i >= 0; i -= THREADS) grad(vload_nt(p + (int64_t)i * N), i * N);
}

__global__ __launch_bounds__(1024) void sum_kernel(const float* __restrict__ terms, int64_t T,
                                                   float* __restrict__ loss) {
  __shared__ double lds[16];
  double sum = 0.0;
#pragma unroll 8
  for (int64_t t = threadIdx.x; t < T; t += 1024) sum += terms[t];
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) *loss = static_cast<float>(sum);
}

// ---------------------------------------------------------------------------
// gradient: a workgroup takes one piece of a row, a vector per lane. Memory
// that many short workgroups write in the order of its addresses goes faster
// than what fewer, longer ones write: 8192 x 128256 bfloat16 takes 571 us
// with one vector per lane (568 when 602 were measured with two and 637 with
// four).
// ---------------------------------------------------------------------------
// One piece of row `row`: coefficient c, statistics st; zeros for a masked row.
// own(g) is the entry at the target, whose softmax's part is g = -c p.
template <class E, class F>
__device__ __forceinline__ void grad_piece(const GradArgs<E>& a, int64_t row, int piece, int y, float c, float2 st,
                                           F own) {
  constexpr int N = Vec<E>::N;
  const int lo = piece * kGradVecs * N;
  const int n = a.V - lo < kGradVecs * N ? a.V - lo : kGradVecs * N;
  const int tid = threadIdx.x;
  const E* p = a.x + row * a.stride + lo;
  E* q = a.dx + row * a.dx_stride + lo;
  const int vecs = n / N;
  const int rest = vecs * N + tid;  // the row's last elements, one per lane
  if (y < 0 || y >= a.V) {
    const typename Vec<E>::type zero = {0u, 0u, 0u, 0u};
    if (tid < vecs) vstore_nt(q + tid * N, zero);
    if (rest < n) q[rest] = Vec<E>::round(0.0f);
    return;
  }
  const float m = at_max(st.x), cs = -c / st.y;
  const int hit = y - lo;
  if (tid < vecs) {
    float f[N];
    Vec<E>::unpack(vload_nt(p + tid * N), f);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = cs * exp_of(f[e] - m);
    if (static_cast<unsigned>(hit - tid * N) < N) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (tid * N + e == hit) f[e] = own(f[e]);
    }
    vstore_nt(q + tid * N, Vec<E>::pack(f));
  }
  if (rest < n) {
    const float g = cs * exp_of(Vec<E>::value(p[rest]) - m);
    q[rest] = Vec<E>::round(rest == hit ? own(g) : g);
  }
}

// s below which a row's entry at the target is not c - c p with p from the
// rounded s: that loses 2^-24 of c, which at 1 - p = 1/5 is 2^-21.7 of the
// entry, and 2^-16 at 2^-8, far below half a step of bfloat16. Below, the
// entry is -c expm1(logp), or target_kernel's.
template <class E>
constexpr float kLikely = sizeof(E) == 2 ? 1.00390625f : 1.25f;

// The entries at the targets of such rows without their log probabilities:
// one workgroup reads the row again and sums the others, then writes the
// entry into dx, which may be x. The gradient of 8192 rows of 128256 bfloat16
// (686 us, one set of inputs over and over) takes 2 us more where no row is
// likely, 225 where half of them are, 427 where all are; with the log
// probabilities nothing.
template <class E>
__global__ __launch_bounds__(256) void target_kernel(GradArgs<E> a, const int32_t* __restrict__ targets,
                                                     const float2* __restrict__ stats, const float* __restrict__ coef,
                                                     const float* __restrict__ grad_out, float scale) {
  constexpr int N = Vec<E>::N;
  __shared__ double lds[4];
  const int64_t row = blockIdx.x;
  const int y = targets[row];
  const float2 st = stats[row];
  if (y < 0 || y >= a.V || !(st.y < kLikely<E>)) return;
  const E* p = a.x + row * a.stride;
  const int tid = threadIdx.x, vecs = a.V / N;
  const LeftOut<E> target(y, vecs);
  const float m = at_max(st.x);
  double sum = 0.0;
#pragma unroll 4
  for (int i = tid; i < vecs; i += 256) {
    float f[N];
    typename Vec<E>::type w = vload(p + (int64_t)i * N);
    target.template from<1>(&w, i, 1);
    Vec<E>::unpack(w, f);
    sum += sum_exp<N>(f, m);
  }
  const int rest = vecs * N + tid;
  if (rest < a.V && rest != y) sum += exp_of(Vec<E>::value(p[rest]) - m);
  sum = block_sum<4>(sum, lds);
  if (tid != 0) return;
  float c = coef[row] * scale;
  if (grad_out != nullptr) c *= *grad_out;
  const double e = exp_of(Vec<E>::value(p[y]) - m);
  a.dx[row * a.dx_stride + y] = Vec<E>::round(static_cast<float>(c * (sum / (sum + e))));
}

template <class E>
__global__ __launch_bounds__(kGradVecs) void logit_grad_kernel(GradArgs<E> a, const int32_t* __restrict__ targets,
                                                               const float2* __restrict__ stats,
                                                               const float* __restrict__ logp,
                                                               const float* __restrict__ coef,
                                                               const float* __restrict__ grad_out, float scale) {
  const int64_t row = blockIdx.x / (unsigned)a.pieces;
  float c = coef[row] * scale;
  if (grad_out != nullptr) c *= *grad_out;
  const float2 st = stats[row];
  const int y = targets[row];
  grad_piece(a, row, blockIdx.x % (unsigned)a.pieces, y, c, st, [&](float g) {
    if (!(st.y < kLikely<E>)) return g + c;
    return logp != nullptr ? -c * expm1f(logp[row]) : Vec<E>::value(a.dx[row * a.dx_stride + y]);
  });
}

// The second half of a policy step by pieces: every workgroup joins the
// pieces of its row and finds its coefficient itself, and one more at the end
// of the grid sums the rows' losses, so that nothing stands between the two
// launches (40 rows of 128256: 16.3 us a call; a kernel between the two took
// 2 us more).
template <class E>
__global__ __launch_bounds__(kGradVecs) void policy_grad_kernel(GradArgs<E> a, RowPieces pieces, int64_t T,
                                                                PolicyArgs policy, float scale,
                                                                float* __restrict__ loss, float* __restrict__ logp) {
  const int sub = threadIdx.x & 3;
  const int64_t row = blockIdx.x / (unsigned)a.pieces;
  if (row == T) {
    __shared__ double lds[kGradVecs / 64];
    double sum = 0.0;
    for (int64_t t = threadIdx.x >> 2; t - (threadIdx.x >> 2) < T; t += kGradVecs / 4) {
      const Joined v = join_row(pieces, t, T, sub);
      if (!v.live || sub != 0) continue;
      sum += policy_token(policy, t, v.logp).x;
    }
    sum = block_sum<kGradVecs / 64>(sum, lds);
    if (threadIdx.x == 0) *loss = static_cast<float>(sum);
    return;
  }
  const int piece = blockIdx.x % (unsigned)a.pieces;
  const Joined v = join_row(pieces, row, T, sub);
  if (piece == 0 && threadIdx.x == 0) logp[row] = v.logp;
  const float c = v.live ? policy_token(policy, row, v.logp).y * scale : 0.0f;
  grad_piece(a, row, piece, policy.targets[row], c, make_float2(v.m, v.sum),
             [&](float) { return -c * expm1f(v.logp); });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxTokens = (int64_t(1) << 25) - 1;  // of the losses on log probabilities
constexpr int kMaxSplits = 64;            // pieces of one row, few enough rows then

// Pieces per row: about as many as give 1024 workgroups (4 per CU), of at
// least 4096 logits each. A preference step of 700 x 128256 bfloat16 takes
// 100.0 us so, 101.1 with 2048 workgroups, 100.8 with 512; 700 x 32000 35.2,
// 37.2, 35.1.
static int row_splits(int64_t T, int64_t V) {
  const int64_t rows = T < 1 ? 1 : T;
  int64_t s = (1024 + rows / 2) / rows;
  const int64_t most = ceil_div(V, 4096);
  s = s < most ? s : most;
  return static_cast<int>(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

struct LossPlan {
  float2* stats;
  MaxSum* part;
  float *hits, *coef;
  size_t bytes;
};

static LossPlan plan_loss(int64_t T, int64_t V, void* ws) {
  LossPlan l{};
  Carver w(ws);
  l.part = static_cast<MaxSum*>(w.take(row_splits(T, V) > 1 ? T * row_splits(T, V) * sizeof(MaxSum) : 0));
  l.hits = static_cast<float*>(w.take(row_splits(T, V) > 1 ? T * sizeof(float) : 0));
  l.stats = static_cast<float2*>(w.take(T * sizeof(float2)));
  l.coef = static_cast<float*>(w.take(T * sizeof(float)));
  l.bytes = w.used;
  return l;
}

static int check_workspace(const LossPlan& l, void* ws, size_t bytes) {
  return !ws || bytes < l.bytes || !aligned(ws, 256) ? LORA_ERR_WORKSPACE : LORA_OK;
}

static RowPieces row_pieces(const lora_mat* x, const int32_t* targets, float2* stats, const LossPlan& l) {
  return {targets, x->cols, row_splits(x->rows, x->cols), l.part, l.hits, stats};
}

// Statistics of the rows, or of their pieces.
static void run_logp(const lora_mat* x, const int32_t* targets, float* logp, float2* stats, const LossPlan& l,
                     hipStream_t st) {
  const int V = static_cast<int>(x->cols);
  const int splits = row_splits(x->rows, V);
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const int piece = static_cast<int>(round_up(ceil_div(V, splits), Vec<E>::N));
    launch(logp_kernel<E>, dim3(x->rows * splits), dim3(256), 0, st, (const E*)x->ptr, x->stride_row, targets, V,
           splits, piece, logp, stats, l.part, l.hits);
  });
}

static void run_join(const lora_mat* x, const int32_t* targets, float* logp, float2* stats, const LossPlan& l,
                     hipStream_t st) {
  if (row_splits(x->rows, x->cols) == 1) return;
  launch(join_kernel, dim3(ceil_div(x->rows, 64)), dim3(256), 0, st, row_pieces(x, targets, stats, l), x->rows, logp);
}

// Few rows are joined by the loss's own workgroup, which saves a launch (about
// 3 us each); more rows are spread over the card by join_kernel.
static bool join_in_loss(int64_t T, int64_t V) { return T > 0 && T <= kJoinRows && row_splits(T, V) > 1; }

// logp: of the rows, or null.
static void run_logit_grad(const lora_mat* x, const int32_t* targets, const float2* stats, const float* logp,
                           const float* coef, const float* grad_out, float scale, const lora_mat* dx, hipStream_t st) {
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const GradArgs<E> a = grad_args<E>(x, dx);
    if (logp == nullptr)
      launch(target_kernel<E>, dim3(x->rows), dim3(256), 0, st, a, targets, stats, coef, grad_out, scale);
    launch(logit_grad_kernel<E>, dim3(x->rows * a.pieces), dim3(kGradVecs), 0, st, a, targets, stats, logp, coef,
           grad_out, scale);
  });
}

// The policy step by rows (one workgroup takes a row from its statistics to
// its gradient, one read of it from HBM) or split (statistics, then the
// gradient, many workgroups to a row). By rows the time is that of one row
// until the card is full, split it is that of all bytes. us a call, no row
// masked, by rows and split:
//   bfloat16  40000 columns: 40 rows 15.0, 13.4; 96 rows 15.1, 14.7
//            128256: 40 rows 24.5, 17.1; 72 rows 24.8, 24.0; 88 rows 25.1, 27.5; 128 rows 25, 35
//   float32   40000: 40 rows 14.7, 13.4; 56 rows 14.9, 15.2
//            128256: 40 rows 26.4, 25.2; 48 rows 26.5, 27.9; 96 rows 29.6, 46.5
// Rows of up to 32000 take the same either way with few of them, and less by
// rows with more (bfloat16, 192 rows: 13.8, 20.0).
static bool policy_by_rows(const lora_mat* x) {
  return x->rows == 0 || x->rows >= (x->dtype == LORA_F32 ? 48 : 80) || x->cols <= 32768;
}

// Waves to a row. us a call of 8192 rows of bfloat16 (4096 of float32), no row
// masked, with 4, 8 and 16 waves:
//   bfloat16  4000 columns 37, 55, 108; 16000: 94, 100, 158; 24000: 143, 141, 191;
//            49152: 320, 289, 306; 64000: 423, 394, 377; 128256: 869, 827, 783
//   float32   4000: 29, 34, 60; 8000: 52, 52, 69; 13000: 87, 81, 85; 24000: 160, 140, 137;
//            32000: 216, 197, 177; 128256: 987, 862, 836
static int policy_waves(const lora_mat* x) {
  const int64_t vecs = x->cols / vec_elems(x->dtype);
  return vecs <= 2560 ? 4 : vecs <= 6144 ? 8 : 16;
}

static void run_policy_rows(const lora_mat* x, const PolicyArgs& a, float scale, float* logp, float* terms,
                            const lora_mat* dx, hipStream_t st) {
  const int V = static_cast<int>(x->cols);
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const int waves = policy_waves(x);
    auto* kernel = waves == 4   ? policy_row_kernel<E, 4, 6>
                   : waves == 8 ? policy_row_kernel<E, 8, 6>
                                : policy_row_kernel<E, 16, 6>;
    launch(kernel, dim3(x->rows), dim3(64 * waves), 0, st, (const E*)x->ptr, x->stride_row, V, a, scale, logp, terms,
           static_cast<E*>(dx->ptr), dx->stride_row);
  });
}

static int check_pref(const int32_t* offsets, int64_t pairs, const float* ref, float beta, float eps,
                      const float* loss) {
  if (!offsets || !ref || !loss) return LORA_ERR_NULL;
  if (pairs < 1 || pairs > (int64_t(1) << 30)) return LORA_ERR_SHAPE;
  if (!std::isfinite(beta) || !(eps >= 0.0f && eps <= 1.0f)) return LORA_ERR_VALUE;
  return LORA_OK;
}

static int check_policy(const lora_policy* p, int64_t T, const float* loss) {
  if (!p || !loss) return LORA_ERR_NULL;
  if (T > 0 && (!p->targets || !p->old_logp || !p->advantages || !p->weights)) return LORA_ERR_NULL;
  if (T > 0 && p->kl_coef != 0.0f && !p->ref_logp) return LORA_ERR_NULL;
  if (!(p->clip_low + p->clip_high >= 0.0f) || !std::isfinite(p->kl_coef)) return LORA_ERR_VALUE;
  return LORA_OK;
}

static PolicyArgs policy_args(const lora_policy* p) {
  return {p->targets,  p->old_logp,  p->kl_coef != 0.0f ? p->ref_logp : nullptr, p->advantages, p->weights,
          p->clip_low, p->clip_high, p->kl_coef};
}

}  // namespace lora

using namespace lora;

extern "C" size_t lora_loss_workspace_bytes(int64_t T, int64_t V) {
  if (T < 0 || V < 0 || T > kMaxRows || V > 0x7FFFFFFF - 8 * kGradVecs) return 0;
  return plan_loss(T, V, nullptr).bytes;
}

extern "C" int lora_token_logp(const lora_mat* logits, const int32_t* targets, float* logp, float* stats,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  const int64_t T = logits->rows;
  if (T == 0) return LORA_OK;
  if (!targets || !logp || !stats || (logits->cols > 0 && !logits->ptr)) return LORA_ERR_NULL;
  const LossPlan l = plan_loss(T, logits->cols, workspace);
  if (int e = check_workspace(l, workspace, workspace_bytes)) return e;
  auto st = static_cast<hipStream_t>(stream);
  run_logp(logits, targets, logp, reinterpret_cast<float2*>(stats), l, st);
  run_join(logits, targets, logp, reinterpret_cast<float2*>(stats), l, st);
  return launch_status();
}

extern "C" int lora_pref_loss(const float* logp, int64_t T, const int32_t* seq_offsets, int64_t pairs,
                              const float* ref_logp, float beta, float label_smoothing, float* loss, float* seq_logp,
                              float* coef, void* stream) {
  if (int e = check_pref(seq_offsets, pairs, ref_logp, beta, label_smoothing, loss)) return e;
  if (T < 0) return LORA_ERR_SHAPE;
  if (T > kMaxTokens) return LORA_ERR_LIMIT;
  if (T > 0 && !logp) return LORA_ERR_NULL;
  launch(pref_kernel<false>, dim3(1), dim3(1024), 0, static_cast<hipStream_t>(stream), RowPieces{},
         const_cast<float*>(logp), T, seq_offsets, pairs, ref_logp, beta, label_smoothing, loss, seq_logp, coef);
  return launch_status();
}

extern "C" int lora_policy_loss(const float* logp, int64_t T, int64_t V, const lora_policy* policy, float* loss,
                                float* coef, void* stream) {
  if (int e = check_policy(policy, T, loss)) return e;
  if (T < 0 || V < 0) return LORA_ERR_SHAPE;
  if (T > kMaxTokens) return LORA_ERR_LIMIT;
  if (T > 0 && !logp) return LORA_ERR_NULL;
  launch(policy_kernel, dim3(1), dim3(1024), 0, static_cast<hipStream_t>(stream), logp, T, V, policy_args(policy),
         loss, coef);
  return launch_status();
}

static int logit_grad(const lora_mat* logits, const int32_t* targets, const float* stats, const float* logp,
                      const float* coef, const float* grad_out, float scale, const lora_mat* dlogits, void* stream) {
  if (!logits || !dlogits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (int e = check_dlogits(logits, dlogits)) return e;
  if (logits->rows == 0 || logits->cols == 0) return LORA_OK;
  if (!targets || !stats || !coef || !logits->ptr || !dlogits->ptr) return LORA_ERR_NULL;
  run_logit_grad(logits, targets, reinterpret_cast<const float2*>(stats), logp, coef, grad_out, scale, dlogits,
                 static_cast<hipStream_t>(stream));
  return launch_status();
}

extern "C" int lora_logit_grad(const lora_mat* logits, const int32_t* targets, const float* stats, const float* coef,
                               const float* grad_out, float scale, const lora_mat* dlogits, void* stream) {
  return logit_grad(logits, targets, stats, nullptr, coef, grad_out, scale, dlogits, stream);
}

extern "C" int lora_logit_grad_logp(const lora_mat* logits, const int32_t* targets, const float* stats,
                                    const float* logp, const float* coef, const float* grad_out, float scale,
                                    const lora_mat* dlogits, void* stream) {
  if (!logp && logits && logits->rows > 0 && logits->cols > 0) return LORA_ERR_NULL;
  return logit_grad(logits, targets, stats, logp, coef, grad_out, scale, dlogits, stream);
}

extern "C" int lora_pref_step(const lora_mat* logits, const int32_t* targets, const int32_t* seq_offsets,
                              int64_t pairs, const float* ref_logp, float beta, float label_smoothing,
                              float grad_scale, float* loss, float* seq_logp, float* logp, const lora_mat* dlogits,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits || !dlogits) return LORA_ERR_NULL;
  if (int e = check_pref(seq_offsets, pairs, ref_logp, beta, label_smoothing, loss)) return e;
  if (int e = check_logits(logits)) return e;
  if (int e = check_dlogits(logits, dlogits)) return e;
  const int64_t T = logits->rows, V = logits->cols;
  if (T > 0 && (!targets || !logp || (V > 0 && (!logits->ptr || !dlogits->ptr)))) return LORA_ERR_NULL;
  const LossPlan l = plan_loss(T, V, workspace);
  if (T > 0)
    if (int e = check_workspace(l, workspace, workspace_bytes)) return e;
  auto st = static_cast<hipStream_t>(stream);
  if (T > 0) run_logp(logits, targets, logp, l.stats, l, st);
  const bool join = join_in_loss(T, V);
  if (T > 0 && !join) run_join(logits, targets, logp, l.stats, l, st);
  launch(join ? pref_kernel<true> : pref_kernel<false>, dim3(1), dim3(1024), 0, st,
         row_pieces(logits, targets, l.stats, l), logp, T, seq_offsets, pairs, ref_logp, beta, label_smoothing, loss,
         seq_logp, l.coef);
  if (T > 0 && V > 0) run_logit_grad(logits, targets, l.stats, logp, l.coef, nullptr, grad_scale, dlogits, st);
  return launch_status();
}

extern "C" int lora_policy_step(const lora_mat* logits, const lora_policy* policy, float grad_scale, float* loss,
                                float* logp, const lora_mat* dlogits, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!logits || !dlogits) return LORA_ERR_NULL;
  const int64_t T = logits->rows, V = logits->cols;
  if (int e = check_policy(policy, T, loss)) return e;
  if (int e = check_logits(logits)) return e;
  if (int e = check_dlogits(logits, dlogits)) return e;
  if (T > 0 && (!logp || (V > 0 && (!logits->ptr || !dlogits->ptr)))) return LORA_ERR_NULL;
  const LossPlan l = plan_loss(T, V, workspace);
  if (T > 0)
    if (int e = check_workspace(l, workspace, workspace_bytes)) return e;
  auto st = static_cast<hipStream_t>(stream);
  const PolicyArgs a = policy_args(policy);
  if (policy_by_rows(logits)) {
    if (T > 0) run_policy_rows(logits, a, grad_scale, logp, l.coef, dlogits, st);
    launch(sum_kernel, dim3(1), dim3(1024), 0, st, (const float*)l.coef, T, loss);
    return launch_status();
  }
  // so few and such long rows are always in pieces
  run_logp(logits, a.targets, logp, l.stats, l, st);
  by_type(logits, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const GradArgs<E> g = grad_args<E>(logits, dlogits);
    launch(policy_grad_kernel<E>, dim3(T * g.pieces + 1), dim3(kGradVecs), 0, st, g,
           row_pieces(logits, a.targets, nullptr, l), T, a, grad_scale, loss, logp);
  });
  return launch_status();
}
