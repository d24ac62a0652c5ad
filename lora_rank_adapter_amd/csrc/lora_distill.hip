// Distillation from a teacher's top logits: the divergence of a row's softmax
// from what the teacher gave of its own (the ids of its likeliest tokens and
// their log probabilities), the weighted loss, and the gradient of the logits.
//
//   p = softmax(x / tau), q_k the teacher's probability of id_k,
//   q_r = 1 - sum q_k, p_r = the sum of p over the tokens that no id names
//   kl = sum q_k (log q_k - log p[id_k]) + q_r (log q_r - log p_r)
//   tau dx_j = Q p_j - sum of q_k with id_k = j        at the teacher's tokens
//            = p_j / p_r (Q p_r - q_r)                 elsewhere, Q = sum q_k + q_r
//
// Without the rest, q is normalised over its ids and q_r is 0, which leaves
// p_j Q elsewhere.
//
// The others' sum is a small part of a row whose likeliest tokens the teacher
// named, so it is never a difference: one bit for each of a row's elements, in
// LDS, says which belong to the teacher, and the pass over the row leaves them
// out. The teacher's tokens and the sums of a row are joined in float64.
//
// Kernels:
//   distill_row_kernel   a workgroup to a row: the divergence, and what the gradient takes
//   distill_grad_kernel  the gradient's rows
//   distill_sum_kernel   the weighted sum of the rows' divergences

#include <type_traits>

#include "lora_softmax.hpp"

namespace lora {

constexpr int kMaxTeacher = 256;       // tokens of a teacher for each row
constexpr int kChunkVecs = 16384;      // vectors of a row whose elements' bits are in LDS at a time
constexpr int kStateHead = 2;          // state of a row: m, a, and a value for each of the teacher's tokens

struct Teacher {
  const int32_t* ids;
  const float* logp;
  int k;
  bool rest;
  double inv_temperature;
};

// A row's elements that the teacher did not name.
struct Others {
  float m;   // what the exponents are relative to
  double s;  // sum of exp((x - m) / tau)
};

// The teacher's tokens of one row, in LDS.
struct Tokens {
  int id[kMaxTeacher];        // -1: none
  float x[kMaxTeacher];       // the row's logits there
  float b[kMaxTeacher];       // tau dx there
  double q[kMaxTeacher];
  int twice, named;           // whether an id occurs twice; how many ids there are
};

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}

struct Row {
  float kl, a;  // tau dx = a exp((x - m) / tau) for the others
};

// By one wave: a row's divergence and gradient factors from the others' sum.
// Entries that name a token twice count both, the token once.
__device__ __forceinline__ Row finish_row(const Teacher& t, int64_t row, int V, Others o, Tokens& k) {
  constexpr int J = kMaxTeacher / 64;
  const int lane = threadIdx.x & 63;
  const float* logp = t.logp + row * t.k;
  double lq[J], lp[J];
  bool on[J], first[J];
  double top = o.s > 0.0 ? (double)o.m : -INFINITY, most = -INFINITY;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int i = lane + 64 * j;
    on[j] = first[j] = i < t.k && k.id[i] >= 0;
    lq[j] = on[j] ? (double)logp[i] : -INFINITY;
    lp[j] = on[j] ? (double)k.x[i] : -INFINITY;
    top = fmax(top, lp[j]);
    most = fmax(most, lq[j]);
    if (on[j] && k.twice)
      for (int e = 0; e < i; ++e) first[j] = first[j] && k.id[e] != k.id[i];
  }
  top = wave_max(top);
  double total = 0.0, z = 0.0;
  if (!t.rest) {
    most = wave_max(most);
#pragma unroll
    for (int j = 0; j < J; ++j) z += on[j] ? exp(lq[j] - most) : 0.0;
    most += log(wave_sum(z));
  }
  int named = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    lp[j] = (lp[j] - top) * t.inv_temperature;
    if (first[j]) total += exp(lp[j]);
    named += __popcll(__ballot(first[j]));
  }
  const double others = o.s > 0.0 ? o.s * exp((o.m - top) * t.inv_temperature) : o.s;
  total = wave_sum(total) + others;
  // a NaN, +inf (their difference from the largest is NaN) or nothing above -inf
  if (!(top > -INFINITY)) total = NAN;
  const double log_total = log(total);
  double q[J], all = 0.0, kl = 0.0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    lp[j] -= log_total;
    if (!t.rest) lq[j] -= most;
    q[j] = on[j] ? exp(lq[j]) : 0.0;
    all += q[j];
    if (on[j] && q[j] != 0.0) kl += q[j] * (lq[j] - lp[j]);
    if (k.twice && lane + 64 * j < t.k) k.q[lane + 64 * j] = q[j];
  }
  all = wave_sum(all);
  kl = wave_sum(kl);
  const double p_rest = others / total;
  double q_rest = 0.0;
  if (t.rest && named < V) {
    q_rest = all < 1.0 ? 1.0 - all : 0.0;
    if (!(all == all)) q_rest = all;
    if (q_rest != 0.0) kl += q_rest * (log(q_rest) - log(p_rest));
    all += q_rest;
  }
  double a = (all * p_rest - q_rest) / o.s;
  if (o.s == 0.0) a = 0.0;                       // the others hold nothing
  if (!(total == total) || !(all == all)) a = kl = NAN;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int i = lane + 64 * j;
    if (i >= t.k) continue;
    double held = q[j];
    if (on[j] && k.twice) {
      held = 0.0;
      for (int e = 0; e < t.k; ++e) held += k.id[e] == k.id[i] ? k.q[e] : 0.0;
    }
    k.b[i] = on[j] ? static_cast<float>(all * exp(lp[j]) - held) : 0.0f;
  }
  return {static_cast<float>(kl), static_cast<float>(a)};
}

// The teacher's tokens of a row and its logits there; whether there is any.
template <class E, int THREADS>
__device__ __forceinline__ bool load_tokens(const Teacher& t, int64_t row, const E* p, int V, Tokens& k) {
  const int tid = threadIdx.x;
  bool on = false;
  if (tid < kMaxTeacher) {
    const int id = tid < t.k ? t.ids[row * t.k + tid] : -1;
    on = id >= 0 && id < V;
    k.id[tid] = on ? id : -1;
    k.x[tid] = on ? Vec<E>::value(p[id]) : 0.0f;
  }
  if (tid == 0) k.twice = 0;
  return __syncthreads_or(on);
}

// Sets the bits of the teacher's tokens among the elements of the vectors
// [base, base + kChunkVecs): bit e of byte v for element e of vector base + v
// (the row's last elements are of one more vector).
template <int N, int THREADS>
__device__ __forceinline__ void mark_tokens(const Teacher& t, Tokens& k, int base, uint32_t* bits) {
  const int tid = threadIdx.x;
  uint4* clear = reinterpret_cast<uint4*>(bits);
  for (int i = tid; i < kChunkVecs / 16; i += THREADS) clear[i] = zero4();
  __syncthreads();
  if (tid < t.k && k.id[tid] >= 0) {
    const int v = k.id[tid] / N - base;
    if (v >= 0 && v < kChunkVecs) {
      const uint32_t bit = 1u << (8 * (v & 3) + k.id[tid] % N);
      if (atomicOr(&bits[v >> 2], bit) & bit) k.twice = 1;
    }
  }
  __syncthreads();
}

template <class E>
__global__ __launch_bounds__(256) void distill_row_kernel(const E* __restrict__ x, int64_t stride, int V, Teacher t,
                                                          Exponent s, float* __restrict__ kl,
                                                          float* __restrict__ state) {
  constexpr int N = Vec<E>::N, THREADS = 256;
  __shared__ Tokens tokens;
  __shared__ __align__(16) uint32_t bits[kChunkVecs / 4];
  __shared__ double lds[4];
  __shared__ float wave_m[4];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const E* p = x + row * stride;
  float* out = state == nullptr ? nullptr : state + row * (t.k + kStateHead);
  if (!load_tokens<E, THREADS>(t, row, p, V, tokens)) {
    if (tid == 0) kl[row] = 0.0f;
    if (out != nullptr)
      for (int i = tid; i < t.k + kStateHead; i += THREADS) out[i] = 0.0f;
    return;
  }
  const int vecs = V / N;
  const uint8_t* byte = reinterpret_cast<const uint8_t*>(bits);
  // f(value) for the others' elements
  auto others = [&](auto f) {
    for (int base = 0; base <= vecs; base += kChunkVecs) {
      mark_tokens<N, THREADS>(t, tokens, base, bits);
      const int end = vecs - base < kChunkVecs ? vecs - base : kChunkVecs;
      for (int i = tid; i < end; i += THREADS) {
        float v[N];
        Vec<E>::unpack(vload(p + (int64_t)(base + i) * N), v);
        const uint32_t off = byte[i];
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (!(off >> e & 1u)) f(v[e]);
      }
      if (end < kChunkVecs && tid < V - vecs * N && !(byte[end] >> tid & 1u)) f(Vec<E>::value(p[vecs * N + tid]));
      __syncthreads();
    }
  };
  float m = -INFINITY;
  others([&](float v) { m = fmaxf(m, v); });
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  if ((tid & 63) == 0) wave_m[tid >> 6] = m;
  __syncthreads();
  m = at_max(fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3])));
  if (tid == 0) tokens.twice = 0;
  double sum = 0.0;
  others([&](float v) { sum += __builtin_amdgcn_exp2f(s.of(v - m)); });
  sum = block_sum<4>(sum, lds);
  if (tid < 64) {
    const Row r = finish_row(t, row, V, Others{m, sum}, tokens);
    if (tid == 0) {
      kl[row] = r.kl;
      if (out != nullptr) {
        out[0] = m;
        out[1] = r.a;
      }
    }
  }
  __syncthreads();
  if (out != nullptr && tid < t.k) out[kStateHead + tid] = tokens.b[tid];
}

// A workgroup takes one piece of a row, a vector per lane; the entries at the
// teacher's tokens follow once the vectors are written.
template <class E>
__global__ __launch_bounds__(kGradVecs) void distill_grad_kernel(GradArgs<E> a, const int32_t* __restrict__ ids, int k,
                                                                 const float* __restrict__ state,
                                                                 const float* __restrict__ coef,
                                                                 const float* __restrict__ grad_out, float scale,
                                                                 Exponent s) {
  constexpr int N = Vec<E>::N;
  const int64_t row = blockIdx.x / (unsigned)a.pieces;
  const int lo = (blockIdx.x % (unsigned)a.pieces) * kGradVecs * N;
  const int n = a.V - lo < kGradVecs * N ? a.V - lo : kGradVecs * N;
  const int tid = threadIdx.x;
  const E* p = a.x + row * a.stride + lo;
  E* q = a.dx + row * a.dx_stride + lo;
  const int vecs = n / N;
  const int rest = vecs * N + tid;  // the row's last elements, one per lane
  const float* st = state + row * (k + kStateHead);
  float c = coef[row] * scale;
  if (grad_out != nullptr) c *= *grad_out;
  const float m = st[0], factor = c == 0.0f || st[1] == 0.0f ? 0.0f : c * st[1];
  if (factor == 0.0f) {
    const typename Vec<E>::type zero = {0u, 0u, 0u, 0u};
    if (tid < vecs) vstore_nt(q + tid * N, zero);
    if (rest < n) q[rest] = Vec<E>::round(0.0f);
  } else {
    if (tid < vecs) {
      float f[N];
      Vec<E>::unpack(vload_nt(p + tid * N), f);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = factor * __builtin_amdgcn_exp2f(s.of(f[e] - m));
      vstore_nt(q + tid * N, Vec<E>::pack(f));
    }
    if (rest < n) q[rest] = Vec<E>::round(factor * __builtin_amdgcn_exp2f(s.of(Vec<E>::value(p[rest]) - m)));
  }
  if (c == 0.0f) return;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid < k) {
    const int at = ids[row * k + tid];
    if (at >= 0 && at < a.V && at >= lo && at - lo < n) q[at - lo] = Vec<E>::round(c * st[kStateHead + tid]);
  }
}

__global__ __launch_bounds__(1024) void distill_sum_kernel(const float* __restrict__ kl,
                                                           const float* __restrict__ weights, int64_t T,
                                                           float* __restrict__ loss) {
  __shared__ double lds[16];
  double sum = 0.0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const float w = weights[t];
    if (w != 0.0f) sum += (double)w * kl[t];
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) *loss = static_cast<float>(sum);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

static size_t state_bytes(int64_t T, int64_t k) {
  return static_cast<size_t>(round_up(T * (k + kStateHead) * (int64_t)sizeof(float), 256));
}

static int check_teacher(const lora_teacher* t, int64_t T) {
  if (!t) return LORA_ERR_NULL;
  if (t->k < 1) return LORA_ERR_SHAPE;
  if (t->k > kMaxTeacher) return LORA_ERR_LIMIT;
  if (!temperature_ok(t->temperature)) return LORA_ERR_VALUE;
  if (T > 0 && (!t->ids || !t->logp)) return LORA_ERR_NULL;
  return LORA_OK;
}

static Teacher teacher_of(const lora_teacher* t) {
  return {t->ids, t->logp, static_cast<int>(t->k), t->rest != 0, 1.0 / t->temperature};
}

static void run_rows(const lora_mat* x, const lora_teacher* t, float* kl, float* state, hipStream_t st) {
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    launch(distill_row_kernel<E>, dim3(x->rows), dim3(256), 0, st, (const E*)x->ptr, x->stride_row,
           static_cast<int>(x->cols), teacher_of(t), exponent_of(t->temperature), kl, state);
  });
}

static void run_grad(const lora_mat* x, const int32_t* ids, int k, const float* state, const float* coef,
                     const float* grad_out, float scale, double temperature, const lora_mat* dx, hipStream_t st) {
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const GradArgs<E> a = grad_args<E>(x, dx);
    launch(distill_grad_kernel<E>, dim3(x->rows * a.pieces), dim3(kGradVecs), 0, st, a, ids, k, state, coef, grad_out,
           static_cast<float>((double)scale / temperature), exponent_of(temperature));
  });
}

}  // namespace lora

using namespace lora;

extern "C" size_t lora_distill_workspace_bytes(int64_t T, int64_t V, int64_t k) {
  if (T < 0 || V < 0 || k < 1 || T > kMaxRows || V > 0x7FFFFFFF - 8 * kGradVecs || k > kMaxTeacher) return 0;
  return state_bytes(T, k) + 256;
}

static int check_distill_workspace(const lora_mat* x, const lora_teacher* t, void* ws, size_t bytes) {
  return !ws || bytes < lora_distill_workspace_bytes(x->rows, x->cols, t->k) || !aligned(ws, 256)
             ? LORA_ERR_WORKSPACE
             : LORA_OK;
}

extern "C" int lora_distill_kl(const lora_mat* logits, const lora_teacher* teacher, float* kl, float* state,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (int e = check_teacher(teacher, logits->rows)) return e;
  if (logits->rows == 0) return LORA_OK;
  if (!kl || (logits->cols > 0 && !logits->ptr)) return LORA_ERR_NULL;
  if (int e = check_distill_workspace(logits, teacher, workspace, workspace_bytes)) return e;
  run_rows(logits, teacher, kl, state, static_cast<hipStream_t>(stream));
  return launch_status();
}

extern "C" int lora_distill_grad(const lora_mat* logits, const int32_t* top_ids, int64_t k, const float* state,
                                 const float* coef, const float* grad_out, float scale, double temperature,
                                 const lora_mat* dlogits, void* stream) {
  if (!logits || !dlogits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (int e = check_dlogits(logits, dlogits)) return e;
  if (k < 1) return LORA_ERR_SHAPE;
  if (k > kMaxTeacher) return LORA_ERR_LIMIT;
  if (!temperature_ok(temperature)) return LORA_ERR_VALUE;
  if (logits->rows == 0 || logits->cols == 0) return LORA_OK;
  if (!top_ids || !state || !coef || !logits->ptr || !dlogits->ptr) return LORA_ERR_NULL;
  run_grad(logits, top_ids, static_cast<int>(k), state, coef, grad_out, scale, temperature, dlogits,
           static_cast<hipStream_t>(stream));
  return launch_status();
}

extern "C" int lora_distill_step(const lora_mat* logits, const lora_teacher* teacher, const float* weights,
                                 float grad_scale, float* loss, float* kl, const lora_mat* dlogits, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!logits || !dlogits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (int e = check_dlogits(logits, dlogits)) return e;
  const int64_t T = logits->rows, V = logits->cols;
  if (int e = check_teacher(teacher, T)) return e;
  if (!loss || (T > 0 && (!weights || !kl || (V > 0 && (!logits->ptr || !dlogits->ptr))))) return LORA_ERR_NULL;
  if (T > 0)
    if (int e = check_distill_workspace(logits, teacher, workspace, workspace_bytes)) return e;
  auto st = static_cast<hipStream_t>(stream);
  float* state = static_cast<float*>(workspace);
  if (T > 0) run_rows(logits, teacher, kl, state, st);
  if (T > 0 && V > 0)
    run_grad(logits, teacher->ids, static_cast<int>(teacher->k), state, weights, nullptr, grad_scale,
             teacher->temperature, dlogits, st);
  launch(distill_sum_kernel, dim3(1), dim3(1024), 0, st, (const float*)kl, weights, T, loss);
  return launch_status();
}
