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
//   distill_row_kernel    a row by one workgroup, to its divergence or to its gradient
//   distill_piece_kernel  the others' sum of a piece of a row
//   distill_join_kernel   the pieces of a row joined: the divergence, and what the gradient takes
//   distill_grad_kernel   the gradient's rows from that
//   distill_sum_kernel    the weighted sum of the rows' divergences

#include <cfloat>
#include <type_traits>

#include "lora_softmax.hpp"

namespace lora {

constexpr int kMaxTeacher = 256;       // tokens of a teacher for each row
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
  float m;   // what the exponents are relative to: kAbove binary orders above the largest x at most
  double s;  // sum of exp((x - m) / tau)
};

// The teacher's tokens of one row, in LDS.
struct Tokens {
  __attribute__((aligned(16))) int id[kMaxTeacher];  // -1: none
  double q[kMaxTeacher]; // if an id occurs twice
  int twice;
};

struct Row {
  double kl, a;  // tau dx = a exp((x - m) / tau) for the others
  float b;       // tau dx at this thread's token
};

// A row's divergence and gradient factors from the others' sum, by all threads
// of a workgroup: thread i has the teacher's i-th token `id`, with the row's
// logit x there and the teacher's log probability. Entries that name a token
// twice count both, the token once. Logarithms are taken of sums, not of
// probabilities, which may be too small for float64.
template <int WAVES>
__device__ __forceinline__ Row finish_row(const Teacher& t, int V, Others o, int id, float x, float logq, Tokens& k) {
  __shared__ float most[2][WAVES];
  __shared__ double sums[5][WAVES];
  const int tid = threadIdx.x, wave = tid >> 6;
  const bool on = id >= 0;
  bool first = on;
  if (on && k.twice)
    for (int e = 0; e < tid; ++e) first = first && k.id[e] != id;
  float top = lane_max(on ? x : -INFINITY), likely = lane_max(logq);
  if ((tid & 63) == 0) {
    most[0][wave] = top;
    most[1][wave] = likely;
  }
  __syncthreads();
  top = o.s > 0.0 ? o.m : -INFINITY;
  likely = -INFINITY;
  for (int w = 0; w < WAVES; ++w) {
    top = fmaxf(top, most[0][w]);
    likely = fmaxf(likely, most[1][w]);
  }
  // the sum that x's token is part of, relative to the largest logit; the teacher's, to its largest
  double lp = ((double)x - top) * t.inv_temperature, lq = logq;
  double p = 0.0, z = 0.0, tokens = first ? 1.0 : 0.0;
  if (wave * 64 < t.k) {
    if (!t.rest) lq -= likely;
    if (first) p = exp(lp);
    if (on) z = exp(lq);
    const double p_sum = lane_total(p), z_sum = lane_total(z);
    tokens = lane_total(tokens);
    if ((tid & 63) == 0) {
      sums[0][wave] = p_sum;
      sums[1][wave] = z_sum;
      sums[2][wave] = tokens;
    }
  }
  __syncthreads();
  const double below = ((double)o.m - top) * t.inv_temperature;
  const double others = o.s > 0.0 ? o.s * exp(below) : o.s;
  double total = others, all = 0.0, named = 0.0;
  for (int w = 0; w * 64 < t.k; ++w) {
    total += sums[0][w];
    all += sums[1][w];
    named += sums[2][w];
  }
  // a NaN, +inf (their difference from the largest is NaN) or nothing above -inf
  if (!(top > -INFINITY)) total = NAN;
  double q = z;
  if (!t.rest) {
    q = z / all;
    lq -= log(all);
    all = all == all ? 1.0 : all;
  }
  const double log_total = log(total);
  lp -= log_total;
  if (wave * 64 < t.k) {
    if (k.twice && tid < t.k) k.q[tid] = q;
    const double part = lane_total(on && q != 0.0 ? q * (lq - lp) : 0.0);
    if ((tid & 63) == 0) sums[3][wave] = part;
  }
  __syncthreads();
  double kl = 0.0;
  for (int w = 0; w * 64 < t.k; ++w) kl += sums[3][w];
  const double p_rest = others / total;
  double q_rest = 0.0;
  if (t.rest && named < V) {
    q_rest = all < 1.0 ? 1.0 - all : all == all ? 0.0 : all;
    if (q_rest != 0.0) kl += q_rest * (log(q_rest) - (o.s > 0.0 ? log(o.s) + below - log_total : log(p_rest)));
    all += q_rest;
  }
  double a = o.s == 0.0 ? 0.0 : (all * p_rest - q_rest) / o.s;  // 0: the others hold nothing
  if (!(total == total) || !(all == all)) a = kl = NAN;
  double given = q;
  if (on && k.twice) {
    given = 0.0;
    for (int e = 0; e < t.k; ++e) given += k.id[e] == id ? k.q[e] : 0.0;
  }
  return {kl, a, on ? static_cast<float>(all * exp(lp) - given) : 0.0f};
}

// Whether a row has a token at all; every wave looks for itself.
__device__ __forceinline__ bool any_token(const Teacher& t, int64_t row, int V) {
  bool on = false;
  for (int i = threadIdx.x & 63; i < t.k; i += 64) on = on || static_cast<unsigned>(t.ids[row * t.k + i]) < (unsigned)V;
  return __ballot(on) != 0;
}

// This thread's token of a row, -1 if it has none.
__device__ __forceinline__ int token_id(const Teacher& t, int64_t row, int V) {
  if ((int)threadIdx.x >= t.k) return -1;
  const int id = t.ids[row * t.k + threadIdx.x];
  return id >= 0 && id < V ? id : -1;
}

// The bits of the teacher's tokens among the elements [lo, lo + n) of a row:
// bit e of byte v for element e of the piece's vector v (the last one may be
// in part). A barrier between the two, and one behind the second.
template <int N, int THREADS>
__device__ __forceinline__ void clear_bits(int n, uint32_t* bits, Tokens& k) {
  uint4* words = reinterpret_cast<uint4*>(bits);
  for (int i = threadIdx.x; i < (n / N + 16) / 16; i += THREADS) words[i] = zero4();
  if (threadIdx.x == 0) k.twice = 0;
}
template <int N>
__device__ __forceinline__ void set_bit(int id, int lo, int n, uint32_t* bits, Tokens& k) {
  if ((int)threadIdx.x < kMaxTeacher) k.id[threadIdx.x] = id;
  if (id < lo || id - lo >= n) return;
  const int v = (id - lo) / N;
  const uint32_t bit = 1u << (8 * (v & 3) + (id - lo) % N);
  if (atomicOr(&bits[v >> 2], bit) & bit) k.twice = 1;
}

// A vector with -inf in the place of the teacher's tokens.
template <class E>
__device__ __forceinline__ void leave_out(float* f, uint32_t off) {
  if (off == 0) return;
#pragma unroll
  for (int e = 0; e < Vec<E>::N; ++e)
    if (off >> e & 1u) f[e] = -INFINITY;
}

template <int N>
__device__ __forceinline__ float sum_exp(const float* f, float z, Exponent s) {
  if constexpr (N == 1)
    return __builtin_amdgcn_exp2f(s.of(f[0] - z));
  else
    return sum_exp<N / 2>(f, z, s) + sum_exp<N / 2>(f + N / 2, z, s);
}

// The largest of the workgroup's v; lds is used once.
template <int WAVES>
__device__ __forceinline__ float block_max(float v, float* lds) {
  v = lane_max(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) v = fmaxf(v, lds[w]);
  return v;
}

template <int WAVES>
struct PassLds {
  float first[WAVES], refs[WAVES];
  double sum[WAVES];
};

// One pass over n elements from p on, but for those whose bits are set. The
// exponents are relative to kAbove binary orders above the largest of the first
// vectors, which the others seldom reach: no running maximum. An exponent far
// above the reference loses precision, so a lane that meets a logit above its own
// moves it kAbove orders above that one, scales its sum and reads those vectors
// anew. At 3 orders one in eight rows of 128256 random logits has such a lane; at
// one nearly every row had, which took 2.5 of the 71 us of 2048 such rows. The last
// H vectors per lane stay in `held` (as read), the elements past the last vector in
// `last`. AGAIN: the elements will be read once more.
constexpr float kAbove = 3.0f;

template <class E, int WAVES, int H, bool AGAIN>
struct OthersPass {
  static constexpr int N = Vec<E>::N, U = 4, THREADS = 64 * WAVES;
  using V4 = typename Vec<E>::type;
  int vecs, body, rest;
  V4 held[H];
  float last;

  static __device__ __forceinline__ V4 load(const E* at) {
    if constexpr (AGAIN) return vload(at);
    return vload_nt(at);
  }

  __device__ __forceinline__ Others run(const E* p, int n, const uint8_t* byte, Exponent s, PassLds<WAVES>& lds) {
    const int tid = threadIdx.x;
    vecs = n / N;
    rest = vecs * N + tid;
    body = vecs > H * THREADS ? vecs - H * THREADS : 0;
    float m = -INFINITY;
    auto largest = [&](V4 v, int i) {
      float f[N];
      Vec<E>::unpack(v, f);
      leave_out<E>(f, byte[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) m = fmaxf(m, f[e]);
    };
    V4 w[U];
    // Loads past the last vector take it once more: behind a condition each would be waited for at once.
    auto before = [](int i, int end) { return (int64_t)(i < end ? i : end - 1) * N; };
    auto hold = [&] {
#pragma unroll
      for (int h = 0; h < H; ++h) held[h] = vload_nt(p + before(body + tid + h * THREADS, vecs));
    };
    last = rest < n ? Vec<E>::value(p[rest]) : -INFINITY;
    const bool left = rest < n && !(byte[vecs] >> tid & 1u);
    if (body > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        w[u] = load(p + before(tid + u * THREADS, body));
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (tid + u * THREADS < body) largest(w[u], tid + u * THREADS);
    } else if (vecs > 0) {
      hold();
      // of bfloat16 the first ones suffice; us a step, the first four and all: 2048 x 20000 bfloat16 42.2 and 44.1,
      // 2048 x 10000 float32 42.2 and 39.3
#pragma unroll
      for (int h = 0; h < (sizeof(E) == 2 && U < H ? U : H); ++h)
        if (tid + h * THREADS < vecs) largest(held[h], tid + h * THREADS);
    }
    if (left) m = fmaxf(m, last);
    m = block_max<WAVES>(m, lds.first);
    // with nothing above -inf so far the first logit that is replaces it
    m = fmaxf(m, -FLT_MAX);
    const float above = kAbove / s.hi;
    float z = m + above;
    double sum = 0.0;
    auto take = [&](V4 v, uint32_t off) {
      float f[N];
      Vec<E>::unpack(v, f);
      leave_out<E>(f, off);
#pragma unroll
      for (int e = 0; e < N; ++e) m = fmaxf(m, f[e]);
      sum += sum_exp<N>(f, z, s);
    };
    // Behind some vectors, `count` of them from i on and up to `end`: the sum anew from what it was before them, if one
    // is above the reference. Read again for it: kept until here they would spill, or take the next ones' room.
    auto settle = [&](double was, int i, int count, int end) {
      if (!(m > z)) return;
      sum = was * __builtin_amdgcn_exp2f(s.of(z - (m + above)));
      z = m + above;
      if constexpr (AGAIN) {
#pragma unroll 1
        for (int u = 0; u < count && i < end; ++u, i += THREADS) take(load(p + (int64_t)i * N), byte[i]);
      } else {
        V4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load(p + before(i + u * THREADS, end));
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < count && i + u * THREADS < end) take(v[u], byte[i + u * THREADS]);
      }
    };
    if (left) sum += __builtin_amdgcn_exp2f(s.of(last - z));
    if (body > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)  // none is above the reference
        if (tid + u * THREADS < body) take(w[u], byte[tid + u * THREADS]);
      int i = tid + U * THREADS;
      uint32_t off[U];  // the vectors' bits, read before the first is used
      if constexpr (AGAIN) {
        for (; i + (U - 1) * THREADS < body; i += U * THREADS) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            w[u] = load(p + (int64_t)(i + u * THREADS) * N);
            off[u] = byte[i + u * THREADS];
          }
          const double was = sum;
#pragma unroll
          for (int u = 0; u < U; ++u) take(w[u], off[u]);
          settle(was, i, U, body);
        }
        for (; i < body; i += THREADS) {
          const double was = sum;
          take(load(p + (int64_t)i * N), byte[i]);
          settle(was, i, 1, body);
        }
      } else {
        // the next four vectors on their way; with the held ones beside them that would spill
        V4 a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = load(p + before(i + u * THREADS, body));
        for (; i + (U - 1) * THREADS < body; i += U * THREADS) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            w[u] = a[u];
            off[u] = byte[i + u * THREADS];
            a[u] = load(p + before(i + (u + U) * THREADS, body));
          }
          sched_fence();
          const double was = sum;
#pragma unroll
          for (int u = 0; u < U; ++u) take(w[u], off[u]);
          settle(was, i, U, body);
        }
        const double was = sum;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + u * THREADS < body) take(a[u], byte[i + u * THREADS]);
        settle(was, i, U, body);
      }
      hold();
    }
#pragma unroll
    for (int g = 0; g < H; g += U) {
      const double was = sum;
#pragma unroll
      for (int h = g; h < g + U && h < H; ++h)
        if (body + tid + h * THREADS < vecs) take(held[h], byte[body + tid + h * THREADS]);
      settle(was, body + tid + g * THREADS, U, vecs);
    }
    // to the largest reference (not to the largest logit: that factor's rounding would be all rows' and all terms')
    const float ref = block_max<WAVES>(z, lds.refs);
    if (sum > 0.0) sum *= __builtin_amdgcn_exp2f(s.of(z - ref));
    sum = lane_total(sum);
    if ((tid & 63) == 0) lds.sum[tid >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int v = 0; v < WAVES; ++v) sum += lds.sum[v];
    return {ref, sum};
  }
};

// A row's divergence and state in memory; zeros for a masked one.
__device__ __forceinline__ void put_row(float* kl, float* state, const Teacher& t, int64_t row, float m, const Row& r) {
  if (threadIdx.x == 0) kl[row] = static_cast<float>(r.kl);
  if (state == nullptr) return;
  float* out = state + row * (t.k + kStateHead);
  if (threadIdx.x == 0) {
    out[0] = m;
    out[1] = static_cast<float>(r.a);
  }
  if ((int)threadIdx.x < t.k) out[kStateHead + threadIdx.x] = r.b;
}

// A row by one workgroup: the divergence, and with GRAD the gradient at once,
// for which the row's last H vectors per lane stay in registers and the others
// are read again, the most recently read first.
template <class E, int WAVES, bool GRAD>
__global__ __launch_bounds__(64 * WAVES, GRAD ? 4 : sizeof(E) == 2 ? 6 : 5) void distill_row_kernel(
    const E* x, int64_t stride, int V, Teacher t, Exponent s, float* __restrict__ kl, float* __restrict__ state,
    const float* __restrict__ weights, float scale, E* dx, int64_t dx_stride) {
  // as many vectors as 128 registers leave room for, four waves' share of a row that they hold whole
  constexpr int N = Vec<E>::N, U = 4, THREADS = 64 * WAVES;
  constexpr int H = !GRAD ? 1 : WAVES == 4 ? 10 : WAVES == 16 ? 14 : sizeof(E) == 2 ? 15 : 16;
  using V4 = typename Vec<E>::type;
  extern __shared__ uint4 dynamic[];
  __shared__ Tokens tokens;
  __shared__ PassLds<WAVES> lds;
  uint32_t* bits = reinterpret_cast<uint32_t*>(dynamic);
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  // dx may be x: no restrict on it, and a vector is stored by the lane that loaded it
  const E* p = x + row * stride;
  E* q = dx + row * dx_stride;
  const int vecs = V / N;
  auto zeros = [&] {
    const V4 zero = {0u, 0u, 0u, 0u};
    for (int i = tid; i < vecs; i += THREADS) vstore_nt(q + (int64_t)i * N, zero);
    if (vecs * N + tid < V) q[vecs * N + tid] = Vec<E>::round(0.0f);
  };
  const int id = token_id(t, row, V);
  clear_bits<N, THREADS>(V, bits, tokens);
  if (!any_token(t, row, V)) {
    put_row(kl, state, t, row, 0.0f, Row{0.0, 0.0, 0.0f});
    if constexpr (GRAD) zeros();
    return;
  }
  const float mine = id >= 0 ? Vec<E>::value(p[id]) : 0.0f;
  const float logq = id >= 0 ? t.logp[row * t.k + tid] : -INFINITY;
  __syncthreads();
  set_bit<N>(id, 0, V, bits, tokens);
  __syncthreads();
  OthersPass<E, WAVES, H, GRAD> pass;
  const Others others = pass.run(p, V, reinterpret_cast<const uint8_t*>(bits), s, lds);
  const Row r = finish_row<WAVES>(t, V, others, id, mine, logq, tokens);
  put_row(kl, state, t, row, others.m, r);
  if constexpr (GRAD) {
    const float c = weights[row] * scale;
    if (c == 0.0f) return zeros();
    // the second pass unpacks the held vectors anew: their float32 values would take twice the registers
#pragma unroll
    for (int h = 0; h < H; ++h) asm volatile("" : "+v"(pass.held[h]));
    const float a = static_cast<float>(r.a), factor = a == 0.0f ? 0.0f : c * a, m = others.m;
    auto grad = [&](V4 w, int i) {
      float f[N];
      Vec<E>::unpack(w, f);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = factor * __builtin_amdgcn_exp2f(s.of(f[e] - m));
      vstore_nt(q + (int64_t)i * N, Vec<E>::pack(f));
    };
    if (pass.rest < V) q[pass.rest] = Vec<E>::round(factor * __builtin_amdgcn_exp2f(s.of(pass.last - m)));
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (pass.body + tid + h * THREADS < vecs) grad(pass.held[h], pass.body + tid + h * THREADS);
    // the lane's vectors of the body, last first
    int i = tid < pass.body ? tid + (pass.body - 1 - tid) / THREADS * THREADS : -1;
    for (; i - (U - 1) * THREADS >= 0; i -= U * THREADS) {
      V4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = vload_nt(p + (int64_t)(i - u * THREADS) * N);
#pragma unroll
      for (int u = 0; u < U; ++u) grad(w[u], i - u * THREADS);
    }
    for (; i >= 0; i -= THREADS) grad(vload_nt(p + (int64_t)i * N), i);
    // the entries at the teacher's tokens, over what the vectors put there
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (id >= 0) q[id] = Vec<E>::round(c * r.b);
  }
}

// ---------------------------------------------------------------------------
// few or long rows in pieces
// ---------------------------------------------------------------------------

struct Pieces {
  Others* part;  // [T][splits]
  float* x;      // [T][k]: the logits at the teacher's tokens (kept here: they may be overwritten)
};

template <class E>
__global__ __launch_bounds__(256) void distill_piece_kernel(const E* __restrict__ x, int64_t stride, int V, int splits,
                                                            int piece, Teacher t, Exponent s, Pieces pieces) {
  constexpr int N = Vec<E>::N, THREADS = 256;
  extern __shared__ uint4 dynamic[];
  __shared__ Tokens tokens;
  __shared__ PassLds<4> lds;
  uint32_t* bits = reinterpret_cast<uint32_t*>(dynamic);
  const int64_t row = blockIdx.x / (unsigned)splits;
  const int sp = (int)(blockIdx.x % (unsigned)splits);
  const int tid = threadIdx.x;
  const int lo = sp * piece;
  const int n = V - lo < piece ? V - lo : piece;
  const E* p = x + row * stride + lo;
  const int id = token_id(t, row, V);
  clear_bits<N, THREADS>(n, bits, tokens);
  if (!any_token(t, row, V)) return;
  if (id >= lo && id - lo < n) pieces.x[row * t.k + tid] = Vec<E>::value(p[id - lo]);
  __syncthreads();
  set_bit<N>(id, lo, n, bits, tokens);
  __syncthreads();
  OthersPass<E, 4, 1, false> pass;
  const Others others = pass.run(p, n, reinterpret_cast<const uint8_t*>(bits), s, lds);
  if (tid == 0) pieces.part[row * splits + sp] = others;
}

// A row's pieces joined, by one workgroup.
__global__ __launch_bounds__(256) void distill_join_kernel(int V, int splits, Teacher t, Pieces pieces,
                                                           float* __restrict__ kl, float* __restrict__ state) {
  __shared__ Tokens tokens;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const int id = token_id(t, row, V);
  tokens.id[tid] = id;
  if (tid == 0) tokens.twice = 0;
  if (!any_token(t, row, V)) return put_row(kl, state, t, row, 0.0f, Row{0.0, 0.0, 0.0f});
  const float mine = id >= 0 ? pieces.x[row * t.k + tid] : 0.0f;
  const float logq = id >= 0 ? t.logp[row * t.k + tid] : -INFINITY;
  const Others v = lane < splits ? pieces.part[row * splits + lane] : Others{-INFINITY, 0.0};
  const float m = at_max(lane_max(v.s > 0.0 ? v.m : -INFINITY));
  const Others all{m, lane_total(v.s > 0.0 ? v.s * exp(((double)v.m - m) * t.inv_temperature) : v.s)};
  __syncthreads();
  bool before = false;
#pragma unroll 4
  for (int e = 0; e < t.k; e += 4) {  // ids past the last are -1
    const int4 v = *reinterpret_cast<const int4*>(tokens.id + e);
    before |= (v.x == id) & (e < tid) | (v.y == id) & (e + 1 < tid) | (v.z == id) & (e + 2 < tid) |
              (v.w == id) & (e + 3 < tid);
  }
  if (before && id >= 0) tokens.twice = 1;
  __syncthreads();
  put_row(kl, state, t, row, m, finish_row<4>(t, V, all, id, mine, logq, tokens));
}

// A row without a token is masked: its divergence is 0 and its weight is not
// used, which shows only where that is not finite. Such a weight on a divergence
// of 0 is rare, and only then the row's ids are looked at.
template <int WAVES>
__device__ __forceinline__ void sum_losses(const float* kl, const float* weights, int64_t T, const int32_t* ids, int k,
                                           int V, float* loss) {
  __shared__ double lds[WAVES];
  double sum = 0.0;
  bool ask = false;
#pragma unroll 8
  for (int64_t t = threadIdx.x; t < T; t += 64 * WAVES) {
    const float w = weights[t];
    if (w != 0.0f) {
      const float v = kl[t];
      const bool plain = v != 0.0f || fabsf(w) < INFINITY;
      sum += plain ? (double)w * v : 0.0;
      ask = ask || !plain;
    }
  }
  if (ask) {
    for (int64_t t = threadIdx.x; t < T; t += 64 * WAVES) {
      if (kl[t] != 0.0f || fabsf(weights[t]) < INFINITY) continue;
      for (int i = 0; i < k; ++i)
        if (static_cast<unsigned>(ids[t * k + i]) < (unsigned)V) sum = NAN;  // not masked: 0 times NaN or infinity
    }
  }
  sum = block_sum<WAVES>(sum, lds);
  if (threadIdx.x == 0) *loss = static_cast<float>(sum);
}

__global__ __launch_bounds__(1024) void distill_sum_kernel(const float* __restrict__ kl,
                                                           const float* __restrict__ weights, int64_t T,
                                                           const int32_t* __restrict__ ids, int k, int V,
                                                           float* __restrict__ loss) {
  sum_losses<16>(kl, weights, T, ids, k, V, loss);
}

// A workgroup takes one piece of a row, a vector per lane; the entries at the
// teacher's tokens follow once the vectors are written. One more at the end of
// the grid sums the rows' losses.
template <class E>
__global__ __launch_bounds__(kGradVecs) void distill_grad_kernel(GradArgs<E> a, const int32_t* __restrict__ ids, int k,
                                                                 const float* __restrict__ state,
                                                                 const float* __restrict__ coef,
                                                                 const float* __restrict__ grad_out, float scale,
                                                                 Exponent s, int64_t T, const float* __restrict__ kl,
                                                                 float* __restrict__ loss) {
  constexpr int N = Vec<E>::N;
  const int64_t row = blockIdx.x / (unsigned)a.pieces;
  if (row == T) return sum_losses<kGradVecs / 64>(kl, coef, T, ids, k, a.V, loss);
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int kMaxPieceVecs = 32768;  // vectors of a row that one workgroup takes: a byte of LDS for each
constexpr int kMaxSplits = 64;
constexpr int64_t kMaxVocab = int64_t(kMaxSplits) * kMaxPieceVecs * 4;

// Pieces of a row: about as many as give 1024 workgroups, of at least 4096
// logits each.
static int piece_splits(int64_t T, int64_t V) {
  const int64_t rows = T < 1 ? 1 : T;
  int64_t splits = (1024 + rows / 2) / rows;
  const int64_t most = ceil_div(V, 4096), least = ceil_div(V, int64_t(kMaxPieceVecs) * 4);
  splits = splits < most ? splits : most;
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  return static_cast<int>(splits > least ? splits : least > 1 ? least : 1);
}

// Whether one workgroup takes a whole row. A few long rows leave most of the
// card idle so; in pieces they take two launches, and three with the gradient,
// which reads all for a second time. us by rows and in pieces, k = 64, no row
// masked; the divergence alone:
//   bfloat16   80000 columns: 8 rows 14.0, 15.8; 96 rows 14.7, 16.0
//             100000: 64 rows 15.8, 16.1; 128 rows 16.1, 17.1
//             128256: 64 rows 17.3, 15.9; 112 rows 17.5, 17.2; 128 rows 17.6, 17.9; 160 rows 17.7, 19.2
//             200000: 128 rows 22.3, 20.2; 160 rows 22.7, 22.6; 192 rows 23.2, 23.8
//   float32    80000: 8 rows 15.0, 15.9; 96 rows 16.0, 16.6
//             100000: 64 rows 17.4, 16.1; 112 rows 18.0, 17.7; 128 rows 18.2, 18.9
//             128256: 96 rows 19.7, 19.2; 128 rows 20.3, 20.5; 160 rows 21.2, 23.0
// and a step:
//   bfloat16   32000: 8 rows 17.3, 20.3; 50000: 8 rows 18.2, 20.4; 96 rows 19.6, 22.6
//              64000: 48 rows 20.8, 20.8; 96 rows 21.2, 23.4
//             100000: 80 rows 26.9, 25.1; 96 rows 27.2, 26.6; 112 rows 27.6, 28.2
//             128256: 80 rows 29.0, 26.8; 96 rows 28.9, 28.9; 112 rows 29.4, 30.3
//             200000: 96 rows 38.2, 36.0; 112 rows 39.2, 38.2; 128 rows 39.4, 41.1
//   float32    32000: 8 rows 17.3, 20.2; 50000: 24 rows 21.0, 20.3; 48 rows 21.9, 21.3; 64 rows 21.9, 22.5
//             128256: 48 rows 29.0, 26.7; 64 rows 29.0, 29.7
// Few rows in pieces wait for the host, which made that 15 to 16 us of a
// divergence and 18 to 20 of a step from run to run.
// Rows of kMaxPieceVecs vectors and more (131072 float32, 262144 bfloat16) go in
// pieces however many they are: a workgroup's bits have no room for them. That
// costs many rows a second read from memory; us a step of 4096 rows right below
// and at that limit: float32 968, 1063; bfloat16 970, 1088.
static bool by_rows(const lora_mat* x, bool grad) {
  if (x->cols / vec_elems(x->dtype) >= kMaxPieceVecs) return false;
  if (grad) return x->cols <= 49152 || x->rows >= (x->dtype == LORA_F32 ? 64 : 104);
  return x->cols <= 81920 || x->rows >= 144;
}

// Waves to a row: with the gradient eight keep 7680 of its vectors in registers
// (8192 of float32), four 2560, sixteen 14336. us a step of 8192 x 128256
// bfloat16, k = 64, a third of the rows masked, by 4, 8 and 16 waves: 755, 697
// and 848 (one workgroup of 16 to a CU leaves nothing beside its serial part).
// Of these 697 the second read takes 24, the exponentials of the second pass 20;
// the rest is 3.6 GB at 5.5 TB/s. Up to 256 long rows, one to a CU, take 16
// waves. us a step of k = 64, 128256 columns, by 16 and by 8: bfloat16 128 rows
// 27.8 and 28.8, 256 rows 32.0 and 37.0; float32 64 rows 28.0 and 32.5, 256 rows
// 57.6 and 62.8. Without the gradient: bfloat16 128 rows 17.8 and 16.3.
static int row_waves(const lora_mat* x, bool grad) {
  const int64_t vecs = x->cols / vec_elems(x->dtype);
  return vecs <= 2560 ? 4 : grad && vecs > 8192 && x->rows <= 256 ? 16 : 8;
}

struct DistillPlan {
  float* state;
  Pieces pieces;
  size_t bytes;
};

static DistillPlan plan_distill(int64_t T, int64_t V, int64_t k, void* ws) {
  DistillPlan l{};
  Carver w(ws);
  l.state = static_cast<float*>(w.take(T * (k + kStateHead) * sizeof(float)));
  l.pieces.part = static_cast<Others*>(w.take(T * piece_splits(T, V) * sizeof(Others)));
  l.pieces.x = static_cast<float*>(w.take(T * k * sizeof(float)));
  l.bytes = w.used > 0 ? w.used : 256;
  return l;
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

static size_t bit_bytes(int64_t elems, int n) { return static_cast<size_t>(round_up(elems / n + 1, 16)); }

// The rows whole: divergences (and states), with dx their gradients too.
static void run_rows(const lora_mat* x, const lora_teacher* t, float* kl, float* state, const float* weights,
                     float scale, const lora_mat* dx, hipStream_t st) {
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const int waves = row_waves(x, dx != nullptr);
    auto* kernel = dx == nullptr ? (waves == 4 ? distill_row_kernel<E, 4, false> : distill_row_kernel<E, 8, false>)
                   : waves == 4  ? distill_row_kernel<E, 4, true>
                   : waves == 8  ? distill_row_kernel<E, 8, true>
                                 : distill_row_kernel<E, 16, true>;
    launch(kernel, dim3(x->rows), dim3(64 * waves), bit_bytes(x->cols, Vec<E>::N), st, (const E*)x->ptr, x->stride_row,
           static_cast<int>(x->cols), teacher_of(t), exponent_of(t->temperature), kl, state, weights, scale,
           dx == nullptr ? (E*)nullptr : (E*)dx->ptr, dx == nullptr ? int64_t(0) : dx->stride_row);
  });
}

// The rows in pieces: divergences and states.
static void run_pieces(const lora_mat* x, const lora_teacher* t, const DistillPlan& l, float* kl, float* state,
                       hipStream_t st) {
  const int splits = piece_splits(x->rows, x->cols), V = static_cast<int>(x->cols);
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const int piece = static_cast<int>(round_up(ceil_div(V, splits), Vec<E>::N));
    launch(distill_piece_kernel<E>, dim3(x->rows * splits), dim3(256), bit_bytes(piece, Vec<E>::N), st,
           (const E*)x->ptr, x->stride_row, V, splits, piece, teacher_of(t), exponent_of(t->temperature), l.pieces);
  });
  launch(distill_join_kernel, dim3(x->rows), dim3(256), 0, st, V, splits, teacher_of(t), l.pieces, kl, state);
}

static void run_grad(const lora_mat* x, const int32_t* ids, int k, const float* state, const float* coef,
                     const float* grad_out, float scale, double temperature, const lora_mat* dx, const float* kl,
                     float* loss, hipStream_t st) {
  by_type(x, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const GradArgs<E> a = grad_args<E>(x, dx);
    launch(distill_grad_kernel<E>, dim3(x->rows * a.pieces + (loss != nullptr)), dim3(kGradVecs), 0, st, a, ids, k,
           state, coef, grad_out, static_cast<float>((double)scale / temperature), exponent_of(temperature), x->rows,
           kl, loss);
  });
}

}  // namespace lora

using namespace lora;

extern "C" size_t lora_distill_workspace_bytes(int64_t T, int64_t V, int64_t k) {
  if (T < 0 || V < 0 || k < 1 || T > kMaxRows || V > kMaxVocab || k > kMaxTeacher) return 0;
  return plan_distill(T, V, k, nullptr).bytes;
}

// The checks that the divergence and the step share; `blocks`: workgroups of 64 * waves of the largest launch (16
// waves take 256 rows at most).
static int check_distill(const lora_mat* x, const lora_teacher* t, bool grad) {
  if (int e = check_teacher(t, x->rows)) return e;
  if (x->cols > kMaxVocab) return LORA_ERR_LIMIT;
  const bool rows = by_rows(x, grad);
  const int64_t blocks = rows ? x->rows : x->rows * piece_splits(x->rows, x->cols);
  return blocks > max_blocks(rows ? 64 * row_waves(x, false) : 256) ? LORA_ERR_LIMIT : LORA_OK;
}

static int check_plan(const DistillPlan& l, void* ws, size_t bytes) {
  return !ws || bytes < l.bytes || !aligned(ws, 256) ? LORA_ERR_WORKSPACE : LORA_OK;
}

extern "C" int lora_distill_kl(const lora_mat* logits, const lora_teacher* teacher, float* kl, float* state,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (int e = check_distill(logits, teacher, false)) return e;
  const int64_t T = logits->rows, V = logits->cols;
  if (T == 0) return LORA_OK;
  if (!kl || (V > 0 && !logits->ptr)) return LORA_ERR_NULL;
  const DistillPlan l = plan_distill(T, V, teacher->k, workspace);
  if (int e = check_plan(l, workspace, workspace_bytes)) return e;
  auto st = static_cast<hipStream_t>(stream);
  if (by_rows(logits, false))
    run_rows(logits, teacher, kl, state, nullptr, 0.0f, nullptr, st);
  else
    run_pieces(logits, teacher, l, kl, state, st);
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
  run_grad(logits, top_ids, static_cast<int>(k), state, coef, grad_out, scale, temperature, dlogits, nullptr, nullptr,
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
  if (int e = check_distill(logits, teacher, true)) return e;
  if (!loss || (T > 0 && (!weights || !kl || (V > 0 && (!logits->ptr || !dlogits->ptr))))) return LORA_ERR_NULL;
  const DistillPlan l = plan_distill(T, V, teacher->k, workspace);
  if (T > 0)
    if (int e = check_plan(l, workspace, workspace_bytes)) return e;
  auto st = static_cast<hipStream_t>(stream);
  if (T > 0 && V > 0 && !by_rows(logits, true)) {
    run_pieces(logits, teacher, l, kl, l.state, st);
    run_grad(logits, teacher->ids, static_cast<int>(teacher->k), l.state, weights, nullptr, grad_scale,
             teacher->temperature, dlogits, kl, loss, st);
    return launch_status();
  }
  if (T > 0)
    run_rows(logits, teacher, kl, nullptr, weights, static_cast<float>((double)grad_scale / teacher->temperature),
             dlogits, st);
  launch(distill_sum_kernel, dim3(1), dim3(1024), 0, st, (const float*)kl, weights, T, teacher->ids,
         static_cast<int>(teacher->k), static_cast<int>(V), loss);
  return launch_status();
}
