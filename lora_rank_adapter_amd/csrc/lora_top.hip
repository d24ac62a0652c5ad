// Log probabilities of given tokens with the entropy and the top alternatives
// of every row of logits, and the gradient of log probability and entropy.
//
//   d_j = (x_j - m) / tau, m the row's largest logit
//   r   = sum of exp(d_j) over all but the first of the largest logits
//   log p_j = d_j - log1p(r),  gap = sum p_j (-d_j),  entropy = log1p(r) + gap
//
// With its 1 left out of the sum, r keeps its own precision in a row whose
// largest logit holds nearly all of the probability, and with it the entropy,
// the log probabilities and their gradients; every term of gap is positive.
//
// Kernels:
//   top_kernel       a workgroup to a row: the statistics, the k largest logits
//   top_grad_kernel  the gradient's rows from the statistics

#include <type_traits>

#include "lora_softmax.hpp"

namespace lora {

constexpr int kMaxTop = 128;  // alternatives of a row

// Unsigned numbers in the order of the values; -0 equals 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

// An alternative as one number: the larger value first, then the lower column.
__device__ __forceinline__ uint64_t entry_of(float x, int column) {
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(column));
}
__device__ __forceinline__ int column_of(uint64_t entry) { return static_cast<int>(0xFFFFFFFFu - (uint32_t)entry); }

// A row's statistics; undefined (a NaN, +inf, or nothing above -inf): NaN.
struct TopStats {
  float m;
  double r, gap;
  __device__ __forceinline__ bool defined() const { return m > -INFINITY && m < INFINITY && r == r; }
};

struct TopOut {
  float *logp, *entropy;
  int32_t* ids;
  float *top, *stats;
  int k;
  double inv_temperature;
};

// What a row gives, by all threads of a workgroup; entries: the k largest in
// order, `count` of them.
__device__ __forceinline__ void put_row(const TopOut& o, int64_t row, const TopStats& v, bool target, float x,
                                        const uint64_t* entries, int count) {
  const bool ok = v.defined();
  const double ls = log1p(v.r);
  if (threadIdx.x == 0) {
    if (o.logp != nullptr)
      o.logp[row] = !target ? 0.0f : ok ? static_cast<float>(((double)x - v.m) * o.inv_temperature - ls) : NAN;
    o.entropy[row] = ok ? static_cast<float>(ls + v.gap) : NAN;
    o.stats[3 * row] = ok ? v.m : NAN;
    o.stats[3 * row + 1] = ok ? static_cast<float>(v.r) : NAN;
    o.stats[3 * row + 2] = ok ? static_cast<float>(v.gap) : NAN;
  }
  if ((int)threadIdx.x < o.k) {
    const int i = threadIdx.x;
    const bool there = ok && i < count;
    const uint64_t e = there ? entries[i] : 0;
    const double d = ((double)value_of(static_cast<uint32_t>(e >> 32)) - v.m) * o.inv_temperature;
    o.ids[row * o.k + i] = there ? column_of(e) : -1;
    o.top[row * o.k + i] = there ? static_cast<float>(d - ls) : ok ? -INFINITY : NAN;
  }
}

// A masked row.
__device__ __forceinline__ void put_masked(const TopOut& o, int64_t row) {
  if (threadIdx.x == 0) {
    o.logp[row] = o.entropy[row] = 0.0f;
    o.stats[3 * row] = o.stats[3 * row + 1] = o.stats[3 * row + 2] = 0.0f;
  }
  if ((int)threadIdx.x < o.k) {
    o.ids[row * o.k + threadIdx.x] = -1;
    o.top[row * o.k + threadIdx.x] = -INFINITY;
  }
}

// f(value, column) for each of the thread's elements of a row.
template <class E, int THREADS, class F>
__device__ __forceinline__ void each_element(const E* p, int V, F f) {
  constexpr int N = Vec<E>::N;
  const int vecs = V / N;
  for (int i = threadIdx.x; i < vecs; i += THREADS) {
    float v[N];
    Vec<E>::unpack(vload(p + (int64_t)i * N), v);
#pragma unroll
    for (int e = 0; e < N; ++e) f(v[e], i * N + e);
  }
  const int rest = vecs * N + threadIdx.x;
  if (rest < V) f(Vec<E>::value(p[rest]), rest);
}

struct Kth {
  uint32_t order;  // of the k-th largest element
  int equal;       // how many of the elements equal to it are among the k
};

// The k-th largest of the elements that each(f) gives f(order) of, by one
// digit of 8 bits after the other; k is at most their number.
template <int THREADS, class Each>
__device__ __forceinline__ Kth kth_largest(Each each, int k, int* hist, int* found) {
  Kth v{0u, k};
  uint32_t mask = 0u;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += THREADS) hist[i] = 0;
    __syncthreads();
    each([&](uint32_t order) {
      if ((order & mask) == v.order) atomicAdd(&hist[order >> shift & 255u], 1);
    });
    __syncthreads();
    if (threadIdx.x < 64) {
      // lane l has the digits 255 - 4 l and the three below
      int c[4], sum = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += c[j] = hist[255 - 4 * threadIdx.x - j];
      int upto = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int other = __shfl_up(upto, d, 64);
        if ((int)threadIdx.x >= d) upto += other;
      }
      int above = upto - sum;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (above < v.equal && v.equal <= above + c[j]) {
          found[0] = 255 - 4 * threadIdx.x - j;
          found[1] = v.equal - above;
        }
        above += c[j];
      }
    }
    __syncthreads();
    v.order |= static_cast<uint32_t>(found[0]) << shift;
    v.equal = found[1];
    mask |= 255u << shift;
  }
  return v;
}

template <class E>
__global__ __launch_bounds__(256) void top_kernel(const E* __restrict__ x, int64_t stride,
                                                  const int32_t* __restrict__ targets, int V, Exponent s, TopOut out) {
  constexpr int N = Vec<E>::N, THREADS = 256;
  __shared__ float wave_m[4];
  __shared__ int wave_at[4];
  __shared__ double lds[4];
  __shared__ int hist[256], found[2], count, wave_ties[4];
  __shared__ uint64_t list[kMaxTop], sorted[kMaxTop];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int y = targets != nullptr ? targets[row] : -1;
  const bool target = y >= 0 && y < V;
  if (targets != nullptr && !target) return put_masked(out, row);
  const E* p = x + row * stride;
  const int vecs = V / N;
  // the first of the largest logits
  float m = -INFINITY;
  int at = 0x7FFFFFFF;
  each_element<E, THREADS>(p, V, [&](float f, int j) {
    if (f > m) {
      m = f;
      at = j;
    }
  });
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const float om = __shfl_xor(m, d, 64);
    const int oat = __shfl_xor(at, d, 64);
    if (om > m || (om == m && oat < at)) {
      m = om;
      at = oat;
    }
  }
  if ((tid & 63) == 0) {
    wave_m[tid >> 6] = m;
    wave_at[tid >> 6] = at;
  }
  if (tid == 0) count = 0;
  __syncthreads();
  m = wave_m[0];
  at = wave_at[0];
  for (int w = 1; w < 4; ++w) {
    if (wave_m[w] > m || (wave_m[w] == m && wave_at[w] < at)) {
      m = wave_m[w];
      at = wave_at[w];
    }
  }
  // the sums over the others
  double r = 0.0, g = 0.0;
  const float z = at_max(m);
  each_element<E, THREADS>(p, V, [&](float f, int j) {
    if (j == at) return;
    const float a = s.of(f - z), e = __builtin_amdgcn_exp2f(a);
    r += e;
    g -= (double)e * fmaxf(a, -256.0f);
  });
  r = block_sum<4>(r, lds);
  g = block_sum<4>(g, lds);
  const TopStats stats{m, r, g * kLn2 / (1.0 + r)};
  // the k largest: all above the k-th, then the first ones equal to it
  const int k = out.k < V ? out.k : V;
  if (k > 0) {
    const Kth kth = kth_largest<THREADS>(
        [&](auto f) { each_element<E, THREADS>(p, V, [&](float v, int) { f(order_of(v)); }); }, k, hist, found);
    each_element<E, THREADS>(p, V, [&](float v, int j) {
      if (order_of(v) > kth.order) list[atomicAdd(&count, 1)] = entry_of(v, j);
    });
    int want = kth.equal, have = k - kth.equal;
    for (int j0 = 0; j0 < V && want > 0; j0 += THREADS) {
      const int j = j0 + tid;
      const bool tie = j < V && order_of(Vec<E>::value(p[j])) == kth.order;
      const uint64_t lanes = __ballot(tie);
      if ((tid & 63) == 0) wave_ties[tid >> 6] = __popcll(lanes);
      __syncthreads();
      int before = __popcll(lanes & ((1ull << (tid & 63)) - 1)), all = 0;
      for (int w = 0; w < 4; ++w) {
        before += w < (tid >> 6) ? wave_ties[w] : 0;
        all += wave_ties[w];
      }
      if (tie && before < want) list[have + before] = entry_of(value_of(kth.order), j);
      have += all < want ? all : want;
      want -= all < want ? all : want;
      __syncthreads();
    }
    __syncthreads();
    if (tid < k) {
      int rank = 0;
      for (int i = 0; i < k; ++i) rank += list[i] > list[tid];
      sorted[rank] = list[tid];
    }
    __syncthreads();
  }
  put_row(out, row, stats, target, target ? Vec<E>::value(p[y]) : 0.0f, sorted, k);
}

// ---------------------------------------------------------------------------
// gradient: with g = d loss / d logp and h = d loss / d entropy of the row,
//   dx_j = (g ([j = y] - p_j) - h p_j (log p_j + entropy)) / tau
// and log p_j + entropy = d_j + gap. A workgroup takes one piece of a row, a
// vector per lane, which writes memory fastest.
// ---------------------------------------------------------------------------
template <class E>
__global__ __launch_bounds__(kGradVecs) void top_grad_kernel(GradArgs<E> a, const int32_t* __restrict__ targets,
                                                             const float* __restrict__ stats,
                                                             const float* __restrict__ dlogp,
                                                             const float* __restrict__ dentropy, Exponent s,
                                                             float inv_temperature) {
  constexpr int N = Vec<E>::N;
  constexpr float kLn2f = static_cast<float>(kLn2);
  const int64_t row = blockIdx.x / (unsigned)a.pieces;
  const int lo = (blockIdx.x % (unsigned)a.pieces) * kGradVecs * N;
  const int n = a.V - lo < kGradVecs * N ? a.V - lo : kGradVecs * N;
  const int tid = threadIdx.x;
  const E* p = a.x + row * a.stride + lo;
  E* q = a.dx + row * a.dx_stride + lo;
  const int vecs = n / N;
  const int rest = vecs * N + tid;  // the row's last elements, one per lane
  const int y = targets != nullptr ? targets[row] : -1;
  const bool live = targets == nullptr || (y >= 0 && y < a.V);
  const float g = live && dlogp != nullptr ? dlogp[row] : 0.0f;
  const float h = live && dentropy != nullptr ? dentropy[row] : 0.0f;
  if (g == 0.0f && h == 0.0f) {
    const typename Vec<E>::type zero = {0u, 0u, 0u, 0u};
    if (tid < vecs) vstore_nt(q + tid * N, zero);
    if (rest < n) q[rest] = Vec<E>::round(0.0f);
    return;
  }
  const float m = stats[3 * row], r = stats[3 * row + 1], gap = stats[3 * row + 2];
  const float c = inv_temperature / (1.0f + r);
  const float c0 = -c * fmaf(h, gap, g), c1 = -c * h * kLn2f;
  const int hit = y - lo;
  auto grad = [&](float f, bool own) {
    const float b = s.of(f - m), e = __builtin_amdgcn_exp2f(b);
    const float held = fmaxf(b, -256.0f);  // e is 0 there, and 0 times -inf is not
    if (!own) return e * fmaf(c1, held, c0);
    // 1 - p from the log probability: it keeps its precision beside a likely token
    const float logp = fmaf(held, kLn2f, -log1pf(r));
    return fmaf(-g * inv_temperature, expm1f(logp), e * fmaf(c1, held, -c * h * gap));
  };
  if (tid < vecs) {
    float f[N], d[N];
    Vec<E>::unpack(vload_nt(p + tid * N), f);
#pragma unroll
    for (int e = 0; e < N; ++e) d[e] = grad(f[e], false);
    if (static_cast<unsigned>(hit - tid * N) < N) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (tid * N + e == hit) d[e] = grad(f[e], true);
    }
    vstore_nt(q + tid * N, Vec<E>::pack(d));
  }
  if (rest < n) q[rest] = Vec<E>::round(grad(Vec<E>::value(p[rest]), rest == hit));
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

}  // namespace lora

using namespace lora;

extern "C" size_t lora_token_top_workspace_bytes(int64_t T, int64_t V, int64_t k) {
  if (T < 0 || V < 0 || k < 0 || T > kMaxRows || V > 0x7FFFFFFF - 8 * kGradVecs || k > kMaxTop) return 0;
  return 256;
}

extern "C" int lora_token_top(const lora_mat* logits, const int32_t* targets, int64_t k, double temperature,
                              float* logp, float* entropy, int32_t* top_ids, float* top_logp, float* stats,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (k < 0) return LORA_ERR_SHAPE;
  if (k > kMaxTop) return LORA_ERR_LIMIT;
  if (!temperature_ok(temperature)) return LORA_ERR_VALUE;
  const int64_t T = logits->rows;
  if (T == 0) return LORA_OK;
  if (!entropy || !stats || (logits->cols > 0 && !logits->ptr)) return LORA_ERR_NULL;
  if ((targets != nullptr) != (logp != nullptr) || (k > 0 && (!top_ids || !top_logp))) return LORA_ERR_NULL;
  const size_t need = lora_token_top_workspace_bytes(T, logits->cols, k);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return LORA_ERR_WORKSPACE;
  const TopOut out{logp, entropy, top_ids, top_logp, stats, static_cast<int>(k), 1.0 / temperature};
  by_type(logits, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    launch(top_kernel<E>, dim3(T), dim3(256), 0, static_cast<hipStream_t>(stream), (const E*)logits->ptr,
           logits->stride_row, targets, static_cast<int>(logits->cols), exponent_of(temperature), out);
  });
  return launch_status();
}

extern "C" int lora_token_top_grad(const lora_mat* logits, const int32_t* targets, const float* stats,
                                   const float* dlogp, const float* dentropy, double temperature,
                                   const lora_mat* dlogits, void* stream) {
  if (!logits || !dlogits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (int e = check_dlogits(logits, dlogits)) return e;
  if (!temperature_ok(temperature)) return LORA_ERR_VALUE;
  if (logits->rows == 0 || logits->cols == 0) return LORA_OK;
  if (!stats || !logits->ptr || !dlogits->ptr || (!targets && dlogp)) return LORA_ERR_NULL;
  by_type(logits, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    const GradArgs<E> a = grad_args<E>(logits, dlogits);
    launch(top_grad_kernel<E>, dim3(logits->rows * a.pieces), dim3(kGradVecs), 0, static_cast<hipStream_t>(stream), a,
           targets, stats, dlogp, dentropy, exponent_of(temperature), static_cast<float>(1.0 / temperature));
  });
  return launch_status();
}
