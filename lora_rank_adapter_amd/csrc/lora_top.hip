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
//   top_kernel       one pass over a row (or one piece of it): the statistics, the k largest logits
//   top_join_kernel  the pieces of a row joined
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

// A row's statistics, or those of a piece of it. A row with a NaN, with +inf or
// with nothing above -inf has no probabilities; r is NaN with a NaN, and 0 in a
// piece with nothing above -inf.
struct TopStats {
  float m;
  double r, gap;  // gap: in a piece times 1 + r
  __device__ __forceinline__ bool defined() const { return m > -INFINITY && m < INFINITY && r == r; }
};

struct TopOut {
  float *logp, *entropy;
  int32_t* ids;
  float *top, *stats;
  int k;
  double inv_temperature;
};

// What a row gives, by all threads of a workgroup; entries: its k largest in
// order, `count` of them.
__device__ __forceinline__ void put_row(const TopOut& o, int64_t row, const TopStats& v, bool target, float x,
                                        const uint64_t* entries, int count) {
  if (threadIdx.x >> 6 > 0 && (int)threadIdx.x >= o.k) return;
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

// ---------------------------------------------------------------------------
// selection of the k largest of a set of entries by a workgroup
// ---------------------------------------------------------------------------

constexpr int kList = 512;    // entries that are put in order at most
constexpr int kDirect = 192;  // and so many without a look at their bins first
constexpr float kFloor = -1e30f;   // logits below (-inf, a mask's lowest values) share one bin

struct Select {
  int hist[256];
  int count;  // entries in the list
  uint32_t low;
  uint64_t list[kList], sorted[kMaxTop];
};

// Room for n more of each lane behind *count, by the whole wave at once.
__device__ __forceinline__ int reserve(int n, int* count) {
  const int upto = lane_sums(n), total = __builtin_amdgcn_readlane(upto, 63);
  int at = 0;
  if (total > 0 && (threadIdx.x & 63) == 63) at = atomicAdd(count, total);
  return __builtin_amdgcn_readlane(at, 63) + upto - n;
}

// 255 bins of equal width from hi down to lo and below, and the one of kFloor.
struct Bins {
  float hi, scale;
  __device__ __forceinline__ Bins(float hi, float lo) : hi(hi), scale(lo < hi ? 254.0f / (hi - lo) : 0.0f) {}
  __device__ __forceinline__ int of(float f) const {
    return f >= kFloor ? (int)fmaxf(fminf((hi - f) * scale, 254.0f), 0.0f) : 255;
  }
};

// The bin of the k-th entry, from bin 0 on; 255 if there are fewer. Every wave
// finds it for itself.
__device__ __forceinline__ int kth_bin(const int* hist, int k) {
  const int lane = threadIdx.x & 63;
  int c[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) sum += c[j] = hist[4 * lane + j];
  const int upto = lane_sums(sum);
  const uint64_t reached = __ballot(upto >= k);
  if (reached == 0) return 255;
  int before = upto - sum, bin = 4 * lane;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    before += c[j];
    if (before < k) ++bin;
  }
  return __builtin_amdgcn_readlane(bin, __builtin_ctzll(reached));
}

template <int THREADS>
__device__ __forceinline__ void clear(Select& l) {
  for (int i = threadIdx.x; i < 256; i += THREADS) l.hist[i] = 0;
  if (threadIdx.x == 0) l.count = 0;
}

// The first k of n entries in order.
template <int THREADS>
__device__ __forceinline__ void sort_list(const uint64_t* list, int n, int k, uint64_t* sorted) {
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const uint64_t e = list[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += list[j] > e;
    if (rank < k) sorted[rank] = e;
  }
  __syncthreads();
}

// The k largest of the entries that each(f) gives f(value, column) of, in order;
// hi is the largest value, lo one that k entries reach. False if too many share
// the k-th's bin. Starts from a cleared l, with a barrier behind it.
template <int THREADS, class Each>
__device__ __forceinline__ bool select_top(Each each, float hi, float lo, int k, Select& l) {
  const Bins bins(hi, lo);
  each([&](float f, int) { atomicAdd(&l.hist[bins.of(f)], 1); });
  __syncthreads();
  const int last = kth_bin(l.hist, k);
  each([&](float f, int column) {
    if (bins.of(f) > last) return;
    const int at = atomicAdd(&l.count, 1);
    if (at < kList) l.list[at] = entry_of(f, column);
  });
  __syncthreads();
  if (l.count > kList) return false;
  sort_list<THREADS>(l.list, l.count, k, l.sorted);
  return true;
}

// The same for any entries, in eight passes over them: the k-th entry by one
// digit of 8 bits after the other, then all from it on. k is at most their number.
template <int THREADS, class Each>
__device__ __forceinline__ void select_exactly(Each each, int k, Select& l) {
  uint64_t kth = 0, mask = 0;
  int want = k;
  for (int shift = 56; shift >= 0; shift -= 8) {
    __syncthreads();
    clear<THREADS>(l);
    __syncthreads();
    // neighbours are often equal: a thread counts a run of them before it adds it
    int run_bin = 0, run = 0;
    each([&](float f, int column) {
      const uint64_t e = entry_of(f, column);
      if ((e & mask) != kth) return;
      const int bin = 255 - (int)(e >> shift & 255);
      if (bin != run_bin) {
        if (run > 0) atomicAdd(&l.hist[run_bin], run);
        run_bin = bin;
        run = 0;
      }
      ++run;
    });
    if (run > 0) atomicAdd(&l.hist[run_bin], run);
    __syncthreads();
    const int bin = kth_bin(l.hist, want);
    for (int i = 0; i < bin; ++i) want -= l.hist[i];
    kth |= static_cast<uint64_t>(255 - bin) << shift;
    mask |= static_cast<uint64_t>(255) << shift;
  }
  each([&](float f, int column) {
    const uint64_t e = entry_of(f, column);
    if (e < kth) return;
    const int at = atomicAdd(&l.count, 1);
    if (at < kList) l.list[at] = e;
  });
  __syncthreads();
  sort_list<THREADS>(l.list, l.count < kList ? l.count : kList, k, l.sorted);
}

// ---------------------------------------------------------------------------
// statistics and alternatives: a workgroup reads its row, or its piece of one,
// once. Its first 32 elements per lane are held while the largest of each lane
// are compared: the k-th of these is reached by k elements at least, so only
// vectors that reach it can matter. They go to a list in LDS, together with
// those of the rest of the row, a few hundred in all, and the k largest are
// found among them. The sums are relative to the largest logit of these first
// elements, no running maximum, but for the vectors that reach it: these are
// listed, and summed behind the loop relative to the largest of their wave. So no
// exponent is far above its reference, which would cost it precision.
//
// The row is read again: for the sums if the reference is 2^24 binary orders away
// from 0, or not all that reach it are listed; for the alternatives if the list
// overflows (logits that rise along the row, a masked beginning: from the k-th of
// the lanes' largest in the whole row on) or holds fewer than k (ties without end,
// a vocabulary masked down to a few tokens: the lowest columns of the next value).
// us a call of 256 rows of 128256 bfloat16, k = 20: random logits 21, rising 48,
// one value throughout 71, masked down to 5 tokens 44, masked in their first
// half 46.
//
// Memory bounds many rows: 5744 of 8192 x 128256 bfloat16 without alternatives
// 231 us (6.4 TB/s; the loop's vector instructions went from 69 to 53 for 8
// logits without a change), 4096 with k = 64 193 us (5.5 TB/s: of a workgroup's
// 40 us half go into the threshold and the selection, when only others load).
// 256 rows are one workgroup per CU: reading takes 13 of the 21 us, the first
// loads, the threshold and the selection the rest.
// ---------------------------------------------------------------------------

constexpr float kFar = 0x1p24f;  // binary orders that the reference may be away from 0
constexpr int kMaxSplits = 64;

// Sums of a vector's exponentials e = 2^a and of e a.
struct VecSums {
  float s, w;
};

template <int N>
__device__ __forceinline__ float tree(const float* f) {
  if constexpr (N == 1)
    return f[0];
  else
    return tree<N / 2>(f) + tree<N / 2>(f + N / 2);
}

// The sums of a vector added to t; a(f) is the exponent of a logit.
template <class E, class F>
__device__ __forceinline__ VecSums add_sums(typename Vec<E>::type v, F a, VecSums t) {
  constexpr int N = Vec<E>::N;
  float f[N];
  Vec<E>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float b = a(f[i]);
    f[i] = __builtin_amdgcn_exp2f(b);
    t.w = fmaf(f[i], b, t.w);
  }
  t.s += tree<N>(f);
  return t;
}

// 0 times -inf is not 0: where a vector holds such an exponent (a logit of
// -inf) w is summed once more with bounds, which costs less than to have them
// everywhere (8192 x 128256: 251 -> 238 us).
template <class E, class F>
__device__ __forceinline__ float bound_w(typename Vec<E>::type v, F a, float w) {
  constexpr int N = Vec<E>::N;
  float f[N];
  Vec<E>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float b = a(f[i]);
    w = fmaf(__builtin_amdgcn_exp2f(b), fmaxf(b, -256.0f), w);
  }
  return w;
}
template <class E, class F>
__device__ __forceinline__ VecSums vec_sums(typename Vec<E>::type v, F a) {
  VecSums t = add_sums<E>(v, a, {0.0f, 0.0f});
  if (t.w != t.w) t.w = bound_w<E>(v, a, 0.0f);
  return t;
}

// Vector i of n elements; -inf past the last.
template <class E>
__device__ __forceinline__ typename Vec<E>::type vec_at(const E* p, int i, int n) {
  constexpr int N = Vec<E>::N;
  constexpr uint32_t low = N == 8 ? 0xFF80FF80u : 0xFF800000u;
  typename Vec<E>::type w = {low, low, low, low};
  if ((i + 1) * N <= n) return vload_nt(p + (int64_t)i * N);
#pragma unroll
  for (int e = 0; e < N - 1; ++e) {
    if (i * N + e >= n) continue;
    if constexpr (N == 8)
      w[e / 2] = e & 1 ? (w[e / 2] & 0xFFFFu) | (uint32_t)p[i * N + e] << 16 : (w[e / 2] & 0xFFFF0000u) | p[i * N + e];
    else
      w[e] = __float_as_uint(p[i * N + e]);
  }
  return w;
}

// fmaxf three at a time, without the instruction that makes a signalling NaN a
// quiet one first (such a row has no probabilities whatever its maximum).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}
template <int N>
__device__ __forceinline__ float vec_max(const float* f) {
  float m = f[0];
#pragma unroll
  for (int i = 1; i < N; i += 2) m = max3(m, f[i], f[i + 1 < N ? i + 1 : i]);
  return m;
}

struct TopPiece {
  double r, gap;
  float m;
};

// Where a piece of a row goes (splits > 1).
struct TopParts {
  TopPiece* stats;    // [T][splits]
  uint64_t* entries;  // [T][splits][k], 0 past the piece's elements
};

template <class E, int WAVES, int HITS>
__global__ __launch_bounds__(64 * WAVES, WAVES == 16 ? 4 : HITS == 256 || sizeof(E) == 2 ? 6 : 5) void top_kernel(
    const E* __restrict__ x, int64_t stride, const int32_t* __restrict__ targets, int V, int splits, int piece,
    Exponent s, TopOut out, TopParts parts) {
  constexpr int N = Vec<E>::N, U = 32 / N, B = 4, THREADS = 64 * WAVES, ROOM = HITS / WAVES;
  constexpr int FEW = WAVES == 4 && HITS > 512 ? 512 : HITS;  // more than 512 and LDS would hold a workgroup less
  using V4 = typename Vec<E>::type;
  __shared__ Select l;
  __shared__ uint4 hit[HITS];  // a part for each wave
  __shared__ int hit_at[HITS];
  __shared__ int overflow, candidates;
  __shared__ uint64_t candidate[FEW];
  __shared__ int wave_n[WAVES];
  __shared__ float wave_hi[WAVES], wave_lo[WAVES];
  __shared__ double wave_s[WAVES], wave_w[WAVES];
  __shared__ TopStats shared;
  const int64_t row = blockIdx.x / (unsigned)splits;
  const int sp = (int)(blockIdx.x % (unsigned)splits);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int y = targets != nullptr ? targets[row] : -1;
  const bool target = y >= 0 && y < V;
  if (targets != nullptr && !target) {
    if (splits == 1) put_masked(out, row);
    return;
  }
  const int lo = sp * piece;
  const int n = V - lo < piece ? V - lo : piece;
  const E* p = x + row * stride + lo;
  const int vecs = (n + N - 1) / N, whole = n / N;
  const int k = out.k < 1 ? 1 : out.k;  // the largest one is needed in any case
  const int kk = k < n ? k : n;

  // Loads past the last vector take it once more: behind a condition each would be waited for at once.
  auto next = [&](int i) { return vload_nt(p + (int64_t)(i < whole ? i : whole - 1) * N); };
  V4 w[U], a[B];  // four vectors are summed at a time, the next four on their way
  if (whole > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = next(tid + u * THREADS);
#pragma unroll
    for (int u = 0; u < B; ++u) a[u] = next(tid + (U + u) * THREADS);
  }
  sched_fence();
  if (tid == 0) {
    overflow = candidates = 0;
    l.sorted[0] = 0;  // of a row without elements
  }
  clear<THREADS>(l);
  float mine = -INFINITY;  // the lane's largest
  auto largest = [&](V4 v) {
    float f[N];
    Vec<E>::unpack(v, f);
    mine = fmaxf(mine, vec_max<N>(f));
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (tid + u * THREADS < whole) largest(w[u]);
  const bool part_of_one = tid == THREADS - 1 && whole < vecs;  // the last vector, in part
  if (part_of_one) largest(vec_at(p, whole, n));
  // A value that the k-th largest of the lanes' reaches; kFloor if fewer than k reach that. hi and low are the largest
  // and the smallest from kFloor on. l is clear before and after.
  float hi, low;
  auto kth_lane = [&](float v) {
    hi = lane_max(v);
    low = lane_min(v >= kFloor ? v : INFINITY);
    if ((tid & 63) == 0) {
      wave_hi[tid >> 6] = hi;
      wave_lo[tid >> 6] = low;
    }
    if (tid == 0) l.low = 0xFFFFFFFFu;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      hi = fmaxf(hi, wave_hi[w]);
      low = fminf(low, wave_lo[w]);
    }
    const int b = Bins(hi, low).of(v);
    atomicAdd(&l.hist[b], 1);
    __syncthreads();
    const int last = kth_bin(l.hist, k);
    if (b <= last) atomicMin(&l.low, order_of(v));
    __syncthreads();
    const float kth = last < 255 ? value_of(l.low) : kFloor;
    clear<THREADS>(l);
    return kth;
  };
  // vectors with an element from here on are listed: all of few
  float reach = kth_lane(mine);
  if (vecs <= 2 * k) reach = -INFINITY;
  const float z = at_max(hi);
  // Two products instead of a difference and two: what `shift` lost to rounding moves all exponents alike, the largest
  // logit's too (by at most two orders up to kFar, beyond which a piece is read again).
  const float shift = -z * s.hi;
  auto exponent = [&](float f) { return fmaf(f, s.lo, fmaf(f, s.hi, shift)); };

  // Every wave lists for itself. A vector that reaches the largest of the first elements may hold the row's largest:
  // its sums are left to the end, when that is known.
  const float first = hi;
  double sum = 0.0, wsum = 0.0;
  int hits = 0;
  auto list = [&](V4 v, int i, bool on) {
    const uint64_t those = __ballot(on);
    if (on) {
      const int at = hits + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(those >> 32),
                                                           __builtin_amdgcn_mbcnt_lo((uint32_t)those, 0));
      if (at < ROOM) {
        hit[wave * ROOM + at] = make_uint4(v[0], v[1], v[2], v[3]);
        hit_at[wave * ROOM + at] = i;
      }
    }
    hits += __popcll(those);
  };
  // the sums of a lane's 32 elements are float32, those of all of them float64
  VecSums part{0.0f, 0.0f};
  auto flush = [&] {
    sum += part.s;
    wsum += part.w;
    part = {0.0f, 0.0f};
  };
  auto late = [&](float m) { return m >= reach && m >= first; };
  // `there` is false for what a lane loaded past the last vector
  auto take = [&](V4 v, int i, bool there) {
    float f[N];
    Vec<E>::unpack(v, f);
    const float m = vec_max<N>(f);
    const VecSums before = part;
    part = add_sums<E>(v, exponent, part);
    const bool on = there && m >= reach;
    if (__any(on)) {
      list(v, i, on);
      mine = on ? max3(mine, m, m) : mine;
      if (on && m >= first) part = before;
    }
    if (!there) part = before;
  };
  // part.w of the vectors that were just taken, where one holds a logit of -inf
  auto bound = [&](const V4* v, auto count, auto taken) {
    if (part.w == part.w) return;
    part.w = 0.0f;
#pragma unroll
    for (int u = 0; u < count(); ++u) {
      V4 x = v[u];
      asm volatile("" : "+v"(x));  // unpacked anew: values kept from above would take registers from all
      float f[N];
      Vec<E>::unpack(x, f);
      if (taken(u) && !late(vec_max<N>(f))) part.w = bound_w<E>(x, exponent, part.w);
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) take(w[u], tid + u * THREADS, tid + u * THREADS < whole);
  bound(w, std::integral_constant<int, U>(), [&](int u) { return tid + u * THREADS < whole; });
  flush();
  if (whole < vecs && wave == WAVES - 1) {
    const V4 v = vec_at(p, whole, n);
    take(v, whole, part_of_one);
    bound(&v, std::integral_constant<int, 1>(), [&](int) { return part_of_one; });
    flush();
  }
  int base = U * THREADS;
  for (; base + B * THREADS <= whole; base += B * THREADS) {
#pragma unroll
    for (int u = 0; u < B; ++u) w[u] = a[u];
    if (base + 2 * B * THREADS <= whole) {  // an address of the whole workgroup
#pragma unroll
      for (int u = 0; u < B; ++u) a[u] = vload_nt(p + (int64_t)(base + (u + B) * THREADS) * N + tid * N);
    } else {
#pragma unroll
      for (int u = 0; u < B; ++u) a[u] = next(base + tid + (u + B) * THREADS);
    }
    sched_fence();
#pragma unroll
    for (int u = 0; u < B; ++u) take(w[u], base + tid + u * THREADS, true);
    bound(w, std::integral_constant<int, B>(), [](int) { return true; });
    flush();
  }
  if (base < whole) {
#pragma unroll
    for (int u = 0; u < B; ++u) take(a[u], base + tid + u * THREADS, base + tid + u * THREADS < whole);
    bound(a, std::integral_constant<int, B>(), [&](int u) { return base + tid + u * THREADS < whole; });
    flush();
  }

  // f(vector, its index, whether the lane has one) once more for the whole piece
  auto scan = [&](auto f) {
    for (int i = tid; i - tid < whole; i += B * THREADS) {
#pragma unroll
      for (int u = 0; u < B; ++u) w[u] = next(i + u * THREADS);
      sched_fence();
#pragma unroll
      for (int u = 0; u < B; ++u) f(w[u], i + u * THREADS, i + u * THREADS < whole);
    }
    if (whole < vecs && wave == WAVES - 1) f(vec_at(p, whole, n), whole, part_of_one);
  };
  auto all = [&](auto f) {
    scan([&](V4 v, int i, bool there) {
      float e[N];
      Vec<E>::unpack(v, e);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (there && i * N + j < n) f(e[j], lo + i * N + j);
    });
  };

  // The k largest, and the sums of the late vectors, relative to the wave's largest: of those a lane keeps the one with
  // its largest logit apart.
  const float most = lane_max(mine), ref = at_max(most);
  auto from_most = [&](float f) { return s.of(f - ref); };
  double late_sum, late_wsum;
  VecSums held;
  V4 held_v;
  float held_m;
  int held_at;
  bool listed, over = false;  // over: the late vectors are not all listed
  for (int turn = 0;; ++turn) {
    if (turn > 0) {
      // Too many, as in logits that rise along the row: anew, from the k-th of the lanes' largest in the whole piece
      // on; if that is a value that many have, from the next one on.
      __syncthreads();
      reach = turn == 1 ? kth_lane(mine) : value_of(order_of(reach) + 1);
      over = !(reach <= first);
      if (tid == 0) overflow = candidates = 0;
      __syncthreads();
      hits = 0;
      scan([&](V4 v, int i, bool there) {
        float f[N];
        Vec<E>::unpack(v, f);
        list(v, i, there && vec_max<N>(f) >= reach);
      });
    }
    late_sum = late_wsum = 0.0;
    held = {0.0f, 0.0f};
    held_m = -INFINITY;
    held_at = -1;
    if (hits > ROOM) {
      if (lane == 0) overflow = 1;
    } else {
      for (int i0 = 0; i0 < hits; i0 += 64) {
        const bool there = i0 + lane < hits;
        const uint4 h = hit[wave * ROOM + (there ? i0 + lane : 0)];
        const int at = hit_at[wave * ROOM + (there ? i0 + lane : 0)];
        const V4 v = {h.x, h.y, h.z, h.w};
        float e[N];
        Vec<E>::unpack(v, e);
        const float m = vec_max<N>(e);
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) bits |= there && e[j] >= reach && at * N + j < n ? 1u << j : 0u;
        if (there && m >= first) {
          VecSums t = vec_sums<E>(v, from_most);
          if (m > held_m || (m == held_m && at < held_at)) {
            const VecSums before = held;
            held = t;
            t = before;
            held_v = v;
            held_m = m;
            held_at = at;
          }
          late_sum += t.s;
          late_wsum += t.w;
        }
        int to = reserve(__popc(bits), &candidates);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (bits >> j & 1u) {
            if (to < FEW) candidate[to] = entry_of(e[j], lo + at * N + j);
            ++to;
          }
      }
    }
    __syncthreads();
    listed = overflow == 0;
    if (listed || turn == 2) break;
  }
  over = over || !listed;
  bool found = listed;
  if (listed) {
    if ((tid & 63) == 0) wave_hi[tid >> 6] = most;
    __syncthreads();
    if (candidates <= kDirect) {
      sort_list<THREADS>(candidate, candidates, kk, l.sorted);
      if (tid == 0) l.count = candidates;
      __syncthreads();
    } else {
      float m = most;
#pragma unroll
      for (int v = 0; v < WAVES; ++v) m = fmaxf(m, wave_hi[v]);
      auto each = [&](auto f) {
        if (candidates <= FEW) {
          for (int i = tid; i < candidates; i += THREADS)
            f(value_of(static_cast<uint32_t>(candidate[i] >> 32)), column_of(candidate[i]));
          return;
        }
        for (int i = lane; i < hits; i += 64) {
          const uint4 h = hit[wave * ROOM + i];
          const int at = hit_at[wave * ROOM + i];
          float e[N];
          Vec<E>::unpack(V4{h.x, h.y, h.z, h.w}, e);
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (e[j] >= reach && at * N + j < n) f(e[j], lo + at * N + j);
        }
      };
      found = select_top<THREADS>(each, m, reach > kFloor ? reach : low, kk, l);
    }
  }
  // Fewer than k from `reach` on, in order: what comes below, value by value (after a mask mostly one), the lowest
  // columns of a value first.
  int have = found ? l.count : 0;
  for (int turn = 0; found && have < kk; ++turn) {
    found = turn < 2;
    if (!found) break;
    float below = -INFINITY;
    bool some = false;
    all([&](float f, int) {
      if (!(f < reach)) return;
      below = fmaxf(below, f);
      some = true;
    });
    below = lane_max(below);
    __syncthreads();
    if ((tid & 63) == 0) wave_hi[tid >> 6] = below;
    if (!__syncthreads_or(some)) break;  // NaNs: the row has no probabilities
    for (int v = 0; v < WAVES; ++v) below = fmaxf(below, wave_hi[v]);
    reach = below;
    for (int i0 = 0; i0 < vecs && have < kk; i0 += THREADS) {
      float e[N];
      Vec<E>::unpack(vec_at(p, i0 + tid < vecs ? i0 + tid : vecs, n), e);
      int mine_too = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) mine_too += e[j] == below && (i0 + tid) * N + j < n;
      const int upto = lane_sums(mine_too);
      if ((tid & 63) == 63) wave_n[tid >> 6] = upto;
      __syncthreads();
      int at = have + upto - mine_too;
      for (int v = 0; v < WAVES; ++v) {
        at += v < (tid >> 6) ? wave_n[v] : 0;
        have += wave_n[v];
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int column = (i0 + tid) * N + j;
        if (e[j] == below && column < n && at < kk) l.sorted[at++] = entry_of(below, lo + column);
      }
      __syncthreads();
    }
  }
  if (!found) {
    select_exactly<THREADS>(all, kk, l);
    have = kk;
  }
  const int top = column_of(l.sorted[0]) - lo;
  const float m = n > 0 ? value_of(static_cast<uint32_t>(l.sorted[0] >> 32)) : -INFINITY;

  // the sums over all but the largest
  // below kFloor nothing was listed behind a beginning of -inf
  const bool again = m > -INFINITY && (over || m < kFloor || !(fabsf(shift) <= kFar));
  const LeftOut<E> without_top(top, vecs);
  auto from_m = [&](float f) { return s.of(f - m); };
  if (again) {
    sum = wsum = 0.0;
    scan([&](V4 v, int i, bool there) {
      without_top.template from<1>(&v, i, 1);
      const VecSums t = vec_sums<E>(v, from_m);
      sum += there ? t.s : 0.0;
      wsum += there ? t.w : 0.0;
    });
  } else {
    if (held_at >= 0 && held_at == top / N) {
      without_top.template from<1>(&held_v, held_at, 1);
      held = vec_sums<E>(held_v, from_most);
    }
    // Both to the largest logit: its exponent relative to the first elements' is d, where there are some above -inf
    // (all is late otherwise); the wave's, relative to it, is b, where there is a late vector. The first factor is
    // float64: it is all terms', so that its rounding would not average out (4096 x 128256, k = 64, 189 -> 191 us).
    const double d = first > -INFINITY ? (double)m * s.hi + ((double)m * s.lo + shift) : 0.0;
    const double by = exp2(-d);
    late_sum += held.s;
    late_wsum += held.w;
    const float b = late_sum == 0.0 ? 0.0f : s.of(ref - m), late_by = __builtin_amdgcn_exp2f(b);
    wsum = by == 0.0 ? 0.0 : (wsum - d * sum) * by;
    sum *= by;
    if (late_by > 0.0f) wsum += (late_wsum + b * late_sum) * late_by;
    sum += late_sum * late_by;
  }
  sum = lane_total(sum);
  wsum = lane_total(wsum);
  if ((tid & 63) == 0) {
    wave_s[tid >> 6] = sum;
    wave_w[tid >> 6] = wsum;
  }
  __syncthreads();
  if (tid == 0) {
    for (int v = 1; v < WAVES; ++v) {
      sum += wave_s[v];
      wsum += wave_w[v];
    }
    // with nothing above -inf the sum is 0 or NaN; m is NaN where nothing could be compared
    if (m > -INFINITY)
      shared = {m, sum, -wsum * kLn2};
    else
      shared = {m, m == -INFINITY ? sum : NAN, 0.0};
  }
  __syncthreads();
  TopStats v = shared;
  if (splits > 1) {
    const int64_t at = row * splits + sp;
    if (tid == 0) parts.stats[at] = {v.r, v.gap, v.m};
    if (tid < k) parts.entries[at * k + tid] = tid < have ? l.sorted[tid] : 0;
    return;
  }
  v.gap /= 1.0 + v.r;
  put_row(out, row, v, target, target ? Vec<E>::value(x[row * stride + y]) : 0.0f, l.sorted, have);
}

// The pieces of a row: their statistics by one wave, the k largest of their
// largest by the workgroup.
template <class E>
__global__ __launch_bounds__(256) void top_join_kernel(const E* __restrict__ x, int64_t stride,
                                                       const int32_t* __restrict__ targets, int V, int splits,
                                                       TopOut out, TopParts parts) {
  __shared__ Select l;
  __shared__ TopStats shared;
  __shared__ float shared_lo;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int y = targets != nullptr ? targets[row] : -1;
  const bool target = y >= 0 && y < V;
  if (targets != nullptr && !target) return put_masked(out, row);
  const int k = out.k < 1 ? 1 : out.k;
  const int kk = k < V ? k : V;
  const uint64_t* entries = parts.entries + row * splits * k;
  clear<256>(l);
  if (tid < 64) {
    const TopPiece* piece = parts.stats + row * splits + tid;
    const bool on = tid < splits;
    const TopStats v = on ? TopStats{piece->m, piece->r, piece->gap} : TopStats{-INFINITY, 0.0, 0.0};
    // what the piece's k-th largest reaches, k entries of the row do
    const uint64_t last = on ? entries[tid * k + k - 1] : 0;
    const float m = lane_max(v.m);
    const float lo = lane_max(last != 0 ? value_of(static_cast<uint32_t>(last >> 32)) : -INFINITY);
    const uint64_t top = __ballot(v.m == m);
    const bool holds = top != 0 && tid == __builtin_ctzll(top);  // the largest logit, whose 1 is not in r
    const double d = ((double)m - v.m) * out.inv_temperature;
    const double f = holds ? 1.0 : v.m > -INFINITY ? exp(-d) : 0.0;
    const double r = lane_total(holds ? v.r : f * (1.0 + v.r));
    const double gap = lane_total(f > 0.0 ? f * (v.gap + (holds ? 0.0 : d * (1.0 + v.r))) : 0.0);
    if (tid == 0) {
      shared = {m, r, gap / (1.0 + r)};
      shared_lo = lo;
    }
  }
  __syncthreads();
  const TopStats v = shared;
  auto each = [&](auto f) {
    const int n = splits * k;
    for (int i = tid; i < n; i += 4 * 256) {
      uint64_t e[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) e[u] = entries[i + u * 256 < n ? i + u * 256 : n - 1];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u * 256 < n && e[u] != 0) f(value_of(static_cast<uint32_t>(e[u] >> 32)), column_of(e[u]));
    }
  };
  if (out.k > 0 && !select_top<256>(each, v.m, shared_lo < kFloor ? kFloor : shared_lo, kk, l))
    select_exactly<256>(each, kk, l);
  put_row(out, row, v, target, target ? Vec<E>::value(x[row * stride + y]) : 0.0f, l.sorted, kk);
}

// ---------------------------------------------------------------------------
// gradient: with g = d loss / d logp and h = d loss / d entropy of the row,
//   dx_j = (g ([j = y] - p_j) - h p_j (log p_j + entropy)) / tau
// and log p_j + entropy = d_j + gap. A workgroup takes one piece of a row, a
// vector per lane, which writes memory fastest. Memory bounds it: 8192 x 128256
// bfloat16 with 2448 rows masked 591 us (1.48 GB read, 2.1 written: 6.05 TB/s),
// 2043 x 32003 float32 77 us.
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

// Workgroups of 4, 8 or (see very_few) 16 waves with room for so many vectors in their list.
struct TopShape {
  int waves, hits;
};
constexpr TopShape kShapes[] = {{4, 256}, {4, 1024}, {8, 1024}};

// Elements of a row in no particular order that list 5/8 of what there is room
// for: with G lanes the k-th largest of their first 32 elements each is reached
// by a share of -log(1 - k / G) / 32 of all. That varies by 1 / sqrt(k).
static int64_t most_elements(const TopShape& v, int k) {
  const double lanes = 64.0 * v.waves;
  return k >= lanes ? 0 : static_cast<int64_t>(v.hits * (5.0 / 8) * 32.0 / -std::log(1.0 - (k < 1 ? 1 : k) / lanes));
}

// The smallest shape that a piece's list fits; a long piece that lists more than
// 256 has room for takes 8 waves, which list half as many: 2048 x 128256
// bfloat16, k = 20, 97 us with 8 waves and 106 with 4; 8192 x 32000, k = 64, 168
// and 147.
static TopShape top_shape(int64_t piece, int k) {
  if (piece <= most_elements(kShapes[0], k)) return kShapes[0];
  return piece <= most_elements(kShapes[1], k) && piece <= 65536 ? kShapes[1] : kShapes[2];
}

// Whether 16 waves take each of very few rows whole: one launch in place of two,
// which the host's time decides (15 us a call, and 18 with the second launch);
// kernels of rows in pieces take about as long. us a call so and in pieces:
//   bfloat16   65536 columns: 1 row, k 20, 15.4 and 18.2; 16 rows, k 5, 15.3 and 18.0, k 128 17.9 and 18.9
//             100000: 1 row, k 5, 15.8 and 17.9, k 20 17.8 and 18.0, k 64 19.5 and 18.1; 16 rows, k 5, 17.9 and 17.9
//             128256: 1 row, k 5, 16.9 and 17.6, k 20 18.3 and 18.1, k 64 19.5 and 17.9; 16 rows, k 5, 18.1 and 18.0,
//             k 20 19.5 and 18.2
//             140000: 1 row, k 5, 18.5 and 17.8
//   float32    65536: 1 row, k 20, 15.3 and 18.5; 16 rows, k 128, 18.5 and 19.0
//             128256: 1 row, k 5, 17.3 and 18.1, k 20 18.7 and 18.4; 16 rows, k 5, 18.7 and 18.0
static bool very_few(int64_t T, int64_t V, int64_t k) {
  return T <= 16 && V > 49152 && V <= (k <= 8 ? 131072 : 65536);
}

// Pieces of a row: one, or of few long rows about as many as give 1024
// workgroups, of at least 8192 logits each; at most what a list has room for. us
// a call in one piece and in such pieces, bfloat16:
//   128256 columns: 128 rows, k = 20, 22.6 and 20.4; 256 rows 23.5 and 25.9
//   32000: 64 rows 14.8 and 16.1
static int64_t top_splits(int64_t T, int64_t V, int k) {
  if (very_few(T, V, k)) return 1;
  const int64_t least = ceil_div(V, most_elements(kShapes[2], k));
  int64_t splits = 1;
  if (V > 49152 && T < 192) {
    const int64_t rows = T < 1 ? 1 : T, most = ceil_div(V, 8192);
    splits = (1024 + rows / 2) / rows;
    splits = splits < most ? splits : most;
    splits = splits < kMaxSplits ? splits : kMaxSplits;
  }
  return splits > least ? splits : least > 1 ? least : 1;
}

struct TopPlan {
  int splits, piece;
  TopShape shape;
  bool fits;  // one launch
  TopParts parts;
  size_t bytes;
};

static TopPlan plan_top(int64_t T, int64_t V, int64_t k, void* ws) {
  TopPlan l{};
  const int64_t splits = top_splits(T, V, static_cast<int>(k));
  l.splits = static_cast<int>(splits);
  l.piece = static_cast<int>(round_up(ceil_div(V, l.splits), 8));
  l.shape = very_few(T, V, k) ? TopShape{16, 1024} : top_shape(l.piece, static_cast<int>(k));
  l.fits = splits <= kMaxSplits && T * splits <= max_blocks(64 * l.shape.waves);
  Carver w(ws);
  const int64_t pieces = l.splits > 1 ? T * l.splits : 0;
  l.parts.stats = static_cast<TopPiece*>(w.take(pieces * sizeof(TopPiece)));
  l.parts.entries = static_cast<uint64_t*>(w.take(pieces * (k < 1 ? 1 : k) * sizeof(uint64_t)));
  l.bytes = w.used > 0 ? w.used : 256;
  return l;
}

constexpr int64_t kMaxVocab = int64_t(1) << 22;  // 64 pieces hold it for any k

}  // namespace lora

using namespace lora;

extern "C" size_t lora_token_top_workspace_bytes(int64_t T, int64_t V, int64_t k) {
  if (T < 0 || V < 0 || k < 0 || T > kMaxRows || V > kMaxVocab || k > kMaxTop) return 0;
  const TopPlan l = plan_top(T, V, k, nullptr);
  return l.fits ? l.bytes : 0;
}

extern "C" int lora_token_top(const lora_mat* logits, const int32_t* targets, int64_t k, double temperature,
                              float* logp, float* entropy, int32_t* top_ids, float* top_logp, float* stats,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits) return LORA_ERR_NULL;
  if (int e = check_logits(logits)) return e;
  if (k < 0) return LORA_ERR_SHAPE;
  if (k > kMaxTop || logits->cols > kMaxVocab) return LORA_ERR_LIMIT;
  if (!temperature_ok(temperature)) return LORA_ERR_VALUE;
  const int64_t T = logits->rows, V = logits->cols;
  const TopPlan l = plan_top(T, V, k, workspace);
  if (!l.fits) return LORA_ERR_LIMIT;
  if (T == 0) return LORA_OK;
  if (!entropy || !stats || (V > 0 && !logits->ptr)) return LORA_ERR_NULL;
  if ((targets != nullptr) != (logp != nullptr) || (k > 0 && (!top_ids || !top_logp))) return LORA_ERR_NULL;
  if (!workspace || workspace_bytes < l.bytes || !aligned(workspace, 256)) return LORA_ERR_WORKSPACE;
  const TopOut out{logp, entropy, top_ids, top_logp, stats, static_cast<int>(k), 1.0 / temperature};
  auto st = static_cast<hipStream_t>(stream);
  by_type(logits, [&](auto* e) {
    using E = std::remove_pointer_t<decltype(e)>;
    auto* kernel = l.shape.hits == 256     ? top_kernel<E, 4, 256>
                   : l.shape.waves == 4  ? top_kernel<E, 4, 1024>
                   : l.shape.waves == 16 ? top_kernel<E, 16, 1024>
                                         : top_kernel<E, 8, 1024>;
    launch(kernel, dim3(T * l.splits), dim3(64 * l.shape.waves), 0, st, (const E*)logits->ptr, logits->stride_row,
           targets, static_cast<int>(V), l.splits, l.piece, exponent_of(temperature), out, l.parts);
    if (l.splits > 1)
      launch(top_join_kernel<E>, dim3(T), dim3(256), 0, st, (const E*)logits->ptr, logits->stride_row, targets,
             static_cast<int>(V), l.splits, out, l.parts);
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
