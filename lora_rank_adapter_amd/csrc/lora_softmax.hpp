// What the kernels on rows of logits share: an element left out of a row's
// vectors, workgroup sums, the pieces that gradients are written in, and the
// checks of logits and their gradients.
#pragma once

#include <cmath>
#include <type_traits>

#include "lora_host.hpp"
#include "lora_rows.hpp"

namespace lora {

__device__ __forceinline__ float at_max(float m) { return m == -INFINITY ? 0.0f : m; }

// Reductions over a wave in registers (DPP: four shifts within a row of 16
// lanes, then the last lane of a row, and of two rows, to the rows after it),
// which take a fraction of the time of shuffles through LDS. f(a, b) joins two
// values; `none` changes nothing. Lane i gets the lanes 0 to i joined.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_move(int none, int v) {
  return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xF, false);
}
template <class F>
__device__ __forceinline__ int lane_scan(int v, int none, F f) {
  v = f(v, dpp_move<0x111, 0xF>(none, v));
  v = f(v, dpp_move<0x112, 0xF>(none, v));
  v = f(v, dpp_move<0x114, 0xF>(none, v));
  v = f(v, dpp_move<0x118, 0xF>(none, v));
  v = f(v, dpp_move<0x142, 0xA>(none, v));
  return f(v, dpp_move<0x143, 0xC>(none, v));
}
__device__ __forceinline__ float lane_max(float v) {
  const int all = lane_scan(__float_as_int(v), __float_as_int(-INFINITY),
                            [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); });
  return __int_as_float(__builtin_amdgcn_readlane(all, 63));
}
__device__ __forceinline__ float lane_min(float v) { return -lane_max(-v); }
__device__ __forceinline__ int lane_sums(int v) {
  return lane_scan(v, 0, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ double lane_total(double v) {
  auto step = [&](auto ctrl, auto rows) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = dpp_move<ctrl(), rows()>(0, (int)u), hi = dpp_move<ctrl(), rows()>(0, (int)(u >> 32));
    v += __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
  };
  using std::integral_constant;
  const integral_constant<int, 0xF> every;
  step(integral_constant<int, 0x111>(), every);
  step(integral_constant<int, 0x112>(), every);
  step(integral_constant<int, 0x114>(), every);
  step(integral_constant<int, 0x118>(), every);
  step(integral_constant<int, 0x142>(), integral_constant<int, 0xA>());
  step(integral_constant<int, 0x143>(), integral_constant<int, 0xC>());
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = __builtin_amdgcn_readlane((int)u, 63), hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

// log2(e) / temperature as a float32 below it and the rest, which is above 0:
// the exponent of 2 of exp(d / temperature) is d hi + d lo, -inf for d = -inf.
struct Exponent {
  float hi, lo;
  __device__ __forceinline__ float of(float d) const { return fmaf(d, hi, d * lo); }
};
constexpr double kLn2 = 0.693147180559945309417;

// Element `at` of a row's piece (-1: it is elsewhere), which the sums leave
// out: -inf takes its place in the loaded vector that holds it.
template <class E>
struct LeftOut {
  static constexpr int N = Vec<E>::N;
  int vector;  // -1: none of the piece's vectors
  uint32_t keep[4], put[4];
  __device__ __forceinline__ LeftOut(int at, int vecs) {
    vector = at >= 0 && at < vecs * N ? at / N : -1;
    const int e = at & (N - 1), word = N == 8 ? e >> 1 : e;
    const uint32_t mask = N == 4 ? 0xFFFFFFFFu : e & 1 ? 0xFFFF0000u : 0x0000FFFFu;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      keep[k] = k == word ? ~mask : 0xFFFFFFFFu;
      put[k] = k == word ? mask & 0xFF80FF80u & (N == 4 ? 0xFFFF0000u : 0xFFFFFFFFu) : 0u;
    }
  }
  // U vectors that are `step` (a power of two) apart, from vector i on
  template <int U>
  __device__ __forceinline__ void from(typename Vec<E>::type* w, int i, int step) const {
    const int d = vector - i;
    if ((d & ~((U - 1) * step)) != 0) return;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (d == u * step) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[u][k] = (w[u][k] & keep[k]) | put[k];
      }
  }
};

// The sum of v over the workgroup's waves, in their order.
template <int WAVES = 16>
__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < WAVES; ++w) total += lds[w];
  __syncthreads();
  return total;
}

// Columns of a gradient that one workgroup writes: a vector per lane.
constexpr int kGradVecs = 256;

template <class E>
struct GradArgs {
  const E* x;
  int64_t stride;
  E* dx;  // may be x: a vector is stored by the lane that loaded it
  int64_t dx_stride;
  int V, pieces;
};

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxBlocks = max_blocks(256);
constexpr int64_t kMaxRows = kMaxBlocks;  // of logits: a workgroup at least for each

inline int check_logits(const lora_mat* m) {
  if (!float_dtype_ok(m->dtype)) return LORA_ERR_DTYPE;
  if (!valid_dims(m)) return LORA_ERR_SHAPE;
  if (m->cols > 1 && m->stride_col != 1) return LORA_ERR_STRIDE;
  if (m->rows > 1 && m->stride_row < m->cols) return LORA_ERR_STRIDE;
  if (!aligned(m->ptr, elem_size(m->dtype))) return LORA_ERR_STRIDE;
  if (m->rows > kMaxRows || m->cols > 0x7FFFFFFF - 8 * kGradVecs) return LORA_ERR_LIMIT;
  return LORA_OK;
}

inline bool temperature_ok(double t) { return t >= 1e-6 && t <= 1e6; }
inline Exponent exponent_of(double temperature) {
  const double scale = 1.4426950408889634074 / temperature;
  float hi = static_cast<float>(scale);
  if (static_cast<double>(hi) >= scale) hi = std::nextafterf(hi, 0.0f);
  return {hi, static_cast<float>(scale - static_cast<double>(hi))};
}

// f with a null pointer of the logits' element type
template <class F>
void by_type(const lora_mat* x, F f) {
  if (x->dtype == LORA_F32)
    f(static_cast<float*>(nullptr));
  else
    f(static_cast<uint16_t*>(nullptr));
}

// Whether two matrices of one shape and type, with rows of consecutive
// elements, are the same memory throughout, or have none in common.
inline bool same_or_apart(const lora_mat* x, const lora_mat* dx) {
  if (x->rows == 0 || x->cols == 0) return true;
  const int64_t es = static_cast<int64_t>(elem_size(x->dtype)), width = x->cols * es;
  const int64_t a = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x->ptr));
  const int64_t b = static_cast<int64_t>(reinterpret_cast<uintptr_t>(dx->ptr));
  const bool pitch = x->rows == 1 || x->stride_row == dx->stride_row;
  if (a == b && pitch) return true;
  const int64_t a_end = a + (x->rows - 1) * x->stride_row * es + width;
  const int64_t b_end = b + (x->rows - 1) * dx->stride_row * es + width;
  if (b >= a_end || a >= b_end) return true;
  if (x->rows == 1 || !pitch) return false;
  // columns of the same rows: each begins where the other has ended
  const int64_t step = x->stride_row * es, shift = ((b - a) % step + step) % step;
  return shift >= width && step - shift >= width;
}

inline int check_dlogits(const lora_mat* x, const lora_mat* dx) {
  if (dx->rows != x->rows || dx->cols != x->cols) return LORA_ERR_SHAPE;
  if (dx->dtype != x->dtype) return LORA_ERR_DTYPE;
  if (int e = check_logits(dx)) return e;
  if (!same_or_apart(x, dx)) return LORA_ERR_STRIDE;
  const int64_t pieces = ceil_div(x->cols, int64_t(kGradVecs) * vec_elems(x->dtype));
  // One more sums a policy loss. This covers rows that a workgroup of 8 or 16 waves takes: they have 11 pieces or more.
  return x->rows * pieces >= kMaxBlocks ? LORA_ERR_LIMIT : LORA_OK;
}

template <class E>
GradArgs<E> grad_args(const lora_mat* x, const lora_mat* dx) {
  const int64_t pieces = ceil_div(x->cols, int64_t(kGradVecs) * Vec<E>::N);
  return {static_cast<const E*>(x->ptr), x->stride_row,          static_cast<E*>(dx->ptr),
          dx->stride_row,                static_cast<int>(x->cols), static_cast<int>(pieces)};
}

}  // namespace lora
