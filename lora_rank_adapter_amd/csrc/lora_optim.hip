// AdamW over many tensors in one launch.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Everything is read and written once: the step is bound by HBM. The tensors
// are described by a table in device memory (their pointers, and for every
// chunk of kChunk elements the tensor it belongs to), so that one grid covers
// all of them whatever their sizes. The states of all tensors are one flat
// array each; a tensor's states start at a multiple of 256 elements.
//
// 8-bit states: 256 elements share a float32 scale, the block's largest
// magnitude over 448, and each element is an e4m3 code (4 significant bits
// over 17 binades). The second moment is stored as its square root, which
// halves its range in binades, and an element above zero never gets the code
// of zero: the step divides by it, and a zero would leave eps alone there.
//
// Kernels:
//   table_kernel   table entries and the chunks' tensors
//   begin_kernel   the step count and the constants that depend on it
//   step_kernel    the update, 256 elements per wave at a time
//   small_step_kernel  constants and update of a few chunks, one workgroup

#include <cmath>

#include "lora_host.hpp"
#include "lora_rows.hpp"

namespace lora {

constexpr int kStateBlock = 256;  // elements that share a scale; one wave's step
constexpr int kChunk = 1024;      // elements of one workgroup, a block for each of its waves
constexpr int kTableBatch = 48;   // entries passed to one table_kernel launch
constexpr int64_t kTableMagic = 0x4164616D57303146;

struct TableHead {
  int64_t magic, elems, tensors, chunks;
  // written by begin_kernel for each step
  float lr, alpha, inv_root, decay;
};
struct TableEntry {
  void* param;
  const void* grad;
  uint16_t* shadow;
  int64_t numel, state;  // elements, first element of its states
  int32_t first_chunk;
  uint8_t param_bf16, grad_bf16, vec, unused;
};
constexpr int64_t kHeadBytes = 256;

struct TableBatch {
  TableEntry e[kTableBatch];
};

__device__ __forceinline__ TableEntry* table_entries(void* table) {
  return reinterpret_cast<TableEntry*>(static_cast<char*>(table) + kHeadBytes);
}
__host__ __device__ inline int64_t chunk_map_offset(int64_t n) {
  return kHeadBytes + (n * (int64_t)sizeof(TableEntry) + 255) / 256 * 256;
}

__global__ __launch_bounds__(256) void table_kernel(TableBatch batch, int first, int64_t n, int64_t elems,
                                                    int64_t chunks, void* __restrict__ table) {
  const TableEntry e = batch.e[blockIdx.x];
  if (threadIdx.x == 0) {
    table_entries(table)[first + blockIdx.x] = e;
    if (first + blockIdx.x == 0) {
      auto* h = static_cast<TableHead*>(table);
      h->magic = kTableMagic;
      h->elems = elems;
      h->tensors = n;
      h->chunks = chunks;
    }
  }
  auto* map = reinterpret_cast<int32_t*>(static_cast<char*>(table) + chunk_map_offset(n));
  const int64_t own = (e.numel + kChunk - 1) / kChunk;
  for (int64_t i = threadIdx.x; i < own; i += 256) map[e.first_chunk + i] = first + (int)blockIdx.x;
}

// The constants need powers in float64; one thread computes them once.
struct BeginArgs {
  int32_t* step;
  double lr, beta1, beta2, decay;
  const float* lr_scale;
};
__device__ __forceinline__ void begin(const BeginArgs& a, TableHead* h) {
  const int t = *a.step + 1;
  *a.step = t;
  const double lr = a.lr_scale != nullptr ? a.lr * (double)*a.lr_scale : a.lr;
  h->alpha = static_cast<float>(lr / (1.0 - pow(a.beta1, (double)t)));
  h->inv_root = static_cast<float>(1.0 / sqrt(1.0 - pow(a.beta2, (double)t)));
  h->decay = static_cast<float>(1.0 - lr * a.decay);
}
__global__ void begin_kernel(void* table, BeginArgs a) { begin(a, static_cast<TableHead*>(table)); }

struct StepArgs {
  void *m, *v;
  float *m_scale, *v_scale;
  const float* grad_scale;
  float b1, c1, b2, c2, eps;  // c = 1 - b, rounded from float64
};

struct StepConst {
  float alpha, inv_root, decay, gs;
};

// Roots and quotients rounded correctly: the approximate instruction's result
// and Newton steps on its residual, which a fused product gives exactly (the
// root checked for every float32 mantissa and both parities of the exponent,
// the quotients for 5 10^7 pairs). Fewer instructions than the compiler's own
// sequences, which count in the 8-bit form: 75.5 M elements take 227 us, 240
// with those, 228 with the approximate results alone. 18.9 M with 32-bit
// states take 97 us in all three.

__device__ __forceinline__ float ordinary_root(float x) {
  const float y = __builtin_amdgcn_rsqf(x), g = x * y;
  return fmaf(fmaf(-g, g, x), 0.5f * y, g);
}
// Below 2^-96 the root is taken of v * 2^64, so that a denormal v keeps its
// root. Zeros, infinities and NaN go through.
__device__ __forceinline__ float any_root(float v) {
  const bool small = v < 0x1p-96f;
  const float r = ordinary_root(small ? v * 0x1p64f : v);
  constexpr int kPositive = 0x180;  // normal or denormal
  return __builtin_amdgcn_classf(v, kPositive) ? (small ? r * 0x1p-32f : r) : v;
}
// Four of each lane; most waves have ordinary values alone (the 8-bit form
// with any_root for all 230 us).
__device__ __forceinline__ void roots(const float* v, float* w) {
  const float low = fminf(fminf(v[0], v[1]), fminf(v[2], v[3]));
  const float high = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
  if (__ballot(!(low >= 0x1p-96f && high < INFINITY)) == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = ordinary_root(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = any_root(v[j]);
  }
}
// b is no denormal (eps, or the root of a v above zero); a denormal quotient
// may be off by one step.
__device__ __forceinline__ float quotient(float a, float b) {
  float y = __builtin_amdgcn_rcpf(b);
  y = fmaf(fmaf(-b, y, 1.0f), y, y);
  const float q = a * y;
  return __builtin_amdgcn_div_fixupf(fmaf(fmaf(-b, q, a), y, q), b, a);
}
__device__ __forceinline__ float over_448(float a) {
  constexpr float y = 1.0f / 448.0f;
  const float q = a * y;
  return __builtin_amdgcn_div_fixupf(fmaf(fmaf(-448.0f, q, a), y, q), 448.0f, a);
}

// Four elements; w receives the roots of the new v.
__device__ __forceinline__ void adamw(float* p, float* m, float* v, const float* g, const StepConst& k,
                                      const StepArgs& a, float* w) {
  // the fused products are written out: a tensor's steps are the same bits in either kernel
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float s = g[j] * k.gs;
    m[j] = fmaf(a.b1, m[j], a.c1 * s);
    v[j] = fmaf(a.b2, v[j], a.c2 * (s * s));
  }
  roots(v, w);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    p[j] = fmaf(p[j], k.decay, -quotient(k.alpha * m[j], fmaf(w[j], k.inv_root, a.eps)));
}

// four codes of one word as values, and back (rounded to nearest even)
__device__ __forceinline__ void fp8_values(uint32_t w, float scale, float* f) {
  f[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * scale;
  f[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * scale;
  f[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * scale;
  f[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * scale;
}
__device__ __forceinline__ uint32_t fp8_codes(const float* f) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true));
}

// The largest of the wave's values: rotations within each row of 16 lanes,
// then the rows' four results.
template <int D>
__device__ __forceinline__ float rotate_max(float v) {
  const int r = __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + D, 0xF, 0xF, false);
  return fmaxf(v, __int_as_float(r));
}
__device__ __forceinline__ float wave_max(float v) {
  const int m = __float_as_int(rotate_max<1>(rotate_max<2>(rotate_max<4>(rotate_max<8>(v)))));
  auto row = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(m, lane)); };
  return fmaxf(fmaxf(row(0), row(16)), fmaxf(row(32), row(48)));
}

// x: 4 values of each lane, one block over the wave. Returns the codes.
__device__ __forceinline__ uint32_t quantise(float* x, bool positive, float* scale) {
  const float amax = wave_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
  // a block below 1e-30 is stored as zeros (448 / amax stays finite above it)
  const bool some = amax >= 1e-30f;
  const float inv = some ? 448.0f / amax : 0.0f;
  *scale = some ? over_448(amax) : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = x[i] * inv;
    x[i] = positive && q > 0.0f ? fmaxf(q, 0.001953125f) : q;
  }
  return fp8_codes(x);
}

// Four elements; NT: non-temporal. Stores always are.
template <bool NT>
__device__ __forceinline__ void load4(const void* p, bool bf16, int64_t i, bool vec, int count, float* f) {
  if (vec && count == 4) {
    f32x4_t v;
    if (bf16) {
      auto* q = reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + i);
      v = Out<uint16_t>::unpack(__builtin_bit_cast(uint2, NT ? __builtin_nontemporal_load(q) : *q));
    } else {
      auto* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
      v = NT ? __builtin_nontemporal_load(q) : *q;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = e < count ? (bf16 ? bf16_value(static_cast<const uint16_t*>(p)[i + e])
                               : static_cast<const float*>(p)[i + e])
                       : 0.0f;
  }
}
__device__ __forceinline__ void store4(void* p, bool bf16, int64_t i, bool vec, int count, const float* f) {
  if (vec && count == 4) {
    const f32x4_t v = {f[0], f[1], f[2], f[3]};
    if (bf16)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x2_t, Out<uint16_t>::pack(v)),
                                  reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p) + i));
    else
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= count) continue;
      if (bf16)
        static_cast<uint16_t*>(p)[i + e] = static_cast<uint16_t>(bf16_bits(f[e]));
      else
        static_cast<float*>(p)[i + e] = f[e];
    }
  }
}

// One wave updates a block of 256 elements of a tensor, 4 per lane: what it
// loads, and the update from there. On tensors that the caches do not hold,
// 18.9 M elements with 32-bit states take 97 us with every access
// non-temporal (99 when 110 were measured with the loads or the stores alone
// and 112 with neither); 75.5 M with 8-bit states 227 us with all but the
// loads of param and grad (229 when it was 237 with those as well and 244 with
// neither stores nor loads of the floats).
template <int BITS>
struct Block {
  static constexpr bool kNt = BITS == 32;
  int64_t i, s;  // the lane's first element, in the tensor and in the states
  int count;     // its elements inside the tensor
  float p[4], g[4], m[4], v[4];
  uint32_t m_code, v_code;
  float m_scale, v_scale;

  __device__ __forceinline__ void load(const TableEntry& e, const StepArgs& a, int64_t block, int lane) {
    i = block + lane * 4;
    s = e.state + i;
    count = e.numel - i < 4 ? (e.numel - i < 0 ? 0 : (int)(e.numel - i)) : 4;
    load4<kNt>(e.param, e.param_bf16, i, e.vec, count, p);
    load4<kNt>(e.grad, e.grad_bf16, i, e.vec, count, g);
    if constexpr (BITS == 8) {
      m_code = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + s));
      v_code = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + s));
      m_scale = a.m_scale[s / kStateBlock];
      v_scale = a.v_scale[s / kStateBlock];
    } else {
      load4<kNt>(a.m, false, s, true, 4, m);
      load4<kNt>(a.v, false, s, true, 4, v);
    }
  }

  __device__ __forceinline__ void update(const TableEntry& e, const StepConst& k, const StepArgs& a, int lane) {
    if constexpr (BITS == 8) {
      fp8_values(m_code, m_scale, m);
      fp8_values(v_code, v_scale, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= v[j];
    }
    float w[4];
    adamw(p, m, v, g, k, a, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BITS == 8) v[j] = w[j];
      // past the tensor's end the states stay zero
      if (j >= count) m[j] = v[j] = 0.0f;
    }
    store4(e.param, e.param_bf16, i, e.vec, count, p);
    if (e.shadow != nullptr) store4(e.shadow, true, i, e.vec, count, p);
    if constexpr (BITS == 8) {
      m_code = quantise(m, false, &m_scale);
      v_code = quantise(v, true, &v_scale);
      __builtin_nontemporal_store(m_code, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + s));
      __builtin_nontemporal_store(v_code, reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + s));
      if (lane == 0) {
        a.m_scale[s / kStateBlock] = m_scale;
        a.v_scale[s / kStateBlock] = v_scale;
      }
    } else {
      store4(a.m, false, s, true, 4, m);
      store4(a.v, false, s, true, 4, v);
    }
  }
};

// A table of other tensors than the states: leave everything as it is.
__device__ __forceinline__ bool foreign(const TableHead* h, int64_t n, int64_t elems) {
  return h->magic != kTableMagic || h->tensors != n || h->elems != elems;
}
__device__ __forceinline__ const int32_t* chunk_map(const void* table, int64_t n) {
  return reinterpret_cast<const int32_t*>(static_cast<const char*>(table) + chunk_map_offset(n));
}

// One block to a wave: 75.5 M elements with 8-bit states take 227 us so (244
// when 265 were measured with two blocks to a wave and 274 with four).
template <int BITS>
__global__ __launch_bounds__(256) void step_kernel(void* table, int64_t n, int64_t elems, StepArgs a) {
  const auto* h = static_cast<const TableHead*>(table);
  if (foreign(h, n, elems) || blockIdx.x >= h->chunks) return;
  const TableEntry e = table_entries(table)[chunk_map(table, n)[blockIdx.x]];
  const StepConst k = {h->alpha, h->inv_root, h->decay, a.grad_scale != nullptr ? *a.grad_scale : 1.0f};
  const int64_t block = (int64_t)(blockIdx.x - e.first_chunk) * kChunk + wave_id() * kStateBlock;
  if (block >= e.numel) return;
  const int lane = threadIdx.x & 63;
  Block<BITS> x;
  x.load(e, a, block, lane);
  x.update(e, k, a, lane);
}

// A few chunks in one workgroup, which computes the constants itself: one
// launch instead of two. Two adapter weights of 4096 elements: 6.2 us a step
// against 8.8; beyond kSmall chunks one CU is too slow for the data.
constexpr int kSmall = 16;

template <int BITS>
__global__ __launch_bounds__(1024) void small_step_kernel(void* table, int64_t n, int64_t elems, BeginArgs b,
                                                          StepArgs a) {
  __shared__ TableHead now;
  if (threadIdx.x == 0) begin(b, &now);
  __syncthreads();
  const auto* h = static_cast<const TableHead*>(table);
  if (foreign(h, n, elems)) return;
  const StepConst k = {now.alpha, now.inv_root, now.decay, a.grad_scale != nullptr ? *a.grad_scale : 1.0f};
  constexpr int kBlocks = kChunk / kStateBlock;  // of a chunk
  for (int64_t u = wave_id(); u < h->chunks * kBlocks; u += 16) {
    const int64_t c = u / kBlocks;
    const TableEntry e = table_entries(table)[chunk_map(table, n)[c]];
    const int64_t block = (c - e.first_chunk) * kChunk + (u % kBlocks) * kStateBlock;
    if (block >= e.numel) continue;
    Block<BITS> x;
    x.load(e, a, block, threadIdx.x & 63);
    x.update(e, k, a, threadIdx.x & 63);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct TableSize {
  int64_t elems, chunks;
  size_t bytes;
};

static int measure(const lora_adamw_tensor* t, int64_t n, TableSize* size) {
  if (n < 0) return LORA_ERR_SHAPE;
  if (n > 0x7FFFFF) return LORA_ERR_LIMIT;
  if (n > 0 && !t) return LORA_ERR_NULL;
  *size = {};
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].numel < 0 || t[i].numel > kMaxOperand / 4) return LORA_ERR_SHAPE;
    size->elems += round_up(t[i].numel, kStateBlock);
    size->chunks += ceil_div(t[i].numel, kChunk);
    if (size->elems > kMaxOperand / 4) return LORA_ERR_SHAPE;
    if (size->chunks > max_blocks(256)) return LORA_ERR_LIMIT;
  }
  size->bytes = static_cast<size_t>(chunk_map_offset(n) + round_up(4 * size->chunks, 256));
  return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" size_t lora_adamw_table_bytes(const lora_adamw_tensor* tensors, int64_t n) {
  TableSize size;
  return measure(tensors, n, &size) == LORA_OK ? size.bytes : 0;
}

extern "C" int64_t lora_adamw_state_elems(const lora_adamw_tensor* tensors, int64_t n) {
  TableSize size;
  return measure(tensors, n, &size) == LORA_OK ? size.elems : 0;
}

extern "C" int lora_adamw_table(const lora_adamw_tensor* tensors, int64_t n, void* table, size_t table_bytes,
                                void* stream) {
  TableSize size;
  if (int e = measure(tensors, n, &size)) return e;
  for (int64_t i = 0; i < n; ++i) {
    const lora_adamw_tensor& t = tensors[i];
    if (!float_dtype_ok(t.param_dtype) || !float_dtype_ok(t.grad_dtype)) return LORA_ERR_DTYPE;
    if (t.shadow && t.param_dtype != LORA_F32) return LORA_ERR_DTYPE;
    if (t.numel > 0 && (!t.param || !t.grad)) return LORA_ERR_NULL;
    if (!aligned(t.param, elem_size(t.param_dtype)) || !aligned(t.grad, elem_size(t.grad_dtype)) ||
        !aligned(t.shadow, 2))
      return LORA_ERR_STRIDE;
  }
  if (size.elems == 0) return LORA_OK;
  if (!table || table_bytes < size.bytes || !aligned(table, 256)) return LORA_ERR_WORKSPACE;
  int64_t state = 0, chunk = 0;
  for (int64_t first = 0; first < n; first += kTableBatch) {
    TableBatch batch = {};
    const int count = static_cast<int>(n - first < kTableBatch ? n - first : kTableBatch);
    for (int i = 0; i < count; ++i) {
      const lora_adamw_tensor& t = tensors[first + i];
      // 4 elements of each operand in one access
      const bool vec = aligned(t.param, 4 * elem_size(t.param_dtype)) && aligned(t.grad, 4 * elem_size(t.grad_dtype)) &&
                       aligned(t.shadow, 8);
      batch.e[i] = {t.param,  t.grad, static_cast<uint16_t*>(t.shadow), t.numel, state, static_cast<int32_t>(chunk),
                    static_cast<uint8_t>(t.param_dtype == LORA_BF16), static_cast<uint8_t>(t.grad_dtype == LORA_BF16),
                    static_cast<uint8_t>(vec), 0};
      state += round_up(t.numel, kStateBlock);
      chunk += ceil_div(t.numel, kChunk);
    }
    launch(table_kernel, dim3(count), dim3(256), 0, static_cast<hipStream_t>(stream), batch, static_cast<int>(first),
           n, size.elems, size.chunks, table);
  }
  return launch_status();
}

extern "C" int lora_adamw_step(const lora_adamw_tensor* tensors, int64_t n, void* table, size_t table_bytes,
                               const lora_adamw_state* state, const lora_adamw_hyper* hyper, void* stream) {
  TableSize size;
  if (int e = measure(tensors, n, &size)) return e;
  if (!state || !hyper) return LORA_ERR_NULL;
  if (state->bits != 8 && state->bits != 32) return LORA_ERR_DTYPE;
  if (!state->step) return LORA_ERR_NULL;
  auto fraction = [](double b) { return b >= 0.0 && b < 1.0; };
  if (!std::isfinite(hyper->lr) || !std::isfinite(hyper->weight_decay) || !fraction(hyper->beta1) ||
      !fraction(hyper->beta2) || !(hyper->eps >= 0.0))
    return LORA_ERR_VALUE;
  if (size.elems > 0) {
    if (!state->m || !state->v || (state->bits == 8 && (!state->m_scale || !state->v_scale))) return LORA_ERR_NULL;
    if (!aligned(state->m, 16) || !aligned(state->v, 16)) return LORA_ERR_STRIDE;
    if (!table || table_bytes < size.bytes || !aligned(table, 256)) return LORA_ERR_WORKSPACE;
  }
  if (size.elems == 0) return LORA_OK;
  const StepArgs a = {state->m, state->v, state->m_scale, state->v_scale, hyper->grad_scale,
                      static_cast<float>(hyper->beta1), static_cast<float>(1.0 - hyper->beta1),
                      static_cast<float>(hyper->beta2), static_cast<float>(1.0 - hyper->beta2),
                      static_cast<float>(hyper->eps)};
  auto st = static_cast<hipStream_t>(stream);
  const BeginArgs b = {state->step, hyper->lr, hyper->beta1, hyper->beta2, hyper->weight_decay, hyper->lr_scale};
  if (size.chunks <= kSmall) {
    launch(state->bits == 8 ? small_step_kernel<8> : small_step_kernel<32>, dim3(1), dim3(1024), 0, st, table, n,
           size.elems, b, a);
    return launch_status();
  }
  launch(begin_kernel, dim3(1), dim3(1), 0, st, table, b);
  launch(state->bits == 8 ? step_kernel<8> : step_kernel<32>, dim3(size.chunks), dim3(256), 0, st, table, n, size.elems,
         a);
  return launch_status();
}
