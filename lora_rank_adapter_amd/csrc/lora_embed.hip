// Embedding lookup with scaling and its gradient.
//
//   out[t] = scale * table[ids[t]]             (zeros for an id outside [0, V))
//   dtable[v] = scale * sum of dy[t] over the tokens t with ids[t] = v
//
// Both move rows and compute next to nothing: they are bound by HBM.
//
// The gradient sums in a fixed order, without float atomics: sort_kernel
// orders the tokens by id (stable) and gives every id its range of the sorted
// list; grad_kernel cuts the list into runs of a fixed length, so that an id
// that fills the batch costs no more than others, and sums each id's tokens
// inside a run; merge_kernel adds the pieces of the ids that span runs.
//
// Kernels:
//   embed_kernel   rows gathered, scaled and stored, 8 elements per lane
//   sort_kernel    stable counting sort of the tokens by id, one launch
//   grad_kernel    sums of each run's ids, zeros of the rows without tokens
//   merge_kernel   pieces of an id added in the order of their runs

#include "lora_host.hpp"
#include "lora_rows.hpp"

namespace lora {

constexpr int kItem = 8;  // elements of a row that one lane handles at a time

template <class E, class O>
__global__ __launch_bounds__(256) void embed_kernel(const int32_t* __restrict__ ids, int64_t T,
                                                    const E* __restrict__ table, int64_t table_stride, int64_t V,
                                                    int64_t D, float scale, O* __restrict__ out, int64_t out_stride,
                                                    int lanes_log2, int items) {
  const int lanes = 1 << lanes_log2;
  const int64_t t = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
  if (t >= T) return;
  const int64_t id = ids[t];
  const bool live = id >= 0 && id < V;
  const E* src = table + (live ? id : 0) * table_stride;
  O* dst = out + t * out_stride;
  int64_t c = ((int64_t)blockIdx.y * items * lanes + (threadIdx.x & (lanes - 1))) * kItem;
  for (int i = 0; i < items; ++i, c += (int64_t)lanes * kItem) {
    if (c + kItem <= D) {
      float f[kItem] = {};
      if (live) load_row<kItem>(src + c, f);
#pragma unroll
      for (int e = 0; e < kItem; ++e) f[e] = live ? f[e] * scale : 0.0f;
      store_row<kItem>(dst + c, f);
    } else {
      for (int64_t e = c; e < D; ++e) dst[e] = Vec<O>::round(live ? Vec<E>::value(src[e]) * scale : 0.0f);
    }
  }
}

// ---------------------------------------------------------------------------
// sort: workgroup b owns the ids [b * bins, (b + 1) * bins) and reads every
// token's id. Wave w takes the w-th part of the tokens and counts its own
// histogram, so that after a scan over (id, wave) each wave knows where its
// tokens of each id go; the second pass places them, a token's rank among the
// equal ids of its 64 found by ballots over the id's bits. The workgroup also
// counts the tokens below its ids, so nothing passes between workgroups.
// ---------------------------------------------------------------------------
constexpr int kBins = 512;
constexpr int kSortWaves = 16;

__global__ __launch_bounds__(1024) void sort_kernel(const int32_t* __restrict__ ids, int T, int V, int bins,
                                                    int32_t* __restrict__ order, int32_t* __restrict__ keys,
                                                    int32_t* __restrict__ start) {
  __shared__ int hist[kSortWaves][kBins];
  __shared__ int below[kSortWaves];
  __shared__ int scan[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int lo = blockIdx.x * bins;
  const int n = V - lo < bins ? V - lo : bins;  // this workgroup's ids
  for (int i = tid; i < kSortWaves * kBins; i += 1024) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int part = (int)((((int64_t)T + kSortWaves - 1) / kSortWaves + 63) / 64 * 64);
  const int64_t first = (int64_t)wave * part;
  const int begin = (int)(first < T ? first : T);
  const int end = T - begin < part ? T : begin + part;

  int less = 0;
  for (int t = begin; t < end; t += 64) {
    const int id = t + lane < end ? ids[t + lane] : -1;
    less += __popcll(__ballot(id >= 0 && id < lo));
    if (id >= lo && id - lo < n) atomicAdd(&hist[wave][id - lo], 1);
  }
  if (lane == 0) below[wave] = less;
  __syncthreads();

  // exclusive positions: over the waves of an id, then over the ids
  int base = 0;
  for (int w = 0; w < kSortWaves; ++w) base += below[w];
  int total = 0;
  if (tid < kBins) {
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = hist[w][tid];
      hist[w][tid] = total;
      total += c;
    }
  }
  int incl = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  if (lane == 63) scan[wave] = incl;
  __syncthreads();
  for (int w = 0; w < wave; ++w) base += scan[w];
  const int at = base + incl - total;
  if (tid < kBins) {
    for (int w = 0; w < kSortWaves; ++w) hist[w][tid] += at;
    if (tid < n) start[lo + tid] = at;
    if (tid == n - 1 && lo + n == V) start[V] = at + total;
  }
  __syncthreads();

  for (int t = begin; t < end; t += 64) {
    const int id = t + lane < end ? ids[t + lane] : -1;
    const bool mine = id >= lo && id - lo < n;
    const uint64_t live = __ballot(mine);
    if (live == 0) continue;
    const int bin = mine ? id - lo : 0;
    uint64_t same = live;
#pragma unroll
    for (int b = 0; b < 9; ++b) {
      const uint64_t bit = __ballot((bin >> b) & 1);
      same &= (bin >> b) & 1 ? bit : ~bit;
    }
    const int head = __ffsll((unsigned long long)same) - 1;
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int pos = 0;
    if (mine && rank == 0) pos = atomicAdd(&hist[wave][bin], __popcll(same));
    pos = __shfl(pos, mine ? head : 0, 64) + rank;
    if (mine) {
      order[pos] = t + lane;
      keys[pos] = id;
    }
  }
}

// ---------------------------------------------------------------------------
// sums: a group of 2^lanes_log2 lanes takes one run of kRun sorted tokens and
// one piece of the columns. An id whose tokens all lie in the run is written
// at once; one that began before the run leaves its sum in part[run][0], one
// that goes on after it in part[run][1].
// ---------------------------------------------------------------------------
constexpr int kRun = 16;

template <class O>
__device__ __forceinline__ void put_row(O* p, const float* f, int count, bool add) {
  if (count == kItem) {
    float g[kItem];
#pragma unroll
    for (int e = 0; e < kItem; ++e) g[e] = f[e];
    if (add) {
      float old[kItem];
      load_row<kItem>(p, old);
#pragma unroll
      for (int e = 0; e < kItem; ++e) g[e] += old[e];
    }
    store_row<kItem>(p, g);
  } else {
    for (int e = 0; e < kItem; ++e)
      if (e < count) p[e] = Vec<O>::round(add ? Vec<O>::value(p[e]) + f[e] : f[e]);
  }
}

template <class E, class O>
__global__ __launch_bounds__(256) void grad_kernel(const int32_t* __restrict__ order, const int32_t* __restrict__ keys,
                                                   const int32_t* __restrict__ start, int64_t V, int64_t D,
                                                   const E* __restrict__ dy, int64_t dy_stride, float scale,
                                                   O* __restrict__ out, int64_t out_stride, bool add,
                                                   float* __restrict__ part, int64_t part_stride, int lanes_log2,
                                                   int pieces, int64_t run_blocks) {
  const int lanes = 1 << lanes_log2;
  const int n = start[V];
  if ((int64_t)blockIdx.x >= run_blocks) {
    // zeros of the rows that no token names
    const int64_t row = ((int64_t)blockIdx.x - run_blocks) * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    if (row >= V || start[row] != start[row + 1]) return;
    const float zero[kItem] = {};
    for (int64_t c = (int64_t)(threadIdx.x & (lanes - 1)) * kItem; c < D; c += (int64_t)lanes * kItem)
      put_row(out + row * out_stride + c, zero, D - c < kItem ? (int)(D - c) : kItem, false);
    return;
  }
  const int64_t group = (int64_t)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
  const int64_t run = group / pieces;
  const int64_t c = ((group % pieces) * lanes + (threadIdx.x & (lanes - 1))) * kItem;
  const int64_t p0 = run * kRun;
  if (p0 >= n || c >= D) return;
  const int p1 = n - p0 < kRun ? n : (int)p0 + kRun;
  const int count = D - c < kItem ? (int)(D - c) : kItem;
  const bool began = p0 > 0 && keys[p0 - 1] == keys[p0];   // the first id began in an earlier run
  const bool goes_on = p1 < n && keys[p1 - 1] == keys[p1];  // the last id goes on in the next
  float sum[kItem] = {};
  bool first = true;
  for (int p = (int)p0; p < p1; ++p) {
    const int key = keys[p];
    const E* src = dy + (int64_t)order[p] * dy_stride + c;
    float f[kItem] = {};
    if (count == kItem) {
      load_row<kItem>(src, f);
    } else {
      for (int e = 0; e < kItem; ++e)
        if (e < count) f[e] = Vec<E>::value(src[e]);
    }
#pragma unroll
    for (int e = 0; e < kItem; ++e) sum[e] += f[e];
    if (p + 1 < p1 && keys[p + 1] == key) continue;
    const bool whole = !(first && began) && !(p + 1 == p1 && goes_on);
    if (whole) {
#pragma unroll
      for (int e = 0; e < kItem; ++e) sum[e] *= scale;
      put_row(out + (int64_t)key * out_stride + c, sum, count, add);
    } else {
      float* q = part + (2 * run + (first && began ? 0 : 1)) * part_stride + c;
      for (int e = 0; e < kItem; ++e)
        if (e < count) q[e] = sum[e];
    }
#pragma unroll
    for (int e = 0; e < kItem; ++e) sum[e] = 0.0f;
    first = false;
  }
}

// One wave per run whose last id began in it and goes on, and 64 columns: the
// id's pieces are part[run][1] and part[r][0] of the runs r that follow.
template <class O>
__global__ __launch_bounds__(256) void merge_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ start,
                                                    int64_t V, int64_t D, const float* __restrict__ part,
                                                    int64_t part_stride, float scale, O* __restrict__ out,
                                                    int64_t out_stride, bool add, int pieces) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave_id();
  const int64_t run = unit / pieces;
  const int64_t c = (unit % pieces) * 64 + (threadIdx.x & 63);
  const int n = start[V];
  const int64_t p1 = (run + 1) * kRun;
  if (p1 >= n || c >= D) return;
  const int key = keys[p1 - 1];
  if (keys[p1] != key || start[key] < run * kRun) return;
  const int64_t last = (start[key + 1] - 1) / kRun;
  float sum = part[(2 * run + 1) * part_stride + c];
  for (int64_t r = run + 1; r <= last; ++r) sum += part[2 * r * part_stride + c];
  O* p = out + (int64_t)key * out_stride + c;
  *p = Vec<O>::round(add ? Vec<O>::value(*p) + sum * scale : sum * scale);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// lanes that share a row: enough for its items, at most a workgroup
static int row_lanes_log2(int64_t D) {
  int l = 0;
  while (l < 8 && (int64_t(kItem) << l) < D) ++l;
  return l;
}

static int check_rows(const lora_mat* m) {
  if (!float_dtype_ok(m->dtype)) return LORA_ERR_DTYPE;
  if (!valid_dims(m)) return LORA_ERR_SHAPE;
  if (m->cols > 1 && m->stride_col != 1) return LORA_ERR_STRIDE;
  if (m->rows > 1 && m->stride_row < m->cols) return LORA_ERR_STRIDE;
  if (!aligned(m->ptr, elem_size(m->dtype))) return LORA_ERR_STRIDE;
  return LORA_OK;
}

constexpr int64_t kMaxTokens = 0x7FFFFFFF - 4096;  // 32-bit token positions, also rounded up to a workgroup's
constexpr int64_t kMaxGrid = 0x7FFFFFFF;

struct GradPlan {
  int64_t runs, part_stride;
  int bins, sort_blocks;
  size_t bytes;
  int32_t *order, *keys, *start;
  float* part;
};

static GradPlan plan_grad(int64_t T, int64_t V, int64_t D, void* ws) {
  GradPlan g{};
  g.runs = ceil_div(T, kRun);
  g.part_stride = round_up(D, 4);
  // 256 workgroups (one per CU) while their ids fit the histogram, more beyond
  g.bins = static_cast<int>(V <= 256 * kBins ? ceil_div(V, 256) : kBins);
  g.sort_blocks = static_cast<int>(ceil_div(V, g.bins));
  Carver w(ws);
  g.order = static_cast<int32_t*>(w.take(T * sizeof(int32_t)));
  g.keys = static_cast<int32_t*>(w.take(T * sizeof(int32_t)));
  g.start = static_cast<int32_t*>(w.take((V + 1) * sizeof(int32_t)));
  g.part = static_cast<float*>(w.take(2 * g.runs * g.part_stride * sizeof(float)));
  g.bytes = w.used;
  return g;
}

static bool grad_sizes_ok(int64_t T, int64_t V, int64_t D) {
  // partial sums: 8 bytes per run and column, within what one operand may span
  return T >= 0 && V >= 0 && D >= 0 && T <= kMaxTokens && V <= kMaxTokens && D <= kMaxOperand &&
         (T == 0 || D == 0 || ceil_div(T, kRun) <= kMaxOperand / (8 * (D + 4)));
}

template <class E, class O>
static int run_grad(const GradPlan& g, const lora_mat* dy, float scale, const lora_mat* out, bool add,
                    hipStream_t st) {
  const int64_t V = out->rows, D = out->cols;
  const int ll = row_lanes_log2(D);
  const int groups = 256 >> ll;
  const int64_t pieces = ceil_div(D, int64_t(kItem) << ll);
  const int64_t run_blocks = ceil_div(g.runs * pieces, groups);
  const int64_t fill_blocks = add ? 0 : ceil_div(V, groups);
  const int64_t merge_pieces = ceil_div(D, 64);
  const int64_t merge_blocks = ceil_div(g.runs * merge_pieces, 4);
  if (run_blocks + fill_blocks > kMaxGrid || merge_blocks > kMaxGrid || pieces > kMaxGrid || merge_pieces > kMaxGrid)
    return LORA_ERR_LIMIT;
  auto* o = static_cast<O*>(out->ptr);
  launch(grad_kernel<E, O>, dim3(run_blocks + fill_blocks), dim3(256), 0, st, (const int32_t*)g.order,
         (const int32_t*)g.keys, (const int32_t*)g.start, V, D, static_cast<const E*>(dy->ptr), dy->stride_row, scale,
         o, out->stride_row, add, g.part, g.part_stride, ll, static_cast<int>(pieces), run_blocks);
  if (g.runs > 1)
    launch(merge_kernel<O>, dim3(merge_blocks), dim3(256), 0, st, (const int32_t*)g.keys, (const int32_t*)g.start, V,
           D, (const float*)g.part, g.part_stride, scale, o, out->stride_row, add, static_cast<int>(merge_pieces));
  return launch_status();
}

}  // namespace lora

using namespace lora;

extern "C" int lora_embed(const int32_t* ids, const lora_mat* table, float scale, const lora_mat* out, void* stream) {
  if (!table || !out) return LORA_ERR_NULL;
  if (table->cols != out->cols) return LORA_ERR_SHAPE;
  if (int e = check_rows(table)) return e;
  if (int e = check_rows(out)) return e;
  if (out->dtype == LORA_BF16 && table->dtype != LORA_BF16) return LORA_ERR_DTYPE;
  const int64_t T = out->rows, V = table->rows, D = out->cols;
  if (T > kMaxTokens || V > kMaxTokens) return LORA_ERR_LIMIT;
  if (T == 0 || D == 0) return LORA_OK;
  if (!ids || !out->ptr || (V > 0 && !table->ptr)) return LORA_ERR_NULL;
  const int ll = row_lanes_log2(D);
  const int64_t blocks = ceil_div(T, 256 >> ll);
  const int64_t steps = ceil_div(D, int64_t(kItem) << ll);
  const int items = steps >= 4 && blocks >= 512 ? 4 : 1;
  if (ceil_div(steps, items) > 65535) return LORA_ERR_LIMIT;
  const dim3 grid(blocks, ceil_div(steps, items));
  auto st = static_cast<hipStream_t>(stream);
  auto go = [&](auto* e, auto* o) {
    using E = std::remove_pointer_t<decltype(e)>;
    using O = std::remove_pointer_t<decltype(o)>;
    launch(embed_kernel<E, O>, grid, dim3(256), 0, st, ids, T, (const E*)e, table->stride_row, V, D, scale, o,
           out->stride_row, ll, items);
  };
  if (table->dtype == LORA_F32)
    go(static_cast<float*>(table->ptr), static_cast<float*>(out->ptr));
  else if (out->dtype == LORA_F32)
    go(static_cast<uint16_t*>(table->ptr), static_cast<float*>(out->ptr));
  else
    go(static_cast<uint16_t*>(table->ptr), static_cast<uint16_t*>(out->ptr));
  return launch_status();
}

extern "C" size_t lora_embed_grad_workspace_bytes(int64_t T, int64_t V, int64_t D) {
  if (!grad_sizes_ok(T, V, D) || V == 0 || D == 0) return 0;
  return plan_grad(T, V, D, nullptr).bytes;
}

extern "C" int lora_embed_grad(const int32_t* ids, const lora_mat* dy, float scale, const lora_mat* dtable,
                               int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dy || !dtable) return LORA_ERR_NULL;
  if (dy->cols != dtable->cols) return LORA_ERR_SHAPE;
  if (int e = check_rows(dy)) return e;
  if (int e = check_rows(dtable)) return e;
  if (dtable->dtype == LORA_BF16 && dy->dtype != LORA_BF16) return LORA_ERR_DTYPE;
  const int64_t T = dy->rows, V = dtable->rows, D = dtable->cols;
  if (!grad_sizes_ok(T, V, D)) return LORA_ERR_LIMIT;
  if (V == 0 || D == 0 || (T == 0 && accumulate)) return LORA_OK;
  if (!dtable->ptr || (T > 0 && (!ids || !dy->ptr))) return LORA_ERR_NULL;
  // without tokens the sort still runs (it writes the empty ranges that the zeros go by)
  const GradPlan g = plan_grad(T, V, D, workspace);
  if (!workspace || workspace_bytes < g.bytes || !aligned(workspace, 256)) return LORA_ERR_WORKSPACE;
  auto st = static_cast<hipStream_t>(stream);
  launch(sort_kernel, dim3(g.sort_blocks), dim3(1024), 0, st, ids, static_cast<int>(T), static_cast<int>(V), g.bins,
         g.order, g.keys, g.start);
  const bool add = accumulate != 0;
  if (dy->dtype == LORA_F32) return run_grad<float, float>(g, dy, scale, dtable, add, st);
  if (dtable->dtype == LORA_F32) return run_grad<uint16_t, float>(g, dy, scale, dtable, add, st);
  return run_grad<uint16_t, uint16_t>(g, dy, scale, dtable, add, st);
}
