// Embedding lookup with scaling and its gradient.
//
//   out[t] = scale * table[ids[t]]             (zeros for an id outside [0, V))
//   dtable[v] = scale * sum of dy[t] over the tokens t with ids[t] = v
//
// Both move rows and compute next to nothing: they are bound by HBM.
//
// The gradient sums in a fixed order, without float atomics: sort_kernel
// groups the tokens by id (stable) and gives every id its range of the
// list; grad_kernel cuts the list into runs of a fixed length, so that an id
// that fills the batch costs no more than others, and sums each id's tokens
// inside a run; merge_kernel adds the pieces of the ids that span runs.
//
// Kernels:
//   embed_kernel   rows gathered, scaled and stored
//   sort_kernel    the tokens grouped by id, one launch
//   grad_kernel    sums of each run's ids, zeros of the rows without tokens
//   merge_kernel   pieces of an id added in the order of their runs
//   few_grad_kernel  all of it for few tokens

#include "lora_host.hpp"
#include "lora_rows.hpp"

namespace lora {

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------

// A lane handles one 16-byte vector of the output's row at a time and U of
// them, `lanes` apart, all loaded before the first is stored. Rows that many
// tokens name are read again from the caches: the loads keep the default
// policy, the stores are non-temporal. 16731 rows of 8192, bfloat16 to
// float32: 144 us for 172 MB fetched and 548 written (5.0 TB/s); all rows
// distinct takes as long, so it is bound by what enters the XCDs.

// N elements of 8 or 16 bytes as float32
template <int N, class E>
__device__ __forceinline__ void load_items(const E* p, float* f) {
  if constexpr (N * sizeof(E) == 8) {
    typedef unsigned int half_t __attribute__((ext_vector_type(2), aligned(2)));
    const half_t w = *reinterpret_cast<const half_t*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    Vec<E>::unpack(vload(p), f);
  }
}

template <class E, class O, int U>
__global__ __launch_bounds__(256) void embed_kernel(const int32_t* __restrict__ ids, int64_t T,
                                                    const E* __restrict__ table, int64_t table_stride, int64_t V,
                                                    int64_t D, float scale, O* __restrict__ out, int64_t out_stride,
                                                    int lanes_log2, unsigned pieces) {
  constexpr int N = Vec<O>::N;
  const int lanes = 1 << lanes_log2;
  // a row's pieces follow each other: the grid writes in the order of the addresses
  const int64_t t = (int64_t)(blockIdx.x / pieces) * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
  if (t >= T) return;
  const int64_t id = ids[t];
  const bool live = id >= 0 && id < V;
  const E* src = table + (live ? id : 0) * table_stride;
  O* dst = out + t * out_stride;
  const int64_t c0 = ((int64_t)(blockIdx.x % pieces) * U * lanes + (threadIdx.x & (lanes - 1))) * N;
  float f[U][N];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + (int64_t)u * lanes * N;
    if (live && c + N <= D) load_items<N>(src + c, f[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + (int64_t)u * lanes * N;
    if (c + N <= D) {
#pragma unroll
      for (int e = 0; e < N; ++e) f[u][e] = live ? f[u][e] * scale : 0.0f;
      vstore_nt(dst + c, Vec<O>::pack(f[u]));
    } else {
      for (int64_t e = c; e < D; ++e) dst[e] = Vec<O>::round(live ? Vec<E>::value(src[e]) * scale : 0.0f);
    }
  }
}

// ---------------------------------------------------------------------------
// sort: groups the tokens by id, those of an id in their order. Four ids in a
// row belong to one workgroup, the next four to the next (frequent ids, often
// the low ones, spread over the card), and the ids' lists follow each other
// by workgroup. Every workgroup reads every token's id. Wave w takes the w-th
// part of the tokens and counts its own histogram, so that after a scan over
// (id, wave) each wave knows where its tokens of each id go; then it places
// them, a token's rank among the equal ids of its 64 found by ballots over
// the id's bits. The workgroup also counts the tokens of the workgroups
// before it, so nothing passes between workgroups.
//
// While counting, a wave lists its workgroup's tokens in shared memory and
// places them from there, 64 at a step. Reading the ids again instead, a
// load would wait for the stores of the steps before it: 16384 tokens over
// 128256 ids take 19 us that way, 9 from the list. A wave with more than
// kList of its tokens in one workgroup's ids reads again.
// ---------------------------------------------------------------------------
// How ids are shared out: blocks_log2 of the workgroups, `bins` ids to each.
struct IdMap {
  int blocks_log2, bins;
  __device__ __forceinline__ int block(int id) const { return (id >> 2) & ((1 << blocks_log2) - 1); }
  __device__ __forceinline__ int bin(int id) const { return (id >> (blocks_log2 + 2) << 2) | (id & 3); }
  __device__ __forceinline__ int id(int block, int bin) const {
    return (bin >> 2 << (blocks_log2 + 2)) | block << 2 | (bin & 3);
  }
  // position of an id in the lists' starts; the end of the last list is at total()
  __device__ __forceinline__ int64_t at(int id) const { return (int64_t)block(id) * bins + bin(id); }
  __device__ __forceinline__ int64_t total() const { return (int64_t)bins << blocks_log2; }
};

constexpr int kBinBits = 9, kBins = 1 << kBinBits;
constexpr int kSortWaves = 16;
constexpr int kList = 1024;                                // tokens that a wave lists
constexpr int64_t kListedPart = int64_t(1) << (32 - kBinBits);  // tokens of a wave that an entry can name

// A wave's ids, 64 at a step, loaded four steps ahead of their use.
struct Ahead {
  int id[4];
  static __device__ __forceinline__ int load(const int32_t* ids, int64_t t, int64_t end) {
    return t < end ? ids[t] : -1;
  }
  __device__ __forceinline__ Ahead(const int32_t* ids, int64_t t, int64_t end, int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) id[k] = load(ids, t + 64 * k + lane, end);
  }
  // the ids of the step at t
  __device__ __forceinline__ int next(const int32_t* ids, int64_t t, int64_t end, int lane) {
    const int now = id[0];
#pragma unroll
    for (int k = 0; k < 3; ++k) id[k] = id[k + 1];
    id[3] = load(ids, t + 256 + lane, end);
    return now;
  }
};

__global__ __launch_bounds__(1024) void sort_kernel(const int32_t* __restrict__ ids, int T, int V, IdMap map,
                                                    int32_t* __restrict__ order, int32_t* __restrict__ keys,
                                                    int32_t* __restrict__ start, int32_t* __restrict__ count) {
  __shared__ int hist[kSortWaves][kBins];
  __shared__ uint32_t list[kSortWaves][kList];
  __shared__ int below[kSortWaves];
  __shared__ int scan[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int block = blockIdx.x;
  // the workgroup of an id, or one past all of them
  auto owner = [&](int id) { return id >= 0 && id < V ? map.block(id) : 0x7FFFFFFF; };
  for (int i = tid; i < kSortWaves * kBins; i += 1024) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int part = (int)((((int64_t)T + kSortWaves - 1) / kSortWaves + 63) / 64 * 64);
  const int64_t first = (int64_t)wave * part;
  const int begin = (int)(first < T ? first : T);
  const int end = T - begin < part ? T : begin + part;

  int less = 0, listed = 0;
  Ahead a(ids, begin, end, lane);
  for (int64_t t = begin; t < end; t += 64) {
    const int id = a.next(ids, t, end, lane);
    const int o = owner(id);
    less += __popcll(__ballot(o < block));
    const bool mine = o == block;
    const uint64_t live = __ballot(mine);
    if (live == 0) continue;
    if (mine) {
      const int bin = map.bin(id);
      atomicAdd(&hist[wave][bin], 1);
      const int at = listed + __popcll(live & ((1ull << lane) - 1));
      if (at < kList) list[wave][at] = (static_cast<uint32_t>(t - begin) + lane) << kBinBits | bin;
    }
    listed += __popcll(live);
  }
  if (lane == 0) below[wave] = less;
  __syncthreads();

  // exclusive positions: over the waves of an id, then over the ids
  int base = 0;
  for (int w = 0; w < kSortWaves; ++w) base += below[w];
  int total = 0, before[kSortWaves] = {};  // tokens of the waves before each, of this thread's id
  if (tid < kBins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) before[w] = hist[w][tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = before[w];
      before[w] = total;
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
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) hist[w][tid] = at + before[w];
    if (tid < map.bins) {
      start[(int64_t)block * map.bins + tid] = at;
      const int id = map.id(block, tid);
      if (id < V) count[id] = total;  // in the order of the ids, for the rows without tokens
    }
    if (tid == map.bins - 1 && block == (1 << map.blocks_log2) - 1) start[map.total()] = at + total;
  }
  __syncthreads();

  auto place = [&](bool mine, int bin, int t) {
    uint64_t same = __ballot(mine);
#pragma unroll
    for (int b = 0; b < kBinBits; ++b) {
      const uint64_t bit = __ballot((bin >> b) & 1);
      same &= (bin >> b) & 1 ? bit : ~bit;
    }
    const int head = __ffsll((unsigned long long)same) - 1;
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int pos = 0;
    if (mine && rank == 0) pos = atomicAdd(&hist[wave][bin], __popcll(same));
    pos = __shfl(pos, mine ? head : 0, 64) + rank;
    if (mine) {
      order[pos] = t;
      keys[pos] = map.id(block, bin);
    }
  };
  if (listed <= kList && part <= kListedPart) {
    for (int i = 0; i < listed; i += 64) {
      const bool mine = i + lane < listed;
      const uint32_t w = mine ? list[wave][i + lane] : 0;
      place(mine, w & (kBins - 1), begin + (int)(w >> kBinBits));
    }
    return;
  }
  a = Ahead(ids, begin, end, lane);
  for (int64_t t = begin; t < end; t += 64) {
    const int id = a.next(ids, t, end, lane);
    const bool mine = owner(id) == block;
    if (__ballot(mine) != 0) place(mine, mine ? map.bin(id) : 0, static_cast<int>(t) + lane);
  }
}

// ---------------------------------------------------------------------------
// sums: a group of 2^lanes_log2 lanes takes one run of kRun sorted tokens and
// one piece of the columns, a vector of dy per lane and token, all of them
// loaded before the first is added. An id whose tokens all lie in the run is
// written at once; one that began before the run leaves its sum in
// part[run][0], one that goes on after it in part[run][1]. Runs of 16 tokens
// held half as many waves in flight (16384 tokens of 64 columns: 10 us, with
// runs of 8 4 us).
// ---------------------------------------------------------------------------
constexpr int kRun = 8;

// `count` of N elements
template <int N, class O>
__device__ __forceinline__ void put_row(O* p, const float* f, int count, bool add) {
  if (count == N) {
    float g[N];
#pragma unroll
    for (int e = 0; e < N; ++e) g[e] = f[e];
    if (add) {
      float old[N];
      load_row<N>(p, old);
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] += old[e];
    }
    store_row<N>(p, g);
  } else {
    for (int e = 0; e < N; ++e)
      if (e < count) p[e] = Vec<O>::round(add ? Vec<O>::value(p[e]) + f[e] : f[e]);
  }
}

struct GradLists {
  const int32_t *order, *keys, *start, *count;
  IdMap map;
  int64_t V, D;
};

// lanes and pieces of a row in the part of the grid that writes zeros
struct FillShape {
  int lanes_log2;
  unsigned pieces;
};

// Zeros of the rows that no token names, one vector per lane: many short
// workgroups in the order of the addresses write 1.05 GB in 153 us, with
// four vectors per lane in 175.
template <class O>
struct FillUnit {
  int64_t row, col;
  __device__ __forceinline__ FillUnit(const FillShape& f, unsigned block) {
    const unsigned unit = (block << (8 - f.lanes_log2)) + (threadIdx.x >> f.lanes_log2);
    row = unit / f.pieces;
    col = (((int64_t)(unit % f.pieces) << f.lanes_log2) + (threadIdx.x & ((1 << f.lanes_log2) - 1))) * Vec<O>::N;
  }
  __device__ __forceinline__ void zero(O* out, int64_t stride, int64_t D) const {
    O* p = out + row * stride + col;
    const typename Vec<O>::type zero = {0u, 0u, 0u, 0u};
    if (col + Vec<O>::N <= D) {
      vstore_nt(p, zero);
    } else {
      for (int e = 0; col + e < D; ++e) p[e] = Vec<O>::round(0.0f);
    }
  }
};

template <class E, class O, bool ADD>
__global__ __launch_bounds__(256, 8) void grad_kernel(GradLists l, const E* __restrict__ dy, int64_t dy_stride,
                                                   float scale, O* __restrict__ out, int64_t out_stride,
                                                   float* __restrict__ part, int64_t part_stride, int lanes_log2,
                                                   unsigned pieces, unsigned run_blocks, FillShape fill) {
  constexpr int N = Vec<E>::N;
  const int lanes = 1 << lanes_log2;
  if (blockIdx.x >= run_blocks) {
    const FillUnit<O> u(fill, blockIdx.x - run_blocks);
    if (u.row < l.V && u.col < l.D && l.count[u.row] == 0) u.zero(out, out_stride, l.D);
    return;
  }
  const int n = l.start[l.map.total()];
  const unsigned group = (blockIdx.x << (8 - lanes_log2)) + (threadIdx.x >> lanes_log2);
  const int64_t run = group / pieces;
  const int64_t c = ((int64_t)(group % pieces) * lanes + (threadIdx.x & (lanes - 1))) * N;
  const int64_t p0 = run * kRun;
  if (p0 >= n || c >= l.D) return;
  const int tokens = n - p0 < kRun ? n - (int)p0 : kRun;
  // the lists' ends are padded to whole runs; what lies past n is not used
  int key[kRun], at[kRun];
#pragma unroll
  for (int j = 0; j < kRun; j += 4) {
    const int4 k = *reinterpret_cast<const int4*>(l.keys + p0 + j);
    const int4 o = *reinterpret_cast<const int4*>(l.order + p0 + j);
    key[j] = k.x, key[j + 1] = k.y, key[j + 2] = k.z, key[j + 3] = k.w;
    at[j] = o.x, at[j + 1] = o.y, at[j + 2] = o.z, at[j + 3] = o.w;
  }
  const int last_key = l.keys[p0 + tokens - 1];
  const bool began = p0 > 0 && l.keys[p0 - 1] == key[0];                        // the first id began in an earlier run
  const bool goes_on = p0 + tokens < n && l.keys[p0 + tokens] == last_key;  // the last id goes on in the next
  float sum[N] = {};
  bool first = true;
  // after token j of id `key`, the last of its id in this run
  auto finish = [&](int j, int key, int count) {
    const bool before = first && began, after = j + 1 == tokens && goes_on;
    if (!before && !after) {
#pragma unroll
      for (int e = 0; e < N; ++e) sum[e] *= scale;
      put_row<N>(out + (int64_t)key * out_stride + c, sum, count, ADD);
    } else {
      put_row<N>(part + (2 * run + (before ? 0 : 1)) * part_stride + c, sum, count, false);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = 0.0f;
    first = false;
  };
  if (l.D - c < N) {
    // the row's last elements
    const int count = (int)(l.D - c);
    for (int j = 0; j < tokens; ++j) {
      const int key_j = l.keys[p0 + j];
      const E* src = dy + (int64_t)l.order[p0 + j] * dy_stride + c;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < count) sum[e] += Vec<E>::value(src[e]);
      if (j + 1 == tokens || l.keys[p0 + j + 1] != key_j) finish(j, key_j, count);
    }
    return;
  }
  typename Vec<E>::type w[kRun];
#pragma unroll
  for (int j = 0; j < kRun; ++j)
    if (j < tokens) w[j] = vload_nt(dy + (int64_t)at[j] * dy_stride + c);
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    if (j >= tokens) break;
    float f[N];
    Vec<E>::unpack(w[j], f);
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] += f[e];
    if (j + 1 == tokens || key[j + 1 < kRun ? j + 1 : j] != key[j]) finish(j, key[j], N);
  }
}

// One workgroup per run whose last id began in it and goes on, and 8 columns
// for each of `lanes` lanes: the id's pieces are part[run][1] and part[r][0]
// of the runs r that follow. The workgroup's 256 / lanes groups take every
// so many-th of them, and the groups' sums are added in order. Most runs have
// nothing to merge: their workgroups only look, which is what bounds it (1023
// runs of 4096 columns 7 us, with 4 columns per lane 10).
constexpr int kMergeCols = 8;

template <class O>
__global__ __launch_bounds__(256) void merge_kernel(GradLists l, const float* __restrict__ part, int64_t part_stride,
                                                    float scale, O* __restrict__ out, int64_t out_stride, bool add,
                                                    int lanes_log2, unsigned pieces) {
  __shared__ f32x4_t sums[2][256];
  const int64_t run = blockIdx.x / pieces;
  const int64_t p1 = (run + 1) * kRun;  // below the padded length of the lists: the last run has no workgroup
  const int n = l.start[l.map.total()], key = l.keys[p1 - 1], next = l.keys[p1];
  if (p1 >= n || next != key) return;
  const int64_t s = l.map.at(key);
  const int from = l.start[s], to = l.start[s + 1];
  if (from < run * kRun) return;
  const int lanes = 1 << lanes_log2, groups = 256 >> lanes_log2;
  const int64_t c = ((int64_t)(blockIdx.x % pieces) * lanes + (threadIdx.x & (lanes - 1))) * kMergeCols;
  const int64_t last = (to - 1) / kRun;  // the id's last run
  f32x4_t sum[2] = {};
  if (c < l.D) {
    for (int64_t r = run + (threadIdx.x >> lanes_log2); r <= last; r += 4 * groups) {
      f32x4_t v[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t k = r + u * groups;
        const float* p = part + (2 * k + (k == run ? 1 : 0)) * part_stride + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) v[u][h] = k <= last ? ld16f(p + 4 * h) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) sum[h] += v[u][h];
    }
  }
  sums[0][threadIdx.x] = sum[0];
  sums[1][threadIdx.x] = sum[1];
  __syncthreads();
  if ((int)threadIdx.x >= lanes || c >= l.D) return;
  for (int g = 1; g < groups; ++g) {
    sum[0] += sums[0][(g << lanes_log2) + threadIdx.x];
    sum[1] += sums[1][(g << lanes_log2) + threadIdx.x];
  }
  float f[kMergeCols];
#pragma unroll
  for (int e = 0; e < kMergeCols; ++e) f[e] = sum[e >> 2][e & 3] * scale;
  put_row<kMergeCols>(out + (int64_t)key * out_stride + c, f, l.D - c < kMergeCols ? (int)(l.D - c) : kMergeCols, add);
}

// ---------------------------------------------------------------------------
// few tokens: one launch. Every workgroup holds all ids; the group of a
// token's lanes sums its id's tokens if it is the first of them, and the
// other workgroups write zeros where no id falls into their rows.
// ---------------------------------------------------------------------------
constexpr int kFewTokens = 64;

template <class E, class O, bool ADD>
__global__ __launch_bounds__(256, 8) void few_grad_kernel(const int32_t* __restrict__ ids, int T, int64_t V, int64_t D,
                                                          const E* __restrict__ dy, int64_t dy_stride, float scale,
                                                          O* __restrict__ out, int64_t out_stride, int lanes_log2,
                                                          unsigned pieces, unsigned run_blocks, FillShape fill) {
  constexpr int N = Vec<E>::N, U = 8;
  __shared__ int held[256];  // the ids, -1 past them; or whether a row is named
  const int tid = threadIdx.x;
  const int mine = tid < T ? ids[tid] : -1;
  if (blockIdx.x >= run_blocks) {
    const FillUnit<O> u(fill, blockIdx.x - run_blocks);
    // the workgroup's rows: as many as it has units, or one that has several pieces
    const int64_t first = ((blockIdx.x - run_blocks) << (8 - fill.lanes_log2)) / fill.pieces;
    const int rows = 256 >> fill.lanes_log2;
    const bool named = mine >= 0 && mine < V && mine >= first && mine - first < rows;
    if (__syncthreads_or(named)) {
      held[tid] = 0;
      __syncthreads();
      if (named) held[mine - first] = 1;
      __syncthreads();
      if (held[u.row - first]) return;
    }
    if (u.row < V && u.col < D) u.zero(out, out_stride, D);
    return;
  }
  held[tid] = mine;
  __syncthreads();
  const unsigned group = (blockIdx.x << (8 - lanes_log2)) + (tid >> lanes_log2);
  const int t = group / pieces;
  const int64_t c = (((int64_t)(group % pieces) << lanes_log2) + (tid & ((1 << lanes_log2) - 1))) * N;
  if (t >= T || c >= D) return;
  const int id = held[t];
  if (id < 0 || id >= V) return;
  bool later = false;
  for (int s = 0; s < t; s += U) {
#pragma unroll
    for (int j = 0; j < U; ++j) later |= s + j < t && held[s + j] == id;
  }
  if (later) return;
  const int count = D - c < N ? (int)(D - c) : N;
  const E* src = dy + c;
  float sum[N] = {};
  for (int s = t; s < T; s += U) {
    bool same[U];
    bool any = false;
#pragma unroll
    for (int j = 0; j < U; ++j) any |= same[j] = held[s + j] == id;  // -1 past the last token
    if (!any) continue;
    if (count == N) {
      typename Vec<E>::type w[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (same[j]) w[j] = vload_nt(src + (int64_t)(s + j) * dy_stride);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (!same[j]) continue;
        float f[N];
        Vec<E>::unpack(w[j], f);
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += f[e];
      }
    } else {
      for (int j = 0; j < U; ++j) {
        if (held[s + j] != id) continue;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < count) sum[e] += Vec<E>::value(src[(int64_t)(s + j) * dy_stride + e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) sum[e] *= scale;
  put_row<N>(out + (int64_t)id * out_stride + c, sum, count, ADD);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// lanes that share a row of D elements: enough for `item` elements each, at most a workgroup
static int row_lanes_log2(int64_t D, int item) {
  int l = 0;
  while (l < 8 && (int64_t(item) << l) < D) ++l;
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
constexpr int64_t kMaxGrid = max_blocks(256);
constexpr int kMaxSortLog2 = 21;  // 2^21 workgroups of 1024: the most that a launch holds
static_assert((int64_t(1) << kMaxSortLog2) <= max_blocks(1024) && (int64_t(2) << kMaxSortLog2) > max_blocks(1024));

struct GradPlan {
  int64_t runs, part_stride;
  IdMap map;
  size_t bytes;
  int32_t *order, *keys, *start, *count;
  float* part;
};

static GradPlan plan_grad(int64_t T, int64_t V, int64_t D, void* ws) {
  GradPlan g{};
  g.runs = ceil_div(T, kRun);
  g.part_stride = round_up(D, kMergeCols);
  // 256 workgroups (one per CU) while their ids fit the histogram, more beyond
  const int64_t quads = ceil_div(V, 4);
  g.map.blocks_log2 = 8;
  while (ceil_div(quads, int64_t(1) << g.map.blocks_log2) > kBins / 4) ++g.map.blocks_log2;
  g.map.bins = static_cast<int>(4 * ceil_div(quads, int64_t(1) << g.map.blocks_log2));
  Carver w(ws);
  g.order = static_cast<int32_t*>(w.take(T * sizeof(int32_t)));
  g.keys = static_cast<int32_t*>(w.take(T * sizeof(int32_t)));
  g.start = static_cast<int32_t*>(w.take(((int64_t(g.map.bins) << g.map.blocks_log2) + 1) * sizeof(int32_t)));
  g.count = static_cast<int32_t*>(w.take(V * sizeof(int32_t)));
  g.part = static_cast<float*>(w.take(2 * g.runs * g.part_stride * sizeof(float)));
  g.bytes = w.used;
  return g;
}

static bool grad_sizes_ok(int64_t T, int64_t V, int64_t D) {
  // partial sums: 8 bytes per run and column, within what one operand may span
  return T >= 0 && V >= 0 && D >= 0 && T <= kMaxTokens && V <= kMaxTokens && D <= kMaxOperand &&
         (T == 0 || D == 0 || ceil_div(T, kRun) <= kMaxOperand / (8 * (D + kMergeCols)));
}

// The grid of a gradient kernel: `items` runs or tokens of the lists, then the rows for zeros.
struct GradGrid {
  int lanes_log2;
  int64_t pieces, item_blocks, fill_blocks;
  FillShape fill;
  int status;
};

template <class E, class O>
static GradGrid grad_grid(int64_t items, int64_t V, int64_t D, bool add) {
  GradGrid g{};
  g.lanes_log2 = row_lanes_log2(D, Vec<E>::N);
  g.pieces = ceil_div(D, int64_t(Vec<E>::N) << g.lanes_log2);
  g.fill.lanes_log2 = row_lanes_log2(D, Vec<O>::N);
  const int64_t fill_pieces = ceil_div(D, int64_t(Vec<O>::N) << g.fill.lanes_log2);
  g.fill.pieces = static_cast<unsigned>(fill_pieces);
  // items, rows and their pieces are counted in 32 bits, rounded up to a workgroup's 256
  constexpr int64_t kMost = 0x7FFFFFFF - 256;
  if (g.pieces > kMost || fill_pieces > kMost || items * g.pieces > kMost || V * fill_pieces > kMost) {
    g.status = LORA_ERR_LIMIT;
    return g;
  }
  g.item_blocks = ceil_div(items * g.pieces, 256 >> g.lanes_log2);
  g.fill_blocks = add ? 0 : ceil_div(V * fill_pieces, 256 >> g.fill.lanes_log2);
  if (g.item_blocks + g.fill_blocks > kMaxGrid) g.status = LORA_ERR_LIMIT;
  return g;
}

template <class E, class O>
static int run_few(const int32_t* ids, const lora_mat* dy, float scale, const lora_mat* out, bool add,
                   hipStream_t st) {
  const int64_t V = out->rows, D = out->cols;
  const GradGrid g = grad_grid<E, O>(dy->rows, V, D, add);
  if (g.status) return g.status;
  launch(add ? few_grad_kernel<E, O, true> : few_grad_kernel<E, O, false>, dim3(g.item_blocks + g.fill_blocks),
         dim3(256), 0, st, ids, static_cast<int>(dy->rows), V, D, static_cast<const E*>(dy->ptr), dy->stride_row,
         scale, static_cast<O*>(out->ptr), out->stride_row, g.lanes_log2, static_cast<unsigned>(g.pieces),
         static_cast<unsigned>(g.item_blocks), g.fill);
  return launch_status();
}

template <class E, class O>
static int run_grad(const GradPlan& g, const int32_t* ids, const lora_mat* dy, float scale, const lora_mat* out,
                    bool add, hipStream_t st) {
  const int64_t T = dy->rows, V = out->rows, D = out->cols;
  const GradGrid grid = grad_grid<E, O>(g.runs, V, D, add);
  if (grid.status) return grid.status;
  int ml = row_lanes_log2(D, kMergeCols);
  ml = ml < 4 ? 4 : ml < 6 ? ml : 6;  // 4 to 16 groups
  const int64_t merge_pieces = ceil_div(D, int64_t(kMergeCols) << ml);
  if (merge_pieces > kMaxGrid || g.runs * merge_pieces > kMaxGrid) return LORA_ERR_LIMIT;
  if (g.map.blocks_log2 > kMaxSortLog2) return LORA_ERR_LIMIT;
  launch(sort_kernel, dim3(1 << g.map.blocks_log2), dim3(1024), 0, st, ids, static_cast<int>(T), static_cast<int>(V),
         g.map, g.order, g.keys, g.start, g.count);
  const GradLists l = {g.order, g.keys, g.start, g.count, g.map, V, D};
  auto* o = static_cast<O*>(out->ptr);
  launch(add ? grad_kernel<E, O, true> : grad_kernel<E, O, false>, dim3(grid.item_blocks + grid.fill_blocks),
         dim3(256), 0, st, l, static_cast<const E*>(dy->ptr), dy->stride_row, scale, o, out->stride_row, g.part,
         g.part_stride, grid.lanes_log2, static_cast<unsigned>(grid.pieces), static_cast<unsigned>(grid.item_blocks),
         grid.fill);
  launch(merge_kernel<O>, dim3((g.runs - 1) * merge_pieces), dim3(256), 0, st, l, (const float*)g.part, g.part_stride,
         scale, o, out->stride_row, add, ml, static_cast<unsigned>(merge_pieces));
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
  const int item = vec_elems(out->dtype);
  const int ll = row_lanes_log2(D, item);
  const int64_t blocks = ceil_div(T, 256 >> ll);
  const int64_t steps = ceil_div(D, int64_t(item) << ll);
  // U vectors of a row per lane where the row has them and the workgroups still fill the card
  const int u = steps >= 4 && blocks >= 512 ? 4 : steps >= 2 && blocks >= 512 ? 2 : 1;
  const int64_t pieces = ceil_div(steps, u);
  if (blocks > kMaxGrid || pieces > kMaxGrid || blocks * pieces > kMaxGrid) return LORA_ERR_LIMIT;
  auto st = static_cast<hipStream_t>(stream);
  auto go = [&](auto* e, auto* o) {
    using E = std::remove_pointer_t<decltype(e)>;
    using O = std::remove_pointer_t<decltype(o)>;
    launch(u == 4 ? embed_kernel<E, O, 4> : u == 2 ? embed_kernel<E, O, 2> : embed_kernel<E, O, 1>,
           dim3(blocks * pieces), dim3(256),
           0, st, ids, T, (const E*)e, table->stride_row, V, D, scale, o, out->stride_row, ll,
           static_cast<unsigned>(pieces));
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
  const GradPlan g = plan_grad(T, V, D, workspace);
  if (!workspace || workspace_bytes < g.bytes || !aligned(workspace, 256)) return LORA_ERR_WORKSPACE;
  auto st = static_cast<hipStream_t>(stream);
  const bool add = accumulate != 0;
  // Few tokens take one launch instead of three: 64 over 128256 x 64 float32 9 us instead of 14 (128 tokens:
  // 12 and 15 with distinct ids, 17 and 14 with one id, whose tokens one group then sums)
  auto go = [&](auto* e, auto* o) {
    using E = std::remove_pointer_t<decltype(e)>;
    using O = std::remove_pointer_t<decltype(o)>;
    return T <= kFewTokens ? run_few<E, O>(ids, dy, scale, dtable, add, st)
                           : run_grad<E, O>(g, ids, dy, scale, dtable, add, st);
  };
  if (dy->dtype == LORA_F32) return go(static_cast<float*>(nullptr), static_cast<float*>(nullptr));
  if (dtable->dtype == LORA_F32) return go(static_cast<uint16_t*>(nullptr), static_cast<float*>(nullptr));
  return go(static_cast<uint16_t*>(nullptr), static_cast<uint16_t*>(nullptr));
}
