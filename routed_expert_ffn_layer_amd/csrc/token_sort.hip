// token_sort.hip -- token rows sorted by expert (dispatch) and back with their weights (combine), and the
// gradients of both and of the gate.
//
// All of it is bound by memory: a token's row is read once and written to its k places, k rows are read
// and one is written, and in the combine's gradient both at once.  The work goes by token, so the row
// that is shared by k pairs is read once and stays in registers; the k places are rows of their own,
// whole cache lines each.  No atomics: every sum has one owner and a fixed order.
//
// Order of the pairs (a stable counting sort, as moe_permute's, but with pairs of no expert left out):
//  * up to kSmallPairs pairs: one launch.  Every workgroup holds all ids in LDS and finds the places of
//    its own token's pairs by counting (ids below; equal ids before), then copies the row.
//  * more: the pairs are cut into at most kMaxChunks chunks, and a workgroup places the pairs of each; then a
//    launch copies the rows.  How many pairs of each expert lie before the chunk, and in all, every workgroup
//    finds by itself: up to kSelfPairs pairs from the ids (they are in L2, and a launch less is worth it: there and
//    back of 2048 pairs 10.9 us instead of 14.2, of 8192 12.7 and 13.3, of 24576 94.6 and 90.0), beyond that from
//    the counts of each chunk that a launch before has written.
#include "kernels.hpp"
#include "row_io.hpp"

#include <algorithm>

namespace moe {

namespace {

constexpr int kSmallPairs = 1024;
constexpr int kSelfPairs = 8192;
constexpr int kMaxChunks = 256;
constexpr int kPlaceThreads = 256;
constexpr int kSortMaxE = 1024;

inline int chunk_pairs(int n) {  // n <= 2^30
  const int per = (n + kMaxChunks - 1) / kMaxChunks;
  return (per + kPlaceThreads - 1) / kPlaceThreads * kPlaceThreads;
}

// Copies the 16-byte group at column col of a row of H elements (fewer at the row's end) to k rows.
template <bool PASS, typename E_, int GROUP = 16 / sizeof(E_)>
__device__ __forceinline__ void copy_group(const E_* __restrict__ src, E_* __restrict__ rows, int64_t rows_ld,
                                           const int* dest, int k, int col, int H) {
  typedef E_ Vec __attribute__((ext_vector_type(GROUP)));
  typedef Vec Any __attribute__((aligned(sizeof(E_))));
  const int n = H - col;
  if (n >= GROUP) {
    const Vec v = *reinterpret_cast<const Any*>(src + col);
#pragma unroll
    for (int j = 0; j < k; ++j) {
      const int p = dest[j];
      if (p >= 0) put<PASS>(reinterpret_cast<Any*>(rows + (int64_t)p * rows_ld + col), v);
    }
  } else {
    for (int i = 0; i < n; ++i) {
      const E_ e = src[col + i];
      for (int j = 0; j < k; ++j) {
        const int p = dest[j];
        if (p >= 0) rows[(int64_t)p * rows_ld + col + i] = e;
      }
    }
  }
}

// Few pairs: places, counts and offsets, and the rows, in one launch of a workgroup per token.
template <typename E_>
__global__ __launch_bounds__(256) void dispatch_small_kernel(DispatchArgs a) {
  __shared__ int s_id[kSmallPairs];
  __shared__ int s_dest[32];
  const int n = a.T * a.k, t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int r = threadIdx.x; r < n; r += 256) {
    const int id = a.ids[r];
    s_id[r] = (unsigned)id < (unsigned)a.E ? id : 0x7fffffff;  // of no expert: above every id
  }
  __syncthreads();
  for (int j = wv; t < a.T && j < a.k; j += 4) {
    const int r = t * a.k + j, id = s_id[r];
    int place = 0;
    for (int q = lane; q < n; q += 64) {
      const int o = s_id[q];
      place += o < id || (o == id && q < r);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) place += __shfl_xor(place, d, 64);
    const bool in = id != 0x7fffffff;
    if (lane == 0) {
      a.inv_rows[r] = in ? place : -1;
      a.sorted_rows[place] = in ? r : -1;  // pairs of no expert come behind all others
      s_dest[j] = in && place < a.n_rows ? place : -1;
    }
  }
  // counts and offsets: a lane per expert, 64 experts a wave, the groups spread over the grid
  for (int g = blockIdx.x * 4 + wv; g * 64 <= a.E; g += gridDim.x * 4) {
    const int e = g * 64 + lane;
    int below = 0, equal = 0;
    for (int q = 0; q < n; ++q) {
      const int o = s_id[q];
      below += o < e;
      equal += o == e;
    }
    if (e < a.E) a.counts[e] = equal;
    if (e <= a.E) a.offsets[e] = below;
  }
  if (t >= a.T) return;  // no tokens at all: one workgroup, for the counts
  __syncthreads();
  const E_* src = static_cast<const E_*>(a.x) + t * a.x_ld;
  for (int col = threadIdx.x * (16 / sizeof(E_)); col < a.H; col += 256 * (16 / sizeof(E_)))
    copy_group<false>(src, static_cast<E_*>(a.rows), a.rows_ld, s_dest, a.k, col, a.H);
}

// Counts of the ids of chunk blockIdx.x -> table[chunk][E].
__global__ __launch_bounds__(kPlaceThreads) void count_kernel(DispatchArgs a, int chunk, int32_t* __restrict__ table) {
  __shared__ int s_cnt[kSortMaxE];
  const int n = a.T * a.k, lo = blockIdx.x * chunk, hi = min(n, lo + chunk);
  for (int e = threadIdx.x; e < a.E; e += kPlaceThreads) s_cnt[e] = 0;
  __syncthreads();
  for (int r = lo + threadIdx.x; r < hi; r += kPlaceThreads) {
    const int id = a.ids[r];
    if ((unsigned)id < (unsigned)a.E) atomicAdd(&s_cnt[id], 1);  // integer counts: any order gives the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kPlaceThreads) table[blockIdx.x * a.E + e] = s_cnt[e];
}

// Places of the pairs of chunk blockIdx.x.  SELF: without a table.
template <bool SELF>
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(DispatchArgs a, int chunk,
                                                              const int32_t* __restrict__ table) {
  constexpr int kWaves = kPlaceThreads / 64;
  __shared__ int s_next[kSortMaxE];            // where the expert's next pair of this chunk goes
  __shared__ int s_all[kSortMaxE];
  __shared__ uint16_t s_wave[kWaves][kSortMaxE];  // pairs of the expert in this round, by wave
  __shared__ int s_sum[kWaves];
  const int n = a.T * a.k, b = blockIdx.x, nb = gridDim.x, E = a.E;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int lo = b * chunk;
  const int hi = min(n, lo + chunk);
  if constexpr (SELF) {
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) s_next[e] = s_all[e] = 0;
    __syncthreads();
    auto add = [&](int r, int id) {  // integer counts: any order gives the same
      if ((unsigned)id < (unsigned)E) atomicAdd(r < lo ? &s_next[id] : &s_all[id], 1);
    };
    const int4* ids4 = reinterpret_cast<const int4*>(a.ids);
#pragma unroll 4
    for (int q = threadIdx.x; q < n / 4; q += kPlaceThreads) {
      const int4 v = ids4[q];
      add(4 * q, v.x);
      add(4 * q + 1, v.y);
      add(4 * q + 2, v.z);
      add(4 * q + 3, v.w);
    }
    if (threadIdx.x < n % 4) add(n / 4 * 4 + threadIdx.x, a.ids[n / 4 * 4 + threadIdx.x]);
    __syncthreads();
  }
  int before[kSortMaxE / kPlaceThreads];
#pragma unroll
  for (int i = 0; i < kSortMaxE / kPlaceThreads; ++i) {
    const int e = i * kPlaceThreads + threadIdx.x;
    before[i] = 0;
    if (e < E) {
      if constexpr (SELF) {
        before[i] = s_next[e];
        s_all[e] += before[i];
      } else {
        int all = 0;
#pragma unroll 32  // loads in flight: the table's columns are the launch's longest chain
        for (int q = 0; q < nb; ++q) {
          const int c = table[q * E + e];
          all += c;
          before[i] += q < b ? c : 0;
        }
        s_all[e] = all;
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s_wave[w][e] = 0;
    }
  }
  __syncthreads();
  // exclusive prefix over the experts: thread i sums experts 4 i .. 4 i + 3, then waves are joined
  constexpr int kPer = kSortMaxE / kPlaceThreads;
  int own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    own[i] = sum;
    sum += e < E ? s_all[e] : 0;
  }
  const int incl = wave_incl_scan(sum);
  if (lane == 63) s_sum[wv] = incl;
  __syncthreads();
  int base = incl - sum;
  for (int w = 0; w < wv; ++w) base += s_sum[w];
  int total = 0;
  for (int w = 0; w < kWaves; ++w) total += s_sum[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < E) {
      s_next[e] = base + own[i];
      if (b == 0) {
        a.counts[e] = s_all[e];
        a.offsets[e] = base + own[i];
      }
    }
  }
  if (b == 0 && threadIdx.x == 0) a.offsets[E] = total;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * kPlaceThreads + threadIdx.x;
    if (e < E) s_next[e] += before[i];
  }
  int nbits = 0;
  while ((1 << nbits) < E) ++nbits;
  const uint64_t lanes_below = lane == 0 ? 0 : ~0ull >> (64 - lane);
  __syncthreads();
  for (; lo < hi; lo += kPlaceThreads) {  // at most 2^30 + 255
    const int r = lo + threadIdx.x;
    const int id = r < hi ? a.ids[r] : -1;
    const bool valid = (unsigned)id < (unsigned)E;
    // lanes of the wave with the same expert
    uint64_t match = __ballot(valid);
    for (int i = 0; i < nbits; ++i) {
      const uint64_t m = __ballot(valid && ((id >> i) & 1));
      match &= ((id >> i) & 1) ? m : ~m;
    }
    const int rank = __popcll(match & lanes_below);
    if (valid && rank == 0) s_wave[wv][id] = (uint16_t)__popcll(match);
    __syncthreads();
    if (valid) {
      int place = s_next[id] + rank;
      for (int w = 0; w < wv; ++w) place += s_wave[w][id];
      a.sorted_rows[place] = r;
      a.inv_rows[r] = place;
    } else if (r < hi) {
      a.inv_rows[r] = -1;
    }
    __syncthreads();
    if (valid && rank == 0) {
      atomicAdd(&s_next[id], (int)s_wave[wv][id]);
      s_wave[wv][id] = 0;
    }
    __syncthreads();
  }
  // the places behind the last pair: -1, shared out over the chunks
  for (int64_t p = (int64_t)total + b * kPlaceThreads + threadIdx.x; p < n; p += (int64_t)nb * kPlaceThreads)
    a.sorted_rows[p] = -1;
}

// Rows of the tokens to their places.  G threads a token.
template <typename E_, int G>
__global__ __launch_bounds__(256) void gather_kernel(DispatchArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  if (t >= a.T) return;
  const E_* src = static_cast<const E_*>(a.x) + t * a.x_ld;
  const int32_t* inv = a.inv_rows + t * a.k;
  constexpr int V = 16 / sizeof(E_);
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    int dest[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      dest[u] = j0 + u < a.k ? inv[j0 + u] : -1;
      if (dest[u] >= a.n_rows) dest[u] = -1;
    }
    for (int col = threadIdx.x % G * V; col < a.H; col += G * V) {
      if (a.pass)
        copy_group<true>(src, static_cast<E_*>(a.rows), a.rows_ld, dest, 8, col, a.H);
      else
        copy_group<false>(src, static_cast<E_*>(a.rows), a.rows_ld, dest, 8, col, a.H);
    }
  }
}

// A token's pairs, lane j holding pair j (k <= 32): its place, -1 where it has none, and its weight.
struct Pairs {
  int place;
  float weight;
  __device__ __forceinline__ Pairs(const CombineRowsArgs& a, int64_t t) {
    const int lane = threadIdx.x & 63;
    const int p = lane < a.k ? a.inv_rows[t * a.k + lane] : -1;
    place = (unsigned)p < (unsigned)a.n_rows ? p : -1;
    weight = a.topk_w && lane < a.k ? a.topk_w[t * a.k + lane] : 1.0f;
  }
  // The whole wave's view of pair j, as scalars.  Only where all lanes are active: a lane that has left a loop
  // need not hold its pair any more.
  __device__ __forceinline__ int at(int j) const { return __builtin_amdgcn_readlane(place, j); }
  __device__ __forceinline__ float w(int j) const {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j));
  }
};

// y[t] = sum_j w[t][j] rows[inv[t][j]] (w null: 1), j ascending, f32.  The rows of 8 pairs are on their way
// together.
template <typename RT, typename YT, int G, bool PASS>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineRowsArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + uniform(threadIdx.x / 64) / (G / 64);
  if (t >= a.T) return;
  const Pairs pairs(a, t);
  const RT* rows = static_cast<const RT*>(a.rows);
  YT* y = static_cast<YT*>(a.y) + t * a.y_ld;
  for (int col0 = 0; col0 < a.H; col0 += G * 8) {  // all lanes stay in: those past the row's end have n <= 0
    const int col = col0 + threadIdx.x % G * 8, n = a.H - col;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      Raw8<RT> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int p = pairs.at(j0 + u);
        if (p >= 0) v[u].template load<PASS>(rows + (int64_t)p * a.rows_ld + col, n);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int p = pairs.at(j0 + u);
        const float w = pairs.w(j0 + u);
        if (p < 0) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[u][i], acc[i]);
      }
    }
    store8(y + col, n, acc);
  }
}

// d_rows[p] = w dy[t], d_w = <dy[t], rows[p]> for the pairs of a token, p = inv[t][j].
template <typename YT, typename RT, int G, bool PASS>
__global__ __launch_bounds__(256) void combine_rows_backward_kernel(CombineRowsArgs a) {
  __shared__ float s_dot[4][8];
  const int wv = uniform(threadIdx.x / 64), lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + wv / (G / 64);
  if (G == 64 && t >= a.T) return;  // no barriers in this form
  const Pairs pairs(a, t);
  const YT* dy = static_cast<const YT*>(a.y) + t * a.y_ld;
  const RT* rows = static_cast<const RT*>(a.rows);
  RT* d_rows = static_cast<RT*>(a.d_rows);
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    float dot[8] = {};
    for (int col0 = 0; col0 < a.H; col0 += G * 8) {  // all lanes stay in
      const int col = col0 + threadIdx.x % G * 8, n = a.H - col;
      Raw8<RT> v[8];
      float d[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int p = pairs.at(j0 + u);
        if (p >= 0) v[u].template load<PASS>(rows + (int64_t)p * a.rows_ld + col, n);
      }
      load8(dy + col, n, d);  // from the caches for the second eight pairs on
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int p = pairs.at(j0 + u);
        const float w = pairs.w(j0 + u);
        if (p < 0) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[u] = fmaf(d[i], v[u][i], dot[u]);  // both 0 past the row's end
          o[i] = w * d[i];
        }
        if (a.pass)
          store8<true>(d_rows + (int64_t)p * a.dr_ld + col, n, o);
        else
          store8(d_rows + (int64_t)p * a.dr_ld + col, n, o);
      }
    }
    float mine = 0.0f;  // lane u: pair j0 + u
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float s = reduce64(dot[u], Add());
      mine = lane == u ? s : mine;
    }
    if constexpr (G > 64) {
      if (lane < 8) s_dot[wv][lane] = mine;
      __syncthreads();
      if (lane < 8) mine = (s_dot[0][lane] + s_dot[1][lane]) + (s_dot[2][lane] + s_dot[3][lane]);
      __syncthreads();
    }
    if (threadIdx.x % G < 8 && j0 + lane < a.k) a.d_w[t * a.k + j0 + lane] = mine;
  }
}

// d_logits[t][e] = sum over j with ids[j] = e of w_j (d_w_j - sum_i w_i d_w_i).  A wave per token: lane j
// holds pair j, then a lane per expert.
__global__ __launch_bounds__(256) void gate_backward_kernel(const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                            const float* __restrict__ d_w, int T, int E, int k,
                                                            float* __restrict__ d_logits) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = threadIdx.x & 63;
  const int id = lane < k ? ids[t * k + lane] : -1;
  const float wj = lane < k ? w[t * k + lane] : 0.0f, dj = lane < k ? d_w[t * k + lane] : 0.0f;
  float s = wj * dj;
  s = reduce64(s, Add());
  const float g = wj * (dj - s);
  for (int e = lane; e - lane < E; e += 64) {
    float v = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int idj = __builtin_amdgcn_readlane(id, j);
      const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), j));
      v += idj == e ? gj : 0.0f;
    }
    if (e < E) d_logits[t * E + e] = v;
  }
}

// Rows that pass the caches by.  Reading: rows of more than the 32 MB of the L2s, read once here (1024 tokens from
// 6144 rows of 4096 bf16 that memory holds 42 -> 34 us, that the last-level cache still holds 33 -> 34).  Writing:
// rows of more than half the 256 MB of the last-level cache (24576 rows of 4096 there and back: 103 -> 90 us).  Up to
// there the next reader loses more than the call gains: gradients of 16384 rows of 4096 30.0 and 30.4 us, with a
// copy of them behind 49 and 57; of 32768 rows of 2048 91 and 106.
inline int64_t row_bytes(int64_t rows, int H, bool bf16) { return rows * H * (bf16 ? 2 : 4); }
inline bool read_past(int64_t bytes) { return bytes > (int64_t)32 << 20; }
inline bool write_past(int64_t bytes) { return bytes > (int64_t)128 << 20; }

// Threads a token: a wave for short rows, else a workgroup.  There and back and gradients (us): 4096 tokens of 2048
// and 4096 bf16 105 + 116 in workgroups, 126 + 127 in waves; 8192 tokens of 1024 37 + 32 in waves, 45 + 35 in workgroups.
inline bool wave_rows(int H) { return H <= 1024; }

}  // namespace

size_t dispatch_workspace_bytes(int T, int k, int E) {
  const int n = T * k;
  if (n <= kSelfPairs) return 0;
  const int chunk = chunk_pairs(n);
  return (size_t)((n + chunk - 1) / chunk) * E * sizeof(int32_t);
}

hipError_t launch_dispatch(DispatchArgs a, int32_t* table, bool bf16, hipStream_t st) {
  const int n = a.T * a.k;
  a.pass = write_past(row_bytes(std::min(n, a.n_rows), a.H, bf16));
  if (n <= kSmallPairs) {
    if (bf16)
      hipLaunchKernelGGL(dispatch_small_kernel<uint16_t>, dim3(a.T > 0 ? a.T : 1), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL(dispatch_small_kernel<uint32_t>, dim3(a.T > 0 ? a.T : 1), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const int chunk = chunk_pairs(n), nb = (n + chunk - 1) / chunk;
  if (n <= kSelfPairs) {
    hipLaunchKernelGGL(place_kernel<true>, dim3(nb), dim3(kPlaceThreads), 0, st, a, chunk, table);
  } else {
    hipLaunchKernelGGL(count_kernel, dim3(nb), dim3(kPlaceThreads), 0, st, a, chunk, table);
    hipLaunchKernelGGL(place_kernel<false>, dim3(nb), dim3(kPlaceThreads), 0, st, a, chunk, table);
  }
  if (wave_rows(a.H)) {
    const dim3 grid((unsigned)((a.T + 3) / 4));
    if (bf16)
      hipLaunchKernelGGL((gather_kernel<uint16_t, 64>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((gather_kernel<uint32_t, 64>), grid, dim3(256), 0, st, a);
  } else if (bf16) {
    hipLaunchKernelGGL((gather_kernel<uint16_t, 256>), dim3(a.T), dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((gather_kernel<uint32_t, 256>), dim3(a.T), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

namespace {

template <typename RT, typename YT, bool PASS>
hipError_t combine_typed(const CombineRowsArgs& a, hipStream_t st) {
  if (wave_rows(a.H))
    hipLaunchKernelGGL((combine_rows_kernel<RT, YT, 64, PASS>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((combine_rows_kernel<RT, YT, 256, PASS>), dim3(a.T), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <typename YT, typename RT, bool PASS>
hipError_t backward_typed(const CombineRowsArgs& a, hipStream_t st) {
  if (wave_rows(a.H))
    hipLaunchKernelGGL((combine_rows_backward_kernel<YT, RT, 64, PASS>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((combine_rows_backward_kernel<YT, RT, 256, PASS>), dim3(a.T), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_rows(const CombineRowsArgs& a, bool rows_bf16, bool y_bf16, hipStream_t st) {
  typedef uint16_t B;
  typedef float F;
  const bool pass = read_past(row_bytes(std::min(a.T * a.k, a.n_rows), a.H, rows_bf16));
  if (rows_bf16) {
    if (y_bf16) return pass ? combine_typed<B, B, true>(a, st) : combine_typed<B, B, false>(a, st);
    return pass ? combine_typed<B, F, true>(a, st) : combine_typed<B, F, false>(a, st);
  }
  if (y_bf16) return pass ? combine_typed<F, B, true>(a, st) : combine_typed<F, B, false>(a, st);
  return pass ? combine_typed<F, F, true>(a, st) : combine_typed<F, F, false>(a, st);
}

hipError_t launch_combine_rows_backward(CombineRowsArgs a, bool dy_bf16, bool rows_bf16, hipStream_t st) {
  typedef uint16_t B;
  typedef float F;
  const int64_t bytes = row_bytes(std::min(a.T * a.k, a.n_rows), a.H, rows_bf16);
  const bool pass = read_past(bytes);
  a.pass = write_past(bytes);
  if (dy_bf16) {
    if (rows_bf16) return pass ? backward_typed<B, B, true>(a, st) : backward_typed<B, B, false>(a, st);
    return pass ? backward_typed<B, F, true>(a, st) : backward_typed<B, F, false>(a, st);
  }
  if (rows_bf16) return pass ? backward_typed<F, B, true>(a, st) : backward_typed<F, B, false>(a, st);
  return pass ? backward_typed<F, F, true>(a, st) : backward_typed<F, F, false>(a, st);
}

hipError_t launch_gate_backward(const int32_t* ids, const float* w, const float* d_w, int T, int E, int k,
                                float* d_logits, hipStream_t st) {
  hipLaunchKernelGGL(gate_backward_kernel, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, st, ids, w, d_w, T, E, k,
                     d_logits);
  return hipGetLastError();
}

}  // namespace moe
