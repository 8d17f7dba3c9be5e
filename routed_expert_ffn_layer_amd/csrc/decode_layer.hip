// decode_layer.hip -- one MoE layer for a few tokens in two kernels: routing with the
// gate/up products, and the down products with the weighted sum.
//
//   ids, w = top-k of the logits and their softmax (or given by the caller)
//   h[p]   = SiLU(Wgate[e] x[t]) * (Wup[e] x[t])          p = t*k + j, e = ids[p]
//   y[t]   = sum_j w[p] * (W2[e] h[p])  (+ the shared expert)
//
// What bounds it: the active experts' weights are read once (HBM) and, for one token,
// the chain launch -> logits -> top-k -> first weights, once per kernel.  Splitting the
// layer at h is forced (every output needs every h); everything else is folded into
// the two kernels: each block repeats the routing for itself (a few hundred pairs at
// most, in LDS), which costs less than a launch, and the block that owns 16 output
// columns holds the products of all pairs in LDS and adds them there, so neither the
// expert rows nor the permutation ever reach memory.
//
// Every sum has a fixed order (K parts in ascending order, then the pairs of a token in
// ascending j), so results are the same on every run.
#include "kernels.hpp"
#include "stream_tile.hpp"
#include "topk.hpp"

namespace moe {

constexpr int kDlMaxPairs = kDecodeLayerMaxPairs, kDlMaxT = kDecodeLayerMaxT;
constexpr int kNoExpert = 0x7fffffff;
constexpr int kGuWaves = 8, kGuTiles = 2;  // gate/up: waves of a block (K parts), row tiles per work item
constexpr int kDnWaves = 16;               // down: waves of a block

// Routing of the batch as a block sees it (LDS).
struct __align__(16) DlPlan {
  int32_t id[kDlMaxPairs];    // expert of pair p
  float w[kDlMaxPairs];       // its gate weight
  int32_t key[kDlMaxPairs];   // the expert if it has a slot, else kNoExpert; padded to a multiple of 4
  int32_t sorted[kDlMaxPairs];  // pairs by (key, p)
  int32_t run_n[kDlMaxPairs];   // by position: pairs of the run that begins here, 0 if none does
  int32_t run_at[kDlMaxPairs];  // first position of run i
  int32_t slot[1024];
};

// Phase 1: ids, gate weights (and the slot table) into LDS.
template <int EPL>
__device__ __forceinline__ void dl_route_t(DlPlan& s, const DecodeLayerArgs& a) {
  for (int t = threadIdx.x >> 6; t < a.T; t += blockDim.x >> 6)
    topk_row<EPL>(a.logits + (size_t)t * a.E, a.E, a.k, s.id + t * a.k, s.w + t * a.k);
}

__device__ __forceinline__ void dl_load_slots(DlPlan& s, const DecodeLayerArgs& a) {
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) s.slot[e] = a.slot_of_expert[e];
}

// Phase 2: sort the pairs by expert (stable) and cut every expert's pairs into runs of
// up to 16.  Pair p's position is the number of pairs with a smaller (key, p): n^2 / threads
// compares of LDS broadcasts.  Returns the number of runs (the same in every thread).
__device__ __forceinline__ int dl_plan(DlPlan& s, const DecodeLayerArgs& a) {
  const int n = a.T * a.k, n4 = (n + 3) & ~3, p = threadIdx.x;
  if (p < n4) {
    int key = kNoExpert;
    if (p < n) {
      const int e = s.id[p];
      if (e >= 0 && e < a.E && s.slot[e] >= 0) key = e;
    }
    s.key[p] = key;
  }
  __syncthreads();
  if (p < n) {
    const int key = s.key[p];
    int less = 0, before = 0, same = 0;
    for (int q = 0; q < n4; q += 4) {
      const int4 kq = *reinterpret_cast<const int4*>(s.key + q);
      less += (kq.x < key) + (kq.y < key) + (kq.z < key) + (kq.w < key);
      same += (kq.x == key) + (kq.y == key) + (kq.z == key) + (kq.w == key);
      before += (kq.x == key && q < p) + (kq.y == key && q + 1 < p) + (kq.z == key && q + 2 < p) +
                (kq.w == key && q + 3 < p);
    }
    const int at = less + before;
    s.sorted[at] = p;
    s.run_n[at] = key != kNoExpert && before % 16 == 0 ? min(16, same - before) : 0;
  }
  __syncthreads();
  int runs = 0;
  const int lane = p & 63;
  const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
  for (int c = 0; c < n; c += 64) {
    const uint64_t m = __ballot(c + lane < n && s.run_n[c + lane] > 0);
    if (c + lane == p && ((m >> lane) & 1)) s.run_at[runs + __popcll(m & below)] = p;
    runs += __popcll(m);
  }
  __syncthreads();
  return runs;
}

template <int WT>
__device__ __forceinline__ int dl_token_offset(int lane, int n, int ld) {
  return min(a_token(lane), n - 1) * ld * 2;
}

// ---------------------------------------------------------------------------
// Gate/up.  Work items (run, kGuTiles row tiles of W13) are dealt to the blocks in turn;
// the 8 waves split K, and the block adds their parts in LDS, applies SwiGLU and writes
// h.  A W13 row tile holds 8 gate rows and the 8 up rows beside them.
// ---------------------------------------------------------------------------
template <int WT>
__global__ __launch_bounds__(64 * kGuWaves) void decode_gate_up(DecodeLayerArgs a) {
  __shared__ DlPlan s;
  __shared__ float red[kGuTiles][kGuWaves][256];  // [tile][K part][token][row]
  const int lane = threadIdx.x & 63, kp = uniform(threadIdx.x >> 6);
  const int n = a.T * a.k;
  dl_load_slots(s, a);
  if (a.logits) {
    if (a.E <= 64) dl_route_t<1>(s, a);
    else if (a.E <= 128) dl_route_t<2>(s, a);
    else if (a.E <= 256) dl_route_t<4>(s, a);
    else if (a.E <= 512) dl_route_t<8>(s, a);
    else dl_route_t<16>(s, a);
  } else {
    for (int p = threadIdx.x; p < n; p += blockDim.x) s.id[p] = a.ids[p];
  }
  __syncthreads();
  if (a.logits && blockIdx.x == 0) {
    for (int p = threadIdx.x; p < n; p += blockDim.x) {
      a.ids[p] = s.id[p];
      a.w[p] = s.w[p];
    }
  }
  const int runs = uniform(dl_plan(s, a));
  const int g_sh = a.shared_w ? (a.I_shared / 8 + kGuTiles - 1) / kGuTiles : 0;
  const int g_rt = (a.I / 8 + kGuTiles - 1) / kGuTiles;
  const int sh_items = (a.T + 15) / 16 * g_sh;
  const int nk = ksteps<WT>(a.H), s0 = kp * nk / kGuWaves, s1 = (kp + 1) * nk / kGuWaves;
  const __amdgpu_buffer_rsrc_t xbuf = make_rsrc(a.x, (size_t)a.T * a.H * 2);
  for (int item = blockIdx.x; item < sh_items + runs * g_rt; item += gridDim.x) {
    const bool shared = item < sh_items;
    const int it = shared ? item : item - sh_items, per = shared ? g_sh : g_rt;
    const int run = it / per, tile0 = (it - run * per) * kGuTiles;
    const int Ie = shared ? a.I_shared : a.I;
    const int at = shared ? run * 16 : uniform(s.run_at[run]);
    const int m = shared ? min(16, a.T - at) : uniform(s.run_n[at]);
    const uint8_t* slot = shared ? a.shared_w : a.slot_pool + (uint64_t)uniform(s.slot[uniform(s.key[uniform(s.sorted[at])])]) * a.slot_stride;
    const Mat w = w13_mat<WT>(slot, a.H, Ie);
    const int tok = min(a_token(lane), m - 1);
    const int row_off = (shared ? at + tok : s.sorted[at + tok] / a.k) * a.H * 2;
    const int tiles = min(kGuTiles, Ie / 8 - tile0);
    for (int t = 0; t < tiles; ++t) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      stream_tile<WT>(w, tile0 + t, s0, s1, xbuf, row_off, acc);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * v < m) red[t][kp][64 * v + lane] = acc[v];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < tiles * m * 8; o += 64 * kGuWaves) {
      const int t = o / (m * 8), i = o / 8 - t * m, c = o & 7;
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int q = 0; q < kGuWaves; ++q) {
        gate += red[t][q][16 * i + c];
        up += red[t][q][16 * i + c + 8];
      }
      const int row = shared ? n + at + i : s.sorted[at + i];
      a.h[(size_t)row * a.h_ld + (tile0 + t) * 8 + c] = f32_to_bf16_rne(silu_f32(gate) * up);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Down and combine.  A block owns one row tile of W2 (16 columns of y) for every pair:
// its waves take (run, K part) tasks in turn, the products of all pairs meet in LDS, and
// the block adds each token's pairs in ascending j.
// ---------------------------------------------------------------------------
template <int WT, bool BF16OUT>
__global__ __launch_bounds__(64 * kDnWaves) void decode_down(DecodeLayerArgs a, int parts) {
  __shared__ DlPlan s;
  extern __shared__ float val[];  // [part][pair, then shared token][16]
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
  const int n = a.T * a.k, rows = n + (a.shared_w ? a.T : 0);
  dl_load_slots(s, a);
  for (int p = threadIdx.x; p < n; p += blockDim.x) {
    s.id[p] = a.ids[p];
    s.w[p] = a.w[p];
  }
  __syncthreads();
  const int runs = uniform(dl_plan(s, a));
  const int sh_runs = a.shared_w ? (a.T + 15) / 16 : 0;
  const int tile = blockIdx.x;
  const __amdgpu_buffer_rsrc_t hbuf = make_rsrc(a.h, (size_t)rows * a.h_ld * 2);
  for (int task = wv; task < (sh_runs + runs) * parts; task += kDnWaves) {
    const int r0 = task / parts, part = task - r0 * parts;
    const bool shared = r0 < sh_runs;
    const int run = shared ? r0 : r0 - sh_runs;
    const int at = shared ? run * 16 : uniform(s.run_at[run]);
    const int m = shared ? min(16, a.T - at) : uniform(s.run_n[at]);
    const int Ie = shared ? a.I_shared : a.I;
    const uint8_t* slot = shared ? a.shared_w : a.slot_pool + (uint64_t)uniform(s.slot[uniform(s.key[uniform(s.sorted[at])])]) * a.slot_stride;
    const Mat w = w2_mat<WT>(slot, a.H, Ie);
    const int tok = min(a_token(lane), m - 1);
    const int row_off = (shared ? n + at + tok : s.sorted[at + tok]) * a.h_ld * 2;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    stream_tile<WT>(w, tile, part * w.nK / parts, (part + 1) * w.nK / parts, hbuf, row_off, acc);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = (lane >> 4) + 4 * v;
      if (i < m) {
        const int row = shared ? n + at + i : s.sorted[at + i];
        val[((size_t)part * rows + row) * 16 + (lane & 15)] = acc[v];
      }
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.T * 16; o += blockDim.x) {
    const int t = o >> 4, c = o & 15;
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int p = t * a.k + j;
      if (s.key[p] == kNoExpert) continue;
      float d = 0.f;
      for (int q = 0; q < parts; ++q) d += val[((size_t)q * rows + p) * 16 + c];
      y = fmaf(s.w[p], d, y);
    }
    if (a.shared_w) {
      float d = 0.f;
      for (int q = 0; q < parts; ++q) d += val[((size_t)q * rows + n + t) * 16 + c];
      y += d;
    }
    const size_t at = (size_t)t * a.H + tile * 16 + c;
    if (BF16OUT)
      static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rne(y);
    else
      static_cast<float*>(a.y)[at] = y;
  }
}

template <int WT>
static hipError_t launch_t(const DecodeLayerArgs& a, bool bf16_out, hipStream_t st) {
  // an upper bound on the work items: every pair its own run
  const int64_t n = (int64_t)a.T * a.k;
  const int64_t bound = (a.shared_w ? (int64_t)(a.T + 15) / 16 * ((a.I_shared / 8 + kGuTiles - 1) / kGuTiles) : 0) +
                        n * ((a.I / 8 + kGuTiles - 1) / kGuTiles);
  const unsigned grid = (unsigned)(bound < 512 ? bound : 512);
  hipLaunchKernelGGL(decode_gate_up<WT>, dim3(grid), dim3(64 * kGuWaves), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int parts = n <= 16 ? 2 : 1;
  const size_t lds = (size_t)parts * (n + (a.shared_w ? a.T : 0)) * 64;
  const dim3 g2(a.H / 16), b2(64 * kDnWaves);
  if (bf16_out)
    hipLaunchKernelGGL((decode_down<WT, true>), g2, b2, lds, st, a, parts);
  else
    hipLaunchKernelGGL((decode_down<WT, false>), g2, b2, lds, st, a, parts);
  return hipGetLastError();
}

hipError_t launch_decode_layer(int wtype, const DecodeLayerArgs& a, bool bf16_out, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  return wtype == W_BF16 ? launch_t<W_BF16>(a, bf16_out, st) : launch_t<W_MXFP4>(a, bf16_out, st);
}

}  // namespace moe
