// decode_layer.hip -- one MoE layer for a few tokens in two kernels: routing with the
// gate/up products, and the down products with the weighted sum.
//
//   ids, w = top-k of the logits and their softmax (or given by the caller)
//   h[p]   = SiLU(Wgate[e] x[t]) * (Wup[e] x[t])          p = t*k + j, e = ids[p]; bf16, or two of them
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
// Pairs are sorted by expert and cut into runs (pairs of one expert that one matrix
// tile serves); a run's weights stream once past all of its tokens.
//
// Every sum has a fixed order (K parts in ascending order, then the pairs of a token in
// ascending j), so results are the same on every run.
//
// Measured: bf16 layer (H = 2048, I = 512, 8 of 256 experts and a shared one) of 16 tokens
// 85 + 42 us, 645 MB, 5.1 TB/s; of one token 13.0 + 7.3 us for 57 MB, about 6 us of the
// first kernel before its first weights; MXFP4 layer (H = 4096, I = 2048, 6 of 256) of 64 tokens
// 103 + 66 us, 20 us of the first kernel for routing and first weights (the separate calls take
// 145 us for the whole layer there: they read W13 once per 32 tokens).
#include "kernels.hpp"
#include "stream_tile.hpp"

namespace moe {

constexpr int kDlMaxPairs = kDecodeLayerMaxPairs;
constexpr int kDlWaves = 16;  // waves of a block, one block per CU
constexpr int kDlThreads = 64 * kDlWaves;
constexpr int kDlTeams = 4;  // gate/up: teams of a block, a tile each
constexpr int kDlHalfTiles = 128;  // row tiles of W2 up to which the down kernel's blocks own half a tile
// Up to this many tokens h is kept as two bf16, h and the remainder of its rounding (16
// significant bits), larger batches round it to bf16.  One rounding of h costs y as much
// as y's own rounding to bf16 (an RMS error of 0.0024 instead of 0.0017); the remainder rides in
// operand rows that a few tokens leave empty, but doubles the h loads that bound the down
// products of many.  MXFP4, h in one and in two parts: 28.2 and 28.9 us a layer at one token,
// 65 and 70 at 8.  With the limit at 32, over eight shapes (H 256 to 7168, 16 to 256 experts), a layer
// of 9 / 16 / 32 tokens takes 2-12 / 3-14 / 5-20% longer in MXFP4 and 0-2 / 0-5 / 0-13% in bf16 (least where
// 256 experts keep HBM busy: 129.6 and 130.2 us at 16 tokens of H = 2048, I = 512, most at H = 7168, I = 2048:
// 491 and 516, 640 and 723 at 32).  Above the limit y has the precision of the separate calls.
constexpr int kDlSplitT = 8;

// A run: pairs of one expert (or tokens of the shared expert) that one matrix tile serves.
struct __align__(16) DlRun {
  uint64_t w;  // the expert's weights
  int32_t at;  // its first position in sorted order (shared expert: its first token)
  int32_t m;   // pairs
};
constexpr int kDlMaxRuns = kDlMaxPairs + kDecodeLayerMaxT;

// What gate/up's first block leaves in the workspace for the second kernel.
struct __align__(16) DlShared {
  int32_t runs, pad[3];
  DlRun run[kDlMaxRuns];        // cut for the second kernel; the shared expert's first
  int32_t sorted[kDlMaxPairs];  // by position: the pair
  int32_t valid[kDlMaxPairs];   // by pair: its expert has a slot
};

size_t decode_layer_plan_bytes() { return sizeof(DlShared); }

// Routing of the batch as a gate/up block sees it (LDS).
struct __align__(16) DlPlan {
  DlRun run[kDlMaxRuns];
  int32_t id[kDlMaxPairs];   // expert of pair p
  int32_t key[kDlMaxPairs];  // the same if it has a slot, else -1
  uint16_t group[1024];      // first position of each expert's pairs
  uint16_t sorted[kDlMaxPairs];  // by position: the pair
};

// Largest of v over the wave, in a scalar register, by six in-register steps (shifts by 1, 2,
// 4, 8 inside a row of 16 lanes, then two broadcasts of a row's last lane).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOE_DPP_MAX(ctrl, rows) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
  MOE_DPP_MAX(0x111, 0xf);  // row_shr:1
  MOE_DPP_MAX(0x112, 0xf);  // row_shr:2
  MOE_DPP_MAX(0x114, 0xf);  // row_shr:4
  MOE_DPP_MAX(0x118, 0xf);  // row_shr:8
  MOE_DPP_MAX(0x142, 0xa);  // row_bcast:15 into rows 1 and 3
  MOE_DPP_MAX(0x143, 0xc);  // row_bcast:31 into rows 2 and 3
#undef MOE_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Inclusive prefix sum over the wave, with the same in-register steps.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
#define MOE_DPP_ADD(ctrl, rows) v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false)
  MOE_DPP_ADD(0x111, 0xf);
  MOE_DPP_ADD(0x112, 0xf);
  MOE_DPP_ADD(0x114, 0xf);
  MOE_DPP_ADD(0x118, 0xf);
  MOE_DPP_ADD(0x142, 0xa);
  MOE_DPP_ADD(0x143, 0xc);
#undef MOE_DPP_ADD
  return v;
}

// Top-k of one token by one wave, lane l holding experts 64 i + l as order-preserving
// keys (zero past E and once taken).  k rounds take the largest key of the wave, the lowest
// index among equals; with up to 256 experts each lane first sorts its own four (larger
// first, then lower index), so that a round looks at the heads only, with more it looks
// for its largest every round (sorting 8 or 16 costs more than it saves).  Then the softmax
// of the k values.  The rounds stay in registers, and k is small, where a bitwise select
// takes 32 rounds whatever k is.
template <int EPL>
__device__ __forceinline__ void topk_few(const float (&row)[EPL], int E, int k, int32_t* ids, float* w) {
  const int lane = threadIdx.x & 63;
  uint32_t key[EPL];
  int grp[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    const uint32_t b = __float_as_uint(row[i]);
    // larger value, larger key; -0.0 and +0.0 the same
    key[i] = e >= E ? 0u : (b << 1) == 0u ? 0x80000000u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    grp[i] = i;
  }
  constexpr bool SORT = EPL <= 4;
#pragma unroll
  for (int i = 1; SORT && i < EPL; ++i)
#pragma unroll
    for (int j = i; j > 0; --j) {
      const bool swap = key[j] > key[j - 1];
      const uint32_t hi = swap ? key[j] : key[j - 1], lo = swap ? key[j - 1] : key[j];
      const int gh = swap ? grp[j] : grp[j - 1], gl = swap ? grp[j - 1] : grp[j];
      key[j - 1] = hi;
      key[j] = lo;
      grp[j - 1] = gh;
      grp[j] = gl;
    }
  uint32_t mine = 0;
  int my_id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t head = key[0];
    int head_grp = grp[0];
#pragma unroll
    for (int i = 1; !SORT && i < EPL; ++i) {
      head_grp = key[i] > head ? i : head_grp;
      head = max(head, key[i]);
    }
    const uint32_t best = wave_max(head);
    uint64_t m = __ballot(head == best);
    if (m & (m - 1)) {  // equal heads: the lowest expert
      const uint32_t inv = head == best ? 0xffffu - (uint32_t)(head_grp * 64 + lane) : 0u;
      m = __ballot(inv == wave_max(inv));
    }
    const int at = __builtin_ctzll(m);
    const int id = __builtin_amdgcn_readlane(head_grp, at) * 64 + at;
    if (lane == at) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if constexpr (SORT) {
          key[i] = i + 1 < EPL ? key[i + 1] : 0u;
          grp[i] = i + 1 < EPL ? grp[i + 1] : 0;
        } else {
          key[i] = i == head_grp ? 0u : key[i];
        }
      }
    }
    if (lane == j) {
      mine = best;
      my_id = id;
    }
  }
  const float v = __uint_as_float((mine & 0x80000000u) ? mine ^ 0x80000000u : ~mine);
  const float top = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 0));
  const float ex = expf(v - top);
  float sum = 0.f;
#pragma unroll 1
  for (int j = 0; j < k; ++j)
    sum += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ex), j));
  if (lane < k) {
    ids[lane] = my_id;
    w[lane] = ex / sum;
  }
}

// Tokens w, w + 16, ... by wave w; a row is requested before the one ahead of it is searched.
template <int EPL>
__device__ __forceinline__ void dl_route(DlPlan& s, float* w, const DecodeLayerArgs& a) {
  const int lane = threadIdx.x & 63;
  float row[EPL], next[EPL];
  auto load = [&](float(&r)[EPL], int t) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = min(i * 64 + lane, a.E - 1);
      r[i] = a.logits[(size_t)min(t, a.T - 1) * a.E + e];
    }
  };
  int t = threadIdx.x >> 6;
  load(row, t);
#pragma unroll 1
  for (; t < a.T; t += kDlWaves) {
    load(next, t + kDlWaves);
    topk_few<EPL>(row, a.E, a.k, s.id + t * a.k, w + t * a.k);
#pragma unroll
    for (int i = 0; i < EPL; ++i) row[i] = next[i];
  }
}

// Groups the pairs by expert, in ascending token order, and cuts every expert's pairs into
// runs of up to P (and, for the second kernel, of up to P2 into `out`, where given).  Each
// expert has a bit mask of the tokens that chose it: its count is the mask's population, a
// pair's place in its group the population below its token, and one scan over the experts
// (thread e holds expert e) places groups and runs.  Given routing may name an expert twice
// in one token, which a mask cannot hold: then every pair counts the pairs before it of the
// same expert instead (n compares each).  Up to 64 pairs take one wave and one barrier
// instead (four barriers: 1.6 us of a 21 us layer at one token).
// slots: the slot table; mask: E 64-bit words; part: kDlWaves words (all LDS).
// Returns the number of runs, the shared expert's included (the same in every thread); ends
// with a barrier.
static_assert(kDlThreads >= 1024 && kDlMaxPairs <= kDlThreads && kDecodeLayerMaxT <= 64, "thread e holds expert e");

__device__ __forceinline__ int dl_plan(DlPlan& s, const int32_t* slots, uint64_t* mask, uint32_t* part,
                                       const DecodeLayerArgs& a, int P, int P2, DlShared* out) {
  const int n = a.T * a.k, p = threadIdx.x, wv = p >> 6, t = p / a.k;
  const int sh1 = a.shared_w ? (a.T + P - 1) / P : 0, sh2 = a.shared_w ? (a.T + P2 - 1) / P2 : 0;
  const uint64_t shared_w = reinterpret_cast<uint64_t>(a.shared_w);
  if (p < sh1) s.run[p] = DlRun{shared_w, p * P, min(P, a.T - p * P)};
  if (out && p < sh2) out->run[p] = DlRun{shared_w, p * P2, min(P2, a.T - p * P2)};
  int e = -1;
  if (p < n) {
    const int id = s.id[p];
    e = id >= 0 && id < a.E && slots[id] >= 0 ? id : -1;
    s.key[p] = e;
  }
  if (n <= 64) {
    // One wave, in registers, groups in order of their first pair: a pair counts its equals
    // (all, and before it), a scan over the groups' first pairs places groups and runs.
    if (wv == 0) {
      int count = 0, before = 0, first = 64;
#pragma unroll 1
      for (int q = 0; q < n; ++q) {
        const bool same = __builtin_amdgcn_readlane(e, q) == e;
        count += same;
        before += same && q < p;
        first = same ? min(first, q) : first;
      }
      const bool head = e >= 0 && before == 0;
      const uint32_t runs1 = head ? (count + P - 1) / P : 0, runs2 = head ? (count + P2 - 1) / P2 : 0;
      const uint32_t packed = (head ? count : 0) | runs1 << 10 | runs2 << 20, scan = wave_scan(packed);
      const uint32_t base = scan - packed;
      if (head) {
        const uint64_t w = reinterpret_cast<uint64_t>(a.slot_pool) + (uint64_t)slots[e] * a.slot_stride;
        const int at = base & 0x3ff, r1 = sh1 + (base >> 10 & 0x3ff), r2 = sh2 + (base >> 20);
#pragma unroll 1
        for (int i = 0; i < (int)runs1; ++i) s.run[r1 + i] = DlRun{w, at + i * P, min(P, count - i * P)};
#pragma unroll 1
        for (int i = 0; out && i < (int)runs2; ++i) out->run[r2 + i] = DlRun{w, at + i * P2, min(P2, count - i * P2)};
      }
      const int group = __shfl((int)(base & 0x3ff), first & 63, 64);
      if (e >= 0) s.sorted[group + before] = (uint16_t)p;
      if (p == 63) {
        part[0] = sh1 + (scan >> 10 & 0x3ff);
        if (out) out->runs = sh2 + (scan >> 20);
      }
    }
    __syncthreads();
    return part[0];
  }
  bool twice = false;
  if (e >= 0) {
    const uint64_t bit = 1ull << t;
    twice = (atomicOr(reinterpret_cast<unsigned long long*>(mask + e), bit) & bit) != 0;
  }
  twice = __syncthreads_or(twice);
  // thread e: pairs of expert e, its runs, and its runs for the second kernel, 10 bits each
  // (sums of at most 512)
  uint32_t count = 0;
  if (p < a.E) {
    if (!twice) {
      count = __popcll(mask[p]);
    } else {
#pragma unroll 1
      for (int q = 0; q < n; ++q) count += s.key[q] == p;
    }
  }
  const uint32_t runs1 = (count + P - 1) / P, runs2 = (count + P2 - 1) / P2;
  const uint32_t packed = count | runs1 << 10 | runs2 << 20, scan = wave_scan(packed);
  if ((p & 63) == 63) part[wv] = scan;
  __syncthreads();
  uint32_t base = 0, total = 0;
#pragma unroll
  for (int q = 0; q < kDlWaves; ++q) {
    const uint32_t v = part[q];
    base += q < wv ? v : 0u;
    total += v;
  }
  base += scan - packed;
  if (count > 0) {
    const uint64_t w = reinterpret_cast<uint64_t>(a.slot_pool) + (uint64_t)slots[p] * a.slot_stride;
    const int at = base & 0x3ff, r1 = sh1 + (base >> 10 & 0x3ff), r2 = sh2 + (base >> 20);
#pragma unroll 1
    for (int i = 0; i < (int)runs1; ++i) s.run[r1 + i] = DlRun{w, at + i * P, min(P, (int)count - i * P)};
#pragma unroll 1
    for (int i = 0; out && i < (int)runs2; ++i) out->run[r2 + i] = DlRun{w, at + i * P2, min(P2, (int)count - i * P2)};
  }
  if (out && p == 0) out->runs = sh2 + (total >> 20);
  if (p < a.E) s.group[p] = base & 0x3ff;
  __syncthreads();
  if (e >= 0) {
    int before = 0;
    if (!twice) {
      before = __popcll(mask[e] & ((1ull << t) - 1));
    } else {
#pragma unroll 1
      for (int q = 0; q < p; ++q) before += s.key[q] == e;
    }
    s.sorted[s.group[e] + before] = (uint16_t)p;
  }
  __syncthreads();
  return sh1 + (total >> 10 & 0x3ff);
}

struct RunRef {
  const uint8_t* w;
  int at, m;
};
__device__ __forceinline__ RunRef read_run(const DlRun* r) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(r);
  RunRef o;
  o.w = (const uint8_t*)((uint64_t)(uint32_t)uniform((int)v[1]) << 32 | (uint32_t)uniform((int)v[0]));
  o.at = uniform((int)v[2]);
  o.m = uniform((int)v[3]);
  return o;
}

// Copies m token rows (H bf16 each, padded with zeros to `padded` 16-byte pieces) into LDS
// rows of row_bytes, by `threads` threads of which this is number `me`; token(i) is row
// i's token.  Four pieces per thread are requested before the first is stored.
template <typename Token>
__device__ __forceinline__ void copy_rows(uint8_t* rows, int row_bytes, const uint16_t* x, int H, int m, int me,
                                          int threads, const Token& token) {
  const int padded = (row_bytes - 16) / 16, total = m * padded;
#pragma unroll 1
  for (int c0 = me; c0 < total; c0 += 4 * threads) {
    u32x4 v[4];
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = min(c0 + j * threads, total - 1), i = c / padded, pc = c - i * padded;
      at[j] = i * row_bytes + pc * 16;
      v[j] = ldg16(x + (size_t)token(i) * H + min(pc, H / 8 - 1) * 8);
      if (pc >= H / 8) v[j] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4*>(rows + at[j]) = v[j];  // the last piece may repeat
  }
}

// ---------------------------------------------------------------------------
// Gate/up.  The row tiles of W13 of all runs form one list, cut into equal contiguous
// ranges, one per block (one block of 16 waves per CU), so a block meets few runs and
// copies each run's token rows into LDS once.  The 16 waves are four teams with a tile
// each; the waves of a team split K (bf16: wave w of 4 takes column steps w, w + 4, ...;
// MXFP4: an even number of consecutive steps, so that one scale word serves two) and
// stream their tiles through `bufs` register buffers of `units` weight fragments: loads run
// across tiles and runs, up to 8 KB in flight per wave, and nothing but weights goes
// through vector memory.  At the end of a turn (a tile per team) the block adds the parts
// in LDS (two buffers, one barrier per turn, which waits for no load), applies SwiGLU and
// writes h.  A W13 row tile holds 8 gate rows and the 8 up rows beside them.
//
// Two things shape the loops.  Every issue requests its loads, past the end from an empty
// buffer, which reads nothing: were they conditional, the wait for a fragment could not count
// the younger loads and would drain the pipeline.  And the code is kept short (few
// buffers, run descriptors ready in LDS, no division): a small launch pays for every
// line of instructions it fetches for the first time.
// ---------------------------------------------------------------------------
template <int WT>
struct GuTune {
  static constexpr int units = WT == W_BF16 ? 4 : 2, bufs = WT == W_BF16 ? 2 : 4;
};

// LDS: DlPlan, the parts of two tiles, the slot table with the gate weights and partial
// ranks, and the token rows.
constexpr int kDlRouting = (1024 + kDlMaxPairs + kDlWaves) * 4;
static int gu_row_bytes(int wtype, int H) { return (wtype == W_MXFP4 ? (H + 127) / 128 * 128 : H) * 2 + 16; }
static constexpr size_t kGuLds = 159 * 1024;  // of 160 KB: the workgroup vote takes a few bytes
static_assert(sizeof(DlPlan) + 2 * kDlWaves * 256 + kDlRouting + kDecodeLayerMaxH * 2 + 16 <= kGuLds, "one token row fits");
static size_t gu_red_bytes(int P) { return (size_t)2 * kDlWaves * 256 * ((P + 3) / 4); }

// Byte offsets and size of one expert's matrices (the slot layout of include/moe.h).
template <int WT>
struct ExpertShape {
  int n13, n2, c13, c2, s13, bytes;  // column steps; bytes of W13, W2 codes and W13 scales; the whole
  __device__ __forceinline__ ExpertShape(int H, int I) {
    n13 = ksteps<WT>(H);
    n2 = ksteps<WT>(I);
    c13 = 2 * I / 16 * n13 * 1024;
    c2 = H / 16 * n2 * 1024;
    s13 = WT == W_MXFP4 ? 2 * I / 16 * ((n13 + 15) / 16) * 1024 : 0;
    bytes = c13 + c2 + s13 + (WT == W_MXFP4 ? H / 16 * ((n2 + 15) / 16) * 1024 : 0);
  }
};

template <int WT, int U>
struct GuBuf {
  u32x4 w[U];
  uint32_t sc[U / 2];
};
static_assert(GuTune<W_MXFP4>::units % 2 == 0, "scale words serve pairs of steps");

// resident: all T token rows fit the LDS rows and are copied there once, beside the top-k.
template <int WT>
__global__ __launch_bounds__(kDlThreads) void decode_gate_up(DecodeLayerArgs a, int P, int P2, int row_bytes, bool resident, bool split) {
  constexpr int U = GuTune<WT>::units, B = GuTune<WT>::bufs;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  DlPlan& s = *reinterpret_cast<DlPlan*>(lds);
  float* red = reinterpret_cast<float*>(lds + sizeof(DlPlan));  // [buffer][element v][part][lane]
  const int red_tile = kDlWaves * 64 * ((P + 3) / 4);
  int32_t* slots = reinterpret_cast<int32_t*>(lds + sizeof(DlPlan) + (size_t)red_tile * 8);
  uint8_t* rows = reinterpret_cast<uint8_t*>(slots) + kDlRouting;
  const int lane = threadIdx.x & 63, g = lane >> 4, kp = uniform(threadIdx.x >> 6);
  const int n = a.T * a.k, p = threadIdx.x;
  uint64_t* masks = reinterpret_cast<uint64_t*>(red);  // until the first tile ends: 8 KB
  {
    const int my_slot = p < a.E ? a.slot_of_expert[p] : -1;  // E <= 1024 = kDlThreads
    float* w = reinterpret_cast<float*>(slots + 1024);
    if (a.logits) {
      if (a.E <= 64) dl_route<1>(s, w, a);
      else if (a.E <= 128) dl_route<2>(s, w, a);
      else if (a.E <= 256) dl_route<4>(s, w, a);
      else if (a.E <= 512) dl_route<8>(s, w, a);
      else dl_route<16>(s, w, a);
    } else if (p < n) {
      s.id[p] = a.ids[p];
    }
    if (p < a.E) {
      slots[p] = my_slot;
      masks[p] = 0;
    }
    if (resident) {  // few tokens: by the waves that have no top-k to do
      const int skip = a.T <= kDlWaves / 2 ? a.T * 64 : 0;
      if (p >= skip)
        copy_rows(rows, row_bytes, a.x, a.H, a.T, p - skip, kDlThreads - skip, [](int i) { return i; });
    }
    __syncthreads();
    if (a.logits && blockIdx.x == 0 && p < n) {
      a.ids[p] = s.id[p];
      a.w[p] = w[p];
    }
  }
  DlShared* out = blockIdx.x == 0 ? static_cast<DlShared*>(a.plan) : nullptr;
  const int runs =
      uniform(dl_plan(s, slots, masks, reinterpret_cast<uint32_t*>(slots + 1024 + kDlMaxPairs), a, P, P2, out));
  if (out && p < n) {
    out->sorted[p] = s.sorted[p];
    out->valid[p] = s.key[p] >= 0;
  }
  constexpr int teams = kDlTeams, parts = kDlWaves / teams;
  const int team = kp / parts, part = kp % parts;
  const int sh_runs = a.shared_w ? (a.T + P - 1) / P : 0;
  const int sh_tiles = a.I_shared / 8, rt_tiles = a.I / 8;
  const int sh_turns = (sh_tiles + teams - 1) / teams, rt_turns = (rt_tiles + teams - 1) / teams;
  const int sh_total = sh_runs * sh_turns, total = sh_total + (runs - sh_runs) * rt_turns;
  const int lo = (int)((int64_t)blockIdx.x * total / gridDim.x), hi = (int)((int64_t)(blockIdx.x + 1) * total / gridDim.x);
  if (lo >= hi) return;
  const ExpertShape<WT> rt(a.H, a.I), sh(a.H, a.I_shared);
  // column steps, units and chunks of units of a wave's tile
  const int nk = rt.n13, nu = (nk + parts - 1) / parts, nc = (nu + U - 1) / U;
  const int step0 = WT == W_MXFP4 ? part * nc * U : part, step_by = WT == W_MXFP4 ? 1 : parts;
  const int run0 = lo < sh_total ? lo / max(sh_turns, 1) : sh_runs + (lo - sh_total) / rt_turns;
  const int turn0 = lo < sh_total ? lo - run0 * sh_turns : lo - sh_total - (run0 - sh_runs) * rt_turns;

  // Issue side: the next chunk to request.
  int iq = lo, ic = 0, irun = run0 - 1, itile = turn0 * teams + team, iper = 0, isc = 0;
  const uint8_t* iw = nullptr;
  int ibytes = 0;
  auto issue_run = [&]() {
    ++irun;
    const bool shared = irun < sh_runs;
    iw = read_run(s.run + irun).w;
    ibytes = shared ? sh.bytes : rt.bytes;
    iper = shared ? sh_tiles : rt_tiles;
    isc = shared ? sh.c13 + sh.c2 : rt.c13 + rt.c2;
  };
  issue_run();
  auto issue = [&](GuBuf<WT, U>& b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = step0 + (ic * U + u) * step_by;
      const bool live = iq < hi && step < nk && itile < iper;
      const __amdgpu_buffer_rsrc_t buf = make_rsrc(iw, live ? ibytes : 0);
      b.w[u] = bld16(buf, lane * 16, live ? (itile * nk + step) * 1024 : 0);
      if constexpr (WT == W_MXFP4)  // steps in pairs from an even one: one word
        if (u % 2 == 0)
          b.sc[u / 2] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
              buf, lane * 16, live ? isc + (itile * ((nk + 15) / 16) + step / 16) * 1024 + step % 16 / 4 * 4 : 0, 0);
    }
    if (++ic == nc) {
      ic = 0;
      ++iq;
      itile += teams;
      if (itile - team >= iper && iq < hi) {
        itile = team;
        issue_run();
      }
    }
  };
  GuBuf<WT, U> buf[B];
#pragma unroll
  for (int b = 0; b < B; ++b) issue(buf[b]);

  // Compute side.
  int q = lo, cc = 0, run = run0 - 1, tile = turn0 * teams + team, per = 0, at = 0, m = 0, half = 0;
  const uint8_t* my_row = rows;
  auto enter_run = [&]() {  // the token rows of the next run into LDS
    ++run;
    const RunRef r = read_run(s.run + run);
    at = r.at;
    m = r.m;
    per = run < sh_runs ? sh_tiles : rt_tiles;
    auto token = [&](int i) { return run < sh_runs ? at + i : s.sorted[at + i] / a.k; };
    const int i = min(a_token(lane), m - 1);
    if (resident) {
      my_row = rows + token(i) * row_bytes;
      return;
    }
    copy_rows(rows, row_bytes, a.x, a.H, m, p, kDlThreads, token);
    my_row = rows + i * row_bytes;
    lds_barrier();
  };
  enter_run();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (;;) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int step = step0 + (cc * U + u) * step_by;
        if (step < nk) {  // a team without a tile multiplies zeros
          if constexpr (WT == W_BF16) {
            acc = mfma16(*reinterpret_cast<const u32x4*>(my_row + step * 64 + 16 * g), as_bf16x8(buf[b].w[u]), acc);
          } else {
            const float sc = scale_of_word(buf[b].sc[u / 2], step);
#pragma unroll
            for (int f = 0; f < 4; ++f)
              acc = mfma16(*reinterpret_cast<const u32x4*>(my_row + step * 256 + 64 * g + 16 * f),
                           fp4x8_to_bf16x8(buf[b].w[u][f], sc), acc);
          }
        }
      }
      issue(buf[b]);
      if (++cc < nc) continue;
      cc = 0;
      float* sums = red + half * red_tile;
      const int nv = (m + 3) / 4;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v < nv) sums[(v * kDlWaves + kp) * 64 + lane] = acc[v];
      acc = f32x4{0.f, 0.f, 0.f, 0.f};
      lds_barrier();
      // element v of a team's tile by wave v + nv (team + teams q) of the 16: lane =
      // (token % 4, stored row)
      const int unit = (kp - q * nv * teams) & (kDlWaves - 1);
      if (unit < nv * teams) {
        const int tm = unit / nv, v = unit - tm * nv, tl = tile - team + tm;
        const float* src = sums + (v * kDlWaves + tm * parts) * 64 + lane;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < parts; ++w) sum += src[w * 64];
        const float up = __shfl_xor(sum, 8, 64);
        const int i = g + 4 * v;
        if (i < m && (lane & 8) == 0 && tl < per) {
          const int row = run < sh_runs ? n + at + i : s.sorted[at + i];
          uint16_t* h = a.h + (size_t)row * (a.h_ld << split) + (lane & 7);
          const float hv = silu_f32(sum) * up;
          const uint16_t hi = f32_to_bf16_rne(hv);
          h[tl * 8] = hi;
          if (split) {  // an infinite or NaN h has no remainder
            const float rest = hv - bf16_bits_to_f32(hi);
            h[a.h_ld + tl * 8] = fabsf(rest) < INFINITY ? f32_to_bf16_rne(rest) : 0;
          }
          if (WT == W_MXFP4 && tl + 1 == per)  // zeros up to the next whole column step
            for (int z = per * 8; z % 128; z += 8) {
              h[z] = 0;
              if (split) h[a.h_ld + z] = 0;
            }
        }
      }
      half ^= 1;
      if (++q >= hi) return;
      tile += teams;
      if (tile - team >= per) {
        tile = team;
        enter_run();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Down and combine.  A block owns one row tile of W2 (16 columns of y) for every pair.
// K is cut into `parts` (a power of two up to 16): wave w takes part w % parts of the runs
// w / parts, w / parts + 16 / parts, ... and streams them (weights, and the run's h
// fragments, which come from L2) without meeting the others; the parts of all pairs
// collect in LDS, and the block adds the parts, then each token's pairs in ascending j.
//
// The vector memory pipe, not HBM, is what a 4-bit stream runs into here (an h fragment
// for every 256 bytes of codes: with four fragment loads and a scale load beside each code
// load the MXFP4 kernel took 86 us at 64 tokens, without them 28; now 62).  Runs are
// therefore short, and a load brings four fragments of 4 rows of h: lane j of a quad, where all
// four would hold the same row, loads its fragment j, so that a load reads whole 64-byte
// pieces (256 consecutive bytes of a row for MXFP4).  Such an operand goes into the products
// of all its fragments' weights as it is: of row 4 i + j of a product only fragment j means
// something, so fragment f adds up in an accumulator of its own, whose element f is the
// row's sum.  A run has 8 rows: 8 tokens, or (SPLIT) 4 tokens and the remainders of their h,
// which add to the same accumulators.
//
// HALF: a block owns 8 columns of y, half a row tile (H / 8 blocks where H / 16 would leave
// CUs idle, as long as the half tiles are one round of blocks: bf16 layer of 16 tokens at
// H = 2048 140 -> 130 us, but MXFP4 layer of 53 tokens at H = 2592 55 -> 70 us).  One 1 KB load
// then holds the 8 rows at two steps, rows at the even step as operand columns 0-7 and at the odd
// one as columns 8-15, and the quads of lanes hold two rows of h at both steps: rows 4 i and
// 4 i + 1 of the result are right in columns 0-7, rows 4 i + 2 and 4 i + 3 in columns 8-15
// (the other products mean nothing), and the two halves add up.  An h load serves half as
// many weights, so this is for blocks that would be too few otherwise.
template <int WT, bool HALF, bool SPLIT>
struct DnTune {
  static constexpr int units = WT == W_BF16 ? 4 : 2;                // steps of a chunk
  static constexpr int wloads = HALF ? units / 2 : units;           // code loads of a chunk
  static constexpr int groups = HALF || WT == W_BF16 ? 1 : 2;       // groups of h loads
  static constexpr int hloads = HALF && WT == W_MXFP4 ? 4 : 2;      // h loads of a group
  static constexpr int bufs = HALF || SPLIT || WT == W_BF16 ? 3 : 2;  // what the registers of 16 waves hold
};

template <int WT, bool HALF, bool SPLIT>
struct DnBuf {
  using Tune = DnTune<WT, HALF, SPLIT>;
  u32x4 w[Tune::wloads], h[Tune::groups][Tune::hloads];
  uint32_t sc;
};

template <int WT, bool HALF, bool SPLIT, bool BF16OUT>
__global__ __launch_bounds__(kDlThreads) void decode_down(DecodeLayerArgs a, int log_parts) {
  using Tune = DnTune<WT, HALF, SPLIT>;
  constexpr int U = Tune::units, NG = Tune::groups, NH = Tune::hloads, B = Tune::bufs, P = SPLIT ? 4 : 8;
  constexpr int COLS = HALF ? 8 : 16, NA = HALF ? 1 : 4;           // columns of y; fragments' accumulators
  constexpr int NR = HALF ? 1 : 2, NS = HALF || SPLIT ? 1 : 2;     // rows a lane reads; sets of accumulators
  __shared__ DlShared s;
  __shared__ float w[kDlMaxPairs];
  extern __shared__ float val[];  // [part][pair, then shared token][COLS]
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, wv = uniform(threadIdx.x >> 6);
  const int n = a.T * a.k, nrows = n + (a.shared_w ? a.T : 0), p = threadIdx.x;
  const int sh_runs = a.shared_w ? (a.T + P - 1) / P : 0;
  const int tile = HALF ? blockIdx.x >> 1 : blockIdx.x;
  const DlShared* in = static_cast<const DlShared*>(a.plan);
  const int runs = in->runs;
  {
    const int pr = min(p, n + sh_runs - 1), pp = min(p, n - 1);  // all loads at once, none conditional
    const u32x4 r = ldg16(in->run + pr);
    const int so = in->sorted[pp], va = in->valid[pp];
    const float wp = a.w[pp];
    if (p < n + sh_runs) *reinterpret_cast<u32x4*>(s.run + p) = r;
    if (p < n) {
      s.sorted[p] = so;
      s.valid[p] = va;
      w[p] = wp;
    }
  }
  __syncthreads();
  const int h_row = (a.h_ld << SPLIT) * 2, hbytes = nrows * h_row;
  const ExpertShape<WT> rt(a.H, a.I), sh(a.H, a.I_shared);
  const int parts = 1 << log_parts, part = wv & (parts - 1), stride = kDlWaves >> log_parts;
  // a part is whole chunks of U steps
  auto part_steps = [&](int nk, int& from, int& to) {
    const int chunks = (nk + U - 1) / U;
    from = (part * chunks >> log_parts) * U;
    to = min(((part + 1) * chunks >> log_parts) * U, nk);
  };
  // this lane's fragment of a tile, and (HALF) the step it takes of a pair
  const int frag = HALF ? 16 * g + 8 * (blockIdx.x & 1) + (c & 7) : lane;
  const int w_step = HALF ? c >> 3 : 0, j = lane & 3, h_step = HALF ? j >> 1 : 0;
  const int w_off = frag * 16 + w_step * 1024;

  // Issue side: run ir, steps is .. ie-1 of it.
  int ir = (wv >> log_parts) - stride, is = 0, ie = 0, i_row[NR], i_w2 = 0, i_sc = 0;
  const uint8_t* iw = nullptr;
  int ibytes = 0;
  auto issue_run = [&]() {
    ir += stride;
    const int r0 = min(ir, runs - 1);
    const bool shared = r0 < sh_runs;
    const RunRef r = read_run(s.run + r0);
    const int nk = shared ? sh.n2 : rt.n2;
    iw = r.w;
    ibytes = shared ? sh.bytes : rt.bytes;
    i_w2 = (shared ? sh.c13 : rt.c13) + tile * nk * 1024;
    i_sc = (shared ? sh.c13 + sh.c2 + sh.s13 : rt.c13 + rt.c2 + rt.s13) + tile * ((nk + 15) / 16) * 1024;
    part_steps(nk, is, ie);
    #pragma unroll
    for (int l = 0; l < NR; ++l) {
      // tokens 0-3, and tokens 4-7 (SPLIT: the remainders of the first)
      const int second = HALF ? j & 1 : l, i = min((c >> 2) + (SPLIT ? 0 : 4 * second), r.m - 1);
      i_row[l] = (shared ? n + r.at + i : s.sorted[r.at + i]) * h_row + (SPLIT ? second * a.h_ld * 2 : 0) +
                 (WT == W_MXFP4 ? 64 : 16) * g;
    }
  };
  auto issue = [&](DnBuf<WT, HALF, SPLIT>& b) {
#pragma unroll
    for (int u = 0; u < U; u += HALF ? 2 : 1) {
      const int step = is + u;
      const bool live = ir < runs && step < ie;
      const __amdgpu_buffer_rsrc_t wbuf = make_rsrc(iw, live ? ibytes : 0), hbuf = make_rsrc(a.h, live ? hbytes : 0);
      // HALF, an odd number of steps: the lanes of the missing one read nothing
      const bool pair = !HALF || step + 1 < ie;
      b.w[HALF ? u / 2 : u] = bld16(wbuf, pair || w_step == 0 ? w_off : kPastEnd, live ? i_w2 + step * 1024 : 0);
      if constexpr (WT == W_MXFP4)
        if (u == 0)
          b.sc = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
              wbuf, frag * 16, live ? i_sc + step / 16 * 1024 + step % 16 / 4 * 4 : 0, 0);
      const int hs = live ? step * (WT == W_MXFP4 ? 256 : 64) : 0;
      if constexpr (HALF && WT == W_BF16) {
        b.h[0][u / 2] = bld16(hbuf, pair || h_step == 0 ? i_row[0] + 64 * h_step : kPastEnd, hs);
      } else if constexpr (HALF) {
#pragma unroll
        for (int f = 0; f < 4; ++f)
          b.h[0][f] = bld16(hbuf, pair || h_step == 0 ? i_row[0] + 256 * h_step + 16 * f : kPastEnd, hs);
      } else if (u < NG) {
        // fragment j (bf16: 64 bytes a step; MXFP4: 16 bytes)
#pragma unroll
        for (int l = 0; l < NH; ++l) b.h[u][l] = bld16(hbuf, i_row[l] + (WT == W_MXFP4 ? 16 : 64) * j, hs);
      }
    }
    is += U;
    if (is >= ie && ir < runs) issue_run();
  };
  int cr = wv >> log_parts, cs = 0, ce = 0, at = 0, m = 0;
  if (cr < runs) {
    auto enter_run = [&]() {
      const RunRef r = read_run(s.run + cr);
      at = r.at;
      m = r.m;
      part_steps(cr < sh_runs ? sh.n2 : rt.n2, cs, ce);
    };
    DnBuf<WT, HALF, SPLIT> buf[B];
    issue_run();
#pragma unroll
    for (int b = 0; b < B; ++b) issue(buf[b]);
    enter_run();
    f32x4 acc[NS][NA];
    auto clear = [&]() {
#pragma unroll
      for (int l = 0; l < NS; ++l)
#pragma unroll
        for (int f = 0; f < NA; ++f) acc[l][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    clear();
    for (bool more = true; more;) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const DnBuf<WT, HALF, SPLIT>& k = buf[b];
        if constexpr (HALF && WT == W_BF16) {
          acc[0][0] = mfma16(k.h[0][0], as_bf16x8(k.w[0]), acc[0][0]);
          if (cs + 2 < ce) acc[0][0] = mfma16(k.h[0][1], as_bf16x8(k.w[1]), acc[0][0]);
        } else if constexpr (HALF) {
          const float sc = e8m0_to_f32(k.sc >> (8 * ((cs & 3) + w_step)) & 0xffu);
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[0][0] = mfma16(k.h[0][f], fp4x8_to_bf16x8(k.w[0][f], sc), acc[0][0]);
        } else if constexpr (WT == W_BF16) {
#pragma unroll
          for (int f = 0; f < 4; ++f)
            if (f == 0 || cs + f < ce)
#pragma unroll
              for (int l = 0; l < NR; ++l) acc[l % NS][f] = mfma16(k.h[0][l], as_bf16x8(k.w[f]), acc[l % NS][f]);
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (cs + u < ce) {
              const float sc = scale_of_word(k.sc, cs + u);
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const bf16x8 wf = fp4x8_to_bf16x8(k.w[u][f], sc);
#pragma unroll
                for (int l = 0; l < NR; ++l) acc[l % NS][f] = mfma16(k.h[u][l], wf, acc[l % NS][f]);
              }
            }
          }
        }
        issue(buf[b]);
        cs += U;
        if (cs < ce) continue;
#pragma unroll
        for (int v = 0; v < (SPLIT ? 1 : 2); ++v) {
          float d;
          if constexpr (HALF) {
            d = c < 8 ? acc[0][0][v] : acc[0][0][v + 2];
            if constexpr (SPLIT) d += c < 8 ? acc[0][0][1] : acc[0][0][3];
            d += __shfl_xor(d, 8, 64);
          } else {
            d = acc[v % NS][0][0];
#pragma unroll
            for (int f = 1; f < NA; ++f) d += acc[v % NS][f][f];
          }
          const int i = g + 4 * v;
          if (i < m && c < COLS) {
            const int row = cr < sh_runs ? n + at + i : s.sorted[at + i];
            val[(part * nrows + row) * COLS + c] = d;
          }
        }
        clear();
        cr += stride;
        more = cr < runs;
        if (!more) break;
        enter_run();
      }
    }
  }
  __syncthreads();
  if (parts > 1) {
    for (int o = threadIdx.x; o < nrows * COLS; o += kDlThreads) {
      float d = val[o];
#pragma unroll 4
      for (int q = 1; q < parts; ++q) d += val[q * nrows * COLS + o];
      val[o] = d;
    }
    __syncthreads();
  }
  for (int o = threadIdx.x; o < a.T * COLS; o += kDlThreads) {
    const int tk = o / COLS, col = o % COLS;
    float y = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < a.k; j0 += 4) {  // four pairs' LDS reads at a time
      float d[4], wj[4];
      int ok[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pr = tk * a.k + min(j0 + j, a.k - 1);
        ok[j] = j0 + j < a.k ? s.valid[pr] : 0;
        wj[j] = w[pr];
        d[j] = val[pr * COLS + col];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ok[j]) y = fmaf(wj[j], d[j], y);
    }
    if (a.shared_w) y += val[(n + tk) * COLS + col];
    const size_t out = (size_t)tk * a.H + blockIdx.x * COLS + col;
    if (BF16OUT)
      static_cast<uint16_t*>(a.y)[out] = f32_to_bf16_rne(y);
    else
      static_cast<float*>(a.y)[out] = y;
  }
}

template <int WT, bool HALF, bool SPLIT>
static hipError_t launch_down(const DecodeLayerArgs& a, bool bf16_out, hipStream_t st) {
  // K parts of the down product: enough (run, part) tasks for the waves when every pair is
  // a run of its own, each part at least one chunk of steps long, and LDS for the parts
  constexpr int COLS = HALF ? 8 : 16;
  const int nrows = a.T * a.k + (a.shared_w ? a.T : 0);
  const int ks = (WT == W_MXFP4 ? 128 : 32) * DnTune<WT, HALF, SPLIT>::units;
  int chunks = (a.I + ks - 1) / ks;
  if (a.shared_w && (a.I_shared + ks - 1) / ks < chunks) chunks = (a.I_shared + ks - 1) / ks;
  int lp = 0;
  while (lp < 4 && 2 << lp <= chunks && nrows << lp < 64 && (size_t)(nrows << lp) * COLS * 8 <= 65536) ++lp;
  const size_t lds = (size_t)(nrows << lp) * COLS * 4;
  const dim3 grid(a.H / COLS), block(kDlThreads);
  if (bf16_out)
    hipLaunchKernelGGL((decode_down<WT, HALF, SPLIT, true>), grid, block, lds, st, a, lp);
  else
    hipLaunchKernelGGL((decode_down<WT, HALF, SPLIT, false>), grid, block, lds, st, a, lp);
  return hipGetLastError();
}

template <int WT>
static hipError_t launch_t(const DecodeLayerArgs& a, bool bf16_out, hipStream_t st) {
  const int n = a.T * a.k;
  const int rb = gu_row_bytes(WT, a.H);
  int P = 16;
  while (P > 1 && sizeof(DlPlan) + gu_red_bytes(P) + kDlRouting + (size_t)P * rb > kGuLds) --P;
  const bool resident = a.T <= P;
  if (P > a.T) P = a.T;  // a token routes to an expert once, unless the caller's routing repeats it
  const size_t lds = sizeof(DlPlan) + gu_red_bytes(P) + kDlRouting + (size_t)P * rb;
  const int64_t sh_turns = (a.I_shared / 8 + kDlTeams - 1) / kDlTeams, rt_turns = (a.I / 8 + kDlTeams - 1) / kDlTeams;
  const int64_t bound = (a.shared_w ? (a.T + P - 1) / P * sh_turns : 0) + n * rt_turns;  // every pair a run
  const unsigned grid = (unsigned)(bound < 256 ? bound : 256);
  const bool half = a.H / 16 <= kDlHalfTiles;
  const bool split = a.T <= kDlSplitT;
  hipLaunchKernelGGL(decode_gate_up<WT>, dim3(grid), dim3(kDlThreads), lds, st, a, P, split ? 4 : 8, rb, resident, split);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (half) return split ? launch_down<WT, true, true>(a, bf16_out, st) : launch_down<WT, true, false>(a, bf16_out, st);
  return split ? launch_down<WT, false, true>(a, bf16_out, st) : launch_down<WT, false, false>(a, bf16_out, st);
}

hipError_t launch_decode_layer(int wtype, const DecodeLayerArgs& a, bool bf16_out, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  return wtype == W_BF16 ? launch_t<W_BF16>(a, bf16_out, st) : launch_t<W_MXFP4>(a, bf16_out, st);
}

}  // namespace moe
