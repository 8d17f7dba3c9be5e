/*
 * moe.h -- C ABI of the MI355X (gfx950) routed-expert MoE layer library, libmoe.so.
 *
 * One MoE layer's routed-expert forward pass, as the hot path of the edge MoE
 * serving engine described in "Meet FreeToken: An Edge-Native MoE Serving Engine
 * that Runs 753B GLM-5.2 on a Single Workstation GPU" (MarkTechPost):
 *
 *   moe_route_topk         top-k gating over router logits
 *   moe_permute            stable permutation of (token, choice) pairs by expert
 *   moe_cache_lookup_fill  global-LRU expert-slot cache in HBM, filled from pinned host memory
 *                          (moe_cache_lookup_fill_split + moe_cache_wait_fills: hits computed during fills)
 *   moe_grouped_ffn        grouped SwiGLU expert FFN (f32, bf16 or MXFP4 weights)
 *   moe_combine            gate-weighted merge of the expert outputs
 *   moe_layer_decode       all of the above for a few tokens in two kernels
 *   moe_layer_stream_*     whole-layer double buffering for prefill
 *   moe_w4_linear          linear product with 4-bit weights and group scales
 *   moe_linear             linear product with f32 or bf16 weights, bias, activation and residual
 *   moe_block_norm         norms before and after a block with its gate and residual
 *   moe_dispatch           token rows sorted by expert; moe_combine_rows: and back, with weights;
 *                          their gradients and the gate's: moe_..._backward
 *
 * Conventions
 *  - Pointers are device pointers unless the name ends in _host.
 *  - Every call returns a moe_status; nothing throws, aborts or exits.  On failure
 *    moe_last_error() holds a message for the calling thread.
 *  - Calls that take a hipStream_t are asynchronous on it, except
 *    moe_cache_lookup_fill(_split) for wave 0 (it waits for the step's expert counts).
 *  - The caller owns every buffer and stream.  The library owns only the opaque
 *    handles (host metadata and HIP events) and allocates no device memory on the
 *    hot path: scratch comes from the caller through moe_grouped_ffn_workspace().
 *  - Device buffers must be 16-byte aligned.
 *  - Shapes: 1 <= E <= 1024, 1 <= k <= min(E, 32), T >= 0, T*k < 2^31,
 *    H and I multiples of 32 for bf16/MXFP4 weights (multiples of 4 for f32).
 *  - Logits must be finite; a NaN logit makes the selection unspecified.
 *
 * Expert slot layout (one expert = one contiguous run of moe_expert_bytes(); the
 * host pool stores experts in this final layout so that a fill is one copy):
 *    f32   :  W13 [2I][H] then W2 [H][I], row-major (rows K-contiguous);
 *             W13 rows 0..I-1 are the gate projection, I..2I-1 the up projection
 *    bf16  :  W13 (2I rows, K = H) then W2 (H rows, K = I), both tiled
 *    MXFP4 :  W13 codes, W2 codes, W13 scales, W2 scales, all tiled
 *  Tiled matrix (R rows, K columns): tiles of 16 rows x KS columns (KS = 32 for
 *  bf16, 128 for MXFP4; K rounded up to a multiple of KS with zero padding),
 *  stored row-tile major then column step; each tile is 64 fragments of 16 bytes
 *  in the order f = 16*g + row%16 with g = (k % KS) / (KS/4): a bf16 fragment is 8
 *  consecutive k, an MXFP4 fragment one 32-element block (OCP MX v1.0 E2M1,
 *  element 2i in the low nibble of byte i).  This is the operand order of the
 *  bf16 MFMA, so a wave reads 1 KB of contiguous memory per load.  MXFP4 E8M0
 *  scales: per row tile the column steps are grouped 16 at a time into 1 KB scale
 *  blocks (the last one padded), row-tile major; in a block, fragment f owns bytes
 *  16f .. 16f+15, byte i being its scale at step 16*block + i, so one 16-byte load
 *  per lane brings its scales for 16 steps.  For bf16 and MXFP4, stored W13
 *  row 16t+q is gate row 8t+q for q < 8 and up row 8t+q-8 otherwise.  W2 is the
 *  down projection.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 1

typedef enum {
  MOE_OK = 0,
  MOE_EINVAL = 1,         /* bad argument (shape, null or misaligned pointer, range) */
  MOE_EUNSUPPORTED = 2,   /* valid request this build does not implement */
  MOE_ECAPACITY = 3,      /* workspace or buffer too small */
  MOE_EHIP = 4,           /* a HIP runtime call or kernel launch failed */
  MOE_ENOMEM = 5,         /* host allocation failed */
  MOE_ESTATE = 6          /* call out of order (e.g. wave w before wave w-1) */
} moe_status;

/* MOE_MXFP4_A8: MXFP4 weights (the MOE_MXFP4 slot layout) with the gate/up
 * activations quantized to MXFP8 (OCP MX v1.0: E4M3 elements, one E8M0 scale per
 * 32 consecutive elements of a token row, X = floor(log2 max|x|) - 8, round to
 * nearest even, clamp to 448) and multiplied on the scaled FP4 x FP8 MFMA; the
 * down projection stays on the exact path (bf16 intermediate).  A precision
 * trade for prefill throughput (the pages' 8,192-token prefill chunks, "Data Check"
 * claim table, Fig 4a row); the other types never lower activation precision. */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_MXFP4 = 2, MOE_MXFP4_A8 = 3 } moe_dtype;

int moe_abi_version(void);
const char* moe_status_str(int status);
const char* moe_last_error(void);

/* Bytes of one expert slot of the given weight type (0 for invalid shapes). */
size_t moe_expert_bytes(int wdt, int H, int I);

/* ------------------------------------------------------------------------- */
/* Top-k gating.  The pages: the model's own routing decides which experts run
 * and the engine leaves it unchanged ("Three mechanisms": bandwidth-adaptive execution; "Key Takeaways").
 * For each token t: the k experts with the largest f32 logits, in descending
 * logit order, equal logits (IEEE equality, -0.0 == +0.0) going to the lower
 * expert index; gate weights are the softmax over the k selected logits (equal,
 * in exact arithmetic, to softmax over all E renormalised over the selection),
 * computed in f32.
 *   logits   [T][E] f32          (read)
 *   topk_ids [T][k] int32        (written)  expert ids, bit-exact
 *   topk_w   [T][k] f32          (written)  gate weights, sum to 1 within rounding */
int moe_route_topk(const float* logits, int T, int E, int k, int32_t* topk_ids, float* topk_w,
                   hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Permutation by expert (the grouping step between routing and the grouped FFN;
 * the pages route each token to its experts, "The gap it targets").  Stable
 * counting sort of the pairs r = t*k + j by topk_ids[r]:
 *   counts      [E]    pairs per expert
 *   offsets     [E+1]  exclusive prefix sum, offsets[E] = T*k
 *   sorted_rows [T*k]  r grouped by expert, ascending r within an expert
 *   inv_rows    [T*k]  position of r in sorted_rows
 * Deterministic, bit-exact.  topk_ids values must lie in [0, E). */
int moe_permute(const int32_t* topk_ids, int T, int k, int E, int32_t* counts, int32_t* offsets,
                int32_t* sorted_rows, int32_t* inv_rows, hipStream_t stream);

/* moe_route_topk followed by moe_permute on the same buffers, with the same
 * arguments, requirements and results; batches of at most 8 tokens run as one
 * workgroup launch (one launch fewer per decode layer). */
int moe_route(const float* logits, int T, int E, int k, int32_t* topk_ids, float* topk_w, int32_t* counts,
              int32_t* offsets, int32_t* sorted_rows, int32_t* inv_rows, hipStream_t stream);

/* Router projection then moe_route: logits[t][e] = sum_h x[t][h] * w_router[e][h]
 * (x [T][H] and w_router [E][H] bf16, f32 accumulation in a fixed order, written
 * to logits [T][E] f32), then top-k gating and the permutation on those logits
 * exactly as moe_route.  H a positive multiple of 8.  The pages leave the model's
 * router as it is ("Three mechanisms", bandwidth-adaptive execution); the plain
 * linear gate of an MoE layer is computed.  Selections follow the f32 logits, so
 * they can differ from an exact-arithmetic selection only where two logits are
 * within the summation error of each other. */
int moe_route_project(const void* x, const void* w_router, int T, int H, int E, int k, float* logits,
                      int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* sorted_rows,
                      int32_t* inv_rows, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Expert-slot cache.  The pages: experts that are not in use are kept in host
 * memory and brought to the GPU only when a token is routed to them ("The gap it
 * targets"); in decode, one recency-ordered cache whose keys cover every MoE
 * layer decides which experts stay on the GPU, driven by what the router picks
 * ("Three mechanisms": semantic-aware caching); host copies of the experts are
 * pinned in the layout the GPU computes from, and serving begins with nothing
 * cached ("Three mechanisms": elastic memory management).
 *
 * Keys are (layer, expert), key = layer*n_experts + expert.  The cache starts
 * empty.  For one (step, layer) the active experts (counts > 0) are accessed
 * hits first, then misses, each group in ascending expert id, hit or miss judged
 * against the state before the step; a miss takes the lowest-index free slot,
 * else evicts the least recently used key.  If more experts are active than
 * there are slots, the accesses run in waves of n_slots: the caller runs the FFN
 * of wave w before asking for wave w+1.  The shared expert is never cached. */
typedef struct moe_cache moe_cache;

typedef struct {
  int n_layers;
  int n_experts;
  int n_slots;
  size_t expert_bytes;  /* bytes copied per fill */
  size_t slot_stride;   /* bytes between slots in slot_pool; >= expert_bytes, multiple of 256 */
  void* slot_pool;      /* device, n_slots*slot_stride bytes; NULL = host-only planning handle */
  const void* host_pool_host;               /* pinned, key-major, expert_bytes per key */
  const void* const* host_expert_ptrs_host; /* optional [n_layers*n_experts] pinned pointers; overrides host_pool_host */
  hipStream_t fill_stream;                  /* side stream the fills run on (device handles) */
} moe_cache_desc;

typedef struct {
  int64_t accesses;     /* distinct active experts of the step (all waves) */
  int64_t hits;
  int64_t misses;
  int64_t cold_misses;  /* misses of keys never accessed before */
  int64_t fill_bytes;   /* bytes copied by this call */
  int32_t n_waves;      /* waves this step needs */
  int32_t wave_accesses;/* accesses in the wave this call handled */
  int64_t inplace;      /* misses of the step computed in place (miss split), not filled */
} moe_cache_stats;

typedef struct {
  int32_t slot;
  int32_t layer;
  int32_t expert;
  int32_t wave;
} moe_fill;

int moe_cache_create(const moe_cache_desc* desc, moe_cache** out);
/* Waits for the handle's in-flight fills, then frees it. */
int moe_cache_destroy(moe_cache* c);

/* Device handle.  counts: device [n_experts] (moe_permute output).  For wave 0
 * the counts are copied to the host and the call waits for them (the only host
 * synchronisation of the layer); waves 1.. must follow in order, each after the
 * FFN of the previous wave has been enqueued on compute_stream.  Writes
 * slot_of_expert (device [n_experts]): the slot of each expert in this wave, -1
 * for the rest.  Fills run on the fill stream after all work enqueued on
 * compute_stream so far (write-after-read on victim slots); compute_stream then
 * waits for them (read-after-write).  stats_host (nullable) receives the
 * counters.  On error no key maps to a slot whose bytes may have been
 * overwritten; the rest of the state is as before the call. */
int moe_cache_lookup_fill(moe_cache* c, int layer, const int32_t* counts, int wave,
                          int32_t* slot_of_expert, moe_cache_stats* stats_host, hipStream_t compute_stream);

/* Split lookup, for computing the resident experts while the misses stream in
 * (the pages: the GPU keeps computing what it holds while missing experts are
 * transferred, "Three mechanisms", bandwidth-adaptive execution).  Same plan,
 * fills, ordering of waves and errors as moe_cache_lookup_fill, but two device
 * tables [n_experts] are written on compute_stream: slot_hits holds the slots of
 * the wave's hits (-1 elsewhere) and may be used at once, since hits are never
 * victims of the wave's misses; slot_misses holds the slots of the wave's filled
 * experts (-1 elsewhere) and may be used only after moe_cache_wait_fills.  The
 * caller runs the FFN over slot_hits, then moe_cache_wait_fills, then the FFN over
 * slot_misses (skipped when stats->fill_bytes is 0); the two FFNs write disjoint
 * output rows, so the layer equals the unsplit one bit for bit.  Both pointers
 * must be 16-byte aligned and distinct. */
int moe_cache_lookup_fill_split(moe_cache* c, int layer, const int32_t* counts, int wave, int32_t* slot_hits,
                                int32_t* slot_misses, moe_cache_stats* stats_host, hipStream_t compute_stream);
/* Miss split (the pages: of a step's misses, a share set by the host-link and
 * host-memory bandwidths crosses into GPU memory and the rest is computed where
 * the weights already are, the partial sums merging exactly; "Three mechanisms",
 * bandwidth-adaptive execution).  On one GPU "where the weights are" is pinned
 * host memory read by the GPU in place.  With fill fraction num/den, of a step's
 * m misses (ascending expert id) the first floor(m*num/den + 1/2) are filled as
 * usual and the others are computed in place: they take no slot, evict nothing
 * and leave the recency order as it is (hits are still refreshed).  Default 1/1
 * (every miss filled).  Between steps only (MOE_ESTATE otherwise);
 * 0 <= num <= den, den >= 1. */
int moe_cache_set_fill_fraction(moe_cache* c, int num, int den);
/* moe_cache_lookup_fill_split plus the step's in-place experts: addr_inplace
 * (device [n_experts] uint64, 16-byte aligned) receives, with wave 0, the
 * device-visible address of the pinned host copy of each in-place expert of the
 * step (0 for every other expert, and everywhere for later waves), for
 * moe_grouped_ffn_addr.  The host copies must be pinned memory the GPU can read
 * (hipHostMalloc).  Same ordering rules as the split lookup; the in-place FFN can
 * run while the fills are in flight (it reads only host memory). */
int moe_cache_lookup_fill_inplace(moe_cache* c, int layer, const int32_t* counts, int wave, int32_t* slot_hits,
                                  int32_t* slot_misses, uint64_t* addr_inplace, moe_cache_stats* stats_host,
                                  hipStream_t compute_stream);
/* The in-place experts of the last step begun (ascending id); experts_host has
 * room for n_experts.  Works on host-only and device handles. */
int moe_cache_step_inplace(const moe_cache* c, int32_t* experts_host, int* n_host);

/* Elastic resize of the slot pool (the pages: the expert pool grows and shrinks
 * with the memory the GPU can spare, "Three mechanisms", elastic memory
 * management).  Between steps only (MOE_ESTATE while a step's waves are open):
 * keeps the min(n_slots, resident) most recently used keys, most recent first in
 * new slots 0, 1, ..., with their recency; the others are dropped (later accesses
 * miss).  Nothing is read from the host pool.  Device handle: slot_pool is the new
 * pool (256-byte aligned, n_slots * slot_stride bytes, stride >= expert_bytes and a
 * multiple of 256, not overlapping the current pool); in-flight fills are waited
 * for, then each kept expert is copied from its old slot on `stream` (after the
 * work already on it); the next lookup makes its compute stream, and through it
 * its fills, wait for those copies, so `stream` may differ from the compute
 * stream; the caller may free the old pool once that work is done.  Host-only handle:
 * slot_pool must be NULL.  moved_from_host (nullable, [n_slots]) receives the old
 * slot of each new slot's expert, -1 for an empty slot.  On error the cache is
 * unchanged. */
int moe_cache_resize(moe_cache* c, int n_slots, void* slot_pool, size_t slot_stride, int32_t* moved_from_host,
                     hipStream_t stream);
/* Makes compute_stream wait for the fills of the last split lookup (no-op if it
 * had none or they were already waited for).  A later lookup on the handle
 * inserts this wait itself if the caller skipped it. */
int moe_cache_wait_fills(moe_cache* c, hipStream_t compute_stream);

/* Same policy without any device work: counts_host in, slot table and the list
 * of fills (slot, layer, expert, wave) out, for the caller to perform.  Works on
 * host-only and device handles.  max_fills >= n_slots is always enough. */
int moe_cache_lookup_host(moe_cache* c, int layer, const int32_t* counts_host, int wave,
                          int32_t* slot_of_expert_host, moe_fill* fills_host, int max_fills,
                          int* n_fills_host, moe_cache_stats* stats_host);

/* Snapshot: key held by each slot (-1 if empty) and its last-use tick. */
int moe_cache_state(const moe_cache* c, int64_t* key_of_slot_host, int64_t* tick_of_slot_host);

/* Test hook for failure handling: make the (n+1)-th fill from now fail with
 * MOE_EHIP without issuing it (n < 0 disables). */
int moe_cache_inject_fill_failure(moe_cache* c, int64_t n);

/* ------------------------------------------------------------------------- */
/* Grouped SwiGLU expert FFN.  The pages: GPU expert compute on cached and filled
 * experts, exact, with precision never lowered ("Three mechanisms";
 * "Key Takeaways").  For every expert e with counts > 0 and slot_of_expert[e] >= 0,
 * for each of its pairs p in [offsets[e], offsets[e+1]) with token t = sorted_rows[p]/k:
 *     out_rows[p] = W2 . ( SiLU(Wgate . x[t]) * (Wup . x[t]) ),   SiLU(z) = z/(1+e^-z)
 * with the expert's weights at slot_pool + slot*slot_stride.  Rows of experts
 * without a slot are not written.  If shared_w is non-null, the shared expert
 * (intermediate I_shared, same layout, always resident) is applied to every
 * token: shared_out[t] = FFN_shared(x[t]).
 *   wdt         weight type (moe_dtype)
 *   x           [T][H] f32 for MOE_F32, bf16 otherwise
 *   out_rows    [T*k][H] f32, indexed by sorted position
 *   shared_out  [T][H] f32 (required iff shared_w)
 *   workspace   >= moe_grouped_ffn_workspace() bytes of device memory
 * Arithmetic: f32 weights use f32 FMA; bf16 and MXFP4 weights use bf16 MFMA
 * with f32 accumulation (MXFP4 is expanded to bf16 exactly), and the SwiGLU
 * intermediate is rounded to bf16.  MOE_MXFP4_A8: gate/up multiply the E2M1
 * weights by the MXFP8 activations exactly (f32 accumulation), H, I and
 * I_shared multiples of 128 (MOE_EUNSUPPORTED otherwise). */
size_t moe_grouped_ffn_workspace(int T, int k, int E, int H, int I, int I_shared, int wdt);
int moe_grouped_ffn(int wdt, const void* slot_pool, size_t slot_stride, const int32_t* slot_of_expert,
                    const void* shared_w, int I_shared, const void* x, const int32_t* offsets,
                    const int32_t* sorted_rows, int T, int k, int E, int H, int I, float* out_rows,
                    float* shared_out, void* workspace, size_t ws_bytes, hipStream_t stream);
/* moe_grouped_ffn over experts addressed one by one instead of through slots:
 * expert_addr (device [E] uint64) holds the address of each expert's weights
 * (same layout as a slot; 16-byte aligned; device memory or pinned host memory
 * the GPU can read), 0 for experts not computed by this call.  Used for the
 * in-place half of the miss split; the results for an expert are bit for bit
 * those of moe_grouped_ffn on a slot holding the same bytes. */
int moe_grouped_ffn_addr(int wdt, const uint64_t* expert_addr, const void* shared_w, int I_shared, const void* x,
                         const int32_t* offsets, const int32_t* sorted_rows, int T, int k, int E, int H, int I,
                         float* out_rows, float* shared_out, void* workspace, size_t ws_bytes, hipStream_t stream);

/* moe_grouped_ffn for callers that cannot allocate device memory (code under
 * HIP graph capture, serving loops or harnesses that forbid hipMalloc): the same
 * arguments and results without the workspace.  The SwiGLU intermediate goes to a
 * fixed array of MOE_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it
 * runs on until the process ends; its device address is looked up on the first
 * call on each device (with that device current).  The call allocates nothing.
 * MOE_ECAPACITY if moe_grouped_ffn_workspace() for the shape exceeds the array
 * (32 MiB: e.g. up to 8192 token-expert pairs at I = 2048).  Every call on one GPU
 * uses the same array, so calls that overlap on one GPU (several streams or
 * threads) race; nothing in it needs clearing between calls. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int moe_grouped_ffn_noalloc(int wdt, const void* slot_pool, size_t slot_stride, const int32_t* slot_of_expert,
                            const void* shared_w, int I_shared, const void* x, const int32_t* offsets,
                            const int32_t* sorted_rows, int T, int k, int E, int H, int I, float* out_rows,
                            float* shared_out, hipStream_t stream);

/* MXFP8 quantization of activations, as MOE_MXFP4_A8 applies it before gate/up
 * (OCP Microscaling Formats v1.0, the format of the pages' MXFP4 build, "Results"):
 * x [T][H] bf16 (H a multiple of 32) -> codes [T][H] E4M3 bytes and scales
 * [T][H/32] E8M0 bytes; per 32-element block of a row X = floor(log2 max|x|) - 8
 * (X = -127 for an all-zero block), scale X + 127, each element x / 2^X rounded to
 * the nearest E4M3 value, ties to even, clamped to +-448.  Deterministic: the codes
 * depend on x alone.  codes 16-byte aligned. */
int moe_mx8_quantize(const void* x, int T, int H, uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* Which kernel family moe_grouped_ffn runs for a shape (the results are the same
 * computation either way): MOE_FFN_WEIGHT_STREAM (decode-sized batches: each
 * expert's weights stream once past its few tokens) or MOE_FFN_GROUPED_GEMM
 * (32 or more (token, expert) pairs per expert on average, bf16 or MXFP4 weights
 * with H, I and I_shared multiples of 128; MOE_MXFP4_A8 always).  -1 for an
 * invalid shape. */
enum { MOE_FFN_WEIGHT_STREAM = 0, MOE_FFN_GROUPED_GEMM = 1 };
int moe_grouped_ffn_kind(int T, int k, int E, int H, int I, int I_shared, int wdt);
/* The two phases of moe_grouped_ffn, same arguments: gate_up writes the SwiGLU
 * intermediate into the workspace, down reads it.  moe_grouped_ffn is exactly
 * gate_up followed by down on the same stream. */
int moe_grouped_ffn_gate_up(int wdt, const void* slot_pool, size_t slot_stride, const int32_t* slot_of_expert,
                            const void* shared_w, int I_shared, const void* x, const int32_t* offsets,
                            const int32_t* sorted_rows, int T, int k, int E, int H, int I, float* out_rows,
                            float* shared_out, void* workspace, size_t ws_bytes, hipStream_t stream);
int moe_grouped_ffn_down(int wdt, const void* slot_pool, size_t slot_stride, const int32_t* slot_of_expert,
                         const void* shared_w, int I_shared, const void* x, const int32_t* offsets,
                         const int32_t* sorted_rows, int T, int k, int E, int H, int I, float* out_rows,
                         float* shared_out, void* workspace, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Combine.  The pages: the partial sums are added without approximation ("Three mechanisms").
 *   y[t] = sum_{j=0..k-1} topk_w[t][j] * out_rows[inv_rows[t*k+j]]  (+ shared_out[t])
 * in f32, j in increasing order (fused multiply-add), then the shared term,
 * then one rounding to ydt (MOE_F32, or MOE_BF16 with round-to-nearest-even).
 * The fixed order makes the result independent of how experts were split into
 * cache waves.  y: [T][H] of ydt. */
int moe_combine(const float* out_rows, const float* topk_w, const int32_t* inv_rows, const float* shared_out,
                int T, int k, int H, void* y, int ydt, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* One layer for a few tokens: routing, expert FFN, shared expert and combine in
 * one call of two kernels (the pages' decode step runs one token through every
 * layer, "The gap it targets"; at that size the launches and round trips between
 * the layer's steps cost as much as the weights).
 *     y[t] = sum_j topk_w[t][j] * FFN_e(x[t]),  e = topk_ids[t][j]  (+ FFN_shared(x[t]))
 * with FFN and weight layouts of moe_grouped_ffn and the order of sums of moe_combine.
 * Up to 8 tokens the SwiGLU intermediate keeps 16 significant bits (a bf16 and a bf16
 * remainder), above it is rounded to bf16 as in moe_grouped_ffn; the K order inside a
 * product differs from moe_grouped_ffn's, so the two agree within rounding, not bit for bit.
 *   logits    [T][E] f32: routed as moe_route_topk does, topk_ids and topk_w [T][k] are
 *             written; NULL: topk_ids and topk_w are read as given (routing of the
 *             caller's own, or of an earlier moe_route)
 *   slot_of_expert  [E]; a pair whose expert has no slot (-1), or whose given id lies
 *             outside [0, E), contributes nothing to y (a cache wave or an expert shard
 *             gives its part of the sum)
 *   y         [T][H] of ydt (MOE_F32 or MOE_BF16)
 *   workspace >= moe_layer_decode_workspace() bytes, written by the call (two calls that
 *             may overlap need one each)
 * bf16 or MXFP4 weights (MOE_EUNSUPPORTED otherwise), T <= MOE_LAYER_DECODE_MAX_T,
 * T*k <= MOE_LAYER_DECODE_MAX_PAIRS, H <= 65536, experts and intermediate under 2 GiB
 * (MOE_EUNSUPPORTED beyond: use the separate calls).
 * Larger batches of 4-bit experts are faster through the separate calls: MXFP4, H = 4096,
 * I = 2048, 6 of 256 experts, 32 tokens 99 us here and 106 there, 48 tokens 137 and 130, 64 tokens
 * 160 and 145 (captured); bf16, H = 2048, I = 512, 8 of 256 and a shared one: within 5% from 16 on.
 * Asynchronous, allocates nothing, may be captured into a graph. */
#define MOE_LAYER_DECODE_MAX_T 64
#define MOE_LAYER_DECODE_MAX_PAIRS 512
size_t moe_layer_decode_workspace(int T, int k, int E, int H, int I, int I_shared, int wdt);
int moe_layer_decode(int wdt, const void* slot_pool, size_t slot_stride, const int32_t* slot_of_expert,
                     const void* shared_w, int I_shared, const void* x, const float* logits, int T, int k, int E,
                     int H, int I, int32_t* topk_ids, float* topk_w, void* y, int ydt, void* workspace,
                     size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Linear product with 4-bit weights, for the dense products around the experts
 * (projections, a head over the vocabulary) of a model whose weights are 4-bit (the
 * pages' MXFP4 build, "Results").
 *     y[t][n] = sum_k x[t][k] * W[n][k]  (+ bias[n])
 *   MOE_MXFP4: W = E2M1(code) * 2^(scale - 127), blocks of 32 along k (OCP MX v1.0), as a bf16
 *              operand: exact, but W of 2^128 and more (scales 253 and 254) is infinite; scale 255 is NaN
 *   MOE_INT4:  W = s * (q - z), q the code 0..15, s (f16) and z (0..255) one per row
 *              and group of `group` = 32, 64 or 128 consecutive k
 * 1 <= N <= 2^30, K a positive multiple of 32 and at most 2^20 (the last group may be
 * partial, group must be 32 for MOE_MXFP4), N * K < 2^40.
 *
 * moe_w4_pack lays the weights out once for the products:
 *   codes   [N][K/2], element 2i of a row in the low nibble of byte i
 *   scales  MOE_MXFP4: E8M0 bytes [N][K/32]; MOE_INT4: f16 [N][ceil(K/group)]
 *   zeros   MOE_INT4: uint8 [N][ceil(K/group)], NULL: 8 everywhere; MOE_MXFP4: NULL
 *   w       moe_w4_bytes() bytes (0 for invalid shapes)
 *
 * moe_w4_linear: x rows of K bf16, x_ld elements apart (x_ld >= K, a multiple of 8, at
 * most 2^22); y rows of N elements of ydt (MOE_F32 or MOE_BF16), y_ld >= N apart, not
 * overlapping x; bias [N] f32 or NULL.  0 <= T <= 2^19: the weights are read once for up to 16
 * tokens, or (many rows) 64, and again for every such batch.  Products are exact, sums
 * are in f32 in a fixed order, one rounding to ydt.  MOE_INT4 sums s (sum x q - z sum x)
 * group by group, so its roundings are relative to the magnitudes s (q + z) |x|; where that comes
 * out infinite or NaN (an infinite x, or x so large that a sum with the codes alone passes the f32
 * range) the output is formed again as the f32 sum of s (q - z) x in ascending k: an infinite x gives the
 * infinity of its products' sign, NaN where q = z.  Tokens concerned take longer.
 * Asynchronous, no workspace. */
enum { MOE_INT4 = 4 };
size_t moe_w4_bytes(int fmt, int N, int K, int group);
int moe_w4_pack(int fmt, const uint8_t* codes, const void* scales, const uint8_t* zeros, int N, int K, int group,
                void* w, hipStream_t stream);
int moe_w4_linear(int fmt, const void* w, int N, int K, int group, const void* x, int64_t x_ld, int T,
                  const float* bias, void* y, int64_t y_ld, int ydt, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Linear product with f32 or bf16 weights, for the dense products around the experts
 * (projections, a dense feed-forward part, a head) of a model whose weights are not 4-bit.
 *     y[t][n] = act( sum_k x[t][k] * w[n][k] + bias[n] ) + res[t][n]
 *   wdt   type of w and x: MOE_BF16 or MOE_F32 (MOE_EUNSUPPORTED otherwise)
 *   w     N rows of K, w_ld elements apart, as a checkpoint holds them: no packing
 *   x     T rows of K, x_ld elements apart
 *   bias  [N] f32 or NULL
 *   act   SiLU z / (1 + e^-z); GELU z P(Z <= z) of a normal Z; GELU_TANH its form with
 *         tanh( sqrt(2 / pi) (z + 0.044715 z^3) )
 *   res   T rows of N of rdt, r_ld apart, or NULL; may be y itself (same start, type and stride)
 *   y     T rows of N of ydt, y_ld apart; apart from that overlaps no operand (MOE_EINVAL)
 * K, w_ld and x_ld multiples of 8 (bf16) or 4 (f32), K, w_ld and x_ld at most 2^20; y_ld and r_ld
 * any (up to 2^36); T and N at most 2^22, T * N at most 2^35.  Products of bf16 are exact, sums are in f32 in an
 * order that the shape fixes, bias, activation and residual are applied in f32 before the one
 * rounding to ydt; f32 weights are multiplied in f32.  GELU's P(Z <= z) is within (1.5 z^2 + 24) 2^-24 of
 * itself for z < 0.  Asynchronous, no workspace, may be captured into a graph. */
enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3, MOE_ACT_GELU_TANH = 4 };
int moe_linear(int wdt, const void* w, int64_t w_ld, int N, int K, const void* x, int64_t x_ld, int T,
               const float* bias, int act, const void* res, int rdt, int64_t r_ld, void* y, int ydt, int64_t y_ld,
               hipStream_t stream);
/* Which kernel moe_linear runs for a shape (the results agree within rounding), as the tile of a workgroup: weight
 * rows * 65536 + tokens.  16 x 4 and 16 x 8: operands straight into registers; 16 x 16: through LDS, each wave for
 * itself; 32 x 32 to 256 x 256: staged by the whole workgroup.  0 for no tokens or an invalid shape. */
int moe_linear_tile(int wdt, int T, int N, int K);

/* ------------------------------------------------------------------------- */
/* The boundary of two blocks (attention, this layer, a dense part) in one call: the norm after
 * a block, its gate, the residual sum, and the norm before the next block.
 *     n = norm_post(block[t]);  r' = res_scale * res[t] + block_scale * gate * n;  x[t] = norm_pre(r')
 *     norm RMS:   v / sqrt(mean(v^2) + eps) * w (+ b);  LAYER: (v - mean(v)) / sqrt(var(v) + eps) * w (+ b)
 *   block    T rows of H of bdt, b_ld apart; NULL: nothing is added to res (the first norm of a model)
 *   gate     of gdt: [H] for every token (gate_ld 0) or T rows gate_ld apart; NULL: 1
 *   res      T rows of H of rdt, r_ld apart; NULL: no residual
 *   post_w, post_b, pre_w, pre_b   [H] f32; NULL: 1 and 0
 *   res_out  T rows of rdt, ro_ld apart, receives r'; NULL: not wanted
 *   x        T rows of xdt, x_ld apart; NULL: no next norm.  Of the f32 r', not of its rounding
 * Results may lie on block, res or a gate of T rows where start, type and stride agree (in place);
 * any other overlap is refused, as far as the addresses show it.  1 <= H <= 32768 (MOE_EUNSUPPORTED
 * beyond), T <= 2^21, strides any from H on (up to 2^36), eps >= 0.  Statistics in f32, exact to its rounding over
 * the whole range of the types.  Asynchronous, no workspace, may be captured. */
enum { MOE_NORM_NONE = 0, MOE_NORM_RMS = 1, MOE_NORM_LAYER = 2 };
int moe_block_norm(const void* block, int bdt, int64_t b_ld, int post_kind, const float* post_w, const float* post_b,
                   const void* gate, int gdt, int64_t gate_ld, float block_scale, const void* res, int64_t r_ld,
                   float res_scale, int pre_kind, const float* pre_w, const float* pre_b, float eps, int T, int H,
                   void* res_out, int rdt, int64_t ro_ld, void* x, int xdt, int64_t x_ld, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Tokens sorted by expert and back, for experts that are not moe_grouped_ffn's (products of
 * the caller, other devices), and the gradients for training a router or such experts.
 *
 * moe_dispatch: permutation and token rows in one call.  counts, offsets, sorted_rows and inv_rows as
 * moe_permute, except that ids outside [0, E) are allowed: such pairs go to no expert (an expert shard,
 * a capacity limit), inv_rows is -1 for them, offsets[E] counts the others, and sorted_rows holds -1
 * from there on.  Then rows[p] = x[sorted_rows[p] / k] for p < min(offsets[E], n_rows); rows behind
 * are left as they were.  x and rows of xdt (MOE_F32 or MOE_BF16), x_ld and rows_ld apart (any from H on,
 * up to 2^36).
 * workspace >= moe_dispatch_workspace() bytes (0 for few pairs: NULL is fine then), written by the call.
 *
 * moe_combine_rows: y[t] = sum_j topk_w[t][j] * rows[inv_rows[t*k+j]], j ascending, in f32, one rounding
 * to ydt.  Pairs whose place is negative or n_rows and beyond contribute nothing; a token without
 * any gets zeros.  Unlike moe_combine, rows may be bf16, strided and fewer than T*k.
 *
 * moe_combine_rows_backward: from dy, for every pair with a place p in [0, n_rows), t its token:
 *     d_rows[p] = topk_w[t][j] * dy[t]  (of rdt),  d_topk_w[t][j] = sum_h dy[t][h] * rows[p][h]  (f32)
 * and d_topk_w = 0 for the other pairs; rows of d_rows that no pair has are left as they were.  d_rows
 * may be rows itself (same start and stride).  No place may occur twice in inv_rows.
 *
 * moe_dispatch_backward: dx[t] = sum_j d_rows[inv_rows[t*k+j]], as moe_combine_rows with weights of 1.
 *
 * moe_gate_backward: gradient of the softmax over the selected logits (moe_route_topk's weights):
 *     d_logits[t][e] = sum over j with topk_ids[t][j] = e of w_j (d_w_j - sum_i w_i d_w_i)
 * for all e (0 where e was not selected; the selection itself has no gradient); [T][E] f32.
 * topk_ids are the router's own, also where moe_dispatch was given a copy with pairs marked as of no expert: the
 * softmax holds those pairs too, and with their d_w of 0 their logits still get -w_j sum_i w_i d_w_i.  With the
 * marked ids that part is lost, since no logit is named for it.  The results of the shards of one batch add up.
 *
 * All: 0 <= T <= 2^21, 1 <= k <= 32, H any positive up to 2^24, n_rows times the rows' distance at most
 * 2^59.  Results that lie on each other or on an operand are refused (MOE_EINVAL), but for d_rows on rows.  No atomics
 * on results: the same inputs give the same bits.  Asynchronous, may be captured (two calls that may overlap need a
 * workspace each). */
size_t moe_dispatch_workspace(int T, int k, int E);
int moe_dispatch(const void* x, int xdt, int64_t x_ld, const int32_t* topk_ids, int T, int k, int E, int H,
                 int32_t* counts, int32_t* offsets, int32_t* sorted_rows, int32_t* inv_rows, void* rows,
                 int64_t rows_ld, int n_rows, void* workspace, size_t ws_bytes, hipStream_t stream);
int moe_dispatch_backward(const void* d_rows, int rdt, int64_t dr_ld, int n_rows, const int32_t* inv_rows, int T,
                          int k, int H, void* dx, int xdt, int64_t dx_ld, hipStream_t stream);
int moe_combine_rows(const void* rows, int rdt, int64_t rows_ld, int n_rows, const float* topk_w,
                     const int32_t* inv_rows, int T, int k, int H, void* y, int ydt, int64_t y_ld, hipStream_t stream);
int moe_combine_rows_backward(const void* dy, int ydt, int64_t dy_ld, const void* rows, int rdt, int64_t rows_ld,
                              int n_rows, const float* topk_w, const int32_t* inv_rows, int T, int k, int H,
                              void* d_rows, int64_t dr_ld, float* d_topk_w, hipStream_t stream);
int moe_gate_backward(const int32_t* topk_ids, const float* topk_w, const float* d_topk_w, int T, int E, int k,
                      float* d_logits, hipStream_t stream);

/* ------------------------------------------------------------------------- */
/* Whole-layer streaming for prefill.  The pages: in prefill, whole layers are
 * copied into one of two device buffers, the next layer arriving while the
 * current one is computed from the other ("Three mechanisms": semantic-aware
 * caching).  Two device banks each hold one layer
 * (layer_bytes); a fill copies one layer from pinned host memory with one
 * hipMemcpyAsync on the fill stream.  Ordering: fill(bank) waits for the last
 * release(bank); acquire(bank) makes the compute stream wait for the last
 * fill(bank); release(bank) marks the compute work enqueued so far as the last
 * reader of the bank.  Typical loop: fill(0, b0); for l: fill(l+1, b(l+1));
 * acquire(b(l)); compute(l); release(b(l)). */
typedef struct moe_layer_stream moe_layer_stream;

typedef struct {
  int n_layers;
  size_t layer_bytes;
  const void* host_layers_host;            /* pinned [n_layers][layer_bytes] */
  const void* const* host_layer_ptrs_host; /* optional [n_layers] pinned pointers; overrides host_layers_host */
  void* banks[2];                          /* device, layer_bytes each */
  hipStream_t fill_stream;
} moe_layer_stream_desc;

int moe_layer_stream_create(const moe_layer_stream_desc* desc, moe_layer_stream** out);
int moe_layer_stream_destroy(moe_layer_stream* s);
int moe_layer_stream_fill(moe_layer_stream* s, int layer, int bank);
int moe_layer_stream_acquire(moe_layer_stream* s, int bank, hipStream_t compute_stream);
int moe_layer_stream_release(moe_layer_stream* s, int bank, hipStream_t compute_stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
