/*
 * tqmoe.h — C ABI of the trellis-quantized MoE grouped GEMM for GB300 (sm_103a).
 *
 * The routed-expert (MoE) product over expert weights stored as 2-bit
 * bitshift-trellis bitstreams, with the trellis decode fused into the multiply.
 *
 * Sources (pages; cited by title and section):
 *  [P1] "fix(qtip): gate the trellis grouped GEMM on m-tile occupancy, not token
 *       count" — "The cause is a threshold, not a kernel defect" (pairs sorted
 *       by expert, sum_e ceil(count_e / TILE_M) m-tiles, each woken expert's
 *       packed bytes staged once per m-tile; the tile-fill closed form), "The
 *       fix" (the amortization predicate), "Tests", post-merge note (the
 *       n <= 8 floor, the GEMV pin).
 *  [P2] "perf(qtip): arch-specialise the trellis grouped GEMM (D16) + close the
 *       silent-failure holes (D18)" — items 1 and 2 of the commit message
 *       (m-tile size; contiguous-run decode seeded by the window identity),
 *       "The two changes" (packed 2-bit bytes cross HBM, decode lands in a
 *       shared-memory tile, full-size weights never materialise), "D18" (every
 *       launcher returns a status, empty grids are errors, unsupported arch is
 *       refused), "The arch witness".
 *  [P3] "fix(ArcLab/ArcQuant): make prefill measurable, then ship the two
 *       kernels it proves were switched off" — launch counters prove which
 *       kernel ran; unknown environment values warn and keep the default.
 *
 * Data model (the pages leave the decode constants open; this library fixes):
 *  - Pair p = t * top_k + j is token t's j-th routed expert topk_ids[t][j].
 *  - Expert e's weight row r (0 <= r < N) is a bitstream of K 2-bit symbols in
 *    packed[e][r][0 .. K/4): symbol i is bits [2(i%4), 2(i%4)+2) of byte i/4.
 *  - The trellis state of symbol i is the L-bit window of the stream ending
 *    with symbol i (bits [2i+2-L, 2i+2), zeros before the row start), i.e.
 *    s_i = (s_{i-1} >> 2) | (c_i << (L-2)), s_{-1} = 0.  The weight is
 *    W_e[r][i] = lut[s_i], lut an fp16 table of 2^L entries.
 *  - Y[t][r] = sum_j topk_w[t][j] * sum_i W_{topk_ids[t][j]}[r][i] * x[t][i].
 *
 * Conventions for every call below:
 *  - Pointers marked (device) are device memory owned by the caller; no call
 *    allocates device memory or keeps a pointer after returning (the one fixed
 *    device array the library holds is described at tq_moe_forward_static).
 *  - Calls taking a stream enqueue work on it and return without waiting;
 *    they never synchronize the device.  The route, tile map, gather,
 *    grouped GEMM and combine kernels are launched as programmatic dependents
 *    of the previous kernel on the stream (they may start while it drains)
 *    and wait for it to finish before touching memory, so stream order holds
 *    as for ordinary launches.  (Inside tq_moe_forward and the grouped arm
 *    of tq_moe_mlp_forward, the first grouped kernel sets up its tensor
 *    memory and stages its LUT before that wait.  Its predecessor there is
 *    always one of this library's own launches, and neither writes the LUT:
 *    the fused route / tile-map launch when the kernel m-tile is at most
 *    TQ_GATHER_MAX_TILE_M, the activation gather above it.)  Status codes
 *    report argument and launch errors only; device-side faults of the data
 *    (an expert id out of range, a tile map over capacity, a wait that timed
 *    out) are recorded in a device error word read by tq_device_error().
 *  - Return value: TQ_OK (0) or a negative TQ_ERR_* code.  A failed call has
 *    launched nothing or reports the launch failure; outputs are then
 *    undefined and must not be read as results.
 *  - Layouts are row-major and dense.  bf16/fp16 values are passed as their
 *    16-bit patterns (uint16_t).
 */
#ifndef TQMOE_H
#define TQMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without the CUDA headers; NULL is the legacy default stream. */
typedef struct CUstream_st* tq_stream_t;

enum tq_status {
  TQ_OK = 0,
  TQ_ERR_INVALID_ARG = -1,      /* null pointer, bad size or alignment          */
  TQ_ERR_UNSUPPORTED_ARCH = -2, /* device or binary lacks sm_103a device code    */
  TQ_ERR_CAPACITY = -3,         /* tile map larger than the caller's capacity    */
  TQ_ERR_LAUNCH = -4,           /* kernel launch failed (cudaGetLastError)       */
  TQ_ERR_CAPTURING = -5,        /* arch witness cannot be taken during capture   */
  TQ_ERR_DEVICE_TIMEOUT = -6,   /* a device-side wait gave up (device error word)*/
  TQ_ERR_CUDA = -7,             /* another CUDA runtime error                     */
  TQ_ERR_WORKSPACE = -8         /* workspace too small or misaligned             */
};

/* Human-readable name of a status code.  Never NULL. */
const char* tq_status_string(int status);

/* ---------------------------------------------------------------------------
 * Arch witness  ([P2] "The arch witness", D18 #12)
 *
 * Launches a one-thread kernel compiled under the same architecture guard as
 * the grouped GEMM and reads back the architecture the running binary carries.
 * Succeeds only if the device is compute capability 10.3 and the binary holds
 * sm_103a device code.  Only a successful answer is cached (per device); the
 * witness is not taken while the calling thread's legacy stream or the given
 * stream is capturing, in which case TQ_ERR_CAPTURING is returned and the
 * next call retries.  Every launcher below checks the cached witness first and
 * takes it if missing.  `device` is a CUDA ordinal; it becomes current.
 * arch_out (host, may be NULL) receives __CUDA_ARCH__ of the device code.
 * ------------------------------------------------------------------------- */
int tq_init(int device);
int tq_arch_witness(int device, int* arch_out);

/* ---------------------------------------------------------------------------
 * Tile fill and the amortization gate  ([P1] "The cause is a threshold",
 * "The fix", post-merge note).  Host-only closed forms in three scalars: safe
 * inside CUDA-graph capture.  All evaluated in fp64.
 * ------------------------------------------------------------------------- */

/* n*k / (E * (1 - (1 - k/E)^n)); 0 for n == 0; NaN on invalid arguments
 * (k < 1, k > E, n < 0). */
double tq_pairs_per_woken_expert(int64_t n, int top_k, int E);

/* 1 if pairs per woken expert >= tile_m (an average m-tile is full), 0 if
 * not or n == 0, TQ_ERR_INVALID_ARG if k < 1, k > E, tile_m < 1 or n < 0. */
int tq_tiles_amortize(int64_t n, int top_k, int E, int tile_m);

/* Smallest n with tq_tiles_amortize(n, ...) == 1 (683 for top-6 of 256 at
 * tile_m 16).  Negative TQ_ERR_INVALID_ARG on invalid arguments. */
int64_t tq_grouped_min_tokens(int top_k, int E, int tile_m);

/* Native m-tile size of the grouped kernel on sm_103a for a routing shape,
 * by the expected pairs per woken expert (ppw, tq_pairs_per_woken_expert):
 * 256 when ppw >= 128 (prefill sizes, where one decode per 256 pairs beats
 * one per 128); 16 when ppw <= 4 (almost no expert has more than 16 pairs,
 * so the m-tiles are the woken experts either way, and at 16 the kernel
 * gathers the token rows itself, saving the pair-sorted copy); else 128
 * (fewer m-tiles, hence fewer decodes, than 16 once experts share more
 * pairs).  Measured on GB300 at 32, 128, 512, 1024 and 8192 tokens of top-6
 * of 256.  The whole-product calls below take tile_m = TQ_TILE_NATIVE to use
 * it: their kernels then run with this tile while the arm selection keeps the
 * pages' TILE_M (TQ_GATE_TILE_M).  Negative on invalid arguments. */
#define TQ_TILE_NATIVE 0
#define TQ_GATE_TILE_M 16
/* Environment (read at each call):
 *   TQ_FORCE_ARM=auto|gemv|grouped|measured  replaces pin = TQ_ARM_AUTO in the
 *       whole-product calls (the pages' env pin of the GEMV arm).
 *   TQ_TILE_M=1..256  the kernel m-tile of whole-product calls made with
 *       tile_m = TQ_TILE_NATIVE (the arm selection keeps TQ_GATE_TILE_M).
 *   TQ_QUIET=1  no engagement log line.
 * An unrecognised value is ignored with one warning on stderr. */
int tq_native_tile_m(int64_t n, int top_k, int E);

/* Upper bound on the number of m-tiles sum_e ceil(count_e / tile_m) for ANY
 * routing of n*top_k pairs: min(P, floor(P / tile_m) + min(E, P)).  Size the
 * tile map with it.  Negative on invalid arguments. */
int64_t tq_tile_map_capacity(int64_t n, int top_k, int E, int tile_m);

/* Arm selection ([P1] post-merge note): TQ_ARM_GEMV when n <= 8 or the tiles
 * do not amortize, TQ_ARM_GROUPED otherwise; `pin` forces an arm.  Negative
 * on invalid arguments.
 * pin = TQ_ARM_MEASURED selects by the crossover measured on GB300 instead
 * ([P3] "Two things that were built, correct, and switched off": the tile-fill
 * gate does not reproduce): this library's grouped kernel decodes each woken
 * expert once per m-tile whatever the tile's fill, so it wins as soon as
 * experts are shared enough; the arms tie near 1.16 pairs per woken expert
 * (V4 up shape, n ~ 14) and the grouped arm is chosen from there on, with no
 * token floor.
 * tq_moe_forward reports TQ_ARM_GEMV or TQ_ARM_GROUPED as the arm used. */
enum tq_arm { TQ_ARM_AUTO = 0, TQ_ARM_GEMV = 1, TQ_ARM_GROUPED = 2, TQ_ARM_MEASURED = 3 };
#define TQ_DECODE_REGIME_MAX_TOKENS 8
#define TQ_MEASURED_CROSSOVER_PPW 1.16
int tq_select_arm(int64_t n, int top_k, int E, int tile_m, int pin);

/* ---------------------------------------------------------------------------
 * Routing sort  ([P1] "The cause is a threshold": the grouped GEMM sorts pairs
 * by expert)
 *
 * topk_ids    (device) int32 [n][top_k], expert ids in [0, E).
 * counts      (device) int32 [E]       out: pairs per expert.
 * offsets     (device) int32 [E + 1]   out: exclusive prefix sum of counts.
 * sorted_pairs(device) int32 [n*top_k] out: pair ids p ordered by expert,
 *             ascending p within an expert (a stable sort).
 * Limits: 1 <= top_k <= E <= 1024, 0 <= n*top_k < 2^31.  An expert id out of
 * range is skipped and sets TQ_ERR_INVALID_ARG in the device error word.
 * One thread block up to 8192 pairs; above that one block per 2048 pairs
 * (at most 64), each sorting a contiguous chunk after counting every pair
 * itself, so no block waits for another.  No scratch memory.
 * ------------------------------------------------------------------------- */
int tq_route(const int32_t* topk_ids, int64_t n, int top_k, int E,
             int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
             tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Device router: per token the top_k experts by fp32 logit (descending;
 * equal logits go to the lower expert id) and their weights, a softmax over
 * the picked logits computed in fp32.  The router GEMM that produces the
 * logits is not part of this library.  Page "The 794 ms decode step,
 * itemised", list of un-owned items: the router runs in fp32.
 *
 * logits   (device) fp32 [n][E]; non-finite values count as -infinity (a row
 *          with no finite logit gets equal weights).
 * topk_ids (device) int32 [n][top_k] out; topk_w (device) fp32 [n][top_k] out.
 * Limits: 1 <= top_k <= min(E, 32), E <= 1024.
 * tq_route_logits = tq_router_topk then tq_route on the ids it wrote.
 * ------------------------------------------------------------------------- */
int tq_router_topk(const float* logits, int64_t n, int E, int top_k,
                   int32_t* topk_ids, float* topk_w, tq_stream_t stream);
int tq_route_logits(const float* logits, int64_t n, int E, int top_k,
                    int32_t* topk_ids, float* topk_w,
                    int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                    tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * m-tile map  ([P1] "The cause is a threshold"; [P2] D18: route and GEMM must
 * agree on tile_m)
 *
 * For experts e ascending with count_e > 0 and i < ceil(count_e / tile_m):
 *   tiles[t] = { e, offsets[e] + i*tile_m, min(tile_m, count_e - i*tile_m) }.
 * offsets   (device) int32 [E + 1] from tq_route.
 * tiles     (device) int32 [cap][3]  out.
 * num_tiles (device) int32 [1]       out: number of tiles written (<= cap).
 * cap: capacity of `tiles` in tiles, >= 1; tq_tile_map_capacity() is always
 * enough.  If the map would exceed cap, only cap tiles are written,
 * *num_tiles = cap and TQ_ERR_CAPACITY is set in the device error word.
 * 1 <= tile_m <= 256 (the grouped kernel's largest m-tile).
 * ------------------------------------------------------------------------- */
int tq_build_tile_map(const int32_t* offsets, int E, int tile_m,
                      int32_t* tiles, int32_t* num_tiles, int64_t cap,
                      tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Activation gather: x_sorted[s][:] = x[sorted_pairs[s] / top_k][:] for every
 * sorted slot s < n*top_k, so that the rows of an m-tile are consecutive
 * (TQ_X_PAIR_SORTED input of tq_grouped_gemm; tq_grouped_gemm_pairs input).
 * x (device) bf16 [n][K]; x_sorted (device) bf16 [n*top_k][K]; both 16-byte
 * aligned; K % 8 == 0.  A pair id out of range gives a zero row and sets
 * TQ_ERR_INVALID_ARG in the device error word.
 * ------------------------------------------------------------------------- */
int tq_gather_rows(const uint16_t* x, const int32_t* sorted_pairs, int64_t n, int top_k, int K,
                   uint16_t* x_sorted, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Everything the grouped GEMM needs, in one launch: tq_route and
 * tq_build_tile_map fused (one block sorts; the tile map takes each expert's
 * slot range from the sort's registers) while the launch's other blocks
 * clear y32[0 .. y32_count) (the fp32 accumulator; 16-byte aligned and
 * y32_count % 4 == 0 for the fused clear, otherwise it is cleared by a
 * separate memset).  x_sorted may be NULL: when given, tq_gather_rows also
 * runs (a second launch; x is unused otherwise).  Results are those of the separate calls.  Arguments as in
 * tq_route, tq_build_tile_map and tq_gather_rows; y32 may be NULL when
 * y32_count == 0.
 * ------------------------------------------------------------------------- */
int tq_prepare(const int32_t* topk_ids, const uint16_t* x, int64_t n, int top_k, int E, int K, int tile_m,
               int32_t* counts, int32_t* offsets, int32_t* sorted_pairs, int32_t* tiles, int32_t* num_tiles,
               int64_t cap, uint16_t* x_sorted, float* y32, int64_t y32_count, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Grouped GEMM  ([P1] m-tiles; [P2] contiguous-run decode, decode fused into
 * the multiply)
 *
 * For every m-tile and every 128-row block of N: TMA stages the expert's
 * packed rows once, warps decode runs of 32 symbols (seeded by the window
 * identity, then stepped) into a bf16 weight tile in tensor memory, TMA
 * copies the tile's activation rows into shared memory, tcgen05 MMAs
 * contract the two (fp32 accumulate), and the epilogue scales by the router
 * weight and adds into y32.
 *
 * x_layout   TQ_X_TOKENS: x (device) bf16 [n][K], the token activations; the
 *            kernel gathers row sorted_pairs[slot] / top_k of each m-tile
 *            slot, four rows per copy.  TQ_X_PAIR_SORTED: x (device) bf16
 *            [n*top_k][K] from tq_gather_rows (row = sorted slot), one box
 *            copy per m-tile and k-step.  Results are identical; the row
 *            gathers cost one copy per four pairs, so for m-tiles above
 *            TQ_GATHER_MAX_TILE_M the separate tq_gather_rows pass is faster
 *            (the whole-product calls choose by that rule).
 * x          16-byte aligned.
 * packed     (device) uint8 [E][N][K/4]; 16-byte aligned.
 * lut        (device) fp16 [2^L] (converted to bf16, nearest-even, on chip).
 * sorted_pairs, tiles, num_tiles: from tq_route / tq_build_tile_map with the
 *            same tile_m.  cap = capacity of `tiles`.
 * topk_w     (device) fp32 [n][top_k] router weights.
 * y32        (device) fp32 [n][N], 16-byte aligned: ACCUMULATED into (y32 += ...); zero it
 *            first for a plain product.  Additions are fp32 atomics, so the
 *            summation order (and the last bits) vary between runs.
 * Requires: K % 64 == 0, N % 128 == 0, L even in [2, 16], 1 <= tile_m <= 256,
 * 1 <= top_k <= E.  Device: compute capability 10.3.
 * ------------------------------------------------------------------------- */
#define TQ_X_TOKENS 0
#define TQ_X_PAIR_SORTED 1
#define TQ_GATHER_MAX_TILE_M 16
int tq_grouped_gemm(const uint16_t* x, int x_layout, const uint8_t* packed, const uint16_t* lut, int L,
                    const int32_t* sorted_pairs, const float* topk_w,
                    const int32_t* tiles, const int32_t* num_tiles, int64_t cap,
                    int64_t n, int top_k, int E, int K, int N, int tile_m,
                    float* y32, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Per-pair GEMV arm  ([P1] "The regression": the per-pair gather GEMV; no
 * de-duplication of experts across pairs)
 *
 * For every pair p (token t = p / top_k, expert e = topk_ids[p]) and every
 * row r: y32[t][r] += topk_w[p] * sum_i W_e[r][i] * x[t][i], fp32 accumulate,
 * fp16 weights widened exactly.  Same layouts as tq_grouped_gemm; needs no
 * routing sort.  Requires K % 64 == 0, K <= 8192, L even in [2, 16].
 * ------------------------------------------------------------------------- */
int tq_gemv(const uint16_t* x, const uint8_t* packed, const uint16_t* lut, int L,
            const int32_t* topk_ids, const float* topk_w,
            int64_t n, int top_k, int E, int K, int N,
            float* y32, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Combine: y[i] = bf16(y32[i]), round to nearest even, for i < count.  The
 * stated numerics of the product: fp32 accumulation, bf16 output (the routed
 * outputs are summed per token in fp32 by the arms above; this call rounds
 * the sum once).  [P1] "The cause is a threshold": the grouped GEMM's output
 * is the per-token combined projection.
 * y32 (device) fp32 [count]; y (device) bf16 [count].
 * ------------------------------------------------------------------------- */
int tq_combine(const float* y32, uint16_t* y, int64_t count, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Whole routed-expert product: arm selection (tq_select_arm with `pin`),
 * then on the grouped arm route + tile map (clearing the fp32 accumulator),
 * the grouped kernel and the combine to bf16 y [n][N]; on the GEMV arm one
 * launch that sums each token's top_k pairs in fp32 registers and writes
 * bf16 y [n][N] directly (the workspace is not touched).
 *
 * workspace (device): caller-owned scratch of at least
 *   tq_moe_workspace_size(n, top_k, E, K, N, tile_m) bytes, 256-byte aligned.
 *   It holds counts, offsets, sorted pairs, the tile map, the fp32
 *   accumulator and, for a kernel m-tile above TQ_GATHER_MAX_TILE_M, the
 *   pair-sorted activations and the sort's inverse (the sorted slot of each
 *   pair, written by the routing launch, through which the activations are
 *   copied in token order: each row of x read once); its contents are
 *   undefined after the call.
 * tile_m: 1..256, the m-tile of both the arm selection and the kernel, or
 *   TQ_TILE_NATIVE (tq_native_tile_m for the kernel, TQ_GATE_TILE_M for the
 *   selection).
 * arm_used (host, may be NULL): receives TQ_ARM_GEMV or TQ_ARM_GROUPED.
 * The first grouped engagement in a process logs the tile fill and the
 * amortization boundary to stderr once (unless TQ_QUIET=1).
 * ------------------------------------------------------------------------- */
size_t tq_moe_workspace_size(int64_t n, int top_k, int E, int K, int N, int tile_m);
int tq_moe_forward(const uint16_t* x, const uint8_t* packed, const uint16_t* lut, int L,
                   const int32_t* topk_ids, const float* topk_w,
                   int64_t n, int top_k, int E, int K, int N, int tile_m, int pin,
                   void* workspace, size_t workspace_bytes,
                   uint16_t* y, int* arm_used, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Whole routed-expert product without allocating: tq_moe_forward with its
 * scratch in a fixed device array inside the library instead of a caller
 * workspace.  The pages have no counterpart; this exists for callers that
 * cannot allocate device memory — e.g. a plugin to which a host framework
 * passes only input and output buffers, or a serving loop that forbids
 * allocation after start-up because cudaMalloc can block and synchronize.
 *
 * Arguments, layouts and results are those of tq_moe_forward minus the
 * workspace.  The scratch is a file-scope device array of
 * TQ_STATIC_SCRATCH_BYTES (16 MiB) that every GPU loading this library holds
 * until the process exits; a shape whose tq_moe_workspace_size() exceeds it
 * is rejected with TQ_ERR_WORKSPACE before anything is launched (at
 * K = 4096, N = 2048, top-6 that is n > 2040 tokens at tile_m 16, where the kernel gathers its own
 * rows, and n > 292 with larger m-tiles, which add the pair-sorted copy of x).  The call allocates nothing (no cudaMalloc,
 * no cudaFree, no allocating library routine).
 *
 * The first call on a device does one-time set-up there: it looks up the
 * array's device address with that device current (cudaGetSymbolAddress) and
 * caches it, and, unless tq_init(device) ran first, takes the arch witness
 * (which creates a private stream, launches one tiny kernel, synchronizes
 * that stream and destroys it) and looks up the driver's tensor-map encoder.
 * That first call can therefore stall the host; make it (or tq_init) at
 * start-up, before any stream capture.  Later calls only enqueue.  Every call on a device shares the one array and
 * it keeps the last call's contents (each call zeroes what must start at
 * zero): calls that overlap on the GPU — on different streams or threads —
 * race and corrupt each other's results; serialize them.
 * ------------------------------------------------------------------------- */
#define TQ_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)
int tq_moe_forward_static(const uint16_t* x, const uint8_t* packed, const uint16_t* lut, int L,
                          const int32_t* topk_ids, const float* topk_w,
                          int64_t n, int top_k, int E, int K, int N, int tile_m, int pin,
                          uint16_t* y, int* arm_used, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * The whole expert MLP (SwiGLU experts).  The routed-expert grouped GEMM
 * above is one of an expert's three projections; these calls chain them:
 *   gate|up_p = W_gu,e x_t,  h_p = silu(gate_p) * up_p,
 *   y_t = sum_j w_tj W_down,e h_(t,j).
 * packed_gu (device) uint8 [E][2I][H/4]: rows 0..I-1 the gate, I..2I-1 the
 * up projection; packed_down (device) uint8 [E][H][I/4]; one LUT each
 * (fp16 [2^L]); the same L.
 *
 * tq_grouped_gemm_pairs: the grouped GEMM with per-pair outputs and no
 *   router weight: out32[slot][:] += W_e x_sorted[slot] for every sorted
 *   slot (out32 (device) fp32 [n*top_k][N], 16-byte aligned, zero it first).
 * tq_swiglu: h[s][i] = bf16(silu(g) * u), g = gate_up[s][i],
 *   u = gate_up[s][I + i]; gate_up (device) fp32 [P][2I], h (device) bf16
 *   [P][I]; I % 4 == 0.
 * tq_moe_mlp_forward: the arm chosen as in tq_moe_forward (tq_select_arm with
 *   `pin`, the gate's TILE_M from `tile_m`; arm_used (host, may be NULL)
 *   receives it).  Grouped arm: route + tile map, gate|up (per pair; token
 *   rows gathered in the kernel, or, above TQ_GATHER_MAX_TILE_M, copied into
 *   pair-sorted order in token order through the sort's inverse, as in
 *   tq_moe_forward), SwiGLU, down (combined per token with the router
 *   weights).  GEMV arm:
 *   gate|up by per-pair GEMVs, SwiGLU, down by per-pair GEMVs on h combined
 *   per token.  Output bf16 y [n][H].  H % 128 == 0, I % 64 == 0 (and
 *   H, I <= 8192 for the GEMV arm).  workspace (device) >=
 *   tq_moe_mlp_workspace_size(...) bytes, 256-byte aligned.
 * ------------------------------------------------------------------------- */
int tq_grouped_gemm_pairs(const uint16_t* x_sorted, const uint8_t* packed, const uint16_t* lut, int L,
                          const int32_t* sorted_pairs, const int32_t* tiles, const int32_t* num_tiles,
                          int64_t cap, int64_t n, int top_k, int E, int K, int N, int tile_m,
                          float* out32, tq_stream_t stream);
int tq_swiglu(const float* gate_up, int64_t P, int I, uint16_t* h, tq_stream_t stream);
size_t tq_moe_mlp_workspace_size(int64_t n, int top_k, int E, int H, int I, int tile_m);
int tq_moe_mlp_forward(const uint16_t* x, const uint8_t* packed_gu, const uint16_t* lut_gu,
                       const uint8_t* packed_down, const uint16_t* lut_down, int L,
                       const int32_t* topk_ids, const float* topk_w,
                       int64_t n, int top_k, int E, int H, int I, int tile_m, int pin,
                       void* workspace, size_t workspace_bytes, uint16_t* y, int* arm_used,
                       tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Dequantize-materialize comparator  ([P1] "Tests": the dequantize path that
 * dispatch falls through to outside the fused arms' ranges; [P2] "The two
 * changes": the fused design never materialises full-size weights).  These
 * calls build that path so it can be measured against the fused arms; the
 * selection of tq_select_arm never picks it.
 *
 * tq_dequantize: w_out[i] = bf16(W_{expert_ids[i]}) for i < m, each a dense
 *   row-major [N][K] matrix: the trellis decode of the bitstreams above and
 *   fp16 -> bf16 nearest-even, bit-identical to the values the fused kernels
 *   feed their MMAs.  expert_ids (device) int32 [m], or NULL for experts
 *   0..m-1 (then m <= E); an id < 0 leaves its slot untouched; an id >= E
 *   leaves it untouched and sets TQ_ERR_INVALID_ARG in the device error word.
 *   packed, lut, w_out (device) 16-byte aligned; K % 8 == 0; L even in
 *   [2, 16].  w_out holds m*N*K bf16 values (16 MiB per expert at
 *   4096 x 2048).
 * tq_grouped_gemm_dense: tq_grouped_gemm with dense bf16 weights
 *   w_dense (device) [E][N][K] (16-byte aligned) in place of packed + lut;
 *   same m-tiles, activation layouts (x, x_layout), MMA and epilogue
 *   (y32 += w * W_e x).
 * tq_moe_forward_dequant: zero y32, route, tile map, dequantize every
 *   expert with at least one pair into slot e of an [E][N][K] bf16 buffer in
 *   the workspace, tq_grouped_gemm_dense, combine to bf16 y [n][N].
 *   workspace (device) >= tq_moe_dequant_workspace_size(...) bytes (the
 *   tq_moe_workspace_size regions followed by E*N*K*2 bytes), 256-byte
 *   aligned.  Requires K % 64 == 0, N % 128 == 0, E <= 1024.
 * ------------------------------------------------------------------------- */
int tq_dequantize(const uint8_t* packed, const uint16_t* lut, int L, const int32_t* expert_ids, int m,
                  int E, int N, int K, uint16_t* w_out, tq_stream_t stream);
int tq_grouped_gemm_dense(const uint16_t* x, int x_layout, const uint16_t* w_dense, const int32_t* sorted_pairs,
                          const float* topk_w, const int32_t* tiles, const int32_t* num_tiles, int64_t cap,
                          int64_t n, int top_k, int E, int K, int N, int tile_m, float* y32,
                          tq_stream_t stream);
size_t tq_moe_dequant_workspace_size(int64_t n, int top_k, int E, int K, int N, int tile_m);
int tq_moe_forward_dequant(const uint16_t* x, const uint8_t* packed, const uint16_t* lut, int L,
                           const int32_t* topk_ids, const float* topk_w,
                           int64_t n, int top_k, int E, int K, int N, int tile_m,
                           void* workspace, size_t workspace_bytes, uint16_t* y, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Element types of the calls below that take more than one.
 * ------------------------------------------------------------------------- */
enum tq_type { TQ_FP32 = 0, TQ_BF16 = 1, TQ_FP16 = 2 };

/* ---------------------------------------------------------------------------
 * Scored router: scores of every expert, a bias that balances the choice,
 * groups, top-k and weights.  Per token t, over its E logits x:
 *   s_i = 1 / (1 + exp(-x_i))  (TQ_SCORE_SIGMOID)  or softmax(x)_i
 *         (TQ_SCORE_SOFTMAX);  c_i = s_i + bias_i.
 *   The experts are `groups` consecutive groups of E / groups; a group's value
 *   is the sum of its two largest c (of its one); the `top_groups` groups of
 *   largest value stay.  The chosen are the top_k largest c of the groups that
 *   stay, in descending order; ties go to the lower index, of groups too.
 *   Weights are the s of the chosen (without the bias), divided by their sum
 *   with `renormalize`, times `scale`.
 * A logit that is not finite is a masked expert: score 0, chosen only when the
 * groups that stay hold fewer than top_k others.  Such a filler, and any other
 * choice beyond the experts left, has weight 0, and so have all of a row's when
 * their sum is 0 (a row with no finite logit).  A NaN in c or in a group's
 * value counts as -infinity.
 * The result of a row depends on that row alone: not on n, the launch or the
 * device's load.  Scores, sums and weights are fp32 throughout.
 *
 * logits   (device) [n] rows of E logits_type values, logits_stride elements
 *          apart (>= E; rows whose base and stride are multiples of 16 bytes
 *          are read fastest, others are correct).
 * bias     (device) fp32 [E], or NULL for none.
 * topk_ids (device) int32 [n][top_k] out; topk_w (device) fp32 [n][top_k] out.
 * Limits: E <= 1024, top_k <= 32, groups <= 32 dividing E, 1 <= top_groups <=
 * groups, top_k <= top_groups * (E / groups).
 *
 * tq_router_scored_backward: the gradient of the logits from grad_w, the
 * gradient of topk_w; topk_ids and topk_w are the forward's outputs for the
 * same logits (the choice itself has no gradient, nor has the bias).  Every
 * element of grad_logits, [n][E] dense in the logits' type, is written.  An id
 * out of range is skipped and sets TQ_ERR_INVALID_ARG in the device error word.
 * ------------------------------------------------------------------------- */
enum tq_score { TQ_SCORE_SOFTMAX = 0, TQ_SCORE_SIGMOID = 1 };
int tq_router_scored(const void* logits, int logits_type, int64_t logits_stride, const float* bias,
                     int64_t n, int E, int top_k, int score, int groups, int top_groups,
                     int renormalize, float scale, int32_t* topk_ids, float* topk_w, tq_stream_t stream);
int tq_router_scored_backward(const void* logits, int logits_type, int64_t logits_stride,
                              const int32_t* topk_ids, const float* topk_w, const float* grad_w,
                              int64_t n, int E, int top_k, int score, int renormalize, float scale,
                              void* grad_logits, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * 4-bit microscaled values.  A row of K values (K % 32 == 0) is kept as E2M1
 * codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign in bit 3), two to a byte, value
 * 2i in the low half of byte i; blocks of consecutive values share a scale:
 *   TQ_FP4_NV  blocks of 16, scale s = e4m3(max|x| / (6 g)), g the 32-bit
 *              global scale (1 when NULL; positive with 6 g finite, or 0, with
 *              which every s is 0, as the g of an all-zero tensor may be);
 *              code = e2m1(x / (s g)), value = code * s * g.
 *   TQ_FP4_MX  blocks of 32, scale s = 2^(floor(log2 max|x|) - 2) as E8M0
 *              (2^-127 at least); code = e2m1(x / s); no global scale (the
 *              pointer must be NULL).
 * Arithmetic is fp32; both roundings are to nearest even and saturate.  NaN is
 * kept as 0 and does not count for the maximum, an infinity counts as the
 * largest finite number.  Values of a block whose scale rounds to 0 are 0.  A
 * scale byte that is NaN (0x7f as E4M3, 0xff as E8M0; the quantiser writes none)
 * makes the values of its block NaN.
 * global_scale, x_scale, h_scale (device) fp32 [1] or NULL; w_scale, gu_scale,
 * down_scale (device) fp32 [E] or NULL.
 *
 * tq_fp4_quantize: x (device) n rows of K x_type values, x_stride elements
 *   apart, base and rows 16-byte aligned -> packed (device) uint8 [n][K/2],
 *   8-byte aligned, and scales (device) uint8 [n][K / block].
 * tq_fp4_dequantize: the values of packed and scales, (code * s) * g rounded
 *   once to out_type; out (device) [n][K], 16-byte aligned.
 * tq_fp4_tile_scales: the products below read block scales in tiles of 128
 *   rows x 4 blocks (512 bytes; byte (row % 32) * 16 + (row % 128 / 32) * 4 +
 *   block % 4), tiles of a group of 128 rows one after another along K, rows
 *   padded to 128 and K to 256 values with zeros.  scales (device) uint8
 *   [E][N][K / block] -> tiled (device), tq_fp4_tiled_scales_size() bytes (0
 *   on invalid arguments; E * N below 2^31 - 1024, as the products take),
 *   16-byte aligned.  Done once, when weights load.
 * ------------------------------------------------------------------------- */
enum tq_fp4_format { TQ_FP4_NV = 0, TQ_FP4_MX = 1 };
int tq_fp4_quantize(const void* x, int x_type, int64_t x_stride, int64_t n, int K, int fmt,
                    const float* global_scale, uint8_t* packed, uint8_t* scales, tq_stream_t stream);
int tq_fp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t n, int K, int fmt,
                      const float* global_scale, void* out, int out_type, tq_stream_t stream);
size_t tq_fp4_tiled_scales_size(int E, int N, int K, int fmt);
int tq_fp4_tile_scales(const uint8_t* scales, int E, int N, int K, int fmt, uint8_t* tiled,
                       tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Products of 4-bit microscaled weights.  The activations are quantised by the
 * call (as by tq_fp4_quantize, x_scale their global scale), multiplied on the
 * block-scaled tensor cores and summed in fp32; the result is rounded once to
 * y_type.  Sums have a fixed order, so results repeat bit for bit.
 *
 * tq_fp4_linear:      y[t] = W x[t], W one matrix: packed [N][K/2].
 * tq_fp4_moe_forward: y[t] = sum_j topk_w[t][j] W_{topk_ids[t][j]} x[t], packed
 *   [E][N][K/2].  A pair whose id is out of range adds nothing and sets
 *   TQ_ERR_INVALID_ARG in the device error word.
 * tq_fp4_moe_mlp_forward: SwiGLU experts, packed_gu [E][2I][H/2] (rows 0..I-1
 *   the gate, I..2I-1 the up projection), packed_down [E][H][I/2]:
 *   h = silu(gate) * up per pair in fp32, quantised with global scale h_scale,
 *   y[t] = sum_j topk_w[t][j] W_down h(t,j).
 * x as in tq_fp4_quantize; packed and tiled_scales (tq_fp4_tile_scales) 16-byte
 * aligned; y (device) dense [n][N] (or [n][H]).  N is any width; K, H and I are
 * multiples of 32.  E <= 1024, top_k <= 32; n * top_k and E * N below
 * 2^31 - 1024, n * top_k * N below 2^58.  Few rows (by a rule on n, top_k,
 * E, K and N) take one launch that needs no workspace.  workspace (device) of
 * at least the matching *_workspace_size() bytes (0 on invalid arguments; 256,
 * or a NULL workspace, where none is needed), 256-byte aligned; its contents
 * are undefined after the call.  The size does not grow with n throughout (K is
 * split where few rows leave the device idle): ask for each n that a workspace
 * is to serve, and take the largest.
 * ------------------------------------------------------------------------- */
size_t tq_fp4_linear_workspace_size(int64_t n, int K, int N, int fmt);
int tq_fp4_linear(const void* x, int x_type, int64_t x_stride, const uint8_t* packed,
                  const uint8_t* tiled_scales, int fmt, const float* w_scale, const float* x_scale,
                  int64_t n, int K, int N, void* workspace, size_t workspace_bytes,
                  void* y, int y_type, tq_stream_t stream);
size_t tq_fp4_moe_workspace_size(int64_t n, int top_k, int E, int K, int N, int fmt);
int tq_fp4_moe_forward(const void* x, int x_type, int64_t x_stride, const uint8_t* packed,
                       const uint8_t* tiled_scales, int fmt, const float* w_scale, const float* x_scale,
                       const int32_t* topk_ids, const float* topk_w,
                       int64_t n, int top_k, int E, int K, int N, void* workspace, size_t workspace_bytes,
                       void* y, int y_type, tq_stream_t stream);
size_t tq_fp4_moe_mlp_workspace_size(int64_t n, int top_k, int E, int H, int I, int fmt);
int tq_fp4_moe_mlp_forward(const void* x, int x_type, int64_t x_stride,
                           const uint8_t* packed_gu, const uint8_t* tiled_gu, const float* gu_scale,
                           const uint8_t* packed_down, const uint8_t* tiled_down, const float* down_scale,
                           int fmt, const float* x_scale, const float* h_scale,
                           const int32_t* topk_ids, const float* topk_w,
                           int64_t n, int top_k, int E, int H, int I, void* workspace, size_t workspace_bytes,
                           void* y, int y_type, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Root-mean-square norm with the residual's addition.  Per row, over its K values:
 *   r = x + residual, rounded to x_type and kept in residual_out (residual NULL:
 *   r = x);  rstd = 1 / sqrt(mean(r^2) + eps);  y = (r * rstd) * weight.
 * The output is y in x's type, or in 8 bits with block scales (codes, scales as
 * tq_fp8_quantize writes them for y before its rounding), or both.  Arithmetic is
 * fp32; the sum of squares carries its rounding errors along, so that rstd is
 * rounded once and results do not depend on the order of a sum.
 * x, residual (device) n rows of K x_type values, *_stride elements apart (>= K);
 *   rows on 16-byte boundaries with K a multiple of 16 are read fastest and are
 *   required for codes.
 * weight       (device) w_type [K], or NULL for ones.
 * residual_out (device) [n][K] of x_type, dense, with a residual; it may be the
 *   residual or x itself where that is dense (in place).
 * y (device) [n][K] of x_type, dense, or NULL; it may be x where that is dense.
 * rstd (device) fp32 [n] or NULL: what the gradient takes.
 * codes (device) uint8 [n][K], 16-byte aligned, and scales (device) fp32
 *   [n][ceil(K / 128)], or both NULL.
 * Outputs that share memory with an input in another way, or with each other, are
 * refused.  Limits: 1 <= K <= TQ_NORM_MAX_WIDTH, eps >= 0 and finite.
 *
 * tq_rms_norm_backward: with x the normed rows (residual_out of the forward call,
 *   or its x), rstd of that call and a = grad_y * weight:
 *   grad_x = rstd * (a - x * rstd^2 * mean(a * x)) + grad_residual, in x_type,
 *   dense [n][K]: the gradient of x and of the residual alike;
 *   grad_weight[k] = sum over rows of grad_y * x * rstd, in w_type, or NULL.
 *   grad_residual (what arrives through residual_out) may be NULL.  Sums are fp32
 *   in a fixed order.  grad_x may be x, grad_y or grad_residual where that is dense;
 *   results and workspace that share other memory with an input or each other are
 *   refused.
 *   workspace (device, 256-byte aligned) of tq_rms_norm_backward_workspace_size()
 *   bytes (0 on invalid arguments); not used without grad_weight.
 * ------------------------------------------------------------------------- */
#define TQ_NORM_MAX_WIDTH 16384
int tq_rms_norm(const void* x, int x_type, int64_t x_stride, const void* residual, int64_t residual_stride,
                const void* weight, int w_type, float eps, int64_t n, int K, void* residual_out, void* y,
                float* rstd, uint8_t* codes, float* scales, tq_stream_t stream);
size_t tq_rms_norm_backward_workspace_size(int64_t n, int K);
int tq_rms_norm_backward(const void* grad_y, int64_t grad_y_stride, const void* x, int x_type, int64_t x_stride,
                         const void* weight, int w_type, const float* rstd, const void* grad_residual,
                         int64_t grad_residual_stride, int64_t n, int K, void* workspace, size_t workspace_bytes,
                         void* grad_x, void* grad_weight, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * 8-bit block-scaled values.  Blocks of rows_per_block x 128 values of a matrix of
 * rows of K (K % 16 == 0; the last block may be short) share an fp32 scale
 * s = max|x| / 448; a value is kept as the E4M3 code of x / s, value = code * s.
 * rows_per_block is 1 (activations) or 128 (weights).  Both quotients are rounded
 * to fp32 and the conversion to nearest even, saturating.  NaN is kept as NaN and
 * does not count for the maximum, an infinity counts as the largest finite number
 * and is kept as 448 (so code * s is that number).  Zeros keep their sign.  In a block
 * with s = 0 all but NaN is kept as 0 (code 0).
 *
 * tq_fp8_quantize: x (device) E matrices of n rows of K x_type values, x_stride
 *   elements apart (matrix e starts at row e * n), base and rows 16-byte aligned ->
 *   codes (device) uint8 [E][n][K], 16-byte aligned, and scales (device) fp32
 *   [E][ceil(n / rows_per_block)][ceil(K / 128)].
 * tq_fp8_dequantize: code * s rounded once to out_type; out (device) [E][n][K],
 *   16-byte aligned.
 * Limits: E * n below 2^31 - 1024; with rows_per_block 128 also E <= 65535.  No
 * output may share memory with an input or the other output.
 * ------------------------------------------------------------------------- */
int tq_fp8_quantize(const void* x, int x_type, int64_t x_stride, int E, int64_t n, int K, int rows_per_block,
                    uint8_t* codes, float* scales, tq_stream_t stream);
int tq_fp8_dequantize(const uint8_t* codes, const float* scales, int E, int64_t n, int K, int rows_per_block,
                      void* out, int out_type, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Products of 8-bit block-scaled rows x (rows_per_block 1) with 8-bit matrices
 * (rows_per_block 128).  The partial sums of each block of 128 are accumulated in
 * fp32, multiplied by the product of both scales, which has to be in fp32's range (the
 * scale of a block with an infinity is 2^119: its weights' scales have to be at most 448,
 * or results are infinite or NaN), and added up in fp32, pair by pair before topk_w
 * multiplies them; the result is rounded once to y_type.  Sums have a fixed order, so
 * results repeat bit for bit.
 *
 * tq_fp8_linear:      y[t] = W x[t], w [N][K], w_scales [ceil(N/128)][ceil(K/128)].
 * tq_fp8_moe_forward: y[t] = sum_j topk_w[t][j] W_{topk_ids[t][j]} x[t], w [E][N][K]
 *   and w_scales [E][..].  A pair whose id is out of range adds nothing and sets
 *   TQ_ERR_INVALID_ARG in the device error word.
 * tq_fp8_moe_mlp_forward: SwiGLU experts, w_gu [E][2I][H] (rows 0..I-1 the gate,
 *   I..2I-1 the up projection), w_down [E][H][I], I a multiple of 128:
 *   h = silu(gate) * up per pair in fp32, kept in 8 bits (blocks of 128 of a row),
 *   y[t] = sum_j topk_w[t][j] W_down h(t,j).  E = 1, top_k = 1: a dense MLP.
 * x, w (device) codes, 16-byte aligned; x_scales (device) fp32 [n][ceil(K/128)];
 * y (device) dense; y and a workspace that is used may not share memory with an input
 * or each other.  K and H are multiples of 16, N is any width.  E <= 1024, top_k <= 32;
 * n * top_k and E * N (E * 2I, E * H) below 2^31 - 1024, n * top_k * N below 2^57.
 * workspace (device) of at least the matching *_workspace_size() bytes (0 on invalid
 * arguments; 256, or a NULL workspace, where none is needed), 256-byte aligned; its
 * contents are undefined after the call.  The size does not grow with n throughout: ask
 * for each n that a workspace is to serve, and take the largest.
 * ------------------------------------------------------------------------- */
size_t tq_fp8_linear_workspace_size(int64_t n, int K, int N);
int tq_fp8_linear(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales, int64_t n, int K,
                  int N, void* workspace, size_t workspace_bytes, void* y, int y_type, tq_stream_t stream);
size_t tq_fp8_moe_workspace_size(int64_t n, int top_k, int E, int K, int N);
int tq_fp8_moe_forward(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                       const int32_t* topk_ids, const float* topk_w, int64_t n, int top_k, int E, int K, int N,
                       void* workspace, size_t workspace_bytes, void* y, int y_type, tq_stream_t stream);
size_t tq_fp8_moe_mlp_workspace_size(int64_t n, int top_k, int E, int H, int I);
int tq_fp8_moe_mlp_forward(const uint8_t* x, const float* x_scales, const uint8_t* w_gu, const float* gu_scales,
                           const uint8_t* w_down, const float* down_scales, const int32_t* topk_ids,
                           const float* topk_w, int64_t n, int top_k, int E, int H, int I, void* workspace,
                           size_t workspace_bytes, void* y, int y_type, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Gated projection in 16 bits (type TQ_BF16 or TQ_FP16), with its gradient:
 *   gate|up = x W_gu^T, h = silu(gate) * up, sums in fp32, h rounded once.
 * x    (device) n rows of H values, x_stride elements apart (a multiple of 8, base
 *   16-byte aligned).
 * w_gu (device) [2I][H], rows 0..I-1 the gate, I..2I-1 the up projection, 16-byte
 *   aligned.  H and I are multiples of 8.
 * h (device) [n][I], 16-byte aligned, or NULL when only gate_up is wanted.
 * gate_up (device) fp32 [n][2I], 16-byte aligned, or NULL: gate and up as the
 *   gradient takes them (fp32: their roundings to 16 bits would be as large as the
 *   one of d below).
 * workspace (device, 256-byte aligned) of tq_swiglu_linear_workspace_size() bytes (0
 *   on invalid arguments; 256, or a NULL workspace, where none is needed).  The size,
 *   and that of the gradient's, does not grow with n throughout: ask for each n that a
 *   workspace is to serve, and take the largest.
 *
 * tq_swiglu_linear_backward: from grad_h (device, [n][I] dense, 16-byte aligned)
 *   dgate = grad_h * up * s * (1 + gate * (1 - s)), dup = grad_h * gate * s,
 *   s = 1 / (1 + exp(-gate)), as rows d = [dgate dup] rounded to the type (the
 *   products' operands have 16 bits), then grad_x = d W_gu (dense [n][H]) and
 *   grad_w_gu = d^T x ([2I][H]), either may be NULL, 16-byte aligned.  gate_up is
 *   the forward call's, or NULL: computed again from x and w_gu.  Sums have a fixed
 *   order.  workspace (device, 256-byte aligned) of
 *   tq_swiglu_linear_backward_workspace_size() bytes (0 on invalid arguments).
 * Outputs and workspace may not share memory with x, w_gu or each other, the workspace
 * not with grad_h or gate_up either (grad_x may lie over those).  Limits: n, 2I and H
 * below 2^31 - 1024, products of two of them below 2^57.
 * ------------------------------------------------------------------------- */
size_t tq_swiglu_linear_workspace_size(int64_t n, int H, int I);
int tq_swiglu_linear(const void* x, int type, int64_t x_stride, const void* w_gu, int64_t n, int H, int I,
                     void* workspace, size_t workspace_bytes, void* h, float* gate_up, tq_stream_t stream);
size_t tq_swiglu_linear_backward_workspace_size(int64_t n, int H, int I, int has_gate_up);
int tq_swiglu_linear_backward(const void* x, int type, int64_t x_stride, const void* w_gu, const float* gate_up,
                              const void* grad_h, int64_t n, int H, int I, void* workspace, size_t workspace_bytes,
                              void* grad_x, void* grad_w_gu, tq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Diagnostics
 * ------------------------------------------------------------------------- */

/* Reads and clears the current device's error word (synchronizes the device).
 * *code (host) receives 0 or the first TQ_ERR_* recorded by a kernel since the
 * last read; *where (host, may be NULL) a kernel-specific location tag. */
int tq_device_error(int* code, int* where);

/* Rate of the resource that bounds the trellis decode: every SM loads the
 * 65536-entry fp16/bf16 `table` (device, 16-byte aligned) into shared memory
 * and its `warps_per_sm` (1..32) warps each perform iters x 16 random 16-bit
 * lookups in it.  cycles (device) [SM count] receives each SM's clock cycles
 * for the lookups; sink (device) [SM count x warps_per_sm x 32] receives one
 * word per thread so no load is dead.  Lookups per clock per SM =
 * warps_per_sm * 32 * iters * 16 / cycles. */
int tq_probe_lut_rate(const uint16_t* table, int warps_per_sm, int iters, uint32_t* sink,
                      unsigned long long* cycles, tq_stream_t stream);

/* The bounded device-side wait ([P2] "The two changes": a failed or stuck
 * launch must surface as an error, never as a silent result): launches one
 * kernel whose single thread waits, through the same bounded mbarrier wait the
 * pipelined kernels use, on a barrier that nothing arrives on, with a limit of
 * timeout_ns (1e3 .. 2e9).  The wait gives up, records TQ_ERR_DEVICE_TIMEOUT
 * (location tag 10) in the device error word and the kernel returns, leaving
 * the context usable.  out (device) int[2], 4-byte aligned: out[0] = 1 if the
 * wait completed (0 expected), out[1] = microseconds waited.  Returns
 * TQ_ERR_INVALID_ARG on a bad argument, else the launch status. */
int tq_probe_wait_timeout(int64_t timeout_ns, int* out, tq_stream_t stream);

/* Host-side counts of successful launches since process start, per kernel:
 * out[0] route, out[1] tile map, out[2] grouped GEMM (trellis or dense),
 * out[3] GEMV, out[4] combine, out[5] activation gather, out[6] router
 * top-k, out[7] dequantize, out[8] route and tile map fused in one launch
 * (clearing y32 in its other blocks), out[9] accumulator clear (the GEMV
 * arms), out[10] SwiGLU ([P3]: counters prove which arm ran). */
#define TQ_NUM_LAUNCH_COUNTERS 11
void tq_launch_counts(int64_t out[TQ_NUM_LAUNCH_COUNTERS]);

/* The same and the counters that came later: out[11] scored router, out[12] its
 * backward, out[13] 4-bit quantise, out[14] dequantise, out[15] scale tiling,
 * out[16] activation staging, out[17] 4-bit GEMM, out[18] combine (of
 * 4- and 8-bit products, and of K splits),
 * out[19] SwiGLU staging, out[20] 4-bit GEMV, out[21] RMS norm, out[22] its
 * gradient, out[23] the sum of its weight's gradient, out[24] 8-bit quantise,
 * out[25] dequantise, out[26] 8-bit product, out[27] product with few rows (8 or 16
 * bits), out[28] 16-bit product, out[29] sum of a gated projection's K splits, out[30]
 * gradient of the gated activation.  Writes the first `capacity` of them and returns how
 * many there are. */
#define TQ_NUM_ALL_LAUNCH_COUNTERS 31
int tq_launch_counts_all(int64_t* out, int capacity);

#ifdef __cplusplus
}
#endif
#endif /* TQMOE_H */
