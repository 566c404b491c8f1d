/*
 * himuon.h -- C ABI of libhimuon, the HiMuon (Hierarchical Muon) optimizer step on
 * AMD Instinct MI355X (gfx950).
 *
 * The operation is the one described in "Hierarchical Muon: Tiled Newton-Schulz
 * Updates for Efficient Muon Optimization" (Abstract): every momentum-gradient
 * matrix is cut into T x T tiles, the same finite Newton-Schulz (NS) map runs on
 * each tile independently, and the tile results are put back in place and applied
 * to the weights.  The page names tile-size-dependent GPU kernels, cross-layer
 * batching, memory-bounded chunking and runtime tile-size schedules as what this
 * structure allows; this library provides each of them.
 *
 * One step, for every layer (W fp32 H x W weights, M momentum, G gradient):
 *   M <- beta * M + G                       (formed as one fp32 fused multiply-add,
 *                                            stored in the momentum dtype, RNE)
 *   for every tile Y of M (row-major grid anchored at (0,0), ragged edge tiles
 *   kept at their own h x w size; T = HIMUON_TILE_FULL or T >= max(H, W) is one
 *   tile per matrix):
 *     X = Y / (||Y||_F + eps), transposed when h > w so that X is r x s, r <= s
 *     K times:  A = X X^T;  X <- a X + (b A + c A^2) X
 *     O_tile = X (transposed back when h > w)
 *   W <- W - lr * O
 * The coefficients (a, b, c) are a parameter: cubic (1.5, -0.5, 0) and quintic
 * (3.4445, -4.7750, 2.0315) are the two shipped settings.
 *
 * Conventions for every entry point:
 *  - returns himuon_status; never throws; never blocks on the GPU except where
 *    stated; a failure leaves a message in himuon_last_error() (per thread).
 *  - matrices are row-major; ld_* are leading dimensions in elements (>= cols).
 *  - all device pointers are owned by the caller and must stay valid while a
 *    step that uses them is in flight.  Layers must not alias one another.
 */
#ifndef HIMUON_H
#define HIMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define HIMUON_API __attribute__((visibility("default")))
#else
#define HIMUON_API
#endif

typedef enum {
  HIMUON_OK = 0,
  HIMUON_EINVAL = -1,       /* bad argument, shape, leading dimension or config   */
  HIMUON_EBUDGET = -2,      /* workspace budget below what one tile needs          */
  HIMUON_ENOMEM = -3,       /* host or device allocation failed                    */
  HIMUON_EDEVICE = -4,      /* HIP runtime error (launch, copy, no device)         */
  HIMUON_EUNSUPPORTED = -5  /* valid request the library does not implement        */
} himuon_status;

/* storage dtype of momentum and gradient */
typedef enum { HIMUON_F32 = 0, HIMUON_BF16 = 1 } himuon_dtype;

/* arithmetic of the NS matrix products (all accumulate in fp32) */
typedef enum {
  HIMUON_PREC_F32 = 0,    /* fp32 operands (fp32 MFMA)                                  */
  HIMUON_PREC_BF16 = 1,   /* operands rounded once to bf16, one bf16 MFMA per product   */
  HIMUON_PREC_BF16X3 = 2, /* operands split x = hi + lo (both bf16), three bf16 products
                             hi*hi + hi*lo + lo*hi per product: fp32-class accuracy at
                             3x the bf16 MFMA work                                       */
  HIMUON_PREC_BF16F8 = 3  /* the same split, with the two correction products hi*lo and
                             lo*hi on e4m3 (fp8) MFMA at twice the bf16 rate: 2x the bf16
                             MFMA time; each fp8 operand carries a power-of-two scale
                             chosen at plan time from bounds on the iterates.  Fused tiles
                             of edge 64 and 128 run it; smaller tiles and the large-tile
                             path run HIMUON_PREC_BF16X3 (256-tiles and 256-blocks with
                             the plain early Gram and square below).  On tiles that fill
                             64 x 64 or 128 x 128, the Gram product of NS step 0 and the
                             square product of steps 0 and 1 use the bf16 hi operands
                             alone, and on dense 128-tiles (full, 16-byte aligned rows)
                             so do the Gram and B X products of step 1 and the B X
                             product of step 0 (never the last step's B X); other
                             128-tiles keep the split square and update.
                             The a X term of each step is added in fp32 from X
                             held to about 2^-17 (bf16 hi + lo, or fp32), not through the
                             e4m3 operands, so rounding noise does not build up in the
                             empty directions of low-rank tiles.  himuon_plan returns
                             HIMUON_EINVAL if the coefficients' iterates are unbounded.   */
} himuon_precision;

#define HIMUON_TILE_FULL 0            /* one tile per matrix: full-matrix Muon        */
#define HIMUON_FLAG_WRITE_UPDATE 1u   /* also store O (fp32) to layer.update          */
/* Test mode: the step runs the momentum update, the gather of every tile (oriented on its
   short side) and the scatter back, with no normalisation and no Newton-Schulz step, so
   O = M as stored.  O, W <- W - lr O and, with HIMUON_FLAG_WRITE_UPDATE, U = O are
   bit-exact copies of the stored momentum whenever the path holds X in fp32
   (HIMUON_PREC_F32) or the state is bf16; it checks tile indexing and reassembly.  The
   plan's steps and coefficients are ignored while it is set.                          */
#define HIMUON_FLAG_IDENTITY_MAP 2u

typedef struct { double a, b, c; } himuon_coeffs;

typedef struct {
  int64_t rows, cols;            /* H, W                                               */
  int64_t ld_w, ld_m, ld_g, ld_u;/* leading dimensions in elements, >= cols            */
  float *weight;                 /* device, fp32 master weights, updated in place      */
  void *momentum;                /* device, state dtype, updated in place              */
  const void *grad;              /* device, state dtype, read only                     */
  float *update;                 /* device fp32 H x W or NULL; written when the plan has
                                    HIMUON_FLAG_WRITE_UPDATE                           */
} himuon_layer;

typedef struct {
  int32_t tile;                  /* T >= 1, or HIMUON_TILE_FULL                        */
  int32_t steps;                 /* K >= 0                                             */
  himuon_coeffs coeffs;          /* (a, b, c)                                          */
  float beta;                    /* momentum factor, e.g. 0.95                         */
  float eps;                     /* normaliser guard, e.g. 1e-7 (>= 0); a zero tile maps
                                    to zero for every eps, 0 included.  ||Y||_F is
                                    formed in fp32; where the sum of squares leaves
                                    [2^-100, 2^100] it is recomputed from the tile
                                    scaled by a power of two, so very large and very
                                    small tiles normalise as in exact arithmetic (on
                                    the large-tile path while ||Y||_F < 2^126)         */
  size_t workspace_budget;       /* bytes of caller workspace the plan may use         */
  himuon_dtype state_dtype;      /* dtype of momentum and grad, same for all layers    */
  himuon_precision precision;    /* arithmetic of the NS products                      */
  uint32_t flags;                /* HIMUON_FLAG_*                                      */
} himuon_config;

typedef struct {
  int32_t tile;                  /* current T (0 = FULL)                               */
  int32_t kernel_tile;           /* LDS tile edge of the fused kernel (32/64/128), or 0
                                    when the large-tile GEMM path runs                 */
  int64_t layers, tiles;         /* tiles of the current partition                     */
  int64_t fused_tiles;           /* tiles run by the fused kernel                      */
  int64_t gemm_tiles;            /* tiles run by the large-tile GEMM path              */
  int64_t chunks;                /* launches groups of the GEMM path (>= 1 if any)     */
  size_t workspace_bytes;        /* workspace one step needs (<= budget)               */
  size_t table_bytes;            /* device bytes of the descriptor tables              */
  double ns_flops;               /* algorithmic NS flops per step:
                                    sum over tiles K (4 r^2 s + 2 r^3 [c != 0])        */
  double issued_flops;           /* MFMA flops issued per step (padding, symmetric
                                    blocks and the BF16X3 split included)              */
  double step_bytes;             /* algorithmic HBM bytes per step: G, M read, M
                                    written (state dtype), W read and written (fp32)   */
} himuon_stats;

typedef struct {
  int32_t layer;                 /* index into the plan's layer list                   */
  int32_t transposed;            /* 1 when h > w (iterated on the transpose)           */
  int64_t row0, col0, rows, cols;/* tile origin and size inside its matrix             */
} himuon_tile;

/* Runtime calls a plan has made so far (for callers that must know which calls allocate
   or wait): device allocations, pinned host allocations, and host waits on the GPU
   (blocking copies, event waits).  himuon_step adds to none of them. */
typedef struct {
  int64_t device_allocs;
  int64_t host_allocs;
  int64_t host_waits;
} himuon_runtime_counts;

typedef struct himuon_plan_s himuon_plan_t;

/* Validate the layers and config and build the tile-descriptor table over all layers
 * (row-major tiles, layers in order), the chunk list of the large-tile path and the
 * workspace layout.  The plan binds to the current HIP device: it allocates the device
 * copy of the tables there and uploads it with a blocking copy.  When no GPU is
 * visible the plan is host-only (stats and tiles work; himuon_step returns EDEVICE).
 * The layer array is copied; the layers' device pointers are not touched.  EINVAL: bad
 * shape/ld/pointer/config, including coefficients that are not finite in fp32, a
 * nonzero c that rounds to zero in fp32, or |b / c| > 2^100 (the kernels accumulate
 * c A^2 + b A as c ((b / c) A + A^2) in fp32); EBUDGET: the budget cannot hold the
 * workspace of the largest single tile; ENOMEM / EDEVICE: the device tables could not be
 * allocated or copied.  */
HIMUON_API himuon_status himuon_plan(const himuon_layer *layers, int32_t n_layers,
                          const himuon_config *cfg, himuon_plan_t **out);

/* Workspace bytes one step of this plan needs (<= cfg.workspace_budget; 0 when every
 * tile runs in the fused kernel). */
HIMUON_API himuon_status himuon_workspace_size(const himuon_plan_t *p, size_t *bytes);

/* Enqueue one full step (momentum, tiled NS, weight update) for every layer on
 * hip_stream (a hipStream_t; NULL = the default stream).  workspace is a device
 * buffer of at least himuon_workspace_size bytes (may be NULL when that is 0).
 * Enqueue only: it allocates nothing and never waits for the GPU, so it may be
 * captured into a HIP graph.  Steps and tile-size changes of one plan go on one
 * stream (or the caller orders them).  EINVAL: workspace too small, non-finite lr,
 * another current device than the plan's; EDEVICE: a launch failed, or the plan is
 * host-only. */
HIMUON_API himuon_status himuon_step(himuon_plan_t *p, void *workspace, size_t ws_bytes,
                          float lr, void *hip_stream);

/* Change T between steps (runtime tile-size schedule).  Rebuilds the tables on the
 * host and enqueues their upload on hip_stream into the plan's second device buffer
 * (the one the steps before the last change read), so steps enqueued later on that
 * stream use the new T and steps already queued keep theirs.  It allocates only when
 * the new tables outgrow that buffer or its pinned staging (outgrown buffers are kept
 * until himuon_plan_destroy), and waits only when the staging is still being read by
 * the upload of the change before the previous one.  A new T whose workspace exceeds
 * the budget gives more chunks, not an error, unless a single tile does not fit
 * (EBUDGET); on any error the plan keeps its current T. */
HIMUON_API himuon_status himuon_set_tile_schedule(himuon_plan_t *p, int32_t tile, void *hip_stream);

/* Runtime calls (allocations, host waits) the plan has made since himuon_plan. */
HIMUON_API himuon_status himuon_plan_runtime_counts(const himuon_plan_t *p, himuon_runtime_counts *out);

/* For callers that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): himuon_step with the large-tile
 * path's workspace taken from a static per-device array of
 * HIMUON_STATIC_WORKSPACE_BYTES (each GPU the library runs on holds its own copy until
 * the process ends) instead of a caller buffer.  It allocates nothing and never waits
 * for the GPU.  Plans that need no workspace (every tile in the fused kernel) run as
 * with himuon_step.  Calls on one GPU share the array, so steps that overlap on one
 * device (on different streams, or from different threads) race on it; the array
 * needs no clearing (each step writes every workspace byte it reads).  EBUDGET: the
 * plan's workspace exceeds HIMUON_STATIC_WORKSPACE_BYTES (plan with a workspace_budget
 * at most that large: the large-tile path then runs in more chunks); other errors as
 * for himuon_step. */
#define HIMUON_STATIC_WORKSPACE_BYTES (64u << 20)
HIMUON_API himuon_status himuon_step_static(himuon_plan_t *p, float lr, void *hip_stream);

/* Counters of the current partition. */
HIMUON_API himuon_status himuon_plan_stats(const himuon_plan_t *p, himuon_stats *out);

/* Copy up to cap tile descriptors (in table order) into out; *n receives the total
 * number of tiles.  out may be NULL with cap 0 to query the count. */
HIMUON_API himuon_status himuon_plan_tiles(const himuon_plan_t *p, himuon_tile *out, int64_t cap,
                                int64_t *n);

/* Release the plan and its device tables.  The caller synchronises the stream of
 * the last step first. */
HIMUON_API void himuon_plan_destroy(himuon_plan_t *p);

/* Message of the last failure on this thread ("" if none). */
HIMUON_API const char *himuon_last_error(void);

/* The momentum and weight update of the step with the map O = M, over one flat run of n
   elements and no tiling: M <- beta M + G (one fp32 fused multiply-add, stored in
   state_dtype with round-to-nearest-even), W <- W - lr M (M as stored).  It moves the
   bytes of a step's memory pass (the momentum and weight lines of the step described at
   the top of this file) and nothing else, so its rate is the HBM rate that read/write mix
   reaches on the device: the reference against which the tiled step's memory pass is
   measured.  For the same values its M and W are bit-exact to himuon_step's with
   HIMUON_FLAG_IDENTITY_MAP (bf16 state, or fp32 state with HIMUON_PREC_F32).  m, g: device arrays of n elements of
   state_dtype (HIMUON_F32 or HIMUON_BF16); w: device fp32, n elements; when all three
   are 16-byte aligned the kernel moves 8 elements per thread and turn.  Enqueued on
   hip_stream.  EINVAL: NULL pointers with n > 0, n < 0, a bad dtype, non-finite beta or
   lr.  EDEVICE: launch failure.                                                       */
HIMUON_API himuon_status himuon_stream_step(void *m, const void *g, float *w, int64_t n,
                                            himuon_dtype state_dtype, float beta, float lr,
                                            void *hip_stream);

/* ---- Sign-Muon, local pieces ----------------------------------------------------
   "Sign-Muon: Communication-Efficient Distributed Muon Optimization" (Figures 1 and 6):
   a worker forms the entrywise sign S in {-1, +1} of its Newton-Schulz direction, packs
   it to one bit per entry for an all-gather, and takes the majority vote of the gathered
   buffers locally.  The collective itself is not part of this library.                */

/* Packs sign(o) of a rows x cols fp32 device matrix (row-major, leading dimension
   ld >= cols) into `bits` (device, 8-byte aligned, ceil(rows * cols / 8) bytes, written
   in full): entry k = i * cols + j is bit k % 8 (least significant first) of byte k / 8,
   1 for o >= 0 (so sign(0) = +1), 0 otherwise (NaN included).  Enqueued on hip_stream.
   EINVAL: NULL pointers with rows * cols > 0, negative sizes, ld < cols, misaligned bits.
   EDEVICE: launch failure.                                                            */
HIMUON_API himuon_status himuon_sign_pack(const float *o, int64_t rows, int64_t cols, int64_t ld,
                                          uint8_t *bits, void *hip_stream);

/* Majority vote over the packed sign buffers of `workers` workers (1..255), worker m's
   buffer at bits + m * stride (device; bits and stride 4-byte aligned, stride >=
   ceil(n / 8)): out[k] = +scale if at least half of the workers have bit k set, else
   -scale, for k < n (a tie counts as +1).  out: device array of n elements of out_dtype
   (HIMUON_F32 or HIMUON_BF16).  Enqueued on hip_stream.  EINVAL on bad arguments,
   EDEVICE on launch failure.                                                          */
HIMUON_API himuon_status himuon_sign_vote(const uint8_t *bits, int32_t workers, int64_t stride, int64_t n,
                                          himuon_dtype out_dtype, void *out, float scale, void *hip_stream);

/* ---- The rest of a training step ----------------------------------------------------
   HiMuon updates a model's matrices.  The entry points below are what stands next to it
   in a training step: the loss with its gradient, the norm of a gradient with its
   clip factor, and AdamW for every parameter that is not a matrix.  They are stateless
   (no plan): the arrays of descriptors are read on the host during the call and may be
   reused at once.  They enqueue only: no allocation, no wait for the GPU, so they may be
   captured into a HIP graph (with the arguments of the capturing call).               */

/* Clipped policy loss with a KL term, over `rows` sampled tokens with `vocab` logits each.
   With z = logits / temperature, lp = z[label] - log sum_j exp z[j],
     rho = exp(lp - old_logp) (1 where old_logp is NULL), u = rho A,
     c = min(max(rho, 1 - clip_low), 1 + clip_high) A,
     kl = exp(ref_logp - lp) - (ref_logp - lp) - 1 (0 where ref_logp is NULL),
     loss = sum over rows of weight (kl_coef kl - min(u, c))
   and, where dlogits is not NULL, with p = softmax(z) and old_logp a constant (where
   it is NULL, too: the gradient at rho = 1),
     dlogits[j] = grad_scale weight / temperature
                  (-(u <= c ? u : 0) + kl_coef (1 - exp(ref_logp - lp))) ((j == label) - p[j]).
   A row whose weight is zero or whose label is outside [0, vocab) is left out: nothing of
   its logits, advantage or log probabilities is read, its logp is 0, its dlogits are 0 and
   it adds nothing to the sums.  Logits of -inf have probability 0; a row with NaN or +inf
   among its logits, or with nothing but -inf, gives NaN.  With kl_coef 0 the KL term is
   only summed (stats[2]): it is no part of loss and gradient, infinite or not.          */
typedef struct {
  int64_t rows, vocab;           /* >= 0, >= 1                                          */
  int64_t ld_logits, ld_dlogits; /* leading dimensions in elements, >= vocab            */
  const void *logits;            /* device, dtype                                       */
  void *dlogits;                 /* device, dtype, or NULL: no gradient.  May be logits
                                    itself (ld_dlogits == ld_logits); must not overlap it
                                    otherwise                                           */
  const int64_t *label;          /* device, rows                                        */
  const float *weight;           /* device, rows                                        */
  const float *advantage;        /* device, rows                                        */
  const float *old_logp;         /* device, rows, or NULL                               */
  const float *ref_logp;         /* device, rows, or NULL                               */
  float *logp;                   /* device, rows: lp                                    */
  float *stats;                  /* device, 4: loss, and the sums over rows of weight
                                    times -min(u, c), kl, and [u > c] (clipped)         */
  himuon_dtype dtype;            /* of logits and dlogits                               */
  double clip_low, clip_high;    /* >= 0, clip_low <= 1                                 */
  double kl_coef;                /* finite                                              */
  double temperature;            /* in [2^-20, 2^20]                                    */
  double grad_scale;             /* finite; multiplies dlogits only                     */
} himuon_policy;

/* Workspace bytes himuon_policy_loss needs for this call (device memory, 16-byte aligned,
   contents immaterial). */
HIMUON_API himuon_status himuon_policy_workspace(const himuon_policy *p, size_t *bytes);

/* Enqueues the loss (and its gradient) on hip_stream.  Sums over rows and over the
   vocabulary have a fixed order: the same call gives the same bits.  EINVAL: NULL
   pointers with rows > 0 (stats always), bad sizes, leading dimensions, scalars or dtype,
   a short or misaligned workspace.  EDEVICE: launch failure.                           */
HIMUON_API himuon_status himuon_policy_loss(const himuon_policy *p, void *workspace, size_t ws_bytes,
                                            void *hip_stream);

/* Entries of a teacher's row at most, and tokens of a vocabulary in the three calls below. */
#define HIMUON_TOP_MOST 1024
#define HIMUON_TOP_VOCAB (1 << 20)

/* Sampling a token from each of `rows` rows of `vocab` logits, from given random numbers.
   With T the row's temperature, e_i = exp((logits[i] - max) / T) and the row's tokens in the order
   of their logits from the largest, equal ones by index (-0 equals 0), the filters keep the first
     n = min(top_k, the smallest n whose e sum to top_p of what the first top_k sum to,
             the number of tokens with e_i >= min_p)
   of them, one at least: top_k outside [1, vocab] and top_p not below 1 keep all, a top_p of 0 or
   less keeps one, min_p not above 0 keeps all and counts as 1 above 1.  The token is the first one,
   by index among those kept, up to which their e sum to more than uniform times the sum over all
   that are kept: with uniform drawn from [0, 1), each with its share of probability (a uniform
   outside of that counts as its nearest end, NaN as 0).  Then
     logp = log of the token's probability under softmax(logits / T), filters aside: old_logp of
            himuon_policy_loss with that temperature,
     kept = the probability that all kept tokens have there.
   T = 0 takes the first of the largest logits (logp 0, kept 1).  Tokens of -inf are never taken (and
   a uniform of 0 passes over tokens with e_i below 2^-1000, and may from 2^-960 down); a row with
   NaN or +inf among its logits or with nothing but -inf, and a row_temperature that is neither 0
   nor in [2^-20, 2^20], give token -1 and NaN.  Borders are decided as 64-bit sums of the formulas
   above decide them. */
typedef struct {
  int64_t rows, vocab;           /* >= 0, in [1, HIMUON_TOP_VOCAB]                      */
  int64_t ld_logits;             /* leading dimension in elements, >= vocab             */
  const void *logits;            /* device, dtype                                       */
  const float *uniform;          /* device, rows                                        */
  const float *row_temperature;  /* device, rows, each: in the place of the number      */
  const int32_t *row_top_k;      /*   below for all rows, or NULL                       */
  const float *row_top_p;
  const float *row_min_p;
  int64_t *token;                /* device, rows                                        */
  float *logp, *kept;            /* device, rows                                        */
  himuon_dtype dtype;
  int32_t top_k;
  double temperature;            /* 0 or in [2^-20, 2^20]                               */
  double top_p, min_p;           /* not NaN                                             */
} himuon_sampling;

/* Workspace bytes himuon_sample needs for this call (device memory, 16-byte aligned, contents
   immaterial; may be 0). */
HIMUON_API himuon_status himuon_sample_workspace(const himuon_sampling *p, size_t *bytes);

/* Enqueues the draws on hip_stream; the same call gives the same bits.  EINVAL: NULL pointers with
   rows > 0, bad sizes, leading dimension, scalars or dtype, a short or misaligned workspace.
   EDEVICE: launch failure. */
HIMUON_API himuon_status himuon_sample(const himuon_sampling *p, void *workspace, size_t ws_bytes, void *hip_stream);

/* The k largest logits of each of `rows` rows, from the largest, equal ones by index (-0 equals 0,
   NaN is larger than every number), with their indices, and what is left:
     rest = log of the sum over all other tokens of exp(logits / temperature),
   -inf where there is none or all are -inf, NaN where NaN or +inf is among them. */
typedef struct {
  int64_t rows, vocab;           /* >= 0, in [1, HIMUON_TOP_VOCAB]                      */
  int64_t ld_logits, ld_top;     /* leading dimensions: of logits, >= vocab; of value and
                                    index, >= k                                         */
  const void *logits;            /* device, dtype                                       */
  void *value;                   /* device, dtype, rows x k                             */
  int64_t *index;                /* device, rows x k                                    */
  float *rest;                   /* device, rows                                        */
  int32_t k;                     /* in [1, min(vocab, HIMUON_TOP_MOST)]                 */
  himuon_dtype dtype;
  double temperature;            /* in [2^-20, 2^20]                                    */
} himuon_top;

/* Workspace bytes himuon_top_logits needs for this call (as above). */
HIMUON_API himuon_status himuon_top_workspace(const himuon_top *p, size_t *bytes);

/* Enqueues the selection on hip_stream; the same call gives the same bits.  Errors as for
   himuon_sample. */
HIMUON_API himuon_status himuon_top_logits(const himuon_top *p, void *workspace, size_t ws_bytes, void *hip_stream);

/* Distillation from a teacher's top logits, over `rows` tokens with `vocab` student logits each.
   Entry j of a row (j < k) names token v_j = index[j] with the teacher's logit value[j]; an entry
   whose index is outside [0, vocab) does not count.  rest, where given, is the log-sum-exp of the
   teacher's other logits over the temperature (himuon_top_logits leaves it), one class more.  With
     q = softmax over the row's entries of value / temperature (and of rest),
     p = softmax(logits / temperature), p_rest = the sum of p over the tokens that no entry names,
     kl = sum_j q_j (log q_j - log p[v_j])  (+ q_rest (log q_rest - log p_rest)),
     loss = sum over rows of weight kl
   and, where dlogits is not NULL,
     dlogits[u] = grad_scale weight / temperature (p[u] - sum of q_j over the entries that name u),
   for a token u that no entry names grad_scale weight / temperature p[u] (1 - q_rest / p_rest)
   (q_rest = 0 without rest).  Terms with q = 0 are 0.  A token that more than one entry names is
   one of the tokens that are named, and each of its entries counts.  A row whose weight is zero, or
   whose teacher has no probability anywhere (no entry that counts and is not -inf, no rest that is
   not -inf), is left out: its kl and dlogits are 0; with weight zero nothing else of it is read.
   Logits of -inf have probability 0 (and an infinite kl where the teacher gives them some); a row
   with NaN or +inf among its student's or its teacher's logits that count, or with nothing but
   -inf, gives NaN. */
typedef struct {
  int64_t rows, vocab;           /* >= 0, in [1, HIMUON_TOP_VOCAB]                      */
  int64_t ld_logits, ld_dlogits; /* leading dimensions in elements, >= vocab            */
  int64_t ld_top;                /* of value and index, >= k                            */
  const void *logits;            /* device, dtype                                       */
  void *dlogits;                 /* device, dtype, or NULL: no gradient.  May be logits
                                    itself (ld_dlogits == ld_logits); must not overlap it
                                    otherwise                                           */
  const void *value;             /* device, value_dtype, rows x k                       */
  const int64_t *index;          /* device, rows x k                                    */
  const float *rest;             /* device, rows, or NULL: q is over the entries alone  */
  const float *weight;           /* device, rows                                        */
  float *kl;                     /* device, rows                                        */
  float *loss;                   /* device, 1                                           */
  int32_t k;                     /* in [1, HIMUON_TOP_MOST]                             */
  himuon_dtype dtype;            /* of logits and dlogits                               */
  himuon_dtype value_dtype;
  double temperature;            /* in [2^-20, 2^20]                                    */
  double grad_scale;             /* finite; multiplies dlogits only                     */
} himuon_distill;

/* Workspace bytes himuon_distill_loss needs for this call (device memory, 16-byte aligned,
   contents immaterial; may be 0). */
HIMUON_API himuon_status himuon_distill_workspace(const himuon_distill *p, size_t *bytes);

/* Enqueues the loss (and its gradient) on hip_stream.  All sums have a fixed order: the same call
   gives the same bits.  EINVAL: NULL pointers with rows > 0 (loss always), bad sizes, leading
   dimensions, scalars or dtypes, a short or misaligned workspace.  EDEVICE: launch failure. */
HIMUON_API himuon_status himuon_distill_loss(const himuon_distill *p, void *workspace, size_t ws_bytes,
                                             void *hip_stream);

/* One tensor of a gradient: n contiguous elements on the device. */
typedef struct {
  int64_t n;
  const void *grad;
} himuon_grad;

/* Workspace bytes of himuon_grad_norm over n_tensors tensors (16-byte aligned).  Its first
   eight bytes must be zero before its first call; every call leaves them zero.  Calls that
   share a workspace go on one stream (or the caller orders them). */
HIMUON_API himuon_status himuon_grad_norm_workspace(int32_t n_tensors, size_t *bytes);

/* out[0] = the 2-norm of all tensors together, out[1] = the factor that clips it:
   min(1, max_norm / (norm + 1e-6)), or NaN where the norm is not finite in exact arithmetic
   (an infinity or a NaN among the elements).  Squares are summed in fp64 in a fixed order, so
   no finite gradient overflows.  out: device, two floats.  EINVAL: bad arguments
   (max_norm is finite and >= 0), short or misaligned workspace.  EDEVICE: launch failure. */
HIMUON_API himuon_status himuon_grad_norm(const himuon_grad *tensors, int32_t n_tensors, himuon_dtype dtype,
                                          double max_norm, float *out, void *workspace, size_t ws_bytes,
                                          void *hip_stream);

/* Elements that share one scale of the 8-bit AdamW states. */
#define HIMUON_ADAMW_BLOCK 256

/* One parameter tensor of an AdamW step: n contiguous elements (any element alignment). */
typedef struct {
  int64_t n;
  void *weight;                  /* device, weight_dtype, updated in place              */
  const void *grad;              /* device, grad_dtype                                  */
  void *m, *v;                   /* device, updated in place; state_bits 32: fp32, the first
                                    and second moment.  state_bits 8: OCP e4m3 bytes, the
                                    first moment and the square root of the second      */
  float *m_scale, *v_scale;      /* device, ceil(n / HIMUON_ADAMW_BLOCK) each, updated in
                                    place: element i of m holds m[i] m_scale[i / 256]
                                    (v, v_scale likewise).  8-bit states only           */
  double weight_decay;           /* decoupled decay of this tensor                      */
} himuon_adamw_tensor;

typedef struct {
  himuon_dtype weight_dtype, grad_dtype;
  int32_t state_bits;            /* 32 or 8                                             */
  double beta1, beta2;           /* in [0, 1)                                           */
  double eps;                    /* >= 1e-30                                            */
} himuon_adamw_config;

/* One AdamW step over all tensors (step number t >= 1), in fp32 per element:
     g <- *grad_scale g (grad_scale: device, one float, or NULL for 1)
     m <- beta1 m + (1 - beta1) g,  v <- beta2 v + (1 - beta2) g^2
     w <- w (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
   with w rounded to nearest even where weight_dtype is bf16.  Where *grad_scale is NaN
   (himuon_grad_norm's factor for a gradient that is not finite) the step changes nothing; t
   is the caller's, who decides whether such a step counts.
   8-bit states: moments and codes are computed in fp32 with every operation rounded on its
   own, in the order of these formulas ((1 - beta2) g first, then times g; r^2 before its
   product with beta2; 448 / peak as the rounded reciprocal times 448), so that any other
   computation in that order gives the same states bit for bit.  Where v overflows fp32 though r
   and g are finite, r is 2^66 times the root of those products of r 2^-66 and g 2^-66 (fp32's
   largest number at most): r is what the states hold.  The weight takes the fp32
   moments; then the step stores m and r = sqrt(v)
   by blocks of 256 elements: peak = the block's largest magnitude, scale = peak / 448, and
   y = |x| 448 / peak rounded to one of its two e4m3 neighbours, up with the probability of
   its distance to the lower one: the upper 16 bits of (i C + dither[k]) mod 2^32, plus one
   half, over 2^16 (i the element's index, k = 0 and C = 0x9E3779B1 for m, k = 1 and C =
   0x85EBCA6B for r) are added to y in units of the neighbours' gap before it is cut off.
   Rounding to nearest would hold a moment still that moves by less than half a gap a step.
   dither: two random numbers of the caller, new ones for each step (host memory; NULL is
   {0, 0}).  A nonzero r is stored as 2^-9 at least, so that no weight is divided by eps
   alone while its m is not zero; a block with peak < 2^-100 is stored as zeros.  Where r is
   not finite, r and an m that is not are stored as the NaN code, and peak is that of the
   block's others: as with 32-bit states only that element is lost.
   table: NULL, or device memory that holds what himuon_adamw_table wrote for these tensors
   and this config: the step is then one launch however many tensors there are; without it
   the descriptors go in the kernel arguments, some 56 (8-bit states) or 72 tensors a launch.
   EINVAL: NULL pointers with n > 0, bad sizes, scalars, dtypes or bits; two tensors
   must not share memory (not checked).  EDEVICE: launch failure.                       */
HIMUON_API himuon_status himuon_adamw_step(const himuon_adamw_tensor *tensors, int32_t n_tensors,
                                           const himuon_adamw_config *cfg, int64_t t, double lr,
                                           const float *grad_scale, const uint32_t *dither, const void *table,
                                           void *hip_stream);

/* Descriptors of many tensors for the device: *bytes is 0 where a table gains nothing (8
   tensors at most), else its size.  himuon_adamw_table writes it into host
   memory (8-byte aligned), from where the caller copies it to device memory (16-byte
   aligned); it holds for as long as no pointer, size or weight_decay of the tensors changes. */
HIMUON_API himuon_status himuon_adamw_table_size(const himuon_adamw_tensor *tensors, int32_t n_tensors,
                                                 const himuon_adamw_config *cfg, size_t *bytes);
HIMUON_API himuon_status himuon_adamw_table(const himuon_adamw_tensor *tensors, int32_t n_tensors,
                                            const himuon_adamw_config *cfg, void *host, size_t bytes);

#ifdef __cplusplus
}
#endif

#endif /* HIMUON_H */
