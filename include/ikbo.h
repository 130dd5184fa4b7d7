/*
 * ikbo.h -- C ABI of libikbo: the IKBO Linear Compression Embedding forward (and its
 * backward) on AMD Instinct MI355X (gfx950), target attention, target attention over
 * cached user histories, and target attention's training.
 *
 * The operation (IKBO recsys blog, "Deep Dive: Linear Compression"; aibriefing
 * article, "kernel deep-dive case 1"):
 *
 *     Y[b] = W_u . U[map[b]]  +  W_c . C[b]          for b < B_c
 *
 * U holds the request-only (user) embeddings at their own batch B_u, C the
 * per-candidate embeddings at batch B_c, and map[b] names the user of
 * candidate b.  The kernels take the two batches "in their natural, mismatched
 * sizes" plus the candidate-to-user map (blog, "Why broadcast is a data-layout
 * problem" and "How the IKBO co-design is built"; aibriefing, RO/NRO paragraph)
 * and never build the replicated tensor U[map].
 *
 * Layouts.  Every tensor is dense row-major (C order) in device memory owned by
 * the caller:
 *     U   [B_u, K_u, D]      C   [B_c, K_c, D]      map [B_c] int32
 *     W_u [M, K_u]           W_c [M, K_c]           Y   [B_c, M, D]
 * U, C, W_u, W_c and Y share one element type (bfloat16 or float32).  Products
 * accumulate in float32; the user partial W_u.U[u] is kept in float32; Y is
 * rounded once (round-to-nearest-even) when it is stored.
 *
 * Threading.  A plan may be used from one host thread and one stream at a
 * time.  Different plans are independent.  No C++ exception crosses this ABI.
 */
#ifndef IKBO_H
#define IKBO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque plan handle; created by ikbo_lce_plan, owned by the library. */
typedef struct ikbo_lce_plan_s *ikbo_lce_plan_t;

/* Status codes returned by every entry point. */
enum {
    IKBO_OK = 0,
    IKBO_ERR_INVALID_ARG = -1,  /* null pointer, bad dimension, shape differs from the plan */
    IKBO_ERR_UNSUPPORTED = -2,  /* valid but not implemented (e.g. D*elt not a multiple of 16 B) */
    IKBO_ERR_HIP = -3,          /* a HIP runtime call failed; see ikbo_last_error_message() */
    IKBO_ERR_ALIGNMENT = -4,    /* a tensor base address is not 16-byte aligned */
    IKBO_ERR_TIMEOUT = -5,      /* device: a candidate tile gave up waiting for its user partial */
    IKBO_ERR_MAP_RANGE = -6,    /* device: some map[b] lies outside [0, B_u) */
    IKBO_ERR_PAGE_RANGE = -7,   /* device: a page, slot, length or position outside its range */
    IKBO_ERR_NO_PAGES = -8,     /* device: a batch needs more pages, table columns or rows than there are */
    IKBO_ERR_NONFINITE = -9     /* device: an infinity or NaN was handed to the 4-bit cache */
};

/* Element type of U, C, W_u, W_c and Y. */
enum { IKBO_DTYPE_BF16 = 0, IKBO_DTYPE_F32 = 1 };

/*
 * Kernel variant.  S0..S4 reproduce the pages' optimisation ladder on CDNA4
 * (blog, "Deep Dive: Linear Compression", stages 1-4; zubnet summary, the
 * four-stage paragraph); all five compute the same Y.
 *   S0  materialise X = [U[map] ; C] in HBM, then one batched GEMM with [W_u | W_c];
 *   S1  decompose by linearity (user GEMM at B_u rows, candidate GEMM at B_c rows),
 *       then materialise P_u[map] and add; unpadded K, 4-byte operand loads;
 *   S2  S1 with K zero-padded and 16-byte operand loads;
 *   S3  user GEMM, then a candidate GEMM whose epilogue gathers P_u[map[b]] by
 *       index and adds it in registers;
 *   S4  one launch: user and candidate tiles overlap, candidate epilogues wait for
 *       their user partial through device-scope release/acquire flags.
 * AUTO selects S4.
 */
enum {
    IKBO_VARIANT_AUTO = 0,
    IKBO_S0_MATERIALISED = 1,
    IKBO_S1_DECOMPOSED = 2,
    IKBO_S2_ALIGNED = 3,
    IKBO_S3_EPILOGUE_FUSED = 4,
    IKBO_S4_PERSISTENT = 5
};

/* Plan flags (host-forced test conditions; production callers pass 0). */
enum {
    IKBO_FLAG_DEBUG_DELAY_USER = 2, /* S4: user tiles sleep before computing (exercises the wait) */
    IKBO_FLAG_DEBUG_SKIP_USER = 4,  /* S4: user tiles publish nothing; candidates time out */
    IKBO_FLAG_BACKWARD = 8,         /* also allocate the workspace of ikbo_lce_backward */
    IKBO_FLAG_DEBUG_POISON_USER = 16 /* each forward first fills the user partials P_u with NaN */
};

/*
 * Create a plan for one shape range ("the compiler needs each operator's
 * dynamic shape range to pick the kernel": blog, co-design section; aibriefing,
 * three-layers paragraph).  Chooses the tile configuration and allocates the
 * device workspace (hipMalloc) on the current device; forward never allocates.
 *   max_B_u, max_B_c  upper bounds of B_u and B_c in later forwards (>= 1, >= 0)
 *   K_u, K_c, M, D    fixed dimensions (>= 1)
 *   dtype             IKBO_DTYPE_*
 *   variant           IKBO_VARIANT_AUTO or IKBO_S*
 * On success stores a handle in *plan and returns IKBO_OK; on failure *plan is
 * left NULL and nothing stays allocated.  Errors: INVALID_ARG, UNSUPPORTED, HIP.
 */
int ikbo_lce_plan(ikbo_lce_plan_t *plan, int max_B_u, int max_B_c, int K_u, int K_c,
                  int M, int D, int dtype, int variant, unsigned flags);

/*
 * Enqueue Y[b] = W_u.U[map[b]] + W_c.C[b] on `stream` (a hipStream_t; NULL =
 * the null stream).  All pointers are device pointers with the layouts above;
 * U, C, W_u, W_c and Y must be 16-byte aligned.  The dimensions must equal the
 * plan's, with 1 <= B_u <= max_B_u and 0 <= B_c <= max_B_c; B_c = 0 is a no-op.
 * Host-side validation errors return before anything is enqueued.  The call is
 * asynchronous: device-side conditions (map entry out of range, S4 wait
 * timeout) are recorded in the plan and reported by ikbo_lce_check; the Y rows
 * of an affected candidate are then unspecified.  Must be called with the
 * plan's device current.
 */
int ikbo_lce_forward(ikbo_lce_plan_t plan, const void *U, const void *C, const int32_t *map,
                     const void *W_u, const void *W_c, void *Y,
                     int B_u, int B_c, int K_u, int K_c, int M, int D, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): the forward above without
 * a plan, calling no hipMalloc, hipFree or other allocating routine.  It computes
 * the same Y as the two-launch gather-add stage (S3) on the streaming engine, and
 * keeps the float32 user partial P_u [B_u, M, D] in a file-scope device array of
 * IKBO_NOALLOC_SCRATCH_BYTES bytes (256 of them reserved) that every GPU the
 * library runs on holds until the process ends.  Limits: bf16 only, D in
 * {32, 64, 128, 160, 192}, and B_u*M*D*4 <= IKBO_NOALLOC_SCRATCH_BYTES - 256;
 * beyond them it returns IKBO_ERR_UNSUPPORTED (ikbo_last_error_message says which)
 * before anything is enqueued.  Arguments, layouts, alignment and the other errors
 * are those of ikbo_lce_forward (the dimensions are not checked against a plan).
 * Every call on one GPU shares that GPU's array: calls that overlap on one GPU
 * (two streams, two host threads) race and may produce wrong Y.  Map entries
 * outside [0, B_u) leave their candidates' Y rows unwritten; this entry point does
 * not report them.  The first call on a device also looks up the array's device
 * address (no allocation).
 */
#define IKBO_NOALLOC_SCRATCH_BYTES (8u << 20)
int ikbo_lce_forward_noalloc(const void *U, const void *C, const int32_t *map,
                             const void *W_u, const void *W_c, void *Y,
                             int B_u, int B_c, int K_u, int K_c, int M, int D, void *stream);

/*
 * Enqueue the gradients of L = <dY, Y> for the forward above (the chain rule of the
 * pages' definition, blog "Deep Dive: Linear Compression", stage 1; the aibriefing
 * article's three-layers paragraph says the kernels serve training when the ratio
 * exceeds 1, but the pages give no training formulas):
 *
 *     dC[b] = W_c^T . dY[b]                    dW_c = sum_b dY[b] . C[b]^T
 *     dU[u] = W_u^T . S[u]                     dW_u = sum_b dY[b] . U[map[b]]^T
 *     S[u]  = sum of dY[b] over the candidates b with map[b] = u
 *
 * The replicated user tensor is not built in this direction either: the user
 * gradient is summed per user first and multiplied at batch B_u.  Requires a plan
 * made with IKBO_FLAG_BACKWARD (bf16, D in {32, 64, 128, 160, 192}; otherwise the
 * plan call returns IKBO_ERR_UNSUPPORTED); the variant does not matter.
 * Layouts (device memory owned by the caller, dense row-major):
 *     dY [B_c, M, D] bf16 (input)         U, C, map, W_u, W_c as for the forward
 *     dU [B_u, K_u, D] bf16 (output)      dC [B_c, K_c, D] bf16 (output)
 *     dW_u [M, K_u] float32 (output)      dW_c [M, K_c] float32 (output)
 * Every output is overwritten, not accumulated into; users that no candidate maps to
 * get dU = 0, and B_c = 0 gives dU = 0 and dW = 0 (dY, C, map and dC may then be NULL).
 * Products accumulate in float32; S is kept in float32 and handed to the bf16 matrix
 * cores as the pair bf16(S) + bf16(S - bf16(S)); dU and dC are rounded once to bf16.
 * Every pointer except map must be 16-byte aligned (map: 4-byte).  Asynchronous, like
 * the forward: map entries outside [0, B_u) are skipped and reported by ikbo_lce_check
 * as IKBO_ERR_MAP_RANGE.  Uses the plan's workspace: do not overlap it with a forward
 * or another backward on the same plan in a different stream.  dC and dU run on two
 * streams that the plan owns, forked from `stream` by events after the work they need
 * and joined back into it before the call returns: work enqueued on `stream` afterwards
 * sees every output (under stream capture the fork and join are captured with it).
 * Errors (before anything is enqueued): INVALID_ARG, ALIGNMENT, UNSUPPORTED, HIP.
 */
int ikbo_lce_backward(ikbo_lce_plan_t plan, const void *dY, const void *U, const void *C,
                      const int32_t *map, const void *W_u, const void *W_c, void *dU, void *dC,
                      float *dW_u, float *dW_c, int B_u, int B_c, int K_u, int K_c, int M, int D,
                      void *stream);

/*
 * Wait for `stream`, then return and clear the device-side status recorded by
 * earlier forwards and backwards on this plan (IKBO_OK, IKBO_ERR_MAP_RANGE or
 * IKBO_ERR_TIMEOUT), or IKBO_ERR_HIP if the wait itself failed.
 */
int ikbo_lce_check(ikbo_lce_plan_t plan, void *stream);

/*
 * Write a NUL-terminated JSON description of the plan (variant, tile sizes,
 * padded K, grid, workspace bytes) into json[0..cap).  Returns the length it
 * needed (excluding the NUL), or a negative status.
 */
int ikbo_lce_plan_info(ikbo_lce_plan_t plan, char *json, size_t cap);

/*
 * Upper bound on the polling iterations a candidate tile spends waiting for a
 * user partial (S4) before it records IKBO_ERR_TIMEOUT and moves on; 0 restores
 * the default.  A test hook: every kernel exits even if a user tile never
 * publishes.
 */
int ikbo_lce_plan_set_spin_limit(ikbo_lce_plan_t plan, uint32_t max_polls);

/* Free the plan and its workspace (synchronises the device first).  NULL is a no-op. */
int ikbo_lce_plan_destroy(ikbo_lce_plan_t plan);

/*
 * IKBO target attention (IKBO recsys blog, "Deep Dive: Flash Attention"): the queries of
 * each candidate attend over the keys and values of its user,
 *
 *     O[b,h] = softmax(scale * Q[b,h] . K[map[b],h]^T) . V[map[b],h]      for b < B_c, h < H
 *
 * with K and V at the user batch B_u, never replicated per candidate.  Layouts (device
 * memory owned by the caller, dense row-major, bf16):
 *     Q, O [B_c, H, L_q, head_dim]      K, V [B_u, H, L_kv, head_dim]      map [B_c] int32
 * Scores, softmax and the weighted sum accumulate in float32 (the softmax weights reach
 * the matrix cores as bf16); O is rounded to bf16 once.  No mask: every query sees all
 * L_kv keys of its user.
 *
 * ikbo_fa_plan: fixed H, L_q, L_kv, head_dim; bf16 only, head_dim 64 or 128, L_q 16, 32
 * or 64 (one wave holds a candidate's queries); any L_kv >= 1.  flags must be 0.
 * Allocates a small workspace (the candidates grouped by user) on the current device.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP.
 */
typedef struct ikbo_fa_plan_s *ikbo_fa_plan_t;
int ikbo_fa_plan(ikbo_fa_plan_t *plan, int max_B_u, int max_B_c, int H, int L_q, int L_kv, int head_dim,
                 int dtype, unsigned flags);

/*
 * Enqueue the attention on `stream`.  scale = 0 means 1/sqrt(head_dim); a negative, NaN or
 * infinite scale is INVALID_ARG.  Q, K, V and O must be 16-byte aligned, map 4-byte.
 * B_c = 0 is a no-op.  Asynchronous: map entries outside [0, B_u) leave their candidates'
 * O unwritten and are reported by ikbo_fa_check as IKBO_ERR_MAP_RANGE.  One plan serves
 * one stream at a time.
 */
int ikbo_fa_forward(ikbo_fa_plan_t plan, const void *Q, const void *K, const void *V, const int32_t *map,
                    void *O, int B_u, int B_c, int H, int L_q, int L_kv, int head_dim, float scale,
                    void *stream);

/*
 * Self + target attention in one launch (blog, "Self + Target Attention Fusion"): besides the
 * candidates' target attention above, the user sequence's own queries attend over the same K
 * and V (no mask, like the target queries):
 *
 *     O_self[u,h] = softmax(scale * Q_self[u,h] . K[u,h]^T) . V[u,h]        for u < B_u
 *
 * Q_self, O_self [B_u, H, L_self, head_dim] bf16 (16-byte aligned); L_self a multiple of L_q
 * (the self queries are taken L_q at a time, as further work of their user, so they share the
 * K/V blocks the user's candidates stage).  L_self = 0 is ikbo_fa_forward; B_c = 0 computes
 * only the self part (Q, map and O may then be NULL).  Otherwise as ikbo_fa_forward.
 */
int ikbo_fa_forward_fused(ikbo_fa_plan_t plan, const void *Q, const void *K, const void *V,
                          const int32_t *map, void *O, const void *Q_self, void *O_self, int B_u,
                          int B_c, int H, int L_q, int L_kv, int L_self, int head_dim, float scale,
                          void *stream);

/* Wait for `stream`, then return and clear the device status (IKBO_OK or IKBO_ERR_MAP_RANGE). */
int ikbo_fa_check(ikbo_fa_plan_t plan, void *stream);

/* Free the plan and its workspace (synchronises the device first).  NULL is a no-op. */
int ikbo_fa_plan_destroy(ikbo_fa_plan_t plan);

/*
 * ---- Cached user histories -------------------------------------------------------------
 *
 * Target attention for users whose histories are kept between requests: K and V of user u
 * are cached in 4 bits in pages of IKBO_KV4_PAGE tokens that a block table names, grow by
 * tokens and have a length of their own.  The calls below hold no plan: every buffer is
 * the caller's, so calls on different streams, devices or captured graphs are independent
 * as long as their buffers are.  All are asynchronous on `stream` and may be captured.
 * Arguments that the host can see are checked before anything is enqueued; conditions in
 * device data set bits of the caller's status word (one uint32 that the caller zeroes
 * once; may not be NULL), which ikbo_kv_status reads.  Strides count elements.  The device
 * that owns the buffers must be current.
 */
#define IKBO_KV4_PAGE 64
#define IKBO_KV_MAX_USERS 4096

/* Wait for `stream`, then return and clear the condition recorded in *status (device memory):
 * IKBO_OK, IKBO_ERR_MAP_RANGE, IKBO_ERR_PAGE_RANGE, IKBO_ERR_NO_PAGES or IKBO_ERR_NONFINITE
 * (the first of these that was set).  Calls on other streams that share the word must be over: what they
 * record meanwhile may be cleared with it. */
int ikbo_kv_status(uint32_t *status, void *stream);

/*
 * Page tables of one step, from the requests' lengths.  Request i holds lens[i] cached tokens
 * and brings counts[i] >= 0 new ones (counts[i] = -1: it leaves, and its pages return).  With
 * have = ceil(lens[i] / page_size), its tokens take the pages
 *     block_table[i][have .. ceil((lens[i] + counts[i]) / page_size))
 * off the head of the ring of free pages, in request order; the pages of leaving requests join
 * the ring's tail in request order and are not handed out by the same call.  state[0] is the
 * ring's head, state[1] the number of free pages behind it (state[2], state[3] belong to the
 * library and start as 0).  Token t of request i gets row  starts[i] + t  of
 *     slots = block_table[i][pos / page_size] * page_size + pos % page_size,
 *     positions = pos = lens[i] + t,  rows = i;
 * the rows from starts[B_u] to capacity are filled with -1.  lens_out[i] = lens[i] + counts[i]
 * (0 for a leaving request); lens_out may be lens or counts, and state_out may be state (updated in
 * place: one step after the other, also on replays of a captured graph).  No other buffers overlap.
 * A step that does not fit (free pages, table columns or capacity: IKBO_ERR_NO_PAGES; a
 * negative or overlong length, a count below -1, a ring state out of range, more free and
 * returned pages than num_pages: IKBO_ERR_PAGE_RANGE) is refused as a whole: slots, positions and rows become -1, starts 0,
 * lens_out = lens, state_out = state, and the table and the ring keep their contents.  A page
 * number outside [0, num_pages) that the table or the ring holds is recorded as PAGE_RANGE and
 * gives slot -1.
 * 1 <= B_u <= IKBO_KV_MAX_USERS, num_pages * page_size < 2^31.
 */
typedef struct ikbo_kv_tables_args {
    const int32_t *counts;      /* [B_u] */
    const int32_t *lens;        /* [B_u] */
    int32_t *lens_out;          /* [B_u] */
    int32_t *block_table;       /* [B_u][table_stride], max_pages columns used */
    int32_t *ring;              /* [num_pages] */
    int32_t *state;             /* [4]: head, free pages, two words of the library's */
    int32_t *state_out;         /* [4]; may be state */
    int32_t *slots, *positions, *rows;   /* [capacity] */
    int32_t *starts;            /* [B_u + 1] */
    uint32_t *status;
    int64_t table_stride;
    int32_t B_u, max_pages, num_pages, page_size, capacity;
} ikbo_kv_tables_args;
int ikbo_kv_tables(const ikbo_kv_tables_args *args, void *stream);

/*
 * Rotary positions of queries and keys.  Pair i < rot_dim/2 of each head at position p turns by
 * the angle p * freq[i]:
 *     (a, b) -> factor * (a cos - b sin,  a sin + b cos)
 * with (a, b) = elements (i, i + rot_dim/2) (IKBO_ROPE_HALF) or (2i, 2i + 1)
 * (IKBO_ROPE_INTERLEAVED); elements from rot_dim on are copied.  inverse = 1 turns by the
 * opposite angle with the same factor: the gradient of the forward rotation.  The angle is
 * formed in 64 bits and reduced to one turn before sine and cosine, so positions may be any
 * int32; the rotation is in float32 and rounds once to the tensors' type (IKBO_DTYPE_*).
 * q, q_out [T][H_q][head_dim] and k, k_out [T][H_k][head_dim] with token and head strides and
 * contiguous heads; an output may be its input (same strides), and may not overlap it
 * otherwise.  H_k = 0 leaves k out.  rot_dim even, 2 <= rot_dim <= head_dim <= 1024.
 */
enum { IKBO_ROPE_HALF = 0, IKBO_ROPE_INTERLEAVED = 1 };
typedef struct ikbo_rope_args {
    const void *q, *k;
    void *q_out, *k_out;
    const int32_t *positions;   /* [T] */
    const double *freq;         /* [rot_dim / 2], radians per position */
    int64_t q_token, q_head, k_token, k_head;                   /* strides of the inputs */
    int64_t q_out_token, q_out_head, k_out_token, k_out_head;   /* strides of the outputs */
    int32_t T, H_q, H_k, head_dim, rot_dim, layout, dtype, inverse;
    float factor;
} ikbo_rope_args;
int ikbo_rope(const ikbo_rope_args *args, void *stream);

/*
 * The 4-bit cache.  tiles [num_pages][H_kv][68 * head_dim bytes], 16-byte aligned; head_dim 64
 * or 128.  The tile of a page and head holds its 64 tokens' keys and values as
 *     K codes [64 tokens][head_dim/2]      byte c: element 2c in the low 4 bits, 2c + 1 in the high
 *     V codes [head_dim/2][64 tokens]      byte (c, t): elements 2c and 2c + 1 of token t
 *     K scales [head_dim/32][64]           token t at 16 (t / 16) + 4 (t % 4) + (t / 4) % 4
 *     V scales [head_dim/32][64]           token t at t
 * (the orders in which the attention's matrix operands read them).  A code is a sign and one of
 * 0, .5, 1, 1.5, 2, 3, 4, 6; 32 consecutive elements x of a token share the scale 2^e, stored as
 * e + 127, with e the smallest in [-125, 125] for which max|x| <= 6 * 2^e; x / 2^e is rounded to
 * the nearest code, ties to the even one, and never beyond +-6.  All values are exact in bf16.
 *
 * ikbo_kv4_write puts k, v [T][H_kv][head_dim] (bf16 or float32, token and head strides) at the
 * slots (page * 64 + offset) of their tokens; a slot of -1 is skipped, others outside the pages
 * are recorded as PAGE_RANGE and skipped.  Slots of one call are distinct (a slot named twice is
 * left with either token's parts).  NaN is stored as 0 and infinity as the largest value; both
 * are recorded as NONFINITE.
 * ikbo_kv4_read gathers the values at the slots into k, v [T][H_kv][head_dim] (bf16 or float32;
 * a float32 value is exact, bf16 likewise); rows of a slot of -1 are left as they were.
 */
typedef struct ikbo_kv4_rows_args {
    void *k, *v;                /* read by the write, written by the read; either may be NULL in a read */
    const int32_t *slots;       /* [T] */
    void *tiles;
    uint32_t *status;
    int64_t k_token, k_head, v_token, v_head;
    int32_t T, H_kv, head_dim, num_pages, dtype;
} ikbo_kv4_rows_args;
int ikbo_kv4_write(const ikbo_kv4_rows_args *args, void *stream);
int ikbo_kv4_read(const ikbo_kv4_rows_args *args, void *stream);

/*
 * Target attention over the cache.  Query l of head h of candidate b, with u = map[b] and the
 * key/value head h / (H_q / H_kv), sees the tokens t of user u with
 *     t < lens[u]   and, if positions are given,   t <= positions[b][l],
 *     O[b,h,l] = sum_t softmax_t(scale * Q[b,h,l] . K[u,t]) V[u,t],
 * and is 0 where it sees none.  Q, O bf16 with candidate, head and query strides and contiguous
 * heads (16-byte aligned rows); map NULL means candidate b belongs to user b (B_c <= B_u).
 * Candidates with map -1 are padding: their O is left as it was; other entries outside [0, B_u)
 * are recorded as MAP_RANGE and left likewise.  Lengths outside [0, 64 * max_pages] are recorded
 * as PAGE_RANGE and clamped, as are page numbers outside [0, num_pages) (page 0 is read then).
 * Scores, softmax and sums are float32 (the weights reach the matrix cores as bf16); O is rounded
 * once.  O may be Q (same strides) and does not overlap it otherwise.  The same call gives the same bits; a row's
 * last bits may depend on the other rows and lengths of the call.  scale = 0 means 1/sqrt(head_dim); negative, NaN and infinite scales are INVALID_ARG.
 * head_dim 64 or 128, H_q a multiple of H_kv, 1 <= B_u <= IKBO_KV_MAX_USERS, L_q >= 1.
 * workspace: ikbo_kv4_attention_workspace bytes, 16-byte aligned, not shared with a call that may
 * overlap; nothing in it has to be kept between calls.
 */
typedef struct ikbo_kv4_attention_args {
    const void *Q;
    void *O;
    const void *tiles;
    const int32_t *block_table; /* [B_u][table_stride], max_pages columns used */
    const int32_t *lens;        /* [B_u] */
    const int32_t *map;         /* [B_c] or NULL */
    const int32_t *positions;   /* [B_c][L_q] or NULL */
    uint32_t *status;
    void *workspace;
    int64_t workspace_bytes;
    int64_t q_cand, q_head, q_query, o_cand, o_head, o_query, table_stride;
    int32_t B_u, B_c, H_q, H_kv, L_q, head_dim, max_pages, num_pages;
    float scale;
} ikbo_kv4_attention_args;
/* Bytes of workspace for these dimensions, or a negative status. */
int64_t ikbo_kv4_attention_workspace(int B_u, int B_c, int H_q, int H_kv, int L_q, int head_dim, int max_pages);
int ikbo_kv4_attention(const ikbo_kv4_attention_args *args, void *stream);

/*
 * ---- Training target attention ----------------------------------------------------------
 *
 * Target attention over dense K and V that keeps the statistics its gradient needs, and the gradient; and dropout from a
 * counter-based generator.  As for the cached histories there is no plan: every buffer is the caller's, calls are
 * asynchronous on `stream`, may be captured, and record conditions in device data in the caller's status word
 * (ikbo_kv_status).  Strides count elements.  The device that owns the buffers must be current.
 *
 * Query l of head h of candidate b, with u = map[b] and the shared head h / (H_q / H_kv), sees the tokens t of user u with
 *     t < lens[u] (L_kv if lens is NULL)   and, if positions are given,   t <= positions[b][l]:
 *
 *     S = scale Q K^T,   lse = ln sum_t exp S,   P = exp(S - lse),   O = (P Z) V
 *
 * with Z the dropout's factors (1 without dropout), and the gradients, for an upstream gradient dO,
 *
 *     dV = (P Z)^T dO,   dP = (dO V^T) Z,   dS = P (dP - rowsum(dO O)),   dQ = scale dS K,   dK = scale dS^T Q
 *
 * dK and dV summed over the user's candidates and queries and the heads that share the head.  A query that sees nothing has
 * O = 0 and lse = -inf, its gradient is 0 and its dO is not read; so are those of candidates whose map entry is -1 (padding) or, recorded
 * as MAP_RANGE, outside [0, B_u).  Tokens from lens[u] on are not read and have dK = dV = 0; lengths outside [0, L_kv] are
 * clamped and recorded as PAGE_RANGE.  A token that some of its user's queries see and others do not has to be finite.
 *
 * Dropout keeps each weight with probability 1 - r / 256, r = round(256 dropout), and divides it by that; r has to be
 * between 1 and 255, or dropout 0.  rng[0] is the seed, the low 32 bits of rng[1] the offset: with the generator Philox4x32
 * of 7 rounds (Salmon, Moraes, Dror, Shaw, 2011), key = the seed's low and high word, the 16 bytes of the counter
 * (2 (t / 32) + (t / 4) % 2, b L_q + l, h, offset) are those of 16 tokens, byte t % 4 of word (t % 32) / 8 that of token t; a
 * weight stays if its byte is at least r.  The backward takes the forward's dropout and rng.
 *
 * Layouts: Q, O, dO, dQ [B_c][H_q][L_q][head_dim], K, V, dK, dV [B_u][H_kv][L_kv][head_dim], bf16 with three strides
 * (multiples of 8, not negative; those of inputs may be 0) and contiguous heads, 16-byte aligned; lse [B_c][H_q][L_q] float32,
 * dense.  Outputs overlap nothing.  Scores, statistics and sums are float32; P and dS reach the matrix cores as bf16; outputs are rounded
 * once.  The same call gives the same bits.  scale = 0 means 1/sqrt(head_dim); negative, NaN and infinite scales are
 * INVALID_ARG.  head_dim 64 or 128, H_q a multiple of H_kv, 1 <= B_u <= IKBO_KV_MAX_USERS; tokens of K and of V at most
 * 2^24 elements apart, 4 L_kv and 4 B_c L_q H_q below 2^31, and no more blocks than a launch holds, else UNSUPPORTED.
 * workspace: ikbo_attention_workspace bytes, 16-byte aligned, not shared with a call that may overlap; nothing in it has
 * to be kept between calls.
 * Without candidates the forward does nothing; the backward writes dK = dV = 0, and needs K and V but no tensor of the candidates.
 */
typedef struct ikbo_attention_args {
    const void *Q, *K, *V;
    void *O;                    /* written by the forward, read by the backward, as lse is */
    float *lse;
    const void *dO;             /* from here to dV: the backward only */
    void *dQ, *dK, *dV;
    const int32_t *map;         /* [B_c] */
    const int32_t *lens;        /* [B_u] or NULL */
    const int32_t *positions;   /* [B_c][L_q] or NULL */
    const int64_t *rng;         /* [2] seed, offset; may be NULL without dropout */
    uint32_t *status;
    void *workspace;
    int64_t workspace_bytes;
    int64_t q_cand, q_head, q_query, k_user, k_head, k_token, v_user, v_head, v_token, o_cand, o_head, o_query;
    int64_t do_cand, do_head, do_query, dq_cand, dq_head, dq_query, dk_user, dk_head, dk_token, dv_user, dv_head, dv_token;
    double dropout;
    int32_t B_u, B_c, H_q, H_kv, L_q, L_kv, head_dim;
    float scale;
} ikbo_attention_args;
/* Bytes of workspace for these dimensions (of the backward if it is not 0), or a negative status. */
int64_t ikbo_attention_workspace(int B_u, int B_c, int H_q, int H_kv, int L_q, int L_kv, int head_dim, int backward);
int ikbo_attention_forward(const ikbo_attention_args *args, void *stream);
int ikbo_attention_backward(const ikbo_attention_args *args, void *stream);

/*
 * Dropout of n elements: y = residual + x / (1 - r / 65536) where an element stays, and residual (0 if NULL) where it does
 * not, with r = round(65536 p) between 1 and 65535, or p = 0.  Element i has the 16 bits i % 8, in order, of the counter
 * (i / 8 low, i / 8 high, 2^32 - 1, offset) of the generator above, and stays if they are at least r.  The gradient of x is
 * the same call on the gradient of y, without residual.  An element that does not stay is not multiplied: NaN and infinity go with it.
 * bf16 or float32 (IKBO_DTYPE_*), dense; y may be x or residual, and overlaps neither otherwise.
 */
typedef struct ikbo_dropout_args {
    const void *x, *residual;
    void *y;
    const int64_t *rng;         /* [2] seed, offset */
    int64_t n;
    double p;
    int32_t dtype;
} ikbo_dropout_args;
int ikbo_dropout(const ikbo_dropout_args *args, void *stream);

/* Static text for a status code. */
const char *ikbo_status_str(int status);

/* Text of the last IKBO_ERR_HIP failure seen by the calling host thread ("" if none). */
const char *ikbo_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* IKBO_H */
