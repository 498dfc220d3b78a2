/*
 * lora.h -- C ABI of liblora.so, the MI355X (gfx950) multi-LoRA adapter
 * execution unit.
 *
 * For a batch of T tokens, each tagged with an adapter slot or with
 * LORA_BASE_ONLY, one lora_apply call computes, per token t,
 *
 *     y[t] = x[t] W^T                                   (base_only)
 *     y[t] = x[t] W^T + (alpha_i / r_i) (x[t] A_i^T) B_i^T   (slot i)
 *
 * over an HBM-resident pool of adapters zero-padded to a common rank.
 *
 * Sources (page title and section):
 *  [P1] xpshop.cn article 492 (multi-tenant LoRA on one private base), sections
 *       二 and 三: one resident base shared by tenants, per-tenant memory quota
 *       as a hard boundary (over-quota mounts are refused, nothing is
 *       evicted), the tenant is mapped to an adapter handle once at request
 *       entry, hot-plug after weight validation, draining unload, refusal on a
 *       base-version mismatch, routing default base_only.
 *  [P3] "Multi-LoRA 在线服务隔离", sections on the request identity (default
 *       deny: a missing mapping is an explicit error, never a fallback; mixed
 *       adapters may share one batch with per-request index mapping) and on
 *       memory accounting (reserve memory before loading; never unload
 *       weights a request still holds).
 *  [P4] "LLM 多 LoRA 推理服务工程 2026": four-layer runtime, the adapter
 *       execution unit paragraph (base linear plus LoRA A/B, fused in one
 *       launch or separate with a residual add); routing layer, the
 *       two-level bucketing paragraph (bucket by adapter; a bucket above a
 *       threshold runs fused, otherwise separate) and the zero-pad paragraph
 *       (A maps hidden to rank, B maps rank to hidden; lower ranks are
 *       zero-padded to the common rank; report the zero-pad share); SRE list
 *       item 11 (the fused/separate threshold is tuned per GPU model).
 *
 * Conventions for every call:
 *  - Every function returns an int status: LORA_OK (0) or a negative LORA_E*
 *    code; lora_strerror() gives its text.  No call aborts the process.
 *  - Matrices are row-major and contiguous, in the nn.Linear [out][in]
 *    convention: W_base is [d_out][d_in], A is [rank][d_in], B is
 *    [d_out][rank].  x is [T][d_in] and y is [T][d_out].
 *  - One element type per pool (lora_dtype) for x, W_base, A, B and y.
 *  - "device" pointers are HIP device memory on the pool's device, 16-byte
 *    aligned.  The caller owns x, W_base, the index array and y, and keeps them
 *    alive until the stream work that uses them completes.
 *  - `stream` is a hipStream_t passed as void*; NULL is the legacy default
 *    stream.
 *  - Control-plane calls (create/destroy/quota/register/unregister/policy/
 *    stats/poll) and lora_apply/lora_route are serialized by a per-pool mutex.
 *    lora_apply and lora_route share the pool's workspace: calls on
 *    different streams must be ordered by the caller (one stream per pool is
 *    the simple contract).
 */
#ifndef LORA_H
#define LORA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- types -- */

typedef struct lora_pool_s *lora_pool; /* opaque; owned by the library */
typedef struct lora_plan_s *lora_plan; /* opaque routing plan; owned by the library */
typedef struct lora_loader_s *lora_loader; /* opaque host-to-slot loader; owned by the library */
typedef struct lora_residency_s *lora_residency; /* opaque slot residency manager */
typedef struct lora_kv_s *lora_kv;     /* opaque quantised key/value cache of one layer */
typedef struct lora_rope_s *lora_rope; /* opaque table of the angles that positions turn keys and queries by */
typedef struct lora_attend_plan_s *lora_attend_plan; /* opaque attention plan of one step's batch */
typedef struct lora_verifier_s *lora_verifier; /* opaque workspace of lora_verify and lora_verify_tree */
typedef struct lora_scorer_s *lora_scorer; /* opaque workspace of lora_logprobs */

typedef enum { LORA_F32 = 0, LORA_F16 = 1, LORA_BF16 = 2 } lora_dtype;

/* Fused/separate policy.  AUTO: a bucket (the tokens of one adapter in one
 * call) with more than `threshold` tokens runs FUSED, otherwise SEPARATE
 * [P4 two-level bucketing].  FUSED / SEPARATE force every bucket. */
typedef enum { LORA_MODE_AUTO = 0, LORA_MODE_FUSED = 1, LORA_MODE_SEPARATE = 2 } lora_mode;

/* Mode recorded per bucket by routing. */
#define LORA_SEG_NONE 0     /* base_only or invalid bucket: no LoRA term */
#define LORA_SEG_FUSED 1    /* LoRA expand added in the base GEMM's epilogue */
#define LORA_SEG_SEPARATE 2 /* base stored first, LoRA added by a residual kernel */

/* token_adapter_idx value for a token that uses the base model only [P1 三]. */
#define LORA_BASE_ONLY (-1)

/* Limits of this build. */
#define LORA_MAX_SLOTS 1024  /* n_slots per pool */
#define LORA_MAX_RANK 64     /* max_rank per pool */

#define LORA_KV_MAX_HEADS 256          /* key/value heads of a cache */
#define LORA_KV_MAX_PAGE 1024          /* tokens of a page (a power of two, at least 16) */
#define LORA_ROPE_MAX_POSITIONS (1 << 24) /* positions of a table of angles */
#define LORA_ROPE_MAX_AXES 4           /* positions of one token */
#define LORA_ATTEND_MAX_TOKENS 65536   /* sequences, groups and new tokens of a plan */
#define LORA_ATTEND_MAX_PAGES (1 << 26) /* pages a plan's sequences and prefixes hold together */
#define LORA_VERIFY_MAX_SEQS 65535     /* sequences of a verifier */
#define LORA_VERIFY_MAX_VOCAB (1 << 21)
#define LORA_SCORE_MAX_ROWS (1 << 20)  /* rows of a scorer */
#define LORA_SCORE_MAX_TOP 32          /* alternatives of a row */
#define LORA_VERIFY_MAX_DRAFTS 63      /* drafted tokens of one sequence */

/* Status codes. */
#define LORA_OK 0
#define LORA_EINVAL (-1)      /* null pointer, bad size, slot out of range, misalignment */
#define LORA_ETOKENS (-2)     /* n_tokens > the pool's max_tokens */
#define LORA_ESLOT_BUSY (-3)  /* register into a slot that is not FREE */
#define LORA_ESLOT_EMPTY (-4) /* unregister a slot that holds no adapter */
#define LORA_ERANK (-5)       /* rank < 1 or rank > the pool's max_rank */
#define LORA_EALPHA (-6)      /* alpha not finite */
#define LORA_EQUOTA (-7)      /* tenant's used + slot bytes > its quota [P1 三; P3 accounting] */
#define LORA_EMISMATCH (-8)   /* shape or dtype does not match the pool's base [P1 三] */
#define LORA_ENOMEM (-9)      /* device or host allocation failed */
#define LORA_EHIP (-10)       /* a HIP runtime call failed; lora_strerror has no detail,
                                 lora_last_hip_error() has the HIP text */
#define LORA_ESCRATCH (-11)   /* lora_apply_noalloc: the call's workspace exceeds
                                 LORA_NOALLOC_SCRATCH_BYTES */

/* Size of the library's static per-device workspace (lora_apply_noalloc). */
#define LORA_NOALLOC_SCRATCH_BYTES (32u << 20)

/* Pool statistics.  The `last_*` fields describe the most recent lora_apply
 * on the pool and are read back from the device (lora_pool_stats
 * synchronizes).  The three concatenation figures of [P4 zero-pad paragraph]
 * are: LoRA rows at the padded rank (last_lora_rows_padded), the launch extent
 * (last_tokens x d_out), and the zero-pad share (last_zero_pad_fraction). */
typedef struct {
    int32_t d_in, d_out, max_rank, n_slots, max_tokens, dtype;
    int32_t active_slots;            /* slots holding a registered adapter */
    int32_t draining_slots;          /* slots being unregistered */
    uint64_t slot_bytes;             /* bytes one slot occupies (and is charged) */
    uint64_t resident_bytes;         /* bytes charged to tenants, all slots */
    uint64_t device_bytes;           /* device memory the pool holds in total */
    int32_t last_tokens;
    int32_t last_adapters;           /* distinct adapters (LoRA buckets) */
    int32_t last_fused_buckets;
    int32_t last_separate_buckets;
    int32_t last_base_only_tokens;
    int32_t last_invalid_tokens;
    int64_t last_lora_rows_padded;   /* sum over LoRA tokens of max_rank */
    int64_t last_lora_rows_true;     /* sum over LoRA tokens of the adapter's rank */
    double last_zero_pad_fraction;   /* 1 - true / padded (0 if no LoRA token) */
} lora_stats;

/* ------------------------------------------------------------ lifecycle -- */

/* Create a pool for one linear layer on the current HIP device: n_slots
 * adapter slots of rank up to max_rank, zero-padded to max_rank [P4 zero-pad],
 * and a workspace for up to max_tokens tokens per call.  Allocates all device
 * memory now; lora_apply never allocates.
 *   d_in, d_out   the base linear's input and output widths.  For LORA_F16 /
 *                 LORA_BF16 both must be multiples of 64; LORA_F32 takes any.
 *   max_rank      1..LORA_MAX_RANK;  n_slots 1..LORA_MAX_SLOTS;
 *   max_tokens    >= 1.
 * The kernels address x, W_base and y through 32-bit byte offsets: each of
 * max_tokens*d_in, d_out*d_in and max_tokens*d_out elements must fit in
 * 4 GiB - 1 bytes, else LORA_EINVAL.
 * Errors: LORA_EINVAL (bad sizes, out == NULL), LORA_ENOMEM, LORA_EHIP. */
int lora_pool_create(int d_in, int d_out, int max_rank, int n_slots, int max_tokens,
                     lora_dtype dtype, lora_pool *out);

/* Wait for every lora_apply / lora_route enqueued on the pool, then free all
 * of its device memory and the handle.  p == NULL is a no-op. */
int lora_pool_destroy(lora_pool p);

/* ------------------------------------------------------- control plane -- */

/* Set a tenant's hard byte quota on this pool [P1 三: vram_quota].  A tenant
 * whose quota was never set has quota 0: every register is refused (default
 * deny, [P3 request identity]).  Lowering a quota below the tenant's current
 * use evicts nothing; later registers are refused.  tenant >= 0. */
int lora_set_tenant_quota(lora_pool p, int32_t tenant, uint64_t bytes);

/* Register an adapter into a FREE slot [P1 三: validate, then attach].
 *   A       device, [rank][d_in], pool dtype
 *   B       device, [d_out][rank], pool dtype
 *   rank    the adapter's true rank, 1..max_rank; rows/columns rank..max_rank-1
 *           of the slot are zero-filled [P4 zero-pad]
 *   alpha   finite; the slot's scale is alpha / rank (the true rank)
 *   stream  the copies are ordered after earlier work on `stream` (so A and B
 *           may have been written there) and complete before the call returns;
 *           A and B may be freed afterwards.
 * The slot turns ACTIVE on the device after every lora_apply / lora_route /
 * lora_plan_route enqueued on the pool before this call (on any stream) and
 * before every one enqueued after it: each call sees the slot either FREE in
 * all of its kernels (its tokens are invalid) or ACTIVE in all of them, never
 * a mix.  The call does not wait for those earlier applies.
 * The slot's bytes (lora_stats.slot_bytes) are reserved against the tenant's
 * quota before anything is copied [P3 accounting]; over quota the call fails
 * with LORA_EQUOTA and nothing else changes [P1 三: never evict another].
 * Errors: LORA_EINVAL (slot out of range, NULL A/B, tenant < 0), LORA_ESLOT_BUSY,
 * LORA_ERANK, LORA_EALPHA, LORA_EQUOTA, LORA_EHIP. */
int lora_register(lora_pool p, int slot, int32_t tenant, const void *A, const void *B,
                  int rank, float alpha, void *stream);

/* Unregister by draining [P1 二/三; P3 accounting: never unload weights a
 * request still holds]: mark the slot DRAINING, wait until every lora_apply
 * enqueued on the pool before this call has completed, then free the slot
 * and return its bytes to its tenant.  Blocks the calling thread; applies
 * from other threads wait on the pool mutex meanwhile.  A token that names
 * the slot in a later call is invalid (see lora_apply).
 * Errors: LORA_EINVAL, LORA_ESLOT_EMPTY, LORA_EHIP. */
int lora_unregister(lora_pool p, int slot);

/* Fused/separate policy [P4 two-level bucketing; SRE item 11].  threshold >= 0
 * is the bucket size above which AUTO runs FUSED.  Default: AUTO with the
 * per-device threshold this build ships for gfx950 (lora_get_policy). */
int lora_set_policy(lora_pool p, lora_mode mode, int threshold);
int lora_get_policy(lora_pool p, lora_mode *mode, int *threshold);

/* For tests of the in-launch shrink.  Calls of 65 .. 2047 tokens whose GEMM
 * tiles leave CUs idle compute h on those CUs inside the GEMM launch; the h
 * consumers of that launch poll a count of finished h units at most `polls`
 * times and, if it is still short, compute every unit themselves (the same
 * code, so the same bits).  polls = 0: they never wait and always compute h
 * themselves; polls = -1: the library's bound (about 0.1-0.3 s).  The
 * outputs do not depend on it.  LORA_EINVAL for a null pool or polls < -1. */
int lora_set_shrink_wait_polls(lora_pool p, int polls);

/* ------------------------------------------------------------ hot path -- */

/* y = x W_base^T + per-token LoRA term, asynchronously on `stream`
 * [P4 execution unit].  Routing, shrink, base GEMM and expand all run on the
 * device; the call neither allocates nor synchronizes.
 *   x                  device, [n_tokens][d_in]
 *   W_base             device, [d_out][d_in]; never retained by the pool
 *   token_adapter_idx  device int32 [n_tokens]: a slot, or LORA_BASE_ONLY
 *   y                  device, [n_tokens][d_out]; must not alias x
 * A token whose index is neither LORA_BASE_ONLY nor a registered slot (at the
 * time the call's routing kernel runs) is invalid: its y row is filled with
 * quiet NaN and the pool's device error counter grows by one; it never falls
 * back to the base or to another adapter [P3 request identity].
 * n_tokens == 0 is a no-op.
 * Errors (host-side, nothing enqueued): LORA_EINVAL, LORA_ETOKENS, LORA_EHIP. */
int lora_apply(lora_pool p, const void *x, const void *W_base,
               const int32_t *token_adapter_idx, int n_tokens, void *y, void *stream);

/* lora_apply for callers that cannot allocate device memory at call time
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same kernels and the same result, bit for bit, but the
 * call's workspace (routing arrays, h parts, split-K partial sums) lives in
 * the library's static per-device array of LORA_NOALLOC_SCRATCH_BYTES,
 * resolved when the first pool was created on the device; the call allocates
 * nothing and creates no HIP object.  Arguments, ordering and errors as
 * lora_apply, plus LORA_ESCRATCH (nothing enqueued) when the call needs more
 * workspace than the array holds: about 4 * splits * T * d_out bytes of
 * split-K partial sums plus the routing arrays and h -- every 7B-shaped
 * projection fits at up to 64 tokens, 4096-wide ones at up to 192, calls of
 * 2048 tokens and more (no split) at any width.  The array is shared by every pool and stream of the
 * device: two lora_apply_noalloc calls that may overlap in time race, so the
 * caller orders them (one stream, or events).  Nothing in it needs to start
 * at zero (every word a kernel reads was written earlier in the same call).
 * The pool's own workspace, the routing lora_last_routing reads and the
 * statistics are unaffected, except the last-call statistics and the error
 * counter, which the call updates as lora_apply does. */
int lora_apply_noalloc(lora_pool p, const void *x, const void *W_base,
                       const int32_t *token_adapter_idx, int n_tokens, void *y, void *stream);

/* Routing alone, asynchronously on `stream` [P4 two-level bucketing]: the
 * per-token histogram and stable segment sort, computed by the same device
 * code lora_apply routes with for this call size (fp16/bf16 calls of at most
 * 64 tokens route inside the decode path's epilogue; this call then runs
 * that routing in a one-wave kernel, others the routing kernel).
 * All outputs are device int32 arrays:
 *   counts[n_slots+2]     tokens per key; key = slot, n_slots = base_only,
 *                         n_slots+1 = invalid
 *   offsets[n_slots+3]    exclusive prefix sum of counts
 *   perm[n_tokens]        perm[p] = token at sorted position p, keys
 *                         ascending, ties in ascending token order
 *   segs[(n_slots+2)*4]   {key, start, len, mode} per non-empty key, keys
 *                         ascending; mode is a LORA_SEG_* value
 *   n_seg[1]              number of records
 * Does not touch the error counter.  Errors: LORA_EINVAL, LORA_ETOKENS, LORA_EHIP. */
int lora_route(lora_pool p, const int32_t *token_adapter_idx, int n_tokens,
               int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *segs,
               int32_t *n_seg, void *stream);

/* The routing the pool's kernels last used [P4 two-level bucketing; "Multi-
 * LoRA 在线服务隔离", request identity: per-request index mapping kept intact
 * in a mixed batch]: copies, asynchronously on `stream` (after the call that
 * built it, also when that ran on another stream), the stable permutation and
 * the bucket records of the last lora_apply on the pool -- or of the last
 * lora_apply_routed of at most 64 fp16/bf16 tokens, which routes in its
 * epilogue; a routed call of more tokens uses its plan's routing and leaves
 * these arrays alone.
 *   *n_tokens  host: tokens of that call (0 if no call has routed yet)
 *   perm       device int32 [*n_tokens] (may be NULL when *n_tokens is 0)
 *   segs       device int32 [(n_slots+2)*4], the first *n_seg records valid
 *   n_seg      device int32 [1]
 * Errors: LORA_EINVAL (NULL pointers), LORA_EHIP. */
int lora_last_routing(lora_pool p, int *n_tokens, int32_t *perm, int32_t *segs, int32_t *n_seg,
                      void *stream);

/* ------------------------------------------------- route once per step -- */

/* A routing plan: the tenant-to-adapter mapping of one batch resolved once,
 * at entry, and reused by every linear of the step instead of being looked
 * up again on the hot path ["xpshop.cn article 492", 二/三: the handle is
 * resolved at request entry; "LLM 多 LoRA 推理服务工程 2026", routing layer:
 * bucketing per batch].  The plan holds a device copy of the token indices
 * and the routing arrays (the same ones lora_apply builds), sized for
 * max_tokens and n_slots.  Allocates once, here.
 * Errors: LORA_EINVAL (sizes out of range, out == NULL), LORA_ENOMEM, LORA_EHIP. */
int lora_plan_create(int max_tokens, int n_slots, lora_plan *out);

/* Waits for the plan's enqueued routing, then frees it.  The caller must not
 * destroy a plan that applies still to run on another stream read. */
int lora_plan_destroy(lora_plan plan);

/* Route a batch into the plan, asynchronously on `stream`, with pool p's slot
 * table and fused/separate policy (p->n_slots must equal the plan's).  Copies
 * token_adapter_idx (device int32 [n_tokens]) into the plan, then runs the
 * routing kernel.  Invalid tokens are counted once, here, on p's error
 * counter.  The plan records p's active slots with their ranks, policy and
 * threshold at this call; lora_apply_routed checks them.
 * Errors: LORA_EINVAL, LORA_ETOKENS (n_tokens > the plan's max_tokens),
 * LORA_EMISMATCH (slot count differs), LORA_EHIP. */
int lora_plan_route(lora_plan plan, lora_pool p, const int32_t *token_adapter_idx, int n_tokens,
                    void *stream);

/* lora_apply for the plan's batch (n_tokens = the plan's), without the
 * routing pass: the plan's routing and token indices are used.  Must follow
 * the lora_plan_route on the same stream (or an event that orders them).
 * The result equals lora_apply's with the same indices bit for bit.  Pool p
 * must match the routing pool in slot count, active slots and their ranks,
 * policy and threshold (as of the route call), else LORA_EMISMATCH and
 * nothing is enqueued: its adapters' values (A, B, alpha) may differ -- one
 * plan serves the pools of every linear of a model.  Leaves p's last-call statistics and
 * error counter unchanged.
 * Errors (host-side, nothing enqueued): LORA_EINVAL (no routed batch,
 * pointers), LORA_ETOKENS, LORA_EMISMATCH, LORA_EHIP. */
int lora_apply_routed(lora_pool p, lora_plan plan, const void *x, const void *W_base, void *y,
                      void *stream);

/* ------------------------------------------------------- async loading -- */

/* The adapter loader ["LLM 多 LoRA 推理服务工程 2026", four-layer runtime,
 * loader paragraph]: moves an adapter from host memory into a pool slot
 * without blocking the hot path -- two pinned host staging buffers and two
 * device staging buffers (double buffering: one copy in flight while the
 * next adapter is staged), a copy stream of its own, and the register-time
 * pad kernel on that stream.  One loader serves any pools of its device.
 * capacity_bytes bounds one adapter's A and B together
 * (rank * (d_in + d_out) * element size).  Allocates once, here.
 * Errors: LORA_EINVAL (capacity 0, out == NULL), LORA_ENOMEM, LORA_EHIP. */
int lora_loader_create(uint64_t capacity_bytes, lora_loader *out);

/* Waits for and commits every pending load, then frees the loader. */
int lora_loader_destroy(lora_loader l);

/* Start loading an adapter into `slot` of pool p from host memory:
 *   A_host  [rank][d_in], B_host [d_out][rank], the pool's dtype, any host
 *           memory (copied into pinned staging before this call returns; the
 *           caller may reuse it at once)
 * The slot is reserved against the tenant's quota at once (the same checks
 * and errors as lora_register, nothing changes on error) and stays LOADING
 * -- tokens naming it are invalid -- until the load is committed by
 * lora_load_poll / lora_load_wait (or by a later load reusing its staging
 * buffer), which makes it ACTIVE -- ordered on the device, as for
 * lora_register, after every call already enqueued on the pool and before
 * every later one, without waiting for them on the host.  When both staging buffers are in flight
 * the call first waits for the older one.  *ticket identifies the load.
 * The caller must wait for its loads before destroying the pool.
 * Errors: LORA_EINVAL (NULL pointers, slot out of range, adapter larger than
 * the loader's capacity), LORA_ESLOT_BUSY, LORA_ERANK, LORA_EALPHA,
 * LORA_EQUOTA, LORA_EHIP. */
int lora_load_async(lora_loader l, lora_pool p, int slot, int32_t tenant, const void *A_host,
                    const void *B_host, int rank, float alpha, uint64_t *ticket);

/* Non-blocking: *done = 1 (and the slot committed, ACTIVE) once the load's
 * copies finished, else 0.  Errors: LORA_EINVAL (unknown ticket), LORA_EHIP. */
int lora_load_poll(lora_loader l, uint64_t ticket, int *done);

/* Blocking: wait for the load's copies, then commit it.  A ticket that was
 * committed already returns LORA_OK.  Errors: LORA_EINVAL, LORA_EHIP. */
int lora_load_wait(lora_loader l, uint64_t ticket);

/* ----------------------------------------------------------- residency -- */

/* Which adapters stay resident when a pool's slots run out
 * ["LLM 多 LoRA 推理服务工程 2026", four-layer runtime, storage-pool
 * paragraph: LRU-K between the HBM tier and the tiers below; "Multi-LoRA 在线
 * 服务隔离", memory-accounting section: evict only versions with no live
 * reference, least recently used first, never weights a request holds, per-
 * tenant resident shares].  The manager takes the slots of pool p that are
 * FREE now (slots registered outside it are never touched) and loads through
 * loader l.  k: accesses of history (LRU-K; 2 is the usual choice).
 * Errors: LORA_EINVAL, LORA_ENOMEM. */
int lora_residency_create(lora_pool p, lora_loader l, int k, lora_residency *out);

/* Frees the manager; resident adapters stay registered in the pool. */
int lora_residency_destroy(lora_residency r);

/* Cap on the slots tenant's adapters may hold at once (unset: no cap).
 * Errors: LORA_EINVAL (tenant < 0, max_slots < 0). */
int lora_residency_set_share(lora_residency r, int32_t tenant, int max_slots);

/* One more holder of adapter `adapter_id` (the caller's identity of a
 * version, e.g. a digest) of `tenant`.  Resident: *slot is its slot,
 * *ticket its load's ticket (0 if committed long ago; lora_load_wait on it
 * returns at once when done).  Not resident: a slot is chosen (a free one
 * within the tenant's share, else the LRU-K victim among unreferenced slots,
 * only the tenant's own when it is at its share), the victim is unloaded
 * (lora_unregister: drains the applies that may read it) and the adapter is
 * loaded there with lora_load_async from A_host / B_host (as there); wait on
 * *ticket before routing tokens to *slot.
 * Errors: LORA_ESLOT_BUSY (every candidate slot is referenced, or the
 * tenant's share is 0; nothing changes), LORA_EINVAL (NULL pointers, id
 * resident for another tenant), and lora_load_async's errors (then the
 * chosen slot is left empty). */
int lora_residency_acquire(lora_residency r, uint64_t adapter_id, int32_t tenant, const void *A_host,
                           const void *B_host, int rank, float alpha, int *slot, uint64_t *ticket);

/* One holder fewer.  Errors: LORA_EINVAL (not resident, or no holder). */
int lora_residency_release(lora_residency r, uint64_t adapter_id);

/* Counters since creation. */
typedef struct {
    uint64_t hits, misses, evictions;
    int32_t resident;  /* slots holding an adapter of the manager */
    int32_t managed;   /* slots the manager may use */
} lora_residency_stats;

int lora_residency_stats_read(lora_residency r, lora_residency_stats *out);

/* ------------------------------------------- the step around the linears -- */

/* What a serving step runs between the query/key/value projections and the
 * output projection, and after the head: the quantised cache, attention over
 * it, and the verification of drafted tokens.  Tokens of one tenant share an
 * adapter, so their keys and values of a common prefix are the same and are
 * held and computed once ["LLM 多 LoRA 推理服务工程 2026", KV reuse section].
 * All calls are asynchronous on `stream` unless they say otherwise, neither
 * allocate nor wait, and may be captured into a HIP graph. */

/* A paged cache of one layer's keys and values in 8 bits, on the current HIP
 * device.  Token slot s is token s % page_size of page s / page_size.  A row
 * (one token of one head, head_dim values x) is held as e4m3 elements and one
 * power of two:
 *     s = the least whole number >= -64 with max|x| <= 448 * 2^s
 *     e = x * 2^-s rounded to e4m3 (nearest, ties to even), stands for e * 2^s
 * A row whose key or value holds a value that is not finite is poisoned: its
 * key and value read back as NaN throughout, and the outputs of every query
 * row that sees it are NaN; no other row's are.  Rows never written are 0.
 *   n_pages >= 1, page_size a power of two of 16 .. LORA_KV_MAX_PAGE,
 *   n_pages * page_size < 2^31; n_kv_heads 1 .. LORA_KV_MAX_HEADS;
 *   head_dim 64 or 128; dtype LORA_F16 or LORA_BF16: of the keys and values
 *   written and read, and of lora_attend's queries and outputs.
 * Bytes: n_pages * page_size * n_kv_heads * 2 * (head_dim + 1).
 * Errors: LORA_EINVAL, LORA_ENOMEM, LORA_EHIP. */
int lora_kv_create(int n_pages, int page_size, int n_kv_heads, int head_dim, lora_dtype dtype, lora_kv *out);

/* Waits for the device, then frees the cache.  kv == NULL is a no-op. */
int lora_kv_destroy(lora_kv kv);

/* Quantise keys and values of n_tokens tokens into their slots.
 *   k, v      device, [n_tokens][n_kv_heads][head_dim], tokens k_stride /
 *             v_stride elements apart (multiples of 8, at least n_kv_heads *
 *             head_dim): parts of a fused projection's output need no copy
 *   slots     device int32 [n_tokens]: the token's slot, or -1: not written.
 *             Any other value outside the cache is not written and counted
 *             (lora_kv_poll_errors).  No slot twice in one call.
 * Errors (nothing enqueued): LORA_EINVAL, LORA_EHIP. */
int lora_kv_write(lora_kv kv, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                  const int32_t *slots, int n_tokens, void *stream);

/* Read slots back: k, v device [n_tokens][n_kv_heads][head_dim], contiguous,
 * the values held, rounded once to the cache's dtype.  A slot outside the
 * cache (-1 among them) reads as NaN and is counted.  Slots may repeat.
 * Errors (nothing enqueued): LORA_EINVAL, LORA_EHIP. */
int lora_kv_read(lora_kv kv, const int32_t *slots, int n_tokens, void *k, void *v, void *stream);

/* A table of angles on the current HIP device: what lora_kv_append turns keys
 * and queries by.  Position p of axis axis[i] turns pair i of a head's elements
 * by the angle p * freq[i]:
 *     (x, y) -> scale * (x cos a - y sin a, x sin a + y cos a)
 *   n_positions  1 .. LORA_ROPE_MAX_POSITIONS: 0 .. n_positions - 1
 *   rot_dim      elements of a head that turn, its first ones: 16 .. 128, a
 *                multiple of 16; the others are left as they are
 *   freq         host [rot_dim / 2], finite, the angles at n_positions - 1 too
 *   axis         host [rot_dim / 2], each 0 .. n_axes - 1; NULL: all 0
 *   n_axes       positions of a token, 1 .. LORA_ROPE_MAX_AXES (a picture's
 *                tokens have a time, a height and a width)
 *   pairs        nonzero: pair i is elements 2 i and 2 i + 1; 0: elements i and
 *                i + rot_dim / 2
 *   scale        above 0, at most 1024
 * Angles are products in fp64, their cosines and sines held to 48 bits.  Bytes:
 * 8 n_positions rot_dim.
 * Allocates once, here, and waits for the device.
 * Errors: LORA_EINVAL, LORA_ENOMEM, LORA_EHIP. */
int lora_rope_create(int n_positions, int rot_dim, const double *freq, const int32_t *axis, int n_axes, int pairs,
                     double scale, lora_rope *out);

/* Waits for the device, then frees the table.  rope == NULL is a no-op. */
int lora_rope_destroy(lora_rope rope);

/* lora_kv_write of keys turned by their positions, and the same tokens'
 * queries turned beside them.
 *   rope       of the cache's device, rot_dim at most head_dim: else
 *              LORA_EMISMATCH
 *   k .. n_tokens  as for lora_kv_write.  A key row is quantised as it would be
 *              from the turned key itself: no 16-bit form comes in between
 *   positions  device int32 [n_axes][n_tokens]
 *   q          device, [n_tokens][n_heads][head_dim], tokens q_stride elements
 *              apart (a multiple of 8, at least n_heads * head_dim), or NULL
 *              (then q_stride, n_heads and the next two are not looked at)
 *   n_heads    1 .. LORA_KV_MAX_HEADS * 32
 *   q_out      the turned queries, rounded once, tokens q_out_stride apart (as
 *              q_stride); q itself with q's stride, or memory of its own
 * A token with a position outside the table: its key and value are poisoned
 * (see lora_kv_create) where it has a slot, its queries are NaN.  It is counted
 * with the invalid slots, unless its slot is -1 (padding, whose queries are
 * turned too).
 * Errors (nothing enqueued): LORA_EINVAL, LORA_EMISMATCH, LORA_EHIP. */
int lora_kv_append(lora_kv kv, lora_rope rope, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                   const int32_t *slots, const int32_t *positions, int n_tokens, const void *q, int64_t q_stride,
                   int n_heads, void *q_out, int64_t q_out_stride, void *stream);

/* Read and clear the count of slots that writes and reads found outside the
 * cache, and of tokens that appends found at positions outside the table.
 * Waits for the device.  Errors: LORA_EINVAL, LORA_EHIP. */
int lora_kv_poll_errors(lora_kv kv, uint64_t *n_invalid_slots);

/* One step's batch, host memory (read before lora_attend_plan_set returns).
 * Sequence s has q_len[s] new tokens, the next q_len[s] rows of q and out,
 * and kv_len[s] tokens of its own in the cache, the new ones among them; page
 * list entries page0[s] .. page0[s + 1] - 1 hold them in order.  It belongs
 * to group[s], whose prefix_len tokens come before its own, or to none (-1).
 * New token j sees the whole prefix and its sequence's own tokens up to
 * itself: the first kv_len[s] - q_len[s] + j + 1.  A token that sees nothing
 * has output 0 and lse -inf. */
typedef struct {
    int32_t n_seqs, n_groups;
    const int32_t *q_len, *kv_len, *group;  /* [n_seqs] */
    const int32_t *pages, *page0;           /* page0 [n_seqs + 1] */
    const int32_t *prefix_len;              /* [n_groups] */
    const int32_t *prefix_pages, *prefix_page0; /* prefix_page0 [n_groups + 1] */
} lora_attend_batch;

/* A plan: how one batch's attention is cut into work for the device, made
 * once a step and used by every layer's lora_attend (the routing plan's
 * counterpart).  It holds the batch's lists and the workspace of partial
 * results, for the largest batch whatever is split of it: about (2 max_tokens
 * n_heads + 40000) (head_dim + 2) 4 bytes on the device (2.2 GB for 65536
 * tokens of 32 heads of 128), and twice the lists in pinned host memory.
 * Allocates once, here.
 *   n_heads a multiple of n_kv_heads, at most 32 times it.
 * Errors: LORA_EINVAL (sizes out of range), LORA_ENOMEM, LORA_EHIP. */
int lora_attend_plan_create(int max_seqs, int max_groups, int max_tokens, int max_pages, int n_heads,
                            int n_kv_heads, int head_dim, lora_attend_plan *out);

/* Waits for the device, then frees the plan.  plan == NULL is a no-op. */
int lora_attend_plan_destroy(lora_attend_plan plan);

/* Plan a batch on caches of kv's geometry: the host cuts it, and the plan goes
 * to the device on `stream` (not while that is being captured: LORA_EINVAL).
 * Waits only while the plan before the last is still on its way there.
 * Every list is checked first: lengths below 0, groups and page ids out of
 * range, fewer pages than a length needs are LORA_EINVAL, more new tokens
 * than max_tokens LORA_ETOKENS, a cache of other heads or head_dim
 * LORA_EMISMATCH; the plan is then empty until the next one, and so is the
 * device's, except after a refusal during a capture, when nothing can be sent.
 * Plan and attention share the plan's memory: calls on one plan on different
 * streams are ordered by the caller.  A captured lora_attend reads the plan as
 * it is when the graph runs, so a graph may be replayed after a new plan, of
 * any number of tokens up to max_tokens: the captured q, out and lse need room
 * for the most that it will meet, and rows past the plan's tokens are not
 * written.  The launch is as large as the plan at capture asks for (one of no
 * tokens: fills the device), so capture with the most work, or with none.  A
 * replay on a cache of another page size or count than the plan's writes NaN
 * for the plan's tokens, and one after a refused plan for those of the last
 * plan that was not refused. */
int lora_attend_plan_set(lora_attend_plan plan, lora_kv kv, const lora_attend_batch *batch, void *stream);

/* As lora_attend_plan_set, for new tokens that form a tree of drafts instead of
 * a chain (or several trees): of its sequence's new tokens, one sees itself and
 * those above it, and no others.  The prefix and the sequence's tokens before
 * the new ones are seen as before, and a new token's key lies where its place
 * in the batch says, whatever its depth.
 *   parent   host int32 [new tokens], in the batch's order: the new token of the
 *            same sequence (0 .. its own place - 1) that it follows, or -1: it
 *            follows the sequence's tokens before the new ones
 * A captured lora_attend may be replayed after plans of either kind.
 * Errors: lora_attend_plan_set's; LORA_EINVAL (parent NULL where there are new
 * tokens, or a value of it out of range); the plan is then empty as there. */
int lora_attend_plan_set_tree(lora_attend_plan plan, lora_kv kv, const lora_attend_batch *batch,
                              const int32_t *parent, void *stream);

/* out = softmax(scale * q k^T) v for the planned batch, the values as the cache
 * holds them, each group's prefix read once for all of its query rows.
 *   kv     a cache of the planned geometry (pages, page size, heads,
 *          head_dim), else LORA_EMISMATCH
 *   q      device, [tokens][n_heads][head_dim], tokens q_stride elements
 *          apart (a multiple of 8); query head h reads key/value head
 *          h / (n_heads / n_kv_heads)
 *   out    device, [tokens][n_heads][head_dim], contiguous; not q
 *   lse    device float [tokens][n_heads], log(sum(exp(scale * q k^T))), or NULL
 * Scores, maxima, sums and outputs are held in fp32; the weights, times the
 * power of two of their value row, are rounded to fp16 for the product with
 * the values: 11 bits down to 2^-21 of the largest, absolute below that, and
 * nothing below 2^-32.  The output is rounded once.
 * A plan of no tokens: nothing is enqueued, and q, out and lse are not looked
 * at, unless the stream is being captured.
 * Errors (nothing enqueued): LORA_EINVAL (no plan set, pointers, strides, scale
 * not finite), LORA_EMISMATCH, LORA_EHIP. */
int lora_attend(lora_kv kv, lora_attend_plan plan, const void *q, int64_t q_stride, float scale, void *out,
                float *lse, void *stream);

/* The workspace of lora_verify and lora_verify_tree, for up to max_seqs sequences a call.
 * Errors: LORA_EINVAL, LORA_ENOMEM, LORA_EHIP. */
int lora_verifier_create(int max_seqs, lora_verifier *out);

/* Waits for the device, then frees it.  v == NULL is a no-op. */
int lora_verifier_destroy(lora_verifier v);

/* Keep or replace drafted tokens.  Sequence s has rows row0[s] .. row0[s + 1] -
 * 1 of p_target, one for each of its n drafted tokens and one for the token
 * after them (n = 0: that one alone); draft and p_draft hold the drafted
 * tokens alone, sequence s's from row0[s] - s.
 *   p_target   device [n_rows][vocab], p_draft device [n_rows - n_seqs][vocab],
 *              probabilities in dtype (any lora_dtype)
 *   draft      device int32 [n_rows - n_seqs]
 *   row0       device int32 [n_seqs + 1], strictly ascending from 0 to n_rows
 *   u          device float [n_rows], of [0, 1)
 * Drafted token i is kept while u[i] * p_draft[i][d] < p_target[i][d], exactly.
 * One token is drawn after the k kept ones, with u[k]: from max(0, p_target -
 * p_draft) of row k if a draft was refused there, from p_target's row n if
 * none was (and where nothing of the difference is above 0): the first index
 * at which the running sum, in fp64, passes u[k] times the whole.
 *   accepted   device int32 [n_seqs]: k
 *   tokens     device int32 [n_rows]: at row0[s], the k kept tokens, the drawn
 *              one, then -1
 * accepted is -1, and the sequence's tokens are -1, where a drafted token lies
 * outside the vocabulary or the row to draw from has no weight (no entry above
 * 0, or a sum that is not finite); also, with no token written, where the
 * sequence's two entries of row0 do not ascend, leave no row for each sequence
 * before and after it, or hold over LORA_VERIFY_MAX_DRAFTS drafts.
 * Errors (nothing enqueued): LORA_EINVAL, LORA_ETOKENS (n_seqs), LORA_EHIP.
 * Calls on one verifier on different streams are ordered by the caller. */
int lora_verify(lora_verifier v, const void *p_target, const void *p_draft, lora_dtype dtype, int vocab,
                const int32_t *draft, const int32_t *row0, const float *u, int n_seqs, int n_rows,
                int32_t *tokens, int32_t *accepted, void *stream);

/* Walk down drafted trees along the target's own draws.  Sequence s has rows
 * row0[s] .. row0[s + 1] - 1, at least one: its new tokens as
 * lora_attend_plan_set_tree has them, the last token already known first (node
 * 0), the drafted ones after it, and after each the target's probabilities of
 * the next.  From node 0 on, a token is drawn from the node's row with the
 * node's u: the first index at which the running sum, in fp64, passes u times
 * the whole.  The first child of the node that holds it is kept and the walk
 * goes on there; where none does, the walk ends.  So every token is distributed
 * as the target's, however the tree was drafted.  Either all rows are read at
 * once or those of the walk one after the other, by the sizes alone and for
 * walks of about six rows: longer ones of large batches take up to three times
 * what all rows at once would.
 *   p_target   device [n_rows][vocab], probabilities in dtype (any lora_dtype);
 *              what is not above 0 counts as nothing
 *   draft      device int32 [n_rows]: the tokens of the nodes (of node 0: not
 *              looked at)
 *   parent     device int32 [n_rows]: as lora_attend_plan_set_tree's.  A node
 *              that is no later one's child (-1, itself, one after it) is
 *              never come to
 *   row0       device int32 [n_seqs + 1], strictly ascending from 0 to n_rows
 *   u          device float [n_rows], of [0, 1)
 *   accepted   device int32 [n_seqs]: how many drafted tokens were kept, k.  It
 *              and the next two share no memory with the inputs or each other
 *   tokens     device int32 [n_rows]: at row0[s] the k kept tokens, then the
 *              last one drawn, then -1
 *   path       device int32 [n_rows]: at row0[s] the k + 1 nodes that these
 *              were drawn at (0 first): the places of the new tokens whose keys
 *              and values stay; then -1
 * accepted is -1, and the sequence's tokens and path are, where a row on the
 * way has no weight (no entry above 0, or a sum that is not finite); also, with
 * nothing else written, where the sequence's two entries of row0 do not ascend
 * or leave no row for each sequence before and after it.  (Sequences that share
 * rows, where a list does not ascend elsewhere, have no answer in particular.)
 * Errors (nothing enqueued): LORA_EINVAL, LORA_ETOKENS (n_seqs), LORA_EHIP.
 * Calls on one verifier on different streams are ordered by the caller. */
int lora_verify_tree(lora_verifier v, const void *p_target, lora_dtype dtype, int vocab, const int32_t *draft,
                     const int32_t *parent, const int32_t *row0, const float *u, int n_seqs, int n_rows,
                     int32_t *tokens, int32_t *path, int32_t *accepted, void *stream);

/* The workspace of lora_logprobs, for up to max_rows rows a call (1 ..
 * LORA_SCORE_MAX_ROWS).  Errors: LORA_EINVAL, LORA_ENOMEM, LORA_EHIP. */
int lora_scorer_create(int max_rows, lora_scorer *out);

/* Waits for the device, then frees it.  s == NULL is a no-op. */
int lora_scorer_destroy(lora_scorer s);

/* Log probabilities under softmax(scale * logits), row by row.  Each logit is
 * read once, and a few neighbourhoods once more where alternatives are asked
 * for; a row of many equal logits is then looked through several times.
 *   logits    device, rows of `vocab` in dtype (any lora_dtype), `stride`
 *             elements apart (at least vocab); vocab 1 .. LORA_VERIFY_MAX_VOCAB
 *   tokens    device int32 [n_rows]: the token to score, or one outside the
 *             vocabulary (-1, say): its log probability is NaN; NULL: every
 *             row's is
 *   scale     2^-64 .. 2^64: one over the temperature
 *   top       alternatives a row, 0 .. LORA_SCORE_MAX_TOP, at most vocab
 *   logprob   device float [n_rows], of the given tokens, or NULL
 *   entropy   device float [n_rows], -sum(p log p), or NULL
 *   top_ids, top_logprobs  device int32, float [n_rows][top]: the largest
 *             logits, the lower index first among equals (+0 and -0 are); not
 *             looked at where top is 0
 * Logits of -inf have probability 0.  A row that holds NaN or +inf, or nothing
 * above -inf, is no distribution: its results are NaN, its top_ids -1.
 * Sums are held in fp32 against each lane's largest logit and joined in a fixed
 * order; no log probability comes out above 0 and no entropy below.  Errors (nothing enqueued): LORA_EINVAL, LORA_ETOKENS (n_rows),
 * LORA_EHIP.
 * Calls on one scorer on different streams are ordered by the caller. */
int lora_logprobs(lora_scorer s, const void *logits, int64_t stride, lora_dtype dtype, int vocab,
                  const int32_t *tokens, float scale, int top, int n_rows, float *logprob, float *entropy,
                  int32_t *top_ids, float *top_logprobs, void *stream);

/* ---------------------------------------------------------- observation -- */

/* Fill *out (synchronizes with every apply enqueued on the pool). */
int lora_pool_stats(lora_pool p, lora_stats *out);

/* Bytes currently charged to `tenant` on this pool ["Multi-LoRA 在线服务隔离",
 * memory-accounting section: resident bytes are accounted per adapter and
 * tenant, and the release gate bounds the accounting error]: the padded slot
 * bytes of the tenant's registered or loading slots.  Host-side; no device
 * call.  Errors: LORA_EINVAL (NULL pointers). */
int lora_tenant_bytes(lora_pool p, int32_t tenant, uint64_t *out);

/* Read and clear the device count of tokens lora_apply / lora_plan_route found
 * invalid ["Multi-LoRA 在线服务隔离", request identity: a missing mapping is an
 * explicit error, never a fallback; their y rows are NaN].  Synchronizes with
 * every call enqueued on the pool.  Errors: LORA_EINVAL, LORA_EHIP. */
int lora_poll_errors(lora_pool p, uint64_t *n_invalid_tokens);

/* Per-stage device time of lora_apply, for measurement.  When enabled, each
 * lora_apply (up to max_calls of them between two reads) records HIP timing
 * events on its own stream before routing and after the routing, shrink,
 * base-GEMM and separate-expand launches; a stage's time is the interval
 * between its two events.  The base-GEMM kernel is also launched with a pair
 * of events that its dispatch records itself (kernel_ms: the kernel's own
 * device time, no launch gaps).  Events are created by lora_profile_enable,
 * not on the hot path.  enable = 0 turns it off and frees the events. */
typedef struct {
    int64_t calls;      /* timed lora_apply calls since the last read */
    double route_ms;    /* summed over those calls */
    double shrink_ms;
    double gemm_ms;     /* base projection with the fused expand.  fp16/bf16
                           calls of at most 64 tokens route and shrink inside
                           their two launches and record no stage marks
                           between them: route_ms, shrink_ms and expand_ms are
                           0 and gemm_ms is the whole call (with the residual
                           expand when a bucket runs SEPARATE).  Longer fp16/
                           bf16 calls may route inside the shrink launch
                           (route_ms 0, shrink_ms both) or shrink inside the
                           GEMM launch (shrink_ms 0, gemm_ms both) */
    double expand_ms;   /* separate residual expand */
    double kernel_ms;   /* device time of the base-GEMM kernel itself (fp16/
                           bf16 pools; 0 for fp32) */
} lora_profile;

int lora_profile_enable(lora_pool p, int enable, int max_calls);

/* Synchronize with the timed calls, fill *out and start a new interval. */
int lora_profile_read(lora_pool p, lora_profile *out);

/* Static text for a status code. */
const char *lora_strerror(int status);

/* Text of the last HIP error seen by this thread inside the library ("" if
 * none). */
const char *lora_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LORA_H */
