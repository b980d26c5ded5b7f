/*
 * gdr.h -- C ABI of libgdr: the chunked gated delta rule forward on GB300 (sm_103a).
 *
 * The operation (per packed segment n and value head h, state S of dk x dv):
 *
 *     S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   S_{start-1} = h0[n,h] or 0
 *     o_t = scale * S_t^T q_t,                                          ht[n,h] = S_last
 *
 * evaluated chunkwise with chunks of 64 tokens, the chunk size of FlashQLA's
 * chunk_gated_delta_rule varlen path ("Findings from integrating FlashQLA's
 * Blackwell GDN kernels into a JAX trainer", section 1: prepare_chunk_indices(cu, 64);
 * "FlashQLA GDN backend produces different tokens from FLA Triton on
 * correctness-test prompts", Setup: chunk_size=64, varlen API).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every data pointer is a DEVICE pointer on the current CUDA device, except
 *   the gdr_tensor_t structs themselves and their `strides` arrays, which live
 *   in host memory and are only read during the call.  The caller owns every
 *   buffer; the library keeps no pointer after a call returns and has no
 *   cache keyed on addresses (the stale-cache failure in "Findings ...",
 *   section 1, cannot occur).
 * - Layouts (row-major by default):
 *       q, k   [T, Hk, dk]  bf16          v, o   [T, H, dv]  bf16
 *       g      [T, H]       f32 (natural-log decay, exp(g) multiplies the state)
 *       beta   [T, H]       bf16          h0, ht [N, H, dk, dv] f32 (row = key dim)
 *   H % Hk == 0 and value head h reads query/key head h / (H / Hk).
 *   dk == dv, with dk in {64, 128}.
 * - `strides == NULL` means compact row-major, as DLPack defines it ("Findings
 *   ...", section 3: stubs that rejected NULL strides).  Explicit strides are
 *   in elements; the innermost stride must be 1.  h0/ht must be compact.
 * - cu_seqlens: DEVICE int32 array of n_seq + 1 offsets into the token axis.
 *   It is never read on the host.  Offsets are clamped to [0, T] and made
 *   non-decreasing by a running maximum, so a malformed array cannot cause an
 *   out-of-bounds access.  Repeated offsets are length-0 ("ghost") segments
 *   ("Findings ...", section 2): they write no o and, when ht is requested,
 *   ht[n] = h0[n] (or zeros).  Tokens outside every segment are not written.
 * - Return value: GDR_OK (0) or a negative gdr_status code.  Nothing is
 *   thrown across the ABI.  Kernels are enqueued on `stream` and the call does
 *   not synchronise; asynchronous device errors surface on the stream.
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of gdr_tensor_t::dtype. */
enum gdr_dtype { GDR_BF16 = 1, GDR_F32 = 2, GDR_I32 = 3 };

/* Status codes. */
enum gdr_status {
  GDR_OK = 0,
  GDR_ERR_NULL = -1,      /* a required pointer or descriptor is NULL          */
  GDR_ERR_DTYPE = -2,     /* wrong element type                                 */
  GDR_ERR_SHAPE = -3,     /* wrong rank or inconsistent extents                 */
  GDR_ERR_STRIDE = -4,    /* innermost stride != 1, negative stride, non-compact state */
  GDR_ERR_DIM = -5,       /* head dimension not supported (dk == dv in {64,128}) */
  GDR_ERR_HEADS = -6,     /* H % Hk != 0                                        */
  GDR_ERR_NSEQ = -7,      /* n_seq < 0 or n_seq inconsistent with h0/ht         */
  GDR_ERR_WORKSPACE = -8, /* workspace NULL, too small or not 256-byte aligned   */
  GDR_ERR_PATH = -9,      /* unknown path, or FUSED requested but unsupported    */
  GDR_ERR_CUDA = -10,     /* a CUDA runtime call or kernel launch failed         */
  GDR_ERR_ALIGN = -11,    /* a base pointer or row stride is not 16-byte aligned */
  GDR_ERR_DEVICE = -12,   /* the current device is not sm_103 (GB300)            */
  GDR_ERR_SCRATCH_LIMIT = -13, /* problem too large for gdr_chunk_out_noalloc's static scratch */
  GDR_ERR_CKPT = -14,          /* checkpoint interval not a positive multiple of 64, or
                                  checkpoint buffer of the wrong type, shape or size  */
  GDR_ERR_OPTION = -15         /* unknown activation, norm or flag, or options that do not go
                                  together                                            */
};

/* Execution paths of the forward. */
enum gdr_path {
  GDR_PATH_AUTO = 0,   /* fused when its alignment preconditions hold, else staged */
  GDR_PATH_FUSED = 1,  /* one persistent kernel per call; intermediates stay on chip.
                          When the (segment, head) pairs are too few to fill the GPU
                          (3 x n_seq x H <= its SM count) and no checkpoints are asked
                          for, segments of 48 chunks or more are cut into 3 to 8
                          pieces that run on different SMs, joined through the affine
                          state map S_out = M S_in + R of each piece (FlashQLA's
                          sequence split, `seq_split_idx`, "Findings ...", section 2) */
  GDR_PATH_STAGED = 2, /* the three stages as separate kernels with HBM intermediates */
  GDR_PATH_FUSED_WHOLE = 3 /* the fused kernel with every (segment, head) in one piece */
};

typedef struct gdr_tensor {
  void *data;             /* device pointer to element [0,...,0]           */
  int32_t dtype;          /* enum gdr_dtype                                  */
  int32_t ndim;           /* 1..4                                            */
  int64_t shape[4];       /* extents, outermost first                        */
  const int64_t *strides; /* host array of ndim strides in elements, or NULL */
} gdr_tensor_t;

/*
 * gdr_chunk_fwd -- the whole forward: q, k, v, g, beta (+ optional h0) -> o (+ optional ht).
 *
 *   q, k    [T, Hk, dk] bf16; v [T, H, dv] bf16; g [T, H] f32; beta [T, H] bf16
 *   scale   multiplies the output (o = scale * S^T q)
 *   h0      [n_seq, H, dk, dv] f32 initial states, or NULL for zero states
 *   cu_seqlens, n_seq   see the conventions above
 *   o       [T, H, dv] bf16 output (round-to-nearest-even); covered tokens only
 *   ht      [n_seq, H, dk, dv] f32 final states, or NULL to skip them
 *           (FlashQLA drops dead h0/ht parameters in this case: "Findings ...", section 4)
 *
 * Runs GDR_PATH_AUTO.  Scratch memory is taken with cudaMallocAsync on `stream`
 * and released with cudaFreeAsync on the same stream.  Errors: any gdr_status.
 */
int gdr_chunk_fwd(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v,
                  const gdr_tensor_t *g, const gdr_tensor_t *beta, float scale,
                  const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                  gdr_tensor_t *o, gdr_tensor_t *ht, cudaStream_t stream);

/* Bytes of device scratch gdr_chunk_fwd_ws needs for these extents and path
 * (GDR_PATH_AUTO sizes for the larger of the two) on the current device: the
 * fused path's sequence split depends on its SM count, and takes up to
 * 24 x n_seq x H x dv x dv x 4 bytes for the pieces' states.  Never fails;
 * returns 0 for negative arguments. */
size_t gdr_chunk_fwd_workspace_bytes(int64_t T, int32_t n_seq, int32_t H, int32_t dk,
                                     int32_t dv, int32_t path);

/*
 * gdr_chunk_fwd_ws -- gdr_chunk_fwd with a caller-owned workspace and an explicit path.
 *   workspace   device pointer, 256-byte aligned, at least
 *               gdr_chunk_fwd_workspace_bytes(T, n_seq, H, dk, dv, path) bytes.
 *               Stream-ordered: it may be reused once the call's work on `stream` is done.
 * Errors: as gdr_chunk_fwd, plus GDR_ERR_WORKSPACE and GDR_ERR_PATH.
 */
int gdr_chunk_fwd_ws(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v,
                     const gdr_tensor_t *g, const gdr_tensor_t *beta, float scale,
                     const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                     gdr_tensor_t *o, gdr_tensor_t *ht, int32_t path, void *workspace,
                     size_t workspace_bytes, cudaStream_t stream);

/*
 * gdr_chunk_fwd_ckpt -- gdr_chunk_fwd_ws that also writes state checkpoints every
 * checkpoint_every_n_tokens tokens of each segment, for prefix caching.  The FlashInfer
 * KDA prefill keeps this surface (state_checkpoints / checkpoint_cu_starts /
 * checkpoint_every_n_tokens kwargs, "feat(cake_kda): add paired recurrent training for
 * SM100a and SM103a", the released inference surface kept by the cherry-picked commit);
 * the pages describe no layout, so the one below is this library's.
 *   checkpoint_every_n_tokens  positive multiple of 64 (the chunk size).
 *   state_checkpoints   [rows, H, dk, dv] fp32 out, compact; rows >=
 *                       gdr_ckpt_count_bound(T, checkpoint_every_n_tokens).  Checkpoint m
 *                       (m = 1 .. floor(len_n / every)) of segment n is the state S
 *                       ([dk][dv], as ht) after the segment's first m * every tokens, in row
 *                       checkpoint_cu_starts[n] + m - 1.  Other rows are not written.
 *   checkpoint_cu_starts  device int32 [n_seq + 1] out: the running sum of
 *                       floor(len_n / every) (lengths after the cu_seqlens reading); the last
 *                       entry is the number of checkpoints written.
 * Workspace as gdr_chunk_fwd_ws.  Errors: as gdr_chunk_fwd_ws, plus GDR_ERR_CKPT.
 */
int gdr_chunk_fwd_ckpt(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v,
                       const gdr_tensor_t *g, const gdr_tensor_t *beta, float scale,
                       const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                       gdr_tensor_t *o, gdr_tensor_t *ht, gdr_tensor_t *state_checkpoints,
                       int32_t *checkpoint_cu_starts, int32_t checkpoint_every_n_tokens,
                       int32_t path, void *workspace, size_t workspace_bytes,
                       cudaStream_t stream);

/* Rows gdr_chunk_fwd_ckpt may write: floor(T / checkpoint_every_n_tokens) (0 for bad
 * arguments). */
int64_t gdr_ckpt_count_bound(int64_t T, int32_t checkpoint_every_n_tokens);

/* Pieces per segment that GDR_PATH_FUSED cuts long segments into on the current
 * device for T tokens in n_seq segments of H value heads (1: no split; else 3..8).
 * The first piece may weigh 2 or 3 of the others (it runs while the others' state
 * maps are formed); a segment of c chunks gets at most floor(c / 16) - (weight - 1)
 * pieces, and stays whole when that is under 3.  Returns 1 when no device can be
 * queried. */
int32_t gdr_fused_split_pieces(int64_t T, int32_t n_seq, int32_t H);

/* The split planner behind gdr_fused_split_pieces, for any machine size: for `units`
 * (segment, value head) pairs on `sms` SMs, the pieces per long segment (1: no split;
 * else 3..8) and, in *lead (may be NULL), the first piece's weight (1..3).  The plan
 * minimises pass A + pass B of the split in units of the whole segment: pass A runs the
 * first pieces (weight `lead`) and, for every middle piece, its state map's offset R and
 * transition M (weight 1 each); pass B the P - 1 later pieces; each pass on `sms` SMs
 * taking units in that order as they come free; ties go to fewer pieces, and no split
 * unless 3 * units <= sms.  Pure host arithmetic; non-positive arguments give 1 and
 * lead 1. */
int32_t gdr_split_plan(int64_t units, int32_t sms, int32_t *lead);

/*
 * gdr_chunk_bwd -- the backward: gradients of gdr_chunk_fwd's outputs with respect to
 * all its inputs.  FlashQLA's GDN kernels serve as a training backend whose backward
 * is bit-reproducible and tolerates length-0 segments ("Findings ...", intro and
 * section 2); the pages print no backward formula, so this is the gradient of the
 * forward defined above (its chunk form is written out in gdr_bwd.cu).
 *
 *   q, k, v, g, beta, scale, h0, cu_seqlens, n_seq
 *           the forward's inputs, as gdr_chunk_fwd takes them (the forward is
 *           recomputed from them; nothing of a previous forward call is kept)
 *   dout    [T, H, dv] bf16, dL/do (read for covered tokens only)
 *   dht     [n_seq, H, dk, dv] f32 compact, dL/dht, or NULL for zero
 *   dq, dk  [T, Hk, dk] f32 compact out (grouped heads: summed over the value heads
 *           that share a query/key head, in head order)
 *   dv      [T, H, dv] f32 compact out
 *   dg, dbeta  [T, H] f32 compact out
 *   dh0     [n_seq, H, dk, dv] f32 compact out, or NULL to skip: the gradient for the
 *           initial state (h0 or the zero state); an empty segment's dh0 is its dht
 *   workspace   device, 256-byte aligned, >= gdr_chunk_bwd_workspace_bytes(...) bytes
 *
 * Tokens outside every segment get zero gradients.  Deterministic: every output
 * element is written by one thread per kernel in a fixed order (no atomics), so
 * results are bit-identical from run to run.  Stream-ordered, no host synchronisation.
 * Errors: as gdr_chunk_fwd_ws (dout is checked like o, dht like ht), GDR_ERR_STRIDE
 * for non-compact outputs, GDR_ERR_WORKSPACE.
 */
int gdr_chunk_bwd(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v,
                  const gdr_tensor_t *g, const gdr_tensor_t *beta, float scale,
                  const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                  const gdr_tensor_t *dout, const gdr_tensor_t *dht, gdr_tensor_t *dq,
                  gdr_tensor_t *dk, gdr_tensor_t *dv, gdr_tensor_t *dg, gdr_tensor_t *dbeta,
                  gdr_tensor_t *dh0, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream);

/* Bytes of device scratch gdr_chunk_bwd needs (0 for bad arguments). */
size_t gdr_chunk_bwd_workspace_bytes(int64_t T, int32_t n_seq, int32_t Hk, int32_t H,
                                     int32_t dk, int32_t dv);

/* Upper bound on the number of 64-token chunks: ceil(T / 64) + n_seq. */
int64_t gdr_chunk_count_bound(int64_t T, int32_t n_seq);

/* Bytes of device scratch each stage entry point below needs (chunk tables). */
size_t gdr_stage_workspace_bytes(int64_t T, int32_t n_seq);

/*
 * Chunk enumeration from cu_seqlens, on the device.
 *   seg_table   [n_seq, 4] int32 out: (start, end, first chunk id, chunk count) per segment
 *   chunk_table [gdr_chunk_count_bound(T, n_seq), 4] int32 out: (segment, first token,
 *               length 1..64, 0) per chunk id; ids are assigned segment by segment.
 *   n_chunks    device int32 out: the number of chunks.
 * Errors: GDR_ERR_NULL, GDR_ERR_NSEQ, GDR_ERR_SHAPE (T < 0), GDR_ERR_CUDA.
 */
int gdr_chunk_index(const int32_t *cu_seqlens, int32_t n_seq, int64_t T, int32_t *seg_table,
                    int32_t *chunk_table, int32_t *n_chunks, cudaStream_t stream);

/*
 * Stage 1, gdr_chunk_prep: per (chunk, value head) with chunk-local index i, j:
 *   G_i  = sum_{t<=i} g_t (chunk-local inclusive cumsum)
 *   A_ij = beta_i exp(G_i - G_j) k_i.k_j (j < i), Tm = (I + A)^-1
 *   W = Tm diag(beta exp(G)) K,  U = Tm diag(beta) V
 * Outputs (compact, covered tokens only): w [T, H, dk] bf16, u [T, H, dv] bf16,
 * gcum [T, H] f32.  workspace: gdr_stage_workspace_bytes(T, n_seq) bytes.
 */
int gdr_chunk_prep(const gdr_tensor_t *k, const gdr_tensor_t *v, const gdr_tensor_t *g,
                   const gdr_tensor_t *beta, const int32_t *cu_seqlens, int32_t n_seq,
                   gdr_tensor_t *w, gdr_tensor_t *u, gdr_tensor_t *gcum, void *workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/*
 * Stage 2, gdr_state_scan: per (segment, value head), sequential over chunks, fp32 state:
 *   h[c] = S (bf16);  V' = U - W S;  S <- exp(G_last) S + (diag(exp(G_last - G)) K)^T V'
 * Inputs: k [T, Hk, dk] bf16, w/u/gcum from stage 1, h0 (or NULL).
 * Outputs: h [gdr_chunk_count_bound, H, dk, dv] bf16 indexed by chunk id,
 * v_new [T, H, dv] bf16 (V'), ht (or NULL).  workspace as for stage 1.
 */
int gdr_state_scan(const gdr_tensor_t *k, const gdr_tensor_t *w, const gdr_tensor_t *u,
                   const gdr_tensor_t *gcum, const gdr_tensor_t *h0,
                   const int32_t *cu_seqlens, int32_t n_seq, gdr_tensor_t *h,
                   gdr_tensor_t *v_new, gdr_tensor_t *ht, void *workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/*
 * Stage 3, gdr_chunk_out: per (chunk, value head):
 *   O = scale [ diag(exp(G)) Q h[c] + (M o Q K^T) V' ],  M_ij = exp(G_i - G_j) for j <= i, else 0
 * Inputs: q, k [T, Hk, dk] bf16, v_new [T, H, dv] bf16, h and gcum as above.
 * Output: o [T, H, dv] bf16, covered tokens only.  workspace as for stage 1.
 */
int gdr_chunk_out(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v_new,
                  const gdr_tensor_t *h, const gdr_tensor_t *gcum, float scale,
                  const int32_t *cu_seqlens, int32_t n_seq, gdr_tensor_t *o, void *workspace,
                  size_t workspace_bytes, cudaStream_t stream);

/*
 * Debug check of cu_seqlens (synchronises `stream`): *n_bad receives the number of
 * offsets that are negative, above T, or below their predecessor, and *first_bad the
 * index of the first such offset (-1 if none).  Errors: GDR_ERR_NULL, GDR_ERR_NSEQ, GDR_ERR_CUDA.
 */
int gdr_debug_check_cu_seqlens(const int32_t *cu_seqlens, int32_t n_seq, int64_t T,
                               int32_t *n_bad, int32_t *first_bad, cudaStream_t stream);

/*
 * Device status word of the fused kernel.  Every bounded wait inside the fused
 * kernel that runs out (after 2 s) sets a nonzero code here: 0x1xx producer,
 * 0x2xx MMA issuer, 0x3xx prep warps, 0x4xx state warps; the CTA then drains its
 * copies and MMAs in flight, releases its Tensor Memory and returns instead of
 * hanging.  The blocks of the gated linear recurrence, which wait for one another, set 0x601
 * (forward) or 0x602 (backward): a block whose wait ran out waits no more and goes on to its end, and
 * those that wait for it do the same, so that a cluster of blocks loses two waits' time at most.
 * gdr_device_status synchronises the current device and
 * reads the word; gdr_clear_device_status resets it.  0 means no wait ran out.
 */
int gdr_device_status(int32_t *status_out);
int gdr_clear_device_status(void);

/*
 * Self-test of the bounded waits: launches one block that waits on an mbarrier
 * nothing ever arrives on.  The wait gives up after `limit_us` microseconds
 * (1..1000000), records GDR_STATUS_WAIT_SELFTEST in the device status word (if it
 * was 0) and the kernel returns normally; the context stays usable.  Read the word
 * with gdr_device_status.  Errors: GDR_ERR_SHAPE for a limit out of range,
 * GDR_ERR_DEVICE, GDR_ERR_CUDA.
 */
#define GDR_STATUS_WAIT_SELFTEST 0x7001
int gdr_debug_wait_selftest(uint32_t limit_us, cudaStream_t stream);
/*
 * The same for the gated linear recurrence's blocks: one that misses another's results in each of `steps`
 * (1..1000000) steps gives up after `limit_us` microseconds (1000..1000000) in the first, waits in none
 * of the others, and records 0x601.
 */
int gdr_debug_rec_wait_selftest(uint32_t limit_us, int32_t steps, cudaStream_t stream);

/*
 * gdr_chunk_out_noalloc -- gdr_chunk_out for callers that cannot allocate device memory.
 *
 * The papers behind this library have no counterpart of this entry point; it exists for
 * embedders that may not call cudaMalloc or hand out a workspace: engines with a fixed,
 * pre-planned memory budget, custom-call hosts that own every buffer, or code that must
 * not touch the allocator while it runs.  It computes exactly what gdr_chunk_out computes,
 * with the same arguments minus the workspace, and calls no cudaMalloc, cudaFree or
 * allocating library routine.
 *
 * Scratch: the chunk tables (segment table, chunk table, chunk count) live in one static
 * device array of GDR_NOALLOC_SCRATCH_BYTES (4 MiB) inside libgdr; every GPU that loads
 * the library holds that array until the process exits.  A problem needs
 * 256 + 16 * max(n_seq, 1) + 16 * gdr_chunk_count_bound(T, n_seq) + 4 * max(n_seq, 1)
 * bytes, each term rounded up to 256 (the chunk count, the segment table, the chunk
 * table and the segment order); larger problems return GDR_ERR_SCRATCH_LIMIT (roughly
 * 260k chunks).
 * The tables are rewritten completely by every call, so nothing needs clearing between
 * calls.  Every call on a device shares the same array: calls whose work overlaps on the
 * GPU (different streams without ordering between them) race and may produce wrong
 * output; order them on one stream or with events.
 *
 * Set-up: the first call on each device (with that device current) looks up the array's
 * device address with cudaGetSymbolAddress and caches it; make that first call before
 * any stream capture on that device.
 *
 * Errors: as gdr_chunk_out (without GDR_ERR_WORKSPACE), plus GDR_ERR_SCRATCH_LIMIT, and
 * GDR_ERR_CUDA if the address lookup fails.
 */
#define GDR_NOALLOC_SCRATCH_BYTES (4u << 20)
int gdr_chunk_out_noalloc(const gdr_tensor_t *q, const gdr_tensor_t *k,
                          const gdr_tensor_t *v_new, const gdr_tensor_t *h,
                          const gdr_tensor_t *gcum, float scale, const int32_t *cu_seqlens,
                          int32_t n_seq, gdr_tensor_t *o, cudaStream_t stream);

/*
 * ---- The operators around the delta rule in a token mixer -------------------------------
 *
 * Short convolution, selective state space, per-head q/k norm with rotation, and the delta
 * rule for single tokens.  Shared conventions, beside those at the top:
 * - Activations are bf16 or f32, all of one call in the same type; sums, states of the state
 *   space and the delta rule, and parameter gradients are f32.
 * - Rows may have any stride >= their extent (innermost contiguous); 16-byte aligned rows take
 *   the fast path, others a slower one with the same results.  States are compact.
 * - Outputs must not overlap inputs or each other.
 * - cu_seqlens NULL with n_seq = 1 means one segment of all T tokens.
 * - Packed calls: tokens outside every segment are not written by a forward and get zero
 *   gradients from a backward; their values, infinities and NaN among them, reach no output.
 * - Single-token calls work on a pool of state slots, in place.  state_indices is a DEVICE
 *   int32 array with each row's slot, or NULL (row i uses slot i).  A slot < 0 or >= the
 *   number of slots marks a padded row: its outputs are zero, no state is touched.  A slot
 *   named by two rows of one call is written by both, in no fixed order.
 * - Deterministic: no atomics on results; parameter gradients are added in a fixed order.
 * - T, B and the channel count are at most 0x7ff00000.
 */
enum gdr_activation { GDR_ACT_NONE = 0, GDR_ACT_SILU = 1, GDR_ACT_SIGMOID = 2 };
enum gdr_norm { GDR_NORM_RMS = 0, GDR_NORM_L2 = 1 };

/*
 * gdr_conv_fwd -- causal convolution of each channel over the tokens of its segment:
 *   u_t = bias + sum_{k < W} weight[c, k] x_{t-W+1+k},   y = u or u sigmoid(u).
 *   x, y    [T, C]; weight [C, W], W = 2, 3 or 4, bias [C] or NULL: f32 or bf16 (both alike)
 *   h0      [n_seq, W - 1, C] in x's type: the inputs before each segment, oldest first, or
 *           NULL for zeros;  ht the same shape, out or NULL: the last W - 1 inputs of each
 *           segment, reaching into h0 where it is shorter (an empty segment: h0's rows)
 * Errors: GDR_ERR_DIM for another W, GDR_ERR_OPTION for an unknown activation.
 */
int gdr_conv_fwd(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
                 const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                 int32_t activation, gdr_tensor_t *y, gdr_tensor_t *ht, cudaStream_t stream);

/*
 * gdr_conv_bwd -- gradients of gdr_conv_fwd (the forward is recomputed).
 *   dy      [T, C], dL/dy;  dht [n_seq, W - 1, C], dL/dht, or NULL for zero: x's type
 *   dx      [T, C] out, dh0 [n_seq, W - 1, C] out or NULL: x's type
 *   dweight [C, W], dbias [C] or NULL: f32 compact out
 *   workspace  256-byte aligned, >= gdr_conv_bwd_workspace_bytes(T, C, W) bytes
 */
int gdr_conv_bwd(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
                 const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                 int32_t activation, const gdr_tensor_t *dy, const gdr_tensor_t *dht,
                 gdr_tensor_t *dx, gdr_tensor_t *dweight, gdr_tensor_t *dbias,
                 gdr_tensor_t *dh0, void *workspace, size_t workspace_bytes,
                 cudaStream_t stream);
size_t gdr_conv_bwd_workspace_bytes(int64_t T, int32_t C, int32_t W);

/*
 * gdr_conv_step -- one token for each of B requests: y from the slot's W - 1 inputs and x,
 * which then moves into the slot (the oldest drops out).
 *   x, y [B, C]; state [slots, W - 1, C] compact, x's type
 */
int gdr_conv_step(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
                  gdr_tensor_t *state, const int32_t *state_indices, int32_t activation,
                  gdr_tensor_t *y, cudaStream_t stream);

/*
 * gdr_ssm_fwd -- selective state space scan, for each channel d, state n and segment:
 *   dt = softplus(dt_raw + dt_bias) (dt_softplus = 0: dt_raw + dt_bias)
 *   h_t = exp(dt A[d, n]) h_{t-1} + dt x B[n],   y = sum_n C[n] h_t + D[d] x,
 *   y *= z sigmoid(z) if z is given.
 *   x, dt, z, y  [T, Dm]; B, C [T, G, N], Dm % G == 0 (channel d reads group d / (Dm / G));
 *   A [Dm, N], D [Dm], dt_bias [Dm]: f32 compact; z, D, dt_bias may be NULL
 *   h0, ht  [n_seq, Dm, N] f32 compact, or NULL (ht of an empty segment: h0's, or zeros)
 *   N = 1 .. 64
 *   workspace  256-byte aligned, >= gdr_ssm_fwd_workspace_bytes(T, Dm, N, G) bytes (may be 0)
 */
int gdr_ssm_fwd(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
                const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
                const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
                const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                gdr_tensor_t *y, gdr_tensor_t *ht, void *workspace, size_t workspace_bytes,
                cudaStream_t stream);
size_t gdr_ssm_fwd_workspace_bytes(int64_t T, int32_t Dm, int32_t N, int32_t G);

/*
 * gdr_ssm_bwd -- gradients of gdr_ssm_fwd (the forward is recomputed).
 *   dy [T, Dm]; dht [n_seq, Dm, N] f32 or NULL
 *   dx, ddt, dz [T, Dm] (dz iff z), dB, dC [T, G, N] compact: out, x's type
 *   dA [Dm, N], dD [Dm] (or NULL), ddt_bias [Dm] (or NULL), dh0 [n_seq, Dm, N] (or NULL):
 *   f32 compact out
 *   workspace  256-byte aligned, >= gdr_ssm_bwd_workspace_bytes(T, Dm, N, G) bytes.  Most of it holds
 *   parts of dB and dC: T x Dm x L^2 / 8 bytes, L = 2, 4, 8, 16 for N up to 8, 16, 32, 64 (at
 *   65,536 x 4,096 0.5 GB for N = 16, 2.1 for 32, 8.6 for 64).
 * Infinities and NaN in one segment's inputs reach no other segment's outputs and gradients; the
 * parameters' gradients sum over all segments.
 */
int gdr_ssm_bwd(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
                const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
                const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
                const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                const gdr_tensor_t *dy, const gdr_tensor_t *dht, gdr_tensor_t *dx,
                gdr_tensor_t *ddt, gdr_tensor_t *dA, gdr_tensor_t *dB, gdr_tensor_t *dC,
                gdr_tensor_t *dD, gdr_tensor_t *dz, gdr_tensor_t *ddt_bias, gdr_tensor_t *dh0,
                void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t gdr_ssm_bwd_workspace_bytes(int64_t T, int32_t Dm, int32_t N, int32_t G);

/*
 * gdr_ssm_step -- one token of gdr_ssm_fwd for each of the rows of x.
 *   x, dt, z, y [rows, Dm]; B, C [rows, G, N]; state [slots, Dm, N] f32 compact, in place
 *   (the fast path takes N % 4 == 0 with A and state 16-byte aligned)
 */
int gdr_ssm_step(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
                 const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
                 const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
                 gdr_tensor_t *state, const int32_t *state_indices, gdr_tensor_t *y,
                 cudaStream_t stream);

/*
 * gdr_qk_fwd -- norm of each row (token, head) of q and k, then the position rotation:
 *   u = x r weight,  r = (mean x^2 + eps)^-1/2 (RMS) or (sum x^2 + eps)^-1/2 (L2)
 *   pairs (a, b) of u's first `rot` elements -> (a cos - b sin, b cos + a sin): element i with
 *   i + rot / 2, or interleaved 2 i with 2 i + 1
 *   q, q_out [T, Hq, d]; k, k_out [T, Hk, d]; d = 1 .. 256;  q_weight, k_weight [d] f32 or
 *   bf16, or NULL (ones)
 *   cos, sin  [places, rot / 2] f32 compact, rot <= d even; both NULL: no rotation
 *   positions DEVICE int32 [T]: each token's row of the tables (clamped to them)
 */
int gdr_qk_fwd(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *q_weight,
               const gdr_tensor_t *k_weight, int32_t norm, float eps, const gdr_tensor_t *cos,
               const gdr_tensor_t *sin, const int32_t *positions, int32_t interleaved,
               gdr_tensor_t *q_out, gdr_tensor_t *k_out, cudaStream_t stream);

/*
 * gdr_qk_bwd -- gradients of gdr_qk_fwd: dq_out, dk_out -> dq, dk (activations' type) and
 * dq_weight, dk_weight [d] f32 (or NULL).  workspace: 256-byte aligned, >=
 * gdr_qk_bwd_workspace_bytes(T, Hq, Hk, d) bytes.
 */
int gdr_qk_bwd(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *q_weight,
               const gdr_tensor_t *k_weight, int32_t norm, float eps, const gdr_tensor_t *cos,
               const gdr_tensor_t *sin, const int32_t *positions, int32_t interleaved,
               const gdr_tensor_t *dq_out, const gdr_tensor_t *dk_out, gdr_tensor_t *dq,
               gdr_tensor_t *dk, gdr_tensor_t *dq_weight, gdr_tensor_t *dk_weight,
               void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t gdr_qk_bwd_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t d);

/*
 * gdr_delta_step -- one token of gdr_chunk_fwd's recurrence for each of B requests, states in
 * place: S = exp(g)(I - beta k k^T) S + beta k v^T, o = scale S^T q.
 *   q, k [B, Hk, dk] bf16; v, o [B, H, dv] bf16; g [B, H] f32; beta [B, H] bf16;
 *   state [slots, H, dk, dv] f32 compact, 16-byte aligned; dk = dv in {64, 128}
 */
int gdr_delta_step(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v,
                   const gdr_tensor_t *g, const gdr_tensor_t *beta, float scale,
                   gdr_tensor_t *state, const int32_t *state_indices, gdr_tensor_t *o,
                   cudaStream_t stream);

/*
 * ---- The operators of a hybrid block beside its mixer ------------------------------------
 *
 * Gated linear recurrence, the norms behind and before a block with its gate and residual scale,
 * and for attention layers between the mixers' the single-token attention over a paged key-value
 * cache, with the cache's block tables, slots and writes.  Conventions as above.
 */

/*
 * gdr_rec_fwd -- gated linear recurrence of each channel over the tokens of its segment:
 *   a_t = exp(A[d] sigmoid(r_t)),  m_t = sqrt(1 - a_t^2) (normalize = 0: 1),
 *   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t (i NULL: no such gate),  y_t = h_t.
 *   x, r, i, y  [T, D];  A [D] f32 compact, <= 0 (above it a > 1: with normalize m is NaN, and
 *     so is y; without it the recurrence is the same formula, of states that grow)
 *   h0, ht  [n_seq, D] f32 compact, or NULL (ht of an empty segment: h0's, or zeros)
 *   checkpoints  [gdr_rec_checkpoint_rows(T), D] f32 compact out, or NULL: what gdr_rec_bwd would
 *                compute again, the state before every eighth token
 * A state that is infinite or NaN is so, one or the other, for the rest of its segment in its channel,
 * however far the decays behind it reach (a product of them that underflowed times an infinity is NaN);
 * the gradients likewise, towards the segment's start.  Other segments and channels see nothing of it.
 */
int gdr_rec_fwd(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
                const gdr_tensor_t *A, int32_t normalize, const gdr_tensor_t *h0,
                const int32_t *cu_seqlens, int32_t n_seq, gdr_tensor_t *y, gdr_tensor_t *ht,
                gdr_tensor_t *checkpoints, cudaStream_t stream);
int64_t gdr_rec_checkpoint_rows(int64_t T);

/*
 * gdr_rec_bwd -- gradients of gdr_rec_fwd.
 *   checkpoints  of the forward with the same inputs, or NULL: they are computed again
 *   dy [T, D]; dht [n_seq, D] f32 or NULL;  dx, dr, di [T, D] (di iff i): out, x's type
 *   dA [D], dh0 [n_seq, D] (or NULL): f32 compact out
 *   workspace  256-byte aligned, >= gdr_rec_bwd_workspace_bytes(...) bytes
 * Where a_t is 1 (A sigmoid(r) = 0) the normaliser has no derivative; its part counts as 0.
 */
int gdr_rec_bwd(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
                const gdr_tensor_t *A, int32_t normalize, const gdr_tensor_t *h0,
                const int32_t *cu_seqlens, int32_t n_seq, const gdr_tensor_t *checkpoints,
                const gdr_tensor_t *dy, const gdr_tensor_t *dht, gdr_tensor_t *dx, gdr_tensor_t *dr,
                gdr_tensor_t *di, gdr_tensor_t *dA, gdr_tensor_t *dh0, void *workspace,
                size_t workspace_bytes, cudaStream_t stream);
size_t gdr_rec_bwd_workspace_bytes(int64_t T, int32_t D, int32_t n_seq, int32_t has_checkpoints);

/*
 * gdr_rec_step -- one token of gdr_rec_fwd for each of the rows of x.
 *   x, r, i, y [rows, D]; state [slots, D] f32 compact, in place.  Rows name different slots: of a slot
 *   that two of them name, either may have read or written first.
 */
int gdr_rec_step(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
                 const gdr_tensor_t *A, int32_t normalize, gdr_tensor_t *state,
                 const int32_t *state_indices, gdr_tensor_t *y, cudaStream_t stream);

/*
 * gdr_gated_norm_fwd -- the norm of each row (token, head) behind a mixer, times its gate:
 *   y = x (mean x^2 + eps)^-1/2 weight f(z),  f(z) = z sigmoid(z) (GDR_ACT_SILU) or sigmoid(z)
 *   (GDR_ACT_SIGMOID)
 *   x, z, y [T, H, d], d = 1 .. 1024; weight [d] f32 or bf16, or NULL (ones).  y may be x or z.
 */
int gdr_gated_norm_fwd(const gdr_tensor_t *x, const gdr_tensor_t *z, const gdr_tensor_t *weight,
                       int32_t activation, float eps, gdr_tensor_t *y, cudaStream_t stream);

/*
 * gdr_gated_norm_bwd -- gradients: dy -> dx, dz [T, H, d] (x's type), dweight [d] f32 (or NULL).
 * workspace: 256-byte aligned, >= gdr_gated_norm_bwd_workspace_bytes(T, H, d) bytes.
 */
int gdr_gated_norm_bwd(const gdr_tensor_t *x, const gdr_tensor_t *z, const gdr_tensor_t *weight,
                       int32_t activation, float eps, const gdr_tensor_t *dy, gdr_tensor_t *dx,
                       gdr_tensor_t *dz, gdr_tensor_t *dweight, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream);
size_t gdr_gated_norm_bwd_workspace_bytes(int64_t T, int32_t H, int32_t d);

/*
 * gdr_residual_norm_fwd -- between two blocks: the norm behind the first, its gate and residual
 * scale, the residual, and the norm before the second:
 *   u = x, or with post = 1  x (mean x^2 + eps)^-1/2 post_weight
 *   h = residual + scale gate u,   y = h (mean h^2 + eps)^-1/2 weight
 *   x, y [T, C], C = 1 .. 16384;  residual (NULL: zeros), h (NULL: not wanted) [T, C]: x's type, or
 *   f32 beside x in bf16;  weight, post_weight, gate [C] f32 or bf16, or NULL (ones).
 *   y is made of h before it is rounded.  h may be the residual, in place, and y may be x.
 */
int gdr_residual_norm_fwd(const gdr_tensor_t *x, const gdr_tensor_t *residual,
                          const gdr_tensor_t *weight, int32_t post, const gdr_tensor_t *post_weight,
                          const gdr_tensor_t *gate, float scale, float eps, gdr_tensor_t *y,
                          gdr_tensor_t *h, cudaStream_t stream);

/*
 * gdr_residual_norm_bwd -- gradients of gdr_residual_norm_fwd (h is computed again from x and the
 * residual).  dy, dx in x's type; dh (NULL: zeros), dresidual (or NULL) in the residual's; dweight,
 * dpost_weight, dgate [C] f32 compact, each or NULL.
 * workspace: 256-byte aligned, >= gdr_residual_norm_bwd_workspace_bytes(T, C) bytes.
 */
int gdr_residual_norm_bwd(const gdr_tensor_t *x, const gdr_tensor_t *residual,
                          const gdr_tensor_t *weight, int32_t post, const gdr_tensor_t *post_weight,
                          const gdr_tensor_t *gate, float scale, float eps, const gdr_tensor_t *dy,
                          const gdr_tensor_t *dh, gdr_tensor_t *dx, gdr_tensor_t *dresidual,
                          gdr_tensor_t *dweight, gdr_tensor_t *dpost_weight, gdr_tensor_t *dgate,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t gdr_residual_norm_bwd_workspace_bytes(int64_t T, int32_t C);

/*
 * gdr_attn_step -- attention of one new token of each of B requests over a paged cache:
 *   o[h] = sum_j p_j v_j,  p = softmax_j(scale q[h].k_j),  query head h reading key head
 *   h / (Hq / Hk), over the keys at places max(0, n - window) .. n - 1 (window = 0: 0 .. n - 1), n =
 *   lengths[b] (clamped to what the table holds).
 *   q, o [B, Hq, d], k_cache, v_cache [pages, page_size, Hk, d] (any strides, innermost contiguous);
 *   d = 1 .. 256, Hq % Hk == 0
 *   block_table  int32 [B, width], rows of any stride: place j of request b is place j % page_size of
 *                page block_table[b, j / page_size]; places on pages < 0 or >= pages are left out
 *   lengths      DEVICE int32 [B], the new token's own key among them
 * A row that sees no key gets zeros, and so does one whose scores all are -infinity; an infinite value of a
 * key that it sees makes its elements infinite (NaN where both signs meet).  What the cache holds at other places is not looked at.
 * width * page_size <= 0x7ff00000.  bf16 with 16-byte aligned cache rows and d % 8 == 0 takes the fast
 * path.  workspace: 256-byte aligned, >= gdr_attn_step_workspace_bytes(B, Hq, Hk, d) bytes.
 */
int gdr_attn_step(const gdr_tensor_t *q, const gdr_tensor_t *k_cache, const gdr_tensor_t *v_cache,
                  const gdr_tensor_t *block_table, const int32_t *lengths, float scale,
                  int32_t window, gdr_tensor_t *o, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream);
size_t gdr_attn_step_workspace_bytes(int32_t B, int32_t Hq, int32_t Hk, int32_t d);

/*
 * gdr_cache_plan -- pages, slots and positions of the new tokens of B requests, in their order.
 *   lengths [B]     tokens that each request has in the cache (below 0: 0)
 *   new_tokens [B]  tokens that it wants to add (below 0: 0)
 *   block_table     int32 [B, width], rows of any stride, in place: the pages that request b needs
 *                   more are written behind the ceil(lengths[b] / page_size) that it has
 *   free_pages      int32 [F]: page numbers; those from *taken on are handed out in order
 *   taken, taken_out   one int32 each: how many of free_pages are handed out, before and after
 *   slots, positions   int32 [max_tokens] out, of the new tokens packed request by request: page *
 *                   page_size + place (-1 on a page < 0, or above 2^31 - 1: gdr_cache_write refuses caches
 *                   of so many places) and the token's place in its request; behind
 *                   the last token -1 and 0
 *   cu_seqlens      int32 [B + 1] out: where each request's new tokens lie in them
 *   lengths_out     int32 [B] out: lengths with the new tokens
 * A request is given fewer tokens than it wants where its row of the table ends, where max_tokens
 * are reached by what the requests before it and it want (each up to its row's end), or where
 * free_pages end; cu_seqlens and lengths_out say how many it was given.  Nothing is left out in
 * slots and positions for what it was not given: token j of request b is at cu_seqlens[b] + j if that
 * is below cu_seqlens[b + 1], and otherwise nowhere.  All arrays are DEVICE arrays, compact but for the table;
 * lengths_out may be lengths, and taken_out taken; a call that reads the same values again writes the
 * same ones.  width * page_size <= 0x7ff00000.
 */
int gdr_cache_plan(const int32_t *lengths, const int32_t *new_tokens, int32_t B,
                   gdr_tensor_t *block_table, const gdr_tensor_t *free_pages, const int32_t *taken,
                   int32_t page_size, int32_t *slots, int32_t *positions, int32_t max_tokens,
                   int32_t *cu_seqlens, int32_t *lengths_out, int32_t *taken_out,
                   cudaStream_t stream);

/*
 * gdr_cache_write -- rows of k and v [T, Hk, d] into k_cache and v_cache [pages, page_size, Hk, d] at
 * slots (DEVICE int32 [T], page * page_size + place); a slot outside the cache: a row that is not
 * written.  A slot named by two rows is written by both, in no fixed order.  pages * page_size <= 2^31.
 */
int gdr_cache_write(const gdr_tensor_t *k, const gdr_tensor_t *v, gdr_tensor_t *k_cache,
                    gdr_tensor_t *v_cache, const int32_t *slots, cudaStream_t stream);

/* Human-readable text for a gdr_status code (static storage). */
const char *gdr_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int gdr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H_ */
