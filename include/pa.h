/*
 * pa.h -- C ABI of libpa: packed (block-diagonal causal) attention on GB300.
 *
 * The operation (mlx-train-perf changelog, entry adding
 * `flash_attention(segments=...)` and the PACKED forward, dQ and dK/dV
 * kernels; mlx-train-perf 0.5.1 README, "Sequence packing" and
 * "Flash-attention training path"): several sequences are packed into one
 * row; a per-token int32 segment id says which sequence each token belongs
 * to, and token i attends token j iff j <= i and seg[i] == seg[j]. No (N, N)
 * mask exists anywhere. The forward saves only the output and its
 * log-sum-exp; the backward recomputes attention tile by tile.
 *
 *   S_ij  = scale * <q_i, k_j>           over visible (i, j) only
 *   lse_i = ln sum_j exp(S_ij)
 *   o_i   = sum_j exp(S_ij - lse_i) v_j
 *   and the gradients of o with respect to q, k and v.
 *
 * Layouts (all contiguous, row-major; same README, "If you maintain a
 * trainer": q/k/v are (B, H, N, D), grouped-query heads mapped contiguously):
 *   q, out, dout, dq : (B, Hq,  N, D) bf16
 *   k, v, dk, dv     : (B, Hkv, N, D) bf16;  query head h reads kv head h / (Hq/Hkv)
 *   lse              : (B, Hq,  N)    fp32, natural log
 *   seg              : (B, N)         int32, shared by all heads. Ids are
 *                      compared for equality only: any values are valid.
 *                      Tile skipping is fastest when each id forms one
 *                      contiguous run, which is what packing produces.
 * Head dim 96 (README, "If you maintain a trainer": head_dim in {64, 96,
 * 128}) runs the 128-wide kernels; the tensors stay 96 wide, the tile loads
 * fill columns 96..127 with zeros and the stores leave them out, so a D = 96
 * call takes about as long as a D = 128 one.
 *
 * Ownership: every pointer is device memory owned by the caller. The library
 * allocates no device memory and keeps no pointer after a call returns. The
 * workspace `ws` (pa_workspace_bytes) holds, in this order and each region
 * starting on a 256-byte boundary: the device status word (uint32 at byte
 * 0); the per-tile segment-range table, (B, N/128) int4 {smallest id,
 * largest id, first key tile whose id range overlaps, last query tile whose
 * id range overlaps} at byte 256; two work lists of B*N/128 int32 entries
 * b*(N/128) + t each, the query tiles and then the key tiles ordered by
 * decreasing walk length; then the backward's per-row delta = rowsum(dO * O)
 * and lse * log2(e). For N % 128 != 0 the table and lists describe the
 * padded row (N rounded up to 128).
 *
 * Execution: every call validates its arguments synchronously and returns an
 * error before launching anything; otherwise it enqueues its kernels on
 * `stream` and returns PA_OK without synchronising. Outputs are overwritten,
 * never accumulated into. There is no fallback path: an unsupported shape or
 * device is refused with a typed status (same README, "When it refuses":
 * typed refusals, never silent fallbacks).
 *
 * Device-side waits are bounded; a pipeline that stalls for ~2 s ends its
 * kernel and sets bits in the workspace status word (pa_device_status).
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pa_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef struct {
  int32_t B;    /* rows (independent packed rows)                    */
  int32_t Hq;   /* query heads                                       */
  int32_t Hkv;  /* key/value heads; Hq % Hkv == 0                    */
  int32_t N;    /* tokens per row (single-step calls: multiple of 128) */
  int32_t D;    /* head dim: 64, 96 or 128                           */
  float scale;  /* softmax scale; <= 0 selects 1/sqrt(D)             */
} pa_dims;

typedef enum {
  PA_OK = 0,
  PA_ERR_NULL = 1,      /* a required pointer is NULL                          */
  PA_ERR_HEAD_DIM = 2,  /* D not in {64, 96, 128}                              */
  PA_ERR_GQA = 3,       /* Hq % Hkv != 0                                       */
  PA_ERR_SHAPE = 4,     /* B, H, N <= 0, sizes overflow int32, a stride < D,
                           or N % 128 != 0 in a single-step call             */
  PA_ERR_ALIGN = 5,     /* a pointer is not 16-byte aligned                    */
  PA_ERR_WORKSPACE = 6, /* ws_bytes < pa_workspace_bytes(dims)                 */
  PA_ERR_ARCH = 7,      /* current device is not compute capability 10.3       */
  PA_ERR_CUDA = 8,      /* a CUDA runtime / driver call or launch failed       */
  PA_ERR_DTYPE = 9,     /* io_dtype is not a pa_io_dtype, or a format not a
                           pa_ckpt_format                                     */
  PA_ERR_HOST_MEMORY = 10 /* a host-side call could not allocate its scratch    */
} pa_status;

/* Device status bits (pa_device_status). */
#define PA_DEVERR_TIMEOUT 0x1u /* a bounded wait expired; bits 8.. name the site */
#define PA_DEVERR_DRAIN 0x2u   /* teardown after a timeout could not drain       */
#define PA_DEVERR_SMEM 0x4u    /* a kernel's shared memory was not 1 KiB aligned;
                                  the kernel did no work                          */

/*
 * Workspace size in bytes for `dims` (0 if dims are invalid), for the calls
 * on contiguous tensors. When N is not a multiple of 128 it also includes
 * room for the staging copies described at pa_fwd_strided; the bf16 calls
 * need only the size for N rounded up to 128, which this never undercuts.
 */
size_t pa_workspace_bytes(const pa_dims* dims);

/*
 * Forward. Writes out (B,Hq,N,D) bf16 and lse (B,Hq,N) fp32.
 * seg (B,N) int32 must not be NULL (use pa_fwd_causal for plain causal).
 */
pa_status pa_fwd(const pa_dims* dims, const void* q, const void* k, const void* v, const int32_t* seg,
                 void* out, float* lse, void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * Backward. Inputs: q, k, v, the forward's out and lse, dout = dL/d(out) and
 * seg. Writes dq (B,Hq,N,D), dk and dv (B,Hkv,N,D), bf16. The gradients of all
 * query heads of a group are summed into their kv head's dk/dv.
 */
pa_status pa_bwd(const pa_dims* dims, const void* q, const void* k, const void* v, const void* out,
                 const void* dout, const float* lse, const int32_t* seg, void* dq, void* dk, void* dv,
                 void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * Plain causal variants (mlx-train-perf 0.5.1 README, "If you maintain a
 * trainer": flash_attention(q, k, v, scale=..., causal=True)). They run the
 * same kernels with every token in one segment, so their results are
 * bit-identical to pa_fwd / pa_bwd on an all-equal seg (the changelog states
 * single-segment packed output is bit-identical to the causal kernels).
 */
pa_status pa_fwd_causal(const pa_dims* dims, const void* q, const void* k, const void* v, void* out,
                        float* lse, void* ws, size_t ws_bytes, pa_stream_t stream);
pa_status pa_bwd_causal(const pa_dims* dims, const void* q, const void* k, const void* v, const void* out,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, void* ws,
                        size_t ws_bytes, pa_stream_t stream);

/*
 * Strided tensors and any N (README, "If you maintain a trainer": q/k/v are
 * (B, H, N, D); a model that holds them as (B, N, H, D) passes that memory
 * with its strides instead of transposing it).
 *
 * Same operation and results as pa_fwd / pa_bwd (seg may be NULL for plain
 * causal), for tensors whose element (b, h, n, c) sits at element offset
 * b*x_b + h*x_h + n*x_n + c: q, out, dout and dq use the q_* strides; k, v,
 * dk and dv the k_* strides. lse stays contiguous (B, Hq, N) fp32 and seg
 * (B, N) int32. Every stride must be >= D and a multiple of 16 bytes (8 bf16
 * or 4 fp32 elements); distinct (b, h, n) rows of an output must not overlap.
 *
 * io_dtype is the element type of q, k, v, out, dout, dq, dk and dv
 * (README, "If you maintain a trainer": the kernels take bf16 or fp32).
 * PA_IO_F32 tensors are rounded to bf16 (nearest even) on the way in and the
 * bf16 results widened exactly on the way out, so an fp32 call returns what
 * the bf16 call returns on the rounded inputs: fp32 is an I/O format here,
 * not a compute precision.
 *
 * How: with bf16 tensors the kernels read and write the caller's tensors in
 * place, whatever their strides and N: they work on Np = N rounded up to
 * 128 tokens through 4-D TMA tensor maps {D, N, H, B} with the given strides,
 * which read the tokens past N as zeros and never store them, and the
 * segment ids are copied into the workspace with the row's last id repeated
 * up to Np (workspace: pa_workspace_bytes for dims with N rounded up to
 * 128). With fp32 tensors the call copies its inputs into bf16 (B, H, Np, D)
 * buffers inside the workspace, runs the kernels there and copies the
 * results out (workspace: pa_workspace_bytes_strided). Either way the extra
 * tokens lie after every real query, so causality hides them; they get zero
 * dO and delta and an infinite lse, so they add nothing to dK and dV, and
 * their outputs are dropped. pa_fwd / pa_bwd and the causal variants take
 * the same in-place path when N % 128 != 0.
 * Errors: as pa_fwd / pa_bwd, plus PA_ERR_NULL (strides), PA_ERR_SHAPE (a
 * stride < D), PA_ERR_ALIGN (a stride not a 16-byte multiple), PA_ERR_DTYPE.
 */
typedef enum { PA_IO_BF16 = 0, PA_IO_F32 = 1 } pa_io_dtype;
typedef struct {
  int64_t q_b, q_h, q_n; /* element strides of q, out, dout, dq */
  int64_t k_b, k_h, k_n; /* element strides of k, v, dk, dv     */
} pa_strides;

size_t pa_workspace_bytes_strided(const pa_dims* dims);
pa_status pa_fwd_strided(const pa_dims* dims, const pa_strides* strides, int32_t io_dtype, const void* q,
                         const void* k, const void* v, const int32_t* seg, void* out, float* lse, void* ws,
                         size_t ws_bytes, pa_stream_t stream);
pa_status pa_bwd_strided(const pa_dims* dims, const pa_strides* strides, int32_t io_dtype, const void* q,
                         const void* k, const void* v, const void* out, const void* dout, const float* lse,
                         const int32_t* seg, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                         pa_stream_t stream);

/*
 * The steps of the path, one kernel each, for callers that schedule or time
 * them individually. pa_fwd is pa_build_tile_table + pa_fwd_tiles; pa_bwd is
 * pa_build_tile_table + pa_bwd_delta + pa_bwd_dq + pa_bwd_dkv, all on one
 * stream, in that order. The later steps read the tile table (and the bwd
 * steps the per-row values of pa_bwd_delta) from `ws`, so they must follow
 * the steps that write it with the same dims and the same seg (NULL seg =
 * plain causal throughout). pa_build_tile_table writes the tile table and
 * the two work lists (the forward, dQ and dK/dV calls take their tiles in
 * that order) and clears the workspace status word. pa_bwd_delta takes the forward's out and lse and stores, per
 * query row, delta = rowsum(dO * O) and lse * log2(e) (the dK/dV step reads
 * that copy; pa_bwd_dkv still validates its lse argument). These calls take
 * contiguous tensors with N % 128 == 0 only (else PA_ERR_SHAPE).
 */
pa_status pa_build_tile_table(const pa_dims* dims, const int32_t* seg, void* ws, size_t ws_bytes,
                              pa_stream_t stream);
pa_status pa_fwd_tiles(const pa_dims* dims, const void* q, const void* k, const void* v, const int32_t* seg,
                       void* out, float* lse, void* ws, size_t ws_bytes, pa_stream_t stream);
pa_status pa_bwd_delta(const pa_dims* dims, const void* out, const void* dout, const float* lse, void* ws,
                       size_t ws_bytes, pa_stream_t stream);
pa_status pa_bwd_dq(const pa_dims* dims, const void* q, const void* k, const void* v, const void* dout,
                    const float* lse, const int32_t* seg, void* dq, void* ws, size_t ws_bytes, pa_stream_t stream);
pa_status pa_bwd_dkv(const pa_dims* dims, const void* q, const void* k, const void* v, const void* dout,
                     const float* lse, const int32_t* seg, void* dk, void* dv, void* ws, size_t ws_bytes,
                     pa_stream_t stream);

/*
 * Single-pass backward (no counterpart on the pages; built to compare with
 * the split dQ / dK-dV design of pa_bwd). One kernel walks the key tiles as
 * pa_bwd_dkv does and also forms each key tile's share of dQ (dS K), which
 * it adds into an fp32 accumulator in the workspace with vector reductions;
 * a last kernel rounds the accumulator to bf16 into dq. Same arguments and
 * operation as pa_bwd; seg may be NULL (plain causal).
 *   - Results: dk and dv are bitwise those of pa_bwd / pa_bwd_causal. dq
 *     matches them within rounding but is not bitwise reproducible from run
 *     to run: the shares of one query row are added in whatever order the
 *     key tiles finish.
 *   - Workspace: pa_bwd_fused_workspace_bytes(dims) = pa_workspace_bytes(dims)
 *     plus B*Hq*N*D*4 bytes for the accumulator (0 if dims are invalid or
 *     N % 128 != 0).
 *   - Errors: as pa_bwd, and PA_ERR_SHAPE when N % 128 != 0 (no staging
 *     copies on this path).
 */
size_t pa_bwd_fused_workspace_bytes(const pa_dims* dims);
pa_status pa_bwd_fused(const pa_dims* dims, const void* q, const void* k, const void* v, const void* out,
                       const void* dout, const float* lse, const int32_t* seg, void* dq, void* dk, void* dv,
                       void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * Backward without a caller workspace, for callers that cannot allocate device
 * memory when they run it: code inside a region where its allocator or memory
 * pool forbids new allocations, or a host runtime that only hands out its own
 * tensors. The pages have no counterpart; this is a deployment convenience.
 *
 * Same arguments and results as pa_bwd (seg may be NULL for plain causal, as
 * in pa_bwd_causal), minus the workspace: the scratch lives in one static
 * device array of PA_NOALLOC_SCRATCH_BYTES (8 MiB) inside the library, held by
 * every GPU that loads the library until the process exits. The call makes no
 * allocation of any kind.
 *   - Limit: the call runs when pa_workspace_bytes(dims) <=
 *     PA_NOALLOC_SCRATCH_BYTES and is refused with PA_ERR_WORKSPACE
 *     otherwise; compare the two before calling. With N % 128 == 0 that is
 *     about 1 million query rows (B*Hq*N: 8 bytes of scratch per row). With
 *     N % 128 != 0 the workspace also holds the staging copies (about
 *     8*D*(1 + Hkv/Hq) + 12 bytes per query row), which caps it far lower:
 *     roughly 4,000 to 6,500 query rows at D = 128.
 *   - The first call on each device looks up the array's device address with
 *     that device current; make that first call before any stream capture.
 *   - Every call on a device shares the one array, which keeps the last call's
 *     contents (the call itself resets what must start at zero). Calls whose
 *     kernels overlap on the GPU -- on different streams, or from different
 *     threads -- race on it and corrupt each other's results: serialise them.
 *   - device_status: if not NULL, the call waits for its kernels and stores
 *     the device status word there (0 = healthy, else PA_DEVERR_* bits);
 *     if NULL, the call returns without synchronising.
 */
#define PA_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
pa_status pa_bwd_noalloc(const pa_dims* dims, const void* q, const void* k, const void* v, const void* out,
                         const void* dout, const float* lse, const int32_t* seg, void* dq, void* dk, void* dv,
                         uint32_t* device_status, pa_stream_t stream);

/*
 * Synchronises `stream`, then returns the workspace's device status word
 * (0 = healthy; PA_DEVERR_* bits otherwise) and clears it. Returns
 * 0xFFFFFFFF if the read itself fails.
 */
uint32_t pa_device_status(const void* ws, pa_stream_t stream);

/*
 * Self-test of the kernels' bounded waits (failure detection without a GPU
 * fault): clears the workspace status word, then launches on `stream` one
 * warp that waits, through the same wait path the kernels use, on an
 * mbarrier that nothing arrives on. After the wait limit (2 s) it gives up,
 * sets PA_DEVERR_TIMEOUT with site 99 in bits 8.. of the status word (the
 * first 4 bytes of `ws`) and exits; the context stays usable. Read the result
 * with pa_device_status.
 * Errors: PA_ERR_NULL (ws), PA_ERR_ALIGN, PA_ERR_WORKSPACE (ws_bytes < 4),
 * PA_ERR_ARCH, PA_ERR_CUDA (launch failed).
 */
pa_status pa_selftest_wait_timeout(void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * Self-test of the forward's FMA-pipe exponential (the softmax's
 * exp(s - m) taken as 2^t with t = (s - m) log2 e; mlx-train-perf 0.5.1
 * README, "Packed attention"): y[i] = 2^x[i] for n fp32 values, computed on
 * `stream` by the device routine the forward kernel can use for part of
 * its keys (Cody-Waite range reduction and a fitted cubic, no MUFU; the
 * build option PA_FWD_FMA_EX2_PAIRS sets how many, none by default).
 * x and y are device pointers to n floats each (4-byte aligned; the caller
 * owns both). Relative error about 1e-4 for results >= 2^-126; inputs <= -127
 * (and -inf) give +0.0; inputs must be below 128. A lane mismatch inside
 * the routine is reported as a NaN in y.
 * Errors: PA_ERR_SHAPE (n < 0), PA_ERR_NULL, PA_ERR_ALIGN, PA_ERR_ARCH,
 * PA_ERR_CUDA. n == 0 returns PA_OK without a device call.
 */
pa_status pa_selftest_exp2_fma(const float* x, float* y, int64_t n, pa_stream_t stream);

/*
 * Host packer (mlx-train-perf changelog, "Added": the packed batch iterator
 * fills fixed rows with (tokens, offset) sequences after a seeded per-epoch
 * shuffle, by first-fit, and emits per-token segment buffers; the packed loss
 * masks segment by segment, so the supervised tokens are those of an
 * unpacked run, per the 0.5.1 README, "Sequence packing"). Host memory only;
 * no CUDA call is made and no GPU is needed.
 *
 * Inputs (host, caller-owned, read only):
 *   lengths[count]  tokens per sequence, each >= 1. count >= 0.
 *   offsets[count]  prompt length per sequence, each >= 0 (>= length means
 *                   nothing of it is supervised); NULL = all 0.
 *   tokens          the sequences' tokens concatenated in input order
 *                   (sum(lengths) values); needed when row_tokens or
 *                   row_targets is set.
 *   rows, N         the output holds `rows` rows of N tokens (rows, N >= 1).
 *   seed, epoch     the shuffle. Draw n of (seed, epoch) is
 *                   m(k + (n + 1) * 0x9E3779B97F4A7C15), k = m(seed * 1000003
 *                   + epoch), m the splitmix64 output function, all mod 2^64;
 *                   for i = count-1 down to 1, position i swaps with position
 *                   draw(i) mod (i + 1).
 * Placement: in shuffled order, each sequence goes whole into the lowest-
 *   numbered row with room for it, behind that row's earlier sequences; one
 *   that fits no row is left out (placement -1). So the rows in use are a
 *   prefix; to pack a whole epoch, pass rows >= count and cut the result into
 *   batches of B rows.
 * Outputs (host, caller-owned, fully overwritten; all but seg may be NULL):
 *   seg[rows*N]         int32, row-major (rows, N): the sequences of a row are
 *                       segments 0, 1, ... in placement order; the unfilled
 *                       tail of a row (an unused row: all of it) is one more
 *                       segment. This is the attention calls' seg.
 *   loss_mask[rows*N]   1 where the token at that position is trained to
 *                       predict the next token of its own sequence and that
 *                       token is past the prompt: position p (0-based within
 *                       its sequence) with offset <= p + 1 <= length - 1.
 *                       0 elsewhere, padding included.
 *   row_tokens[rows*N]  the packed tokens; pad_token in the padding.
 *   row_targets[rows*N] where loss_mask is 1, the token that position is
 *                       trained to predict (the next token of its own
 *                       sequence); -1 elsewhere, which pa_lce_fwd ignores.
 *   placement[count]    int64 flat index row*N + start of each input
 *                       sequence (input order), or -1 when it was left out.
 *   rows_used           1 + the highest row holding a sequence (0 if none).
 *   placed_tokens       tokens placed in all rows.
 * Errors: PA_ERR_NULL (seg; lengths when count > 0; tokens when row_tokens
 * or row_targets is set and count > 0), PA_ERR_SHAPE (count < 0, rows or N < 1, a length
 * < 1 or an offset < 0), PA_ERR_HOST_MEMORY (its O(count + rows) scratch
 * could not be allocated). Nothing is written on error.
 */
pa_status pa_pack_first_fit(const int32_t* lengths, const int32_t* offsets, int32_t count, const int32_t* tokens,
                            int32_t pad_token, int32_t rows, int32_t N, uint64_t seed, uint64_t epoch,
                            int32_t* seg, uint8_t* loss_mask, int32_t* row_tokens, int32_t* row_targets,
                            int64_t* placement, int32_t* rows_used, int64_t* placed_tokens);

/*
 * Fused linear cross-entropy, forward (mlx-train-perf 0.5.1 README, "The
 * fused cross-entropy loss" and "If you maintain a trainer":
 * linear_cross_entropy(hidden, head, targets)). With logits z = H W^T it
 * writes, per token i,
 *   lse[i]          = log sum_v exp(z[i, v])
 *   target_logit[i] = z[i, targets[i]]
 *   nll[i]          = lse[i] - target_logit[i]
 * without storing z: the tensor cores form 128 x 128 logit tiles in TMEM
 * and the epilogue folds each into a running maximum and sum.
 *   hidden       : (N, D) bf16, row-major      head : (V, D) bf16, row-major
 *   targets      : (N) int32; a target outside [0, V) is ignored: its nll
 *                  and target_logit are 0 (lse is still written)
 *   nll, lse, target_logit : (N) fp32
 * N, V >= 1; D a multiple of 64 in [64, 16384]. Device pointers, caller-owned,
 * 16-byte aligned; ws >= pa_lce_workspace_bytes(N, V, D) bytes (its first 4
 * bytes are the device status word read by pa_device_status). Asynchronous
 * on `stream`, like the attention calls.
 * Errors: PA_ERR_SHAPE, PA_ERR_NULL, PA_ERR_ALIGN, PA_ERR_WORKSPACE,
 * PA_ERR_ARCH, PA_ERR_CUDA.
 */
size_t pa_lce_workspace_bytes(int32_t N, int32_t V, int32_t D);
pa_status pa_lce_fwd(int32_t N, int32_t V, int32_t D, const void* hidden, const void* head, const int32_t* targets,
                     float* nll, float* lse, float* target_logit, void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * Fused linear cross-entropy, backward (same README section: the backward
 * recomputes the logit tiles it needs instead of reading a stored matrix).
 * For L = sum_i g[i] * nll[i] it writes
 *   dz[i, v]     = g[i] * (exp(z[i, v] - lse[i]) - [v == targets[i]])
 *   dhidden[i]   = sum_v dz[i, v] head[v]          (N, D) bf16, overwritten
 *   dhead[v]     = sum_i dz[i, v] hidden[i]        (V, D) bf16, overwritten;
 *                  pass NULL when the head does not train (then only
 *                  dhidden is computed)
 * lse (N) fp32 is the forward's; g (N) fp32 is dL/dnll per token (for a
 * masked mean, mask[i] / count). A target outside [0, V) contributes
 * nothing (its row of dz is 0, whatever g[i] is).
 * How: the vocabulary is taken in chunks of Vc rows (8192 for N <= 16384,
 * fewer for longer inputs, so that the two dz buffers of a chunk stay within
 * 512 MiB); per chunk one kernel recomputes the chunk's logits on the tensor
 * cores and writes dz in bf16 (tokens x Vc and Vc x tokens), and two tcgen05
 * GEMMs form dhead's rows of the chunk and add the chunk's share of dhidden
 * to an fp32 accumulator in the workspace. The chunks run in a fixed order,
 * so results do not depend on timing. Nothing of size N x V is stored.
 * Arguments as pa_lce_fwd (16-byte aligned device pointers, caller-owned);
 * ws >= pa_lce_bwd_workspace_bytes(N, V, D), its first 4 bytes the status
 * word. Asynchronous on `stream`.
 * Errors: PA_ERR_SHAPE, PA_ERR_NULL, PA_ERR_ALIGN, PA_ERR_WORKSPACE,
 * PA_ERR_ARCH, PA_ERR_CUDA.
 */
size_t pa_lce_bwd_workspace_bytes(int32_t N, int32_t V, int32_t D);
pa_status pa_lce_bwd(int32_t N, int32_t V, int32_t D, const void* hidden, const void* head, const int32_t* targets,
                     const float* lse, const float* g, void* dhidden, void* dhead, void* ws, size_t ws_bytes,
                     pa_stream_t stream);

/*
 * Log probabilities of given tokens, with the entropy and the most likely
 * alternatives (beside the fused cross-entropy: a policy's loss takes the log
 * probability of each token that was sampled and an entropy bonus, not a mean
 * NLL). With z = H W^T / temperature, never stored, per token i
 *   lse[i]     = ln sum_v exp(z[i, v])
 *   logp[i]    = z[i, targets[i]] - lse[i]
 *   entropy[i] = -sum_v p ln p,  p = exp(z[i, v] - lse[i])
 *   top_ids[i, k], top_logp[i, k]  the `top` largest logits' vocabulary rows and
 *                log probabilities, largest first, the lower row first among equals
 *   hidden  : (N, D) bf16, row-major      head : (V, D) bf16, row-major
 *   targets : (N) int32; outside [0, V) the token is not scored: its logp is 0
 *             (its other outputs are written all the same)
 *   logp, lse, entropy : (N) fp32;  top_ids (N, top) int32, top_logp (N, top) fp32
 * N, V in [1, 2^30]; D a multiple of 64 in [64, 16384]; top in [0, 32] and <= V
 * (0: no alternatives, their pointers are not used); temperature > 0. Any N is
 * one pass over the head: a single token costs the reading of it.
 * Alternatives are ranked by the unscaled logits as the tensor cores' fp32
 * sums give them. Logits of -inf or NaN are no alternatives: a token with fewer
 * others than `top` has id -1 and log probability -inf in the places left. A
 * NaN or +inf logit makes the token's lse, logp and entropy NaN. Finite logits
 * may have any size, a mask's lowest values included. A token's sums keep what
 * their additions round off, so logp of a likely token carries what all the
 * unlikely ones add, to about 1e-6. The logits themselves are the tensor cores'
 * fp32 sums, which are cut towards zero at each 16 of D, by about 2e-8 of the sum
 * (normals at D = 4096: lse is 2e-5 off for logits of up to 10 and 2e-4 for logits
 * of up to 43, and a tenth of that at D = 256).
 * Device pointers, caller-owned, 16-byte aligned; ws >=
 * pa_logp_workspace_bytes(N, V, D, top), its first 4 bytes the status word.
 * Asynchronous on `stream`; results do not depend on timing.
 * Errors: PA_ERR_SHAPE, PA_ERR_NULL, PA_ERR_ALIGN, PA_ERR_WORKSPACE,
 * PA_ERR_ARCH, PA_ERR_CUDA.
 */
size_t pa_logp_workspace_bytes(int32_t N, int32_t V, int32_t D, int32_t top);
pa_status pa_logp_fwd(int32_t N, int32_t V, int32_t D, float temperature, int32_t top, const void* hidden,
                      const void* head, const int32_t* targets, float* logp, float* lse, float* entropy,
                      int32_t* top_ids, float* top_logp, void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * How pa_logp_fwd cuts its work on a device of `sms` SMs (host only, for tests
 * and profiling): plan[0] 1 where two CTAs form one product of 256 tokens, 0
 * where one forms 128; plan[1] the splits of the vocabulary; plan[2] the units
 * of 32 vocabulary rows of a split, plan[3] those of a logit tile (at most 8).
 * A function of its arguments alone. Errors: PA_ERR_SHAPE, PA_ERR_NULL.
 */
pa_status pa_logp_plan(int32_t N, int32_t V, int32_t D, int32_t sms, int32_t* plan);

/*
 * Its backward: for L = sum_i g_logp[i] * logp[i] + g_entropy[i] * entropy[i]
 *   dz[i, v]   = (g_logp[i] ([v == targets[i]] - p) - g_entropy[i] p (ln p + entropy[i])) / temperature
 *   dhidden[i] = sum_v dz[i, v] head[v]      (N, D) bf16, overwritten
 *   dhead[v]   = sum_i dz[i, v] hidden[i]    (V, D) bf16, overwritten; NULL when
 *                the head does not train
 * lse and entropy are the forward's at the same temperature; g_entropy may be
 * NULL (all 0), entropy then too. A target outside [0, V) leaves only the
 * entropy's part; a token without any gradient has a dhidden row of exact
 * zeros. Every row of hidden is a factor in dhead, so a padding row holds
 * finite values even where its gradient is 0. The vocabulary is taken in chunks
 * as in pa_lce_bwd (the logits are formed again, dz of a chunk is held in bf16,
 * up to 128 tokens as the sum of two bf16 terms), in a fixed order: the same
 * call gives the same bits (with dhead NULL, dhidden of up to 128 tokens is
 * summed in another order).
 * How exact: an element of dz is off by at most 2^-16 of itself up to 128
 * tokens and by 2^-8 (its rounding to bf16) from 129 on, where a second term
 * would double two of the three products; the results are rounded to bf16. Of
 * a gradient's norm that is about 1.7e-3 (the results' rounding alone) and
 * 2.4e-3. p is formed from lse in fp32, which adds about 2^-22 |lse| of p (and
 * is taken as 1 where it comes out larger).
 * ws >= pa_logp_bwd_workspace_bytes(N, V, D): up to 262,144 tokens a chunk's dz
 * takes at most 128 MiB of it and its transposed copy 256 MiB (laid out with
 * dhead NULL too), beside dhidden's fp32 accumulators. Arguments, execution and
 * errors otherwise as pa_logp_fwd.
 */
size_t pa_logp_bwd_workspace_bytes(int32_t N, int32_t V, int32_t D);
pa_status pa_logp_bwd(int32_t N, int32_t V, int32_t D, float temperature, const void* hidden, const void* head,
                      const int32_t* targets, const float* lse, const float* entropy, const float* g_logp,
                      const float* g_entropy, void* dhidden, void* dhead, void* ws, size_t ws_bytes,
                      pa_stream_t stream);

/*
 * Activation checkpoints in 8 bits: what the backward needs of the forward,
 * kept at half the size of bf16 in between. The last dimension of a tensor is
 * cut into blocks of `block` elements (32, 64 or 128; a row's last block may
 * be short). Per block
 *   scale = max |x| / top          fp32; top = 127 (PA_CKPT_INT8) or 448 (PA_CKPT_E4M3)
 *   code  = x / scale              rounded once, to nearest even: an int8 in
 *                                  [-127, 127], or a float8 of 4 exponent and 3 mantissa bits
 * and loading gives code * scale, rounded to the tensor's type. A block of
 * zeros has scale 0. A block that holds an infinity or a NaN has scale NaN and
 * codes 0: it comes back as NaN throughout.
 *   x      : (B, H, N, C), element (b, h, n, c) at b*s_b + h*s_h + n*s_n + c, bf16 or fp32
 *            (io_dtype); the source of a save, the destination of a load.
 *            C is a multiple of 8. Strides of dimensions larger than one are
 *            >= C and multiples of 16 bytes; rows of a destination do not overlap.
 *   codes  : (B, H, N, C) bytes, contiguous
 *   scales : (B, H, N, ceil(C / block)) fp32, contiguous
 * One launch for up to PA_CKPT_MAX_TENSORS tensors of one type (q, k, v and
 * out of a layer, say). No workspace. Pointers 16-byte aligned; at most
 * 2^31 - 4096 groups of eight elements per tensor, short blocks counted whole.
 * Errors: PA_ERR_NULL, PA_ERR_SHAPE (also count and block), PA_ERR_DTYPE
 * (io_dtype, format), PA_ERR_ALIGN, PA_ERR_ARCH, PA_ERR_CUDA.
 */
#define PA_CKPT_MAX_TENSORS 8
typedef enum { PA_CKPT_INT8 = 0, PA_CKPT_E4M3 = 1 } pa_ckpt_format;
typedef struct {
  void* x;
  void* codes;
  float* scales;
  int32_t B, H, N, C;
  int64_t s_b, s_h, s_n;
} pa_ckpt_tensor;
pa_status pa_ckpt_save(int32_t count, const pa_ckpt_tensor* tensors, int32_t io_dtype, int32_t format, int32_t block,
                       pa_stream_t stream);
pa_status pa_ckpt_load(int32_t count, const pa_ckpt_tensor* tensors, int32_t io_dtype, int32_t format, int32_t block,
                       pa_stream_t stream);

/*
 * Attention backward from 8-bit checkpoints: pa_bwd with q, k, v and out given
 * as pa_ckpt_save left them (C = D, the four in one format and block). With ^
 * for what a load gives, q^, k^ and v^ in bf16 and out^ unrounded:
 *   P = exp(scale <q^, k^> - lse) over visible pairs, lse the forward's
 *   delta_i = <dout_i, out^_i>,  and the gradients from those as in pa_bwd.
 * One launch brings q^, k^ and v^ into the workspace and forms delta from
 * out's codes; out^ is never stored. P and dS enter the products in bf16 (dS
 * from P unrounded): with the results' own rounding, about 2.4e-3 of each
 * gradient's norm.
 *   q, out : codes (B, Hq, N, D), scales (B, Hq, N, ceil(D / block));  k, v with Hkv
 *   dout, dq, dk, dv : bf16, contiguous, or with `strides` as in pa_bwd_strided
 *            (dout and dq the q_* strides, dk and dv the k_* ones); NULL = contiguous
 *   lse    : (B, Hq, N) fp32;  seg (B, N) int32, or NULL for plain causal; any N
 * ws >= pa_bwd_ckpt_workspace_bytes(dims) (0 if dims are invalid).
 * Errors: as pa_bwd_strided, and PA_ERR_SHAPE (block, or more than 2^31 - 4096
 * groups of eight elements in q), PA_ERR_DTYPE (format).
 */
typedef struct {
  const void* codes;
  const float* scales;
} pa_ckpt;
size_t pa_bwd_ckpt_workspace_bytes(const pa_dims* dims);
pa_status pa_bwd_ckpt(const pa_dims* dims, const pa_strides* strides, int32_t format, int32_t block,
                      const pa_ckpt* q, const pa_ckpt* k, const pa_ckpt* v, const pa_ckpt* out, const void* dout,
                      const float* lse, const int32_t* seg, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                      pa_stream_t stream);

/*
 * Rotary positions: what the attention's queries and keys are turned by before
 * they meet. The first `rot` elements of a head form rot / 2 pairs; at position p
 * pair i, of frequency f_i radians a position, becomes
 *   y1 = a (x1 cos(p f_i) - x2 sin(p f_i)),   y2 = a (x2 cos(p f_i) + x1 sin(p f_i))
 * and the elements past rot stay as they are. PA_ROPE_HALF pairs element i with
 * i + rot / 2, PA_ROPE_INTERLEAVED 2i with 2i + 1.
 *
 * pa_rotary_frequencies (host only) fills f_i = theta^(-2i / rot), i < rot / 2, with
 * `scaling` for contexts longer than those trained on:
 *   PA_ROPE_PLAIN   as they are
 *   PA_ROPE_LINEAR  f_i / factor
 *   PA_ROPE_BASE    theta * factor^(rot / (rot - 2)) in theta's place: the slowest
 *                   pair comes out factor times slower, the fastest as it was
 *   PA_ROPE_BANDS   by the turns r_i = original f_i / (2 pi) that a pair makes over
 *                   the `original` context: f_i / factor up to r_i = low, f_i from
 *                   r_i = high on, linear in r_i between. (Some models' ramp is linear
 *                   in the pair's index i between two rounded ones instead: theirs are other
 *                   frequencies, to be given to pa_rotary_init as they are.)
 * Arguments that a scaling does not name are not looked at.
 * pa_rotary_init (host only) makes the description that the kernels take, from any
 * frequencies (finite) and the amplitude a (1 as a rule). The angle is formed
 * from a 64-bit binary fraction of a turn, so that of the given frequencies (of 2^40 radians
 * at most) is as exact at far positions as at near ones: about 5e-8 radians. What
 * pa_rotary_frequencies rounds to doubles is off by 2^-53 of itself before that.
 *   rot : a multiple of 8 in [8, 128]
 * Errors: PA_ERR_NULL, PA_ERR_SHAPE (rot; theta, factor, original or frequencies
 * not finite and positive, negative frequencies allowed in pa_rotary_init; low >=
 * high; PA_ROPE_BASE with rot 2 or less; an amplitude that is not finite),
 * PA_ERR_DTYPE (layout or scaling).
 */
#define PA_ROPE_MAX_PAIRS 64
#define PA_ROPE_MAX_TENSORS 4
typedef enum { PA_ROPE_HALF = 0, PA_ROPE_INTERLEAVED = 1 } pa_rope_layout;
typedef enum { PA_ROPE_PLAIN = 0, PA_ROPE_LINEAR = 1, PA_ROPE_BASE = 2, PA_ROPE_BANDS = 3 } pa_rope_scaling;
typedef struct {
  int32_t rot, layout;
  float amplitude;
  int32_t ready;                      /* set by pa_rotary_init                   */
  uint64_t turns[PA_ROPE_MAX_PAIRS];  /* 2^64 * (f_i / 2 pi), whole turns dropped */
} pa_rotary;
pa_status pa_rotary_frequencies(int32_t rot, int32_t scaling, double theta, double factor, double original, double low,
                                double high, double* frequencies);
pa_status pa_rotary_init(pa_rotary* rotary, int32_t rot, int32_t layout, const double* frequencies, double amplitude);

/*
 * Positions of packed rows: positions[b, n] = n minus the first token of the run of
 * equal ids that token n of row b lies in. So each segment of a packed row counts
 * from 0 (an id that comes back later in the row starts a run of its own there).
 *   seg, positions : (B, N) int32, contiguous, 16-byte aligned, apart; B * N < 2^31
 * Errors: PA_ERR_SHAPE, PA_ERR_NULL, PA_ERR_ALIGN, PA_ERR_ARCH, PA_ERR_CUDA.
 */
pa_status pa_positions(int32_t B, int32_t N, const int32_t* seg, int32_t* positions, pa_stream_t stream);

/*
 * Rotates up to PA_ROPE_MAX_TENSORS tensors (q and k of a layer, say) in one launch.
 * `backward` non-zero takes gradients back: the rotation by minus the angle with
 * the same amplitude, so dx is written from dy given as x.
 *   x, y : (B, H, N, D), element (b, h, n, c) at b*x_b + h*x_h + n*x_n + c (y_* for y),
 *          bf16 or fp32 (io_dtype, one for all); y may be x with the same strides and
 *          overlaps no tensor of the call otherwise. fp32 arithmetic; bf16 results are
 *          rounded once. Strides of dimensions larger than one are >= D and
 *          multiples of 16 bytes.
 *   positions : (B, N) int32, any values, 4-byte aligned; NULL: position n
 * D a multiple of 8 in [rot, 256]; B * N < 2^31; H in [1, 65535].
 * Errors: PA_ERR_NULL, PA_ERR_SHAPE (also count, and a rotary that pa_rotary_init did
 * not fill), PA_ERR_DTYPE, PA_ERR_ALIGN, PA_ERR_ARCH, PA_ERR_CUDA.
 */
typedef struct {
  const void* x;
  void* y;
  int32_t H;
  int64_t x_b, x_h, x_n, y_b, y_h, y_n;
} pa_rope_tensor;
pa_status pa_rope(const pa_rotary* rotary, int32_t count, const pa_rope_tensor* tensors, int32_t B, int32_t N, int32_t D,
                  int32_t io_dtype, const int32_t* positions, int32_t backward, pa_stream_t stream);

/*
 * A paged cache of keys and values, for generating from the model that is trained.
 * The cache is a pool of pages of `page` tokens; sequence s holds its token j in row
 * j % page of page page_table[s, j / page]. A step brings T rows of new tokens,
 * the sequences' one behind the other: rows q_start[s] .. q_start[s + 1] - 1 are
 * sequence s's last tokens, kv_len[s] its tokens with the new ones counted. So
 * row i of them has position kv_len[s] - (q_start[s + 1] - q_start[s]) + i. One new
 * token a sequence, a few, a chunk of a prompt, none, and any mixture are alike.
 *   q          : (T, Hq, D) bf16     element (t, h, c) at t*q_t + h*q_h + c
 *   k, v       : (T, Hkv, D) bf16    the new tokens', at t*n_t + h*n_h + c
 *   out, q_out : (T, Hq, D) bf16     at t*o_t + h*o_h + c
 *   k_pages, v_pages : (pages, Hkv, page, D) bf16, at p*p_p + h*p_h + n*p_n + c; either
 *                order of heads and tokens in memory, by the strides
 *   page_table : (S, width) int32    q_start : (S + 1) int32, rising    kv_len : (S) int32
 * The three are read on the device, so a captured step is replayed with new
 * lengths. Whatever they hold, no call reads or writes outside the tensors
 * described: q_start is taken within [0, T], a negative kv_len as 0, and tokens past
 * width * page, or on a page number outside [0, pages), are not in the cache:
 * they are neither written nor attended (pages given back at the start of a long
 * context, say, marked with -1). Rows of q before q_start[0] and from q_start[S] on
 * belong to nobody: their outputs stay as they were.
 * D is 64, 96 or 128; page 16, 32, 64, 128 or 256; S, pages, width >= 1; T <= 2^30 (0
 * returns PA_OK without a launch); width * page < 2^31 - 256; S < 2^24. Strides of dimensions
 * larger than one are >= D and multiples of 8; pointers are 16-byte aligned (page_table,
 * q_start and kv_len 4-byte aligned).
 */
typedef struct {
  int32_t S, T, Hq, Hkv, D;
  int32_t pages, page, width;
  float scale; /* softmax scale; <= 0 selects 1/sqrt(D) */
} pa_paged_dims;
typedef struct {
  int64_t q_t, q_h, n_t, n_h, o_t, o_h, p_p, p_h, p_n;
} pa_paged_strides;

/*
 * Writes the new tokens' keys and values into their places in the cache, the keys
 * rotated on the way, and their queries rotated into q_out. `rotary` NULL: nothing is
 * rotated. q may be NULL, q_out then too; q_out may be q with the same strides.
 * positions (T) int32 replaces the tokens' places as what they are rotated by; NULL:
 * their places. A token that has no place in the cache leaves only its q_out. Two
 * tokens of one place (a page listed for two sequences) leave either's value in each element.
 * Errors: PA_ERR_NULL, PA_ERR_HEAD_DIM, PA_ERR_GQA, PA_ERR_SHAPE (also rot > D),
 * PA_ERR_ALIGN, PA_ERR_ARCH, PA_ERR_CUDA.
 */
pa_status pa_paged_append(const pa_paged_dims* dims, const pa_paged_strides* strides, const pa_rotary* rotary,
                          const void* q, const void* k, const void* v, const int32_t* page_table, const int32_t* q_start,
                          const int32_t* kv_len, const int32_t* positions, void* q_out, void* k_pages, void* v_pages,
                          pa_stream_t stream);

/*
 * Attention of the new tokens over the cache (which holds theirs too, see
 * pa_paged_append). For row i of sequence s, at position p, over the keys j <= p that
 * are in the cache, query head h reading kv head h / (Hq / Hkv):
 *   lse[t, h] = ln sum_j exp(scale <q, k_j>)      out = sum_j exp(scale <q, k_j> - lse) v_j
 * A row that sees no key has out 0 and lse -inf. lse (T, Hq) fp32, contiguous. What a page
 * holds past a sequence's tokens may be anything (NaN too); the keys and values
 * up to kv_len are finite. P enters the second product in bf16; sums and maxima are
 * fp32. Hq / Hkv is at most 128.
 * ws >= pa_paged_workspace_bytes(D) bytes, its first 4 the status word (T 0 launches
 * nothing and leaves it as it is); a workspace belongs to one stream at a time. The same call
 * gives the same bits.
 * Errors: PA_ERR_NULL, PA_ERR_HEAD_DIM, PA_ERR_GQA (also Hq / Hkv > 128), PA_ERR_SHAPE, PA_ERR_ALIGN,
 * PA_ERR_WORKSPACE, PA_ERR_ARCH, PA_ERR_CUDA.
 */
size_t pa_paged_workspace_bytes(int32_t D);
pa_status pa_paged_fwd(const pa_paged_dims* dims, const pa_paged_strides* strides, const void* q, const void* k_pages,
                       const void* v_pages, const int32_t* page_table, const int32_t* q_start, const int32_t* kv_len,
                       void* out, float* lse, void* ws, size_t ws_bytes, pa_stream_t stream);

/*
 * Self-test of how pa_paged_fwd deals out its work (host only, no device call): `units`
 * becomes what a step costs, in the units that the kernel would count it in, by the
 * kernel's own arithmetic. q_start (S + 1) and kv_len (S) are host memory here. The kernel adds
 * the costs up in 32 bits, so with rising q_start the sum is below 2^32, whatever kv_len holds.
 * Errors: PA_ERR_NULL, PA_ERR_HEAD_DIM, PA_ERR_GQA, PA_ERR_SHAPE.
 */
pa_status pa_selftest_paged_units(const pa_paged_dims* dims, const int32_t* q_start, const int32_t* kv_len, uint64_t* units);

/* Static, human-readable name of a status code. */
const char* pa_status_string(pa_status s);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
