/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact, IO-aware, tiled attention library.
 *
 * The library computes exact scaled-dot-product attention
 *     O = softmax(tau * Q K^T + mask) V
 * tile by tile with the online-softmax recurrence (running row max m, running
 * row sum l, accumulator rescaled by exp(m_old - m_new)), never writes the
 * N x N score or probability matrix to memory, and saves only O and the per-row
 * logsumexp.  The backward pass recomputes the probability tiles on chip from
 * Q, K, V and the logsumexp.  Sources of the method:
 *   - "FlashAttention: Fast and Memory-Efficient Exact Attention with
 *     IO-Awareness" (Dao et al., 2022), as summarised on tonho.wtf (section
 *     "como funciona": the recurrence, the saved statistics, recomputation in
 *     the backward pass and D_i = dO_i . O_i) and agihunt.info (the fused
 *     forward/backward kernels, on-chip masking and dropout replay, and the
 *     block-sparse variant);
 *   - marketmaker.cc "Flash Attention" post (Q-outer loop, causal tile
 *     skipping, the PyTorch (batch, heads, seq, head_dim) interface);
 *   - lynx-cortex "FlashAttention como una optimizacion de roofline" (the
 *     Q-outer loop with deferred normalisation used by the forward kernel).
 *
 * Conventions shared by every entry point
 *   - Tensors Q, O, dO, dQ are logical [B, H, N, d] arrays of one dtype,
 *     addressed as base + b*stride_b + h*stride_h + n*stride_n + c (element
 *     strides; the head dimension is contiguous).  K, V, dK, dV are
 *     [B, H_kv, N, d] arrays of the same dtype with the kv_stride_* strides;
 *     H_kv = H (multi-head attention) unless grouped-query attention is asked
 *     for.  LSE is a contiguous float32 [B, H, N] array.
 *   - Grouped-query attention (living-dl-book, "Atencao eficiente", section
 *     6): the H query heads form H_kv groups of g = H / H_kv heads, and every
 *     head of group k reads K/V head k, i.e. query head h reads K/V head h / g;
 *     g = 1 is multi-head and g = H multi-query attention.  dK and dV of a
 *     shared head are the sums over its g query heads.
 *   - Sliding window (lynx-cortex, "Problemas de practica", the
 *     sliding-window exercise), read as the local causal window: with
 *     window = w > 0 and causal set, key j is visible to query i iff
 *     i - w < j <= i; whole K/V tiles outside every window of a query tile
 *     are skipped.
 *   - Head dimension: d = 64 for every dtype; d = 128 for float16 and
 *     bfloat16 (the pages name d = 128 as the case where the on-chip tile
 *     budget gets tight: marketmaker.cc, "O que isso custou"; lynx-cortex,
 *     "Lo que Flash forward no hace").  Other values, and d = 128 with
 *     float32, return FA_ERR_UNSUPPORTED.
 *   - Ownership: the caller owns every buffer and the stream.  The library
 *     never allocates, frees or synchronises device memory, except that
 *     fa_check_status synchronises the stream it is given.  Work is enqueued
 *     asynchronously on `stream` (a cudaStream_t; NULL = legacy default
 *     stream).  All pointers named "device" must be device-accessible.
 *   - Errors found on the host (shapes, alignment, unsupported combinations,
 *     too small a workspace, a failed launch) are returned synchronously and
 *     nothing is enqueued.  There is no silent fallback to another algorithm:
 *     every unsupported combination returns FA_ERR_UNSUPPORTED.
 *   - Device-side waits are bounded; a wait that runs out records
 *     FA_ERR_TIMEOUT in the workspace status word, the kernel releases its
 *     resources and exits, and fa_check_status reports it.
 *   - Re-entrant: no global mutable state.  Concurrent calls need separate
 *     workspaces.
 */
#ifndef FA_GB300_FA_H
#define FA_GB300_FA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,   /* null pointer, bad shape, bad probability ...   */
  FA_ERR_UNSUPPORTED = 2,   /* valid request this build does not implement    */
  FA_ERR_MISALIGNED = 3,    /* base pointer or stride breaks the 16-B rule    */
  FA_ERR_WORKSPACE = 4,     /* workspace NULL or smaller than the query says  */
  FA_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed              */
  FA_ERR_TIMEOUT = 6        /* a bounded device-side wait ran out             */
} fa_status;

typedef enum { FA_DT_F32 = 0, FA_DT_F16 = 1, FA_DT_BF16 = 2 } fa_dtype;

typedef struct {
  int32_t B, H, N, d;        /* batch, heads, sequence length, head dim         */
  int32_t dtype;             /* fa_dtype of Q,K,V,O,dO,dQ,dK,dV                 */
  int64_t stride_b;          /* element strides shared by all [B,H,N,d] tensors */
  int64_t stride_h;
  int64_t stride_n;
  float scale;               /* tau; <= 0 selects 1/sqrt(d)                     */
  int32_t causal;            /* nonzero: key j visible to query i iff j <= i    */
  const int32_t *seqlens_k;  /* device [B] or NULL: keys j >= L_b are masked     */
  float dropout_p;           /* in [0, 1); 0 disables dropout                   */
  uint64_t seed;             /* Philox4x32-10 key = (lo32(seed), hi32(seed))    */
  uint64_t offset;           /* Philox counter words 2,3 = (lo32, hi32)(offset) */
  const uint8_t *block_mask; /* device [nb][nb] (nb = ceil(N/block_size)),
                                nonzero = keep the block; or NULL (dense)       */
  int32_t block_size;        /* must be 128 when block_mask != NULL             */
  float *o_f32;              /* optional device [B,H,N,d] contiguous float32:
                                fa_fwd also writes O before its final rounding
                                to the storage dtype (parity diagnostics)       */
  void *prof_start;          /* optional cudaEvent_t pair: when both are set,   */
  void *prof_stop;           /* they are recorded on `stream` right before and
                                right after the main attention kernel of the
                                call (profiling; not owned by the library)      */
  /* -- ABI 1.1 -- zero-filled by callers of 1.0, which keeps their meaning */
  int32_t H_kv;              /* K/V heads; H % H_kv == 0; 0 selects H           */
  int64_t kv_stride_b;       /* element strides of K, V, dK, dV [B,H_kv,N,d];   */
  int64_t kv_stride_h;       /* all three 0 selects stride_b/h/n, allowed only  */
  int64_t kv_stride_n;       /* when H_kv == H                                  */
  int32_t window;            /* w > 0: key j visible to query i only if
                                i - w < j (requires causal); 0 = no window     */
  /* -- ABI 1.3 -- zero-filled by older callers, which keeps their meaning */
  int32_t fwd_kernel;        /* forward kernel at head dimension 64:
                                0 = chosen by the library (see fa_fwd);
                                1 = one 128-row query tile per CTA, two CTAs
                                    per SM; 2 = two query tiles per CTA
                                    sharing their K/V tiles.  Both compute
                                    the same result; other values and other
                                    head dimensions ignore it             */
} fa_params;

/* ---------------------------------------------------------------------------
 * fa_fwd_workspace_size / fa_bwd_workspace_size
 * Bytes of device workspace fa_fwd / fa_bwd need for `p` (0 is never
 * returned: the status word is always present).  Pure host function.
 * The backward workspace holds the float32 dQ accumulator [B,H,N,d] (16-bit
 * dtypes), D = rowsum(dO o O) [B,H,N], block lists and the status word.
 * ------------------------------------------------------------------------- */
size_t fa_fwd_workspace_size(const fa_params *p);
size_t fa_bwd_workspace_size(const fa_params *p);

/* ---------------------------------------------------------------------------
 * fa_fwd -- forward pass.
 * Computes, for every (b, h) head, O = P~ V with P = softmax(tau Q K^T) over
 * the visible keys (causal AND key-padding AND block mask), P~ = Z o P/(1-p)
 * when dropout is on, and LSE_i = m_i + ln l_i (natural log, tau-scaled
 * scores; -inf for a row with no visible key, whose O row is 0).
 * Method: Q-outer tiling with the online-softmax recurrence and deferred
 * normalisation (lynx-cortex, "El algoritmo Flash (forward)"; marketmaker.cc,
 * "O algoritmo de atencao do Flash"), whole future / masked / sparse tiles
 * skipped (marketmaker.cc, "O mascaramento causal"; agihunt.info, block-sparse
 * paragraph), dropout applied on chip (agihunt.info, fused-kernel paragraph).
 *   q, k, v : device [B,H,N,d] inputs (strides in p)
 *   o       : device [B,H,N,d] output, same dtype and strides
 *   lse     : device float32 [B,H,N] output
 *   ws      : device workspace of ws_bytes >= fa_fwd_workspace_size(p)
 * Dropout element (b,h,i,j) is kept iff the 16-bit slice (j & 7) of
 * Philox4x32-10(counter = (j>>3, (b*H+h)*N+i, lo32(offset), hi32(offset)),
 * key = (lo32(seed), hi32(seed))) is >= round(p * 65536); slice t is half
 * (t & 1) of output word (t >> 1), low half first.  Requires B*H*N < 2^32.
 * At head dimension 64 with fwd_kernel = 0 the library runs the one-tile
 * kernel unless the query tiles average at least 64 key tiles (dense or
 * causal, no window, no block mask) and the two-tile grid fills at least four
 * waves of the GPU, where sharing K/V tiles between two query tiles wins.
 * ------------------------------------------------------------------------- */
fa_status fa_fwd(const fa_params *p, const void *q, const void *k, const void *v,
                 void *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fa_bwd -- backward pass by recomputation (tonho.wtf, "como funciona": only
 * O, the softmax statistics and the RNG state are kept; S and P are rebuilt
 * on chip; D_i = dO_i . O_i replaces a length-N reduction).
 * For upstream gradient dO it computes, with the same mask and dropout
 * replay as fa_fwd:
 *   dV = P~^T dO;  dP = Z o (dO V^T)/(1-p);  D_i = dO_i . O_i;
 *   dS = P o (dP - D);  dQ = tau dS K;  dK = tau dS^T Q.
 *   q,k,v,o,dout : device [B,H,N,d] inputs;  lse: device float32 [B,H,N]
 *                  from fa_fwd with the same p
 *   dq,dk,dv     : device [B,H,N,d] outputs (same dtype and strides)
 *   ws           : device workspace, ws_bytes >= fa_bwd_workspace_size(p)
 * ------------------------------------------------------------------------- */
fa_status fa_bwd(const fa_params *p, const void *q, const void *k, const void *v,
                 const void *o, const void *dout, const float *lse,
                 void *dq, void *dk, void *dv, void *ws, size_t ws_bytes,
                 void *stream);

/* ---------------------------------------------------------------------------
 * fa_bwd_noalloc -- fa_bwd for callers that cannot allocate device memory.
 * The FlashAttention pages have no counterpart; this is an interface
 * convenience around the same backward kernels.
 * Some callers cannot hand fa_bwd a workspace: code running inside a memory
 * pool it does not own, hooks where allocation is forbidden, or plain C
 * programs without a device allocator.  This entry point takes the
 * backward pass's scratch (dQ accumulator, padded LSE / D rows, status word)
 * from a fixed 64 MiB array compiled into the library's device image; every
 * device that loads the library holds that array until the process exits.
 * Arguments are those of fa_bwd without ws / ws_bytes.
 *   - Returns FA_ERR_WORKSPACE, enqueuing nothing, when
 *     fa_bwd_workspace_size(p) exceeds 64 MiB.  For 16-bit inputs the
 *     scratch is about 264 bytes per query row at d = 64 and 520 at
 *     d = 128 (float32 dQ accumulator, LSE and D), so B*H*N may reach about
 *     254,000 rows at d = 64 and 129,000 at d = 128; float32 inputs need
 *     8 bytes per row.  Block-sparse masks add their block lists.
 *   - The array's device address is looked up on every call (with the
 *     calling thread's current device).  The first call on a device also
 *     loads the library's device image there; make that first call before
 *     any stream capture.
 *   - All calls on a device share the array and leave their contents in it;
 *     what must start at zero is cleared on the stream by each call, but
 *     calls whose GPU work overlaps (unordered streams) race on it.
 *   - It calls no cudaMalloc, cudaFree or other allocating routine.
 *   - A bounded device wait that gives up records FA_ERR_TIMEOUT in the
 *     array's status word: read it with fa_noalloc_check_status.
 * ------------------------------------------------------------------------- */
fa_status fa_bwd_noalloc(const fa_params *p, const void *q, const void *k, const void *v,
                         const void *o, const void *dout, const float *lse,
                         void *dq, void *dk, void *dv, void *stream);

/* fa_noalloc_check_status -- fa_check_status for fa_bwd_noalloc: synchronises
 * `stream`, then returns the status word the last fa_bwd_noalloc on the
 * current device left in the fixed array (FA_OK, or FA_ERR_TIMEOUT if a
 * bounded device wait ran out; the gradients are then undefined).
 * FA_ERR_CUDA if the stream reported an error. */
fa_status fa_noalloc_check_status(void *stream);

/* fa_noalloc_scratch -- the current device's address and size of the fixed
 * array fa_bwd_noalloc uses (for diagnostics: e.g. to run
 * fa_selftest_wait_timeout on it).  Allocates nothing. */
fa_status fa_noalloc_scratch(void **addr, size_t *bytes);

/* ---------------------------------------------------------------------------
 * fa_check_status -- synchronises `stream`, then reads the status word the
 * last fa_fwd/fa_bwd on `ws` left: FA_OK, or FA_ERR_TIMEOUT if a bounded
 * device wait ran out (outputs are then undefined).  FA_ERR_CUDA if the
 * stream reported an error.
 * ------------------------------------------------------------------------- */
fa_status fa_check_status(const void *ws, void *stream);

/* ---------------------------------------------------------------------------
 * fa_dropout_mask -- writes the dropout keep-mask fa_fwd/fa_bwd use for rows
 * row0 .. row0+nrows-1 of head (b, h): out[r][j] = 1 if kept, else 0, for
 * j in [0, N).  out: device uint8 [nrows][N].  Same mapping as fa_fwd.
 * For testing the mapping bit for bit; the attention kernels never store Z.
 * ------------------------------------------------------------------------- */
fa_status fa_dropout_mask(const fa_params *p, int32_t b, int32_t h, int32_t row0,
                          int32_t nrows, uint8_t *out, void *stream);

/* ---------------------------------------------------------------------------
 * fa_selftest_wait_timeout -- exercises the bounded device-side wait that
 * every attention kernel uses, without any attention work and without a
 * fault: one CTA of two warps waits on mbarriers that nothing arrives at,
 * the second warp starting one second after the first.  The first wait
 * gives up after the library's limit (2 s of %globaltimer), records
 * FA_ERR_TIMEOUT in the status word at the start of `ws` and raises the
 * CTA's abort flag; the second wait then returns on that flag, about one
 * second after it began.  The kernel exits normally and the context stays
 * usable.
 *   ws    : device workspace of >= 256 bytes (the status word is cleared
 *           first, as fa_fwd / fa_bwd do)
 *   out   : device int32[2]: 1 where a warp's wait returned "gave up"
 *   out_ns: device uint64[1]: nanoseconds the second warp waited
 * fa_check_status(ws) then returns FA_ERR_TIMEOUT.  For tests of the
 * failure path; it takes about two seconds.
 * ------------------------------------------------------------------------- */
fa_status fa_selftest_wait_timeout(void *ws, int32_t *out, uint64_t *out_ns, void *stream);

/* ---------------------------------------------------------------------------
 * FP8 forward (ABI 1.2).
 * FlashAttention-3's low-precision path (living-dl-book, "Atencao Eficiente
 * em Escala", section 10; marketmaker.cc, "FA3: Mecanica da tremonha", item
 * 3): Q, K and V are quantised to FP8 one tile at a time, with one scale per
 * tile, after a random Hadamard-style rotation of every row that spreads
 * outlying coordinates; the rotation is undone after the products.  Here:
 *   - FP8 is E4M3 (largest finite 448), round to nearest even, saturating;
 *   - the rotation is M = diag(signs) H_d / sqrt(d) (H_d the Sylvester
 *     Hadamard matrix); Q, K and V rows are all rotated; the scores are
 *     unchanged (M M^T = I) and O is rotated back, O = O' M^T;
 *   - a block is 128 rows x d of one head, scale = amax / 448, codes =
 *     E4M3(x * (448 / amax)); per_tensor = 1 uses the whole tensor's amax
 *     for every block and is the pages' baseline;
 *   - both products run in E4M3 on the tensor cores; the probabilities of
 *     key tile t are rounded to E4M3 as E4M3(exp(S - m) * 256 * sv_t / SV)
 *     with m the running row max (the accumulator is rescaled whenever m
 *     grows), sv_t the V scale of tile t and SV the largest V scale of the
 *     head; the row sum uses the unrounded probabilities;
 *   - head dimension 64 or 128, float16 or bfloat16 inputs and output; causal,
 *     key padding, block-sparse masks, the sliding window and grouped K/V
 *     heads as in fa_fwd; dropout returns FA_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t per_tensor;        /* 0: one scale per 128-row block; 1: per tensor   */
  const int8_t *signs;       /* device int8 [d] of +1 / -1, 16-byte aligned:
                                rotate rows by diag(signs) H_d / sqrt(d);
                                NULL: no rotation                              */
} fa_fp8_params;

/* Byte offsets (multiples of 256) of the parts of the quantised buffer:
 *   q8  : uint8 [B,H,N,d]      E4M3 codes of the (rotated) Q rows
 *   k8  : uint8 [B,H_kv,N,d]   of K
 *   v8t : uint8 [B,H_kv,d,Np]  of V, transposed (keys contiguous), Np = N
 *                              rounded up to 128, zero on keys >= N
 *   sq  : float [B,H,nt]       dequantisation scale of each 128-row tile,
 *   sk, sv : float [B,H_kv,nt] nt = ceil(N / 128)
 *   amax: float [4]            scratch of the per-tensor mode
 * total is the buffer size. */
typedef struct {
  size_t q8, k8, v8t, sq, sk, sv, amax, total;
} fa_fp8_layout;

/* Fills *out for the problem p (a pure host function). */
fa_status fa_fp8_buffer_layout(const fa_params *p, fa_fp8_layout *out);

/* fa_fp8_quantize -- quantises q, k, v ([B,H,N,d] / [B,H_kv,N,d] 16-bit
 * tensors with the strides of p) into buf (device, 16-byte aligned,
 * buf_bytes >= layout.total).  The float32 order of operations is fixed:
 * sign flip, butterfly stages h = 1, 2, ..., d/2, multiply by 1/sqrt(d),
 * block amax, inv = 448 / amax, x * inv, E4M3 rounding. */
fa_status fa_fp8_quantize(const fa_params *p, const fa_fp8_params *f, const void *q, const void *k,
                          const void *v, void *buf, size_t buf_bytes, void *stream);

/* fa_fwd_fp8 -- the forward pass on a buffer fa_fp8_quantize filled with
 * the same p and f (f->signs rotates O back).  o: device [B,H,N,d] output in
 * p->dtype with p's strides; lse: device float32 [B,H,N] (natural log of
 * the scores of the dequantised operands); ws: ws_bytes >=
 * fa_fwd_workspace_size(p).  p->o_f32, if set, receives O before its final
 * rounding. */
fa_status fa_fwd_fp8(const fa_params *p, const fa_fp8_params *f, const void *buf, size_t buf_bytes,
                     void *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Rotary positions (ABI 1.4).
 * fa_rope turns the first `rot` columns of every row of q and k by the row's
 * position, one pair of columns at a time:
 *     (x0, x1) -> m (x0 cos a - x1 sin a, x1 cos a + x0 sin a),  a = p f_i,
 * with p the token's position, f_i = inv_freq[i] the pair's inverse frequency
 * (radians per position) and m = mscale.  Pair i is columns (i, i + rot/2), or
 * (2i, 2i + 1) when `interleaved` is set; columns from rot on are copied.
 * `backward` flips the sign of sin, which makes the map the transpose of the
 * forward one: applied to dQ and dK after the attention's backward pass it
 * gives the gradients of the unrotated q and k.
 *   - q, q_out are [B,H,N,d] and k, k_out [B,H_kv,N,d] tensors of one dtype
 *     (float32, float16, bfloat16), each with its own element strides; the
 *     last dimension is contiguous.  H_kv = 0: no k.  Inputs may be broadcast
 *     (stride 0).  An output may be its own input (same base, same strides);
 *     any other overlap of an output with an input is an error of the caller.
 *   - d is a multiple of 8 up to 256, rot even, 2 <= rot <= d.
 *   - Bases and strides follow the 16-byte rule (a dimension of one element
 *     may have any stride).
 *   - positions: device int32 (or int64 with positions_i64) array, the
 *     position of token n of sequence b at b*pos_stride_b + n*pos_stride_n
 *     (pos_stride_b = 0: the same for every sequence); NULL: start + n.
 *     Positions may be negative.  The angle is reduced to a fraction of a
 *     turn exactly, in 64-bit integers, so it does not lose accuracy with
 *     the position (float64's own 2^-53 of p f remains).
 *   - inv_freq: device float64 [rot/2], read on the stream.  A NaN or infinite
 *     frequency makes its pair's two columns NaN at every position.
 *   - Products and sums are float32, rounded once to the dtype.
 *   - No workspace, one launch.  B*N*d < 2^32 - 4096.
 * ------------------------------------------------------------------------- */
typedef enum { FA_ROPE_NONE = 0, FA_ROPE_LINEAR = 1, FA_ROPE_NTK = 2, FA_ROPE_YARN = 3 } fa_rope_scaling;

typedef struct {
  int32_t B, H, H_kv, N, d;
  int32_t rot;               /* rotated leading columns, even                   */
  int32_t dtype;             /* fa_dtype                                        */
  int32_t interleaved;       /* 0: pairs (i, i + rot/2); else (2i, 2i + 1)      */
  int32_t backward;          /* nonzero: the transposed rotation                */
  int32_t positions_i64;     /* positions are int64                             */
  int64_t q_stride_b, q_stride_h, q_stride_n;
  int64_t k_stride_b, k_stride_h, k_stride_n;
  int64_t q_out_stride_b, q_out_stride_h, q_out_stride_n;
  int64_t k_out_stride_b, k_out_stride_h, k_out_stride_n;
  const void *positions;     /* device, or NULL                                 */
  int64_t pos_stride_b, pos_stride_n;
  int64_t start;             /* position of token 0 when positions is NULL      */
  const double *inv_freq;    /* device float64 [rot/2]                          */
  float mscale;              /* factor on cos and sin (1 for plain rotations)   */
} fa_rope_params;

fa_status fa_rope(const fa_rope_params *p, const void *q, const void *k, void *q_out, void *k_out, void *stream);

/* fa_rope_frequencies -- inverse frequencies and mscale of a rotation of rot
 * columns, written to HOST memory (a pure host function):
 *   FA_ROPE_NONE    base^(-2i/rot)
 *   FA_ROPE_LINEAR  the same divided by factor (positions interpolated)
 *   FA_ROPE_NTK     base replaced by base * factor^(rot/(rot-2)): the slowest
 *                   pair is slowed by factor, the fastest not at all
 *   FA_ROPE_YARN    pairs that turn more than beta_fast times within
 *                   original_len positions are kept, those that turn less
 *                   than beta_slow times are divided by factor, a linear ramp
 *                   over the pair index between; mscale = 0.1 ln(factor) + 1
 * factor >= 1; original_len, beta_fast > beta_slow > 0 matter to YARN only. */
fa_status fa_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, int64_t original_len,
                              double beta_fast, double beta_slow, double *inv_freq, float *mscale);

/* ---------------------------------------------------------------------------
 * Differential attention (ABI 1.4).
 * Head pair h (of H) has two score maps over one set of values:
 *     P_m = softmax(tau Q_m K_m^T + mask), m = 1, 2;   O = (P_1 - lam[h] P_2) V.
 *   - q: [B,2H,N,64], the pair's maps in heads 2h and 2h + 1; k: [B,2H_kv,N,64]
 *     alike; v: [B,H_kv,N,128]; o, o2: [B,H,N,128] (one stride set for both);
 *     lse: contiguous float32 [B,2H,N], natural log, one row set per map.
 *     Query pair h reads K/V pair h / (H / H_kv); H_kv = 0 selects H.
 *   - float16 or bfloat16, d = 64 (128 value columns); others return
 *     FA_ERR_UNSUPPORTED.  lam: device float32 [H], any finite values for which
 *     the dtype holds O, P_1 - lam P_2 and the gradients (float16 ends at 65504).
 *   - Masks: causal, seqlens_k (keys j >= L_b are masked; K and V rows there
 *     may hold anything, NaN included), window (causal only).  A query row
 *     that sees no key has O = 0, O_2 = 0, both logsumexps -inf and no part
 *     in any gradient.  Its q and dO rows, like every K and V row that is not
 *     masked, should be finite all the same: the tile products take masked
 *     places times zero, which spreads a NaN or infinity over its tile.
 *   - Weights are rounded to the dtype before the product with V, which is
 *     summed in float32 and normalised by the sum of the rounded weights.
 *   - 2*B*H*N < 2^32.  16-byte rule for bases and strides (a dimension of one
 *     element may have any stride).
 * fa_diff_fwd writes o, lse and, when o2 is not NULL, the second map's own
 * output O_2 = P_2 V, which the backward pass needs.
 * fa_diff_bwd takes o, o2 and lse of a forward call with the same p and inputs
 * and writes, for the upstream gradient dout [B,H,N,128] (do_stride_*):
 *     dP = dO V^T, D_m = rowsum(P_m o dP), dS_1 = P_1 o (dP - D_1),
 *     dS_2 = -lam P_2 o (dP - D_2), dV = (P_1 - lam P_2)^T dO,
 *     dQ_m = tau dS_m K_m, dK_m = tau dS_m^T Q_m, dlam = -sum D_2
 * with dq, dk, dv in q's, k's and v's strides (no broadcast strides) and dlam
 * float32 [H].  D_m comes from dO and the rounded O and O_2, so a row whose
 * exact dS vanishes (one visible key) gets a residue of their rounding.  For head
 * pairs with |lam| > 2, where that residue would outgrow dS_1, D_1 is summed from
 * float32 P_1 and dP instead, which makes the backward pass of such pairs about
 * 1.7 times as long.  dQ is
 * accumulated in float32 in the order in which the key tiles finish: its last
 * bit may differ from run to run; every other output repeats bit for bit.
 * Workspace: fa_diff_*_workspace_size bytes, 16-byte aligned; status word at
 * its start, read by fa_check_status.  Nothing persists in it between calls.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t B, H, H_kv, N, d;  /* H: head pairs; d = 64 columns per map           */
  int32_t dtype;
  int32_t causal, window;    /* as in fa_params                                 */
  float scale;               /* tau; <= 0 selects 1/sqrt(d)                     */
  const int32_t *seqlens_k;  /* device [B] or NULL                              */
  const float *lam;          /* device float32 [H]                              */
  int64_t q_stride_b, q_stride_h, q_stride_n;
  int64_t k_stride_b, k_stride_h, k_stride_n;
  int64_t v_stride_b, v_stride_h, v_stride_n;
  int64_t o_stride_b, o_stride_h, o_stride_n;
  int64_t do_stride_b, do_stride_h, do_stride_n;   /* fa_diff_bwd only          */
} fa_diff_params;

size_t fa_diff_fwd_workspace_size(const fa_diff_params *p);
size_t fa_diff_bwd_workspace_size(const fa_diff_params *p);
fa_status fa_diff_fwd(const fa_diff_params *p, const void *q, const void *k, const void *v, void *o, void *o2,
                      float *lse, void *ws, size_t ws_bytes, void *stream);
fa_status fa_diff_bwd(const fa_diff_params *p, const void *q, const void *k, const void *v, const void *o,
                      const void *o2, const void *dout, const float *lse, void *dq, void *dk, void *dv, float *dlam,
                      void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Attention over a shared prefix (ABI 1.4): B sequences that continue one
 * prefix, T new tokens of each (T = 1: one decoding step).
 *   - q, o: [B,H,T,d]; k_prefix, v_prefix: [H_kv,P,d], one copy for the batch;
 *     k, v: [B,H_kv,M,d], each sequence's own cache, of which the first
 *     L_b = seqlens_k[b] rows are filled, the T new tokens' rows among them
 *     (L_b is taken into [0, M]).  lse: contiguous float32 [B,H,T], natural log.
 *   - Query t of sequence b sees every prefix key and its own keys
 *     j <= L_b - T + t.  A query that sees no key has O = 0 and lse -inf.
 *     Query head h reads K/V head h / (H / H_kv); H_kv = 0 selects H.
 *   - P = 0 (plain cached attention) and M = 0 (only the prefix) are allowed;
 *     the pointers of an empty part may be NULL.
 *   - Cache rows at or past L_b may hold anything, NaN included, and are
 *     not written.
 *   - float16, bfloat16; d = 64 or 128.  Weights are rounded to the dtype
 *     before the product with V; sums, statistics and joins are float32.
 *   - lam: differential attention over the same prefix and caches (fa_diff_fwd's
 *     step for few tokens).  H and H_kv then count head pairs: q is
 *     [B,2H,T,64], k_prefix [2H_kv,P,64], k [B,2H_kv,M,64] with the two maps of
 *     pair h in heads 2h and 2h + 1, v_prefix [H_kv,P,128], v [B,H_kv,M,128],
 *     o [B,H,T,128], lse [B,2H,T], and O = O_1 - lam[h] O_2.  d = 64 only.
 *   - Results repeat bit for bit; they do not depend on what else runs.
 *   - B*H*T (twice that with lam) < 2^26, P and M <= 2^28.  16-byte rule for bases and strides (a
 *     dimension of one element may have any stride); offsets are 64-bit.
 * The prefix is read once per K/V head for up to 64 query rows together (256 where
 * there is much work) of all B * H / H_kv * T, not once per sequence.  Workspace:
 * fa_prefix_workspace_size bytes, 16-byte aligned, nothing persists in it;
 * status word at its start, read by fa_check_status.
 * ------------------------------------------------------------------------- */
typedef struct {
  int32_t B, H, H_kv, T;
  int32_t P, M;              /* prefix keys; rows of each own cache             */
  int32_t d, dtype;
  float scale;               /* tau; <= 0 selects 1/sqrt(d)                     */
  const int32_t *seqlens_k;  /* device [B]                                      */
  int64_t q_stride_b, q_stride_h, q_stride_n;
  int64_t o_stride_b, o_stride_h, o_stride_n;
  int64_t k_stride_b, k_stride_h, k_stride_n;
  int64_t v_stride_b, v_stride_h, v_stride_n;
  int64_t kp_stride_h, kp_stride_n;
  int64_t vp_stride_h, vp_stride_n;
  const float *lam;          /* NULL, or device float32 [H]: differential form  */
} fa_prefix_params;

size_t fa_prefix_workspace_size(const fa_prefix_params *p);
fa_status fa_prefix_fwd(const fa_prefix_params *p, const void *q, const void *k_prefix, const void *v_prefix,
                        const void *k, const void *v, void *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char *fa_status_string(fa_status s);

/* Library ABI version (major * 100 + minor): 101 adds H_kv, kv_stride_*
 * and window to fa_params; 102 adds the FP8 forward; 103 adds fwd_kernel,
 * fa_noalloc_check_status and fa_noalloc_scratch; 104 adds fa_rope,
 * fa_diff_* and fa_prefix_*. */
int32_t fa_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FA_GB300_FA_H */
