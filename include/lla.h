/*
 * lla.h -- C ABI of the Looped Latent Attention (LLA) decode library for NVIDIA
 * B200 (sm_100a).
 *
 * What the method computes (pages cited by title and section):
 *   "Looped Latent Attention: Cross-Loop KV Compression for Looped Transformers"
 *   (gist.science explainer), Technisches Resümee / Kernmechanismus:
 *     encode                c    = (x - mu) W_down
 *     loop-specific decode  x^_t = c W_up,t^T + mu_t
 *   where x = [x_1; ...; x_T] is one token's pre-RoPE K (or V) for every loop.
 *   "Looped Latent Attention: 跨循环 KV 压缩精读" (cc.laoqi.cc close reading),
 *   §二.1 symbol table (W_down is (T d_head) x r, W_up,t is d_head x r),
 *   §二.2 eq. (4) (exact ratio 2 T d_head / (r_k + r_v)), §二.3 (compress before
 *   RoPE, rotate the rebuilt K at its position), §二.6 (LLA-2D folds the heads
 *   into one latent of input width T H d_head; the latent-store path keeps only
 *   latents and rebuilds on read).
 *
 * Conventions
 *   - Loops are 0-based (t = 0 .. T-1); the pages count from 1.
 *   - Row vectors, as on the pages.  Every matrix is row-major, C order.
 *   - bf16 values are passed as their uint16_t bit patterns.
 *   - RoPE is the split-half layout: pair (i, i + d/2) rotates by angle
 *     pos * rope_base^(-2 i / d).  Scores are scaled by sm_scale (1/sqrt(d) when 0).
 *   - The in-flight token (the one whose loops are still running) is not in the
 *     latent cache: its loop-t K and V are passed exactly (k_self, v_self) and it
 *     attends to itself at q_pos.  It is encoded with lla_encode after its last loop.
 *
 * Ownership and execution
 *   - Every buffer is allocated by the caller.  Pointers named d_* or documented
 *     as "device" must be device memory of the current CUDA device; the library
 *     never allocates device memory, never synchronises the device, and enqueues
 *     work only on `stream` (a cudaStream_t passed as void*; NULL = legacy stream).
 *   - Device pointers must be 16-byte aligned; tensors are dense (no strides).
 *   - Functions are thread-safe; calls on one stream run in order.
 *
 * Errors
 *   Every int-returning function returns LLA_OK (0) or a negative code.  On error
 *   nothing was enqueued, and lla_last_error() (thread-local) describes it.
 *   Errors found on the device (positions outside the RoPE table, ctx_len outside
 *   [0, n_cap], cache slots outside the cache) never fault: the offending element
 *   is skipped or clamped and a bit is set in a device status word (see below).
 */
#ifndef LLA_H_
#define LLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LLA_OK 0
#define LLA_ERR_INVALID (-1)     /* null pointer, bad size, misaligned pointer, t >= T ... */
#define LLA_ERR_UNSUPPORTED (-2) /* shape outside the supported set (see lla_cfg) */
#define LLA_ERR_TOO_SMALL (-3)   /* packed / table / workspace buffer too small */
#define LLA_ERR_CUDA (-4)        /* a CUDA call or kernel launch failed */

#define LLA_MODE_PER_HEAD 0 /* one (c_k, c_v) pair per token, layer and head */
#define LLA_MODE_2D 1       /* LLA-2D: one (c_k, c_v) pair per token and layer */

/* Device status bits (see lla_decode_attn / lla_encode). */
#define LLA_STATUS_POSITION_RANGE 1 /* a history position or q_pos outside [0, rope_max_pos) */
#define LLA_STATUS_CTX_RANGE 2      /* ctx_len[b] outside [0, n_cap] (clamped) */
#define LLA_STATUS_SLOT_RANGE 4     /* an encode slot outside [0, n_slots) (skipped) */
#define LLA_STATUS_TIMEOUT 8        /* a kernel wait timed out; that call's output is invalid */
#define LLA_STATUS_PAGE_RANGE 16    /* a page outside [0, n_pages), or a free list out of bounds */
#define LLA_STATUS_PAGES_SHORT 32   /* lla_page_map: a sequence was not served */
#define LLA_STATUS_NONFINITE 64     /* lla_q8_append: a NaN or an infinity among keys or values */
#define LLA_STATUS_ROPE_TABLE 128   /* lla_decode_attn: a table of scaled frequencies; output invalid */

/*
 * Codec geometry of one shared layer.
 * Supported: 1 <= T <= 64; 1 <= H <= 128; d_head in {32, 64, 96, 128};
 * r_k, r_v multiples of 8 in [8, 256]; rope_base > 1; sm_scale >= 0;
 * d_rope in {0, 32, 64, d_head} (see the field).
 */
typedef struct lla_cfg {
  int32_t T;        /* loops */
  int32_t H;        /* attention heads (K/V heads; MHA) */
  int32_t d_head;   /* head width d */
  int32_t r_k;      /* K latent width */
  int32_t r_v;      /* V latent width */
  int32_t mode;     /* LLA_MODE_PER_HEAD or LLA_MODE_2D */
  float rope_base;  /* RoPE base, e.g. 10000 */
  float sm_scale;   /* softmax scale; 0 selects 1/sqrt(d_head) */
  int32_t d_rope;   /* 0: RoPE over the whole head (the method's default).  Otherwise the
                       decoupled RoPE of the close reading, Appendix J: only the first
                       d_rope dims of q and k rotate, as a rotary vector of their own width
                       (pairs (i, i + d_rope/2), angle pos * rope_base^(-2 i / d_rope)),
                       and the other dims form a NoPE content path that decode absorbs into
                       the query.  Supported: 32 or 64, below d_head, decode on the
                       tensor-core path (per head and LLA-2D); d_rope == d_head is the
                       default RoPE. */
} lla_cfg;

/* Last error message of the calling thread ("" if none). Never NULL. */
const char* lla_last_error(void);

/* Library version string ("lla-b200 <major>.<minor> ..."); 0.2 added lla_cfg.d_rope,
 * the full-memory fast path and the eviction calls; 0.3 the rotary, page and 8-bit cache calls. */
const char* lla_version(void);

/* ------------------------------------------------------------------------ */
/* Bookkeeping (host only, exact integers).                                  */
/* ------------------------------------------------------------------------ */

/*
 * Exact compression ratio of the persistent cache as a reduced fraction num/den.
 * Per head: 2 T d_head / (r_k + r_v)  (close reading §二.2 eq. (4); gist.science
 * "Zentrale Beiträge").  LLA-2D: 2 T H d_head / (r_k + r_v)  (close reading §二.6).
 */
int lla_ratio(const lla_cfg* cfg, int64_t* num, int64_t* den);

/*
 * Bytes of bf16 latent cache for `tokens` tokens over `layers` layers:
 * (r_k + r_v) * H * tokens * layers * 2 per head, (r_k + r_v) * tokens * layers * 2
 * for LLA-2D.  Also the uncompressed loop-indexed cache (2 T H d_head scalars per
 * token and layer) when teacher != 0.  Fails with LLA_ERR_INVALID on overflow.
 */
int lla_cache_bytes(const lla_cfg* cfg, int64_t tokens, int64_t layers, int teacher,
                    int64_t* bytes);

/* ------------------------------------------------------------------------ */
/* Codec packing (once per layer).                                            */
/* ------------------------------------------------------------------------ */

/* Size in bytes of the packed codec buffer for cfg (0 if cfg is unsupported). */
size_t lla_codec_packed_bytes(const lla_cfg* cfg);

/*
 * Pack fp32 codec parameters (device pointers) into the library's internal
 * device layout.  Inputs (row-major fp32):
 *   per head:  W_down_{k,v} [H][T*d][r],  W_up_{k,v} [H][T][d][r],  mu_{k,v} [H][T*d]
 *   LLA-2D:    W_down_{k,v} [T*H*d][r],   W_up_{k,v} [T][H][d][r],  mu_{k,v} [T*H*d]
 *   (concatenation order: loop-major, then head for LLA-2D, then the d entries.)
 * The packed buffer (`packed`, device, >= lla_codec_packed_bytes(cfg)) holds W_up
 * and mu in fp32, W_down rounded to bf16 (round to nearest even; stored twice: row
 * major, and cut into the tensor-core encode's operand tiles), and the encode bias
 * mu W_down computed with that rounded W_down.  Inputs may be freed once the stream
 * has passed this call.
 */
int lla_codec_pack(const lla_cfg* cfg, const float* W_down_k, const float* W_down_v,
                   const float* W_up_k, const float* W_up_v, const float* mu_k,
                   const float* mu_v, void* packed, size_t packed_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* RoPE table (once per d_head / base / maximum position).                    */
/* ------------------------------------------------------------------------ */

/* Size in bytes of the RoPE table covering positions [0, max_pos). */
size_t lla_rope_table_bytes(const lla_cfg* cfg, int32_t max_pos);

/*
 * Fill `table` (device) with (cos, sin) of pos * rope_base^(-2i/d_head) for
 * pos < max_pos, i < d_head/2, as fp32 pairs [max_pos][d_head/2][2].  Angles are
 * formed and reduced in fp64 and rounded once to fp32, so large positions keep
 * full fp32 accuracy (close reading §二.3: full-dimension RoPE on the rebuilt K).
 */
int lla_rope_table(const lla_cfg* cfg, int32_t max_pos, void* table, size_t table_bytes,
                   void* stream);

/* ------------------------------------------------------------------------ */
/* Encode: codec write of finished tokens.                                    */
/* ------------------------------------------------------------------------ */

/*
 * c = (x - mu) W_down, rounded to bf16, for n_tok finished tokens
 * (gist.science, Kernmechanismus, latent storage; close reading §二.6 for LLA-2D).
 *   x_k, x_v  device bf16 [n_tok][T][H][d]: each token's pre-RoPE K / V rows for all
 *             loops (the concatenation x = [x_0; ...; x_{T-1}] per head, or over
 *             (t, h) for LLA-2D).
 *   slot      device int64 [n_tok]: destination row of each token in the cache.
 *   c_k, c_v  device bf16 caches with n_slots rows: per head [n_slots][H][r_k] and
 *             [n_slots][H][r_v]; LLA-2D [n_slots][r_k] and [n_slots][r_v].  A
 *             cache laid out [B][n_cap][...] is addressed by slot = b * n_cap + j.
 *   status    optional device int32 (may be NULL): LLA_STATUS_SLOT_RANGE is OR-ed
 *             in when a slot is outside [0, n_slots); that token is skipped.
 * n_tok == 0 is a no-op.
 */
int lla_encode(const lla_cfg* cfg, const void* packed, int64_t n_tok, const uint16_t* x_k,
               const uint16_t* x_v, const int64_t* slot, int64_t n_slots, uint16_t* c_k,
               uint16_t* c_v, int32_t* status, void* stream);

/* ------------------------------------------------------------------------ */
/* Decode attention over the latent cache at loop t.                          */
/* ------------------------------------------------------------------------ */

/*
 * Workspace bytes needed by lla_decode_attn for (cfg, B, n_cap).  The workspace
 * must be zero-filled once before its first use; the library keeps it consistent
 * afterwards.  Its first two int32 words are the device status: word 0 collects
 * the bits of the call in flight, word 1 holds the final bits of the last
 * completed call (LLA_STATUS_* values).
 */
size_t lla_decode_workspace_bytes(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/*
 * out[b][h] = attention of the loop-t query over the history rebuilt from the
 * latents plus the in-flight token (gist.science Kernmechanismus, loop-specific
 * reconstruction; close reading §二.3, RoPE after reconstruction):
 *   k_j  = RoPE(c_k,j W_up,k,t,h^T + mu_k,t,h, positions[b][j])
 *   s_j  = sm_scale * RoPE(q, q_pos[b]) . k_j ,  s_self likewise with k_self
 *   p    = softmax over {s_j : j < ctx_len[b]} and s_self
 *   out  = W_up,v,t,h (sum_j p_j c_v,j) + (sum_j p_j) mu_v,t,h + p_self v_self
 * (values are summed in latent space and up-projected once; equal to rebuilding
 * each V because the weights are linear in the rebuilt values.)
 *   packed        codec from lla_codec_pack (device)
 *   rope_table    table from lla_rope_table covering [0, rope_max_pos) (device); one from
 *                 lla_rope_table_scaled sets LLA_STATUS_ROPE_TABLE
 *   t             loop index, 0 <= t < T
 *   B, n_cap      batch and cache capacity per sequence (n_cap >= 0)
 *   ctx_len       device int32 [B]: history length of each sequence (<= n_cap)
 *   q, k_self, v_self  device fp32 [B][H][d]: the in-flight token's loop-t query,
 *                 key and value, pre-RoPE
 *   positions     device int32 [B][n_cap]: position of each history token
 *   q_pos         device int32 [B]: position of the in-flight token
 *   c_k, c_v      device bf16 latent caches: per head [B][n_cap][H][r_k] / [..][r_v];
 *                 LLA-2D [B][n_cap][r_k] / [B][n_cap][r_v].  Rows at or past ctx_len[b]
 *                 never reach the output, whatever they hold (NaN included).
 *   out           device fp32 [B][H][d]
 *   ws            device workspace of >= lla_decode_workspace_bytes(cfg, B, n_cap)
 * Work is launched on `stream` only; there is no host synchronisation.
 */
int lla_decode_attn(const lla_cfg* cfg, const void* packed, const void* rope_table,
                    int32_t rope_max_pos, int32_t t, int32_t B, int32_t n_cap,
                    const int32_t* ctx_len, const float* q, const float* k_self,
                    const float* v_self, const int32_t* positions, const int32_t* q_pos,
                    const uint16_t* c_k, const uint16_t* c_v, float* out, void* ws,
                    size_t ws_bytes, void* stream);

/*
 * lla_decode_attn for callers that cannot allocate device memory.
 *
 * The paper has no counterpart to this entry point; it exists for deployment.
 * Some callers cannot call cudaMalloc or any other allocator when they run
 * decode: code inside an allocator-free region of a host runtime, plugins that
 * are handed only their input and output buffers, or servers that forbid
 * allocation after start-up so that their memory use stays fixed.  This call
 * computes exactly what lla_decode_attn computes (same kernels, same arguments
 * and layouts) but takes no workspace: its split partials and status words live
 * in a fixed device array of 8 MiB (8388608 bytes) that the library holds on
 * every GPU where it is loaded, until the process exits.
 *   - Shapes whose workspace (lla_decode_workspace_bytes) exceeds 8 MiB are
 *     rejected with LLA_ERR_TOO_SMALL, and every argument lla_decode_attn checks
 *     is checked, before anything is enqueued: a rejected call leaves the array
 *     and status_out untouched.  B == 0 enqueues nothing.
 *   - The first call on a device looks up the array's device address with that
 *     device current (cudaGetSymbolAddress); make that first call before any
 *     stream capture.  Later calls reuse the address while the device keeps the
 *     same CUDA context, and look it up again after a device reset.
 *   - All calls share the one array and it keeps the last call's contents.  Each
 *     call clears the status words it needs; calls that overlap on the GPU (on
 *     different streams, or from different threads) race on the array and must
 *     be serialised by the caller.
 *   - status_out: optional device int32 (may be NULL) that receives this call's
 *     LLA_STATUS_* bits, written on `stream` after the kernels.
 * It allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 */
int lla_decode_attn_noalloc(const lla_cfg* cfg, const void* packed, const void* rope_table,
                            int32_t rope_max_pos, int32_t t, int32_t B, int32_t n_cap,
                            const int32_t* ctx_len, const float* q, const float* k_self,
                            const float* v_self, const int32_t* positions,
                            const int32_t* q_pos, const uint16_t* c_k, const uint16_t* c_v,
                            float* out, int32_t* status_out, void* stream);

/*
 * Number of kernel launches one lla_decode_attn call makes for (cfg, B, n_cap)
 * (for launch accounting by callers); -1 if the shape is unsupported.
 */
int lla_decode_launches(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/* ------------------------------------------------------------------------ */
/*
 * Eviction composed with the latent cache: a sink + window retention budget
 * (close reading §四.10, Table 9: 4 sink tokens + a 256-token window; Appendix J:
 * a 1024-token budget).  The first `sink` history tokens and the `window` most
 * recent ones are kept, each at its own position.  A sequence's cache rows then
 * act as sink + window slots: history position p < sink lives in slot p, and
 * p >= sink in slot sink + (p - sink) mod window, overwriting the position that
 * just left the window.  Each slot's positions entry holds its token's position
 * and the decode reads slots [0, ctx_len) with ctx_len = min(n, sink + window);
 * attention over a set does not depend on slot order, so lla_decode_attn is
 * used unchanged.  No data moves when a token is evicted.
 */

/* Slot (row within its sequence) of history position pos; host only, exact.
 * Returns -1 when sink < 0, window < 1 or pos < 0. */
int64_t lla_evict_slot(int32_t sink, int32_t window, int64_t pos);

/*
 * Decode-time append under eviction, one new history token per sequence:
 *   pos        device int32 [B]: history position of each sequence's new token
 *              (its index in the history: the previous ctx_len when nothing was
 *              evicted yet); pos < 0 leaves the sequence untouched and writes
 *              slot -1 (lla_encode then skips it).
 *   slot       device int64 [B] (out): flat cache row b * n_cap + slot for lla_encode.
 *   positions  device int32 [B][n_cap] (in/out): the slot's entry is set to pos.
 *   ctx_len    device int32 [B] (out): min(pos + 1, sink + window).
 * Requires B >= 0, n_cap >= 1, sink >= 0, window >= 1 and sink + window <= n_cap
 * (LLA_ERR_INVALID otherwise); pointers 8-byte (slot) or 4-byte aligned.
 * Enqueued on `stream`; B == 0 is a no-op.
 */
int lla_evict_append(int32_t B, int32_t n_cap, int32_t sink, int32_t window, const int32_t* pos,
                     int64_t* slot, int32_t* positions, int32_t* ctx_len, void* stream);

/* ------------------------------------------------------------------------ */
/* Full-memory fast path: rebuild once, then ordinary attention.              */
/* ------------------------------------------------------------------------ */

/*
 * The close reading ("Looped Latent Attention: 跨循环 KV 压缩精读", §四.9, Table 5
 * and the paragraph after it) contrasts the latent store (keep only latents,
 * rebuild on every read) with a full-memory fast path that keeps the complete
 * rebuilt K/V, giving up the cache saving for speed.  Per §二.3 the codec works
 * on pre-RoPE K and the model rotates the rebuilt key at its position before it
 * is cached, so the full cache holds rotated keys.
 *
 * Full cache of one loop t: k_full and v_full, each device bf16 [B][H][n_cap][d]
 * (head-major: one (sequence, head) history is a contiguous run of rows).
 */

/* Bytes of one of k_full / v_full for (cfg, B, n_cap); 0 if the arguments are invalid. */
size_t lla_full_kv_bytes(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/*
 * Rebuild rows of the loop-t full cache from the latent cache:
 *   k_full[b][h][j] = bf16(RoPE(c_k[b][j](h) W_up,k,t,h^T + mu_k,t,h, positions[b][j]))
 *   v_full[b][h][j] = bf16(c_v[b][j](h) W_up,v,t,h^T + mu_v,t,h)
 * for each row b * n_cap + j listed in slot[0 .. n_rows) (device int64), or for
 * rows 0 .. n_rows-1 when slot is NULL (n_rows <= B * n_cap; B * n_cap rebuilds the
 * whole cache once).  c_k, c_v and positions are laid out as for lla_decode_attn;
 * packed and rope_table as for lla_decode_attn.  status (optional device int32)
 * collects LLA_STATUS_SLOT_RANGE (a slot outside [0, B * n_cap): skipped) and
 * LLA_STATUS_POSITION_RANGE (a position outside the table: clamped).  Runs on the
 * CUDA cores; it is a once-per-token conversion, not a per-step cost.
 */
int lla_full_rebuild(const lla_cfg* cfg, const void* packed, const void* rope_table,
                     int32_t rope_max_pos, int32_t t, int32_t B, int32_t n_cap,
                     const int32_t* positions, const uint16_t* c_k, const uint16_t* c_v,
                     const int64_t* slot, int64_t n_rows, uint16_t* k_full, uint16_t* v_full,
                     int32_t* status, void* stream);

/* Workspace bytes for lla_full_decode_attn (zero-filled once before first use; its
 * first two int32 words are the status words described at lla_decode_workspace_bytes). */
size_t lla_full_decode_workspace_bytes(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/* Kernel launches one lla_full_decode_attn call makes (1 or 2), or -1 if invalid. */
int lla_full_decode_launches(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/*
 * out[b][h] = ordinary decode attention over the full cache plus the in-flight token:
 *   s_j   = sm_scale * RoPE(q, q_pos[b]) . k_full[b][h][j]   (j < ctx_len[b])
 *   s_self = sm_scale * RoPE(q, q_pos[b]) . RoPE(k_self, q_pos[b])
 *   out   = sum_j p_j v_full[b][h][j] + p_self v_self,  p = softmax(s, s_self)
 *   q, k_self, v_self  device fp32 [B][H][d], pre-RoPE; q_pos, ctx_len device int32 [B]
 *   k_full, v_full     device bf16 [B][H][n_cap][d] (may be NULL when n_cap == 0)
 *   out                device fp32 [B][H][d]
 * The cfg's codec fields (T, r_k, r_v, mode) are not used.  B * H * n_cap must stay
 * below 2^31 rows (LLA_ERR_UNSUPPORTED otherwise).  Device-side range problems set
 * LLA_STATUS_POSITION_RANGE / LLA_STATUS_CTX_RANGE in the workspace status word.
 */
int lla_full_decode_attn(const lla_cfg* cfg, const void* rope_table, int32_t rope_max_pos,
                         int32_t B, int32_t n_cap, const int32_t* ctx_len, const float* q,
                         const float* k_self, const float* v_self, const int32_t* q_pos,
                         const uint16_t* k_full, const uint16_t* v_full, float* out, void* ws,
                         size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Rotary positions as operators.                                             */
/* ------------------------------------------------------------------------ */

#define LLA_ROPE_HALF 0        /* pairs (i, i + rd/2) */
#define LLA_ROPE_INTERLEAVED 1 /* pairs (2i, 2i + 1) */

#define LLA_F32 0
#define LLA_BF16 1

/*
 * Frequencies for contexts longer than the trained one.  With theta_i =
 * rope_base^(-2i/rd), rd the rotary dims (d_rope, or d_head when d_rope is 0), and
 * s = factor (>= 1), position p turns pair i by p times
 *   NONE    theta_i
 *   LINEAR  theta_i / s
 *   NTK     (rope_base * s^(rd/(rd-2)))^(-2i/rd)
 *   YARN    theta_i (1 - r_i) + theta_i / s * r_i, with the ramp r_i rising from 0 at
 *           pair max(floor(at(beta_fast)), 0) to 1 at min(ceil(at(beta_slow)), rd - 1),
 *           at(n) = rd ln(orig_len / (2 pi n)) / (2 ln rope_base), the pair that turns n
 *           times over the orig_len positions trained on.
 * The tables stay plain rotations: the attention factor that goes with YARN,
 * f = (0.1 ln s + 1)^2 on the rotary dims' part of a score, belongs in lla_cfg.sm_scale where the
 * whole head rotates; where only d_rope dims do, multiply those dims of the queries by f.
 */
#define LLA_ROPE_SCALE_NONE 0
#define LLA_ROPE_SCALE_LINEAR 1
#define LLA_ROPE_SCALE_NTK 2
#define LLA_ROPE_SCALE_YARN 3

typedef struct lla_rope_scaling {
  int32_t kind;      /* LLA_ROPE_SCALE_* */
  int32_t orig_len;  /* YARN: trained context, >= 1 */
  double factor;     /* s, finite and >= 1 */
  double beta_fast;  /* YARN; 0 selects 32 */
  double beta_slow;  /* YARN; 0 selects 1; below beta_fast */
} lla_rope_scaling;

/*
 * lla_rope_table with scaled frequencies (same layout, size and accuracy).  Such a
 * table serves lla_rope_apply, the lla_q8_* and the lla_full_* calls, which take their
 * angles from it.  lla_decode_attn does not: its kernels form the history's angles from
 * rope_base, and a scaled table would turn only the query by other ones.  So a table whose
 * frequencies differ (kind not NONE, factor not 1) has a sine of -0 at position 0 of pair 0,
 * which changes no rotation, and lla_decode_attn sets LLA_STATUS_ROPE_TABLE for it.  (NTK alone
 * can be had there: rope_base times s^(rd/(rd-2)).)
 */
int lla_rope_table_scaled(const lla_cfg* cfg, const lla_rope_scaling* scaling, int32_t max_pos,
                          void* table, size_t table_bytes, void* stream);

/*
 * y = x rotated at its positions, on rows of n_heads heads of d_head:
 *   (y_a, y_b) = (x_a c - x_b s, x_a s + x_b c) on the pairs (a, b) of `layout` among the
 *   rotary dims, (c, s) the table's row at positions[token]; other dims are copied.
 * inverse != 0 rotates back, which is also the gradient: dL/dx = inverse rotation of dL/dy.
 *   x, y       device, dtype LLA_F32 or LLA_BF16 (arithmetic in fp32, each product and
 *              each sum rounded): token i's heads
 *              start at element i * stride and are contiguous; strides in elements, whole
 *              multiples of 16 bytes, at least n_heads * d_head.  y == x with the same
 *              stride rotates in place; rows of x and y must not overlap otherwise
 *              (LLA_ERR_INVALID), but may alternate in one buffer with one stride.
 *   positions  device int32 [n_tok]; outside [0, rope_max_pos) they are clamped and
 *              LLA_STATUS_POSITION_RANGE is OR-ed into status (device int32, may be NULL).
 * 1 <= n_heads <= 4096; n_tok == 0 is a no-op.
 */
int lla_rope_apply(const lla_cfg* cfg, const void* rope_table, int32_t rope_max_pos,
                   int32_t layout, int32_t inverse, int32_t dtype, int64_t n_tok,
                   int32_t n_heads, const int32_t* positions, const void* x, int64_t x_stride,
                   void* y, int64_t y_stride, int32_t* status, void* stream);

/* ------------------------------------------------------------------------ */
/* Pages: block tables and slot maps from request lengths.                    */
/* ------------------------------------------------------------------------ */

/*
 * A paged cache keeps sequence b's token j in row j % page of page
 * block_table[b][j / page].  One call grows and shrinks every sequence of a batch:
 *   n_new      device int32 [B]: n_new[b] > 0 appends that many tokens, < 0 drops the last
 *              -n_new[b] (all of them when it holds fewer), 0 leaves the sequence.
 *   ctx_len    device int32 [B] (in/out): the lengths.
 *   block_table device int32 [B][max_pages] (in/out): entries [0, ceil(len/page)) are the
 *              sequence's pages; entries given back become -1, others are not touched.
 *   free_list  device int32 [n_pages] (in/out), n_free device int32 [1] (in/out): the pages
 *              free_list[0 .. n_free) are free; the top is taken first.
 *   tok_start  device int32 [B + 1] (out): the appended tokens of sequence b are tokens
 *              tok_start[b] .. tok_start[b + 1] of the batch (prefix sums).
 *   slot       device int64 [tok_cap] (out): each token's row page_id * page + offset in the
 *              cache; -1 past the last token.  positions device int32 [tok_cap] (out): its
 *              index in its sequence; 0 past the last token.
 * Pages given back are free for the same call.  Growing sequences are served in order:
 * one whose pages, with all that was asked before it, exceed the free ones, or whose
 * tokens likewise exceed tok_cap, is left as it was (LLA_STATUS_PAGES_SHORT; the tokens after
 * it move up in tok_start, see row_start at lla_q8_append_rows), and so is
 * one that would pass max_pages * page tokens or whose ctx_len is outside that range
 * (LLA_STATUS_CTX_RANGE).  Dropping the tokens a call just appended restores free_list,
 * n_free, ctx_len and block_table (whose new entries become -1).  A page index outside
 * [0, n_pages) is kept as -1 and sets LLA_STATUS_PAGE_RANGE; tokens in it get slot -1.
 * page in {16, 32, 64, 128}; B <= 65535; max_pages * page and tok_cap below 2^31.  slot and
 * positions may be NULL when tok_cap == 0.  Pointers 4-byte (slot 8-byte) aligned; status
 * (device int32, may be NULL) collects the bits.  No buffer may overlap another.
 */
int lla_page_map(int32_t B, int32_t page, int32_t max_pages, int32_t n_pages, int32_t* ctx_len,
                 const int32_t* n_new, int32_t* block_table, int32_t* free_list, int32_t* n_free,
                 int64_t tok_cap, int32_t* tok_start, int64_t* slot, int32_t* positions,
                 int32_t* status, void* stream);

/* ------------------------------------------------------------------------ */
/* Paged 8-bit cache: exact keys and values, one scale per page and head.     */
/* ------------------------------------------------------------------------ */

/*
 * The 8-bit cache keeps a token's own keys and values of one loop and layer (close
 * reading §三.2's kv_quant, without the latent codec) in int8, value = code * scale:
 *   k, v             device int8 [n_pages][H][page][d_head]; keys are stored rotated
 *   k_scale, v_scale device fp32 [n_pages][H]
 * half the bytes of the lla_full cache, in pages that sequences of any length share.
 * The cfg's codec fields (T, r_k, r_v, mode) are not used; H, d_head, d_rope, rope_base
 * and sm_scale are.  A value is off by at most half its page's scale per rounding.
 */
typedef struct lla_q8_cache {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int32_t n_pages;
  int32_t page;      /* tokens per page: 16, 32, 64 or 128 */
} lla_q8_cache;

/* Bytes of k (or of v) for n_pages pages; 0 if the arguments are invalid. */
size_t lla_q8_cache_bytes(const lla_cfg* cfg, int32_t n_pages, int32_t page);

/*
 * Append tokens: rows tok_start[b] .. tok_start[b + 1] of k and v are the last tokens of
 * sequence b, whose length with them is ctx_len[b] (as lla_page_map leaves them).  A sequence
 * that lla_page_map refused has no rows there: where k and v hold some all the same, call
 * lla_q8_append_rows.
 *   k, v       dtype LLA_F32 or LLA_BF16, rows of H heads of d_head, k_stride / v_stride
 *              elements apart (as lla_rope_apply's); n_tok rows are there to read.
 *   rope_table, rope_max_pos, layout, positions [n_tok]: keys are rotated in fp32 on the way,
 *              as by lla_rope_apply.  rope_table NULL: keys come rotated, positions unused.
 * Per page and head, with amax the largest magnitude among the new tokens' values, in fp32
 * (every product rounded; amax / 127 is amax * fp32(1 / 127), value / scale is
 * value * fp32(1 / scale), so that codes repeat bit by bit from elementary operations):
 *   page without earlier tokens   scale = amax / 127
 *   page with earlier tokens      scale kept if amax / 127 <= scale, else it becomes
 *                                 max(amax / 127, 1.25 scale) and the codes of the earlier
 *                                 tokens are rounded again; later rows are not touched
 *   code = round(value / scale), ties to even.
 * An amax of 1e-30 or less asks for a scale of 0, whose values read as zeros.  A scale found
 * on a page that is below 7.8e-33 or not finite, which no append leaves, counts as 0: what the
 * earlier tokens held reads as zeros.  NaN is stored as 0 and an infinity as the largest code
 * (amax looks at finite values), with LLA_STATUS_NONFINITE.  A page must belong to one
 * appended sequence only: written from two, its contents are unspecified.
 * Sequences whose tok_start or ctx_len do not fit (LLA_STATUS_CTX_RANGE) and pages
 * outside the cache (LLA_STATUS_PAGE_RANGE) are skipped.  B <= 65535.  With no token, page or
 * table entry at all (B, n_tok, n_pages or max_pages 0) nothing is enqueued and no bit set.
 */
int lla_q8_append(const lla_cfg* cfg, const lla_q8_cache* cache, const void* rope_table,
                  int32_t rope_max_pos, int32_t layout, int32_t dtype, int32_t B,
                  int32_t max_pages, const int32_t* ctx_len, const int32_t* block_table,
                  int32_t n_tok, const int32_t* tok_start, const int32_t* positions,
                  const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  int32_t* status, void* stream);

/*
 * lla_q8_append for k and v whose rows were laid out before the call that grew the sequences:
 * sequence b's tokens are rows row_start[b], row_start[b] + 1, ... of k and v (device int32 [B];
 * 0, 1, .. B - 1 for a decode step with a row per sequence).  lla_page_map packs tok_start over
 * the sequences that it served, so after a refusal (or beside a sequence that did not grow) token
 * tok_start[b] is no longer row tok_start[b]: without row_start every later sequence would store
 * another one's keys and values.  A sequence whose rows do not lie within the n_tok rows is
 * skipped (LLA_STATUS_CTX_RANGE).  positions stay in the order of tok_start.
 */
int lla_q8_append_rows(const lla_cfg* cfg, const lla_q8_cache* cache, const void* rope_table,
                       int32_t rope_max_pos, int32_t layout, int32_t dtype, int32_t B,
                       int32_t max_pages, const int32_t* ctx_len, const int32_t* block_table,
                       int32_t n_tok, const int32_t* tok_start, const int32_t* positions,
                       const int32_t* row_start, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int32_t* status, void* stream);

/*
 * Rows of the cache as bf16: k_out, v_out [n_rows][H][d_head] = code * scale of row slot[i]
 * (page_id * page + offset, as lla_page_map's slots).  A slot outside the cache leaves its
 * output row as it was (LLA_STATUS_SLOT_RANGE).
 */
int lla_q8_read(const lla_cfg* cfg, const lla_q8_cache* cache, int64_t n_rows,
                const int64_t* slot, uint16_t* k_out, uint16_t* v_out, int32_t* status,
                void* stream);

/* Workspace bytes of lla_q8_decode_attn for sequences of up to n_cap tokens (zero-filled
 * once before first use); 0 if the arguments are invalid.  Its int32 word 1 holds the final
 * status bits of the last completed call, as at lla_decode_workspace_bytes; word 0 is not used. */
size_t lla_q8_decode_workspace_bytes(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/* Kernel launches one lla_q8_decode_attn call makes, or -1 if invalid. */
int lla_q8_decode_launches(const lla_cfg* cfg, int32_t B, int32_t n_cap);

/*
 * Decode attention, one token per sequence, over the 8-bit cache and the in-flight token:
 *   s_j    = sm_scale * RoPE(q, q_pos[b]) . k_j (j < ctx_len[b]),  s_self likewise
 *   out    = sum_j p_j v_j + p_self v_self,  p = softmax(s, s_self)
 *   q, k_self, v_self, out   dtype [B][H][d_head]; k_self and v_self both NULL: the history
 *              alone (a sequence of length 0 then gives zeros)
 *   ctx_len [B], block_table [B][max_pages], q_pos [B] device int32 (q_pos unused and
 *              rope_table NULL when q and k_self come rotated)
 *   ws         >= lla_q8_decode_workspace_bytes(cfg, B, max_pages * page)
 * Tokens of a page outside the cache are left out (LLA_STATUS_PAGE_RANGE); what the cache
 * holds past ctx_len[b] or in pages of other sequences does not reach the output.
 * Softmax, weights and sums are held in fp32.  A score is an exact integer dot product per 16
 * dims (12 with d_head 96), in which each element of q is held to 2^-24 of the largest of
 * those dims (at or below 1e-30 they count as zeros), times fp32 scales.
 * B <= 65535; B * H * (max_pages * page / 32 + 16) at most 2^31 - 4097 (LLA_ERR_UNSUPPORTED).
 */
int lla_q8_decode_attn(const lla_cfg* cfg, const lla_q8_cache* cache, const void* rope_table,
                       int32_t rope_max_pos, int32_t layout, int32_t dtype, int32_t B,
                       int32_t max_pages, const int32_t* ctx_len, const int32_t* block_table,
                       const void* q, const void* k_self, const void* v_self,
                       const int32_t* q_pos, void* out, void* ws, size_t ws_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LLA_H_ */
