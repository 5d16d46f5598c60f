/*
 * fox.h — C ABI of the forget-gated causal softmax attention library (libfox.so).
 *
 * The operation (Forgetting Transformer, FoX). Per batch b and head h, with
 * tokens t = 0..N-1:
 *   f_t = sigmoid(z_t),  a_t = log f_t,  c_t = sum_{l<=t} a_l
 *   D_ij = c_i - c_j          (bias_from_j = 0, the default; D_ii = 0)
 *   D_ij = c_i - c_{j-1}      (bias_from_j = 1; c_{-1} = 0)
 *   S_ij = scale * q_i . k_j + D_ij  for j <= i  (causal; j > i excluded unless non_causal)
 *   LSE_i = ln sum_{j<=i} exp(S_ij),  O_i = sum_{j<=i} exp(S_ij - LSE_i) v_j
 * Sources: "Forgetting Transformer (FoX) Attention" module source
 * (frankenstein-transformer docs, fox_attn: module docstring formula and
 * ForgettingAttention.forward — sigmoid gate, log, cumsum, outer difference,
 * causal mask, scaled logits + bias, softmax, attn @ v); foxwindow README,
 * "The window is a first-passage time" (score form with the sum from j+1);
 * fast-transformers "Creating a custom attention layer", "New Attention"
 * (attention-only call on projected, head-split inputs, [batch, length,
 * heads, dim] layout). The backward is the chain rule through the same
 * formula; the gate gradient is d a_t = sum_{s>=t} (R_s - C_s) (+ C_t under
 * bias_from_j = 1), R/C the row/column sums of dS, and dz_t = d a_t * sigmoid(-z_t).
 *
 * Layout (all row-major, contiguous, device memory):
 *   q, k, v, o, dO, dq, dk, dv : [B, N, H, d], element type per params.dtype
 *   z, lse, dz                  : [B, N, H] fp32
 * Alignment: q, k, v, o, dO, dq, dk, dv 16-byte aligned; z, lse, dz 4-byte
 * aligned; workspace 256-byte aligned.
 *
 * Ownership and threading: the caller owns every buffer, the workspace
 * included. The library allocates no device memory, keeps no state between
 * calls except a lazily-resolved driver entry point, and never synchronises
 * (fox_check_error excepted). All work is enqueued on `stream` (a
 * cudaStream_t; NULL means the legacy default stream) of the current device.
 * Outputs are fully overwritten. Calls on different streams must use
 * different workspaces.
 *
 * Errors: every call validates its arguments on the host and returns a
 * fox_status without touching the GPU when they are wrong. Device-side waits
 * are bounded; a wait that gives up sets a bit in the workspace's error word
 * (reset by each fox_fwd / fox_bwd call) and the kernel exits cleanly;
 * fox_check_error reports it.
 */
#ifndef FOX_H_
#define FOX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fox_status {
  FOX_OK = 0,
  FOX_ERR_INVALID_ARG = 1, /* null pointer, negative size, misalignment, bad flag or dtype */
  FOX_ERR_UNSUPPORTED = 2, /* well-formed but not implemented (d not in {64, 128}; fp32 backward;
                              non_causal or tile_skip with fp32; tile_skip with non_causal;
                              other page sizes; a batch beyond the limits of its counts) */
  FOX_ERR_WORKSPACE = 3,   /* workspace null, misaligned or smaller than the size query */
  FOX_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
  FOX_ERR_TIMEOUT = 5,     /* a device-side bounded wait gave up (from fox_check_error) */
  FOX_ERR_DEVICE = 6       /* another device-side error bit was set (from fox_check_error), e.g. a
                              V value outside the fp16 range of the forward's P V product, or a
                              length or page id that does not fit (paged cache) */
} fox_status;

enum { FOX_DTYPE_BF16 = 0, FOX_DTYPE_F32 = 1 };

typedef struct fox_params {
  int B;           /* batch size, >= 0 */
  int N;           /* sequence length, >= 0 (any value; no multiple-of-tile requirement) */
  int H;           /* heads, >= 0; q, k and v have the same head count */
  int d;           /* head dimension: 64 or 128 */
  int dtype;       /* FOX_DTYPE_BF16 (tensor cores) or FOX_DTYPE_F32 (forward only) */
  float scale;     /* multiplies q.k only; 0 selects d^-1/2 (module __init__: head_dim ** -0.5) */
  int bias_from_j; /* 0: D_ij = sum_{l=j+1}^{i} log f_l (module code, foxwindow); 1: sum_{l=j}^{i} (module docstring) */
  int non_causal;  /* 0: causal (the module's "decoder" mode, the default); 1: every key, the module's
                      "encoder" mode, where the same outer difference D_ij = c_i - c_j (positive for
                      j > i) biases keys after the query too. bf16 forward and backward only. */
  int tile_skip;   /* 0: visit every causal tile pair (default). 1: skip the (query tile, key tile)
                      pairs whose every weight the decay bound puts below 2^-150 of its row's
                      largest (see fox_tile_span); outputs are bit-identical to tile_skip = 0 for
                      the forward, dK and dV, and equal up to the order of fp32 atomic sums for dQ
                      and dz. Causal bf16 only (FOX_ERR_UNSUPPORTED otherwise). */
  int gate_ready;  /* fox_bwd only (ignored elsewhere). 0: the backward runs its own gate scan (default).
                      1: the workspace already holds the gate terms of this z, written by a fox_fwd
                      (or fox_fwd_xgate, fox_gate_proj, fox_gate_scan) call with the same B, N, H and
                      bias_from_j on the same workspace, and nothing has written the workspace since:
                      the backward skips the scan and reads them. The workspace must then be at least
                      the larger of the fox_fwd and fox_bwd sizes. The backward also leaves the
                      workspace's error word as the forward left it (errors of both calls accumulate
                      until fox_check_error clears them). With a workspace that does not hold them, the
                      results are wrong (nothing faults: every index comes from B, N, H). */
} fox_params;

/*
 * Workspace bytes for these params (0 if params are invalid).
 * fox_fwd_workspace_bytes: the gate terms plus, for bf16, an fp16 copy of V
 *   (B*N*H*d*2 bytes), which fox_fwd writes once and the attention kernel reads.
 * fox_fwd_min_workspace_bytes: the gate terms alone, the least fox_fwd accepts.
 *   With less than fox_fwd_workspace_bytes the attention kernel converts every
 *   V tile it loads on chip instead (same results, bit for bit; slower).
 * fox_bwd_workspace_bytes: everything fox_bwd needs (more than the forward's).
 */
size_t fox_fwd_workspace_bytes(const fox_params* p);
size_t fox_fwd_min_workspace_bytes(const fox_params* p);
size_t fox_bwd_workspace_bytes(const fox_params* p);

/*
 * Forward. Reads q, k, v [B,N,H,d] and gate logits z [B,N,H] (fp32; +inf
 * allowed and means f = 1; -inf and NaN are outside the domain). Writes
 * O [B,N,H,d] (params.dtype; bf16 rounded to nearest even) and
 * LSE [B,N,H] (fp32, natural log, bias included).
 * Steps: gate log-sigmoid + per-head prefix scan into the workspace, V to fp16
 * into the workspace (when it has room, see above), then the fused causal
 * attention kernel. B*H == 0 or N == 0 returns FOX_OK with no work.
 * Workspace: at least fox_fwd_min_workspace_bytes(p), else FOX_ERR_WORKSPACE.
 * Precision (bf16): S = Q K^T in bf16 with fp32 accumulation, the softmax in
 * fp32, and P V in fp16 (P on chip and V converted to fp16, fp32 accumulation),
 * so that the weights carry 11 significant bits instead of bf16's 8. Every bf16
 * V value of magnitude 2^-14 .. 65280 converts exactly; smaller ones round to a
 * multiple of 2^-24; a V value of magnitude 65536 or more sets a device error
 * bit (fox_check_error then returns FOX_ERR_DEVICE).
 */
fox_status fox_fwd(const fox_params* p, const void* q, const void* k, const void* v, const float* z, void* o,
                   float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gate projection ("Forgetting Transformer (FoX) Attention" module source:
 * f_proj = Linear(hidden_size, num_heads, bias=True), f = sigmoid(f_proj(x))):
 *   z[b,t,h] = sum_e x[b,t,e] W_f[h,e] + b_f[h]
 * x: [B,N,hidden] bf16. W_f: [H,hidden] bf16 (the Linear's weight layout).
 * b_f: [H] fp32. z: [B,N,H] fp32. All arrays are device pointers.
 * One kernel computes the 128-token x H blocks of z on the tensor cores
 * (fp32 accumulation) and runs the gate scan of fox_fwd on them in the same
 * pass, so fox_fwd_xgate's gate terms never round-trip through z.
 * Requires dtype bf16, hidden a positive multiple of 8, and H <= 256.
 * Workspace: fox_fwd_workspace_bytes(p) (its gate terms are also written).
 */
fox_status fox_gate_proj(const fox_params* p, int hidden, const void* x, const void* w_f, const float* b_f, float* z,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Forward from the layer input's gate projection instead of z: the fused
 * projection + gate scan above, then the attention as in fox_fwd. Writes
 * O, LSE and, when z is not null, z for the backward (fox_bwd takes z).
 * The same requirements as fox_gate_proj apply; tile_skip is honoured.
 */
fox_status fox_fwd_xgate(const fox_params* p, int hidden, const void* q, const void* k, const void* v, const void* x,
                         const void* w_f, const float* b_f, float* z, void* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Backward (bf16 only). Reads q, k, v, z, the forward's O and LSE, and the
 * upstream gradient dO; writes dq, dk, dv [B,N,H,d] bf16 and dz [B,N,H] fp32.
 * Steps: gate scan (skipped with p->gate_ready), the fp32 dQ accumulator in the
 * workspace cleared (a stream-ordered cudaMemsetAsync), Delta_i = dO_i . O_i,
 * the fused recompute-and-backward attention kernel (dK, dV, dQ accumulator and
 * the row and column sums of dS), the dQ conversion and the reverse gate scan
 * (one pass: a decoupled look-back across 128-token blocks or, with at least
 * one (b, 4-head) sequence per SM, one CTA walking each whole sequence).
 * With non_causal = 1, Delta is not taken from the bf16 O: a pass of its own
 * forms Delta_i = sum_j P_ij dP_ij from S = Q K^T and dP = dO V^T with P
 * recomputed from LSE, in fp32 (the gate gradient is a small difference of
 * large sums of dS there, and the bf16 rounding of O moves it by percents).
 * The extra pass costs about one forward.
 */
fox_status fox_bwd(const fox_params* p, const void* q, const void* k, const void* v, const float* z, const void* o,
                   const float* lse, const void* dO, void* dq, void* dk, void* dv, float* dz, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * The gate step alone: log f_t = log sigmoid(z_t) and its prefix sum along the
 * sequence per (b, h) ("Forgetting Transformer (FoX) Attention" module source,
 * ForgettingAttention.forward: sigmoid of the gate logits, log, cumsum), as the
 * first launches of fox_fwd and fox_bwd compute them. The gate terms are left in
 * the workspace; when c is not NULL the cumulative log gate
 *   c[b,t,h] = sum_{l<=t} log sigmoid(z[b,l,h])   (natural log, fp32, [B,N,H])
 * is written as well. No later call reads the workspace's gate terms (fox_fwd and
 * fox_bwd always recompute them): the call exists to check and time this step on
 * its own, at sizes where the attention itself would not fit. Only B, N, H and
 * bias_from_j are read from p. z is [B,N,H] fp32. Workspace:
 * fox_gate_scan_workspace_bytes(p) (the same as fox_fwd's for the same B, N, H).
 */
size_t fox_gate_scan_workspace_bytes(const fox_params* p);
fox_status fox_gate_scan(const fox_params* p, const float* z, float* c, void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * The gate gradient from the row and column sums of dS, the last step of
 * fox_bwd: with R[b,h,t] = sum_j dS_tj and C[b,h,t] = sum_i dS_it,
 *   d a_t = sum_{s>=t} (R_s - C_s)          (bias_from_j = 0)
 *   d a_t = sum_{s>=t} (R_s - C_s) + C_t    (bias_from_j = 1)
 *   dz[b,t,h] = d a_t * sigmoid(-z[b,t,h])  (d/dz log sigmoid(z) = sigmoid(-z))
 * (chain rule through D_ij = c_i - c_j of the module's forward; the suffix form
 * holds with or without the causal mask). R, C: [B,H,N] fp32, each (b, h) row
 * contiguous; z, dz: [B,N,H] fp32. The sums are fp32 within 128-token blocks and
 * double-float (two fp32 values, about 48 bits) across them. Only B, N, H and
 * bias_from_j are read from p. Workspace (block sums): fox_gate_bwd_workspace_bytes(p).
 */
size_t fox_gate_bwd_workspace_bytes(const fox_params* p);
fox_status fox_gate_bwd(const fox_params* p, const float* z, const float* R, const float* C, float* dz,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Epsilon-effective window of every query row (foxwindow README, "The window is
 * a first-passage time"): with X_t = -log sigmoid(z_t) and L = ln(1/eps),
 *   window[b,i,h] = inf{ n >= 1 : X_i + X_{i-1} + ... + X_{i-n+1} > L },
 * one more than the largest distance n whose decay prod_{t=i-n+1..i} f_t is
 * still >= eps; -1 if the whole prefix (n = i+1) does not pass L. Uses the
 * score form's sum from j+1 (bias_from_j, d, dtype and scale are ignored).
 * z is [B,N,H] fp32, window [B,N,H] int32; 0 < eps < 1. The prefix sums and
 * the comparisons are fp64. Workspace: fox_window_workspace_bytes(p).
 */
size_t fox_window_workspace_bytes(const fox_params* p);
fox_status fox_window(const fox_params* p, const float* z, double eps, int32_t* window, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * Tile spans of the decay-aware tile skip (tile_skip = 1). The bias falls
 * monotonically with distance because every log f_t < 0 (foxwindow README,
 * "The window is a first-passage time"). So for query tile I (rows
 * 128I..128I+127) and an earlier key tile J, in log2 units,
 *   U(I,J) = scale log2e qmax_I (kmax_{<=J} + kmax_I) + (colterm(128I) - colterm(128J+127)) log2e
 * bounds x_ij - max_j' x_ij' over the pair. Here:
 *   - qmax_T, kmax_T are the largest row norms of q, k in tile T;
 *   - kmax_{<=J} is the largest kmax over tiles 0..J;
 *   - colterm(t) = c_t, or c_{t-1} when bias_from_j = 1.
 * Pairs with U < -150 are skipped. Every weight in such a pair is then
 * below 2^-150 of its row's largest, and the kernels' flushing exp2 makes it
 * exactly 0. Outputs, int32 [B*H][nT] with nT = ceil(N/128):
 *   jmin[bh][I]  first key tile that query tile I visits. It is made
 *                non-decreasing in I by a suffix minimum, which only keeps
 *                more pairs.
 *   imax[bh][J]  last query tile that key tile J serves:
 *                the largest I with jmin[bh][I] <= J.
 * q, k: [B,N,H,d] bf16; z: [B,N,H] fp32; causal bf16 params only.
 * Workspace: fox_fwd_workspace_bytes(p). jmin and imax are device pointers,
 * written by stream-ordered copies.
 */
fox_status fox_tile_span(const fox_params* p, const void* q, const void* k, const float* z, int32_t* jmin,
                         int32_t* imax, void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---- Answering token by token: a paged cache, and attention over it ----
 *
 * The cache is a pool of pages of page_size tokens each, in device memory that the caller owns:
 *   k, v  [num_pages, Hkv, page_size, d]  element type dtype
 *   g     [num_pages, H, page_size] fp32  sum of log sigmoid(z) from the page's first token to this one
 *   gbase [num_pages, H, 2] fp32          the sum over every earlier token of the sequence (high, low):
 *                                         c of a token = gbase[0] + gbase[1] + g (natural log)
 * H query heads share Hkv key heads: query head h reads key head h / (H / Hkv). The gate has one
 * logit a query head, as everywhere in this library.
 * Nothing has to be initialised: a page's slots are read only once tokens were appended to them.
 * Precision of c_i - c_j: each of the two g is the nearest fp32 of its sum, so off by 2^-24 |g|, where the sum was
 * formed by one call of at most 8 tokens a sequence, or with g_low (fox_cache_append_low); by 11 times that where one
 * call brought more tokens. A call that goes on in a page that holds tokens adds to the rounded g: without g_low each
 * such call adds one rounding, 2^-24 |g| for the largest |g| of the page, to the difference of all tokens before it and all
 * after. That matters for tokens appended one at a time behind a strong gate in their page: over n of them c_i - c_j
 * may be off by n 2^-24 |g|, 1e-3 for 127 tokens behind z = -132, 0.08 behind z = -1e4 (with g_low by 0.0012).
 */
typedef struct fox_cache {
  int num_pages; /* >= 1 */
  int page_size; /* 16, 32, 64 or 128 */
  int H;         /* query heads, a multiple of Hkv */
  int Hkv;       /* key heads, >= 1 */
  int d;         /* 64 or 128 */
  int dtype;     /* FOX_DTYPE_BF16 or FOX_DTYPE_F32 */
  void* k;       /* 16-byte aligned, as v, g and gbase */
  void* v;
  float* g;
  float* gbase;
} fox_cache;

/*
 * One step's sequences. Each brings its newest tokens: `rows` rows of q, k, v, z in all, the
 * sequences' rows one after the other. All arrays are device memory and read when the work runs, so
 * that a captured step can be replayed on new contents.
 * With a shared prefix, every sequence begins with the same prefix_len tokens, held once in the
 * pages of prefix_table; `table` then names the pages of each sequence's later tokens, the first of
 * which starts a page of its own. The new tokens are never the prefix's (it is appended beforehand,
 * as a sequence without a prefix).
 * Two sequences of one append must not name the same page for their new tokens.
 */
typedef struct fox_batch {
  int B;                       /* sequences, 0 .. 2048 */
  int max_new;                 /* >= the new tokens of any sequence (ignored without cu_new), >= 1 */
  int table_stride;            /* entries of a sequence's row of `table`, >= 1 */
  int prefix_len;              /* tokens of the shared prefix; 0: none */
  const int32_t* cu_new;       /* [B + 1] first row of each sequence, rising from 0; rows behind cu_new[B] are
                                  left as they are. NULL: rows / B rows each (rows a multiple of B) */
  const int32_t* lens;         /* [B] tokens of each sequence, the prefix and the new ones among them.
                                  0: an idle sequence (padding); its rows are not appended, and attend to nothing */
  const int32_t* table;        /* [B, table_stride] page ids */
  const int32_t* prefix_table; /* [ceil(prefix_len / page_size)] page ids, or NULL with prefix_len 0 */
} fox_batch;

/*
 * Workspace of fox_cache_append and fox_decode for these arguments (0 if they are invalid): the
 * error word, and for fox_decode counters and the partial results of keys split among the SMs. It
 * depends on sizes only, never on the contents of lens: some rows * H * d * 4 bytes, more where sequences bring few.
 * fox_cache_append uses its first 256 bytes alone, and takes no more. Its first FOX_CACHE_ZERO_BYTES must be zero
 * before its first call with these two functions (any other use in between, a call of fox_fwd for
 * instance, makes it a new one); they leave the counters zero, and only ever add bits to the error word, the
 * first 4 bytes, which fox_check_error reads and clears: a length, row range, page id or position
 * outside what the arguments allow sets one. The sequence, or the token, is then skipped, or an
 * unknown page read as page 0; its outputs are not meaningful, and no other sequence is touched (rows that two
 * sequences claim, by a cu_new that falls, are neither's).
 * Calls that may run at the same time (other streams, captured graphs) need workspaces of their own.
 * After a call whose device wait gave up (FOX_ERR_TIMEOUT) the header has to be made zero again.
 */
#define FOX_CACHE_ZERO_BYTES 16384
size_t fox_cache_workspace_bytes(const fox_cache* c, const fox_batch* s, int rows);

/* Rotation of the first `dim` channels of k (and q) by the angles of the token's position in its sequence. */
typedef struct fox_rotary {
  const float* cos;  /* [max_pos, dim / 2] fp32, 16-byte aligned, as sin */
  const float* sin;
  int max_pos;       /* positions that the tables hold */
  int dim;           /* 0 (none), or a multiple of 16 up to d */
  int pairs;         /* 0: channel i with i + dim / 2;  1: channel 2i with 2i + 1 */
  const void* q;     /* [rows, H, d] to rotate with the same angles, or NULL */
  int64_t q_stride;  /* elements from one row of q to the next */
  void* q_out;       /* [rows, H, d] contiguous, apart from q, k, v, z, cos and sin */
} fox_rotary;

/*
 * Appends the new tokens: K (rotated when rot is given; products and sums in fp32, rounded once), V and
 * the gates' running sums go to the pages of positions lens[b] - n_b .. lens[b] - 1. Calling it again
 * with the same arguments writes the same values. k, v: rows of [Hkv, d], row strides in elements
 * (multiples of 16 bytes, 16-byte aligned); z: rows of [H] fp32, any stride >= H. rot may be NULL.
 * Every value of the range that fox_fwd takes for z is allowed.
 */
fox_status fox_cache_append(const fox_cache* c, const fox_batch* s, int rows, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const float* z, int64_t z_stride, const fox_rotary* rot,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * fox_cache_append with the gates' running sums in two parts: g_low [num_pages, H, page_size] fp32 holds what the
 * rounding of g leaves of each sum, so that tokens appended one at a time add to the sum and not to its rounded value.
 * Needs no initialisation, and every append to the cache should be given it: a slot whose g_low is not its g's (more
 * than half a step of g) counts as 0 there. fox_decode does not read it. NULL: as fox_cache_append.
 */
fox_status fox_cache_append_low(const fox_cache* c, const fox_batch* s, int rows, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, const float* z, int64_t z_stride,
                                const fox_rotary* rot, float* g_low, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Attention of the new tokens over the cache (their own K, V and gates appended before): row i of
 * sequence b at position pos attends to the sequence's keys 0 .. pos with the scores of fox_fwd,
 *   x_ij = scale q_i . k_j + c_i - c_j   (c_{j-1} under bias_from_j = 1).
 * q: rows of [H, d], q_stride elements apart (multiples of 16 bytes; 16-byte aligned).
 * o: [rows, H, d] of the cache's type; lse: [rows, H] fp32, natural log; q, o and lse apart from each other. Rows of idle
 * sequences get O = 0 and LSE = -inf. scale 0 selects d^-1/2.
 * A shared prefix of a bf16 cache is, where that saves more than it costs (B * prefix_len * Hkv * d * 4 bytes
 * above 72 MB, counted once for every 16 rows that a sequence brings a key head), multiplied once with the rows of
 * all sequences: its weights and V then pass through fp16 as in fox_fwd, so that |v| >= 65536 in its pages sets the
 * error word, and V below 2^-14 is held in steps of 2^-24. Otherwise, and in fp32, every sequence walks it, with V as
 * it is.
 * Nothing behind a row's position is used for it, whatever K, V and the gates hold there (new tokens further on, slots
 * behind the sequence's end). The same arguments and
 * contents give the same bits; how a row's sums are ordered follows from the lengths of the whole batch.
 */
fox_status fox_decode(const fox_cache* c, const fox_batch* s, int rows, const void* q, int64_t q_stride, float scale,
                      int bias_from_j, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Forward without a caller-provided workspace, for callers that cannot
 * allocate device memory where they run this code (a plugin in a host
 * application that owns all device memory, a latency-bound loop that cannot
 * take an allocation's implicit synchronisation). The pages have no
 * counterpart: this is a library convenience, not part of the method.
 * Same arguments and results as fox_fwd, minus the workspace: the scratch
 * for the gate terms is a fixed array of fox_noalloc_scratch_bytes() (16 MiB)
 * compiled into the library, which every GPU that loads the library holds
 * until the process exits. Problems whose fox_fwd_min_workspace_bytes exceeds
 * it return FOX_ERR_WORKSPACE without touching the GPU; the fp16 copy of V is
 * used when fox_fwd_workspace_bytes fits too. Allocates nothing
 * (no cudaMalloc, cudaFree or allocating library call). The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) with that
 * device current; make that first call before any stream capture. All calls
 * share the one array and the last call's contents stay in it: each call
 * rewrites it completely (the error word included), and calls whose work
 * overlaps on the GPU race on it. The device address is cached per device for
 * the life of the process: a cudaDeviceReset() on a device destroys the array
 * with the context, and fox_fwd_noalloc must not be called on that device
 * again in the same process.
 */
fox_status fox_fwd_noalloc(const fox_params* p, const void* q, const void* k, const void* v, const float* z,
                           void* o, float* lse, void* stream);
size_t fox_noalloc_scratch_bytes(void);
/*
 * fox_check_error for fox_fwd_noalloc: synchronises `stream`, reads and clears
 * the error word of the fixed scratch array of the current device (the one the
 * last fox_fwd_noalloc on that device used), with fox_check_error's results.
 * Allocates nothing.
 */
fox_status fox_noalloc_check_error(void* stream);

/*
 * Synchronises `stream`, reads and clears the device error word of
 * `workspace` (the one passed to the last fox_fwd / fox_bwd on it).
 * Returns FOX_OK, FOX_ERR_TIMEOUT or FOX_ERR_DEVICE, or FOX_ERR_CUDA if the
 * stream itself reports an error.
 */
fox_status fox_check_error(void* workspace, void* stream);

/*
 * Self-test of the device-side error path (the pages have no counterpart: this
 * checks the library's own failure reporting). One kernel on `stream` waits on
 * an mbarrier that nothing arrives at, with the attention kernels' bounded-wait
 * code and a limit of limit_us microseconds (1 .. 100000), while a second wait
 * of 16x that limit must be released by the first one's abort flag. Afterwards
 * the workspace's error word holds the timeout bit of the first wait only, so
 * fox_check_error(workspace, stream) returns FOX_ERR_TIMEOUT and clears it; the
 * next two 32-bit words of the header hold what each wait returned (0 = gave
 * up). Nothing faults; the context stays usable. workspace: >= 256 bytes,
 * 256-byte aligned (any fox_* workspace qualifies). Returns FOX_ERR_INVALID_ARG
 * for a limit out of range.
 */
fox_status fox_selftest_wait_timeout(unsigned limit_us, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Kernel-level timing, for benchmarks. Between fox_trace_begin() and
 * fox_trace_end(), every kernel launch this library enqueues (from any host
 * thread) is bracketed by two CUDA events recorded on its stream; events are
 * created on first use and reused. fox_trace_end() stops recording, waits for
 * the recorded events, writes up to max_records {kernel name, milliseconds}
 * in launch order into `out` (may be NULL), and returns the number of
 * launches recorded, or -1 if a CUDA event call failed. Names are static strings.
 */
typedef struct fox_trace_record {
  const char* kernel;
  float ms;
} fox_trace_record;
fox_status fox_trace_begin(void);
int fox_trace_end(fox_trace_record* out, int max_records);

/* Static string naming a status. */
const char* fox_status_string(fox_status s);

/* Library ABI version (major * 100 + minor). */
int fox_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FOX_H_ */
