/*
 * hq.h — C ABI of libhq.so: hybrid-precision attention on NVIDIA B200 (sm_100a).
 *
 * What the library computes is the hot path of HyQuant ("HyQuant:
 * Hybrid-Precision Quantization for LLM Attention"):
 *
 *   - keys are split three ways: vertical-line (VL) positions and a recent
 *     window stay FP16, every other position is stored 4-bit (K4V4)
 *     (agihunt.info digest of the paper, method paragraph; repository README,
 *     Overview);
 *   - decode attention runs over that hybrid cache with dequantisation fused
 *     into the online-softmax KV scan, so no FP16 copy of the cache is ever
 *     materialised (digest, prefill/decode paragraph; README Overview item 3);
 *   - the VL set is the top-rho (default 5 %) of the non-window prefix by
 *     accumulated column attention mass, re-identified every 64 tokens from at
 *     most 64 buffered FP16 queries (digest, method paragraph; README Overview
 *     item 1 and "Overhead");
 *   - new tokens are staged and merged into the hybrid layout later (digest,
 *     prefill/decode paragraph);
 *   - prefill is one FlashAttention-style causal pass whose quantised tiles run
 *     on low-precision tensor cores while VL and window tiles stay FP16, under a
 *     single online softmax (digest, prefill/decode paragraph; README Overview
 *     item 2).
 *
 * K4V4 layout (the pages name the format but print no layout; this library
 * fixes it): per token and head, D = 128 values in 4 groups of 32;
 * scale = fp16(fp32(max - min) / 15), zero = min (fp16);
 * q = clamp(rint_even((x - zero) / scale), 0, 15) with float32 RN arithmetic
 * (q = 0 when scale == 0); two nibbles per byte, low nibble first; the
 * dequantised value is zero + q * scale.
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers, 16-byte aligned, owned by the
 *     caller; the library allocates nothing.  Its only state is the last error
 *     message of each host thread (hq_last_error) and, for
 *     hq_decode_attn_noalloc alone, a fixed device scratch array of its own.
 *   - fp16 tensors are passed as uint16_t* (IEEE binary16 bit patterns).
 *   - Calls are asynchronous on `stream`.  Arguments are validated on the host
 *     before anything is launched; on a non-HQ_OK status nothing was launched.
 *   - Conditions that depend on device-resident lengths (a full staging area,
 *     an exhausted capacity) cannot be seen by the host: the kernels skip their
 *     work and OR a HQ_DEVERR_* bit into state[b][HQ_STATE_ERR] of the sequence
 *     concerned; read it after synchronising.  No kernel traps or spins
 *     without a bound.
 *   - Sequences are independent: each batch row b has its own lengths (a row
 *     of the state array), so one call serves a batch of sequences of
 *     different lengths.  The K4V4 store may be paged (page_table), so that the
 *     pages of a sequence need not be contiguous.  A single sequence is
 *     addressed by a descriptor whose pointers are offset to its row (B = 1),
 *     e.g. to install its prefix while the others keep decoding.
 */
#ifndef HQ_H
#define HQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HQ_ABI_VERSION 4
#define HQ_HEAD_DIM 128       /* D: the only head size built */
#define HQ_GROUP 32           /* K4V4 group length along D */
#define HQ_STAGE 64           /* staged tokens before a merge = reselection period */
#define HQ_QBUF 64            /* buffered queries kept for the column-mass estimate */
#define HQ_MAX_GQA 8          /* query heads per kv head supported by the decode kernel */
/* K4V4 store page: 64 positions of one (batch, kv head), one contiguous block */
#define HQ_PAGE_POSITIONS 64
#define HQ_PAGE_BYTES 10304
#define HQ_PAGE_KCODES 0        /* [64][D/2] K codes, row r = position 64 j + r */
#define HQ_PAGE_VCODES 4096     /* [64][D/2] V codes */
#define HQ_PAGE_KSZ 8192        /* [64][D/32] uint32 K (scale bits | zero bits << 16) */
#define HQ_PAGE_VSZ 9216        /* [64][D/32] uint32 V (scale | zero << 16) */
#define HQ_PAGE_VLMASK 10240    /* 2 uint32: bit r of word r/32 <=> position 64 j + r is a vertical line */
#define HQ_PAGE_VLBASE 10248    /* int32: VL-store row of the page's first vertical line (valid when the bitmap is non-zero) */
/* Other code widths (k_bits, v_bits in {2, 4, 8}; README Mode reference: K8V8,
 * K4V2, K2V4 beside K4V4).  Same scale/zero rule with 2^bits - 1 levels and
 * 8 / bits codes per byte, lowest bits first.  A page of 64 positions is cut
 * into sub-pages of HQ_PAGE_SUBPOS(kb, vb) positions (64, or 32 when kb + vb >
 * 8), each laid out [K codes][V codes][K (scale|zero) words][V words] with
 * 16 * bits bytes of codes per position; the bitmap and the first-VL row follow
 * the sub-pages.  For kb = vb = 4 this is exactly the HQ_PAGE_* layout above. */
#define HQ_PAGE_SUBPOS(kb, vb) (((kb) + (vb)) > 8 ? 32 : 64)
#define HQ_PAGE_SUBBYTES(kb, vb) (HQ_PAGE_SUBPOS(kb, vb) * (16 * (kb) + 16 * (vb) + 32))
#define HQ_PAGE_MASK_OFF(kb, vb) ((64 / HQ_PAGE_SUBPOS(kb, vb)) * HQ_PAGE_SUBBYTES(kb, vb))
#define HQ_PAGE_BYTES_KV(kb, vb) (((HQ_PAGE_MASK_OFF(kb, vb) + 16) + 63) / 64 * 64)
/* FP16 ring length for a window W: W + HQ_STAGE rounded up to a multiple of 16 */
#define HQ_RING_LEN(W) ((((W) + HQ_STAGE) + 15) / 16 * 16)

typedef struct CUstream_st* hq_stream_t;  /* same type as cudaStream_t */

#if defined(__GNUC__)
#define HQ_API __attribute__((visibility("default")))
#else
#define HQ_API
#endif

typedef enum hq_status {
  HQ_OK = 0,
  HQ_ERR_INVALID = 1,      /* null/misaligned pointer, bad shape or argument */
  HQ_ERR_UNSUPPORTED = 2,  /* valid request this build does not implement (e.g. D != 128) */
  HQ_ERR_WORKSPACE = 3,    /* workspace missing or smaller than hq_*_workspace_bytes() */
  HQ_ERR_CAPACITY = 4,     /* a host-visible size exceeds the cache's capacity */
  HQ_ERR_CUDA = 5          /* a CUDA runtime call or launch failed */
} hq_status;

/* device-side error bits, OR-ed into state[b][HQ_STATE_ERR] */
#define HQ_DEVERR_STAGING_FULL 0x1u  /* decode with HQ_STAGE tokens staged: select + merge first */
#define HQ_DEVERR_CAPACITY 0x2u      /* T would exceed cap */
#define HQ_DEVERR_VL_CAPACITY 0x4u   /* k = ceil(rho * n) exceeds vl_cap (clamped) */
#define HQ_DEVERR_TIMEOUT 0x8u       /* a bounded wait gave up (never expected) */
#define HQ_DEVERR_PAGE 0x10u         /* a page-table entry outside [0, n_pages): pool page 0 was read
                                        instead (the outputs of that sequence are unspecified) and
                                        nothing was written through the entry */

/* words of one sequence's row of the device-resident state (int32[B][HQ_STATE_WORDS]) */
enum {
  HQ_STATE_T = 0,         /* current length: positions 0 .. T-1 are cached */
  HQ_STATE_NPACKED = 1,   /* positions 0 .. n_packed-1 have a K4V4 record */
  HQ_STATE_NVL = 2,       /* rows in the VL store */
  HQ_STATE_NQ = 3,        /* valid buffered queries (<= HQ_QBUF) */
  HQ_STATE_KSEL = 4,      /* entries written to vl_sel by the last hq_select_vlines */
  HQ_STATE_ERR = 5,       /* HQ_DEVERR_* bits */
  HQ_STATE_WORDS = 8
};

/*
 * The hybrid KV cache of one attention layer.  Every array is caller-owned
 * device memory laid out as stated ([..] = row-major shape, innermost last).
 * R = HQ_RING_LEN(W) is the FP16 ring length (W + HQ_STAGE rounded up to 16).
 *
 *   pages     uint8  [B, Hkv, cap/64, PB]  (page_table == NULL) or a page pool uint8 [n_pages, PB]
 *             (page_table != NULL), PB = HQ_PAGE_BYTES_KV(k_bits, v_bits): the packed store, one page per
 *             64 positions (layout HQ_PAGE_* for K4V4, sub-pages for the other widths): codes
 *             of both K and V, their per-group (scale, zero) words and the VL bitmap of the
 *             page's positions, so that one contiguous copy brings a whole (sub-)page on chip,
 *             then the VL-store row of the page's first vertical line (at
 *             HQ_PAGE_MASK_OFF(k_bits, v_bits) + 8); the bytes after it up to PB are padding
 *   kf, vf    fp16   [B, Hkv, vl_cap, D]  VL store rows, in vl_pos order
 *   vl_pos    int32  [B, Hkv, vl_cap]     VL positions, ascending (first n_vl valid)
 *   kr, vr    fp16   [B, Hkv, R, D]       recent window + staging; position p at slot p % R
 *   qbuf      fp16   [B, Hq, HQ_QBUF, D]  buffered decode queries; position p at slot p % HQ_QBUF
 *   vl_sel    int32  [B, Hkv, vl_cap]     output of hq_select_vlines, input of hq_pack_merge
 *   state     int32  [B, HQ_STATE_WORDS]  device-resident lengths of each sequence (HQ_STATE_*)
 *   page_table int32 [B, Hkv, cap/64]    optional (NULL: pages is the dense [B, Hkv, cap/64, ..]
 *             array): entry (b, h, j) is the pool page holding positions 64 j .. 64 j + 63
 *             of sequence b, kv head h; 4-byte aligned; entries of pages no position
 *             reaches are not read.  Pages of different (b, h) must be distinct.
 *   score_acc float [B, Hkv, cap]        optional running column-mass scores (NULL: each
 *             reselection ranks its own column mass).  When set, the prefix selection
 *             (init mode) stores its column mass there (zero past the scored prefix) and
 *             every decode-mode reselection adds its column mass to it and ranks the sums
 *             (README Overview item 1, "running column-mass score").
 *   qlse      float [B, Hq, HQ_QBUF]     optional (NULL: not kept): each decode step stores the
 *             log-sum-exp (base 2, over its T + 1 logits q.k / sqrt(D)) of its query next to
 *             the query itself (slot T % HQ_QBUF).  A decode-mode reselection whose buffered
 *             queries all came after the last merge (so they saw the keys exactly as the
 *             reselection does) takes its row normalisers from here instead of a first
 *             pass over the keys.  Decode steps with sm_scale != 1/sqrt(D) store NaN.
 *
 * Limits checked by hq_cache_validate(): D == 128; Hq % Hkv == 0 and
 * Hq / Hkv <= HQ_MAX_GQA; W >= 0; 0 <= rho_bp <= 10000; cap a positive
 * multiple of 128; vl_cap a positive multiple of 16; with a page table,
 * n_pages >= 1; (k_bits, v_bits) one of (4, 4), (8, 8), (4, 2), (2, 4).
 * Pages are HQ_PAGE_BYTES_KV(k_bits, v_bits) bytes.
 * Fields W and rho_bp fix the method's window and VL ratio (basis points:
 * 500 = 5 %).  The fp16 positions in [n_packed, T) live in the ring, VL rows
 * in kf/vf, every other position < n_packed is read from its K4V4 record.
 */
typedef struct hq_cache {
  int32_t B, Hq, Hkv, D;
  int32_t W, rho_bp, cap, vl_cap;
  uint8_t* pages;
  uint16_t* kf;
  uint16_t* vf;
  int32_t* vl_pos;
  uint16_t* kr;
  uint16_t* vr;
  uint16_t* qbuf;
  int32_t* vl_sel;
  int32_t* state;
  int32_t* page_table;
  float* score_acc;
  float* qlse;
  int32_t n_pages;
  int32_t k_bits;     /* code bits of packed keys: 4 (0 means 4), 8 or 2 */
  int32_t v_bits;     /* code bits of packed values: 4 (0 means 4), 8 or 2 */
  int32_t reserved;   /* 0 */
} hq_cache;

/* Operation codes for hq_workspace_bytes. */
enum { HQ_OP_SELECT = 0, HQ_OP_MERGE = 1, HQ_OP_DECODE = 2 };

HQ_API int32_t hq_abi_version(void);
HQ_API const char* hq_status_str(hq_status s);

/* After a call returned HQ_ERR_CUDA: which step failed and the CUDA error name
 * (e.g. "prefill launch: cudaErrorLaunchOutOfResources").  Per host thread;
 * the string stays valid until the next failing call on that thread. */
HQ_API const char* hq_last_error(void);

/* Host-side check of a cache descriptor (shapes, limits, 16-byte alignment of
 * every pointer).  Returns HQ_OK or HQ_ERR_INVALID / HQ_ERR_UNSUPPORTED. */
HQ_API hq_status hq_cache_validate(const hq_cache* c);

/* Bytes of device workspace an operation needs for this cache; `L` is the
 * prefix length for an init-mode select/merge (ignored otherwise).
 * HQ_OP_DECODE and HQ_OP_MERGE workspaces start with completion counters:
 * zero-fill the workspace once before its first use; the kernels return the
 * counters to zero at the end of every call.  A workspace must not be shared
 * by calls that can run at the same time. */
HQ_API size_t hq_workspace_bytes(const hq_cache* c, int32_t op, int32_t L);

/*
 * Reset every sequence of the descriptor to empty: its state row to 0, the
 * VL bitmap of each of its pages (through the page table, if any) cleared and
 * its running scores (score_acc, if any) zeroed.
 */
HQ_API hq_status hq_cache_reset(const hq_cache* c, hq_stream_t stream);

/*
 * Vertical-line selection (digest, method paragraph; README Overview item 1).
 * For every (b, kv head): column mass
 *     score_j = sum over the group's query heads h and buffered queries i of
 *               softmax_{j' <= p_i}(q_{h,i} . k_{j'} * sm_scale)[j],
 * for j in the non-window prefix [0, n), n = T - W, sm_scale = 1/sqrt(D);
 * then the k = ceil(n * rho_bp / 10000) largest scores (ties -> lower
 * position) are written to c->vl_sel in ascending position order and k to
 * state[b][HQ_STATE_KSEL]; every sequence b uses its own T, n and k.
 *
 * Init mode (k_dense != NULL): keys are the dense FP16 prefix
 *   k_dense [B, Hkv, L, D], T = L; queries q_ext [B, Hq, nq, D] sit at
 *   positions L-nq .. L-1 (1 <= nq <= HQ_QBUF, nq <= L).  The cache's state
 *   is not read.
 * Decode mode (k_dense == NULL, q_ext == NULL): keys are the cache in its
 *   current representation (VL rows FP16, other packed positions
 *   dequantised, ring FP16), T and the buffered queries come from state/qbuf.
 * scores_out (optional, may be NULL): float [B, Hkv, cap] receives the scores
 *   (entries >= n are unspecified).
 * Errors: HQ_ERR_INVALID for bad pointers/shapes; k > vl_cap is clamped and
 *   flagged with HQ_DEVERR_VL_CAPACITY.
 */
HQ_API hq_status hq_select_vlines(const hq_cache* c, const uint16_t* k_dense, int32_t L,
                           const uint16_t* q_ext, int32_t nq, float* scores_out,
                           void* ws, size_t ws_bytes, hq_stream_t stream);

/*
 * Staging -> hybrid merge (digest, prefill/decode paragraph).
 * Init mode (k_dense, v_dense != NULL, both [B, Hkv, L, D] FP16): install a
 *   prefix of L tokens: positions [0, L-W) get their K4V4 records, the last
 *   min(W, L) positions go to the ring, the VL store is filled from c->vl_sel
 *   (state[b][HQ_STATE_KSEL] entries, FP16 rows taken from the dense prefix);
 *   every row b of state becomes T = L, n_packed = max(L-W, 0), n_q = 0.
 *   Requires L <= cap.  Sequences of different prefix lengths are installed
 *   one at a time through single-sequence descriptors.
 * Merge mode (both NULL): positions [n_packed, T-W) leave the window and get
 *   their K4V4 records; the VL store is rebuilt from c->vl_sel: a row keeps the
 *   position's current FP16 value when it has one (old VL row or ring),
 *   otherwise it is the dequantised record rounded once to FP16; n_packed
 *   becomes max(n_packed, T-W).  Records are never rewritten.  Each sequence
 *   uses its own lengths.
 */
HQ_API hq_status hq_pack_merge(const hq_cache* c, const uint16_t* k_dense, const uint16_t* v_dense,
                        int32_t L, void* ws, size_t ws_bytes, hq_stream_t stream);

/*
 * One decode step (digest, prefill/decode paragraph; README Overview item 3):
 * append k_new, v_new [B, Hkv, D] at position T (ring) and q [B, Hq, D] to
 * the query buffer, then
 *     out[b, h] = softmax(q[b,h] . K^T * sm_scale) V
 * over all T+1 positions, each key/value in its stored representation
 * (dequantisation fused into the scan; split-K over the sequence with a
 * log-sum-exp merge).  out: fp16 [B, Hq, D].  Increments T.  Every sequence
 * b attends over its own T_b + 1 positions.
 * If HQ_STAGE tokens of sequence b are already staged (T - n_packed == W +
 * HQ_STAGE) or T == cap, nothing of that sequence is written (its out rows
 * included) and HQ_DEVERR_STAGING_FULL / _CAPACITY is set in its state row;
 * the other sequences proceed.  B * Hkv <= 2048 (else HQ_ERR_UNSUPPORTED).
 * After a HQ_DEVERR_TIMEOUT the workspace's counters may not be zero: zero
 * the workspace again before the next call.
 */
HQ_API hq_status hq_decode_attn(const hq_cache* c, const uint16_t* q, const uint16_t* k_new,
                         const uint16_t* v_new, uint16_t* out, float sm_scale,
                         void* ws, size_t ws_bytes, hq_stream_t stream);

/*
 * Hybrid causal prefill (digest, prefill/decode paragraph; README Overview
 * item 2, modes "vquant_vert" / "hybrid_full"): for query i and key j <= i,
 *   j is a window key if i - W < j <= i, else a VL key if j is in vl_pos[b, kvh],
 *   else a quantised key;
 * window and VL keys use FP16 Q, K, V; quantised keys use, by qk_format,
 *   HQ_PREFILL_E4M3:    FP8 e4m3 Q, K, V with one float32 scale per (b, head,
 *                       128 positions) (scale = amax / 448, values stored as
 *                       e4m3_RN_sat(x / scale));
 *   HQ_PREFILL_INT8_QK: INT8 Q, K with one float32 scale per (b, head, 128
 *                       positions) (scale = amax / 127, codes
 *                       clamp(rint_even(x / scale), -127, 127)) and FP16 V
 *                       (README Overview item 2, the INT8-QK / FP16-PV kernels);
 * one softmax covers all three classes.
 *   q [B, Hq, L, D], k, v [B, Hkv, L, D], out [B, Hq, L, D]: fp16
 *   vl_pos int32 [B, Hkv, vl_stride], first n_vl entries ascending, < L
 *     (0 <= n_vl <= min(vl_stride, L))
 * Workspace: at least hq_prefill_workspace_bytes(B, Hq, Hkv, L, D, vl_stride)
 * bytes, 16-byte aligned; one call's workspace must not be shared with a call
 * that can run at the same time.  It holds, in this order (each region starting
 * on a 1024-byte boundary, Lp = L rounded up to a multiple of 128):
 *   bytes [0, 4)  uint32 error word, cleared by the call: non-zero when a
 *                 bounded wait of the kernel gave up (never expected; the
 *                 output is then incomplete); read it after synchronising;
 *   e4m3 (or INT8) codes of Q [B, Hq, Lp, D], e4m3 (or INT8) codes of K
 *   [B, Hkv, Lp, D], fp16 values fp16(fp32(e4m3(V / scale)) * scale) of V
 *   [B, Hkv, Lp, D] (e4m3 format only), then the per-block scales and gathered
 *   VL rows (internal).
 * Rows past L of the three coded tensors are zero.
 */
HQ_API size_t hq_prefill_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t L, int32_t D, int32_t vl_stride);
enum { HQ_PREFILL_E4M3 = 0, HQ_PREFILL_INT8_QK = 1 };
HQ_API hq_status hq_prefill_attn(int32_t B, int32_t Hq, int32_t Hkv, int32_t L, int32_t D,
                          const uint16_t* q, const uint16_t* k, const uint16_t* v,
                          const int32_t* vl_pos, int32_t n_vl, int32_t vl_stride, int32_t W,
                          int32_t qk_format, float sm_scale, uint16_t* out, void* ws, size_t ws_bytes,
                          hq_stream_t stream);

/*
 * Allocation-free decode step.  The paper has no counterpart: this is a
 * deployment variant of hq_decode_attn for callers that may not allocate
 * device memory at all, such as a plugin inside a serving engine that owns all
 * device memory, or a latency-critical loop where cudaMalloc / cudaFree would
 * synchronise the device.  Arguments and result are those of hq_decode_attn,
 * minus the workspace: the library uses a fixed scratch array of
 * HQ_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds until the
 * process exits.
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make that first call before any stream capture.
 *     After the device is reset (cudaDeviceReset, or its primary context
 *     released and created again) the next call sees a new context and looks
 *     the address up again: make that call before any capture as well.
 *   - All calls on a device share the array and it keeps the last call's
 *     contents; each call clears what must start at zero itself.  Calls whose
 *     executions can overlap on the GPU (unordered streams) race on the array:
 *     order them on one stream.
 *   - Returns HQ_ERR_WORKSPACE when this cache's decode workspace
 *     (hq_workspace_bytes(c, HQ_OP_DECODE, 0)) exceeds HQ_NOALLOC_SCRATCH_BYTES;
 *     nothing is launched then.  It never calls cudaMalloc or cudaFree.
 */
#define HQ_NOALLOC_SCRATCH_BYTES (4u << 20)
HQ_API hq_status hq_decode_attn_noalloc(const hq_cache* c, const uint16_t* q, const uint16_t* k_new,
                                        const uint16_t* v_new, uint16_t* out, float sm_scale, hq_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions, and a plain 8-bit cache with its attention.  They have no
 * counterpart in the method: they are what a serving layer needs around it
 * (rotated queries and keys go into every attention call of this library) and
 * the uniform low-precision cache that the hybrid one is weighed against.
 * ------------------------------------------------------------------------ */

/* Element types of the calls below (f16: IEEE binary16, bf16: bfloat16). */
enum { HQ_F16 = 0, HQ_BF16 = 1, HQ_F32 = 2 };

/* Which elements of a head form a pair: (i, i + rot/2), or (2i, 2i + 1). */
enum { HQ_ROPE_HALF = 0, HQ_ROPE_INTERLEAVED = 1 };

/* Frequencies of the rot/2 pairs, w_i radians per position.  With
 * w_i = base^(-2i/rot), f = factor and t_i = orig_len * w_i / 2 pi (the turns
 * pair i makes in the original context):
 *   PLAIN   w_i
 *   LINEAR  w_i / f                               (position interpolation)
 *   NTK     the base is base * f^(rot/(rot-2))    (rot > 2)
 *   YARN    (1 - r_i) w_i + r_i w_i / f, r_i = clamp((i - a)/max(c - a, 0.001), 0, 1),
 *           a = max(floor(d(high)), 0), c = min(ceil(d(low)), rot - 1),
 *           d(x) = rot ln(orig_len / (2 pi x)) / (2 ln base); amp = 1 + 0.1 ln f for f > 1
 *           (Peng et al. 2023, "YaRN"; defaults high = 32, low = 1)
 *   BANDS   (1 - r_i) w_i / f + r_i w_i, r_i = clamp((t_i - low)/(high - low), 0, 1)
 *           (defaults high = 4, low = 1)
 */
enum { HQ_ROPE_PLAIN = 0, HQ_ROPE_LINEAR = 1, HQ_ROPE_NTK = 2, HQ_ROPE_YARN = 3, HQ_ROPE_BANDS = 4 };

/*
 * Host-only: the table that hq_rope reads, written to HOST memory; the caller
 * copies it to the device once.  freqs[i] = the fraction of a turn that pair i
 * makes per position, as a 64-bit fixed-point fraction (unit 2^-64), so that
 * position * freqs[i] modulo 2^64 is the angle modulo one turn, exact for any
 * position.  *amp receives the factor of the rotated values (1 except YARN).
 * low, high: 0 = the kind's default.  Requires rot even, 2 <= rot <= 65536,
 * base > 1, factor >= 1, orig_len > 0 for YARN and BANDS, 0 < low < high there.
 */
HQ_API hq_status hq_rope_freqs(int32_t rot, double base, int32_t kind, double factor, double orig_len, double low,
                               double high, uint64_t* freqs, float* amp);

#define HQ_ROPE_MAX_DIM 512

/* One tensor of a hq_rope call: x, y [B, T, H, D] with strides in elements, D contiguous. */
typedef struct hq_rope_tensor {
  const void* x;
  void* y;
  int64_t x_batch, x_tok, x_head;
  int64_t y_batch, y_tok, y_head;
  int32_t H;
  int32_t reserved; /* 0 */
} hq_rope_tensor;

/*
 * Rotary positions of q and (optionally, k != NULL) k in one launch: for each
 * pair (u, v) of the first `rot` elements of a head,
 *     (u, v) -> amp * (u cos a - v sin a, v cos a + u sin a),  a = w_i * pos[b, t],
 * and elements rot .. D-1 are copied.  grad != 0 applies the transposed
 * rotation instead (a -> -a): the gradient of x from that of y.
 *   dtype HQ_F16, HQ_BF16 or HQ_F32 (the arithmetic is float32)
 *   pos   int32 [B, T] contiguous, any sign; freqs uint64 [rot/2] on the device
 * y may equal x with the same strides (in place); otherwise they must not
 * overlap.  D <= HQ_ROPE_MAX_DIM, rot even, 0 < rot <= D.  B, T or H of 0: nothing
 * is done.  Any element-aligned pointers and strides are accepted; 16-byte
 * alignment of rows, D % 8 == 0 and rot % 16 == 0 (4 and 8 for f32) take the
 * 16-byte path.
 */
HQ_API hq_status hq_rope(int32_t dtype, int32_t B, int32_t T, int32_t D, int32_t rot, int32_t layout, int32_t grad,
                         const hq_rope_tensor* q, const hq_rope_tensor* k, const int32_t* pos, const uint64_t* freqs,
                         float amp, hq_stream_t stream);

/* 8-bit block cache: code formats.  Over the 64 x D values of a block (64
 * positions of one sequence and kv head; K and V apart), in float32:
 *   E4M3  s = amax / 448, code = e4m3_RN_sat(x / s)
 *   INT8  s = amax / 127, code = clamp(rint_even(x / s), -127, 127)
 * s = 1 when amax is 0; a block holding an infinity or NaN gets s = NaN (and
 * codes 0): what reads it sees NaN. */
enum { HQ_KV8_E4M3 = 0, HQ_KV8_INT8 = 1 };

/* Page of 64 positions of one (sequence, kv head).  Element (r, d) of K stands
 * at byte HQ_KV8_K_INDEX(r, d), of V at HQ_KV8_V + HQ_KV8_V_INDEX(r, d): the
 * orders in which the matrix instructions of hq_kv8_attn take them, 16 bytes a
 * thread. */
#define HQ_KV8_PAGE_BYTES 16448
#define HQ_KV8_V 8192
#define HQ_KV8_KSCALE 16384 /* float32 */
#define HQ_KV8_VSCALE 16388 /* float32; the bytes from 16392 on are padding */
#define HQ_KV8_MAX_BATCH 1024
#define HQ_KV8_MAX_HEADS 1024
#define HQ_KV8_TAIL 128     /* positions of the 16-bit tail: the two newest blocks */
#define HQ_KV8_K_INDEX(r, d) (((((r) / 8) * 2 + (d) / 64) * 8 + (r) % 8) * 64 + (d) % 64)
#define HQ_KV8_V_INDEX(r, d)                                                                                     \
  (((r) / 16) * 2048 + ((d) / 32) * 512 + (((d) % 8) * 4 + (r) % 8 / 2) * 16 + ((d) / 16 % 2) * 8 + ((d) / 8 % 2) * 4 + \
   ((r) / 8 % 2) * 2 + (r) % 2)

/*
 * The 8-bit block cache of one attention layer (caller-owned device memory).
 * Lengths are not part of it: every call takes them, since all layers of a
 * model share them.
 *   pages      uint8 [B, Hkv, cap/64, HQ_KV8_PAGE_BYTES] (page_table == NULL) or
 *              a pool [n_pages, HQ_KV8_PAGE_BYTES], 16-byte aligned
 *   page_table int32 [B, Hkv, cap/64] or NULL: pool page of positions 64 j .. 64 j + 63;
 *              entries that no position reaches are not read.  Pages that an append
 *              completes must belong to one (b, h) only; full pages may be shared.
 *   tail_k, tail_v fp16 [B, Hkv, 2, 64 * D]: position p of the two newest blocks, in
 *              half (p / 64) % 2 in the page's element order; zero-filled before first use
 *   tail_scale float [B, Hkv, 2, 128]: (K, V) scale of the tail's row of position p at p % 128.
 *              A row's value is fp16 * scale: scale is 1 for fp16 rows; for bf16 rows the
 *              power of two that brings the row's largest magnitude to [2^14, 2^15), so that
 *              every bit of a bf16 row within 2^-29 of its largest value is kept; NaN (and
 *              zeros in the row) when the row holds an infinity or NaN
 *   err        int32 [B]: HQ_DEVERR_* bits, OR-ed; zero-filled by the caller
 * Positions of a block that is complete (all 64 cached) are read from its page,
 * those of the incomplete last block from the tail.  Codes always come from the
 * 16-bit values, however the tokens were split over appends.
 * Limits: D == 128, cap a positive multiple of 128, B <= HQ_KV8_MAX_BATCH,
 * Hkv <= HQ_KV8_MAX_HEADS.
 */
typedef struct hq_kv8_cache {
  int32_t B, Hkv, D, cap;
  int32_t fmt;     /* HQ_KV8_E4M3 or HQ_KV8_INT8 */
  int32_t n_pages; /* pool pages (page_table != NULL) */
  uint8_t* pages;
  int32_t* page_table;
  uint16_t* tail_k;
  uint16_t* tail_v;
  float* tail_scale;
  int32_t* err;
} hq_kv8_cache;

/* device-side error bit of the calls below: cu is not ascending within [0, N], a sequence
 * has more new tokens than max_new, or kv_len is smaller than its new tokens */
#define HQ_DEVERR_ROWS 0x20u

HQ_API hq_status hq_kv8_validate(const hq_kv8_cache* c);

/*
 * Append: sequence b's new tokens are rows cu[b] .. cu[b+1]-1 of k, v [N, Hkv, D]
 * (HQ_F16 or HQ_BF16; strides in elements, multiples of 8; D contiguous) and take
 * positions kv_len[b] - n_b .. kv_len[b] - 1, n_b = cu[b+1] - cu[b]: kv_len counts the
 * new tokens.  Blocks that become complete are quantised into their pages, the newest
 * two blocks' rows stand in the tail.  A call goes on where the last one ended, or up to
 * 64 positions before the furthest one appended (drafted tokens that were rejected, more
 * than once if need be): the rows from there on are replaced; or it starts the sequence
 * anew at any multiple of 64 (a slot used again): the furthest one then counts from there,
 * and no later call goes back past that start but to start anew again.
 * Elsewhere a block's earlier 16-bit rows are gone, which no call can tell.  Rows of both
 * element types may follow one another.  cu int32 [B+1], kv_len int32 [B] (device).  A sequence with
 * kv_len > cap (HQ_DEVERR_CAPACITY) or inconsistent rows (HQ_DEVERR_ROWS) is left as it is;
 * where cu descends, so that rows belong to two sequences, so may others be.
 */
HQ_API hq_status hq_kv8_append(const hq_kv8_cache* c, int32_t dtype, const void* k, int64_t k_tok, int64_t k_head,
                               const void* v, int64_t v_tok, int64_t v_head, int32_t N, const int32_t* cu,
                               const int32_t* kv_len, hq_stream_t stream);

/*
 * Read back: positions start .. start+n-1 of every sequence, dequantised (code * scale
 * in float32, rounded once), as k_out, v_out [B, Hkv, n, D] of dtype HQ_F16, HQ_BF16 or
 * HQ_F32 (one set of strides in elements for both, multiples of 8; D contiguous).  Rows
 * at or past kv_len[b] are left as they are, or zeroed with zero_rest != 0.
 */
HQ_API hq_status hq_kv8_read(const hq_kv8_cache* c, int32_t dtype, const int32_t* kv_len, int32_t start, int32_t n,
                             void* k_out, void* v_out, int64_t o_batch, int64_t o_head, int64_t o_tok,
                             int32_t zero_rest, hq_stream_t stream);

/* Device workspace of hq_kv8_attn for these sizes (0: invalid).  Its first
 * HQ_KV8_WS_ZERO bytes are counters: zero them once before its first use; the kernels
 * return them to zero.  Calls that follow one another may share a workspace, whatever
 * their caches and sizes; calls that can run at the same time must not. */
#define HQ_KV8_WS_ZERO 4096
HQ_API size_t hq_kv8_attn_workspace_bytes(const hq_kv8_cache* c, int32_t Hq, int32_t max_new);

/*
 * Attention of each sequence's newest tokens over its cache (they must have been
 * appended): query row cu[b] + i (i < n_b <= max_new) sits at position
 * t = kv_len[b] - n_b + i and attends to positions j <= t, with window > 0 only to
 * j > t - window:
 *     out[row, h] = sum_j p_j v_j,  p = softmax_j(q[row, h] . k_j * sm_scale),
 * each key and value as cached (read through the page table; no 16-bit copy is made).
 * Query head h reads kv head h / (Hq / Hkv).
 *   q, out [N, Hq, D] HQ_F16 or HQ_BF16, strides in elements (multiples of 8), D
 *          contiguous; they must not overlap
 *   lse    float [N, Hq] contiguous or NULL: log2 of the softmax's denominator,
 *          log2 sum_j 2^(s_j), s_j = q.k_j * sm_scale * log2 e
 * Sums, softmax and accumulators are float32.  Weights times value scales enter the value
 * product as fp16 beside the largest of them: to 2^-11 of each, down to 2^-20 of that
 * largest one, below in steps of 2^-30 of it; keys whose p_j lies below 2^-126 of the
 * largest count as 0.  A bf16 query enters as fp16 at a power of two of its row: elements
 * below 2^-29 of the row's largest lose bits.  A row of q that is not finite gives NaN.
 * HQ_ERR_UNSUPPORTED where the blocks of all tasks may pass 32 bits: a call is taken while
 * B * Hkv * (cap / 64 + 14) * max(2, Hq / Hkv * max_new / 256 + 1) is below 4e9.
 * Rows outside [cu[0], cu[B]) and rows of a sequence that is skipped
 * (HQ_DEVERR_CAPACITY, HQ_DEVERR_ROWS) are left as they are.  A copy that does not land
 * within about a second ends its block's work: every sequence whose output lacks a part
 * for it, or was not begun, has HQ_DEVERR_TIMEOUT.
 */
HQ_API hq_status hq_kv8_attn(const hq_kv8_cache* c, int32_t dtype, const void* q, int64_t q_tok, int64_t q_head,
                             int32_t Hq, int32_t N, const int32_t* cu, const int32_t* kv_len, int32_t max_new,
                             int32_t window, float sm_scale, void* out, int64_t o_tok, int64_t o_head, float* lse,
                             void* ws, size_t ws_bytes, hq_stream_t stream);

/*
 * Measurement helper (no counterpart in the method): reads `bytes` (a multiple
 * of 16) of device memory at `src` (16-byte aligned) with 16-byte streaming
 * loads from sms * ctas_per_sm CTAs of 512 threads (1 <= ctas_per_sm <= 4),
 * and XORs what it read into *sink (device, 4-byte aligned) so the loads are
 * kept.  Timing it over a buffer far larger than L2 gives the read-only HBM
 * bandwidth ceiling that a scan such as the decode step can approach.
 */
HQ_API hq_status hq_diag_stream_read(const void* src, size_t bytes, uint32_t* sink, int32_t ctas_per_sm,
                                     hq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HQ_H */
