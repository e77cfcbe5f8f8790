/*
 * mbd.h -- C ABI of libmbd: weight-only low-bit decode GEMV for MI355X (gfx950).
 *
 * Sources the operations follow (cited by page title and section):
 *   [Bonsai2]    "Ternary Bonsai 2" hands-on walkthrough, 27B model to 6 GB:
 *                section 1.2 (block_ternary absmean quantizer, block 128),
 *                sections 3.4 and 5.5 (all-zero blocks: scale 1, flagged).
 *   [GPT54-INT4] "GPT-5.4 small-model compression in practice", section 3.2
 *                (INT4 group 128: scale = max|w| / 7, codes clamped to [-7, 7]).
 *   [Cassandra]  review of "Cassandra: Enabling Reasoning LLMs at Edge via
 *                Self-Speculative Decoding": 3.1 (bf16 fields), 3.2 (Wanda value
 *                pruning + bitmap, mantissa truncation, speculation + verification
 *                = original bits, draft zero-fill, target restore), 3.3 (unary
 *                exponent code by frequency rank; MX shared exponent), 3.5
 *                (chunked parallel unary decode with carried boundary state).
 *   [Bolt]       "Nemotron 3.5 Bolt teardown", background: decode time is set by
 *                the weight bytes read per token.
 *
 * Conventions shared by every call:
 *   - W is [M][K] row-major (row = output channel, K contiguous).  Activations
 *     x / X are bf16 bit patterns [B][K]; outputs y / Y are fp32 [B][M].
 *   - Pointers named *host* are CPU memory; every other data pointer is device
 *     memory owned by the caller (e.g. a torch tensor).  The library never keeps
 *     a pointer after a call returns and never allocates device memory.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Device calls only
 *     enqueue work; they never synchronise.  Argument, shape and alignment errors
 *     are reported synchronously before anything is enqueued; a launch failure
 *     returns MBD_EHIP.
 *   - Kernels trust packed data that mbd_validate() accepted; corrupt device
 *     data gives unspecified (but in-bounds) results.
 *   - Thread-safe and reentrant.  mbd_last_error() is a per-thread message for the
 *     most recent failing call on that thread.  No C++ exception crosses the ABI.
 */
#ifndef MBD_H
#define MBD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t mbd_status;
#define MBD_OK      0
#define MBD_EINVAL  1   /* null pointer, unknown format, bad parameter        */
#define MBD_ESHAPE  2   /* K % 128 != 0 (K % 32 for MX32), B outside [1, 16] */
#define MBD_EALIGN  3   /* device pointer not aligned as documented           */
#define MBD_ERANGE  4   /* bf16 Inf/NaN in W, or a scale that overflows fp16  */
#define MBD_EFORMAT 5   /* packed sections inconsistent (mbd_validate)        */
#define MBD_EHIP    6   /* HIP launch or runtime error                        */
#define MBD_ENOMEM  7   /* host allocation failed                             */

typedef enum {
    MBD_TERNARY_B128 = 1,   /* [Bonsai2] 1.2: 2-bit codes + fp16 scale per 128      */
    MBD_INT4_G128    = 2,   /* [GPT54-INT4] 3.2: 4-bit codes + fp16 scale per 128   */
    MBD_CASSANDRA    = 3,   /* [Cassandra] 3.2-3.3: bit-split speculation / verify  */
    MBD_MX32         = 4,   /* [Cassandra] 3.3: shared max exponent per 32 values   */
    MBD_TERNARY_SKIP = 5,   /* [Bonsai2] 1.2 + 3.4 / 5.5: ternary, all-zero blocks
                               flagged and not stored                              */
    MBD_CASSANDRA_MX = 6    /* [Cassandra] 3.3 Cassandra-2: speculation data with the
                               kept exponents as MX-32 instead of unary codes      */
} mbd_format;

/* ------------------------------------------------------------------ packing
 * Offline, CPU only.  Section layouts (all little-endian):
 *
 * MBD_TERNARY_B128  (sec 0) "codes"  uint32 [M*K/16]: a word holds 16 consecutive
 *                                    elements of a row, the even ones in the low half
 *                                    and the odd ones in the high half: code q+1 of
 *                                    element t of the word at bit 2*(t/2) (+16 if t
 *                                    is odd); code 3 is never written.  Word order is
 *                                    tile-interleaved (below), blocks taken in pairs
 *                                    (2h, 2h+1): unit (m, kq) of a pair is 16 bytes,
 *                                    2 words of block 2h then 2 of block 2h+1 (columns
 *                                    32kq..+32 of each); an odd last block is stored
 *                                    alone in 8-byte units.
 *                   (sec 1) "scales" fp16 [M][K/128]: fp16(mean|w| of the block),
 *                                    round to nearest even; 1.0 for an all-zero
 *                                    block (whose codes are all q = 0).
 *                   q = clamp(round_half_even(w / scale), -1, 1).
 * MBD_INT4_G128     (sec 0) "codes"  uint32 [M*K/8]: a word holds 8 consecutive
 *                                    elements of a row, evens in the low half, odds
 *                                    in the high half: code q+8 of element t of the
 *                                    word at bit 4*(t/2) (+16 if t is odd); code 0 is
 *                                    never written.  Word order is tile-interleaved
 *                                    (below); unit (m, kq) of group g is 16 bytes,
 *                                    the 4 words of columns 128g + 32kq .. +32.
 *                   (sec 1) "scales" fp16 [M][K/128]: fp16(max|w| / 7); 1.0 for
 *                                    an all-zero group.  q = clamp(rne(w/s), -7, 7).
 *                   Tile-interleaved order: rows in tiles of 16 (the last tile of a
 *                   matrix holds the R <= 16 rows left).  A tile holds its groups
 *                   (ternary: group pairs) in order; each is R*4 units, unit (row m
 *                   of the tile, quarter kq) at index kq*R + m, so that the 64 lanes
 *                   of a wave, lane = 16*kq + m, read one contiguous run.  A stack of
 *                   n_mats matrices (mbd_pack_params.n_mats) is tiled matrix by
 *                   matrix: its sections are the concatenation of each matrix's.
 * MBD_TERNARY_SKIP  The MBD_TERNARY_B128 quantizer and word encoding; a block whose
 *                   codes are all q = 0 ([Bonsai2] 3.4 / 5.5: all-zero, scale 1) is
 *                   flagged and its codes are not stored.  tiles = ceil(M / 16).
 *                   (sec 0) "codes"  uint32: the stored blocks, 32 bytes each, tile
 *                                    by tile, block column g by g; the nz stored
 *                                    blocks of (tile, g), ranked r by tile row, as
 *                                    4*nz units of 8 bytes, unit (r, kq) at index
 *                                    kq*nz + r holding columns 32kq .. +32 (2 words).
 *                   (sec 1) "scales" fp16 [M][K/128], as MBD_TERNARY_B128.
 *                   (sec 2) "slabs"  uint32 [tiles][K/128]: bit m (m < R) set when
 *                                    tile row m's block is stored (clear = the
 *                                    all-zero flag); bits 16-31: blocks stored in
 *                                    this tile before column g.  K <= 524288.
 *                   (sec 3) "tile_base" uint32 [tiles+1]: blocks stored before
 *                                    tile t; the last entry is the total.
 * MBD_CASSANDRA     Wanda keep count floor(K*keep_num/keep_den) per row, score
 *                   |w| * act_norm[k], ties to the lower k; 3 high mantissa bits
 *                   kept; 4096-element flat tiles.  f = m*K + k is the flat index.
 *                   (sec 0) "bitmap"   uint32 [ceil(M*K/32)]: keep bit of f at bit f%32
 *                   (sec 1) "spec_nib" uint32 [ceil(kept/8)]: kept values in flat
 *                                      order, (S<<3)|(M>>4), nibble i at bits 4*(i%8)
 *                   (sec 2) "unary"    uint32: rank r of each kept exponent written as
 *                                      r zeros then a one, LSB-first, kept flat order
 *                   (sec 3) "codebook" uint8 [n_sym]: rank -> exponent, ranks by
 *                                      descending count, ties to the smaller exponent
 *                   (sec 4) "bitoff"   uint64 [T+1]: unary bits before tile t
 *                   (sec 5) "kprefix"  uint32 [T+1]: kept values before tile t
 *                   (sec 6) "lo_nib"   uint32 [ceil(kept/8)]: verification, M & 15
 *                   (sec 7) "pruned"   uint16 [M*K - kept]: verification, raw bits
 *                   Sections 0-5 are the speculation data, 6-7 the verification data.
 * MBD_CASSANDRA_MX  Speculation data only, the MBD_CASSANDRA keep rule and bitmap;
 *                   the kept values in kept flat order form groups of 32 (the last
 *                   may be short).  A kept value (S, E, H = 3 high mantissa bits)
 *                   has significand sig = E ? 8 + H : H and e' = max(E, 1); X is
 *                   the largest e' of its group; mag = sig >> (X - e'), 0 once the
 *                   shift reaches 4.  Draft value (-1)^S * mag * 2^(X - 130), exact
 *                   in bf16 (-0.0 when mag = 0 and S = 1); pruned positions +0.0.
 *                   (sec 0) "bitmap"  as MBD_CASSANDRA
 *                   (sec 1) "mx_nib"  uint32 [ceil(kept/8)]: mag of kept value i at
 *                                     bits 4*(i%8) of word i/8
 *                   (sec 2) "mx_sign" uint32 [ceil(kept/32)]: S of kept value i at
 *                                     bit i%32 of word i/32
 *                   (sec 3) "mx_exp"  uint8 [ceil(kept/32)]: X of each group
 *                   (sec 4) "kprefix" uint32 [T+1]: kept values before tile t
 *                   mbd_spec_decode and mbd_spec_gemv take it; mbd_gemv does not
 *                   (no verification data).
 * MBD_MX32          (sec 0) "mx_exp"  uint8 [M][K/32]: X = max over the group of
 *                                     max(E, 1)
 *                   (sec 1) "mx_sign" uint32 [M][K/32]: bit i = sign of element i
 *                   (sec 2) "mx_mag"  uint8 [M][K]: (E ? 128|M : M) >> (X - max(E,1)),
 *                                     0 when the shift is 8 or more.
 *                   Value = (-1)^S * mag * 2^(X - 134), exact in bf16.
 *
 * Every section buffer is zero padded: `padded_bytes` (a multiple of 256, at least
 * `bytes` + 256) is the size to copy to the device; kernels may read the padding.
 */
typedef struct {
    int32_t keep_num;   /* Cassandra keep fraction numerator   (default 3)  */
    int32_t keep_den;   /* Cassandra keep fraction denominator (default 10) */
    int64_t n_mats;     /* TERNARY / INT4: the M rows are n_mats stacked matrices
                           of M / n_mats rows each (default 1; 0 means 1)   */
} mbd_pack_params;

typedef struct mbd_packed mbd_packed;   /* opaque, owns the host section buffers */

typedef struct {
    const char* name;       /* static string, e.g. "codes"                   */
    const void* data;       /* host pointer owned by the mbd_packed handle   */
    uint64_t bytes;         /* meaningful bytes                              */
    uint64_t padded_bytes;  /* bytes to copy to the device (zero padded)     */
} mbd_section;

typedef struct {
    int32_t fmt;
    int32_t n_sym;          /* Cassandra codebook size                       */
    int64_t M, K;
    int64_t n_kept;         /* Cassandra kept values                         */
    int64_t unary_bits;     /* Cassandra unary stream length in bits         */
    int64_t n_tiles;        /* Cassandra 4096-element tiles                  */
    double bpw;             /* all sections' meaningful bits / (M*K)         */
    double spec_bpw;        /* Cassandra speculation sections (0-5) / (M*K)  */
    double exp_entropy_bits;/* Cassandra: Shannon entropy of kept exponents  */
    double unary_avg_bits;  /* Cassandra: unary bits per kept value          */
    double zero_fraction;   /* ternary: fraction of q == 0                   */
} mbd_stats;

/* Pack a bf16 weight.  w_bf16_host [M][K] and act_norm_host [K] (fp32, Cassandra
 * only, else may be NULL) are borrowed for the call.  params may be NULL (defaults).
 * On success *out is a new handle; free it with mbd_packed_free().
 * Errors: EINVAL (null / unknown fmt / bad params), ESHAPE (M < 1, K < 1 or K not a
 * multiple of 128 (32 for MX32)), ERANGE (Inf/NaN in W, fp16 scale overflow, non-finite
 * or negative act_norm), ENOMEM. */
mbd_status mbd_pack(int32_t fmt, const uint16_t* w_bf16_host, int64_t M, int64_t K,
                    const float* act_norm_host, const mbd_pack_params* params,
                    mbd_packed** out);

/* Copy up to `cap` section descriptors into arr (section order as documented above)
 * and the total count into *n.  Pointers stay valid until mbd_packed_free(h).  The
 * sections are the saved form of a quantized weight: codes and scales stored apart
 * ([GPT54-INT4] 3.2, the weight saved with its scales; [Bonsai2] 3.6, export of the
 * packed model), or the speculation and verification parts ([Cassandra] 3.2: the
 * draft loads the first only, the target both).  cap = 0 only reports *n.
 * Errors: EINVAL (NULL h or n, or arr NULL with cap > 0). */
mbd_status mbd_packed_sections(const mbd_packed* h, mbd_section* arr, int32_t cap, int32_t* n);
/* Format statistics of a handle ([Cassandra] 3.3: exponent entropy of the kept
 * values and average unary code length; bits per weight of all sections and of
 * the speculation sections; [Bonsai2] 1.2: fraction of ternary zeros).
 * Errors: EINVAL (NULL argument). */
mbd_status mbd_packed_stats(const mbd_packed* h, mbd_stats* out);
/* Full CPU consistency check of a handle's sections (codes in range, bitmap row
 * counts, tile table vs unary stream, codebook ranks): the conditions under which
 * the decode of [Cassandra] 3.5 and the dequantization of [Bonsai2] 1.2 and
 * [GPT54-INT4] 3.2 are defined.  EFORMAT on failure, EINVAL for NULL. */
mbd_status mbd_validate(const mbd_packed* h);
/* Releases the handle and its host sections; NULL is a no-op. */
void mbd_packed_free(mbd_packed* h);

/* ------------------------------------------------------------------ device data
 * Raw device pointers to byte copies (padded_bytes) of the packed sections, in the
 * documented section order.  Section base pointers must be 16-byte aligned.
 * n_mats > 1 describes n_mats matrices of identical shape stacked back to back in
 * each section (ternary / INT4 only; used by the expert GEMV). */
#define MBD_MAX_SECTIONS 8
typedef struct {
    int32_t fmt;
    int32_t n_sym;
    int64_t M, K;
    int64_t n_kept;
    int64_t n_mats;
    const void* sec[MBD_MAX_SECTIONS];
} mbd_dweights;

/* Dense dequantized weight w_out fp32 [M][K] (TERNARY, TERNARY_SKIP, INT4, MX32):
 * q*s ([Bonsai2] 1.2, the ternary value is the code times its block scale;
 * [GPT54-INT4] 3.2, the INT4 value is the code times its group scale) or
 * (-1)^S*mag*2^(X-134) ([Cassandra] 3.3, the MX value is the shifted significand at
 * the shared exponent), all exact in fp32.  w_out 16-byte aligned, caller-owned.
 * Errors: EINVAL (NULL, unknown format), ESHAPE, EALIGN, EHIP. */
mbd_status mbd_dequant(const mbd_dweights* w, float* w_out, void* stream);

/* Fused dequant-GEMV / skinny GEMM: y[b][m] = sum_k deq(W)[m][k] * x[b][k] with fp32
 * accumulation ([Bolt] background; [Bonsai2] 1.2; [GPT54-INT4] 3.2).
 * TERNARY and INT4: B in [1, 16].  MX32: B in [1, 16] (MFMA bf16, the Cassandra-2
 * verify GEMM).  CASSANDRA: the target-side verify GEMM over the restored weight
 * (speculation + verification data merged on the fly, [Cassandra] 3.2), B in [1, 16].
 * x: bf16 [B][K], 16-byte aligned.  y: fp32 [B][M], 4-byte aligned.  TERNARY,
 * TERNARY_SKIP and INT4 at B > 4 address the activations with 32-bit element
 * offsets: B·K of 2^32 or more returns MBD_ESHAPE. */
mbd_status mbd_gemv(const mbd_dweights* w, const uint16_t* x, int32_t B, float* y,
                    void* stream);

/* Expert GEMV over n_mats stacked TERNARY or INT4 matrices (MoE; [Bolt] routes each
 * token to a subset of experts).  route [T][k] int32 expert ids in [0, n_mats) with
 * distinct ids per token.  x bf16: [T][K] (x_per_pair = 0) or [T][k][K]
 * (x_per_pair = 1).  y fp32 [T][k][M]: y[t][j] = W[route[t][j]] @ x_row.  An
 * expert's weights are read once per group of up to 16 tokens routed to it.  At
 * most 4096 experts (MBD_ESHAPE beyond).  Ids outside [0, n_mats) leave their y
 * rows unwritten; an id repeated within a token is outside this contract (with at
 * most 16 tokens, pairs past an expert's 16th may be left unwritten).  ws: device workspace of at least
 * mbd_moe_workspace_bytes(n_mats, T, k) bytes, 16-byte aligned, contents
 * overwritten.  Calls that share a workspace must not overlap.  With T > 1 the
 * activations are addressed with 32-bit element offsets: x's rows (T, or T·k with
 * x_per_pair) times K of 2^32 or more returns MBD_ESHAPE. */
mbd_status mbd_moe_workspace_bytes(int64_t n_mats, int32_t T, int32_t k, uint64_t* bytes);
mbd_status mbd_moe_gemv(const mbd_dweights* experts, const int32_t* route, int32_t T,
                        int32_t k, const uint16_t* x, int32_t x_per_pair, float* y,
                        void* ws, uint64_t ws_bytes, void* stream);

/* mbd_moe_gemv for callers that cannot allocate device memory or pass a workspace
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same kernels and results, with the grouping tables in a static
 * device array of the library (1 MiB per device, held until the process ends; its
 * address is looked up once per device on the first call there).  Routes whose
 * workspace (mbd_moe_workspace_bytes) exceeds 1 MiB return MBD_ESHAPE.  Every call
 * on one device shares that array: calls that overlap on a device race (serialise
 * them on one stream).  No allocation of any kind, host or device. */
mbd_status mbd_moe_gemv_noalloc(const mbd_dweights* experts, const int32_t* route, int32_t T,
                                int32_t k, const uint16_t* x, int32_t x_per_pair, float* y,
                                void* stream);

/* Draft weights from the speculation data only ([Cassandra] 3.2, path b): bf16
 * w_spec [M][K]; kept values get (S<<15)|(E<<7)|(M_hi<<4), pruned values +0.0.
 * Sections 6-7 are not read and may be NULL.  w_spec 16-byte aligned. */
mbd_status mbd_spec_decode(const mbd_dweights* w, uint16_t* w_spec, void* stream);

/* Draft GEMV fused with speculation decode: y = W_spec x, B in [1, 16]. */
mbd_status mbd_spec_gemv(const mbd_dweights* w, const uint16_t* x, int32_t B, float* y,
                         void* stream);

/* Bit-exact original weights from speculation + verification data ([Cassandra]
 * 3.2, path c): bf16 w_out [M][K], 16-byte aligned. */
mbd_status mbd_verify_restore(const mbd_dweights* w, uint16_t* w_out, void* stream);

/* ------------------------------------------------------------------ device encoder
 * [Cassandra] 3.2-3.3 (and 3.5, the online encoder the paper builds in hardware):
 * the eight MBD_CASSANDRA sections of a bf16 weight already in device memory,
 * bit-identical to mbd_pack(MBD_CASSANDRA) with the same keep fraction.
 * w: bf16 [M][K] device, 16-byte aligned; act_norm: fp32 [K] device; K % 128 == 0,
 * M*K < 2^32.  ws: device workspace of mbd_encode_workspace_bytes(M) bytes,
 * 16-byte aligned, shared by both calls (contents overwritten).
 * mbd_encode_plan runs the pruning and the exponent histogram and returns the
 * section sizes; it SYNCHRONISES `stream` to read two totals back, and reports
 * MBD_ERANGE for Inf/NaN in w or a negative / non-finite act_norm entry.
 * mbd_encode_cassandra then writes every section: sec[i] is a device buffer of at
 * least plan->padded_bytes[i] bytes, 16-byte aligned (padding zeroed by the call).
 * It only enqueues work; w and act_norm must be those the plan was made from (the
 * unary stream is cut at the planned size otherwise).  Calls that share a
 * workspace must not overlap. */
typedef struct {
    int64_t n_kept;
    int64_t unary_bits;
    int64_t n_tiles;
    int32_t n_sym;
    int32_t reserved;
    uint64_t bytes[8];         /* meaningful bytes of each section, MBD_CASSANDRA order */
    uint64_t padded_bytes[8];  /* buffer bytes the encode call writes               */
} mbd_encode_plan_t;
mbd_status mbd_encode_workspace_bytes(int64_t M, uint64_t* bytes);
mbd_status mbd_encode_plan(const uint16_t* w, const float* act_norm, int64_t M, int64_t K,
                           int32_t keep_num, int32_t keep_den, void* ws, uint64_t ws_bytes,
                           mbd_encode_plan_t* plan, void* stream);
mbd_status mbd_encode_cassandra(const uint16_t* w, const float* act_norm, int64_t M, int64_t K,
                                int32_t keep_num, int32_t keep_den, const mbd_encode_plan_t* plan,
                                void* const* sec, void* ws, uint64_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ KV cache
 * The other half of what a decode step reads: a paged cache of 8-bit keys and values.
 * A pool of n_blocks blocks holds block_size tokens each; a request's block table
 * names its blocks in order.  Each (block, KV head) has one fp32 scale for its keys
 * and one for its values; a value is code * scale.
 *
 * Formats, x the value to store, s the scale, amax the largest finite |x| among the
 * tokens that one call brings to a (block, head):
 *   MBD_KV_INT8  code = clamp(rne(x / s), -127, 127); wanted s = amax * (1/127), the
 *                constant rounded to fp32, quotient and product rounded to fp32.
 *   MBD_KV_E4M3  code = e4m3fn(x / s), nearest even, saturating at 448; wanted s =
 *                the smallest power of two, at least 2^-126, with amax <= 448 s.
 * amax = 0 wants s = 0 (codes 0).  NaN is stored as 0; an infinity as the largest code.
 * A slot is block * block_size + place in the block.  A block's tokens are appended
 * in order, so a token at place o finds o live tokens before it: the first call that
 * reaches a block at place 0 sets the wanted scale; later calls take
 * s' = max(s, wanted), and where that is larger than s the live codes become
 * rne(code * fl32(s / s')) (for E4M3 a power of two, so exact above its subnormals).
 *
 * Codes: uint8 [n_blocks][n_heads][block_size/16] tiles of 16 tokens x head_dim, in the
 * order in which a wave's 64 lanes feed them to the matrix cores 16 bytes each.  Byte
 * of (token t of the tile, channel d):
 *   keys    (d/64)*1024 + (d/16%4)*256 + t*16 + d%16
 *   values  (d/64)*1024 + (t/4)*256 + (d/4%16)*16 + d%4*4 + t%4
 * Scales: fp32 [n_blocks][n_heads].  None of it needs to be cleared before use.  */
typedef enum { MBD_KV_INT8 = 1, MBD_KV_E4M3 = 2 } mbd_kv_format;
typedef enum { MBD_BF16 = 1, MBD_F32 = 2 } mbd_dtype;

typedef struct {
    int32_t fmt;          /* mbd_kv_format                              */
    int32_t block_size;   /* tokens a block: 16, 32, 64, 128 or 256     */
    int32_t n_heads;      /* KV heads, 1..65535                         */
    int32_t head_dim;     /* 64, 128, 192 or 256                        */
    int64_t n_blocks;     /* n_blocks * block_size < 2^31               */
    void* k_codes;        /* device, 16-byte aligned; offsets may pass  */
    void* v_codes;        /*   32 bits                                  */
    float* k_scale;       /* device, 4-byte aligned                     */
    float* v_scale;
} mbd_kv_cache;

/* Block tables of n_seqs requests over one pool, and its free blocks as a stack:
 * free_blocks[0 .. n_free) are free, the last is taken first. */
typedef struct {
    int32_t n_seqs;       /* 1..4096                                    */
    int32_t block_size;   /* 16, 32, 64, 128 or 256                     */
    int32_t max_blocks;   /* columns of the block table                 */
    int32_t n_blocks;     /* length of free_blocks; ids are below it    */
    int32_t* block_table; /* device [n_seqs][max_blocks]                */
    int32_t* free_blocks; /* device [n_blocks]                          */
} mbd_kv_pool;

/* One step's bookkeeping, from request lengths, in one call: which blocks each request
 * gets, and where each of its new tokens goes.  All arrays are device int32.
 *   in   new_tokens [n_seqs]  tokens that the request brings; negative: it has ended,
 *                             and its blocks go back to the pool
 *        lens [n_seqs]        tokens it has cached; held [n_seqs] blocks it holds
 *        n_free [1]
 *   out  seq_start [n_seqs+1] exclusive prefix sum of max(new_tokens, 0), at most T:
 *                             the rows of the step's packed [T] token batch
 *        slots [T]            slot of each new token; -1 for tokens of a request that
 *                             is not served and for rows past seq_start[n_seqs]
 *        positions [T]        its place in its request (lens + j), or -1; may be NULL
 *        lens_out, held_out [n_seqs], n_free_out [1]: after the step (may be the
 *                             same buffers as lens, held, n_free)
 *        status [n_seqs]      0 served, or nothing to do; 1 the pool has too few
 *                             blocks; 2 more than max_blocks columns; 3 its tokens end
 *                             past T; 4 lens or held cannot be (negative, held above
 *                             max_blocks, lens above held blocks' tokens)
 * Ended requests' blocks are pushed in request order, each in table order, before any
 * is taken.  Requests take blocks in order, all that they need or none: one is served
 * if it needs none, or if what it and the requests before it need (those of status 1
 * among them) is there.  A request not served keeps lens, held and its table row.
 * Rows of ended requests stay as they were, with lens_out = held_out = 0.  A request
 * whose lens was lowered (rejected drafts) keeps its blocks and fills them again.
 * Errors: EINVAL (NULL), ESHAPE (n_seqs, block_size, max_blocks or n_blocks < 1,
 * either times block_size 2^31 or more, T < 0), EALIGN (4 bytes), EHIP. */
mbd_status mbd_kv_slots(const mbd_kv_pool* pool, const int32_t* new_tokens, const int32_t* lens,
                        const int32_t* held, const int32_t* n_free, int32_t T, int32_t* seq_start,
                        int32_t* slots, int32_t* positions, int32_t* lens_out, int32_t* held_out,
                        int32_t* n_free_out, int32_t* status, void* stream);

/* Quantise T tokens' keys and values into the cache (rules above).  k, v: device
 * [T][n_heads][head_dim] of dtype (MBD_BF16 or MBD_F32, e.g. rows of mbd_gemv's y),
 * 16-byte aligned; k_stride, v_stride: elements from one token to the next, multiples
 * of 8, at least n_heads * head_dim (so both may be slices of one projection).  slots
 * [T] device int32: the slot of each token; a slot outside the cache skips its token.
 * The tokens that a call brings to one block stand next to each other in rising slots
 * (as mbd_kv_slots writes them); otherwise that block's codes and scale are unspecified.
 * T = 0 does nothing; T is at most 2^24.  Errors: EINVAL, ESHAPE, EALIGN, EHIP. */
mbd_status mbd_kv_append(const mbd_kv_cache* cache, const void* k, const void* v, int32_t dtype,
                         int64_t k_stride, int64_t v_stride, const int32_t* slots, int32_t T,
                         void* stream);

/* Dense keys and values of cached tokens: k_out, v_out [T][n_heads][head_dim] of dtype,
 * 16-byte aligned: code * scale in fp32, then rounded to dtype.  Any slots in any order;
 * rows of slots outside the cache stay as they were.  Errors as mbd_kv_append. */
mbd_status mbd_kv_gather(const mbd_kv_cache* cache, const int32_t* slots, int32_t T, int32_t dtype,
                         void* k_out, void* v_out, void* stream);

/* Attention of each request's newest tokens over its cache, causal:
 *   u_ij = cap(scale * q_i . k_j) + slope_h * (j - i),  cap(x) = softcap * tanh(x / softcap)
 *   o_i  = sum_j softmax_j(u_ij) v_j   over j <= i, i - j < window, j in a block with an id
 * i, j positions in the request.  softcap = 0: no cap; window = 0: no window; slopes
 * NULL: no distance bias. */
typedef struct {
    int32_t n_heads;      /* query heads, a multiple of the cache's; query head h reads
                             KV head h / (n_heads / cache n_heads); at most 256 of them
                             a KV head                                                  */
    int32_t n_seqs;       /* 1..4096                                                    */
    int32_t max_blocks;   /* columns of the block table                                 */
    int32_t T;            /* rows of q, out and lse                                     */
    int32_t max_new;      /* most new tokens of one request, >= 1: 1 for decode, N+1 to
                             verify N drafts, more for prompts                          */
    int32_t window;       /* >= 0                                                       */
    float scale, softcap; /* scale in [-2^64, 2^64]; softcap 0, or 2^-64 to 2^64 and
                             |scale| / softcap at most 2^126                            */
    const float* slopes;  /* device fp32 [n_heads], or NULL                             */
    int64_t q_stride;     /* elements from one token's row to the next, a multiple of 8 */
    int64_t out_stride;   /*   and at least n_heads * head_dim                          */
} mbd_kv_attn_args;

/* seq_start [n_seqs+1], lens [n_seqs], block_table [n_seqs][max_blocks]: device int32.
 * Request i's queries are rows seq_start[i] .. seq_start[i+1] of q [T][n_heads][head_dim]
 * (bf16, 16-byte aligned); they are its last tokens: row j of n_i stands at position
 * lens[i] - n_i + j, its own key and value already appended.  lens is taken as at most
 * max_blocks * block_size, seq_start as within [0, T].  Block ids outside the cache
 * are left out, as if masked.  A query that sees nothing (position below 0, all
 * blocks left out) gets o = 0, lse = -inf.  Rows of a request that mbd_kv_slots did not
 * serve are taken as its last cached tokens: they mean nothing, their caller drops them.
 * out bf16 [T][n_heads][head_dim], 16-byte aligned: as the x of mbd_gemv where out_stride
 * = n_heads * head_dim.  lse fp32 [T][n_heads], natural logarithm of the softmax's sum, or
 * NULL.  Rows of no request, and a request's rows past its first max_new, stay as they
 * were.  Sums and statistics are fp32 (so a product q . k of codes, an uncapped score times
 * log2(e), and 2^8 times the sum of a channel's |v| over the tokens a query sees have to
 * stay below 2^127); softmax weights times value scales enter the second product as bf16, each off
 * by at most 2^-8 of itself.  The order of every sum depends on the arguments alone.
 * ws: device workspace of mbd_kv_attn_workspace_bytes, 16-byte aligned, contents
 * overwritten; may be NULL where that is 0.  One made for the most n_seqs, max_new and
 * max_blocks of a program serves its smaller calls of the same heads too.  Calls that
 * share a workspace must not overlap.  Errors: EINVAL, ESHAPE (T above 2^24, max_blocks *
 * block_size above 2^30, n_seqs * max_blocks * block_size / 16 of 2^31 or more, KV heads
 * times tiles of query rows of 2^24 or more, n_seqs times those of max_new above 2^28),
 * EALIGN, EHIP. */
mbd_status mbd_kv_attn_workspace_bytes(const mbd_kv_cache* cache, int32_t n_heads, int32_t n_seqs,
                                       int32_t max_new, int32_t max_blocks, uint64_t* bytes);
mbd_status mbd_kv_attn(const mbd_kv_cache* cache, const mbd_kv_attn_args* args, const uint16_t* q,
                       const int32_t* seq_start, const int32_t* lens, const int32_t* block_table,
                       uint16_t* out, float* lse, void* ws, uint64_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ measurement aid
 * Streaming-read probe, not a step of the method: reads `bytes` of device memory at
 * src (16-byte aligned, a multiple of 16) with `blocks` x `threads` threads (threads
 * a multiple of 64, at most 1024), 16-byte non-temporal loads, eight in flight per
 * thread.  The measured rate is the practical ceiling of the weight-streaming kernels
 * ([Bolt] background: a decode step's time is the weight bytes it reads).  sink:
 * device uint32 [blocks], never written in practice (it keeps the loads alive).
 * Errors: EINVAL, EALIGN, ESHAPE, EHIP. */
mbd_status mbd_probe_stream_read(const void* src, uint64_t bytes, uint32_t* sink, int32_t blocks,
                                 int32_t threads, void* stream);

const char* mbd_status_str(mbd_status s);
const char* mbd_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MBD_H */
