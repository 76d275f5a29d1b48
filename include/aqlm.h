/*
 * aqlm.h - C ABI of libaqlm.so: the AQLM 2-bit quantized linear layer on
 * AMD Instinct MI355X (gfx950).
 *
 * Representation ("The AQLM Quantization Algorithm, Explained", section
 * "What is Multi-Codebook Quantization (MCQ)?" and Figure 2): a weight matrix
 * W of shape [out][in] (W.X convention, rows are output channels) is cut
 * row-wise into groups of g consecutive inputs.  Group j of row i is the sum
 * of M codewords, one from each of M codebooks of 2^B fp16 codewords of
 * length g, then multiplied by the row's fp16 scale:
 *
 *     W[i][j*g + t] = s[i] * sum_{m=0}^{M-1} C_m[ code[i][j][m] ][t]
 *
 * Schemes ("Key AQLM quantization parameters" on the same page: (M, B, g)
 * are free hyperparameters, and e.g. (1, 4), (2, 8), ..., (8, 32) at B = 8
 * all cost 2 bits per weight): 1 <= M <= AQLM_MAX_CODEBOOKS, 1 <= B <= 16,
 * g in {1, 2, 4, 8, 16, 32}.  The two named there as XBit-MxB at g = 8,
 * (1, 16, 8) "1x16" and (2, 8, 8) "2x8", run tuned kernels; every other
 * triple runs general kernels with the same semantics, except that the GEMV
 * of the other 2-bit triples with B = 8 ((1, 8, 4), (4, 8, 16), and
 * (8, 8, 32) above batch 8) runs the tuned 2x8 kernel when in % 8 == 0, and
 * the prefill GEMM of (1, 8, 4) the tuned 2x8 pipeline when in % 64 == 0.
 *
 * Memory layouts (all arrays contiguous, row-major, DEVICE pointers):
 *   codes      [out][in/g][M]  uint8 for B <= 8; 16-bit (int16) for
 *                              9 <= B <= 16.  The codeword index is the low
 *                              B bits of the stored pattern read as unsigned
 *                              (the page notes that a B that is not a
 *                              multiple of 8 leaves bits of its bytes unused)
 *   codebooks  [M][2^B][g]     fp16 (IEEE binary16, passed as opaque 16-bit
 *                              storage)
 *   scales     [out]           fp16
 *   x          [batch][in]     fp16 activations
 *   y          [batch][out]    fp16 outputs (decode: W16 [out][in])
 *
 * Ownership: the caller owns every buffer.  No entry point keeps a pointer
 * after it returns, and none allocates device memory.
 *
 * Asynchrony: every call validates its arguments on the host, enqueues its
 * kernels on `stream` (a hipStream_t; NULL means the null stream) and
 * returns.  Execution errors surface at the caller's next synchronisation.
 * Calls are reentrant and thread-safe.  A call with out == 0 (or, for GEMV
 * and GEMM, batch == 0) enqueues nothing and returns AQLM_OK once the scheme
 * and shape are valid; its pointers may then be NULL.
 *
 * Numerics: GEMV and GEMM accumulate in fp32 and round y to fp16 once
 * (nearest-even).  Decode is bit-exact: per weight, the fp32 sum of the M
 * codewords (codebook 0 first, then m ascending, the sum starting from
 * codebook 0's codeword), times the fp32 scale, rounded to fp16 nearest-even
 * with subnormals kept.
 */
#ifndef AQLM_H
#define AQLM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    AQLM_OK = 0,
    AQLM_ERR_NULL = 1,   /* a required pointer is NULL (or decode got x != NULL) */
    AQLM_ERR_SHAPE = 2,  /* out/in/batch negative or out of range, in % g != 0 */
    AQLM_ERR_SCHEME = 3, /* (M, B, g) outside 1..AQLM_MAX_CODEBOOKS x 1..16 x {1,2,4,8,16,32} */
    AQLM_ERR_ALIGN = 4,  /* codes, codebooks, x or y not 16-byte aligned, scales not 2-byte aligned */
    AQLM_ERR_HIP = 5,    /* the HIP runtime reported an error at launch */
    AQLM_ERR_SCRATCH = 6, /* more scratch needed than an allocation-free entry point holds */
    AQLM_ERR_ACT = 7     /* an activation that is none of aqlm_act */
} aqlm_status;

/* Largest `in` accepted (inputs per row). */
#define AQLM_MAX_IN (1 << 20)
/* Most codebooks (M) a scheme may have. */
#define AQLM_MAX_CODEBOOKS 8
/* Largest batch of aqlm_linear_gemv. */
#define AQLM_GEMV_MAX_BATCH 16

/*
 * y[b][i] = sum_k W[i][k] * x[b][k] for b < batch, with W decoded on the fly
 * (Figure 2 of the MCQ section: weights are dequantized after being fetched,
 * then multiplied).  Decode-phase matrix-vector product: 1 <= batch <= 16.
 * Requires 1 <= in <= AQLM_MAX_IN, in % g == 0, out <= 2^31 - 16.
 */
int aqlm_linear_gemv(const void* codes, const void* codebooks, const void* scales,
                     const void* x, void* y, int M, int B, int g,
                     int64_t out, int64_t in, int64_t batch, void* stream);

/* Most layers one aqlm_linear_gemv_fused call takes. */
#define AQLM_FUSED_MAX_LAYERS 8

/*
 * n_layers decode-phase products that share the activations x, in one launch:
 *
 *     y_l[b][i] = sum_k W_l[i][k] * x[b][k]   for l < n_layers, b < batch,
 *
 * e.g. the q, k and v projections of an attention block, or the gate and up
 * projections of its MLP, which all multiply the same hidden state.  Layer l
 * has its own codes[l], codebooks[l], scales[l], outs[l] rows and output
 * ys[l] ([batch][outs[l]]); all layers share (M, B, g), in, batch and x.
 * codes, codebooks, scales, outs and ys are HOST arrays of n_layers entries;
 * the pointers they hold are device pointers with the layouts above.  The
 * library reads the arrays during the call and keeps nothing.
 *
 * Each layer is validated exactly as by aqlm_linear_gemv and the first
 * failing layer's status is returned (nothing is enqueued then); a layer
 * with outs[l] == 0 is skipped.  1 <= n_layers <= AQLM_FUSED_MAX_LAYERS
 * (else AQLM_ERR_SHAPE); a NULL array gives AQLM_ERR_NULL.  The results are
 * bit-identical to n_layers separate aqlm_linear_gemv calls; fusing pays the
 * launch and the per-workgroup start-up latencies once for the group.  (The
 * triples whose GEMV runs a general kernel are served by one launch per
 * layer.)
 */
int aqlm_linear_gemv_fused(int n_layers, const void* const* codes, const void* const* codebooks,
                           const void* const* scales, const int64_t* outs, const void* x,
                           void* const* ys, int M, int B, int g, int64_t in, int64_t batch,
                           void* stream);

/*
 * Same product for a prefill batch of `batch` >= 1 tokens (batch <= 2^31 - 1):
 * W tiles are decoded into LDS and fed to fp16 matrix cores with fp32
 * accumulation.
 */
int aqlm_linear_gemm(const void* codes, const void* codebooks, const void* scales,
                     const void* x, void* y, int M, int B, int g,
                     int64_t out, int64_t in, int64_t batch, void* stream);

/*
 * The same prefill product in two passes, following the page's statement that
 * the product with the activations runs on the dequantized half-precision
 * weights ("The AQLM Quantization Algorithm, Explained", MCQ section, Figure
 * 2): the weights are decoded once into `workspace` (W16[out][in] fp16,
 * bit-exact as aqlm_linear_decode writes them, the scale applied), then a
 * dense fp16 matrix-core product y = x W16^T runs with fp32 accumulation and
 * one rounding to fp16.  Each weight is decoded once instead of once per
 * 256-token tile.  workspace is caller-owned device memory, 16-byte aligned,
 * of at least aqlm_gemm_dequant_workspace_bytes bytes; its contents are
 * overwritten, and calls that share it must not run concurrently.  Every
 * argument is validated as by aqlm_linear_gemm, and out * (in / g) <
 * 2^32 (else AQLM_ERR_SHAPE).  A NULL or undersized workspace gives
 * AQLM_ERR_NULL / AQLM_ERR_SHAPE, a misaligned one AQLM_ERR_ALIGN.  When
 * in % 64 != 0 the call runs aqlm_linear_gemm instead and does not touch the
 * workspace.
 */
int aqlm_linear_gemm_dequant(const void* codes, const void* codebooks, const void* scales,
                             const void* x, void* y, void* workspace, int64_t workspace_bytes,
                             int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);

/* Bytes of workspace aqlm_linear_gemm_dequant needs (out * in * 2; 0 when in % 64 != 0). */
int aqlm_gemm_dequant_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t* bytes);

/*
 * Writes the dequantized fp16 weights W16[out][in] to y (bit-exact as stated
 * above).  x must be NULL; batch is ignored.
 */
int aqlm_linear_decode(const void* codes, const void* codebooks, const void* scales,
                       const void* x, void* y, int M, int B, int g,
                       int64_t out, int64_t in, int64_t batch, void* stream);

/* ---------------------------------------------------------------------------
 * Bit-packed codes ("Key AQLM quantization parameters" on the same page: a B
 * that is not a multiple of 8 leaves unused bits in the bytes that hold each
 * code; packing drops them, so e.g. (1, 12, 4) stores 3 bits per weight in its
 * codes instead of 4).  Packed layout: the codes in their stored order
 * ([out][in/g][M] flattened, code n = (i * in/g + j) * M + m) form one bit
 * stream, code n in bits [n B, n B + B), least significant bit first; bit b is
 * bit b % 32 of 32-bit word b / 32 (little-endian words); the stream is padded
 * with zero bits to a whole word.  Rows are not padded (a row may start inside
 * a word).  The buffer holds aqlm_packed_codes_bytes bytes and is 4-byte
 * aligned.
 *
 * aqlm_linear_{gemv,gemm,decode}_packed take such a stream as `codes` and
 * otherwise the arguments, validation and results of aqlm_linear_{gemv,gemm,
 * decode} (decode bit-exact; every scheme of AQLM_ERR_SCHEME's range runs the
 * general kernels); a misaligned stream gives AQLM_ERR_ALIGN.  aqlm_pack_codes
 * writes the stream of whole-byte codes [out][in/g][M] (the low B bits of each
 * stored code; every word of the stream, padding bits zero).
 */
int aqlm_packed_codes_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t* bytes);
int aqlm_pack_codes(const void* codes, void* packed, int M, int B, int g, int64_t out, int64_t in, void* stream);
int aqlm_linear_gemv_packed(const void* codes, const void* codebooks, const void* scales, const void* x, void* y,
                            int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);
int aqlm_linear_gemm_packed(const void* codes, const void* codebooks, const void* scales, const void* x, void* y,
                            int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);
int aqlm_linear_decode_packed(const void* codes, const void* codebooks, const void* scales, const void* x, void* y,
                              int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);

/* ---------------------------------------------------------------------------
 * Building the representation ("The AQLM quantization procedure" on the same
 * page: per layer, the codes are learned first with fixed codebooks that a
 * residual k-means initialises).  The page's learning loss is lost and needs
 * calibration data; these are its data-free counterparts on plain weights:
 *
 *   target of a group    W[i][j*g .. j*g+g) / s_i, one fp32 division each;
 *   code of codebook m   the nearest codeword (squared Euclidean distance,
 *                        sum_t (r_t - c_t)^2 in fp32, t ascending, no fused
 *                        multiply-add, lowest index on a tie) to the target
 *                        minus the codewords chosen for codebooks 0 .. m-1.
 *
 * w is [out][in] fp16 (16-byte aligned), scales [out] fp16 (the page does not
 * say how scales are initialised; the caller gives them), codes and
 * codebooks as above.  Both calls accept every scheme the products accept.
 * out == 0 enqueues nothing.  Results are deterministic and bit-identical to
 * the plain CPU definition.
 */

/* Greedy residual codes for w with the given codebooks; writes codes. */
int aqlm_encode_greedy(const void* w, const void* scales, const void* codebooks, void* codes,
                       int M, int B, int g, int64_t out, int64_t in, void* stream);

/* Largest iteration count aqlm_kmeans_init accepts. */
#define AQLM_KMEANS_MAX_ITERS 10000

/* Bytes of device workspace aqlm_kmeans_init needs for the scheme (into *bytes). */
int aqlm_kmeans_workspace_bytes(int M, int B, int g, int64_t* bytes);

/*
 * Residual k-means: for m = 0 .. M-1, Lloyd's algorithm (`iters` rounds of
 * assign + update) on what codebooks 0 .. m-1 leave of every group's target,
 * seeded with the leftovers of groups seeds[m][0 .. 2^B-1] (device int64
 * [M][2^B], group index = row * in/g + j, clamped into range); writes the fp16
 * codebooks [M][2^B][g] and the codes of the greedy encoding against them.
 * A centroid is the mean of its members, summed exactly as integers in units
 * of 2^-24 and divided in float64, then rounded to fp32; an empty cluster
 * keeps its centroid; codebook m is the fp16 rounding of the centroids.  The
 * sums are exact while every target satisfies |W/s| < 2^29 / n_groups
 * (n_groups = out * in / g; e.g. |W/s| < 256 with 2^21 groups).  A target at
 * or above that bound, or not finite, cannot be summed exactly: the call then
 * does not produce wrapped sums but NaN codebooks (from the first k-means round
 * that meets such a target on; every later codebook too), and the codes
 * assigned against them are 0.  `workspace` is caller-owned device memory of
 * at least aqlm_kmeans_workspace_bytes bytes (16-byte aligned); its contents
 * on entry do not matter.
 */
int aqlm_kmeans_init(const void* w, const void* scales, const int64_t* seeds, void* codebooks, void* codes,
                     void* workspace, int64_t workspace_bytes, int M, int B, int g,
                     int64_t out, int64_t in, int iters, void* stream);

/* ---------------------------------------------------------------------------
 * 1x16 at batch 1 over slice lists ("Key AQLM quantization parameters" on the
 * same page: 1x16 is the scheme with 2^16 codewords, and its decoding is the
 * slower one because of them).  The product above gathers a 16-byte codeword
 * per code from the 1 MiB codebook; these calls instead regroup the codes of
 * a layer once, at load time, so that a workgroup can keep one eighth of the
 * codebook (8192 codewords, 128 KB) in LDS and read only the codes that fall
 * in it.  Only (M, B, g) = (1, 16, 8) (else AQLM_ERR_SCHEME); 8 <= in <=
 * AQLM_MAX_IN, in % 8 == 0, out <= AQLM_LISTS_MAX_OUT and out * in/8 <=
 * 2^32 - 1 (else AQLM_ERR_SHAPE).
 *
 * Layout (all device memory, 16-byte aligned, owned by the caller):
 *   rows form tiles of 64; the groups j of a row form J = ceil(G / 1024)
 *   blocks of Gb = ceil(G / J) groups (G = in / 8); for every unit
 *   u = (s * J + k) * ceil(out / 64) + rt (slice s < 8, block k, row tile
 *   rt), row 64 rt + l lists its codes c with c >> 13 == s and j in block k,
 *   ascending in j, as uint32 entries ((j - k Gb) << 13) | (c & 8191); the
 *   64 lists are padded to the longest, L, with Z << 13 (Z = Gb rounded up
 *   to a multiple of 64) and stored as entries[(off + t) * 64 + l].
 *   table: uint32 pairs (off, L) per unit, then the total number of steps
 *   (sum of L) as a uint64; entries take 256 bytes per step.
 *
 * Building: aqlm_lists_plan(codes, table) writes the table (asynchronous);
 * the caller reads the total (the uint64 at byte aqlm_lists_table_bytes - 8)
 * after synchronising, allocates total * 256 bytes of entries and calls
 * aqlm_lists_fill.  A fill or product whose entries_bytes is smaller than a
 * unit's off + L needs leaves that unit out (no access beyond entries_bytes);
 * a table that does not belong to the codes gives wrong results, never an
 * access outside the buffers.  The product needs a caller workspace of
 * aqlm_lists_workspace_bytes (fp32 partial sums, overwritten by every call;
 * calls that share a workspace must not run concurrently).
 *
 * Result: y = W x for batch 1 (batch 0 enqueues nothing), accumulated in
 * fp32, rounded to fp16 once; deterministic (the summation order is fixed by
 * out and in), but not bit-identical to aqlm_linear_gemv, which adds in
 * another order.
 */
#define AQLM_LISTS_MAX_OUT (1 << 30)

/* Bytes of the table of a layer (into *bytes). */
int aqlm_lists_table_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t* bytes);
/* Bytes of workspace aqlm_linear_gemv_lists needs for the shape (into *bytes). */
int aqlm_lists_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t* bytes);
/* Writes the table of codes [out][in/8] (int16) into table.  codes may be NULL when out == 0. */
int aqlm_lists_plan(const void* codes, void* table, int M, int B, int g, int64_t out, int64_t in, void* stream);
/* Writes the entries of codes, placed by table, into entries (entries_bytes long). */
int aqlm_lists_fill(const void* codes, const void* table, void* entries, int64_t entries_bytes, int M, int B, int g,
                    int64_t out, int64_t in, void* stream);
/* y[0][i] = sum_k W[i][k] x[0][k] over the slice lists (codebooks, scales, x, y as for aqlm_linear_gemv). */
int aqlm_linear_gemv_lists(const void* table, const void* entries, int64_t entries_bytes, const void* codebooks,
                           const void* scales, const void* x, void* y, void* workspace, int64_t workspace_bytes, int M,
                           int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);

/*
 * n_layers slice-list products that share x (q/k/v, gate/up) in one launch of
 * the product and one of the reduction: y_l = W_l x for l < n_layers, batch 1.
 * tables, entries, entries_bytes, codebooks, scales, outs and ys are HOST
 * arrays of n_layers entries (pointers in them are device pointers, laid out
 * as for aqlm_linear_gemv_lists); the library reads them during the call.
 * Each layer is validated as by aqlm_linear_gemv_lists; a layer with
 * outs[l] == 0 is skipped.  workspace (16-byte aligned) holds the layers'
 * partial sums one after another, each rounded up to 256 bytes:
 * aqlm_lists_fused_workspace_bytes gives its size.  Results are bit-identical to separate aqlm_linear_gemv_lists calls.
 * 1 <= n_layers <= AQLM_FUSED_MAX_LAYERS (else AQLM_ERR_SHAPE); a NULL array
 * gives AQLM_ERR_NULL.
 */
int aqlm_linear_gemv_lists_fused(int n_layers, const void* const* tables, const void* const* entries,
                                 const int64_t* entries_bytes, const void* const* codebooks, const void* const* scales,
                                 const int64_t* outs, const void* x, void* const* ys, void* workspace,
                                 int64_t workspace_bytes, int M, int B, int g, int64_t in, int64_t batch,
                                 void* stream);
/* Bytes of workspace aqlm_linear_gemv_lists_fused needs for the layers' outs (host array). */
int aqlm_lists_fused_workspace_bytes(int n_layers, const int64_t* outs, int M, int B, int g, int64_t in,
                                     int64_t* bytes);

/*
 * For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): aqlm_linear_gemv_lists
 * without the workspace argument.  The fp32 partial sums go to a static device
 * array of the library, AQLM_LISTS_NOALLOC_SCRATCH_BYTES long, that every GPU the
 * library runs on holds until the process ends; the call allocates and frees
 * nothing (its first call on a device looks the array's address up once).  A
 * layer whose partial sums (aqlm_lists_workspace_bytes) exceed the array gives
 * AQLM_ERR_SCRATCH and enqueues nothing; 4 MiB covers e.g. every Llama-2-7B and
 * 70B projection.  Every call on one GPU shares that GPU's array: calls that
 * overlap on one GPU (other streams, other host threads) race and must be
 * serialised by the caller.  Each call writes every partial it reads, so the
 * array needs no clearing between calls.  Other arguments, validation and
 * results are those of aqlm_linear_gemv_lists (bit-identical to it).
 */
#define AQLM_LISTS_NOALLOC_SCRATCH_BYTES (4 << 20)
int aqlm_linear_gemv_lists_noalloc(const void* table, const void* entries, int64_t entries_bytes,
                                   const void* codebooks, const void* scales, const void* x, void* y, int M, int B,
                                   int g, int64_t out, int64_t in, int64_t batch, void* stream);

/* ---------------------------------------------------------------------------
 * Fused products: what a feed-forward block does right after its quantized
 * projections, done before their results leave the kernel, and the gradients
 * of both with respect to their inputs and biases (the quantized weights are
 * frozen: codes, codebooks and scales get no gradient).
 *
 *   aqlm_linear_act           z = W x + bias;  y = act(z) + residual
 *   aqlm_gated                zg = Wg x + bg;  zu = Wu x + bu;  y = act(zg) * zu
 *   aqlm_linear_act_backward  dz = dy * act'(z);  dx = dz W;  dbias = sum_b dz[b]
 *   aqlm_gated_backward       dzg = dy * zu * act'(zg);  dzu = dy * act(zg);
 *                             dx = dzg Wg + dzu Wu;  dbias likewise
 *
 * act is one of aqlm_act; gelu is z (1 + erf(z / sqrt 2)) / 2, gelu_tanh its
 * tanh form z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2, silu is
 * z / (1 + exp(-z)).  relu's slope at 0 is 0.
 *
 * Arrays: codes, codebooks, scales, x as above, every scheme with codes in
 * whole bytes; bias [out] fp16; residual, z, y, dy [batch][out] fp16; x, dx
 * [batch][in] fp16; dbias [out] fp16.  bias, residual and z (forward) may be
 * NULL: no bias, no residual, the pre-activations not kept.  residual may be y
 * itself (the residual stream updated in place); no other arrays may overlap.
 * The gated calls take host arrays of two entries, gate then up, of one
 * scheme, out and in; their bias and z arrays may be NULL as a whole or per
 * entry.  bias and dbias need 2-byte alignment, everything else 16 bytes.
 *
 * Backward: z holds the pre-activations that the forward call kept; NULL for
 * aqlm_linear_act_backward with AQLM_ACT_NONE.  dbias NULL: not wanted (gated:
 * both or neither).  dx, dbias are overwritten, not added to.  out == 0 gives
 * dx = 0, batch == 0 gives dbias = 0 (sums over nothing).
 *
 * Sizes: 0 <= out <= AQLM_ACT_MAX_OUT, 1 <= in <= AQLM_MAX_IN, in % g == 0,
 * 0 <= batch <= 2^31 - 257, out * ceil(in / 64) * 8 < 2^32 and
 * out * (in / g) < 2^32 (else AQLM_ERR_SHAPE).  An activation outside aqlm_act
 * gives AQLM_ERR_ACT.
 *
 * Workspace: caller-owned device memory, 16-byte aligned, of at least the
 * bytes that the _workspace_bytes call of the same shape gives (0 for some
 * shapes: NULL is then accepted; an undersized one gives AQLM_ERR_SHAPE).  The
 * bytes of a larger batch of the same call, scheme, out and in are never
 * fewer, so a workspace for the largest batch serves every smaller one.  Its
 * contents on entry do not matter; calls that share it, captured graphs
 * included, must not run concurrently.
 *
 * Numerics: products are accumulated in fp32; bias, activation, gate and
 * residual are applied in fp32; y, and z where it is kept, are rounded to fp16
 * once, y from the unrounded z.  With M = 1 the codewords are multiplied as
 * they are and the row scale is applied in fp32.  With M > 1 a weight is
 * rounded to fp16 once at most:
 *   - batch 1..16, 2x8 up to 512 tokens (gated: 384) and 4x8 g16 up to 320
 *     (gated: 256): not at all (codewords multiplied one by one; the general
 *     schemes decode in fp32; layers of fewer than 64 weights: batch 1..16 only);
 *   - else the decoded weight that aqlm_linear_decode gives.
 * Backward, small batches (2x8 to 256 tokens, 1x16 and 4x8 g16 to 128) multiply
 * the codewords as they are, one by one, by dz times the row's scale.  Larger
 * ones do so for M = 1 and multiply the decoded weights by dz for M > 1; with
 * AQLM_ACT_NONE, one layer and out % 64 == 0 they multiply the decoded weights
 * by dy as it is, for every M.  dz, times the scale where it takes it, is
 * rounded to fp16 once, in units of a power of two per token and 512 rows that
 * its largest finite value in them fixes, so that it does not leave fp16's
 * range: elements down to 2^-9 of the token's largest keep all their bits,
 * smaller ones are off by at most 2^-19 of it.  dbias sums the fp32 values in
 * a fixed order.  Decoded weights beyond fp16's range are infinite, and those
 * below 2^-14 lose bits; non-finite values reach the outputs that they take
 * part in and no others.  Results are deterministic.
 */
typedef enum {
    AQLM_ACT_NONE = 0,
    AQLM_ACT_RELU = 1,
    AQLM_ACT_SILU = 2,
    AQLM_ACT_GELU = 3,
    AQLM_ACT_GELU_TANH = 4
} aqlm_act;

/* Largest out of the fused products. */
#define AQLM_ACT_MAX_OUT (1 << 24)

int aqlm_linear_act_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes);
int aqlm_linear_act(const void* codes, const void* codebooks, const void* scales, const void* x, const void* bias,
                    const void* residual, void* z, void* y, void* workspace, int64_t workspace_bytes, int act, int M,
                    int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);

int aqlm_gated_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes);
int aqlm_gated(const void* const* codes, const void* const* codebooks, const void* const* scales, const void* x,
               const void* const* bias, void* const* z, void* y, void* workspace, int64_t workspace_bytes, int act,
               int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);

int aqlm_linear_act_backward_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch,
                                             int64_t* bytes);
int aqlm_linear_act_backward(const void* codes, const void* codebooks, const void* scales, const void* dy,
                             const void* z, void* dx, void* dbias, void* workspace, int64_t workspace_bytes, int act,
                             int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream);

int aqlm_gated_backward_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes);
int aqlm_gated_backward(const void* const* codes, const void* const* codebooks, const void* const* scales,
                        const void* dy, const void* const* z, void* dx, void* const* dbias, void* workspace,
                        int64_t workspace_bytes, int act, int M, int B, int g, int64_t out, int64_t in, int64_t batch,
                        void* stream);

/*
 * The forward calls over slice lists (1x16, batch 0 or 1): table, entries and
 * entries_bytes as for aqlm_linear_gemv_lists, workspace of
 * aqlm_lists_fused_workspace_bytes for one layer, or for two of the same out.
 * The epilogue runs in the reduction of the partial sums; numerics otherwise
 * as aqlm_linear_gemv_lists.
 */
int aqlm_linear_act_lists(const void* table, const void* entries, int64_t entries_bytes, const void* codebooks,
                          const void* scales, const void* x, const void* bias, const void* residual, void* z, void* y,
                          void* workspace, int64_t workspace_bytes, int act, int M, int B, int g, int64_t out,
                          int64_t in, int64_t batch, void* stream);
int aqlm_gated_lists(const void* const* tables, const void* const* entries, const int64_t* entries_bytes,
                     const void* const* codebooks, const void* const* scales, const void* x, const void* const* bias,
                     void* const* z, void* y, void* workspace, int64_t workspace_bytes, int act, int M, int B, int g,
                     int64_t out, int64_t in, int64_t batch, void* stream);

/* ---------------------------------------------------------------------------
 * MX4: layers in microscaled 4-bit floating point (4.25 bits per weight), the
 * format that the matrix cores multiply as it is stored.  For the layers that
 * a 2-bit model keeps at more bits, and for products with 4-bit activations.
 *
 *   aqlm_mx4_quantize  fp16 rows [rows][in] to codes and scales
 *   aqlm_mx4_decode    and back: W16 [rows][in]
 *   aqlm_mx4_linear    y = act(W x + bias) + residual, x in fp16 or in MX4
 *
 * A row is cut into blocks of 32 consecutive values.  Value i of block b is
 * q 2^(s[b] - 127): q, one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, is a 4-bit float
 * (sign, two exponent bits of bias 1, one mantissa bit), s the block's scale
 * byte (255: the block is NaN).
 *   codes   [rows][in / 2]   uint8, value 2i in the low half of byte i
 *   scales  [rows][in / 32]  uint8
 * in % 32 == 0, 32 <= in <= AQLM_MAX_IN.  codes, fp16 arrays: 16-byte aligned,
 * bias 2-byte, scales at any address.
 *
 * Quantization: 2^(s - 127) = 2^(floor(log2 max |v|) - 2) over the block;
 * v / 2^(s - 127) is rounded to nearest (ties to even) and is 6 at most.  A
 * block of zeros has s = 0, one that holds an infinity or NaN s = 255 and
 * codes 0.  Decoding rounds q 2^(s - 127) to fp16 once (nearest even, 0 and
 * infinity where it leaves fp16's range); what aqlm_mx4_quantize wrote is
 * decoded without rounding.  rows == 0 enqueues nothing.
 *
 * aqlm_mx4_linear: x_scales NULL: x is fp16 [batch][in]; else x holds MX4
 * codes [batch][in / 2] and x_scales their scales [batch][in / 32].  bias [out]
 * and residual [batch][out] fp16 may be NULL; residual may be y itself; no
 * other arrays may overlap.  act is one of aqlm_act.  0 <= out <=
 * AQLM_ACT_MAX_OUT, 0 <= batch <= AQLM_MX4_MAX_BATCH, fewer than 2^31 tiles
 * of 128 outputs x 128 tokens (else AQLM_ERR_SHAPE).
 * out == 0 or batch == 0 enqueues nothing.  Workspace: as for the fused
 * products above, of aqlm_mx4_linear_workspace_bytes bytes (x_mx4: whether x
 * is in MX4); a larger batch never needs fewer.
 *
 * Numerics: neither weights nor activations are rounded.  Products are
 * accumulated in fp32; bias, activation and residual are applied in fp32 and y
 * is rounded to fp16 once.  Next to fp16 activations a weight block of scale 0
 * counts as zero, and blocks of scales outside 104..140 (0.5 2^-23 to 6 2^13:
 * quantized blocks whose largest value is below 2^-21, or foreign ones) cost
 * up to ten times the time of others.  A block of x with an infinity or NaN makes its
 * token's outputs NaN, a weight block of scale 255 its row's; non-finite bias and
 * residual values reach the outputs that they take part in.  Results are
 * deterministic.
 */
#define AQLM_MX4_MAX_BATCH (1 << 30)

int aqlm_mx4_quantize(const void* w, void* codes, void* scales, int64_t rows, int64_t in, void* stream);
int aqlm_mx4_decode(const void* codes, const void* scales, void* w, int64_t rows, int64_t in, void* stream);
int aqlm_mx4_linear_workspace_bytes(int x_mx4, int64_t out, int64_t in, int64_t batch, int64_t* bytes);
int aqlm_mx4_linear(const void* codes, const void* scales, const void* x, const void* x_scales, const void* bias,
                    const void* residual, void* y, void* workspace, int64_t workspace_bytes, int act, int64_t out,
                    int64_t in, int64_t batch, void* stream);

/* ---------------------------------------------------------------------------
 * Mixture of experts, for serving: the router, and a whole layer for few
 * tokens.
 *
 *   aqlm_moe_route    l = x R^T;  scores, the k experts of every token and
 *                     their weights
 *   aqlm_moe          y_t = residual_t
 *   aqlm_moe_mx4            + sum_{j<k} w_tj Wd_e (act(Wg_e x_t) * (Wu_e x_t)),
 *                     e = ids_tj
 *
 * aqlm_moe_route: x [tokens][in], router R [experts][in] fp16; ids
 * [tokens][k] int32 and weights [tokens][k] fp32 are written, best expert
 * first.  Scores: softmax of a token's logits, or 1 / (1 + exp(-l)) of each.
 * The experts are those of the k largest scores, plus bias [experts] (fp32,
 * or NULL) where it is given; equal ones: the lowest index first.  weights are
 * the scores without the bias, divided by their sum over the k when renorm is
 * not 0, times scale.  in % 8 == 0, k <= experts, 0 <= tokens <=
 * AQLM_ROUTE_MAX_TOKENS.  The choice is the one of logits and scores in 64
 * bits (softmax scores without a bias: of the logits) and does not depend on
 * the batch.  So are the weights, except where
 * tokens * experts * in >= 2^29 (and no softmax with a bias): there they come
 * from logits with sums of 64 products in fp32, added in 64 bits, off by at
 * most 2^-17 |x| |R_e| and usually by about 2^-22.  A NaN score ranks below all
 * others; a token with a NaN logit has NaN weights under softmax.
 *
 * aqlm_moe: the experts' layers in one AQLM scheme, three host arrays of three
 * entries (gate, up, down), each stacked over the experts: codes
 * [experts][rows][n/g][M], codebooks [experts][M][2^B][g], scales
 * [experts][rows], for gate and up rows = inner, n = in, for down rows = in,
 * n = inner.  aqlm_moe_mx4: the same in MX4, codes [experts][rows][n / 2],
 * scales [experts][rows][n / 32].  x, y, residual [tokens][in] fp16 (residual
 * may be NULL, or y itself; no other arrays may overlap), ids, weights as
 * aqlm_moe_route writes them.  A token may name an expert twice, and an id
 * that is no expert (-1, say) adds nothing.  in and inner are multiples of g
 * (MX4: 32), 0 <= tokens, tokens * k <= AQLM_MOE_MAX_PAIRS.  Larger batches:
 * sort the tokens by expert and use the products above.
 *
 * Codes, codebooks, x, y, residual and workspace need 16-byte alignment, AQLM
 * scales 2, ids, weights and bias 4, MX4 scales none.  Workspaces as for the
 * fused products above.
 *
 * Numerics: aqlm_moe multiplies every codeword on its own (no weight is
 * rounded), aqlm_moe_mx4 as aqlm_mx4_linear.  The hidden vector
 * act(.) * (.) is kept to 2^-22 of each element or 2^-28, whichever is larger
 * (infinite beyond 2^8 * 65504).  Sums are fp32, over a token's choices in their
 * order; y is rounded to fp16 once.  Results are deterministic.
 */
#define AQLM_MOE_MAX_EXPERTS 512
#define AQLM_MOE_MAX_K 16
#define AQLM_MOE_MAX_PAIRS 1024
#define AQLM_ROUTE_MAX_TOKENS (1 << 24)

typedef enum {
    AQLM_SCORE_SOFTMAX = 0,
    AQLM_SCORE_SIGMOID = 1
} aqlm_score;

int aqlm_moe_route_workspace_bytes(int64_t experts, int64_t in, int64_t k, int64_t tokens, int64_t* bytes);
/* score: one of aqlm_score (else AQLM_ERR_ACT). */
int aqlm_moe_route(const void* x, const void* router, const float* bias, int32_t* ids, float* weights, void* workspace,
                   int64_t workspace_bytes, int score, int renorm, float scale, int64_t experts, int64_t in, int64_t k,
                   int64_t tokens, void* stream);

int aqlm_moe_workspace_bytes(int M, int B, int g, int64_t experts, int64_t in, int64_t inner, int64_t k, int64_t tokens,
                             int64_t* bytes);
int aqlm_moe(const void* const* codes, const void* const* codebooks, const void* const* scales, const void* x,
             const int32_t* ids, const float* weights, const void* residual, void* y, void* workspace,
             int64_t workspace_bytes, int act, int M, int B, int g, int64_t experts, int64_t in, int64_t inner, int64_t k,
             int64_t tokens, void* stream);

int aqlm_moe_mx4_workspace_bytes(int64_t experts, int64_t in, int64_t inner, int64_t k, int64_t tokens, int64_t* bytes);
int aqlm_moe_mx4(const void* const* codes, const void* const* scales, const void* x, const int32_t* ids,
                 const float* weights, const void* residual, void* y, void* workspace, int64_t workspace_bytes, int act,
                 int64_t experts, int64_t in, int64_t inner, int64_t k, int64_t tokens, void* stream);

/* Static, human-readable name of a status code. */
const char* aqlm_status_str(int status);

/* hipError_t of the calling thread's last AQLM_ERR_HIP (0 if none). */
int aqlm_last_hip_error(void);

/* Library version, e.g. "0.1.0". */
const char* aqlm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* AQLM_H */
