/*
 * exl3.h — C ABI of libexl3.so, a single-GPU (sm_103a) implementation of the
 * EXL3-style trellis-quantized linear layer
 *
 *     y = had_r_128( had_r_128(x * su) . W ) * sv
 *
 * Sources of the operations (page title, section):
 *   [P1] vLLM PR #316, "[EXL3] dispatch prefill-shaped GEMMs to
 *        reconstruct+hgemm (+113 % prefill, decode unchanged)": sections
 *        "Problem", "Kernel measurements", "Change".
 *   [P2] vLLM PR #314, "[EXL3] allow CUDA-graph decode for dense checkpoints
 *        by priming exl3_gemm autotune": sections "Problem", "Change".
 *   [P3] pegainfer PR #1046, "perf(qwen35): align the logits GEMM width so
 *        the output projection stops landing on an align-1 sm_75 kernel":
 *        sections "Summary", "Review follow-ups", "Testing".
 *
 * Storage format of W (the pages leave it open; this library fixes it):
 *   W is K x n_stored. It is stored as 16x16 tiles ordered row-major over
 *   (k/16, n/16), weights row-major inside a tile. Tile t owns 16*bits
 *   little-endian uint16 words at trellis[t*16*bits ...], a circular stream
 *   of 256*bits bits read MSB-first inside each word. Weight i of a tile
 *   has as its 16-bit state the circular window of stream bits ending at bit
 *   (i+1)*bits-1 (earliest bit = most significant). Its value is
 *       u = state*89226354 + 64248484 (mod 2^32)
 *       u = (u & 0x8FFF8FFF) ^ 0x3B603B60
 *       w = RNE_fp16( fp32(fp16 bits u[15:0]) + fp32(fp16 bits u[31:16]) ).
 *   had_r_128 is the orthonormal 128-point Walsh-Hadamard transform in
 *   natural (Sylvester) order, H[i][j] = (-1)^popcount(i&j) / sqrt(128),
 *   applied to every 128-wide block.
 *
 * General conventions:
 *   - Every data pointer is a caller-owned DEVICE pointer that must be
 *     16-byte aligned. The library never allocates or frees device memory
 *     and never synchronizes a stream except in exl3_get_device_status.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).
 *   - Matrices are row-major and densely packed unless a leading dimension
 *     is stated.
 *   - Arguments are validated before anything is launched; a rejected call
 *     launches nothing and returns the named status. A failed launch
 *     returns EXL3_ERR_CUDA.
 *   - exl3_init(device) must run once per device, with that device
 *     current, before any other call that touches it and before any CUDA
 *     graph capture: it loads every kernel and sets their attributes, so
 *     no later call loads modules, allocates or queries the device.
 *   - Consecutive kernels of one call overlap their launches through
 *     programmatic dependent launch; each waits for its predecessor before
 *     touching memory it shares with it. The last kernel of a call lets the
 *     next kernel in the stream begin early as well: a caller kernel that
 *     opts into programmatic stream serialization must, as that contract
 *     requires, wait on its grid dependency (cudaGridDependencySynchronize)
 *     before reading this call's outputs. Ordinary launches are unaffected.
 *   - Supported trellis widths: bits in 1..8.
 *   - Shapes: K % 128 == 0, K <= 131072, n_gemm % 128 == 0,
 *     n_gemm <= n_stored, n_stored % 128 == 0, n_stored <= 2^24; others
 *     return EXL3_ERR_INVALID_ARG.
 */
#ifndef EXL3_H_
#define EXL3_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EXL3_OK = 0,
    EXL3_ERR_INVALID_ARG = 1,        /* a shape, size or enum is out of range */
    EXL3_ERR_ALIGNMENT = 2,          /* a pointer is NULL or not 16-byte aligned */
    EXL3_ERR_UNSUPPORTED_BITS = 3,   /* bits is not a supported trellis width */
    EXL3_ERR_WORKSPACE_TOO_SMALL = 4,/* workspace_bytes below the required size */
    EXL3_ERR_NOT_INITIALIZED = 5,    /* exl3_init was not called for the current device */
    EXL3_ERR_CUDA = 6,               /* a CUDA runtime call or a launch failed */
    EXL3_ERR_DEVICE_TIMEOUT = 7,     /* a kernel gave up a bounded wait (see exl3_get_device_status) */
    EXL3_ERR_NOALLOC_TOO_LARGE = 8,  /* the problem needs more scratch than the fixed no-alloc buffer holds */
    EXL3_ERR_OUT_OF_BOUNDS = 9,      /* bounds-checked build only: a kernel's index left its buffer */
    EXL3_ERR_DEVICE_INDEX = 10       /* a page number, length or row range read on the device is out of range */
} exl3_status;

typedef enum { EXL3_F16 = 0, EXL3_F32 = 1 } exl3_dtype;

/* Layout of a reconstructed weight slice. */
typedef enum {
    EXL3_LAYOUT_KN = 0, /* w[k][j] = W[k][n0+j], K rows of n_cols, ld = n_cols */
    EXL3_LAYOUT_NK = 1  /* w[j][k] = W[k][n0+j], n_cols rows of K, ld = K (GEMM operand layout) */
} exl3_layout;

/* Columns reconstructed per prefill chunk; bounds the scratch at
 * 32768*K*2 bytes ([P1] "Change": 336 MB at K = 5120). */
#define EXL3_RECONSTRUCT_CHUNK_COLS 32768

/*
 * exl3_init: one-time set-up for `device` (made current by this call).
 * Loads all kernels, raises their shared-memory limits and caches the SM
 * count. Idempotent. Call before any stream capture ([P2] "Change": every
 * lazy initialisation must happen before capture).
 * Errors: EXL3_ERR_INVALID_ARG (no such device), EXL3_ERR_CUDA.
 */
exl3_status exl3_init(int device);

/* Static English text for a status code (never NULL). */
const char *exl3_status_string(int status);

/* 1 if `bits` is a supported trellis width, else 0. Host only. */
int exl3_supported_bits(int bits);

/*
 * Logits GEMM width for an odd decodable vocabulary: n_decodable rounded up
 * to a multiple of 128, clamped to n_stored ([P3] "Summary": 248077 ->
 * 248192 <= 248320). Returns -1 on invalid input. Host only.
 */
int64_t exl3_aligned_logits_width(int64_t n_decodable, int64_t n_stored);

/*
 * The decode-shaped path's work split for a (K, n_gemm) geometry on a GPU
 * with `num_sms` SMs, for calls of at most 8 rows: the whole (128-column
 * n-block x 16-row k slab) space is cut into equal contiguous ranges, one
 * per warp (stream-K); *splits receives the largest number of warps that
 * share one n-block (its partial-sum slots) and *ctas_per_split the number
 * of CTAs launched. Returns 0, or -1 on invalid input. Host only.
 */
int exl3_decode_plan(int64_t K, int64_t n_gemm, int num_sms, int *splits, int *ctas_per_split);

/*
 * The kernels a prefill-shaped call (m_threshold > 0 and M >= m_threshold)
 * of M rows takes on a layer n_gemm columns wide, on a GPU with `num_sms`
 * SMs: 1 for the fused prefill kernel, whose producer warps decode the
 * trellis straight into the tensor-core operand (the "dequant fused into
 * the GEMM" of [P1] "The remaining gap is structural"), used for
 * M <= 512 on layers with at least 0.3 x num_sms column blocks of 256; 0 for
 * reconstruct (32768-column chunks) followed by the tensor-core GEMM.
 * Both apply the input and output rotations, sv and the logits mask.
 * Returns -1 on invalid input (M < 1, n_gemm not a positive multiple of
 * 128, num_sms < 1). Host only.
 */
int exl3_prefill_path(int64_t M, int64_t n_gemm, int num_sms);

/*
 * Workspace bytes an exl3_linear / exl3_logits_masked call with M <= M_max
 * needs on a GPU with `num_sms` streaming multiprocessors. The workspace is
 * laid out as: split-K partial sums (shared by the decode-shaped kernels
 * and, when a prefill-shaped call is possible, the prefill GEMM's split
 * tail tiles: at most 3 x num_sms fp32 128 x 256 tiles) and rotated
 * activations; then, when a prefill-shaped call is possible (m_threshold > 0
 * and M_max >= m_threshold), the rotated activations (M_max x K fp16) and
 * one reconstruct chunk (min(n_gemm, 32768) x K fp16) ([P1] "Change": one
 * scratch per geometry, reused by every layer of that geometry on one
 * stream). Returns 0 for invalid arguments. Host only.
 */
size_t exl3_linear_workspace_bytes_for(int64_t M_max, int64_t K, int64_t n_gemm, int bits,
                                       int64_t m_threshold, int num_sms);

/* Same, for the current device's SM count (queried, not allocated). */
size_t exl3_linear_workspace_bytes(int64_t M_max, int64_t K, int64_t n_gemm, int bits,
                                   int64_t m_threshold);

/*
 * Clears a workspace (cudaMemsetAsync on `stream`). Optional: no call needs
 * particular initial workspace contents; it only makes a fresh buffer's
 * contents defined.
 */
exl3_status exl3_workspace_init(void *workspace, size_t workspace_bytes, void *stream);

/*
 * exl3_hadamard128: y = RNE_fp16( had_r_128(x * pre_scale) ) on every
 * 128-block of each row ([P1] "Kernel measurements": the had_r_128 stage).
 *   x, y:       rows x cols fp16 (may alias for an in-place transform).
 *   pre_scale:  cols fp16, or NULL for none (su of the layer).
 *   cols % 128 == 0, rows >= 0.
 * Arithmetic: fp32, butterfly stages h = 1, 2, 4, ..., 64, then one multiply
 * by fp32(1/sqrt(128)), then round to nearest even.
 */
exl3_status exl3_hadamard128(const void *x, void *y, const void *pre_scale, int64_t rows,
                             int64_t cols, void *stream);

/*
 * exl3_reconstruct: decode columns [n0, n0+n_cols) of W from the trellis
 * ([P1] "Kernel measurements", "Change": reconstruct / reconstruct_slice).
 *   trellis: tiles of the K x n_stored matrix (format above), uint16.
 *   w:       fp16 output in `layout` (exl3_layout).
 *   n0 % 128 == 0, n_cols % 128 == 0, n0 + n_cols <= n_stored.
 * Output is bit-exact with the format definition.
 */
exl3_status exl3_reconstruct(const uint16_t *trellis, int bits, int64_t K, int64_t n_stored,
                             int64_t n0, int64_t n_cols, void *w, int layout, void *stream);

/*
 * Weight-side rotation variant ([P1] "Kernel measurements":
 * reconstruct_had_slice). Moves both rotations and both scales onto the
 * weight, W' = diag(su) . had_r_128(K) . W . had_r_128(N) . diag(sv), so the
 * prefill-shaped layer is the plain product y = x . W'. The pages give no
 * arithmetic for it; this library defines it per 128 x 128 block of W as
 * fp32(w) -> fast WHT of each column along k (fp32, stages h = 1 .. 64)
 * -> * fp32(su[k]) -> fast WHT of each row along n -> * 2^-7 (exact)
 * -> * fp32(sv[n]) -> round to nearest even fp16, and the output is
 * bit-exact with that definition.
 *
 * exl3_reconstruct_rotated: columns [n0, n0+n_cols) of W' into `w`
 *   (fp16, `layout` as exl3_reconstruct); su: K fp16, sv: n_stored fp16.
 *   K % 128 == 0, n0 % 128 == 0, n_cols % 128 == 0, n0 + n_cols <= n_stored.
 *
 * exl3_weight_rotated_workspace_bytes: scratch for
 *   exl3_linear_weight_rotated (one 32768-column W'^T slice), 0 if invalid.
 *
 * exl3_linear_weight_rotated: y = x . W'[:, :n_gemm], reconstructing W' in
 *   32768-column slices into the caller's workspace and running the
 *   tensor-core GEMM without input or output rotation. x: M x K fp16 (not
 *   rotated); y: M x n_gemm (`y_dtype`), ld = n_gemm; fp32 accumulation.
 *   It differs from exl3_linear by where the fp16 roundings fall (W' instead
 *   of x'): max|y - y_linear| / rms(y_linear) stays below 3e-3.
 *   Errors as exl3_linear (EXL3_ERR_WORKSPACE_TOO_SMALL below the size above).
 */
exl3_status exl3_reconstruct_rotated(const uint16_t *trellis, int bits, int64_t K, int64_t n_stored,
                                     int64_t n0, int64_t n_cols, const void *su, const void *sv, void *w,
                                     int layout, void *stream);
size_t exl3_weight_rotated_workspace_bytes(int64_t K, int64_t n_gemm);
exl3_status exl3_linear_weight_rotated(const void *x, int64_t M, int64_t K, const uint16_t *trellis, int bits,
                                       int64_t n_stored, int64_t n_gemm, const void *su, const void *sv, void *y,
                                       int y_dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * exl3_linear: y = had_r_128( RNE_fp16(had_r_128(x * su)) . W[:, :n_gemm] )
 *                  * sv[:n_gemm]
 *   x:     M x K fp16.            su: K fp16.         sv: n_stored fp16.
 *   y:     M x n_gemm, `y_dtype` (EXL3_F32 or EXL3_F16 = RNE of the fp32
 *          result), ld = n_gemm.
 *   m_threshold: path choice made inside this call on its own M ([P1]
 *          "Change": the dispatch must live inside the op, not in a branch
 *          a tracer can freeze). M < m_threshold, or m_threshold == 0,
 *          takes the decode-shaped path, where the trellis is decoded
 *          inside the GEMM and never materialised: for M <= 16 a stream-K
 *          kernel with the decoded weights as the mma.sync operand; for
 *          larger M one tensor-core (tcgen05) kernel per 256 rows whose
 *          producer warps decode straight into the MMA operand buffers.
 *          Otherwise the prefill-shaped path runs had_r_128, then either
 *          (M <= 512 on a layer with at least 0.3 x SMs column blocks of
 *          256) one fused tensor-core kernel whose producer warps decode
 *          straight into the MMA operand, 512 rows per decoded tile, or
 *          reconstruct (32768-column chunks into the workspace) followed by
 *          a tensor-core GEMM; both apply the output rotation, sv and the
 *          mask in their epilogue. On one GB300 the prefill-shaped path is
 *          faster from M = 384 (4-bit 5120 -> 17408) and from M = 768
 *          (4-bit 17408 -> 5120).
 *   workspace: device buffer of at least
 *          exl3_linear_workspace_bytes(M, K, n_gemm, bits, m_threshold)
 *          bytes, cleared once by exl3_workspace_init. Calls that share a
 *          workspace must be ordered (same stream, or synchronised).
 * Accumulation is fp32. M == 0 is a no-op.
 */
exl3_status exl3_linear(const void *x, int64_t M, int64_t K, const uint16_t *trellis, int bits,
                        int64_t n_stored, int64_t n_gemm, const void *su, const void *sv, void *y,
                        int y_dtype, int64_t m_threshold, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * exl3_logits_masked: the logits projection with the pad mask and greedy
 * selection fused behind one entry point, so the GEMM cannot be reached
 * without the mask ([P3] "Review follow-ups": output_logits_into owns both).
 *   logits: M x n_gemm fp32 (ld = n_gemm), = exl3_linear's fp32 output with
 *           columns [n_decodable, n_gemm) forced to -inf.
 *   argmax: M int32, the first index of each row's maximum.
 *   1 <= n_decodable <= n_gemm. Other arguments as exl3_linear.
 */
exl3_status exl3_logits_masked(const void *x, int64_t M, int64_t K, const uint16_t *trellis,
                               int bits, int64_t n_stored, int64_t n_gemm, int64_t n_decodable,
                               const void *su, const void *sv, float *logits, int32_t *argmax,
                               int64_t m_threshold, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word, which holds the first device-side error since the last read:
 * EXL3_ERR_DEVICE_TIMEOUT if a kernel gave up one of its bounded waits,
 * EXL3_ERR_OUT_OF_BOUNDS if a check of the bounds-checked build failed,
 * EXL3_ERR_DEVICE_INDEX if a serving call met a page number, length or row
 * range on the device that its buffers do not hold (it was not followed; the
 * call's outputs for that sequence are undefined); EXL3_OK otherwise.
 * The word is one per device, shared by every stream and workspace on it
 * (some entry points that wait on the device have no workspace): with
 * several streams, a timeout is reported to whichever caller reads first.
 */
exl3_status exl3_get_device_status(void *stream);

/*
 * exl3_silu_mul: out = RNE_fp16(silu(gate) * up) elementwise (fp32 math,
 * silu(a) = a / (1 + exp(-a))), n % 8 == 0. The glue between the gate/up
 * and down projections of a dense MLP ([P1] follow-up comment: gate + up +
 * down per layer); not itself part of the trellis layer.
 */
exl3_status exl3_silu_mul(const void *gate, const void *up, void *out, int64_t n, void *stream);

/*
 * Self-test of the failure-detection path: launches one kernel that waits
 * on a barrier nothing will complete, gives up after limit_us microseconds
 * (1 .. 2,000,000) and records EXL3_ERR_DEVICE_TIMEOUT in the device error
 * word, which exl3_get_device_status then returns. The kernel always
 * returns on its own; it neither traps nor faults. The pages have no
 * counterpart; it exercises the bounded waits every pipelined kernel uses.
 */
exl3_status exl3_selftest_wait_timeout(uint32_t limit_us, void *stream);

/*
 * Bounds-checked build. The same sources compiled with EXL3_DEBUG_BOUNDS=1
 * give libexl3_bounds.so, with the same entry points. Before each access,
 * its kernels check against the extents implied by the launch's arguments:
 *   - every computed global index;
 *   - every shared-memory address and mbarrier;
 *   - every TMA coordinate and bulk-copy span;
 *   - every TMEM column.
 * A failed check skips the access (a load reads zero) and records
 * EXL3_ERR_OUT_OF_BOUNDS in the device error word. It also prints the
 * source line once. The check stands in for a memory checker; the pages
 * have no counterpart to it.
 *
 * exl3_bounds_checked: 1 in the bounds-checked library, 0 in libexl3.so.
 * Host only.
 *
 * exl3_selftest_bounds: checks that every kernel translation unit of the
 * bounds-checked build reports to the device error word. It launches one
 * probe kernel per unit, on `stream`. Each probe submits an index equal to
 * its extent to the checks and touches no memory. After each probe the
 * word is read and cleared.
 *   *units_total   receives the number of units probed.
 *   *units_reported receives how many recorded EXL3_ERR_OUT_OF_BOUNDS.
 * In libexl3.so it launches nothing and sets both to 0.
 * An error already pending in the word is returned (and cleared) before
 * any probe runs.
 * Synchronises `stream`.
 * Errors: EXL3_ERR_INVALID_ARG (NULL pointer), EXL3_ERR_NOT_INITIALIZED,
 * EXL3_ERR_CUDA.
 */
int exl3_bounds_checked(void);
exl3_status exl3_selftest_bounds(int *units_reported, int *units_total, void *stream);

/*
 * exl3_linear_decode_noalloc: the decode-shaped linear layer for callers
 * that cannot allocate device memory: a
 * plugin inside a host program that owns every device buffer, or code that
 * must not call cudaMalloc at run time because it synchronises the whole
 * device. The caller passes only inputs and outputs; the split-K partial
 * sums and rotated activations live in a fixed 24 MiB buffer inside the
 * library (a static device array that every GPU which loads libexl3.so
 * keeps until the process exits). The pages have no counterpart to this
 * entry point.
 *   Arguments as exl3_linear, without m_threshold and workspace; the same
 *   shape, row-count, bit-width and alignment rules, with the same status
 *   codes.
 *   Kernels: the rows run in groups of up to 16 through the 16-row
 *   decode-shaped kernel (exactly what exl3_linear runs for M <= 16). For
 *   M > 16 exl3_linear switches to its tensor-core kernel, which needs a
 *   rotated copy of all M rows in the workspace; this entry point instead
 *   repeats the 16-row kernel ceil(M/16) times, so its cost grows about
 *   ceil(M/16)-fold over the M = 16 call (results agree with exl3_linear
 *   within the layer tolerance, not bit for bit).
 *   Limit: exl3_linear_workspace_bytes(16, K, n_gemm, bits, 0) must not
 *   exceed EXL3_NOALLOC_SCRATCH_BYTES (24 MiB; the MLP projections fit, a
 *   248192-wide logits layer does not); larger problems return
 *   EXL3_ERR_NOALLOC_TOO_LARGE and launch nothing.
 *   The first call on a device looks up the buffer's device address, so
 *   make that first call before any stream capture. No call needs the
 *   buffer to start at zero. Every call shares the one buffer
 *   and it keeps the last call's contents, so calls that may overlap on the
 *   GPU (different streams, no ordering) race: order them. It never calls
 *   cudaMalloc, cudaFree or any allocating routine. exl3_init must have run.
 */
#define EXL3_NOALLOC_SCRATCH_BYTES ((size_t)24 << 20)
exl3_status exl3_linear_decode_noalloc(const void *x, int64_t M, int64_t K, const uint16_t *trellis,
                                       int bits, int64_t n_stored, int64_t n_gemm, const void *su,
                                       const void *sv, void *y, int y_dtype, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Serving operators: what a decode step needs between the projections (an
 * 8-bit paged key/value cache and the attention that reads it) and after the
 * logits (penalties, biases and a grammar mask before a token is chosen).
 * Everything sizes depend on per step (lengths, rows of each sequence, page
 * numbers) lives on the device, so a captured graph serves every step whose
 * bounds (rows, max_rows, max_pages) it was captured with.
 * ---------------------------------------------------------------------------
 *
 * Matrices (codes, q, k, v, out, logits) and `weight` are 16-byte aligned;
 * scales, lse and integer arrays by their elements (4 bytes). A NULL or
 * misaligned pointer returns EXL3_ERR_ALIGNMENT, except in a call without rows
 * (or, to evict, without sequences), which does nothing and looks at none.
 *
 * The cache holds E4M3 codes in blocks (pages) of 64 tokens. A block holds,
 * for each key/value head, 64 x head_dim codes and ONE scale, a power of two;
 * keys and values have blocks of the same number in two buffers:
 *     value[page][head][token][d] = code * scale[page][head].
 * A block's scale is 2^e, e the smallest integer in -32 .. 8 with
 * max |x| <= 448 * 2^e over the finite values it holds (448 is E4M3's largest
 * value; every finite fp16 fits), and never smaller than it was while the
 * block held older tokens. Powers of two make a change of scale exact except
 * where a code becomes subnormal.
 */
#define EXL3_KV8_BLOCK 64

typedef struct {
    void *k, *v;             /* E4M3, n_pages x n_kv_heads x 64 x head_dim */
    float *k_scale, *v_scale;/* n_pages x n_kv_heads */
    float *weight;           /* n_pages x n_kv_heads x 64: accumulated attention weight, or NULL */
    int64_t n_pages;         /* at least 1; n_pages * n_kv_heads * 64 < 2^31 */
    int32_t n_kv_heads;      /* 1 .. 1024 */
    int32_t head_dim;        /* 64 or 128 */
} exl3_kv8_cache;

/*
 * The sequences of one call. Row r of a call's q / k / v matrices belongs to
 * the sequence s with q_start[s] <= r < q_start[s + 1]; its rows are the last
 * tokens of the sequence: row q_start[s] + i stands at position
 * kv_len[s] - (q_start[s + 1] - q_start[s]) + i. kv_len counts this call's
 * own tokens too.
 */
typedef struct {
    const int32_t *page_table; /* n_seqs x max_pages: page of tokens 64 j .. 64 j + 63 of a sequence */
    const int32_t *kv_len;     /* n_seqs, each at most 64 * max_pages */
    const int32_t *q_start;    /* n_seqs + 1, not decreasing, from 0 to rows */
    int32_t n_seqs;            /* 0 .. 65535 */
    int32_t max_pages;
    int32_t rows;              /* rows of this call, all sequences */
    int32_t max_rows;          /* the most rows that one sequence has */
} exl3_kv8_batch;

/*
 * exl3_kv8_append: quantizes this call's keys and values into the cache.
 *   k, v: rows x (n_kv_heads * head_dim) fp16, leading dimensions ldk, ldv
 *         (elements, multiples of 8, at least the width): column ranges of
 *         one fused projection's output will do.
 * Each block that receives tokens gets the scale above. Where it grows, the
 * older tokens' codes are rescaled, E4M3(code * 2^(e_old - e)); new codes are
 * E4M3(x * 2^-e), both rounded to nearest even. New tokens before position 0
 * (kv_len below the sequence's rows) are dropped and recorded as
 * EXL3_ERR_DEVICE_INDEX. Infinities saturate at
 * +-448 * 2^e; NaN is stored as NaN (E4M3 has one) and takes no part in the
 * scale. Slots past a sequence's length keep what they held. The cache's
 * `weight` of the new tokens is set to 0 where the cache has one.
 * Blocks that receive tokens must not be shared between sequences.
 */
exl3_status exl3_kv8_append(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const void *k, int64_t ldk,
                            const void *v, int64_t ldv, void *stream);

/*
 * exl3_kv8_attention: attention of this call's rows over the cached tokens.
 *     s[t] = scale * sum_d q[d] key[t][d];  s = softcap * tanh(s / softcap) if softcap > 0
 *     out  = sum_t softmax(s)[t] value[t]
 * over the positions t that the row sees: those up to its own (causal != 0)
 * or the whole sequence.
 *   q:    rows x (n_heads * head_dim) fp16, leading dimension ldq (multiple
 *         of 8). n_heads is a multiple of n_kv_heads; query head h reads
 *         key/value head h / (n_heads / n_kv_heads).
 *   out:  rows x (n_heads * head_dim) fp16 (RNE of fp32), leading dimension
 *         ldo (multiple of 8).
 *   lse:  rows x n_heads fp32, log sum_t exp(s[t]); or NULL.
 * A row that sees no token gives out = 0 and lse = -inf. What lies past a
 * sequence's length in its last block is never used, whatever its bytes are.
 * A NaN among the values of a sequence may reach every row that attends to
 * the sequence in this call, also rows before its position.
 * Sums, maxima and the softmax are fp32; the probabilities enter the product
 * with the values as fp16, scaled so that one of 2^-26 of a row's largest has all
 * its 11 bits and one of 2^-37 still counts.
 *   scale: finite; softcap: 0 (off) or finite and at least 1e-30. A capped score
 *         has an error of 2^-19 of itself at most, besides that of the products.
 *   workspace: exl3_kv8_attention_workspace_bytes bytes (0 for invalid
 *         arguments; it goes by rows, max_rows, the heads and head_dim),
 *         contents undefined before and after. Calls that share one must be
 *         ordered.
 * Up to 48 rows of a sequence and key/value head (max_rows x heads of a group)
 * go through a kernel bound by reading the cache, once for each 16 rows; more go
 * through one for 256 rows at a time. Both split long sequences over all SMs by the
 * lengths that they find on the device, and the result does not depend on
 * scheduling. max_rows decides for the whole call: single tokens beside a long
 * chunk are better served by a call of their own.
 * With more than 48 rows, keys and values are held relative to the largest scale of
 * the blocks that are worked on together, in fp16: what is below 2^-25 of that
 * block's largest value (448 scales) is lost, whether a row sees that block or not.
 */
size_t exl3_kv8_attention_workspace_bytes(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, int32_t n_heads);
exl3_status exl3_kv8_attention(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const void *q, int64_t ldq,
                               int32_t n_heads, float scale, float softcap, int causal, void *out, int64_t ldo,
                               float *lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * exl3_kv8_weigh: adds to the cache's `weight` of every token that a row of
 * this call sees the attention that it gets,
 *     weight[t] += sum over rows and query heads of the group: exp(s[t] - lse),
 * with s as in exl3_kv8_attention and lse as that call returned it (rows whose
 * lse is -inf add nothing). Each sequence's sum for a token is formed in a fixed
 * order: the result does not depend on scheduling, except where sequences of the
 * call share a block, whose sums are added to its weights in any order.
 */
exl3_status exl3_kv8_weigh(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const void *q, int64_t ldq,
                           int32_t n_heads, float scale, float softcap, int causal, const float *lse, void *stream);

/*
 * exl3_kv8_evict: cuts sequences back to `budget` tokens. For each sequence
 * and key/value head it keeps the last min(recent, kv_len) tokens and, of the
 * others, those with the largest `weight` (ties: the lower position; a NaN
 * weight counts as the lowest) until min(budget, kv_len) are kept, and writes
 * them, in their order, to the blocks of dst_pages.
 *   batch:     page_table, kv_len, n_seqs and max_pages of the sequences as
 *              they are (q_start, rows and max_rows are not read).
 *   dst_pages: n_seqs x ceil(budget / 64) page numbers, none of them a page
 *              of `batch` and none twice: the sequences' new page table. The
 *              old pages are the caller's to reuse after this call.
 *   kept:      n_seqs x n_kv_heads x budget int32: the positions kept, then -1.
 *   new_len:   n_seqs int32: min(budget, kv_len).
 * A new block's scale is the largest of its tokens' scales (their codes are
 * rescaled, E4M3(code * 2^(e_old - e))); weights move along; slots past
 * new_len keep what they held. 1 <= budget, 0 <= recent <= budget.
 * Positions are a sequence's own afterwards: a later append continues at
 * new_len.
 */
exl3_status exl3_kv8_evict(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const int32_t *dst_pages,
                           int32_t budget, int32_t recent, int32_t *kept, int32_t *new_len, void *stream);

/*
 * exl3_logits_adjust: penalties, biases and a grammar mask on logits, and the
 * greedy choice from what is left. For row m and token t < n, with c the times
 * that t occurs in the generated part of the row's history and `seen` whether
 * it occurs in it at all:
 *     l = seen ? (l > 0 ? l / repetition : l * repetition) : l
 *     l = l - (frequency * c + (c > 0 ? presence : 0))
 *     l = l + bias[t]
 *     l = -inf where the mask forbids t
 * in fp32, each operation rounded by itself.
 */
typedef struct {
    const int32_t *history;        /* token ids of all rows; ids outside 0 .. n-1 are ignored */
    const int32_t *history_start;  /* M + 1: row m's ids are history[history_start[m]] ... (both NULL: no history) */
    const int32_t *generated_from; /* M: index in the row's history of the first generated token, or NULL (0) */
    const float *repetition;       /* M, each > 0, or NULL (1) */
    const float *presence;         /* M, or NULL (0) */
    const float *frequency;        /* M, or NULL (0) */
    const int32_t *bias_id;        /* token ids; entries of the same id add up in their order */
    const float *bias_value;
    const int32_t *bias_start;     /* M + 1 (all three NULL: no biases) */
    const uint32_t *allowed;       /* M x ceil(n / 32) words, bit t % 32 of word t / 32 set: allowed; or NULL */
    int32_t history_size;          /* entries of `history` */
    int32_t bias_size;             /* entries of `bias_id` */
} exl3_logits_rules;

/*
 *   logits, out: M x n fp32, leading dimensions ldl, ldo (multiples of 4, at
 *          least n): exl3_logits_masked's logits with n = n_decodable. They may
 *          be the same buffer, with ldl = ldo. Columns from n on are neither read nor written.
 *   argmax: M int32: the first index of the row's maximum (a NaN is never
 *          the maximum); -1 where no token is left (all -inf or NaN).
 *   1 <= n <= 2^19, 0 <= M <= 65535; at most 2^29 history and 2^29 bias entries.
 */
exl3_status exl3_logits_adjust(const float *logits, int64_t ldl, int64_t M, int64_t n, const exl3_logits_rules *rules,
                               float *out, int64_t ldo, int32_t *argmax, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Step operators: what a serving step does around its projections before the
 * cache is read. exl3_kv8_plan makes a step's lengths, row ranges, block tables,
 * positions and slots; exl3_rms_norm stands before a projection; exl3_qk_rotary
 * between the projection of queries, keys and values and exl3_kv8_append;
 * exl3_prompt_attention attends over prompts that begin in this step, which have
 * all their keys and values at hand in fp16. It reads no cache: a sequence that has
 * tokens there (a running one, or the rest of a prompt) would attend over this step's
 * rows alone. A step that takes both kinds goes through exl3_kv8_attention as a whole,
 * or is planned as two, prompts (the running ones with 0 tokens) and single tokens.
 * ---------------------------------------------------------------------------
 *
 * exl3_kv8_plan: the step's batch from its requests, on the device.
 *   batch:      page_table (n_seqs x max_pages), kv_len and q_start are WRITTEN; n_seqs,
 *               max_pages, rows and max_rows bound the step.
 *   tokens:     n_seqs int32: the new tokens of each sequence in this step; 0: none;
 *               negative: the sequence has ended.
 *   cached:     n_seqs int32: its tokens in the cache before this step, 0 .. 64 * max_pages;
 *               may be the batch's kv_len. The first ceil(cached / 64) entries of its row of
 *               page_table are its pages; what lies behind them is not read.
 *   free_pages: a stack of free_capacity entries, of which the first *free_count are the
 *               numbers of free pages; the last of them is taken first. free_left receives
 *               how many are left (one int32; may be free_count).
 *   First the pages of ended sequences go onto the stack, in the order of the sequences
 *   and of their blocks; their kv_len becomes 0. Then the sequences are served in their
 *   order: kv_len = cached + tokens, and the blocks that this needs beyond those that it
 *   has get pages from the stack, in order of sequence and block. A sequence does not
 *   fit where pages run out, where the rows of this and the earlier sequences exceed
 *   batch->rows, or its own batch->max_rows, or cached + tokens exceeds 64 * max_pages.
 *   From the first one that does not fit on, sequences get no rows and keep kv_len = cached
 *   (ended ones have ended all the same); *served is the number of sequences before it
 *   (n_seqs: all).
 *   q_start:    the rows' ranges, n_seqs + 1.
 *   position, slot: batch->rows int32. Row r of sequence s stands at position
 *               kv_len[s] - (q_start[s + 1] - r) and in slot
 *               64 * page_table[s][position / 64] + position % 64. Rows from
 *               q_start[n_seqs] on have -1 in both.
 * A `cached` out of its range is recorded as EXL3_ERR_DEVICE_INDEX: the sequence does not
 * fit, and its kv_len becomes 0. So is a page number outside 0 .. n_pages - 1 that a row
 * needs (its slot is -1, and a page so taken from the stack is entered as -1), a
 * *free_count outside 0 .. free_capacity (it is brought into it), and pages given back
 * beyond free_capacity (they are dropped).
 * The other arrays must not overlap. n_pages: 1 .. 2^25 - 1; rows, free_capacity below 2^30.
 */
exl3_status exl3_kv8_plan(const exl3_kv8_batch *batch, const int32_t *tokens, const int32_t *cached, int32_t *free_pages,
                          int32_t free_capacity, const int32_t *free_count, int32_t *free_left, int64_t n_pages,
                          int32_t *position, int32_t *slot, int32_t *served, void *stream);

/*
 * exl3_rms_norm: the residual's addition and the root-mean-square norm of each row,
 *     h = x + residual
 *     y = h / sqrt(sum h^2 / cols + eps) * (weight + weight_offset)
 * in fp32 from inputs to outputs, each rounded once: residual_out = h, y in fp16, and
 * 8-bit codes with a scale for each `group` columns,
 *     scale = max(max |y| / 448, 2^-40) over the group's finite values, code = E4M3(y / scale),
 * nearest even, infinities saturating, NaN to NaN.
 */
typedef struct {
    const void *x;         /* rows x cols, x_dtype */
    const void *residual;  /* rows x cols, residual_dtype; NULL: none */
    void *residual_out;    /* rows x cols, residual_dtype; NULL: not written (and always without a residual) */
    const void *weight;    /* cols fp16; NULL: the factor is 1, without the offset */
    void *y;               /* rows x cols fp16; NULL: not written */
    void *codes;           /* rows x cols E4M3; NULL, with scales: not written */
    float *scales;         /* rows x (cols / group) fp32 */
    int64_t rows, cols;    /* rows >= 0 (below 2^31); cols a multiple of 8, 8 .. 32768 */
    int64_t ldx, ldr, ldro, ldy, ldc; /* leading dimensions in elements: multiples of 8, at least cols, below 2^31 */
    int32_t x_dtype, residual_dtype;  /* exl3_dtype */
    int32_t group;         /* with codes: 32, 64 or 128, which divides cols, or cols itself */
    float eps, weight_offset;         /* finite, eps >= 0 */
} exl3_norm;
/*
 * At least one of residual_out, y and codes is written. An output may be an input's own
 * buffer where type and leading dimension are the same; otherwise they must not overlap.
 * The squares' sum must stay in fp32.
 */
exl3_status exl3_rms_norm(const exl3_norm *norm, void *stream);

/*
 * exl3_qk_rotary: rotates the query and key heads of each row by its position, after a
 * root-mean-square norm of each head where weights are given. With x a head, after
 *     x = x / sqrt(sum x^2 / head_dim + eps) * (weight + weight_offset)      (if normed)
 * its first rot_dim elements turn in pairs i = 0 .. rot_dim / 2 - 1:
 *     a' = a cos - b sin,  b' = b cos + a sin
 *     (a, b) = (x[i], x[i + rot_dim / 2]), or (x[2 i], x[2 i + 1]) if interleaved,
 * and the others stay. fp32, rounded once.
 *   x, out:   rows x ((q_heads + k_heads) * head_dim) fp16: the query heads, then the key
 *             heads, as a fused projection gives them; leading dimensions ldx, ldo
 *             (multiples of 8). out may be x, with ldo = ldx; otherwise they must not overlap.
 *   position: rows int32, as exl3_kv8_plan gives them: a row with a negative one is left
 *             as it is in out; one of n_positions or more is recorded as
 *             EXL3_ERR_DEVICE_INDEX and treated so.
 *   cos_sin:  n_positions x rot_dim fp32, 16-byte aligned: for each position the cosines
 *             of the pairs' angles, then their sines. rot_dim: a multiple of 16, 16 .. head_dim.
 *   q_weight, k_weight: head_dim fp16 each, or both NULL (no norm; with no key heads,
 *             k_weight may be NULL too).
 *   head_dim: 64 or 128. q_heads, k_heads: at least 0, together 1 .. 65535.
 */
exl3_status exl3_qk_rotary(const void *x, int64_t ldx, void *out, int64_t ldo, int64_t rows, int32_t q_heads,
                           int32_t k_heads, int32_t head_dim, const int32_t *position, const float *cos_sin,
                           int64_t n_positions, int32_t rot_dim, int interleaved, const void *q_weight,
                           const void *k_weight, float eps, float weight_offset, void *stream);

/*
 * exl3_prompt_attention: attention of each row over the rows of its own sequence,
 *     s[t] = scale * sum_d q[d] k[t][d];  s = softcap * tanh(s / softcap) if softcap > 0
 *     out  = sum_t softmax(s)[t] v[t]
 * over the rows t of the sequence up to its own (causal != 0) or all of them. Sequences
 * lie one behind the other: rows q_start[s] .. q_start[s + 1] - 1 (n_seqs + 1 int32 on the
 * device, 0 <= q_start, not decreasing, at most rows).
 *   q, out:  rows x (n_heads * head_dim) fp16, leading dimensions ldq, ldo.
 *   k, v:    rows x (n_kv_heads * head_dim) fp16, leading dimensions ldk, ldv. All
 *            leading dimensions are multiples of 8: column ranges of one fused
 *            projection's output will do. Query head h reads key/value head
 *            h / (n_heads / n_kv_heads), at most 128 query heads one of them.
 *   lse:     rows x n_heads fp32, log sum_t exp(s[t]); or NULL.
 * A sequence's rows are all that it attends over: one with tokens in the cache does not belong here.
 * Rows of no sequence are left as they are in out and lse, and whatever they hold in q, k
 * and v reaches no other row; so it is with the rows that a row does not see, infinities and
 * NaN among them. A row that sees an infinity or NaN in v gets it in that column (or NaN).
 * A row whose scores are all minus infinity gets zeros, and -inf in lse.
 * A sequence whose range is not in the rows is recorded as EXL3_ERR_DEVICE_INDEX and
 * left out.
 * Sums, maxima and the softmax are fp32; the probabilities enter the product with the
 * values as fp16, scaled so that one of 2^-22 of a row's largest has all its 11 bits and
 * one of 2^-33 still counts. The result does not depend on scheduling. Scores of any size
 * that fp32 holds are taken as they are; beyond it they are infinite.
 *   head_dim: 64 or 128; scale: finite; softcap: 0 (off) or finite and at least 1e-30 (a
 *   capped score has an error of 2^-19 of itself at most, besides that of the products);
 *   n_seqs: 0 .. 65535; rows * n_heads below 2^31. out must not overlap q, k or v.
 */
exl3_status exl3_prompt_attention(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                  int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, const int32_t *q_start,
                                  int32_t n_seqs, int64_t rows, float scale, float softcap, int causal, void *out,
                                  int64_t ldo, float *lse, void *stream);

/*
 * exl3_selftest_bounds, for the translation units of the serving and step operators.
 */
exl3_status exl3_selftest_bounds_serving(int *units_reported, int *units_total, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_H_ */
