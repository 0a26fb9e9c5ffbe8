/*
 * tq2.h -- C ABI of the packed low-bit weight GEMM library for GB300 (sm_103a).
 *
 * One operation sits under two consumers:
 *
 *     out[m,n] = sum_k x[m,k] * W[n,k]
 *
 *  1. W in the ternary block format BlockTQ2_0_g128
 *     ("oxibonsai-kernels 0.2.1, src/gpu_backend/metal_graph/tests_gemm_tq2.rs",
 *     test test_encode_gemm_tq2_matches_reference): each 128-wide block of a
 *     weight row holds 32 bytes of 2-bit codes, 4 per byte, least significant
 *     first, code c meaning c-1 in {-1,0,+1}, and one f16 scale d;
 *     W[n,k] = (c-1)*d.
 *  2. The binary low-rank layer blr
 *     ("cortiq-engine 0.8.43, src/gpu_wgpu/train_mm.rs", module doc,
 *     blr_forward, blr_backward): W = diag(h) S_U diag(l) S_V^T diag(g) with
 *     the +-1 factors S_U, S_V stored as 1-bit bitmaps.
 *
 * Conventions for every entry point
 *   - Every call returns a tq2_status; nothing aborts the process.  Argument
 *     and shape errors are detected on the host before anything is launched.
 *     tq2_last_error() gives a one-line message for the calling thread.
 *   - "stream" is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Compute calls are asynchronous on that stream unless stated.
 *   - "DEVICE" pointers are CUDA device memory owned by the caller (for
 *     instance torch tensors); "HOST" pointers are ordinary host memory.
 *   - All float data is IEEE binary32, row-major, densely packed, but for the
 *     calls that take a tq2_dtype and a row stride.
 *   - Device-side waits inside the kernels are bounded (about one second);
 *     when one runs out the kernel records TQ2_ETIMEOUT and returns early.
 *     tq2_device_status() reports (and clears) that record.
 *   - Activations are staged to f16 on the GPU; entries must be finite with
 *     |v| < 65504 or the results are not finite.
 */
#ifndef TQ2_GB300_H
#define TQ2_GB300_H

#include <stdint.h>

#if defined(__GNUC__)
#define TQ2_API __attribute__((visibility("default")))
#else
#define TQ2_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TQ2_OK = 0,
    TQ2_EINVAL = 1,          /* null pointer or bad argument value            */
    TQ2_ESHAPE = 2,          /* sizes break a documented shape rule           */
    TQ2_ENOMEM = 3,          /* device or host allocation failed              */
    TQ2_ECUDA = 4,           /* a CUDA runtime/driver call failed             */
    TQ2_ETIMEOUT = 5,        /* a bounded device-side wait ran out            */
    TQ2_EUNSUPPORTED = 6     /* no kernel for this device or configuration    */
} tq2_status;

/* Opaque weight handle; the library owns the device planes behind it. */
typedef struct tq2_weight* tq2_handle;

/* Kernel selection for tq2_gemm_path (tests and benchmarks). */
typedef enum {
    TQ2_PATH_AUTO = 0,       /* M <= 16: skinny kernel; otherwise tensor path */
    TQ2_PATH_SKINNY = 1,     /* decode-in-register kernel, f32 activations, M <= 16 */
    TQ2_PATH_TENSOR = 2      /* tcgen05 kernel, activations staged to f16     */
} tq2_path;

/* Static string for a status code. */
TQ2_API const char* tq2_status_string(int status);

/* Message of the last failure on the calling thread ("" if none). */
TQ2_API const char* tq2_last_error(void);

/* Library build identification, e.g. "tq2-gb300 sm_103a". */
TQ2_API const char* tq2_version(void);

/*
 * Synchronize `stream`, then report and clear the device-side error record
 * (TQ2_ETIMEOUT if a bounded wait in any kernel ran out since the last call,
 * TQ2_ECUDA if the stream reports an error, else TQ2_OK).
 */
TQ2_API tq2_status tq2_device_status(void* stream);

/*
 * Give back to the device what the library's memory pool of the current
 * device holds and no call is using.  moe_route (plans of many tokens) and
 * moe_experts take their scratch from that pool, and it keeps what they took
 * (gigabytes after a call of many tokens) for the next call; the scratch of
 * work still pending on a stream is in use.  The next call takes memory from
 * the device again.  Not during a capture.
 */
TQ2_API tq2_status tq2_release_scratch(void);

/*
 * tq2_debug_wait_timeout -- test export for the error path above: launches
 * one thread that waits, with a bound of limit_ns, on a shared-memory
 * barrier that nothing completes.  When the bound runs out it records the
 * timeout exactly as the library's kernels do and returns, so the next
 * tq2_device_status on that stream reports TQ2_ETIMEOUT (and clears it)
 * while the context stays usable.  Nothing faults, traps or hangs.
 *   limit_ns  0 < limit_ns <= 1e9 (the kernels' own bound), else TQ2_EINVAL.
 *   stream    asynchronous on it.
 */
TQ2_API tq2_status tq2_debug_wait_timeout(uint64_t limit_ns, void* stream);

/* ------------------------------------------------------------------------ */
/* Ternary TQ2 weights                                                       */
/* ------------------------------------------------------------------------ */

/*
 * tq2_upload -- copy BlockTQ2_0_g128 blocks to the device and repack them.
 * Passage: the public SoA cache path get_or_upload_tq2_weight_soa(key, aos)
 * of test test_encode_gemm_tq2_matches_reference ("oxibonsai-kernels 0.2.1,
 * tests_gemm_tq2.rs").
 *
 *   aos     HOST, N*(K/128) blocks of 34 bytes, row-major (block kb of row n
 *           at index n*(K/128)+kb).  Block = { uint8 qs[32]; f16 d (little
 *           endian) }; code i of qs[j] (bits 2i..2i+1) is element 4j+i of
 *           the block.  The caller keeps ownership; the bytes are copied.
 *   N, K    weight rows and inner dimension; N >= 1, K >= 128, K % 128 == 0,
 *           N*K < 2^40.  Else TQ2_ESHAPE.
 *   out     receives the handle (set to NULL on failure).
 *   stream  used for the copy and the repack kernel; the call synchronizes
 *           it before returning, so `aos` may be freed afterwards.
 *
 * Device layout behind the handle ("SoA"): a code plane uint8[N][K/4]
 * holding each row's qs bytes in K order, and a scale plane uint16[N][K/128]
 * of f16 bits, each followed by a little zeroed padding.  The tensor-core
 * path (M > 8) reads two further copies made here: the codes stage-tiled
 * (uint8[ceil(N/128)][K/64][128][16], a 64-code stage of 128 rows
 * contiguous) and the scales block-major (uint16[K/128][ceil(N/128)*128]),
 * rows past N zero; so a handle holds about 2*N*K/4 + N*K/64 bytes.  Codes
 * are not validated: code 3 decodes as +2 (3-1).
 */
TQ2_API tq2_status tq2_upload(const void* aos, int64_t N, int64_t K, tq2_handle* out, void* stream);

/* Release the handle and its device memory (NULL is accepted).  The caller
 * must make sure no work that reads it is still pending. */
TQ2_API tq2_status tq2_free(tq2_handle h);

/* Shape of a handle. */
TQ2_API tq2_status tq2_shape(tq2_handle h, int64_t* N, int64_t* K);

/*
 * tq2_gemm -- out[m,n] = sum_k x[m,k] * W[n,k].
 * Passage: encode_gemm_tq2(&handle, &input, &mut out, m, n, k) and its CPU
 * reference ("oxibonsai-kernels 0.2.1, tests_gemm_tq2.rs",
 * test_encode_gemm_tq2_matches_reference: out is row-major [M][N]).
 *
 *   x       DEVICE float[M][K], row-major, 16-byte aligned.
 *   out     DEVICE float[M][N], row-major, overwritten.
 *   M       0 <= M <= 2^24 (M == 0 is a no-op returning TQ2_OK); on the
 *           tensor path also M*K < 2^31.  Else TQ2_ESHAPE.
 *   N, K    must equal the handle's shape, else TQ2_ESHAPE.
 *   stream  asynchronous on this stream.  Internal scratch (f16 copies of
 *           x) is taken from the stream-ordered allocator of the current
 *           device and released on the same stream.
 *
 * M <= 16 runs the skinny kernel: each f32 activation is carried as two f16
 * terms, hi = f16(x) and lo = f16(x - hi), whose sum differs from x by at
 * most about 2^-22 |x| (the weights are exact), with f32 accumulation:
 * |error| <= 2^-12 sum_k |x[m,k] W[n,k]| + 1e-7 per element, which is within
 * the pages' 1e-3 at K <= 4096 for unit-scale data.  For M <= 8 and
 * MT*K <= 32768, with MT = M rounded up to 1, 2, 4 or 8, it is a single
 * kernel with no scratch (the fused GEMV); that kernel decodes
 * codes with an offset that it removes per 128-block, so the rounding of a
 * block that holds a nonzero weight scales with that block's sum of |x|
 * (tested within the bound above on weights with 99 % zeros and x up to 256x
 * unit scale).  On every path a block whose codes are all 1 contributes
 * exactly 0, so an all-zero row gives exactly 0.
 * M > 16 runs the tensor-core kernel: activations rounded to f16
 * (nearest-even), weights exact in f16, f32 accumulation;
 * |error| <= 1e-2 * sum_k |x[m,k] W[n,k]|.
 */
TQ2_API tq2_status tq2_gemm(tq2_handle h, const float* x, float* out, int64_t M, int64_t N, int64_t K,
                    void* stream);

/* tq2_gemm with an explicit kernel choice (tq2_path).  TQ2_PATH_SKINNY
 * requires M <= 16 (else TQ2_ESHAPE). */
TQ2_API tq2_status tq2_gemm_path(tq2_handle h, const float* x, float* out, int64_t M, int64_t N, int64_t K,
                         int path, void* stream);

/*
 * tq2_gemm_tensor_tuned -- the tensor-core path of tq2_gemm with its tile
 * shape chosen by the caller (tuning sweeps; no counterpart on the pages).
 *
 *   bn      tokens per tile: 0 = the library's choice, else a multiple of 16
 *           in 16..256 (one that is not a multiple of 32 must be >= M), or
 *           384 when N > 128.
 *   splits  K splits: 0 = the library's choice, else 1..16 and <= K/64.  With
 *           more than one split the partial sums are added into the
 *           (zeroed) output with atomic adds: two splits give the same bits
 *           in either order, more than two may differ between runs by
 *           rounding (all within the tensor-path bound of tq2_gemm).
 *   Other arguments and errors as tq2_gemm on its tensor path; a bad bn or
 *   splits returns TQ2_EINVAL.
 */
TQ2_API tq2_status tq2_gemm_tensor_tuned(tq2_handle h, const float* x, float* out, int64_t M, int64_t N,
                                         int64_t K, int bn, int splits, void* stream);

/*
 * tq2_gemm_grouped -- G independent decode-shape GEMMs in one launch:
 * out_g[m,n] = sum_k x_g[m,k] * W_g[n,k] for g < G, each as tq2_gemm with
 * M <= 8 computes it (same kernel, same per-output arithmetic, so results
 * are bit-identical to G separate tq2_gemm calls).  One launch streams all
 * G weights, so independent projections that read the same activations
 * (or different ones) do not pay G kernel launches and G dependency waits.
 *
 *   hs      HOST array of G handles; all must have the same K.
 *   xs      HOST array of G DEVICE pointers, float[M][K] each, 16-byte aligned.
 *   outs    HOST array of G DEVICE pointers, float[M][N_g] each (overwritten).
 *   G       1..64;  1 <= M <= 8 with MT*K <= 32768, MT = M rounded up to
 *           1, 2, 4 or 8 (x is held in shared memory);  K the handles' K.
 *           Else TQ2_ESHAPE.
 *   stream  asynchronous; no scratch is allocated.
 */
TQ2_API tq2_status tq2_gemm_grouped(const tq2_handle* hs, const float* const* xs, float* const* outs, int G,
                                    int64_t M, int64_t K, void* stream);

/*
 * tq2_unpack -- rebuild the AoS bytes from the device planes (round trip of
 * tq2_upload).  aos_out: HOST buffer of N*(K/128)*34 bytes.  Synchronous.
 */
TQ2_API tq2_status tq2_unpack(tq2_handle h, void* aos_out, void* stream);

/*
 * tq2_dequant_f16 -- W[n,k] = (c-1)*d as f16 bits, exact (code x scale is
 * representable in f16; "oxibonsai-kernels 0.2.1, tests_gemm_tq2.rs", the
 * v10 parity test notes that f16 staging of code x scale is exact).
 *   w   DEVICE uint16[N][K], overwritten.  Debug / test export.
 */
TQ2_API tq2_status tq2_dequant_f16(tq2_handle h, uint16_t* w, void* stream);

/*
 * tq2_quantize -- the ternary producer: f32 weights -> BlockTQ2_0_g128 blocks.
 * Passage: the 2-bit FakeQuantize helpers of "rlx-mlx 0.2.13,
 * src/lower/helpers.rs" (fq_q_max gives q_max = 1 for 2 bits; the scale is
 * max|w| / q_max floored at 1e-12; the value is round(w / scale) clamped to
 * [-q_max, q_max]), applied per 128-element block of a row in f32:
 *   s = max(max|w|, 1e-12);  q = clamp(round_half_even(w / s), -1, 1);
 *   code = q + 1;  d = f16(s), nearest with ties to even.
 * The block granularity and the half-to-even rounding are readings: the page
 * reduces per channel or per tensor and stores no codes.
 *
 *   w        DEVICE float32[N][K], row-major, finite values (NaN or Inf give
 *            unspecified codes).  Read only.
 *   N, K     N >= 1, K >= 128, K % 128 == 0, N*K < 2^40.  Else TQ2_ESHAPE.
 *   aos_out  DEVICE, N*(K/128) blocks of 34 bytes in the tq2_upload layout
 *            (block kb of row n at index n*(K/128)+kb), overwritten.  Copy
 *            it to the host and pass it to tq2_upload to use the weights.
 *   stream   the launch is asynchronous on it.
 * Null pointers: TQ2_EINVAL.
 */
TQ2_API tq2_status tq2_quantize(const float* w, int64_t N, int64_t K, void* aos_out, void* stream);

/*
 * tq2_gemm_skinny_static -- the skinny GEMM (M <= 16) without any device
 * allocation.  The pages have no counterpart to this call; it exists for
 * callers that must not allocate while they run a GEMM: plugin or custom-op
 * interfaces that forbid allocation inside their enqueue call, serving
 * processes that reserve all device memory up front, and real-time loops in
 * which an allocator call could stall or fail.
 *
 *   Same arguments as tq2_gemm with 1 <= M <= 16; it runs the same kernel
 *   as tq2_gemm (the fused GEMV where that applies, which needs no scratch,
 *   else the staged skinny kernel), so its results equal tq2_gemm's bit for
 *   bit.
 *   The handle must live on the current device, else TQ2_EINVAL.
 *   Scratch (staged kernel only): a fixed 1 MiB device array inside the
 *   library (one per GPU that loads it, held until the process exits) holds
 *   the staged f16 fragments of x, ceil(M/4)*K*16 bytes; larger requests (for example K > 16384 at
 *   M = 16, K > 65536 at M <= 4) return TQ2_ESHAPE.  No cudaMalloc,
 *   cudaFree or stream-ordered allocation is made.
 *   The first call on a device looks up the array's device address on the
 *   current device (cudaGetSymbolAddress) and caches it for the life of the
 *   process; make that first call before any stream capture, and do not call
 *   this function on a device after resetting it (cudaDeviceReset).
 *   Every call shares the one array: calls whose work may overlap on the GPU
 *   (different streams, or different threads without ordering) race on it.
 *   Nothing in it needs clearing between calls: each call writes every byte
 *   it later reads.
 */
TQ2_API tq2_status tq2_gemm_skinny_static(tq2_handle h, const float* x, float* out, int64_t M, int64_t N,
                                          int64_t K, void* stream);

/* ------------------------------------------------------------------------ */
/* Binary low-rank layer (blr)                                               */
/* ------------------------------------------------------------------------ */

/*
 * blr_expand_bits -- sign bitmap to an f16 +-1 plane (bit-exact).
 * Passage: kernels expand_n / expand_t ("cortiq-engine 0.8.43,
 * train_mm.rs"): bitmap [rows][r/32] u32, bit j of word w is rank 32w+j,
 * a set bit is +1.0, a clear bit -1.0.
 *   bits       DEVICE uint32[rows][r/32].
 *   plane_f16  DEVICE uint16[rows][r] (transpose == 0) or [r][rows]
 *              (transpose != 0), f16 bits, overwritten.
 *   rows >= 1; r >= 32, r % 32 == 0.
 */
TQ2_API tq2_status blr_expand_bits(const uint32_t* bits, int64_t rows, int64_t r, uint16_t* plane_f16,
                           int transpose, void* stream);

/*
 * blr_forward -- one path of the binary low-rank layer, forward.
 * Passage: blr_forward and the module doc ("cortiq-engine 0.8.43,
 * train_mm.rs"):  a = (x.g) S_V,  c = (a.l) S_U^T,  y = h.c
 * (elementwise products broadcast over tokens).
 *
 *   bits_u  DEVICE uint32[d_out][r/32]  (S_U, [d_out][r])
 *   bits_v  DEVICE uint32[d_in][r/32]   (S_V, [d_in][r])
 *   h       DEVICE float[d_out];  l  DEVICE float[r];  g  DEVICE float[d_in]
 *   x       DEVICE float[T][d_in]
 *   y       DEVICE float[T][d_out], overwritten
 *   a_save  DEVICE float[T][r], overwritten with a (needed by blr_backward)
 *   c_save  DEVICE float[T][d_out] overwritten with c, or NULL (then
 *           blr_backward recomputes c from a_save)
 *   T >= 1; d_in, d_out multiples of 64; r >= 128, r % 128 == 0 (the page
 *   requires a multiple of 128); T*max(d_in, d_out) < 2^31, T*r < 2^28 and
 *   d_in, d_out <= 2^20.  Else TQ2_ESHAPE.  x, g and l must be 16-byte
 *   aligned (TQ2_EINVAL otherwise).
 * The activations x.g and a.l are staged to f16 (nearest-even); the GEMMs
 * accumulate in f32.  Scratch comes from the stream-ordered allocator.
 */
TQ2_API tq2_status blr_forward(const uint32_t* bits_u, const uint32_t* bits_v, const float* h,
                       const float* l, const float* g, const float* x, float* y,
                       float* a_save, float* c_save, int64_t T, int64_t d_in, int64_t d_out,
                       int64_t r, void* stream);

/*
 * blr_backward -- one path of the binary low-rank layer, backward.
 * Passage: blr_backward and the module doc ("cortiq-engine 0.8.43,
 * train_mm.rs"):
 *   dh += sum_t dy.c     b   = (dy.h) S_U     dl += sum_t a.b
 *   dx' = (b.l) S_V^T    dg += sum_t x.dx'    dx  = g.dx'
 *
 *   x, dy         DEVICE float[T][d_in], float[T][d_out]
 *   a_save        DEVICE float[T][r] from blr_forward on the same x
 *   c_save        DEVICE float[T][d_out] from blr_forward, or NULL (recompute)
 *   dx            DEVICE float[T][d_in], overwritten
 *   dh, dl, dg    DEVICE float[d_out], float[r], float[d_in]; ACCUMULATED
 *                 (+=) as on the page; the caller zeroes them.
 *   gscale        power of two (1.0 allowed) multiplying the gradients while
 *                 they are staged in f16, divided back out after each GEMM
 *                 (the page keeps gradients out of the f16 subnormals this
 *                 way).  Else TQ2_EINVAL.
 * Column sums use a fixed reduction order (deterministic run to run).
 * Shape rules as blr_forward; dy, h, l and a_save must be 16-byte aligned.
 */
TQ2_API tq2_status blr_backward(const uint32_t* bits_u, const uint32_t* bits_v, const float* h,
                        const float* l, const float* g, const float* x, const float* dy,
                        const float* a_save, const float* c_save, float* dx, float* dh,
                        float* dl, float* dg, int64_t T, int64_t d_in, int64_t d_out,
                        int64_t r, float gscale, void* stream);

/*
 * Several paths of one blr layer, y = sum_p diag(h_p) S_U,p diag(l_p) S_V,p^T
 * diag(g_p) x.  Passage: blr_forward / blr_backward over layer.paths and the
 * two-path combine scale_acc2 ("cortiq-engine 0.8.43, train_mm.rs"): the
 * paths are taken in order, the first writes y (dx) and each later one adds
 * its product to it, each product and each sum rounded to f32 separately
 * (no fused multiply-add): for two paths y = fl(fl(h0.c0) + fl(h1.c1)), the
 * page's one-pass two-path rounding; for more, fl(fl(y + fl(h_p.c_p))) in
 * path order, as the page's scale_acc passes.
 *
 * One path: its bitmaps and vectors (DEVICE, layouts as blr_forward), its
 * forward outputs a_save (required) and c_save (may be NULL), and its
 * gradient accumulators dh, dl, dg (DEVICE, += as in blr_backward; used by
 * blr_backward_paths only).
 */
typedef struct {
    const uint32_t* bits_u;
    const uint32_t* bits_v;
    const float* h;
    const float* l;
    const float* g;
    float* a_save;
    float* c_save;
    float* dh;
    float* dl;
    float* dg;
} blr_path;

#define BLR_MAX_PATHS 64

/*
 * blr_forward_paths -- forward of a layer of P paths (1 <= P <= BLR_MAX_PATHS).
 *   paths   HOST array of P blr_path (read during the call only).
 *   x       DEVICE float[T][d_in], shared by all paths.
 *   y       DEVICE float[T][d_out], overwritten with the combined output.
 * Shape rules as blr_forward.  x and each path's g and l must be 16-byte
 * aligned.  With P = 1 the result is blr_forward's bit for bit.
 */
TQ2_API tq2_status blr_forward_paths(const blr_path* paths, int P, const float* x, float* y, int64_t T,
                             int64_t d_in, int64_t d_out, int64_t r, void* stream);

/*
 * blr_backward_paths -- backward of the layer of the last blr_forward_paths
 * on the same x: each path's dh, dl, dg accumulate (+=), dx (DEVICE
 * float[T][d_in]) is overwritten with sum_p g_p.dx'_p rounded as described
 * above.  gscale as blr_backward; dy and each path's h, l and a_save must be
 * 16-byte aligned.
 */
TQ2_API tq2_status blr_backward_paths(const blr_path* paths, int P, const float* x, const float* dy, float* dx,
                              int64_t T, int64_t d_in, int64_t d_out, int64_t r, float gscale,
                              void* stream);

/*
 * blr_sign_grads -- the gradients of the loss with respect to one path's
 * signs, G_U = diag(h) dy^T a diag(l) ([d_out][r]) and
 * G_V = diag(g) x^T b diag(l) ([d_in][r]) with b = (dy.h) S_U.
 * Passage: blr_backward's sign-training step and the test
 * blr_sign_flip_exact ("cortiq-engine 0.8.43, train_mm.rs"): the token axis
 * is the GEMMs' K, the operands dy.h.gs, a.l, x.g and b.l.gs are staged
 * transposed in f16, and flipping sign s of U[i,k] changes L = 1/2|y - y*|^2
 * by -2 s G_U[i,k] + 2 h_i^2 l_k^2 sum_t a_tk^2 (V likewise).
 *
 *   bits_u        DEVICE uint32[d_out][r/32] (S_U; S_V is not needed)
 *   h, l, g       DEVICE float[d_out], float[r], float[d_in]
 *   x, dy         DEVICE float[T][d_in], float[T][d_out]
 *   a_save        DEVICE float[T][r] from blr_forward on the same x
 *   gu, gv        DEVICE float[d_out][r], float[d_in][r], overwritten
 *   gscale        power of two multiplying the dy-side operands while they
 *                 are staged in f16, divided back out (as blr_backward);
 *                 dy.h.gs and b.l.gs must stay inside the f16 range (a
 *                 value beyond 65504 stages as inf).
 * Shape rules as blr_forward; x, dy, a_save, h, l and g must be 16-byte
 * aligned (TQ2_EINVAL otherwise).
 */
TQ2_API tq2_status blr_sign_grads(const uint32_t* bits_u, const float* h, const float* l, const float* g,
                          const float* x, const float* dy, const float* a_save, float* gu, float* gv,
                          int64_t T, int64_t d_in, int64_t d_out, int64_t r, float gscale, void* stream);

/* ------------------------------------------------------------------------ */
/* 4-bit weights with group scales                                           */
/* ------------------------------------------------------------------------ */

/* Element types of activations, logits and outputs. */
typedef enum { TQ2_F32 = 0, TQ2_F16 = 1, TQ2_BF16 = 2 } tq2_dtype;

/* Opaque handle of E 4-bit matrices of the same shape (E = 1: one weight). */
typedef struct q4_weight* q4_handle;

/*
 * q4_upload -- lay out 4-bit weights for the products below:
 *     W[e,n,k] = (c - z) * d,   c = codes[e,n,k],  z, d of the group k/group.
 *
 *   codes   uint8[E][N][K/2], the code of an even k in the low half of its
 *           byte, of the odd k after it in the high half.
 *   scales  f16 bits [E][N][K/group]; any sign.
 *   zeros   uint8[E][N][K/group], 0..15 (the upper four bits are ignored), or
 *           NULL: every zero point is 8.
 *           All three in HOST or in DEVICE memory (each by itself); codes
 *           2-byte aligned.  Copied: the caller keeps ownership.
 *   E, N, K, group   E, N >= 1, E <= 1024, group 32, 64 or 128, K >= group a
 *           multiple of it, K <= 32768, N <= 2^24, N*K <= 2^36.  Else
 *           TQ2_ESHAPE.
 *   out     receives the handle (NULL on failure).
 *   stream  used for the copies and the layout kernel, after work queued on
 *           it; the call synchronizes it before returning.
 *
 * The handle holds one copy in 16-row x 256-k blocks (codes, then the block's
 * scales and zero points), N padded to 128 rows and K to 256, and a bound of
 * each matrix's row norms, the spread of those norms and the weights' largest
 * magnitude (for moe_experts).
 */
TQ2_API tq2_status q4_upload(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t E,
                             int64_t N, int64_t K, int group, q4_handle* out, void* stream);

/* Release the handle and its device memory (NULL is accepted).  The caller
 * must make sure no work that reads it is still pending. */
TQ2_API tq2_status q4_free(q4_handle h);

/* Shape of a handle (each pointer may be NULL). */
TQ2_API tq2_status q4_shape(q4_handle h, int64_t* E, int64_t* N, int64_t* K, int* group);

/*
 * q4_dequant -- W as the products see it: DEVICE float[E][N][K], overwritten;
 * exact ((c - z) * d has at most 16 significant bits).  Asynchronous.
 */
TQ2_API tq2_status q4_dequant(q4_handle h, float* w, void* stream);

/*
 * q4_quantize -- plain weights to codes, scales and zero points, all in the
 * layout q4_upload takes.  Per group of a row, in f32:
 *   zeros given:  lo = min(w, 0), hi = max(w, 0), d = f16((hi - lo) / 15),
 *                 z = clamp(rint(-lo / d), 0, 15), c = clamp(rint(w / d) + z, 0, 15)
 *   zeros NULL:   d = f16(max|w| / 7), c = clamp(rint(w / d) + 8, 0, 15)
 * with the rounded d (at most 65504) and halves to even; where d = 0, c = z
 * (z = 0, or 8 without zero points).
 *
 *   w       DEVICE, dtype (tq2_dtype), [rows][K] dense, finite (NaN or Inf
 *           give unspecified codes).  rows >= 1, K and group as q4_upload.
 *   codes, scales, zeros   DEVICE, overwritten; codes 4-byte aligned, w and
 *           scales aligned to their elements (else TQ2_EINVAL).
 * Asynchronous.
 */
TQ2_API tq2_status q4_quantize(const void* w, int dtype, int64_t rows, int64_t K, int group, uint8_t* codes,
                               uint16_t* scales, uint8_t* zeros, void* stream);

/*
 * q4_gemm -- out[m,n] = sum_k x[m,k] W[n,k], for a handle with E = 1.
 *
 *   x       DEVICE, dtype, M rows of K, ldx >= K elements apart.
 *   out     DEVICE, dtype (that of x), M rows of N, ldo >= N elements apart,
 *           overwritten; must not overlap x.
 *   M       0 <= M <= 2^20 (0: nothing is done).
 *   x and out need only their element's alignment (else TQ2_EINVAL); rows that
 *   are 16-byte aligned are fetched faster.
 * Weights and f16 / bf16 activations enter the products exactly; f32
 * activations as two f16 parts of a row scaled by a power of two, whose sum
 * is within 2^-22 |x[m,k]| + 2^-38 max_k |x[m,k]| of x.  Accumulation is in
 * f32 and the result is rounded once to dtype.  The order of the additions
 * depends on the shape and the GPU alone, so results are the same from run to
 * run.  A row of x with NaN or Inf has NaN or Inf in its own row of out only.
 * Meant for decode batches: up to 32 rows of f16 or bf16 (16 of f32) read the
 * weights once, larger M runs as launches of so many rows (of fewer, where they
 * do not fit the shared memory of eight SMs).  Asynchronous, no scratch.
 */
TQ2_API tq2_status q4_gemm(q4_handle h, const void* x, int64_t ldx, void* out, int64_t ldo, int dtype, int64_t M,
                           void* stream);

/* ------------------------------------------------------------------------ */
/* Mixture of experts                                                        */
/* ------------------------------------------------------------------------ */

/* Scores of a router. */
typedef enum { MOE_SOFTMAX = 0, MOE_SIGMOID = 1 } moe_score;

/*
 * moe_route -- a router's selection, its weights and the order of its slots.
 *
 * Per token (row of logits), in f32: expert e is available where its logit
 * and its bias are neither -inf nor NaN; +inf counts as the largest f32.
 *   p     softmax of the available logits, or their sigmoid 1/(1+exp(-l)),
 *         each operation rounded to f32 (so saturated scores tie); 0 for the
 *         others.  The softmax sum adds neighbouring experts first (a binary
 *         tree over the row, padded with zeros to a power of two).
 *   s     p + bias: what the selection goes by.
 *   groups > 1 and top_groups < groups: E/groups neighbouring experts form a
 *         group; its value is the sum of its two largest s (of one, where only
 *         one is available).  Only the top_groups groups of largest value take part.
 *   ids   the k experts of largest s, in that order.  Ties, among groups too,
 *         go to the lower index.  -1 where fewer are available.
 *   w     p of the selected (0 beside -1), divided by max(their sum,
 *         2^-126) if renorm, times scale.
 * The slots t*k+j with an expert, ordered by expert and then by slot, are the
 * plan that moe_experts takes: those of expert e are
 * slots[offsets[e]] .. slots[offsets[e+1]-1]; slots past offsets[E] are -1.
 *
 *   logits   DEVICE, dtype, T rows of E, ld >= E elements apart.
 *   bias     DEVICE float[E] or NULL (zero).
 *   ids      DEVICE int32[T][k];  weights  DEVICE float[T][k].
 *   offsets  DEVICE int32[E+1];  slots  DEVICE int32[T*k]; or both NULL: no plan.
 *   0 <= T, T*k <= 2^24;  1 <= E <= 1024;  1 <= k <= 32, k <= E;  groups
 *   divides E and is at most 32;  1 <= top_groups <= groups.  Else TQ2_ESHAPE.
 *   score a moe_score, scale finite, pointers aligned to their elements.  Else
 *   TQ2_EINVAL.
 * Asynchronous; scratch (for a plan of many tokens) from the library's
 * stream-ordered pool.
 */
TQ2_API tq2_status moe_route(const void* logits, int64_t ld, int dtype, const float* bias, int64_t T, int E, int k,
                             int score, int groups, int top_groups, int renorm, float scale, int32_t* ids,
                             float* weights, int32_t* offsets, int32_t* slots, void* stream);

/*
 * moe_route_backward -- gradient of moe_route's weights to its logits (the
 * selection is piecewise constant and the bias takes no part in the weights).
 * With g_j = scale * dweights[j] and p as above, sums over the selected j, S = sum_i p_i:
 *   q_j = g_j without renorm;  (g_j - sum_i g_i p_i / S) / S with renorm;  g_j / 2^-126 with
 *   renorm where S < 2^-126 (the weights are divided by a constant there)
 *   softmax:  dlogits[e] = p_e (q_e - sum_j q_j p_j)      (q_e = 0 unless selected;
 *             with renorm and S >= 2^-126 the sum is 0 and only the selected get a gradient)
 *   sigmoid:  dlogits[e] = p_e (1 - p_e) q_e
 * ids as moe_route returned them; a slot of -1 takes no part.  dweights: DEVICE
 * float[T][k], the loss's gradient to the weights; for the output of moe_experts that
 * is out's gradient times the slot's own expert output, which is the caller's to
 * compute (moe_experts returns the weighted sum alone).  dlogits: DEVICE,
 * dtype, T rows of E, ldd >= E elements apart, overwritten; may be logits itself
 * (ldd = ld), else overlaps none of the inputs.  Limits as moe_route.
 * Asynchronous, no scratch.
 */
TQ2_API tq2_status moe_route_backward(const void* logits, int64_t ld, int dtype, const float* bias,
                                      const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd,
                                      int64_t T, int E, int k, int score, int renorm, float scale, void* stream);

/*
 * moe_experts -- the routed experts' gated products:
 *   out[t] = sum_j weights[t,j] * Down_e ( silu(Gate_e x[t]) * (Up_e x[t]) ),  e = ids[t,j],
 * over the j with ids[t,j] >= 0 (a token without any gets 0); silu(v) = v/(1+exp(-v)).
 *
 *   gate, up  handles of E matrices F x D, the same group and zero-point form.
 *   down      handle of E matrices D x F.
 *   x         DEVICE, dtype, T rows of D, ldx >= D elements apart.
 *   ids, weights, offsets, slots   DEVICE, a plan of moe_route for these E:
 *             int32[T][k], float[T][k], int32[E+1], int32[T*k].  Of any other
 *             contents the result is unspecified (offsets and slots are
 *             clamped to their ranges: nothing outside the arrays is touched).
 *   out       DEVICE, dtype, T rows of D, ldo >= D elements apart,
 *             overwritten; must not overlap x.
 *   0 <= T, T*k <= 2^24, 1 <= k <= 32, (T*k + E) * max(D, 2F) < 2^35, shapes
 *   that fit each other: else TQ2_ESHAPE.  Pointers aligned to their elements:
 *   else TQ2_EINVAL.
 *
 * Calls of f32, and those of f16 and bf16 with at most 4 slots a matrix on
 * average (T*k <= 4 E) or with a weight that may exceed 65504, the largest of
 * f16 (|d| max(z, 15-z) in any of the handles): Gate and Up take x as q4_gemm
 * takes it; the gated product is kept in f32 and enters Down as f32 activations
 * do (for f16 and bf16 as its first f16 part alone, within 2^-11 of its
 * magnitude).
 * Other f16 and bf16 calls: the weights are rounded to f16, rows of x and of
 * the gated product are f16 scaled by a power of two each (of x so that its
 * largest element is just below 2^15; of the gated product by a bound of it,
 * |x|^2 times Gate's and Up's largest row norms in the matrix, so that elements
 * below 2^-28 of that bound lose bits), and a product's sum over k runs in f32.
 * Where Gate's largest row norm over its smallest (but 0) in some matrix, times
 * Up's, times D is above 2^24, a row of the gated product is scaled by its own
 * maximum instead, like a row of x.
 * Either way a token's sum over j runs in the order of j, in f32, and is
 * rounded once to dtype.
 * Scratch from the library's stream-ordered pool, which keeps it
 * (tq2_release_scratch): T*k rows of D floats, and of F
 * floats (f16 and bf16 calls with many slots: of F and of D halves, and of F
 * floats where gated rows are scaled by themselves).  Asynchronous.
 */
TQ2_API tq2_status moe_experts(q4_handle gate, q4_handle up, q4_handle down, const void* x, int64_t ldx, int dtype,
                               const int32_t* ids, const float* weights, const int32_t* offsets,
                               const int32_t* slots, void* out, int64_t ldo, int64_t T, int k, void* stream);

/* ------------------------------------------------------------------------ */
/* 8-bit cache of keys and values                                            */
/* ------------------------------------------------------------------------ */

/*
 * The cache: a pool of blocks of `tokens` tokens, in the caller's DEVICE memory.
 *   codes   uint8[blocks][2][heads][tokens][dim] (keys, then values), 16-byte aligned.
 *   scales  float[blocks][2][heads]: one scale for a block's tokens in a head, >= 0 or NaN
 *           (attention may take one below 2^-103, less than kv8_write makes, for 0, and takes Inf for NaN).
 * A code c stands for (c - 128) * scale.
 *   tokens 16, 32, 64 or 128;  dim 64 or 128;  1 <= heads <= 1024;  blocks >= 1 with
 *   blocks * 2 * heads * tokens < 2^31.  Else TQ2_ESHAPE.
 */
typedef struct {
    uint8_t* codes;
    float* scales;
    int64_t blocks;
    int heads, tokens, dim;
} kv8_cache;

/*
 * Sequences of a call (the arrays in DEVICE memory, read when the kernels run, so a captured
 * call follows what they hold at its replay):
 *   table    int32, a row of `width` block numbers a sequence, rows `ld` >= width elements
 *            apart: token t of sequence s lies in block table[s*ld + t/tokens], at t % tokens.
 *   offsets  int32[seqs+1], ascending: rows offsets[s] .. offsets[s+1]-1 of the call's other
 *            arrays are sequence s's last tokens.
 *   lens     int32[seqs]: tokens of each sequence, those n = offsets[s+1]-offsets[s] among
 *            them; row offsets[s]+j is at position lens[s]-n+j.
 *   1 <= seqs, 1 <= width, width * tokens <= 2^30.  Else TQ2_ESHAPE.
 * Entries of any contents are safe: offsets outside the rows and lengths outside the table are
 * clamped to them, ranges that go back are empty, and a block number outside the pool names
 * no block.  Entries past a sequence's tokens are not read.
 */
typedef struct {
    const int32_t* table;
    int64_t ld;
    const int32_t* offsets;
    const int32_t* lens;
    int width, seqs;
} kv8_batch;

/*
 * kv8_write -- quantise the sequences' last tokens as they enter their blocks.
 *
 * Per block, head, and keys or values, each operation rounded to f32, halves to even: with
 * M the largest magnitude of the new tokens, d0 the block's scale where it holds
 * tokens of the sequence before the new ones (0 where not),
 *     d = max(d0, M / 127)   (M below 2^-96 counts as 0)
 *     c = 128 + clamp(rint(x * (1 / d)), -127, 127)          of the new tokens
 *     c = 128 + rint((c - 128) * (d0 / d))                   of those before, where d > d0
 * (d = 0: c = 128; 1 / d is the largest f32 at most).  Codes past the new tokens keep what they hold, which nothing reads.
 * A NaN or Inf among the new tokens leaves the block's scale NaN: every value of that
 * block and head reads as NaN until a write begins the block anew.
 *
 *   c, b    HOST structs, read during the call.
 *   k, v    DEVICE, dtype (tq2_dtype), T rows of `heads` heads of dim neighbouring elements;
 *           kt, kh and vt, vh: elements from row to row and from head to head.  Fetched
 *           faster where 16-byte aligned throughout.
 *   0 <= T, T * heads * dim < 2^40.
 * Tokens without a position (n > lens[s]) or without a block are not written.  What a
 * block of two sequences (shared, or named twice) holds after both were written into it
 * is unspecified.  Asynchronous, no scratch.
 */
TQ2_API tq2_status kv8_write(const kv8_cache* c, const kv8_batch* b, const void* k, int64_t kt, int64_t kh,
                             const void* v, int64_t vt, int64_t vh, int dtype, int64_t T, void* stream);

/*
 * kv8_read -- the sequences' last tokens as values: k[offsets[s]+j][head] = (c - 128) * scale, rounded
 * to f32 and then to dtype.  Arguments as kv8_write's; k and v are written, and keep what they
 * hold in rows without a position, without a block, or of no sequence.  Asynchronous, no scratch.
 */
TQ2_API tq2_status kv8_read(const kv8_cache* c, const kv8_batch* b, void* k, int64_t kt, int64_t kh, void* v,
                            int64_t vt, int64_t vh, int dtype, int64_t T, void* stream);

/*
 * kv8_attention -- attention of the sequences' last tokens over the cache.
 *
 * Query head h of a row reads head h / (Hq / heads) of the cache:
 *     s_t = scale * sum_d q[row][h][d] k_t[d],   p = softmax of s over the seen tokens t,
 *     out[row][h] = sum_t p_t v_t,   lse[row][h] = ln sum_t exp(s_t).
 * Of tokens 0 .. lens[s]-1, those with a block, a row at position i sees
 *     causal:  t <= i, and t > i - window where window > 0;      else all.
 * A row that sees none has out 0 and lse -Inf.
 *
 *   q, out  DEVICE, dtype, T rows of Hq heads of dim neighbouring elements; qt, qh and ot, oh:
 *           elements from row to row and from head to head.  out must not overlap q. Rows of no
 *           sequence are left as they are, in lse too.
 *   lse     DEVICE float[T][Hq] or NULL.
 *   Hq      a multiple of heads, T <= 2^30, T * Hq <= 2^31 - 512, and fewer than 2^38 tiles of 128 rows (T * Hq / heads)
 *           by 128 tokens of the tables; seqs <= 2^24.  Else TQ2_ESHAPE.
 *   scale   finite, and times log2(e) too;  causal 0 or 1;  window >= 0, 0 unless causal.  Else TQ2_EINVAL.
 *   max_q   a bound of the sequences' rows that the choice of kernels goes by (0: T); results
 *           of longer ones are right too, but slower.  Give it where it is known: without one, decoded tokens whose
 *           rows (T * Hq / heads) are more than 32 in all count as a prompt, and run or launch its kernels too.
 * f16 and bf16 queries and the codes enter the products exactly (elements below 2^-29 of their
 * row's largest lose bits), f32 queries within 2^-22 of each element and 2^-39 of the row's
 * largest (both: of 2^-112 where that is larger).  Scores have to be in f32's range.  A token's weight times its block's scale is rounded to f16 for bf16 results (2^-11), to two
 * f16 parts for f16 and f32 ones (2^-22), and to 2^-30 of the row's largest at the least (where values are
 * all zeros, a weight times 2^-40 of a neighbour's scale may be the largest).  Sums
 * are f32, results rounded once.  A row of q with NaN or Inf gives NaN in its own row alone; a NaN scale reaches the rows
 * that see a token of its block: out, and lse where it is the keys'.  The order of additions depends on lengths, shapes and the
 * GPU alone, so results are the same from run to run.  Asynchronous; scratch from the
 * library's stream-ordered pool.
 */
TQ2_API tq2_status kv8_attention(const kv8_cache* c, const kv8_batch* b, const void* q, int64_t qt, int64_t qh,
                                 void* out, int64_t ot, int64_t oh, int dtype, float* lse, int64_t T, int Hq,
                                 float scale, int causal, int64_t window, int64_t max_q, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ2_GB300_H */
