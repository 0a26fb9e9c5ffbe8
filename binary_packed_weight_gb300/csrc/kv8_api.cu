// kv8_api.cu -- the C ABI of the 8-bit cache: argument checks, scratch, and
// the choice of the attention's path.
#include <cmath>

#include "../../include/tq2.h"
#include "kv8.cuh"

namespace tq2 {
namespace {

tq2_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return TQ2_OK;
    return (tq2_status)set_error(e == cudaErrorMemoryAllocation ? TQ2_ENOMEM : TQ2_ECUDA, "%s: %s", what,
                                 cudaGetErrorString(e));
}

// What the three calls have in common: the cache and the sequences as the kernels see them.
tq2_status view(const kv8_cache* c, const kv8_batch* b, int dtype, int64_t T, const char* where, Kv8View* out) {
    if (!c || !b || !c->codes || !c->scales || !b->table || !b->offsets || !b->lens)
        return (tq2_status)set_error(TQ2_EINVAL, "%s: null pointer", where);
    if (dtype != TQ2_F32 && dtype != TQ2_F16 && dtype != TQ2_BF16)
        return (tq2_status)set_error(TQ2_EINVAL, "%s: unknown dtype %d", where, dtype);
    int logB = 4;
    while (logB < 7 && (1 << logB) < c->tokens) ++logB;
    if ((1 << logB) != c->tokens || (c->dim != 64 && c->dim != 128) || c->heads < 1 || c->heads > 1024 ||
        c->blocks < 1 || c->blocks > ((int64_t)1 << 30) || c->blocks * 2 * c->heads * c->tokens >= ((int64_t)1 << 31))
        return (tq2_status)set_error(TQ2_ESHAPE,
                                     "%s: need tokens 16, 32, 64 or 128, dim 64 or 128, 1 <= heads <= 1024, blocks >= 1 "
                                     "and blocks*2*heads*tokens < 2^31 (blocks=%lld heads=%d tokens=%d dim=%d)",
                                     where, (long long)c->blocks, c->heads, c->tokens, c->dim);
    if (b->seqs < 1 || b->width < 1 || b->ld < b->width || (int64_t)b->width * c->tokens > ((int64_t)1 << 30))
        return (tq2_status)set_error(TQ2_ESHAPE,
                                     "%s: need seqs >= 1, 1 <= width <= ld, width*tokens <= 2^30 (seqs=%d width=%d ld=%lld)",
                                     where, b->seqs, b->width, (long long)b->ld);
    if (T < 0 || T >= ((int64_t)1 << 31))
        return (tq2_status)set_error(TQ2_ESHAPE, "%s: bad T=%lld", where, (long long)T);
    if (off_element(c->codes, 16) || off_element(c->scales, 4) || off_element(b->table, 4) ||
        off_element(b->offsets, 4) || off_element(b->lens, 4))
        return (tq2_status)set_error(TQ2_EINVAL, "%s: codes must be 16-byte aligned, the others to their elements", where);
    *out = Kv8View{c->codes, c->scales, b->table, b->offsets, b->lens, b->ld, (int)c->blocks, c->heads, logB, c->dim,
                   b->width, b->seqs, (int)T};
    return TQ2_OK;
}

tq2_status move(const kv8_cache* c, const kv8_batch* b, void* k, int64_t kt, int64_t kh, void* v, int64_t vt,
                int64_t vh, int dtype, int64_t T, void* stream, const char* where,
                cudaError_t (*launch)(const Kv8View&, const Kv8Rows&, cudaStream_t)) {
    Kv8View w;
    const tq2_status st = view(c, b, dtype, T, where, &w);
    if (st != TQ2_OK) return st;
    if (T * c->heads * c->dim >= ((int64_t)1 << 40))
        return (tq2_status)set_error(TQ2_ESHAPE, "%s: %lld rows are too many for one call", where, (long long)T);
    if (T == 0) return TQ2_OK;
    if (!k || !v) return (tq2_status)set_error(TQ2_EINVAL, "%s: null pointer", where);
    if (off_element(k, element_size(dtype)) || off_element(v, element_size(dtype)))
        return (tq2_status)set_error(TQ2_EINVAL, "%s: k and v must be element-aligned", where);
    return cuda_status(launch(w, Kv8Rows{k, v, kt, kh, vt, vh, dtype}, reinterpret_cast<cudaStream_t>(stream)), where);
}

// Scratch of one call, given back on the same stream whatever happens.
struct Scratch {
    void* p = nullptr;
    cudaStream_t st;
    explicit Scratch(cudaStream_t s) : st(s) {}
    ~Scratch() {
        if (p) cudaFreeAsync(p, st);
    }
};

}  // namespace
}  // namespace tq2

using namespace tq2;

extern "C" {

tq2_status kv8_write(const kv8_cache* c, const kv8_batch* b, const void* k, int64_t kt, int64_t kh, const void* v,
                     int64_t vt, int64_t vh, int dtype, int64_t T, void* stream) {
    return move(c, b, const_cast<void*>(k), kt, kh, const_cast<void*>(v), vt, vh, dtype, T, stream, "kv8_write",
                launch_kv8_write);
}

tq2_status kv8_read(const kv8_cache* c, const kv8_batch* b, void* k, int64_t kt, int64_t kh, void* v, int64_t vt,
                    int64_t vh, int dtype, int64_t T, void* stream) {
    return move(c, b, k, kt, kh, v, vt, vh, dtype, T, stream, "kv8_read", launch_kv8_read);
}

tq2_status kv8_attention(const kv8_cache* c, const kv8_batch* b, const void* q, int64_t qt, int64_t qh, void* out,
                         int64_t ot, int64_t oh, int dtype, float* lse, int64_t T, int Hq, float scale, int causal,
                         int64_t window, int64_t max_q, void* stream) {
    Kv8Attention a{};
    const tq2_status bad = view(c, b, dtype, T, "kv8_attention", &a.c);
    if (bad != TQ2_OK) return bad;
    // (a row's position less the window, each of 2^30 at most, is a number of 32 bits)
    // (and so is the end of the last, part-full tile of rows)
    if (Hq < c->heads || Hq % c->heads || T > ((int64_t)1 << 30) || T * Hq > ((int64_t)1 << 31) - 512)
        return (tq2_status)set_error(TQ2_ESHAPE,
                                     "kv8_attention: Hq=%d must be a multiple of heads=%d with T <= 2^30 and T*Hq <= 2^31 - 512", Hq,
                                     c->heads);
    const float scale2 = scale * 1.4426950408889634f;        // powers of 2 from here on
    if (!std::isfinite(scale2) || (causal != 0 && causal != 1) || window < 0 || (window && !causal) || max_q < 0)
        return (tq2_status)set_error(TQ2_EINVAL,
                                     "kv8_attention: need a finite scale (times log2(e) too), causal 0 or 1, window >= 0 (0 unless causal), "
                                     "max_q >= 0 (scale=%g causal=%d window=%lld max_q=%lld)",
                                     (double)scale, causal, (long long)window, (long long)max_q);
    // tiles of 128 rows by 128 tokens are counted in 32 bits a CTA
    if (((double)T * (Hq / c->heads) / 128 + b->seqs) * c->heads * ((double)b->width * c->tokens / 128 + 1) >= 0x1p38)
        return (tq2_status)set_error(TQ2_ESHAPE, "kv8_attention: T=%lld rows over tables of %lld tokens are too many for one call",
                                     (long long)T, (long long)b->width * c->tokens);
    // each of a CTA's warps walks sequences without rows by itself, and none may be a second ahead of the others
    if (b->seqs > 1 << 24)
        return (tq2_status)set_error(TQ2_ESHAPE, "kv8_attention: %d sequences are too many for one call", b->seqs);
    if (T == 0) return TQ2_OK;
    if (!q || !out) return (tq2_status)set_error(TQ2_EINVAL, "kv8_attention: null pointer");
    if (off_element(q, element_size(dtype)) || off_element(out, element_size(dtype)) || off_element(lse, 4))
        return (tq2_status)set_error(TQ2_EINVAL, "kv8_attention: q, out and lse must be element-aligned");
    const uint32_t box = (uint32_t)(c->tokens < 64 ? c->tokens : 64);
    if (!make_tensor_map_2d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, c->codes, (uint64_t)c->dim,
                            (uint64_t)c->blocks * 2 * c->heads * c->tokens, (uint64_t)c->dim, (uint32_t)c->dim, box,
                            c->dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return (tq2_status)set_error(TQ2_ECUDA, "kv8_attention: the cache cannot be mapped for TMA");
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.qt = qt;
    a.qh = qh;
    a.ot = ot;
    a.oh = oh;
    a.dtype = dtype;
    a.G = Hq / c->heads;
    const int64_t size = (int64_t)element_size(dtype);
    a.qvec = (((int64_t)(uintptr_t)q | qt * size | qh * size) & 15) == 0;
    a.scale = scale2;
    a.causal = causal;
    a.window = window < ((int64_t)1 << 30) ? (int)window : 0;  // no sequence is longer
    // Rows of a sequence (queries * G): few go the streaming way, many the tensor cores'.  Which sequences have how
    // many the host does not know, so where both may be there both kernels are launched, each for its own; but where the
    // tables hold little, all go one way.  (8 sequences of 4096 tokens, 8 heads of 128, G = 4, bf16: 16 rows 24 us
    // streaming and 42 on the tensor cores, 32 rows 37 / 43, 64 rows 62 / 44.  f32, passes of 8 rows: 34 / 60, 58 / 61,
    // 103 / 63.  The second pair of kernels costs 7 us; few rows' codes stream at 5 TB/s and pass the tensor
    // cores at half of that, so 32 MB are worth it.)
    const int64_t rows = (max_q && max_q < T ? max_q : T) * a.G;
    const double held = 2.0 * b->seqs * b->width * c->tokens * c->heads * c->dim;
    // Warps of the tensor path that a piece of work leaves idle wait for the next one, and no wait may last a second: a
    // piece of 2^24 tokens takes 0.3 to 0.4 s (where scales are 2^40 apart 0.65, f32 0.7), a walk over 2^18 sequences
    // without rows as long.  Beyond those, all stream, where nothing waits for more than a chunk.
    const bool longest = (int64_t)b->width * c->tokens > 1 << 24 || b->seqs > 1 << 18;
    const bool few = rows <= KV8_FEW_ROWS || longest;
    a.few = few ? 0x7fffffff : b->seqs == 1 || held <= 32 << 20 ? 0 : KV8_FEW_ROWS;
    a.narrow = rows <= 8;
    const size_t stream_bytes = (kv8_stream_scratch(a) + 255) / 256 * 256;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Scratch mem(st);
    cudaError_t e = scratch_alloc(&mem.p, stream_bytes + (few ? 0 : kv8_umma_scratch(a)), st);
    if (e != cudaSuccess) {
        mem.p = nullptr;
        return cuda_status(e, "kv8_attention: scratch");
    }
    if (!few) e = launch_kv8_umma(a, static_cast<char*>(mem.p) + stream_bytes, st);
    if (e == cudaSuccess && a.few) e = launch_kv8_stream(a, mem.p, st);
    return cuda_status(e, "kv8_attention");
}

}  // extern "C"
