// kv8_cache.cu -- new tokens into the 8-bit cache, and tokens out of it.
//
// A CTA takes a block of B tokens in one head, of the keys or of the values: all
// that shares a scale.  Its new values stay in registers between the maximum
// and the codes, so each is read once.  Both kernels move bytes and little else: 65536 tokens
// of 8 heads of 128 are read as bf16 at 6.4 TB/s (63 us; 96 % of the measured copy).  The write
// has one exchange of the maximum between a CTA's loads and its stores, which the SM's other CTAs
// cover in part, and 21 instructions a value: 13518 tokens as bf16 at 3.9 TB/s (21.4 us, issue slots 73 % busy).
// A decoded token: 4.1 us, launch and four dependent reads.  f32 is read back at 4.1 TB/s (163 us for the tokens above).
#include <cfloat>

#include "kv8.cuh"

namespace tq2 {
namespace {

constexpr int CHUNK = 16;       // elements a thread takes at a time: 16 codes are one 16-byte store
constexpr int MAX_THREADS = 256;

// A block's chunks, one, two or four a thread.
int chunks_of(const Kv8View& c) { return (c.D << c.logB) / CHUNK; }
int threads_of(const Kv8View& c) { return chunks_of(c) < MAX_THREADS ? chunks_of(c) : MAX_THREADS; }

// CTAs of a writing SM: what bounds it is a CTA's chain of loads, maximum and stores, so as many as hold their values.
template <class T, int PER>
constexpr int ctas() { return PER * sizeof(T) <= 4 ? 5 : PER * sizeof(T) <= 8 ? 3 : 2; }

// Blocks of a sequence are dealt over gridDim.z CTAs: enough for a lone prompt to fill the GPU, and no more than twice
// the average sequence's blocks (10 sequences of 1500 tokens in blocks of 16, with a CTA for every block there could be:
// 5.6 us, so 4.1).
dim3 grid_of(const Kv8View& c) {
    const int64_t most = 2 * (int64_t)c.T / ((int64_t)c.seqs << c.logB) + 1;
    const int64_t fill = (int64_t)kv8_sm_count() * 32 / ((int64_t)c.seqs * c.H * 2) + 1;
    return dim3((unsigned)c.seqs, (unsigned)(c.H * 2), (unsigned)(most < fill ? most : fill));
}

// Values below 2^-96 count as zeros, so that a scale and its reciprocal are normal numbers.
constexpr float SMALLEST = 0x1p-96f;

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* shared) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();                                         // the last block's maximum has been read
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    v = shared[0];
    for (int i = 1; i < warps; ++i) v = max(v, shared[i]);
    return v;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    // whole numbers of -127..127 above 1.5 * 2^23 have their value in the low byte
    const float magic = 12583040.f;                          // 1.5 * 2^23 + 128
    const uint32_t lo = __byte_perm(__float_as_uint(a + magic), __float_as_uint(b + magic), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(c + magic), __float_as_uint(d + magic), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

__device__ __forceinline__ float code_of(float x, float inverse) {
    return fminf(fmaxf(rintf(__fmul_rn(x, inverse)), -127.f), 127.f);
}

template <class T, int PER>
__global__ void __launch_bounds__(MAX_THREADS, ctas<T, PER>())
kv8_write_kernel(const Kv8View c, const T* k, const T* v, int64_t kt, int64_t kh, int64_t vt, int64_t vh, bool vec) {
    __shared__ uint32_t shared[MAX_THREADS / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int s = blockIdx.x, head = blockIdx.y >> 1, kv = blockIdx.y & 1;
    const Kv8Seq q = kv8_seq(c, s);
    if (q.n == 0 || q.len == 0) return;
    const T* x = kv ? v : k;
    const int64_t xt = kv ? vt : kt, xh = kv ? vh : kh;
    const int B = 1 << c.logB, logR = c.D == 128 ? 3 : 2, chunks = 1 << (logR + c.logB);   // a row's chunks, a block's
    const int start = q.len - q.n;                           // below 0: tokens that no position is left for
    const int first = max(start, 0);
    constexpr int W = CHUNK * (int)sizeof(T) / 16;
    for (int b = (first >> c.logB) + blockIdx.z; (b << c.logB) < q.len; b += gridDim.z) {
        const int base = b << c.logB;
        const int lo = max(first - base, 0), hi = min(q.len - base, B);   // new tokens of the block
        // the values stay as they came between the maximum and the codes
        uint4 raw[PER][W];
        const T* from = x + (q.q0 + (base - start)) * xt + head * xh;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = threadIdx.x + i * blockDim.x, token = at >> logR;
#pragma unroll
            for (int k = 0; k < W; ++k) raw[i][k] = make_uint4(0, 0, 0, 0);
            if (at < chunks && token >= lo && token < hi) {
                const T* p = from + token * xt + (at & ((1 << logR) - 1)) * CHUNK;
                if (vec) {
#pragma unroll
                    for (int k = 0; k < W; ++k) raw[i][k] = __ldcs(reinterpret_cast<const uint4*>(p) + k);
                } else {
                    T* e = reinterpret_cast<T*>(raw[i]);
#pragma unroll
                    for (int k = 0; k < CHUNK; ++k) e[k] = p[k];
                }
            }
        }
        const int block = kv8_block(c, s, base);
        float* where = c.scales + ((int64_t)max(block, 0) * 2 + kv) * c.H + head;
        const float before = lo > 0 && block >= 0 ? *where : 0.f;
        uint32_t peak = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const T* e = reinterpret_cast<const T*>(raw[i]);
#pragma unroll
            for (int k = 0; k < CHUNK; ++k) peak = max(peak, __float_as_uint(kv8_wide(e[k])) & 0x7fffffffu);
        }
        peak = block_max(peak, shared);                      // (behind it, every thread has read the scale)
        if (block < 0) continue;
        const float most = __uint_as_float(peak);
        // a value that is no number leaves none in the block
        const float fresh = peak >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                                                : most >= SMALLEST ? __fdiv_rn(most, 127.f) : 0.f;
        const bool bad = isnan(before) || isnan(fresh);
        const float now = bad ? __uint_as_float(0x7fffffffu) : fmaxf(before, fresh);
        const float inverse = now > 0.f ? fminf(__fdiv_rn(1.f, now), FLT_MAX) : 0.f;
        const bool coarser = lo > 0 && now > before;
        const float ratio = coarser ? __fdiv_rn(before, now) : 1.f;
        if (threadIdx.x == 0 && (lo == 0 || bad || coarser)) *where = now;
        uint4* codes = reinterpret_cast<uint4*>(c.codes + kv8_row(c, block, kv, head) * c.D);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = threadIdx.x + i * blockDim.x, token = at >> logR;
            if (at >= chunks || token >= hi) continue;
            if (token >= lo) {
                const T* e = reinterpret_cast<const T*>(raw[i]);
                uint4 w;
                uint32_t* o = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = pack4(code_of(kv8_wide(e[4 * j]), inverse), code_of(kv8_wide(e[4 * j + 1]), inverse),
                                 code_of(kv8_wide(e[4 * j + 2]), inverse), code_of(kv8_wide(e[4 * j + 3]), inverse));
                codes[at] = w;
            } else if (coarser) {
                uint4 w = codes[at];
                uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float z[4];
#pragma unroll
                    for (int l = 0; l < 4; ++l) z[l] = code_of((float)((int)(e[j] >> (8 * l) & 255u) - 128), ratio);
                    e[j] = pack4(z[0], z[1], z[2], z[3]);
                }
                codes[at] = w;
            }
        }
    }
}

template <class T>
__global__ void __launch_bounds__(MAX_THREADS)
kv8_read_kernel(const Kv8View c, T* k, T* v, int64_t kt, int64_t kh, int64_t vt, int64_t vh, bool vec) {
    pdl_launch_dependents();
    pdl_wait();
    const int s = blockIdx.x, head = blockIdx.y >> 1, kv = blockIdx.y & 1;
    const Kv8Seq q = kv8_seq(c, s);
    if (q.n == 0 || q.len == 0) return;
    T* x = kv ? v : k;
    const int64_t xt = kv ? vt : kt, xh = kv ? vh : kh;
    const int B = 1 << c.logB, per_row = c.D / CHUNK, chunks = per_row << c.logB;
    const int start = q.len - q.n, first = max(start, 0);
    for (int b = (first >> c.logB) + blockIdx.z; (b << c.logB) < q.len; b += gridDim.z) {
        const int block = kv8_block(c, s, b << c.logB);
        if (block < 0) continue;
        const int base = b << c.logB;
        const int lo = max(first - base, 0), hi = min(q.len - base, B);
        const float scale = c.scales[((int64_t)block * 2 + kv) * c.H + head];
        const uint4* codes = reinterpret_cast<const uint4*>(c.codes + kv8_row(c, block, kv, head) * c.D);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = threadIdx.x + i * blockDim.x, token = at / per_row;
            if (at >= chunks || token < lo || token >= hi) continue;
            const uint4 w = codes[at];
            const uint32_t* e = reinterpret_cast<const uint32_t*>(&w);
            float y[CHUNK];
#pragma unroll
            for (int j = 0; j < CHUNK; ++j)
                y[j] = __fmul_rn((float)((int)(e[j / 4] >> (8 * (j & 3)) & 255u) - 128), scale);
            kv8_store16(x + (q.q0 + (base + token - start)) * xt + head * xh + (at % per_row) * CHUNK, vec, y);
        }
    }
}

bool vectors(const Kv8Rows& r) {
    const int64_t size = (int64_t)element_size(r.dtype);
    const int64_t all = (int64_t)(uintptr_t)r.k | (int64_t)(uintptr_t)r.v | r.kt * size | r.kh * size | r.vt * size | r.vh * size;
    return (all & 15) == 0;
}

template <class T>
cudaError_t write_as(const Kv8View& c, const Kv8Rows& r, cudaStream_t st) {
    auto kernel = chunks_of(c) > 2 * MAX_THREADS ? kv8_write_kernel<T, 4>
                  : chunks_of(c) > MAX_THREADS ? kv8_write_kernel<T, 2> : kv8_write_kernel<T, 1>;
    return launch_pdl(kernel, grid_of(c), dim3(threads_of(c)), 0, st, c, static_cast<const T*>(r.k),
                      static_cast<const T*>(r.v), r.kt, r.kh, r.vt, r.vh, vectors(r));
}
template <class T>
cudaError_t read_as(const Kv8View& c, const Kv8Rows& r, cudaStream_t st) {
    return launch_pdl(kv8_read_kernel<T>, grid_of(c), dim3(threads_of(c)), 0, st, c, static_cast<T*>(r.k),
                      static_cast<T*>(r.v), r.kt, r.kh, r.vt, r.vh, vectors(r));
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8View& c, const Kv8Rows& r, cudaStream_t st) {
    if (r.dtype == TQ2_F32) return write_as<float>(c, r, st);
    if (r.dtype == TQ2_F16) return write_as<__half>(c, r, st);
    return write_as<__nv_bfloat16>(c, r, st);
}

cudaError_t launch_kv8_read(const Kv8View& c, const Kv8Rows& r, cudaStream_t st) {
    if (r.dtype == TQ2_F32) return read_as<float>(c, r, st);
    if (r.dtype == TQ2_F16) return read_as<__half>(c, r, st);
    return read_as<__nv_bfloat16>(c, r, st);
}

}  // namespace tq2
