// q4_api.cu -- the C ABI of the 4-bit weights and of the routed experts:
// argument checks, device memory of the handles, scratch, launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <new>

#include "../../include/tq2.h"
#include "q4.cuh"
#include "tq2_internal.h"

namespace tq2 {

constexpr int MAX_DEVICES = 64;
static std::atomic<cudaMemPool_t> pools[MAX_DEVICES];   // of scratch, by device

// The library's stream-ordered pool of a device: like the device's default
// pool, except that freed scratch stays reserved over synchronizations (the
// default pool gives it back to the driver at each one, and the next call
// pays for mapping it again).
cudaError_t scratch_pool(cudaMemPool_t* pool) {
    static std::mutex lock;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= MAX_DEVICES) return cudaDeviceGetDefaultMemPool(pool, dev);
    *pool = pools[dev].load(std::memory_order_acquire);
    if (*pool) return cudaSuccess;
    std::lock_guard<std::mutex> hold(lock);
    *pool = pools[dev].load(std::memory_order_relaxed);
    if (*pool) return cudaSuccess;
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    // The first call may be part of a capture.  Making a pool is no work of a stream, but this thread may
    // not do it during one unless it says so.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    e = cudaMemPoolCreate(pool, &props);
    uint64_t keep = ~uint64_t(0);
    if (e == cudaSuccess) e = cudaMemPoolSetAttribute(*pool, cudaMemPoolAttrReleaseThreshold, &keep);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) e = back;
    if (e != cudaSuccess) return e;
    pools[dev].store(*pool, std::memory_order_release);
    return cudaSuccess;
}

cudaError_t scratch_alloc(void** p, size_t bytes, cudaStream_t st) {
    cudaMemPool_t pool = nullptr;
    cudaError_t e = scratch_pool(&pool);
    if (e != cudaSuccess) return e;
    return cudaMallocFromPoolAsync(p, bytes, pool, st);
}

cudaError_t launch_q4_stream(const Q4Stream& a, cudaStream_t st) {
    if (a.group == 32) return launch_q4_stream_g32(a, st);
    if (a.group == 64) return launch_q4_stream_g64(a, st);
    return launch_q4_stream_g128(a, st);
}

namespace {

tq2_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return TQ2_OK;
    return (tq2_status)set_error(e == cudaErrorMemoryAllocation ? TQ2_ENOMEM : TQ2_ECUDA, "%s: %s", what,
                                 cudaGetErrorString(e));
}

bool dtype_ok(int dtype) { return dtype == TQ2_F32 || dtype == TQ2_F16 || dtype == TQ2_BF16; }

bool format_ok(int64_t K, int group) {
    return (group == 32 || group == 64 || group == 128) && K >= group && K % group == 0 && K <= 32768;
}

// A plane as a device pointer: copied to *tmp if it is in host memory.
cudaError_t to_device(const void* p, size_t bytes, void** tmp, const void** dev, cudaStream_t st) {
    *tmp = nullptr;
    cudaPointerAttributes at = {};
    cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) return e;
    if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) {
        *dev = p;
        return cudaSuccess;
    }
    e = cudaMallocAsync(tmp, bytes, st);
    if (e != cudaSuccess) {
        *tmp = nullptr;
        return e;
    }
    *dev = *tmp;
    return cudaMemcpyAsync(*tmp, p, bytes, cudaMemcpyHostToDevice, st);
}

// out[t] = sum_j weights[t,j] y[t*k+j] over the routed j, in order.  A thread
// takes four columns of a token and reads its k rows four at a time, so that
// enough of the k*D*4 bytes a token are in flight to stream them (2048 tokens, k = 8,
// D = 2048: 134 MB in 26.2 us from DRAM).
template <class T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T>
__global__ void __launch_bounds__(256)
moe_combine_kernel(const float* __restrict__ y, const int32_t* __restrict__ ids, const float* __restrict__ weights,
                   T* __restrict__ out, int64_t ldo, int64_t T_, int D, int k) {
    pdl_launch_dependents();
    pdl_wait();
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 4;
    if (c >= D) return;                                    // (D is a multiple of 32)
    for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const float* p = y + t * k * D + c;
        for (int j0 = 0; j0 < k; j0 += 4) {
            float4 v[4];
            float w[4];
            bool on[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = j0 + i;
                on[i] = j < k && ids[t * k + j] >= 0;
                w[i] = on[i] ? weights[t * k + j] : 0.f;
                if (on[i]) v[i] = __ldcs(reinterpret_cast<const float4*>(p + (int64_t)j * D));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (on[i]) {
                    s[0] = fmaf(w[i], v[i].x, s[0]);
                    s[1] = fmaf(w[i], v[i].y, s[1]);
                    s[2] = fmaf(w[i], v[i].z, s[2]);
                    s[3] = fmaf(w[i], v[i].w, s[3]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) out[t * ldo + c + i] = round_to<T>(s[i]);
    }
}

template <class T>
cudaError_t launch_combine(const float* y, const int32_t* ids, const float* w, void* out, int64_t ldo, int64_t T_,
                           int D, int k, cudaStream_t st) {
    const unsigned gy = (unsigned)((D + 1023) / 1024);
    const unsigned gx = (unsigned)(T_ < 16384 ? T_ : 16384);
    return launch_pdl(moe_combine_kernel<T>, dim3(gx, gy), dim3(256), 0, st, y, ids, w, reinterpret_cast<T*>(out),
                      ldo, T_, D, k);
}

// Average rows of a matrix above which f16 and bf16 calls take the tensor-core
// path: beyond, the streaming products need a second tile of columns (64 experts of
// 2048x1024 bf16, groups of 128, 4 / 4.9 rows each: streaming 66 / 85 us, tensor cores
// 67 / 68; the one shape that was measured).
constexpr int64_t MOE_TENSOR_ROWS = 4;

// Whether every weight is an f16 number, as the tensor-core path decodes them; the streaming products scale the
// integers' sums in f32 and take any.  (A group's scale may be up to 65504, its weights 15 times that.)
bool fits_f16(const q4_weight* w) { return w->most <= 65504.f; }

// Whether the gated rows need a scale of their own.  The tensor-core path scales them as it
// makes them, by the bound |x|^2 |Gate row| |Up row| of the matrix's largest rows.  Products
// are about 1/sqrt(D) of |x| |row|, so values of a matrix's smallest rows are spread_gate
// spread_up D below the bound; f16 keeps 2^28 below it without losing bits, and four
// of its binades are left to rows of x that meet the weights less than chance would.
// (Of outputs to which all rows contribute alike, D = 7168: off by 2.1e-4 up to a spread
// of 2^11, 6.7e-4 at 2^14, 4e-2 at 2^20.)  With a pass of its own the scale is the row's
// maximum: 64 experts of 2048x1024 bf16, top 8, 2048 tokens 208 -> 241 us, 64 tokens 68 -> 72.
bool own_scale(const q4_weight* gate, const q4_weight* up) {
    return !((double)gate->spread * up->spread * (double)gate->K <= 0x1p24);
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

Q4Stream stream_of(const q4_weight* w) {
    Q4Stream a{};
    a.w0 = w->blocks;
    a.mstride = w->mstride;
    a.N = w->N;
    a.K = w->K;
    a.nkc = (int)w->nkc;
    a.zeros = w->zeros ? 1 : 0;
    a.group = w->group;
    a.E = (int)w->E;
    return a;
}

}  // namespace
}  // namespace tq2

using namespace tq2;

extern "C" {

tq2_status tq2_release_scratch(void) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < MAX_DEVICES) {
        cudaMemPool_t pool = pools[dev].load(std::memory_order_acquire);
        if (pool) e = cudaMemPoolTrimTo(pool, 0);
    }
    return cuda_status(e, "tq2_release_scratch");
}

tq2_status q4_upload(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t E, int64_t N,
                     int64_t K, int group, q4_handle* out, void* stream) {
    if (out) *out = nullptr;
    if (!codes || !scales || !out) return (tq2_status)set_error(TQ2_EINVAL, "q4_upload: null pointer");
    if (E < 1 || E > 1024 || N < 1 || N > (1 << 24) || !format_ok(K, group) || N * K > ((int64_t)1 << 36))
        return (tq2_status)set_error(TQ2_ESHAPE,
                                     "q4_upload: need 1 <= E <= 1024, 1 <= N <= 2^24, group 32, 64 or 128, K a "
                                     "multiple of it up to 32768, N*K <= 2^36 (E=%lld N=%lld K=%lld group=%d)",
                                     (long long)E, (long long)N, (long long)K, group);
    if (off_element(codes, 2) || off_element(scales, 2))
        return (tq2_status)set_error(TQ2_EINVAL, "q4_upload: codes and scales must be 2-byte aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    q4_weight* w = new (std::nothrow) q4_weight();
    if (!w) return (tq2_status)set_error(TQ2_ENOMEM, "q4_upload: host allocation");
    w->E = E;
    w->N = N;
    w->K = K;
    w->group = group;
    w->zeros = zeros != nullptr;
    w->nkc = (K + Q4_K - 1) / Q4_K;
    w->mstride = (N + 127) / 128 * 8 * w->nkc * q4_block_bytes(group, w->zeros);
    const size_t ngroups = (size_t)E * N * (K / group);
    void* tmp[3] = {nullptr, nullptr, nullptr};
    const void* dev[3] = {nullptr, nullptr, nullptr};
    // the bounds sit behind the blocks
    const size_t blocks_bytes = ((size_t)E * w->mstride + 255) / 256 * 256;
    cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&w->blocks), blocks_bytes + q4_bounds(E) * 4);
    if (e == cudaSuccess) w->bound = reinterpret_cast<float*>(w->blocks + blocks_bytes);
    if (e == cudaSuccess) e = to_device(codes, (size_t)E * N * (K / 2), &tmp[0], &dev[0], st);
    if (e == cudaSuccess) e = to_device(scales, ngroups * 2, &tmp[1], &dev[1], st);
    if (e == cudaSuccess && zeros) e = to_device(zeros, ngroups, &tmp[2], &dev[2], st);
    if (e == cudaSuccess)
        e = launch_q4_pack(static_cast<const uint8_t*>(dev[0]), static_cast<const uint16_t*>(dev[1]),
                           static_cast<const uint8_t*>(dev[2]), w, st);
    if (e == cudaSuccess)
        e = launch_q4_bound(static_cast<const uint8_t*>(dev[0]), static_cast<const uint16_t*>(dev[1]),
                            static_cast<const uint8_t*>(dev[2]), w, st);
    float bounds[q4_bounds(1024)];
    if (e == cudaSuccess) e = cudaMemcpyAsync(bounds, w->bound, q4_bounds(E) * 4, cudaMemcpyDeviceToHost, st);
    for (void* p : tmp)
        if (p) cudaFreeAsync(p, st);
    const cudaError_t done = cudaStreamSynchronize(st);        // the caller's planes are read, whatever happened
    if (e == cudaSuccess) e = done;
    if (e != cudaSuccess) {
        cudaFree(w->blocks);
        delete w;
        return cuda_status(e, "q4_upload");
    }
    for (int64_t i = 0; i < E; ++i)
        if (bounds[i] > w->spread * bounds[E + i]) w->spread = bounds[i] / bounds[E + i];
    w->most = bounds[2 * E];
    *out = w;
    return TQ2_OK;
}

tq2_status q4_free(q4_handle h) {
    if (!h) return TQ2_OK;
    cudaError_t e = cudaFree(h->blocks);
    delete h;
    return cuda_status(e, "q4_free");
}

tq2_status q4_shape(q4_handle h, int64_t* E, int64_t* N, int64_t* K, int* group) {
    if (!h) return (tq2_status)set_error(TQ2_EINVAL, "q4_shape: null handle");
    if (E) *E = h->E;
    if (N) *N = h->N;
    if (K) *K = h->K;
    if (group) *group = h->group;
    return TQ2_OK;
}

tq2_status q4_dequant(q4_handle h, float* w, void* stream) {
    if (!h || !w) return (tq2_status)set_error(TQ2_EINVAL, "q4_dequant: null pointer");
    if (off_element(w, 4)) return (tq2_status)set_error(TQ2_EINVAL, "q4_dequant: w must be 4-byte aligned");
    return cuda_status(launch_q4_dequant(h, w, reinterpret_cast<cudaStream_t>(stream)), "q4_dequant");
}

tq2_status q4_quantize(const void* w, int dtype, int64_t rows, int64_t K, int group, uint8_t* codes,
                       uint16_t* scales, uint8_t* zeros, void* stream) {
    if (!w || !codes || !scales) return (tq2_status)set_error(TQ2_EINVAL, "q4_quantize: null pointer");
    if (!dtype_ok(dtype)) return (tq2_status)set_error(TQ2_EINVAL, "q4_quantize: unknown dtype %d", dtype);
    if (rows < 1 || rows > ((int64_t)1 << 34) || !format_ok(K, group))
        return (tq2_status)set_error(TQ2_ESHAPE, "q4_quantize: bad shape (rows=%lld K=%lld group=%d)",
                                     (long long)rows, (long long)K, group);
    if (off_element(codes, 4) || off_element(scales, 2) || off_element(w, element_size(dtype)))
        return (tq2_status)set_error(TQ2_EINVAL, "q4_quantize: codes must be 4-byte aligned, w and scales element-aligned");
    return cuda_status(launch_q4_quantize(w, dtype, rows, K, group, codes, scales, zeros,
                                          reinterpret_cast<cudaStream_t>(stream)),
                       "q4_quantize");
}

tq2_status q4_gemm(q4_handle h, const void* x, int64_t ldx, void* out, int64_t ldo, int dtype, int64_t M,
                   void* stream) {
    if (!h) return (tq2_status)set_error(TQ2_EINVAL, "q4_gemm: null handle");
    if (!dtype_ok(dtype)) return (tq2_status)set_error(TQ2_EINVAL, "q4_gemm: unknown dtype %d", dtype);
    if (M < 0 || M > (1 << 20)) return (tq2_status)set_error(TQ2_ESHAPE, "q4_gemm: bad M=%lld", (long long)M);
    if (M == 0) return TQ2_OK;
    if (!x || !out) return (tq2_status)set_error(TQ2_EINVAL, "q4_gemm: null pointer");
    if (off_element(x, element_size(dtype)) || off_element(out, element_size(dtype)))
        return (tq2_status)set_error(TQ2_EINVAL, "q4_gemm: x and out must be element-aligned");
    if (h->E != 1)
        return (tq2_status)set_error(TQ2_ESHAPE, "q4_gemm: the handle holds %lld matrices, not one", (long long)h->E);
    if (ldx < h->K || ldo < h->N)
        return (tq2_status)set_error(TQ2_ESHAPE, "q4_gemm: row strides %lld, %lld are shorter than K=%lld, N=%lld",
                                     (long long)ldx, (long long)ldo, (long long)h->K, (long long)h->N);
    Q4Stream a = stream_of(h);
    a.x = x;
    a.ldx = ldx;
    a.xmode = dtype == TQ2_F32 ? Q4_X_SPLIT : Q4_X_RAW16;
    a.bf16 = dtype == TQ2_BF16;
    a.out = out;
    a.ldo = ldo;
    a.otype = dtype;
    a.M = (int)M;
    a.tokens = (int)(M < 32 ? M : 32);
    return cuda_status(launch_q4_stream(a, reinterpret_cast<cudaStream_t>(stream)), "q4_gemm");
}

tq2_status moe_experts(q4_handle gate, q4_handle up, q4_handle down, const void* x, int64_t ldx, int dtype,
                       const int32_t* ids, const float* weights, const int32_t* offsets, const int32_t* slots,
                       void* out, int64_t ldo, int64_t T, int k, void* stream) {
    if (!gate || !up || !down) return (tq2_status)set_error(TQ2_EINVAL, "moe_experts: null handle");
    if (!dtype_ok(dtype)) return (tq2_status)set_error(TQ2_EINVAL, "moe_experts: unknown dtype %d", dtype);
    if (T < 0 || T > (1 << 24) || k < 1 || k > 32 || T * k > (1 << 24))
        return (tq2_status)set_error(TQ2_ESHAPE, "moe_experts: bad T=%lld, k=%d", (long long)T, k);
    const int64_t D = gate->K, F = gate->N, E = gate->E;
    if (up->K != D || up->N != F || up->E != E || down->K != F || down->N != D || down->E != E ||
        up->group != gate->group || up->zeros != gate->zeros)
        return (tq2_status)set_error(TQ2_ESHAPE,
                                     "moe_experts: gate, up and down do not fit (%lldx%lldx%lld, %lldx%lldx%lld, "
                                     "%lldx%lldx%lld, or gate's and up's groups)",
                                     (long long)E, (long long)F, (long long)D, (long long)up->E, (long long)up->N,
                                     (long long)up->K, (long long)down->E, (long long)down->N, (long long)down->K);
    if (ldx < D || ldo < D)
        return (tq2_status)set_error(TQ2_ESHAPE, "moe_experts: row strides %lld, %lld are shorter than D=%lld",
                                     (long long)ldx, (long long)ldo, (long long)D);
    // a launch's row tiles are counted in 32 bits, of one row of x a pass at worst
    if ((T * k + E) * (D > 2 * F ? D : 2 * F) >= ((int64_t)1 << 35))
        return (tq2_status)set_error(TQ2_ESHAPE, "moe_experts: %lld slots of D=%lld, F=%lld are too many for one call",
                                     (long long)(T * k), (long long)D, (long long)F);
    if (T == 0) return TQ2_OK;
    if (!x || !ids || !weights || !offsets || !slots || !out)
        return (tq2_status)set_error(TQ2_EINVAL, "moe_experts: null pointer");
    if (off_element(x, element_size(dtype)) || off_element(out, element_size(dtype)) || off_element(ids, 4) ||
        off_element(weights, 4) || off_element(offsets, 4) || off_element(slots, 4))
        return (tq2_status)set_error(TQ2_EINVAL, "moe_experts: pointers must be element-aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t S = T * k;
    auto combine = [&](const float* y) {
        if (dtype == TQ2_F32) return launch_combine<float>(y, ids, weights, out, ldo, T, (int)D, k, st);
        if (dtype == TQ2_F16) return launch_combine<__half>(y, ids, weights, out, ldo, T, (int)D, k, st);
        return launch_combine<__nv_bfloat16>(y, ids, weights, out, ldo, T, (int)D, k, st);
    };
    Scratch mem(st);
    const size_t ybytes = ((size_t)S * D * 4 + 255) / 256 * 256;
    if (dtype != TQ2_F32 && S > MOE_TENSOR_ROWS * E && fits_f16(gate) && fits_f16(up) && fits_f16(down)) {
        const bool own = own_scale(gate, up);
        cudaError_t e = scratch_alloc(&mem.p, ybytes + moe_tensor_scratch(S, D, F, own), st);
        if (e != cudaSuccess) {
            mem.p = nullptr;
            return cuda_status(e, "moe_experts: scratch");
        }
        const MoeTensor m{gate, up, down, x, ldx, dtype, ids, offsets, slots, (int)S, k, static_cast<float*>(mem.p),
                          own};
        e = launch_moe_tensor(m, static_cast<char*>(mem.p) + ybytes, st);
        if (e == cudaSuccess) e = combine(m.y);
        return cuda_status(e, "moe_experts: tensor path");
    }
    cudaError_t e = scratch_alloc(&mem.p, ybytes + (size_t)S * F * 4, st);
    if (e != cudaSuccess) {
        mem.p = nullptr;
        return cuda_status(e, "moe_experts: scratch");
    }
    float* y = static_cast<float*>(mem.p);
    float* hid = reinterpret_cast<float*>(static_cast<char*>(mem.p) + ybytes);
    // rows of one expert: the average, and room for the spread around it
    const int64_t mean = (S + E - 1) / E;
    const int64_t spread = (mean + 2 * (int64_t)ceil(sqrt((double)mean)) + 7) / 8 * 8;
    const int64_t most = spread < T ? spread : T;
    Q4Stream a = stream_of(gate);
    a.w1 = up->blocks;
    a.pair = 1;
    a.x = x;
    a.ldx = ldx;
    a.xmode = dtype == TQ2_F32 ? Q4_X_SPLIT : Q4_X_RAW16;
    a.bf16 = dtype == TQ2_BF16;
    a.out = hid;                                              // by position of the plan
    a.ldo = F;
    a.otype = TQ2_F32;
    a.offsets = offsets;
    a.slots = slots;
    a.nslots = (int)S;
    a.xdiv = k;
    a.tokens = (int)(most < 32 ? most : 32);
    e = launch_q4_stream(a, st);
    if (e != cudaSuccess) return cuda_status(e, "moe_experts: gate and up");
    Q4Stream b = stream_of(down);
    b.x = hid;
    b.ldx = F;
    b.xmode = dtype == TQ2_F32 ? Q4_X_SPLIT : Q4_X_SCALED;
    b.out = y;                                                // by slot
    b.ldo = D;
    b.otype = TQ2_F32;
    b.oslot = 1;
    b.offsets = offsets;
    b.slots = slots;
    b.nslots = (int)S;
    b.tokens = a.tokens;
    b.after = 1;
    e = launch_q4_stream(b, st);
    if (e != cudaSuccess) return cuda_status(e, "moe_experts: down");
    e = combine(y);
    return cuda_status(e, "moe_experts: combine");
}

}  // extern "C"
