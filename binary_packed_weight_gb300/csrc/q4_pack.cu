// q4_pack.cu -- producers of the 4-bit weights: quantization, the device
// layout of q4.cuh from plain code planes, and its inverse.
//
// All three stream their operands once; none is on a decode path.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/tq2.h"
#include "q4.cuh"
#include "tq2_internal.h"

namespace tq2 {

namespace {

// One thread per 16 bytes of a block's codes; thread 0..15 of a block's first
// chunk also write its scales and zero points.
__global__ void __launch_bounds__(128)
q4_pack_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
               const uint8_t* __restrict__ zeros, uint8_t* __restrict__ blocks, int64_t N, int64_t K, int64_t nkc,
               int G, int64_t mstride, int64_t nblocks) {
    const int lane = threadIdx.x & 31, c = threadIdx.x >> 5;
    const int ng = Q4_K / G;
    const int64_t e = blockIdx.y;
    const int64_t kg = K / G;
    const int blk = q4_block_bytes(G, zeros != nullptr);
    codes += e * N * (K / 2);
    scales += e * N * kg;
    if (zeros) zeros += e * N * kg;
    blocks += e * mstride;
    for (int64_t b = blockIdx.x; b < nblocks; b += gridDim.x) {
        const int64_t sub = b & 7, kc = (b >> 3) % nkc, rt = ((b >> 3) / nkc) * 8 + sub;
        uint8_t* out = blocks + b * blk;
        const int g = lane & 7, t = lane >> 3;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = kc * 256 + c * 64 + 32 * (j & 1) + 8 * t, r = rt * 16 + g + 8 * (j >> 1);
            uint32_t p = zeros ? 0u : 0x88888888u;             // padding: the code of its zero point
            if (r < N && k < K) {
                const uint16_t* src = reinterpret_cast<const uint16_t*>(codes + r * (K / 2) + k / 2);
                p = src[0] | ((uint32_t)src[1] << 16);         // code i of k+i in bits 4i
            }
            w[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[j] |= ((p >> (4 * i)) & 15u) << (4 * (i >> 1) + 16 * (i & 1));
        }
        *reinterpret_cast<uint4*>(out + c * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        for (int i = threadIdx.x; i < 16 * ng; i += 128) {
            const int64_t r = rt * 16 + (i & 15), gi = kc * ng + (i >> 4);
            const bool in = r < N && gi < kg;
            const int at = q4_scale_index(i & 15, i >> 4, ng);
            reinterpret_cast<uint16_t*>(out + Q4_CODES)[at] = in ? scales[r * kg + gi] : (uint16_t)0;
            if (zeros) out[Q4_CODES + 32 * ng + at] = in ? (zeros[r * kg + gi] & 15) : 0;
        }
    }
}

// A warp a row: its 2-norm from the integers' squares, which are exact, each eight of
// them scaled by d^2; (1 + 2^-10) times that, so that no rounding makes a bound too small.
// A matrix's largest and smallest (of rows that are not 0) and the largest |d| max|c - z|
// of all are kept as the bits of non-negative floats: they have the floats' order,
// extremes have none of their own, and a largest NaN stays.
__global__ void __launch_bounds__(256)
q4_bound_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                const uint8_t* __restrict__ zeros, float* __restrict__ bound, int64_t N, int64_t K, int gshift) {
    __shared__ int cta[3];
    const int lane = threadIdx.x & 31;
    int* of = reinterpret_cast<int*>(bound);
    if (threadIdx.x < 3) cta[threadIdx.x] = threadIdx.x == 1 ? 0x7F7F7F7F : 0;
    __syncthreads();
    const int64_t kg = K >> gshift;
    codes += (int64_t)blockIdx.y * N * (K / 2);
    scales += (int64_t)blockIdx.y * N * kg;
    if (zeros) zeros += (int64_t)blockIdx.y * N * kg;
    int most = 0, least = 0x7F7F7F7F, weight = 0;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < N; r += (int64_t)gridDim.x * 8) {
        float s = 0.f;
        const uint16_t* row = reinterpret_cast<const uint16_t*>(codes + r * (K / 2));
#pragma unroll 4
        for (int k = lane * 8; k < (int)K; k += 256) {
            const uint32_t p = row[k / 4] | ((uint32_t)row[k / 4 + 1] << 16);
            const int64_t g = r * kg + (k >> gshift);
            const int z = zeros ? zeros[g] & 15 : 8;
            const float d = __half2float(__ushort_as_half(scales[g]));
            // sum (c - z)^2 = sum c^2 - 2 z sum c + 8 z^2
            const uint32_t lo = p & 0x0F0F0F0Fu, hi = (p >> 4) & 0x0F0F0F0Fu;
            const int c1 = (int)__dp4a(lo, 0x01010101u, __dp4a(hi, 0x01010101u, 0u));
            const int q = (int)__dp4a(lo, lo, __dp4a(hi, hi, 0u)) - 2 * z * c1 + 8 * z * z;
            weight = max(weight, __float_as_int(d * (float)max(z, 15 - z)) & 0x7FFFFFFF);
            s = fmaf(d * d, (float)q, s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int norm = __float_as_int(sqrtf(s) * (1.f + 0x1p-10f)) & 0x7FFFFFFF;
        most = max(most, norm);
        if (norm > 0) least = min(least, norm);
    }
    weight = __reduce_max_sync(0xffffffffu, weight);
    if (lane == 0) {
        atomicMax(cta, most);
        atomicMin(cta + 1, least);
        atomicMax(cta + 2, weight);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        atomicMax(of + blockIdx.y, cta[0]);
        atomicMin(of + gridDim.y + blockIdx.y, cta[1]);
        atomicMax(of + 2 * gridDim.y, cta[2]);
    }
}

// One thread per (row, 8 k): out[e][row][k..k+7], exact in f32 (5 + 11 bits).
__global__ void __launch_bounds__(256)
q4_dequant_kernel(const uint8_t* __restrict__ blocks, float* __restrict__ out, int64_t N, int64_t K, int64_t nkc,
                  int G, int zeros, int64_t mstride) {
    const int ng = Q4_K / G;
    const int blk = q4_block_bytes(G, zeros != 0);
    blocks += blockIdx.y * mstride;
    out += (int64_t)blockIdx.y * N * K;
    const int64_t total = N * (K / 8);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / (K / 8), k = (i % (K / 8)) * 8;
        const int r = (int)(row & 15);
        const int kk = (int)(k & 255);
        const uint8_t* b = blocks + q4_block_index(row >> 4, k >> 8, nkc) * blk;
        const int t = (kk & 31) >> 3;
        const uint32_t w = reinterpret_cast<const uint32_t*>(b + (kk >> 6) * 512 + (t * 8 + (r & 7)) * 16)
            [2 * (r >> 3) + ((kk >> 5) & 1)];
        const int at = q4_scale_index(r, kk / G, ng);
        const float d = __half2float(reinterpret_cast<const __half*>(b + Q4_CODES)[at]);
        const int z = zeros ? b[Q4_CODES + 32 * ng + at] : 8;
        float* o = out + row * K + k;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (float)((int)((w >> (4 * (i >> 1) + 16 * (i & 1))) & 15u) - z) * d;
    }
}

__device__ __forceinline__ float load_as_float(const void* p, int dtype, int64_t i) {
    if (dtype == TQ2_F32) return reinterpret_cast<const float*>(p)[i];
    if (dtype == TQ2_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// G/8 lanes per group, eight values a lane.  The scale is rounded to f16
// first and the codes are taken against the rounded scale.
__global__ void __launch_bounds__(256)
q4_quantize_kernel(const void* __restrict__ w, int dtype, int64_t ngroups, int G, uint8_t* __restrict__ codes,
                   uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
    const int lpg = G / 8;
    const int64_t nthreads = ngroups * lpg;
    const int64_t round = (nthreads + 31) / 32 * 32;          // whole warps, for the shuffles
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < round;
         i += (int64_t)gridDim.x * blockDim.x) {
        const bool in = i < nthreads;
        float v[8], lo = 0.f, hi = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = in ? load_as_float(w, dtype, i * 8 + j) : 0.f;
            lo = fminf(lo, v[j]);
            hi = fmaxf(hi, v[j]);
        }
        for (int o = lpg / 2; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        // with zero points the codes span [lo, hi] (0 included), else [-max, max] over -7..7
        const float want = zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
        const __half d16 = __float2half_rn(fminf(want, 65504.0f));
        const float d = __half2float(d16);
        const float z = zeros ? (d > 0.f ? fminf(fmaxf(rintf(-lo / d), 0.f), 15.f) : 0.f) : 8.f;
        uint32_t pack = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = d > 0.f ? fminf(fmaxf(rintf(v[j] / d) + z, 0.f), 15.f) : z;
            pack |= (uint32_t)q << (4 * j);
        }
        if (!in) continue;
        reinterpret_cast<uint32_t*>(codes)[i] = pack;
        if (i % lpg == 0) {
            scales[i / lpg] = __half_as_ushort(d16);
            if (zeros) zeros[i / lpg] = (uint8_t)z;
        }
    }
}

unsigned grid_of(int64_t blocks) {
    if (blocks < 1) blocks = 1;
    return (unsigned)(blocks < 4096 ? blocks : 4096);
}

}  // namespace

cudaError_t launch_q4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const q4_weight* w,
                           cudaStream_t st) {
    const int64_t nblocks = (w->N + 127) / 128 * 8 * w->nkc;
    q4_pack_kernel<<<dim3(grid_of(nblocks), (unsigned)w->E), 128, 0, st>>>(codes, scales, zeros, w->blocks, w->N,
                                                                         w->K, w->nkc, w->group, w->mstride, nblocks);
    return cudaGetLastError();
}

cudaError_t launch_q4_bound(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const q4_weight* w,
                            cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(w->bound, 0, q4_bounds(w->E) * 4, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(w->bound + w->E, 0x7F, (size_t)w->E * 4, st);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((w->N + 7) / 8 < 1024 ? (w->N + 7) / 8 : 1024);
    q4_bound_kernel<<<dim3(grid, (unsigned)w->E), 256, 0, st>>>(codes, scales, zeros, w->bound, w->N, w->K,
                                                               w->group == 32 ? 5 : w->group == 64 ? 6 : 7);
    return cudaGetLastError();
}

cudaError_t launch_q4_dequant(const q4_weight* w, float* out, cudaStream_t st) {
    q4_dequant_kernel<<<dim3(grid_of((w->N * (w->K / 8) + 255) / 256), (unsigned)w->E), 256, 0, st>>>(
        w->blocks, out, w->N, w->K, w->nkc, w->group, w->zeros ? 1 : 0, w->mstride);
    return cudaGetLastError();
}

cudaError_t launch_q4_quantize(const void* w, int dtype, int64_t rows, int64_t K, int group, uint8_t* codes,
                               uint16_t* scales, uint8_t* zeros, cudaStream_t st) {
    const int64_t ngroups = rows * (K / group);
    q4_quantize_kernel<<<grid_of((ngroups * (group / 8) + 255) / 256), 256, 0, st>>>(w, dtype, ngroups, group, codes,
                                                                                  scales, zeros);
    return cudaGetLastError();
}

}  // namespace tq2
