// kv8.cuh -- the 8-bit cache of keys and values as its kernels see it.
//
// Codes are uint8[blocks][2][H][B][D] (keys, then values), with one f32 scale for
// the B tokens of a block in a head, float[blocks][2][H]: x = (c - 128) * scale.
// A sequence's tokens lie in the blocks of its row of the table, B at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"
#include "tq2_internal.h"

namespace tq2 {

struct Kv8View {
    uint8_t* codes;
    float* scales;
    const int32_t* table;
    const int32_t* offsets;
    const int32_t* lens;
    int64_t ld;       // of the table's rows
    int blocks, H, logB, D;
    int width, seqs;
    int T;            // rows of the call's new tokens or queries
};

// New tokens or queries of a sequence: rows q0 .. q0+n-1, at positions len-n .. len-1.  Offsets
// and lengths of any contents stay inside the rows and the table.
struct Kv8Seq {
    int q0, n, len;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8View& c, int s) {
    Kv8Seq r;
    r.q0 = min(max(c.offsets[s], 0), c.T);
    r.n = min(max(c.offsets[s + 1], r.q0), c.T) - r.q0;
    const int64_t most = (int64_t)c.width << c.logB;
    const int len = max(c.lens[s], 0);
    r.len = len < most ? len : (int)most;
    return r;
}

// The block of a token, or -1 where the table names none.
__device__ __forceinline__ int kv8_block(const Kv8View& c, int s, int token) {
    const int b = c.table[s * c.ld + (token >> c.logB)];
    return (unsigned)b < (unsigned)c.blocks ? b : -1;
}

// First code of a block's head: kv 0 keys, 1 values.
__device__ __forceinline__ int64_t kv8_row(const Kv8View& c, int block, int kv, int head) {
    return (((int64_t)block * 2 + kv) * c.H + head) << c.logB;
}

template <class T>
__device__ __forceinline__ T kv8_round(float v);
template <>
__device__ __forceinline__ float kv8_round<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half kv8_round<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 kv8_round<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float kv8_wide(float v) { return v; }
__device__ __forceinline__ float kv8_wide(__half v) { return __half2float(v); }
__device__ __forceinline__ float kv8_wide(__nv_bfloat16 v) { return __bfloat162float(v); }

// Sixteen neighbouring elements as f32; vec: p is 16-byte aligned.
template <class T>
__device__ __forceinline__ void kv8_load16(const T* p, bool vec, float (&x)[16]) {
    constexpr int N = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < 16 / N; ++i) {
            const uint4 w = reinterpret_cast<const uint4*>(p)[i];
            const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int j = 0; j < N; ++j) x[i * N + j] = kv8_wide(e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = kv8_wide(p[i]);
    }
}

template <class T>
__device__ __forceinline__ void kv8_store16(T* p, bool vec, const float (&x)[16]) {
    constexpr int N = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < 16 / N; ++i) {
            uint4 w;
            T* e = reinterpret_cast<T*>(&w);
#pragma unroll
            for (int j = 0; j < N; ++j) e[j] = kv8_round<T>(x[i * N + j]);
            reinterpret_cast<uint4*>(p)[i] = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = kv8_round<T>(x[i]);
    }
}

// The two codes in bytes B0, B0+1 of w as an f16 pair c - 128: a byte under the
// exponent of 1024 is 1024 + c, exact.
template <int B0>
__device__ __forceinline__ uint32_t kv8_pair(uint32_t w) {
    const uint32_t v = __byte_perm(w, 0x64646464u, B0 == 0 ? 0x4140 : 0x4342);
    const uint32_t bias = 0x64806480u;                       // 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// ------------------------------------------------------------ launches ----
inline int kv8_sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    return n;
}

// Keys and values of a write or a read: strides in elements.
struct Kv8Rows {
    void *k, *v;
    int64_t kt, kh, vt, vh;
    int dtype;
};
cudaError_t launch_kv8_write(const Kv8View& c, const Kv8Rows& r, cudaStream_t st);
cudaError_t launch_kv8_read(const Kv8View& c, const Kv8Rows& r, cudaStream_t st);

struct Kv8Attention {
    Kv8View c;
    CUtensorMap map;            // codes as rows of D bytes, boxes of min(B, 64) rows
    const void* q;
    void* out;
    float* lse;                 // [T][Hq] or NULL
    int64_t qt, qh, ot, oh;     // strides in elements
    int dtype, G;               // query heads a head of the cache
    int qvec;                   // rows of q are 16-byte aligned
    int narrow;                 // no sequence has more than 8 rows
    float scale;                // softmax scale * log2(e)
    int causal, window;
    int few;                    // sequences of at most so many rows (queries * G) are the streaming path's
};
constexpr int KV8_FEW_ROWS = 32;  // of a sequence: where there are no more, the streaming path is faster
size_t kv8_stream_scratch(const Kv8Attention& a);
cudaError_t launch_kv8_stream(const Kv8Attention& a, void* scratch, cudaStream_t st);
unsigned int read_clear_dev_error_kv8_stream(cudaStream_t st);
size_t kv8_umma_scratch(const Kv8Attention& a);
cudaError_t launch_kv8_umma(const Kv8Attention& a, void* scratch, cudaStream_t st);
unsigned int read_clear_dev_error_kv8_umma(cudaStream_t st);

}  // namespace tq2
