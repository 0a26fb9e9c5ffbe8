// q4.cuh -- the 4-bit weight format of the library and its device layout.
//
//   W[n,k] = (c[n,k] - z[n,k/G]) * d[n,k/G],   c, z in 0..15, d f16,
//
// G = 32, 64 or 128 consecutive k to a group; without zero points z = 8.
//
// Device layout of one matrix ("blocks"): 16 rows x 256 k to a block, blocks in
// the order [128-row tile][256-k chunk][16-row tile of the 8], rows padded to
// a multiple of 128 and k to a multiple of 256 with codes equal to their zero
// point and scale 0, so padding contributes exactly nothing.  A block holds
//   codes   [4 chunks of 64 k][4 t][8 g][16 bytes]         2048 bytes
//   scales  f16 [8 rows g][256/G groups][row g, row g+8]
//   zeros   u8  the same                                  (if there are any)
// so all of a block that a lane of the products needs is a few wide loads.
// The 16 bytes at (t*8 + g)*16 of a chunk belong to lane (g, t) (lane 4g + t of
// the streaming products): words j = 0, 1 hold row g, words 2, 3 row g+8, and
// word j holds k = 32*(j%2) + 8t + i, i = 0..7, one nibble each:
//   bits 0..3: i=0   4..7: i=2   8..11: i=4   12..15: i=6
//   bits 16..19: i=1   20..23: i=3   24..27: i=5   28..31: i=7
// so a word masked with 0x000F000F << 4f is the pair (k+2f, k+2f+1): an A
// register of mma.m16n8k16, or a column of a row's f16 pairs in tensor memory.
// One 16-byte load feeds four MMAs, whose k index maps to eight consecutive k
// of a lane: its B fragments of 32 k are 16 bytes of one activation row.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace tq2 {

constexpr int Q4_ROWS = 16;            // rows of a block
constexpr int Q4_K = 256;              // k of a block
constexpr int Q4_CODES = Q4_ROWS * Q4_K / 2;

__host__ __device__ constexpr int q4_groups(int G) { return Q4_K / G; }
__host__ __device__ constexpr int q4_block_bytes(int G, bool zeros) {
    return Q4_CODES + Q4_ROWS * q4_groups(G) * (zeros ? 3 : 2);
}
// Place of row r (0..15) and group gi of a block among its scales (zeros).
__host__ __device__ constexpr int q4_scale_index(int r, int gi, int ng) { return ((r & 7) * ng + gi) * 2 + (r >> 3); }
// Block index of 16-row tile rt and 256-k chunk kc (nkc chunks a row).
__host__ __device__ inline int64_t q4_block_index(int64_t rt, int64_t kc, int64_t nkc) {
    return ((rt >> 3) * nkc + kc) * 8 + (rt & 7);
}

// The integer weights of four pairs of a word.  f16: a nibble under the
// exponent of 1024 is 1024 + c (low) or 1024 + 16 c (bits 4..7), and
// 1 * (1024 + c) - (1024 + z) and (1024 + 16 c) / 16 - (64 + z) are exact.  bf16
// has 7 mantissa bits: every nibble is shifted low and read as 128 + c.
// (M is a value of the register file that the compiler cannot see through: as a
// literal it is loaded anew for every word.)
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t m) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(m));
    return r;
}
template <bool BF>
__device__ __forceinline__ uint32_t q4_exponent() {
    uint32_t m;
    if (BF) asm volatile("mov.b32 %0, 0x43004300;" : "=r"(m));
    else asm volatile("mov.b32 %0, 0x64006400;" : "=r"(m));
    return m;
}
// What a row's zero point takes off: z0 from plain nibbles, z1 from those in bits 4..7 (f16).
struct Q4Zero {
    uint32_t z0, z1;
};
template <bool BF>
__device__ __forceinline__ Q4Zero q4_zero(uint32_t z) {
    const uint32_t zz = z * 0x00010001u;
    if (BF) return {zz + 0x43004300u, 0u};
    return {zz + 0x64006400u, zz * 16u + 0xD400D400u};      // 1024 + z; -(64 + z), whose ulp is 1/16
}
template <bool BF>
__device__ __forceinline__ void q4_decode(uint32_t w, uint32_t m, const Q4Zero& z, uint32_t (&a)[4]) {
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    const uint32_t w8 = w >> 8;
    const uint32_t v[4] = {and_or<LO>(w, m), BF ? and_or<LO>(w >> 4, m) : and_or<HI>(w, m), and_or<LO>(w8, m),
                           BF ? and_or<LO>(w >> 12, m) : and_or<HI>(w8, m)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF) {
            const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v[i]),
                                             *reinterpret_cast<const __nv_bfloat162*>(&z.z0));
            a[i] = *reinterpret_cast<const uint32_t*>(&r);
        } else if (i & 1) {
            const __half2 s = __float2half2_rn(0.0625f);
            const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v[i]), s,
                                      *reinterpret_cast<const __half2*>(&z.z1));
            a[i] = *reinterpret_cast<const uint32_t*>(&r);
        } else {
            const __half2 r =
                __hsub2(*reinterpret_cast<const __half2*>(&v[i]), *reinterpret_cast<const __half2*>(&z.z0));
            a[i] = *reinterpret_cast<const uint32_t*>(&r);
        }
    }
}

// This file's error record, read and cleared.  Until one of its kernels has been launched there is nothing
// in it, and a program that uses other calls pays for no round trip (nor for loading the kernels).
static std::atomic<bool> g_launched{false};
[[maybe_unused]] static unsigned int read_clear_record(cudaStream_t st) {
    if (!g_launched.load(std::memory_order_acquire)) return 0;
    unsigned int v = 0;
    const unsigned int none = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_dev_error, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess) return 0;
    cudaStreamSynchronize(st);
    if (v) cudaMemcpyToSymbolAsync(g_dev_error, &none, sizeof(none), 0, cudaMemcpyHostToDevice, st);
    return v;
}

// A plan's values, kept inside their ranges whatever it holds.
// (Read from L2: a kernel that starts before the one ahead of it has ended may read a plan.)
__device__ __forceinline__ int plan_offset(const int* offsets, int nslots, int e) {
    return min(max(__ldcg(offsets + e), 0), nslots);
}
__device__ __forceinline__ int plan_slot(const int* slots, int nslots, int p) {
    return min(max(__ldcg(slots + p), 0), nslots - 1);
}

}  // namespace tq2

// Device memory of a 4-bit weight: E matrices of N x K.
struct q4_weight {
    int64_t E = 0, N = 0, K = 0;
    int group = 0;
    bool zeros = false;
    int64_t nkc = 0;                   // 256-k chunks of a row
    int64_t mstride = 0;               // bytes of one matrix
    uint8_t* blocks = nullptr;
    float* bound = nullptr;            // [E] no row of W[e] has a larger 2-norm
    float spread = 1.f;                // within a matrix at most: largest row norm / smallest that is not 0
    float most = 0.f;                  // no weight is larger in magnitude (Inf or NaN where a scale is)
};

namespace tq2 {

// q4_pack.cu
cudaError_t launch_q4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const q4_weight* w,
                           cudaStream_t st);
// bound[E], each matrix's smallest row norm that is not 0 [E] and the largest weight [1], one after the other
constexpr size_t q4_bounds(int64_t E) { return (size_t)(2 * E + 1); }
cudaError_t launch_q4_bound(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const q4_weight* w,
                            cudaStream_t st);
cudaError_t launch_q4_dequant(const q4_weight* w, float* out, cudaStream_t st);
cudaError_t launch_q4_quantize(const void* w, int dtype, int64_t rows, int64_t K, int group, uint8_t* codes,
                               uint16_t* scales, uint8_t* zeros, cudaStream_t st);

// What one launch of the streaming product computes (q4_stream.cuh).
enum Q4XMode : int {
    Q4_X_RAW16 = 0,                    // x is f16 (bf16): rows copied as they are
    Q4_X_SCALED = 1,                   // x is f32: one f16 part, scaled by a power of two per row
    Q4_X_SPLIT = 2                     // x is f32: two f16 parts (hi + lo), scaled by a power of two per row
};
struct Q4Stream {
    const uint8_t* w0;                 // blocks of the matrices
    const uint8_t* w1;                 // pair: blocks of the second (up) matrices of the same shape
    int64_t mstride;
    int64_t N, K;
    int nkc, zeros, group;
    const void* x;
    int64_t ldx;                       // elements between rows
    int xmode, bf16;
    void* out;
    int64_t ldo;
    int otype;                         // tq2_dtype of out
    int pair;                          // out = silu(w0 x) * (w1 x)
    int E, M;                          // matrices; rows of x when there is no plan
    const int* offsets;                // plan (or NULL): E+1 row ranges of the matrices
    const int* slots;                  // position -> slot
    int nslots;                        // slots of the plan, routed or not
    int xdiv;                          // x row of position p: slots[p] / xdiv; 0: p itself
    int oslot;                         // out row of position p: slots[p]; 0: p itself
    int tokens;                        // rows expected of one matrix at most (sizes the column tiles)
    int after;                         // the last kernel of the stream is a product over the same plan
};
cudaError_t launch_q4_stream(const Q4Stream& a, cudaStream_t st);
cudaError_t launch_q4_stream_g32(const Q4Stream& a, cudaStream_t st);
cudaError_t launch_q4_stream_g64(const Q4Stream& a, cudaStream_t st);
cudaError_t launch_q4_stream_g128(const Q4Stream& a, cudaStream_t st);
unsigned int read_clear_dev_error_q4_g32(cudaStream_t st);
unsigned int read_clear_dev_error_q4_g64(cudaStream_t st);
unsigned int read_clear_dev_error_q4_g128(cudaStream_t st);

// moe_umma.cu: the routed experts on the tensor cores (f16 and bf16 rows).
struct MoeTensor {
    const q4_weight *gate, *up, *down;
    const void* x;
    int64_t ldx;
    int dtype;
    const int* ids;
    const int* offsets;
    const int* slots;
    int nslots, k;
    float* y;                          // [slot][D]
    bool own_scale;                    // gated rows are scaled by their own maximum, in a pass of their own
};
size_t moe_tensor_scratch(int64_t nslots, int64_t D, int64_t F, bool own_scale);
cudaError_t launch_moe_tensor(const MoeTensor& m, void* scratch, cudaStream_t st);
unsigned int read_clear_dev_error_moe_umma(cudaStream_t st);

}  // namespace tq2
