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
//   codes   [4 chunks of 64 k][32 lanes][16 bytes]       2048 bytes
//   scales  f16 [8 rows g][256/G groups][row g, row g+8]
//   zeros   u8  the same                                  (if there are any)
// so all of a block that a lane of the products needs is a few wide loads.
// The 16 bytes of lane (g = lane/4, t = lane%4) are four words j; word j holds
// k = 32*(j/2) + 8t + 4*(j%2) + {0,1,2,3} of rows g and g+8, one nibble each:
//   bits  0.. 3 row g   k+0     16..19 row g   k+1
//   bits  4.. 7 row g+8 k+0     20..23 row g+8 k+1
//   bits  8..11 row g   k+2     24..27 row g   k+3
//   bits 12..15 row g+8 k+2     28..31 row g+8 k+3
// so a word masked with 0x000F000F << 4i is the pair a_i of the A fragment of
// mma.m16n8k16, one 16-byte load feeds four MMAs, and the MMA's k index maps
// to eight consecutive k for a lane: its B fragments of 32 k are 16 bytes of
// one activation row.
#pragma once

#include <cstddef>
#include <cstdint>
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

}  // namespace tq2

// Device memory of a 4-bit weight: E matrices of N x K.
struct q4_weight {
    int64_t E = 0, N = 0, K = 0;
    int group = 0;
    bool zeros = false;
    int64_t nkc = 0;                   // 256-k chunks of a row
    int64_t mstride = 0;               // bytes of one matrix
    uint8_t* blocks = nullptr;
    int device = 0;
};

namespace tq2 {

// q4_pack.cu
cudaError_t launch_q4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const q4_weight* w,
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
};
cudaError_t launch_q4_stream(const Q4Stream& a, cudaStream_t st);
cudaError_t launch_q4_stream_g32(const Q4Stream& a, cudaStream_t st);
cudaError_t launch_q4_stream_g64(const Q4Stream& a, cudaStream_t st);
cudaError_t launch_q4_stream_g128(const Q4Stream& a, cudaStream_t st);
unsigned int read_clear_dev_error_q4_g32(cudaStream_t st);
unsigned int read_clear_dev_error_q4_g64(cudaStream_t st);
unsigned int read_clear_dev_error_q4_g128(cudaStream_t st);

}  // namespace tq2
