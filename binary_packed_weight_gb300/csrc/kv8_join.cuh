// kv8_join.cuh -- what both attention paths of the 8-bit cache share: the even cut of
// their work over the CTAs, and the kernel that joins what a cut divided.
#pragma once

#include "kv8.cuh"

namespace tq2 {

// CTAs' shares of `total` units: as even as can be, over as many CTAs as have `least` each.
struct Kv8Cut {
    long long base, more;
    int ctas;
    __device__ __forceinline__ Kv8Cut(long long total, int grid, int least) {
        const long long useful = total < least ? total > 0 : total / least;
        ctas = useful < grid ? (int)useful : grid;
        base = ctas ? total / ctas : 0;
        more = ctas ? total - base * ctas : 0;
    }
    __device__ __forceinline__ long long begin(int c) const { return c * base + (c < more ? c : more); }
    __device__ __forceinline__ int of(long long unit) const {
        const long long fat = more * (base + 1);
        return (int)(unit < fat ? unit / (base + 1) : more + (unit - fat) / base);
    }
};

// A tile of rows that a cut divided, noted by the CTA that has the first piece: that CTA's last
// piece (part 2 cta + 1), and the first ones (parts 2 (cta + i)) of the pieces-1 CTAs behind it.
struct Kv8Joint {
    int s, head, tile, pieces;
};

// A part: R references m of the values' sums, R sums l of the weights, R references n of those, R rows of D values' sums.
__host__ __device__ constexpr size_t kv8_part_floats(int rows, int D) { return (size_t)rows * (D + 3); }

// A row's values' sums, of 2^(s_t - m) v_t, and its weights' sum, of 2^(s_t - n), have references of their own: the first
// follows the largest weight times scale, and what is far below it is dropped there, but not from the second,
// whatever the scales are (blocks of zeros among large values; nothing but zeros, for a million tokens).  Where the
// scales at hand are at least 2^(m - n - NEAR), one exponential serves both: what it flushes to
// zero is below 2^(NEAR - 126) in the second, and it adds 2^(NEAR + RAISE) there at most.  Elsewhere the second has its own.
constexpr float KV8_NEAR = 40.f, KV8_FAR = 0x1p40f;          // an exponent, and the factor

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// What f16 left of a and b.
__device__ __forceinline__ uint32_t rest_half2(float a, float b, uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_half2(a - f.x, b - f.y);
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// One of the barrier's arrivals, when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A wait of a whole warp: where it runs out, or another role has given up, all lanes learn so and the other roles are told.
__device__ __forceinline__ bool kv8_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, bool spin) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, abort_flag, spin));
    if (!ok) *abort_flag = 1;
    return ok;
}

__device__ __forceinline__ float kv8_none() { return __int_as_float(0xff800000); }

// The power of two that takes a row of queries' largest element to 2^14 .. 2^15, in f16's range (below 2^-112: less far).
__device__ __forceinline__ int kv8_power(float most) { return min(max(141 - (int)(__float_as_uint(most) >> 23), -113), 126); }

// Where row r of a sequence's head goes in out; its place in lse.
__device__ __forceinline__ int64_t kv8_out_row(const Kv8Attention& a, int q0, int head, int r, int64_t* lse) {
    const int token = q0 + r / a.G, h = head * a.G + r % a.G;
    *lse = (int64_t)token * a.c.H * a.G + h;
    return token * a.ot + h * a.oh;
}
__device__ __forceinline__ float kv8_lse(float n, float l) {
    return l > 0.f || isnan(l) ? (log2f(l) + n) * 0.69314718055994531f : kv8_none();
}
// Factor that takes sums of reference m to those of reference top; sums without a reference are 0 or NaN.
__device__ __forceinline__ float kv8_factor(float m, float top) { return m == kv8_none() ? 1.f : exp2_fast(m - top); }
// What takes a row's values' sums to its result.
__device__ __forceinline__ float kv8_inverse(float m, float n, float l) { return l == 0.f ? 0.f : exp2_fast(m - n) / l; }

// The pieces' sums, each warp's in the order of the tokens and then those of the WPR warps that share a row: one
// where a row has few pieces and there are many rows, several where one sequence was cut over the whole GPU.
constexpr int KV8_JOIN_WARPS = 8;
template <class T, int D, int RM, int WPR>
__global__ void __launch_bounds__(KV8_JOIN_WARPS * 32)
kv8_join_kernel(const __grid_constant__ Kv8Attention a, const float* parts, const Kv8Joint* joints) {
    constexpr int RPB = KV8_JOIN_WARPS / WPR, PER = D / 32;  // rows a block at a time; a lane's columns
    constexpr size_t PART = kv8_part_floats(RM, D);
    __shared__ float os[KV8_JOIN_WARPS][D], ls[KV8_JOIN_WARPS];
    pdl_launch_dependents();
    pdl_wait();
    const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = warp % WPR;
    const Kv8Joint j = joints[cta];
    if (j.pieces == 0) return;
    const Kv8Seq q = kv8_seq(a.c, j.s);
    const int rows = min(q.n * a.G - j.tile * RM, RM);
    const float* first = parts + ((size_t)cta * 2 + 1) * PART;
    const float* rest = parts + (size_t)cta * 2 * PART;
    for (int r0 = blockIdx.y * RPB; r0 < rows; r0 += gridDim.y * RPB) {
        const int r = r0 + warp / WPR;
        const bool live = r < rows;
        float top = kv8_none(), top_n = kv8_none(), sum = 0.f, o[PER];
#pragma unroll
        for (int c = 0; c < PER; ++c) o[c] = 0.f;
        if (live) {
            for (int i = lane; i < j.pieces; i += 32) {
                const float* p = i ? rest + i * 2 * PART : first;
                top = fmaxf(top, p[r]);
                top_n = fmaxf(top_n, p[2 * RM + r]);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                top_n = fmaxf(top_n, __shfl_xor_sync(0xffffffffu, top_n, d));
            }
#pragma unroll 8
            for (int i = share; i < j.pieces; i += WPR) {
                const float* p = i ? rest + i * 2 * PART : first;
                const float f = kv8_factor(p[r], top);
                sum = fmaf(p[RM + r], kv8_factor(p[2 * RM + r], top_n), sum);
#pragma unroll
                for (int c = 0; c < PER; ++c) o[c] = fmaf(p[3 * RM + r * D + lane + 32 * c], f, o[c]);
            }
        }
        if (WPR > 1) {
#pragma unroll
            for (int c = 0; c < PER; ++c) os[warp][lane + 32 * c] = o[c];
            if (lane == 0) ls[warp] = sum;
            __syncthreads();
            if (share == 0) {
#pragma unroll
                for (int k = 1; k < WPR; ++k) {
                    sum += ls[warp + k];
#pragma unroll
                    for (int c = 0; c < PER; ++c) o[c] += os[warp + k][lane + 32 * c];
                }
            }
            __syncthreads();
        }
        if (live && share == 0) {
            int64_t at_lse;
            T* dst = static_cast<T*>(a.out) + kv8_out_row(a, q.q0, j.head, j.tile * RM + r, &at_lse);
            const float inv = kv8_inverse(top, top_n, sum);
#pragma unroll
            for (int c = 0; c < PER; ++c) dst[lane + 32 * c] = kv8_round<T>(o[c] * inv);
            if (lane == 0 && a.lse) a.lse[at_lse] = kv8_lse(top_n, sum);
        }
    }
}

}  // namespace tq2
