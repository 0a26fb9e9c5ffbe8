// q4_stream.cuh -- products of few activation rows with 4-bit weights.
//
//   out[m,n] = sum_k x[m,k] (c[n,k] - z[n,k/G]) d[n,k/G]
//            = sum_groups d[n,g] * sum_{k in g} x[m,k] (c[n,k] - z[n,g])
//
// The inner sums run on mma.sync with integer weights c - z, which are exact
// in f16 (bf16), and with x as it is (f16, bf16) or as two f16 parts whose sum
// is x to 2^-22 (f32; scaled per row by a power of two so that neither the
// f16 range nor its subnormals cut it); a group's sum is scaled by its d in
// f32.  So the only roundings are those of f32 accumulation.
//
// The weights are read once and bound the time.  The matrix is cut into units
// of 16-row tiles over the whole of k; a CTA walks a contiguous range of
// units, its eight warps splitting k (KS) and tiles (RT).  Each warp streams
// its own blocks into a private shared-memory ring by bulk copies issued a
// ring ahead (one contiguous block of q4.cuh each), so warps wait for each
// other only at the end of a unit, where the k parts are added in a fixed
// order.  The activations sit in shared memory for the CTA's whole life (one
// matrix) or per matrix of the plan.
//
// With a plan (offsets, slots) matrix e multiplies the rows of positions
// offsets[e]..offsets[e+1]; `pair` runs two matrices over the same rows and
// stores silu(first) * second.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/tq2.h"
#include "q4.cuh"
#include "tq2_internal.h"

namespace tq2 {

constexpr int Q4_WARPS = 8;
constexpr int Q4_MAX_DEPTH = 12;
constexpr int Q4_RED_PITCH = 20;       // floats of a 16-row column in the reduction buffer (conflict-free)

struct Q4Kernel {
    Q4Stream a;
    int tok;                           // rows of x a pass takes
    int parts;                         // f16 columns of a row
    int KS, RT, RU;                    // k splits x row tiles of the warps; units of a pass
    int depth;
    int pitch;                         // bytes of an activation column in shared memory
    int xvec;                          // rows of x are 16-byte aligned
    int off_prefix, off_scale, off_red, off_x, off_ring;   // shared-memory layout
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

template <bool BF>
__device__ __forceinline__ void q4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_16816_pure(d, a, b0, b1);
}

// The integer weights of a word as an A fragment.  f16: a nibble under the
// exponent of 1024 is 1024 + c (low) or 1024 + 16 c (bits 4..7); subtracting
// 1024 + z (1024 + 16 z) is exact, and rows g+8 come out times 16, which their
// scale takes back.  bf16 has 7 mantissa bits: every nibble is shifted low
// and read as 128 + c.
template <bool BF>
__device__ __forceinline__ void q4_decode(uint32_t w, uint32_t z0, uint32_t z1, uint32_t (&a)[4]) {
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    if (BF) {
        constexpr uint32_t M = 0x43004300u;
        const uint32_t v[4] = {(w & LO) | M, ((w >> 4) & LO) | M, ((w >> 8) & LO) | M, ((w >> 12) & LO) | M};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v[i]),
                                       *reinterpret_cast<const __nv_bfloat162*>((i & 1) ? &z1 : &z0));
            a[i] = *reinterpret_cast<uint32_t*>(&r);
        }
    } else {
        constexpr uint32_t M = 0x64006400u;
        const uint32_t w8 = w >> 8;
        const uint32_t v[4] = {(w & LO) | M, (w & HI) | M, (w8 & LO) | M, (w8 & HI) | M};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v[i]),
                                *reinterpret_cast<const __half2*>((i & 1) ? &z1 : &z0));
            a[i] = *reinterpret_cast<uint32_t*>(&r);
        }
    }
}

// A plan's values, kept inside their ranges whatever it holds.
__device__ __forceinline__ int q4_offset(const Q4Stream& a, int e) { return min(max(a.offsets[e], 0), a.nslots); }
__device__ __forceinline__ int q4_slot(const Q4Stream& a, int p) { return min(max(a.slots[p], 0), a.nslots - 1); }

// The plan's work: pass j (rows p0 .. p0+cnt of matrix e).
struct Q4Pass {
    int e, p0, cnt;
};
__device__ __forceinline__ Q4Pass q4_pass(const Q4Kernel& k, const int* prefix, int j) {
    Q4Pass p;
    if (!k.a.offsets) {
        p.e = 0;
        p.p0 = j * k.tok;
        p.cnt = min(k.tok, k.a.M - p.p0);
        return p;
    }
    int lo = 0, hi = k.a.E;                               // prefix[lo] <= j < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= j) lo = mid; else hi = mid;
    }
    p.e = lo;
    p.p0 = q4_offset(k.a, lo) + (j - prefix[lo]) * k.tok;
    p.cnt = min(k.tok, q4_offset(k.a, lo + 1) - p.p0);
    return p;
}

__device__ __forceinline__ int64_t q4_xrow(const Q4Kernel& k, int p) {
    return k.a.xdiv ? q4_slot(k.a, p) / k.a.xdiv : p;
}

// Activation rows of a pass into shared memory: column (row i, part q) at
// (i*parts + q)*pitch, f16 or bf16 in k order.  Rows are copied by the copy
// engine where they are 16-byte aligned; f32 rows are scaled to a largest
// magnitude of 2^14..2^15 and split.  Every thread of the CTA calls it.
__device__ __forceinline__ bool q4_stage_x(const Q4Kernel& k, uint8_t* smem, const Q4Pass& p, uint64_t* xbar,
                                           uint32_t& xphase) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* xs = smem + k.off_x;
    float* inv = reinterpret_cast<float*>(smem + k.off_scale);
    int* top = reinterpret_cast<int*>(inv + 32);
    const int K = (int)k.a.K;
    bool ok = true;
    fence_proxy_async_shared();
    __syncthreads();                                       // the previous rows and their scales are done with
    if (k.a.xmode == Q4_X_RAW16) {
        if (k.xvec) {
            if (warp == 0) {
                if (lane == 0) mbar_arrive_expect_tx(xbar, (uint32_t)(p.cnt * K * 2));
                __syncwarp();
                if (lane < p.cnt)
                    bulk_load(xs + lane * k.pitch,
                              reinterpret_cast<const uint16_t*>(k.a.x) + q4_xrow(k, p.p0 + lane) * k.a.ldx,
                              (uint32_t)K * 2, xbar);
            }
            ok = mbar_wait(xbar, xphase);
            xphase ^= 1u;
        } else {
            for (int i = warp; i < p.cnt; i += Q4_WARPS) {
                const uint16_t* src = reinterpret_cast<const uint16_t*>(k.a.x) + q4_xrow(k, p.p0 + i) * k.a.ldx;
                for (int c = lane; c < K; c += 32) reinterpret_cast<uint16_t*>(xs + i * k.pitch)[c] = src[c];
            }
            __syncthreads();
        }
        return ok;
    }
    if (tid < 32) top[tid] = 0;
    __syncthreads();
    // nw warps a row
    const int nw = p.cnt > 4 ? 1 : p.cnt > 2 ? 2 : p.cnt > 1 ? 4 : 8;
    const int step = nw * 32 * 4, first = ((warp & (nw - 1)) * 32 + lane) * 4;
    for (int i = warp / nw; i < p.cnt; i += Q4_WARPS / nw) {
        const float* src = reinterpret_cast<const float*>(k.a.x) + q4_xrow(k, p.p0 + i) * k.a.ldx;
        float m = 0.f;
        for (int c = first; c < K; c += step) {
            float4 v;
            if (k.xvec) v = *reinterpret_cast<const float4*>(src + c);
            else v = make_float4(src[c], src[c + 1], src[c + 2], src[c + 3]);
            m = fmaxf(fmaxf(fmaxf(m, fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) atomicMax(top + i, __float_as_int(m));  // m >= 0: the order of its bits; a maximum has no order
    }
    __syncthreads();
    const bool split = k.a.xmode == Q4_X_SPLIT;
    for (int i = warp / nw; i < p.cnt; i += Q4_WARPS / nw) {
        const float* src = reinterpret_cast<const float*>(k.a.x) + q4_xrow(k, p.p0 + i) * k.a.ldx;
        // 2^(14 - exponent of the maximum), kept a normal number; 1 for a row of zeros or one with infinities
        const int be = (top[i] >> 23) & 255;
        int se = 127 + 14 - (be - 127);
        if (be == 0) se = 253;
        if (top[i] == 0 || be == 255) se = 127;
        se = se > 253 ? 253 : se;
        const float s = __int_as_float(se << 23);
        if (lane == 0 && (warp & (nw - 1)) == 0) inv[i] = __int_as_float((254 - se) << 23);
        uint8_t* hi = xs + i * k.parts * k.pitch;
        uint8_t* lo = hi + k.pitch;
        for (int c = first; c < K; c += step) {
            float4 v;
            if (k.xvec) v = *reinterpret_cast<const float4*>(src + c);
            else v = make_float4(src[c], src[c + 1], src[c + 2], src[c + 3]);
            const float f[4] = {v.x * s, v.y * s, v.z * s, v.w * s};
            __half h[4], l[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                h[q] = __float2half_rn(f[q]);
                l[q] = __hisinf(h[q]) ? __ushort_as_half(0) : __float2half_rn(f[q] - __half2float(h[q]));
            }
            *reinterpret_cast<uint2*>(hi + c * 2) = *reinterpret_cast<uint2*>(h);
            if (split) *reinterpret_cast<uint2*>(lo + c * 2) = *reinterpret_cast<uint2*>(l);
        }
    }
    __syncthreads();
    return true;
}

template <int G, int NT, int RP, bool BF>
__global__ void __launch_bounds__(Q4_WARPS * 32, NT * RP <= 2 ? 2 : 1)
q4_stream_kernel(const __grid_constant__ Q4Kernel k) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NG = Q4_K / G;
    constexpr int NB = NT * RP <= 2 ? 2 : 1;               // reduction buffers
    constexpr int RED = Q4_WARPS * RP * NT * 8 * Q4_RED_PITCH;
    const Q4Stream& a = k.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int ks = warp & (k.KS - 1), rtw = warp / k.KS;
    const int blk = q4_block_bytes(G, a.zeros != 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem) + warp * Q4_MAX_DEPTH;
    uint64_t* xbar = reinterpret_cast<uint64_t*>(smem) + Q4_WARPS * Q4_MAX_DEPTH;
    int* prefix = reinterpret_cast<int*>(smem + k.off_prefix);
    const float* inv = reinterpret_cast<const float*>(smem + k.off_scale);
    float* red = reinterpret_cast<float*>(smem + k.off_red);
    uint8_t* ring = smem + k.off_ring + (size_t)warp * k.depth * RP * blk;
    const int nrt = (int)((a.N + 15) / 16);
    const int tpw = a.pair ? 1 : RP;                       // row tiles of a warp
    const int nkc = a.nkc;

    if (lane == 0)
        for (int d = 0; d < k.depth; ++d) mbar_init(&bars[d], 1);
    if (tid == 0) {
        mbar_init(xbar, 1);
        fence_mbar_init();
    }
    // k past the row's end is zero for the kernel's whole life
    for (int c = 0; c < k.tok * k.parts; ++c)
        for (int i = (int)a.K + 2 * tid; i < nkc * Q4_K; i += 2 * Q4_WARPS * 32)
            *reinterpret_cast<uint32_t*>(smem + k.off_x + c * k.pitch + i * 2) = 0u;
    if (lane == 0) fence_mbar_init();
    __syncthreads();
    pdl_launch_dependents();

    int passes;
    if (a.offsets) {
        pdl_wait();                                        // the plan is an earlier kernel's
        if (warp == 0) {
            int run = 0;
            for (int e0 = 0; e0 < a.E; e0 += 32) {
                const int e = e0 + lane;
                const int n = e < a.E ? max(q4_offset(a, e + 1) - q4_offset(a, e) + k.tok - 1, 0) / k.tok : 0;
                int s = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, s, o);
                    if (lane >= o) s += up;
                }
                if (e < a.E) prefix[e] = run + s - n;
                run += __shfl_sync(0xffffffffu, s, 31);
            }
            if (lane == 0) prefix[a.E] = run;
        }
        __syncthreads();
        passes = prefix[a.E];
    } else {
        passes = (a.M + k.tok - 1) / k.tok;
    }
    const int64_t units = (int64_t)passes * k.RU;
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);

    // the unit's blocks of this warp: chunk 0 of its row tiles, NULL past the last tile
    auto tiles = [&](int u, const uint8_t* (&b)[RP]) {
        const int j = u / k.RU, ru = u - j * k.RU;
        const int64_t e = a.offsets ? q4_pass(k, prefix, j).e : 0;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            const int rt = (ru * k.RT + rtw) * tpw + (a.pair ? 0 : r);
            const uint8_t* w = a.pair && r ? a.w1 : a.w0;
            b[r] = rt < nrt ? w + e * a.mstride + (q4_block_index(rt, 0, nkc)) * blk : nullptr;
        }
    };
    // the part of k a warp takes turns with the row unit, so that no warp always has the longer one
    auto first_chunk = [&](int u) { return (ks + u % k.RU) & (k.KS - 1); };
    // producer side: the next block to fetch
    int pu = u0, pkc = u0 < u1 ? first_chunk(u0) : 0, pit = 0, pslot = 0;
    const uint8_t* pb[RP];
    auto seek = [&]() {                                    // to the next unit with a tile of this warp
        while (pu < u1) {
            tiles(pu, pb);
            pkc = first_chunk(pu);
            if (pb[0]) return;
            ++pu;
        }
    };
    auto fetch = [&]() {
        if (pu >= u1) return;
        if (lane == 0) {
            const bool two = RP == 2 && pb[RP - 1] != nullptr;
            mbar_arrive_expect_tx(&bars[pslot], (uint32_t)(two ? 2 * blk : blk));
            uint8_t* dst = ring + (size_t)pslot * RP * blk;
            bulk_load(dst, pb[0] + (int64_t)pkc * 8 * blk, (uint32_t)blk, &bars[pslot]);
            if (two) bulk_load(dst + blk, pb[RP - 1] + (int64_t)pkc * 8 * blk, (uint32_t)blk, &bars[pslot]);
        }
        ++pit;
        if (++pslot == k.depth) pslot = 0;
        pkc += k.KS;
        if (pkc >= nkc) {
            ++pu;
            seek();
        }
    };
    seek();
    for (int d = 0; d < k.depth; ++d) fetch();
    if (!a.offsets) pdl_wait();                            // x is an earlier kernel's; the weights are not

    uint32_t xphase = 0, ph = 0;
    int slot = 0, it = 0;
    bool ok = true;
    int cur = -1;
    Q4Pass pass{0, 0, 0};
    const uint32_t xaddr = smem_u32(smem + k.off_x) + t * 16 + g * k.pitch;
    const uint32_t raddr = smem_u32(ring);
    int buf = 0;

    for (int u = u0; u < u1; ++u) {
        const int j = u / k.RU, ru = u - j * k.RU;
        if (j != cur) {
            cur = j;
            pass = q4_pass(k, prefix, j);
            if (!q4_stage_x(k, smem, pass, xbar, xphase)) ok = false;
        }
        const int cols = pass.cnt * k.parts;
        const int rt0 = (ru * k.RT + rtw) * tpw;
        float tot[RP][NT][4];
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[r][n][i] = 0.f;
        if (rt0 < nrt) {
            for (int kc = first_chunk(u); kc < nkc; kc += k.KS) {
                if (ok && !mbar_wait(&bars[slot], ph)) ok = false;
                const uint32_t base = raddr + (uint32_t)(slot * RP * blk);
                const uint8_t* sc = ring + (size_t)slot * RP * blk + Q4_CODES;
                float acc[RP][NT][4];
                float d0[RP], d1[RP];
                uint32_t z0[RP], z1[RP];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 wv[RP];
#pragma unroll
                    for (int r = 0; r < RP; ++r) wv[r] = lds128(base + (uint32_t)(r * blk + c * 512 + lane * 16));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        constexpr int HG = G / 32;             // halves of a group
                        const int half = c * 2 + h, gi = half / HG;
                        if (half % HG == 0) {
#pragma unroll
                            for (int r = 0; r < RP; ++r) {
                                const uint8_t* s = sc + r * blk;
                                d0[r] = __half2float(reinterpret_cast<const __half*>(s)[gi * 16 + g]);
                                d1[r] = __half2float(reinterpret_cast<const __half*>(s)[gi * 16 + g + 8]);
                                uint32_t za = 8, zb = 8;
                                if (a.zeros) {
                                    za = s[NG * 32 + gi * 16 + g];
                                    zb = s[NG * 32 + gi * 16 + g + 8];
                                }
                                if (BF) {
                                    z0[r] = 0x43004300u + za * 0x00010001u;
                                    z1[r] = 0x43004300u + zb * 0x00010001u;
                                } else {
                                    z0[r] = 0x64006400u + za * 0x00010001u;
                                    z1[r] = 0x64006400u + zb * 0x00100010u;
                                    d1[r] *= 0.0625f;
                                }
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.f;
                            }
                        }
                        uint4 b[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            b[n] = make_uint4(0, 0, 0, 0);
                            if (n * 8 + g < cols)
                                b[n] = lds128(xaddr + (uint32_t)(n * 8 * k.pitch + kc * 512 + c * 128 + h * 64));
                        }
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                            for (int r = 0; r < RP; ++r) {
                                uint32_t f[4];
                                q4_decode<BF>(h ? (jj ? wv[r].w : wv[r].z) : (jj ? wv[r].y : wv[r].x), z0[r], z1[r],
                                              f);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    if (n == 0 || n * 8 < cols)
                                        q4_mma<BF>(acc[r][n], f, jj ? b[n].z : b[n].x, jj ? b[n].w : b[n].y);
                            }
                        if (half % HG == HG - 1) {
#pragma unroll
                            for (int r = 0; r < RP; ++r)
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    tot[r][n][0] = fmaf(acc[r][n][0], d0[r], tot[r][n][0]);
                                    tot[r][n][1] = fmaf(acc[r][n][1], d0[r], tot[r][n][1]);
                                    tot[r][n][2] = fmaf(acc[r][n][2], d1[r], tot[r][n][2]);
                                    tot[r][n][3] = fmaf(acc[r][n][3], d1[r], tot[r][n][3]);
                                }
                        }
                    }
                }
                // the values are used: the slot is refilled through the async proxy
                fence_proxy_async_shared();
                __syncwarp();
                ++it;
                if (++slot == k.depth) { slot = 0; ph ^= 1u; }
                if (ok) fetch();
            }
        }
        // k parts and row tiles meet: [warp][r][column][16 rows]
        float* rb = red + buf * RED + warp * (RED / Q4_WARPS);
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n > 0 && n * 8 >= cols) continue;
                float* q = rb + ((r * NT + n) * 8 + 2 * t) * Q4_RED_PITCH + g;
                q[0] = tot[r][n][0];
                q[Q4_RED_PITCH] = tot[r][n][1];
                q[8] = tot[r][n][2];
                q[Q4_RED_PITCH + 8] = tot[r][n][3];
            }
        __syncthreads();
        const int rows = k.RT * tpw * 16;
        for (int i = tid; i < rows * pass.cnt; i += Q4_WARPS * 32) {
            const int m = i / rows, row = i - m * rows;
            const int64_t n = (int64_t)ru * rows + row;
            if (n >= a.N) continue;
            const int tile = row >> 4, w0 = (a.pair ? tile : tile / RP) * k.KS, r0 = a.pair ? 0 : tile % RP;
            auto sum = [&](int r) {                        // k parts in order, then the parts of x
                float v = 0.f;
                for (int q = 0; q < k.parts; ++q) {
                    const float* s = red + buf * RED + w0 * (RED / Q4_WARPS) +
                                     (r * NT * 8 + m * k.parts + q) * Q4_RED_PITCH + (row & 15);
                    for (int w = 0; w < k.KS; ++w) v += s[w * (RED / Q4_WARPS)];
                }
                return a.xmode == Q4_X_RAW16 ? v : v * inv[m];
            };
            float v = sum(r0);
            if (a.pair) {
                const float up = sum(RP - 1);
                v = v / (1.0f + expf(-v)) * up;
            }
            const int p = pass.p0 + m;
            const int64_t o = (a.oslot ? (int64_t)q4_slot(a, p) : (int64_t)p) * a.ldo + n;
            if (a.otype == TQ2_F32) reinterpret_cast<float*>(a.out)[o] = v;
            else if (a.otype == TQ2_F16) reinterpret_cast<__half*>(a.out)[o] = __float2half_rn(v);
            else reinterpret_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
        }
        if (NB == 1) __syncthreads();
        else buf ^= 1;
    }
    // every copy issued has landed before the CTA can exit (all were waited for unless a wait ran out)
    if (!ok)
        for (; it < pit; ++it) {
            mbar_wait(&bars[slot], ph);
            if (++slot == k.depth) { slot = 0; ph ^= 1u; }
        }
}

template <int G, int NT, int RP, bool BF>
cudaError_t q4_stream_launch(Q4Kernel& k, int tok, cudaStream_t st) {
    const Q4Stream& a = k.a;
    int dev = 0, sms = 152, optin = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    const int blk = q4_block_bytes(G, a.zeros != 0);
    const int nrt = (int)((a.N + 15) / 16), tpw = a.pair ? 1 : RP;
    k.tok = tok;
    // warps: split k while each warp keeps two chunks a unit, or while units would not fill the GPU
    int ks = 1;
    while (ks < Q4_WARPS && a.nkc >= 4 * ks) ks *= 2;
    while (ks < Q4_WARPS && a.nkc >= 2 * ks && (nrt + tpw * (Q4_WARPS / ks) - 1) / (tpw * (Q4_WARPS / ks)) * (a.offsets ? a.E : 1) < sms)
        ks *= 2;
    k.KS = ks;
    k.RT = Q4_WARPS / ks;
    k.RU = (nrt + tpw * k.RT - 1) / (tpw * k.RT);
    auto up = [](int v) { return (v + 127) / 128 * 128; };
    constexpr int NB = NT * RP <= 2 ? 2 : 1;
    k.off_prefix = up((Q4_WARPS * Q4_MAX_DEPTH + 1) * 8);
    k.off_scale = up(k.off_prefix + (a.offsets ? (a.E + 1) * 4 : 0));
    k.off_red = up(k.off_scale + 64 * 4);
    k.off_x = up(k.off_red + NB * Q4_WARPS * RP * NT * 8 * Q4_RED_PITCH * 4);
    k.off_ring = up(k.off_x + tok * k.parts * k.pitch);
    const int slot = Q4_WARPS * RP * blk;
    // two CTAs an SM when three ring slots a warp fit beside the rows (the
    // next launch on the stream then starts its weights early), else one
    const int half = (optin + 1024) / 2 - 1024;
    const int occ = NT * RP <= 2 && k.off_ring + 3 * slot <= half ? 2 : 1;
    k.depth = ((occ == 2 ? half : optin) - k.off_ring) / slot;
    if (k.depth > (occ == 2 ? 6 : Q4_MAX_DEPTH)) k.depth = occ == 2 ? 6 : Q4_MAX_DEPTH;
    if (k.depth < 1) return cudaErrorInvalidValue;
    const size_t smem = (size_t)k.off_ring + (size_t)k.depth * slot;
    cudaError_t e = cudaFuncSetAttribute(q4_stream_kernel<G, NT, RP, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    int64_t units = a.offsets ? (int64_t)sms * occ : (int64_t)((a.M + tok - 1) / tok) * k.RU;
    const int grid = (int)(units < (int64_t)sms * occ ? units : (int64_t)sms * occ);
    return launch_pdl(q4_stream_kernel<G, NT, RP, BF>, dim3((unsigned)grid), dim3(Q4_WARPS * 32), smem, st, k);
}

// The variant by sizes: column tiles (NT) for the rows a pass takes, limited
// by what shared memory holds beside two ring slots a warp; two row tiles a
// warp (RP) share the activations' shared-memory reads.
template <int G>
cudaError_t q4_stream_run(const Q4Stream& a, cudaStream_t st) {
    Q4Kernel k{};
    k.a = a;
    k.parts = a.xmode == Q4_X_SPLIT ? 2 : 1;
    k.pitch = a.nkc * Q4_K * 2 + 64;
    const int el = a.xmode == Q4_X_RAW16 ? 2 : 4;
    k.xvec = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (a.ldx * el) % 16 == 0;
    int dev = 0, optin = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    const int blk = q4_block_bytes(G, a.zeros != 0);
    const int nrt = (int)((a.N + 15) / 16);
    auto room = [&](int nt, int rp) {                      // columns that fit
        const int nb = nt * rp <= 2 ? 2 : 1;
        const int fixed = 2048 + (a.offsets ? (a.E + 1) * 4 : 0) + nb * Q4_WARPS * rp * nt * 8 * Q4_RED_PITCH * 4 +
                          2 * Q4_WARPS * rp * blk;
        const int c = (optin - fixed) / k.pitch;
        return c < 8 * nt ? (c < 0 ? 0 : c) : 8 * nt;
    };
    const int want = a.tokens * k.parts;
    auto tokens = [&](int nt, int rp) {
        const int c = room(nt, rp) / k.parts;
        return c < a.tokens ? c : a.tokens;
    };
    if (want > 16 && tokens(4, 2) > tokens(2, 2) && tokens(2, 2) > 0)
        return a.bf16 ? q4_stream_launch<G, 4, 2, true>(k, tokens(4, 2), st)
                      : q4_stream_launch<G, 4, 2, false>(k, tokens(4, 2), st);
    if (want > 8 && tokens(2, 2) > tokens(1, 2) && tokens(1, 2) > 0)
        return a.bf16 ? q4_stream_launch<G, 2, 2, true>(k, tokens(2, 2), st)
                      : q4_stream_launch<G, 2, 2, false>(k, tokens(2, 2), st);
    int sms = 152;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const bool wide = tokens(1, 2) > 0 && (a.pair || nrt >= 8 * sms);
    const int tok = wide ? tokens(1, 2) : tokens(1, 1);
    if (tok < 1 || (a.pair && !wide)) return cudaErrorInvalidValue;
    if (wide)
        return a.bf16 ? q4_stream_launch<G, 1, 2, true>(k, tok, st) : q4_stream_launch<G, 1, 2, false>(k, tok, st);
    return a.bf16 ? q4_stream_launch<G, 1, 1, true>(k, tok, st) : q4_stream_launch<G, 1, 1, false>(k, tok, st);
}

}  // namespace tq2
