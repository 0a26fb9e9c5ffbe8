// moe_umma.cu -- the routed experts' products for many tokens, on tcgen05.
//
// Per matrix e of the plan, rows p of its positions, W = (c - z) d:
//   hidden[p] = silu(Gate x[p]) * (Up x[p]),   y[slot(p)] = Down hidden[p]
//
// Both products are D[n, p] = sum_k W[n,k] act[p,k] with 128 weight rows and up
// to 192 positions a tile, f16 operands and f32 accumulators in tensor memory:
//   * warp 0 streams the activations (B, 64 k a stage, 128-byte swizzle) by TMA;
//   * warp 3 streams the packed blocks of 256 k by bulk copies;
//   * warps 4..11 decode a block's rows, one weight row a thread, and store
//     them as the A operand in tensor memory (rounding (c - z) d to f16 is
//     the only rounding of the weights);
//   * warp 1 issues the MMAs into one of two accumulators; warps 12..15 and
//     16..19 drain one each while the other fills.
// A tile of the first product holds 64 rows of Gate and the same 64 of Up: lanes
// 0..15 of each quarter are Gate's, 16..31 Up's, so one shuffle meets the two.
//
// f16 holds the activations because each row is scaled by a power of two: a
// row of x so that its largest magnitude is 2^14..2^15, a hidden row by its
// bound |x|^2 bound(Gate) bound(Up) (Cauchy-Schwarz; silu(v) <= |v|), which
// can only be too large, by about 2^16 for ordinary rows, and leaves 13 binades
// of full precision below them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/tq2.h"
#include "q4.cuh"
#include "tq2_internal.h"

namespace tq2 {

namespace {

constexpr int MU_THREADS = 640;
constexpr int MU_BN = 192;                 // positions of a tile: two accumulators and four A stages fill 512 columns
constexpr int MU_B = 6;                    // 64-k stages of activations
constexpr int MU_A = 4;                    // 64-k stages of decoded weights (32 columns each)
constexpr int MU_RAW = 3;                  // 256-k stages of packed blocks
constexpr int MU_B_STAGE = MU_BN * 128;    // 24 KB
constexpr int MU_ACOL = 2 * MU_BN;         // first tensor-memory column of the A stages

struct MuBars {
    uint64_t b_full[MU_B], b_empty[MU_B], a_full[MU_A], a_empty[MU_A], raw_full[MU_RAW], raw_empty[MU_RAW];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem_base;
    int abort;
    float2 scale[2][MU_BN];                // epilogue: a tile's scales and output rows
    int row[2][MU_BN];
};

// Slot and phase parity of a ring's next item.
template <int S>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    bool first = true;                     // no slot has been used twice yet
    __device__ __forceinline__ void next() {
        if (++s == S) {
            s = 0;
            ph ^= 1u;
            first = false;
        }
    }
};

struct MuArgs {
    const uint8_t* w0;
    const uint8_t* w1;                     // pair: Up
    int64_t mstride;
    int nkc, zeros, E, nslots;
    int N;                                 // output columns (F, or D)
    int row_tiles;                         // tiles along them
    int nk;                                // 64-k stages of a tile
    const int* offsets;
    const int* slots;
    const float2* scales;                  // [position] of a row of x: 1/scale; of the hidden row: scale
    __half* hidden;                        // pair: [position][N]
    float* y;                              // else: [slot][N]
};

struct MuTile {
    int e, p0, cnt, r;
};

// Barrier of the four warps of epilogue group b.
__device__ __forceinline__ void epi_bar(int b) { asm volatile("bar.sync %0, 128;" ::"r"(1 + b) : "memory"); }

template <int G, bool PAIR>
__global__ void __launch_bounds__(MU_THREADS, 1)
moe_umma_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ MuArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    constexpr int NG = Q4_K / G;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int blk = q4_block_bytes(G, a.zeros != 0);
    uint8_t* raw_ring = smem + MU_B * MU_B_STAGE;
    MuBars* bars = reinterpret_cast<MuBars*>(raw_ring + MU_RAW * 8 * blk);
    int* prefix = reinterpret_cast<int*>(bars + 1);        // token tiles before each matrix
    int* offs = prefix + a.E + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < MU_B; ++s) {
            mbar_init(&bars->b_full[s], 1);
            mbar_init(&bars->b_empty[s], 1);               // the MMA warp's commit
        }
        for (int s = 0; s < MU_A; ++s) {
            mbar_init(&bars->a_full[s], 4);                // the stage's decoder warps
            mbar_init(&bars->a_empty[s], 1);
        }
        for (int r = 0; r < MU_RAW; ++r) {
            mbar_init(&bars->raw_full[r], 1);
            mbar_init(&bars->raw_empty[r], 8);             // every decoder warp
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 4);
        }
        bars->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&xmap);
    }
    if (warp == 2) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    if (warp == 1) {
        pdl_wait();                                        // the plan is an earlier kernel's
        int run = 0;
        for (int e0 = 0; e0 <= a.E; e0 += 32) {
            const int e = e0 + lane;
            const int o = e <= a.E ? plan_offset(a.offsets, a.nslots, e) : 0;
            const int n = e < a.E ? max(plan_offset(a.offsets, a.nslots, e + 1) - o + MU_BN - 1, 0) / MU_BN : 0;
            int s = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += up;
            }
            if (e <= a.E) {
                prefix[e] = run + s - n;
                offs[e] = o;
            }
            run += __shfl_sync(0xffffffffu, s, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort;
    const int total = prefix[a.E] * a.row_tiles;

    // tile t: row tiles fastest; a matrix's positions are cut evenly
    auto tile_at = [&](int t) {
        MuTile m;
        const int tt = t / a.row_tiles;
        m.r = t - tt * a.row_tiles;
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= tt) lo = mid; else hi = mid;
        }
        m.e = lo;
        const int i = tt - prefix[lo], n = prefix[lo + 1] - prefix[lo], c = offs[lo + 1] - offs[lo];
        const int each = c / n, more = c - each * n;
        m.p0 = offs[lo] + i * each + min(i, more);
        m.cnt = each + (i < more ? 1 : 0);
        return m;
    };

    if (warp == 0) {
        if (lane == 0) {                                   // ---- activations
            pdl_wait();
            Ring<MU_B> b;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const MuTile m = tile_at(t);
                const int boxes = (m.cnt + 31) / 32;
                for (int ks = 0; ks < a.nk; ++ks, b.next()) {
                    if (!b.first && !mbar_wait_or_abort(&bars->b_empty[b.s], b.ph ^ 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars->b_full[b.s], (uint32_t)boxes * 4096u);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(smem + b.s * MU_B_STAGE + i * 4096, &xmap, &bars->b_full[b.s], ks * 64,
                                    m.p0 + 32 * i);
                }
            }
            // after a wait that ran out: the copies already issued land before the CTA can exit
            if (!ok)
                for (int i = 0; i < MU_B; ++i)
                    mbar_wait(&bars->b_full[i], i < b.s ? b.ph : b.ph ^ 1u);
        }
    } else if (warp == 3) {
        if (lane == 0) {                                   // ---- packed blocks
            Ring<MU_RAW> r;
            bool ok = true;
            const uint32_t bytes = 8u * (uint32_t)blk;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const MuTile m = tile_at(t);
                // first of the tile's blocks of a chunk: 8 row tiles of one matrix, or 4 of each of two
                const int rt = PAIR ? m.r * 4 : m.r * 8;
                const int64_t first = (int64_t)m.e * a.mstride + q4_block_index(rt, 0, a.nkc) * blk;
                for (int kc = 0; kc * 4 < a.nk; ++kc, r.next()) {
                    if (!r.first && !mbar_wait_or_abort(&bars->raw_empty[r.s], r.ph ^ 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars->raw_full[r.s], bytes);
                    uint8_t* dst = raw_ring + (size_t)r.s * bytes;
                    const int64_t at = first + (int64_t)kc * 8 * blk;
                    if (PAIR) {
                        bulk_load(dst, a.w0 + at, bytes / 2, &bars->raw_full[r.s]);
                        bulk_load(dst + bytes / 2, a.w1 + at, bytes / 2, &bars->raw_full[r.s]);
                    } else {
                        bulk_load(dst, a.w0 + at, bytes, &bars->raw_full[r.s]);
                    }
                }
            }
            if (!ok)
                for (int i = 0; i < MU_RAW; ++i)
                    mbar_wait(&bars->raw_full[i], i < r.s ? r.ph : r.ph ^ 1u);
        }
    } else if (warp == 1) {                                // ---- MMA issuer (the whole warp, elect.sync)
        auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, abort_flag, true)) != 0;
        };
        Ring<MU_B> b;
        Ring<MU_A> w;
        Ring<2> acc;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x, acc.next()) {
            const MuTile m = tile_at(t);
            const uint32_t idesc = idesc_f16_f32(128, (uint32_t)((m.cnt + 15) / 16 * 16));
            const uint32_t dcol = tmem + (uint32_t)(acc.s * MU_BN);
            if (!acc.first && !wait_all(&bars->acc_empty[acc.s], acc.ph ^ 1u)) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            for (int ks = 0; ks < a.nk; ++ks, b.next(), w.next()) {
                if (!wait_all(&bars->b_full[b.s], b.ph) || !wait_all(&bars->a_full[w.s], w.ph)) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t bdesc = sdesc_kmajor_sw128(smem_u32(smem + b.s * MU_B_STAGE));
                const uint32_t acol = tmem + MU_ACOL + (uint32_t)(w.s * 32);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    umma_f16_ts_elect(dcol, acol + (uint32_t)(j * 8), bdesc + (uint64_t)(2 * j), idesc,
                                      (ks > 0 || j > 0) ? 1u : 0u);
                umma_commit_elect(&bars->b_empty[b.s]);
                umma_commit_elect(&bars->a_empty[w.s]);
            }
            if (!ok) break;
            umma_commit_elect(&bars->acc_full[acc.s]);
        }
    } else if (warp >= 4 && warp < 12) {                   // ---- decoders
        // quarter q of the rows, stages of parity h; rows 0..15 of a quarter are one
        // 16-row tile's, 16..31 the next one's (pair: Gate's and Up's)
        const int q = warp & 3, h = (warp - 4) >> 2;
        const int row = lane & 15, g = row & 7, hi = row >> 3;
        const int b = PAIR ? (lane >> 4) * 4 + q : q * 2 + (lane >> 4);
        const uint32_t expo = q4_exponent<false>();
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + MU_ACOL;
        Ring<MU_RAW> r;
        int it0 = 0;                                       // stages of the tiles before
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            for (int kc = 0; kc * 4 < a.nk && ok; ++kc, r.next()) {
                if (!mbar_wait_or_abort(&bars->raw_full[r.s], r.ph, abort_flag)) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                const uint8_t* src = raw_ring + (size_t)r.s * 8 * blk + b * blk;
                const uint8_t* sc = src + Q4_CODES + q4_scale_index(row, 0, NG) * 2;
                const uint8_t* zp = src + Q4_CODES + 32 * NG + q4_scale_index(row, 0, NG);
                for (int c = h; c < 4; c += 2) {
                    const int ks = kc * 4 + c;
                    if (ks >= a.nk) break;
                    uint32_t v[32];
                    __half2 d[2];
                    Q4Zero z[2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (half == 1 && G > 32) {
                            d[1] = d[0];
                            z[1] = z[0];
                            break;
                        }
                        const int gi = (c * 2 + half) / (G / 32);
                        d[half] = __half2half2(*reinterpret_cast<const __half*>(sc + gi * 4));
                        z[half] = q4_zero<false>(a.zeros ? zp[gi * 2] : 8u);
                    }
#pragma unroll
                    for (int tt = 0; tt < 4; ++tt) {
                        const uint2 w = *reinterpret_cast<const uint2*>(src + c * 512 + (tt * 8 + g) * 16 + hi * 8);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t p[4];
                            q4_decode<false>(half ? w.y : w.x, expo, z[half], p);
#pragma unroll
                            for (int f = 0; f < 4; ++f) {
                                const __half2 m = __hmul2(*reinterpret_cast<const __half2*>(&p[f]), d[half]);
                                v[16 * half + 4 * tt + f] = *reinterpret_cast<const uint32_t*>(&m);
                            }
                        }
                    }
                    const int it = it0 + ks, s = it % MU_A;
                    if (it >= MU_A &&
                        !mbar_wait_or_abort(&bars->a_empty[s], (uint32_t)(it / MU_A - 1) & 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    tmem_st_32x32b_x32(lane_addr + (uint32_t)(s * 32), v);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->a_full[s]);
                }
                // the values are used: the slot is refilled through the async proxy
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->raw_empty[r.s]);
            }
            it0 += a.nk;
        }
    } else if (warp >= 12) {                               // ---- epilogue: group b drains accumulator b
        const int q = warp & 3, b = (warp - 12) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * MU_BN);
        const float2* scale = bars->scale[b];
        const int* orow = bars->row[b];
        pdl_wait();
        uint32_t ph = 0;
        for (int t = blockIdx.x + b * gridDim.x; t < total; t += 2 * gridDim.x, ph ^= 1u) {
            const MuTile m = tile_at(t);
            epi_bar(b);                                    // the last tile's scales and rows are done with
            for (int i = tid - (12 + 4 * b) * 32; i < m.cnt; i += 128) {
                bars->scale[b][i] = a.scales[m.p0 + i];
                if (!PAIR) bars->row[b][i] = plan_slot(a.slots, a.nslots, m.p0 + i);
            }
            epi_bar(b);
            if (!mbar_wait_or_abort(&bars->acc_full[b], ph, abort_flag)) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            // pair: this lane finishes 16 of 32 positions of its row, else all of them
            const bool upper = PAIR && lane >= 16;
            const int n = PAIR ? m.r * 64 + q * 16 + (lane & 15) : m.r * 128 + q * 32 + lane;
            const bool mine = n < a.N;
            for (int cc = 0; cc < m.cnt; cc += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(lane_addr + (uint32_t)cc, v);
                tmem_wait_ld();
                if (cc + 32 >= m.cnt) {                    // accumulator read: hand it back
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->acc_empty[b]);
                }
                if (PAIR) {
                    const int c0 = cc + (upper ? 16 : 0), left = mine ? m.cnt - c0 : 0;
                    __half* out = a.hidden + (int64_t)(m.p0 + c0) * a.N + n;
#pragma unroll
                    for (int i = 0; i < 16; ++i, out += a.N) {
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[16 + i], 16);
                        const float2 sc = scale[c0 + i];
                        const float gt = __uint_as_float(upper ? other : v[i]) * sc.x;
                        const float up = __uint_as_float(upper ? v[16 + i] : other) * sc.x;
                        const float hv = __fdividef(gt, 1.0f + __expf(-gt)) * up;
                        if (i < left) *out = __float2half_rn(hv * sc.y);
                    }
                } else if (mine) {
                    float* out = a.y + n;
                    const int left = m.cnt - cc;
                    if (left >= 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            out[(int64_t)orow[cc + i] * a.N] = __uint_as_float(v[i]) * scale[cc + i].y;
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < left) out[(int64_t)orow[cc + i] * a.N] = __uint_as_float(v[i]) * scale[cc + i].y;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Eight elements of a row.
template <class T>
__device__ __forceinline__ void load8(const T* p, bool vec, float (&f)[8]) {
    T raw[8];
    if (vec) {
        *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)raw[i];
}

// A warp a position: its row of x as f16, scaled, and the scales.  Two passes
// over the row, the second from L1; a token's rows share its lines in L2.
template <class T>
__global__ void __launch_bounds__(256)
moe_stage_kernel(const T* __restrict__ x, int64_t ldx, int vec, int D, const int* __restrict__ offsets,
                 const int* __restrict__ slots, int nslots, int k, int E, const float* __restrict__ bound0,
                 const float* __restrict__ bound1, __half* __restrict__ xs, float2* __restrict__ first,
                 float2* __restrict__ second) {
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int end = plan_offset(offsets, nslots, E);
    for (int p = blockIdx.x * 8 + (threadIdx.x >> 5); p < end; p += gridDim.x * 8) {
        const T* row = x + (int64_t)(plan_slot(slots, nslots, p) / k) * ldx;
        float m = 0.f, ss = 0.f, f[8];
#pragma unroll 4
        for (int c = lane * 8; c < D; c += 256) {
            load8(row + c, vec != 0, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
        }
        m = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(m)));   // m >= 0: its bits have its order
        const int be = (__float_as_int(m) >> 23) & 255;
        int se = be == 0 ? 253 : 127 + 14 - (be - 127);
        if (m == 0.f || be == 255) se = 127;
        se = se > 253 ? 253 : se;
        const float s = __int_as_float(se << 23);
#pragma unroll 4
        for (int c = lane * 8; c < D; c += 256) {
            load8(row + c, vec != 0, f);
            __half2 h[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] *= s;
                ss = fmaf(f[i], f[i], ss);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            *reinterpret_cast<uint4*>(xs + (int64_t)p * D + c) = *reinterpret_cast<uint4*>(h);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) {
            int lo = 0, hi = E;                            // the position's matrix
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (plan_offset(offsets, nslots, mid) <= p) lo = mid; else hi = mid;
            }
            // exponent of the hidden row's bound, x's own scale taken out
            const float b = ss * bound0[lo] * bound1[lo];
            const int e = ((__float_as_int(b) >> 23) & 255) - 127 - 2 * (se - 127);
            int hs = 127 + 14 - e;
            if (b == 0.f) hs = 127;
            hs = hs < 1 ? 1 : hs > 253 ? 253 : hs;
            const float inv = __int_as_float((254 - se) << 23);
            first[p] = make_float2(inv, __int_as_float(hs << 23));
            second[p] = make_float2(0.f, __int_as_float((254 - hs) << 23));
        }
    }
}

template <int G, bool PAIR>
cudaError_t launch_umma_moe(const CUtensorMap& xmap, const MuArgs& a, cudaStream_t st) {
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const size_t smem = 1024 + (size_t)MU_B * MU_B_STAGE + (size_t)MU_RAW * 8 * q4_block_bytes(G, a.zeros != 0) +
                        sizeof(MuBars) + (size_t)(2 * (a.E + 1)) * 4;
    cudaError_t e = cudaFuncSetAttribute(moe_umma_kernel<G, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_umma_kernel<G, PAIR>, dim3((unsigned)sms), dim3(MU_THREADS), smem, st, xmap, a);
}

template <bool PAIR>
cudaError_t launch_by_group(int group, const CUtensorMap& xmap, const MuArgs& a, cudaStream_t st) {
    if (group == 32) return launch_umma_moe<32, PAIR>(xmap, a, st);
    if (group == 64) return launch_umma_moe<64, PAIR>(xmap, a, st);
    return launch_umma_moe<128, PAIR>(xmap, a, st);
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// f16 rows of x and of the hidden values by position, and two scales each.
size_t moe_tensor_scratch(int64_t nslots, int64_t D, int64_t F) {
    return round256((size_t)nslots * D * 2) + round256((size_t)nslots * F * 2) + 2 * round256((size_t)nslots * 8);
}

cudaError_t launch_moe_tensor(const MoeTensor& m, void* scratch, cudaStream_t st) {
    const int64_t S = m.nslots, D = m.gate->K, F = m.gate->N;
    char* at = static_cast<char*>(scratch);
    __half* xs = reinterpret_cast<__half*>(at);
    at += round256((size_t)S * D * 2);
    __half* hid = reinterpret_cast<__half*>(at);
    at += round256((size_t)S * F * 2);
    float2* first = reinterpret_cast<float2*>(at);
    at += round256((size_t)S * 8);
    float2* second = reinterpret_cast<float2*>(at);
    int64_t grid = (S + 7) / 8;
    if (grid > 152 * 16) grid = 152 * 16;
    const int vec = (reinterpret_cast<uintptr_t>(m.x) & 15) == 0 && m.ldx % 8 == 0;
    cudaError_t e;
    const int E = (int)m.gate->E;
    if (m.dtype == TQ2_F16)
        e = launch_pdl(moe_stage_kernel<__half>, dim3((unsigned)grid), dim3(256), 0, st,
                       static_cast<const __half*>(m.x), m.ldx, vec, (int)D, m.offsets, m.slots, (int)S, m.k, E,
                       static_cast<const float*>(m.gate->bound), static_cast<const float*>(m.up->bound), xs, first,
                       second);
    else
        e = launch_pdl(moe_stage_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(256), 0, st,
                       static_cast<const __nv_bfloat16*>(m.x), m.ldx, vec, (int)D, m.offsets, m.slots, (int)S, m.k, E,
                       static_cast<const float*>(m.gate->bound), static_cast<const float*>(m.up->bound), xs, first,
                       second);
    if (e != cudaSuccess) return e;
    CUtensorMap xmap, hmap;
    if (!make_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xs, (uint64_t)D, (uint64_t)S, (uint64_t)D * 2, 64u,
                            32u, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map_2d(&hmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, hid, (uint64_t)F, (uint64_t)S, (uint64_t)F * 2,
                            64u, 32u, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    MuArgs a{};
    a.w0 = m.gate->blocks;
    a.w1 = m.up->blocks;
    a.mstride = m.gate->mstride;
    a.nkc = (int)m.gate->nkc;
    a.zeros = m.gate->zeros ? 1 : 0;
    a.E = E;
    a.nslots = (int)S;
    a.N = (int)F;
    a.row_tiles = (int)((F + 63) / 64);
    a.nk = (int)((D + 63) / 64);
    a.offsets = m.offsets;
    a.slots = m.slots;
    a.scales = first;
    a.hidden = hid;
    e = launch_by_group<true>(m.gate->group, xmap, a, st);
    if (e != cudaSuccess) return e;
    MuArgs b = a;
    b.w0 = m.down->blocks;
    b.w1 = nullptr;
    b.mstride = m.down->mstride;
    b.nkc = (int)m.down->nkc;
    b.zeros = m.down->zeros ? 1 : 0;
    b.N = (int)D;
    b.row_tiles = (int)((D + 127) / 128);
    b.nk = (int)((F + 63) / 64);
    b.scales = second;
    b.hidden = nullptr;
    b.y = m.y;
    return launch_by_group<false>(m.down->group, hmap, b, st);
}

unsigned int read_clear_dev_error_moe_umma(cudaStream_t st) {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_dev_error, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess) return 0;
    cudaMemcpyToSymbolAsync(g_dev_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    cudaStreamSynchronize(st);
    return v;
}

}  // namespace tq2
