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
// The weights are read once and bound the time.  A CTA takes a contiguous range
// of 16-row tiles; the blocks (tiles x 256-k chunks) of one pass over its rows
// of x are one sequence that is cut evenly among its sixteen warps, so a warp's
// part may begin and end inside a tile.  A warp reads its blocks straight into
// registers, one block ahead of the one it multiplies (34 KB in flight on an
// SM).  Tiles that it has to itself it stores from registers; of the at most
// two that it shares it leaves its part in shared memory, and after the last
// block those parts are added in a fixed order.  Only there do warps wait for
// each other.  The activations sit in shared memory for the CTA's whole life
// (one matrix) or per pass of the plan.
//
// Long rows of x do not fit shared memory whole: a cluster of CTAs then takes
// the tiles together, each CTA a range of k, and the CTAs' sums of a tile meet
// through distributed shared memory, in the order of their ranks.
//
// A decode call lasts a few microseconds, so what a warp does once counts as
// much as the blocks (two to six a warp): there is one copy of the block's code,
// the work is cut with shifts and host-side reciprocals, and more rows than
// fit are further launches.
//
// Bound: one row by the launch and one pass of latency (1x4096x4096 f32 5.4 us a
// call).  8x11008x4096 bf16 takes 8.2 us (2.9 TB/s) and 16x14336x4096 bf16 12.7 (2.5 TB/s):
// 400 to 490 warp instructions a block are 3.7 and 6.0 us of that, if every scheduler
// issued in every cycle.  The rest is the start, rows of x that the first MMA waits for,
// the one block of look-ahead and the closing sums; how it divides is not measured.
//
// With a plan the accumulators of two or four column tiles do not fit 128 registers
// beside a pass's bookkeeping: those variants spill (four tiles, groups of 128: 284 bytes
// stored, 340 loaded a thread).  f32 calls of more than 4 rows a pass use them, and
// 16-bit ones of more than 8 whose weights pass f16.
//
// With a plan (offsets, slots; PLAN) matrix e multiplies the rows of positions
// offsets[e]..offsets[e+1]; `pair` takes tiles of two matrices in turn over the
// same rows and stores silu(first) * second.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <mutex>

#include "../../include/tq2.h"
#include "q4.cuh"
#include "tq2_internal.h"

namespace tq2 {

constexpr int Q4_WARPS = 16;
constexpr int Q4_RED_PITCH = 20;       // floats of a 16-row column in the reduction buffer (conflict-free)

struct Q4Kernel {
    Q4Stream a;
    int tok;                           // rows of x a pass takes
    int parts;                         // f16 columns of a row
    int tiles;                         // 16-row tiles of a pass (both matrices' of a pair)
    int each, more;                    // no plan: tiles of a CTA, and CTAs that take one more
    int split, teams;                  // no plan: CTAs of a cluster, each with a range of k; clusters
    int pitch;                         // bytes of an activation column in shared memory
    int xvec;                          // rows of x are 16-byte aligned
    int off_prefix, off_slots, off_scale, off_red, off_sum, off_x;   // shared-memory layout (off_slots 0: none)
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

// The same with a zero accumulator.
template <bool BF>
__device__ __forceinline__ void q4_mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ int q4_offset(const Q4Stream& a, int e) { return plan_offset(a.offsets, a.nslots, e); }
__device__ __forceinline__ int q4_slot(const Q4Stream& a, int p) { return plan_slot(a.slots, a.nslots, p); }
constexpr int Q4_PLAN_SLOTS = 512;     // plans of at most this many slots are kept in shared memory whole

// Pass j of the plan: rows p0 .. p0+cnt of matrix e.
struct Q4Pass {
    int e, p0, cnt;
};
__device__ __forceinline__ Q4Pass q4_pass(const Q4Kernel& k, const int* prefix, int j) {
    const int* offs = prefix + k.a.E + 1;
    int lo = 0, hi = k.a.E;                               // prefix[lo] <= j < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= j) lo = mid; else hi = mid;
    }
    Q4Pass p;
    p.e = lo;
    p.p0 = offs[lo] + (j - prefix[lo]) * k.tok;
    p.cnt = min(k.tok, offs[lo + 1] - p.p0);
    return p;
}

// Slot and x row of position p.
__device__ __forceinline__ int q4_slot_of(const Q4Kernel& k, const uint8_t* smem, int p) {
    return k.off_slots ? reinterpret_cast<const int*>(smem + k.off_slots)[p] : q4_slot(k.a, p);
}
__device__ __forceinline__ int64_t q4_xrow(const Q4Kernel& k, const uint8_t* smem, int p) {
    return k.a.xdiv ? q4_slot_of(k, smem, p) / k.a.xdiv : p;
}

// Activation rows of a pass into shared memory: column (row i, part q) at
// (i*parts + q)*pitch, f16 or bf16 in k order.  Rows are copied by the copy
// engine where they are 16-byte aligned; f32 rows are scaled to a largest
// magnitude of 2^14..2^15 and split.  Only k = k0 .. k0 + K of the rows is taken.
// Every thread of the CTA calls it.
__device__ __forceinline__ bool q4_stage_x(const Q4Kernel& k, uint8_t* smem, const Q4Pass& p, int k0, int K,
                                           uint64_t* xbar, uint32_t& xphase) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* xs = smem + k.off_x;
    float* inv = reinterpret_cast<float*>(smem + k.off_scale);
    int* top = reinterpret_cast<int*>(inv + 32);
    int* orow = top + 32;
    __syncthreads();                                       // the previous rows and their scales are done with
    if (warp == Q4_WARPS - 1 && lane < p.cnt) orow[lane] = k.a.oslot ? q4_slot_of(k, smem, p.p0 + lane) : p.p0 + lane;
    if (k.a.xmode == Q4_X_RAW16) {
        if (!k.xvec) {
            for (int i = warp; i < p.cnt; i += Q4_WARPS) {
                const uint16_t* src = reinterpret_cast<const uint16_t*>(k.a.x) + q4_xrow(k, smem, p.p0 + i) * k.a.ldx + k0;
                for (int c = lane; c < K; c += 32) reinterpret_cast<uint16_t*>(xs + i * k.pitch)[c] = src[c];
            }
            __syncthreads();
            return true;
        }
        if (warp == 0) {
            if (lane == 0) mbar_arrive_expect_tx(xbar, (uint32_t)(p.cnt * K * 2));
            __syncwarp();
            if (lane < p.cnt)
                bulk_load(xs + lane * k.pitch,
                          reinterpret_cast<const uint16_t*>(k.a.x) + q4_xrow(k, smem, p.p0 + lane) * k.a.ldx + k0,
                          (uint32_t)K * 2, xbar);
        }
        const bool ok = mbar_wait(xbar, xphase);
        xphase ^= 1u;
        __syncthreads();                                   // (the output rows)
        return ok;
    }
    if (tid < 32) top[tid] = 0;
    __syncthreads();
    // nw warps a row, which read it twice (the second time from L1)
    const int nw = p.cnt > 8 ? 1 : p.cnt > 4 ? 2 : p.cnt > 2 ? 4 : p.cnt > 1 ? 8 : 16;
    const int step = nw * 128, first = ((warp & (nw - 1)) * 32 + lane) * 4;
    const bool split = k.a.xmode == Q4_X_SPLIT;
    auto load = [&](const float* src, int c) {
        return k.xvec ? *reinterpret_cast<const float4*>(src + c)
                      : make_float4(src[c], src[c + 1], src[c + 2], src[c + 3]);
    };
    for (int i0 = 0; i0 < p.cnt; i0 += Q4_WARPS / nw) {
        const int i = i0 + warp / nw;
        const bool on = i < p.cnt;
        const float* src = reinterpret_cast<const float*>(k.a.x) + (on ? q4_xrow(k, smem, p.p0 + i) * k.a.ldx + k0 : 0);
        float m = 0.f;
        if (on) {
#pragma unroll 2
            for (int c = first; c < K; c += step) {
                const float4 f = load(src, c);
                m = fmaxf(fmaxf(fmaxf(m, fabsf(f.x)), fmaxf(fabsf(f.y), fabsf(f.z))), fabsf(f.w));
            }
        }
        // m >= 0: as integers its bits have its order; a maximum does not depend on the order it is taken in
        const int wm = __reduce_max_sync(0xffffffffu, __float_as_int(m));
        if (on && lane == 0) atomicMax(top + i, wm);
        __syncthreads();
        if (!on) continue;
        // 2^(14 - exponent of the maximum), kept a normal number; 1 for a row of zeros or one with infinities
        const int be = (top[i] >> 23) & 255;
        int se = be == 0 ? 253 : 127 + 14 - (be - 127);
        if (top[i] == 0 || be == 255) se = 127;
        se = se > 253 ? 253 : se;
        const float s = __int_as_float(se << 23);
        if (lane == 0 && (warp & (nw - 1)) == 0) inv[i] = __int_as_float((254 - se) << 23);
        uint8_t* hi = xs + i * k.parts * k.pitch;
        uint8_t* lo = hi + k.pitch;
#pragma unroll 2
        for (int c = first; c < K; c += step) {
            const float4 u = load(src, c);
            const float f[4] = {u.x * s, u.y * s, u.z * s, u.w * s};
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

__device__ __forceinline__ uint4 ldg_stream128(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// What a lane holds of a block: codes, scales and zero points.
template <int G>
struct Q4Block {
    static constexpr int NG = Q4_K / G;
    uint4 w[4];
    uint32_t s[NG];                    // group: scales of rows g (low) and g+8
    uint32_t z[NG / 2];                // two groups: zero points of rows g, g+8 each
    __device__ __forceinline__ void load(const uint8_t* b, int lane, int zeros) {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = ldg_stream128(b + c * 512 + ((lane & 3) * 8 + (lane >> 2)) * 16);
        const uint8_t* p = b + Q4_CODES + (lane >> 2) * (4 * NG);
        if (NG == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            s[0] = v.x;
            s[NG - 1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < NG / 4; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
                s[(4 * i) % NG] = v.x;
                s[(4 * i + 1) % NG] = v.y;
                s[(4 * i + 2) % NG] = v.z;
                s[(4 * i + 3) % NG] = v.w;
            }
        }
        if (zeros) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(b + Q4_CODES + 32 * NG + (lane >> 2) * (2 * NG));
#pragma unroll
            for (int i = 0; i < NG / 2; ++i) z[i] = __ldg(q + i);
        } else {
#pragma unroll
            for (int i = 0; i < NG / 2; ++i) z[i] = 0x08080808u;
        }
    }
};

template <int G, int NT, bool BF, bool PLAN>
__global__ void __launch_bounds__(Q4_WARPS * 32, 1) q4_stream_kernel(const __grid_constant__ Q4Kernel k) {
    extern __shared__ __align__(128) uint8_t smem[];
    const Q4Stream& a = k.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t blk = (uint32_t)q4_block_bytes(G, a.zeros != 0);
    uint64_t* xbar = reinterpret_cast<uint64_t*>(smem);
    int* nshared = reinterpret_cast<int*>(smem + 8);
    int4* shared_units = reinterpret_cast<int4*>(smem + 16);   // unit, first and last warp
    int* prefix = reinterpret_cast<int*>(smem + k.off_prefix);
    const float* inv = reinterpret_cast<const float*>(smem + k.off_scale);
    const int* orow = reinterpret_cast<const int*>(inv + 64);
    float* red = reinterpret_cast<float*>(smem + k.off_red);
    float* csum = reinterpret_cast<float*>(smem + k.off_sum);  // cluster: [tile][row of x][16 rows]
    // this CTA's range of k, in chunks
    const int split = PLAN ? 1 : k.split, rank = split > 1 ? (int)(blockIdx.x % split) : 0;
    const int c0 = split > 1 ? a.nkc * rank / split : 0;
    const int nkc = split > 1 ? a.nkc * (rank + 1) / split - c0 : a.nkc;
    const int kl = min((int)a.K - c0 * Q4_K, nkc * Q4_K);

    if (tid == 0) {
        mbar_init(xbar, 1);
        fence_mbar_init();
    }
    if (kl != nkc * Q4_K) {                                // k past the row's end is zero for the kernel's whole life
        for (int c = 0; c < k.tok * k.parts; ++c)
            for (int i = kl + 2 * tid; i < nkc * Q4_K; i += 2 * Q4_WARPS * 32)
                *reinterpret_cast<uint32_t*>(smem + k.off_x + c * k.pitch + i * 2) = 0u;
        fence_proxy_async_shared();
    }
    __syncthreads();
    // The plan may be the last kernel's.  Where that is the product before this one, the plan is older and read at
    // once: that product lets this one start only when it has waited for the plan itself.
    if (PLAN && !a.after) pdl_wait();
    pdl_launch_dependents();

    // the CTA's tiles (whole units: a tile, or a pair of them)
    const int two = PLAN && a.pair ? 2 : 1;
    int u0, u1;
    if (PLAN) {
        int* offs = prefix + a.E + 1;
        for (int e = tid; e <= a.E; e += Q4_WARPS * 32) offs[e] = q4_offset(a, e);
        if (k.off_slots && tid < a.nslots) reinterpret_cast<int*>(smem + k.off_slots)[tid] = q4_slot(a, tid);
        __syncthreads();
        if (warp == 0) {
            int run = 0;
            bool down = false;                             // ranges that go back are no plan: nothing is done
            for (int e0 = 0; e0 <= a.E; e0 += 32) {
                const int e = e0 + lane;
                const int rows = e < a.E ? offs[e + 1] - offs[e] : 0;
                const int n = (rows + k.tok - 1) / k.tok;
                down |= rows < 0;
                int s = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, s, d);
                    if (lane >= d) s += up;
                }
                if (e <= a.E) prefix[e] = run + s - n;
                run += __shfl_sync(0xffffffffu, s, 31);
            }
            __syncwarp();
            if (__any_sync(0xffffffffu, down) && lane == 0) prefix[a.E] = 0;
        }
        __syncthreads();
        const unsigned jobs = (unsigned)prefix[a.E], units = (unsigned)(k.tiles / two), grid = gridDim.x;
        const unsigned b = blockIdx.x;
        if (jobs > 0 && 4 * jobs <= grid) {
            // few passes: each has CTAs to itself (one that spans two passes stages x twice, 5 us on the path)
            const unsigned per = grid / jobs, wide = grid - per * jobs;   // `wide` passes get one more
            const unsigned cut = wide * (per + 1);
            const unsigned n = b < cut ? per + 1 : per, c = b < cut ? b : b - cut;
            const unsigned j = (b < cut ? 0 : wide) + c / n, i = c - c / n * n;
            u0 = (int)(j * units + units * i / n) * two;
            u1 = (int)(j * units + units * (i + 1) / n) * two;
        } else {
            const unsigned all = jobs * units, each = all / grid, more = all - each * grid;
            u0 = (int)(b * each + min(b, more)) * two;
            u1 = u0 + (int)(each + (b < more ? 1u : 0u)) * two;
        }
    } else {
        const int b = split > 1 ? blockIdx.x / split : blockIdx.x;
        u0 = b * k.each + min(b, k.more);
        u1 = u0 + k.each + (b < k.more ? 1 : 0);
    }
    if (u0 >= u1) {                                        // uniform
        if (PLAN && a.after) pdl_wait();                   // (a kernel never ends before the ones it follows)
        return;
    }

    // The tiles of one pass; warp w takes their blocks L*w/16 .. L*(w+1)/16.
    struct Batch {
        int j, first, n;                                   // pass, first tile of the pass, tiles
        int i0, i1;                                        // blocks of this warp
        const uint8_t* w;                                  // the pass's matrix
    };
    auto batch_at = [&](int u) {
        Batch b;
        b.j = PLAN ? u / k.tiles : 0;
        b.first = u - b.j * k.tiles;
        b.n = min(u1 - u, k.tiles - b.first);
        const int L = b.n * nkc;
        b.i0 = L * warp / Q4_WARPS;
        b.i1 = L * (warp + 1) / Q4_WARPS;
        b.w = a.w0;
        if (PLAN) b.w += (int64_t)q4_pass(k, prefix, b.j).e * a.mstride;
        return b;
    };
    const int64_t second = PLAN && a.pair ? a.w1 - a.w0 : 0;
    auto tile_of = [&](int i) { return i / nkc; };
    auto block_ptr = [&](const Batch& b, int tl, int kc) {
        const int tile = b.first + tl, rt = two == 2 ? tile >> 1 : tile;
        const uint32_t index = (uint32_t)(((rt >> 3) * a.nkc + c0 + kc) * 8 + (rt & 7));
        const uint8_t* p = b.w + (int64_t)index * blk;
        return two == 2 && (tile & 1) ? p + second : p;
    };
    auto first_ptr = [&](const Batch& b) {
        const int tl = tile_of(b.i0);
        return block_ptr(b, tl, b.i0 - tl * nkc);
    };
    Batch b = batch_at(u0);
    Q4Block<G> cur;
    if (b.i0 < b.i1) cur.load(first_ptr(b), lane, a.zeros);
    if (!PLAN || a.after) pdl_wait();                      // x is the last kernel's; the weights are not

    const uint32_t expo = q4_exponent<BF>();
    uint32_t xphase = 0;
    int staged = -1;
    Q4Pass pass{0, 0, a.M};
    uint32_t xa[NT];
    int cols = 0;

    auto store = [&](float v, int m, int row, int tl) {
        if (split > 1) {
            csum[(tl * pass.cnt + m) * 16 + (row & 15)] = v;
            return;
        }
        if (row >= a.N) return;
        const int64_t o = (int64_t)orow[m] * a.ldo + row;
        if (PLAN || a.otype == TQ2_F32) reinterpret_cast<float*>(a.out)[o] = v;
        else if (a.otype == TQ2_F16) reinterpret_cast<__half*>(a.out)[o] = __float2half_rn(v);
        else reinterpret_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
    };

    for (int u = u0;;) {
        if (b.j != staged) {
            staged = b.j;
            if (PLAN) pass = q4_pass(k, prefix, b.j);
            q4_stage_x(k, smem, pass, c0 * Q4_K, kl, xbar, xphase);   // a wait that ran out is on record; the rest is harmless
            cols = pass.cnt * k.parts;
            // columns past the last one repeat it and are not stored
#pragma unroll
            for (int n = 0; n < NT; ++n)
                xa[n] = smem_u32(smem + k.off_x) + t * 16 + min(n * 8 + g, cols - 1) * k.pitch;
        }
        const int un = u + b.n;
        const bool again = PLAN && un < u1;
        Batch next{};
        if (again) next = batch_at(un);
        const int L = b.n * nkc, U = two * nkc;
        const int seg = cols * Q4_RED_PITCH;               // floats of a part of a tile
        float tot[NT][4], hold[PLAN ? NT : 1][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[n][i] = 0.f;
        int tl = tile_of(b.i0), kc = b.i0 - tl * nkc;
        if (PLAN && b.i0 == b.i1 && again && next.i0 < next.i1) cur.load(first_ptr(next), lane, a.zeros);

#pragma unroll 1
        for (int i = b.i0; i < b.i1; ++i) {
            Q4Block<G> ahead;
            const bool last = kc + 1 == nkc;
            if (i + 1 < b.i1) ahead.load(block_ptr(b, last ? tl + 1 : tl, last ? 0 : kc + 1), lane, a.zeros);
            else if (again && next.i0 < next.i1) ahead.load(first_ptr(next), lane, a.zeros);
            const uint32_t xo = (uint32_t)kc * 512u;
            float acc[NT][4];
            float d0, d1;
            Q4Zero z0, z1;
#pragma unroll
            for (int h = 0; h < 8; ++h) {                  // 32 k
                constexpr int HG = G / 32;
                const int gi = h / HG;
                if (h % HG == 0) {
                    const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&cur.s[gi]));
                    d0 = d.x;
                    d1 = d.y;
                    const uint32_t zz = cur.z[gi / 2] >> (gi % 2 * 16);
                    z0 = q4_zero<BF>(zz & 255u);
                    z1 = q4_zero<BF>((zz >> 8) & 255u);
                }
                uint4 x[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n == 0 || n * 8 < cols) x[n] = lds128(xa[n] + xo + h * 64);
                const uint4& w = cur.w[h >> 1];
                uint32_t p[4], q[4];                       // pairs of rows g and g+8
                q4_decode<BF>((h & 1) ? w.y : w.x, expo, z0, p);
                q4_decode<BF>((h & 1) ? w.w : w.z, expo, z1, q);
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const uint32_t f[4] = {p[2 * jj], q[2 * jj], p[2 * jj + 1], q[2 * jj + 1]};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n == 0 || n * 8 < cols) {
                            if (h % HG == 0 && jj == 0) q4_mma0<BF>(acc[n], f, x[n].x, x[n].y);
                            else q4_mma<BF>(acc[n], f, jj ? x[n].z : x[n].x, jj ? x[n].w : x[n].y);
                        }
                }
                if (h % HG == HG - 1) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n == 0 || n * 8 < cols) {
                            tot[n][0] = fmaf(acc[n][0], d0, tot[n][0]);
                            tot[n][1] = fmaf(acc[n][1], d0, tot[n][1]);
                            tot[n][2] = fmaf(acc[n][2], d1, tot[n][2]);
                            tot[n][3] = fmaf(acc[n][3], d1, tot[n][3]);
                        }
                }
            }
            cur = ahead;
            if (last || i + 1 == b.i1) {
                const int unit = two == 2 ? tl >> 1 : tl, half = tl & (two - 1);
                if (unit * U >= b.i0 && (unit + 1) * U <= b.i1) {   // this warp has the unit to itself
                    if (PLAN && half + 1 < two) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 4; ++c) hold[PLAN ? n : 0][c] = tot[n][c];
                    } else {
                        const int row = ((b.first + tl) / two) * 16 + g;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                // split rows: columns 2t, 2t+1 are the two parts of row n*4 + t
                                const int m = k.parts == 2 ? n * 4 + t : n * 8 + 2 * t + c;
                                if (m >= pass.cnt || (k.parts == 2 && c == 1)) continue;
                                const float s = a.xmode == Q4_X_RAW16 ? 1.f : inv[m];
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    float v = tot[n][2 * r + c];
                                    if (k.parts == 2) v += tot[n][2 * r + 1];
                                    v *= s;
                                    if (PLAN && a.pair) {
                                        float f = hold[PLAN ? n : 0][2 * r + c];
                                        if (k.parts == 2) f += hold[PLAN ? n : 0][2 * r + 1];
                                        f *= s;
                                        v = f / (1.0f + expf(-f)) * v;
                                    }
                                    store(v, m, row + 8 * r, tl);
                                }
                            }
                    }
                } else {                                   // its part of the tile: [column][16 rows]
                    const int slot = 2 * warp + (b.i0 >= unit * U ? 0 : 1);
                    float* q = red + (slot * two + half) * seg + 2 * t * Q4_RED_PITCH + g;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (n * 8 + 2 * t + c < cols) {
                                q[(n * 8 + c) * Q4_RED_PITCH] = tot[n][c];
                                q[(n * 8 + c) * Q4_RED_PITCH + 8] = tot[n][2 + c];
                            }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.f;
            }
            kc = last ? 0 : kc + 1;
            tl = last ? tl + 1 : tl;
        }
        // the units that warps share: warp w's part begins inside one
        if (warp == 0) {
            const int at = L * lane / Q4_WARPS, before = L * (lane - 1) / Q4_WARPS;
            const int unit = (two == 2 ? tile_of(at) >> 1 : tile_of(at)), start = unit * U;
            // the first boundary strictly inside the unit lists it
            const bool mine = lane > 0 && lane < Q4_WARPS && at > start && (lane == 1 || before <= start);
            const uint32_t who = __ballot_sync(0xffffffffu, mine);
            if (mine) {
                int lastw = lane;
                while (lastw + 1 < Q4_WARPS && L * (lastw + 1) / Q4_WARPS < start + U) ++lastw;
                shared_units[__popc(who & ((1u << lane) - 1u))] = make_int4(unit, lane - 1, lastw, 0);
            }
            if (lane == 0) *nshared = __popc(who);
        }
        __syncthreads();
        // sixteen lanes a unit and row of x: parts in the order of the warps, then of x
        const int nu = *nshared;
        const float rnu = 1.0f / (float)nu;
        for (int q = tid >> 4; q < nu * pass.cnt; q += Q4_WARPS * 2) {
            const int m = (int)(((float)q + 0.5f) * rnu);
            const int4 su = shared_units[q - m * nu];
            const int row = (b.first / two + su.x) * 16 + (tid & 15);
            auto sum = [&](int half) {
                const int ts = su.x * U + half * nkc, te = ts + nkc;
                float v = 0.f;
#pragma unroll 1
                for (int w = su.y; w <= su.z; ++w) {
                    const int w0 = L * w / Q4_WARPS, w1 = L * (w + 1) / Q4_WARPS;
                    if (max(w0, ts) >= min(w1, te)) continue;   // no block of this tile
                    const float* s = red + ((2 * w + (w0 >= su.x * U ? 0 : 1)) * two + half) * seg +
                                     m * k.parts * Q4_RED_PITCH + (tid & 15);
                    v += s[0];
                    if (k.parts == 2) v += s[Q4_RED_PITCH];
                }
                return a.xmode == Q4_X_RAW16 ? v : v * inv[m];
            };
            float v = sum(0);
            if (PLAN && a.pair) {
                const float up = sum(1);
                v = v / (1.0f + expf(-v)) * up;
            }
            store(v, m, row, su.x);
        }
        if (split > 1) {
            // the CTAs' sums, in the order of their ranks; each CTA finishes its share
            cluster_sync();
            for (int i = rank * Q4_WARPS * 32 + tid; i < b.n * pass.cnt * 16; i += split * Q4_WARPS * 32) {
                float v = 0.f;
                for (int c = 0; c < split; ++c)
                    v += __uint_as_float(ld_dsmem_u32(mapa_shared(smem_u32(csum + i), (uint32_t)c)));
                const int q = i >> 4, tl = q / pass.cnt, m = q - tl * pass.cnt, row = (b.first + tl) * 16 + (i & 15);
                if (row >= a.N) continue;
                const int64_t o = (int64_t)m * a.ldo + row;
                if (a.otype == TQ2_F32) reinterpret_cast<float*>(a.out)[o] = v;
                else if (a.otype == TQ2_F16) reinterpret_cast<__half*>(a.out)[o] = __float2half_rn(v);
                else reinterpret_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
            }
            cluster_sync();                                // a CTA stays while others read its sums
        }
        if (!again) break;
        u = un;
        b = next;
        fence_proxy_async_shared();                        // the next pass's rows come through the async proxy
    }
}

struct Q4Device {
    int sms, smem;
    int clusters[4];                   // of 1, 2, 4, 8 CTAs that fit the GPU at once, one CTA an SM
};
// Attributes of a device never change: asked once.  (Clusters do not cross the
// hardware's groups of SMs, so fewer fit than the SMs would say.)
template <int G>
const Q4Device& q4_device() {
    static Q4Device known[64];
    static std::mutex lock;
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev > 63) dev = 63;
    Q4Device& d = known[dev];
    if ((ready.load(std::memory_order_acquire) >> dev) & 1) return d;
    std::lock_guard<std::mutex> hold(lock);
    cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&d.smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    cudaFuncSetAttribute(q4_stream_kernel<G, 1, false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem);
    d.clusters[0] = d.sms;
    for (int i = 1; i < 4; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)d.sms / 8 * 8);
        cfg.blockDim = dim3(Q4_WARPS * 32);
        cfg.dynamicSmemBytes = (size_t)d.smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << i;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, q4_stream_kernel<G, 1, false, false>, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = 1;
        }
        d.clusters[i] = n;
    }
    ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return d;
}

// Shared memory of a launch that takes `tok` rows a pass over clusters of `split`.
inline int q4_smem(const Q4Stream& a, int parts, int tok, int split, const Q4Device& dev, Q4Kernel* k) {
    auto up = [](int v) { return (v + 127) / 128 * 128; };
    const int pitch = (a.nkc + split - 1) / split * Q4_K * 2 + 64;
    const int tiles = (int)((a.N + 15) / 16) * (a.pair ? 2 : 1);
    const int fit = dev.clusters[split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3];
    const int teams = tiles < fit ? tiles : fit;
    const int prefix = up(16 + 16 * Q4_WARPS);
    const int slots = up(prefix + (a.offsets ? 2 * (a.E + 1) * 4 : 0));
    const bool held = a.offsets && a.nslots <= Q4_PLAN_SLOTS;
    const int scale = up(slots + (held ? a.nslots * 4 : 0));
    const int red = scale + 3 * 32 * 4;
    const int sum = up(red + 2 * Q4_WARPS * (a.pair ? 2 : 1) * tok * parts * Q4_RED_PITCH * 4);
    const int64_t x = sum + (split > 1 ? (int64_t)(tiles / teams + 1) * tok * 64 : 0);
    const int64_t end = (x + 127) / 128 * 128 + (int64_t)tok * parts * pitch;
    if (k) {
        k->tiles = tiles;
        k->split = split;
        k->teams = teams;
        k->each = tiles / teams;
        k->more = tiles - k->each * teams;
        k->pitch = pitch;
        k->off_prefix = prefix;
        k->off_slots = held ? slots : 0;
        k->off_scale = scale;
        k->off_red = red;
        k->off_sum = sum;
        k->off_x = up((int)x);
        return (int)end;
    }
    return end > dev.smem ? dev.smem + 1 : (int)end;
}

template <int G, int NT, bool BF, bool PLAN>
cudaError_t q4_stream_launch(Q4Kernel& k, int tok, int split, const Q4Device& dev, cudaStream_t st) {
    const Q4Stream& a = k.a;
    k.tok = tok;
    const int smem = q4_smem(a, k.parts, tok, split, dev, &k);
    if (smem > dev.smem) return cudaErrorInvalidValue;
    const int grid = PLAN ? dev.sms : k.teams * split;
    static std::atomic<uint64_t> raised{0};                // devices whose limit of this kernel is raised
    int d = 0;
    cudaGetDevice(&d);
    if (smem > 48 * 1024 && (d >= 64 || !((raised.load(std::memory_order_relaxed) >> d) & 1))) {
        cudaError_t e = cudaFuncSetAttribute(q4_stream_kernel<G, NT, BF, PLAN>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, dev.smem);
        if (e != cudaSuccess) return e;
        if (d < 64) raised.fetch_or(uint64_t(1) << d, std::memory_order_relaxed);
    }
    if (PLAN)
        return launch_pdl(q4_stream_kernel<G, NT, BF, PLAN>, dim3((unsigned)grid), dim3(Q4_WARPS * 32), (size_t)smem,
                          st, k);
    // rows beyond a pass: further launches
    const int M = a.M;
    const size_t xs = (a.xmode == Q4_X_RAW16 ? 2 : 4) * (size_t)a.ldx, os = (a.otype == TQ2_F32 ? 4 : 2) * (size_t)a.ldo;
    cudaError_t e = cudaSuccess;
    for (int m = 0; m < M && e == cudaSuccess; m += tok) {
        Q4Kernel p = k;
        p.a.M = M - m < tok ? M - m : tok;
        p.a.x = static_cast<const char*>(a.x) + m * xs;
        p.a.out = static_cast<char*>(a.out) + m * os;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(Q4_WARPS * 32);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)split;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = split > 1 ? 2 : 1;
        e = cudaLaunchKernelEx(&cfg, q4_stream_kernel<G, NT, BF, PLAN>, p);
    }
    return e;
}

template <int G, int NT>
cudaError_t q4_stream_pick(Q4Kernel& k, int tok, int split, const Q4Device& dev, cudaStream_t st) {
    if (k.a.offsets)
        return k.a.bf16 ? q4_stream_launch<G, NT, true, true>(k, tok, 1, dev, st)
                        : q4_stream_launch<G, NT, false, true>(k, tok, 1, dev, st);
    return k.a.bf16 ? q4_stream_launch<G, NT, true, false>(k, tok, split, dev, st)
                    : q4_stream_launch<G, NT, false, false>(k, tok, split, dev, st);
}

// The variant by sizes: the rows a pass takes, as far as shared memory holds
// their columns (f32 rows take two each), and the column tiles (NT) they need.
// Without a plan k is split over the clusters that let a pass take most rows
// (13 rows of 10624 f32 and 106 columns: 41.8 us in passes, 11.9 in a cluster of
// 4), and further while that gives idle SMs a CTA of at least 32 chunks a tile.
template <int G>
cudaError_t q4_stream_run(const Q4Stream& a, cudaStream_t st) {
    g_launched.store(true, std::memory_order_release);
    Q4Kernel k{};
    k.a = a;
    k.parts = a.xmode == Q4_X_SPLIT ? 2 : 1;
    const int el = a.xmode == Q4_X_RAW16 ? 2 : 4;
    k.xvec = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (a.ldx * el) % 16 == 0;
    const Q4Device& dev = q4_device<G>();
    const int most = a.tokens * k.parts < 32 ? a.tokens : 32 / k.parts;
    auto rows = [&](int split) {
        int tok = most;
        while (tok > 0 && q4_smem(a, k.parts, tok, split, dev, nullptr) > dev.smem) --tok;
        return tok;
    };
    int split = 1, tok = rows(1);
    if (!a.offsets) {
        const int tiles = (int)((a.N + 15) / 16);
        for (int s = 2; s <= 8 && tok < most && a.nkc >= s; s *= 2) {
            const int n = rows(s);                         // (many columns: a CTA's sums of them take space too)
            if (n > tok) {
                tok = n;
                split = s;
            }
        }
        for (int i = split == 1 ? 1 : split == 2 ? 2 : 3; i < 4 && split < 8 && tiles <= dev.clusters[i] &&
                                                       a.nkc >= 64 * split && rows(2 * split) >= tok; ++i)
            tok = rows(split *= 2);
    }
    if (tok < 1) return cudaErrorInvalidValue;
    if (tok * k.parts > 16) return q4_stream_pick<G, 4>(k, tok, split, dev, st);
    if (tok * k.parts > 8) return q4_stream_pick<G, 2>(k, tok, split, dev, st);
    return q4_stream_pick<G, 1>(k, tok, split, dev, st);
}

}  // namespace tq2
