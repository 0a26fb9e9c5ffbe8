// kv8_umma.cu -- attention of many rows over the 8-bit cache on tcgen05: prompts,
// chunks of prompts, an encoder's states.
//
// Mathematics: as the streaming path (kv8_stream.cu), with the whole weight
// 2^(w_t - m), w_t = (scale log2(e) ks) (q . c) + log2 vs, in f16, and
// l = sum 2^(w_t - m) / vs.  ks and vs are constant over 16 columns, so per score that is
// half a packed multiply-add, one exponential and half a packed sum.
//
// A CTA takes 256 rows (f32: 128), a row being a query token and one of the heads
// that share a head of the cache, over tiles of 128 tokens.  Warps: one brings packed
// tiles by TMA, four decode them (code - 128, exact in f16) into the swizzled layout of the MMAs'
// operands, one issues S = Q K^T (both from shared memory) and O += P V (P from tensor
// memory, over S's columns), and a group of four for every 128 rows does the softmax, a
// thread a row, while the MMAs work for the other group.  f32 queries are two f16 parts, f32
// and f16 results' weights too (twice the MMAs of that product).  All tiles of
// all rows are cut evenly over the CTAs; what a cut divides is joined afterwards.
//
// The MMAs are issued in the order Q K^T, P V, Q K^T .. of a group, and execute in that order: P V
// reads P before the next scores take its place, and scores that are there mean that the
// last P V is done, so the group may rescale O.
#include <type_traits>

#include "kv8_join.cuh"
#include "q4.cuh"

namespace tq2 {
namespace {

constexpr int KT = 128;         // tokens of a tile
constexpr int THREADS = 512;
constexpr int DECODERS = 4;     // warps
constexpr int BUFS = 4;         // decoded tiles: keys and values in turn
constexpr int CONS = 4;         // tiles whose scales are at hand
constexpr int LEAST = 2;        // tiles of a CTA, where there are fewer than all CTAs take
constexpr float HEAD = 6.f, RAISE = 14.f;                    // as kv8_stream.cu
constexpr float TINY = 0x1p-103f;

template <class T, int D>
struct Form {
    static constexpr bool SPLIT = sizeof(T) == 4;
    static constexpr bool TWO = !std::is_same<T, __nv_bfloat16>::value;   // parts of a weight
    static constexpr int NQ = SPLIT ? 1 : 2;                 // groups of 128 rows
    static constexpr int ROWS = NQ * 128;
    static constexpr int RAW = D == 128 ? 2 : 6;             // packed tiles
    static constexpr int SLAB = KT * 128;                    // 128 rows of 64 f16
    static constexpr int TILE = SLAB * (D / 64);             // 128 rows of D f16
};

template <class T, int D>
struct __align__(1024) Shared {
    uint8_t q[2][Form<T, D>::TILE];                          // by group (f32: by part)
    uint8_t kv[BUFS][Form<T, D>::TILE];
    uint8_t raw[Form<T, D>::RAW][KT * D];
    float4 cons[CONS][KT / 16];                              // ks, log2 vs, 1 / vs; w: values count
    float2 scales[CONS][8];                                  // of keys and values, by piece; -1: nothing there
    uint64_t raw_full[Form<T, D>::RAW], raw_empty[Form<T, D>::RAW];
    uint64_t kv_full[BUFS], kv_empty[BUFS], cons_full[CONS];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], idle;
    long long sums[THREADS / 32], rest;
    uint32_t tmem;
    int seq, head, tile, at;
    volatile int abort;
};

// Rows of one head of a sequence in tiles of ROWS, and the KV tiles each of them goes over.
struct Seq {
    Kv8Seq q;
    int rows, tiles;
};
template <int ROWS>
__device__ __forceinline__ Seq seq_of(const Kv8Attention& a, int s) {
    Seq r;
    r.q = kv8_seq(a.c, s);
    r.rows = r.q.n * a.G;
    r.tiles = r.rows <= a.few ? 0 : (r.rows + ROWS - 1) / ROWS;
    return r;
}
// First tile of 128 tokens that some row of a tile sees, and the number of them (at least one).
template <int ROWS>
__device__ __forceinline__ int2 span_of(const Kv8Attention& a, const Seq& s, int tile) {
    const int r0 = tile * ROWS, r1 = min(r0 + ROWS, s.rows) - 1, p = s.q.len - s.q.n;
    const int hi = a.causal ? min(s.q.len, p + r1 / a.G + 1) : s.q.len;
    const int lo = a.window ? max(p + r0 / a.G - a.window + 1, 0) : 0;
    const int first = lo / KT;
    return make_int2(first, max((hi + KT - 1) / KT - first, 1));
}

// A CTA's way through its share: pieces of `run` tiles of one tile of rows.
template <int ROWS>
struct Walk {
    long long left;
    int s, head, tile, at;      // at: tiles of the current rows that are behind
    Seq q;
    int2 span;
    int run;
    __device__ __forceinline__ void open(const Kv8Attention& a) {
        span = span_of<ROWS>(a, q, tile);
        run = (int)min((long long)(span.y - at), left);
    }
    __device__ __forceinline__ void next(const Kv8Attention& a) {
        left -= run;
        if (left == 0) return;
        at = 0;                                              // the piece ended its rows
        if (++tile == q.tiles) {
            tile = 0;
            if (++head == a.c.H) {
                head = 0;
                do q = seq_of<ROWS>(a, ++s);
                while (q.tiles == 0);
            }
        }
        open(a);
    }
};

// KV tiles of one head of the warp's sequences s0 + lane (a lane's own; 0 where there is none).
template <int ROWS>
__device__ __forceinline__ long long lane_units(const Kv8Attention& a, int s, int end, Seq& q, int lane) {
    long long u = 0;
    q.tiles = 0;
    if (s < end) q = seq_of<ROWS>(a, s);
    const bool many = q.tiles > 4;
    if (!many)
        for (int t = 0; t < q.tiles; ++t) u += span_of<ROWS>(a, q, t).y;
    for (uint32_t rest = __ballot_sync(0xffffffffu, many); rest; rest &= rest - 1) {
        const int owner = __ffs(rest) - 1;
        const Seq o = seq_of<ROWS>(a, __shfl_sync(0xffffffffu, s, owner));
        long long sum = 0;
        for (int t = lane; t < o.tiles; t += 32) sum += span_of<ROWS>(a, o, t).y;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == owner) u = sum;
    }
    return u;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

using F2 = unsigned long long;  // two f32
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_parts(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max16(const uint32_t* v) {
    auto f = [&](int i) { return __uint_as_float(v[i]); };
    const float a = max3(f(0), f(1), f(2)), b = max3(f(3), f(4), f(5)), c = max3(f(6), f(7), f(8));
    const float d = max3(f(9), f(10), f(11)), e = max3(f(12), f(13), f(14));
    return max3(max3(a, b, c), max3(d, e, f(15)), kv8_none());
}

// Scores are read from tensor memory twice (64 columns take 50 cycles) rather than held: the loops stay short, which
// the instruction caches of warps in four different roles ask for.

// The largest exponent of a row's 128 weights.  ALL: the row sees all tokens, else those of columns lo .. hi-1.
template <bool ALL>
__device__ __forceinline__ float tile_top(uint32_t s_addr, const float4* cons, float qa, int lo, int hi) {
    float t = kv8_none();
#pragma unroll 1
    for (int c = 0; c < KT; c += 64) {
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(s_addr + c, v[0]);
        tmem_ld_32x32b_x32(s_addr + c + 32, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float4 k = cons[c / 16 + h];
            const float ks = k.x * qa;
            uint32_t* x = &v[h >> 1][16 * (h & 1)];
            if (ALL) {
                t = fmaxf(t, fmaf(max16(x), ks, k.y));
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int col = c + 16 * h + e;
                    t = fmaxf(t, col >= lo && col < hi ? fmaf(__uint_as_float(x[e]), ks, k.y) : kv8_none());
                }
            }
        }
    }
    return t;
}

// The row's weights relative to ref, in place of its scores: 32 tokens' are 16 columns (and 16 of second
// parts).  Returns l with their sum.
template <bool TWO, bool ALL>
__device__ __forceinline__ float tile_weights(uint32_t s_addr, const float4* cons, float qa, float ref, float l, int lo,
                                              int hi) {
#pragma unroll 1
    for (int c = 0; c < KT; c += 64) {
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(s_addr + c, v[0]);
        tmem_ld_32x32b_x32(s_addr + c + 32, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t ph[16], pl[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 k = cons[c / 16 + 2 * g + h];
                const float ks = k.x * qa, off = k.y - ref;
                const F2 ks2 = f2(ks, ks), off2 = f2(off, off);
                F2 sum = f2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t* at = &v[g][16 * h + 2 * e];
                    const float2 x = f2_parts(f2_fma(f2(__uint_as_float(at[0]), __uint_as_float(at[1])), ks2, off2));
                    float e0 = exp2_fast(x.x), e1 = exp2_fast(x.y);
                    if (!ALL) {
                        const int col = c + 32 * g + 16 * h + 2 * e;
                        e0 = col >= lo && col < hi ? e0 : 0.f;
                        e1 = col + 1 >= lo && col + 1 < hi ? e1 : 0.f;
                    }
                    sum = f2_add(sum, f2(e0, e1));
                    ph[8 * h + e] = pack_half2(e0, e1);
                    if (TWO) pl[8 * h + e] = rest_half2(e0, e1, ph[8 * h + e]);
                }
                const float2 both = f2_parts(sum);
                l = fmaf(both.x + both.y, k.z, l);
            }
            tmem_st_32x32b_x16(s_addr + c + 32 * g, ph);
            if (TWO) tmem_st_32x32b_x16(s_addr + c + 32 * g + 16, pl);
        }
    }
    return l;
}

// A warp's 32 rows of queries, scaled by a power of two to 2^14 .. 2^15, into the layout of an MMA operand (the scores of
// the rows before are there, so nobody reads those any more).  Returns the power of the lane's row.
template <class T, int D>
__device__ __forceinline__ int load_queries(const Kv8Attention& a, Shared<T, D>& sm, const Walk<Form<T, D>::ROWS>& w, int qi,
                                            int warp, int lane) {
    using F = Form<T, D>;
    constexpr int EL = 16 / (int)sizeof(T), LPR = D / EL, RPP = 32 / LPR;   // a lane's elements, lanes a row, rows a pass
    constexpr int DEEP = 8;                     // passes whose loads are in flight
    const int in_row = lane % LPR, el = in_row * EL;
    int power = 0;
#pragma unroll 1
    for (int p0 = 0; p0 < 32 / RPP; p0 += DEEP) {
        uint4 raw[DEEP];
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const int r = w.tile * F::ROWS + qi * 128 + warp * 32 + (p0 + d) * RPP + lane / LPR;
            const int token = min(r, w.q.rows - 1) / a.G, h = min(r, w.q.rows - 1) - token * a.G;
            const T* p = static_cast<const T*>(a.q) + (int64_t)(w.q.q.q0 + token) * a.qt + (int64_t)(w.head * a.G + h) * a.qh + el;
            if (a.qvec) {
                raw[d] = *reinterpret_cast<const uint4*>(p);
            } else {
                T* e = reinterpret_cast<T*>(&raw[d]);
#pragma unroll
                for (int k = 0; k < EL; ++k) e[k] = p[k];
            }
        }
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const int i = warp * 32 + (p0 + d) * RPP + lane / LPR;          // of the group
            const bool live = w.tile * F::ROWS + qi * 128 + i < w.q.rows;
            const T* u = reinterpret_cast<const T*>(&raw[d]);
            float x[EL], most = 0.f;
#pragma unroll
            for (int k = 0; k < EL; ++k) {
                x[k] = live ? kv8_wide(u[k]) : 0.f;
                most = fmaxf(most, fabsf(x[k]));
            }
#pragma unroll
            for (int k = 1; k < LPR; k <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
            const int e = min(max(141 - (int)(__float_as_uint(most) >> 23), -112), 126);
            const float up = copysignf(__uint_as_float((uint32_t)(e + 127) << 23), a.scale);
            const int of = __shfl_sync(0xffffffffu, e, (lane - (p0 + d) * RPP) * LPR & 31);
            if (lane / RPP == p0 + d) power = of;
            uint32_t h[EL / 2], l[EL / 2];
#pragma unroll
            for (int k = 0; k < EL / 2; ++k) {
                h[k] = pack_half2(x[2 * k] * up, x[2 * k + 1] * up);
                if (F::SPLIT) l[k] = rest_half2(x[2 * k] * up, x[2 * k + 1] * up, h[k]);
            }
            const int off = (el / 64) * F::SLAB + i * 128 + (el % 64 / 8 ^ (i & 7)) * 16 + el % 8 * 2;
            if constexpr (F::SPLIT) {
                *reinterpret_cast<uint2*>(sm.q[0] + off) = make_uint2(h[0], h[1]);
                *reinterpret_cast<uint2*>(sm.q[1] + off) = make_uint2(l[0], l[1]);
            } else {
                *reinterpret_cast<uint4*>(sm.q[qi] + off) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full[qi]);
    return power;
}

template <class T, int D>
__global__ void __launch_bounds__(THREADS, 1)
kv8_umma_kernel(const __grid_constant__ Kv8Attention a, float* parts, Kv8Joint* joints) {
    using F = Form<T, D>;
    constexpr int ROWS = F::ROWS;
    constexpr uint32_t S_COL = 0, O_COL = 256;
    extern __shared__ __align__(1024) uint8_t raw_shared[];
    Shared<T, D>& sm = *reinterpret_cast<Shared<T, D>*>(raw_shared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < F::RAW; ++i) {
            mbar_init(&sm.raw_full[i], 33);
            mbar_init(&sm.raw_empty[i], DECODERS);
        }
        for (int i = 0; i < BUFS; ++i) {
            mbar_init(&sm.kv_full[i], DECODERS);
            mbar_init(&sm.kv_empty[i], 1);
        }
        for (int i = 0; i < CONS; ++i) mbar_init(&sm.cons_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 4);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 128);
            mbar_init(&sm.o_full[i], 1);
        }
        mbar_init(&sm.idle, 1);
        sm.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.map);
    }
    pdl_launch_dependents();
    pdl_wait();

    // the whole list's length (a head's times H), and where this CTA's share begins
    const int S = a.c.seqs, per = (S + THREADS / 32 - 1) / (THREADS / 32);
    const int slice_end = min((warp + 1) * per, S);
    long long mine = 0;
    Seq q;
    for (int s = warp * per; s < slice_end; s += 32) mine += lane_units<ROWS>(a, s + lane, slice_end, q, lane);
#pragma unroll
    for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    mine *= a.c.H;
    if (lane == 0) sm.sums[warp] = mine;
    __syncthreads();
    long long total = 0, before = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += sm.sums[i];
        total += sm.sums[i];
    }
    const Kv8Cut cut(total, gridDim.x, LEAST);
    const int cta = blockIdx.x;
    if (cta >= cut.ctas) {
        if (tid == 0) joints[cta].pieces = 0;
        return;
    }
    const long long begin = cut.begin(cta);
    if (before <= begin && begin < before + mine) {
        for (int s = warp * per; s < slice_end; s += 32) {
            const long long u = lane_units<ROWS>(a, s + lane, slice_end, q, lane);
            const long long incl = warp_scan(u * a.c.H, lane);
            const uint32_t past = __ballot_sync(0xffffffffu, before + incl > begin);
            if (!past) {
                before += __shfl_sync(0xffffffffu, incl, 31);
                continue;
            }
            const int owner = __ffs(past) - 1;
            const long long in = begin - before - __shfl_sync(0xffffffffu, incl - u * a.c.H, owner);
            const long long uh = __shfl_sync(0xffffffffu, u, owner);
            q = seq_of<ROWS>(a, s + owner);
            long long left = in % uh;
            for (int t = 0;; t += 32) {
                const long long c = t + lane < q.tiles ? span_of<ROWS>(a, q, t + lane).y : 0;
                const long long sum = warp_scan(c, lane);
                const uint32_t there = __ballot_sync(0xffffffffu, sum > left);
                if (!there) {
                    left -= __shfl_sync(0xffffffffu, sum, 31);
                    continue;
                }
                const int o = __ffs(there) - 1;
                left -= __shfl_sync(0xffffffffu, sum - c, o);
                if (lane == 0) {
                    sm.seq = s + owner;
                    sm.head = (int)(in / uh);
                    sm.tile = t + o;
                    sm.at = (int)left;
                }
                break;
            }
            break;
        }
    }
    if (warp == 2) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    Walk<ROWS> w;
    w.left = cut.begin(cta + 1) - begin;
    const long long units = w.left;
    w.s = sm.seq;
    w.head = sm.head;
    w.tile = sm.tile;
    w.at = sm.at;
    w.q = seq_of<ROWS>(a, w.s);
    w.open(a);
    volatile int* abort_flag = &sm.abort;
    const int logB = a.c.logB, rows_piece = min(1 << logB, KT / 2), pieces = KT / rows_piece;

    if (warp == 0) {                                         // ---- packed tiles
        int st = 0;
        uint32_t ph = 0;
        long long g = 0;
        bool wrapped = false, ok = true;
        fence_proxy_async_shared();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        for (; ok && w.left; w.next(a)) {
            const int from = a.window ? max(w.q.q.len - w.q.q.n - a.window + 1, 0) : 0;
            for (int i = 0; ok && i < w.run; ++i, ++g) {
                const int token = (w.span.x + w.at + i) * KT + lane * rows_piece;
                int block = -1;
                if (lane < pieces && token < w.q.q.len && token + rows_piece > from) block = kv8_block(a.c, w.s, token);
                const uint32_t here = __ballot_sync(0xffffffffu, block >= 0);
                const int inside = token & ((1 << logB) - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!mbar_wait_or_abort(&sm.raw_empty[st], ph ^ 1, abort_flag, true)) {
                        sm.abort = 1;
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[st], __popc(here) * (uint32_t)(rows_piece * D));
                    if (block >= 0)
                        tma_load_2d(sm.raw[st] + lane * rows_piece * D, &a.map, &sm.raw_full[st], 0,
                                    (int)(kv8_row(a.c, block, kv, w.head) + inside));
                    if (kv == 0) {
                        float2* sc = &sm.scales[g & (CONS - 1)][lane & 7];
                        if (block >= 0) {
                            const float* src = a.c.scales + (int64_t)block * 2 * a.c.H + w.head;
                            cp_async4(&sc->x, src);
                            cp_async4(&sc->y, src + a.c.H);
                        } else if (lane < pieces) {
                            *sc = make_float2(0.f, -1.f);
                        }
                    }
                    cp_async_arrive(&sm.raw_full[st]);
                    if (++st == F::RAW) st = 0, ph ^= 1, wrapped = true;
                }
            }
        }
        if (!ok)                                             // copies in flight end before the shared memory goes
            for (int u = 0; u < F::RAW; ++u)
                if (u < st || wrapped) mbar_wait(&sm.raw_full[u], u < st ? ph : ph ^ 1);
    } else if (warp == 1) {                                  // ---- MMA issuer
        constexpr uint32_t s_idesc = idesc_f16_f32(128, KT), o_idesc = idesc_f16_f32_bmn(128, D);
        uint32_t q_ph[2] = {0, 0}, p_ph[2] = {0, 0};
        long long g = 0;
        bool ok = true;
        auto scores = [&](int qi, int buf) {
            if (elect_one()) {
                const uint32_t qb = smem_u32(sm.q[F::SPLIT ? 0 : qi]), kb = smem_u32(sm.kv[buf]);
#pragma unroll
                for (int part = 0; part < (F::SPLIT ? 2 : 1); ++part)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * F::SLAB + (k & 3) * 32;
                        umma_f16_ss(tmem + S_COL + 128 * qi, sdesc_kmajor_sw128(qb + part * F::TILE + off),
                                    sdesc_kmajor_sw128(kb + off), s_idesc, part || k);
                    }
                umma_commit(&sm.s_full[qi]);
            }
            __syncwarp();
        };
        auto values = [&](int qi, int buf, bool more) {
            if (elect_one()) {
                const uint32_t vb = smem_u32(sm.kv[buf]);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
#pragma unroll
                    for (int part = 0; part < (F::TWO ? 2 : 1); ++part)
                        umma_f16_ts(tmem + O_COL + D * qi, tmem + S_COL + 128 * qi + 32 * (k >> 1) + 16 * part + 8 * (k & 1),
                                    sdesc_mnmajor_sw128(vb + k * 2048, F::SLAB, 1024), o_idesc, more || k || part);
            }
            __syncwarp();
        };
        auto done = [&](uint64_t* bar) {
            if (elect_one()) umma_commit(bar);
            __syncwarp();
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok && !mbar_wait_or_abort(bar, parity, abort_flag, true)) {
                sm.abort = 1;
                ok = false;
            }
            return ok;
        };
        for (; ok && w.left; w.next(a)) {
            const int nq = w.q.rows - w.tile * ROWS > 128 ? F::NQ : 1;
            for (int i = 0; ok && i < w.run; ++i, ++g) {
                const int kb = (int)(2 * g) & 3, vb = kb + 1;
                const uint32_t ph = (uint32_t)(g >> 1) & 1;
                if (i == 0) {
                    for (int qi = 0; qi < nq && ok; ++qi) {
                        if (!wait(&sm.q_full[qi], q_ph[qi])) break;
                        q_ph[qi] ^= 1;
                        if (qi == 0 && !wait(&sm.kv_full[kb], ph)) break;
                        tc_fence_after();
                        scores(qi, kb);
                    }
                    if (!ok) break;
                    done(&sm.kv_empty[kb]);
                }
                const int kn = kb ^ 2;
                const uint32_t phn = (uint32_t)((g + 1) >> 1) & 1;
                for (int qi = 0; qi < nq && ok; ++qi) {
                    if (!wait(&sm.p_full[qi], p_ph[qi])) break;
                    p_ph[qi] ^= 1;
                    if (qi == 0 && !wait(&sm.kv_full[vb], ph)) break;
                    tc_fence_after();
                    values(qi, vb, i > 0);
                    if (qi == nq - 1) done(&sm.kv_empty[vb]);
                    if (i + 1 < w.run) {
                        if (qi == 0 && !wait(&sm.kv_full[kn], phn)) break;
                        tc_fence_after();
                        scores(qi, kn);
                        if (qi == nq - 1) done(&sm.kv_empty[kn]);
                    } else {
                        done(&sm.o_full[qi]);
                    }
                }
            }
        }
        if (!ok) {                                           // MMAs in flight end before their operands go
            done(&sm.idle);
            mbar_wait(&sm.idle, 0);
        }
    } else if (warp >= 12) {                                 // ---- decoders: 32 tokens of a tile each
        const int dw = warp - 12;
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (long long g = 0; ok && g < units; ++g) {
            const int slot = (int)g & (CONS - 1);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const int buf = ((int)(2 * g) & 3) + kv;
                if (!mbar_wait_or_abort(&sm.raw_full[st], ph, abort_flag, true) ||
                    !mbar_wait_or_abort(&sm.kv_empty[buf], ((uint32_t)(g >> 1) & 1) ^ 1, abort_flag, true)) {
                    sm.abort = 1;
                    ok = false;
                    break;
                }
                if (kv == 0 && dw == 0) {
                    if (lane < KT / 16) {
                        const float2 sc = sm.scales[slot][lane * 16 / rows_piece];
                        float4 c = make_float4(sc.x, log2f(sc.y), 1.f / sc.y, 1.f);
                        if (isnan(sc.y)) c.z = 1.f;
                        if (sc.y < TINY) c = make_float4(sc.x, -103.f, 0x1p103f, 0.f);   // values that are all zeros
                        if (sc.y < 0.f) c = make_float4(0.f, kv8_none(), 1.f, 0.f);      // no block: nobody sees it
                        sm.cons[slot][lane] = c;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.cons_full[slot]);
                } else if (kv && !mbar_wait_or_abort(&sm.cons_full[slot], (uint32_t)(g / CONS) & 1, abort_flag, true)) {
                    sm.abort = 1;
                    ok = false;
                    break;
                }
                const uint8_t* src = sm.raw[st];
                uint8_t* dst = sm.kv[buf];
                // Eight rows of 64 packed bytes a step.  Lanes 0..3 and 4..7 of a phase take rows r and r ^ 5: their swizzled
                // 16-byte pieces lie in different halves of a line, and those of f16 in its even and odd pieces.
                constexpr int DEEP = 4;                      // steps whose loads are in flight
                const int in8 = (lane >> 3) ^ ((lane >> 2 & 1) * 5), c = lane & 3;
                const int row0 = dw * 32 + in8;
                const int from = row0 * D + (D == 128 ? c ^ in8 : c ^ (in8 >> 1 & 3)) * 16;
                const int to = row0 * 128 + (2 * c ^ in8) * 16;
                const bool any_zero = kv && __any_sync(0xffffffffu, lane < 2 && sm.cons[slot][dw * 2 + (lane & 1)].w == 0.f);
#pragma unroll 1
                for (int x0 = 0; x0 < D / 16; x0 += DEEP) {
                    uint4 u[DEEP];
#pragma unroll
                    for (int x = 0; x < DEEP; ++x) {
                        const int block = (x0 + x) & 3, slab = (x0 + x) >> 2;      // of 8 rows, of 64 columns
                        u[x] = *reinterpret_cast<const uint4*>(src + (from ^ (slab * 64)) + block * 8 * D);
                        if (any_zero && sm.cons[slot][dw * 2 + (block >> 1)].w == 0.f)
                            u[x] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
                    }
#pragma unroll
                    for (int x = 0; x < DEEP; ++x) {
                        const int block = (x0 + x) & 3, slab = (x0 + x) >> 2;
                        uint8_t* p = dst + slab * F::SLAB + block * 1024;
                        *reinterpret_cast<uint4*>(p + to) =
                            make_uint4(kv8_pair<0>(u[x].x), kv8_pair<2>(u[x].x), kv8_pair<0>(u[x].y), kv8_pair<2>(u[x].y));
                        *reinterpret_cast<uint4*>(p + (to ^ 16)) =
                            make_uint4(kv8_pair<0>(u[x].z), kv8_pair<2>(u[x].z), kv8_pair<0>(u[x].w), kv8_pair<2>(u[x].w));
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.kv_full[buf]);
                    mbar_arrive(&sm.raw_empty[st]);
                }
                if (++st == F::RAW) st = 0, ph ^= 1;
            }
        }
    } else if (warp >= 4 && warp < 4 + 4 * F::NQ) {          // ---- softmax: a thread a row
        const int qi = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t s_addr = tmem + S_COL + 128 * qi + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_addr = tmem + O_COL + D * qi + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t s_ph = 0, o_ph = 0;
        long long g = 0;
        bool ok = true;
        const float NONE = kv8_none();
        Kv8Joint joint{0, 0, 0, 0};
        // pieces that have rows for this group
        auto skip = [&] {
            while (w.left && w.q.rows - w.tile * ROWS <= 128 * qi) {
                g += w.run;
                w.next(a);
            }
        };
        skip();
        int power = 0;
        if (w.left) power = load_queries<T, D>(a, sm, w, qi, warp & 3, lane);
        while (w.left) {
            const int r = w.tile * ROWS + qi * 128 + row;
            const bool live = r < w.q.rows;
            const int pos = w.q.q.len - w.q.q.n + (live ? r : w.tile * ROWS) / a.G;
            const int row_hi = a.causal ? min(w.q.q.len, pos + 1) : w.q.q.len;
            const int row_lo = a.window ? max(pos - a.window + 1, 0) : 0;
            const float qa = fabsf(a.scale) * __uint_as_float((uint32_t)(127 - power) << 23);
            // tokens [safe_lo, safe_hi) are seen by all of the warp's rows
            const int safe_hi = __reduce_min_sync(0xffffffffu, live ? row_hi : 0x7fffffff);
            const int safe_lo = __reduce_max_sync(0xffffffffu, live ? row_lo : 0);

            float m = NONE, l = 0.f;
            for (int i = 0; i < w.run; ++i, ++g) {
                const int base = (w.span.x + w.at + i) * KT, slot = (int)g & (CONS - 1);
                // (scores that are there mean that the slot's phase is this tile's)
                if (!mbar_wait_or_abort(&sm.s_full[qi], s_ph, abort_flag, true) ||
                    !mbar_wait_or_abort(&sm.cons_full[slot], (uint32_t)(g / CONS) & 1, abort_flag, true)) {
                    sm.abort = 1;
                    ok = false;
                    break;
                }
                s_ph ^= 1;
                tc_fence_after();
                const float4* cons = sm.cons[slot];
                const bool inside = base >= safe_lo && base + KT <= safe_hi;
                const int lo = row_lo - base, hi = row_hi - base;
                float t = inside ? tile_top<true>(s_addr, cons, qa, lo, hi) : tile_top<false>(s_addr, cons, qa, lo, hi);
                const bool raise = t > m + RAISE;
                if (__any_sync(0xffffffffu, raise)) {
                    const float now = raise ? t - HEAD : m;
                    const float f = raise ? exp2_fast(m - now) : 1.f;
                    m = now;
                    l *= f;
                    if (i > 0) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_addr + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st_32x32b_x16(o_addr + 16 * c, o);
                        }
                    }
                }
                const float ref = m == NONE ? 0.f : m;
                l = inside ? tile_weights<F::TWO, true>(s_addr, cons, qa, ref, l, lo, hi)
                           : tile_weights<F::TWO, false>(s_addr, cons, qa, ref, l, lo, hi);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sm.p_full[qi]);
            }
            if (!ok) break;
            // ---- where the row's result goes, or its part of one; the next rows' queries meanwhile
            const bool whole = w.run == w.span.y;
            int64_t at_lse = 0;
            T* out = static_cast<T*>(a.out) + kv8_out_row(a, w.q.q, w.head, live ? r : 0, &at_lse);
            float* part = parts + ((size_t)cta * 2 + (w.at == 0 ? 1 : 0)) * kv8_part_floats(ROWS, D);
            if (!whole && w.at == 0) {
                // the rows' other pieces: as many CTAs as the rest of their tiles reaches into
                const long long from = cut.begin(cta + 1) - w.run;
                joint = Kv8Joint{w.s, w.head, w.tile, cut.of(from + w.span.y - 1) - cta + 1};
            }
            w.next(a);
            skip();
            if (w.left) power = load_queries<T, D>(a, sm, w, qi, warp & 3, lane);
            if (!mbar_wait_or_abort(&sm.o_full[qi], o_ph, abort_flag, true)) {
                sm.abort = 1;
                ok = false;
                break;
            }
            o_ph ^= 1;
            tc_fence_after();
            const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
            const int pr = qi * 128 + row;
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(o_addr + 32 * c, v);
                tmem_wait_ld();
                float y[2][16];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e >> 4][e & 15] = __uint_as_float(v[e]) * inv;
                if (live && whole) {
                    kv8_store16(out + 32 * c, vec, y[0]);
                    kv8_store16(out + 32 * c + 16, vec, y[1]);
                } else if (live) {
                    float* to = part + 2 * ROWS + (size_t)pr * D + 32 * c;
                    kv8_store16(to, true, y[0]);
                    kv8_store16(to + 16, true, y[1]);
                }
            }
            if (live && whole && a.lse) a.lse[at_lse] = kv8_lse(m, l);
            if (live && !whole) part[pr] = m, part[ROWS + pr] = l;
            tc_fence_before();
        }
        if (warp == 4 && lane == 0) joints[cta] = ok ? joint : Kv8Joint{0, 0, 0, 0};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

// One CTA a SM, and none that could never have a tile.
int grid_of(const Kv8Attention& a) {
    const int64_t rows = (int64_t)a.c.T * a.G;
    const int64_t most = (rows / 128 + a.c.seqs) * a.c.H * ((((int64_t)a.c.width << a.c.logB) + KT - 1) / KT);
    const int64_t full = kv8_sm_count();
    return (int)(most < full ? most : full);
}

template <class T, int D>
cudaError_t run(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    constexpr int ROWS = Form<T, D>::ROWS;
    static_assert(sizeof(Shared<T, D>) <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(kv8_umma_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Shared<T, D>));
    if (e != cudaSuccess) return e;
    const int grid = grid_of(a);
    float* parts = static_cast<float*>(scratch);
    Kv8Joint* joints = reinterpret_cast<Kv8Joint*>(parts + (size_t)grid * 2 * kv8_part_floats(ROWS, D));
    g_launched.store(true, std::memory_order_release);
    e = launch_pdl(kv8_umma_kernel<T, D>, dim3(grid), dim3(THREADS), sizeof(Shared<T, D>), st, a, parts, joints);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv8_join_kernel<T, D, ROWS>, dim3(grid, ROWS / 32), dim3(256), 0, st, a, (const float*)parts,
                      (const Kv8Joint*)joints);
}

template <class T>
cudaError_t run_d(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    return a.c.D == 64 ? run<T, 64>(a, scratch, st) : run<T, 128>(a, scratch, st);
}

}  // namespace

size_t kv8_umma_scratch(const Kv8Attention& a) {
    const int rows = a.dtype == TQ2_F32 ? 128 : 256;
    return (size_t)grid_of(a) * (2 * kv8_part_floats(rows, a.c.D) * sizeof(float) + sizeof(Kv8Joint));
}

cudaError_t launch_kv8_umma(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    if (a.dtype == TQ2_F32) return run_d<float>(a, scratch, st);
    if (a.dtype == TQ2_F16) return run_d<__half>(a, scratch, st);
    return run_d<__nv_bfloat16>(a, scratch, st);
}

unsigned int read_clear_dev_error_kv8_umma(cudaStream_t st) { return read_clear_record(st); }

}  // namespace tq2
